"""Predictor-guided, neuron-aware sparse FFN for one AMD MI355X (gfx950).

The compute path is the HIP library libsffn.so (C ABI in include/sffn.h); this package only binds it
(``_lib``), packs stored layouts (``pack``) and drives a resident layer stack (``stack``), of FFN layers or with the
attention half and a paged K/V cache in front of each. There is no CPU fallback: calls fail if the library is missing.
"""
from ._lib import (  # noqa: F401
    ACT_RELU, ACT_REGLU, EXPORTS, SffnError, add_rmsnorm, attn, attn_path, attn_workspace_size, forward, forward_q4,
    kv_read, kv_write, lib, mask_words, predict, status_string, workspace_size,
)

__all__ = ["ACT_RELU", "ACT_REGLU", "EXPORTS", "SffnError", "add_rmsnorm", "attn", "attn_path", "attn_workspace_size",
           "forward", "forward_q4", "kv_read", "kv_write", "lib", "mask_words", "predict", "status_string",
           "workspace_size"]
