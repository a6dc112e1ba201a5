"""Which lengths an eviction takes: a sequence's own count may not be overwritten by the cached one's, and the refusal says so."""
import pytest

from activation_sparse_ffn_predictor_amd import _lib
from test_attention_abi_cpu import kv
from test_layer_ops_abi_cpu import A, EVICT, call


@pytest.mark.parametrize("lens", [dict(plen=A, len_out=A), dict(plen=2 * A, len_out=2 * A)])
def test_seq_len_is_not_overwritten(lens):
    """Both in place (the binding's kv_len for what is left out), and both the same other tensor."""
    assert call("sffn_kv_evict", dict(EVICT, cache=kv()), lens) == 6
    text = _lib.lib().sffn_last_error().decode()
    assert "kv_len_out" in text and "seq_len" in text, text


def test_other_overlaps_say_so():
    assert call("sffn_kv_evict", dict(EVICT, cache=kv()), dict(src=4 * A)) == 6
    assert "overlaps" in _lib.lib().sffn_last_error().decode()
