"""Build libsffn.so (gfx950) in-tree: one hipcc compile per source, then a shared-library link; and _bind.so, the
CPython binding of the attention half (host code only)."""
import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libsffn.so")
BUILD = os.path.join(HERE, "_build")
SOURCES = ["api.hip", "predict.hip", "forward.hip", "forward_q4.hip", "union.hip", "union_rows.hip", "union_down.hip",
           "fused.hip", "decode.hip", "attn_api.hip", "norm.hip", "kv_cache.hip", "attn_few.hip", "attn_many.hip"]

# -packed-fp32-ops: keep the compiler from forming packed fp32 arithmetic (scalar fp32 only).
HIPFLAGS = ["-O3", "--offload-arch=gfx950", "-fPIC", "-std=c++17", "-Wall", "-Wno-unused-function",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-munsafe-fp-atomics"]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".hip", ".o"))
    cmd = ["hipcc", *HIPFLAGS, "-I", os.path.join(HERE, "..", "include"), "-c", os.path.join(SRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile {src} failed:\n{r.stdout}{r.stderr}")
    return obj


def build_binding() -> str:
    """_bind.so from csrc/bind.cpp, against the installed torch's headers and libraries (torch is imported before it)."""
    from torch.utils.cpp_extension import include_paths, library_paths
    out = os.path.join(HERE, "_bind.so")
    inc = [*include_paths(), os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
           sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           *(a for p in inc for a in ("-isystem", p)), os.path.join(SRC, "bind.cpp"), "-o", out + ".tmp",
           *("-L" + p for p in library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile bind.cpp failed:\n{r.stdout}{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding.result()
    tmp = OUT + ".tmp"
    cmd = ["hipcc", "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print("built", OUT)
    return OUT


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
