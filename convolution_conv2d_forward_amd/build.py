"""Build libconv2d.so for gfx950 with hipcc (in-tree, next to this file).

    python convolution_conv2d_forward_amd/build.py [-v]

Every HIP source is compiled with packed-fp32 instructions disabled
(``-Xclang -target-feature -Xclang -packed-fp32-ops``); hipcc's host pass
warns that it does not know that feature, which is harmless.
"""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libconv2d.so")
MARSHAL = os.path.join(HERE, "_marshal.so")   # tensor checks of the Python binding
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["conv2d_api.cpp", "igemm_f32.hip", "igemm_bf16.hip", "depthwise.hip", "qpointwise.hip",
           "direct.hip", "fused_pw_dw.hip", "fused_dw_pw.hip", "grouped.hip", "qdepthwise.hip",
           "qfused_dw_pw.hip", "qfused_pw_dw.hip", "igemm_i8.hip", "probe_copy.hip", "winograd_f32.hip",
           "winograd4_f32.hip", "pointwise_f32.hip", "pw_gemm_f32.hip", "pw_narrow_f32.hip", "small_f32.hip",
           "attention_api.cpp", "linear.hip", "linear_rows.hip", "linear_f32.hip", "linear_bf16.hip", "qk_rope.hip",
           "attention_any.hip", "attention_f32.hip", "attention_bf16.hip", "attention_rows.hip", "decoder_api.cpp",
           "kv_cache.hip", "block_norm.hip", "paged_attention.hip", "paged_rows_f32.hip", "paged_rows_f32_e4m3.hip",
           "paged_rows_bf16.hip", "paged_rows_bf16_e4m3.hip", "paged_tile_f32.hip", "paged_tile_f32_e4m3.hip",
           "paged_tile_bf16.hip", "paged_tile_bf16_e4m3.hip"]

FLAGS = ["-O3", "-std=c++17", "--offload-arch=gfx950", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-ffp-contract=fast"]


def _compile(src, verbose):
    out = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", out]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, flush=True)
    return out


def _build_marshal(verbose):
    """The binding's tensor checks, against the headers of the installed torch (host code only).  The C library needs
    neither, so without torch they are left out, with a note: the Python binding, which uses torch, says so too."""
    import sysconfig

    try:
        import torch
    except ImportError as e:
        print(f"_marshal.so is not built: {e}", flush=True)
        return
    root = os.path.dirname(os.path.abspath(torch.__file__))
    tmp = MARSHAL + ".tmp"
    cmd = [HIPCC, "-x", "c++", "-no-hip-rt", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-I" + os.path.join(root, d) for d in ("include", "include/torch/csrc/api/include")),
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "marshal.cpp"), "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on marshal.cpp:\n{r.stdout}{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    workers = min(len(SOURCES), max(1, min(8, os.cpu_count() or 1)))
    with ThreadPoolExecutor(workers) as ex:
        marshal = ex.submit(_build_marshal, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        marshal.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
