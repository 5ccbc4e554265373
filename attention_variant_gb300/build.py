"""Build the CUDA library in-tree: attention_variant_gb300/_build/libflattn.so.

Every translation unit under csrc/ is compiled for sm_103a only, in parallel,
then linked into one shared library with the CUDA runtime linked statically
(so loading it needs no libcudart and no GPU; calls that need a device fail
with FL_ERR_NO_DEVICE instead).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libflattn.so")
SOURCES = ["api.cu", "fwd_standard.cu", "fwd_diff.cu", "fwd_evo.cu", "fwd_decode.cu", "score_expr.cu",
           "bwd_standard.cu", "bwd_diff.cu", "rope.cu", "kv_plan.cu", "fwd_chunk.cu", "kv_fp8.cu",
           "fwd_chunk_fp8.cu"]
# Sources of the standard kernel, embedded in the library for the runtime
# compilation of score_mod expressions (score_expr.cu).
JIT_SOURCES = ["fwd_standard.cu", "bwd_standard.cu", "common.cuh", "ptx.cuh", "softmax_tile.cuh",
               "launch.h", "rtc_compat.cuh", "fastdiv.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "nvcc")


def _flags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-I", BUILD, *extra]


def write_jit_sources(path: str) -> None:
    """The kernel sources the runtime compiler needs, as C++ raw strings."""
    delim = "FL_SRC"
    parts = ["// generated by build.py from csrc/: do not edit\n",
             "struct JitSource { const char *name; const char *text; };\n",
             "static const JitSource kJitSources[] = {\n"]
    for name in JIT_SOURCES:
        text = open(os.path.join(CSRC, name)).read()
        if f"){delim}\"" in text:
            raise RuntimeError(f"{name} contains the raw-string delimiter")
        parts.append(f'    {{"{name}", R"{delim}({text}){delim}"}},\n')
    parts.append("};\n")
    tmp = path + f".tmp{os.getpid()}"
    with open(tmp, "w") as f:
        f.write("".join(parts))
    os.replace(tmp, path)


def _inputs_mtime() -> float:
    paths = [os.path.join(ROOT, "include", "fl_attn.h")]
    paths += [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return max(os.path.getmtime(p) for p in paths)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _inputs_mtime():
        return LIB
    write_jit_sources(os.path.join(BUILD, "jit_sources.inc"))

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC, *_flags(extra_flags), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
