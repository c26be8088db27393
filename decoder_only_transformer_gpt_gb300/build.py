"""Build the CUDA library libgpt_gb300.so in-tree with nvcc for sm_103a, and the
module _calls.so that calls it with torch's tensors.

Each translation unit under csrc/ is compiled in parallel, then linked into
one shared library next to this file. The library knows no torch type and is
built without torch; where there is one, the module (csrc/py_calls.cpp, host
code only) is compiled beside the others and linked behind the library. Rebuilds
only when a source or header is newer than either (or when forced), and the
module alone when it was built against another torch or Python.

    python -m decoder_only_transformer_gpt_gb300.build [--force] [--verbose]
"""
import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgpt_gb300.so")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_FOR = os.path.join(BUILD, "calls_for.txt")    # what _calls.so was built against

SOURCES = ["k_gemm_tc.cu", "k_attn_tc.cu", "k_rowwise.cu", "k_simt.cu", "k_decode.cu", "tmap.cu", "gpt_api.cu",
           "gpt_forward.cu", "gptk.cu", "gptk_noalloc.cu", "k_backward.cu", "k_attn_bwd_tc.cu", "gpt_backward.cu",
           "k_paged.cu", "gptk_paged.cu", "k_attn_window_tc.cu", "k_attn_window_bwd_tc.cu", "gptk_window.cu",
           "k_append.cu", "k_paged4.cu", "k_logprobs.cu", "gptk_logprobs.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
          "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def calls_for() -> str:
    """The torch and the Python whose headers and libraries the module is built against (without an import of torch)."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"torch {version} in {importlib.util.find_spec('torch').origin}, {sysconfig.get_config_var('SOABI')}\n"


def _newer_than_sources(made: str) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in _deps())


def calls_up_to_date() -> bool:
    if not has_torch():
        return True
    if not _newer_than_sources(CALLS) or not os.path.exists(CALLS_FOR):
        return False
    with open(CALLS_FOR) as f:
        return f.read() == calls_for()


def up_to_date() -> bool:
    return _newer_than_sources(LIB) and calls_up_to_date()


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def compile_calls() -> str:
    """The object file of the module, against this machine's Python, torch and CUDA headers."""
    import torch
    obj = os.path.join(BUILD, "py_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-unknown-pragmas",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(_torch_dir(), "include"), "-isystem", cuda,
           "-c", os.path.join(CSRC, "py_calls.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for py_calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def link_calls(obj: str) -> None:
    """_calls.so, which finds the library next to itself and torch's libraries where `import torch` has loaded them."""
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libgpt_gb300.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _calls.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(calls_for())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    if not force and _newer_than_sources(LIB):
        link_calls(compile_calls())
        return LIB
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *CFLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        calls = ex.submit(compile_calls) if has_torch() else None
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_verbose:
        for obj, log in results:
            if log.strip():
                print(f"--- {os.path.basename(obj)}\n{log}", file=sys.stderr)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if calls:
        link_calls(calls.result())
    else:
        print("no torch: the library alone, without _calls.so (the binding needs both)", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas", action="store_true", help="print register and shared-memory usage")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas))
