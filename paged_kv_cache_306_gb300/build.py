"""Build libpa.so in-tree for sm_103a with nvcc.

    python -m paged_kv_cache_306_gb300.build [--force]

Each translation unit is compiled in parallel, then linked into
paged_kv_cache_306_gb300/_build/libpa.so.  Rebuilds only when a source or header
is newer than the library.  Beside it goes the CPython extension that marshals the
FP4 calls (csrc/fp4_calls.cpp), built for the Python and torch at hand, by itself where
only it is missing; without a compiler or their headers it is left out, and the binding
takes its ctypes path.  A build that failed leaves its message beside it and is tried
again when the library is rebuilt, or by the command above.
"""
import argparse
import concurrent.futures as cf
import contextlib
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libpa.so")
SOURCES = ["api.cu", "cache_ops.cu", "decode_f32.cu", "decode_f16.cu", "decode_bf16.cu", "decode_fp8.cu", "decode_noalloc.cu",
           "prefill.cu", "fp4_cache.cu", "fp4_decode.cu", "block_manager.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def calls_path():
    """Where the FP4 calls' extension for this Python, torch and source lies (built or not); None without torch.

    The extension calls the library through the prototypes it was compiled with, so its name carries a digest of
    them: one that was compiled from another header, by this environment or another, is never loaded."""
    try:
        import torch
    except ImportError:
        return None
    h = hashlib.sha256()
    for f in (os.path.join(CSRC, "fp4_calls.cpp"), os.path.join(INCLUDE, "pa.h")):
        with open(f, "rb") as src:
            h.update(src.read())
    return os.path.join(OUT_DIR, f"_fp4_calls-{torch.__version__}-{sys.version_info[0]}{sys.version_info[1]}-"
                                 f"{h.hexdigest()[:12]}.so")


def _build_calls(out):
    """Compile the FP4 calls' extension; returns an error text, or None."""
    import torch
    t = os.path.dirname(torch.__file__)
    py = sysconfig.get_paths()["include"]
    try:
        cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    except RuntimeError as e:
        return str(e)
    gxx = shutil.which("g++")
    for need in (gxx, os.path.join(py, "Python.h"), os.path.join(t, "include", "ATen", "core", "Tensor.h")):
        if not need or not os.path.exists(need):
            return f"{need or 'g++'} not found"
    lib = os.path.join(t, "lib")
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-I", py,
           "-isystem", os.path.join(t, "include"), "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", cuda, os.path.join(CSRC, "fp4_calls.cpp"), "-o", out + ".tmp", "-L", lib, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        return r.stderr
    os.replace(out + ".tmp", out)
    return None


def _nvcc():
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]
    return any(os.path.getmtime(d) > t for d in deps)


def _calls_missing():
    calls = calls_path()
    return bool(calls) and not os.path.exists(calls)


def _make_calls():
    """Build the FP4 calls' extension, or leave the reason beside its place."""
    calls = calls_path()
    mark = calls + ".failed"
    os.makedirs(OUT_DIR, exist_ok=True)
    failed = _build_calls(calls)
    # what earlier sources left of this environment's extension
    for end in ("", ".failed"):
        for f in glob.glob(glob.escape(calls.rsplit("-", 1)[0]) + "*.so" + end):
            if f != calls or failed:
                with contextlib.suppress(FileNotFoundError):  # (another process builds too)
                    os.remove(f)
    if failed:
        with open(mark, "w") as f:
            f.write(failed)


def _report_calls():
    """Say so where the binding works without the extension, a few microseconds a call slower."""
    calls = calls_path()
    if calls and os.path.exists(calls + ".failed"):
        with open(calls + ".failed") as f:
            why = f.read().strip().splitlines() or ["no message"]
        print(f"FP4 calls' extension not built ({why[-1][:200]}): the ctypes path is used")


def _compile(nvcc, src, extra):
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, r


def build(force=False, verbose=False, extra_flags=(), retry=False):
    """Compile and link libpa.so; return its path.  retry: the FP4 calls' extension even if it failed before."""
    stale = force or _stale()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        made = None
        if calls_path() and (stale or _calls_missing() and (retry or not os.path.exists(calls_path() + ".failed"))):
            made = ex.submit(_make_calls)
        if stale:
            _build_lib(verbose, extra_flags)
        if made:
            made.result()
    _report_calls()
    return LIB


def _build_lib(verbose, extra_flags):
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    objs = []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        for src, obj, r in ex.map(lambda s: _compile(nvcc, s, list(extra_flags)), SOURCES):
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
            if verbose and r.stderr:
                print(r.stderr)
            objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra, retry=True))
