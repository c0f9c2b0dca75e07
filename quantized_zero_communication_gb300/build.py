"""Build ``libzpp.so`` in-tree with nvcc for sm_103a, and the Python extension ``_tensors`` with
the host compiler against torch's headers (no torch extension machinery).

Each translation unit compiles in parallel into ``_build/``; the objects link into one
shared library (CUDA runtime linked statically). Numerics flags: -fmad=false (no FMA
contraction), IEEE division and square root, denormals kept.
"""
import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libzpp.so")
EXT = os.path.join(PKG, "_tensors.so")
EXT_ABI = os.path.join(BUILD, "_tensors.abi")  # what EXT was compiled against
SOURCES = ["zpp_abi.cu", "quant.cu", "reorder_quant.cu", "reorder_tensors_f16.cu",
           "reorder_tensors_bf16.cu", "dequant.cu", "qgz.cu", "adamw.cu", "grad_norm.cu",
           "matvec.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++20", "-O3", "-lineinfo", "-fmad=false", "-prec-div=true", "-prec-sqrt=true",
         "-ftz=false", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libzpp")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return files + [os.path.join(INCLUDE, "zpp.h"), __file__]


def _stale(out):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in _inputs())


def ext_abi():
    """The torch and the Python that the extension is for; None without a torch with CUDA (the C
    library needs none)."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    if torch.version.cuda is None:
        return None
    return f"torch {torch.__version__}, Python {sysconfig.get_config_var('SOABI')}"


def built_ext_abi():
    """Those that the extension in place was compiled against; None if that is not known."""
    try:
        with open(EXT_ABI) as f:
            return f.read()
    except OSError:
        return None


def _build_ext():
    import torch
    root = os.path.dirname(torch.__file__)
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(CSRC, "tensor_access.cpp"), "-o", tmp, "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(root, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling tensor_access.cpp failed:\n{r.stderr}")
    if os.path.exists(EXT_ABI):
        os.remove(EXT_ABI)
    os.replace(tmp, EXT)
    with open(EXT_ABI, "w") as f:
        f.write(ext_abi())


def build(force: bool = False, verbose: bool = False) -> str:
    """Brings libzpp.so up to date, and the extension where torch is there; an extension that does not
    compile is an error, raised once the library is in place."""
    lib = force or _stale(LIB)
    abi = ext_abi()
    ext = abi is not None and (force or _stale(EXT) or built_ext_abi() != abi)
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(1) as ex:
        made = ex.submit(_build_ext) if ext else None
        if lib:
            _build_lib(verbose)
        if made:
            made.result()
    return LIB


def _build_lib(verbose):
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src),
               "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        for _, log in results:
            print(log)


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
