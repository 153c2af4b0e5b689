"""Builds liblsa.so (the C-ABI CUDA library) in-tree for sm_100a, and _binding.so, the native
marshalling of its short calls (csrc/binding.cpp, against torch's headers).

    python -m learned_sparse_kv_b200.build [--force] [--verbose]
"""
import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblsa.so")
BINDING = os.path.join(HERE, "_binding.so")
STAMP = os.path.join(OBJ, "binding.torch")      # the torch and Python that the binding was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC,-O2",
         "-I", os.path.join(ROOT, "include")]


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "lsa.h")]


def _torch_dir():
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _torch_version():
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sys.version}\n{f.read()}"


def _note_torch():
    with open(STAMP, "w") as f:
        f.write(_torch_version())


def _binding_fits():
    """Is the binding there, and built for this torch?"""
    try:
        with open(STAMP) as f:
            return os.path.exists(BINDING) and f.read() == _torch_version()
    except OSError:
        return False


def _build_binding():
    _link_binding(_compile_binding())
    _note_torch()


def _compile_binding():
    """binding.cpp -> binding.o, next to the CUDA objects."""
    torch = os.path.join(_torch_dir(), "include")
    inc = [torch, os.path.join(torch, "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"]]
    obj = os.path.join(OBJ, "binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall", *[f"-isystem{i}" for i in inc], "-c",
           os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the compiler failed for binding.cpp:\n{r.stderr}")
    return obj


def _link_binding(obj):
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{HERE}", "-llsa", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def _compile(src, verbose):
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    return obj, r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles every csrc/*.cu and links liblsa.so, then the binding; skips the work when up to date."""
    if not force and os.path.exists(LIB) and os.path.exists(BINDING):
        t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
        if all(os.path.getmtime(p) <= t for p in _deps()):
            if not _binding_fits():
                os.makedirs(OBJ, exist_ok=True)
                _build_binding()
            return LIB
    os.makedirs(OBJ, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
        binding = binding.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    _note_torch()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
