"""Build libpkv.so in-tree with nvcc for sm_103a, and _torch_calls.so with g++.

Each translation unit compiles in its own process (in parallel), then nvcc
links the shared library and g++ the Python module that calls it with torch
tensors (against the installed torch's headers and libraries; without a torch
the library is built alone).  The CUDA runtime is linked statically; the
driver's tensor-map encoder is looked up at run time, so the library loads
on a machine without a GPU (the host scheduler works there).
"""
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
CALLS = os.path.join(HERE, "_torch_calls.so")

SOURCES = ["abi.cu", "append.cu", "decode.cu", "decode_static.cu", "prefill.cu", "prefill_tc.cu", "mixed.cu",
           "tables.cu", "rope.cu", "window_decode.cu", "window_prefill.cu", "host_sched.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pkv.h"), __file__]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc(), "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
           "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cu"):
        cmd[1:1] = ARCH + ["--expt-relaxed-constexpr"]
        if verbose_ptxas:
            cmd.insert(1, "-Xptxas=-v")
    else:
        cmd[1:1] = ["-x", "c++"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), res.stderr))
    if verbose_ptxas and res.stderr:
        print(res.stderr)
    return obj


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found")
    return list(spec.submodule_search_locations)[0]


def _torch_built_for():
    """What _torch_calls.so is made for: the Python and the torch that import it.  None without a torch."""
    try:
        torch = _torch_dir()
    except RuntimeError:
        return None
    text = "%s\n%s\n" % (sysconfig.get_config_var("SOABI"), torch)
    version = os.path.join(torch, "version.py")
    if os.path.exists(version):
        with open(version) as f:
            text += f.read()
    return text


def _run(what: str, cmd) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, " ".join(cmd), res.stderr))


def _compile_calls() -> str:
    torch, obj = _torch_dir(), os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    _run("g++", ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", os.path.join(torch, "include"), "-I",
                 os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I",
                 sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), "-c",
                 os.path.join(CSRC, "torch_calls.cpp"), "-o", obj])
    return obj


def _link_calls(obj: str) -> None:
    tmp = CALLS + ".tmp.%d" % os.getpid()
    _run("link", ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN", "-L",
                  os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, CALLS)


def _link(objs) -> None:
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-lrt", "-ldl", "-lpthread"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), res.stderr))
    os.replace(tmp, LIB)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """libpkv.so where it is older than its sources; then _torch_calls.so where it is, or was made for another torch or
    Python.  libpkv.so needs no torch: without one it is built alone (the calls of _torch_calls.so say what is missing),
    and where _torch_calls.so cannot be made it is in its place before the error is raised."""
    newest = _inputs_mtime()
    fresh = lambda p: not force and os.path.exists(p) and os.path.getmtime(p) >= newest   # noqa: E731
    made_for, wanted = os.path.join(BUILD, "torch_calls.for"), _torch_built_for()
    lib_fresh, calls_fresh = fresh(LIB), wanted is None
    if fresh(CALLS) and os.path.exists(made_for):
        with open(made_for) as f:
            calls_fresh = calls_fresh or f.read() == wanted
    if lib_fresh and calls_fresh:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = [] if lib_fresh else [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        calls = None if calls_fresh else ex.submit(_compile_calls)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if objs:
        _link(objs)
    if calls is not None:
        _link_calls(calls.result())
        with open(made_for, "w") as f:
            f.write(wanted)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
