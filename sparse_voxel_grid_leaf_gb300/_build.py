"""Builds libtb.so in-tree with nvcc for sm_103a (GB300), and _seq.so, the
Python entry points of its sequence operators, with the host compiler where
torch is installed.

The translation units compile in parallel and are linked with the static
CUDA runtime, so the library needs only the NVIDIA driver at run time.
"""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtb.so")
SEQ, SEQ_OBJ = os.path.join(HERE, "_seq.so"), os.path.join(BUILD, "tb_seq_py.o")
SOURCES = ["tb_api.cu", "tb_prepass.cu", "tb_chain.cu", "tb_noalloc.cu", "tb_kmap.cu",
           "tb_seq_api.cu", "tb_rotary.cu", "tb_norm.cu", "tb_linattn.cu",
           "tb_linattn_chunk.cu", "tb_linattn_split.cu", "tb_conv.cu", "tb_scan.cu",
           "tb_scan_join.cu", "tb_scan_backward.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is needed to build libtb.so")


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch():
    """The folder of the installed torch, or None."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec else None


def _torch_version(root):
    """What _seq.so is built for, as text: it links torch's C++ ABI, which differs between versions."""
    with open(os.path.join(root, "version.py")) as f:
        return f.read()


def _torch_command(root):
    """The compiler command of _seq.so up to its inputs, and torch's library folder."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "c++"
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden"] + [x for i in inc for x in ("-isystem", i)], \
        os.path.join(root, "lib")


def build(force=False, verbose=False, extra_flags=()):
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    headers.append(os.path.join(os.path.dirname(HERE), "include", "tb.h"))
    objs = []
    jobs = []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", path, "-o", obj])

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return r

    built = len(jobs)
    seq_src, torch = os.path.join(CSRC, "tb_seq_py.cpp"), _torch()
    if torch:
        cxx, torch_lib = _torch_command(torch)
        made_for, target = SEQ_OBJ + ".torch", " ".join(cxx) + "\n" + _torch_version(torch)
        other = True
        if os.path.exists(made_for):
            with open(made_for) as f:
                other = f.read() != target
        if force or other or _stale(SEQ_OBJ, [seq_src] + headers):
            jobs.append([*cxx, "-c", seq_src, "-o", SEQ_OBJ])
    else:
        print("torch is not installed: _seq.so, the Python entry points of the sequence operators, is left out",
              file=sys.stderr)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        list(ex.map(run, jobs))
    if force or built or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if torch and (force or other or _stale(SEQ, [SEQ_OBJ, LIB])):
        tmp = SEQ + ".tmp%d" % os.getpid()
        run([cxx[0], "-shared", "-o", tmp, SEQ_OBJ, "-L", HERE, "-l:libtb.so", "-Wl,-rpath,$ORIGIN", "-L", torch_lib,
             "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"])
        os.replace(tmp, SEQ)
        with open(made_for, "w") as f:
            f.write(target)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
