"""Build libpkv.so and its Python binding in-tree for sm_103a (GB300).

Each CUDA translation unit under csrc/ is compiled with nvcc in parallel,
then linked into paged_kv_cache_mapping_gb300/libpkv.so (static CUDA
runtime, so the library loads without a GPU; the driver is opened at the
first CUDA call).  Beside them g++ compiles csrc/pkv_binding.cpp, the CPython
module that marshals PyTorch tensors for the calls made once per layer of a
speculative step.  Run ``python -m paged_kv_cache_mapping_gb300.build``.
"""
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
BINDING_SRC = os.path.join(CSRC, "pkv_binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "binding_for.txt")  # what the binding was built against
SOURCES = ["pkv_api.cu", "pkv_append.cu", "pkv_plan.cu", "pkv_decode.cu", "pkv_prefill.cu", "pkv_f32.cu", "pkv_static_ws.cu", "pkv_prefill_tc.cu", "pkv_blocks.cu",
           "pkv_spec_api.cu", "pkv_rope.cu", "pkv_tree.cu", "pkv_tree_tc.cu", "pkv_tree_wide.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def binding_command(out: str):
    """g++ on the binding, against the headers and libraries of the PyTorch that is installed."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    system = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{os.path.join(ROOT, 'include')}",
            *(f"-isystem{d}" for d in system), BINDING_SRC, "-o", out, f"-L{os.path.join(root, 'lib')}",
            f"-Wl,-rpath,{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def binding_target() -> str:
    """The Python and PyTorch that a binding links against (PyTorch is not imported for this)."""
    torch = importlib.util.find_spec("torch").origin
    with open(os.path.join(os.path.dirname(torch), "version.py")) as f:
        return "\n".join([sys.version, torch, f.read()])


def _binding_stale() -> bool:
    if _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "pkv.h"), __file__]) or not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        return f.read() != binding_target()


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers += [os.path.join(ROOT, "include", f) for f in ("pkv.h", "pkv_blocks.h")]
    objs, jobs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s, *headers, __file__]):
            cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", s, "-o", o]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    bind_tmp = BINDING + f".tmp{os.getpid()}"
    new_binding = force or _binding_stale()
    if new_binding:
        jobs.append(binding_command(bind_tmp))
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
    for cmd, r in zip(jobs, results):
        if verbose or r.returncode != 0 or ptxas_info:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    bound = not new_binding or results.pop().returncode == 0
    if any(r.returncode != 0 for r in results):
        raise RuntimeError("nvcc failed")
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    if not bound:  # the library does not need it
        raise RuntimeError("the binding's compiler failed (libpkv.so is built)")
    if new_binding:
        os.replace(bind_tmp, BINDING)
        with open(BINDING_FOR, "w") as f:
            f.write(binding_target())
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv, force="--force" in sys.argv))
