"""In-tree build of libmk.so for sm_103a with nvcc (no cmake, no torch extension machinery).

The translation units compile in parallel; the shared library links the CUDA runtime
statically, so loading it needs no CUDA driver (host-only entry points such as
mk_plan work on a machine without a GPU).  Beside it a small extension module passes torch
tensors to the paged operators; it wants g++ and a torch with CUDA, and where either is missing
libmk.so is built alone (paged.py then does not import).
"""
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_objs")
LIB = os.path.join(HERE, "libmk.so")
EXT = os.path.join(HERE, "_mk_torch.so")  # the paged operators on torch tensors (paged.py)
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = [f"mk_k_{d}_{s}{m}{t}.cu" for d in ("f16", "bf16") for s in ("counter", "sentinel") for m in ("", "_ms")
           for t in ("", "_am", "_tc")] + ["mk_kernel.cu", "mk_host.cu", "mk_plan.cpp", "mk_tmap.cpp", "mk_noalloc.cu",
                                           "mk_append.cu", "mk_attend.cu", "mk_pages.cu", "mk_select.cu",
                                           "mk_tree.cu", "mk_accept.cu", "mk_blocks.cu"]


def _nvcc():
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "mk.h"))
    files.append(os.path.abspath(__file__))
    return files


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _torch_of():
    """(folder, what identifies it) of the torch an extension would be built against, or (None, why there is none)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        spec = None
    if spec is None or not spec.submodule_search_locations:
        return None, "torch is not installed"
    root = list(spec.submodule_search_locations)[0]
    if not os.path.exists(os.path.join(root, "lib", "libc10_cuda.so")):
        return None, "torch is without CUDA"
    if shutil.which("g++") is None:
        return None, "g++ is missing"
    with open(os.path.join(root, "version.py")) as f:
        return root, f"{sys.version_info[:2]} {root}\n{f.read()}"


def _extension_command(nvcc):
    """The compile of the torch extension module (host code; torch's headers, libmk.so linked after)."""
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)) if os.path.isabs(nvcc) else "/usr/local/cuda", "include")
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda]
    obj = os.path.join(OBJ, "mk_torch.o")
    comp = ["g++", "-O2", "-std=c++17", "-fPIC", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    comp += [f"-I{d}" for d in inc] + ["-c", os.path.join(CSRC, "mk_torch.cpp"), "-o", obj]
    lib = os.path.join(root, "lib")
    link = ["g++", "-shared", obj, "-o", EXT + ".tmp", f"-L{HERE}", "-l:libmk.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}",
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return comp, link


def build(force=False, verbose=False, ptxas_info=False):
    """Compile and link libmk.so, and the torch extension where it can be, if any source (or torch) changed; returns
    the library's path."""
    deps = _deps()
    root, torch_id = _torch_of()
    stamp = os.path.join(OBJ, "mk_torch.stamp")  # the torch that the extension was built against
    need_lib = force or _stale(LIB, deps)
    need_ext = root is not None and (force or _stale(EXT, deps) or not os.path.exists(stamp) or open(stamp).read() != torch_id)
    if need_lib and root is None:
        print(f"the torch extension of the paged operators (paged.py) is not built: {torch_id}", file=sys.stderr)
    if not need_lib and not need_ext:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", CSRC, "-I", INCLUDE]

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + common + ARCH + ["-lineinfo", "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cu"):
            cmd += ["-Xcudafe", "--diag_suppress=177"]
            if ptxas_info:
                cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    logs = ""
    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        if need_ext:
            ext_compile, ext_link = _extension_command(nvcc)
            ext = ex.submit(subprocess.run, ext_compile, capture_output=True, text=True)
        results = list(ex.map(compile_one, SOURCES)) if need_lib else []
    if need_lib:
        logs = "".join(r[1] for r in results)
        if verbose and logs:
            print(logs, file=sys.stderr)
        tmp = LIB + ".tmp"
        cmd = [nvcc, "-shared"] + ARCH + ["-o", tmp] + [r[0] for r in results]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if need_ext:  # (libmk.so is in place by now, whatever becomes of it)
        if ext.result().returncode != 0:
            raise RuntimeError(f"g++ failed on mk_torch.cpp:\n{ext.result().stdout}\n{ext.result().stderr}")
        r = subprocess.run(ext_link, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of the torch extension failed:\n{r.stdout}\n{r.stderr}")
        os.replace(EXT + ".tmp", EXT)
        with open(stamp, "w") as f:
            f.write(torch_id)
    return (LIB, logs) if ptxas_info else LIB


if __name__ == "__main__":
    out = build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(out if isinstance(out, str) else out[1])
