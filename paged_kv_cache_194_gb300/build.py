"""Build step for libpkv.so: compiles csrc/*.cu for sm_103a with nvcc (one
process per translation unit, in parallel) and links a shared library next to
this file.  The CUDA runtime is linked statically and the driver is never
linked, so the library loads on machines without a GPU driver (its entry
points then fail with a CUDA error instead).

Beside it goes _pkvstep.so, the CPython module of csrc_python/ (argument checks
on torch tensors), compiled with the host compiler against torch's headers and
linked to libpkv.so."""
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkv.so")
STEP_SRC = os.path.join(HERE, "csrc_python", "step_calls.cpp")
STEP_LIB = os.path.join(HERE, "_pkvstep.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _cxx() -> str:
    for c in (os.environ.get("CXX"), shutil.which("g++"), shutil.which("c++")):
        if c:
            return c
    raise RuntimeError("no C++ compiler")


def _torch_dir() -> str:
    import torch  # (its headers and libraries only)

    return os.path.dirname(torch.__file__)


def _torch_include():
    inc = os.path.join(_torch_dir(), "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include")]


def _torch_lib() -> str:
    return os.path.join(_torch_dir(), "lib")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps():
    out = [os.path.join(INCLUDE, "pkv.h")]
    out += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return out


def _stale(target, inputs):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(i) > t for i in inputs)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(OBJ, exist_ok=True)
    deps = _deps()
    jobs = []
    objs = []
    step_obj = os.path.join(OBJ, "step_calls_python.o")
    step_stale = force or _stale(step_obj, [STEP_SRC, os.path.join(INCLUDE, "pkv.h"),
                                             os.path.join(_torch_dir(), "version.py"), os.path.abspath(__file__)])
    if step_stale:
        jobs.append([_cxx(), "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE,
                     "-isystem", sysconfig.get_paths()["include"]]
                    + [x for p in _torch_include() for x in ("-isystem", p)] + ["-c", STEP_SRC, "-o", step_obj])
    for src in sources():
        obj = os.path.join(OBJ, os.path.splitext(os.path.basename(src))[0] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + deps):
            if src.endswith(".cpp"):  # host-only C++
                cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-c", src, "-o", obj]
            else:
                cmd = [nvcc] + ARCH + FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
            jobs.append(cmd)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = [ex.submit(subprocess.run, cmd, capture_output=True, text=True) for cmd in jobs]
            for cmd, f in zip(jobs, futs):
                r = f.result()
                if verbose or r.returncode != 0:
                    sys.stderr.write(r.stdout + r.stderr)
                if r.returncode != 0:
                    raise RuntimeError("nvcc failed: " + " ".join(cmd))
    if force or len(jobs) > int(step_stale) or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, LIB)
    if step_stale or _stale(STEP_LIB, [step_obj]):
        tmp = STEP_LIB + ".tmp%d" % os.getpid()
        r = subprocess.run([_cxx(), "-shared", "-o", tmp, step_obj, "-L", HERE, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN",
                            "-L", _torch_lib(), "-ltorch_python", "-ltorch_cpu", "-lc10"], capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(tmp, STEP_LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
