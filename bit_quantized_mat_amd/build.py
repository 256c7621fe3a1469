"""Build step for the HIP library: compiles every ``csrc/*.hip`` source for
gfx950 into ``bit_quantized_mat_amd/libbqm.so`` (in-tree, so the built
library travels with the source tree), and the Python bindings of its attention
and token sides, ``binding/attention.cpp`` and ``binding/tokens.cpp``, into
``_attention.so`` and ``_tokens.so`` beside it."""
import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbqm.so")
# calibration kernels used only by bench.py (empty dispatch, streaming read)
PROBE_SRC = os.path.join(HERE, "probes", "probes.hip")
PROBE_LIB = os.path.join(HERE, "libbqm_probes.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    # no packed-fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # every fp32 operation rounds once, as written; fused multiply-adds only
    # where the source calls fmaf (HIP's default would also fuse a product
    # with its fp16 conversion, rounding once instead of twice)
    "-ffp-contract=off",
    "-Wall", "-Wno-unused-function",
]


BINDING_SRC = os.path.join(HERE, "binding", "attention.cpp")
BINDING_LIB = os.path.join(HERE, "_attention.so")
TOKENS_SRC = os.path.join(HERE, "binding", "tokens.cpp")
CXX = os.environ.get("CXX", "g++")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


OBJ_DIR = os.path.join(HERE, "_build")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)


def _compile(srcs, out, verbose):
    """Each source to its own object (in parallel: every translation unit
    holds its own kernels and launchers), then one shared library."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    inc = ["-I", os.path.join(HERE, "..", "include")]
    objs = [os.path.join(OBJ_DIR, os.path.basename(s) + ".%d.o" % os.getpid()) for s in srcs]
    jobs = max(1, min(len(srcs), int(os.environ.get("MAX_JOBS", os.cpu_count() or 1))))
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        list(ex.map(lambda so: _run([HIPCC, *FLAGS, *inc, "-c", so[0], "-o", so[1]], verbose),
                    zip(srcs, objs)))
    tmp = out + ".tmp%d" % os.getpid()
    try:
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp], verbose)
        os.replace(tmp, out)
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)


def _binding_includes():
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    return [root, os.path.join(root, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"]]


def _binding_lacks():
    """What the binding's build needs, beside the C library, and does not find; or None."""
    if shutil.which(CXX) is None:
        return CXX
    try:
        inc = _binding_includes()
    except ImportError:
        return "torch"
    for d, f in ((inc[0], "torch/csrc/utils/pybind.h"), (inc[2], "Python.h")):
        if not os.path.exists(os.path.join(d, f)):
            return f
    return None


def _bindings():
    """(source, library) of each binding."""
    return [(BINDING_SRC, BINDING_LIB),
            (TOKENS_SRC, os.path.join(os.path.dirname(BINDING_LIB), "_tokens.so"))]


def _compile_binding(src, obj, verbose):
    """A binding's object: host code against torch's headers."""
    import torch
    inc = _binding_includes()
    _run([CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
          *[a for i in inc for a in ("-isystem", i)], "-c", src, "-o", obj], verbose)


def _link_binding(obj, out, verbose):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp%d" % os.getpid()
    _run([CXX, "-shared", obj, "-o", tmp, "-L" + HERE, "-l:" + os.path.basename(LIB), "-L" + lib,
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib],
         verbose)
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    """Compile the library, its Python bindings and the benchmark's probe
    library (always recompiles); returns the library path. The C libraries need
    hipcc alone: where what the bindings need is not there, they are left out (and
    older ones taken away), and the Python names of the attention and token sides
    raise when called."""
    lacks = _binding_lacks()
    if lacks:
        _compile(sources(), LIB, verbose)
        _compile([PROBE_SRC], PROBE_LIB, verbose)
        for _, lib in _bindings():
            if os.path.exists(lib):
                os.remove(lib)
        print("bit_quantized_mat_amd: built without the Python bindings of the attention and token "
              "sides (%s not found)" % lacks, file=sys.stderr)
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    made = [(src, os.path.join(OBJ_DIR, os.path.basename(src) + ".%d.o" % os.getpid()), lib)
            for src, lib in _bindings()]
    try:
        with concurrent.futures.ThreadPoolExecutor(len(made)) as ex:
            bindings = [ex.submit(_compile_binding, src, obj, verbose) for src, obj, _ in made]
            _compile(sources(), LIB, verbose)
            _compile([PROBE_SRC], PROBE_LIB, verbose)
            for b in bindings:
                b.result()
        for _, obj, lib in made:
            _link_binding(obj, lib, verbose)
    finally:
        for _, obj, _ in made:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
