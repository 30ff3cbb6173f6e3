"""Build ``libbitlinear.so`` in-tree for sm_100a with nvcc, and the native
torch binding ``_native.so`` over it with the host compiler.

    python bit_linear_layers_b200/build.py [--verbose-ptxas]

(Run it by path: importing the package loads the library it builds.)

nvcc cross-compiles, so this runs on machines without a GPU.
"""
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", f) for f in ("bl_api.cu", "bl_norm.cu", "bl_norm_grad.cu")]
LIB = os.path.join(PKG, "libbitlinear.so")
BINDING_SRC = os.path.join(PKG, "csrc", "bl_binding.cpp")
BINDING = os.path.join(PKG, "_native.so")
INCLUDE = os.path.join(ROOT, "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-Wall",
    "--expt-relaxed-constexpr",
]


def sources():
    d = os.path.join(PKG, "csrc")
    return [os.path.join(d, f) for f in sorted(os.listdir(d)) if f.endswith((".cu", ".cuh", ".cpp"))]


def build(verbose_ptxas: bool = False, out: str = LIB) -> str:
    nvcc = os.environ.get("NVCC", "nvcc")
    flags = (["-Xptxas=-v"] if verbose_ptxas else []) + NVCC_FLAGS
    with tempfile.TemporaryDirectory() as tmp:  # the translation units side by side
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SRCS]
        running = [subprocess.Popen([nvcc, *flags, "-I", INCLUDE, "-c", "-o", o, s]) for s, o in zip(SRCS, objs)]
        failed = [s for s, p in zip(SRCS, running) if p.wait() != 0]
        if failed:
            raise RuntimeError(f"nvcc failed on {', '.join(failed)}")
        subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", out, *objs], check=True)
    if out == LIB:
        build_binding()
    return out


def build_binding(out: str = BINDING) -> str:
    """The torch binding: links the C ABI library beside it and torch's own libraries."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths(device_type="cuda")]
    libs = cpp_extension.library_paths(device_type="cpu")
    # the system's g++, whatever $CXX names: exceptions cross into torch's libraries, so both have to use the
    # one shared libstdc++ (a compiler that links its own statically gives a binding that crashes on a refusal)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{p}" if p != INCLUDE else f"-I{p}" for p in inc), "-o", out, BINDING_SRC,
           f"-L{PKG}", "-l:libbitlinear.so", *(f"-L{p}" for p in libs), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN", *(f"-Wl,-rpath,{p}" for p in libs)]
    subprocess.run(cmd, check=True)
    return out


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    deps = sources() + [os.path.join(INCLUDE, "bitlinear.h")]
    return any(os.path.getmtime(p) > t for p in deps)


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv))
