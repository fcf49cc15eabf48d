"""Build step for the HIP libraries: the translation units under csrc/ are
compiled in parallel with ``hipcc`` for gfx950 and linked into
``ssim_loss_amd/libssim_loss_amd.so``, those under train/csrc/ (the training
operators) into ``ssim_loss_amd/train/libssim_train_amd.so``.  The second
library's binding to torch, train/csrc/bind*.cpp, becomes the Python module
``ssim_loss_amd/train/_bind.so``.

Packed-FP32 instructions are switched off (``-packed-fp32-ops``); the kernels
are written so that nothing depends on them.  Floating-point contraction is
limited to single expressions (``-ffp-contract=on``, not HIP's default of
fusing across statements): every fused multiply-add the arithmetic relies on
is written out, and a product stored to a variable must stay rounded -- the
forward's blurs by parts are exact on constant windows only if, say, a
squared difference is rounded before the difference from its neighbour is
taken.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
HEADERS = sorted(glob.glob(os.path.join(CSRC, "*.hpp")))
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libssim_loss_amd.so")
ARCH = "gfx950"

TRAIN = os.path.join(PKG, "train")
TRAIN_CSRC = os.path.join(TRAIN, "csrc")
TRAIN_INCLUDE = os.path.join(TRAIN, "include")
TRAIN_SOURCES = sorted(glob.glob(os.path.join(TRAIN_CSRC, "*.hip")))
TRAIN_LIB_PATH = os.path.join(TRAIN, "libssim_train_amd.so")
BIND_PATH = os.path.join(TRAIN, "_bind.so")
BIND_SOURCES = sorted(glob.glob(os.path.join(TRAIN_CSRC, "bind*.cpp")))


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def compile_flags(extra: list[str] | None = None) -> list[str]:
    return [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-ffp-contract=on",
            "-I", INCLUDE, "-I", CSRC, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            *(extra or [])]


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def _build_library(sources: list[str], flags: list[str], verbose: bool, build_dir: str,
                   lib_path: str, link: tuple = ()) -> str:
    os.makedirs(build_dir, exist_ok=True)
    cc = hipcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        _run([cc, *flags, "-c", "-o", obj, src], verbose)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(sources))) as pool:
        objs = list(pool.map(compile_one, sources))
    tmp = lib_path + ".tmp"
    _run([cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *link, "-o", tmp, *objs], verbose)
    os.replace(tmp, lib_path)
    return lib_path


def build(verbose: bool = False, extra: list[str] | None = None, build_dir: str = BUILD_DIR,
          lib_path: str = LIB_PATH) -> str:
    """Compile every csrc/*.hip and link lib_path.  `extra` compile flags go
    to every translation unit (a variant build, e.g. with host-side
    sanitizers, names its own build_dir and lib_path)."""
    return _build_library(SOURCES, compile_flags(extra), verbose, build_dir, lib_path)


def build_train(verbose: bool = False, extra: list[str] | None = None,
                build_dir: str = os.path.join(BUILD_DIR, "train"),
                lib_path: str = TRAIN_LIB_PATH) -> str:
    """Compile every train/csrc/*.hip and link lib_path; `extra` as for build."""
    flags = compile_flags(["-I", TRAIN_INCLUDE, "-I", TRAIN_CSRC, *(extra or [])])
    # (by this name the binding asks for it)
    soname = f"-Wl,-soname,{os.path.basename(TRAIN_LIB_PATH)}"
    return _build_library(TRAIN_SOURCES, flags, verbose, build_dir, lib_path, (soname,))


def build_bind(verbose: bool = False) -> str:
    """Compile train/csrc/bind*.cpp against torch's headers and link them with
    the training library, which they find beside themselves."""
    import torch

    inside = os.path.dirname(torch.__file__)
    tmp = BIND_PATH + ".tmp"
    includes = [os.path.join(inside, "include"),
                os.path.join(inside, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"),
                "/opt/rocm/include", sysconfig.get_paths()["include"]]
    compiler = [shutil.which("g++") or shutil.which("c++")]
    if compiler == [None]:  # (torch's names are those of g++, and of clang up to this version)
        compiler = [os.path.join(os.path.dirname(hipcc()), "amdclang++"), "-fclang-abi-compat=17"]
    cmd = [*compiler, "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared",
           "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", TRAIN_INCLUDE,
           *(a for d in includes if os.path.isdir(d) for a in ("-isystem", d)),
           "-o", tmp, *BIND_SOURCES,
           "-L", os.path.join(inside, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch",
           "-ltorch_python", TRAIN_LIB_PATH, "-Wl,-rpath,$ORIGIN"]
    _run(cmd, verbose)
    os.replace(tmp, BIND_PATH)
    return BIND_PATH


def build_all(verbose: bool = False) -> list[str]:
    """Both libraries, which need hipcc alone, and the binding where torch for
    ROCm is installed."""
    built = [build(verbose), build_train(verbose)]
    try:
        import torch

        missing = not torch.version.hip
    except ImportError:
        missing = True
    if missing:
        print("the training operators' binding is not built: it needs torch for ROCm", file=sys.stderr)
        return built
    return [*built, build_bind(verbose)]


if __name__ == "__main__":
    print(*build_all(verbose=True), sep="\n")
