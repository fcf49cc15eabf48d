"""The training operators' host code under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU.

The library is rebuilt with both on the host pass only (device code is built as
usual), and child processes that preload the ASan runtime run its host tests,
and random lists of tensors through the planning of launches: there the
runtime's device query and launch are replaced by a stub that takes any launch.
Any report ends the child with an error.  Skipped where the toolchain or the
runtime is absent."""
import importlib
import os
import subprocess
import sys

import pytest

from test_sanitize_host import REPORTS, _asan_runtime, _run

HOST_TESTS = ["tests/test_train_host.py", "tests/test_train_groups_host.py"]

STUB = r"""
#include <hip/hip_runtime_api.h>
#include <string.h>
static long launches = 0, bad = 0;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* p, int) {
  memset(p, 0, sizeof(*p));
  p->warpSize = 64;
  p->multiProcessorCount = 256;
  strcpy(p->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void** args, size_t lds, hipStream_t) {
  ++launches;
  bad += !f || !args || !args[0] || lds != 0 || g.x < 1 || g.y < 1 || g.z != 1 || g.y > 65535 || b.x < 64 ||
         b.x > 1024 || b.x % 64 != 0 || b.y != 1 || (unsigned long)g.x * b.x > 0xffffffffUL;
  return hipSuccess;
}
long stub_launches(void) { return launches; }
long stub_bad(void) { return bad; }
}
"""

LISTS = r"""
import ctypes, os, random, sys
sys.path[:0] = [os.path.join(os.getcwd(), "tests"), os.getcwd()]
import ssim_loss_amd as S
from test_train_host import AdamItem, AdamOptions, ClipItem, NormGrads, NormInputs
lib, stub = S.train.lib(), ctypes.CDLL(os.environ["HIP_STUB"])
stub.stub_launches.restype = stub.stub_bad.restype = ctypes.c_long
rng = random.Random(1)
spread = lambda most: int(2 ** rng.uniform(0, most))
calls = 0
for _ in range(3000):
    at = [1 << 20]
    packed = rng.random() < 0.5
    def place(nbytes, align):
        at[0] += -at[0] % (align if packed else 512)
        here = at[0]
        at[0] += nbytes
        return here
    count, most = rng.choice([1, 2, 7, 8, 9, 64, 65, 113, 145, 400]), rng.choice([2, 13, 24, 33])
    sizes = [rng.choice([0, spread(most), spread(most), spread(most)]) for _ in range(count)]
    kinds = [rng.randrange(3) for _ in range(rng.choice([1, 1, 3]))]
    kind = lambda k: kinds[k % len(kinds)]
    eb = lambda d: 2 if d else 4
    norm, ws, step = 64, 1024, 128
    grads = [place(n * eb(kind(k)), eb(kind(k))) for k, n in enumerate(sizes)]
    outs = [place(n * eb(kind(k)), eb(kind(k))) for k, n in enumerate(sizes)] if rng.random() < 0.5 else grads
    items = (ClipItem * count)(*[ClipItem(g, o, n, kind(k), 0)
                                 for k, (g, o, n) in enumerate(zip(grads, outs, sizes))])
    assert lib.ssim_clip_grads(items, count, 1.0, norm, ws, None) == 0
    assert lib.ssim_grad_norm(items, count, norm, ws, None) == 0
    masters = rng.random() < 0.5
    held = [[place(n * w, w) for n in sizes] for w in (4, 4, 4)]
    params = [place(n * eb(kind(k)), eb(kind(k))) for k, n in enumerate(sizes)]
    items = (AdamItem * count)(*[AdamItem(grads[k], params[k], held[0][k], held[1][k],
                                          held[2][k] if masters else None, n, kind(k), kind(k))
                                 for k, n in enumerate(sizes)])
    clips = rng.random() < 0.5
    o = AdamOptions(1e-3, 0.9, 0.99, 1e-8, 0.1, 1.0 if clips else float("inf"), None)
    assert lib.ssim_adamw_step(items, count, ctypes.byref(o), step, norm if clips else None, ws, None) == 0
    rows, each, width = spread(16), rng.choice([1, 2, 3, spread(12)]), min(16384, spread(14.1))
    dtype = rng.randrange(3)
    given = NormInputs(1 << 45, 2 << 45, rng.choice([None, 3 << 45]), 4096, 4096, 4096, rows * each, width,
                       each, 1e-6, rng.choice([0, dtype]), dtype, rng.randrange(2), 0)
    assert lib.ssim_block_norm_forward(ctypes.byref(given), 5 << 45, 6 << 45, 7 << 45, None) == 0
    assert lib.ssim_block_norm_workspace_bytes(ctypes.byref(given)) % 16 == 0
    wanted = NormGrads(8 << 45, 9 << 45, 10 << 45 if given.gate else None, 12 << 45, 13 << 45, 14 << 45)
    assert lib.ssim_block_norm_backward(ctypes.byref(given), 7 << 45, 15 << 45, 16 << 45, ctypes.byref(wanted),
                                        17 << 45, None) == 0
    calls += 5
assert stub.stub_launches() >= calls and stub.stub_bad() == 0, (stub.stub_launches(), stub.stub_bad())
print("lists done", stub.stub_launches())
"""


@pytest.fixture(scope="module")
def sanitized(tmp_path_factory):
    runtime = _asan_runtime()
    if runtime is None:
        pytest.skip("clang's AddressSanitizer runtime is not installed")
    if not os.path.exists("/opt/rocm/bin/hipcc"):
        pytest.skip("hipcc is not installed")
    # the module, not the package's build() of the same name
    build = importlib.import_module("ssim_loss_amd.build")
    d = tmp_path_factory.mktemp("sanitize_train")
    host_only = ["-g", "-fno-omit-frame-pointer",
                 "-Xarch_host", "-fsanitize=address,undefined",
                 "-Xarch_host", "-fno-sanitize-recover=undefined"]
    lib = build.build_train(extra=host_only, build_dir=str(d / "obj"),
                            lib_path=str(d / "libssim_train_amd.so"))
    (d / "stub.cpp").write_text(STUB)
    stub = str(d / "libstub.so")
    subprocess.run([build.hipcc(), "-x", "c++", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", "-shared", "-fPIC",
                    "-o", stub, str(d / "stub.cpp")], check=True)
    env = dict(os.environ)
    env.update(LD_PRELOAD=runtime, SSIM_TRAIN_AMD_LIB=lib, HIP_STUB=stub,
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", PYTHONDONTWRITEBYTECODE="1")
    return {"runtime": runtime, "lib": lib, "stub": stub, "env": env}


def clean(result):
    out = result.stdout + result.stderr
    assert result.returncode == 0, out[-6000:]
    for report in REPORTS:
        assert report not in out, out[-6000:]
    return result.stdout


def test_the_sanitized_library_is_the_one_loaded(sanitized):
    code = "import ssim_loss_amd as S; S.train.lib(); print(open('/proc/self/maps').read())"
    maps = clean(_run([sys.executable, "-c", code], sanitized["env"], timeout=300))
    assert sanitized["lib"] in maps and sanitized["runtime"] in maps


def test_host_tests_under_asan_ubsan(sanitized):
    out = clean(_run([sys.executable, "-m", "pytest", *HOST_TESTS, "-q", "-x", "-k", "not binding",
                      "-p", "no:cacheprovider"], sanitized["env"]))
    assert " passed" in out


def test_lists_and_shapes_under_asan_ubsan(sanitized):
    env = {**sanitized["env"], "LD_PRELOAD": sanitized["runtime"] + ":" + sanitized["stub"]}
    assert "lists done" in clean(_run([sys.executable, "-c", LISTS], env))
