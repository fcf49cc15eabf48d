"""The host code of rotary positions, attention and the gated layer under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU: the host tests, and
random shapes through the checks, the planning and the launches, with the
runtime's device query and launch replaced by a stub that takes any launch."""
import sys

from test_sanitize_host import _run
from test_sanitize_train_host import clean, sanitized  # noqa: F401

SHAPES = r"""
import ctypes, os, random, sys
sys.path[:0] = [os.path.join(os.getcwd(), "tests"), os.getcwd()]
import ssim_loss_amd as S
from test_block_host import (I32, I64, AttentionInputs, GatedGrads, GatedInputs, RotaryInputs)
lib, stub = S.train.lib(), ctypes.CDLL(os.environ["HIP_STUB"])
stub.stub_launches.restype = stub.stub_bad.restype = ctypes.c_long
rng = random.Random(2)
spread = lambda most: int(2 ** rng.uniform(0, most))
at = lambda k: k << 45
calls = 0
for _ in range(4000):
    dtype = rng.randrange(3)
    heads_kv = rng.choice([1, 2, 3, 8, 40])
    group = rng.choice([1, 1, 2, 5, 16])
    batch, tokens = rng.choice([1, 2, 7, 64]), spread(17)
    # rotary
    dim = rng.choice([2, 7, 64, 72, 128, 512, spread(9)])
    axes, left = [], max(dim, 2) // 2
    dim = max(dim, 2)
    for _ in range(rng.randint(1, 4)):
        if left:
            axes.append(2 * rng.randint(1, left))
            left -= axes[-1] // 2
    st = lambda n, h, d: (I64 * 3)(n * h * d, h * d, d)
    q_heads = heads_kv * group
    tokens = max(1, min(tokens, (1 << 38) // (batch * q_heads * dim)))  # (what 288 GB can hold)
    r = RotaryInputs(at(1), rng.choice([None, at(2)]), at(3), st(tokens, q_heads, dim), st(tokens, heads_kv, dim),
                     (I64 * 2)(rng.choice([0, tokens * len(axes)]), len(axes)), batch, tokens, q_heads, heads_kv, dim, len(axes),
                     (I32 * 4)(*axes), rng.randrange(2), rng.randrange(3), dtype, rng.randrange(2), rng.choice([1.5, 1e4]))
    assert lib.ssim_rotary(ctypes.byref(r), at(4), at(5) if r.k else None, None) == 0, (batch, tokens, q_heads, heads_kv, dim, axes)
    # attention
    dim = 8 * rng.randint(1, 16)
    n, m = rng.choice([0, 1, spread(14)]), rng.choice([0, 1, spread(14)])
    a = AttentionInputs(at(1), at(2), at(3), rng.choice([None, at(4)]), rng.choice([None, at(4) + 4096]), st(n, q_heads, dim),
                        st(m, heads_kv, dim), st(m, heads_kv, dim), batch, n, m, q_heads, heads_kv, dim, rng.randrange(2), dtype, 0,
                        0.125)
    assert lib.ssim_attention_workspace_bytes(ctypes.byref(a)) % 16 == 0
    assert lib.ssim_attention_forward(ctypes.byref(a), at(5), at(6), at(7), at(8), None) == 0
    assert lib.ssim_attention_backward_workspace_bytes(ctypes.byref(a)) % 16 == 0
    assert lib.ssim_attention_backward(ctypes.byref(a), at(5), at(6), at(7), at(9), at(10), at(11), at(12), at(8), None) == 0
    # the gated layer
    rows, width, hidden = rng.choice([0, 1, 64, 65, spread(18)]), spread(14), spread(14)
    g = GatedInputs(at(1) + rng.choice([0, 0, 4]), at(2), at(3), rng.choice([None, at(4)]), rng.choice([None, at(5)]), rows, width,
                    hidden, rng.randrange(3), dtype)
    assert lib.ssim_gated_linear_workspace_bytes(ctypes.byref(g)) % 16 == 0
    assert lib.ssim_gated_linear_forward(ctypes.byref(g), at(6), at(7), at(8), at(9), None) == 0
    assert lib.ssim_gated_linear_backward_workspace_bytes(ctypes.byref(g)) % 16 == 0
    some = GatedGrads(*[rng.choice([None, at(10 + k)]) for k in range(3)], at(13) if g.b_gate else None, at(14) if g.b_up else None)
    assert lib.ssim_gated_linear_backward(ctypes.byref(g), at(7), at(8), at(15), ctypes.byref(some), at(9), None) == 0
    calls += 5
assert stub.stub_launches() >= calls and stub.stub_bad() == 0, (stub.stub_launches(), stub.stub_bad())
print("shapes done", stub.stub_launches())
"""


def test_host_tests_under_asan_ubsan(sanitized):  # noqa: F811
    out = clean(_run([sys.executable, "-m", "pytest", "tests/test_block_host.py", "-q", "-x",
                      "-k", "not binding and not oracle and not tangent and not tracers", "-p", "no:cacheprovider"], sanitized["env"]))
    assert " passed" in out


def test_shapes_under_asan_ubsan(sanitized):  # noqa: F811
    env = {**sanitized["env"], "LD_PRELOAD": sanitized["runtime"] + ":" + sanitized["stub"]}
    assert "shapes done" in clean(_run([sys.executable, "-c", SHAPES], env))
