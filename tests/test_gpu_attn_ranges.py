"""Attention whose probabilities or values reach far: heavy keys whose values are zero, so that what is left is
the sum of small probabilities, and values near the top of bfloat16.  The bounds are those of
every other test: each probability to the rounding that its operator states, whatever its size."""
import numpy as np
import pytest

from attn_cases import HALF_UNIT, Paged, attention, bound, check, rounded
from gpu_cases import host, say, torch_dev
from test_gpu_attn_prompt import call, on_gpu

pytestmark = pytest.mark.gpu


def far_rows(r, n, H, D, at, gap):
    """Rows k, v of which row `at` stands `gap` nats before the others for a query whose channel 0 is 1 (scale 1), and
    has values of zero."""
    k, v = (r.standard_normal((n, H, D)).astype(np.float32) for _ in "kv")
    k *= 0.25
    k[:, :, 0] = 0.0
    k[at] = 0.0
    k[at, :, 0] = gap
    v[at] = 0.0
    return k, v


def queries(r, n, H, D):
    q = (r.standard_normal((n, H, D)) * 0.25).astype(np.float32)
    q[:, :, 0] = 1.0
    return q


def decode(fmt, seqs, q, D, page, seed, what, heads):
    torch = torch_dev()
    Hq, Hkv = q.shape[1], seqs[0][0].shape[1]
    c = Paged(fmt, seqs, Hkv, D, page, seed)
    got = host(c.decode(torch.from_numpy(q).cuda(), scale=1.0))
    worst = 0.0
    for i, (k, v) in enumerate(c.rows):
        for h in heads:
            j = h * Hkv // Hq
            want, A, S = attention(q[i, h:h + 1], k[:, j], v[:, j], 1.0, np.ones((1, len(k)), bool))
            worst = max(worst, check(got[i, h:h + 1], want, bound(want, A, S, D, len(k), "f32", 0.0, 8), f"{what} sequence {i} head {h}"))
    say(f"  worst error / bound {worst:.3g}")


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("gap", [8, 15, 20, 30, 60])
def test_decode_small_probabilities(fmt, gap):
    """The heavy key first, in the middle and last; 4200 keys in long parts (many key heads) and 601 in short ones."""
    say(f"decode small probabilities {fmt} gap={gap}")
    r = np.random.Generator(np.random.PCG64(gap))
    for n, Hkv, Hq, D, places, heads in ((601, 2, 4, 64, (0, 311, 600), range(4)), (4200, 64, 64, 32, (0, 2100, 4199), (0, 31, 63))):
        seqs = [far_rows(r, n, Hkv, D, at, gap) for at in places]
        decode(fmt, seqs, queries(r, len(seqs), Hq, D), D, 16, gap + n, f"{fmt} gap {gap}", heads)


def test_decode_values_near_the_top_of_bfloat16():
    """Every weighted sum with probabilities up to 1 fits float32 (5000 values below 2^114); scores rise by 7.8 powers of two
    after the first tile, which is less than the running maximum follows at once."""
    say("decode values of 2^113 .. 2^114")
    r = np.random.Generator(np.random.PCG64(4))
    n, Hkv, D = 5000, 64, 32
    k = (r.standard_normal((n, Hkv, D)) * 2.0 ** -6).astype(np.float32)
    k[:, :, 0] = 5.375
    k[:128, :, 0] = 0.0
    v = (r.uniform(0.5, 0.99, (n, Hkv, D)) * 2.0 ** 114).astype(np.float32)
    decode("bf16", [(k, v)], queries(r, 1, Hkv, D), D, 64, 5, "large values", (0, 17, 63))


def prompt(q, k, v, type_, D, what):
    m, n = len(q), len(k)
    cu = [np.array([0, x], np.int32) for x in (m, n)]
    got = host(call(*(on_gpu(x, type_) for x in (q, k, v)), *cu, scale=1.0).float())
    seen = np.arange(n)[None] <= np.arange(m)[:, None] + (n - m)
    worst = 0.0
    for h in range(q.shape[1]):
        want, A, S = attention(q[:, h], k[:, 0], v[:, 0], 1.0, seen)
        worst = max(worst, check(got[:, h], want, bound(want, A, S, D, n, type_, HALF_UNIT[type_], 2), f"{what} head {h}"))
    say(f"  worst error / bound {worst:.3g}")


@pytest.mark.parametrize("type_,gap", [("f16", 8), ("f16", 11), ("f16", 14), ("f16", 16), ("bf16", 16), ("bf16", 30), ("bf16", 60)])
def test_prompt_small_probabilities(type_, gap):
    """The heavy key is the first one, so every query sees it; probabilities down to e^-17 of the largest (binary16)."""
    say(f"prompt small probabilities {type_} gap={gap}")
    r = np.random.Generator(np.random.PCG64(gap))
    D, m, n = 64, 70, 2100
    k, v = (rounded(x, type_) for x in far_rows(r, n, 1, D, 0, gap))
    q = rounded(queries(r, m, 2, D) * np.where(np.arange(D) == 0, 1.0, 0.3).astype(np.float32), type_)
    s = q[:, :, 1:].reshape(-1, D - 1) @ k[:, 0, 1:].T
    assert np.abs(s).max() < 1.0  # so that all probabilities lie within a nat of e^-gap
    prompt(q, k, v, type_, D, f"{type_} gap {gap}")


def test_prompt_values_near_the_top_of_bfloat16():
    say("prompt values of 2^113 .. 2^114")
    r = np.random.Generator(np.random.PCG64(6))
    D, m, n = 64, 40, 4000
    k = (r.standard_normal((n, 1, D)) * 2.0 ** -6).astype(np.float32)
    k[:, :, 0] = 5.375
    k[:64, :, 0] = 0.0
    k = rounded(k, "bf16")
    v = rounded(r.uniform(0.5, 0.99, (n, 1, D)) * 2.0 ** 114, "bf16")
    prompt(rounded(queries(r, m, 2, D), "bf16"), k, v, "bf16", D, "large values")
