"""Chunk attention whose scores are so large that float32 no longer holds the difference from their maximum to a whole number:
the key with the largest score by far takes all, and its values are the result.

Keys are one row of signs times sizes of which each is 2^-6 larger than the next smaller one, in any order; queries are that row times a
power of two.  A query is looked at where its largest score passes the next one by 2^-8 of itself, which is past what 16-bit keys
and Q8_0's operands (2 * 2^-11) and float32 sums (136 * 2^-24) may change it by, and by 64: nothing but the largest key's probability is left.
What remains is the rounding of its values: as operands over Q8_0 (2^-11), the sum over keys that hold it once (2^-20 allowed), the result's.
"""
import numpy as np
import pytest

from attn_cases import HALF_UNIT, Paged, rounded
from gpu_cases import host, say
from test_gpu_attn_chunk import KINDS, call, on_gpu
from window_cases import seen_of

pytestmark = pytest.mark.gpu

SIZES = {"f16": [2.0 ** 8, 2.0 ** 15], "bf16": [2.0 ** 8, 2.0 ** 15, 2.0 ** 30, 2.0 ** 80]}


def largest(s):
    """The place of the largest score, or None where the next one is too near"""
    at = int(s.argmax())
    rest = np.delete(s, at)
    far = s[at] - rest.max(initial=-np.inf)
    return at if np.isfinite(s[at]) and far >= max(2.0 ** -8 * abs(s[at]), 64.0) else None


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("scale", [1.0, -1.0])
@pytest.mark.parametrize("Hq,Hkv,D,seqs,window,sinks", [(4, 2, 64, [(1, 3), (70, 300), (40, 900)], 0, 0), (40, 8, 128, [(9, 1000)], 0, 0),
                                                        (16, 1, 64, [(300, 700)], 0, 0), (4, 2, 96, [(100, 800), (7, 1000)], 150, 4)])
def test_the_largest_score_takes_all(Hq, Hkv, D, seqs, window, sinks, scale, fmt, type_):
    for size in SIZES[type_]:
        say(f"large scores {fmt} {type_} {seqs} Hq={Hq} Hkv={Hkv} D={D} window={window} scale={scale} size={size}")
        r = np.random.Generator(np.random.PCG64(D))
        kv, q = [], []
        for m, n in seqs:
            sign, c = r.choice([-1.0, 1.0], (1, Hkv, D)), 2.0 ** 15 * (1 + 2.0 ** -6) ** -r.permutation(1000)[:n]
            kv.append(((c[:, None, None] * sign).astype(np.float32), r.standard_normal((n, Hkv, D)).astype(np.float32)))
            q.append(np.repeat(sign, Hq // Hkv, axis=1) * np.ones((m, 1, 1)) * size * scale)
        c = Paged(fmt, kv, Hkv, D, 16, 5)
        q = rounded(np.concatenate(q), type_)
        got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks, scale=scale).float())
        a = looked_at = 0
        for i, (m, n) in enumerate(seqs):
            seen = seen_of(m, n, window, sinks)
            k, v = c.rows[i]
            score = np.abs(k[:, 0, 0]).astype(np.float64) * size * D
            for x in range(m):
                top = largest(np.where(seen[x], score, -np.inf))
                if top is not None:
                    want = v[top, np.arange(Hq) * Hkv // Hq]
                    limit = (HALF_UNIT[type_] + (2.0 ** -11 if fmt == "q8_0" else 0) + 2.0 ** -20) * 1.01 * np.abs(want) + 2.0 ** -24
                    assert (np.abs(got[a + x] - want) <= limit).all(), f"sequence {i} query {x}"
                    looked_at += 1
            assert np.isfinite(got[a:a + m]).all()
            a += m
        assert looked_at > a / 2


@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (64, 2)])
@pytest.mark.parametrize("type_", ["f16", "bf16"])
def test_large_scores_beside_values_far_apart(type_, Hq, Hkv):
    """The same over Q8_0 where the last key's values are 2^28 times the others', so that the last tile is computed by itself; its
    largest scores come before, in, and behind that tile's.  (Other keys' probabilities are below e^-64: 2^28 times them is nothing.)"""
    D, seqs = 64, [(70, 300), (60, 64)]
    for size in SIZES[type_]:
        r = np.random.Generator(np.random.PCG64(11))
        kv, q = [], []
        for m, n in seqs:
            sign, c = r.choice([-1.0, 1.0], (1, Hkv, D)), 2.0 ** 15 * (1 + 2.0 ** -6) ** -r.permutation(1000)[:n]
            v = r.standard_normal((n, Hkv, D)).astype(np.float32) * 1e-3
            v[-1] *= 2.0 ** 28
            kv.append(((c[:, None, None] * sign).astype(np.float32), v))
            q.append(np.repeat(sign, Hq // Hkv, axis=1) * np.ones((m, 1, 1)) * size)
        c = Paged("q8_0", kv, Hkv, D, 16, 5)
        q = rounded(np.concatenate(q), type_)
        got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], scale=1.0).float())
        a = looked_at = 0
        for i, (m, n) in enumerate(seqs):
            seen = seen_of(m, n, 0, 0)
            k, v = c.rows[i]
            score = np.abs(k[:, 0, 0]).astype(np.float64) * size * D
            for x in range(m - 1):
                top = largest(np.where(seen[x], score, -np.inf))
                if top is not None:
                    want = v[top, np.arange(Hq) * Hkv // Hq]
                    limit = (HALF_UNIT[type_] + 2.0 ** -11 + 2.0 ** -20) * 1.01 * np.abs(want) + 2.0 ** -24
                    assert (np.abs(got[a + x] - want) <= limit).all(), f"sequence {i} query {x} size {size}"
                    looked_at += 1
            a += m
        assert looked_at > a / 2
