"""Causal attention of packed prompts on the GPU against float64."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import HALF_UNIT, attention, bound, check, rounded, torch_type
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu


def make(seqs, Hq, Hkv, D, type_, seed, width=1.0):
    """seqs: (queries, keys) of each -> q, k, v (as the type holds them, float32), cu_q, cu_k"""
    r = np.random.Generator(np.random.PCG64(seed))
    tq, tk = sum(m for m, _ in seqs), sum(n for _, n in seqs)
    q, k, v = (rounded(r.standard_normal((t, h, D)) * w, type_) for t, h, w in ((tq, Hq, width), (tk, Hkv, 1.0), (tk, Hkv, 1.0)))
    cu = [np.concatenate([[0], np.cumsum([s[i] for s in seqs])]).astype(np.int32) for i in (0, 1)]
    return q, k, v, *cu


def on_gpu(x, type_):
    torch = torch_dev()
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch_type(type_)).cuda()


def call(q, k, v, cu_q, cu_k, **kw):
    torch = torch_dev()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    nvq.nvq_attn_prompt(q, k, v, torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda(), out, **kw)
    return out


def compare(got, q, k, v, cu_q, cu_k, scale, causal, type_, what, some=None):
    D, Hq, Hkv = q.shape[2], q.shape[1], k.shape[1]
    worst = 0.0
    for b in range(len(cu_q) - 1):
        a, e, x, y = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        m, n = e - a, y - x
        seen = np.ones((m, n), bool) if not causal else np.arange(n)[None] <= np.arange(m)[:, None] + (n - m)
        pick = np.arange(m) if some is None or m <= some else np.unique(np.linspace(0, m - 1, some).astype(int))
        for h in range(Hq):
            want, A, S = attention(q[a:e][pick, h], k[x:y, h * Hkv // Hq], v[x:y, h * Hkv // Hq], scale, seen[pick])
            worst = max(worst, check(got[a:e][pick, h], want, bound(want, A, S, D, n, type_, HALF_UNIT[type_], 2), f"{what} sequence {b} head {h}"))
            assert (got[a:e][pick, h][~seen[pick].any(1)] == 0).all()
    say(f"  worst error / bound {worst:.3g}")


def run(seqs, Hq, Hkv, D, type_, seed, causal=True, scale=None, width=1.0, some=None):
    say(f"prompt {seqs} Hq={Hq} Hkv={Hkv} D={D} {type_} causal={causal} scale={scale}")
    x = make(seqs, Hq, Hkv, D, type_, seed, width)
    got = host(call(*(on_gpu(a, type_) for a in x[:3]), *x[3:], causal=causal, scale=scale).float())
    compare(got, *x, D ** -0.5 if scale is None else scale, causal, type_, str(seqs), some)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(m, type_):
    run([(m, m)], 2, 1, 128, type_, m)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_widths(D, type_):
    run([(70, 70), (5, 140)], 3, 1, D, type_, D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (10, 2), (40, 8)])
def test_head_layouts(Hq, Hkv):
    run([(45, 45), (130, 131)], Hq, Hkv, 64, "bf16", Hq)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_with_prefixes_and_empty_rows(type_, causal):
    """No queries, no keys, fewer keys than queries (rows that see nothing), one query behind a long prefix."""
    run([(0, 0), (17, 17), (0, 9), (40, 0), (100, 30), (1, 700), (129, 257), (200, 199)], 4, 2, 64, type_, 5, causal)


def test_many_sequences():
    r = np.random.Generator(np.random.PCG64(6))
    run([(int(m), int(m + p)) for m, p in zip(r.integers(0, 30, 140), r.integers(0, 20, 140))], 2, 1, 32, "f16", 7)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("width,scale", [(200.0, None), (1e-3, None), (1.0, -0.4), (1.0, 0.0)])
def test_ranges(type_, width, scale):
    run([(150, 190)], 2, 1, 64, type_, 11, scale=scale, width=width)


def test_longer_prompt():
    run([(1500, 1500)], 4, 2, 128, "bf16", 12, some=40)


def test_strides_and_rows_outside_the_sequences():
    """Columns of a fused row, a tensor with heads first; rows before, between and behind the sequences are not
    written, and what keys and values hold there does not matter."""
    torch = torch_dev()
    seqs, Hq, Hkv, D = [(60, 60), (33, 80)], 4, 2, 64
    q, k, v, cu_q, cu_k = make(seqs, Hq, Hkv, D, "bf16", 13)
    want = call(*(on_gpu(a, "bf16") for a in (q, k, v)), cu_q, cu_k)
    tq, tk = q.shape[0] + 20, k.shape[0] + 30
    y = torch.full((max(tq, tk), (Hq + 2 * Hkv) * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = torch.full((Hq, tq, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    big = [y[:tq, :Hq * D].unflatten(1, (Hq, D)), y[:tk, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)),
           torch.full((Hkv, tk, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)]
    cq, ck = cu_q + 7, cu_k + 11
    big[0][7:7 + q.shape[0]] = on_gpu(q, "bf16")
    for t, x in ((big[1], k), (big[2], v)):
        t[11:11 + k.shape[0]] = on_gpu(x, "bf16")
    nvq.nvq_attn_prompt(*big, torch.from_numpy(cq).cuda(), torch.from_numpy(ck).cuda(), out)
    assert torch.equal(out[7:7 + q.shape[0]], want)
    assert (out[:7] == 7).all() and (out[7 + q.shape[0]:] == 7).all()


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128, 160, 256])
def test_non_finite_rows_reach_only_queries_that_see_them(D, type_):
    """An infinity or NaN in one channel of a value row shows in that channel of the queries that see the row, in a key
    row in all of theirs; queries before it in the same tile, and those that see no key, are as if it were not there."""
    q, k, v, cu_q, cu_k = make([(200, 260), (40, 30), (70, 70)], 4, 2, D, type_, 17 + D)
    for row, ch, x in ((63, 1, np.inf), (130, 3, np.nan), (259, 5, np.inf), (262, 0, np.nan), (359, 31, -np.inf)):
        v[row, :, ch] = x
    k[350, 1, 7] = np.nan
    got = host(call(*(on_gpu(a, type_) for a in (q, k, v)), cu_q, cu_k).float())
    for b in range(3):
        a, e, x, y = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        m, n = e - a, y - x
        seen = np.arange(n)[None] <= np.arange(m)[:, None] + (n - m)
        for h in range(4):
            with np.errstate(invalid="ignore"):
                want, A, S = attention(q[a:e, h], k[x:y, h // 2], v[x:y, h // 2], D ** -0.5, seen)
                limit = bound(want, A, S, D, n, type_, HALF_UNIT[type_], 2)
            ok = np.isfinite(want)
            assert (np.isfinite(got[a:e, h]) == ok).all(), f"sequence {b} head {h}"
            assert (np.isnan(got[a:e, h]) == np.isnan(want)).all() and (got[a:e, h][np.isinf(want)] == want[np.isinf(want)]).all()
            assert (np.abs(got[a:e, h] - want)[ok] <= limit[ok]).all(), f"sequence {b} head {h}"
            assert 0 < ok.sum() < ok.size and (got[a:e, h][~seen.any(1)] == 0).all()


@pytest.mark.parametrize("x", [np.inf, np.nan])
def test_non_finite_channel(x):
    """One channel of every value row: it alone is that in every result, and zero where no key is seen."""
    q, k, v, cu_q, cu_k = make([(150, 150), (40, 20)], 2, 1, 96, "bf16", 18)
    want = host(call(*(on_gpu(a, "bf16") for a in (q, k, v)), cu_q, cu_k).float())
    v[:, :, 37] = x
    got = host(call(*(on_gpu(a, "bf16") for a in (q, k, v)), cu_q, cu_k).float())
    assert (got[170:, :, 37] == x).all() or np.isnan(x) and np.isnan(got[170:, :, 37]).all()
    assert (got[:150, :, 37] == x).all() or np.isnan(x) and np.isnan(got[:150, :, 37]).all()
    assert (got[150:170] == 0).all()
    rest = np.arange(96) != 37
    # (rounded at two maxima at most 2^8 apart: twice the half unit of a probability, and the result's own)
    assert np.abs(got - want)[..., rest].max() <= 4 * HALF_UNIT["bf16"] * np.abs(v[..., rest]).max()


def test_offsets_outside_the_tensors_are_cut():
    torch = torch_dev()
    q, k, v, cu_q, cu_k = make([(40, 40)], 2, 1, 64, "f16", 14)
    x = [on_gpu(a, "f16") for a in (q, k, v)]
    want = call(*x, cu_q, cu_k)
    assert torch.equal(call(*x, np.array([-5, 1000], np.int32), np.array([-9, 1 << 30], np.int32)), want)
    assert (call(*x, np.array([30, 10], np.int32), cu_k) == 7).all()


def test_deterministic_and_on_another_stream():
    torch = torch_dev()
    q, k, v, cu_q, cu_k = make([(300, 300), (64, 500)], 4, 2, 128, "bf16", 15)
    x = [on_gpu(a, "bf16") for a in (q, k, v)]
    want = call(*x, cu_q, cu_k)
    assert torch.equal(call(*x, cu_q, cu_k), want)
    cq, ck = torch.from_numpy(cu_q).cuda(), torch.from_numpy(cu_k).cuda()
    out = torch.empty_like(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    nvq.nvq_attn_prompt(*x, cq, ck, out, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)


def test_one_token_prompt_equals_decode():
    """The same query over the same keys by the two operators, within both bounds."""
    torch = torch_dev()
    q, k, v, cu_q, cu_k = make([(1, 200)], 10, 2, 128, "f16", 16)
    got = call(*(on_gpu(a, "f16") for a in (q, k, v)), cu_q, cu_k)
    kc, vc = (torch.zeros((4, 2, 64, 128), dtype=torch.float16, device="cuda") for _ in "kv")
    nvq.nvq_kv_write(on_gpu(k, "f16"), on_gpu(v, "f16"), torch.arange(200, device="cuda"), kc, vc)
    out = torch.empty_like(got)
    nvq.nvq_attn_decode(on_gpu(q, "f16"), kc, vc, torch.arange(4, dtype=torch.int32, device="cuda")[None],
                        torch.tensor([200], dtype=torch.int32, device="cuda"), out)
    assert float((got.float() - out.float()).abs().max()) < 3 * 2.0 ** -11 * float(np.abs(v).max())
