"""Attention of several new tokens per sequence over the paged cache, against float64.

Bounds: those of attn_cases with the probabilities' half unit (bfloat16 over a bfloat16 cache, binary16 otherwise), and over
Q8_0 what window_cases.limits adds for the operands' rounding."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import HALF_UNIT, Paged, attention, rounded, torch_type
from gpu_cases import host, say, torch_dev
from window_cases import Hidden, compare, limits, seen_of

pytestmark = pytest.mark.gpu

KINDS = [("q8_0", "bf16"), ("q8_0", "f16"), ("f16", "f16"), ("bf16", "bf16")]
P_UNIT = {"q8_0": HALF_UNIT["f16"], "f16": HALF_UNIT["f16"], "bf16": HALF_UNIT["bf16"]}


def cu_of(new):
    torch = torch_dev()
    return torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()


def call(c, q, new, out=None, window=0, sinks=0, cu=None, **kw):
    torch = torch_dev()
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    nvq.nvq_attn_chunk(q, c.kc, c.vc, c.table, cu_of(new) if cu is None else cu, c.lengths, out, c.kd, c.vd, window=window, sinks=sinks, **kw)
    return out


def data(fmt, type_, seqs, Hq, Hkv, D, page, seed, window=0, sinks=0, width_q=1.0, width_k=1.0, width_v=1.0, rows_of=None):
    """seqs: (new, keys) -> cache (what nobody sees is unusable), q (as the type holds it), what is seen"""
    r = np.random.Generator(np.random.PCG64(seed))
    rows_of = rows_of or (lambda n, w: r.standard_normal((n, Hkv, D)) * w)
    kv = [(rows_of(n, width_k).astype(np.float32), rows_of(n, width_v).astype(np.float32)) for _, n in seqs]
    seen = [seen_of(m, n, window, sinks) for m, n in seqs]
    c = Hidden(fmt, kv, seen, Hkv, D, page, seed + 1)
    return c, rounded(r.standard_normal((sum(m for m, _ in seqs), Hq, D)) * width_q, type_), seen


def on_gpu(q, type_):
    torch = torch_dev()
    return torch.from_numpy(np.ascontiguousarray(q)).to(torch_type(type_)).cuda()


def run(fmt, type_, seqs, Hq, Hkv, D, page, seed, window=0, sinks=0, scale=None, some=None, **kw):
    say(f"chunk {fmt} {type_} {seqs} Hq={Hq} Hkv={Hkv} D={D} page={page} window={window}+{sinks} scale={scale} {list(kw)}")
    c, q, seen = data(fmt, type_, seqs, Hq, Hkv, D, page, seed, window, sinks, **kw)
    got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks, scale=scale).float())
    worst, a = 0.0, 0
    for i, (m, n) in enumerate(seqs):
        worst = max(worst, compare(got[a:a + m], q[a:a + m], c.rows[i], seen[i], D ** -0.5 if scale is None else scale, fmt, type_, P_UNIT[fmt],
                                   f"sequence {i}", some))
        a += m
    say(f"  worst error / bound {worst:.3g}")


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("m", [1, 2, 31, 32, 33, 127, 128, 129, 300])
@pytest.mark.parametrize("prefix", [0, 1, 63])
def test_lengths(m, prefix, fmt, type_):
    run(fmt, type_, [(m, m + prefix)], 2, 1, 64, 16, m)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 193])
def test_single_tokens(n, fmt, type_):
    run(fmt, type_, [(1, n)], 5, 1, 128, 16, n)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_widths(D, fmt, type_):
    run(fmt, type_, [(70, 70), (5, 140)], 3, 1, D, 32, D)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("D", [32, 96, 128, 224, 256])
def test_head_widths_split(D, fmt, type_):
    run(fmt, type_, [(9, 700), (3, 2000)], 6, 2, D, 64, D)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (10, 2), (40, 8), (129, 1), (200, 2)])
def test_head_layouts(Hq, Hkv, fmt, type_):
    """(more query heads to a key head than a workgroup has rows, too)"""
    run(fmt, type_, [(9, 45), (30, 131), (1, 5)], Hq, Hkv, 64, 16, Hq)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_mixed_batch(page, fmt, type_):
    """No queries, no keys, fewer keys than queries (rows that see nothing), single tokens behind long prefixes, pieces of prompts."""
    run(fmt, type_, [(0, 0), (17, 17), (0, 9), (40, 0), (100, 30), (1, 700), (129, 257), (1, 1), (200, 1199), (3, 3000)], 4, 2, 64, page, 5)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (15, 4), (16, 16), (17, 0), (64, 1), (63, 64), (65, 65), (128, 130), (200, 4), (1000, 2), (5, 4000)])
def test_windows(window, sinks, fmt, type_):
    run(fmt, type_, [(0, 50), (1, 300), (40, 40), (130, 700), (65, 80), (20, 10), (1, 1), (7, 2000)], 5, 1, 64, 16, window + sinks, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt,type_", KINDS)
def test_windows_over_many_heads(fmt, type_):
    run(fmt, type_, [(300, 900), (1, 2000)], 40, 8, 128, 64, 9, window=256, sinks=4, some=30)


def test_many_sequences():
    r = np.random.Generator(np.random.PCG64(6))
    seqs = [(int(m), int(m + p)) for m, p in zip(r.choice([0, 1, 1, 1, 30], 140), r.integers(0, 200, 140))]
    run("f16", "f16", seqs, 2, 1, 32, 16, 7)
    run("q8_0", "bf16", seqs, 2, 1, 32, 16, 8, window=40, sinks=3)


@pytest.mark.parametrize("fmt,type_", KINDS)
def test_long_splits(fmt, type_):
    run(fmt, type_, [(16, 9000), (1, 40), (130, 5000)], 5, 1, 128, 64, 12, some=20)


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("kw", [dict(width_q=200.0), dict(width_q=1e-3), dict(scale=-0.4), dict(scale=0.0), dict(width_q=1e-4, scale=1e3),
                                dict(width_k=1e-3), dict(width_v=1e-3), dict(width_v=1e4), dict(width_k=1e3, width_q=1e-2)])
def test_ranges(kw, fmt, type_):
    """(over 16 bits the widths stay inside binary16's normal range; values' results too)"""
    run(fmt, type_, [(70, 190), (2, 600)], 2, 1, 64, 16, 11, **kw)


@pytest.mark.parametrize("kw", [dict(width_v=3e5), dict(width_k=3e5, width_q=1e-5), dict(width_v=1e-5), dict(width_q=1e-30, width_k=1e5, scale=1e25),
                                dict(width_q=1e20, width_k=1e-5, scale=1e-15)])
def test_q8_0_ranges_past_binary16(kw):
    """Values and keys that binary16 does not hold (scales do), bfloat16 queries of any size."""
    run("q8_0", "bf16", [(70, 190), (2, 600)], 2, 1, 64, 16, 11, **kw)


def test_q8_0_value_powers_that_change_along_the_keys():
    """Values that grow, and that shrink, by 9 orders of magnitude from key to key; keys' blocks of all sizes."""
    def growing(n, w):
        x = r.standard_normal((n, 1, 64))
        return x * 10.0 ** np.linspace(*sign, n)[:, None, None] if w == 2.0 else x * r.choice([1e-3, 1.0], (n, 1, 1))

    for sign in ((-5, 4), (4, -5), (0, 4)):
        r = np.random.Generator(np.random.PCG64(3))
        run("q8_0", "bf16", [(40, 500), (1, 1500)], 2, 1, 64, 16, 13, width_v=2.0, rows_of=growing)


def test_strides_and_rows_outside_the_sequences():
    """Queries as columns of a fused row, an output with heads first; rows before and behind the sequences are not written."""
    torch = torch_dev()
    seqs, Hq, Hkv, D = [(60, 90), (33, 80)], 4, 2, 64
    c, q, _ = data("bf16", "bf16", seqs, Hq, Hkv, D, 16, 13)
    new = [m for m, _ in seqs]
    want = call(c, on_gpu(q, "bf16"), new)
    tq = q.shape[0] + 20
    y = torch.full((tq, (Hq + 2 * Hkv) * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    big = y[:, :Hq * D].unflatten(1, (Hq, D))
    big[7:7 + q.shape[0]] = on_gpu(q, "bf16")
    out = torch.full((Hq, tq, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    call(c, big, None, out=out, cu=cu_of(new) + 7)
    assert torch.equal(out[7:7 + q.shape[0]], want)
    assert (out[:7] == 7).all() and (out[7 + q.shape[0]:] == 7).all()
    call(c, big, None, out=out, cu=torch.tensor([-5, 60 + 7, 1 << 30], dtype=torch.int32, device="cuda"))  # cut to the rows
    assert torch.isfinite(out[7:60 + 7].float()).all()


@pytest.mark.parametrize("fmt,type_", KINDS)
@pytest.mark.parametrize("window", [0, 70])
def test_non_finite_rows_reach_only_queries_that_see_them(window, fmt, type_):
    """An infinity or NaN in one channel of a value row shows in that channel (Q8_0: block) of the queries that see the row, in
    a key row in all of theirs; the other queries of the tile are as if it were not there."""
    torch = torch_dev()
    Hq, Hkv, D, sinks = 4, 2, 64, 3
    seqs = [(200, 260), (40, 30), (70, 70), (3, 900)]
    r = np.random.Generator(np.random.PCG64(17))
    kv = [[r.standard_normal((n, Hkv, D)).astype(np.float32) for _ in "kv"] for _, n in seqs]
    for b, row, ch, x in ((0, 63, 1, np.inf), (0, 130, 33, np.nan), (0, 259, 5, np.inf), (1, 2, 0, np.nan), (2, 50, 31, -np.inf), (3, 898, 40, np.nan),
                          (0, 1, 60, np.inf)):
        kv[b][1][row, :, ch] = x
    kv[2][0][60, 1, 7] = np.nan
    c = Paged(fmt, [tuple(x) for x in kv], Hkv, D, 16, 18)
    q = rounded(r.standard_normal((sum(m for m, _ in seqs), Hq, D)), type_)
    got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks).float())
    a = 0
    for b, (m, n) in enumerate(seqs):
        seen = seen_of(m, n, window, sinks)
        k, v = c.rows[b]
        for h in range(Hq):
            with np.errstate(invalid="ignore"):
                want, A, S = attention(q[a:a + m, h], k[:, h // 2], v[:, h // 2], D ** -0.5, seen)
                limit = limits(want, A, S, D, n, fmt, type_, P_UNIT[fmt])
            o, ok = got[a:a + m, h], np.isfinite(want)
            assert (np.isfinite(o) == ok).all(), f"sequence {b} head {h}"
            if fmt != "q8_0":
                assert (o[np.isinf(want)] == want[np.isinf(want)]).all()
            assert (np.abs(np.where(ok, o, 0) - np.where(ok, want, 0))[ok] <= limit[ok]).all(), f"sequence {b} head {h}"
            assert 0 < ok.sum() < ok.size and (o[~seen.any(1)] == 0).all()
        a += m


@pytest.mark.parametrize("fmt,type_", KINDS)
def test_lengths_and_pages_that_are_wrong(fmt, type_):
    torch = torch_dev()
    seqs = [(30, 500), (4, 900), (20, 60), (6, 300)]
    c, q, _ = data(fmt, type_, seqs, 4, 2, 64, 16, 19)
    new, x = [m for m, _ in seqs], on_gpu(q, type_)
    want = call(c, x, new)
    c.lengths[0], c.lengths[1] = -1, c.max_pages * 16 + 1
    got = call(c, x, new)
    assert got[:34].isnan().all() and torch.equal(got[34:], want[34:])
    c.lengths[0], c.lengths[1] = 500, 900
    c.table[0, 3], c.table[1, 900 // 16], c.table[2, 60 // 16] = c.n_pages, -1, 1 << 30  # seen by all; by the last queries
    got = call(c, x, new)
    assert got[:30].isnan().all() and got[33].isnan().all() and got[53].isnan().all() and torch.equal(got[54:], want[54:])


def test_deterministic_captured_and_on_another_stream():
    torch = torch_dev()
    seqs = [(30, 1500), (1, 3000), (200, 300)]
    c, q, _ = data("q8_0", "bf16", seqs, 4, 2, 128, 64, 21)
    new, x = [m for m, _ in seqs], on_gpu(q, "bf16")
    want = call(c, x, new)
    assert torch.equal(call(c, x, new), want)
    cu, out, s = cu_of(new), torch.empty_like(want), torch.cuda.Stream()
    torch.cuda.synchronize()
    call(c, x, new, out=out, cu=cu, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)
    need = nvq.nvq_attn_chunk_workspace_bytes(nvq.NVQ_KV_Q8_0, 3, 231, 4, 2, 128, c.max_pages, 64)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    with pytest.raises(nvq.NvqError, match="workspace"):
        call(c, x, new, workspace=ws[:need - 16])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, x, new, out=out, cu=cu, workspace=ws)
    for n in (1500, 30, 700):
        c.lengths[0] = n
        x.copy_(torch.randn_like(x))
        want = call(c, x, new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("fmt,type_", KINDS)
def test_pieces_equal_the_whole_prompt_and_decode(fmt, type_):
    """One prompt whole and in pieces, and its last token by the decode operator, within the bounds of both."""
    torch = torch_dev()
    n, Hq, Hkv, D = 400, 10, 2, 128
    c, q, _ = data(fmt, type_, [(n, n)], Hq, Hkv, D, 16, 22)
    x = on_gpu(q, type_)
    whole = call(c, x, [n])
    a = 0
    for m in (1, 100, 130, 168, 1):
        c.lengths.fill_(a + m)
        part = call(c, x[a:a + m], [m])
        assert float((part.float() - whole[a:a + m].float()).abs().max()) <= 6 * HALF_UNIT[type_] * float(np.abs(c.rows[0][1]).max())
        a += m
    one = torch.empty_like(x[:1])
    nvq.nvq_attn_decode(x[n - 1:], c.kc, c.vc, c.table, c.lengths, one, c.kd, c.vd)
    assert float((one.float() - whole[n - 1:].float()).abs().max()) <= 6 * HALF_UNIT[type_] * float(np.abs(c.rows[0][1]).max())


def test_rows_past_32_bit_offsets():
    """A cache of over 4 GiB whose sequence sits in its last pages."""
    torch = torch_dev()
    Hkv, D, page, n = 8, 256, 4096, 5000
    n_pages = (1 << 32) // (Hkv * D * page) + 3
    kc, vc = (torch.zeros((n_pages, Hkv, page, D), dtype=torch.int8, device="cuda") for _ in "kv")
    kd, vd = (torch.zeros((n_pages, Hkv, page, D // 32), dtype=torch.float16, device="cuda") for _ in "kv")
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    at = torch.arange(n, device="cuda")
    k, v = (torch.randn((n, Hkv, D), device="cuda") for _ in "kv")
    nvq.nvq_kv_write(k, v, table[0].long()[at // page] * page + at % page, kc, vc, kd, vd)
    small = [torch.cat([x[n_pages - 1:], x[n_pages - 2:n_pages - 1]]) for x in (kc, vc, kd, vd)]
    q = torch.randn((20, 16, D), device="cuda").bfloat16()
    a, b = torch.empty_like(q), torch.empty_like(q)
    cu, lens = cu_of([20]), torch.tensor([n], dtype=torch.int32, device="cuda")
    nvq.nvq_attn_chunk(q, kc, vc, table, cu, lens, a, kd, vd)
    nvq.nvq_attn_chunk(q, *small[:2], torch.tensor([[0, 1]], dtype=torch.int32, device="cuda"), cu, lens, b, *small[2:])
    assert torch.equal(a, b) and float(a.float().abs().max()) > 0


def test_offsets_that_do_not_ascend_write_nothing_outside():
    """4096 sequences that each claim all 8192 queries: 2^32 key tiles in all, which the work's plan does not count.  What is
    computed is anybody's; the workspace's neighbour and the rows behind are left alone."""
    torch = torch_dev()
    B, Tq, D, page, pages = 4096, 8192, 32, 65536, 64
    say("chunk offsets that do not ascend")
    kc, vc = (torch.zeros((1, 1, page, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    table = torch.zeros((B, pages), dtype=torch.int32, device="cuda")
    lengths = torch.full((B,), page * pages - 1, dtype=torch.int32, device="cuda")
    cu = (torch.arange(B + 1, device="cuda") % 2 * Tq).int()
    cu[::2] = -5
    q = torch.ones((Tq, 1, D), dtype=torch.bfloat16, device="cuda")
    rows = torch.full((Tq + 64, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    need = nvq.nvq_attn_chunk_workspace_bytes(nvq.NVQ_KV_BF16, B, Tq, 1, 1, D, pages, page)
    room = torch.full((need + (64 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    nvq.nvq_attn_chunk(q, kc, vc, table, cu, lengths, rows[:Tq], workspace=room[:need])
    torch.cuda.synchronize()
    assert bool((room[need:] == 0x5A).all()) and bool((rows[Tq:] == 7.0).all())
