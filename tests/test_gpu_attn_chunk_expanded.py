"""Chunk attention over Q8_0 with so many queries to a sequence (1024 rows of query and head, on average) that the cache's rows
are turned into binary16 first: the same tests, at sizes that go that way."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import Paged, attention, rounded
from gpu_cases import host, torch_dev
from test_gpu_attn_chunk import P_UNIT, call, data, on_gpu, run
from window_cases import limits, seen_of

pytestmark = pytest.mark.gpu


def goes_that_way(seqs, Hq, Hkv):
    return sum(m for m, _ in seqs) * (Hq // Hkv) >= 1024 * len(seqs)


def go(type_, seqs, Hq, Hkv, D, page, seed, **kw):
    assert goes_that_way(seqs, Hq, Hkv)
    run("q8_0", type_, seqs, Hq, Hkv, D, page, seed, **kw)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_widths(D, type_):
    go(type_, [(70, 70), (60, 140)], 16, 1, D, 32, D, some=25)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 1024])
def test_mixed_batch(page, type_):
    go(type_, [(0, 0), (17, 17), (0, 90), (40, 0), (100, 30), (1, 700), (129, 257), (1, 1), (100, 1199), (3, 3000)], 64, 2, 64, page, 5, some=12)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 5), (15, 4), (17, 0), (64, 1), (65, 65), (128, 130), (200, 4), (1000, 2), (5, 4000)])
def test_windows(window, sinks):
    go("bf16", [(0, 50), (1, 300), (40, 40), (130, 700), (65, 80), (20, 10), (7, 2000)], 32, 1, 64, 16, window + sinks, window=window, sinks=sinks, some=15)


def test_several_key_heads_and_splits():
    go("bf16", [(260, 5000), (200, 3000)], 40, 8, 128, 64, 9, some=12)
    go("f16", [(260, 5000)], 20, 4, 96, 64, 10, window=700, sinks=20, some=12)


@pytest.mark.parametrize("kw", [dict(width_q=200.0), dict(scale=-0.4), dict(scale=0.0), dict(width_v=3e5), dict(width_k=3e5, width_q=1e-5),
                                dict(width_v=1e-5), dict(width_q=1e-30, width_k=1e5, scale=1e25), dict(width_q=1e20, width_k=1e-5, scale=1e-15)])
def test_ranges(kw):
    go("bf16", [(70, 190), (60, 600)], 16, 1, 64, 16, 11, some=25, **kw)


@pytest.mark.parametrize("way", [(-5, 4), (4, -5), (0, 4)])
def test_powers_that_change_along_the_keys(way):
    r = np.random.Generator(np.random.PCG64(3))

    def rows(n, w):
        x = r.standard_normal((n, 1, 64))
        return x * 10.0 ** np.linspace(*way, n)[:, None, None] if w == 2.0 else x * r.choice([1e-3, 1.0], (n, 1, 1))

    go("bf16", [(70, 500), (60, 1500)], 16, 1, 64, 16, 13, width_v=2.0, rows_of=rows, some=25)


@pytest.mark.parametrize("more", [1.0, 1e-4])
def test_smallest_scales(more):
    """Blocks whose scale is the smallest that there is, 2^-24, or 0; and a sequence of zeros alone."""
    r = np.random.Generator(np.random.PCG64(4))

    def rows(n, w):
        return np.clip(r.standard_normal((n, 1, 64)) * w, -3.2 * w, 3.2 * w) * (more if w < 1 else 1.0)

    go("bf16", [(70, 200), (60, 700)], 16, 1, 64, 16, 14, width_v=2.5e-6, rows_of=rows, some=25)


@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("window", [0, 70])
def test_non_finite_rows_reach_only_queries_that_see_them(window, type_):
    Hq, Hkv, D, sinks = 32, 2, 64, 3
    seqs = [(200, 260), (40, 30), (70, 70), (3, 900)]
    assert goes_that_way(seqs, Hq, Hkv)
    r = np.random.Generator(np.random.PCG64(17))
    kv = [[r.standard_normal((n, Hkv, D)).astype(np.float32) for _ in "kv"] for _, n in seqs]
    for b, row, ch, x in ((0, 63, 1, np.inf), (0, 130, 33, np.nan), (0, 259, 5, np.inf), (1, 2, 0, np.nan), (2, 50, 31, -np.inf), (3, 898, 40, np.nan)):
        kv[b][1][row, :, ch] = x
    kv[2][0][60, 1, 7] = np.nan
    c = Paged("q8_0", [tuple(x) for x in kv], Hkv, D, 16, 18)
    q = rounded(r.standard_normal((sum(m for m, _ in seqs), Hq, D)), type_)
    got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks).float())
    a = 0
    for b, (m, n) in enumerate(seqs):
        seen = seen_of(m, n, window, sinks)
        k, v = c.rows[b]
        for h in (0, 15, 16, 31):
            with np.errstate(invalid="ignore"):
                want, A, S = attention(q[a:a + m, h], k[:, h // 16], v[:, h // 16], D ** -0.5, seen)
                limit = limits(want, A, S, D, n, "q8_0", type_, P_UNIT["q8_0"])
            o, ok = got[a:a + m, h], np.isfinite(want)
            assert (np.isfinite(o) == ok).all(), f"sequence {b} head {h}"
            assert (np.abs(np.where(ok, o, 0) - np.where(ok, want, 0))[ok] <= limit[ok]).all(), f"sequence {b} head {h}"
            assert 0 < ok.sum() < ok.size and (o[~seen.any(1)] == 0).all()
        a += m


def test_lengths_and_pages_that_are_wrong():
    seqs = [(90, 500), (40, 900), (80, 120), (60, 300)]
    c, q, _ = data("q8_0", "bf16", seqs, 32, 2, 64, 16, 19)
    assert goes_that_way(seqs, 32, 2)
    new, x = [m for m, _ in seqs], on_gpu(q, "bf16")
    want = call(c, x, new)
    c.lengths[0], c.lengths[1] = -1, c.max_pages * 16 + 1
    got = call(c, x, new)
    torch = torch_dev()
    assert got[:130].isnan().all() and torch.equal(got[130:], want[130:])
    c.lengths[0], c.lengths[1] = 500, 900
    c.table[0, 3], c.table[1, 900 // 16], c.table[2, 119 // 16] = c.n_pages, -1, 1 << 30  # seen by all; by the last queries
    got = call(c, x, new)
    assert got[:90].isnan().all() and got[129].isnan().all() and got[209].isnan().all() and torch.equal(got[210:], want[210:])


def test_same_as_without():
    """The queries of one sequence among so many others that nothing is turned first: equal but for the order of the sums."""
    torch = torch_dev()
    seqs = [(100, 900)] + [(1, 1)] * 12
    c, q, _ = data("q8_0", "bf16", seqs, 16, 1, 128, 64, 23)
    assert not goes_that_way(seqs, 16, 1) and goes_that_way(seqs[:1], 16, 1)
    x, new = on_gpu(q, "bf16"), [m for m, _ in seqs]
    all_ = call(c, x, new)
    c.table, c.lengths = c.table[:1].contiguous(), c.lengths[:1].contiguous()
    one = call(c, x[:100], new[:1])
    assert float((one.float() - all_[:100].float()).abs().max()) <= 2 * 2.0 ** -8 * float(one.float().abs().max())


def test_captured():
    torch = torch_dev()
    seqs = [(130, 1500), (100, 300)]
    c, q, _ = data("q8_0", "bf16", seqs, 32, 2, 128, 64, 21)
    assert goes_that_way(seqs, 32, 2)
    new, x = [m for m, _ in seqs], on_gpu(q, "bf16")
    from test_gpu_attn_chunk import cu_of

    cu, out = cu_of(new), torch.empty_like(x)
    ws = torch.full((nvq.nvq_attn_chunk_workspace_bytes(nvq.NVQ_KV_Q8_0, 2, 230, 32, 2, 128, c.max_pages, 64),), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, x, new, out=out, cu=cu, workspace=ws)
    for n in (1500, 140, 700):
        c.lengths[0] = n
        x.copy_(torch.randn_like(x))
        want = call(c, x, new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
