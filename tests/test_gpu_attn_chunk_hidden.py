"""Chunk attention over Q8_0 where keys and values that a query does not see are larger by many orders of magnitude than those it
sees: the bounds are those of any other call, in both forms (rows taken as they are, or turned into binary16 first).

What the operands of a tile lose where its seen rows themselves lie far apart is not looked at here: a query's own rows are of one size.
"""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import HALF_UNIT, Paged, rounded
from gpu_cases import host, say, torch_dev
from test_gpu_attn_chunk import call, on_gpu
from test_gpu_attn_chunk_expanded import goes_that_way
from window_cases import Hidden, compare, seen_of

pytestmark = pytest.mark.gpu

P_UNIT = HALF_UNIT["f16"]
FORMS = {"direct": (4, 2), "turned": (64, 2)}  # query and key heads


def rows(r, n, Hkv, D, width):
    return (r.standard_normal((n, Hkv, D)) * width).astype(np.float32)


def queries(r, m, Hq, D, type_, width_k):
    """Scores of width 1 over keys of that width"""
    return rounded(r.standard_normal((m, Hq, D)) / width_k, type_)


def compare_all(got, q, c, seqs, seen, D, type_, some=12):
    a = 0
    for i, (m, _) in enumerate(seqs):
        pick = np.arange(m) if m <= 4 * some else np.unique(np.r_[np.arange(8), np.linspace(0, m - 1, some).astype(int), np.arange(m - 8, m)])
        worst = compare(got[a:a + m][pick], q[a:a + m][pick], c.rows[i], seen[i][pick], D ** -0.5, "q8_0", type_, P_UNIT, f"sequence {i}")
        say(f"  sequence {i}: worst error / bound {worst:.3g}")
        a += m


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("type_", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(20, 3), (100, 0), (1000, 5)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_nobody_sees(D, window, sinks, type_, form):
    """Between the first keys and the windows: codes of 127 with the largest scale that there is."""
    Hq, Hkv = FORMS[form]
    seqs = [(70, 2000), (33, 500), (40, 45)]
    assert goes_that_way(seqs, Hq, Hkv) == (form == "turned")
    say(f"hidden rows {form} {type_} D={D} window={window}+{sinks}")
    width = 1e-2
    r = np.random.Generator(np.random.PCG64(D + window))
    seen = [seen_of(m, n, window, sinks) for m, n in seqs]
    c = Hidden("q8_0", [(rows(r, n, Hkv, D, width), rows(r, n, Hkv, D, width)) for _, n in seqs], seen, Hkv, D, 16, 3)
    for d in (c.kd, c.vd):
        d[d.isnan()] = 65504.0
    q = queries(r, sum(m for m, _ in seqs), Hq, D, type_, width)
    got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks).float())
    compare_all(got, q, c, seqs, seen, D, type_)


def later(r, n, Hkv, D, width, at, far):
    """Rows of one width, those of `at` larger by the factor `far`"""
    x = rows(r, n, Hkv, D, width)
    x[at] *= far
    return x


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("far", [2.0 ** 17, 2.0 ** 20, 2.0 ** 28])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 2)])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_later_rows(D, window, sinks, far, which, form):
    """The last row, and one in the middle of the pieces, are larger than all others: queries before them are as exact as ever.  (Behind
    them a query's own rows lie far apart: looked at up to the documented 2^15, not here.)"""
    Hq, Hkv = FORMS[form]
    seqs = [(90, 90), (70, 700), (40, 2100)]
    assert goes_that_way(seqs, Hq, Hkv) == (form == "turned")
    say(f"later {which} {form} D={D} far={far} window={window}+{sinks}")
    r = np.random.Generator(np.random.PCG64(D))
    width = 1e-3
    large = [(n - m // 2, n - 1) for m, n in seqs]
    kv = [(later(r, n, Hkv, D, width, list(at) if which == "keys" else [], far), later(r, n, Hkv, D, width, list(at) if which == "values" else [], far))
          for (m, n), at in zip(seqs, large)]
    c = Paged("q8_0", kv, Hkv, D, 16, 4)
    type_ = "bf16"
    q = queries(r, sum(m for m, _ in seqs), Hq, D, type_, width)
    got = host(call(c, on_gpu(q, type_), [m for m, _ in seqs], window=window, sinks=sinks).float())
    a = 0
    for i, ((m, n), at) in enumerate(zip(seqs, large)):
        before = np.unique(np.linspace(0, at[0] - (n - m) - 1, 9).astype(int))
        seen = seen_of(m, n, window, sinks)[before]
        assert not seen[:, list(at)].any()
        worst = compare(got[a:a + m][before], q[a:a + m][before], c.rows[i], seen, D ** -0.5, "q8_0", type_, P_UNIT, f"sequence {i}")
        say(f"  sequence {i}: worst error / bound {worst:.3g}")
        assert np.isfinite(got[a:a + m]).all()
        a += m


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("D", [64, 128])
def test_all_queries_of_a_tile_with_rows_far_apart(D, form):
    """Values of one half of the channels larger by 2^28 than the other half's, in one row: every query, those that see it too, keeps
    its other channels' bits where the tile is not seen by all."""
    Hq, Hkv = FORMS[form]
    seqs = [(60, 60), (64, 64 * 4)]
    assert goes_that_way(seqs, Hq, Hkv) == (form == "turned")
    r = np.random.Generator(np.random.PCG64(5))
    kv = [(rows(r, n, Hkv, D, 1.0), rows(r, n, Hkv, D, 1e-3)) for _, n in seqs]
    for (m, n), x in zip(seqs, kv):
        x[1][n - 30, :, :D // 2] *= 2.0 ** 28
    c = Paged("q8_0", kv, Hkv, D, 16, 4)
    q = queries(r, sum(m for m, _ in seqs), Hq, D, "bf16", 1.0)
    got = host(call(c, on_gpu(q, "bf16"), [m for m, _ in seqs]).float())
    compare_all(got, q, c, seqs, [seen_of(m, n, 0, 0) for m, n in seqs], D, "bf16")


@pytest.mark.parametrize("form", FORMS)
def test_what_is_not_finite_beside_rows_far_apart(form):
    """A NaN and a large row in one tile: NaN in its block of the queries that see it, nothing of either in the others'; a page
    outside the cache makes NaN of the queries that see its keys."""
    torch = torch_dev()
    Hq, Hkv, D = *FORMS[form], 64
    seqs = [(80, 80), (60, 300)]
    r = np.random.Generator(np.random.PCG64(6))
    kv = [(rows(r, n, Hkv, D, 1e-3), rows(r, n, Hkv, D, 1e-3)) for _, n in seqs]
    for (m, n), x in zip(seqs, kv):
        x[1][n - 20, :, 33] = np.nan
        x[1][n - 9] *= 2.0 ** 28
        x[0][n - 8] *= 2.0 ** 28
    c = Paged("q8_0", kv, Hkv, D, 16, 7)
    q = queries(r, sum(m for m, _ in seqs), Hq, D, "bf16", 1e-3)
    new, x = [m for m, _ in seqs], on_gpu(q, "bf16")
    got = host(call(c, x, new).float())
    a = 0
    for i, (m, n) in enumerate(seqs):
        o, seen = got[a:a + m], seen_of(m, n, 0, 0)
        assert np.isnan(o[seen[:, n - 20]][:, :, 32:]).all() and np.isfinite(o[:, :, :32]).all() and np.isfinite(o[~seen[:, n - 20]]).all()
        before = np.flatnonzero(~seen[:, n - 20])[::7]
        compare(o[before], q[a:a + m][before], tuple(np.nan_to_num(y, nan=0.0) for y in c.rows[i]), seen[before], D ** -0.5, "q8_0", "bf16", P_UNIT, f"{i}")
        a += m
    assert not got[:, :, :32].max() == 0
    c.table[1, 299 // 16] = c.n_pages + 3
    got = call(c, x, new)
    assert got[80 + 48:].isnan().all() and got[:80, :, :32].isfinite().all()  # keys 288 on are seen by queries 48 on


@pytest.mark.parametrize("form", FORMS)
def test_rows_far_apart_captured(form):
    """Replays over rows whose sizes change from call to call equal the calls."""
    torch = torch_dev()
    Hq, Hkv, D = *FORMS[form], 128
    seqs = [(70, 900), (40, 40)]
    r = np.random.Generator(np.random.PCG64(8))
    c = Paged("q8_0", [(rows(r, n, Hkv, D, 1e-3), rows(r, n, Hkv, D, 1e-3)) for _, n in seqs], Hkv, D, 16, 9)
    q = on_gpu(queries(r, 110, Hq, D, "bf16", 1e-3), "bf16")
    cu, out = torch.tensor([0, 70, 110], dtype=torch.int32, device="cuda"), torch.empty_like(q)
    ws = torch.empty(nvq.nvq_attn_chunk_workspace_bytes(nvq.NVQ_KV_Q8_0, 2, 110, Hq, Hkv, D, c.max_pages, 16), dtype=torch.uint8, device="cuda")
    call(c, q, None, cu=cu, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, q, None, out=out, cu=cu, workspace=ws)
    last = int(c.slots[899])
    for size in (1.0, 2.0 ** 20, 0.0, 2.0 ** 27):
        d = c.vd[last // 16, :, last % 16]
        d.fill_(size * 2.0 ** -13)
        want = call(c, q, None, cu=cu)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and bool(out.isfinite().all())
