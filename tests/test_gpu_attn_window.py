"""Attention of one new token over a sliding window and the first keys of the paged cache, against float64."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import Paged, rounded, torch_type
from gpu_cases import host, say, torch_dev
from window_cases import Hidden, compare, seen_of

pytestmark = pytest.mark.gpu


def call(c, q, window, sinks, **kw):
    torch = torch_dev()
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    nvq.nvq_attn_decode_window(q, c.kc, c.vc, c.table, c.lengths, out, c.kd, c.vd, window=window, sinks=sinks, **kw)
    return out


def run(fmt, type_, lens, window, sinks, Hq, Hkv, D, page, seed, hide=True):
    torch = torch_dev()
    say(f"window {window}+{sinks} {fmt} {type_} lens={lens} Hq={Hq} Hkv={Hkv} D={D} page={page}")
    r = np.random.Generator(np.random.PCG64(seed))
    seqs = [tuple(r.standard_normal((n, Hkv, D)).astype(np.float32) for _ in "kv") for n in lens]
    seen = [seen_of(1, n, window, sinks) for n in lens]
    c = Hidden(fmt, seqs, seen, Hkv, D, page, seed + 1) if hide else Paged(fmt, seqs, Hkv, D, page, seed + 1)
    q = rounded(r.standard_normal((len(lens), Hq, D)), type_)
    got = host(call(c, torch.from_numpy(q).to(torch_type(type_)).cuda(), window, sinks).float())
    worst = 0.0
    for i, rows in enumerate(c.rows):
        worst = max(worst, compare(got[i:i + 1], q[i:i + 1], rows, seen[i], D ** -0.5, fmt, type_, None, f"sequence {i}"))
    say(f"  worst error / bound {worst:.3g}")


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64, 65, 100, 127, 128, 129, 300]


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (1, 16), (15, 4), (16, 0), (16, 16), (17, 17), (32, 4), (33, 31), (48, 1), (100, 33), (64, 200),
                                          (500, 4), (0, 9)])
def test_windows_at_group_tile_and_page_edges(fmt, window, sinks):
    run(fmt, "f32", EDGES, window, sinks, 5, 1, 64, 16, 100 * window + sinks)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_types_and_pages(fmt, type_, page):
    run(fmt, type_, [700, 90, 0, 333], 130, 20, 10, 2, 128, page, 7 + page)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_widths(fmt, D):
    run(fmt, "f32", [40, 301], 90, 5, 6, 2, D, 32, 100 + D)


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (17, 1), (40, 8), (16, 16)])
def test_head_layouts(fmt, Hq, Hkv):
    run(fmt, "f32", [177, 5], 60, 3, Hq, Hkv, 64, 16, 7 * Hq + Hkv)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("lens,window,sinks,Hq,Hkv", [([5000], 2000, 40, 5, 1), ([9000, 1000, 3], 4096, 4, 16, 16), ([3000, 2999, 0, 2600], 2500, 600, 80, 16)])
def test_windows_that_are_split(fmt, lens, window, sinks, Hq, Hkv):
    run(fmt, "f32", lens, window, sinks, Hq, Hkv, 64, 64, sum(lens))


def test_many_sequences():
    r = np.random.Generator(np.random.PCG64(3))
    run("q8_0", "f16", [int(x) for x in r.choice([0, 0, 1, 3, 20, 40, 400], 150)], 33, 4, 2, 1, 64, 16, 4)


def test_no_window_is_plain_decode():
    """Window 0, windows of everything and first keys that are everything: nvq_attn_decode's bits."""
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(5))
    seqs = [tuple(r.standard_normal((n, 2, 64)).astype(np.float32) for _ in "kv") for n in (700, 30, 0)]
    c = Paged("q8_0", seqs, 2, 64, 16, 6)
    q = torch.from_numpy(r.standard_normal((3, 4, 64)).astype(np.float32)).cuda()
    want = c.decode(q)
    room = c.max_pages * 16
    for window, sinks in ((0, 0), (0, 5), (room, 0), (room + 1, 3), (1 << 40, 1 << 40), (5, room), (room - 1, room)):
        assert torch.equal(call(c, q, window, sinks), want)


def test_workspaces_lengths_and_pages_that_are_wrong():
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(7))
    seqs = [tuple(r.standard_normal((n, 2, 64)).astype(np.float32) for _ in "kv") for n in (900, 500, 400)]
    c = Paged("bf16", seqs, 2, 64, 16, 8)
    q = torch.from_numpy(r.standard_normal((3, 4, 64)).astype(np.float32)).cuda()
    want = call(c, q, 200, 4)
    need = nvq.nvq_attn_decode_workspace_bytes(3, 4, 2, 64, -(-(200 + 4 + 30) // 16), 16)
    assert 0 < need < nvq.nvq_attn_decode_workspace_bytes(3, 4, 2, 64, c.max_pages, 16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(call(c, q, 200, 4, workspace=ws), want)
    with pytest.raises(nvq.NvqError, match="workspace"):
        call(c, q, 200, 4, workspace=ws[:16])
    c.lengths[0], c.lengths[1] = -1, c.max_pages * 16 + 1
    got = call(c, q, 200, 4)
    assert got[:2].isnan().all() and torch.equal(got[2], want[2])
    c.lengths[0], c.lengths[1] = 900, 500
    c.table[0, 880 // 16], c.table[1, 0], c.table[2, 10] = c.n_pages, -1, -1  # in the window; a first key's; between them (keys 160 .. 175)
    got = call(c, q, 200, 4)
    assert got[:2].isnan().all() and torch.equal(got[2], want[2])


def test_captured_and_on_another_stream():
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(9))
    seqs = [tuple(r.standard_normal((n, 2, 64)).astype(np.float32) for _ in "kv") for n in (900, 300)]
    c = Paged("q8_0", seqs, 2, 64, 16, 10)
    q = torch.from_numpy(r.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
    want = call(c, q, 300, 4)
    s, out = torch.cuda.Stream(), torch.empty_like(q)
    torch.cuda.synchronize()
    nvq.nvq_attn_decode_window(q, c.kc, c.vc, c.table, c.lengths, out, c.kd, c.vd, window=300, sinks=4, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(out, want)
    ws = torch.empty(max(16, nvq.nvq_attn_decode_workspace_bytes(2, 4, 2, 64, c.max_pages, 16)), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nvq.nvq_attn_decode_window(q, c.kc, c.vc, c.table, c.lengths, out, c.kd, c.vd, window=300, sinks=4, workspace=ws)
    for n in (900, 650, 7):
        c.lengths[0] = n
        q.copy_(torch.randn_like(q))
        want = call(c, q, 300, 4)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
