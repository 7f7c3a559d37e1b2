"""Attention of one new token over the paged cache, on the GPU against float64."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import Paged, attention, bound, check, rounded, torch_type
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu


def rows(r, n, H, D, width=1.0):
    return (r.standard_normal((n, H, D)) * width).astype(np.float32)


def run(fmt, type_, lens, Hq, Hkv, D, page, seed, width_q=1.0, width_v=1.0, scale=None, what="", rows_of=rows):
    torch = torch_dev()
    say(f"decode {what} fmt={fmt} type={type_} lens={lens} Hq={Hq} Hkv={Hkv} D={D} page={page}")
    r = np.random.Generator(np.random.PCG64(seed))
    seqs = [(rows_of(r, n, Hkv, D), rows_of(r, n, Hkv, D, width_v)) for n in lens]
    c = Paged(fmt, seqs, Hkv, D, page, seed + 1)
    q = rounded(r.standard_normal((len(lens), Hq, D)) * width_q, type_)
    got = host(c.decode(torch.from_numpy(q).to(torch_type(type_)).cuda(), scale=scale).float())
    scale = D ** -0.5 if scale is None else scale
    worst = 0.0
    for i, (k, v) in enumerate(c.rows):
        for h in range(Hq):
            j = h * Hkv // Hq
            want, A, S = attention(q[i, h:h + 1], k[:, j], v[:, j], scale, np.ones((1, len(k)), bool))
            worst = max(worst, check(got[i, h:h + 1], want, bound(want, A, S, D, len(k), type_, 0.0, 8), f"{what} sequence {i} head {h}"))
            if len(k) == 0:
                assert (got[i, h] == 0).all()
    say(f"  worst error / bound {worst:.3g}")


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129]


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
def test_lengths_at_tile_and_page_edges(fmt, type_):
    run(fmt, type_, EDGES, 10, 2, 128, 16, 11)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_head_widths(fmt, D):
    run(fmt, "f32", [1, 40, 301], 6, 2, D, 32, 100 + D)


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (5, 1), (16, 1), (17, 1), (40, 8), (70, 2)])
def test_head_layouts(fmt, Hq, Hkv):
    run(fmt, "f32", [77, 5], Hq, Hkv, 64, 16, 7 * Hq + Hkv)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("lens,page", [([255, 256, 257, 511, 0, 513], 64), ([5000], 64), ([3001, 1, 2048, 0, 700], 256)])
def test_lengths_that_are_split(fmt, lens, page):
    run(fmt, "f32", lens, 5, 1, 128, page, sum(lens))


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", [([20011, 900], 16, 16, 64, 64), ([21500], 80, 16, 128, 256), ([5000, 0, 3900], 128, 64, 32, 16),
                                                ([4100], 64, 32, 256, 16), ([9000, 31], 64, 32, 96, 32)])
def test_parts_of_many_tiles(fmt, lens, Hq, Hkv, D, page):
    """Many key heads, so that the parts are long: every wavefront takes 3 to 12 tiles in turn, over both slots."""
    run(fmt, "f32", lens, Hq, Hkv, D, page, sum(lens) + D)


def test_many_sequences():
    """More sequences than a wavefront has lanes, most of them short or empty."""
    r = np.random.Generator(np.random.PCG64(3))
    run("q8_0", "f16", [int(x) for x in r.choice([0, 0, 1, 3, 20, 400], 150)], 2, 1, 64, 16, 4)


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("width_q,width_v,scale", [(300.0, 1.0, None), (1e-3, 1.0, None), (1.0, 6e4 / 5, None), (1.0, 1e-4, None), (1.0, 1.0, -0.3),
                                                   (1.0, 1.0, 0.0), (1e-20, 1.0, 1e20)])
def test_ranges(fmt, width_q, width_v, scale):
    """Sharp and flat scores, value scales near both ends of binary16, scales that are negative, zero and large."""
    run(fmt, "f32", [33, 600], 4, 2, 64, 16, 21, width_q, width_v, scale)


def test_value_scales_that_grow_along_the_sequence():
    """Value blocks over 9 orders of magnitude, the largest ones last, so that what is summed is rescaled on the way."""
    def growing(r, n, H, D, width=1.0):
        x = r.standard_normal((n, H, D))
        return (x * 10.0 ** np.linspace(-5, 4, n)[:, None, None] if width == 2.0 else x).astype(np.float32)

    run("q8_0", "f32", [900], 4, 1, 64, 16, 31, width_v=2.0, rows_of=growing)


def test_scores_that_grow_along_the_sequence():
    """The running maximum moves in every step."""
    def growing(r, n, H, D, width=1.0):
        return (r.standard_normal((n, H, D)) * np.linspace(0.01, 30, n)[:, None, None]).astype(np.float32)

    for fmt in ("q8_0", "f16"):
        run(fmt, "f32", [700], 4, 1, 64, 16, 33, rows_of=growing)


def _small(fmt="q8_0", lens=(50, 20), Hq=4, Hkv=2, D=64, page=16, seed=9):
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(seed))
    c = Paged(fmt, [(rows(r, n, Hkv, D), rows(r, n, Hkv, D)) for n in lens], Hkv, D, page, seed)
    q = torch.from_numpy(rows(r, len(lens), Hq, D)).cuda()
    return c, q


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
def test_lengths_and_pages_out_of_range_give_nan(fmt):
    torch = torch_dev()
    c, q = _small(fmt, lens=(50, 20, 30, 40))
    want = c.decode(q)
    c.lengths[0], c.lengths[1] = -1, c.max_pages * 16 + 1
    c.table[2, 1] = c.n_pages
    got = c.decode(q)
    assert got[:3].isnan().all() and torch.equal(got[3], want[3])
    c.table[2, 1] = -1
    assert c.decode(q)[2].isnan().all()


def test_non_finite_keys_and_values_show():
    torch = torch_dev()
    for where in ("kc", "vc"):
        c, q = _small("f16")
        want = c.decode(q)
        getattr(c, where)[c.table[0, 0], 0, 3, 7] = float("nan")  # key head 0 of sequence 0
        got = c.decode(q)
        assert not torch.isfinite(got[0, :2]).all(dim=1).any()
        assert torch.equal(got[1], want[1]) and torch.equal(got[0, 2:], want[0, 2:])


def test_strided_queries_same_bits_and_deterministic():
    torch = torch_dev()
    c, q = _small(lens=(3000, 700), Hq=10, Hkv=2)
    want = c.decode(q)
    wide = torch.zeros((2, 3, 10, 64), device="cuda")
    wide[:, 1] = q
    assert torch.equal(c.decode(wide[:, 1]), want)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)
    for _ in range(3):
        assert torch.equal(c.decode(turned), want)


def test_on_another_stream_and_with_a_workspace():
    torch = torch_dev()
    c, q = _small(lens=(3000, 700))
    want = c.decode(q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.decode(q, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)
    need = nvq.nvq_attn_decode_workspace_bytes(2, 4, 2, 64, c.max_pages, 16)
    assert need > 0
    guard = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.decode(q, workspace=guard[:need]), want)
    assert (guard[need:] == 0x5A).all()
    with pytest.raises(nvq.NvqError) as e:
        c.decode(q, workspace=guard[:need - 16])
    assert e.value.status == -7


def test_in_a_graph():
    """Write, attend, replayed with eager work between: each replay sees the cache as it is then."""
    torch = torch_dev()
    c, q = _small(lens=(400, 333))
    k, v = (torch.randn((2, 2, 64), device="cuda") for _ in "kv")
    slots = torch.stack([c.table[0, 24].long() * 16 + 15, c.table[1, 20].long() * 16 + 12])
    out = torch.empty_like(q)

    def work():
        nvq.nvq_kv_write(k, v, slots, c.kc, c.vc, c.kd, c.vd)
        c.decode(q, out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for i in range(4):
        k.normal_(), v.normal_(), q.normal_()
        g.replay()
        got = out.clone()
        out.fill_(3.0)
        work()
        torch.cuda.synchronize()
        assert torch.equal(got, out), i


def test_cache_past_32_bit_offsets():
    torch = torch_dev()
    H, D, page = 8, 256, 4096
    n_pages = (1 << 32) // (H * D * page) + 2
    kc, vc = (torch.zeros((n_pages, H, page, D), dtype=torch.int8, device="cuda") for _ in "kv")
    kd, vd = (torch.zeros((n_pages, H, page, D // 32), dtype=torch.float16, device="cuda") for _ in "kv")
    r = np.random.Generator(np.random.PCG64(8))
    n = 300
    k, v = (torch.from_numpy(rows(r, n, H, D)).cuda() for _ in "kv")
    nvq.nvq_kv_write(k, v, (n_pages - 1) * page + torch.arange(n, device="cuda"), kc, vc, kd, vd)
    q = torch.from_numpy(rows(r, 1, 2 * H, D)).cuda()
    out, low = torch.empty_like(q), torch.empty_like(q)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    nvq.nvq_attn_decode(q, kc, vc, torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda"), lengths, out, kd, vd)
    nvq.nvq_kv_write(k, v, torch.arange(n, device="cuda"), kc, vc, kd, vd)
    nvq.nvq_attn_decode(q, kc, vc, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), lengths, low, kd, vd)
    assert torch.equal(out, low) and float(out.abs().max()) > 0
