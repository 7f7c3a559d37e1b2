"""Norms and position rotation of heads, into rows and into the paged cache, against float64.

Bounds.  A sum of squares takes 2 D/32 + 4 float32 roundings at most, its root half of them, the mean, eps, the
root and the two products by it and by the weight 5 more: a normed value is off by (D/32 + 7) 2^-24
of itself.  A turned one is the difference of two products of such values: off by (D/32 + 10) 2^-24 of
the sum of their magnitudes.  The result is rounded to its type.
"""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import HALF_UNIT, SMALLEST, check, rounded, torch_type
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu

PAIRS = {"halves": nvq.NVQ_ROPE_HALVES, "neighbours": nvq.NVQ_ROPE_NEIGHBOURS}


def want_rows(x, w, eps, table, positions, R, pairs, sections=None):
    """Float64 rows [T, H, D] and the sum of magnitudes that each is made of."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, size = x.copy(), np.abs(x)
    positions = np.atleast_2d(positions)
    axis = [a for a, n in enumerate(sections if sections else [R // 2]) for _ in range(n)]
    for c in range(R // 2):
        i, j = (c, c + R // 2) if pairs == "halves" else (2 * c, 2 * c + 1)
        p = positions[axis[c]]
        ok = (p >= 0) & (p < len(table))
        row = table[np.where(ok, p, 0)].astype(np.float64)
        co, si = (np.where(ok, row[:, k], np.nan)[:, None] for k in (c, R // 2 + c))
        y[..., i], y[..., j] = x[..., i] * co - x[..., j] * si, x[..., j] * co + x[..., i] * si
        size[..., i] = np.abs(x[..., i] * co) + np.abs(x[..., j] * si)
        size[..., j] = np.abs(x[..., j] * co) + np.abs(x[..., i] * si)
    return y, size


def limit(y, size, D, out):
    e = (D / 32 + 10) * 2.0 ** -24 * size
    return e + HALF_UNIT[out] * (np.abs(y) + e) + SMALLEST[out]


def data(T, H, D, type_, seed, width=1.0):
    r = np.random.Generator(np.random.PCG64(seed))
    return rounded(r.standard_normal((T, H, D)) * r.choice([0.1, 1.0, 5.0], (T, H, 1)) * width, type_)


def dev(x, type_="f32"):
    torch = torch_dev()
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch_type(type_)).cuda()


def ints(x):
    torch = torch_dev()
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def weights(D, seed):
    r = np.random.Generator(np.random.PCG64(seed))
    return (1 + r.standard_normal(D) / 4).astype(np.float32)


CASES = [  # T, Hq, Hkv, D, R, pairs, type, out, norm
    (1, 5, 1, 128, 128, "halves", "f32", "f32", True), (1, 1, 1, 32, 32, "neighbours", "f32", "f32", False),
    (37, 3, 3, 64, 64, "halves", "f32", "bf16", True), (21, 4, 2, 96, 96, "halves", "f16", "f16", True),
    (130, 8, 8, 128, 64, "halves", "bf16", "bf16", True), (64, 2, 1, 128, 32, "halves", "bf16", "f32", False),
    (19, 5, 1, 160, 160, "neighbours", "f16", "f32", True), (7, 3, 1, 192, 96, "halves", "f32", "f16", True),
    (9, 2, 2, 224, 224, "halves", "bf16", "f16", True), (33, 4, 2, 256, 256, "halves", "bf16", "bf16", True),
    (5, 7, 3, 256, 128, "neighbours", "f32", "f32", True), (11, 3, 1, 64, 4, "halves", "f32", "f32", True),
    (11, 3, 1, 64, 12, "halves", "f32", "f32", False), (11, 3, 1, 96, 20, "neighbours", "f32", "f32", True),
    (300, 40, 8, 128, 128, "halves", "bf16", "bf16", True), (257, 6, 2, 64, 64, "neighbours", "f16", "bf16", False)]


@pytest.mark.parametrize("T,Hq,Hkv,D,R,pairs,type_,out,norm", CASES)
def test_rows(T, Hq, Hkv, D, R, pairs, type_, out, norm):
    torch = torch_dev()
    say(f"rope T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} {pairs} {type_} -> {out} norm={norm}")
    P = 5000
    table = nvq.nvq_rope_table(P, R)
    r = np.random.Generator(np.random.PCG64(T + D))
    at = r.integers(0, P, T)
    x = [data(T, h, D, type_, 10 * T + h) for h in (Hq, Hkv)]
    w = [weights(D, i) if norm else None for i in (1, 2)]
    o = [torch.full(a.shape, 7.0, dtype=torch_type(out), device="cuda") for a in x]
    nvq.nvq_qk_norm_rope(dev(x[0], type_), dev(x[1], type_), dev(table), ints(at), *o, *(None if a is None else dev(a) for a in w),
                         eps=1e-5, pairs=PAIRS[pairs])
    for a, ww, got in zip(x, w, o):
        y, size = want_rows(a, ww, 1e-5, table, at, R, pairs)
        check(host(got.float()), y, limit(y, size, D, out), "rows")


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("sections", [[5, 27], [8, 12, 12], [0, 32], [10, 0, 22], [3, 4, 5, 20], [32, 0, 0, 0]])
def test_axes(sections, pairs):
    torch = torch_dev()
    T, H, D, R, P = 23, 3, 64, 64, 700
    table = nvq.nvq_rope_table(P, R, base=500.0)
    at = np.random.Generator(np.random.PCG64(3)).integers(0, P, (len(sections), T))
    x = data(T, H, D, "f32", 5)
    q, k = (torch.empty((T, H, D), device="cuda") for _ in "qk")
    nvq.nvq_qk_norm_rope(dev(x), dev(x), dev(table), ints(at), q, k, k_weight=dev(weights(D, 1)), pairs=PAIRS[pairs], sections=sections)
    for got, w in ((q, None), (k, weights(D, 1))):
        y, size = want_rows(x, w, 1e-6, table, at, R, pairs, sections)
        check(host(got), y, limit(y, size, D, "f32"), "rows")


def test_table_and_far_positions():
    """The table against the angle in exact arithmetic reduced in double; far positions use their own rows."""
    P, R = 131072, 64
    table = nvq.nvq_rope_table(P, R)
    inv = 10000.0 ** (-np.arange(R // 2) * 2.0 / R)
    for p in (0, 1, 4095, 100001, P - 1):
        angle = p * inv
        assert np.abs(table[p, :R // 2] - np.cos(angle)).max() <= 2.0 ** -24 and np.abs(table[p, R // 2:] - np.sin(angle)).max() <= 2.0 ** -24
    assert np.array_equal(nvq.nvq_rope_table(9, R, inv_freq=inv), table[:9])
    torch = torch_dev()
    at = np.array([P - 1, 0, 100001, 65536])
    x = data(4, 2, 64, "f32", 6)
    q = torch.empty((4, 2, 64), device="cuda")
    nvq.nvq_qk_norm_rope(dev(x), None, dev(table), ints(at), q, None)
    y, size = want_rows(x, None, 0, table, at, R, "halves")
    check(host(q), y, limit(y, size, 64, "f32"), "far")


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_positions_outside_the_table(pairs):
    """NaN in the pairs that such a position turns, and nowhere else; nothing is read there."""
    torch = torch_dev()
    table = nvq.nvq_rope_table(50, 32)
    at = np.array([[3, -1, 50, 7, 1 << 30, -(1 << 31)], [4, 5, 6, -2, 3, 2]])
    x = data(6, 2, 64, "f32", 7)
    q = torch.empty((6, 2, 64), device="cuda")
    nvq.nvq_qk_norm_rope(dev(x), None, dev(table), ints(at), q, None, pairs=PAIRS[pairs], sections=[6, 10])
    y, size = want_rows(x, None, 0, table, at, 32, pairs, [6, 10])
    got = host(q)
    assert (np.isnan(got) == np.isnan(y)).all() and 0 < np.isnan(y).sum() < y.size
    ok = np.isfinite(y)
    assert (np.abs(got - y)[ok] <= limit(y, size, 64, "f32")[ok]).all()


@pytest.mark.parametrize("pairs,R", [("halves", 128), ("halves", 64), ("halves", 20), ("neighbours", 128)])
@pytest.mark.parametrize("T", [1, 700])
def test_in_place_strides_and_one_side(pairs, R, T):
    """Columns of one fused row turned in place; outputs with heads first; queries or keys alone: the same bits."""
    torch = torch_dev()
    Hq, Hkv, D = 5, 2, 128
    table, at = dev(nvq.nvq_rope_table(900, R)), ints(np.arange(T) + 100)
    y = torch.randn((T, (Hq + 2 * Hkv) * D), device="cuda").bfloat16()
    q, k = y[:, :Hq * D].unflatten(1, (Hq, D)), y[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    w = dict(q_weight=dev(weights(D, 1)), k_weight=dev(weights(D, 2)), pairs=PAIRS[pairs])
    want = [torch.empty(x.shape, dtype=x.dtype, device="cuda") for x in (q, k)]
    nvq.nvq_qk_norm_rope(q.contiguous(), k.contiguous(), table, at, *want, **w)
    first = [torch.empty((x.shape[1], T, D), dtype=x.dtype, device="cuda").transpose(0, 1) for x in (q, k)]
    nvq.nvq_qk_norm_rope(q, k, table, at, *first, **w)
    alone = [torch.empty_like(x) for x in want]
    nvq.nvq_qk_norm_rope(q, None, table, at, alone[0], None, **w)
    nvq.nvq_qk_norm_rope(None, k, table, at, None, alone[1], **w)
    rest = y[:, (Hq + Hkv) * D:].clone()
    nvq.nvq_qk_norm_rope(q, k, table, at, q, k, **w)
    for a in (first, alone, (q, k)):
        assert all(torch.equal(b, c) for b, c in zip(a, want))
    assert torch.equal(y[:, (Hq + Hkv) * D:], rest)


def test_norm_of_zeros_and_of_large_rows():
    torch = torch_dev()
    x = np.zeros((3, 1, 64), np.float32)
    x[1], x[2] = 1e15, 1e-15
    o = torch.empty((3, 1, 64), device="cuda")
    nvq.nvq_qk_norm_rope(dev(x), None, dev(nvq.nvq_rope_table(1, 4)), ints([0, 0, 0]), o, None, q_weight=dev(np.ones(64, np.float32)), eps=1e-6)
    got = host(o)
    assert (got[0] == 0).all() and np.abs(got[1] - 1).max() < 2e-6 and np.abs(got[2] / 1e-12 - 1).max() < 2e-6


def cache(fmt, n_pages, H, page, D):
    torch = torch_dev()
    shape = (n_pages, H, page, D)
    kc, vc = (torch.full(shape, 3, dtype=torch.int8 if fmt == "q8_0" else torch_type(fmt), device="cuda") for _ in "kv")
    if fmt != "q8_0":
        return kc, vc, None, None
    return kc, vc, *(torch.full((*shape[:3], D // 32), 3.0, dtype=torch.float16, device="cuda") for _ in "kv")


@pytest.mark.parametrize("fmt", ["q8_0", "f16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,pairs,type_,out,norm", CASES)
def test_cache_rows_are_those_of_the_single_steps(T, Hq, Hkv, D, R, pairs, type_, out, norm, fmt):
    """Bit for bit what nvq_kv_write makes of the turned rows in float32; queries as nvq_qk_norm_rope's; other cache rows
    untouched; slots that name no row write nothing."""
    torch = torch_dev()
    say(f"rope write T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} {pairs} {type_} -> {out}, {fmt} norm={norm}")
    P, page = 5000, 16
    r = np.random.Generator(np.random.PCG64(T + D))
    table, at = dev(nvq.nvq_rope_table(P, R)), ints(r.integers(0, P, T))
    q, k, v = (dev(data(T, h, D, type_, T + i), type_) for i, h in enumerate((Hq, Hkv, Hkv)))
    w = dict(q_weight=dev(weights(D, 1)), k_weight=dev(weights(D, 2))) if norm else {}
    n_pages = -(-T // page) + 2
    slots = r.permutation(n_pages * page)[:T]
    if T > 4:
        slots[[1, 3]] = -1, n_pages * page + 5
    slots = torch.from_numpy(slots).cuda()
    turned, want_q = torch.empty(k.shape, device="cuda"), torch.empty(q.shape, dtype=torch_type(out), device="cuda")
    nvq.nvq_qk_norm_rope(None, k, table, at, None, turned, pairs=PAIRS[pairs], **w)
    nvq.nvq_qk_norm_rope(q, None, table, at, want_q, None, pairs=PAIRS[pairs], **w)
    want, got = cache(fmt, n_pages, Hkv, page, D), cache(fmt, n_pages, Hkv, page, D)
    nvq.nvq_kv_write(turned, v.float(), slots, *want)
    got_q = torch.empty_like(want_q)
    nvq.nvq_rope_kv_write(q, k, v, table, at, slots, got_q, *got, pairs=PAIRS[pairs], **w)
    assert torch.equal(got_q, want_q)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
    nvq.nvq_rope_kv_write(None, k, v, table, at, slots, None, *got, pairs=PAIRS[pairs], **w)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)


def test_a_position_outside_reads_back_as_nan():
    torch = torch_dev()
    k = torch.randn((3, 2, 64), device="cuda")
    table, slots = dev(nvq.nvq_rope_table(10, 32)), torch.arange(3, device="cuda")
    c = cache("q8_0", 1, 2, 16, 64)
    nvq.nvq_rope_kv_write(None, k, k, table, ints([4, 10, 5]), slots, None, *c)
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    nvq.nvq_kv_read(c[0], c[1], slots, ko, vo, c[2], c[3])
    assert ko[1, :, :32].isnan().all() and not ko[1, :, 32:].isnan().any() and not ko[[0, 2]].isnan().any() and not vo.isnan().any()


def test_empty_calls():
    torch = torch_dev()
    x = torch.empty((0, 2, 64), device="cuda")
    table, at = dev(nvq.nvq_rope_table(10, 32)), ints([])
    nvq.nvq_qk_norm_rope(x, x, table, at, x, x)
    c = cache("q8_0", 1, 2, 16, 64)
    nvq.nvq_rope_kv_write(x, x, x, table, at, torch.empty(0, dtype=torch.int64, device="cuda"), x, *c)
    assert all((a == 3).all() for a in c)


def test_more_rows_than_one_launch_takes():
    """Over 2^28 rows: the last token's, in the second launch, use their own positions and slots."""
    torch = torch_dev()
    H, D = 1, 32
    T = (1 << 27) + 1000
    one = torch.randn((1, H, D), device="cuda").half()
    k = one.expand(T, H, D)
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    at[-3:], slots[-3:] = torch.tensor([5, 6, 7], device="cuda"), torch.tensor([0, 20, 31], device="cuda")
    table = dev(nvq.nvq_rope_table(10, 32))
    c, want = cache("f16", 2, H, 16, D), cache("f16", 2, H, 16, D)
    nvq.nvq_rope_kv_write(None, k, k, table, at, slots, None, *c)
    nvq.nvq_rope_kv_write(None, k[-3:], k[-3:], table, at[-3:].contiguous(), slots[-3:].contiguous(), None, *want)
    assert torch.equal(c[0], want[0]) and torch.equal(c[1], want[1]) and not torch.equal(c[0][0, 0, 0], c[0][1, 0, 15])


def test_captured_and_on_another_stream():
    torch = torch_dev()
    T, Hq, Hkv, D, page = 9, 4, 2, 64, 16
    table, at = dev(nvq.nvq_rope_table(100, 64)), ints(np.arange(T))
    q, k, v = (torch.randn((T, h, D), device="cuda") for h in (Hq, Hkv, Hkv))
    slots = torch.arange(T, device="cuda")
    c, o = cache("q8_0", 1, Hkv, page, D), torch.empty_like(q)

    def call(c, o, **kw):
        nvq.nvq_rope_kv_write(q, k, v, table, at, slots, o, *c, **kw)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(c, o, stream=s.cuda_stream)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(c, o)
    for i in range(3):
        q.copy_(torch.randn_like(q)), k.copy_(torch.randn_like(k)), at.add_(7)
        want, wo = cache("q8_0", 1, Hkv, page, D), torch.empty_like(o)
        call(want, wo)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and all(torch.equal(a, b) for a, b in zip(c, want))
