"""The paged key-value cache on the GPU: codes and scales bit for bit against the oracle's
Q8_0, the row order against the header's rule, pages, slots, strides and types."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import place_of, rounded, torch_type
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu


def cache(fmt, n_pages, H, page, D, fill=0):
    torch = torch_dev()
    shape = (n_pages, H, page, D)
    kc, vc = (torch.full(shape, fill, dtype=torch.int8 if fmt == "q8_0" else torch_type(fmt), device="cuda") for _ in "kv")
    if fmt != "q8_0":
        return kc, vc, None, None
    return kc, vc, *(torch.full((*shape[:3], D // 32), fill, dtype=torch.float16, device="cuda") for _ in "kv")


@pytest.mark.parametrize("T,H,D,page,type_", [
    (1, 1, 32, 16, "f32"), (1, 8, 128, 64, "f32"), (37, 3, 96, 16, "f16"), (130, 8, 128, 32, "bf16"), (5, 2, 256, 64, "f32"),
    (19, 5, 64, 128, "bf16"), (7, 1, 160, 16, "f32"), (6, 2, 192, 16, "f16"), (9, 2, 224, 32, "f32")])
def test_q8_0_rows_match_the_oracle(oracle, T, H, D, page, type_):
    torch = torch_dev()
    say(f"kv q8_0 T={T} H={H} D={D} page={page} {type_}")
    r = np.random.Generator(np.random.PCG64(T * 1000 + D))
    n_pages = -(-T // page) + 2
    slots = r.permutation(n_pages * page)[:T]
    x = [rounded(r.standard_normal((T, H, D)) * r.choice([1e-6, 1e-3, 1.0, 300.0], (T, H, 1)), type_) for _ in "kv"]
    x[0][0, 0, :32] = 0.0  # a block of zeros
    dev = [torch.from_numpy(a).to(torch_type(type_)).cuda() for a in x]
    kc, vc, kd, vd = cache("q8_0", n_pages, H, page, D, fill=3)
    sl = torch.from_numpy(slots).cuda()
    nvq.nvq_kv_write(dev[0], dev[1], sl, kc, vc, kd, vd)
    back = [torch.full((T, H, D), 9.0, dtype=torch.float32, device="cuda") for _ in "kv"]
    nvq.nvq_kv_read(kc, vc, sl, back[0], back[1], kd, vd)
    at = place_of(D)
    for a, codes, scales, b in ((x[0], kc, kd, back[0]), (x[1], vc, vd, back[1])):
        qo, do, _ = oracle.quantize_q8_0(a.reshape(T * H, D))
        codes, scales = host(codes), host(scales).view(np.uint16)
        got = codes[slots // page, :, slots % page][:, :, at].reshape(T * H, D)
        sc = scales[slots // page, :, slots % page].reshape(T * H, D // 32)
        assert (got == qo).all() and (sc == do).all()
        want = qo.astype(np.float32) * np.repeat(do.view(np.float16).astype(np.float32), 32, axis=1)
        assert (host(b).reshape(T * H, D) == want).all()
        # every other row is untouched
        rest = np.ones((n_pages, page), bool)
        rest[slots // page, slots % page] = False
        assert (codes.transpose(0, 2, 1, 3)[rest] == 3).all() and (scales.view(np.float16).transpose(0, 2, 1, 3)[rest] == 3).all()


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("type_", ["f32", "f16", "bf16"])
def test_16_bit_rows(fmt, type_):
    torch = torch_dev()
    T, H, D, page = 23, 3, 96, 16
    r = np.random.Generator(np.random.PCG64(5))
    x = [torch.from_numpy(r.standard_normal((T, H, D)).astype(np.float32)).to(torch_type(type_)) for _ in "kv"]
    kc, vc, _, _ = cache(fmt, 4, H, page, D)
    slots = torch.from_numpy(r.permutation(4 * page)[:T])
    nvq.nvq_kv_write(x[0].cuda(), x[1].cuda(), slots.cuda(), kc, vc)
    back = [torch.empty((T, H, D), dtype=torch_type(type_), device="cuda") for _ in "kv"]
    nvq.nvq_kv_read(kc, vc, slots.cuda(), *back)
    for a, c, b in zip(x, (kc, vc), back):
        want = a.float().to(torch_type(fmt))
        assert torch.equal(c.cpu()[slots // page, :, slots % page], want)
        assert torch.equal(b.cpu(), want.float().to(torch_type(type_)))


@pytest.mark.parametrize("fmt", ["q8_0", "f16"])
def test_slots_that_name_no_row(fmt):
    """Negative slots and slots past the cache write nothing; they read back as zeros and as NaN."""
    torch = torch_dev()
    T, H, D, page = 6, 2, 64, 16
    k, v = (torch.randn((T, H, D), device="cuda") for _ in "kv")
    kc, vc, kd, vd = cache(fmt, 2, H, page, D, fill=5)
    slots = torch.tensor([-1, 31, 32, -(1 << 62), 1 << 62, 0], device="cuda")
    nvq.nvq_kv_write(k, v, slots, kc, vc, kd, vd)
    touched = torch.zeros((2, page), dtype=torch.bool)
    touched[1, 15] = touched[0, 0] = True
    for c in (kc, vc):
        rows = c.cpu().transpose(1, 2)
        assert (rows[~touched] == 5).all() and not (rows[touched] == 5).all()
    ko, vo = (torch.full((T, H, D), 2.0, device="cuda") for _ in "kv")
    nvq.nvq_kv_read(kc, vc, slots, ko, vo, kd, vd)
    for o, x in ((ko.cpu(), k.cpu()), (vo.cpu(), v.cpu())):
        assert (o[[0, 3]] == 0).all() and o[[2, 4]].isnan().all()
        assert (o[[1, 5]] - x[[1, 5]]).abs().max() <= x.abs().max() / 127


def test_strided_rows_and_empty_calls():
    """Columns of one fused row, heads before tokens, one key broadcast to all tokens; no rows at all."""
    torch = torch_dev()
    T, Hq, H, D, page = 21, 5, 2, 64, 16
    y = torch.randn((T, (Hq + 2 * H) * D), device="cuda")
    k = y[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    v = torch.randn((H, T, D), device="cuda").transpose(0, 1)
    slots = torch.arange(T, device="cuda") + 3
    out = []
    for kk, vv in ((k, v), (k.contiguous(), v.contiguous())):
        c = cache("q8_0", 2, H, page, D)
        nvq.nvq_kv_write(kk, vv, slots, *c)
        out.append(c)
    assert all(torch.equal(a, b) for a, b in zip(*out))
    c = cache("q8_0", 2, H, page, D)
    one = torch.randn((1, H, D), device="cuda")
    nvq.nvq_kv_write(one.expand(T, H, D), one.expand(T, H, D), slots, *c)
    ko = torch.empty((T, 3 * H, D), device="cuda")
    nvq.nvq_kv_read(c[0], c[1], slots, ko[:, H:2 * H], ko[:, 2 * H:], c[2], c[3])
    assert torch.equal(ko[:, H:2 * H], ko[:, 2 * H:]) and (ko[:, H:2 * H] == ko[:1, H:2 * H]).all()
    none = torch.empty((0, H, D), device="cuda")
    nvq.nvq_kv_write(none, none, slots[:0], *c)
    nvq.nvq_kv_read(c[0], c[1], slots[:0], none, none, c[2], c[3])


def test_non_finite_blocks_read_back_as_nan():
    torch = torch_dev()
    k = torch.randn((3, 1, 64), device="cuda")
    k[0, 0, 5], k[1, 0, 40], k[2, 0, 3] = float("inf"), float("nan"), -float("inf")
    c = cache("q8_0", 1, 1, 16, 64)
    slots = torch.arange(3, device="cuda")
    nvq.nvq_kv_write(k, k, slots, *c)
    o, p = torch.empty_like(k), torch.empty_like(k)
    nvq.nvq_kv_read(c[0], c[1], slots, o, p, c[2], c[3])
    bad = torch.zeros((3, 1, 64), dtype=torch.bool)
    bad[0, 0, :32] = bad[1, 0, 32:] = bad[2, 0, :32] = True
    assert torch.equal(o.isnan().cpu(), bad) and torch.equal(p.isnan().cpu(), bad)


def test_rows_past_32_bit_offsets():
    """A cache of over 4 GiB: the last page's rows land there and nowhere else."""
    torch = torch_dev()
    H, D, page = 8, 256, 4096
    n_pages = (1 << 32) // (H * D * page) + 3
    kc, vc = (torch.zeros((n_pages, H, page, D), dtype=torch.int8, device="cuda") for _ in "kv")
    kd, vd = (torch.zeros((n_pages, H, page, D // 32), dtype=torch.float16, device="cuda") for _ in "kv")
    k, v = (torch.randn((2, H, D), device="cuda") for _ in "kv")
    slots = torch.tensor([(n_pages - 1) * page + page - 1, n_pages // 2 * page], device="cuda")
    nvq.nvq_kv_write(k, v, slots, kc, vc, kd, vd)
    for c in (kc, vc):
        assert int((c[n_pages - 1, :, page - 1] != 0).sum()) > 0.9 * H * D
        assert int((c[:2] != 0).sum()) == 0
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    nvq.nvq_kv_read(kc, vc, slots, ko, vo, kd, vd)
    assert (ko - k).abs().max() < 0.05 and (vo - v).abs().max() < 0.05
