"""Cache calls of more rows than one launch takes (2^28 of 16 threads each)."""
import pytest

import gemm_q8_act_amd as nvq
from gpu_cases import torch_dev

pytestmark = pytest.mark.gpu


def test_rows_past_one_launch():
    """4200 tokens of 65536 heads of 32, all the same rows (strides of 0); slots name rows at both ends and on both sides
    of 2^28 rows, all others none."""
    torch = torch_dev()
    T, H, D, page = 4200, 65536, 32, 16
    assert T * H > 1 << 28
    kc, vc = (torch.zeros((1, H, page, D), dtype=torch.float16, device="cuda") for _ in "kv")
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    tokens = [0, 1, 4094, 4095, 4096, 4097, T - 2, T - 1]
    for i, t in enumerate(tokens):
        slots[t] = 2 * i + 1
    k, v = (torch.randn((1, H, D), dtype=torch.float16, device="cuda") for _ in "kv")
    k0, v0 = (torch.zeros_like(k).expand(T - 100, H, D) for _ in "kv")
    nvq.nvq_kv_write(k.expand(T, H, D), v.expand(T, H, D), slots, kc, vc)
    for c, x in ((kc, k), (vc, v)):
        assert (c[0, :, 1::2] == x[0, :, None]).all() and (c[0, :, 0::2] == 0).all()
    # the rows' own offsets: tokens from 100 on get other rows, all of them in one tensor's pages past the first launch's
    nvq.nvq_kv_write(k0, v0, slots[100:], kc, vc)
    for c, x in ((kc, k), (vc, v)):
        assert (c[0, :, [1, 3]] == x[0, :, None]).all() and (c[0, :, 5::2] == 0).all()


def test_read_past_one_launch():
    torch = torch_dev()
    T, H, D, page = 4200, 65536, 32, 16
    kc, vc = (torch.randn((1, H, page, D), dtype=torch.float16, device="cuda") for _ in "kv")
    slots = torch.arange(T, device="cuda") % page
    ko, vo = (torch.full((T, H, D), 7.0, dtype=torch.float16, device="cuda") for _ in "kv")
    nvq.nvq_kv_read(kc, vc, slots, ko, vo)
    for c, o in ((kc, ko), (vc, vo)):
        for t in (0, 1, 15, 16, 4094, 4095, 4096, 4097, T - 1):
            assert torch.equal(o[t], c[0, :, t % page]), t
        assert not (o[:, 0] == 7).all(dim=1).any()
