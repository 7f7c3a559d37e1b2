"""Norms and rotation into the cache at every head width, each with every way that its pairs can lie: bit for bit what the
single steps (nvq_qk_norm_rope into float32 rows, nvq_kv_write) make of the same rows."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from gpu_cases import say, torch_dev
from test_gpu_rope import PAIRS, cache, data, dev, ints, weights

pytestmark = pytest.mark.gpu

# all of a head's channels turned, half of them, and a number that ends inside a block
WIDTHS = [(D, R, pairs) for D in range(32, 257, 32) for R in (D, D // 2, D // 2 - 12 if D > 32 else 4) for pairs in PAIRS]


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
@pytest.mark.parametrize("D,R,pairs", WIDTHS)
def test_cache_rows_at_every_width(D, R, pairs, fmt):
    torch = torch_dev()
    say(f"rope write D={D} R={R} {pairs} {fmt}")
    T, Hq, Hkv, page, P = 21, 3, 2, 16, 300
    r = np.random.Generator(np.random.PCG64(D + R))
    table, at = dev(nvq.nvq_rope_table(P, R)), ints(r.integers(0, P, T))
    q, k, v = (dev(data(T, h, D, "f32", D + i)) for i, h in enumerate((Hq, Hkv, Hkv)))
    w = dict(q_weight=dev(weights(D, 1)), k_weight=dev(weights(D, 2)), pairs=PAIRS[pairs])
    slots = torch.from_numpy(r.permutation(3 * page)[:T]).cuda()
    turned, want_q, got_q = torch.empty_like(k), torch.empty_like(q), torch.empty_like(q)
    nvq.nvq_qk_norm_rope(q, k, table, at, want_q, turned, **w)
    want, got = cache(fmt, 3, Hkv, page, D), cache(fmt, 3, Hkv, page, D)
    nvq.nvq_kv_write(turned, v, slots, *want)
    nvq.nvq_rope_kv_write(q, k, v, table, at, slots, got_q, *got, **w)
    assert torch.equal(got_q, want_q)
    assert all(torch.equal(a, b) for a, b in zip(got, want) if a is not None)
