"""Norms of heads so small that their squares leave float32's normal range, or float32, with an eps as small or none."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import check
from gpu_cases import host, torch_dev
from test_gpu_rope import dev, ints, limit, want_rows, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-39, 1e-31])
@pytest.mark.parametrize("D,R,pairs", [(64, 64, "halves"), (96, 96, "halves"), (64, 32, "neighbours")])
def test_norms_of_small_heads(D, R, pairs, eps):
    """Of widths 1e-36 to 1e-12: bounds as for any other width (subnormal inputs are given as float32 holds them)."""
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(D))
    x = (r.standard_normal((13, 1, D)) * 10.0 ** -np.arange(12, 38, 2)[:, None, None]).astype(np.float32)
    table, at = nvq.nvq_rope_table(50, R), r.integers(0, 50, len(x))
    o = torch.empty(x.shape, device="cuda")
    w = weights(D, 1)
    nvq.nvq_qk_norm_rope(dev(x), None, dev(table), ints(at), o, None, q_weight=dev(w), eps=eps,
                         pairs={"halves": nvq.NVQ_ROPE_HALVES, "neighbours": nvq.NVQ_ROPE_NEIGHBOURS}[pairs])
    y, size = want_rows(x, w, float(np.float32(eps)), table, at, R, pairs)
    check(host(o), y, limit(y, size, D, "f32"), "small heads")
