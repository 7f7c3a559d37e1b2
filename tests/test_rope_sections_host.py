"""The rotation's binding with one position axis: its sections, if given, are all pairs."""
import pytest

import gemm_q8_act_amd as nvq


@pytest.mark.parametrize("sections", [[5], [16], [0], (7,)])
def test_one_axis_with_other_sections_is_refused(sections):
    import torch

    x, t, p = torch.zeros((3, 1, 32)), torch.zeros((10, 16)), torch.zeros((1, 3), dtype=torch.int32)
    s, c, d = torch.zeros(3, dtype=torch.int64), torch.zeros((2, 1, 16, 32), dtype=torch.int8), torch.zeros((2, 1, 16, 1), dtype=torch.float16)
    for at in (p, p[0]):
        with pytest.raises(ValueError, match="sections"):
            nvq.nvq_qk_norm_rope(x, x, t, at, x, x, sections=sections)
        with pytest.raises(ValueError, match="sections"):
            nvq.nvq_rope_kv_write(x, x, x, t, at, s, x, c, c, d, d, sections=sections)
