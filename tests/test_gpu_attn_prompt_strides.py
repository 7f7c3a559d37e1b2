"""Prompt attention over key and value tensors of one row, whose token stride has no meaning."""
import numpy as np
import pytest

from gpu_cases import torch_dev
from test_gpu_attn_prompt import call, make, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [0, 8, 1 << 31])
def test_single_row_with_any_token_stride(stride):
    torch = torch_dev()
    q, k, v, cu_q, cu_k = make([(1, 1), (0, 0), (0, 0)], 4, 2, 64, "bf16", 3)
    v[0, 1, 5] = np.inf
    q, k, v = (on_gpu(x, "bf16") for x in (q, k, v))
    want = call(q, k, v, cu_q, cu_k)
    assert torch.equal(want, v.repeat_interleave(2, dim=1))  # one key: its own values
    odd = [x.as_strided((1, 2, 64), (stride, 64, 1)) for x in (k, v)]
    assert torch.equal(call(q, *odd, cu_q, cu_k), want)
