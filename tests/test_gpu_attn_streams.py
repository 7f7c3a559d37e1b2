"""The attention entries on a stream other than torch's current one."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import Paged
from gpu_cases import torch_dev

pytestmark = pytest.mark.gpu


def test_scratch_is_not_memory_that_the_current_stream_still_writes():
    """A tensor of the scratch's size is let go of while the current stream has yet to fill it; a call on another
    stream, which does not wait for that, must not work in its memory."""
    torch = torch_dev()
    r = np.random.Generator(np.random.PCG64(1))
    seqs = [tuple(r.standard_normal((n, 2, 64)).astype(np.float32) for _ in "kv") for n in (3000, 700)]
    c = Paged("q8_0", seqs, 2, 64, 16, 2)
    q = torch.from_numpy(r.standard_normal((2, 4, 64)).astype(np.float32)).cuda()
    want = c.decode(q)
    need = nvq.nvq_attn_decode_workspace_bytes(2, 4, 2, 64, c.max_pages, 16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = torch.full(q.shape, 7.0, device="cuda")
        torch.cuda.synchronize()
        gone = torch.empty(need, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(2_000_000)
        gone.fill_(0xFF)
        del gone
        c.decode(q, got, stream=s.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
