"""The tiled products' binding, without a GPU: where the scratch that it allocates comes from."""
import numpy as np
import pytest

import gemm_q8_act_amd as nvq


@pytest.mark.parametrize("name", ["nvfp4", "q4_1", "q4_k", "q5_k", "q6_k", "iq4_xs"])
def test_scratch_is_asked_for_with_the_calls_stream(monkeypatch, name):
    """(torch's current stream may have work waiting that still writes the memory that it would be handed.)"""
    import torch

    class Asked(Exception):
        pass

    def scratch(nbytes, stream, like):
        raise Asked(nbytes, stream, like)

    def empty(*a, **kw):
        raise AssertionError("scratch from the current stream")

    M, N, K = 16, 4096, 4096
    q, d, b = torch.zeros((M, K), dtype=torch.int8), torch.zeros((M, K // 32), dtype=torch.int16), torch.zeros((M, K // 16), dtype=torch.int16)
    w = torch.zeros(getattr(nvq, f"nvq_{name}_weight_bytes")(N, K), dtype=torch.uint8)
    y = torch.zeros((M, N))
    before = {"nvfp4": (w, 1.0, q, d), "q6_k": (w, q, d), "iq4_xs": (w, np.zeros(16, np.int8), q, d)}.get(name, (w, q, d, b))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(nvq, "_workspace", scratch)
    with pytest.raises(Asked) as e:
        getattr(nvq, f"nvq_gemm_{name}")(*before, y, stream=5)
    assert e.value.args[0] == nvq.nvq_gemm_workspace_bytes(getattr(nvq, f"NVQ_FMT_{name.upper()}"), M, N, K)
    assert e.value.args[1] == 5 and e.value.args[2] is y
