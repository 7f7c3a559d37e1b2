"""The attention layer example's own refusals, without a GPU: tokens past its cache would be indexed past its page
table on the device."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def example(monkeypatch):
    monkeypatch.syspath_prepend(os.path.join(ROOT, "examples"))
    import attention_layer

    return attention_layer


def test_tokens_past_the_cache_are_refused_before_anything_runs(example):
    import torch

    layer = example.AttentionLayer.__new__(example.AttentionLayer)  # (the weights want a GPU; a refusal needs none)
    layer.n, layer.max_tokens = 30, 32
    layer._product = layer._slots = lambda *a: pytest.fail("the call went on")
    layer.w_qkv = layer.s_qkv = layer.rows = None
    for x in (torch.zeros((3, 8)), torch.zeros((0, 8))):
        with pytest.raises(ValueError, match="cache"):
            layer.prompt(x)
    layer.n = 32
    with pytest.raises(ValueError, match="cache"):
        layer.step(torch.zeros((1, 8)))


@pytest.mark.parametrize("args", [["--prompt", "1"], ["--steps", "0"]])
def test_arguments_that_leave_a_piece_empty_are_refused(example, monkeypatch, args):
    monkeypatch.setattr(sys, "argv", ["attention_layer.py", *args])
    monkeypatch.setattr(example, "AttentionLayer", lambda *a, **kw: pytest.fail("went on"))
    with pytest.raises(SystemExit):
        example.main()
