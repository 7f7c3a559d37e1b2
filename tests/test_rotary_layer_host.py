"""The rotary layer example's own refusals, without a GPU."""
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

    layer = example.RotaryLayer.__new__(example.RotaryLayer)  # (the weights want a GPU; a refusal needs none)
    layer.n, layer.max_tokens = 30, 32
    layer._product = layer._slots = layer._append = lambda *a: pytest.fail("the call went on")
    layer.w_qkv = layer.s_qkv = layer.rows = None
    for x in (torch.zeros((3, 8)), torch.zeros((0, 8))):
        with pytest.raises(ValueError, match="cache"):
            layer.prompt(x)
    layer.n = 32
    with pytest.raises(ValueError, match="cache"):
        layer.step(torch.zeros((1, 8)))


@pytest.mark.parametrize("args", [["--window", "16"], ["--sinks", "2"], ["--rotary", "--window", "-1"], ["--rotary", "--sinks", "-1"]])
def test_window_arguments_that_fit_no_layer_are_refused(example, monkeypatch, args):
    monkeypatch.setattr(sys, "argv", ["attention_layer.py", *args])
    for kind in ("AttentionLayer", "RotaryLayer"):
        monkeypatch.setattr(example, kind, lambda *a, **kw: pytest.fail("went on"))
    with pytest.raises(SystemExit):
        example.main()
