"""The cache and attention entries' binding, without a GPU: its first call, from one thread and from several."""
import threading

import pytest

import gemm_q8_act_amd as nvq


def _refused():
    """A call that gets past the library and is refused for its arguments."""
    import torch

    x = torch.zeros((3, 1, 32))
    c, d = torch.zeros((2, 1, 16, 32), dtype=torch.int8), torch.zeros((2, 1, 16, 1), dtype=torch.float16)
    nvq.nvq_kv_write(x.double(), x, torch.zeros(3, dtype=torch.int64), c, c, d, d)


@pytest.fixture
def unloaded(monkeypatch):
    real = nvq.lib()
    monkeypatch.setattr(nvq, "_lib", None)
    monkeypatch.setattr(nvq, "_torch", None)
    return real


def test_a_library_that_cannot_be_loaded_is_named_every_time(unloaded, monkeypatch):
    def missing():
        raise ImportError("libnvq.so not built")

    monkeypatch.setattr(nvq, "lib", missing)
    for _ in range(2):
        with pytest.raises(ImportError, match="not built"):
            _refused()


def test_first_calls_of_several_threads(unloaded, monkeypatch):
    """A second thread's first call while the library is loading waits for it as the first one's does."""
    inside, go = threading.Event(), threading.Event()

    def slow():
        inside.set()
        assert go.wait(30)
        nvq._lib = unloaded
        return unloaded

    monkeypatch.setattr(nvq, "lib", slow)
    errors = []

    def call():
        try:
            _refused()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=call) for _ in range(4)]
    threads[0].start()
    assert inside.wait(30)
    for t in threads[1:]:
        t.start()
    threads[1].join(1.0)  # what would not wait for the library has ended by then
    go.set()
    for t in threads:
        t.join(30)
    assert len(errors) == 4 and all(type(e) is ValueError for e in errors), errors


@pytest.mark.parametrize("stream,want", [(None, 77), (77, 77), (5, 5), (0, 0)])
def test_scratch_comes_from_the_stream_that_uses_it(monkeypatch, stream, want):
    """torch's allocator hands memory out in the order of the stream that is current when it is asked: scratch of a call
    on another stream has to be asked for there, or work still waiting on the current one writes over it."""
    import contextlib
    import types

    import torch

    current, asked = [77], []

    @contextlib.contextmanager
    def on(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def empty(n, dtype, device):
        asked.append((n, current[-1], device))
        return types.SimpleNamespace(record_stream=lambda s: None)

    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=current[-1]))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda d=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: types.SimpleNamespace(cuda_stream=p))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(nvq, "_torch", torch)
    assert nvq._workspace(4096, stream, types.SimpleNamespace(device="cuda:0")) is not None
    assert asked == [(4096, want, "cuda:0")] and current == [77]
    assert nvq._workspace(0, stream, None) is None


def test_calls_of_more_threads_than_a_launch_takes_are_refused():
    """A launch takes fewer than 2^32 threads (256 to a workgroup, 512 to one that joins parts); a longer one is cut short
    without an error, so the entries refuse what would need it."""
    from test_attention_host import ALIGN, NULL, SHAPE, P, decode, prompt

    ws = nvq.nvq_attn_decode_workspace_bytes
    # 128 keys at most: no parts to join
    assert decode(B=1 << 21, max_pages=2, q=None) == SHAPE and decode(B=(1 << 21) - 1, max_pages=2, q=None) == NULL
    assert decode(B=1 << 20, Hq=8 * 17, max_pages=2, q=None) == SHAPE and decode(B=(1 << 20) - 1, Hq=8 * 17, max_pages=2, q=None) == NULL
    # 256 keys: parts
    assert decode(B=1 << 20, max_pages=4, q=None) == SHAPE and ws(1 << 20, 40, 8, 128, 4, 64) == 0
    assert decode(B=(1 << 20) - 1, max_pages=4, q=None) == NULL and ws((1 << 20) - 1, 40, 8, 128, 4, 64) > 0
    assert prompt(B=1 << 19, Hq=32, cu_q=P + 2) == SHAPE and "query tiles" in nvq.last_error()
    assert prompt(B=1, Tq=1 << 29, Hq=8, cu_q=P + 2) == SHAPE
    assert prompt(B=(1 << 19) - 1, Hq=32, cu_q=P + 2) == ALIGN


def test_a_width_of_zero_is_the_librarys_refusal(monkeypatch):
    """(Not a division by zero in the default scale.)"""
    import torch

    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # CPU tensors' own
    q, c, d = torch.zeros((1, 2, 0)), torch.zeros((2, 1, 16, 0), dtype=torch.int8), torch.zeros((2, 1, 16, 0), dtype=torch.float16)
    t, n = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    h, cu = torch.zeros((4, 2, 0), dtype=torch.float16), torch.tensor([0, 4], dtype=torch.int32)
    for call in (lambda: nvq.nvq_attn_decode(q, c, c, t, n, q, d, d, stream=0), lambda: nvq.nvq_attn_prompt(h, h, h, cu, cu, h, stream=0)):
        with pytest.raises(nvq.NvqError) as e:
            call()
        assert e.value.status == -2
