"""The chunk and window attention entries' argument checks and workspace sizes, without a GPU."""
import ctypes

import pytest

import gemm_q8_act_amd as nvq

P = 1 << 20  # an aligned address that no check may follow
NULL, SHAPE, RANGE, ALIGN, WORKSPACE = -1, -2, -3, -4, -7


def window(**kw):
    a = dict(fmt=0, type=0, q=P, q_sb=5120, q_sh=128, B=2, Hq=40, Hkv=8, D=128, kc=P, vc=P, kd=P, vd=P, n_pages=10, page=64, table=P,
             max_pages=100, lengths=P, scale=0.1, window=1000, sinks=4, out=P, ws=P, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return nvq.lib().nvq_attn_decode_window(*a.values())


def chunk(strides=(5120, 128, 5120, 128), **kw):
    a = dict(fmt=0, type=2, q=P, strides=(ctypes.c_int64 * 4)(*strides) if strides else None, B=2, Tq=10, Hq=40, Hkv=8, D=128, kc=P, vc=P, kd=P, vd=P,
             n_pages=10, page=64, table=P, max_pages=100, cu_q=P, lengths=P, scale=0.1, window=0, sinks=0, out=P, ws=P, ws_bytes=1 << 40, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return nvq.lib().nvq_attn_chunk(*a.values())


CACHE = [(NULL, dict(q=None)), (NULL, dict(table=None)), (NULL, dict(lengths=None)), (NULL, dict(out=None)), (NULL, dict(kc=None)), (NULL, dict(vd=None)),
         (RANGE, dict(fmt=9)), (RANGE, dict(fmt=-1)), (RANGE, dict(type=5)), (RANGE, dict(fmt=2)), (RANGE, dict(window=-1)), (RANGE, dict(sinks=-1)),
         (SHAPE, dict(D=100)), (SHAPE, dict(D=0)), (SHAPE, dict(D=288)), (SHAPE, dict(Hq=41)), (SHAPE, dict(Hq=0)), (SHAPE, dict(Hkv=0)), (SHAPE, dict(B=-1)),
         (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=1 << 24)), (SHAPE, dict(page=24)), (SHAPE, dict(n_pages=0)), (ALIGN, dict(q=P + 8)),
         (ALIGN, dict(out=P + 8)), (ALIGN, dict(table=P + 2)), (ALIGN, dict(lengths=P + 1)), (ALIGN, dict(kc=P + 8)), (ALIGN, dict(ws=P + 8)),
         (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100))]


@pytest.mark.parametrize("want,kw", CACHE + [(ALIGN, dict(q_sb=5122)), (SHAPE, dict(B=1 << 20, max_pages=1 << 6))])
def test_window_refusals(want, kw):
    assert window(**kw) == want
    assert "nvq_attn_decode_window" in nvq.last_error()


@pytest.mark.parametrize("want,kw", CACHE + [
    (NULL, dict(cu_q=None)), (NULL, dict(strides=None)), (RANGE, dict(type=0)), (RANGE, dict(fmt=1, kd=None, vd=None)), (SHAPE, dict(Tq=-1)),
    (SHAPE, dict(Tq=1 << 30)), (SHAPE, dict(Tq=1 << 29)), (SHAPE, dict(B=1 << 22, max_pages=1)), (SHAPE, dict(B=1 << 20, max_pages=1 << 12)),
    (ALIGN, dict(cu_q=P + 2)), (ALIGN, dict(strides=(5124, 128, 5120, 128))), (ALIGN, dict(strides=(5120, 132, 5120, 128))),
    (SHAPE, dict(strides=(5120, 128, 0, 128))), (SHAPE, dict(strides=(5120, 128, 5120, 64))), (SHAPE, dict(strides=(-5120, 128, 5120, 128)))])
def test_chunk_refusals(want, kw):
    assert chunk(**kw) == want
    assert "nvq_attn_chunk" in nvq.last_error()


def test_nothing_to_do_is_ok():
    assert window(B=0, q=None, ws=None) == 0 and chunk(B=0, q=None, ws=None) == 0 and chunk(Tq=0, q=None, cu_q=None, ws=None) == 0


def test_workspaces():
    ws = nvq.nvq_attn_chunk_workspace_bytes
    assert ws(1, 16, 40, 8, 128, 1, 64) == 0 and ws(0, 16, 40, 8, 128, 8, 64) == 0 and ws(1, 16, 41, 8, 128, 8, 64) == 0
    assert ws(1, 1, 40, 8, 128, 1024, 64) > 0 and ws(1, 1, 40, 8, 128, 1024, 64, -1) == 0
    # what the header promises: the bytes of more are enough for fewer, and those of no window for any
    sizes = [(B, T, pages, w, s) for B in (1, 3, 64) for T in (1, 7, 26, 600) for pages in (2, 9, 300) for w in (0, 1, 100, 5000) for s in (0, 4, 300)]
    of = {x: ws(x[0], x[1], 40, 8, 128, x[2], 64, x[3], x[4]) for x in sizes}
    for (B, T, pages, w, s), n in of.items():
        assert n <= of[(64, 600, 300, 0, 0)] and n <= of[(B, T, pages, 0, 0)]
        for x in ((3, T, pages, w, s), (B, 600, pages, w, s), (B, T, 300, w, s)):
            if B <= x[0]:
                assert n <= of[x], ((B, T, pages, w, s), x)
    assert max(of.values()) < 140 << 20


def test_binding_refusals():
    import torch

    c, d = torch.zeros((2, 1, 16, 32), dtype=torch.int8), torch.zeros((2, 1, 16, 1), dtype=torch.float16)
    q = torch.zeros((4, 2, 32), dtype=torch.float16)
    t, n, cu = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    for a in ((q, c, c, t.long(), cu, n, q, d, d), (q, c, c, t, cu[:1], n, q, d, d), (q, c, c, t, cu, n[:0], q, d, d), (q, c, c, t, cu, n, q.float(), d, d),
              (q[:, :, :16], c, c, t, cu, n, q, d, d), (q, c, c, t[0], cu, n, q, d, d), (q, c, c, t, cu.long(), n, q, d, d), (q, c, c, t, cu, n, q[:3], d, d),
              (q, c, c, t, cu, n, q, None, d), (q, c, c, t, cu, n, None, d, d), (None, c, c, t, cu, n, q, d, d), (q, c, c, None, cu, n, q, d, d)):
        with pytest.raises(ValueError):
            nvq.nvq_attn_chunk(*a)
    x = torch.zeros((1, 2, 32))
    for a in ((x, c, c, t.long(), n, x, d, d), (x, c, c, t, n[:0], x, d, d), (x, c, c, t, n, x.half(), d, d)):
        with pytest.raises(ValueError):
            nvq.nvq_attn_decode_window(*a, window=3)
