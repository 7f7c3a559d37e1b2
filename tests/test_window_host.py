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
    q8, f16 = nvq.NVQ_KV_Q8_0, nvq.NVQ_KV_F16
    assert ws(f16, 1, 16, 40, 8, 128, 1, 64) == 0 and ws(f16, 0, 16, 40, 8, 128, 8, 64) == 0 and ws(f16, 1, 16, 41, 8, 128, 8, 64) == 0
    assert ws(f16, 1, 1, 40, 8, 128, 1024, 64) > 0 and ws(f16, 1, 1, 40, 8, 128, 1024, 64, -1) == 0 and ws(9, 1, 1, 40, 8, 128, 1024, 64) == 0
    # partial results: no more than the parts of 2048 workgroups, 128 rows of float32 each
    for B, T, pages, w, s in ((b, t, p, w, s) for b in (1, 3, 64) for t in (1, 7, 26, 600) for p in (2, 9, 300) for w in (0, 1, 100, 5000) for s in (0, 4, 300)):
        n = ws(f16, B, T, 40, 8, 128, pages, 64, w, s)
        assert 0 <= n <= 2048 * (128 * 128 * 4 + 1024) and ws(q8, B, T, 40, 8, 128, pages, 64, w, s) >= n
    # Q8_0 turned into binary16 first: keys and values of 64-key tiles, and 16 bytes a tile, from 1024 rows a sequence on
    one = 64 * 128 * 4 + 16
    for B, T, pages, want in ((1, 204, 300, 0), (1, 205, 300, 300), (2, 409, 300, 0), (2, 410, 300, 600), (1, 4096, 4096, 4096), (1, 4096, 4097, 0), (9000, 9000 * 205, 1, 0)):
        more = ws(q8, B, T, 40, 8, 128, pages, 64) - ws(f16, B, T, 40, 8, 128, pages, 64)
        assert more == 8 * want * one, (B, T, pages)


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
