"""The cache and attention entries' argument checks, without a GPU: every refusal is decided
before any HIP call."""
import ctypes

import pytest

import gemm_q8_act_amd as nvq

P = 1 << 20  # an aligned address that no check may follow


def kv(name="nvq_kv_write", **kw):
    a = dict(fmt=0, type=0, k=P, k_st=1024, k_sh=128, v=P, v_st=1024, v_sh=128, slots=P, T=4, H=8, D=128, kc=P, vc=P, kd=P, vd=P,
             n_pages=10, page=64, stream=None)
    a.update(kw)
    return getattr(nvq.lib(), name)(*a.values())


def decode(**kw):
    a = dict(fmt=0, type=0, q=P, q_sb=5120, q_sh=128, B=2, Hq=40, Hkv=8, D=128, kc=P, vc=P, kd=P, vd=P, n_pages=10, page=64, table=P,
             max_pages=100, lengths=P, scale=0.1, out=P, ws=P, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return nvq.lib().nvq_attn_decode(*a.values())


def prompt(strides=(5120, 128, 1024, 128, 1024, 128, 5120, 128), **kw):
    a = dict(type=2, q=P, k=P, v=P, out=P, strides=(ctypes.c_int64 * 8)(*strides) if strides else None, cu_q=P, cu_k=P, B=2, Tq=10, Tk=10,
             Hq=40, Hkv=8, D=128, scale=0.1, causal=1, stream=None)
    a.update(kw)
    return nvq.lib().nvq_attn_prompt(*a.values())


NULL, SHAPE, RANGE, ALIGN, WORKSPACE = -1, -2, -3, -4, -7


@pytest.mark.parametrize("name", ["nvq_kv_write", "nvq_kv_read"])
@pytest.mark.parametrize("want,kw", [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(slots=None)), (NULL, dict(kc=None)), (NULL, dict(vc=None)), (NULL, dict(kd=None)),
    (NULL, dict(vd=None)), (RANGE, dict(fmt=3)), (RANGE, dict(fmt=-1)), (RANGE, dict(type=3)), (RANGE, dict(type=-1)), (RANGE, dict(fmt=1)),
    (SHAPE, dict(D=0)), (SHAPE, dict(D=48)), (SHAPE, dict(D=288)), (SHAPE, dict(H=0)), (SHAPE, dict(H=65537)), (SHAPE, dict(T=-1)),
    (SHAPE, dict(T=1 << 33)), (SHAPE, dict(page=8)), (SHAPE, dict(page=48)), (SHAPE, dict(page=1 << 17)), (SHAPE, dict(n_pages=0)),
    (SHAPE, dict(n_pages=1 << 31)), (SHAPE, dict(k_st=-1024)), (ALIGN, dict(k=P + 4)), (ALIGN, dict(v=P + 8)), (ALIGN, dict(k_st=1026)),
    (ALIGN, dict(v_sh=130)), (ALIGN, dict(kc=P + 8)), (ALIGN, dict(vd=P + 2)), (ALIGN, dict(slots=P + 4)), (ALIGN, dict(type=1, k_st=1028))])
def test_cache_refusals(name, want, kw):
    assert kv(name, **kw) == want
    assert name in nvq.last_error()


@pytest.mark.parametrize("kw", [dict(k_st=64, k_sh=64), dict(v_st=0), dict(v_sh=0), dict(k_sh=64), dict(k_st=128, k_sh=128), dict(v_st=960)])
def test_read_refuses_rows_that_overlap(kw):
    assert kv("nvq_kv_read", **kw) == SHAPE
    assert "overlap" in nvq.last_error()


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(q=None)), (NULL, dict(table=None)), (NULL, dict(lengths=None)), (NULL, dict(out=None)), (NULL, dict(kc=None)), (NULL, dict(kd=None)),
    (RANGE, dict(fmt=9)), (RANGE, dict(type=5)), (RANGE, dict(fmt=2)), (SHAPE, dict(D=100)), (SHAPE, dict(Hq=41)), (SHAPE, dict(Hq=0)),
    (SHAPE, dict(Hkv=0)), (SHAPE, dict(B=-1)), (SHAPE, dict(max_pages=0)), (SHAPE, dict(max_pages=1 << 30)), (SHAPE, dict(max_pages=1 << 23)), (SHAPE, dict(B=1 << 20, max_pages=1 << 6)),
    (SHAPE, dict(page=24)), (ALIGN, dict(q=P + 8)), (ALIGN, dict(q_sb=5122)), (ALIGN, dict(out=P + 8)), (ALIGN, dict(table=P + 2)),
    (ALIGN, dict(lengths=P + 1)), (ALIGN, dict(ws=P + 8)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=100))])
def test_decode_refusals(want, kw):
    assert decode(**kw) == want
    assert "nvq_attn_decode" in nvq.last_error()


@pytest.mark.parametrize("want,kw", [
    (NULL, dict(q=None)), (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(out=None)), (NULL, dict(cu_q=None)), (NULL, dict(cu_k=None)),
    (NULL, dict(strides=None)), (RANGE, dict(type=0)), (RANGE, dict(type=3)), (SHAPE, dict(D=33)), (SHAPE, dict(D=512)), (SHAPE, dict(Hq=39)),
    (SHAPE, dict(Hkv=0)), (SHAPE, dict(B=-1)), (SHAPE, dict(Tq=-1)), (SHAPE, dict(Tk=1 << 30)), (ALIGN, dict(q=P + 2)), (ALIGN, dict(out=P + 8)),
    (ALIGN, dict(cu_q=P + 2)), (ALIGN, dict(strides=(5124, 128, 1024, 128, 1024, 128, 5120, 128))),
    (SHAPE, dict(strides=(5120, 128, 1024, 128, 1024, 128, 0, 128))), (SHAPE, dict(strides=(5120, 128, 1024, 128, 1024, 128, 5120, 64))),
    (SHAPE, dict(strides=(5120, -128, 1024, 128, 1024, 128, 5120, 128))), (SHAPE, dict(strides=(5120, 128, 1 << 24, 128, 1024, 128, 5120, 128))),
    (SHAPE, dict(strides=(5120, 128, 1024, 128, 1 << 25, 128, 5120, 128)))])
def test_prompt_refusals(want, kw):
    assert prompt(**kw) == want
    assert "nvq_attn_prompt" in nvq.last_error()


def test_nothing_to_do_is_ok():
    assert kv(T=0, k=None, v=None, slots=None) == 0 and decode(B=0, q=None, ws=None) == 0
    assert prompt(B=0, cu_q=None) == 0 and prompt(Tq=0, q=None) == 0


def test_decode_workspace_sizes():
    ws = nvq.nvq_attn_decode_workspace_bytes
    assert ws(1, 40, 8, 128, 2, 64) == 0                 # at most 128 keys: one part to a sequence
    one = 8 * 64 * 16 + 2 * 16 * 4                       # a part: 128 channels and 2 statistics of 16 heads
    assert ws(1, 40, 8, 128, 4, 64) == 2 * 8 * one       # 256 keys: two parts
    assert ws(4, 40, 8, 128, 4, 64) == 4 * 2 * 8 * one
    assert ws(1, 34, 2, 128, 4, 64) == 2 * 2 * 2 * one   # 17 heads to a key head: two tiles of heads
    assert ws(1, 41, 8, 128, 8, 64) == 0 and ws(1, 40, 8, 100, 8, 64) == 0 and ws(0, 40, 8, 128, 8, 64) == 0


def test_binding_refusals():
    import torch

    c = torch.zeros((2, 1, 16, 32), dtype=torch.int8)
    d = torch.zeros((2, 1, 16, 1), dtype=torch.float16)
    x = torch.zeros((3, 1, 32))
    s = torch.zeros(3, dtype=torch.int64)
    for a in ((x.double(), x, s, c, c, d, d), (x, x.half(), s, c, c, d, d), (x, x, s.int(), c, c, d, d), (x, x, s, c, c, None, d),
              (x, x, s, c.half(), c, None, None), (x, x, s, c.half(), c.half(), d, d), (x, x[:2], s, c, c, d, d),
              (x.transpose(0, 2).reshape(1, 3, 32).transpose(0, 1)[:, :, ::2], x, s, c, c, d, d), (x, x, s, c[0], c[0], d, d)):
        with pytest.raises(ValueError):
            nvq.nvq_kv_write(*a)
    q = torch.zeros((2, 1, 32))
    t, n = torch.zeros((2, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for a in ((q, c, c, t.long(), n, q, d, d), (q, c, c, t, n[:1], q, d, d), (q, c, c, t, n, q.half(), d, d), (q[:, :, :16], c, c, t, n, q, d, d),
              (q, c, c, t[:1], n, q, d, d)):
        with pytest.raises(ValueError):
            nvq.nvq_attn_decode(*a)
    h = torch.zeros((4, 2, 32), dtype=torch.float16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for a in ((h, h, h.bfloat16(), cu, cu, h), (h, h, h[:2], cu, cu, h), (h, h, h, cu, cu.long(), h), (h, h, h, cu[:0], cu, h), (h, h, h, cu, cu, h[:3]),
              (h, h, h, cu, torch.zeros(3, dtype=torch.int32), h)):
        with pytest.raises(ValueError):
            nvq.nvq_attn_prompt(*a)
