"""The rotation entries' argument checks and table, without a GPU: every refusal is decided before any HIP call."""
import ctypes

import numpy as np
import pytest

import gemm_q8_act_amd as nvq

P = 1 << 20  # an aligned address that no check may follow
NULL, SHAPE, RANGE, ALIGN = -1, -2, -3, -4


def three(*x):
    return (ctypes.c_int32 * len(x))(*x)


def rows(**kw):
    a = dict(type=0, out_type=0, q=P, q_st=5120, q_sh=128, k=P, k_st=1024, k_sh=128, T=4, Hq=40, Hkv=8, D=128, qw=P, kw=P, eps=1e-6, table=P, P=100,
             R=128, pairs=0, positions=P, axes=1, sections=None, qo=P, qo_st=5120, qo_sh=128, ko=P, ko_st=1024, ko_sh=128, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return nvq.lib().nvq_qk_norm_rope(*a.values())


def write(**kw):
    a = dict(fmt=0, type=0, out_type=0, q=P, q_st=5120, q_sh=128, k=P, k_st=1024, k_sh=128, v=P, v_st=1024, v_sh=128, T=4, Hq=40, Hkv=8, D=128, qw=P,
             kw=P, eps=1e-6, table=P, P=100, R=128, pairs=0, positions=P, axes=1, sections=None, slots=P, qo=P, qo_st=5120, qo_sh=128, kc=P, vc=P,
             kd=P, vd=P, n_pages=10, page=64, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return nvq.lib().nvq_rope_kv_write(*a.values())


BOTH = [(NULL, dict(table=None)), (NULL, dict(positions=None)), (NULL, dict(q=None)), (NULL, dict(qo=None)), (NULL, dict(axes=2)),
        (RANGE, dict(type=3)), (RANGE, dict(type=-1)), (RANGE, dict(out_type=3)), (RANGE, dict(pairs=2)), (RANGE, dict(pairs=-1)),
        (RANGE, dict(eps=-1.0)), (RANGE, dict(eps=float("nan"))), (RANGE, dict(eps=float("inf"))), (RANGE, dict(axes=0)),
        (RANGE, dict(axes=5, sections=three(1, 1, 1, 1, 60))), (RANGE, dict(sections=three(64))), (RANGE, dict(axes=2, sections=three(32, 31))),
        (RANGE, dict(axes=2, sections=three(-1, 65))), (RANGE, dict(axes=3, sections=three(32, 32, 32))),
        (RANGE, dict(axes=3, sections=three(1 << 30, 1 << 30, 64))), (SHAPE, dict(R=0)), (SHAPE, dict(R=2)), (SHAPE, dict(R=66)), (SHAPE, dict(R=132)),
        (SHAPE, dict(P=0)), (SHAPE, dict(P=1 << 31)), (SHAPE, dict(D=100)), (SHAPE, dict(D=288)), (SHAPE, dict(D=0)), (SHAPE, dict(Hq=0)),
        (SHAPE, dict(Hq=65537)), (SHAPE, dict(Hkv=0)), (SHAPE, dict(T=-1)), (SHAPE, dict(T=1 << 28)), (SHAPE, dict(q_st=-5120)), (SHAPE, dict(k_sh=1 << 41)),
        (SHAPE, dict(qo_st=5000)), (SHAPE, dict(qo_st=128, qo_sh=128)), (ALIGN, dict(q=P + 4)), (ALIGN, dict(k=P + 8)), (ALIGN, dict(qo=P + 2)),
        (ALIGN, dict(q_st=5121)), (ALIGN, dict(k_sh=130)), (ALIGN, dict(qo_sh=130)), (ALIGN, dict(out_type=1, qo_st=5124)), (ALIGN, dict(table=P + 4)),
        (ALIGN, dict(positions=P + 2)), (ALIGN, dict(qw=P + 4)), (ALIGN, dict(kw=P + 8))]


@pytest.mark.parametrize("want,kw", BOTH + [(NULL, dict(k=None)), (NULL, dict(ko=None)), (NULL, dict(q=None, qo=None, k=None, ko=None)),
                                            (ALIGN, dict(ko=P + 4)), (SHAPE, dict(ko_sh=64))])
def test_rows_refusals(want, kw):
    assert rows(**kw) == want
    assert "nvq_qk_norm_rope" in nvq.last_error()


@pytest.mark.parametrize("want,kw", BOTH + [
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(slots=None)), (NULL, dict(kc=None)), (NULL, dict(vc=None)), (NULL, dict(kd=None)),
    (RANGE, dict(fmt=3)), (RANGE, dict(fmt=1)), (SHAPE, dict(page=24)), (SHAPE, dict(n_pages=0)), (ALIGN, dict(slots=P + 4)), (ALIGN, dict(v=P + 8)),
    (ALIGN, dict(v_st=1026)), (ALIGN, dict(kc=P + 8))])
def test_write_refusals(want, kw):
    assert write(**kw) == want
    assert "nvq_rope_kv_write" in nvq.last_error()


def test_nothing_to_do_is_ok():
    none = dict(T=0, q=None, k=None, table=None, positions=None, qw=None, kw=None)
    assert rows(**none, qo=None, ko=None) == 0 and write(**none, v=None, slots=None, qo=None) == 0


def test_table():
    t = nvq.nvq_rope_table(40, 8, base=100.0)
    angle = np.arange(40)[:, None] * 100.0 ** (-np.arange(4) / 4.0)
    assert t.shape == (40, 8) and np.abs(t - np.concatenate([np.cos(angle), np.sin(angle)], 1)).max() <= 2.0 ** -24
    for a, kw in (((0, 8), {}), ((10, 6), {}), ((10, 0), {}), ((10, 260), {}), ((-1, 8), {}), ((10, 8), dict(inv_freq=[1.0, 2.0])), ((10, 8), dict(base=0.0)),
                  ((10, -4), {})):
        with pytest.raises((ValueError, nvq.NvqError)):
            nvq.nvq_rope_table(*a, **kw)
    f = ctypes.c_double * 4
    assert nvq.lib().nvq_rope_table(None, 3, 8, P) == NULL and nvq.lib().nvq_rope_table(f(), 3, 8, None) == NULL


def test_binding_refusals():
    import torch

    x, s = torch.zeros((3, 1, 32)), torch.zeros(3, dtype=torch.int64)
    t, p = torch.zeros((10, 16)), torch.zeros(3, dtype=torch.int32)
    c, d = torch.zeros((2, 1, 16, 32), dtype=torch.int8), torch.zeros((2, 1, 16, 1), dtype=torch.float16)
    for a, kw in (((x, x, t, p, x, None), {}), ((None, None, t, p, None, None), {}), ((x, None, t, p, None, None), {}), ((x.double(), x, t, p, x, x), {}),
                  ((x, x.half(), t, p, x, x), {}), ((x, x, t.double(), p, x, x), {}), ((x, x, t[0], p, x, x), {}), ((x, x, t, p.long(), x, x), {}),
                  ((x, x, t, p[:2], x, x), {}), ((x, x, t, p, x[:2], x), {}), ((x, x, t, p, x, x.half()), {}), ((x, x, t, p, x, x), dict(sections=[4, 4])),
                  ((x, x, t, p.expand(2, 3).contiguous(), x, x), {}), ((x, x, t, p, x, x), dict(q_weight=torch.zeros(31))),
                  ((x, x, t, p, x, x), dict(k_weight=torch.zeros(32).half())), ((x, x[:, :, ::2], t, p, x, x), {}), ((x[0], x, t, p, x, x), {})):
        with pytest.raises(ValueError):
            nvq.nvq_qk_norm_rope(*a, **kw)
    for a in ((x, x, x, t, p, s, None, c, c, d, d), (None, x, x, t, p, s, x, c, c, d, d), (x, x, x, t, p, s.int(), x, c, c, d, d),
              (x, x, x.half(), t, p, s, x, c, c, d, d), (x, x, x, t, p, s, x, c, c, None, d), (x, x, x, t, p[:1], s, x, c, c, d, d),
              (x, x, x, None, p, s, x, c, c, d, d), (x, x, x, t, None, s, x, c, c, d, d), (x.half(), x, x, t, p, s, x, c, c, d, d)):
        with pytest.raises(ValueError):
            nvq.nvq_rope_kv_write(*a)
