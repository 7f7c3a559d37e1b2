"""Shared helpers of the cache and attention tests: seeded inputs, the operators in float64
(numpy, one sequence and head at a time), and the bounds that their formulas give.

Bounds.  With exact p_j = exp(s_j - max), A = sum p_j |v_j| / sum p_j (per output channel) and
S = max_j scale * sum_d |q_d k_jd|, an error e in every score changes a result by at most 2 e A, and a
relative error f in every probability or product by at most 2 f A.
  float32 accumulation of a score: e <= (D + 8) 2^-24 S (D products, the scale, base 2 and the
  difference from the maximum, whose size is at most 2 S), two-term operands 2^-21 S;
  sums over L keys in float32: f <= (L / 8 + 64) 2^-24 (at least 16 partial sums run side by side in
  decode's four wavefronts, 2 in the prompt's), exponential and two-term operands 2^-20;
  probabilities rounded to 16 bits: f <= the type's half unit; the result rounded to its type.
"""
from __future__ import annotations

import numpy as np

import gemm_q8_act_amd as nvq
from gpu_cases import torch_dev

HALF_UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SMALLEST = {"f32": 1e-37, "f16": 2.0 ** -24, "bf16": 1e-37}


def torch_type(name):
    torch = torch_dev()
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def rounded(x: np.ndarray, type_: str) -> np.ndarray:
    """float32 values as the type holds them, as float32."""
    torch = torch_dev()
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch_type(type_)).float().numpy()


def place_of(D: int) -> np.ndarray:
    """The byte of a quantised row that holds each channel (from the header's rule, channel by channel)."""
    nb = D // 32
    at = np.empty(D, np.int64)
    for b in range(nb):
        for n in range(16):
            for e in range(2):
                at[32 * b + 2 * n + e] = 2 * nb * n + 2 * b + e
    return at


def attention(q, k, v, scale, seen):
    """One head in float64: q [m, D], k, v [n, D], seen bool [m, n] -> (out, A, S)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    m, D = q.shape
    out, A, S = np.zeros((m, v.shape[1])), np.zeros((m, v.shape[1])), np.zeros((m, 1))
    for i in range(m):
        j = np.flatnonzero(seen[i])
        if not len(j):
            continue
        s = scale * (k[j] @ q[i])
        p = np.exp(s - s.max())
        out[i] = p @ v[j] / p.sum()
        A[i] = p @ np.abs(v[j]) / p.sum()
        S[i] = abs(scale) * (np.abs(k[j]) @ np.abs(q[i])).max()
    return out, A, S


def bound(out, A, S, D, L, out_type, p_unit, streams):
    e = ((D + 8) * 2.0 ** -24 + 2.0 ** -21) * S
    f = (L / streams + 64) * 2.0 ** -24 + 2.0 ** -20 + p_unit
    return 2 * (e + f) * A * 1.0001 + HALF_UNIT[out_type] * (np.abs(out) + 2 * (e + f) * A) + SMALLEST[out_type]


def check(got, want, limit, what):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got - want)
    worst = float((err / limit).max()) if err.size else 0.0
    assert (err <= limit).all(), f"{what}: {int((err > limit).sum())} of {err.size} outside the bound (worst {worst:.3g})"
    if np.abs(want).max(initial=0) > 0:
        assert np.abs(got).max() > 0, f"{what}: output all zero"
    return worst


class Paged:
    """Sequences of rows k, v [n, Hkv, D] written into a shuffled paged cache by nvq_kv_write; every row that is
    not written holds NaN (NaN scales over codes of 127 in a Q8_0 cache).  rows[i]: (k, v) as the cache holds them."""

    def __init__(self, fmt, seqs, Hkv, D, page, seed, spare=2, write_type="f32"):
        torch = torch_dev()
        r = np.random.Generator(np.random.PCG64(seed))
        need = [-(-len(k) // page) for k, _ in seqs]
        self.n_pages = max(1, sum(need) + spare)
        ids = r.permutation(self.n_pages)
        self.max_pages = max(1, max(need))
        table = np.full((len(seqs), self.max_pages), -7, np.int32)  # entries behind the end are never read
        shape = (self.n_pages, Hkv, page, D)
        if fmt == "q8_0":
            self.kc, self.vc = (torch.full(shape, 127, dtype=torch.int8, device="cuda") for _ in "kv")
            self.kd, self.vd = (torch.full((*shape[:3], D // 32), float("nan"), dtype=torch.float16, device="cuda") for _ in "kv")
        else:
            self.kc, self.vc = (torch.full(shape, float("nan"), dtype=torch_type(fmt), device="cuda") for _ in "kv")
            self.kd = self.vd = None
        at, slots = 0, []
        for i, n in enumerate(need):
            table[i, :n] = ids[at:at + n]
            at += n
            j = np.arange(len(seqs[i][0]))
            slots.append(table[i, j // page].astype(np.int64) * page + j % page)
        slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
        self.slots = torch.from_numpy(slots).cuda()
        self.table = torch.from_numpy(table).cuda()
        self.lengths = torch.tensor([len(k) for k, _ in seqs], dtype=torch.int32, device="cuda")
        k, v = (torch.from_numpy(np.ascontiguousarray(np.concatenate([s[i] for s in seqs]), np.float32)).to(torch_type(write_type)).cuda()
                for i in (0, 1))
        nvq.nvq_kv_write(k, v, self.slots, self.kc, self.vc, self.kd, self.vd)
        kb, vb = (torch.empty(x.shape, dtype=torch.float32, device="cuda") for x in (k, v))
        nvq.nvq_kv_read(self.kc, self.vc, self.slots, kb, vb, self.kd, self.vd)
        kb, vb = kb.cpu().numpy(), vb.cpu().numpy()
        self.rows, at = [], 0
        for s in seqs:
            self.rows.append((kb[at:at + len(s[0])], vb[at:at + len(s[0])]))
            at += len(s[0])

    def decode(self, q, out=None, **kw):
        torch = torch_dev()
        if out is None:
            out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        nvq.nvq_attn_decode(q, self.kc, self.vc, self.table, self.lengths, out, self.kd, self.vd, **kw)
        return out
