"""Shared helpers of the chunk and window attention tests: who sees what, and what nobody sees made unusable."""
from __future__ import annotations

import numpy as np

from attn_cases import Paged, attention, bound, check
from gpu_cases import host, torch_dev

U16 = 2.0 ** -11  # binary16's half unit


def seen_of(m, n, window, sinks):
    """[m, n]: what the m last of n tokens see (m may pass n)."""
    p = np.arange(m)[:, None] + (n - m)
    j = np.arange(n)[None]
    seen = j <= p
    return seen & ((j > p - window) | (j < sinks)) if window else seen


class Hidden(Paged):
    """A paged cache whose rows that no query sees are NaN (those of pages with none of them seen lose their table entry too):
    seen[i] bool [queries, keys] of sequence i."""

    def __init__(self, fmt, seqs, seen, Hkv, D, page, seed, **kw):
        super().__init__(fmt, seqs, Hkv, D, page, seed, **kw)
        table = host(self.table).copy()
        for i, s in enumerate(seen):
            n = s.shape[1]
            any_ = s.any(0)
            for x in range(-(-n // page)):
                rows = any_[x * page:(x + 1) * page]
                at = int(table[i, x])
                for off in np.flatnonzero(~rows):
                    for c, d in ((self.kc, self.kd), (self.vc, self.vd)):
                        if d is None:
                            c[at, :, off] = float("nan")
                        else:
                            c[at, :, off], d[at, :, off] = 127, float("nan")
                if not rows.any():
                    table[i, x] = (-7, 1 << 30, self.n_pages)[x % 3]
        torch = torch_dev()
        self.table = torch.from_numpy(table).cuda()


def limits(want, A, S, D, L, fmt, type_, p_unit):
    """Bounds of attn_cases.bound with what the operands' rounding over Q8_0 adds in the chunk kernel: key and value elements to
    binary16's half unit, which is at most U16 S in a score and U16 A in a result."""
    limit = bound(want, A, S, D, L, type_, p_unit, 2)
    return limit + (2 * U16 * S + U16) * A * 1.01 if fmt == "q8_0" else limit


def compare(got, q, rows, seen, scale, fmt, type_, p_unit, what, some=None):
    """got, q [m, Hq, D] of one sequence against float64."""
    m, Hq, D = q.shape
    k, v = rows
    worst = 0.0
    pick = np.arange(m) if some is None or m <= some else np.unique(np.linspace(0, m - 1, some).astype(int))
    for h in range(Hq):
        j = h * k.shape[1] // Hq
        want, A, S = attention(q[pick, h], k[:, j], v[:, j], scale, seen[pick])
        limit = bound(want, A, S, D, len(k), type_, 0.0, 8) if p_unit is None else limits(want, A, S, D, len(k), fmt, type_, p_unit)
        worst = max(worst, check(got[pick, h], want, limit, f"{what} head {h}"))
        assert (got[pick, h][~seen[pick].any(1)] == 0).all()
    return worst
