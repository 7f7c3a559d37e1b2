"""Decode attention over a Q8_0 cache for every number of columns that a query head can take (by the heads to a key
head and the width): with few heads the idle columns carry the value scales of further blocks."""
import numpy as np
import pytest

from attn_cases import Paged, attention, bound, check
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G", [1, 4, 5, 8, 16, 17])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_heads_and_widths(D, G):
    """A sequence of one part, one of several with at least three tiles to a wavefront (32 key heads, so that parts are
    long), an empty one; all query heads of the first, a middle and the last key head."""
    torch = torch_dev()
    lens, Hkv, page = [77, 4400, 0], 32, 16
    Hq = G * Hkv
    say(f"decode q8_0 columns D={D} G={G}")
    r = np.random.Generator(np.random.PCG64(1000 * D + G))
    # widths that differ from block to block: a scale of the wrong block shows
    width = (10.0 ** np.linspace(-1, 1, D // 32)).repeat(32).astype(np.float32)
    seqs = [(r.standard_normal((n, Hkv, D)).astype(np.float32), r.standard_normal((n, Hkv, D)).astype(np.float32) * width) for n in lens]
    c = Paged("q8_0", seqs, Hkv, D, page, D + G)
    q = r.standard_normal((len(lens), Hq, D)).astype(np.float32)
    got = host(c.decode(torch.from_numpy(q).cuda()))
    worst = 0.0
    for i, (k, v) in enumerate(c.rows):
        for j in (0, 13, Hkv - 1):
            for h in range(j * G, j * G + G):
                want, A, S = attention(q[i, h:h + 1], k[:, j], v[:, j], D ** -0.5, np.ones((1, len(k)), bool))
                worst = max(worst, check(got[i, h:h + 1], want, bound(want, A, S, D, len(k), "f32", 0.0, 8), f"sequence {i} head {h}"))
        if not len(k):
            assert (got[i] == 0).all()
    say(f"  worst error / bound {worst:.3g}")
