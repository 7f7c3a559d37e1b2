"""The attention layer example against the same chain in float64: the products by the oracle,
the cache's rows by the oracle's Q8_0, attention from the formula.

Bounds (relative 2-norm of the layer's output).  Decode: attention agrees to about 1e-6, which moves a
Q8_0 code of its output (step 1/127 of the block's largest) by one for about one in 10^4 values, so the
product of the codes moves by about 10^-2 * 1/127 / 0.3 = 3e-4: 1e-3.  Prompt: the probabilities and the
attention's output are rounded to bfloat16 (2^-9 each, twice), and codes move with it: 1e-2."""
import os
import sys

import numpy as np
import pytest

from attn_cases import attention, rounded
from gemm_q8_act_amd import synth
from gpu_cases import host, say, torch_dev

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def relative(a, b):
    return float(np.linalg.norm(a - b) / np.linalg.norm(b))


@pytest.mark.parametrize("hidden,heads,kv_heads,head_dim,page", [(256, 4, 2, 64, 16), (320, 5, 1, 128, 64)])
def test_layer(oracle, hidden, heads, kv_heads, head_dim, page):
    torch = torch_dev()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from attention_layer import AttentionLayer
    finally:
        sys.path.pop(0)
    pieces, steps = (40, 21), 5
    total = sum(pieces) + steps
    layer = AttentionLayer(hidden, heads, kv_heads, head_dim, total, page=page, seed=5)
    x = synth.activations(total, hidden, 6)
    xd = torch.from_numpy(x).cuda()
    got, at = [], 0
    for m in pieces:
        got.append(host(layer.prompt(xd[at:at + m])))
        at += m
    for i in range(at, total):
        got.append(host(layer.step(xd[i:i + 1])))

    def product(logical, a):
        codes, scales, s = logical
        qo, do, _ = oracle.quantize_q8_0(np.ascontiguousarray(a, np.float32))
        return oracle.matmul_nvfp4(codes, scales, s, qo, do)[0]

    y = product(layer.qkv_logical, x).astype(np.float32).reshape(total, heads + 2 * kv_heads, head_dim)
    q, k, v = y[:, :heads], y[:, heads:heads + kv_heads], y[:, heads + kv_heads:]

    def cached(rows):
        qo, do, _ = oracle.quantize_q8_0(np.ascontiguousarray(rows.reshape(-1, head_dim)))
        return (qo.astype(np.float32) * np.repeat(do.view(np.float16).astype(np.float32), 32, axis=1)).reshape(rows.shape)

    kc, vc = cached(k), cached(v)
    at = 0
    for i, m in enumerate([*pieces, *[1] * steps]):
        n = at + m
        step = i >= len(pieces)
        if step:  # float32 queries over the cache
            qq, kk, vv = q[at:n], kc[:n], vc[:n]
        else:     # bfloat16: the cache's rows for the prefix, the new ones as they are
            qq = rounded(q[at:n], "bf16")
            kk, vv = (rounded(np.concatenate([c[:at], r[at:n]]), "bf16") for c, r in ((kc, k), (vc, v)))
        seen = np.arange(n)[None] <= np.arange(m)[:, None] + at
        a = np.stack([attention(qq[:, h], kk[:, h * kv_heads // heads], vv[:, h * kv_heads // heads], head_dim ** -0.5, seen)[0]
                      for h in range(heads)], axis=1)
        a = a.reshape(m, -1).astype(np.float32)
        want = product(layer.o_logical, a if step else rounded(a, "bf16"))
        r = relative(got[i].astype(np.float64), want.astype(np.float64))
        say(f"piece {i}: {m} tokens behind {at}: relative difference {r:.2e}")
        assert r < (1e-3 if step else 1e-2)
        at = n
