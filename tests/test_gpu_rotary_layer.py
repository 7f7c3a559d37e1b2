"""Norms, rotation, cache, chunk and window attention together: the example's layer, stage by stage, and a serving step of
several sequences captured once and replayed.

Every stage of the layer is checked on what the stage before handed it (a share of the places where a value quantised in
between lies on the edge of two codes gives the other code, so an end-to-end bound would be one on their number).  Cached
keys: half a code's step, and the binary16 scale's half unit at 127 steps; values: bit for bit.
"""
import os
import sys

import numpy as np
import pytest

import gemm_q8_act_amd as nvq
from attn_cases import check
from gemm_q8_act_amd import synth
from gpu_cases import host, say, torch_dev
from test_gpu_attn_chunk import P_UNIT
from test_gpu_rope import limit, want_rows
from window_cases import compare, seen_of

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("hidden,heads,kv_heads,head_dim,page,window,sinks",
                         [(256, 4, 2, 64, 16, 0, 0), (320, 5, 1, 128, 64, 24, 3), (256, 2, 2, 96, 16, 33, 0)])
def test_layer(oracle, monkeypatch, hidden, heads, kv_heads, head_dim, page, window, sinks):
    torch = torch_dev()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        from attention_layer import RotaryLayer
    finally:
        sys.path.pop(0)
    pieces, steps = (40, 21), 5
    total = sum(pieces) + steps
    layer = RotaryLayer(hidden, heads, kv_heads, head_dim, total, page=page, seed=5, window=window, sinks=sinks)
    x = synth.activations(total, hidden, 6)
    xd = torch.from_numpy(x).cuda()
    calls = []  # of the three operators: their arguments

    def recorded(name):
        call = getattr(nvq, name)

        def run(*a, **kw):
            call(*a, **kw)
            calls.append((name, a))
        monkeypatch.setattr(nvq, name, run)

    for name in ("nvq_rope_kv_write", "nvq_attn_chunk", "nvq_attn_decode_window"):
        recorded(name)

    def product(logical, rows, got, what):
        codes, scales, s = logical
        qo, do, _ = oracle.quantize_q8_0(np.ascontiguousarray(rows, np.float32))
        want, size = oracle.matmul_nvfp4(codes, scales, s, qo, do)
        assert (np.abs(got - want) <= 1e-5 * size + 1e-6).all(), what

    def cached(rows):
        qo, do, _ = oracle.quantize_q8_0(np.ascontiguousarray(rows.reshape(-1, head_dim)))
        return (qo.astype(np.float32) * np.repeat(do.view(np.float16).astype(np.float32), 32, axis=1)).reshape(rows.shape)

    turns, at, weights = host(layer.turns), 0, [host(w) for w in layer.norms]
    for m in [*pieces, *[1] * steps]:
        step, n = at >= sum(pieces), at + m
        calls.clear()
        out = host((layer.step if step else layer.prompt)(xd[at:n])).astype(np.float64)
        (first, write), (second, attend) = calls
        assert first == "nvq_rope_kv_write" and second == ("nvq_attn_decode_window" if step else "nvq_attn_chunk")
        say(f"{m} tokens behind {at}: {second}")
        q, k, v = (host(r) for r in write[:3])
        product(layer.qkv_logical, x[at:n], np.concatenate([q, k, v], axis=1).reshape(m, -1), "QKV product")
        type_ = "f32" if step else "bf16"
        place = np.arange(at, n)
        want, size = want_rows(q, weights[0], 1e-6, turns, place, head_dim, "halves")
        turned = host(attend[0].float())
        check(turned, want, limit(want, size, head_dim, type_), "queries")
        rows = [torch.empty((n, kv_heads, head_dim), dtype=torch.float32, device="cuda") for _ in "kv"]
        nvq.nvq_kv_read(*layer.codes, layer._slots(0, n), *rows, *layer.scales)
        kc, vc = (host(r) for r in rows)
        want, size = want_rows(k, weights[1], 1e-6, turns, place, head_dim, "halves")
        unit = np.abs(want).reshape(m, kv_heads, -1, 32).max(-1).repeat(32, axis=-1) / 127
        check(kc[at:], want, (0.501 + 127 * 2.0 ** -11) * unit + 2 * limit(want, size, head_dim, "f32"), "keys in the cache")
        assert (vc[at:] == cached(v)).all()
        a = host((attend[5] if step else attend[6]).float())
        compare(a, turned, (kc, vc), seen_of(m, n, window, sinks), head_dim ** -0.5, "q8_0", type_, None if step else P_UNIT["q8_0"],
                f"{m} tokens behind {at}")
        product(layer.o_logical, a.reshape(m, -1), out, "O product")
        at = n


@pytest.mark.parametrize("cache", ["q8_0", "bf16"])
def test_captured_serving_step(cache):
    """Three sequences, one with a piece of its prompt, two with a token each: one launch sequence captured, replayed while all
    the numbers it reads move on, every replay against the eager calls on a second cache."""
    torch = torch_dev()
    Hq, Hkv, D, page, pages, window, sinks, piece = 6, 2, 128, 16, 12, 40, 5, 9
    g = torch.Generator("cuda").manual_seed(3)

    def make():
        shape = (3 * pages, Hkv, page, D)
        if cache == "q8_0":
            return ([torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in "kv"],
                    [torch.zeros((*shape[:3], D // 32), dtype=torch.float16, device="cuda") for _ in "kv"])
        return [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in "kv"], [None, None]

    table = torch.randperm(3 * pages, generator=g, device="cuda").int().view(3, pages)
    turns = torch.from_numpy(nvq.nvq_rope_table(pages * page, D)).cuda()
    weights = dict(q_weight=1 + torch.randn(D, generator=g, device="cuda") / 4, k_weight=1 + torch.randn(D, generator=g, device="cuda") / 4)
    counts = [piece, 1, 1]
    T = sum(counts)
    cu_q = torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32, device="cuda")
    owner = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(counts, device="cuda"))
    y = torch.empty((T, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")
    lengths = torch.zeros(3, dtype=torch.int32, device="cuda")
    positions = torch.zeros(T, dtype=torch.int32, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")

    def set_inputs(i):
        """Replay i: the prompt's sequence has i * piece tokens already, the others 20 + i and 3 + i (as far as those go: the rows before were
        never written, and are zeros in both caches)."""
        y.normal_(generator=g)
        old = [i * piece, 20 + i, 3 + i]
        at = np.concatenate([np.arange(o, o + m) for o, m in zip(old, counts)])
        positions.copy_(torch.from_numpy(at.astype(np.int32)))
        p = positions.long()
        slots.copy_(table.long()[owner, p // page] * page + p % page)
        lengths.copy_(torch.tensor([o + m for o, m in zip(old, counts)], dtype=torch.int32))

    def step(codes, scales, q, a, b):
        nvq.nvq_rope_kv_write(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], turns, positions, slots, q, *codes, *scales, **weights)
        nvq.nvq_attn_chunk(q, *codes, table, cu_q, lengths, a, *scales, window=window, sinks=sinks)
        nvq.nvq_attn_decode_window(q[piece:], *codes, table[1:], lengths[1:], b, *scales, window=window, sinks=sinks)

    def outputs():
        return [torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda") for n in (T, T, 2)]

    largest = 0.0  # value so far
    eager, replayed = make(), make()
    want, got = outputs(), outputs()
    set_inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*replayed, *got)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*replayed, *got)
    for i in range(6):
        set_inputs(i)
        largest = max(largest, float(y[:, Hq + Hkv:].abs().max()) * 1.01)
        step(*eager, *want)
        graph.replay()
        torch.cuda.synchronize()
        say(f"replay {i}")
        for x, z in zip(want, got):
            assert torch.equal(x, z)
        # A token through the chunk kernel and through the decode kernel.  The chunk kernel rounds weights to its type (2^-8 at
        # most) and, over Q8_0, both operands of a score to binary16: 2 * 2^-11 of |q| |k| scale, where normed heads are
        # sqrt(D) times their weights long at most (1.05: the cache's own rounding).  Both results are rounded.
        x, z = want[1][piece:].float(), want[2].float()
        score = 2 * 2.0 ** -11 * 1.05 * D ** 0.5 * float(weights["q_weight"].abs().max() * weights["k_weight"].abs().max())
        assert ((x - z).abs() <= (2.0 ** -8 + score) * largest + 2.0 ** -8 * (x.abs() + z.abs())).all()
    for x, z in zip([*eager[0], *[s for s in eager[1] if s is not None]], [*replayed[0], *[s for s in replayed[1] if s is not None]]):
        assert torch.equal(x, z)


@pytest.mark.parametrize("fmt", ["q8_0", "bf16"])
def test_pages_past_32_bit_offsets(fmt):
    """The same tokens written to, and read from, the last pages of a cache of more than 4 GiB a tensor and a small one."""
    torch = torch_dev()
    Hq, Hkv, D, page, n = 10, 2, 128, 256, 700
    pages = -(-n // page)
    g = torch.Generator("cuda").manual_seed(9)
    y = torch.randn((n, Hq + 2 * Hkv, D), generator=g, device="cuda")
    turns = torch.from_numpy(nvq.nvq_rope_table(n, D)).cuda()
    at = torch.arange(n, device="cuda")
    results = []
    for n_pages in (pages, (1 << 32) // (Hkv * page * D * (1 if fmt == "q8_0" else 2)) + pages + 5):
        say(f"pages past 32 bits: {fmt} {n_pages}")
        dtype = torch.int8 if fmt == "q8_0" else torch.bfloat16
        codes = [torch.empty((n_pages, Hkv, page, D), dtype=dtype, device="cuda") for _ in "kv"]
        scales = [torch.empty((n_pages, Hkv, page, D // 32), dtype=torch.float16, device="cuda") if fmt == "q8_0" else None for _ in "kv"]
        table = (n_pages - 1 - torch.arange(pages, device="cuda"))[None].int()
        q = torch.empty((n, Hq, D), dtype=torch.bfloat16, device="cuda")
        nvq.nvq_rope_kv_write(y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:], turns, at.int(), table[0].long()[at // page] * page + at % page, q, *codes,
                              *scales)
        lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
        a, b = torch.empty_like(q), torch.empty_like(q[-1:])
        nvq.nvq_attn_chunk(q, *codes, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"), lengths, a, *scales, window=400, sinks=3)
        nvq.nvq_attn_decode_window(q[-1:], *codes, table, lengths, b, *scales, window=400, sinks=3)
        results.append([host(x.float()) for x in (q, a, b)])
        del codes, scales
    for x, z in zip(*results):
        assert np.isfinite(x).all() and (x == z).all()
