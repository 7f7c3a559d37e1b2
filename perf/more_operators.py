"""Cases and plain forms of the operators that positions and long contexts need around the paged
key-value cache: norms of query and key heads with the position rotation, the same on the way into
the cache, attention of several new tokens per sequence over the cache, and attention
with a sliding window and first tokens that stay visible.

``own = False`` computes each operator from its formula with elementary torch operations in
float32; ``own = True`` calls the library.  ``exact`` computes it in float64.

Sizes: the layer workload of this repository has a QKV product of 7168 rows, which is 40 query
heads and 8 key and 8 value heads of 128; the other head layouts and lengths are generic.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PLACES = 32768  # rows of the rotation table
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    heads = dict(hq=40, hkv=8, d=128)
    return [
        # a decode step's new token behind the QKV product: the smallest call, all latency
        dict(name="norm rope 1 token", op="rope", type="f32", out="f32", tokens=1, norm=True, rot=128, pairs="halves", axes=1, **heads),
        # a 2048-token prompt as the float32 QKV product leaves it, turned to the attention's type
        dict(name="norm rope 2048 f32 to bf16", op="rope", type="f32", out="bf16", tokens=2048, norm=True, rot=128, pairs="halves", axes=1, **heads),
        # a packed batch of prompts with images: three axes, an odd number of rows
        dict(name="norm rope 16411 3 axes bf16", op="rope", type="bf16", out="bf16", tokens=16411, norm=True, rot=128, pairs="halves", axes=3, **heads),
        # a decode step's token on its way into the cache: latency
        dict(name="append 1 token q8_0", op="append", kv="q8_0", type="f32", out="f32", tokens=1, norm=False, rot=128, pairs="halves", axes=1, page=64, **heads),
        # a prompt's rows into the quantised cache, norms and rotation on the way
        dict(name="append 2048 norm q8_0", op="append", kv="q8_0", type="f32", out="bf16", tokens=2048, norm=True, rot=128, pairs="halves", axes=1, page=64, **heads),
        # a packed batch into a 16-bit cache, half of the channels turned, neighbouring pairs
        dict(name="append 16411 bf16", op="append", kv="bf16", type="bf16", out="bf16", tokens=16411, norm=False, rot=64, pairs="neighbours", axes=1, page=16, **heads),
        # a few speculated tokens behind a short conversation: latency
        dict(name="chunk 16 of 500 q8_0", op="chunk", kv="q8_0", type="bf16", batch=1, tokens=16, prefix=484, ragged=False, window=0, sinks=0, page=64, mix=1, **heads),
        # a mixed batch: single tokens and pieces of prompts behind prefixes of all lengths
        dict(name="chunk 24 mixed bf16", op="chunk", kv="bf16", type="bf16", batch=24, tokens=1100, prefix=4000, ragged=True, window=0, sinks=0, page=16, mix=2, **heads),
        # the next piece of one long prompt
        dict(name="chunk 2048 of 16384 q8_0", op="chunk", kv="q8_0", type="bf16", batch=1, tokens=2048, prefix=14336, ragged=False, window=0, sinks=0, page=64, mix=3, **heads),
        # a piece of a long prompt in a layer with a window, a head width of 64
        dict(name="chunk 1024 window 4096 f16", op="chunk", kv="f16", type="f16", batch=1, tokens=1024, prefix=15000, ragged=False, window=4096, sinks=4, page=32, mix=4, hq=32, hkv=4, d=64),
        # one token of one very long conversation in a layer with a window: latency
        dict(name="window 4096 of 131071 q8_0", op="window", kv="q8_0", type="f32", batch=1, length=131071, ragged=False, window=4096, sinks=4, page=64, mix=5, **heads),
        # a full serving batch over a bfloat16 cache, ragged
        dict(name="window 4096 of 64x8192 bf16", op="window", kv="bf16", type="bf16", batch=64, length=8192, ragged=True, window=4096, sinks=16, page=16, mix=6, **heads),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "chunk", "window"))
    hq, hkv = rng.choice(((40, 8), (32, 8), (32, 4), (16, 16), (64, 8), (20, 4), (16, 1)))
    d = rng.choice((64, 96, 128, 128, 256))
    heads = dict(hq=hq, hkv=hkv, d=d)
    if op in ("rope", "append"):
        case = dict(op=op, type=rng.choice(("f32", "f16", "bf16")), out=rng.choice(("f32", "f16", "bf16")), tokens=_log_int(rng, 1, min(16384, 16384 * 56 * 128 // ((hq + 2 * hkv) * d) // 2)),
                    norm=rng.random() < 0.5, rot=rng.choice((d, d, d // 2)), pairs=rng.choice(("halves", "halves", "neighbours")), axes=rng.choice((1, 1, 3)), **heads)
        return case if op == "rope" else dict(case, kv=rng.choice(("q8_0", "q8_0", "f16", "bf16")), page=rng.choice((16, 32, 64, 256)))
    kv = rng.choice(("q8_0", "q8_0", "f16", "bf16"))
    sinks = rng.choice((0, 4, rng.randrange(1, 130)))
    page, mix = rng.choice((16, 32, 64, 256)), rng.randrange(1 << 20)
    if op == "window":
        batch = _log_int(rng, 1, 64)
        most = min(131071, 64 * 8192 * 8 * 128 // (batch * hkv * d))
        return dict(op=op, kv=kv, type=rng.choice(("f32", "f16", "bf16")), batch=batch, length=_log_int(rng, 1, most), ragged=rng.random() < 0.7,
                    window=_log_int(rng, 1, 4096), sinks=sinks, page=page, mix=mix, **heads)
    batch, tokens, prefix = _log_int(rng, 1, 24), _log_int(rng, 1, 2048), _log_int(rng, 1, 14336) - 1
    while batch * hq * min(tokens, 2 * -(-tokens // batch)) * (prefix + tokens) * d > 40 * 2048 * 16384 * 128:
        batch, tokens, prefix = max(1, batch // 2), max(1, tokens // 2), prefix // 2
    return dict(op=op, kv=kv, type=rng.choice(("f16", "bf16")) if kv == "q8_0" else kv, batch=batch, tokens=tokens, prefix=prefix, ragged=rng.random() < 0.7,
                window=rng.choice((0, 0, _log_int(rng, 1, 4096))), sinks=sinks, page=page, mix=mix, **heads)


def _lengths(case):
    """window: the sequences' lengths.  Ragged: uniform in 0 .. length, the first one whole."""
    if not case["ragged"]:
        return [case["length"]] * case["batch"]
    r = random.Random(case["mix"])
    return [case["length"]] + [r.randint(0, case["length"]) for _ in range(case["batch"] - 1)]


def _chunks(case):
    """chunk: (new tokens, keys) of each sequence.  Ragged: half of the sequences bring one token or none, the others share what is left
    (none more than twice its part), behind prefixes of 0 .. prefix."""
    n, b = case["tokens"], case["batch"]
    if not case["ragged"]:
        return [(n * (i + 1) // b - n * i // b, n * (i + 1) // b - n * i // b + case["prefix"]) for i in range(b)]
    r = random.Random(case["mix"])
    new = [min(1, r.randint(0, 4)) if i % 2 else r.randint(1, 2 * -(-n // b)) for i in range(b)]
    return [(m, m + r.randint(0, case["prefix"])) for m in new]


def _seen(case, m, n):
    """Keys that the m last of n tokens see, summed."""
    w, s = case["window"], case["sinks"]
    p = np.arange(n - m, n, dtype=np.int64)
    return int((p + 1 if not w else np.minimum(p + 1, w) + np.minimum(s, np.maximum(p + 1 - w, 0))).sum())


def _touched(case, m, n):
    """Keys that any of the m last of n tokens sees."""
    w, s = case["window"], case["sinks"]
    if m == 0:
        return 0
    lo = max(0, n - m + 1 - w) if w else 0
    return n - lo + min(s, lo)


def _sections(case):
    """Pairs of each axis."""
    half = case["rot"] // 2
    return [half] if case["axes"] == 1 else [half // 4, half - half // 4 - half // 8 * 3, half // 8 * 3]


def _row_bytes(case):
    return case["d"] * 2 if case["kv"] != "q8_0" else case["d"] + case["d"] // 32 * 2


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] in ("rope", "append"):
        size, out, n = TYPES[case["type"]].itemsize, TYPES[case["out"]].itemsize, case["tokens"]
        both = 4 * n * (case["rot"] + case["axes"]) + (8 * d if case["norm"] else 0)  # the table's rows, positions, weights
        if case["op"] == "rope":
            return {"bytes": n * (hq + hkv) * d * (size + out) + both, "flops": 0}
        back = 2 if case["kv"] == "q8_0" else 1  # (a quantised cache is read back)
        return {"bytes": n * (hq * d * (size + out) + 2 * hkv * (d * size + back * _row_bytes(case))) + both + 8 * n * back
                + (2 * n * hkv * d * 2 if back == 2 else 0), "flops": 0}
    size = TYPES[case["type"]].itemsize
    seqs = [(1, n) if n else (0, 0) for n in _lengths(case)] if case["op"] == "window" else _chunks(case)
    rows = case["batch"] if case["op"] == "window" else sum(m for m, _ in seqs)
    keys = sum(_touched(case, m, n) for m, n in seqs)
    return {"bytes": 2 * keys * hkv * _row_bytes(case) + 2 * rows * hq * d * size + 4 * keys // case["page"] + 8 * len(seqs),
            "flops": 4 * sum(_seen(case, m, n) for m, n in seqs) * hq * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _interleave(x):
    """Rows [..., D] in the order of the quantised cache: place 2 * (D/32) * n + 2 * b + e holds element 32 b + 2 n + e."""
    return x.unflatten(-1, (-1, 16, 2)).transpose(-3, -2).flatten(-3)


def _quantise(x):
    """Q8_0 of float32 rows [..., D]: codes (whole numbers, float32) and binary16 scales [..., D/32].  The divisor is a tensor: a division by a
    Python number would be a product with its rounded reciprocal."""
    x = x.unflatten(-1, (-1, 32))
    d = x.abs().amax(-1, keepdim=True) / torch.full((1,), 127.0, device=x.device)
    q = torch.where(d > 0, torch.round(x / d).clamp(-127, 127), torch.zeros((), device=x.device))
    return q.flatten(-2), d.squeeze(-1).to(torch.float16)


def _page_table(lens, page, g):
    """Pages of the sequences in shuffled order, as an allocator hands them out; entries behind a sequence's end are 0."""
    need = [-(-n // page) for n in lens]
    ids = torch.randperm(sum(need) + 3, generator=g)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table.cuda(), len(ids)


def _cache(kv, n_pages, hkv, page, d, r):
    """A cache full of keys or values of a normal distribution whose width differs from channel to channel."""
    codes = torch.empty((n_pages, hkv, page, d), dtype=torch.int8 if kv == "q8_0" else TYPES[kv], device="cuda")
    scales = torch.empty((n_pages, hkv, page, d // 32), dtype=torch.float16, device="cuda") if kv == "q8_0" else None
    width = torch.rand((hkv, 1, d), generator=r, device="cuda") * 1.5 + 0.25
    step = max(1, (1 << 26) // (hkv * page * d))
    for i in range(0, n_pages, step):
        x = torch.randn((min(step, n_pages - i), hkv, page, d), generator=r, device="cuda") * width
        if kv == "q8_0":
            q, scales[i:i + step] = _quantise(x)
            codes[i:i + step] = _interleave(q).to(torch.int8)
        else:
            codes[i:i + step] = x.to(codes.dtype)
    return codes, scales


def _rotation(rot):
    """The table that a program makes once: a row's cosines, then its sines, of place * 10000^(-2 c / rot)."""
    c = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(PLACES, dtype=torch.float64, device="cuda")[:, None] * 10000.0 ** (-2 * c / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def prepare(case, seed):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    t = TYPES[case["type"]]
    r = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.Generator().manual_seed(seed)
    s = dict(case=case)
    if case["op"] in ("rope", "append"):
        n = case["tokens"]
        # queries, keys and values as the fused QKV product leaves them: columns of one row, wider in some channels
        qkv = (torch.randn((n, (hq + 2 * hkv) * d), generator=r, device="cuda") * (torch.rand(((hq + 2 * hkv) * d,), generator=r, device="cuda") * 3 + 0.25)).to(t)
        s["q"], s["k"], s["v"] = (qkv[:, a * d:(a + h) * d].unflatten(1, (h, d)) for a, h in ((0, hq), (hq, hkv), (hq + hkv, hkv)))
        s["weights"] = [1 + torch.randn((d,), generator=r, device="cuda") / 4 for _ in "qk"] if case["norm"] else [None, None]
        s["table"], s["sections"] = _rotation(case["rot"]), _sections(case)
        first = int(torch.randint(0, PLACES - n, (1,), generator=g))
        i = torch.arange(n)
        # one axis: a prompt behind what came before it; three: an image's frames, rows and columns
        places = i[None] + first if case["axes"] == 1 else torch.stack([first + i // 1024, i // 32 % 32, i % 32])
        s["positions"] = places.to(torch.int32).cuda()
        s["axis"] = torch.arange(case["axes"], device="cuda").repeat_interleave(torch.tensor(s["sections"], device="cuda"))
        if case["op"] == "append":
            page, kv = case["page"], case["kv"]
            n_pages = -(-n // page) + 1
            at = i + (page // 3 if n + page // 3 <= n_pages * page else 0)  # prompts do not begin at a page's start
            s["slots"] = (torch.randperm(n_pages, generator=g)[at // page] * page + at % page).cuda()
            shape = (n_pages, hkv, page, d)
            s["codes"] = [torch.zeros(shape, dtype=torch.int8 if kv == "q8_0" else TYPES[kv], device="cuda") for _ in "kv"]
            s["scales"] = [torch.zeros((*shape[:3], d // 32), dtype=torch.float16, device="cuda") if kv == "q8_0" else None for _ in "kv"]
        return s
    seqs = [(1, n) for n in _lengths(case)] if case["op"] == "window" else _chunks(case)
    lens = [n for _, n in seqs]
    s["table"], n_pages = _page_table(lens, case["page"], g)
    s["q"] = torch.randn((sum(m for m, _ in seqs), hq, d), generator=r, device="cuda").to(t)
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu_q"] = torch.tensor([sum(m for m, _ in seqs[:j]) for j in range(len(seqs) + 1)], dtype=torch.int32, device="cuda")
    s["most"] = max(m for m, _ in seqs)
    caches = [_cache(case["kv"], n_pages, hkv, case["page"], d, r) for _ in "kv"]
    s["codes"], s["scales"] = [c for c, _ in caches], [x for _, x in caches]
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    return {"rope": _run_rope, "append": _run_append, "chunk": _run_chunk, "window": _run_window}[case["op"]](state, case)


def _back(case):
    """The type that a quantised cache's rows are read back in."""
    return torch.bfloat16 if case["out"] == "bf16" else torch.float16


def _turned(x, weight, s, case):
    """Rows [T, H, D], normed and turned, in float32."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    rot = case["rot"]
    pair = torch.arange(rot // 2, device="cuda")
    place = s["positions"].long()[s["axis"]].T  # [T, pairs]
    cos, sin = (s["table"][place, pair + i][:, None] for i in (0, rot // 2))
    if case["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)


def _more(s, case, nvq):
    return dict(q_weight=s["weights"][0], k_weight=s["weights"][1], eps=EPS, pairs=nvq.NVQ_ROPE_HALVES if case["pairs"] == "halves" else nvq.NVQ_ROPE_NEIGHBOURS,
                sections=None if case["axes"] == 1 else s["sections"])


def _run_rope(s, case):
    out = TYPES[case["out"]]
    if own:
        import gemm_q8_act_amd as nvq

        q, k = (torch.empty(s[x].shape, dtype=out, device="cuda") for x in "qk")
        nvq.nvq_qk_norm_rope(s["q"], s["k"], s["table"], s["positions"], q, k, **_more(s, case, nvq))
        return q, k
    return tuple(_turned(s[x], w, s, case).to(out) for x, w in zip("qk", s["weights"]))


def _run_append(s, case):
    out, back = TYPES[case["out"]], _back(case)
    (kc, vc), (kd, vd) = s["codes"], s["scales"]
    if own:
        import gemm_q8_act_amd as nvq

        q = torch.empty(s["q"].shape, dtype=out, device="cuda")
        nvq.nvq_rope_kv_write(s["q"], s["k"], s["v"], s["table"], s["positions"], s["slots"], q, kc, vc, kd, vd, **_more(s, case, nvq))
        if kd is None:
            return q, kc, vc
        k, v = (torch.empty(s[x].shape, dtype=back, device="cuda") for x in "kv")
        nvq.nvq_kv_read(kc, vc, s["slots"], k, v, kd, vd)
        return q, k, v
    q = _turned(s["q"], s["weights"][0], s, case).to(out)
    page, off = s["slots"] // case["page"], s["slots"] % case["page"]
    if kd is None:
        kc[page, :, off], vc[page, :, off] = _turned(s["k"], s["weights"][1], s, case).to(kc.dtype), s["v"].float().to(vc.dtype)
        return q, kc, vc
    return q, _through(_turned(s["k"], s["weights"][1], s, case), kc, kd, page, off).to(back), _through(s["v"].float(), vc, vd, page, off).to(back)


def _through(x, codes, scales, page, off):
    """Rows written into the quantised cache, and as it holds them."""
    q, d = _quantise(x)
    codes[page, :, off] = _interleave(q).to(torch.int8)
    scales[page, :, off] = d
    return _rows(codes[page, :, off], scales[page, :, off])


def _rows(codes, scales):
    """Cache rows [..., D] as float32."""
    if scales is None:
        return codes.float()
    x = codes.float().unflatten(-1, (16, -1, 2)) * scales.float()[..., None, :, None]
    return x.transpose(-3, -2).flatten(-3)


def _softmax_product(s, seen, v):
    """Rows of scores, of which each sees what `seen` says, times v; a row that sees nothing gives zeros."""
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total == 0, 1.0, total)


def _run_chunk(s, case):
    (kc, vc), (kd, vd) = s["codes"], s["scales"]
    q = s["q"]
    if own:
        import gemm_q8_act_amd as nvq

        out = torch.empty_like(q)
        nvq.nvq_attn_chunk(q, kc, vc, s["table"], s["cu_q"], s["lengths"], out, kd, vd, window=case["window"], sinks=case["sinks"])
        return out
    hkv, d, most = case["hkv"], case["d"], s["most"]
    table, n, cu = s["table"].long(), s["lengths"].long(), s["cu_q"].long()
    b, g = table.shape[0], case["hq"] // hkv
    k, v = (_rows(c[table], x if x is None else x[table]).transpose(1, 2).flatten(2, 3) for c, x in ((kc, kd), (vc, vd)))  # [B, Hkv, L, D]
    i, m = torch.arange(most, device="cuda"), cu[1:] - cu[:-1]
    row = (cu[:-1, None] + i).clamp_(max=q.shape[0] - 1)  # every sequence's rows, filled up to the longest
    qs = q[row].float().view(b, most, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * most, d) * (1 / math.sqrt(d))
    p, j = (i + (n - m)[:, None])[:, :, None], torch.arange(k.shape[2], device="cuda")
    seen = j <= p
    if case["window"]:
        seen &= (j > p - case["window"]) | (j < case["sinks"])
    o = _softmax_product(torch.matmul(qs, k.transpose(-1, -2)).view(b, hkv, g, most, -1), seen[:, None, None], v[:, :, None])
    o = o.permute(0, 3, 1, 2, 4).reshape(b, most, -1, d)
    return o[i < m[:, None]].to(q.dtype)


def _run_window(s, case):
    (kc, vc), (kd, vd) = s["codes"], s["scales"]
    q = s["q"]
    if own:
        import gemm_q8_act_amd as nvq

        out = torch.empty_like(q)
        nvq.nvq_attn_decode_window(q, kc, vc, s["table"], s["lengths"], out, kd, vd, window=case["window"], sinks=case["sinks"])
        return out
    hkv, d, n = case["hkv"], case["d"], s["lengths"].long()[:, None]
    first = torch.arange(case["sinks"], device="cuda")[None]
    start = (n - case["window"]).clamp(min=0)
    last = start + torch.arange(min(case["window"], case["length"]), device="cuda")
    seen = torch.cat([first < torch.minimum(start, n), last < n], 1)  # [B, sinks + window]
    at = torch.cat([first.expand(n.shape[0], -1), last], 1)
    at = torch.where(seen, at, 0)
    page, off = s["table"].long().gather(1, at // case["page"]), at % case["page"]
    k, v = (_rows(c[page, :, off], x if x is None else x[page, :, off]).transpose(1, 2) for c, x in ((kc, kd), (vc, vd)))  # [B, Hkv, keys, D]
    scores = torch.matmul(q.float().view(q.shape[0], hkv, -1, d) * (1 / math.sqrt(d)), k.transpose(-1, -2))
    return _softmax_product(scores, seen[:, None, None], v).reshape(q.shape).to(q.dtype)


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------

def _exact_turned(x, weight, s, case):
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    half = case["rot"] // 2
    y = x.clone()
    axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    for c in range(half):
        i, j = (c, c + half) if case["pairs"] == "halves" else (2 * c, 2 * c + 1)
        row = s["table"][s["positions"][axis[c]].long()].double()
        co, si = row[:, c, None], row[:, half + c, None]
        y[..., i], y[..., j] = x[..., i] * co - x[..., j] * si, x[..., j] * co + x[..., i] * si
    return y


def _exact_quantised(x):
    blocks = x.reshape(*x.shape[:2], -1, 32)
    step = blocks.abs().max(-1, keepdim=True).values / 127
    return (torch.round(blocks / step) * torch.from_numpy(step.cpu().numpy().astype(np.float16).astype(np.float64)).cuda()).reshape(x.shape)


def _exact_rows(codes, scales):
    """Cache rows [n, H, D] (interleaved codes or plain numbers) in float64."""
    if scales is None:
        return codes.double()
    d = codes.shape[-1]
    at = torch.arange(d)
    nb = d // 32
    place = 2 * nb * (at % 32 // 2) + 2 * (at // 32) + at % 2
    return codes.double()[..., place.to(codes.device)] * scales.double()[..., (at // 32).to(codes.device)]


def _exact_attention(q, k, v, case, n):
    """q [m, Hq, D], the last m tokens' of the n of k and v [n, Hkv, D], in float64."""
    m, hq, d = q.shape
    out = torch.zeros_like(q)
    if n == 0 or m == 0:
        return out
    j, p = torch.arange(n, device="cuda")[None], torch.arange(n - m, n, device="cuda")[:, None]
    hidden = j > p
    if case["window"]:
        hidden |= (p - j >= case["window"]) & (j >= case["sinks"])
    for h in range(hq):
        i = h * k.shape[1] // hq
        s = q[:, h] @ k[:, i].T / math.sqrt(d)
        s[hidden] = -math.inf
        out[:, h] = torch.softmax(s, -1).nan_to_num(0.0) @ v[:, i]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_exact_turned(s[x], w, s, case) for x, w in zip("qk", s["weights"]))
    if case["op"] == "append":
        q, k = (_exact_turned(s[x], w, s, case) for x, w in zip("qk", s["weights"]))
        if case["kv"] == "q8_0":
            return q, _exact_quantised(k), _exact_quantised(s["v"].double())
        page, off = s["slots"] // case["page"], s["slots"] % case["page"]
        caches = [c.double() for c in s["codes"]]
        for c, x in zip(caches, (k, s["v"].double())):
            c[page, :, off] = x
        return q, *caches
    seqs = [(1, n) for n in _lengths(case)] if case["op"] == "window" else _chunks(case)
    out, a = [], 0
    for i, (m, n) in enumerate(seqs):
        at = torch.arange(n, device="cuda")
        page, off = s["table"][i].long()[at // case["page"]], at % case["page"]
        k, v = (_exact_rows(c[page, :, off], x if x is None else x[page, :, off]) for c, x in zip(s["codes"], s["scales"]))
        out.append(_exact_attention(s["q"][a:a + m].double(), k, v, case, n))
        a += m
    return torch.cat(out)
