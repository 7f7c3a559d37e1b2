"""The attention half of a transformer layer on this library: NVFP4 QKV and O products with
the paged Q8_0 key-value cache and both attention operators between them.

  python examples/attention_layer.py [--prompt 2048] [--steps 32] [--hidden 5120] [--heads 40] [--kv-heads 8]

A prompt goes through the tiled products and nvq_attn_prompt, its keys and values into the cache;
a second piece of the same prompt attends to the first one's rows, read back from the cache; then
tokens are decoded one at a time: fused quantisation + GEMV, nvq_kv_write, nvq_attn_decode, fused
GEMV.  Weights are random (no checkpoint is read); position embeddings, which belong between
the QKV product and the cache, are left out.
"""
import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_q8_act_amd as nvq  # noqa: E402
from gemm_q8_act_amd import synth  # noqa: E402


class AttentionLayer:
    """Weights, cache and one sequence's place in it."""

    def __init__(self, hidden, heads, kv_heads, head_dim, max_tokens, page=64, seed=0):
        self.hidden, self.heads, self.kv_heads, self.head_dim, self.page = hidden, heads, kv_heads, head_dim, page
        self.rows = (heads + 2 * kv_heads) * head_dim
        self.w_qkv, self.s_qkv, self.qkv_logical = self._weights(self.rows, hidden, seed + 1)
        self.w_o, self.s_o, self.o_logical = self._weights(hidden, heads * head_dim, seed + 2)
        pages = -(-max_tokens // page)
        self.max_tokens = pages * page
        shape = (pages, kv_heads, page, head_dim)
        self.codes = [torch.zeros(shape, dtype=torch.int8, device="cuda") for _ in "kv"]
        self.scales = [torch.zeros((*shape[:3], head_dim // 32), dtype=torch.float16, device="cuda") for _ in "kv"]
        ids = np.random.Generator(np.random.PCG64(seed)).permutation(pages).astype(np.int32)
        self.table = torch.from_numpy(ids).cuda()[None]  # one sequence: every page, in an allocator's order
        self.workspace = torch.empty(max(16, nvq.nvq_attn_decode_workspace_bytes(1, heads, kv_heads, head_dim, pages, page)), dtype=torch.uint8,
                                     device="cuda")
        self.length = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.n = 0

    def _weights(self, N, K, seed):
        """Random weights with the per-tensor scale that gives products of unit width, as a trained layer's roughly have
        (without it the softmax would pick one key): packed, scale, logical."""
        codes, scales, _ = synth.nvfp4_weights(N, K, seed)
        w = torch.from_numpy(nvq.nvq_pack_nvfp4(codes, scales)).cuda()
        y = self._product(w, 1.0, torch.from_numpy(synth.activations(8, K, seed)).cuda(), N)
        s = float(np.float32(1.0 / float(y.square().mean().sqrt())))
        return w, s, (codes, scales, s)

    def _room(self, count):
        if count < 1 or self.n + count > self.max_tokens:
            raise ValueError("%d tokens behind %d: the cache takes 1 to %d more" % (count, self.n, self.max_tokens - self.n))

    def _slots(self, first, count):
        at = torch.arange(first, first + count, device="cuda")
        return self.table[0].long()[at // self.page] * self.page + at % self.page

    def _split(self, y):
        h, k, d = self.heads, self.kv_heads, self.head_dim
        y = y.unflatten(1, (h + 2 * k, d))
        return y[:, :h], y[:, h:h + k], y[:, h + k:]

    def _product(self, w, s, x, rows):
        """[M, K] float32 -> [M, rows]: Q8_0 quantisation, then the GEMV or the tiled product by M."""
        M, K = x.shape
        q = torch.empty((M, K), dtype=torch.int8, device="cuda")
        d = torch.empty((M, K // 32), dtype=torch.int16, device="cuda")
        nvq.nvq_quantize_act_q8_0(x, q, d)
        y = torch.empty((M, rows), dtype=torch.float32, device="cuda")
        (nvq.nvq_gemv_nvfp4 if M <= nvq.NVQ_GEMV_MAX_M else nvq.nvq_gemm_nvfp4)(w, s, q, d, y)
        return y

    def prompt(self, x):
        """x [M, hidden] float32, the next M tokens: [M, hidden].  What is already in the cache is read back."""
        M, prefix = x.shape[0], self.n
        self._room(M)
        q, k, v = self._split(self._product(self.w_qkv, self.s_qkv, x, self.rows))
        nvq.nvq_kv_write(k, v, self._slots(prefix, M), *self.codes, *self.scales)
        keys, values = (torch.empty((prefix + M, self.kv_heads, self.head_dim), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        nvq.nvq_kv_read(*self.codes, self._slots(0, prefix), keys[:prefix], values[:prefix], *self.scales)
        keys[prefix:], values[prefix:] = k, v
        self.n += M
        self.length.fill_(self.n)
        cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (M, prefix + M))
        a = torch.empty((M, self.heads, self.head_dim), dtype=torch.bfloat16, device="cuda")
        nvq.nvq_attn_prompt(q.bfloat16(), keys, values, cu_q, cu_k, a)
        return self._product(self.w_o, self.s_o, a.flatten(1).float(), self.hidden)

    def step(self, x):
        """x [1, hidden] float32, the next token: [1, hidden]."""
        self._room(1)
        y = torch.empty((1, self.rows), dtype=torch.float32, device="cuda")
        nvq.nvq_gemv_nvfp4_fused(self.w_qkv, self.s_qkv, x, y)
        q, k, v = self._split(y)
        nvq.nvq_kv_write(k, v, self._slots(self.n, 1), *self.codes, *self.scales)
        self.n += 1
        self.length += 1
        a = torch.empty((1, self.heads, self.head_dim), dtype=torch.float32, device="cuda")
        nvq.nvq_attn_decode(q, *self.codes, self.table, self.length, a, *self.scales, workspace=self.workspace)
        out = torch.empty((1, self.hidden), dtype=torch.float32, device="cuda")
        nvq.nvq_gemv_nvfp4_fused(self.w_o, self.s_o, a.flatten(1), out)
        return out


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--prompt", type=int, default=2048)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--heads", type=int, default=40)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--head-dim", type=int, default=128)
    a = p.parse_args()
    if a.prompt < 2 or a.steps < 1:
        p.error("a prompt of two tokens or more (it goes in two pieces) and a step or more")
    layer = AttentionLayer(a.hidden, a.heads, a.kv_heads, a.head_dim, a.prompt + a.steps + 1)
    x = torch.from_numpy(synth.activations(a.prompt + a.steps, a.hidden, 3)).cuda()
    half = a.prompt // 2
    for name, run in (("first half of the prompt", lambda: layer.prompt(x[:half])), ("second half", lambda: layer.prompt(x[half:a.prompt])),
                      ("%d decode steps" % a.steps, lambda: [layer.step(x[i:i + 1]) for i in range(a.prompt, a.prompt + a.steps)][-1])):
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = run()
        torch.cuda.synchronize()
        print("%s: %.3f ms, output %s, rms %.3f" % (name, 1e3 * (time.perf_counter() - t), list(y.shape), float(y.square().mean().sqrt())), flush=True)


if __name__ == "__main__":
    main()
