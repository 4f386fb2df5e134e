"""One attention layer decoding step by step on quantized weights with a
bounded cache: the q|k|v and o products over packed images (gemm_mixed_w),
rotary positions and the cache write (rope_append), attention of the new
token with its weights accumulated (paged_attention), and eviction once a
sequence passes its budget (cache_evict).

    python examples/decode_layer.py [--steps 200] [--budget 128]

prints the cache lengths and the time of a step on one GPU."""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_block_bit_amd as gbb  # noqa: E402


class DecodeLayer:
    """Attention of a pre-norm decoder layer for `batch` sequences.  budget:
    slots a sequence keeps per kv head; `slack` more are let in before an
    eviction, so that it runs once in `slack` steps."""

    def __init__(self, batch, q_heads, kv_heads, head_dim, budget, recent, slack=16, page=64, n_pos=4096, bits=4.0,
                 layout="half", dtype=torch.float16, seed=0):
        self.batch, self.q_heads, self.kv_heads, self.head_dim = batch, q_heads, kv_heads, head_dim
        self.budget, self.recent, self.slack, self.layout = budget, recent, slack, layout
        self.hidden = q_heads * head_dim
        g = np.random.default_rng(seed)

        def packed(n, k):
            w = (g.standard_normal((n, k)) / np.sqrt(k)).astype(np.float16)
            image, _, _ = gbb.pack_blocks(w, gbb.allocate_bits(w, bits))
            return torch.from_numpy(image).cuda()

        self.qkv_rows = (q_heads + 2 * kv_heads) * head_dim
        self.qkv, self.o = packed(self.qkv_rows, self.hidden), packed(self.hidden, self.hidden)
        self.table = torch.from_numpy(gbb.rope_table(head_dim, n_pos, 500000.0)).cuda()
        # budget + slack slots a sequence, its pages given out once
        self.max_len = budget + slack
        per = -(-self.max_len // page)
        scale = torch.full((kv_heads,), 8.0 / 448, device="cuda") if dtype == torch.float8_e4m3fn else None
        self.cache = gbb.PagedCache.empty(batch * per, page, kv_heads, head_dim, dtype, "cuda", True, scale, scale)
        self.block_table = torch.randperm(batch * per).to(torch.int32).view(batch, per).cuda()
        self.lengths = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.positions = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.rows = torch.arange(batch, device="cuda")
        self.length = 0          # the lengths' common value, known without a copy from the GPU

    def step(self, x):
        """x fp16 [batch][hidden] -> fp16 [batch][hidden]."""
        page = self.cache.page
        qkv = gbb.gemm_mixed_w(self.qkv, self.qkv_rows, self.hidden, x)
        slots = self.block_table[self.rows, (self.lengths // page).long()] * page + self.lengths % page
        q = gbb.rope_append(self.cache, qkv, self.q_heads, self.positions, slots, self.table, layout=self.layout)
        self.positions += 1
        self.lengths += 1
        self.length += 1
        out = gbb.paged_attention(self.cache, q, self.block_table, self.lengths, self.max_len,
                                  weights_out=self.cache.weights)
        y = gbb.gemm_mixed_w(self.o, self.hidden, self.hidden, out.view(self.batch, self.hidden))
        if self.length == self.max_len:
            self.lengths = gbb.cache_evict(self.cache, self.block_table, self.lengths, self.max_len, self.budget,
                                           self.recent)
            self.length = self.budget
        return y


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--budget", type=int, default=128)
    a = ap.parse_args()
    layer = DecodeLayer(a.batch, 32, 8, 128, a.budget, a.budget // 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.steps, a.batch, layer.hidden, generator=g, device="cuda").half()
    layer.step(x[0])
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    for i in range(1, a.steps):
        y = layer.step(x[i])
        if i % 50 == 0:
            print(f"step {i}: lengths {layer.lengths.tolist()}, |y| {y.float().norm().item():.3f}", flush=True)
    t[1].record()
    torch.cuda.synchronize()
    print(f"{t[0].elapsed_time(t[1]) / max(1, a.steps - 1) * 1e3:.1f} us a step, {a.steps} tokens seen, "
          f"{layer.length} kept a sequence")


if __name__ == "__main__":
    main()
