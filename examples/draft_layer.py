"""One attention layer that reads ragged prompts and decodes by verifying trees
of drafted tokens, on quantized weights: the q|k|v and o products over packed
images (gemm_mixed_w), norms of the q and k heads with rotary positions and the
cache write (rope_append), attention of prompts and trees (paged_attention_tokens)
and of single tokens (paged_attention), and the cut of the cache to the drafted
tokens that were accepted (cache_keep).

    python examples/draft_layer.py [--steps 50] [--drafted 25]

prints the cache lengths and the time of a step on one GPU."""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_block_bit_amd as gbb  # noqa: E402


def tree_of(parents):
    """Each new token's row: itself and its ancestors (parents[i] < i, -1 where
    the last cached token is the parent) -> bool [n][n]."""
    m = np.zeros((len(parents), len(parents)), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def tree_words(trees):
    """Trees of several sequences -> int32 [tokens][words]."""
    words = max(1, max(-(-len(t) // 32) for t in trees))
    rows = np.zeros((sum(len(t) for t in trees), 32 * words), bool)
    at = 0
    for t in trees:
        rows[at:at + len(t), :len(t)] = t
        at += len(t)
    return np.packbits(rows, axis=1, bitorder="little").view(np.int32)


class DraftLayer:
    """Attention of a pre-norm decoder layer for `batch` sequences of up to
    max_len slots."""

    def __init__(self, batch, q_heads, kv_heads, head_dim, max_len, page=64, bits=4.0, layout="half", softcap=0.0,
                 window=0, dtype=torch.float16, seed=0):
        self.batch, self.q_heads, self.kv_heads, self.head_dim = batch, q_heads, kv_heads, head_dim
        self.max_len, self.layout, self.scores = max_len, layout, dict(softcap=softcap, window=window)
        self.hidden = q_heads * head_dim
        g = np.random.default_rng(seed)

        def packed(n, k):
            w = (g.standard_normal((n, k)) / np.sqrt(k)).astype(np.float16)
            image, _, _ = gbb.pack_blocks(w, gbb.allocate_bits(w, bits))
            return torch.from_numpy(image).cuda()

        self.qkv_rows = (q_heads + 2 * kv_heads) * head_dim
        self.qkv, self.o = packed(self.qkv_rows, self.hidden), packed(self.hidden, self.hidden)
        self.q_norm, self.k_norm = (torch.from_numpy(g.uniform(0.5, 1.5, head_dim).astype(np.float32)).cuda() for _ in range(2))
        self.table = torch.from_numpy(gbb.rope_table(head_dim, max_len, 500000.0)).cuda()
        per = -(-max_len // page)
        scale = torch.full((kv_heads,), 8.0 / 448, device="cuda") if dtype == torch.float8_e4m3fn else None
        self.cache = gbb.PagedCache.empty(batch * per, page, kv_heads, head_dim, dtype, "cuda", False, scale, scale)
        self.pages = torch.from_numpy(g.permutation(batch * per).astype(np.int32)).view(batch, per)
        self.block_table = self.pages.cuda()
        self.lengths = [0] * batch

    def extend(self, x, new, trees=None):
        """x fp16 [sum(new)][hidden], new[b] tokens of sequence b one after the
        other, or where `trees` is given a tree of drafted ones each (tree_of)
        -> fp16 [sum(new)][hidden]."""
        page, T = self.cache.page, sum(new)
        slots, positions = [], []
        for b, n in enumerate(new):
            at = self.lengths[b] + np.arange(n)
            slots.append(self.pages[b].numpy()[at // page] * page + at % page)
            positions.append(self.lengths[b] + trees[b].sum(1) - 1 if trees else at)
            self.lengths[b] += n
        slots, positions, starts, lengths = (
            torch.from_numpy(np.asarray(a, np.int32)).cuda()
            for a in (np.concatenate(slots), np.concatenate(positions), np.cumsum([0] + list(new)), self.lengths))
        qkv = gbb.gemm_mixed_w(self.qkv, self.qkv_rows, self.hidden, x)
        q = gbb.rope_append(self.cache, qkv, self.q_heads, positions, slots, self.table, layout=self.layout,
                            q_norm=self.q_norm, k_norm=self.k_norm)
        if trees is None and set(new) == {1}:
            out = gbb.paged_attention(self.cache, q, self.block_table, lengths, self.max_len, **self.scores)
        else:
            tree = torch.from_numpy(tree_words(trees)).cuda() if trees else None
            out = gbb.paged_attention_tokens(self.cache, q, starts, self.block_table, lengths, self.max_len, tree=tree,
                                             **self.scores)
        return gbb.gemm_mixed_w(self.o, self.hidden, self.hidden, out.view(T, self.hidden))

    def keep(self, drafted, kept):
        """Of the drafted[b] newest tokens those numbered kept[b] stay."""
        most = max(1, max(len(k) for k in kept))
        rows = np.zeros((self.batch, most), np.int32)
        for b, k in enumerate(kept):
            rows[b, :len(k)] = k
        lengths, drafted_, rows, counts = (torch.from_numpy(np.asarray(a, np.int32)).cuda()
                                           for a in (self.lengths, drafted, rows, [len(k) for k in kept]))
        after = gbb.cache_keep(self.cache, self.block_table, lengths, drafted_, rows, counts)
        self.lengths = [n - d + len(k) for n, d, k in zip(self.lengths, drafted, kept)]
        return after


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafted", type=int, default=25)
    a = ap.parse_args()
    g = np.random.default_rng(1)
    new = [int(n) for n in g.integers(100, 1000, a.batch)]
    layer = DraftLayer(a.batch, 32, 8, 128, max(new) + (a.steps + 1) * a.drafted)
    noise = torch.Generator(device="cuda").manual_seed(1)
    layer.extend(torch.randn(sum(new), layer.hidden, generator=noise, device="cuda").half(), new)
    x = torch.randn(a.batch * a.drafted, layer.hidden, generator=noise, device="cuda").half()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    accepted = 0
    for i in range(a.steps + 1):
        if i == 1:
            t[0].record()
        trees = [tree_of([-1] + [int(g.integers(0, j)) for j in range(1, a.drafted)]) for _ in range(a.batch)]
        y = layer.extend(x, [a.drafted] * a.batch, trees)
        # as if the path to one of the drafted tokens were the one accepted
        kept = [np.flatnonzero(tree[int(g.integers(a.drafted))]) for tree in trees]
        layer.keep([a.drafted] * a.batch, kept)
        accepted += sum(len(k) for k in kept)
        if i % 10 == 0:
            print(f"step {i}: lengths {layer.lengths}, |y| {y.float().norm().item():.3f}", flush=True)
    t[1].record()
    torch.cuda.synchronize()
    print(f"{t[0].elapsed_time(t[1]) / max(1, a.steps) * 1e3:.1f} us a step, {accepted / (a.steps + 1) / a.batch:.2f} tokens "
          f"a step and sequence")


if __name__ == "__main__":
    main()
