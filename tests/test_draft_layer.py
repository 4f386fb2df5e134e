"""The example's layer, call by call against the 64-bit oracle on the state each
call starts from: ragged prompts, trees of drafted tokens, the cut to the kept
ones and single tokens together, with norms of the q and k heads."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import new_tokens as on

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("draft_layer", os.path.join(ROOT, "examples", "draft_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trees_as_words():
    m = example()
    tree = m.tree_of([-1, 0, 0, 2, -1])
    assert tree.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]]
    chain = np.tril(np.ones((40, 40), bool))
    words = m.tree_words([tree, chain]).view(np.uint32)
    assert words.shape == (45, 2) and words[3].tolist() == [0b1101, 0]
    assert words[5].tolist() == [1, 0] and words[44].tolist() == [2 ** 32 - 1, 255]


@pytest.mark.gpu
@pytest.mark.parametrize("options", [dict(), dict(layout="interleaved", softcap=4.0), dict(window=20),
                                     dict(dtype=torch.float8_e4m3fn)], ids=str)
def test_layer_against_oracle(options):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    m = example()
    B, hq, hkv, D, page = 3, 4, 2, 64, 16
    layer = m.DraftLayer(B, hq, hkv, D, 200, page=page, **options)
    c, bt, eps = layer.cache, layer.pages.numpy(), 1e-6
    es = {1: torch.uint8, 2: torch.int16}[c.k.element_size()]
    unit = 2.0 ** -4 if es is torch.uint8 else 2.0 ** -11
    scales = np.ones(hkv) if c.k_scale is None else c.k_scale.double().cpu().numpy()
    wide = lambda t: t.double().cpu().numpy() * scales[None, :, None, None]  # noqa: E731
    wo = gbb.dequant(layer.o, layer.hidden, layer.hidden)[1].double().cpu().numpy()
    norms = [w.double().cpu().numpy() for w in (layer.q_norm, layer.k_norm)]
    table = layer.table.double().cpu().numpy()
    g = np.random.default_rng(3)

    def extend(new, trees=None):
        T, before, was = sum(new), list(layer.lengths), [t.clone() for t in (c.k, c.v)]
        x = torch.from_numpy(g.standard_normal((T, layer.hidden)).astype(np.float16)).cuda()
        qkv = gbb.gemm_mixed_w(layer.qkv, layer.qkv_rows, layer.hidden, x).double().cpu().numpy().reshape(T, hq + 2 * hkv, D)
        y = layer.extend(x, new, trees).double().cpu().numpy()
        assert layer.lengths == [a + n for a, n in zip(before, new)]
        at = np.concatenate([a + np.arange(n) for a, n in zip(before, new)])
        pos = np.concatenate([a + (t.sum(1) - 1 if trees else np.arange(n))
                              for a, n, t in zip(before, new, trees or new)])
        q, k = (on.norm_rope(h, w, eps, pos[None], [D // 2], table, layer.layout)
                for h, w in ((qkv[:, :hq], norms[0]), (qkv[:, hq:hq + hkv], norms[1])))
        of = np.repeat(np.arange(B), new)
        pg, off = bt[of, at // page], at % page
        # the new slots hold the tokens (one rounding; 2^-16 covers the fp32 before
        # it, 2^-6 scale the smallest e4m3 steps), and no others changed
        kw, vw = wide(c.k), wide(c.v)
        for got, ref in ((kw[pg, :, off], k), (vw[pg, :, off], qkv[:, hq + hkv:])):
            floor = (0 if es is torch.int16 else 2.0 ** -10) * scales.max()
            assert np.all(np.abs(got - ref) <= unit * np.abs(ref) * (1 + 2.0 ** -10) + 2.0 ** -16 * np.abs(ref).max() + floor)
        same = torch.ones(c.k.shape[:3], dtype=torch.bool, device="cuda")
        same[torch.from_numpy(pg).cuda().long(), :, torch.from_numpy(off).cuda()] = False
        assert all(torch.equal(t.view(es)[same], o.view(es)[same]) for t, o in zip((c.k, c.v), was))
        # attention over the cache as it is: q's own rounding moves a score by at
        # most 2^-11 of sum |q k| (2^-10 with all that is smaller), an output by
        # twice that of sum p |v|, and the roundings of P and of the output add 2^-10
        starts = np.cumsum([0] + list(new)).tolist()
        bits = None
        if trees:
            bits = np.zeros((T, max(new)), bool)
            for b, t in enumerate(trees):
                bits[starts[b]:starts[b + 1], :new[b]] = t
        out, _, mass, parts = on.attention_tokens(q, kw, vw, starts, bt, layer.lengths, D ** -0.5, tree=bits, **layer.scores)
        e = (2.0 ** -9 * parts[0][..., None] + 2.0 ** -10) * mass
        ref = out.reshape(T, -1) @ wo.T
        # the o product: exact terms, its output's rounding, and its bar of 2e-3
        tol = e.reshape(T, -1) @ np.abs(wo).T + 2e-3 * np.abs(ref).max()
        assert np.all(np.abs(y - ref) <= tol), np.max(np.abs(y - ref) / tol)

    def keep(drafted, kept):
        arrays, lengths = [t.view(es).cpu().numpy() for t in (c.k, c.v)], list(layer.lengths)
        most = max(1, max(len(k) for k in kept))
        rows = np.zeros((B, most), np.int64)
        for b, k in enumerate(kept):
            rows[b, :len(k)] = k
        want, after = on.cache_keep(arrays, bt, lengths, drafted, rows, [len(k) for k in kept], bt.size, page)
        assert layer.keep(drafted, kept).tolist() == after == layer.lengths
        for t, w in zip((c.k, c.v), want):
            assert np.array_equal(t.view(es).cpu().numpy(), w)

    extend([37, 5, 60])                          # ragged prompts
    extend([0, 20, 3])                           # a chunk more of two of them
    for _ in range(3):
        new = [7, 12, 1]
        trees = [m.tree_of([-1] + [int(g.integers(-1, j)) for j in range(1, n)]) for n in new]
        extend(new, trees)
        keep(new, [np.flatnonzero(t[int(g.integers(len(t)))]) for t in trees])
        extend([1, 1, 1])
    keep([1, 1, 1], [[], [0], []])               # a token taken back
    extend([1, 1, 1])
