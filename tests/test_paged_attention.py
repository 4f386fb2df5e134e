"""Attention of one new token over the paged cache against the 64-bit oracle.

Tolerances, per output element.  With e the largest error of a score, P = sum
p |v| (p normalised) and n slots: a probability is off by a factor of at most
1 + 2 e + 2^-20 (its own and the normalisation's exponentials) and, as the
matrix cores' operand, by 2^-16 (bf16 in two parts; fp16 in two is finer);
sums of n terms in fp32 add n 2^-24.  So before the output's own rounding the
error is at most (2 e + 2^-16 + 2^-19 + 2 n 2^-24) P.  A score is a sum of D
exact products in fp32, e <= (D + 4) 2^-24 scale sum |q k| + 2^-20: the last
term is the rounding of a score below 2^4 in the exponent's base 2."""
import ctypes

import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


class Setup:
    """A cache of random keys and values with pages in no order, unused memory
    filled with NaN (every code of it, e4m3 included)."""

    def __init__(self, lengths, hq, hkv, D, dt="f16", ct="f16", page=16, seed=0, tracked=False, max_len=None, spare=2):
        g = np.random.default_rng(seed)
        self.lengths, self.hq, self.dt, self.D = list(lengths), hq, dt, D
        self.max_len = max_len or max(1, max(lengths))
        per = -(-self.max_len // page)
        used = [-(-max(0, n) // page) for n in lengths]
        pages = max(1, sum(used)) + spare
        order = g.permutation(pages)
        bt = np.full((len(lengths), per), 2 ** 31 - 1, np.int64)   # what is not used is never looked at
        at = 0
        for b, n in enumerate(used):
            bt[b, :n] = order[at:at + n]
            at += n
        self.bt = bt.astype(np.int32)
        nan = torch.full((pages, hkv, page, D), float("nan"))
        self.kw = {}
        if ct == "e4m3":
            self.ks, self.vs = g.uniform(0.01, 0.03, hkv).astype(np.float32), g.uniform(0.01, 0.03, hkv).astype(np.float32)
            self.kw = dict(k_scale=torch.from_numpy(self.ks).to(dev()), v_scale=torch.from_numpy(self.vs).to(dev()))
        else:
            self.ks = self.vs = np.ones(hkv, np.float32)
        k, v = nan.clone(), nan.clone()
        for b, n in enumerate(lengths):
            for j in range(max(0, n)):
                p, o = self.bt[b, j // page], j % page
                k[p, :, o] = torch.from_numpy(g.standard_normal((hkv, D)).astype(np.float32) / self.ks[:, None])
                v[p, :, o] = torch.from_numpy(g.standard_normal((hkv, D)).astype(np.float32) / self.vs[:, None])
        clamp = (lambda x: torch.clamp(x, -448, 448)) if ct == "e4m3" else (lambda x: x)   # keeps NaN
        self.k, self.v = clamp(k).to(DT[ct]), clamp(v).to(DT[ct])
        self.q = torch.from_numpy((2 * g.standard_normal((len(lengths), hq, D))).astype(np.float32)).to(DT[dt])
        w = torch.from_numpy(g.random((pages, hkv, page)).astype(np.float32)) if tracked else None
        self.w = w
        self.cache = gbb.PagedCache(self.k.to(dev()), self.v.to(dev()), weights=None if w is None else w.to(dev()), **self.kw)
        self.btd = torch.from_numpy(self.bt).to(dev())
        self.lend = torch.tensor(lengths, dtype=torch.int32, device=dev())

    def run(self, **kw):
        return gbb.paged_attention(self.cache, self.q.to(dev()), self.btd, self.lend, self.max_len, **kw)

    def wide(self):
        k = np.nan_to_num(self.k.double().numpy()) * self.ks[None, :, None, None].astype(np.float64)
        v = np.nan_to_num(self.v.double().numpy()) * self.vs[None, :, None, None].astype(np.float64)
        return self.q.double().numpy(), k, v

    def oracle(self, scale=None):
        q, k, v = self.wide()
        scale = self.D ** -0.5 if scale is None else scale
        lens = [min(max(0, n), self.max_len) for n in self.lengths]
        out, lse, w, mass, dots = od.paged_attention(q, k, v, self.bt, lens, scale)
        e = (self.D + 4) * 2.0 ** -24 * abs(scale) * dots + 2.0 ** -20
        n = np.array(lens)[:, None]
        return out, lse, w, mass, e, n

    def check(self, got, scale=None, lse=None, weights=None):
        out, ref_lse, w, mass, e, n = self.oracle(scale)
        pre = (2 * e + 2.0 ** -16 + 2.0 ** -19 + 2 * n * 2.0 ** -24)[..., None] * mass
        tol = pre + UNIT[self.dt] * (np.abs(out) + pre) + 2.0 ** -25
        got = got.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - out) <= tol), np.max(np.abs(got - out) / tol)
        if lse is not None:
            x = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(x), np.isneginf(ref_lse))
            some = ~np.isneginf(ref_lse)
            bound = (e + n * 2.0 ** -24 + 2.0 ** -20)[some] + 2.0 ** -22 * np.abs(ref_lse[some])
            assert np.all(np.abs(x[some] - ref_lse[some]) <= bound)
        if weights is not None:
            # a probability's relative error, summed over the query heads, and the sum's rounding
            got_w, base = weights.double().cpu().numpy(), self.w.double().numpy()
            rel = float((2 * e + n * 2.0 ** -24 + 2.0 ** -19).max()) if e.size else 0.0
            group = self.hq // self.cache.kv_heads
            assert np.all(np.abs(got_w - base - w) <= rel * w + (group + 1) * 2.0 ** -24 * (base + w))
            assert np.array_equal(got_w[w == 0], base[w == 0])


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 300]


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 64, 256])
def test_lengths_around_tiles_and_pages(page, D, dt, ct):
    s = Setup(LENGTHS, 4, 2, D, dt, ct, page, seed=page + D)
    lse = torch.zeros(len(LENGTHS), 4, device=dev())
    got = s.run(lse=lse)
    s.check(got, lse=lse)
    assert not got[0].any()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (3, 1), (5, 1), (16, 2), (14, 2), (16, 1), (17, 1), (40, 1), (96, 2), (128, 1)])
def test_groups(hq, hkv, dt, ct):
    s = Setup([70, 0, 129, 400], hq, hkv, 64, dt, ct, 32, seed=hq, tracked=True)
    lse, w = torch.zeros(4, hq, device=dev()), s.w.to(dev())
    s.check(s.run(lse=lse, weights_out=w), lse=lse, weights=w)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [5000], [4097, 3, 0, 2600], [9000] * 3])
def test_split_and_joined(lengths, D, dt, ct):
    """Contexts of many runs, with and without weights; out of place, then in
    place, give the same bits."""
    s = Setup(lengths, 4, 1, D, dt, ct, 64, seed=len(lengths) + D, tracked=True)
    lse, w = torch.zeros(len(lengths), 4, device=dev()), s.w.to(dev())
    got = s.run(lse=lse)
    s.check(got, lse=lse)
    both = s.run(weights_out=w)
    s.check(both, weights=w)
    assert torch.equal(both, got)
    s.run(weights_out=s.cache.weights)
    assert torch.equal(s.cache.weights, w)


@pytest.mark.gpu
def test_pages_that_are_not_there():
    """Missing pages, negative or too large, inside and at both ends, and a
    sequence of nothing else."""
    s = Setup([200, 90, 64, 33], 4, 2, 128, page=16, seed=3, tracked=True)
    s.bt[0, 0], s.bt[0, 5], s.bt[0, 12] = -1, s.k.shape[0], -2 ** 31
    s.bt[1, 1:3] = 2 ** 31 - 1
    s.bt[2, :] = -1
    s.btd = torch.from_numpy(s.bt).to(dev())
    lse, w = torch.zeros(4, 4, device=dev()), s.w.to(dev())
    got = s.run(lse=lse, weights_out=w)
    s.check(got, lse=lse, weights=w)
    assert not got[2].any() and torch.isneginf(lse[2]).all()


@pytest.mark.gpu
def test_lengths_are_clamped():
    s = Setup([64, 0, 64], 2, 1, 64, page=16, seed=4)
    s.lend = torch.tensor([2 ** 31 - 1, -7, 64], dtype=torch.int32, device=dev())
    s.check(s.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 40.0])
def test_scales(scale, dt):
    """Uniform, peaked and reversed probabilities.  The tolerance's 2^-20 is
    that of a score below 2^4; a larger one is rounded to 2^-24 of itself."""
    s = Setup([1, 40, 700], 4, 2, 64, dt, dt, seed=6)
    got = s.run(scale=scale)
    out, _, _, mass, e, n = s.oracle(scale)
    q, k, _ = s.wide()
    biggest = abs(scale) * np.abs(q).sum(-1).max() * np.abs(k).max()
    pre = (2 * e + 2.0 ** -23 * biggest + 2.0 ** -16 + 2.0 ** -19 + 2 * n * 2.0 ** -24)[..., None] * mass
    tol = pre + UNIT[dt] * (np.abs(out) + pre) + 2.0 ** -25
    assert np.all(np.abs(got.double().cpu().numpy() - out) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_small_probabilities_are_kept(dt):
    """One slot far above 4000 equal ones that carry a third of the mass
    together, each 2^-13: what they add must not be lost to a 16-bit operand."""
    n, D = 4001, 64
    s = Setup([n], 1, 1, D, dt, dt, page=64, seed=8)
    k = torch.zeros_like(s.k)
    p, o = s.bt[0, 7], 5
    k[p, 0, o, 0] = 8.0
    s.k = k
    s.q.zero_()
    s.q[0, 0, 0] = 8.0 * np.log(2.0) * 13 / 8   # score 9.0 after the 1/8 scale: about 2^13 of the rest
    s.cache.k.copy_(k.to(dev()))
    s.check(s.run())


@pytest.mark.gpu
def test_infinities_and_nan():
    d = dev()
    s = Setup([40, 40, 40, 40], 1, 1, 64, page=16, seed=9)
    s.q[:, 0, 0] = 1.0
    k = s.cache.k
    at = lambda b, j: (int(s.bt[b, j // 16]), 0, j % 16)  # noqa: E731
    for j in range(40):   # all scores -inf: zeros
        k[at(0, j)] = 0.0
        k[at(0, j)][0] = float("-inf")
    k[at(1, 20)][0] = float("-inf")    # one score -inf: that slot takes no part
    k[at(2, 20)][0] = float("nan")     # one score NaN: the sequence is NaN
    k[at(3, 20)][0] = float("inf")     # one score +inf: inf - inf, NaN as in any softmax
    lse = torch.zeros(4, 1, device=d)
    got = s.run(lse=lse)
    assert not got[0].any() and torch.isneginf(lse[0]).all()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    q, kk, v = s.wide()
    j = np.array([x for x in range(40) if x != 20])
    kk, v = kk[s.bt[1][j // 16], 0, j % 16], v[s.bt[1][j // 16], 0, j % 16]
    sc = kk @ q[1, 0] / 8
    p = np.exp(sc - sc.max())
    ref = p @ v / p.sum()
    assert np.abs(got[1, 0].double().cpu().numpy() - ref).max() <= 2.0 ** -11 * 4 + 2.0 ** -12


@pytest.mark.gpu
def test_strided_queries_given_outputs_streams_and_repeats():
    """q inside a wider row, an output and a workspace of the caller, another
    stream: the same bits each time."""
    d = dev()
    s = Setup([700, 33, 0, 1500], 8, 2, 128, "bf16", "bf16", 32, seed=10, tracked=True)
    first = s.run()
    s.check(first)
    wide = torch.randn(4, 8 * 128 + 64, device=d).bfloat16()
    q = wide[:, 32:32 + 1024].unflatten(1, (8, 128))
    q.copy_(s.q)
    need = gbb.paged_attention_workspace(s.cache, 4, 8, s.max_len, True)
    ws = torch.zeros(need, dtype=torch.uint8, device=d)
    out, w = torch.full_like(first, float("nan")), s.w.to(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            assert gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len, out=out, weights_out=w, workspace=ws) is out
    side.synchronize()
    assert torch.equal(out, first)
    s.check(out, weights=w)
    for bad in (0, need - 1):
        with pytest.raises(gbb.GbbError) as e:
            gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len, weights_out=w, workspace=ws[:bad])
        assert e.value.status in (-1, -5)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_all_sizes():
    d = dev()
    a = Setup([3000], 4, 1, 128, seed=11, page=64, tracked=True)
    b = Setup([20, 5000, 7], 6, 2, 64, seed=12, page=16, tracked=True)
    size = max(gbb.paged_attention_workspace(a.cache, 1, 4, 3000, True), gbb.paged_attention_workspace(b.cache, 3, 6, 5000, True))
    ws = torch.zeros(size, dtype=torch.uint8, device=d)
    for _ in range(3):
        for s in (a, b):
            w = s.w.to(d)
            s.check(s.run(workspace=ws), None)
            s.check(s.run(workspace=ws, weights_out=w), weights=w)


@pytest.mark.gpu
def test_in_a_graph():
    """Captured once, replayed with other queries, lengths and pages, with
    eager work between the replays."""
    d = dev()
    s = Setup([900, 40], 4, 2, 64, seed=13, page=32, tracked=True)
    q, out, w = s.q.to(d), torch.empty(2, 4, 64, device=d, dtype=torch.float16), s.w.to(d)
    ws = torch.zeros(gbb.paged_attention_workspace(s.cache, 2, 4, s.max_len, True), dtype=torch.uint8, device=d)
    call = lambda: gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len, out=out, weights_out=w, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(4):
        s.q = torch.roll(s.q, 1, 0) * (1 - i / 8)
        s.lengths = [900 - 211 * i, 40 - 13 * i]
        q.copy_(s.q)
        s.lend.copy_(torch.tensor(s.lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        s.check(out, weights=w)
        eager_w = s.w.to(d)
        assert torch.equal(s.run(weights_out=eager_w), out) and torch.equal(eager_w, w)
        w.copy_(s.w)


@pytest.mark.gpu
def test_a_capture_keeps_its_workspace_to_itself(monkeypatch):
    """Captured without a workspace: replays beside eager calls give the eager
    bits, and nothing of the graph's memory stays for calls outside it."""
    s = Setup([900, 40], 4, 2, 64, seed=14)
    q, out = s.q.to(dev()), torch.zeros(2, 4, 64, device=dev(), dtype=torch.float16)
    kept = {}
    monkeypatch.setattr(gbb.paged, "_ws_cache", kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len, out=out)
    assert not kept
    for i in range(4):
        s.q = torch.roll(s.q, 1, 0) * (1 - i / 8)
        q.copy_(s.q)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(out)
        assert torch.equal(s.run(), out)


@pytest.mark.gpu
def test_one_head_of_any_stride():
    """The stride of a dimension of one element says nothing."""
    s = Setup([70, 5], 1, 1, 64, seed=15)
    first = s.run()
    q = s.q.to(dev()).as_strided((2, 1, 64), (64, 7, 1))
    assert torch.equal(gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len), first)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Pages whose byte offsets pass 2^32 in a cache of 6 GiB a side."""
    d = dev()
    D, page, pages = 128, 64, 400000
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory")
    k = torch.empty(pages, 1, page, D, dtype=torch.float16, device=d)
    v = torch.empty(pages, 1, page, D, dtype=torch.float16, device=d)
    s = Setup([200], 4, 1, D, page=page, seed=14, tracked=True)
    far = torch.tensor([pages - 1, 0, 262144 + 3, 399000], dtype=torch.int64)
    for i, p in enumerate(far.tolist()):
        k[p], v[p] = s.cache.k[int(s.bt[0, i])], s.cache.v[int(s.bt[0, i])]
    big = gbb.PagedCache(k, v)
    got = gbb.paged_attention(big, s.q.to(d), far.to(torch.int32).to(d)[None], s.lend, 200)
    assert torch.equal(got, s.run())
    # and the write of a token there
    table = torch.from_numpy(gbb.rope_table(128, 4)).to(d)
    qkv = torch.randn(1, 6 * 128, device=d, dtype=torch.float16)
    slot = torch.tensor([(pages - 1) * page + 63], dtype=torch.int32, device=d)
    gbb.rope_append(big, qkv, 4, torch.zeros(1, dtype=torch.int32, device=d), slot, table)
    assert torch.equal(v[-1, 0, 63], qkv[0, 640:]) and torch.equal(k[-1, 0, 63], qkv[0, 512:640])


def test_argument_refusals():
    """Checked before anything touches a device."""
    L, C = gbb.lib(), gbb.binding._PagedCache
    base = dict(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4,
                page=16, kv_heads=2, head_dim=64)

    def call(c=None, q=8 << 20, qt=256, dt=0, B=2, hq=4, bt=9 << 20, mp=4, ln=10 << 20, ml=64, sc=1.0, o=11 << 20, lse=None,
             w=None, ws=1 << 24, wb=1 << 30):
        cc = C(**{**base, **(c or {})})
        return L.gbb_paged_attention(ctypes.byref(cc), q, qt, dt, B, hq, bt, mp, ln, ml, sc, o, lse, w, ws, wb, None)

    assert call(B=0) == 0
    for bad in (dict(c=dict(v=None)), dict(c=dict(dtype=2)), dict(dt=3), dict(dt=1), dict(B=-1), dict(ml=0), dict(mp=0),
                dict(sc=float("nan")), dict(q=None), dict(o=None), dict(bt=None), dict(ln=None), dict(w=64),
                dict(o=8 << 20), dict(c=dict(v_scale=64))):
        assert call(**bad) == -1, bad
    for bad in (dict(c=dict(page=8)), dict(c=dict(head_dim=32)), dict(hq=5), dict(hq=2 * 129), dict(ml=65), dict(qt=128),
                dict(B=1 << 22), dict(c=dict(kv_heads=1 << 15), hq=1 << 15)):
        assert call(**bad) == -2, bad
    for bad in (dict(q=(8 << 20) + 2), dict(o=(11 << 20) + 8), dict(qt=260), dict(lse=2), dict(bt=(9 << 20) + 1)):
        assert call(**bad) == -4, bad
    long = dict(mp=64, ml=1024, c=dict(num_pages=64))
    assert call(ws=None, **long) == -1
    assert call(wb=16, **long) == -5
    assert call(ws=(1 << 24) + 8, **long) == -4
    cc = C(**base)
    assert L.gbb_paged_attention_workspace(ctypes.byref(cc), 2, 5, 64, 0) == 0
    assert L.gbb_paged_attention_workspace(None, 2, 4, 64, 0) == 0
    small, big = (L.gbb_paged_attention_workspace(ctypes.byref(cc), 2, 4, 10000, w) for w in (0, 1))
    assert 0 < small < big


def test_weights_out_that_overlaps_in_part_is_refused():
    L, C = gbb.lib(), gbb.binding._PagedCache
    w = 3 << 20   # never read; 4 pages of 2 kv heads of 16 slots: 512 bytes
    c = C(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=w, positions=None, dtype=0, num_pages=4, page=16,
          kv_heads=2, head_dim=64)
    for at in (w + 4, w + 508, w - 508):
        assert L.gbb_paged_attention(ctypes.byref(c), 8 << 20, 256, 0, 2, 4, 9 << 20, 4, 10 << 20, 64, 1.0, 11 << 20,
                                     None, at, 1 << 24, 1 << 30, None) == -1
