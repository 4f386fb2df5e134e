"""Attention of several new tokens per sequence over the paged cache, and of
single ones with capped, biased or windowed scores, against the 64-bit oracle.

Tolerances, per output element, with u = 2^-24, P = sum p |v| and n slots.  A
score is a sum of D exact products in fp32: (D + 4) u scale sum |q k|; a cap adds
at most 2^-21 of itself, a bias and the exponent's base 2 two roundings of the
largest score and bias: 4 u (|s| + bias) + 2^-20.  With e the sum of these a
probability is off by a factor of at most 1 + 2 e + 2^-19; as the matrix cores'
operand it is rounded once to the type of q (half a step, 2^-11 or 2^-8), or in
calls of few rows carries 16 bits or more; sums of n terms add 2 n u.  So
before the output's own rounding the error is at most (2 e + half a step + 2^-18
+ 2 n u) P."""
import ctypes

import numpy as np
import pytest

from oracle import new_tokens as on

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]
U = 2.0 ** -24


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def random_tree(g, n):
    """bool [n][n]: ancestors and itself."""
    m = np.zeros((n, n), bool)
    for i in range(n):
        parent = int(g.integers(-1, i))
        if parent >= 0:
            m[i] = m[parent]
        m[i, i] = True
    return m


def words_of(bits, words):
    """bool [T][any] -> int32 [T][words]."""
    out = np.zeros((bits.shape[0], words), np.uint32)
    for j in range(min(bits.shape[1], 32 * words)):
        out[:, j // 32] |= bits[:, j].astype(np.uint32) << np.uint32(j % 32)
    return out.view(np.int32)


class Setup:
    """Contexts and new tokens of several sequences in a cache with pages in no
    order, unused memory filled with NaN.  gap: tokens before, between the last
    and the end that belong to nobody."""

    def __init__(self, context, new, hq, hkv, D, dt="f16", ct="f16", page=16, seed=0, gap=(0, 0), q_scale=2.0, **options):
        g = np.random.default_rng(seed)
        self.hq, self.hkv, self.D, self.dt, self.ct, self.page = hq, hkv, D, dt, ct, page
        self.new = list(new)
        self.lengths = [c + n for c, n in zip(context, new)]
        self.max_len = max(1, max(self.lengths))
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32) + gap[0]
        self.T = int(self.starts[-1]) + gap[1]
        per = -(-self.max_len // page)
        used = [-(-n // page) for n in self.lengths]
        pages = max(1, sum(used)) + 2
        order = g.permutation(pages)
        bt, at = np.full((len(new), per), 2 ** 31 - 1, np.int64), 0
        for b, n in enumerate(used):
            bt[b, :n] = order[at:at + n]
            at += n
        self.bt = bt.astype(np.int32)
        self.ks = self.vs = np.ones(hkv, np.float32)
        self.kw = {}
        if ct == "e4m3":
            self.ks, self.vs = g.uniform(0.01, 0.03, hkv).astype(np.float32), g.uniform(0.01, 0.03, hkv).astype(np.float32)
            self.kw = dict(k_scale=torch.from_numpy(self.ks).to(dev()), v_scale=torch.from_numpy(self.vs).to(dev()))
        k, v = np.full((2, pages, hkv, page, D), np.nan, np.float32)
        for b, n in enumerate(self.lengths):
            j = np.arange(n)
            for x, s in ((k, self.ks), (v, self.vs)):
                x[self.bt[b, j // page], :, j % page] = g.standard_normal((n, hkv, D)) / s[None, :, None]
        clamp = (lambda x: torch.clamp(x, -448, 448)) if ct == "e4m3" else (lambda x: x)
        self.k, self.v = (clamp(torch.from_numpy(x)).to(DT[ct]) for x in (k, v))
        self.q = torch.from_numpy((q_scale * g.standard_normal((self.T, hq, D))).astype(np.float32)).to(DT[dt])
        self.options, self.g = options, g
        self.to_device()

    def to_device(self):
        d = dev()
        self.cache = gbb.PagedCache(self.k.to(d), self.v.to(d), **self.kw)
        self.btd, self.qd = torch.from_numpy(self.bt).to(d), self.q.to(d)
        self.lend = torch.tensor(self.lengths, dtype=torch.int32, device=d)
        self.startd = torch.from_numpy(self.starts).to(d)

    def arguments(self):
        d, o = dev(), {}
        for name, x in self.options.items():
            if name == "tree":
                bits, words = x
                o[name] = torch.from_numpy(words_of(bits, words)).to(d)
            elif isinstance(x, np.ndarray):
                o[name] = torch.from_numpy(x.astype(np.float32 if name == "slopes" else np.int32)).to(d)
            else:
                o[name] = x
        return o

    def run(self, **kw):
        return gbb.paged_attention_tokens(self.cache, self.qd, self.startd, self.btd, self.lend, self.max_len,
                                          **{**self.arguments(), **kw})

    def wide(self):
        k = np.nan_to_num(self.k.double().numpy()) * self.ks[None, :, None, None].astype(np.float64)
        v = np.nan_to_num(self.v.double().numpy()) * self.vs[None, :, None, None].astype(np.float64)
        return self.q.double().numpy(), k, v

    def oracle(self):
        q, k, v = self.wide()
        o = dict(self.options)
        scale = o.pop("scale", self.D ** -0.5)
        if "tree" in o:
            bits, words = o["tree"]
            o["tree"] = bits[:, :32 * words]
        if "slopes" in o:
            o["slopes"] = o["slopes"].astype(np.float32).astype(np.float64)
        return on.attention_tokens(q, k, v, self.starts.tolist(), self.bt, self.lengths, scale, **o)

    def check(self, got, lse=None, ref=None):
        out, ref_lse, mass, (dots, scores, bias) = ref or self.oracle()
        mine = ~np.isnan(ref_lse[:, 0])
        e = (self.D + 4) * U * dots + 2.0 ** -21 * self.options.get("softcap", 0.0) + 4 * U * (scores + bias) + 2.0 ** -20
        n = 2 * self.max_len * U
        pre = (2 * e + UNIT[self.dt] + 2.0 ** -18 + n)[..., None] * mass
        tol = pre + UNIT[self.dt] * (np.abs(out) + pre) + 2.0 ** -25
        got = got.double().cpu().numpy()
        assert np.all(np.isfinite(got[mine]))
        bad = np.abs(got[mine] - out[mine]) > tol[mine]
        assert not bad.any(), (np.argwhere(bad)[:4], np.max(np.abs(got[mine] - out[mine]) / tol[mine]))
        if lse is not None:
            x = lse.double().cpu().numpy()
            assert np.array_equal(np.isneginf(x[mine]), np.isneginf(ref_lse[mine]))
            some = mine[:, None] & ~np.isneginf(ref_lse)
            bound = (e + n + 2.0 ** -19)[some] + 2.0 ** -22 * np.abs(ref_lse[some])
            assert np.all(np.abs(x[some] - ref_lse[some]) <= bound)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_tokens_and_contexts_around_tiles(page, D, dt, ct):
    context = [0, 0, 1, 15, 16, 31, 63, 64, 65, 0, 130, 7]
    new = [1, 33, 2, 17, 16, 1, 3, 32, 31, 0, 5, 64]
    s = Setup(context, new, 4, 2, D, dt, ct, page, seed=page + D)
    lse = torch.zeros(s.T, 4, device=dev())
    s.check(s.run(lse=lse), lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("new", [1, 2, 7, 8, 9, 40, 130])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (5, 1), (14, 2), (40, 1), (128, 1)])
def test_groups_and_rows(hq, hkv, new, dt, ct):
    """Every number of waves, rows that end anywhere in a tile."""
    s = Setup([70, 3], [new, max(1, new // 2)], hq, hkv, 64, dt, ct, 32, seed=hq + new)
    lse = torch.zeros(s.T, hq, device=dev())
    s.check(s.run(lse=lse), lse)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,ct", PAIRS)
def test_split_over_the_slots(dt, ct, D):
    """Few rows behind long contexts: runs of slots and their join."""
    for context, new, hkv in (([3000], [5], 1), ([2500, 0, 700], [40, 1, 3], 2), ([4100], [300], 1)):
        s = Setup(context, new, 4, hkv, D, dt, ct, 64, seed=D + len(new))
        lse = torch.zeros(s.T, 4, device=dev())
        first = s.run(lse=lse)
        s.check(first, lse)
        again = torch.zeros_like(lse)
        assert torch.equal(s.run(lse=again), first) and torch.equal(again, lse)


@pytest.mark.gpu
def test_a_chunk_of_a_prompt_is_the_prompt():
    """A prompt at once, in two chunks, and token by token with the single
    token's operator: the same values up to the rounding of probabilities."""
    s = Setup([0], [200], 4, 2, 128, "f16", "f16", 32, seed=1)
    whole = s.run()
    s.check(whole)
    late = gbb.paged_attention_tokens(s.cache, s.qd[77:], torch.tensor([0, 123], dtype=torch.int32, device=dev()), s.btd,
                                      s.lend, 200)
    one = torch.cat([gbb.paged_attention(s.cache, s.qd[i:i + 1], s.btd, torch.tensor([i + 1], dtype=torch.int32, device=dev()),
                                         200) for i in (0, 1, 150)])
    bound = 2 * (2.0 ** -11 + 2.0 ** -17) * 8   # two roundings each of P and the output, |v| below 8 or so
    assert (late.double() - whole[77:].double()).abs().max() <= bound
    assert (one.double() - whole[[0, 1, 150]].double()).abs().max() <= bound


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,new", [(2, 2, [90, 3, 17]), (8, 1, [7, 0, 2]), (4, 1, [10, 40, 0])])
def test_masks(hq, hkv, new, dt):
    """Every mask alone and together, rows that see nothing among them."""
    context = [100, 40, 0]
    T = sum(new)
    g = np.random.default_rng(T)
    lengths = np.array(context) + np.array(new)
    of = np.repeat(np.arange(3), new)
    first = g.integers(-5, lengths.max() + 20, T)
    first[: T // 3] = 30
    prefix = np.array([120, 43, 2 ** 31 - 1])
    slopes = 2.0 ** -np.arange(1, hq + 1)
    for o in (dict(first=first), dict(prefix=prefix), dict(window=1), dict(window=33), dict(window=2 ** 31 - 1),
              dict(first=first, prefix=prefix), dict(prefix=prefix, window=20), dict(slopes=slopes),
              dict(softcap=5.0), dict(softcap=500.0), dict(softcap=30.0, slopes=slopes, first=first, prefix=prefix, window=50),
              dict(first=np.full(T, 2 ** 31 - 1)), dict(first=(lengths[of] - 1))):
        s = Setup(context, new, hq, hkv, 64, dt, dt, 16, seed=len(o), **o)
        lse = torch.zeros(T, hq, device=dev())
        got = s.run(lse=lse)
        s.check(got, lse)
    assert s.options["first"] is not None


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_trees(D, dt, ct):
    context, new = [37, 0, 130, 64], [25, 70, 1, 33]
    g = np.random.default_rng(D)
    bits = np.zeros((sum(new), max(new)), bool)
    at = 0
    for n in new:
        bits[at:at + n, :n] = random_tree(g, n)
        bits[at:at + n, n:] = g.random((n, max(new) - n)) < 0.5    # bits past the sequence's tokens do not count
        at += n
    slopes = 2.0 ** -np.arange(1, 5)
    for o in (dict(), dict(slopes=slopes), dict(window=5), dict(window=40, slopes=slopes, softcap=20.0),
              dict(first=g.integers(0, 150, sum(new)))):
        for words in (3, 4):
            s = Setup(context, new, 4, 2, D, dt, ct, 32, seed=D + words, tree=(bits, words), **o)
            lse = torch.zeros(s.T, 4, device=dev())
            s.check(s.run(lse=lse), lse)
    s = Setup(context, new, 4, 2, D, dt, ct, 32, seed=D, tree=(bits, 1))   # tokens from the 33rd on are seen by none
    s.check(s.run())


@pytest.mark.gpu
def test_trees_that_are_chains_and_trees_of_any_bits():
    n, ctx = 70, 50
    chain = np.tril(np.ones((n, n), bool))
    s = Setup([ctx], [n], 4, 1, 64, seed=4, tree=(chain, 3), slopes=2.0 ** -np.arange(1, 5), window=30)
    plain = Setup([ctx], [n], 4, 1, 64, seed=4, slopes=2.0 ** -np.arange(1, 5), window=30)
    # (not the same bits: tiles start at other slots, so probabilities are
    # rounded relative to other running maxima; both are held to one oracle)
    ref = plain.oracle()
    s.check(s.run(), ref=ref)
    plain.check(plain.run(), ref=ref)
    g = np.random.default_rng(5)
    for bits in (g.random((n, n)) < 0.3, np.zeros((n, n), bool), np.ones((n, n), bool)):
        s = Setup([ctx], [n], 4, 1, 64, seed=6, tree=(bits, 3), slopes=2.0 ** -np.arange(1, 5))
        s.check(s.run())
        s = Setup([0], [n], 4, 1, 64, seed=6, tree=(bits, 3))   # no context: an empty row sees nothing
        lse = torch.zeros(n, 4, device=dev())
        s.check(s.run(lse=lse), lse)


@pytest.mark.gpu
def test_a_large_tree_behind_a_long_context():
    n = 600
    bits = random_tree(np.random.default_rng(7), n)
    s = Setup([1500], [n], 2, 2, 64, "bf16", "bf16", 64, seed=8, tree=(bits, 19), window=700)
    s.check(s.run())


@pytest.mark.gpu
def test_outputs_of_nobodys_tokens_are_left_alone():
    s = Setup([40, 9], [50, 3], 4, 2, 64, seed=9, gap=(7, 11))
    s.q[:7], s.q[-11:] = float("nan"), float("nan")
    s.to_device()
    out, lse = torch.full_like(s.qd, 3.0), torch.full((s.T, 4), 3.0, device=dev())
    assert s.run(out=out, lse=lse) is out
    s.check(out, lse)
    for x in (out, lse):
        assert (x[:7] == 3.0).all() and (x[-11:] == 3.0).all()


@pytest.mark.gpu
def test_starts_and_lengths_that_make_no_sense_stay_in_bounds():
    """Starts outside the tokens are clamped, falling ones mean none; lengths
    are clamped too, and more new tokens than slots leave the first ones nothing."""
    s = Setup([30, 20], [40, 10], 4, 2, 64, seed=10)
    want = s.run()
    out = torch.full_like(s.qd, 3.0)
    gbb.paged_attention_tokens(s.cache, s.qd, torch.tensor([-5, 40, 2 ** 31 - 1], dtype=torch.int32, device=dev()), s.btd,
                               s.lend, 70, out=out)
    assert torch.equal(out, want)
    out.fill_(3.0)
    gbb.paged_attention_tokens(s.cache, s.qd, torch.tensor([40, 30, 20], dtype=torch.int32, device=dev()), s.btd, s.lend, 70,
                               out=out)
    assert (out == 3.0).all()
    short = torch.tensor([25, -3], dtype=torch.int32, device=dev())
    out = s.run()
    gbb.paged_attention_tokens(s.cache, s.qd, s.startd, s.btd, short, 70, out=out)
    assert not out[:15].any() and not out[40:].any() and out[15:40].any(-1).any(-1).all()
    s.lengths = [25, 10]
    s.new = [25, 10]
    s.starts = np.array([0, 25, 35], np.int32)
    s.q = s.q[15:50]
    s.T = 35
    s.to_device()
    ref = s.run()
    assert (ref[:25].double() - out[15:40].double()).abs().max() <= 2.0 ** -9 * 8


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 24, 25, 30, 64, 65, 2 ** 31 - 1])
def test_more_tokens_than_slots(window):
    """Those before the first slot see what their sequence shares (a window
    counts from where they would lie), or what the tree gives them."""
    n, length = 40, 25
    o = dict(window=window) if window else {}
    s = Setup([length - n, 0], [n, 3], 4, 2, 64, seed=12, prefix=np.array([20, 0]), slopes=2.0 ** -np.arange(1, 5), **o)
    lse = torch.zeros(s.T, 4, device=dev())
    s.check(s.run(lse=lse), lse)
    bits = np.zeros((n + 3, n), bool)
    bits[:n] = random_tree(np.random.default_rng(13), n)
    bits[n:, :3] = True
    s = Setup([length - n, 0], [n, 3], 4, 2, 64, seed=14, tree=(bits, 2), slopes=2.0 ** -np.arange(1, 5), **o)
    s.check(s.run(lse=lse), lse)


@pytest.mark.gpu
def test_pages_that_are_not_there():
    s = Setup([150, 60, 0], [60, 9, 40], 4, 2, 128, page=16, seed=11)
    s.bt[0, 0], s.bt[0, 5], s.bt[0, 12] = -1, s.k.shape[0], -2 ** 31
    s.bt[1, 1:3] = 2 ** 31 - 1
    s.bt[2, :] = -1
    s.to_device()
    lse = torch.zeros(s.T, 4, device=dev())
    got = s.run(lse=lse)
    s.check(got, lse)
    assert not got[69:].any() and torch.isneginf(lse[69:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("new", [5, 60])
def test_what_is_not_seen_may_hold_anything(new, dt, ct):
    """NaN and infinities in slots that some rows see and others do not: they
    reach those that see them and no others."""
    n = 70 + new
    bits = np.tril(np.ones((new, new), bool))
    bits[:, 2] = False
    bits[2, 2] = True
    first = np.full(new, 20)
    s = Setup([70], [new], 4, 1, 64, dt, ct, 16, seed=12, tree=(bits, 3), first=first)
    ref = s.oracle()
    clean = s.run()
    s.check(clean, ref=ref)

    def poison(slot, value, which="kv"):
        p, o = int(s.bt[0, slot // 16]), slot % 16
        for name in which:
            t = getattr(s.cache, name)
            t[p, 0, o] = torch.full((64,), value, device=dev()).to(t.dtype)
    inf = float("inf") if ct != "e4m3" else float("nan")
    for slot, value in ((0, float("nan")), (5, inf), (19, float("nan"))):   # left padding: seen by none
        poison(slot, value)
    assert torch.equal(s.run(), clean)
    poison(72, float("nan"))                                                # drafted token 2: seen by itself alone
    got = s.run()
    rest = [i for i in range(new) if i != 2]
    assert torch.isnan(got[2]).all() and torch.equal(got[rest], clean[rest])
    if ct != "e4m3":   # infinities of either sign, and of both, where V alone has them
        s = Setup([10], [new], 4, 1, 64, dt, ct, 16, seed=13)
        clean = s.run()
        at = 10 + new - 2
        poison(at, float("-inf"), "v")
        got = s.run()
        assert torch.equal(got[:-2], clean[:-2]) and torch.isneginf(got[-2:]).all()
        poison(at + 1, float("inf"), "v")
        got = s.run()
        assert torch.equal(got[:-2], clean[:-2]) and torch.isneginf(got[-2]).all() and torch.isnan(got[-1]).all()
    assert n > 70


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3])
def test_scales(scale, dt):
    s = Setup([40], [90], 4, 2, 64, dt, dt, seed=14, scale=scale)
    s.check(s.run())
    s = Setup([40], [9], 1, 1, 64, dt, dt, seed=14, scale=scale, softcap=3.0)
    s.check(s.run())


@pytest.mark.gpu
def test_strided_queries_workspaces_streams_and_repeats():
    d = dev()
    s = Setup([700, 33, 0, 1500], [3, 9, 0, 30], 8, 2, 128, "bf16", "bf16", 32, seed=15)
    first = s.run()
    s.check(first)
    rows = torch.randn(s.T, 8 * 128 + 64, device=d).bfloat16()
    q = rows[:, 32:32 + 1024].unflatten(1, (8, 128))
    q.copy_(s.q)
    need = gbb.paged_attention_tokens_workspace(s.cache, s.T, 4, 8, s.max_len)
    assert need > 0
    ws = torch.zeros(need, dtype=torch.uint8, device=d)
    out = torch.full_like(first, float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            assert gbb.paged_attention_tokens(s.cache, q, s.startd, s.btd, s.lend, s.max_len, out=out, workspace=ws) is out
            gbb.paged_attention(s.cache, q[:4], s.btd, s.lend, s.max_len, workspace=torch.zeros_like(ws))
    side.synchronize()
    assert torch.equal(out, first)
    for bad in (0, need - 1):
        with pytest.raises(gbb.GbbError) as e:
            s.run(workspace=ws[:bad])
        assert e.value.status in (-1, -5)


@pytest.mark.gpu
def test_one_workspace_for_calls_of_all_kinds():
    """Single tokens and several, of many sizes, in turn on one workspace."""
    d = dev()
    a = Setup([3000], [4], 4, 1, 128, seed=16, page=64)
    b = Setup([20, 5000, 7], [1, 60, 2], 6, 2, 64, seed=17)
    size = max(gbb.paged_attention_tokens_workspace(x.cache, x.T, len(x.new), x.hq, x.max_len) for x in (a, b))
    size = max([size] + [gbb.paged_attention_workspace(x.cache, len(x.new), x.hq, x.max_len) for x in (a, b)])
    ws = torch.zeros(size, dtype=torch.uint8, device=d)
    want = [x.run() for x in (a, b)]
    single = [gbb.paged_attention(x.cache, x.qd[:len(x.new)], x.btd, x.lend, x.max_len) for x in (a, b)]
    for _ in range(3):
        for x, w, o in zip((a, b), want, single):
            assert torch.equal(x.run(workspace=ws), w)
            assert torch.equal(gbb.paged_attention(x.cache, x.qd[:len(x.new)], x.btd, x.lend, x.max_len, workspace=ws), o)


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_in_a_graph(given):
    d = dev()
    s = Setup([900, 40], [6, 20], 4, 2, 64, seed=18, page=32, window=500)
    out = torch.empty_like(s.qd)
    kw = {}
    if given:
        need = gbb.paged_attention_tokens_workspace(s.cache, s.T, 2, 4, s.max_len, window=500)
        kw = dict(workspace=torch.zeros(need, dtype=torch.uint8, device=d))
    s.run(out=out, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(out=out, **kw)
    lengths = s.lengths
    for i in range(4):
        s.q = torch.roll(s.q, 1, 0) * (1 - i / 8)
        s.lengths = [lengths[0] - 211 * i, lengths[1] - 9 * i]
        s.qd.copy_(s.q)
        s.lend.copy_(torch.tensor(s.lengths, dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        s.check(out)
        assert torch.equal(s.run(), out)


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    d = dev()
    D, page, pages = 128, 64, 400000
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("not enough memory")
    k = torch.empty(pages, 1, page, D, dtype=torch.float16, device=d)
    v = torch.empty(pages, 1, page, D, dtype=torch.float16, device=d)
    s = Setup([120], [80], 4, 1, D, page=page, seed=19)
    far = torch.tensor([pages - 1, 0, 262144 + 3, 399000], dtype=torch.int64)
    for i, p in enumerate(far.tolist()):
        k[p], v[p] = s.cache.k[int(s.bt[0, i])], s.cache.v[int(s.bt[0, i])]
    big = gbb.PagedCache(k, v)
    got = gbb.paged_attention_tokens(big, s.qd, s.startd, far.to(torch.int32).to(d)[None], s.lend, 200)
    assert torch.equal(got, s.run())
    kept = torch.tensor([[3, 70]], dtype=torch.int32, device=d)
    n = gbb.cache_keep(big, far.to(torch.int32).to(d)[None], s.lend, torch.tensor([80], dtype=torch.int32, device=d), kept,
                       torch.tensor([2], dtype=torch.int32, device=d))
    assert n.tolist() == [122]
    assert torch.equal(k[0, 0, 57], s.cache.k[int(s.bt[0, 2]), 0, 62]) and torch.equal(v[0, 0, 56], s.cache.v[int(s.bt[0, 1]), 0, 59])


# ----------------------------------------------------------------------------
# single tokens
# ----------------------------------------------------------------------------
def single(s, **kw):
    """The newest token of each sequence with the single token's operator."""
    return gbb.paged_attention(s.cache, s.qd, s.btd, s.lend, s.max_len, **{**s.arguments(), **kw})


SHAPED = [dict(softcap=5.0), dict(softcap=300.0), dict(window=1), dict(window=16), dict(window=100), dict(window=2 ** 31 - 1),
          dict(slopes=True), dict(softcap=30.0, slopes=True, window=77)]


@pytest.mark.gpu
@pytest.mark.parametrize("options", SHAPED, ids=lambda o: "+".join(o))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,ct", PAIRS)
def test_single_tokens(dt, ct, D, options):
    lengths = [0, 1, 2, 16, 17, 63, 64, 129, 300, 2500]
    o = dict(options)
    if o.get("slopes"):
        o["slopes"] = 2.0 ** -np.arange(1, 5)
    s = Setup([max(0, n - 1) for n in lengths], [min(1, n) for n in lengths], 4, 2, D, dt, ct, 16, seed=D, **o)
    full = torch.zeros(10, 4, D, dtype=s.q.dtype)
    full[1:] = s.q
    args, q = s.arguments(), full.to(dev())
    lse = torch.zeros(10, 4, device=dev())
    got = gbb.paged_attention(s.cache, q, s.btd, s.lend, s.max_len, lse=lse, **args)
    s.check(got[1:], lse[1:])
    assert not got[0].any() and torch.isneginf(lse[0]).all()
    # the same from the weights' launch, and the weights themselves
    w = torch.rand(s.k.shape[:3], device=dev())
    cache = gbb.PagedCache(s.cache.k, s.cache.v, weights=w, **s.kw)
    wo = torch.full_like(w, -1.0)
    again = gbb.paged_attention(cache, q, s.btd, s.lend, s.max_len, weights_out=wo, **args)
    assert torch.equal(again, got)
    qw, k, _ = s.wide()
    window, cap = o.get("window", 0), o.get("softcap", 0.0)
    touched = np.zeros(w.shape, bool)
    for b, n in enumerate(lengths):
        if not n:
            continue
        j = np.arange(n)
        pg, off = s.bt[b, j // 16], j % 16
        touched[pg, :, off] = True
        sc = np.einsum("hd,jhd->hj", qw[b - 1].reshape(4, D), np.repeat(k[pg, :, off], 2, 1)) * D ** -0.5
        e = (D + 4) * U * np.abs(sc).max() * 40 + 2.0 ** -19
        if cap:
            sc = cap * np.tanh(sc / cap)
            e += 2.0 ** -21 * cap
        if "slopes" in o:
            sc = sc - o["slopes"][:, None] * (n - 1 - j)
            e += 4 * U * (np.abs(sc).max() + n)
        if window:
            sc = np.where(n - 1 - j < window, sc, -np.inf)
        p = np.exp(sc - sc.max(1, keepdims=True))
        p = (p / p.sum(1, keepdims=True)).reshape(2, 2, n).sum(1)
        base = w.double().cpu().numpy()[pg, :, off]
        have = wo.double().cpu().numpy()[pg, :, off]
        assert np.all(np.abs(have - base - p.T) <= (2 * e + 2.0 ** -18 + 2 * n * U) * p.T + 4 * U * (base + p.T))
    assert (wo.cpu().numpy()[~touched] == -1.0).all()


@pytest.mark.gpu
def test_single_token_slots_before_the_window_may_hold_anything():
    for ct in ("f16", "e4m3"):
        s = Setup([299], [1], 4, 1, 64, "f16", ct, 16, seed=20, window=50)
        clean = single(s)
        s.check(clean)
        for j in list(range(240, 250)) + [0, 100]:
            s.cache.k[int(s.bt[0, j // 16]), 0, j % 16] = torch.full((64,), float("nan"), device=dev()).to(s.cache.k.dtype)
            s.cache.v[int(s.bt[0, j // 16]), 0, j % 16] = torch.full((64,), float("nan"), device=dev()).to(s.cache.k.dtype)
        assert torch.equal(single(s), clean)


@pytest.mark.gpu
def test_windows_of_any_size_split_and_whole():
    """Windows that end anywhere in a tile, in contexts of one and many runs."""
    for n in (40, 1000, 9000):
        for window in (1, 15, 31, 33, 500, 4096, 8999, 9000, 9001):
            s = Setup([n - 1], [1], 4, 1, 64, "bf16", "bf16", 16, seed=n, window=window)
            lse = torch.zeros(1, 4, device=dev())
            s.check(single(s, lse=lse), lse)
            need = gbb.paged_attention_workspace(s.cache, 1, 4, n, window=window)
            given = torch.zeros(max(16, need), dtype=torch.uint8, device=dev())
            assert torch.equal(single(s, workspace=given), single(s))


# ----------------------------------------------------------------------------
# refusals
# ----------------------------------------------------------------------------
def test_argument_refusals():
    """Checked before anything touches a device."""
    L, C, O = gbb.lib(), gbb.binding._PagedCache, gbb.binding._AttentionOptions  # noqa: E741
    base = dict(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4,
                page=16, kv_heads=2, head_dim=64)

    def tokens(c=None, o=None, q=8 << 20, qt=256, dt=0, T=6, B=2, hq=4, st=12 << 20, bt=9 << 20, mp=4, ln=10 << 20, ml=64, sc=1.0,
               out=11 << 20, lse=None, ws=1 << 24, wb=1 << 30):
        cc = C(**{**base, **(c or {})})
        oo = None if o is None else ctypes.byref(O(**o))
        return L.gbb_paged_attention_tokens(ctypes.byref(cc), q, qt, dt, T, B, hq, st, bt, mp, ln, ml, sc, oo, out, lse, ws, wb,
                                            None)

    def one(o, **kw):
        cc = C(**base)
        return L.gbb_paged_attention_options(ctypes.byref(cc), 8 << 20, 256, 0, 2, 4, 9 << 20, 4, 10 << 20, 64, 1.0,
                                             ctypes.byref(O(**o)), 11 << 20, None, None, 1 << 24, 1 << 30, None)

    assert tokens(B=0) == 0 and tokens(T=0) == 0
    for bad in (dict(c=dict(v=None)), dict(c=dict(dtype=2)), dict(dt=1), dict(T=-1), dict(B=-1), dict(ml=0), dict(mp=0),
                dict(sc=float("inf")), dict(q=None), dict(out=None), dict(st=None), dict(bt=None), dict(ln=None),
                dict(out=8 << 20), dict(o=dict(softcap=-1.0)), dict(o=dict(softcap=float("nan"))), dict(o=dict(softcap=1e-35)),
                dict(o=dict(window=-1)), dict(o=dict(tree=1 << 20, tree_words=1, prefix=1 << 20)),
                dict(o=dict(softcap=1e35)), dict(sc=1e25, o=dict(softcap=1e-10)), dict(sc=-1e35)):
        assert tokens(**bad) == -1, bad
    for bad in (dict(c=dict(page=8)), dict(c=dict(head_dim=32)), dict(hq=5), dict(hq=2 * 129), dict(ml=65), dict(qt=128),
                dict(T=1 << 23), dict(B=1 << 23), dict(o=dict(tree=1 << 20, tree_words=0)),
                dict(o=dict(tree=1 << 20, tree_words=1 << 20))):
        assert tokens(**bad) == -2, bad
    for bad in (dict(q=(8 << 20) + 2), dict(out=(11 << 20) + 8), dict(qt=260), dict(lse=2), dict(st=(12 << 20) + 1),
                dict(o=dict(slopes=2)), dict(o=dict(first=2)), dict(o=dict(prefix=2)), dict(o=dict(tree=2, tree_words=1))):
        assert tokens(**bad) == -4, bad
    long = dict(mp=64, ml=1024, c=dict(num_pages=64))
    assert tokens(ws=None, **long) == -1
    assert tokens(wb=16, **long) == -5
    assert tokens(ws=(1 << 24) + 8, **long) == -4
    for o in (dict(first=1 << 20), dict(prefix=1 << 20), dict(tree=1 << 20, tree_words=1), dict(window=-1), dict(softcap=-2.0), dict(softcap=1e35),
              dict(softcap=float("inf"))):
        assert one(o) == -1, o
    assert one(dict(slopes=2)) == -4
    cc = C(**base)
    need = L.gbb_paged_attention_tokens_workspace
    assert need(ctypes.byref(cc), 6, 2, 5, 64, 0, 0) == 0 and need(None, 6, 2, 4, 64, 0, 0) == 0
    assert need(ctypes.byref(cc), 0, 2, 4, 64, 0, 0) == 0 and need(ctypes.byref(cc), 6, 2, 4, 10000, -1, 0) == 0
    assert 0 < need(ctypes.byref(cc), 6, 2, 4, 2000, 0, 0) < need(ctypes.byref(cc), 64, 2, 4, 10000, 0, 0)
    window = L.gbb_paged_attention_options_workspace
    assert window(ctypes.byref(cc), 2, 4, 10000, 0, 0) == L.gbb_paged_attention_workspace(ctypes.byref(cc), 2, 4, 10000, 0)
    assert window(ctypes.byref(cc), 2, 4, 10000, 0, -1) == 0


def test_binding_refusals():
    """Shapes and types, without a GPU: tensors of the CPU are refused first."""
    k = torch.zeros(2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        gbb.PagedCache(k, k)
    gbb.paged._resolve()
    with pytest.raises((TypeError, ValueError)):
        gbb.paged._options(0, 4, 0.0, torch.zeros(4), 0)
    assert gbb.paged._options(0, 4, 0.0, None, 0) is None
    assert gbb.paged._options(0, 4, 0.0, None, 2 ** 32 + 5)._obj.window == 2 ** 31 - 1   # not 5
