"""The attention kernel by its plans: run lengths, waves, ways of joining and
numbers of query heads that other tests' sizes do not reach, each type and
head size, against the 64-bit oracle.

Which plan a size takes follows from pairs of (sequence, kv head) and the
bound on the lengths, on the host; the number of runs shows in the
workspace's size and is asserted beside every case (on a GPU of 256 compute
units, which is also what the library plans for without one).

Tolerances, per output element.  With e the largest error of a score, P = sum
p |v| (p normalised) and n terms to a sum: a probability is off by a factor of
at most 1 + 2 e + 2^-20 (its own and the normalisation's exponentials; its
parts for the matrix cores hold 22 bits or more) and sums of n terms in fp32
add n 2^-24, for the output's and the probabilities' sum.  A run has at most
4096 slots and there are at most 256 of them to join, so n <= 4352.  A score
is a sum of D exact products in fp32, e <= (D + 4) 2^-24 scale sum |q k| +
2^-20: the last term is the rounding of a score below 2^4 in the exponent's
base 2."""
import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
PAIRS = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


def runs(B, hq, hkv, D, max_len):
    """Runs of a sequence in the library's plan, from its workspace: 16 KiB of
    counters, then 8 bytes and D floats a (query head, run), in pieces of 256
    bytes."""
    C = gbb.binding._PagedCache
    c = C(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4, page=16,
          kv_heads=hkv, head_dim=D)   # never read
    import ctypes
    have = gbb.lib().gbb_paged_attention_workspace(ctypes.byref(c), B, hq, max_len, 0)
    up = lambda n: (n + 255) & ~255  # noqa: E731
    for n in range(1, 300):
        rows = B * hq * n
        if have == (0 if n == 1 else 16384 + up(8 * rows) + up(4 * D * rows)):
            return n
    raise AssertionError(have)


class Case:
    """Random keys and values in pages in no order; what no sequence uses is
    NaN, and so are the slots past a length."""

    def __init__(self, lengths, hq, hkv, D, dt, ct, max_len, page=64, seed=0):
        g = np.random.default_rng(seed)
        d = torch.device("cuda", 0)
        self.lengths, self.hq, self.hkv, self.D, self.dt, self.max_len = list(lengths), hq, hkv, D, dt, max_len
        B, per = len(lengths), -(-max_len // page)
        used = [-(-n // page) for n in lengths]
        pages = sum(used) + 2
        order = g.permutation(pages)
        self.bt = np.full((B, per), 2 ** 31 - 1, np.int32)   # what is not used is never looked at
        there, at = np.zeros((pages, page), bool), 0
        for b, n in enumerate(used):
            self.bt[b, :n] = order[at:at + n]
            at += n
            j = np.arange(lengths[b])
            there[self.bt[b, j // page], j % page] = True
        self.ks, self.vs = np.ones(hkv, np.float32), np.ones(hkv, np.float32)
        kw = {}
        if ct == "e4m3":
            self.ks, self.vs = (g.uniform(0.01, 0.03, hkv).astype(np.float32) for _ in range(2))
            kw = dict(k_scale=torch.from_numpy(self.ks).to(d), v_scale=torch.from_numpy(self.vs).to(d))

        def made(scale):
            x = g.standard_normal((pages, hkv, page, D), np.float32) / scale[None, :, None, None]
            if ct == "e4m3":
                x = np.clip(x, -448, 448)
            x = torch.from_numpy(np.where(there[:, None, :, None], x, np.float32(np.nan)))
            return x.to(DT[ct])
        self.k, self.v = made(self.ks), made(self.vs)
        self.q = torch.from_numpy(2 * g.standard_normal((B, hq, D), np.float32)).to(DT[dt])
        self.w = torch.from_numpy(g.random((pages, hkv, page), np.float32))
        self.cache = gbb.PagedCache(self.k.to(d), self.v.to(d), weights=self.w.to(d), **kw)
        self.qd, self.btd = self.q.to(d), torch.from_numpy(self.bt).to(d)
        self.lend = torch.tensor(self.lengths, dtype=torch.int32, device=d)

    def run(self, **kw):
        return gbb.paged_attention(self.cache, self.qd, self.btd, self.lend, self.max_len, **kw)

    def check(self):
        """With the log-sums; with weights the same bits, out of place and in
        place."""
        B = len(self.lengths)
        lse = torch.zeros(B, self.hq, device="cuda")
        got = self.run(lse=lse)
        w, lse2 = self.w.cuda(), torch.zeros(B, self.hq, device="cuda")
        assert torch.equal(self.run(weights_out=w, lse=lse2), got) and torch.equal(lse2, lse)
        self.run(weights_out=self.cache.weights)
        assert torch.equal(self.cache.weights, w)
        assert torch.equal(self.run(), got)   # and again

        wide = lambda x, s: np.nan_to_num(x.double().numpy()) * s[None, :, None, None].astype(np.float64)  # noqa: E731
        out, ref_lse, added, mass, dots = od.paged_attention(self.q.double().numpy(), wide(self.k, self.ks), wide(self.v, self.vs),
                                                             self.bt, self.lengths, self.D ** -0.5)
        e = (self.D + 4) * 2.0 ** -24 * self.D ** -0.5 * dots + 2.0 ** -20
        n = np.minimum(np.array(self.lengths), 4096 + 256)[:, None]
        pre = (2 * e + 2.0 ** -20 + 2 * n * 2.0 ** -24)[..., None] * mass
        tol = pre + UNIT[self.dt] * (np.abs(out) + pre) + 2.0 ** -25
        x = got.double().cpu().numpy()
        assert np.all(np.isfinite(x))
        assert np.all(np.abs(x - out) <= tol), np.max(np.abs(x - out) / tol)
        x = lse.double().cpu().numpy()
        some = ~np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(x), ~some)
        assert np.all(np.abs(x[some] - ref_lse[some]) <= (e + n * 2.0 ** -24 + 2.0 ** -20)[some] + 2.0 ** -22 * np.abs(ref_lse[some]))
        x, base = w.double().cpu().numpy(), self.w.double().numpy()
        rel = float((2 * e + n * 2.0 ** -24 + 2.0 ** -19).max())
        assert np.all(np.abs(x - base - added) <= rel * added + (self.hq // self.hkv + 1) * 2.0 ** -24 * (base + added))
        assert np.array_equal(x[added == 0], base[added == 0])


# name: (lengths, query heads, kv heads, bound, runs)
SIZES = {
    # four waves a workgroup, runs of 128 and 256
    "short runs": ([700, 33, 0, 1500, 128, 129], 4, 2, 1500, 12),
    "runs of 256": ([2300, 256, 257, 1], 2, 1, 4000, 16),
    # the pairs alone fill the chip: whole contexts, four waves and eight
    "whole, four waves": ([600, 0, 1, 599, 33] + [17] * 140, 4, 2, 600, 1),
    "whole, eight waves": ([4096, 3001, 0, 2048, 100] + [9] * 130, 4, 2, 4096, 1),
    # runs of 2048 and of 4096
    "runs of 2048": ([10000, 2049, 4096, 0, 2048] + [5] * 25, 4, 2, 10000, 5),
    "runs of 4096": ([20000, 4097, 4096, 0, 12288] + [5] * 12, 4, 2, 20000, 5),
    # one launch joins more than 16 runs, and 64
    "20 runs": ([20000, 17000, 1025, 0], 4, 1, 20000, 20),
    "64 runs": ([65536, 1024], 2, 1, 65536, 64),
    # a second launch joins: more than 64 runs
    "69 runs": ([70000, 5000, 0, 66000], 4, 1, 70000, 69),
    "137 runs": ([140000], 2, 1, 140000, 137),
}


@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_plans_are_those_meant(name, D):
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("another number of compute units")
    lengths, hq, hkv, max_len, want = SIZES[name]
    assert runs(len(lengths), hq, hkv, D, max_len) == want


@pytest.mark.gpu
@pytest.mark.parametrize("name", SIZES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,ct", PAIRS)
def test_plan(name, D, dt, ct):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lengths, hq, hkv, max_len, _ = SIZES[name]
    Case(lengths, hq, hkv, D, dt, ct, max_len, page=128 if max_len > 20000 else 32, seed=D + len(lengths)).check()


GROUPS = {
    "whole": ([70, 0, 129, 400], 1, 400, 1),
    "runs": ([3000, 17, 0, 1025], 1, 3000, 12),
    "runs, two kv heads": ([2500, 40, 1200], 2, 2600, 11),
    "second launch": ([70000, 40], 1, 70000, 69),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name,group", [(n, g) for g in (17, 40, 128) for n in GROUPS if g == 17 or n != "second launch"])
@pytest.mark.parametrize("dt,ct,D", [("f16", "f16", 64), ("bf16", "bf16", 128), ("f16", "e4m3", 256), ("bf16", "e4m3", 64)])
def test_more_than_16_query_heads(name, group, dt, ct, D):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lengths, hkv, max_len, _ = GROUPS[name]
    Case(lengths, group * hkv, hkv, D, dt, ct, max_len, seed=group).check()


@pytest.mark.parametrize("name", GROUPS)
def test_groups_take_several_runs(name):
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("another number of compute units")
    lengths, hkv, max_len, want = GROUPS[name]
    assert runs(len(lengths), 17 * hkv, hkv, 64, max_len) == want


@pytest.mark.gpu
@pytest.mark.parametrize("ct", ["f16", "e4m3"])
def test_more_sequences_than_counters(ct):
    """4400 pairs, of which a few are split: a second launch joins them."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lengths = [5000, 0, 2049, 2048, 1] * 2 + [3, 0, 18, 7, 1] * 218
    assert len(lengths) * 4 > 4096
    Case(lengths, 4, 4, 64, "f16", ct, 5000, page=16, seed=1).check()


def test_more_sequences_than_counters_are_split():
    assert runs(1100, 4, 4, 64, 5000) == 3
