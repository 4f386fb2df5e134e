"""Every kind of launch of the attention of several new tokens: two waves a
workgroup with all types, head sizes, masks and shapes of scores, and runs that the
last workgroup of a row tile joins.  Bounds as in test_paged_attention_tokens.py,
without the half step of one operand where there are two."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_paged_attention_bits import check_fine  # noqa: E402
from test_paged_attention_tokens import PAIRS, U, UNIT, Setup, dev, random_tree  # noqa: E402

HQ, HKV = 12, 4
# 32 sequences of 4 kv heads, 3 to 63 rows each: two waves (on 256 CUs), both of them with rows
NEW = [1, 2, 11, 3, 21, 1, 0, 2] * 4
CONTEXT = [130, 0, 70, 33, 64, 15, 40, 1] * 4


def two_waves(D, dt, ct, **options):
    return Setup(CONTEXT, NEW, HQ, HKV, D, dt, ct, 16, seed=D + len(options), **options)


def check(s, missing=()):
    for b, page in missing:
        s.bt[b, page] = -1
    if missing:
        s.to_device()
    lse = torch.zeros(s.T, s.hq, device=dev())
    got = s.run(lse=lse)
    s.check(got, lse)
    check_fine(s, got, 22 if s.dt == "f16" else 16, telling=False)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_waves(D, dt, ct):
    g, T = np.random.default_rng(D), sum(NEW)
    slopes = 2.0 ** -np.arange(1, HQ + 1)
    first = g.integers(-5, 160, T)
    first[::7] = 2 ** 31 - 1                                    # rows that see nothing
    prefix = np.resize(np.array([140, 1, 75, 0]), len(NEW))
    check(two_waves(D, dt, ct))
    check(two_waves(D, dt, ct, window=40, softcap=20.0), [(0, 7), (2, 4), (4, 5)])
    check(two_waves(D, dt, ct, slopes=slopes, first=first))
    check(two_waves(D, dt, ct, prefix=prefix, softcap=300.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_two_waves_of_trees(D, dt, ct):
    g, T = np.random.default_rng(D + 1), sum(NEW)
    bits, at = np.zeros((T, 32), bool), 0
    for n in NEW:
        bits[at:at + n, :n] = random_tree(g, n)
        bits[at:at + n, n:] = g.random((n, 32 - n)) < 0.5       # bits past the sequence's tokens do not count
        at += n
    slopes = 2.0 ** -np.arange(1, HQ + 1)
    check(two_waves(D, dt, ct, tree=(bits, 1)), [(0, 0), (2, 4)])
    check(two_waves(D, dt, ct, tree=(bits, 1), slopes=slopes, window=30))
    check(two_waves(D, dt, ct, tree=(bits, 1), softcap=5.0, first=g.integers(0, 100, T)))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("tree", [False, True])
def test_two_runs_joined_by_the_last_workgroup(tree, D, dt, ct):
    """Too few slots for a second launch, in four waves: one operand and two."""
    for new in (9, 70):
        o = dict(tree=(random_tree(np.random.default_rng(new), new), 3)) if tree else {}
        s = Setup([390], [new], 4, 2, D, dt, ct, 64, seed=D + new, **o)
        words = 3 if tree else 0
        assert gbb.paged_attention_tokens_workspace(s.cache, s.T, 1, 4, s.max_len, tree_words=words) > 0
        lse = torch.zeros(s.T, 4, device=dev())
        got = s.run(lse=lse)
        s.check(got, lse)
        again = torch.zeros_like(lse)
        assert torch.equal(s.run(lse=again), got) and torch.equal(again, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts_of_a_batch_in_several_runs(D, dt, ct):
    """More row tiles than two a CU, behind more than 4096 slots: the definition in
    64 bits on the GPU, a kv head at a time."""
    hq, hkv, page = 64, 8, 64
    new, context = [112] * 8, [4400, 4200, 0, 4096, 1000, 4300, 17, 3900]
    g = torch.Generator(device=dev()).manual_seed(D)
    per = -(-(max(context) + 112) // page)
    shape = (8 * per, hkv, page, D)
    k, v = (torch.randn(shape, generator=g, device=dev()) for _ in range(2))
    scales = torch.full((hkv,), 0.02, device=dev()) if ct == "e4m3" else None
    if ct == "e4m3":
        k, v = k / 0.02, v / 0.02
    kind = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
    k, v = (x.clamp(-448, 448).to(kind[ct]) for x in (k, v))
    cache = gbb.PagedCache(k, v, scales, scales)
    q = (2 * torch.randn(sum(new), hq, D, generator=g, device=dev())).to(kind[dt])
    bt = torch.randperm(8 * per, generator=g, device=dev()).to(torch.int32).view(8, per)
    lengths = torch.tensor([c + 112 for c in context], dtype=torch.int32, device=dev())
    starts = torch.arange(9, dtype=torch.int32, device=dev()) * 112
    max_len = max(context) + 112
    assert gbb.paged_attention_tokens_workspace(cache, sum(new), 8, hq, max_len) > 0
    lse = torch.zeros(sum(new), hq, device=dev())
    got = gbb.paged_attention_tokens(cache, q, starts, bt, lengths, max_len, lse=lse)
    unit, n = UNIT[dt], 2 * max_len * U
    factor = float(scales[0]) if scales is not None else 1.0
    for b, c in enumerate(context):
        rows = slice(112 * b, 112 * (b + 1))
        slots = torch.arange(c + 112, device=dev())
        pages = bt[b].long()[slots // page]
        seen = slots[None, :] <= c + torch.arange(112, device=dev())[:, None]
        for h in range(hkv):
            kk, vv = (x[pages, h, slots % page].double() * factor for x in (k, v))
            for x in range(h * 8, h * 8 + 8):
                qq = q[rows, x].double()
                s = (qq @ kk.T.contiguous() * D ** -0.5).masked_fill(~seen, float("-inf"))
                dots = (qq.abs() @ kk.abs().T.contiguous() * D ** -0.5).masked_fill(~seen, 0.0).amax(1)
                e = (D + 4) * U * dots + 4 * U * s.masked_fill(~seen, 0.0).abs().amax(1) + 2.0 ** -20
                p = s.softmax(1)
                out, mass = p @ vv, p @ vv.abs()
                pre = (2 * e + unit + 2.0 ** -18 + n)[:, None] * mass
                tol = pre + unit * (out.abs() + pre) + 2.0 ** -25
                assert ((got[rows, x].double() - out).abs() <= tol).all()
                ref = s.logsumexp(1)
                assert ((lse[rows, x].double() - ref).abs() <= e + n + 2.0 ** -19 + 2.0 ** -22 * ref.abs()).all()
