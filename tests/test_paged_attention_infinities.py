"""Infinities and NaN of V in attention of several new tokens: they reach the
rows that see them with a weight above 0 and no others, whatever the number of
waves, runs and rows of the call.  Weights of 0 are made by scores 110 or more below
another (exp(-110) is 0 in 32 bits), all others lie within 2^-16 of their row's
largest."""
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_paged_attention_tokens import PAIRS, Setup, dev, random_tree, words_of  # noqa: E402

import numpy as np  # noqa: E402

INF, NAN = float("inf"), float("nan")


def two_waves(**kw):
    """Sequences and kv heads enough for two waves a workgroup (256 CUs)."""
    context = [70, 3, 40, 64] * 4
    new = kw.pop("new", [4, 9, 1, 5] * 4)
    return Setup(context, new, 32, 8, **{**dict(D=64, page=16, q_scale=0.25), **kw})


def four_waves(context=70, new=40, **kw):
    return Setup([context], [new], 4, 1, **{**dict(D=64, page=16, q_scale=0.25), **kw})


def put(s, b, slot, value, which="v", head=0):
    t = getattr(s.cache, which)
    row = t[int(s.bt[b, slot // s.page]), head, slot % s.page]
    row.copy_(torch.full((s.D,), value, device=dev()).to(t.dtype) if not torch.is_tensor(value) else value.to(t.dtype))


def head_of(s, out, b, head=0):
    """Outputs of sequence b's rows of a kv head, and all others."""
    group = s.hq // s.hkv
    mine = torch.zeros(out.shape[:2], dtype=torch.bool)
    mine[int(s.starts[b]):int(s.starts[b + 1]), head * group:(head + 1) * group] = True
    return out[mine.to(out.device)], out[~mine.to(out.device)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("make", [two_waves, four_waves])
def test_an_infinity_that_all_rows_see(make, D, dt):
    """In a tile that every row sees whole, where the weights' second operand is
    0 or negative."""
    s = make(D=D, dt=dt, ct=dt, seed=D)
    lse = torch.zeros(s.T, s.hq, device=dev())
    clean = s.run(lse=lse)
    s.check(clean, lse)
    for value in (INF, -INF):
        put(s, 0, 5, value)
        again = torch.zeros_like(lse)
        mine, rest = head_of(s, s.run(lse=again), 0)
        assert (mine == value).all() and torch.equal(rest, head_of(s, clean, 0)[1]) and torch.equal(again, lse)
    put(s, 0, 5, INF)
    put(s, 0, 37, -INF)
    mine, rest = head_of(s, s.run(), 0)
    assert torch.isnan(mine).all() and torch.equal(rest, head_of(s, clean, 0)[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("far", ["before", "behind"])
@pytest.mark.parametrize("make", [two_waves, four_waves])
def test_a_weight_that_rounds_to_zero(make, far, dt, ct):
    """A slot far below the others counts as not seen, whether its tile comes
    after the one with the largest score or before it."""
    s = make(dt=dt, ct=ct, seed=3)
    s.q[:, :s.hq // s.hkv] = 1.0
    s.to_device()
    slot = 5
    if ct == "e4m3":                                            # as large as the scales let it, with more of q
        s.qd[:, :s.hq // s.hkv] = 4.0
    high = 400.0 if ct == "e4m3" else 30.0                      # scores of 120 or more, and of 30 D / sqrt(D) = 240
    put(s, 0, *((slot, -high) if far == "before" else (69, high)), "k")
    put(s, 0, slot, 1.0)
    clean = s.run()
    assert torch.isfinite(clean.float()).all()
    for value in ((NAN,) if ct == "e4m3" else (INF, -INF, NAN)):
        put(s, 0, slot, value)
        assert torch.equal(s.run(), clean)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("context", [450, 3000])
def test_runs_that_hold_an_infinity(context, dt, ct):
    """A run's infinity through the join by the last workgroup (two runs) and by
    the second launch: at a weight above 0 and at one of 0."""
    s = four_waves(context=context, new=5, dt=dt, ct=ct, seed=context)
    assert gbb.paged_attention_tokens_workspace(s.cache, 5, 1, 4, s.max_len) > 0
    value = NAN if ct == "e4m3" else INF
    s.check(s.run())
    put(s, 0, 7, value)
    got = s.run()
    assert (torch.isnan(got) if ct == "e4m3" else got == INF).all()
    put(s, 0, 7, 1.0)
    s.qd.fill_(4.0)
    put(s, 0, context - 20, 30.0 if ct != "e4m3" else 400.0, "k")
    clean = s.run()
    assert torch.isfinite(clean.float()).all()
    put(s, 0, 7, value)
    assert torch.equal(s.run(), clean)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
def test_a_drafted_token_that_holds_nan(dt, ct):
    """Seen by its own row alone, with two waves a workgroup."""
    new = [40] + [3] * 15
    bits = np.zeros((sum(new), 40), bool)
    at = 0
    for n in new:
        bits[at:at + n, :n] = random_tree(np.random.default_rng(n), n)
        at += n
    bits[:40, 2] = False
    bits[2, 2] = True
    assert words_of(bits, 2).shape == (sum(new), 2)
    s = two_waves(new=new, dt=dt, ct=ct, seed=5, tree=(bits, 2))
    clean = s.run()
    s.check(clean)
    for which in "kv":
        put(s, 0, 72, NAN, which)
        got = s.run()
        keep = torch.ones(got.shape[:2], dtype=torch.bool, device=dev())
        keep[2, :4] = False
        assert torch.isnan(got[2, :4]).all() and torch.equal(got[keep], clean[keep])
