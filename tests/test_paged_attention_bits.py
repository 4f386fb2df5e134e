"""How many bits of the probabilities reach the output, apart from the bounds that
allow for one 16-bit operand: the weighted sum of values that nearly cancel.

Scores hardly differ up to a bias by distance, and V alternates in sign between
slots that lie next to each other, of one size each pair.  An output is then sum
p |v| times what a step between neighbours leaves, below the half step that one
operand would be off by for each of them.  With u = 2^-24 and the operands' 22 bits (fp16) or 16 and 24 (bf16)
an output is off by at most (2^-bits + 2 n u + 2^-18) sum p |v| and half a step of
its own."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_paged_attention_tokens import PAIRS, U, UNIT, Setup, dev, random_tree  # noqa: E402


def check_fine(s, got, bits, telling=True):
    """Setup.check without its half step of the operand."""
    out, ref_lse, mass, (dots, scores, bias) = s.oracle()
    mine = ~np.isnan(ref_lse[:, 0])
    e = (s.D + 4) * U * dots + 2.0 ** -21 * s.options.get("softcap", 0.0) + 4 * U * (scores + bias) + 2.0 ** -20
    pre = (2 * e + 2.0 ** -bits + 2.0 ** -18 + 2 * s.max_len * U)[..., None] * mass
    tol = pre + UNIT[s.dt] * (np.abs(out) + pre) + 2.0 ** -25
    got = got.double().cpu().numpy()
    assert np.all(np.isfinite(got[mine]))
    error = np.abs(got[mine] - out[mine])
    assert (error <= tol[mine]).all(), np.max(error / tol[mine])
    # a bound that a single operand can miss: most of what is allowed lies below its half step
    assert not telling or np.median(tol[mine] / (UNIT[s.dt] * mass[mine] + 1e-300)) < 0.7


def cancelling(s):
    """V's neighbours of opposite sign, so that outputs are far below sum p |v|."""
    for b, n in enumerate(s.lengths):
        for j in range(1, n, 2):
            at, last = (int(s.bt[b, j // s.page]), slice(None), j % s.page), (int(s.bt[b, (j - 1) // s.page]), slice(None), (j - 1) % s.page)
            s.v[at] = (-s.v[last].float()).to(s.v.dtype)
    s.q *= 0.02          # scores that hardly differ
    s.to_device()
    return s


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("drafted", ["tokens", "tree"])
def test_drafts_of_one_user(drafted, D, dt, ct):
    """A row tile a kv head (four waves), in one run and in several."""
    for context, new in ((200, 2), (500, 25), (1000, 7)):
        o = {}
        if drafted == "tree":
            o["tree"] = (random_tree(np.random.default_rng(new), new), 1)
        s = cancelling(Setup([context], [new], 8, 2, D, dt, ct, 64, seed=D + new, slopes=np.full(8, 2.0 ** -6), **o))
        check_fine(s, s.run(), 22 if dt == "f16" else 16)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,ct", PAIRS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_drafts_of_a_batch(D, dt, ct):
    """Two waves a workgroup."""
    s = cancelling(Setup([150, 70, 33, 200] * 4, [2, 5, 1, 3] * 4, 16, 8, D, dt, ct, 32, seed=D, slopes=np.full(16, 2.0 ** -6)))
    check_fine(s, s.run(), 22 if dt == "f16" else 16)


@pytest.mark.gpu
@pytest.mark.parametrize("options", [dict(softcap=5.0), dict(window=100), dict(slopes=True), dict(softcap=30.0, slopes=True, window=150)],
                         ids=lambda o: "+".join(o))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dt,ct", PAIRS)
def test_single_tokens(dt, ct, D, options):
    o = dict(options)
    if o.get("slopes"):
        o["slopes"] = np.full(4, 2.0 ** -6)
    lengths = [200, 64, 333, 1500]
    s = cancelling(Setup([n - 1 for n in lengths], [1] * 4, 4, 2, D, dt, ct, 16, seed=D, **o))
    got = gbb.paged_attention(s.cache, s.qd, s.btd, s.lend, s.max_len, **s.arguments())
    check_fine(s, got, 22 if dt == "f16" else 24)
