"""How many bits of a probability the attention kernel's products carry.

Head h has three slots: two with score 0 and one with score -x_h, so that p =
(1, 1, e) / (2 + e) with e = exp(-x_h).  In column h the values are -hi, -lo
and 1, where hi is e rounded to the cache's type and lo what that drops,
rounded again.  So the output there is (e - hi - lo) / (2 + e): what is left
of e after two roundings, and zero if e itself is held in two such parts.

Tolerance.  The exponential's argument is below 16 in base 2 with its offset
of 14, so its rounding is at most 2^-21 and e's relative error ln 2 * 2^-21;
its score's rounding adds ln 2 * 2^-22 (|x_h| < 2.8, below 4 in base 2), the
exponential 2^-23, and each of the products' fp32 sums and the division 2^-24
of the largest term.  Together less than 2^-20.3 e / (2 + e), then bf16's own
rounding of the output."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).bfloat16().double().numpy()


def steps():
    """16 bf16 scores in [0.4, 2.8] whose exponential leaves much after two
    roundings to bf16: at least 0.7 of the largest remainder, 2^-18 e."""
    x = bf16(np.linspace(0.4, 2.8, 4000))
    x = np.unique(x)
    e = np.exp(-x)
    hi = bf16(e)
    lo = bf16(e - hi)
    rest = np.abs(e - hi - lo) / 2.0 ** np.floor(np.log2(e))
    return x[np.argsort(-rest)[:16]]


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
def test_bf16_products_keep_the_bits_of_a_probability(D):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    x = steps()
    e = np.exp(-x)
    hi = bf16(e)
    lo = bf16(e - hi)
    want = (e - hi - lo) / (2 + e)
    # what two parts lose is well above the tolerance
    tol = 2.0 ** -20.3 * e / (2 + e)
    assert np.all(np.abs(want) >= 1.5 * tol)
    q = torch.zeros(1, 16, D, dtype=torch.bfloat16)
    q[0, :, 0] = torch.from_numpy(x).bfloat16()
    k, v = (torch.zeros(1, 1, 16, D, dtype=torch.bfloat16) for _ in range(2))
    k[0, 0, 2, 0] = -1.0
    heads = np.arange(16)
    for slot, values in enumerate((-hi, -lo, np.ones(16))):
        v[0, 0, slot, heads] = torch.from_numpy(values).bfloat16()
    cache = gbb.PagedCache(k.cuda(), v.cuda())
    got = gbb.paged_attention(cache, q.cuda(), torch.zeros(1, 1, dtype=torch.int32, device="cuda"),
                              torch.tensor([3], dtype=torch.int32, device="cuda"), 3, scale=1.0)
    got = got[0].double().cpu().numpy()[heads, heads]
    assert np.all(np.abs(got - want) <= tol + 2.0 ** -8 * np.abs(want)), (got, want)
