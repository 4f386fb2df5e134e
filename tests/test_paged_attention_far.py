"""Attention of several new tokens where lengths come near the largest that are
accepted: max_len up to 2^31 - 1 - 8192."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_paged_attention_tokens import Setup, dev  # noqa: E402

LARGEST = 2 ** 31 - 1 - 8192


def test_runs_past_31_bits():
    """What the kernel has to hold for: the runs of a plan for the largest
    max_len (64 of them at most) start, from a first slot near the end, past
    2^31, where a sum in 32 bits is negative and below every length."""
    chunk = ((LARGEST + 15 + 63) // 64 + 63) & ~63
    low = (LARGEST - 300) & ~15
    wrapped = (low + chunk + 2 ** 31) % 2 ** 32 - 2 ** 31
    assert wrapped < 0 and low + chunk > 2 ** 31 and chunk >= LARGEST - low   # the second run: nothing of it is left


@pytest.mark.gpu
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("window", [0, 200])
def test_first_slots_near_the_largest_length(window, tree):
    """The last slots of a sequence of the largest length, those before hidden
    by `first`: as if the sequence had nothing else."""
    d, page, n, length = dev(), 256, 5, 300
    options = dict(window=window) if window else {}
    if tree:
        options["tree"] = (np.tril(np.ones((n, n), bool)), 1)
    s = Setup([length - n], [n], 2, 1, 64, page=page, seed=1, **options)
    pages = -(-LARGEST // page)
    base = (pages - 3) * page                                   # base + length <= LARGEST
    bt = torch.full((1, pages), -1, dtype=torch.int32, device=d)
    bt[0, pages - 3:pages - 1] = s.btd[0]
    lengths = torch.tensor([base + length], dtype=torch.int32, device=d)
    first = torch.full((n,), base, dtype=torch.int32, device=d)
    lse = torch.zeros(n, 2, device=d)
    got = gbb.paged_attention_tokens(s.cache, s.qd, s.startd, bt, lengths, LARGEST, lse=lse, first=first, **s.arguments())
    s.check(got, lse)
