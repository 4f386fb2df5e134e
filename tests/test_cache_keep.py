"""What is left of drafted tokens in the cache, exact against the oracle."""
import ctypes

import numpy as np
import pytest

from oracle import new_tokens as on

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


BITS = {torch.float16: torch.int16, torch.bfloat16: torch.int16, torch.float8_e4m3fn: torch.uint8}


def keep(lengths, drafted, kept, counts, dtype=torch.float16, page=16, hkv=3, D=64, tracked=True, holes=(), seed=0):
    """Runs it on random caches (any bits) and compares all of the cache."""
    g = np.random.default_rng(seed)
    B, most = len(lengths), len(kept[0]) if len(kept) else 0
    per = -(-max(1, max(lengths)) // page)
    pages = B * per + 1
    bt = g.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    for b, i in holes:
        bt[b, i] = -1 if i % 2 else pages
    kind = BITS[dtype]
    top = 256 if kind is torch.uint8 else 1 << 15
    k, v = (torch.from_numpy(g.integers(0, top, (pages, hkv, page, D))).to(kind) for _ in range(2))
    w = torch.from_numpy(g.random((pages, hkv, page)).astype(np.float32)) if tracked else None
    p = torch.from_numpy(g.integers(0, 1 << 20, (pages, hkv, page)).astype(np.int32)) if tracked else None
    d = dev()
    cache = gbb.PagedCache(k.to(d).view(dtype), v.to(d).view(dtype), weights=None if w is None else w.to(d),
                           positions=None if p is None else p.to(d))
    i32 = lambda x: torch.tensor(np.asarray(x, np.int64).astype(np.int32), device=d)  # noqa: E731
    kept = np.asarray(kept, np.int64).reshape(B, most)
    n = gbb.cache_keep(cache, torch.from_numpy(bt).to(d), i32(lengths), i32(drafted), i32(kept), i32(counts))
    arrays = [x if x is None else x.numpy() for x in (k, v, w, p)]
    want, new = on.cache_keep(arrays, bt, list(lengths), list(drafted), kept, list(counts), pages, page)
    assert n.tolist() == new
    for got, ref in zip((cache.k.view(kind), cache.v.view(kind), cache.weights, cache.positions), want):
        assert (got is None) == (ref is None)
        if ref is not None:
            assert np.array_equal(got.cpu().numpy(), ref)
    return new


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", list(BITS), ids=str)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 256])
def test_keep(page, D, dtype):
    g = np.random.default_rng(page + D)
    lengths = [70, 33, 1, 40, 300, 16, 0, 25]
    drafted = [25, 33, 1, 1, 280, 16, 0, 25]
    counts = [6, 20, 1, 0, 150, 16, 0, 24]
    kept = np.full((8, 150), -7)
    for b in range(8):
        kept[b, :counts[b]] = np.sort(g.choice(max(1, drafted[b]), counts[b], replace=False))
    for tracked in (False, True):
        new = keep(lengths, drafted, kept, counts, dtype, page, 3, D, tracked, seed=D)
    assert new == [n - d + c for n, d, c in zip(lengths, drafted, counts)]


@pytest.mark.gpu
def test_last_token_of_a_long_draft_and_all_of_it():
    keep([1000], [600], [[599]], [1])
    keep([1000], [600], [list(range(600))], [600])
    keep([1000], [600], [list(range(1, 600)) + [0]], [599])
    keep([5, 9], [3, 2], np.zeros((2, 0)), [0, 0])


@pytest.mark.gpu
def test_what_makes_no_sense_is_left_alone():
    kept = [[0, 3, 5], [0, 3, 3], [3, 1, 5], [0, 1, 9], [-1, 1, 2], [0, 1, 2], [0, 1, 2], [0, 2, 4], [0, 2, 4]]
    lengths = [40, 40, 40, 40, 40, 40, 2, 40, 2 ** 20]
    drafted = [9, 9, 9, 9, 9, 9, 9, 9, 9]
    counts = [3, 3, 3, 3, 3, 4, 3, -1, 3]
    lengths[8] = 48
    new = keep(lengths, drafted, kept, counts, holes=[(8, 2)])
    assert new == [34, 40, 40, 40, 40, 40, 2, 40, 48]
    # a length beyond the pages, and a missing page that nothing moves through
    d = dev()
    cache = gbb.PagedCache.empty(4, 16, 1, 64, torch.float16, d)
    cache.k.copy_(torch.randn(cache.k.shape, device=d))
    before = cache.k.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)  # noqa: E731
    n = gbb.cache_keep(cache, i32([[0, 1]]), i32([33]), i32([5]), i32([[1]]), i32([1]))
    assert n.tolist() == [33] and torch.equal(cache.k, before)
    n = gbb.cache_keep(cache, i32([[-1, 1]]), i32([30]), i32([10]), i32([[4]]), i32([1]))
    assert n.tolist() == [21] and torch.equal(cache.k[1, 0, 4], before[1, 0, 8])


@pytest.mark.gpu
def test_in_a_graph_on_another_stream_with_a_given_output():
    d = dev()
    cache = gbb.PagedCache.empty(4, 16, 2, 64, torch.bfloat16, d, tracked=True)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=d)  # noqa: E731
    bt, lengths, drafted, kept, counts, out = i32([[2, 0, 1]]), i32([40]), i32([9]), i32([[1, 4, 8]]), i32([3]), i32([0])
    call = lambda: gbb.cache_keep(cache, bt, lengths, drafted, kept, counts, lengths_out=out)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert call() is out
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        rows = [[0, 2, 3], [1, 4, 8], [6, 7, 8]][i]
        cache.k.copy_(torch.randn(cache.k.shape, device=d))
        cache.positions.copy_(torch.randint(0, 99, cache.positions.shape, device=d))
        k, p = cache.k.clone(), cache.positions.clone()
        kept.copy_(torch.tensor([rows]))
        graph.replay()
        torch.cuda.synchronize()
        slot = lambda s: (int(bt[0, s // 16]), slice(None), s % 16)  # noqa: E731
        for j, r in enumerate(rows):
            assert torch.equal(cache.k[slot(31 + j)], k[slot(31 + r)]) and torch.equal(cache.positions[slot(31 + j)], p[slot(31 + r)])
        assert out.tolist() == [34]


def test_argument_refusals():
    L, C = gbb.lib(), gbb.binding._PagedCache
    c = C(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4, page=16,
          kv_heads=2, head_dim=64)

    def call(c=c, B=2, bt=9 << 20, mp=4, ln=10 << 20, dr=11 << 20, kp=12 << 20, mk=3, ct=13 << 20, out=14 << 20):
        return L.gbb_cache_keep(None if c is None else ctypes.byref(c), B, bt, mp, ln, dr, kp, mk, ct, out, None)

    assert call(B=0) == 0
    for bad in (dict(c=None), dict(B=-1), dict(mp=0), dict(mk=-1), dict(bt=None), dict(ln=None), dict(dr=None), dict(kp=None),
                dict(ct=None), dict(out=None), dict(out=10 << 20), dict(out=(11 << 20) + 4), dict(out=13 << 20),
                dict(out=(12 << 20) + 20), dict(out=(9 << 20) + 28)):
        assert call(**bad) == -1, bad
    assert call(B=1 << 22) == -2
    for bad in (dict(bt=2), dict(ln=2), dict(dr=2), dict(kp=2), dict(ct=2), dict(out=2)):
        assert call(**bad) == -4, bad
