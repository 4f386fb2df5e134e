"""Eviction by accumulated attention weight against the oracle: everything is
a selection or a copy, so everything is compared bit for bit."""
import ctypes

import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


def setup(lengths, hkv, D, page, ct, seed, weight="heavy", spare=2):
    g = np.random.default_rng(seed)
    per = max(1, -(-max(lengths) // page))
    used = [-(-max(0, n) // page) for n in lengths]
    pages = sum(used) + spare
    order = g.permutation(pages)
    bt = np.full((len(lengths), per), -5, np.int32)
    at = 0
    for b, n in enumerate(used):
        bt[b, :n] = order[at:at + n]
        at += n
    raw = lambda: g.integers(0, 256, (pages, hkv, page, D * (1 if ct == "e4m3" else 2)), np.uint8)  # noqa: E731
    k, v = (torch.from_numpy(raw()).view(DT[ct]) for _ in range(2))
    shape = (pages, hkv, page)
    w = {"heavy": lambda: np.exp(2 * g.standard_normal(shape)), "ties": lambda: g.integers(0, 3, shape),
         "equal": lambda: np.full(shape, 0.25), "wild": lambda: g.choice([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, -1.0, 1e-45, -1e-45, 3e38, -3e38], shape),
         "close": lambda: 1 + g.integers(0, 300, shape) * 2.0 ** -23}[weight]().astype(np.float32)
    pos = np.full(shape, -1, np.int32)
    for b, n in enumerate(lengths):
        for h in range(hkv):
            p = g.permutation(3 * max(0, n))[:max(0, n)]
            for j in range(max(0, n)):
                pos[bt[b, j // page], h, j % page] = p[j]
    return k, v, w, pos, bt


def run_and_check(lengths, hkv, D, page, ct, budget, recent, seed, weight="heavy", in_place=True, max_len=None, table=None):
    k, v, w, pos, bt = setup(lengths, hkv, D, page, ct, seed, weight)
    if table:
        table(bt)
    d = dev()
    max_len = max_len or max(1, max(lengths))
    want = od.cache_evict(bits(k), bits(v), w, pos, bt, [min(n, max_len) for n in lengths], budget, recent)
    c = gbb.PagedCache(k.to(d), v.to(d), weights=torch.from_numpy(w).to(d), positions=torch.from_numpy(pos).to(d))
    w0, p0 = c.weights.clone(), c.positions.clone()
    out = {} if in_place else dict(weights_out=torch.full_like(w0, -3.0), positions_out=torch.full_like(p0, -9))
    n = gbb.cache_evict(c, torch.from_numpy(bt).to(d), torch.tensor(lengths, dtype=torch.int32, device=d), max_len, budget,
                        recent, **out)
    assert np.array_equal(n.cpu().numpy(), want[4])
    assert np.array_equal(bits(c.k), want[0]) and np.array_equal(bits(c.v), want[1])
    want_w, want_p = want[2].astype(np.float32), want[3]
    if not in_place:
        assert torch.equal(c.weights.view(torch.int32), w0.view(torch.int32)) and torch.equal(c.positions, p0)
        named = np.zeros(w.shape, bool)   # slots below the lengths, of sequences whose pages are all there
        for b, ln in enumerate(lengths):
            ln = min(max(0, ln), max_len)
            pg = bt[b, :-(-ln // page)]
            if ((pg >= 0) & (pg < w.shape[0])).all():
                j = np.arange(ln)
                named[bt[b, j // page], :, j % page] = True
        want_w, want_p = np.where(named, want_w, -3.0).astype(np.float32), np.where(named, want_p, -9)
    got_w, got_p = (out["weights_out"], out["positions_out"]) if out else (c.weights, c.positions)
    # values rather than bits: a NaN's payload may differ
    assert np.array_equal(got_w.cpu().numpy(), want_w, equal_nan=True)
    assert np.array_equal(got_p.cpu().numpy(), want_p)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("ct,D,page", [("f16", 64, 16), ("f16", 128, 64), ("bf16", 256, 32), ("e4m3", 64, 256), ("e4m3", 128, 16)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (16, 4), (17, 17), (63, 0), (64, 10), (200, 32)])
def test_ragged(budget, recent, ct, D, page, in_place):
    run_and_check([0, 1, 15, 16, 17, 64, 65, 129, 200, 201, 333], 2, D, page, ct, budget, recent, budget + recent, in_place=in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("weight", ["ties", "equal", "wild", "close"])
@pytest.mark.parametrize("budget,recent", [(5, 0), (100, 20), (500, 500), (699, 3)])
def test_ties_and_special_weights(budget, recent, weight, in_place):
    run_and_check([700, 40, 501], 3, 64, 32, "f16", budget, recent, budget, weight, in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["heavy", "equal"])
@pytest.mark.parametrize("n,budget,recent", [(1024, 1023, 100), (1025, 1024, 100), (2049, 2048, 256), (4100, 1000, 128),
                                             (5000, 4900, 0), (9000, 64, 64)])
def test_long(n, budget, recent, weight):
    run_and_check([n, n - 1, budget, budget + 1], 2, 64, 64, "f16", budget, recent, n, weight)


@pytest.mark.gpu
@pytest.mark.parametrize("weight", ["heavy", "ties", "equal", "wild", "close"])
@pytest.mark.parametrize("budget,recent,in_place", [(1, 0, True), (4096, 100, False), (4095, 0, True), (4100, 4100, True),
                                                    (8192, 1000, True), (8999, 5, False), (5000, 64, False)])
def test_rows_over_several_workgroups(budget, recent, in_place, weight):
    """Rows above 32768 slots (a bound on the lengths above it takes short ones
    the same way), with the new length at, before and after the bounds of
    4096 slots that workgroups take."""
    run_and_check([33000, 9000, 8192, 4097, 8193, 100, 0], 1, 64, 64, "e4m3", budget, recent, budget, weight, in_place)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 70, 515])
def test_long_row_with_a_missing_page(page):
    def table(bt):
        bt[0, page] = -3
    run_and_check([33000, 8800], 1, 64, 64, "e4m3", 4500, 8, page, table=table)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,budget,recent", [(12000, 11950, 64), (12000, 40, 10), (16384, 16383, 0), (16385, 16384, 100),
                                             (20000, 7000, 1000), (32768, 20000, 0), (32768, 32767, 5)])
def test_rows_in_registers(n, budget, recent, in_place):
    run_and_check([n, n // 3, budget + 1], 1, 64, 128, "e4m3", budget, recent, n, "ties", in_place, max_len=n)


@pytest.mark.gpu
def test_one_very_long_sequence():
    run_and_check([40000], 1, 64, 256, "e4m3", 3000, 500, 40)


@pytest.mark.gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_missing_pages_leave_the_sequence(in_place):
    def table(bt):
        bt[0, 3], bt[1, 0] = -1, 10 ** 6
    run_and_check([100, 60, 80], 2, 64, 16, "f16", 40, 8, 7, in_place=in_place, table=table)


@pytest.mark.gpu
def test_lengths_above_the_bound_are_clamped():
    run_and_check([90, 70, 10], 2, 64, 16, "f16", 40, 8, 8, max_len=64)


@pytest.mark.gpu
def test_repeated_states_and_positions():
    """Equal positions (more slots than `recent` are the newest) and an int32
    range of positions."""
    d = dev()
    k, v, w, pos, bt = setup([120], 1, 64, 16, "f16", 9)
    for p in (np.zeros_like(pos), np.where(np.arange(pos.size).reshape(pos.shape) % 2, 2 ** 31 - 1, -2 ** 31).astype(np.int32)):
        want = od.cache_evict(bits(k), bits(v), w, p, bt, [120], 30, 10)
        c = gbb.PagedCache(k.to(d), v.to(d), weights=torch.from_numpy(w).to(d), positions=torch.from_numpy(p).to(d))
        n = gbb.cache_evict(c, torch.from_numpy(bt).to(d), torch.tensor([120], dtype=torch.int32, device=d), 120, 30, 10)
        assert n.item() == 30 and np.array_equal(bits(c.k), want[0]) and np.array_equal(c.positions.cpu().numpy(), want[3])
        assert np.array_equal(c.weights.cpu().numpy(), want[2].astype(np.float32))


@pytest.mark.gpu
def test_same_bits_on_a_stream_in_a_graph_and_again():
    d = dev()
    lengths = [500, 37, 260]
    k, v, w, pos, bt = setup(lengths, 2, 128, 32, "f16", 11)
    new = lambda: gbb.PagedCache(k.to(d), v.to(d), weights=torch.from_numpy(w).to(d), positions=torch.from_numpy(pos).to(d))  # noqa: E731
    btd, ld = torch.from_numpy(bt).to(d), torch.tensor(lengths, dtype=torch.int32, device=d)
    a = new()
    first = gbb.cache_evict(a, btd, ld, 500, 100, 10)
    b = new()
    ws = torch.empty(gbb.cache_evict_workspace(b, 3, 500, 100), dtype=torch.uint8, device=d).fill_(0xA5)
    n = torch.empty(3, dtype=torch.int32, device=d)
    w_out, p_out = b.weights.clone(), b.positions.clone()
    call = lambda: gbb.cache_evict(b, btd, ld, 500, 100, 10, w_out, p_out, n, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        n.zero_()
        w_out.fill_(0)
        b.k.copy_(k)
        b.v.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, first) and torch.equal(b.k.view(torch.int16), a.k.view(torch.int16))
        assert torch.equal(b.v.view(torch.int16), a.v.view(torch.int16))
        for s, ln in zip(range(3), lengths):
            j = torch.arange(ln, device=d)
            at = (btd[s].long()[j // 32], slice(None), j % 32)
            assert torch.equal(w_out[at], a.weights[at]) and torch.equal(p_out[at], a.positions[at])
    with pytest.raises(gbb.GbbError) as e:
        gbb.cache_evict(b, btd, ld, 500, 100, 10, w_out, p_out, n, ws[:-256])
    assert e.value.status == -5


@pytest.mark.gpu
def test_attention_does_not_see_the_order():
    """The kept slots in their new places give the attention of the same
    tokens in order, to the rounding of the sums' order (fp32 sums of 64
    terms and one fp16 rounding of values below 4)."""
    d = dev()
    g = np.random.default_rng(12)
    k, v, w, pos, bt = setup([160], 1, 64, 16, "f16", 12)
    k, v = (torch.from_numpy(g.standard_normal(k.shape).astype(np.float16)) for _ in range(2))
    c = gbb.PagedCache(k.to(d), v.to(d), weights=torch.from_numpy(w).to(d), positions=torch.from_numpy(pos).to(d))
    q = torch.randn(1, 2, 64, device=d, dtype=torch.float16)
    btd = torch.from_numpy(bt).to(d)
    n = gbb.cache_evict(c, btd, torch.tensor([160], dtype=torch.int32, device=d), 160, 64, 8)
    got = gbb.paged_attention(c, q, btd, n, 160)
    left = c.positions.cpu().numpy()
    kept = set(left[bt[0, np.arange(64) // 16], 0, np.arange(64) % 16].tolist())
    assert len(kept) == 64
    old = [j for j in range(160) if pos[bt[0, j // 16], 0, j % 16] in kept]
    kk, vv = (x.double().numpy()[bt[0, np.array(old) // 16], 0, np.array(old) % 16] for x in (k, v))
    s = q[0].double().cpu().numpy() @ kk.T / 8
    p = np.exp(s - s.max(-1, keepdims=True))
    ref = p @ vv / p.sum(-1, keepdims=True)
    assert np.abs(got[0].double().cpu().numpy() - ref).max() <= 2.0 ** -11 * 4 + 2.0 ** -13


def test_argument_refusals():
    """Checked before anything touches a device."""
    L, C = gbb.lib(), gbb.binding._PagedCache
    W, P = 3 << 20, 4 << 20
    base = dict(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=W, positions=P, dtype=0, num_pages=4, page=16,
                kv_heads=2, head_dim=64)

    def call(c=None, B=2, bt=9 << 20, mp=4, ln=10 << 20, ml=64, budget=32, recent=4, lo=11 << 20, wo=W, po=P, ws=1 << 24, wb=1 << 30):
        cc = C(**{**base, **(c or {})})
        return L.gbb_cache_evict(ctypes.byref(cc), B, bt, mp, ln, ml, budget, recent, lo, wo, po, ws, wb, None)

    assert call(B=0) == 0
    for bad in (dict(c=dict(k=None)), dict(c=dict(weights=None)), dict(c=dict(positions=None)), dict(B=-1), dict(bt=None),
                dict(ln=None), dict(ml=0), dict(budget=0), dict(recent=-1), dict(recent=33), dict(lo=None), dict(wo=None),
                dict(po=None), dict(lo=10 << 20), dict(lo=(10 << 20) + 4), dict(wo=W + 16), dict(po=P - 16), dict(ws=None)):
        assert call(**bad) == -1, bad
    for bad in (dict(c=dict(page=48)), dict(c=dict(head_dim=80)), dict(ml=65), dict(B=1 << 20, c=dict(kv_heads=8))):
        assert call(**bad) == -2, bad
    for bad in (dict(bt=(9 << 20) + 2), dict(lo=(11 << 20) + 1), dict(wo=(12 << 20) + 2), dict(ws=(1 << 24) + 4)):
        assert call(**bad) == -4, bad
    assert call(wb=16) == -5
    cc = C(**base)
    assert L.gbb_cache_evict_workspace(ctypes.byref(cc), 2, 64, 0) == 0
    assert L.gbb_cache_evict_workspace(ctypes.byref(cc), 2, 64, 32) > 0
