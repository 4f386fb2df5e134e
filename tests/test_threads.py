"""Calls of several Python threads on one stream.  A call's launches meet in a
workspace that the binding keeps per stream, so no other call's may come
between them."""
import threading
import time

import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


class Library:
    """Stands for an entry point: says which calls overlapped on a buffer."""

    def __init__(self, at):
        self.at, self.inside, self.overlapped, self.calls = at, {}, 0, 0   # at: the workspace among the arguments

    def __call__(self, *args):
        at = args[self.at]
        self.calls += 1
        if self.inside.setdefault(at, 0):
            self.overlapped += 1
        self.inside[at] += 1
        time.sleep(0.005)
        self.inside[at] -= 1
        return 0


class Buffer:
    def __init__(self, n):
        self.n = n

    def data_ptr(self):
        return id(self)

    def numel(self):
        return self.n


def in_threads(n, work):
    start, errors = threading.Barrier(n), []

    def one(i):
        start.wait()
        try:
            work(i)
        except BaseException as e:   # told to the test below
            errors.append(e)

    threads = [threading.Thread(target=one, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_paged_calls_on_one_stream_do_not_overlap(monkeypatch):
    call = Library(at=-3)
    monkeypatch.setattr(gbb.paged, "_ws_cache", {})
    monkeypatch.setattr(gbb.paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(gbb.paged, "_current_device", lambda: 0)
    monkeypatch.setattr(gbb.paged, "_capturing", lambda: False)
    monkeypatch.setattr(gbb.paged, "_buffer", lambda kind, n, device: Buffer(n))
    in_threads(4, lambda i: [gbb.paged._with_workspace("evict", 0, None, call, (), lambda: 16) for _ in range(5)])
    assert call.calls == 20 and len(call.inside) == 1 and not call.overlapped


def test_paged_calls_grow_one_buffer(monkeypatch):
    """A call that finds the buffer too small replaces it for all threads."""
    seen = []

    def call(ws, n, stream):
        seen.append(n)
        return 0 if n >= 2 << 20 else -5
    monkeypatch.setattr(gbb.paged, "_ws_cache", {})
    monkeypatch.setattr(gbb.paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(gbb.paged, "_current_device", lambda: 0)
    monkeypatch.setattr(gbb.paged, "_capturing", lambda: False)
    monkeypatch.setattr(gbb.paged, "_buffer", lambda kind, n, device: Buffer(n))
    in_threads(4, lambda i: gbb.paged._with_workspace("attention", 0, None, call, (), lambda: 2 << 20))
    assert sorted(seen) == [1 << 20] + [2 << 20] * 4


def test_product_calls_on_one_stream_do_not_overlap(monkeypatch):
    call = Library(at=-4)

    class FakeTorch:
        uint8 = float16 = None
        zeros = staticmethod(lambda n, dtype, device: Buffer(n))

        class cuda:
            current_device = staticmethod(lambda: 0)
            current_stream = staticmethod(lambda device: type("S", (), {"cuda_stream": 0}))

    class FakeLib:
        gbb_gemm_mixed_w_path = call
        gbb_gemm_mixed_w_path_workspace = staticmethod(lambda N, K, M, path: 64)
    x = type("X", (), {"shape": (1, 128), "dim": lambda self: 2, "device": "gpu", "get_device": lambda self: 0})()
    for name, value in (("_ws_cache", {}), ("_torch", lambda: FakeTorch), ("lib", lambda: FakeLib),
                        ("_dev_ptr", lambda *a: 0), ("_stream", lambda t: 0)):
        monkeypatch.setattr(gbb.binding, name, value)
    in_threads(4, lambda i: [gbb.gemm_mixed_w(x, 64, 128, x, out=x) for _ in range(5)])
    assert call.calls == 20 and len(call.inside) == 1 and not call.overlapped


@pytest.mark.gpu
def test_evictions_and_weighted_attention_of_two_threads():
    """Two threads, one stream, caches of different sizes, calls that take two
    launches each: the bits of the same calls one after the other."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d = torch.device("cuda", 0)

    def setup(seed, n, hkv, D, page, budget):
        g = torch.Generator(device=d).manual_seed(seed)
        pages = -(-n // page)
        c = gbb.PagedCache.empty(pages, page, hkv, D, torch.float16, d, tracked=True)
        c.k.normal_(generator=g)
        c.v.normal_(generator=g)
        c.weights.uniform_(generator=g)
        bt = torch.randperm(pages, generator=g, device=d).to(torch.int32)[None]
        at = torch.arange(n, dtype=torch.int32, device=d)
        c.positions[bt[0, at.long() // page].long(), :, at.long() % page] = at[:, None].expand(n, hkv)
        q = torch.randn(1, 2 * hkv, D, generator=g, device=d).half()
        return c, q, bt, torch.tensor([n], dtype=torch.int32, device=d), n, budget

    cases = [setup(1, 3000, 2, 64, 64, 1200), setup(2, 1500, 5, 128, 16, 400)]

    def steps(case, rounds):
        c, q, bt, ln, n, budget = case
        keep = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
        out = []
        for _ in range(rounds):
            for t, k in zip((c.k, c.v, c.weights, c.positions), keep):
                t.copy_(k)
            o = gbb.paged_attention(c, q, bt, ln, n, weights_out=c.weights)
            gbb.cache_evict(c, bt, ln, n, budget, 50)
            out.append([t.clone() for t in (o, c.k, c.v, c.weights, c.positions)])
        for t, k in zip((c.k, c.v, c.weights, c.positions), keep):
            t.copy_(k)
        return out

    want = [steps(c, 1)[0] for c in cases]
    got = [None, None]

    def work(i):
        got[i] = steps(cases[i], 30)
    in_threads(2, work)
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            for a, b in zip(result, want[i]):
                assert np.array_equal(a.cpu().view(torch.int16 if a.element_size() == 2 else torch.int32).numpy(),
                                      b.cpu().view(torch.int16 if b.element_size() == 2 else torch.int32).numpy())
