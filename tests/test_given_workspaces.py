"""A caller's workspace: all of its bytes are given to the library, so a view
with gaps, whose other bytes belong to someone else, is refused."""
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


def never(*args):
    raise AssertionError("the library was called")


def views():
    buf = torch.zeros(64, 256, dtype=torch.uint8)   # on the CPU: GPU -1 to these checks
    return [buf[:, :128], buf.t(), buf[::2], torch.zeros(1, 1, dtype=torch.uint8).expand(1, 4096)]


@pytest.mark.parametrize("i", range(4))
def test_views_with_gaps_are_refused(i, monkeypatch):
    ws = views()[i]
    monkeypatch.setattr(gbb.paged, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(gbb.paged, "_current_device", lambda: -1)
    with pytest.raises(ValueError, match="contiguous"):
        gbb.paged._with_workspace("evict", -1, ws, never, (), never)


@pytest.mark.parametrize("i", range(4))
def test_views_with_gaps_are_refused_by_products(i, monkeypatch):
    ws = views()[i]
    x = torch.zeros(1, 128, dtype=torch.float16)

    class FakeLib:
        gbb_gemm_mixed_w_path = gbb_gemm_w48a8_split = never
        gbb_gemm_mixed_w_path_workspace = gbb_gemm_mixed_w_64x64_path_workspace = staticmethod(lambda *a: 64)
        gbb_gemm_mixed_w_64x64_path = gbb_gemm_mixed_w_batched = gbb_graph_create = never
        gbb_gemm_mixed_w_batched_workspace = gbb_gemm_mixed_w_workspace = staticmethod(lambda *a: 64)
    monkeypatch.setattr(gbb.binding, "lib", lambda: FakeLib)
    monkeypatch.setattr(gbb.binding, "_dev_ptr", lambda *a: 0)
    monkeypatch.setattr(gbb.binding, "_stream", lambda t: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    y = torch.zeros(1, 64, dtype=torch.float16)
    for call in (lambda: gbb.gemm_mixed_w(x, 64, 128, x, y, ws), lambda: gbb.gemm_mixed_w_64x64(x, 64, 128, x, y, ws),
                 lambda: gbb.gemm_w48a8(x, 64, 128, 0, x, x, out=y, workspace=ws),
                 lambda: gbb.Batched([(x, 64, 128, x, y)], ws), lambda: gbb.Graph([(x, 64, 128, x, y)], ws)):
        with pytest.raises(ValueError, match="contiguous"):
            call()


def test_the_bytes_of_a_whole_one():
    ws = torch.zeros(4, 256, dtype=torch.float32)
    assert gbb.binding._given(ws, -1) == (ws.data_ptr(), 4096)
    assert gbb.binding._given(ws[1:3], -1) == (ws.data_ptr() + 1024, 2048)
    with pytest.raises(ValueError, match="GPU 0"):
        gbb.binding._given(ws, 0)


@pytest.mark.parametrize("kind,cleared", [("attention", 16384), ("evict", 0)])
@pytest.mark.parametrize("captured", [False, True])
def test_only_counters_are_cleared(kind, cleared, captured, monkeypatch):
    """What a new workspace costs, in every replay of a graph that captured a
    call without one: its counters, not its size."""
    big, written = 300 << 20, []

    class Bytes:
        def __init__(self, n):
            self.n = n

        def __getitem__(self, part):
            return Bytes(len(range(self.n)[part]))

        def zero_(self):
            written.append(self.n)
            return self

        def numel(self):
            return self.n

        def data_ptr(self):
            return 0

    class FakeTorch:
        uint8 = None
        empty = staticmethod(lambda n, dtype, device: Bytes(n))
        zeros = staticmethod(lambda n, dtype, device: Bytes(n).zero_())
        device = staticmethod(lambda *a: None)
    for name, value in (("_torch", lambda: FakeTorch), ("_ws_cache", {}), ("_raw_stream", lambda d: 0),
                        ("_capturing", lambda: captured)):
        monkeypatch.setattr(gbb.paged, name, value)

    def call(ws, n, stream):
        return 0 if n >= big else -5
    gbb.paged._with_workspace(kind, 0, None, call, (), lambda: big)
    assert sum(written) == cleared * (1 if captured else 2)   # else: the first one was too small


@pytest.mark.gpu
@pytest.mark.parametrize("n,max_len", [(5000, 5000), (70, 70000), (40000, 70000)])
@pytest.mark.parametrize("weights", [False, True])
def test_attention_asks_for_zero_counters_only(n, max_len, weights):
    """Runs joined in the launch, by a second one, and with weights, over a
    workspace of NaN behind the counters: the bits of a zero one, twice."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d = torch.device("cuda", 0)
    torch.manual_seed(n)
    cache = gbb.PagedCache.empty(-(-max_len // 256), 256, 1, 64, torch.float16, d, tracked=True)
    cache.k.normal_()
    cache.v.normal_()
    q = torch.randn(1, 4, 64, device=d).half()
    bt = torch.randperm(cache.num_pages, device=d).to(torch.int32)[None]
    ln = torch.tensor([n], dtype=torch.int32, device=d)
    need = gbb.paged_attention_workspace(cache, 1, 4, max_len, weights)
    results = []
    for fill in (0, 255, 255):
        if fill == 0 or len(results) == 1:
            ws = torch.full((need,), fill, dtype=torch.uint8, device=d)
            ws[:16384] = 0
        w, lse = (torch.zeros_like(cache.weights) if weights else None), torch.zeros(1, 4, device=d)
        out = gbb.paged_attention(cache, q, bt, ln, max_len, lse=lse, weights_out=w, workspace=ws)
        assert torch.isfinite(out).all() and not ws[:16384].any()
        results.append([out, lse] + ([w] if weights else []))
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


def test_tensors_of_the_cpu_are_refused_as_such():
    """Before a GPU is asked for anything, with or without one."""
    x, y, image = torch.zeros(1, 128, dtype=torch.float16), torch.zeros(1, 64, dtype=torch.float16), torch.zeros(64, dtype=torch.uint8)
    for call in (lambda: gbb.gemm_mixed_w(image, 64, 128, x), lambda: gbb.gemm_mixed_w_64x64(image, 64, 128, x),
                 lambda: gbb.gemm_mixed_w_noalloc(image, 64, 128, x), lambda: gbb.Batched([(image, 64, 128, x, y)]),
                 lambda: gbb.Graph([(image, 64, 128, x, y)]), lambda: gbb.quant_act_i8(x), lambda: gbb.dequant(image, 64, 128),
                 lambda: gbb.gemm_w48a8(image, 64, 128, 0, x.to(torch.int8), x)):
        with pytest.raises(TypeError, match="torch tensor on a GPU"):
            call()
