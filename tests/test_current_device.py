"""Calls on tensors of a GPU that is not the current one.  The library launches
on the current GPU and plans for it, so the binding has to make the tensors'
GPU the current one for the call and leave the caller's as it was.  Here with
tensors of the CPU, whose index is -1, beside a current GPU 0, and a library
that says which GPU was current."""
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


@pytest.fixture
def where(monkeypatch):
    """[(what was called, the current GPU then)]"""
    state, seen = {"current": 0}, []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["current"] = state["current"], self.index

        def __exit__(self, *a):
            state["current"] = self.before

    class FakeLib:
        def __getattr__(self, name):
            def call(*args):
                seen.append((name, state["current"]))
                return 64 if name.endswith("_workspace") else 0
            return call

    def capturing():
        seen.append(("capturing", state["current"]))
        return False

    def current():
        return state["current"]
    gbb.paged._resolve()
    fake = FakeLib()
    stream = type("S", (), {"cuda_stream": 0})()
    for owner, name, value in (
            (torch.cuda, "device", device), (torch.cuda, "current_device", current),
            (torch.cuda, "current_stream", lambda d=None: stream), (gbb.binding, "lib", lambda: fake),
            (gbb.binding, "_dev_ptr", lambda t, *a: t.data_ptr()), (gbb.binding, "_ws_cache", {}),
            (gbb.paged, "lib", lambda: fake), (gbb.paged, "_ws_cache", {}), (gbb.paged, "_resolve", lambda: None),
            (gbb.paged, "_raw_stream", lambda d: 0), (gbb.paged, "_capturing", capturing),
            (gbb.paged, "_current_device", current), (gbb.paged, "_device_of", lambda t, name: t.get_device()),
            (gbb.paged, "_buffer", lambda kind, n, d: torch.zeros(n, dtype=torch.uint8))):
        monkeypatch.setattr(owner, name, value, raising=False)
    yield seen
    assert state["current"] == 0
    assert seen and all(at == -1 for _, at in seen), seen


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def cache():
    k, v = (torch.zeros(2, 2, 16, 64, dtype=torch.float16) for _ in range(2))
    return gbb.PagedCache(k, v, weights=torch.zeros(2, 2, 16), positions=i32(2, 2, 16))


def test_rope(where):
    gbb.rope(torch.zeros(3, 2, 64), i32(3), torch.zeros(8, 32, 2))
    gbb.rope_append(cache(), torch.zeros(3, 8 * 64, dtype=torch.float16), 4, i32(3), i32(3), torch.zeros(8, 32, 2))


@pytest.mark.parametrize("workspace", [None, torch.zeros(64, dtype=torch.uint8)])
def test_attention_and_eviction(where, workspace):
    c, q = cache(), torch.zeros(1, 4, 64, dtype=torch.float16)
    gbb.paged_attention(c, q, i32(1, 2), i32(1), 32, workspace=workspace)
    gbb.cache_evict(c, i32(1, 2), i32(1), 32, 8, 2, workspace=workspace)
    if workspace is None:
        assert ("capturing", -1) in where


def test_plans(where):
    assert gbb.paged_attention_workspace(cache(), 1, 4, 32) == 64


@pytest.mark.parametrize("workspace", [None, torch.zeros(64, dtype=torch.uint8)])
def test_products(where, workspace):
    x, xq, image = torch.zeros(2, 128, dtype=torch.float16), torch.zeros(2, 128, dtype=torch.int8), torch.zeros(64, dtype=torch.uint8)
    y = torch.zeros(2, 64, dtype=torch.float16)
    gbb.gemm_mixed_w(image, 64, 128, x, workspace=workspace)
    gbb.gemm_mixed_w_64x64(image, 64, 128, x, workspace=workspace)
    gbb.gemm_mixed_w_noalloc(image, 64, 128, x)
    gbb.gemm_w48a8(image, 64, 128, 0, xq, x, workspace=workspace)
    gbb.gemm_w48a8(image, 64, 128, 0, xq, x, split=False)
    gbb.quant_act_i8(x)
    gbb.w48_group_acc(image, 64, 128, 0, xq)
    gbb.unpack_codes(image, 64, 128)
    gbb.dequant(image, 64, 128)
    gbb.Batched([(image, 64, 128, x, y)], workspace).launch()
    g = gbb.Graph([(image, 64, 128, x, y)], workspace)
    g.launch()
    g._g = None   # nothing to destroy
