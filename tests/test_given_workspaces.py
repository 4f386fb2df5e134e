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
