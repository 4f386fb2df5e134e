"""The rotary positions in torch's differentiation: the gradient is the
transposed rotation, in place too, and a write that is not differentiated is
seen by what saved the memory before."""
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")


@pytest.fixture
def calls(monkeypatch):
    """`transpose` of the library's calls, on tensors of the CPU."""
    seen = []

    class FakeLib:
        @staticmethod
        def gbb_rope(*args):
            seen.append(args[-2])
            return 0
    gbb.paged._resolve()
    for name, value in (("lib", lambda: FakeLib), ("_raw_stream", lambda d: 0), ("_current_device", lambda: -1),
                        ("_device_of", lambda t, name: t.get_device())):
        monkeypatch.setattr(gbb.paged, name, value)
    return seen


@pytest.mark.parametrize("transpose", [False, True])
def test_what_is_differentiated(calls, transpose):
    x = torch.zeros(3, 2, 64, requires_grad=True)
    rest = (torch.zeros(3, dtype=torch.int32), torch.zeros(8, 32, 2))
    y = gbb.rope(x, *rest, transpose=transpose)
    assert y.requires_grad and calls == [int(transpose)]
    y.sum().backward()   # a gradient with strides 0
    assert x.grad is not None and x.grad.shape == x.shape and calls == [int(transpose), int(not transpose)]
    with torch.no_grad():
        assert not gbb.rope(x, *rest).requires_grad
    assert not gbb.rope(x.detach(), *rest).requires_grad
    assert len(calls) == 4


def test_writes_are_seen(calls):
    rest = (torch.zeros(3, dtype=torch.int32), torch.zeros(8, 32, 2))
    w = torch.zeros(3, 2, 64, requires_grad=True)
    x = torch.zeros(3, 2, 64)
    z = w * x   # x is saved for w's gradient
    gbb.rope(x, *rest, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.sum().backward()
    with pytest.raises(RuntimeError, match="leaf"):
        gbb.rope(w, *rest, out=w)
    y = w + 0.0
    before = y._version
    assert gbb.rope(y, *rest, out=y) is y and y.requires_grad and y._version > before
    out = torch.zeros(3, 2, 64)
    assert gbb.rope(w, *rest, out=out) is out and out.requires_grad
    with torch.inference_mode():
        u = torch.zeros(3, 2, 64)
        assert gbb.rope(u, *rest, out=u) is u


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gradients(dtype, layout):
    """Bit for bit the transposed call's, through new, given and in-place
    outputs, of views, and for a second derivative."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d = torch.device("cuda", 0)
    torch.manual_seed(0)
    table = torch.from_numpy(gbb.rope_table(48, 64, attention=1.1)).to(d)
    pos = torch.tensor([5, 0, 63, -1, 9], dtype=torch.int32, device=d)   # the fourth token is padding
    x = torch.randn(5, 3, 80, device=d).to(dtype).requires_grad_()
    go = torch.randn(5, 3, 80, device=d).to(dtype)
    want = gbb.rope(go, pos, table, layout=layout, transpose=True)
    assert not want[3].any()
    value = gbb.rope(x.detach(), pos, table, layout=layout)
    for way in ("new", "given", "in place", "heads outside"):
        x.grad = None
        h = x * 1.0
        if way == "heads outside":
            h = h.transpose(0, 1).contiguous().transpose(0, 1)
        out = {"new": None, "given": torch.empty_like(value), "in place": h, "heads outside": h}[way]
        y = gbb.rope(h, pos, table, layout=layout, out=out)
        assert torch.equal(y, value)
        y.backward(go)
        assert torch.equal(x.grad, want), way
    # the map is linear: the gradient of <rope(g), v> with respect to g is rope's transpose of v
    g = go.clone().requires_grad_()
    first, = torch.autograd.grad(gbb.rope(x, pos, table, layout=layout), x, g, create_graph=True)
    second, = torch.autograd.grad(first, g, value)
    assert torch.equal(second, gbb.rope(value, pos, table, layout=layout))


@pytest.mark.gpu
def test_gradient_against_differences():
    """As in the linear map's own test: a central difference is exact but for
    fp32's rounding, here through autograd's backward pass."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    d = torch.device("cuda", 0)
    torch.manual_seed(1)
    table = torch.from_numpy(gbb.rope_table(64, 4096)).to(d)
    pos = torch.randint(0, 4096, (6,), device=d, dtype=torch.int32)
    x, v, go = (torch.randn(6, 3, 96, device=d) for _ in range(3))
    x.requires_grad_()
    (gbb.rope(x, pos, table) * go).sum().backward()
    h = 2.0 ** -3
    with torch.no_grad():
        f = lambda t: (gbb.rope(t, pos, table).double() * go.double()).sum().item()  # noqa: E731
        num = (f(x + h * v) - f(x - h * v)) / (2 * h)
        ana = (x.grad.double() * v.double()).sum().item()
        bound = (2.0 ** -22 * 2 * (x.abs() + h * v.abs()).max().item() * go.abs().sum().item()) / h + 1e-6 * abs(ana)
    assert abs(num - ana) <= bound


def test_what_is_no_tensor_is_refused_as_before():
    with pytest.raises(TypeError, match="x must be a torch tensor on a GPU"):
        gbb.rope([1.0], None, None)
