"""Norms of heads with rotary positions of one or several axes, their gradient
and the cache write, against the 64-bit oracle.

Tolerances.  With u = 2^-24: a sum of D squares in fp32 is within D u of exact
relatively, its inverse root within D u / 2 + 3 u, so a normed and weighted
element is within (D / 2 + 6) u of itself, and a rotated one within (D / 2 + 9) u
times (|n1| + |n2|) |table| (n the normed pair), before its one rounding.  The
gradient: g is within 3 u (|dy1| + |dy2|) |table|; mean(g w xh) is a sum of D
terms, within (D + 12) u mean|g w xh|; so dx is within (D + 16) u r (|g w| + |xh|
mean|g w xh|) with |g| taken as (|dy1| + |dy2|) |table|.  dw sums N terms, each
within (D / 2 + 12) u, in fp32 in any order: (D / 2 + 12 + N) u times the sum of
their magnitudes."""
import ctypes

import numpy as np
import pytest

from oracle import decode_step as od
from oracle import new_tokens as on

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -149}
U = 2.0 ** -24
EPS = 1e-6


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def wide(t):
    return t.detach().double().cpu().numpy()


def pair_sum(a, half, layout):
    """|a| summed over each element's pair (itself alone beyond the pairs)."""
    out = np.abs(a).astype(np.float64)
    for i in range(half):
        x, y = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        out[..., x] = out[..., y] = np.abs(a[..., x]) + np.abs(a[..., y])
    return out


class Case:
    def __init__(self, T, H, D, rot, layout="half", dt="f16", wt="f32", sections=None, seed=0, padding=()):
        g = np.random.default_rng(seed)
        self.layout, self.dt, self.sections, self.n_pos = layout, dt, sections, 50
        self.axes = 1 if sections is None else len(sections)
        self.table = (gbb.rope_table(rot, self.n_pos) * 1.25).astype(np.float32)
        pos = g.integers(0, self.n_pos, (self.axes, T)).astype(np.int32)
        for t in padding:
            if t < T:
                pos[t % self.axes, t] = (-1, self.n_pos, 2 ** 31 - 1, -2 ** 31)[t % 4]
        self.pos = pos
        f = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32))  # noqa: E731
        self.x = (f(T, H, D) * torch.from_numpy(np.exp(g.uniform(-6, 3, (T, H, 1))).astype(np.float32))).to(DT[dt])
        self.dy = f(T, H, D).to(DT[dt])
        self.w = None if wt is None else (1 + 0.5 * f(D)).to(DT[dt] if wt == "same" else DT[wt])
        self.D, self.half = D, rot // 2

    def dev(self, *names):
        pos = self.pos if self.sections is not None else self.pos[0]
        d = {"positions": torch.from_numpy(pos.copy()), "table": torch.from_numpy(self.table)}
        return [x.to(dev()) if x is not None else None
                for x in (d.get(n) if n in d else getattr(self, n) for n in names)]

    def axis_sections(self):
        return self.sections or (self.half,)

    def check_forward(self, got, x=None, norm=True):
        x = wide(self.x if x is None else x)
        w = None if self.w is None or not norm else wide(self.w)
        args = (self.pos, self.axis_sections(), self.table, self.layout)
        ref = on.norm_rope(x, w, EPS, *args) if norm else on.rope_axes(x, *args)
        n = x
        if norm:
            n = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * (1 if w is None else w)
        pre = (self.D / 2 + 9 if norm else 3) * U * pair_sum(n, self.half, self.layout) * 1.25
        tol = pre + UNIT[self.dt] * (np.abs(ref) + pre) + TINY[self.dt]
        bad = np.abs(wide(got) - ref) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], (np.abs(wide(got) - ref) / tol).max())

    def check_grad(self, dx, dw):
        x, dy = wide(self.x), wide(self.dy)
        w = None if self.w is None else wide(self.w)
        rx, rw, mass = on.norm_rope_grad(x, dy, w, EPS, self.pos, self.axis_sections(), self.table, self.layout)
        if dx is not None:
            r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
            gw = pair_sum(dy, self.half, self.layout) * 1.25 * (1 if w is None else np.abs(w))
            u = np.abs(x) * r
            pre = (self.D + 16) * U * r * (gw + u * (gw * u).mean(-1, keepdims=True))
            tol = pre + UNIT[self.dt] * (np.abs(rx) + pre) + TINY[self.dt]
            assert np.all(np.abs(wide(dx) - rx) <= tol), (np.abs(wide(dx) - rx) / tol).max()
        if dw is not None:
            N = x.shape[0] * x.shape[1]
            g = pair_sum(dy, self.half, self.layout) * 1.25
            terms = (g * np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)).sum((0, 1))
            pre = (self.D / 2 + 12 + N) * U * terms
            unit = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dw.dtype]
            tol = pre + unit * (np.abs(rw) + pre) + 2.0 ** -25
            assert np.all(np.abs(wide(dw) - rw) <= tol), (np.abs(wide(dw) - rw) / tol).max()


SHAPES = [(1, 1, 2, 2), (3, 2, 64, 64), (5, 3, 80, 40), (17, 5, 96, 24), (9, 7, 128, 128), (33, 2, 250, 50),
          (4, 3, 256, 128), (2, 2, 1024, 1024), (3, 1, 1024, 10), (2, 33, 66, 66), (130, 1, 128, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_norm_and_gradient(shape, layout, dt):
    T, H, D, rot = shape
    for wt in ("f32", "same", None):
        c = Case(T, H, D, rot, layout, dt, wt, seed=D + T, padding=(2, 5, 7))
        x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
        x.requires_grad_()
        if w is not None:
            w.requires_grad_()
        y = gbb.norm_rope(x, w, p, t, eps=EPS, layout=layout)
        c.check_forward(y)
        y.backward(dy)
        assert x.grad.dtype == x.dtype and (w is None or w.grad.dtype == w.dtype)
        c.check_grad(x.grad, None if w is None else w.grad)
        with torch.no_grad():
            assert torch.equal(gbb.norm_rope(x, w, p, t, eps=EPS, layout=layout), y)


SECTIONS = [(16, 8, 8), (0, 32), (10, 0, 0, 22), (32,), (1, 31)]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("sections", SECTIONS, ids=str)
def test_axes(sections, layout, dt):
    for D in (64, 72):
        c = Case(21, 3, D, 64, layout, dt, sections=sections, seed=len(sections), padding=(1, 6, 8))
        x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
        c.check_forward(gbb.rope(x, p, t, layout=layout, sections=sections), norm=False)
        x.requires_grad_()
        w.requires_grad_()
        y = gbb.norm_rope(x, w, p, t, eps=EPS, layout=layout, sections=list(sections))
        c.check_forward(y)
        c.check_grad(*torch.autograd.grad(y, (x, w), dy))
        turned = gbb.rope(x, p, t, layout=layout, sections=sections)
        back = torch.autograd.grad(turned, x, dy)[0]
        assert torch.equal(back, gbb.rope(dy, p, t, layout=layout, sections=sections, transpose=True))


@pytest.mark.gpu
def test_one_axis_given_as_a_section_is_rope():
    c = Case(40, 6, 128, 128, "half", "bf16", sections=(64,), seed=3, padding=(3,))
    x, p, t = c.dev("x", "positions", "table")
    assert torch.equal(gbb.rope(x, p, t, sections=(64,)), gbb.rope(x, p[0].contiguous(), t))
    assert torch.equal(gbb.rope(x, p, t, sections=(64,), transpose=True), gbb.rope(x, p[0].contiguous(), t, transpose=True))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_strides_and_places(dt):
    """Views of a wider row, odd offsets, heads outermost, broadcast inputs, in
    place, a given output."""
    c = Case(11, 4, 64, 64, "half", dt, seed=5)
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    want = gbb.norm_rope(x, w, p, t)
    c.check_forward(want)
    for off in (0, 1, 2, 8):
        row = torch.full((11, 4 * 64 + 24), float("nan"), device=x.device, dtype=x.dtype)
        view = row[:, off:off + 256].unflatten(1, (4, 64))
        view.copy_(x)
        got = gbb.norm_rope(view, w, p, t)
        c.check_forward(got)
        assert gbb.norm_rope(view, w, p, t, out=view) is view
        assert torch.equal(view, got)
        assert torch.isnan(row[:, :off]).all() and torch.isnan(row[:, off + 256:]).all()
    heads = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert torch.equal(gbb.norm_rope(heads, w, p, t), want)
    out = torch.empty_like(heads)
    assert gbb.norm_rope(heads, w, p, t, out=out) is out and torch.equal(out, want)
    shifted = torch.empty(65, device=x.device)[1:]   # a weight at an odd address
    shifted.copy_(w)
    c.check_forward(gbb.norm_rope(x, shifted, p, t))
    # one head read by all, and its gradient the sum over them
    one = x[:, :1].clone().requires_grad_()
    y = gbb.norm_rope(one.expand(11, 4, 64), w, p, t)
    parts = [gbb.norm_rope(one, w, p, t) for _ in range(4)]
    assert torch.equal(y, torch.cat(parts, 1))
    g = torch.autograd.grad(y, one, dy)[0]
    each = [torch.autograd.grad(q, one, dy[:, i:i + 1].contiguous())[0].double() for i, q in enumerate(parts)]
    total = sum(each)
    assert (g.double() - total).abs().max() <= 8 * UNIT[dt] * sum(e.abs() for e in each).max()
    # a gradient that is one number everywhere
    leaf = x.clone().requires_grad_()
    flat = torch.autograd.grad(gbb.norm_rope(leaf, w, p, t).sum(), leaf)[0]
    assert torch.equal(flat, torch.autograd.grad(gbb.norm_rope(leaf, w, p, t), leaf, torch.ones_like(x))[0])


@pytest.mark.gpu
def test_gradient_against_differences():
    """fp32, central differences of a scalar function in 64 bits: within the
    kernel's error and h^2."""
    c = Case(3, 2, 16, 8, "interleaved", "f32", seed=9, sections=(1, 3))
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    x.requires_grad_()
    w.requires_grad_()
    gx, gw = torch.autograd.grad(gbb.norm_rope(x, w, p, t, eps=EPS, layout="interleaved", sections=(1, 3)), (x, w), dy)
    f = lambda a, b: (on.norm_rope(a, b, EPS, c.pos, (1, 3), c.table, "interleaved") * wide(dy)).sum()  # noqa: E731
    x0, w0 = wide(x), wide(w)
    for got, base, which in ((wide(gx), x0, 0), (wide(gw), w0, 1)):
        scale = np.abs(got).max()
        for i in np.ndindex(base.shape):
            size = np.sqrt((x0[i[:2]] ** 2).mean()) if which == 0 else 1.0
            h = 1e-4 * size
            up, dn = base.copy(), base.copy()
            up[i] += h
            dn[i] -= h
            d = (f(up, w0) - f(dn, w0) if which == 0 else f(x0, up) - f(x0, dn)) / (2 * h)
            assert abs(got[i] - d) <= 1e-5 * max(scale, abs(d))


@pytest.mark.gpu
def test_what_is_asked_for():
    """Gradients of x or of the weight alone; many tokens, whose weight
    gradient is summed over all workgroups, the same bits each time."""
    c = Case(3000, 3, 64, 64, "half", "bf16", seed=11, padding=(100,))
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    w1 = w.clone().requires_grad_()
    y = gbb.norm_rope(x, w1, p, t)
    dw = torch.autograd.grad(y, w1, dy)[0]
    x1 = x.clone().requires_grad_()
    dx = torch.autograd.grad(gbb.norm_rope(x1, w, p, t), x1, dy)[0]
    c.check_grad(dx, dw)
    for _ in range(3):
        ax, aw = x.clone().requires_grad_(), w.clone().requires_grad_()
        gx, gw = torch.autograd.grad(gbb.norm_rope(ax, aw, p, t), (ax, aw), dy)
        assert torch.equal(gx, dx) and torch.equal(gw, dw)
    none = x[:0].clone().requires_grad_()
    w2 = w.clone().requires_grad_()
    y = gbb.norm_rope(none, w2, p[:0], t)
    gx, gw = torch.autograd.grad(y, (none, w2), torch.zeros_like(y))
    assert gx.shape == (0, 3, 64) and not gw.any()
    with pytest.raises(ValueError):
        gbb.norm_rope(x1, w, p, t, out=torch.empty_like(x))
    y = gbb.norm_rope(x1, w, p, t)
    g = torch.autograd.grad(y, x1, dy.clone().requires_grad_(), create_graph=True)[0]
    with pytest.raises(RuntimeError):
        g.sum().backward()
    z = x.clone().requires_grad_() * 1
    y = gbb.norm_rope(z, w, p, t)
    z.add_(1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


@pytest.mark.gpu
def test_nan_stays_in_its_head_and_out_of_padding():
    c = Case(6, 2, 64, 64, "half", "f16", seed=12, padding=(1,))
    c.x[1] = float("nan")
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    x[4, 1, 3] = float("nan")
    w1, x1 = w.clone().requires_grad_(), x.clone().requires_grad_()
    y = gbb.norm_rope(x1, w1, p, t)
    bad = torch.isnan(y).any(-1)
    assert not y[1].any() and bad.sum() == 1 and bad[4, 1]
    dx, dw = torch.autograd.grad(y, (x1, w1), dy)
    assert not dx[1].any() and torch.isnan(dx).any(-1).sum() == 1 and torch.isnan(dw).all()
    x1 = x[:4].clone().requires_grad_()   # without that head the padding's NaN reaches nothing
    dx, dw = torch.autograd.grad(gbb.norm_rope(x1, w1, p[:4], t), (x1, w1), dy[:4])
    assert torch.isfinite(dw).all() and torch.isfinite(dx).all()
    zero = torch.zeros(2, 1, 64, device=x.device)
    assert not gbb.norm_rope(zero, w, p[2:4].clone(), t, eps=EPS).any()


@pytest.mark.gpu
def test_forward_and_backward_in_a_graph():
    c = Case(700, 4, 128, 128, "half", "bf16", seed=13)
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    x.requires_grad_()
    w.requires_grad_()
    step = lambda: torch.autograd.grad(gbb.norm_rope(x, w, p, t), (x, w), dy)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gx, gw = step()
    for i in range(4):
        with torch.no_grad():
            x.mul_(-0.5).add_(0.1 * i)
        graph.replay()
        torch.cuda.synchronize()
        ex, ew = step()
        assert torch.equal(ex, gx) and torch.equal(ew, gw)


# ----------------------------------------------------------------------------
# on the way into the cache
# ----------------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 64), (128, 10), (256, 256), (256, 2)])
@pytest.mark.parametrize("dt,ct", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
def test_append(dt, ct, D, rot, layout):
    hq, hkv, page, pages, T = 6, 2, 16, 4, 29
    g = np.random.default_rng(D + rot)
    first = rot // 4
    for sections, wt in ((None, "same"), ((first, rot // 2 - first), "f32"), ((first, rot // 2 - first), None)):
        ctype = DT.get(ct, torch.float8_e4m3fn)
        kw, ks, vs = {}, np.ones(hkv), np.ones(hkv)
        if ct == "e4m3":
            ks, vs = g.uniform(0.01, 0.03, hkv).astype(np.float32), g.uniform(0.01, 0.03, hkv).astype(np.float32)
            kw = dict(k_scale=torch.from_numpy(ks).to(dev()), v_scale=torch.from_numpy(vs).to(dev()))
        cache = gbb.PagedCache.empty(pages, page, hkv, D, ctype, dev(), tracked=True, **kw)
        cache.weights.fill_(7.0)
        slots = g.permutation(pages * page)[:T].astype(np.int32)
        slots[3], slots[4] = -1, pages * page
        axes = 1 if sections is None else 2
        pos = g.integers(0, 40, (axes, T)).astype(np.int32)
        pos[-1, 5] = 40
        table = gbb.rope_table(rot, 40)
        qkv = torch.from_numpy((2 * g.standard_normal((T, (hq + 2 * hkv) * D))).astype(np.float32)).to(DT[dt])
        ws = [None, None]
        if wt is not None:
            ws = [torch.from_numpy((1 + 0.5 * g.standard_normal(D)).astype(np.float32)).to(DT[dt] if wt == "same" else DT[wt])
                  for _ in range(2)]
        wd = [None if w is None else w.to(dev()) for w in ws]
        dpos = torch.from_numpy(pos if sections else pos[0]).to(dev())
        q = gbb.rope_append(cache, qkv.to(dev()), hq, dpos, torch.from_numpy(slots).to(dev()),
                            torch.from_numpy(table).to(dev()), layout=layout, q_norm=wd[0], k_norm=wd[1], eps=EPS,
                            sections=sections)
        x = wide(qkv).reshape(T, hq + 2 * hkv, D)
        sec = sections or (rot // 2,)

        def want(part, w):
            if w is None:
                return on.rope_axes(part, pos, sec, table, layout), part
            w = wide(w)
            return (on.norm_rope(part, w, EPS, pos, sec, table, layout),
                    part / np.sqrt((part * part).mean(-1, keepdims=True) + EPS) * w)
        (rq, nq), (rk, nk) = want(x[:, :hq], ws[0]), want(x[:, hq:hq + hkv], ws[1])
        padding = np.isin(np.arange(T), [3, 4, 5])
        rq[padding] = 0.0
        pre = (D / 2 + 9) * U * pair_sum(nq, rot // 2, layout)
        assert np.all(np.abs(wide(q) - rq) <= pre + UNIT[dt] * (np.abs(rq) + pre) + TINY[dt])
        stay = np.ones((pages, page), bool)
        for t in np.flatnonzero(~padding):
            pg, off = slots[t] // page, slots[t] % page
            stay[pg, off] = False
            pk = (D / 2 + 9) * U * pair_sum(nk, rot // 2, layout)[t]
            for got, ref, pre, sc in ((cache.k, rk[t], pk, ks), (cache.v, x[t, hq + hkv:], 0.0, vs)):
                have = wide(got)[pg, :, off]
                if ct == "e4m3":
                    ref, pre = ref / sc[:, None], pre / sc[:, None] + U * np.abs(ref / sc[:, None])
                    # a value near a border may go either way
                    low, high = (od.e4m3_values()[od.e4m3_encode(ref + s * pre)] for s in (-1, 1))
                    assert np.all((have >= low) & (have <= high))
                else:
                    assert np.all(np.abs(have - ref) <= pre + UNIT[ct] * (np.abs(ref) + pre) + TINY[ct])
            assert (cache.positions.cpu().numpy()[pg, :, off] == pos[0, t]).all()
            assert not cache.weights.cpu().numpy()[pg, :, off].any()
        mask = torch.from_numpy(stay)[:, None].expand(-1, hkv, -1).to(dev())
        assert not cache.k.float()[mask].any() and not cache.v.float()[mask].any()
        assert (cache.positions[mask] == -1).all() and (cache.weights[mask] == 7.0).all()


def test_argument_refusals():
    """Checked before anything touches a device."""
    L = gbb.lib()
    x, y, z, p, t, w = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20, 6 << 20   # never read
    sec = lambda *n: (ctypes.c_int * len(n))(*n)  # noqa: E731

    def axes(x=x, y=y, T=4, H=1, D=64, p=p, axes=2, s=sec(16, 16), t=t, n=8, rot=64, lay=0):
        return L.gbb_rope_axes(x, 64, 64, y, 64, 64, 0, T, H, D, p, axes, s, t, n, rot, lay, 0, None)

    def norm(x=x, y=y, dt=0, T=4, D=64, w=w, wd=2, eps=1e-6, p=p, axes=1, s=None, t=t, rot=64):
        return L.gbb_norm_rope(x, 64, 64, y, 64, 64, dt, T, 1, D, w, wd, eps, p, axes, s, t, 8, rot, 0, None)

    def grad(x=x, dy=y, dx=z, xt=64, dxt=64, dt=0, T=4, H=1, w=w, wd=2, eps=1e-6, p=p, dw=7 << 20, ws=8 << 20, wb=1 << 30):
        return L.gbb_norm_rope_grad(x, xt, 64, dy, 64, 64, dx, dxt, 64, dt, T, H, 64, w, wd, eps, p, 1, None, t, 8, 64, 0,
                                    dw, ws, wb, None)

    assert axes(T=0) == 0 and norm(T=0) == 0 and grad(dx=None, dw=None) == 0
    for call, bad in ((axes, dict(axes=0)), (axes, dict(axes=5)), (axes, dict(s=None)), (axes, dict(s=sec(-1, 33))),
                      (axes, dict(p=None)), (axes, dict(y=x + 2)), (norm, dict(wd=1)), (norm, dict(wd=3)),
                      (norm, dict(eps=-1.0)), (norm, dict(eps=float("nan"))), (norm, dict(eps=float("inf"))),
                      (norm, dict(x=None)), (norm, dict(dt=3)), (grad, dict(dy=None)), (grad, dict(dx=x)),
                      (grad, dict(dx=y + 2)), (grad, dict(ws=None)), (grad, dict(wd=1)), (grad, dict(w=None, wd=1)),
                      (grad, dict(xt=-1))):
        assert call(**bad) == -1, bad
    for call, bad in ((axes, dict(s=sec(16, 15))), (axes, dict(s=sec(2 ** 31 - 1, 2 ** 31 - 1))), (axes, dict(rot=66)),
                      (norm, dict(D=65)), (norm, dict(rot=3)), (grad, dict(dxt=32))):
        assert call(**bad) == -2, bad
    for call, bad in ((norm, dict(w=w + 2)), (norm, dict(w=w + 1, wd=0)), (norm, dict(x=x + 1)), (grad, dict(dw=(7 << 20) + 2)),
                      (grad, dict(ws=(8 << 20) + 4)), (grad, dict(dx=z + 1))):
        assert call(**bad) == -4, bad
    assert grad(wb=16) == -5
    assert L.gbb_norm_rope_grad_workspace(0, 1, 64) == 0 and L.gbb_norm_rope_grad_workspace(4, 1, 65) == 0


def test_append_argument_refusals():
    L, C = gbb.lib(), gbb.binding._PagedCache
    c = C(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4, page=16,
          kv_heads=2, head_dim=64)

    def call(T=4, hq=4, qw=3 << 20, kw=4 << 20, wd=0, eps=1e-6, p=16 << 20, axes=1, s=None, sl=17 << 20, q=32 << 20):
        return L.gbb_norm_rope_append(ctypes.byref(c), 8 << 20, 512, 0, T, hq, qw, kw, wd, eps, p, axes, s, sl, 18 << 20, 8,
                                      64, 0, q, None)

    assert call(T=0) == 0
    for bad in (dict(qw=None), dict(kw=None), dict(wd=1), dict(eps=-1.0), dict(p=None), dict(axes=2), dict(sl=None),
                dict(q=8 << 20), dict(T=-1)):
        assert call(**bad) == -1, bad
    for bad in (dict(hq=3), dict(T=1 << 23)):
        assert call(**bad) == -2, bad
    for bad in (dict(qw=(3 << 20) + 1), dict(kw=(4 << 20) + 2, wd=2), dict(q=(32 << 20) + 8)):
        assert call(**bad) == -4, bad


def test_binding_refusals():
    """Of tensors of the CPU and of sections that make no sense, without a GPU."""
    x, w, p, t = torch.zeros(2, 1, 64), torch.zeros(64), torch.zeros(2, dtype=torch.int32), torch.zeros(4, 32, 2)
    for call in (lambda: gbb.norm_rope(x, w, p, t), lambda: gbb.rope(x, p, t, sections=(32,))):
        with pytest.raises(TypeError):
            call()
    gbb.paged._resolve()
    for bad in ((), (1,) * 5):
        with pytest.raises(ValueError):
            gbb.paged._axes(p, bad, -1, 2)
