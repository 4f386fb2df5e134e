"""Rotary positions and the cache write: tables against the formulas (CPU),
kernels against the 64-bit oracle (GPU).

Tolerances.  A rotated element is two fp32 products and their sum, so it is
within 3 * 2^-24 (|x1| + |x2|) * |table| of exact before its one rounding to
the output's type (half a unit in the last place, relative 2^-11, 2^-8 or
2^-24, or half the smallest subnormal)."""
import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}

SCALINGS = [dict(), dict(scaling="linear", factor=4.0),
            dict(scaling="bands", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
            dict(scaling="yarn", factor=16.0, original_len=4096.0, low=1.0, high=32.0)]


# ----------------------------------------------------------------------------
# tables (host)
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s.get("scaling", "plain"))
@pytest.mark.parametrize("rot,n_pos,base", [(2, 1, 10000.0), (64, 1000, 10000.0), (128, 9000, 500000.0)])
def test_table_against_formulas(rot, n_pos, base, scaling):
    att = 1.25 if scaling else 1.0
    got = gbb.rope_table(rot, n_pos, base, attention=att, **scaling)
    assert got.shape == (n_pos, rot // 2, 2) and got.dtype == np.float32
    ref = od.rope_table(rot, n_pos, base, attention=att, **scaling)
    # one rounding to fp32 (half a unit in each value's own last place), and
    # an angle below 2^14 whose 64-bit rounding is below 2^-38
    assert np.all(np.abs(got - ref) <= 0.5 * np.spacing(np.abs(got)) + att * 2.0 ** -37)


def test_scaled_frequencies_meet_their_ends():
    """Short waves keep their frequency, long ones are divided by the factor."""
    for s in SCALINGS[2:]:
        f = [od.rope_frequency(i, 128, 500000.0, **s) * 500000.0 ** (2 * i / 128) for i in range(64)]
        assert abs(f[0] - 1) < 1e-12 and abs(f[-1] - 1 / s["factor"]) < 1e-12
        assert all(a >= b - 1e-12 for a, b in zip(f, f[1:]))
        got = gbb.rope_table(128, 2, 500000.0, **s)[1]   # position 1: the angle is the frequency
        want = np.array([od.rope_frequency(i, 128, 500000.0, **s) for i in range(64)])
        assert np.abs(np.arctan2(got[:, 1], got[:, 0]) - want).max() <= 2.0 ** -23


@pytest.mark.parametrize("kw", [dict(rot=3), dict(rot=0), dict(n_pos=0), dict(base=1.0), dict(base=float("nan")),
                                dict(attention=0.0), dict(attention=float("inf")),
                                dict(scaling="linear", factor=0.5), dict(scaling="bands", factor=2.0),
                                dict(scaling="bands", factor=2.0, original_len=8.0, low=4.0, high=4.0),
                                dict(scaling="yarn", factor=2.0, original_len=8.0, low=0.0)])
def test_table_refusals(kw):
    args = dict(rot=8, n_pos=4, base=10000.0)
    args.update(kw)
    with pytest.raises(gbb.GbbError) as e:
        gbb.rope_table(**args)
    assert e.value.status == -1


def test_oracle_e4m3_against_torch():
    """The oracle's 8-bit codes against torch's conversion, over all codes,
    their midpoints and random values in range."""
    val = od.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(val, nan=1e9), np.nan_to_num(t, nan=1e9))
    g = np.random.default_rng(0)
    x = np.concatenate([val[~np.isnan(val)], (val[:126] + val[1:127]) / 2, -(val[:126] + val[1:127]) / 2,
                        g.standard_normal(4000) * np.exp(g.uniform(-8, 5, 4000))]).astype(np.float32)
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(od.e4m3_encode(x), want)
    assert np.array_equal(od.e4m3_encode([1e9, -np.inf, 460.0]), [126, 254, 126])


def test_rope_argument_refusals():
    """Checked before anything touches a device."""
    L = gbb.lib()
    x, y, p, t = 1 << 20, 2 << 20, 3 << 20, 4 << 20   # never read

    def call(x=x, xt=64, xh=64, y=y, yt=64, yh=64, dt=0, T=4, H=1, D=64, p=p, t=t, n=8, rot=64, lay=0):
        return L.gbb_rope(x, xt, xh, y, yt, yh, dt, T, H, D, p, t, n, rot, lay, 0, None)

    assert call(T=0) == 0
    for bad in (dict(dt=3), dict(T=-1), dict(H=0), dict(D=0), dict(x=None), dict(y=None), dict(p=None), dict(t=None),
                dict(n=0), dict(lay=2), dict(xt=-1), dict(y=x + 2)):
        assert call(**bad) == -1, bad
    for bad in (dict(D=65), dict(D=2048), dict(rot=66), dict(rot=0), dict(rot=3), dict(yt=32), dict(H=2, yh=32, yt=128)):
        assert call(**bad) == -2, bad
    for bad in (dict(x=x + 1), dict(y=y + 1), dict(dt=2, x=x + 2), dict(t=t + 4)):
        assert call(**bad) == -4, bad


def test_append_argument_refusals():
    L = gbb.lib()
    C = gbb.binding._PagedCache
    import ctypes
    base = dict(k=1 << 20, v=2 << 20, k_scale=None, v_scale=None, weights=None, positions=None, dtype=0, num_pages=4,
                page=16, kv_heads=2, head_dim=64)

    def call(c=None, qkv=8 << 20, stride=512, dt=0, T=4, hq=4, p=16 << 20, s=17 << 20, t=18 << 20, n=8, rot=64, lay=0,
             q=32 << 20):
        cc = C(**{**base, **(c or {})})
        return L.gbb_rope_append(ctypes.byref(cc), qkv, stride, dt, T, hq, p, s, t, n, rot, lay, q, None)

    assert call(T=0) == 0
    assert L.gbb_rope_append(None, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, None) == -1
    for bad in (dict(c=dict(k=None)), dict(c=dict(dtype=2)), dict(c=dict(k_scale=64)), dict(c=dict(num_pages=0)),
                dict(c=dict(kv_heads=0)), dict(dt=1), dict(dt=2), dict(T=-1), dict(qkv=None), dict(q=None), dict(s=None),
                dict(p=None), dict(t=None), dict(n=0), dict(lay=5), dict(q=8 << 20)):
        assert call(**bad) == -1, bad
    for bad in (dict(c=dict(page=24)), dict(c=dict(page=512)), dict(c=dict(head_dim=96)), dict(hq=3), dict(hq=0),
                dict(hq=2 * 129), dict(stride=504), dict(rot=66), dict(c=dict(num_pages=1 << 28)), dict(T=1 << 23)):
        assert call(**bad) == -2, bad
    for bad in (dict(qkv=(8 << 20) + 8), dict(q=(32 << 20) + 8), dict(stride=516), dict(c=dict(k=8)),
                dict(s=(17 << 20) + 2), dict(c=dict(weights=2))):
        assert call(**bad) == -4, bad


# ----------------------------------------------------------------------------
# kernels
# ----------------------------------------------------------------------------
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def check_rotated(got, x, pos, table, layout, transpose, dt):
    """got against the oracle of x (fp64 values of the inputs)."""
    ref = od.rope(x, pos, table, layout, transpose)
    pair = np.zeros_like(ref)   # |x1| + |x2| of the element's pair
    half = table.shape[1]
    for i in range(half):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        pair[..., a] = pair[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    before = 3 * 2.0 ** -24 * pair * np.abs(table).max()
    tol = before + UNIT[dt] * (np.abs(ref) + before) + TINY[dt]
    assert np.all(np.abs(got - ref) <= tol), np.max(np.abs(got - ref) / tol)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 32, 128, 128), (7, 3, 64, 64), (5, 2, 96, 24), (3, 5, 80, 20),
                                       (2, 1, 10, 6), (33, 9, 256, 128), (2, 2, 1024, 2), (2, 1, 1024, 1024),
                                       (300, 4, 64, 32)])
def test_rope_against_oracle(T, H, D, rot, dt, layout):
    g = np.random.default_rng(T * D + rot)
    n_pos = 131072
    x = torch.from_numpy(g.standard_normal((T, H, D)).astype(np.float32)).to(DT[dt])
    table = gbb.rope_table(rot, n_pos, 500000.0)
    pos = g.integers(0, n_pos, T).astype(np.int32)
    pos[-1] = n_pos - 1
    xd, pd, td = x.to(dev()), torch.from_numpy(pos).to(dev()), torch.from_numpy(table).to(dev())
    xs = x.double().numpy()
    for transpose in (False, True):
        y = gbb.rope(xd, pd, td, layout=layout, transpose=transpose)
        check_rotated(y.double().cpu().numpy(), xs, pos, table.astype(np.float64), layout, transpose, dt)
        z = xd.clone()   # in place gives the same bits
        assert gbb.rope(z, pd, td, layout=layout, transpose=transpose, out=z) is z
        assert torch.equal(z, y)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("off,head", [(0, 72), (2, 70), (1, 67)])
def test_rope_strides_and_odd_addresses(off, head, layout):
    """Views with gaps between heads, starting at any element: the widest
    loads the addresses allow, down to one element."""
    g = np.random.default_rng(off)
    T, H, D = 9, 3, 64
    table = gbb.rope_table(32, 64)
    pos = torch.arange(T, dtype=torch.int32, device=dev()) * 7
    for dt in ("f16", "f32"):
        buf = torch.from_numpy(g.standard_normal(20000).astype(np.float32)).to(DT[dt]).to(dev())
        x = buf[off:].as_strided((T, H, D), (H * head + 5, head, 1))
        out = torch.zeros(20000, dtype=DT[dt], device=dev())
        y = out[off:].as_strided((T, H, D), (H * head + 3, head, 1))
        gbb.rope(x, pos, torch.from_numpy(table).to(dev()), layout=layout, out=y)
        check_rotated(y.double().cpu().numpy(), x.double().cpu().numpy(), pos.cpu().numpy(), table.astype(np.float64),
                      layout, False, dt)
        y.zero_()
        assert not out.any()   # nothing outside the heads was written


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 4), (6, 1), (6, 4)])
def test_rope_heads_outside_tokens(T, H):
    """Views of [H][T][D] memory, in place and as the output: the same bits as
    the contiguous call."""
    d = dev()
    table = torch.from_numpy(gbb.rope_table(64, 16)).to(d)
    pos = torch.arange(T, dtype=torch.int32, device=d) + 3
    x = torch.randn(H, T, 64, device=d, dtype=torch.bfloat16)
    want = gbb.rope(x.transpose(0, 1).contiguous(), pos, table)
    assert torch.equal(gbb.rope(x.transpose(0, 1), pos, table), want)
    y = torch.zeros_like(x)
    gbb.rope(x.transpose(0, 1), pos, table, out=y.transpose(0, 1))
    assert torch.equal(y.transpose(0, 1), want)
    v = x.transpose(0, 1)
    assert torch.equal(gbb.rope(v, pos, table, out=v), want)


def test_rope_heads_outside_tokens_that_overlap():
    L = gbb.lib()
    x, y, p, t = 1 << 20, 2 << 20, 3 << 20, 4 << 20   # never read
    for yt, yh in ((64, 64 * 4 - 1), (63, 1024), (64, 64)):   # 4 tokens of 2 heads of 64
        assert L.gbb_rope(x, 64, 256, y, yt, yh, 0, 4, 2, 64, p, t, 8, 64, 0, 0, None) == -2


@pytest.mark.gpu
def test_rope_broadcast_input_padding_and_empty():
    d = dev()
    table = torch.from_numpy(gbb.rope_table(64, 16)).to(d)
    x = torch.randn(1, 1, 64, device=d, dtype=torch.float16).expand(5, 3, 64)
    pos = torch.tensor([3, -1, 16, 2 ** 31 - 1, 15], dtype=torch.int32, device=d)
    y = gbb.rope(x, pos, table)
    assert torch.equal(y, gbb.rope(x.contiguous(), pos, table))
    assert not y[1:4].any() and y[0].any() and y[4].any()
    assert gbb.rope(x[:0], pos[:0], table).shape == (0, 3, 64)
    nan = torch.full((1, 1, 64), float("nan"), device=d)
    assert not gbb.rope(nan, pos[1:2], table).any()   # padding is zero whatever it held


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_against_differences(layout):
    """The map is linear, so a central difference along a random direction is
    exact but for fp32 rounding; it has to be the direction's product with the
    transposed map of the output's gradient."""
    g = np.random.default_rng(5)
    T, H, D, rot, h = 6, 3, 96, 64, 2.0 ** -3
    table = torch.from_numpy(gbb.rope_table(rot, 4096, scaling="linear", factor=2.0, attention=1.1)).to(dev())
    pos = torch.from_numpy(g.integers(0, 4096, T).astype(np.int32)).to(dev())
    x, d, go = (torch.from_numpy(g.standard_normal((T, H, D)).astype(np.float32)).to(dev()) for _ in range(3))
    f = lambda v: gbb.rope(v, pos, table, layout=layout).double()  # noqa: E731
    num = ((f(x + h * d) - f(x - h * d)) * go.double()).sum().item() / (2 * h)
    grad = gbb.rope(go, pos, table, layout=layout, transpose=True)
    ana = (grad.double() * d.double()).sum().item()
    # each of the difference's values carries at most 2^-22 (|x1| + |x2|) 1.1
    # of rounding (inputs x + h d and outputs), over 2 h
    bound = (2.0 ** -22 * 1.1 * 2 * (x.abs() + h * d.abs()).max().item() * go.abs().sum().item()) / h + 1e-6 * abs(ana)
    assert abs(num - ana) <= bound


CACHES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")]


def make_cache(pages, page, hkv, D, dt, ct, tracked, g):
    d = dev()
    kw = {}
    if ct == "e4m3":
        kw = dict(k_scale=torch.from_numpy(g.uniform(0.01, 0.05, hkv).astype(np.float32)).to(d),
                  v_scale=torch.from_numpy(g.uniform(0.01, 0.05, hkv).astype(np.float32)).to(d))
    c = gbb.PagedCache.empty(pages, page, hkv, D, torch.float8_e4m3fn if ct == "e4m3" else DT[dt], d, tracked, **kw)
    if tracked:
        c.weights.fill_(7.0)
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt,ct", CACHES)
@pytest.mark.parametrize("T,hq,hkv,D,rot,page", [(1, 32, 8, 128, 128, 64), (19, 6, 2, 64, 64, 16), (40, 1, 1, 256, 64, 32),
                                                 (5, 12, 4, 64, 20, 16), (6, 3, 3, 128, 2, 256)])
def test_append_against_oracle(T, hq, hkv, D, rot, page, dt, ct, layout):
    g = np.random.default_rng(T + D + rot)
    n_pos, pages = 5000, 4 + T // page
    c = make_cache(pages, page, hkv, D, dt, ct, True, g)
    width = (hq + 2 * hkv) * D
    buf = torch.from_numpy(g.standard_normal((T, width + 24)).astype(np.float32)).to(DT[dt]).to(dev())
    qkv = buf[:, 8:8 + width]   # rows inside wider ones
    table = gbb.rope_table(rot, n_pos)
    pos = g.integers(0, n_pos, T).astype(np.int32)
    slots = g.permutation(pages * page)[:T].astype(np.int32)
    pad = [] if T < 4 else [1, 3]
    if pad:
        pos[1], slots[3] = -1, pages * page   # two padding tokens
    q = gbb.rope_append(c, qkv, hq, torch.from_numpy(pos).to(dev()), torch.from_numpy(slots).to(dev()),
                        torch.from_numpy(table).to(dev()), layout=layout)
    x = qkv.double().cpu().numpy().reshape(T, -1, D)
    real = [t for t in range(T) if t not in pad]
    tab = table.astype(np.float64)
    qn = q.double().cpu().numpy()
    check_rotated(qn[real], x[real, :hq], pos[real], tab, layout, False, dt)
    assert not qn[pad].any()
    pg, off = slots[real] // page, slots[real] % page
    k, v = x[real, hq:hq + hkv], x[real, hq + hkv:]
    other = np.ones((pages, page), bool)
    other[pg, off] = False
    assert np.array_equal((c.weights.cpu().numpy() == 7).transpose(0, 2, 1), np.repeat(other[..., None], hkv, 2))
    assert np.array_equal(c.positions.cpu().numpy()[pg, :, off], np.repeat(pos[real][:, None], hkv, 1))
    assert (c.positions.cpu().numpy().transpose(0, 2, 1)[other] == -1).all()
    if ct != "e4m3":
        ck, cv = c.k.double().cpu().numpy(), c.v.double().cpu().numpy()
        check_rotated(ck[pg, :, off], k, pos[real], tab, layout, False, dt)
        assert np.array_equal(cv[pg, :, off], v)
        assert not ck.transpose(0, 2, 1, 3)[other].any() and not cv.transpose(0, 2, 1, 3)[other].any()
        return
    ks, vs = (s.cpu().numpy()[None, :, None] for s in (c.k_scale, c.v_scale))
    codes = c.v.view(torch.uint8).cpu().numpy()
    want = od.e4m3_encode(v.astype(np.float32) / vs)   # the fp32 quotient, one rounding
    assert np.array_equal(codes[pg, :, off], want)
    ref = np.clip(od.rope(k, pos[real], tab, layout) / ks, -448, 448)
    got = c.k.double().cpu().numpy()[pg, :, off]
    # fp32 work before the rounding to 3 mantissa bits (half a unit: 2^-4) or subnormals of 2^-9
    pre = 2.0 ** -21 * 2 * np.abs(k).max() / ks
    assert np.all(np.abs(got - ref) <= np.maximum(2.0 ** -4 * (np.abs(ref) + pre), 2.0 ** -10) + pre)
    assert not c.k.view(torch.uint8).cpu().numpy().transpose(0, 2, 1, 3)[other].any()


@pytest.mark.gpu
def test_append_e4m3_saturates_and_keeps_nan():
    d = dev()
    c = gbb.PagedCache.empty(1, 16, 1, 64, torch.float8_e4m3fn, d)   # no scales: 1
    table = torch.from_numpy(gbb.rope_table(64, 1)).to(d)            # position 0: no turn
    qkv = torch.zeros(1, 192, dtype=torch.float16, device=d)
    qkv[0, 64:70] = torch.tensor([1e4, -1e4, float("inf"), float("-inf"), 448.0, 0.001], dtype=torch.float16)
    qkv[0, 128:131] = torch.tensor([float("nan"), 500.0, 17.0], dtype=torch.float16)
    z = torch.zeros(1, dtype=torch.int32, device=d)
    gbb.rope_append(c, qkv, 1, z, z, table)
    k, v = c.k.float()[0, 0, 0], c.v.float()[0, 0, 0]
    # an infinity meets 0 * sin in its pair: what is asked of k is the finite ones
    assert k[0] == 448 and k[1] == -448 and k[4] == 448 and k[5] == 2.0 ** -9 * round(0.001 * 512)
    assert torch.isnan(v[0]) and v[1] == 448 and v[2] == 16


@pytest.mark.gpu
def test_append_refusals_in_the_binding():
    d = dev()
    c = gbb.PagedCache.empty(2, 16, 2, 64, torch.float16, d)
    table = torch.from_numpy(gbb.rope_table(64, 8)).to(d)
    i = torch.zeros(3, dtype=torch.int32, device=d)
    qkv = torch.zeros(3, 8 * 64, dtype=torch.float16, device=d)
    gbb.rope_append(c, qkv, 4, i, torch.arange(3, dtype=torch.int32, device=d), table)
    for bad in (lambda: gbb.rope_append(c, qkv[:, :-1], 4, i, i, table), lambda: gbb.rope_append(c, qkv, 4, i[:2], i, table),
                lambda: gbb.rope_append(c, qkv, 4, i, i, table[:, :, 0]), lambda: gbb.rope_append(c, qkv, 4, i, i, table, layout="x"),
                lambda: gbb.rope_append(c, qkv.t(), 4, i, i, table), lambda: gbb.rope(qkv, i, table)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gbb.rope_append(c, qkv, 4, i.long(), i, table), lambda: gbb.rope_append(c, qkv.double(), 4, i, i, table),
                lambda: gbb.rope_append(c, qkv.cpu(), 4, i, i, table),
                lambda: gbb.PagedCache(torch.zeros(1, 1, 16, 64, device=d), torch.zeros(1, 1, 16, 64, device=d))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(gbb.GbbError):
        gbb.rope_append(c, qkv.bfloat16(), 4, i, i, table)
