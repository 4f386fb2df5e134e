"""Rotary positions and the cache write with so many tokens that a workgroup
takes several groups of heads of its tokens in turn (a thread keeps its angles
over them).  In calls of 40 tokens every group of heads has a workgroup of its own
here; those are the reference bit for bit, and the oracle for a part."""
import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda", 0)


def near(got, x, pos, table, layout, dt, transpose=False):
    """As for a single token: fp32 work on two products, one rounding."""
    ref = od.rope(x, pos, table, layout, transpose)
    before = 3 * 2.0 ** -24 * 2 * np.abs(x).max() * np.abs(table).max()
    assert np.all(np.abs(got - ref) <= before + UNIT[dt] * (np.abs(ref) + before) + 2.0 ** -25)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,H,D,rot", [(1100, 80, 128, 128), (1029, 70, 64, 20), (4100, 9, 256, 64), (1500, 3, 1024, 1022)])
def test_rope(T, H, D, rot, dt, layout):
    d = dev()
    torch.manual_seed(T + rot)
    table = gbb.rope_table(rot, 512)
    x = torch.randn(T, H, D, device=d).to(DT[dt])
    pos = torch.randint(0, 512, (T,), device=d, dtype=torch.int32)
    td = torch.from_numpy(table).to(d)
    for transpose in (False, True):
        y = gbb.rope(x, pos, td, layout=layout, transpose=transpose)
        parts = [gbb.rope(x[t:t + 40], pos[t:t + 40], td, layout=layout, transpose=transpose) for t in range(0, T, 40)]
        assert torch.equal(y, torch.cat(parts))
    some = [0, 1, T // 2, T - 1]
    near(y[some].double().cpu().numpy(), x[some].double().cpu().numpy(), pos[some].cpu().numpy(), table.astype(np.float64),
         layout, dt, True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dt,ct", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("T,hq,hkv,D,rot,page", [(1100, 64, 8, 128, 128, 64), (1029, 72, 4, 64, 20, 16), (2050, 12, 12, 256, 64, 32),
                                                 (1200, 6, 3, 128, 2, 256)])
def test_append(T, hq, hkv, D, rot, page, dt, ct, layout):
    d = dev()
    torch.manual_seed(T + rot)
    table = gbb.rope_table(rot, 512)
    td = torch.from_numpy(table).to(d)
    pages = -(-T // page) + 2
    qkv = torch.randn(T, (hq + 2 * hkv) * D, device=d).to(DT[dt])
    pos = torch.randint(0, 512, (T,), device=d, dtype=torch.int32)
    slots = torch.randperm(pages * page, device=d)[:T].to(torch.int32)
    pos[7], slots[T - 2] = -1, -1   # padding tokens
    scale = torch.rand(hkv, device=d) * 0.02 + 0.01 if ct == "e4m3" else None

    def cache():
        c = gbb.PagedCache.empty(pages, page, hkv, D, torch.float8_e4m3fn if ct == "e4m3" else DT[ct], d, True, scale, scale)
        c.weights.fill_(7.0)
        return c
    a, b = cache(), cache()
    q = gbb.rope_append(a, qkv, hq, pos, slots, td, layout=layout)
    parts = [gbb.rope_append(b, qkv[t:t + 40], hq, pos[t:t + 40], slots[t:t + 40], td, layout=layout) for t in range(0, T, 40)]
    assert torch.equal(q, torch.cat(parts))
    bits = torch.uint8 if ct == "e4m3" else torch.int16
    assert torch.equal(a.k.view(bits), b.k.view(bits)) and torch.equal(a.v.view(bits), b.v.view(bits))
    assert torch.equal(a.weights, b.weights) and torch.equal(a.positions, b.positions)
    assert not q[7].any() and not q[T - 2].any() and (a.weights == 0).sum().item() == (T - 2) * hkv
    some = [0, 8, T // 2, T - 1]
    x = qkv.view(T, -1, D)[some].double().cpu().numpy()
    near(q[some].double().cpu().numpy(), x[:, :hq], pos[some].cpu().numpy(), table.astype(np.float64), layout, dt)
    at = slots[some].long()
    if ct != "e4m3":
        k, v = a.k[at // page, :, at % page], a.v[at // page, :, at % page]
        near(k.double().cpu().numpy(), x[:, hq:hq + hkv], pos[some].cpu().numpy(), table.astype(np.float64), layout, dt)
        assert np.array_equal(v.double().cpu().numpy(), x[:, hq + hkv:])
