"""The example's decoding layer, step by step against the 64-bit oracle on
the state each step starts from: products, rotary positions, cache, attention,
weights and eviction together."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import decode_step as od

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("layout,dtype", [("half", torch.float16), ("interleaved", torch.float16),
                                          ("half", torch.float8_e4m3fn)])
def test_layer_against_oracle(layout, dtype):
    torch.manual_seed(0)
    B, hq, hkv, D, budget, slack = 3, 4, 2, 64, 24, 5
    layer = example().DecodeLayer(B, hq, hkv, D, budget, 6, slack, page=16, n_pos=256, layout=layout, dtype=dtype)
    c = layer.cache
    weight = [gbb.dequant(im, n, layer.hidden)[1].double().cpu().numpy() for im, n in ((layer.qkv, layer.qkv_rows), (layer.o, layer.hidden))]
    table = layer.table.double().cpu().numpy()
    bt = layer.block_table.cpu().numpy()
    es = {1: torch.uint8, 2: torch.int16}[c.k.element_size()]
    sc = np.ones(hkv) if c.k_scale is None else c.k_scale.double().cpu().numpy()
    wide = lambda t: t.double().cpu().numpy() * sc[None, :, None, None]  # noqa: E731
    g = np.random.default_rng(2)
    evicted = 0
    for step in range(70):
        x = torch.from_numpy(g.standard_normal((B, layer.hidden)).astype(np.float16)).cuda()
        length, lengths = layer.length, layer.lengths.cpu().numpy()
        before = [t.clone() for t in (c.k, c.v, c.weights, c.positions)]
        evicts = length + 1 == layer.max_len
        keep = {}
        if evicts:   # the state between attention and eviction
            real = gbb.cache_evict

            def spy(cache, *a, **k):
                keep.update(state=[t.clone() for t in (cache.k, cache.v, cache.weights, cache.positions)], lengths=a[1].clone())
                return real(cache, *a, **k)
            gbb.cache_evict = spy
        try:
            y = layer.step(x).double().cpu().numpy()
        finally:
            if evicts:
                gbb.cache_evict = real
        k, v, w, p = keep["state"] if evicts else (c.k, c.v, c.weights, c.positions)
        assert (lengths == length).all()
        # the new token: 2e-3 is the products' bar, on top of the cache's rounding
        qkv = (x.double().cpu().numpy() @ weight[0].T).reshape(B, hq + 2 * hkv, D)
        pos = np.full(B, step)
        turned = od.rope(qkv[:, :hq + hkv], pos, table, layout)
        page, off = bt[np.arange(B), length // 16], length % 16
        unit = 2.0 ** -4 if es is torch.uint8 else 2.0 ** -11
        top = np.abs(qkv).max()
        for t, ref in ((k, turned[:, hq:]), (v, qkv[:, hq + hkv:])):
            got = wide(t)[page, :, off]
            assert np.abs(got - ref).max() <= unit * top + 4e-3 * top
        assert (p.cpu().numpy()[page, :, off] == step).all()
        # nothing but the new slots changed in the cache
        same = torch.ones(k.shape[:3], dtype=torch.bool, device="cuda")
        same[torch.from_numpy(page).cuda().long(), :, off] = False
        assert torch.equal(k.view(es)[same], before[0].view(es)[same]) and torch.equal(v.view(es)[same], before[1].view(es)[same])
        assert torch.equal(p[same], before[3][same])
        # attention over the cache as it is, and the o product
        out, _, add, _, _ = od.paged_attention(turned[:, :hq], wide(k), wide(v), bt, lengths + 1, D ** -0.5)
        ref = out.reshape(B, -1) @ weight[1].T
        assert np.abs(y - ref).max() <= 1e-2 * np.abs(ref).max()
        base = before[2].double().cpu().numpy()
        base[page, :, off] = 0.0
        assert np.abs(w.double().cpu().numpy() - base - add).max() <= 2e-2
        if evicts:
            evicted += 1
            # the eviction is exact on that state
            want = od.cache_evict(k.view(es).cpu().numpy(), v.view(es).cpu().numpy(), w.cpu().numpy(), p.cpu().numpy(), bt,
                                  keep["lengths"].cpu().numpy(), budget, 6)
            for got, ref in zip((c.k.view(es), c.v.view(es), c.weights, c.positions), want):
                assert np.array_equal(got.cpu().numpy(), ref.astype(got.cpu().numpy().dtype))
            assert layer.lengths.tolist() == [budget] * B
    assert evicted >= 8
