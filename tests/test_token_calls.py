"""Calls around prompts and drafts as programs make them: of several threads,
with gradients written over their inputs, with a cache's every call on a stream
of its own and in one graph."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
gbb = pytest.importorskip("gemm_block_bit_amd")

from test_norm_rope import EPS, Case  # noqa: E402
from test_paged_attention_tokens import Setup, random_tree  # noqa: E402
from test_threads import in_threads  # noqa: E402

pytestmark = pytest.mark.gpu


def test_several_threads_on_one_stream():
    """Each thread's calls, of one new token and of several, have the results
    that they have alone: those of one stream share a workspace."""
    sets = [Setup([900 + 100 * i], [2 + 30 * i], 4, 1, 128, "bf16", "bf16", 16, seed=i) for i in range(4)]
    want = [s.run() for s in sets]
    got = [[] for _ in sets]
    stream = torch.cuda.current_stream()

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i].append(sets[i].run())
    in_threads(len(sets), work)
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for w, xs in zip(want, got) for x in xs)


@pytest.mark.parametrize("D,rot,layout,dt", [(128, 128, "half", "bf16"), (64, 10, "interleaved", "f32"), (80, 40, "half", "f16"),
                                             (6, 2, "half", "f16"), (1000, 1000, "interleaved", "f32")])
def test_a_gradient_in_place_of_the_output_s(D, rot, layout, dt):
    c = Case(70, 3, D, rot, layout, dt, seed=D, padding=(5,))
    x, w, p, t, dy = c.dev("x", "w", "positions", "table", "dy")
    T, H = x.shape[:2]
    code = {"f16": 0, "bf16": 1, "f32": 2}[dt]
    need = gbb.lib().gbb_norm_rope_grad_workspace(T, H, D)
    ws = torch.empty(need, dtype=torch.uint8, device=x.device)

    def grad(dx):
        dw = torch.empty(D, device=x.device)
        args = (x.data_ptr(), H * D, D, dy.data_ptr(), H * D, D, dx.data_ptr(), H * D, D, code, T, H, D, w.data_ptr(), 2, EPS,
                p.data_ptr(), 1, None, t.data_ptr(), t.shape[0], rot, {"half": 0, "interleaved": 1}[layout], dw.data_ptr(),
                ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert gbb.lib().gbb_norm_rope_grad(*args) == 0
        return dw
    dx = torch.empty_like(x)
    dw = grad(dx)
    c.check_grad(dx, dw)
    assert torch.equal(grad(dy), dw) and torch.equal(dy, dx)


@pytest.mark.parametrize("B,n", [(8, 12300), (3, 12300), (1, 600), (2, 150)])
def test_runs_joined_in_the_launch_and_by_a_second(B, n):
    """Many row tiles and few, in several runs: sequences of one length and of
    others, on the same pages."""
    hkv, D, page = 64, 64, 64
    s = Setup([n - 1], [1], hkv, hkv, D, page=page, seed=n + B)
    d = s.qd.device
    lengths = [n, n, n // 3, 70, n, 1, n - 100, 4200][:B]
    g = np.random.default_rng(B)
    q = torch.from_numpy((2 * g.standard_normal((B, hkv, D))).astype(np.float16))
    s.q, s.T, s.lengths, s.new, s.starts, s.bt = q, B, lengths, [1] * B, np.arange(B + 1, dtype=np.int32), s.bt.repeat(B, 0)
    s.to_device()
    lse = torch.zeros(B, hkv, device=d)
    out = s.run(lse=lse)
    s.check(out, lse)
    for _ in range(3):                            # the same bits each time
        assert torch.equal(s.run(), out)


def test_a_step_of_drafts_in_a_graph():
    """Norms and append, attention of a tree, the cut to the kept tokens and
    attention of the next token captured together; every replay, with eager work
    between, is the eager step on the state it starts from."""
    new, ctx, hq, hkv, D, page = [12, 5], [700, 90], 8, 2, 64, 16
    g = np.random.default_rng(1)
    bits = np.zeros((17, 12), bool)
    bits[:12, :12], bits[12:, :5] = random_tree(g, 12), random_tree(g, 5)
    s = Setup(ctx, new, hq, hkv, D, page=page, seed=2, tree=(bits, 1), softcap=20.0)
    d = s.qd.device
    qkv = torch.from_numpy(g.standard_normal((17, (hq + 2 * hkv) * D)).astype(np.float16)).to(d)
    norms = [torch.from_numpy(g.uniform(0.5, 1.5, D).astype(np.float32)).to(d) for _ in range(2)]
    table = torch.from_numpy(gbb.rope_table(D, 1024, 500000.0)).to(d)
    at = [np.arange(c, c + n) for c, n in zip(ctx, new)]
    slots = np.concatenate([s.bt[b][a // page] * page + a % page for b, a in enumerate(at)])
    slots = torch.from_numpy(slots.astype(np.int32)).to(d)
    positions = torch.from_numpy(np.concatenate(at).astype(np.int32)).to(d)
    kept = torch.tensor([[0, 3, 7, 11], [1, 2, 4, 0]], dtype=torch.int32, device=d)
    counts, drafted = torch.tensor([4, 3], dtype=torch.int32, device=d), torch.tensor(new, dtype=torch.int32, device=d)
    tree = s.arguments()["tree"]

    def step():
        q = gbb.rope_append(s.cache, qkv, hq, positions, slots, table, q_norm=norms[0], k_norm=norms[1])
        out = gbb.paged_attention_tokens(s.cache, q, s.startd, s.btd, s.lend, s.max_len, tree=tree, softcap=20.0)
        after = gbb.cache_keep(s.cache, s.btd, s.lend, drafted, kept, counts)
        one = gbb.paged_attention(s.cache, q[:2], s.btd, after, s.max_len, softcap=20.0, window=300)
        return out, after, one

    start = s.cache.k.clone(), s.cache.v.clone()

    def restore(x):
        qkv.copy_(x)
        s.cache.k.copy_(start[0])
        s.cache.v.copy_(start[1])
    inputs = [qkv.clone(), qkv.flip(0).contiguous(), 0.5 * qkv]
    want = []
    for x in inputs:
        restore(x)
        want.append([t.clone() for t in step()] + [s.cache.k.clone(), s.cache.v.clone()])
    assert want[0][1].tolist() == [704, 93]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):                            # two graphs, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for i in range(6):
        graph, out = graphs[i % 2]
        restore(inputs[i % 3])
        graph.replay()
        got = list(out) + [s.cache.k, s.cache.v]
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[i % 3])), i
        restore(inputs[i % 3])
        assert torch.equal(step()[0], want[i % 3][0])
        torch.cuda.synchronize()
