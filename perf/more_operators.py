"""Cases of the operators that bring prompts, drafted tokens and more kinds of
models to the paged cache: norms of q and k heads with rotary positions of one
or several axes (with gradients, and on their way into the cache), attention of
single tokens, prompts and trees of drafted tokens whose scores are capped,
biased by distance or masked, and the cut of the cache to the drafted tokens
that were accepted.

`own = False` computes them in plain torch operations in 32 bits, rounded once
at the end; `own = True` calls the library.  Head counts and head sizes are
those of the Llama-3-8B (32 query heads, 8 kv heads of 128) and Llama-3-70B
(64, 8, 128) layers that the rest of this repository measures, and generic ones.

Caches are [pages][kv heads][page][head size] (fp16, bf16, or e4m3 with one
scale per kv head).  Slot s of a cache is token s % page of page s // page.
"""
import numpy as np
import torch

own = False

F16, BF16, F32, E4M3 = "f16", "bf16", "f32", "e4m3"
DTYPES = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
SIZE = {F16: 2, BF16: 2, F32: 4, E4M3: 1}
BASE = 500000.0          # rotary base of the tables
EPS = 1e-6               # of the norms


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # a training step's normed and rotated queries over a long sequence, with the gradients
        _turn("norm rope gradient 16384", tokens=16384, heads=32, dim=128, rot=128, layout="half", dtype=BF16,
              weight=F32, axes=1, grad=True),
        # one odd-sized image's queries in a vision tower: time, height and width, no norm
        _turn("rope 3 axes of 37 x 37", tokens=1369, heads=16, dim=80, rot=80, layout="half", dtype=F16, weight=None,
              axes=3, grad=False),
        # one user's next token on its way into the cache
        _append("append normed 1 token", tokens=1, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", dtype=F16,
                cache=F16, page=64, axes=1),
        # a prompt of text and images into an 8-bit cache
        _append("append normed 4097 3 axes", tokens=4097, q_heads=64, kv_heads=8, dim=128, rot=128,
                layout="interleaved", dtype=BF16, cache=E4M3, page=32, axes=3),
        # one user's next token after a short context, biased by distance
        _attend("token 1 x 1000 bias", mode="token", batch=1, new=1, context=999, ragged=False, q_heads=32, kv_heads=8,
                dim=128, dtype=F16, cache=F16, page=16, cap=0.0, bias=True, window=0, document=0, prefix=False,
                lse=False),
        # a serving batch in a layer with a cap and a sliding window
        _attend("token 32 cap window", mode="token", batch=32, new=1, context=16383, ragged=True, q_heads=64,
                kv_heads=8, dim=128, dtype=BF16, cache=BF16, page=64, cap=50.0, bias=False, window=4096, document=0,
                prefix=False, lse=True),
        # one long prompt in a layer with a cap
        _attend("prompt 8192 cap", mode="prompt", batch=1, new=8192, context=0, ragged=False, q_heads=32, kv_heads=8,
                dim=128, dtype=BF16, cache=BF16, page=64, cap=50.0, bias=False, window=0, document=0, prefix=False,
                lse=False),
        # chunks of several prompts behind what the cache holds of them, packed documents, a prefix seen both ways
        _attend("prompt 6 ragged documents", mode="prompt", batch=6, new=1500, context=2000, ragged=True, q_heads=12,
                kv_heads=12, dim=64, dtype=F16, cache=F16, page=32, cap=0.0, bias=True, window=0, document=1000,
                prefix=True, lse=True),
        # one user's drafted tree
        _attend("tree 1 x 25 of 4000", mode="tree", batch=1, new=25, context=4000, ragged=False, q_heads=32,
                kv_heads=8, dim=128, dtype=F16, cache=F16, page=64, cap=0.0, bias=False, window=0, document=0,
                prefix=False, lse=False),
        # a serving batch's trees over long contexts in an 8-bit cache
        _attend("tree 16 x 64 ragged e4m3", mode="tree", batch=16, new=64, context=16384, ragged=True, q_heads=64,
                kv_heads=8, dim=128, dtype=BF16, cache=E4M3, page=128, cap=0.0, bias=False, window=0, document=0,
                prefix=False, lse=False),
        # what one user's tree leaves behind
        _keep("keep 6 of 25", batch=1, kv_heads=8, dim=128, cache=F16, page=64, context=4000, new=25, most=6,
              tracked=False),
        # a batch's, in a cache that is evicted from
        _keep("keep up to 17 of 64 tracked", batch=64, kv_heads=8, dim=128, cache=BF16, page=32, context=1000, new=64,
              most=17, tracked=True),
    ]


def _turn(name, **k):
    return {"name": name, "op": "turn", **k}


def _append(name, **k):
    return {"name": name, "op": "append", **k}


def _attend(name, **k):
    return {"name": name, "op": "attend", **k}


def _keep(name, **k):
    return {"name": name, "op": "keep", **k}


def _spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(low * (high / low) ** rng.random()))))


def draw(rng):
    op = rng.choice(["turn", "append", "token", "token", "prompt", "prompt", "tree", "tree", "keep"])
    layout = rng.choice(["half", "interleaved"])
    axes = rng.choice([1, 1, 2, 3])
    if op == "turn":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.choice([1, 5, 8, 12, 32, 64])
        dtype = rng.choice([F16, BF16, F32])
        return {"op": op, "tokens": _spread(rng, 1, min(16384, 2 ** 25 // (heads * dim))), "heads": heads, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]), "layout": layout, "dtype": dtype,
                "weight": rng.choice([None, dtype, F32]), "axes": axes, "grad": rng.random() < 0.5}
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    dtype = rng.choice([F16, BF16])
    cache = rng.choice([dtype, dtype, E4M3])
    if op == "keep":
        new = _spread(rng, 1, 256)
        return {"op": op, "batch": _spread(rng, 1, 128), "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page,
                "context": _spread(rng, 1, 2000), "new": new, "most": _spread(rng, 1, new), "tracked": rng.random() < 0.5}
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        return {"op": op, "tokens": _spread(rng, 1, min(8192, 2 ** 26 // ((q_heads + 2 * kv_heads) * dim))),
                "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rng.choice([dim, dim, dim // 2]),
                "layout": layout, "dtype": dtype, "cache": cache, "page": page, "axes": axes}
    bias = rng.random() < 0.3
    case = {"op": "attend", "mode": op, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "cache": cache, "page": page, "ragged": rng.random() < 0.6, "cap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "bias": bias, "lse": rng.random() < 0.3}
    if op == "token":
        batch = _spread(rng, 1, 128)
        context = _spread(rng, 1, min(65536, 2 ** 27 // (batch * kv_heads * dim))) - 1
        window = rng.choice([0, _spread(rng, 1, 8192)])
        return {**case, "batch": batch, "new": 1, "context": context, "window": window, "document": 0, "prefix": False}
    if op == "tree":
        batch, new = _spread(rng, 1, 32), _spread(rng, 2, 128)
        # at most as many pairs of a query head and a slot as the largest listed prompt has
        most = min(2 ** 27 // (batch * kv_heads * dim), 2 ** 30 // (batch * new * q_heads) * 128 // dim)
        context = _spread(rng, 1, max(1, min(65536, most) - new))
        window = rng.choice([0, 0, _spread(rng, 16, 4096)])
        return {**case, "batch": batch, "new": new, "context": context, "window": window, "document": 0, "prefix": False}
    batch = _spread(rng, 1, 16)
    new = _spread(rng, 2, max(2, min(8192, 2 ** 25 // (batch * q_heads * dim))))
    most = 2 ** 30 // (batch * new * q_heads) * 128 // dim - new
    context = rng.choice([0, _spread(rng, 1, max(1, min(16384, most)))])
    return {**case, "batch": batch, "new": new, "context": context, "window": rng.choice([0, 0, _spread(rng, 16, 4096)]),
            "document": rng.choice([0, 0, _spread(rng, 16, 4096)]), "prefix": rng.random() < 0.3}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _table(rot, n_pos):
    """fp32 [n_pos][rot/2][2]: cos and sin of position times frequency, from 64 bits."""
    f = BASE ** (-2.0 * np.arange(rot // 2) / rot)
    a = np.arange(n_pos)[:, None] * f[None, :]
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)).cuda()


def _randn(gen, *shape, dtype=torch.float16, scale=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def _sections(rot, axes):
    """Pairs per axis: a quarter for time, the rest shared by height and width."""
    half = rot // 2
    if axes == 1:
        return None
    first = half // 4 if axes == 3 else half // 2
    second = (half - first) // 2 if axes == 3 else half - first
    return (first, second) if axes == 2 else (first, second, half - first - second)


def _positions(case, gen, n_pos):
    """int32 [T], or [axes][T]: text, then an image's rows and columns."""
    t = torch.arange(case["tokens"], device="cuda", dtype=torch.int32)
    start = torch.randint(0, n_pos - case["tokens"], (1,), generator=gen, device="cuda", dtype=torch.int32)
    if case["axes"] == 1:
        return start + t
    wide = max(1, int(case["tokens"] ** 0.5))
    return torch.stack([start + t // (wide * wide), start + t // wide, start + t % wide][3 - case["axes"]:]).contiguous()


def _even(low, high, n, gen, ragged):
    """int32 [n]: high, or whole numbers spread evenly over [low, high] in an order of the seed's."""
    if not ragged or n == 1:
        return torch.full((n,), high, dtype=torch.int32, device="cuda")
    x = low + torch.arange(n, device="cuda") * (high - low) // (n - 1)
    return x[torch.randperm(n, generator=gen, device="cuda")].to(torch.int32)


def _cache(case, gen, num_pages):
    shape = (num_pages, case["kv_heads"], case["page"], case["dim"])
    s = {"k_scale": None, "v_scale": None}
    if case["cache"] == E4M3:
        for n in ("k", "v"):
            scale = torch.rand(case["kv_heads"], generator=gen, device="cuda") * 0.02 + 0.01
            s[n + "_scale"] = scale
            x = _randn(gen, *shape, dtype=torch.float32) / scale.view(1, -1, 1, 1)
            s[n] = x.clamp(-448, 448).to(DTYPES[E4M3])
    else:
        s["k"], s["v"] = (_randn(gen, *shape, dtype=DTYPES[case["cache"]]) for _ in range(2))
    return s


def _tree(gen_np, new, words):
    """uint32 [new][words]: each token's ancestors and itself in a random tree; a parent is one of the last few tokens
    or the root's own (several first tokens)."""
    m = np.zeros((new, words), np.uint32)
    for i in range(new):
        parent = int(gen_np.integers(max(-1, i - 8), i)) if i else -1
        if parent >= 0:
            m[i] = m[parent]
        m[i, i // 32] |= np.uint32(1 << (i % 32))
    return m


def _handle(s):
    import gemm_block_bit_amd as gbb
    return gbb.PagedCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], weights=s.get("weights"),
                          positions=s.get("positions"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62))
    s = {"case": case}
    {"turn": _prepare_turn, "append": _prepare_append, "attend": _prepare_attend, "keep": _prepare_keep}[case["op"]](
        s, case, gen, int(seed))
    if own and case["op"] != "turn":
        s["cache"] = _handle(s)
    return s


def _prepare_turn(s, case, gen, seed):
    n_pos = max(4096, 2 * case["tokens"])
    s["table"], s["positions_of"] = _table(case["rot"], n_pos), _positions(case, gen, n_pos)
    s["sections"] = _sections(case["rot"], case["axes"])
    dtype = DTYPES[case["dtype"]]
    s["x"] = _randn(gen, case["tokens"], case["heads"], case["dim"], dtype=dtype, scale=1.5)
    s["weight"] = None
    if case["weight"]:
        s["weight"] = (1.0 + 0.2 * _randn(gen, case["dim"], dtype=torch.float32)).to(DTYPES[case["weight"]])
    if case["grad"]:
        s["dy"] = _randn(gen, case["tokens"], case["heads"], case["dim"], dtype=dtype)
        if own:   # leaves of the user's graph
            s["x"].requires_grad_()
            if s["weight"] is not None:
                s["weight"].requires_grad_()


def _prepare_append(s, case, gen, seed):
    n_pos = max(4096, 2 * case["tokens"])
    s["table"], s["positions_of"] = _table(case["rot"], n_pos), _positions(case, gen, n_pos)
    s["sections"] = _sections(case["rot"], case["axes"])
    per = -(-case["tokens"] // case["page"])
    s |= _cache(case, gen, per + 3)
    dtype = DTYPES[case["dtype"]]
    heads = case["q_heads"] + 2 * case["kv_heads"]
    s["qkv"] = _randn(gen, case["tokens"], heads * case["dim"], dtype=dtype, scale=1.5)
    s["q_norm"], s["k_norm"] = ((1.0 + 0.2 * _randn(gen, case["dim"], dtype=torch.float32)).to(dtype) for _ in range(2))
    pages = torch.randperm(per + 3, generator=gen, device="cuda")[:per].to(torch.int32)
    t = torch.arange(case["tokens"], device="cuda", dtype=torch.int32)
    s["slots"] = pages[(t // case["page"]).long()] * case["page"] + t % case["page"]


def _prepare_attend(s, case, gen, seed):
    batch, page = case["batch"], case["page"]
    s["max_len"] = case["context"] + case["new"]
    per = -(-s["max_len"] // page)
    s["block_table"] = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32).view(batch, per)
    context = _even(0, case["context"], batch, gen, case["ragged"])
    new = torch.ones_like(context)
    if case["mode"] != "token":
        new = _even(1 if case["mode"] == "tree" else 0, case["new"], batch, gen, case["ragged"])
    s["lengths"] = context + new
    s["starts"] = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
    tokens = int(new.sum())
    s |= _cache(case, gen, batch * per)
    # scores of standard deviation 2: some keys matter, most do not; of 12 with a cap, so that it is felt
    s["q"] = _randn(gen, tokens, case["q_heads"], case["dim"], dtype=DTYPES[case["dtype"]],
                    scale=12.0 if case["cap"] else 2.0)
    if case["bias"]:   # slopes of a geometric series over the heads
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, case["q_heads"] + 1, device="cuda").float() / case["q_heads"])
    seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), new.long())
    slot = (context[seq] + torch.arange(tokens, device="cuda") - s["starts"][seq]).to(torch.int32)
    if case["document"]:   # documents of one length, at borders of the seed's
        at = torch.randint(0, case["document"], (batch,), generator=gen, device="cuda", dtype=torch.int32)[seq]
        s["first"] = (slot - (slot + at) % case["document"]).clamp(min=0).to(torch.int32)
    if case["prefix"]:
        s["prefix"] = (s["lengths"] // 4).to(torch.int32)
    if case["mode"] == "tree":
        words = -(-case["new"] // 32)
        rng = np.random.default_rng(seed)
        rows = [_tree(rng, n, words) for n in new.tolist()]
        s["tree"] = torch.from_numpy(np.concatenate(rows).view(np.int32)).cuda()
    if case["lse"]:
        s["lse"] = torch.empty(tokens, case["q_heads"], device="cuda")


def _prepare_keep(s, case, gen, seed):
    batch, page = case["batch"], case["page"]
    per = -(-(case["context"] + case["new"]) // page)
    s["block_table"] = torch.randperm(batch * per, generator=gen, device="cuda").to(torch.int32).view(batch, per)
    context = _even(0, case["context"], batch, gen, True)
    s["new"] = _even(1, case["new"], batch, gen, True)
    s["lengths"] = context + s["new"]
    s |= _cache(case, gen, batch * per)
    # the accepted path: some of the drafted tokens in their order
    rng = np.random.default_rng(seed)
    kept, counts = np.zeros((batch, case["most"]), np.int32), np.zeros(batch, np.int32)
    for b, n in enumerate(s["new"].tolist()):
        counts[b] = rng.integers(0, min(n, case["most"]) + 1) if batch > 1 else min(n, case["most"])
        kept[b, : counts[b]] = np.sort(rng.choice(n, counts[b], replace=False))
    s["kept"], s["counts"] = torch.from_numpy(kept).cuda(), torch.from_numpy(counts).cuda()
    if case["tracked"]:
        s["weights"] = torch.rand(s["k"].shape[:3], generator=gen, device="cuda")
        s["positions"] = torch.randint(0, 1 << 20, s["k"].shape[:3], generator=gen, device="cuda", dtype=torch.int32)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_turn(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    if s["weight"] is None:
        y = gbb.rope(s["x"], s["positions_of"], s["table"], layout=c["layout"], sections=s["sections"])
    else:
        y = gbb.norm_rope(s["x"], s["weight"], s["positions_of"], s["table"], eps=EPS, layout=c["layout"],
                          sections=s["sections"])
    if not c["grad"]:
        return [y]
    leaves = [s["x"]] if s["weight"] is None else [s["x"], s["weight"]]
    return [y.detach(), *torch.autograd.grad(y, leaves, s["dy"])]


def _own_append(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    q = gbb.rope_append(s["cache"], s["qkv"], c["q_heads"], s["positions_of"], s["slots"], s["table"],
                        layout=c["layout"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, sections=s["sections"])
    return [q, s["k"], s["v"]]


def _own_attend(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    options = {"lse": s.get("lse"), "softcap": c["cap"], "slopes": s.get("slopes"), "window": c["window"]}
    if c["mode"] == "token":
        out = gbb.paged_attention(s["cache"], s["q"], s["block_table"], s["lengths"], s["max_len"], **options)
    else:
        out = gbb.paged_attention_tokens(s["cache"], s["q"], s["starts"], s["block_table"], s["lengths"], s["max_len"],
                                         first=s.get("first"), prefix=s.get("prefix"), tree=s.get("tree"), **options)
    return [out, s.get("lse")]


def _own_keep(s):
    import gemm_block_bit_amd as gbb
    n = gbb.cache_keep(s["cache"], s["block_table"], s["lengths"], s["new"], s["kept"], s["counts"])
    return [s["k"], s["v"], s.get("weights"), s.get("positions"), n]


def _angles(s):
    """fp32 [T][rot/2][2] of every token and pair."""
    table, positions = s["table"], s["positions_of"].long()
    if s["sections"] is None:
        return table[positions]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"))
    return table[positions[axis].T, torch.arange(table.shape[1], device="cuda")]


def _rotate(x, cs, layout, transpose=False):
    """fp32 [T][H][D] rotated by fp32 cs [T][rot/2][2]."""
    rot = 2 * cs.shape[1]
    c, sn = cs[:, None, :, 0], -cs[:, None, :, 1] if transpose else cs[:, None, :, 1]
    y = x.clone()
    first = slice(0, rot // 2) if layout == "half" else slice(0, rot, 2)
    second = slice(rot // 2, rot) if layout == "half" else slice(1, rot, 2)
    y[..., first] = x[..., first] * c - x[..., second] * sn
    y[..., second] = x[..., second] * c + x[..., first] * sn
    return y


def _plain_turn(s):
    c, cs = s["case"], _angles(s)
    x = s["x"].float()
    if s["weight"] is None:
        out = [_rotate(x, cs, c["layout"]).to(s["x"].dtype)]
        if c["grad"]:
            out.append(_rotate(s["dy"].float(), cs, c["layout"], True).to(s["x"].dtype))
        return out
    w = s["weight"].float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    unit = x * r
    out = [_rotate(unit * w, cs, c["layout"]).to(s["x"].dtype)]
    if c["grad"]:
        g = _rotate(s["dy"].float(), cs, c["layout"], True)
        gw = g * w
        dx = r * (gw - unit * (gw * unit).mean(-1, keepdim=True))
        dw = (g * unit).sum((0, 1), dtype=torch.float64)
        out += [dx.to(s["x"].dtype), dw.to(s["weight"].dtype)]
    return out


def _stored(x, scale, dtype):
    """fp32 [T][kv heads][D] as the cache holds it."""
    return x.to(dtype) if scale is None else (x / scale.view(1, -1, 1)).clamp(-448, 448).to(dtype)


def _plain_append(s):
    c = s["case"]
    x = s["qkv"].float().view(c["tokens"], -1, c["dim"])
    nq, nk = c["q_heads"], c["kv_heads"]
    w = torch.cat([s["q_norm"].float().expand(nq, -1), s["k_norm"].float().expand(nk, -1)])
    qk = x[:, :nq + nk]
    qk = qk * torch.rsqrt((qk * qk).mean(-1, keepdim=True) + EPS) * w
    turned = _rotate(qk, _angles(s), c["layout"])
    at = s["slots"].long()
    page, offset = at // c["page"], at % c["page"]
    bits = {1: torch.uint8, 2: torch.int16}[s["k"].element_size()]   # rows are moved as they are
    s["k"].view(bits)[page, :, offset] = _stored(turned[:, nq:], s["k_scale"], s["k"].dtype).view(bits)
    s["v"].view(bits)[page, :, offset] = _stored(x[:, nq + nk:], s["v_scale"], s["v"].dtype).view(bits)
    return [turned[:, :nq].to(s["qkv"].dtype), s["k"], s["v"]]


def _gathered(cache, scale, table):
    """fp32 [batch][kv heads][slots][D] of the pages in `table`."""
    x = cache.float()[table.long()].transpose(1, 2)
    x = x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])
    return x if scale is None else x * scale.view(1, -1, 1, 1)


def _plain_attend(s):
    """All sequences as a padded batch: `n` rows of tokens, every slot a column."""
    c = s["case"]
    batch, group = c["batch"], c["q_heads"] // c["kv_heads"]
    starts, length = s["starts"].long(), s["lengths"].long()
    new, n = starts.diff(), c["new"]
    i = torch.arange(n, device="cuda")
    real = i < new[:, None]                                        # [batch][n]
    token = torch.where(real, starts[:-1, None] + i, 0)
    q = s["q"].float()[token] * c["dim"] ** -0.5                   # [batch][n][q heads][D]
    q = q.view(batch, n, c["kv_heads"], group, -1).permute(0, 2, 1, 3, 4).reshape(batch, c["kv_heads"], n * group, -1)
    k, v = _gathered(s["k"], s["k_scale"], s["block_table"]), _gathered(s["v"], s["v_scale"], s["block_table"])
    score = torch.matmul(q.contiguous(), k.transpose(-1, -2).contiguous())
    score = score.view(batch, c["kv_heads"], n, group, -1)
    slot = torch.arange(k.shape[2], device="cuda")
    ctx = (length - new)[:, None, None]
    own_slot = ctx + i[:, None]                                    # [batch][n][1]
    behind = own_slot - slot                                       # how far a slot lies behind the token
    there = (slot < length[:, None, None]) & real[..., None]
    if c["mode"] == "tree":
        j = (slot - ctx).clamp(min=0, max=32 * s["tree"].shape[1] - 1)          # [batch][1][slots]
        word = s["tree"].long()[token].gather(2, (j // 32).expand(batch, n, -1))
        drafted = slot >= ctx
        bit = ((word >> (j % 32)) & 1).bool() & drafted & there
        # distances along the tree: the visible drafted tokens behind the slot
        after = bit.long().flip(-1).cumsum(-1).flip(-1) - bit.long()
        behind = torch.where(drafted, after, ctx - 1 - slot + bit.sum(-1, keepdim=True))
        there = there & (bit | ~drafted)
    else:
        seen = behind >= 0
        if c["prefix"]:
            seen = seen | (slot < s["prefix"].long()[:, None, None])
        there = there & seen
        behind = behind.abs()
    if c["window"]:
        there = there & (behind < c["window"])
    if c["document"]:
        there = there & (slot >= s["first"].long()[token][..., None])
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    if c["bias"]:
        slope = s["slopes"].view(1, c["kv_heads"], 1, group, 1)
        score = score - slope * behind[:, None, :, None, :].float()
    score = torch.where(there[:, None, :, None, :], score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total == 0, 1.0, total)).view(batch, c["kv_heads"], n * group, -1)
    o = torch.matmul(p, v.contiguous()).view(batch, c["kv_heads"], n, group, -1)
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, n, c["q_heads"], -1)[real].to(s["q"].dtype)
    lse = None
    if c["lse"]:
        lse = (top + torch.log(total))[..., 0].permute(0, 2, 1, 3).reshape(batch, n, -1)[real]
    return [o, lse]


def _plain_keep(s):
    c = s["case"]
    page, most = c["page"], c["most"]
    table, kept = s["block_table"].long(), s["kept"].long()
    ctx = (s["lengths"] - s["new"]).long()[:, None]
    i = torch.arange(most, device="cuda")
    moves = i < s["counts"][:, None]
    # a row that does not move takes its own place's contents
    dst = (ctx + i).clamp(max=table.shape[1] * page - 1)
    src = torch.where(moves, ctx + kept, dst)
    head = torch.arange(c["kv_heads"], device="cuda")[None, None, :]
    seq = torch.arange(c["batch"], device="cuda")[:, None]
    to = (table[seq, dst // page][..., None], head, (dst % page)[..., None])
    frm = (table[seq, src // page][..., None], head, (src % page)[..., None])
    bits = {1: torch.uint8, 2: torch.int16}[s["k"].element_size()]   # rows are moved as they are
    for x in (s["k"].view(bits), s["v"].view(bits)) + ((s["weights"], s["positions"]) if c["tracked"] else ()):
        x[to] = x[frm]
    return [s["k"], s["v"], s.get("weights"), s.get("positions"), (ctx[:, 0] + s["counts"]).to(torch.int32)]


_run_own = {"turn": _own_turn, "append": _own_append, "attend": _own_attend, "keep": _own_keep}
_run_plain = {"turn": _plain_turn, "append": _plain_append, "attend": _plain_attend, "keep": _plain_keep}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def _shares(case):
    """What a sequence has of the largest context and of the most new tokens, (context, new) of equal shares of the batch."""
    if not case["ragged"] or case["batch"] == 1:
        return [(case["context"], case["new"])]
    even = np.arange(case["batch"]) / (case["batch"] - 1)
    if case["mode"] == "token":
        return [(c, 1) for c in case["context"] * even]
    # contexts and new tokens are dealt out apart: every context with the mean of the new tokens and their mean square
    return [(c, n) for c in (case["context"] * even)[:: max(1, case["batch"] // 8)] for n in case["new"] * even]


def work(case):
    op = case["op"]
    if op in ("turn", "append"):
        t, es = case["tokens"], SIZE[case["dtype"]]
        angles = 4 * t * case["axes"] + 4 * t * case["rot"]
        if op == "turn":
            n = t * case["heads"]
            norm = case["weight"] is not None
            passes = 2 + ((3 if norm else 2) if case["grad"] else 0)
            weight = case["dim"] * SIZE[case["weight"]] * (2 if case["grad"] else 1) if norm else 0
            flops = n * (3 * case["rot"] + (4 * case["dim"] if norm else 0)) * (2.5 if case["grad"] else 1)
            return {"bytes": passes * n * case["dim"] * es + angles + weight, "flops": flops}
        kv = 2 * t * case["kv_heads"] * case["dim"]
        q = t * case["q_heads"] * case["dim"]
        turned = t * (case["q_heads"] + case["kv_heads"])
        return {"bytes": (2 * q + kv) * es + kv * SIZE[case["cache"]] + angles + 4 * t,
                "flops": turned * (3 * case["rot"] + 4 * case["dim"])}
    row = case["dim"] * SIZE[case["cache"]]
    if op == "keep":
        even = [1 + (case["new"] - 1) * b / max(1, case["batch"] - 1) for b in range(case["batch"])]
        if case["batch"] == 1:
            moved = min(case["new"], case["most"])
        else:
            moved = sum(min(n, case["most"]) / 2 for n in even)
        return {"bytes": moved * (case["kv_heads"] * (4 * row + (16 if case["tracked"] else 0)) + 4) + 16 * case["batch"],
                "flops": 0}
    shares = _shares(case)
    pairs = slots = rows = 0.0
    for ctx, new in shares:
        n = max(0, int(round(new)))
        s = ctx + np.arange(n)
        if case["mode"] == "tree":   # the context, and about a tree's depth of it
            seen = np.full(n, ctx + min(n, 4 * np.log2(1 + n))) if n else np.zeros(0)
            first = 0.0
        else:
            low = np.zeros(n)
            if case["document"]:     # a document's border lies anywhere
                low = np.maximum(low, s - (case["document"] - 1) / 2)
            if case["window"]:
                low = np.maximum(low, s + 1 - case["window"])
            seen = s + 1 - low
            if case["prefix"]:
                seen = seen + np.maximum(0, (ctx + n) / 4 - (s + 1))
            first = low.min() if n else 0.0
        if case["window"]:
            seen = np.minimum(seen, case["window"] * (2 if case["prefix"] else 1))
            first = max(first, ctx - case["window"]) if n else 0.0
        pairs += seen.sum()
        slots += ctx + n - first if n else 0.0
        rows += n
    scale = case["batch"] / len(shares)
    pairs, slots, rows = pairs * scale, slots * scale, rows * scale
    b = 2 * slots * case["kv_heads"] * row + 4 * slots / case["page"] + 8 * case["batch"]
    b += rows * case["q_heads"] * (2 * case["dim"] * SIZE[case["dtype"]] + (4 if case["lse"] else 0))
    return {"bytes": b, "flops": 4 * pairs * case["q_heads"] * case["dim"]}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"turn": _exact_turn, "append": _exact_append, "attend": _exact_attend, "keep": _exact_keep}[case["op"]](s)


def _pairs_of(s):
    """64-bit complex [T][1][rot/2]: cos + i sin of each pair's own axis."""
    p = s["positions_of"]
    rows = [s["table"].index_select(0, one) for one in (p if p.dim() == 2 else p[None])]
    z, at = [], 0
    for row, n in zip(rows, s["sections"] or (rows[0].shape[1],)):
        z.append(row[:, at:at + n])
        at += n
    return torch.view_as_complex(torch.cat(z, 1).double().contiguous())[:, None]


def _turned(x, z, layout):
    """64-bit [T][H][D]: each pair as a complex number, times z."""
    half = z.shape[-1]
    body, rest = x[..., :2 * half], x[..., 2 * half:]
    if layout == "half":
        w = torch.complex(body[..., :half].contiguous(), body[..., half:].contiguous()) * z
        return torch.cat([w.real, w.imag, rest], -1)
    w = torch.view_as_complex(body.reshape(*body.shape[:-1], half, 2).contiguous()) * z
    return torch.cat([torch.view_as_real(w).flatten(-2), rest], -1)


def _normed(x, w):
    return w * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _exact_turn(s):
    c = s["case"]
    x = s["x"].detach().double().requires_grad_(c["grad"])
    w = None if s["weight"] is None else s["weight"].detach().double().requires_grad_(c["grad"])
    y = _turned(x if w is None else _normed(x, w), _pairs_of(s), c["layout"])
    if not c["grad"]:
        return [y]
    return [y.detach(), *torch.autograd.grad(y, [x] if w is None else [x, w], s["dy"].double())]


def _exact_append(s):
    c = s["case"]
    nq, nk = c["q_heads"], c["kv_heads"]
    x, z = s["qkv"].double().unflatten(1, (-1, c["dim"])), _pairs_of(s)
    q = _turned(_normed(x[:, :nq], s["q_norm"].double()), z, c["layout"])
    k, v = _turned(_normed(x[:, nq:nq + nk], s["k_norm"].double()), z, c["layout"]), x[:, nq + nk:]
    if s["k_scale"] is not None:
        k = torch.clamp(k / s["k_scale"].double()[None, :, None], -448.0, 448.0)
        v = torch.clamp(v / s["v_scale"].double()[None, :, None], -448.0, 448.0)
    out = [q]
    for cache, rows in ((s["k"], k), (s["v"], v)):
        flat = cache.double().transpose(1, 2).flatten(0, 1).index_copy(0, s["slots"].long(), rows)   # [slot][kv head][D]
        out.append(flat.unflatten(0, (-1, c["page"])).transpose(1, 2).contiguous())
    return out


def _exact_attend(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -torch.inf, dtype=torch.float64, device="cuda")
    starts = s["starts"].tolist()
    for b, n in enumerate(s["lengths"].tolist()):
        t0, t1 = starts[b], starts[b + 1]
        if t0 == t1 or not n:
            continue
        new, ctx = t1 - t0, n - (t1 - t0)
        pages = s["block_table"][b, : -(-n // c["page"])].long()
        place = ctx + torch.arange(new, device="cuda")
        j = torch.arange(n, device="cuda")
        if c["mode"] == "tree":
            words = s["tree"][t0:t1].cpu().numpy().view(np.uint32)
            bits = np.unpackbits(words.view(np.uint8), axis=1, bitorder="little")[:, :new].astype(np.int64)
            depth = bits.sum(1)
            later = depth[:, None] - bits.cumsum(1)
            back = np.concatenate([(ctx - 1 + depth)[:, None] - np.arange(ctx)[None, :], later], 1)
            back = torch.from_numpy(back).cuda()
            seen = torch.from_numpy(np.concatenate([np.ones((new, ctx), bool), bits.astype(bool)], 1)).cuda()
        else:
            back = (place[:, None] - j[None, :])
            seen = back >= 0
            if c["prefix"]:
                seen |= (j < int(s["prefix"][b]))[None, :]
            back = back.abs()
        if c["window"]:
            seen &= back < c["window"]
        if c["document"]:
            seen &= j[None, :] >= s["first"][t0:t1, None]
        for h in range(c["kv_heads"]):
            k = s["k"][pages, h].double().flatten(0, 1)[:n]
            v = s["v"][pages, h].double().flatten(0, 1)[:n]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for g in range(h * group, (h + 1) * group):
                score = (s["q"][t0:t1, g].double() @ k.T) / c["dim"] ** 0.5
                if c["cap"]:
                    score = c["cap"] * torch.tanh(score / c["cap"])
                if c["bias"]:
                    score = score - float(s["slopes"][g]) * back
                score = score.masked_fill(~seen, -torch.inf)
                total = torch.logsumexp(score, -1)
                lse[t0:t1, g] = total
                p = torch.exp(score - torch.where(torch.isinf(total), 0.0, total)[:, None])
                out[t0:t1, g] = p @ v
    return [out, lse if c["lse"] else None]


def _exact_keep(s):
    c, page = s["case"], s["case"]["page"]
    bits = {1: torch.uint8, 2: torch.int16}[s["k"].element_size()]
    table = s["block_table"].cpu().numpy().astype(np.int64)
    kept, counts, new = (s[n].cpu().numpy() for n in ("kept", "counts", "new"))
    k, v = (s[n].view(bits).cpu().numpy() for n in ("k", "v"))
    w = s["weights"].double().cpu().numpy() if c["tracked"] else None
    for b, n in enumerate(s["lengths"].tolist()):
        src = n - new[b] + kept[b, : counts[b]].astype(np.int64)
        dst = n - new[b] + np.arange(counts[b])
        for x in (k, v) if w is None else (k, v, w):
            x[table[b, dst // page], :, dst % page] = x[table[b, src // page], :, src % page].copy()
    wide = lambda x: torch.from_numpy(x).view(s["k"].dtype).cuda().double()  # noqa: E731
    return [wide(k), wide(v), None if w is None else torch.from_numpy(w).cuda(), None, None]
