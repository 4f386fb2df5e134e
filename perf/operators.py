"""Cases of the decoding step's operators around the quantized products: rotary
positions (alone, and fused with the write of k and v into a paged cache),
attention of one new token over that cache, and eviction from it by
accumulated attention weight.

`own = False` computes them in plain torch operations in 32 bits, rounded once
at the end; `own = True` calls the library.  Head counts and head sizes are
those of the Llama-3-8B (32 query heads, 8 kv heads of 128) and Llama-3-70B
(64, 8, 128) layers that the rest of this repository measures, and generic ones.

Caches are [pages][kv heads][page][head size] (fp16, bf16, or e4m3 with one
scale per kv head), with fp32 weights and int32 positions [pages][kv heads][page]
where the cache is tracked.  Slot s of a cache is token s % page of page s // page.
"""
import numpy as np
import torch

own = False

F16, BF16, F32, E4M3 = "f16", "bf16", "f32", "e4m3"
DTYPES = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32, E4M3: torch.float8_e4m3fn}
BASE = 500000.0          # rotary base of the tables


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one user's next token: the smallest call a decoding step makes
        _append("append 1 token", tokens=1, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half", dtype=F16,
                cache=F16, page=64, tracked=False),
        # a decoding batch of odd size into an 8-bit cache that will be evicted from
        _append("append 33 tokens e4m3", tokens=33, q_heads=64, kv_heads=8, dim=128, rot=128, layout="interleaved",
                dtype=BF16, cache=E4M3, page=32, tracked=True),
        # a long prompt's tokens on their way into the cache
        _append("append 8192 tokens", tokens=8192, q_heads=64, kv_heads=8, dim=128, rot=128, layout="half",
                dtype=BF16, cache=BF16, page=64, tracked=False),
        # part of an odd-sized head rotated, a short ragged run of tokens
        _rope("rope part of 96", tokens=777, heads=12, dim=96, rot=24, layout="interleaved", dtype=F16,
              transpose=False),
        # the gradient of a long sequence's queries in training
        _rope("rope gradient 16384", tokens=16384, heads=32, dim=128, rot=128, layout="half", dtype=BF16,
              transpose=True),
        # one user's next token after a short context, small pages
        _attention("attention 1 x 1000", batch=1, q_heads=32, kv_heads=8, dim=128, dtype=F16, cache=F16, page=16,
                   max_len=1000, ragged=False, lse=False, weights=False),
        # a serving batch of ragged contexts
        _attention("attention 32 ragged", batch=32, q_heads=64, kv_heads=8, dim=128, dtype=BF16, cache=BF16, page=64,
                   max_len=8192, ragged=True, lse=False, weights=False),
        # two very long contexts in an 8-bit cache, with the log-sums that joining parts of a context takes
        _attention("attention 2 x 131072 e4m3", batch=2, q_heads=32, kv_heads=8, dim=128, dtype=BF16, cache=E4M3,
                   page=128, max_len=131072, ragged=False, lse=True, weights=False),
        # one kv head per query head, small heads, many short ragged contexts
        _attention("attention 96 mha 64", batch=96, q_heads=12, kv_heads=12, dim=64, dtype=F16, cache=F16, page=32,
                   max_len=2047, ragged=True, lse=False, weights=False),
        # a batch whose attention weights decide what is evicted later
        _attention("attention 16 weights", batch=16, q_heads=32, kv_heads=8, dim=128, dtype=F16, cache=F16, page=64,
                   max_len=4097, ragged=True, lse=False, weights=True),
        # the steady state of a bounded cache: one token over the budget in every sequence
        _evict("evict 1 of 2049", batch=32, kv_heads=8, dim=128, cache=F16, page=64, max_len=2049, ragged=False,
               budget=2048, recent=256, aged=True),
        # a long prompt cut to what is worth keeping
        _evict("evict 32768 to 4096", batch=2, kv_heads=8, dim=128, cache=F16, page=64, max_len=32768, ragged=False,
               budget=4096, recent=512, aged=False),
    ]


def _rope(name, **k):
    return {"name": name, "op": "rope", **k}


def _append(name, **k):
    return {"name": name, "op": "append", **k}


def _attention(name, **k):
    return {"name": name, "op": "attention", **k}


def _evict(name, **k):
    return {"name": name, "op": "evict", **k}


def _spread(rng, low, high):
    """A whole number in [low, high], spread over its logarithm."""
    n = int(round(low * (high / low) ** rng.random()))
    n = max(low, min(high, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "evict"])
    layout = rng.choice(["half", "interleaved"])
    if op == "rope":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.choice([1, 5, 8, 12, 32, 64])
        return {"op": op, "tokens": _spread(rng, 1, min(16384, 2 ** 26 // (heads * dim))), "heads": heads, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim // 4]), "layout": layout, "dtype": rng.choice([F16, BF16, F32]),
                "transpose": rng.random() < 0.5}
    dim, page = rng.choice([64, 128, 128, 256]), rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 12])
    dtype = rng.choice([F16, BF16])
    cache = rng.choice([dtype, dtype, E4M3])
    if op == "evict":
        batch = _spread(rng, 1, 64)
        max_len = _spread(rng, 32, min(65536, 2 ** 27 // (batch * kv_heads * dim)))
        budget = max_len - 1 if rng.random() < 0.3 else _spread(rng, 16, max_len)
        return {"op": op, "batch": batch, "kv_heads": kv_heads, "dim": dim, "cache": cache, "page": page,
                "max_len": max_len, "ragged": rng.random() < 0.5, "budget": budget,
                "recent": rng.choice([0, budget // 8, budget // 2]), "aged": rng.random() < 0.5}
    q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        return {"op": op, "tokens": _spread(rng, 1, min(8192, 2 ** 26 // ((q_heads + 2 * kv_heads) * dim))),
                "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "rot": rng.choice([dim, dim, dim // 2]),
                "layout": layout, "dtype": dtype, "cache": cache, "page": page, "tracked": rng.random() < 0.5}
    batch = _spread(rng, 1, 128)
    max_len = _spread(rng, 1, min(131072, 2 ** 27 // (batch * kv_heads * dim)))
    return {"op": op, "batch": batch, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "cache": cache, "page": page, "max_len": max_len, "ragged": rng.random() < 0.6,
            "lse": rng.random() < 0.3, "weights": rng.random() < 0.3}


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


def _lengths(case, gen):
    """int32 [batch]: max_len, or ragged ones of which the first is max_len."""
    n = torch.full((case["batch"],), case["max_len"], dtype=torch.int32, device="cuda")
    if case["ragged"]:
        n[1:] = torch.randint(0, case["max_len"] + 1, (case["batch"] - 1,), generator=gen, device="cuda",
                              dtype=torch.int32)
    return n


def _block_table(case, gen):
    """int32 [batch][pages of max_len]: a cache whose pages were given out in no order."""
    per = -(-case["max_len"] // case["page"])
    return torch.randperm(case["batch"] * per, generator=gen, device="cuda").to(torch.int32).view(case["batch"], per)


def _cache(case, gen, num_pages):
    shape = (num_pages, case["kv_heads"], case["page"], case["dim"])
    s = {"num_pages": num_pages, "k_scale": None, "v_scale": None}
    if case["cache"] == E4M3:
        s["k_scale"] = torch.rand(case["kv_heads"], generator=gen, device="cuda") * 0.02 + 0.01
        s["v_scale"] = torch.rand(case["kv_heads"], generator=gen, device="cuda") * 0.02 + 0.01
        per_head = {n: s[n].view(1, -1, 1, 1) for n in ("k_scale", "v_scale")}
        s["k"] = (_randn(gen, *shape, dtype=torch.float32) / per_head["k_scale"]).clamp(-448, 448).to(DTYPES[E4M3])
        s["v"] = (_randn(gen, *shape, dtype=torch.float32) / per_head["v_scale"]).clamp(-448, 448).to(DTYPES[E4M3])
    else:
        s["k"] = _randn(gen, *shape, dtype=DTYPES[case["cache"]])
        s["v"] = _randn(gen, *shape, dtype=DTYPES[case["cache"]])
    return s


def _handle(s):
    import gemm_block_bit_amd as gbb
    return gbb.PagedCache(s["k"], s["v"], k_scale=s["k_scale"], v_scale=s["v_scale"], weights=s.get("weights"),
                          positions=s.get("positions"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2654435761 % (1 << 62))
    s = {"case": case}
    if case["op"] in ("rope", "append"):
        n_pos = max(4096, 2 * case["tokens"])
        s["table"] = _table(case["rot"], n_pos)
        start = torch.randint(0, n_pos - case["tokens"], (1,), generator=gen, device="cuda", dtype=torch.int32)
        s["positions_of"] = start + torch.arange(case["tokens"], device="cuda", dtype=torch.int32)
    if case["op"] == "rope":
        s["x"] = _randn(gen, case["tokens"], case["heads"], case["dim"], dtype=DTYPES[case["dtype"]])
    elif case["op"] == "append":
        per = -(-case["tokens"] // case["page"])
        s |= _cache(case, gen, per + 3)
        heads = case["q_heads"] + 2 * case["kv_heads"]
        s["qkv"] = _randn(gen, case["tokens"], heads * case["dim"], dtype=DTYPES[case["dtype"]])
        pages = torch.randperm(per + 3, generator=gen, device="cuda")[:per].to(torch.int32)
        t = torch.arange(case["tokens"], device="cuda", dtype=torch.int32)
        s["slots"] = pages[(t // case["page"]).long()] * case["page"] + t % case["page"]
        if case["tracked"]:
            s["weights"] = torch.rand(s["k"].shape[:3], generator=gen, device="cuda")
            s["positions"] = torch.full(s["k"].shape[:3], -1, device="cuda", dtype=torch.int32)
    else:
        s["block_table"], s["lengths"] = _block_table(case, gen), _lengths(case, gen)
        s |= _cache(case, gen, s["block_table"].numel())
        if case["op"] == "attention":
            # scores of standard deviation 2: some keys matter, most do not
            s["q"] = _randn(gen, case["batch"], case["q_heads"], case["dim"], dtype=DTYPES[case["dtype"]], scale=2.0)
            if case["weights"]:
                s["weights"] = torch.rand(s["k"].shape[:3], generator=gen, device="cuda")
                s["weights_out"] = s["weights"].clone()
            if case["lse"]:
                s["lse"] = torch.empty(case["batch"], case["q_heads"], device="cuda")
        else:
            # attention mass is heavy-tailed; tokens nothing ever attended to are exactly equal
            w = torch.exp(1.5 * torch.randn(s["k"].shape[:3], generator=gen, device="cuda"))
            s["weights"] = torch.where(w < 0.15, torch.zeros_like(w), w)
            s["positions"] = torch.full(s["k"].shape[:3], -1, device="cuda", dtype=torch.int32)
            n = s["block_table"].shape[1] * case["page"]
            pos = torch.arange(n, device="cuda", dtype=torch.int32).expand(case["batch"], case["kv_heads"], n)
            if case["aged"]:   # evictions before this one left the slots in no order of age
                order = torch.rand(case["batch"], case["kv_heads"], case["max_len"], generator=gen, device="cuda")
                pos = torch.nn.functional.pad(2 * order.argsort(-1).to(torch.int32), (0, n - case["max_len"]))
            p = pos.reshape(case["batch"], case["kv_heads"], -1, case["page"]).permute(0, 2, 1, 3)
            s["positions"][s["block_table"].long()] = p.contiguous()
            s["weights_out"], s["positions_out"] = s["weights"].clone(), s["positions"].clone()
    if own and case["op"] != "rope":
        s["cache"] = _handle(s)
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_rope(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    return gbb.rope(s["x"], s["positions_of"], s["table"], layout=c["layout"], transpose=c["transpose"])


def _own_append(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    q = gbb.rope_append(s["cache"], s["qkv"], c["q_heads"], s["positions_of"], s["slots"], s["table"],
                        layout=c["layout"])
    return [q, s["k"], s["v"]] + ([s["positions"], s["weights"]] if c["tracked"] else [])


def _own_attention(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    out = gbb.paged_attention(s["cache"], s["q"], s["block_table"], s["lengths"], c["max_len"], lse=s.get("lse"),
                              weights_out=s.get("weights_out"))
    return [out, s.get("lse"), s.get("weights_out")]


def _own_evict(s):
    import gemm_block_bit_amd as gbb
    c = s["case"]
    n = gbb.cache_evict(s["cache"], s["block_table"], s["lengths"], c["max_len"], c["budget"], c["recent"],
                        weights_out=s["weights_out"], positions_out=s["positions_out"])
    return [s["k"], s["v"], s["weights_out"], s["positions_out"], n]


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


def _plain_rope(s):
    c = s["case"]
    cs = s["table"][s["positions_of"].long()]
    return _rotate(s["x"].float(), cs, c["layout"], c["transpose"]).to(s["x"].dtype)


def _stored(x, scale, dtype):
    """fp32 [T][kv heads][D] as the cache holds it."""
    return x.to(dtype) if scale is None else (x / scale.view(1, -1, 1)).clamp(-448, 448).to(dtype)


def _plain_append(s):
    c = s["case"]
    x = s["qkv"].float().view(c["tokens"], -1, c["dim"])
    cs = s["table"][s["positions_of"].long()]
    turned = _rotate(x[:, :c["q_heads"] + c["kv_heads"]], cs, c["layout"])
    at = s["slots"].long()
    page, offset = at // c["page"], at % c["page"]
    bits = {1: torch.uint8, 2: torch.int16}[s["k"].element_size()]   # rows are moved as they are
    s["k"].view(bits)[page, :, offset] = _stored(turned[:, c["q_heads"]:], s["k_scale"], s["k"].dtype).view(bits)
    s["v"].view(bits)[page, :, offset] = _stored(x[:, c["q_heads"] + c["kv_heads"]:], s["v_scale"],
                                                 s["v"].dtype).view(bits)
    out = [turned[:, :c["q_heads"]].to(s["qkv"].dtype), s["k"], s["v"]]
    if c["tracked"]:
        s["positions"][page, :, offset] = s["positions_of"][:, None].expand(-1, c["kv_heads"])
        s["weights"][page, :, offset] = 0.0
        out += [s["positions"], s["weights"]]
    return out


def _gathered(cache, scale, table):
    """fp32 [batch][kv heads][slots][D] of the pages in `table`."""
    x = cache.float()[table.long()].transpose(1, 2)
    x = x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])
    return x if scale is None else x * scale.view(1, -1, 1, 1)


def _plain_attention(s):
    c = s["case"]
    q = s["q"].float().view(c["batch"], c["kv_heads"], -1, c["dim"])
    k, v = _gathered(s["k"], s["k_scale"], s["block_table"]), _gathered(s["v"], s["v_scale"], s["block_table"])
    score = torch.matmul(k, (q * c["dim"] ** -0.5).transpose(-1, -2).contiguous()).transpose(-1, -2).contiguous()
    slot = torch.arange(k.shape[2], device="cuda")
    there = (slot[None, :] < s["lengths"][:, None])[:, None, None, :]
    score = torch.where(there, score, -torch.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    out = torch.matmul(p, v).view(c["batch"], c["q_heads"], c["dim"]).to(s["q"].dtype)
    lse = (top + torch.log(total)).view(c["batch"], c["q_heads"]) if c["lse"] else None
    weights = None
    if c["weights"]:
        add = p.sum(2).view(c["batch"], c["kv_heads"], -1, c["page"]).transpose(1, 2)
        weights = s["weights_out"]
        weights[s["block_table"].long()] = s["weights"][s["block_table"].long()] + add
    return [out, lse, weights]


def _plain_evict(s):
    c = s["case"]
    table, page = s["block_table"].long(), c["page"]
    flat = lambda x: x[table].transpose(1, 2).reshape(c["batch"], c["kv_heads"], -1)  # noqa: E731
    weight, position = flat(s["weights"]), flat(s["positions"])
    slot = torch.arange(weight.shape[-1], device="cuda")
    length = s["lengths"].long()[:, None, None]
    there = slot < length
    newest = torch.where(there, position, -1).amax(-1, keepdim=True)
    rank = torch.where(position > newest - c["recent"], torch.inf, weight)
    rank = torch.where(there, torch.where(torch.isnan(weight), -torch.inf, rank), -torch.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(there.expand_as(rank)).scatter(-1, order, slot.expand_as(order) < c["budget"]) & there
    stay = torch.clamp(length, max=c["budget"])
    hole, source = ~kept & (slot < stay), kept & (slot >= stay)
    # the i-th dropped slot below the new length takes the i-th kept slot above it
    most = max(1, min(c["budget"], c["max_len"] - c["budget"]))
    number = lambda m: torch.where(m, m.long().cumsum(-1) - 1, most).clamp(max=most)  # noqa: E731
    empty = torch.zeros(*rank.shape[:2], most + 1, dtype=torch.long, device="cuda")
    dst = empty.scatter(-1, number(hole), slot.expand_as(order))[..., :most]
    src = empty.scatter(-1, number(source), slot.expand_as(order))[..., :most]
    moves = hole.sum(-1, keepdim=True)
    i = torch.arange(most, device="cuda")
    last = torch.minimum(i.expand_as(dst), (moves - 1).clamp(min=0))   # past the last move: the last move again
    dst, src = dst.gather(-1, last), src.gather(-1, last)
    dst, src = torch.where(moves > 0, dst, 0), torch.where(moves > 0, src, 0)
    head = torch.arange(c["kv_heads"], device="cuda")[None, :, None]
    seq = torch.arange(c["batch"], device="cuda")[:, None, None]
    to = (table[seq, dst // page], head, dst % page)
    frm = (table[seq, src // page], head, src % page)
    bits = {1: torch.uint8, 2: torch.int16}[s["k"].element_size()]   # rows are moved as they are
    for x in (s["k"].view(bits), s["v"].view(bits)):
        x[to] = x[frm]
    w = weight.scatter(-1, dst, weight.gather(-1, src))
    p = position.scatter(-1, dst, position.gather(-1, src))
    w = torch.where(there, torch.where(slot < stay, w, 0.0), weight)
    p = torch.where(there, torch.where(slot < stay, p, -1), position)
    paged = lambda x: x.view(c["batch"], c["kv_heads"], -1, page).transpose(1, 2)  # noqa: E731
    s["weights_out"][table], s["positions_out"][table] = paged(w), paged(p)
    return [s["k"], s["v"], s["weights_out"], s["positions_out"], stay.view(-1).to(torch.int32)]


_run_own = {"rope": _own_rope, "append": _own_append, "attention": _own_attention, "evict": _own_evict}
_run_plain = {"rope": _plain_rope, "append": _plain_append, "attention": _plain_attention, "evict": _plain_evict}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    size = {F16: 2, BF16: 2, F32: 4, E4M3: 1}
    if case["op"] in ("rope", "append"):
        t = case["tokens"]
        angles = 4 * t + 4 * t * case["rot"]
        if case["op"] == "rope":
            n = t * case["heads"]
            return {"bytes": 2 * n * case["dim"] * size[case["dtype"]] + angles, "flops": 3 * n * case["rot"]}
        kv = 2 * t * case["kv_heads"] * case["dim"]
        q = t * case["q_heads"] * case["dim"]
        extra = 4 * t + (8 * t * case["kv_heads"] if case["tracked"] else 0)
        return {"bytes": (2 * q + kv) * size[case["dtype"]] + kv * size[case["cache"]] + angles + extra,
                "flops": 3 * t * (case["q_heads"] + case["kv_heads"]) * case["rot"]}
    # ragged lengths are uniform in [0, max_len] but for the first
    tokens = case["max_len"] * (1 + (case["batch"] - 1) * (0.5 if case["ragged"] else 1.0))
    row = case["dim"] * size[case["cache"]]
    if case["op"] == "attention":
        b = 2 * tokens * case["kv_heads"] * row + 4 * tokens / case["page"] + 4 * case["batch"]
        b += 2 * case["batch"] * case["q_heads"] * case["dim"] * size[case["dtype"]]
        b += (8 * tokens * case["kv_heads"] if case["weights"] else 0) + (4 * case["batch"] * case["q_heads"] if case["lse"] else 0)
        return {"bytes": b, "flops": 4 * tokens * case["q_heads"] * case["dim"]}
    # of the kept slots of a sequence, the share that lies above the new length moves
    n = case["max_len"]
    lengths = [n] + [n * (i + 0.5) / 64 for i in range(64)] if case["ragged"] else [n]
    scale = [1.0] + [(case["batch"] - 1) / 64.0] * 64 if case["ragged"] else [float(case["batch"])]
    b = 8 * case["batch"]
    for ln, times in zip(lengths, scale):
        over = max(0.0, ln - case["budget"])
        recent = min(case["recent"], ln)
        free = max(0.0, case["budget"] - recent)
        if case["aged"] or recent == 0:
            moved = case["budget"] * over / ln if ln else 0.0
        else:   # the protected slots are the last ones
            inside = min(recent, over)
            moved = inside + free * max(0.0, over - recent) / max(1.0, ln - recent)
        b += times * case["kv_heads"] * (16 * ln + 4 * moved * row)
        b += times * 4 * ln / case["page"]
    return {"bytes": b, "flops": 0}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "append": _exact_append, "attention": _exact_attention, "evict": _exact_evict}[case["op"]](s)


def _turned(x, angle_pairs, layout, sign):
    """64-bit [T][H][D]: each pair as a complex number, times cos + i sin."""
    half = angle_pairs.shape[1]
    z = torch.view_as_complex(angle_pairs.double().contiguous())
    z = (z.conj() if sign < 0 else z)[:, None, :]
    body, rest = x[..., :2 * half].double(), x[..., 2 * half:].double()
    if layout == "half":
        w = torch.complex(body[..., :half].contiguous(), body[..., half:].contiguous()) * z
        return torch.cat([w.real, w.imag, rest], -1)
    w = torch.view_as_complex(body.reshape(*body.shape[:-1], half, 2).contiguous()) * z
    return torch.cat([torch.view_as_real(w).flatten(-2), rest], -1)


def _exact_rope(s):
    c = s["case"]
    return _turned(s["x"], s["table"].index_select(0, s["positions_of"]), c["layout"], -1 if c["transpose"] else 1)


def _exact_append(s):
    c = s["case"]
    nq, nk = c["q_heads"], c["kv_heads"]
    x = s["qkv"].unflatten(1, (-1, c["dim"]))
    cs = s["table"].index_select(0, s["positions_of"])
    q, k, v = _turned(x[:, :nq], cs, c["layout"], 1), _turned(x[:, nq:nq + nk], cs, c["layout"], 1), x[:, nq + nk:].double()
    if s["k_scale"] is not None:
        k = torch.clamp(k / s["k_scale"].double()[None, :, None], -448.0, 448.0)
        v = torch.clamp(v / s["v_scale"].double()[None, :, None], -448.0, 448.0)
    out = [q]
    for cache, new in ((s["k"], k), (s["v"], v)):
        rows = cache.double().transpose(1, 2).flatten(0, 1)      # [slot][kv head][D]
        rows = rows.index_copy(0, s["slots"].long(), new)
        out.append(rows.unflatten(0, (-1, c["page"])).transpose(1, 2).contiguous())
    if c["tracked"]:
        out.append(None)
        zero = s["weights"].double().transpose(1, 2).flatten(0, 1).index_fill(0, s["slots"].long(), 0.0)
        out.append(zero.unflatten(0, (-1, c["page"])).transpose(1, 2).contiguous())
    return out


def _exact_attention(s):
    c = s["case"]
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(c["batch"], c["q_heads"], c["dim"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["q_heads"]), -torch.inf, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if c["weights"] else None
    for b, n in enumerate(s["lengths"].tolist()):
        pages = s["block_table"][b, : -(-n // c["page"])].long()
        if not n:
            continue
        for h in range(c["kv_heads"]):
            k = s["k"][pages, h].double().flatten(0, 1)[:n]
            v = s["v"][pages, h].double().flatten(0, 1)[:n]
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            heads = slice(h * group, (h + 1) * group)
            score = (s["q"][b, heads].double() @ k.T) / c["dim"] ** 0.5
            lse[b, heads] = torch.logsumexp(score, -1)
            p = torch.softmax(score, -1)
            out[b, heads] = p @ v
            if weights is not None:
                i = torch.arange(n, device="cuda")
                weights[pages[i // c["page"]], h, i % c["page"]] += p.sum(0)
    return [out, lse if c["lse"] else None, weights]


def _exact_evict(s):
    c = s["case"]
    page, budget = c["page"], c["budget"]
    k, v, w, p = (s[n].cpu() for n in ("k", "v", "weights", "positions"))
    # no arithmetic on k and v: their rows move, and are widened afterwards
    bits = {1: torch.uint8, 2: torch.int16}[k.element_size()]
    k, v = k.view(bits).numpy(), v.view(bits).numpy()
    w64, table = w.double().numpy(), s["block_table"].cpu().numpy().astype(np.int64)
    p = p.numpy()
    w_out = w64.copy()
    for b, n in enumerate(s["lengths"].tolist()):
        i = np.arange(n)
        pg, off = table[b, i // page], i % page
        for h in range(c["kv_heads"]):
            if n <= budget:
                continue
            wt, ps = w64[pg, h, off], p[pg, h, off]
            old = ps <= ps.max() - c["recent"]
            # protected first, then by weight, the lower slot before the higher one
            best = np.lexsort((i, -np.where(old, wt, 0.0), old))[:budget]
            kept = np.zeros(n, bool)
            kept[best] = True
            dst, src = np.flatnonzero(~kept[:budget]), budget + np.flatnonzero(kept[budget:])
            w_out[pg[dst], h, off[dst]] = wt[src]
            w_out[pg[budget:], h, off[budget:]] = 0.0
            for x in (k, v):
                x[pg[dst], h, off[dst]] = x[pg[src], h, off[src]]
    wide = lambda x: torch.from_numpy(x).view(s["k"].dtype).cuda().double()  # noqa: E731
    return [wide(k), wide(v), torch.from_numpy(w_out).cuda(), None, None]
