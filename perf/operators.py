"""Measured cases of the decoder-block operators around the adapted linear layer.

The adapted layer computes the projections of a transformer block for a batch
of requests; the four operators here are what a serving step does between
them: give every request its cache pages and its new tokens their slots
(``resize``), rotate queries and keys by position and write keys and values
into the paged cache (``append``), attend from one new token of each request
over its cached tokens (``attend``), and close a sub-block with its norms,
gate and residual (``norm``).  Head counts and widths are those of the
Llama-3-8B projections (q 4096, k and v 1024: 32 query and 8 key/value heads
of 128), batch sizes those of the decode and prefill workloads, or generic.

Every case is a dict of plain values.  ``prepare`` draws its inputs from the
seed, ``run`` makes one call on them (the framework's where ``own`` is true,
elementary torch operations in 32 bits otherwise) and ``exact`` repeats the
call from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_contexts = {}
FP8_MAX = 448.0


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's chat request on an otherwise idle server: latency only
        _attend("attend_one_request", n=1, lo=777, hi=777, page=16),
        # the 64-request decode batch, contexts spread over a few hundred to 8K tokens
        _attend("attend_decode_64", n=64, lo=200, hi=8192, page=16),
        # many short requests, some of them not started yet (no cached token),
        # pages of 64 tokens with the heads of one token beside each other
        _attend("attend_short_256", n=256, lo=1, hi=1000, empty=16, page=64, token_major=True),
        # few long documents: the batch alone cannot fill the GPU
        _attend("attend_long_4", n=4, lo=100003, hi=131072, page=16),
        # an 8-bit cache under a larger model's heads (eight queries to a key)
        _attend("attend_fp8_64", n=64, lo=500, hi=16384, q_heads=64, page=32, kind="fp8"),
        # a 32-bit context: as many keys as queries, a sliding window, odd pages
        _attend("attend_window_fp32", n=24, lo=30, hi=3000, q_heads=16, kv_heads=16, dim=64, page=24, kind="fp32",
                window=1000),
        # a decode step: every request takes one more token
        _resize("resize_decode_64", n=64, lo=200, hi=8192, page=16),
        # a large mixed step: most requests decode, some end, some begin with a prompt
        _resize("resize_mixed_4096", n=4096, lo=1, hi=4096, page=16, ends=16, begins=32, prompt=1024),
        # the decode batch's keys, values and queries
        _append("append_decode_64", n=64, page=16),
        # a prompt batch with images and video frames in it (three position axes),
        # padded to a fixed length as under a captured graph
        _append("append_prefill_axes", n=8772, page=16, axes=3, pad=37),
        # the decode batch: norm after attention, residual, norm before the feed-forward block
        _norm("norm_decode_64", n=64, d=4096, post=True),
        # the prompt batch, with a per-channel gate and a residual scale
        _norm("norm_prefill_8772", n=8772, d=4096, post=True, gate="vector", scale=0.5),
    ]


def _attend(name, n, lo, hi, page, empty=0, q_heads=32, kv_heads=8, dim=128, kind="bf16", token_major=False,
            window=0, softcap=0.0):
    return {"name": name, "op": "attend", "n": n, "lo": lo, "hi": hi, "empty": empty, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "kind": kind, "token_major": token_major,
            "window": window, "softcap": softcap}


def _resize(name, n, lo, hi, page, ends=0, begins=0, prompt=1, tight=False):
    return {"name": name, "op": "resize", "n": n, "lo": lo, "hi": hi, "page": page, "ends": ends,
            "begins": begins, "prompt": prompt, "tight": tight}


def _append(name, n, page, q_heads=32, kv_heads=8, dim=128, rot=None, axes=1, interleaved=False, kind="bf16",
            token_major=False, pad=0):
    return {"name": name, "op": "append", "n": n, "page": page, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "rot": dim if rot is None else rot, "axes": axes, "interleaved": interleaved,
            "kind": kind, "token_major": token_major, "pad": pad}


def _norm(name, n, d, post=False, gate="none", layer=False, scale=1.0, kind="bf16"):
    return {"name": name, "op": "norm", "n": n, "d": d, "post": post, "gate": gate, "layer": layer,
            "scale": scale, "kind": kind}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over their logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "resize", "append", "norm"])
    if op == "attend":
        kind = rng.choice(["bf16", "bf16", "fp8", "fp32"])
        heads = rng.choice([1, 2, 4, 8, 8, 16])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 8, 16])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        n = _spread(rng, 1, 512)
        token = 2 * heads * dim * {"bf16": 2, "fp8": 1, "fp32": 4}[kind]
        most = max(16, min(131072, int(1.5e9) // (n * token)))
        hi = _spread(rng, 1, most)
        c = _attend("", n=n, lo=max(1, hi // rng.choice([1, 2, 16, 64])), hi=hi, empty=rng.choice([0, 0, 5]),
                    q_heads=heads * group, kv_heads=heads, dim=dim, page=rng.choice([1, 8, 16, 16, 24, 32, 64, 256]),
                    kind=kind, token_major=rng.random() < 0.4,
                    window=_spread(rng, 1, 4096) if rng.random() < 0.25 else 0,
                    softcap=rng.choice([0.0, 0.0, 0.0, 30.0]))
    elif op == "resize":
        hi = _spread(rng, 1, 8192)
        c = _resize("", n=_spread(rng, 1, 4096), lo=max(1, hi // 32), hi=hi, page=rng.choice([1, 8, 16, 24, 64, 256]),
                    ends=rng.choice([0, 3, 16]), begins=rng.choice([0, 4, 32]), prompt=_spread(rng, 1, 1024),
                    tight=rng.random() < 0.3)
    elif op == "append":
        heads, dim = rng.choice([1, 2, 8, 16]), rng.choice([64, 80, 96, 128, 128, 256])
        group = rng.choice([1, 2, 4, 7, 8])
        n = max(1, min(_spread(rng, 1, 16384), int(8772 * 6144 / ((group + 2) * heads * dim))))
        c = _append("", n=n, page=rng.choice([1, 8, 16, 24, 64]), q_heads=heads * group, kv_heads=heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), axes=rng.choice([1, 1, 2, 3]),
                    interleaved=rng.random() < 0.3, kind=rng.choice(["bf16", "bf16", "fp32"]),
                    token_major=rng.random() < 0.4, pad=rng.choice([0, 0, 3]) if n > 8 else 0)
        if c["kind"] == "fp32":
            c["n"] = max(1, c["n"] // 2)
            c["pad"] = min(c["pad"], c["n"] // 3)
    else:
        d = rng.choice([64, 257, 1000, 1024, 2880, 4096, 4096, 5120, 8192, 14336])
        kind = rng.choice(["bf16", "bf16", "fp32"])
        n = max(1, min(_spread(rng, 1, 16384), int(8772 * 4096 / d) // (2 if kind == "fp32" else 1)))
        c = _norm("", n=n, d=d, post=rng.random() < 0.6, gate=rng.choice(["none", "none", "vector", "rows"]),
                  layer=rng.random() < 0.25, scale=rng.choice([1.0, 1.0, 0.22]), kind=kind)
        if c["gate"] == "rows":
            c["n"] = max(1, c["n"] * 4 // 5)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _type(case):
    return torch.float32 if case["kind"] == "fp32" else torch.bfloat16


def _normal(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _lengths(n, lo, hi, empty=0):
    """The batch's lengths: lo to hi, even over their logarithm, the longest
    hi itself; every ``empty``-th request has none."""
    at = (np.arange(n) + 0.5) / n
    lens = np.round(np.exp(np.log(lo) + at * (np.log(hi + 0.5) - np.log(lo)))).astype(np.int64).clip(lo, hi)
    lens[-1] = hi
    if empty:
        lens[::empty] = 0
    return lens


def _pages(lens, page):
    return (lens + page - 1) // page


def _table(rs, lens, page, spare, cols=None):
    """(block table, pages of the pool): every request's pages at random
    places of the pool, -1 beyond its last."""
    need = _pages(lens, page)
    total = int(need.sum()) + spare
    order = rs.permutation(total).astype(np.int32)
    cols = max(1, int(need.max(initial=0))) if cols is None else cols
    table = np.full((len(lens), cols), -1, np.int32)
    table[np.arange(cols)[None, :] < need[:, None]] = order[:int(need.sum())]
    return table, total, order


def _inputs(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"attend": _attend_inputs, "resize": _resize_inputs, "append": _append_inputs,
            "norm": _norm_inputs}[case["op"]](case, rs, gen)


def _attend_inputs(case, rs, gen):
    lens = rs.permutation(_lengths(case["n"], case["lo"], case["hi"], case["empty"]))
    table, total, _ = _table(rs, lens, case["page"], 8)
    H, P, D = case["kv_heads"], case["page"], case["dim"]
    shape = (total, P, H, D) if case["token_major"] else (total, H, P, D)
    s = {"kv_len": torch.from_numpy(lens.astype(np.int32)).cuda(), "block_table": torch.from_numpy(table).cuda(),
         "q": _normal(gen, (case["n"], case["q_heads"], D), _type(case), 1.5)}
    # a recycled page holds anything beyond its request's last token: not a number, here
    rows = np.nonzero(lens % P)[0]
    last = torch.from_numpy(table[rows, lens[rows] // P].astype(np.int64)).cuda()
    tail = (torch.arange(P, device="cuda")[None, :] >= torch.from_numpy(lens[rows] % P).cuda()[:, None])
    page_at, off_at = last[:, None].expand(-1, P)[tail], torch.arange(P, device="cuda")[None, :].expand(len(rows), P)[tail]
    for name in ("k", "v"):
        if case["kind"] == "fp8":
            pool = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
            flat = pool.view(-1)
            for i in range(0, flat.numel(), 1 << 27):
                part = flat[i:i + (1 << 27)]
                part.copy_(_normal(gen, (part.numel(),), torch.bfloat16, 16.0).clamp_(-FP8_MAX, FP8_MAX))
            bits, nan = pool.view(torch.uint8), 0x7F
            s[name + "_scale"] = (torch.rand(H, device="cuda", generator=gen) * 0.05 + 0.04)
        else:
            pool = _normal(gen, shape, _type(case))
            bits, nan = pool, float("nan")
            s[name + "_scale"] = None
        if case["token_major"]:
            bits[page_at, off_at] = nan
        else:
            bits[page_at, :, off_at] = nan
        s[name] = pool
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(case["n"], case["q_heads"], device="cuda")
    return s


def _resize_inputs(case, rs, gen):
    n, page = case["n"], case["page"]
    old = _lengths(n, case["lo"], case["hi"])
    new = old + 1
    at = np.arange(n)
    if case["begins"]:
        old[at % case["begins"] == 1] = 0
        new[at % case["begins"] == 1] = 1 + (at[at % case["begins"] == 1] * 7919) % case["prompt"]
    if case["ends"]:
        new[at % case["ends"] == 0] = 0
    mix = rs.permutation(n)
    old, new = old[mix], new[mix]
    cols = max(1, int(_pages(np.maximum(old, new), page).max()))
    grow = int(np.maximum(_pages(new, page) - _pages(old, page), 0).sum())
    freed = int(np.maximum(_pages(old, page) - _pages(new, page), 0).sum())
    spare = max(0, grow - freed) // 2 if case["tight"] else grow + 64
    table, total, order = _table(rs, old, page, spare, cols)
    free = np.full(max(total, 1), -1, np.int32)
    free[:spare] = order[total - spare:]
    tokens = int(np.maximum(new - old, 0).sum())
    room = max(1, tokens + tokens // 16 + 1)       # the step's fixed number of token rows, as under a captured graph
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    one = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"len_in": dev(old), "len_new": dev(new), "block_table": dev(table), "free_pages": dev(free),
            "free_in": dev([spare]), "free_out": one(1), "len_out": one(n), "cu_new": one(n + 1),
            "slot_map": one(room), "positions": one(room), "token_req": one(room)}


def _append_inputs(case, rs, gen):
    n, H, P, D = case["n"], case["kv_heads"], case["page"], case["dim"]
    total = -(-n * 5 // 4 // P) + 1
    slots = rs.permutation(total)[:-(-n // P)].astype(np.int64)       # whole pages, as a prompt takes them
    slots = (slots[:, None] * P + np.arange(P)[None, :]).reshape(-1)[:n]
    if case["pad"]:
        slots[n - case["pad"]:] = -1
    shape = (total, P, H, D) if case["token_major"] else (total, H, P, D)
    places = 32768
    inv = 500000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])
    angle = np.arange(places)[:, None] * inv[None, :]
    pos = np.stack([rs.randint(0, places >> (3 * a), n) for a in range(case["axes"])])
    dt = _type(case)
    qkv = _normal(gen, (n, case["q_heads"] + 2 * H, D), dt)   # one projection's rows: q, k and v are strided views
    s = {"slot_map": torch.from_numpy(slots.astype(np.int32)).cuda(),
         "positions": torch.from_numpy(pos.astype(np.int32)).cuda(),
         "cos_sin": torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda(),
         "q": qkv[:, :case["q_heads"]], "k": qkv[:, case["q_heads"]:case["q_heads"] + H],
         "v": qkv[:, case["q_heads"] + H:],
         "q_out": torch.empty(n, case["q_heads"], D, dtype=dt, device="cuda"),
         "axis_of_pair": torch.from_numpy(np.repeat(np.arange(case["axes"]), _sections(case))).cuda()}
    # one page more than the pool shows: the plain form's place for padding rows
    s["k_pool"], s["v_pool"] = (torch.zeros((total + 1,) + shape[1:], dtype=dt, device="cuda") for _ in range(2))
    return s


def _sections(case):
    """Pairs of each position axis: the first takes what the others leave."""
    pairs, axes = case["rot"] // 2, case["axes"]
    rest = [pairs // 3] * (axes - 1)
    return [pairs - sum(rest)] + rest


def _norm_inputs(case, rs, gen):
    n, d, dt = case["n"], case["d"], _type(case)
    vec = lambda mean: _normal(gen, (d,), torch.float32, 0.1) + mean  # noqa: E731
    s = {"y": _normal(gen, (n, d), dt, 0.7), "residual": _normal(gen, (n, d), dt, 3.0), "pre_w": vec(1.0),
         "post_w": vec(1.0) if case["post"] else None,
         "pre_b": vec(0.0) if case["layer"] else None,
         "post_b": vec(0.0) if case["layer"] and case["post"] else None,
         "gate": {"none": lambda: None, "vector": lambda: vec(0.5),
                  "rows": lambda: _normal(gen, (n, d), dt, 0.5)}[case["gate"]](),
         "out": torch.empty(n, d, dtype=dt, device="cuda"),
         "residual_out": torch.empty(n, d, dtype=dt, device="cuda")}
    return s


def _context(kind):
    """The framework's context, one for each type, as a server holds it."""
    import lora_normal_form_gb300 as scute
    kind = "fp32" if kind == "fp32" else "bf16"
    if kind not in _contexts:
        _contexts[kind] = scute.Context(dtype=kind, max_tokens=128, max_adapters=1, max_layers=1)
    return _contexts[kind]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:      # the handles that a server keeps for its cache and its positions
        import lora_normal_form_gb300 as scute
        s["ctx"] = _context(case.get("kind", "bf16"))
        if case["op"] == "attend":
            s["cache"] = scute.KvCache(s["k"], s["v"], s["block_table"], token_major=case["token_major"],
                                       k_scale=s["k_scale"], v_scale=s["v_scale"])
        elif case["op"] == "append":
            s["cache"] = scute.KvCache(s["k_pool"][:-1], s["v_pool"][:-1], token_major=case["token_major"])
            s["rope"] = scute.Rope(s["cos_sin"], s["positions"], sections=_sections(case),
                                   interleaved=case["interleaved"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if not own:
        return {"attend": _attend_plain, "resize": _resize_plain, "append": _append_plain,
                "norm": _norm_plain}[case["op"]](case, s)
    ctx = s["ctx"]
    if case["op"] == "attend":
        ctx.paged_attention(s["cache"], s["q"], s["kv_len"], s["out"], lse=s["lse"], window=case["window"],
                            softcap=case["softcap"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "resize":
        ctx.kv_resize(s["len_in"], s["len_new"], s["block_table"], case["page"], s["free_pages"], s["free_in"],
                      s["free_out"], s["len_out"], s["cu_new"], s["slot_map"], s["positions"], s["token_req"])
        return {k: s[k] for k in ("block_table", "free_pages", "free_out", "len_out", "cu_new", "slot_map",
                                  "positions", "token_req")}
    if case["op"] == "append":
        ctx.kv_append(s["cache"], s["slot_map"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], rope=s["rope"])
        return {"q": s["q_out"], "k": s["k_pool"][:-1], "v": s["v_pool"][:-1]}
    ctx.residual_norm(s["y"], s["out"], residual=s["residual"], residual_out=s["residual_out"], pre_w=s["pre_w"],
                      pre_b=s["pre_b"], post_w=s["post_w"], post_b=s["post_b"], gate=s["gate"],
                      scale=case["scale"], eps=1e-5, layer=case["layer"])
    return {"out": s["out"], "residual": s["residual_out"]}


def _gathered(case, s, name):
    """The pool's pages of every request, [n, heads, tokens, dim] in 32 bits."""
    pool, at = s[name], s["block_table"].clamp(min=0).long()
    x = pool.view(torch.uint8)[at].view(pool.dtype) if case["kind"] == "fp8" else pool[at]
    x = x.permute(0, 3, 1, 2, 4) if case["token_major"] else x.permute(0, 2, 1, 3, 4)
    x = x.float().reshape(case["n"], case["kv_heads"], -1, case["dim"])
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][None, :, None, None]
    return x


def _attend_plain(case, s):
    n, H, D = case["n"], case["kv_heads"], case["dim"]
    k = _gathered(case, s, "k")
    at = torch.arange(k.shape[2], device=k.device)[None, :]
    length = s["kv_len"][:, None]
    seen = at < length
    if case["window"]:
        seen = seen & (at >= length - case["window"])
    score = torch.matmul(s["q"].float().view(n, H, -1, D), k.transpose(2, 3)) * D ** -0.5
    del k
    if case["softcap"]:
        score = case["softcap"] * torch.tanh(score / case["softcap"])
    score = torch.where(seen[:, None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], _gathered(case, s, "v"), 0.0)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return {"out": out.view(n, -1, D).to(s["q"].dtype), "lse": (top + torch.log(total)).view(n, -1)}


def _resize_plain(case, s):
    page, old, new, table = case["page"], s["len_in"], s["len_new"], s["block_table"]
    n, cols, room = case["n"], table.shape[1], s["slot_map"].numel()
    have, want = (old + page - 1) // page, (new + page - 1) // page
    drop, need = (have - want).clamp(min=0), (want - have).clamp(min=0)
    drop_at, need_at = drop.cumsum(0) - drop, need.cumsum(0) - need
    # pages of shrinking requests go on top of the free list
    col = torch.arange(cols, device=table.device)[None, :]
    free = torch.cat([s["free_pages"], s["free_pages"].new_zeros(1)])   # one place more, for what is not kept
    going = (col >= want[:, None]) & (col < have[:, None])
    place = s["free_in"].long() + drop_at[:, None] + col - want[:, None]
    dump = free.numel() - 1
    free[torch.where(going, place, dump).view(-1)] = table.view(-1)
    left = s["free_in"] + drop.sum()
    # growing requests are served while pages and token rows last
    fits = (need == 0) | (need_at + need <= left)
    add = torch.where(fits, (new - old).clamp(min=0), 0)
    add = torch.where(add.cumsum(0) <= room, add, 0)
    grown = add > 0
    taken = torch.where(grown, need, 0).sum()
    coming = grown[:, None] & (col >= have[:, None]) & (col < want[:, None])
    source = left.long() - 1 - need_at[:, None] - (col - have[:, None])
    table.copy_(torch.where(coming, free[torch.where(coming, source, 0)], table))
    left = left - taken
    # above the count the list keeps what it held
    above = torch.arange(dump, device=table.device) >= left
    s["free_pages"].copy_(torch.where(above, s["free_pages"], free[:dump]))
    length = torch.where(new > old, old + add, new)
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    token = torch.arange(room, device=table.device)
    req = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    real = req < n
    req = req.clamp(max=n - 1)
    pos = torch.where(real, old[req] + token - cu[req], 0)
    slot = table[req, (pos // page).clamp(max=cols - 1)] * page + pos % page
    return {"block_table": table, "free_pages": s["free_pages"], "free_out": left.int(), "len_out": length.int(),
            "cu_new": cu.int(), "slot_map": torch.where(real, slot, -1).int(), "positions": pos.int(),
            "token_req": torch.where(real, req, -1).int()}


def _turned(case, x, cos, sin):
    """x [n, heads, dim] in 32 bits with its first ``rot`` values turned."""
    rot = case["rot"]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _append_plain(case, s):
    half = case["rot"] // 2
    at = s["positions"].long()[s["axis_of_pair"]].t()                    # [n, pairs]
    cos, sin = s["cos_sin"][:, :half].gather(0, at), s["cos_sin"][:, half:].gather(0, at)
    dt, pages, page = s["q"].dtype, s["k_pool"].shape[0] - 1, case["page"]
    slot = s["slot_map"].long()
    where = torch.where(slot >= 0, slot // page, pages), torch.where(slot >= 0, slot % page, 0)
    for name, x in (("k_pool", _turned(case, s["k"].float(), cos, sin).to(dt)), ("v_pool", s["v"])):
        if case["token_major"]:
            s[name][where[0], where[1]] = x
        else:
            s[name][where[0], :, where[1]] = x
    q = _turned(case, s["q"].float(), cos, sin).to(dt)
    return {"q": q, "k": s["k_pool"][:-1], "v": s["v_pool"][:-1]}


def _normed(case, x, w, b):
    if case["layer"]:
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-5) * w
    return x + b if b is not None else x


def _norm_plain(case, s):
    y = s["y"].float()
    if case["post"]:
        y = _normed(case, y, s["post_w"], s["post_b"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    h = s["residual"].float() + case["scale"] * y
    return {"out": _normed(case, h, s["pre_w"], s["pre_b"]).to(s["out"].dtype), "residual": h.to(s["out"].dtype)}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "fp8": 1, "fp32": 4}.get(case.get("kind"), 4)
    io = 4 if case.get("kind") == "fp32" else 2
    if case["op"] == "attend":
        lens = _lengths(case["n"], case["lo"], case["hi"], case["empty"])
        seen = np.minimum(lens, case["window"]) if case["window"] else lens
        first = lens - seen
        pages = _pages(lens, case["page"]) - first // case["page"]
        rows = case["n"] * case["q_heads"]
        return {"bytes": int(seen.sum()) * 2 * case["kv_heads"] * case["dim"] * size + rows * (case["dim"] * 2 * io + 4)
                + 4 * int(pages.sum()) + 4 * case["n"],
                "flops": 4 * int(seen.sum()) * case["q_heads"] * case["dim"]}
    if case["op"] == "resize":
        old = _lengths(case["n"], case["lo"], case["hi"])
        new, at = old + 1, np.arange(case["n"])
        if case["begins"]:
            old[at % case["begins"] == 1] = 0
            new[at % case["begins"] == 1] = 1 + (at[at % case["begins"] == 1] * 7919) % case["prompt"]
        if case["ends"]:
            new[at % case["ends"] == 0] = 0
        pages = int(np.abs(_pages(new, case["page"]) - _pages(old, case["page"])).sum())
        tokens = int(np.maximum(new - old, 0).sum())
        return {"bytes": 16 * case["n"] + 8 * pages + 12 * (tokens + tokens // 16 + 1) + 4 * case["n"] + 16,
                "flops": 8 * case["n"] + 6 * tokens}
    if case["op"] == "append":
        n, kept = case["n"], case["n"] - case["pad"]
        heads = case["q_heads"] * n + 2 * case["kv_heads"] * kept
        return {"bytes": 2 * heads * case["dim"] * io + 4 * n * (1 + case["axes"]) + min(n, 32768) * case["rot"] * 4,
                "flops": 3 * (case["q_heads"] * n + case["kv_heads"] * kept) * case["rot"]}
    n, d = case["n"], case["d"]
    vectors = 1 + case["post"] + case["layer"] * (1 + case["post"]) + (case["gate"] == "vector")
    return {"bytes": n * d * io * (4 + (case["gate"] == "rows")) + 4 * d * vectors,
            "flops": n * d * (8 + 4 * case["post"])}


# --------------------------------------------------------------------------
# the definitions in 64 bits, one request or row at a time where the plain
# form works on whole batches
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "resize":
        return None         # whole numbers: the outputs have to be equal as they are
    s = _inputs(case, seed)
    return {"attend": _attend_exact, "append": _append_exact, "norm": _norm_exact}[case["op"]](case, s)


def _attend_exact(case, s):
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    G = case["q_heads"] // H
    out = torch.zeros(case["n"], case["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["n"], case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    table, ones = s["block_table"].cpu().numpy(), torch.ones(H, dtype=torch.float64, device="cuda")
    ks = ones if s["k_scale"] is None else s["k_scale"].double()
    vs = ones if s["v_scale"] is None else s["v_scale"].double()
    bits = (lambda x: x.view(torch.uint8)) if case["kind"] == "fp8" else (lambda x: x)
    for r, length in enumerate(s["kv_len"].tolist()):
        first = max(0, length - case["window"]) if case["window"] else 0
        if length == first:
            continue
        t = np.arange(first, length)
        page, off = torch.from_numpy(table[r, t // P].astype(np.int64)).cuda(), torch.from_numpy(t % P).cuda()
        for h in range(H):
            pick = (lambda x: x[page, off, h]) if case["token_major"] else (lambda x: x[page, h, off])
            k = pick(bits(s["k"])).view(s["k"].dtype).to(torch.float64) * ks[h]
            v = pick(bits(s["v"])).view(s["v"].dtype).to(torch.float64) * vs[h]
            a = (s["q"][r, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(D)
            if case["softcap"]:
                a = case["softcap"] * torch.tanh(a / case["softcap"])
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(a, 1)
            out[r, h * G:(h + 1) * G] = torch.softmax(a, 1) @ v
    return {"out": out, "lse": lse}


def _append_exact(case, s):
    sizes, n = _sections(case), case["n"]
    pool = {x: s[x][:-1].double() for x in ("k_pool", "v_pool")}
    cos_sin, pos = s["cos_sin"].double(), s["positions"].long()
    turned = {x: s[x].double() for x in ("q", "k")}
    pair = 0
    for axis, size in enumerate(sizes):
        for i in range(pair, pair + size):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
            z = torch.complex(cos_sin[pos[axis], i], cos_sin[pos[axis], case["rot"] // 2 + i])[:, None]
            for x in turned.values():
                w = torch.complex(x[:, :, a].clone(), x[:, :, b].clone()) * z
                x[:, :, a], x[:, :, b] = w.real, w.imag
        pair += size
    kept = torch.nonzero(s["slot_map"] >= 0)[:, 0]
    slot = s["slot_map"][kept].long()
    page, off = slot // case["page"], slot % case["page"]
    for name, x in (("k_pool", turned["k"]), ("v_pool", s["v"].double())):
        if case["token_major"]:
            pool[name][page, off] = x[kept]
        else:
            pool[name][page, :, off] = x[kept]
    return {"q": turned["q"], "k": pool["k_pool"], "v": pool["v_pool"]}


def _norm_exact(case, s):
    def norm(x, w, b):
        if case["layer"]:
            var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
            x, ms = x - mean, var
        else:
            ms = (x * x).sum(1, keepdim=True) / x.shape[1]
        x = x / torch.sqrt(ms + 1e-5) * w.double()
        return x if b is None else x + b.double()

    t = s["y"].double()
    if s["post_w"] is not None:
        t = norm(t, s["post_w"], s["post_b"])
    if s["gate"] is not None:
        t = t * s["gate"].double()
    h = torch.add(s["residual"].double(), t, alpha=case["scale"])
    return {"out": norm(h, s["pre_w"], s["pre_b"]), "residual": h}
