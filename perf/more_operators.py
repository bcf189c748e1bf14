"""Measured cases of the operators for caches whose pages several requests share.

A serving step that branches (several samples of one prompt, beam search, a
system prompt in front of every request) needs more than one page list for each
request: rows of the block table that continue other rows, sharing their full
pages and copying the last one (``fork``); one new token of each request over a
context whose beginning is the same for a group of requests (``shared``); over
the first tokens of a context and its last ones (``sinks``); and the cache
write of models that norm every head's queries and keys before they are turned
(``append``).  Head counts and widths are those of the Llama-3-8B projections
(32 query and 8 key/value heads of 128), batch sizes those of the decode and
prefill workloads, or generic.

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
        # one long chat whose model keeps its first tokens and a window: latency only
        _sinks("sinks_one_request", n=1, lo=20011, hi=20011, window=1024, sinks=4, page=16),
        # the 64-request decode batch of such a model, most contexts longer than its window
        _sinks("sinks_decode_64", n=64, lo=200, hi=32768, window=4096, sinks=4, page=16),
        # an 8-bit cache, a batch of uneven contexts, a whole page and a half of first tokens
        _sinks("sinks_fp8_200", n=200, lo=30, hi=5000, window=1000, sinks=24, page=16, kind="fp8", empty=16),
        # two samples of one prompt: latency
        _shared("shared_two_samples", groups=1, per=2, lo=1536, hi=1536, own=40, page=16),
        # the 64-request decode batch behind one long system prompt
        _shared("shared_decode_64", groups=1, per=64, lo=8192, hi=8192, own=512, page=16),
        # ten adapters' system prompts of 500 to 4000 tokens, 8-bit cache, pages of 64
        # tokens with the heads of one token beside each other, some rows idle
        _shared("shared_adapters_250", groups=10, per=25, lo=512, hi=4032, own=1000, page=64, kind="fp8",
                token_major=True, empty=16),
        # many questions about one long document
        _shared("shared_document_32", groups=1, per=32, lo=131072, hi=131072, own=300, page=32),
        # the decode batch's queries, keys and values, normed by head
        _append("append_norm_decode_64", n=64, page=16),
        # a prompt batch, padded to a fixed length as under a captured graph
        _append("append_norm_prefill_8772", n=8772, page=16, pad=37),
        # beam search: 16 prompts of 4 beams choose which beams go on
        _fork("fork_beams_64", prompts=16, width=4, lo=200, hi=8192, own=256, page=16, layers=2),
        # one prompt becomes 64 samples
        _fork("fork_samples_64", prompts=1, width=64, lo=8189, hi=8189, own=1, page=16, layers=4, samples=True),
        # a large batch of short beams, some prompts end, some rows give tokens back
        _fork("fork_beams_4096", prompts=1024, width=4, lo=17, hi=512, own=64, page=16, layers=1, ends=16, cut=8),
    ]


def _sinks(name, n, lo, hi, window, sinks, page, empty=0, q_heads=32, kv_heads=8, dim=128, kind="bf16",
           token_major=False):
    return {"name": name, "op": "sinks", "n": n, "lo": lo, "hi": hi, "empty": empty, "window": window,
            "sinks": sinks, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "kind": kind,
            "token_major": token_major}


def _shared(name, groups, per, lo, hi, own, page, empty=0, alone=0, q_heads=32, kv_heads=8, dim=128, kind="bf16",
            token_major=False):
    return {"name": name, "op": "shared", "groups": groups, "per": per, "lo": lo, "hi": hi, "own": own,
            "empty": empty, "alone": alone, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
            "kind": kind, "token_major": token_major}


def _append(name, n, page, q_heads=32, kv_heads=8, dim=128, rot=None, interleaved=False, layer=False, each=False,
            kind="bf16", token_major=False, pad=0):
    return {"name": name, "op": "append", "n": n, "page": page, "q_heads": q_heads, "kv_heads": kv_heads,
            "dim": dim, "rot": dim if rot is None else rot, "interleaved": interleaved, "layer": layer,
            "each": each, "kind": kind, "token_major": token_major, "pad": pad}


def _fork(name, prompts, width, lo, hi, own, page, layers, samples=False, ends=0, cut=0, tight=False, kv_heads=8,
          dim=128, kind="bf16", token_major=False):
    return {"name": name, "op": "fork", "prompts": prompts, "width": width, "lo": lo, "hi": hi, "own": own,
            "page": page, "layers": layers, "samples": samples, "ends": ends, "cut": cut, "tight": tight,
            "kv_heads": kv_heads, "dim": dim, "kind": kind, "token_major": token_major}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over their logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


_SIZE = {"bf16": 2, "fp8": 1, "fp32": 4}


def draw(rng):
    op = rng.choice(["sinks", "shared", "shared", "append", "fork"])
    if op in ("sinks", "shared"):
        kind = rng.choice(["bf16", "bf16", "fp8", "fp32"])
        heads, group = rng.choice([1, 2, 4, 8, 8]), rng.choice([1, 2, 3, 4, 4, 7, 8, 16])
        dim, page = rng.choice([64, 80, 96, 128, 128, 128, 256]), rng.choice([1, 8, 16, 16, 24, 32, 64, 256])
        token, major = 2 * heads * dim * _SIZE[kind], rng.random() < 0.4
    if op == "sinks":
        n, window, sinks = _spread(rng, 1, 512), _spread(rng, 1, 8192), _spread(rng, 1, 256)
        most = max(16, min(131072, int(9e8) // (n * token)))
        hi = _spread(rng, 1, most)
        window = max(1, min(window, int(4e9) // (n * heads * dim * 8)))
        c = _sinks("", n=n, lo=max(1, hi // rng.choice([1, 2, 16, 64])), hi=hi, window=window, sinks=sinks,
                   page=page, empty=rng.choice([0, 0, 5]), q_heads=heads * group, kv_heads=heads, dim=dim, kind=kind,
                   token_major=major)
    elif op == "shared":
        groups, per = rng.choice([1, 1, 2, 5, 12]), _spread(rng, 1, 96)
        n = groups * per
        most = min(131072, int(5e8) // (groups * token), int(6e10) // (4 * n * heads * group * dim))
        hi = _spread(rng, 1, max(16, most))
        c = _shared("", groups=groups, per=per, lo=max(1, hi // rng.choice([1, 1, 4])), hi=hi,
                    own=_spread(rng, 1, max(2, min(1024, int(3e8) // (n * token)))), page=page,
                    empty=rng.choice([0, 0, 7]), alone=rng.choice([0, 0, 3]), q_heads=heads * group, kv_heads=heads,
                    dim=dim, kind=kind, token_major=major)
    elif op == "append":
        heads, dim = rng.choice([1, 2, 8, 16]), rng.choice([64, 80, 96, 128, 128, 256])
        group = rng.choice([1, 2, 4, 7, 8])
        n = max(1, min(_spread(rng, 1, 16384), int(8772 * 6144 / ((group + 2) * heads * dim))))
        c = _append("", n=n, page=rng.choice([1, 8, 16, 24, 64]), q_heads=heads * group, kv_heads=heads, dim=dim,
                    rot=rng.choice([dim, dim, dim // 2]), interleaved=rng.random() < 0.3, layer=rng.random() < 0.3,
                    each=rng.random() < 0.3, kind=rng.choice(["bf16", "bf16", "fp32"]),
                    token_major=rng.random() < 0.4, pad=rng.choice([0, 0, 3]) if n > 8 else 0)
        if c["kind"] == "fp32":
            c["n"] = max(1, c["n"] // 2)
            c["pad"] = min(c["pad"], c["n"] // 3)
    else:
        prompts, width, heads = _spread(rng, 1, 512), rng.choice([1, 2, 4, 5, 16]), rng.choice([1, 2, 8])
        dim, page, layers = rng.choice([64, 80, 128]), rng.choice([1, 8, 16, 24, 64]), rng.choice([1, 2, 3])
        kind = rng.choice(["bf16", "bf16", "fp32"])
        token = 2 * heads * dim * _SIZE[kind] * layers
        prompts = max(1, min(prompts, int(5e8) // (width * page * token)))
        own_most = max(1, min(256, int(6e8) // (prompts * width * token)))
        hi = _spread(rng, 1, max(1, min(8192, int(6e8) // (prompts * token))))
        c = _fork("", prompts=prompts, width=width, lo=max(1, hi // rng.choice([1, 4, 32])), hi=hi,
                  own=_spread(rng, 1, own_most), page=page, layers=layers, samples=rng.random() < 0.3,
                  ends=rng.choice([0, 3, 16]), cut=rng.choice([0, 0, 5]), tight=rng.random() < 0.2, kv_heads=heads,
                  dim=dim, kind=kind, token_major=rng.random() < 0.4)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _type(case):
    return torch.float32 if case["kind"] == "fp32" else torch.bfloat16


def _normal(gen, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _lengths(n, lo, hi, empty=0):
    """The batch's lengths: lo to hi, even over their logarithm, the longest
    hi itself; every ``empty``-th request has none."""
    at = (np.arange(n) + 0.5) / n
    lens = np.round(np.exp(np.log(lo) + at * (np.log(hi + 0.5) - np.log(lo)))).astype(np.int64).clip(lo, hi)
    lens[-1] = hi
    if empty:
        lens[::empty] = 0
    return lens


def _ceil(a, b):
    return (a + b - 1) // b


def _pool_shape(case, pages):
    H, P, D = case["kv_heads"], case["page"], case["dim"]
    return (pages, P, H, D) if case["token_major"] else (pages, H, P, D)


def _pools(case, gen, pages, holes):
    """Key and value pools with their scales; ``holes`` (page, first token that
    holds nothing yet): a recycled page holds anything there, not a number here."""
    s, P = {}, case["page"]
    page = torch.from_numpy(np.array([p for p, _ in holes], np.int64)).cuda()
    first = torch.from_numpy(np.array([t for _, t in holes], np.int64)).cuda()
    off = torch.arange(P, device="cuda")[None, :].expand(len(holes), P)
    tail = off >= first[:, None]
    page, off = page[:, None].expand(-1, P)[tail], off[tail]
    for name in ("k", "v"):
        if case["kind"] == "fp8":
            pool = torch.empty(_pool_shape(case, pages), dtype=torch.float8_e4m3fn, device="cuda")
            flat = pool.view(-1)
            for i in range(0, flat.numel(), 1 << 27):
                part = flat[i:i + (1 << 27)]
                part.copy_(_normal(gen, (part.numel(),), torch.bfloat16, 16.0).clamp_(-FP8_MAX, FP8_MAX))
            bits, nan = pool.view(torch.uint8), 0x7F
            s[name + "_scale"] = torch.rand(case["kv_heads"], device="cuda", generator=gen) * 0.05 + 0.04
        else:
            pool = _normal(gen, _pool_shape(case, pages), _type(case))
            bits, nan = pool, float("nan")
            s[name + "_scale"] = None
        if case["token_major"]:
            bits[page, off] = nan
        else:
            bits[page, :, off] = nan
        s[name] = pool
    return s


def _inputs(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"sinks": _sinks_inputs, "shared": _shared_inputs, "append": _append_inputs,
            "fork": _fork_inputs}[case["op"]](case, rs, gen)


def _attention_buffers(case, s, n, gen):
    s["q"] = _normal(gen, (n, case["q_heads"], case["dim"]), _type(case), 1.5)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(n, case["q_heads"], device="cuda")
    return s


def _sinks_inputs(case, rs, gen):
    lens = rs.permutation(_lengths(case["n"], case["lo"], case["hi"], case["empty"]))
    need, P = _ceil(lens, case["page"]), case["page"]
    total = int(need.sum()) + 8
    order, cols = rs.permutation(total).astype(np.int32), max(1, int(need.max(initial=0)))
    table = np.full((case["n"], cols), -1, np.int32)
    table[np.arange(cols)[None, :] < need[:, None]] = order[:int(need.sum())]
    rows = np.nonzero(lens % P)[0]
    s = _pools(case, gen, total, [(table[r, lens[r] // P], lens[r] % P) for r in rows])
    s["kv_len"], s["block_table"] = _dev(lens), _dev(table)
    return _attention_buffers(case, s, case["n"], gen)


def _group_plan(case):
    """Tokens that each group's requests share (whole pages), requests in all
    (those behind the last group share nothing), and own tokens of each."""
    P, n = case["page"], case["groups"] * case["per"] + case["alone"]
    common = np.maximum(1, _lengths(case["groups"], case["lo"], case["hi"]) // P) * P
    own_len = _lengths(n, 1, case["own"])
    return common, n, own_len


def _shared_inputs(case, rs, gen):
    P, per = case["page"], case["per"]
    common, n, own_len = _group_plan(case)
    own_len = rs.permutation(own_len)
    base = np.concatenate([np.repeat(common, per), np.zeros(case["alone"], np.int64)])
    lens = base + own_len
    if case["empty"]:
        lens[1::case["empty"]] = 0
    own_pages = np.where(lens > 0, _ceil(own_len, P), 0)
    total = int(common.sum() // P + own_pages.sum()) + 8
    order, at = rs.permutation(total).astype(np.int32), 0
    table = np.full((n, max(1, int(_ceil(base + own_len, P).max()))), -1, np.int32)
    for g in range(case["groups"]):
        k = int(common[g]) // P
        table[g * per:(g + 1) * per, :k] = order[at:at + k]      # an idle row still names its group's pages
        at += k
    holes = []
    for r in range(n):
        k, first = int(own_pages[r]), int(base[r]) // P
        table[r, first:first + k] = order[at:at + k]
        at += k
        if lens[r] % P:
            holes.append((table[r, lens[r] // P], lens[r] % P))
    s = _pools(case, gen, total, holes)
    s["kv_len"], s["block_table"], s["common"] = _dev(lens), _dev(table), _dev(common)
    s["start"] = _dev(np.arange(case["groups"] + 1) * per)
    return _attention_buffers(case, s, n, gen)


def _append_inputs(case, rs, gen):
    n, H, P, D = case["n"], case["kv_heads"], case["page"], case["dim"]
    total = -(-n * 5 // 4 // P) + 1
    slots = rs.permutation(total)[:-(-n // P)].astype(np.int64)       # whole pages, as a prompt takes them
    slots = (slots[:, None] * P + np.arange(P)[None, :]).reshape(-1)[:n]
    if case["pad"]:
        slots[n - case["pad"]:] = -1
    places = 32768
    inv = 500000.0 ** (-np.arange(0, case["rot"], 2) / case["rot"])
    angle = np.arange(places)[:, None] * inv[None, :]
    dt = _type(case)
    qkv = _normal(gen, (n, case["q_heads"] + 2 * H, D), dt)   # one projection's rows: q, k and v are strided views
    weight = lambda heads: _normal(gen, (heads, D) if case["each"] else (D,), torch.float32, 0.2) + 1.0  # noqa: E731
    s = {"slot_map": _dev(slots), "positions": _dev(rs.randint(0, places, n)),
         "cos_sin": torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda(),
         "q": qkv[:, :case["q_heads"]], "k": qkv[:, case["q_heads"]:case["q_heads"] + H],
         "v": qkv[:, case["q_heads"] + H:], "q_w": weight(case["q_heads"]), "k_w": weight(H),
         "q_out": torch.empty(n, case["q_heads"], D, dtype=dt, device="cuda")}
    # one page more than the pool shows: the plain form's place for padding rows
    s["k_pool"], s["v_pool"] = (torch.zeros(_pool_shape(case, total + 1), dtype=dt, device="cuda") for _ in range(2))
    return s


def _fork_inputs(case, rs, gen):
    P, width, n = case["page"], case["width"], case["prompts"] * case["width"]
    prompt = rs.permutation(_lengths(case["prompts"], case["lo"], case["hi"]))
    if case["samples"]:                       # a row for each prompt, continued by `width` rows
        len_in, source = prompt, np.repeat(np.arange(case["prompts"]), width)
        shared = np.zeros(len(prompt), np.int64)
    else:                                     # beams: the prompt's full pages are shared, the rest a beam's own
        base = np.repeat(prompt, width)
        len_in = base + np.repeat(rs.randint(1, case["own"] + 1, case["prompts"]), width)
        source = np.repeat(np.arange(case["prompts"]), width) * width + rs.randint(0, width, n)
        shared = base // P if width > 1 else 0 * base
    if case["ends"]:
        source[(source // (1 if case["samples"] else width)) % case["ends"] == 0] = -1
    len_new = np.where(source >= 0, len_in[source], 0)
    if case["cut"]:                           # rows that give tokens back (a speculation that failed)
        who = np.arange(n) % case["cut"] == 1
        len_new[who] = np.maximum(len_new[who] - 1 - np.arange(n)[who] * 7919 % (2 * P + 3), 0)
    need = _ceil(len_in, P)
    # a pool of one size whatever the seed, so that some of its pages are others'
    if case["samples"]:
        total = int(need.sum())
    elif width == 1:
        total = int(_ceil(prompt + case["own"], P).sum())
    else:
        total = int((prompt // P).sum()) + n * _ceil(P - 1 + case["own"], P)
    spare = n // 8 if case["tight"] else n + 16
    total += spare
    order, at = rs.permutation(total).astype(np.int32), 0
    table = np.full((len(len_in), _ceil(case["hi"] + case["own"], P) + 1), -1, np.int32)
    extra = np.zeros(total, np.int32)
    for r in range(len(len_in)):
        k = int(shared[r])
        if k and r % width:
            table[r, :k] = table[r - 1, :k]
            extra[table[r, :k]] += 1
        elif k:
            table[r, :k] = order[at:at + k]
            at += k
        own_k = int(need[r]) - k
        table[r, k:k + own_k] = order[at:at + own_k]
        at += own_k
    free = np.full(total, -1, np.int32)
    free[:spare] = order[total - spare:]
    dt, whole = _type(case), lambda *k: torch.zeros(*k, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"table_in": _dev(table), "len_in": _dev(len_in), "source": _dev(source), "len_new": _dev(len_new),
         "table_out": whole(n, table.shape[1]) - 1, "len_out": whole(n), "book0": _dev(np.concatenate([extra, free])),
         "free_in": _dev([spare]), "free_out": whole(1), "copy_from": whole(n), "copy_to": whole(n),
         "copy_tokens": whole(n)}
    # counts and free list, which a step changes in place: brought back before every pass
    s["book"] = s["book0"].clone()
    s["extra"], s["free"] = s["book"][:total], s["book"][total:]
    # one page more than the pools show: the plain form's place for rows that copy nothing
    s["k"], s["v"] = ([_normal(gen, _pool_shape(case, total + 1), dt) for _ in range(case["layers"])] for _ in range(2))
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
    if own:      # the handles that a server keeps for its cache, its positions and its weights
        import lora_normal_form_gb300 as scute
        ctx = s["ctx"] = _context(case["kind"])
        major = case["token_major"]
        if case["op"] in ("sinks", "shared"):
            s["cache"] = scute.KvCache(s["k"], s["v"], s["block_table"], token_major=major, k_scale=s["k_scale"],
                                       v_scale=s["v_scale"])
            if case["op"] == "shared":
                work = ctx.shared_work(s["cache"], s["q"].shape[0], case["q_heads"])
                s["prefix"] = scute.Shared(s["start"], s["common"], work)
        elif case["op"] == "append":
            s["cache"] = scute.KvCache(s["k_pool"][:-1], s["v_pool"][:-1], token_major=major)
            s["rope"] = scute.Rope(s["cos_sin"], s["positions"], interleaved=case["interleaved"])
            s["norm"] = scute.HeadNorm(s["q_w"], s["k_w"], eps=1e-6, layer=case["layer"])
        else:
            s["caches"] = scute.KvCaches([scute.KvCache(k[:-1], v[:-1], token_major=major)
                                          for k, v in zip(s["k"], s["v"])])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    case = s["case"]
    if case["op"] == "fork":
        s["book"].copy_(s["book0"])
    if not own:
        return {"sinks": _sinks_plain, "shared": _shared_plain, "append": _append_plain,
                "fork": _fork_plain}[case["op"]](case, s)
    ctx = s["ctx"]
    if case["op"] == "sinks":
        ctx.paged_attention(s["cache"], s["q"], s["kv_len"], s["out"], lse=s["lse"], window=case["window"],
                            sinks=case["sinks"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "shared":
        ctx.paged_attention(s["cache"], s["q"], s["kv_len"], s["out"], lse=s["lse"], shared=s["prefix"])
        return {"out": s["out"], "lse": s["lse"]}
    if case["op"] == "append":
        ctx.kv_append(s["cache"], s["slot_map"], s["k"], s["v"], q=s["q"], q_out=s["q_out"], rope=s["rope"],
                      norm=s["norm"])
        return {"q": s["q_out"], "k": s["k_pool"][:-1], "v": s["v_pool"][:-1]}
    ctx.kv_fork(s["table_in"], s["len_in"], s["source"], s["table_out"], s["len_out"], case["page"], s["extra"],
                s["free"], s["free_in"], s["free_out"], s["copy_from"], s["copy_to"], s["copy_tokens"],
                len_new=s["len_new"])
    ctx.kv_copy(s["caches"], s["copy_from"], s["copy_to"], s["copy_tokens"])
    return _fork_outputs(s)


def _fork_outputs(s):
    out = {k: s[k] for k in ("table_out", "len_out", "extra", "free", "free_out", "copy_from", "copy_to",
                             "copy_tokens")}
    out["k"], out["v"] = [x[:-1] for x in s["k"]], [x[:-1] for x in s["v"]]
    return out


def _picked(case, s, name, page, off):
    """Tokens ``off`` of pages ``page`` (of one shape) in 32 bits, heads first:
    [.., heads, tokens, dim]."""
    pool = s[name].view(torch.uint8) if case["kind"] == "fp8" else s[name]
    x = pool[page, off] if case["token_major"] else pool.permute(0, 2, 1, 3)[page, off]
    x = x.view(s[name].dtype).float().transpose(-3, -2)
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"][:, None, None]
    return x


def _joined(q, parts, scale):
    """Attention of q [.., rows, dim] over several parts (keys, values, which
    count) together: (out, lse)."""
    scores = [torch.where(seen, torch.matmul(q, k.transpose(-2, -1)) * scale, -math.inf) for k, _, seen in parts]
    top = torch.stack([x.amax(-1, keepdim=True) for x in scores]).amax(0)
    top = torch.where(top == -math.inf, 0.0, top)
    weights = [torch.exp(x - top) for x in scores]
    total = sum(w.sum(-1, keepdim=True) for w in weights)
    out = sum(torch.matmul(w, torch.where(seen.transpose(-2, -1), v, 0.0)) for w, (_, v, seen) in zip(weights, parts))
    return out / torch.where(total == 0, 1.0, total), (top + torch.log(total))[..., 0]


def _sinks_plain(case, s):
    n, H, D, P = case["n"], case["kv_heads"], case["dim"], case["page"]
    length = s["kv_len"].long()[:, None]
    S, W = min(case["sinks"], case["hi"]), min(case["window"], case["hi"])
    first = torch.arange(S, device="cuda")[None, :].expand(n, S)
    last = length - W + torch.arange(W, device="cuda")[None, :]
    at = torch.cat([first, last], 1)
    seen = torch.cat([first < length, last >= S], 1)        # the window's part among the first tokens counts once
    at = torch.where(seen, at, 0)
    page = s["block_table"].long().gather(1, at // P).clamp(min=0)
    k, v = (_picked(case, s, x, page, at % P) for x in ("k", "v"))
    out, lse = _joined(s["q"].float().view(n, H, -1, D), [(k, v, seen[:, None, None, :])], D ** -0.5)
    return {"out": out.reshape(n, -1, D).to(s["q"].dtype), "lse": lse.reshape(n, -1)}


def _shared_plain(case, s):
    common, n, _ = _group_plan(case)
    H, D, P, per = case["kv_heads"], case["dim"], case["page"], case["per"]
    G, table, length = case["q_heads"] // H, s["block_table"].long(), s["kv_len"].long()
    out = torch.empty(n, H, G, D, device="cuda")
    lse = torch.empty(n, H, G, device="cuda")
    q = s["q"].float().view(n, H, G, D)
    spans = [(g * per, (g + 1) * per, int(common[g])) for g in range(case["groups"])]
    if case["alone"]:
        spans.append((n - case["alone"], n, 0))
    for r0, r1, T in spans:
        R = r1 - r0
        # the requests' own tokens
        at = T + torch.arange(case["own"], device="cuda")[None, :].expand(R, -1)
        seen = at < length[r0:r1, None]
        page = table[r0:r1].gather(1, torch.where(seen, at // P, 0)).clamp(min=0)
        k, v = (_picked(case, s, x, page, at % P) for x in ("k", "v"))                  # [R, H, own, D]
        score = torch.matmul(q[r0:r1], k.transpose(2, 3)) * D ** -0.5                   # [R, H, G, own]
        score = torch.where(seen[:, None, None, :], score, -math.inf)
        top = score.amax(-1, keepdim=True)
        if T:
            # what they share, every request's rows in one product
            t = torch.arange(T, device="cuda")
            pk, pv = (_picked(case, s, x, table[r0, t // P].clamp(min=0), t % P) for x in ("k", "v"))
            rows = q[r0:r1].permute(1, 0, 2, 3).reshape(H, R * G, D)
            first = torch.matmul(rows, pk.transpose(1, 2)) * D ** -0.5
            first = first.view(H, R, G, T).permute(1, 0, 2, 3)                           # [R, H, G, T]
            first = torch.where((length[r0:r1] > 0)[:, None, None, None], first, -math.inf)
            top = torch.maximum(top, first.amax(-1, keepdim=True))
        ref = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(score - ref)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, torch.where(seen[:, None, :, None], v, 0.0))
        if T:
            p = torch.exp(first - ref)
            total = total + p.sum(-1, keepdim=True)
            p = p.permute(1, 0, 2, 3).reshape(H, R * G, T)
            o = o + torch.matmul(p, pv).view(H, R, G, D).permute(1, 0, 2, 3)
        out[r0:r1] = o / torch.where(total == 0, 1.0, total)
        lse[r0:r1] = (ref + torch.log(total))[..., 0]
    return {"out": out.view(n, -1, D).to(s["q"].dtype), "lse": lse.view(n, -1)}


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
    half, at = case["rot"] // 2, s["positions"].long()
    cos, sin = s["cos_sin"][at, :half], s["cos_sin"][at, half:]
    dt, pages, page = s["q"].dtype, s["k_pool"].shape[0] - 1, case["page"]
    slot = s["slot_map"].long()
    where = torch.where(slot >= 0, slot // page, pages), torch.where(slot >= 0, slot % page, 0)

    def normed(x, w):
        x = x.float()
        if case["layer"]:
            x = x - x.mean(-1, keepdim=True)
        return _turned(case, x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w, cos, sin).to(dt)

    for name, x in (("k_pool", normed(s["k"], s["k_w"])), ("v_pool", s["v"])):
        if case["token_major"]:
            s[name][where[0], where[1]] = x
        else:
            s[name][where[0], :, where[1]] = x
    return {"q": normed(s["q"], s["q_w"]), "k": s["k_pool"][:-1], "v": s["v_pool"][:-1]}


def _fork_plain(case, s):
    P, table, old = case["page"], s["table_in"].long(), s["len_in"].long()
    (n_in, cols), n = table.shape, s["source"].numel()
    pages = s["extra"].numel()
    dump = pages                                   # counted and thrown away
    source = s["source"].long()
    new = torch.where(source >= 0, torch.minimum(s["len_new"].long(), old[source]), 0)
    full, rest = new // P, new % P
    col = torch.arange(cols, device="cuda")[None, :]
    rows = table[source]                           # (source -1: the last row, of which nothing is taken)
    # owners beyond the first: one less for every page of the old rows, one more for
    # every page that a new row takes whole
    extra = torch.cat([s["extra"], s["extra"].new_zeros(1)])
    lost = torch.where(col < (old + P - 1)[:, None] // P, table, dump)
    kept = torch.where(col < full[:, None], rows, dump)
    extra.index_add_(0, lost.view(-1), extra.new_full((lost.numel(),), -1))
    extra.index_add_(0, kept.view(-1), extra.new_full((kept.numel(),), 1))
    extra[dump] = 0
    # a last page in part goes to the first row that wants it where nobody holds it,
    # and is copied for the others
    at = torch.arange(n, device="cuda")
    last = torch.where(rest > 0, rows.gather(1, full.clamp(max=cols - 1)[:, None])[:, 0], dump)
    wants = (rest > 0) & (extra[last] < 0)
    first = torch.full((pages + 1,), n, dtype=torch.long, device="cuda")
    first.scatter_reduce_(0, torch.where(wants, last, dump), at, "amin")
    first[dump] = n
    stays = wants & (first[last] == at)
    extra = torch.where(first < n, 0, extra)
    # pages without owners go on top of the list, by number; copies are taken from its top
    gone = extra[:pages] < 0
    rank = gone.cumsum(0) - gone.long()
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    start = s["free_in"].long()
    place = torch.where(gone, start + rank, pages).clamp(max=pages)
    number = torch.arange(pages, dtype=torch.int32, device="cuda")
    free[place] = number
    left = start + gone.sum()
    copies = (rest > 0) & ~stays
    nth = copies.cumsum(0) - copies.long()
    given = copies & (nth < left)
    page_to = torch.where(given, free[torch.where(given, left - 1 - nth, pages)].long(), -1)
    left = left - given.sum()
    extra = torch.where(extra < 0, 0, extra)[:pages]
    above = torch.arange(pages, device="cuda") >= left
    s["free"].copy_(torch.where(above, s["free"], free[:pages]))
    s["extra"].copy_(extra)
    # the new rows; a row that got no page for its last tokens ends at its full ones
    has_last = stays | given
    last_page = torch.where(stays, last, page_to)
    out = torch.where(col < full[:, None], rows, s["table_out"].long())
    out = torch.where((col == full[:, None]) & has_last[:, None], last_page[:, None], out)
    s["table_out"].copy_(out)
    s["len_out"].copy_(torch.where(has_last, new, full * P))
    s["free_out"].copy_(left)
    s["copy_from"].copy_(torch.where(given, last, -1))
    s["copy_to"].copy_(page_to)
    s["copy_tokens"].copy_(torch.where(given, rest, 0))
    # the copied pages' tokens, in every layer's pools
    src, dst = torch.where(given, last, dump), torch.where(given, page_to, dump)
    token = torch.arange(P, device="cuda")
    token = token[None, :, None, None] if case["token_major"] else token[None, None, :, None]
    for pool in (*s["k"], *s["v"]):
        pool[dst] = torch.where(token < torch.where(given, rest, 0)[:, None, None, None], pool[src], pool[dst])
    return _fork_outputs(s)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = _SIZE[case["kind"]]
    io = 4 if case["kind"] == "fp32" else 2
    if case["op"] == "sinks":
        lens = _lengths(case["n"], case["lo"], case["hi"], case["empty"])
        seen = np.minimum(lens, case["window"] + np.minimum(case["sinks"], np.maximum(lens - case["window"], 0)))
        rows = case["n"] * case["q_heads"]
        return {"bytes": int(seen.sum()) * 2 * case["kv_heads"] * case["dim"] * size
                + rows * (case["dim"] * 2 * io + 4) + 4 * int(_ceil(seen, case["page"]).sum()) + 4 * case["n"],
                "flops": 4 * int(seen.sum()) * case["q_heads"] * case["dim"]}
    if case["op"] == "shared":
        common, n, own_len = _group_plan(case)
        idle = len(range(1, n, case["empty"])) if case["empty"] else 0
        own_tokens = int(own_len.sum()) * (n - idle) // n
        each = int(common.sum()) * case["per"] * (n - idle) // n
        rows = n * case["q_heads"]
        return {"bytes": (int(common.sum()) + own_tokens) * 2 * case["kv_heads"] * case["dim"] * size
                + rows * (case["dim"] * 2 * io + 4) + 4 * (int(common.sum()) + own_tokens) // case["page"] + 8 * n,
                "flops": 4 * (each + own_tokens) * case["q_heads"] * case["dim"]}
    if case["op"] == "append":
        n, kept = case["n"], case["n"] - case["pad"]
        heads = case["q_heads"] * n + 2 * case["kv_heads"] * kept
        normed = case["q_heads"] * n + case["kv_heads"] * kept
        return {"bytes": 2 * heads * case["dim"] * io + 8 * n + min(n, 32768) * case["rot"] * 4 + 8 * case["dim"],
                "flops": normed * (3 * case["rot"] + 4 * case["dim"])}
    P, width, n = case["page"], case["width"], case["prompts"] * case["width"]
    rows_in = case["prompts"] if case["samples"] else n
    mean = int(_lengths(case["prompts"], case["lo"], case["hi"]).mean()) + (0 if case["samples"] else case["own"] // 2)
    copied = max(1, n - rows_in // 2) if case["samples"] else max(1, n // 3)
    if P == 1:
        copied = 0
    token = 4 * case["kv_heads"] * case["dim"] * size * case["layers"]       # keys and values, read and written
    return {"bytes": 4 * (rows_in + n) * _ceil(mean, P) + 24 * n + copied * (P // 2) * token,
            "flops": 2 * (rows_in + n) * _ceil(mean, P) + 8 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits, one request or row at a time where the plain
# form works on whole batches
# --------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "fork":
        return None         # whole numbers and copies: the outputs have to be equal as they are
    s = _inputs(case, seed)
    return _append_exact(case, s) if case["op"] == "append" else _attention_exact(case, s)


def _attention_exact(case, s):
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    n, G = s["q"].shape[0], case["q_heads"] // H
    out = torch.zeros(n, case["q_heads"], D, dtype=torch.float64, device="cuda")
    lse = torch.full((n, case["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")
    table, one = s["block_table"].cpu().numpy(), [1.0] * H
    ks = one if s["k_scale"] is None else s["k_scale"].tolist()
    vs = one if s["v_scale"] is None else s["v_scale"].tolist()
    bits = (lambda x: x.view(torch.uint8)) if case["kind"] == "fp8" else (lambda x: x)
    for r, length in enumerate(s["kv_len"].tolist()):
        t = np.arange(length)
        if case["op"] == "sinks":
            t = t[(t < case["sinks"]) | (t >= length - case["window"])]
        if not len(t):
            continue
        page, off = torch.from_numpy(table[r, t // P].astype(np.int64)).cuda(), torch.from_numpy(t % P).cuda()
        for h in range(H):
            pick = (lambda x: x[page, off, h]) if case["token_major"] else (lambda x: x[page, h, off])
            k = pick(bits(s["k"])).view(s["k"].dtype).to(torch.float64) * ks[h]
            v = pick(bits(s["v"])).view(s["v"].dtype).to(torch.float64) * vs[h]
            a = (s["q"][r, h * G:(h + 1) * G].double() @ k.T) / math.sqrt(D)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(a, 1)
            out[r, h * G:(h + 1) * G] = torch.softmax(a, 1) @ v
    return {"out": out, "lse": lse}


def _append_exact(case, s):
    pool = {x: s[x][:-1].double() for x in ("k_pool", "v_pool")}
    cos_sin, pos, half = s["cos_sin"].double(), s["positions"].long(), case["rot"] // 2
    ready = {}
    for name in ("q", "k"):
        x = s[name].double()
        if case["layer"]:
            var, mean = torch.var_mean(x, dim=2, correction=0, keepdim=True)
            x = (x - mean) / torch.sqrt(var + 1e-6)
        else:
            x = x / torch.sqrt((x * x).sum(2, keepdim=True) / case["dim"] + 1e-6)
        ready[name] = x * s[name + "_w"].double()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.complex(cos_sin[pos, i], cos_sin[pos, half + i])[:, None]
        for x in ready.values():
            w = torch.complex(x[:, :, a].clone(), x[:, :, b].clone()) * z
            x[:, :, a], x[:, :, b] = w.real, w.imag
    kept = torch.nonzero(s["slot_map"] >= 0)[:, 0]
    slot = s["slot_map"][kept].long()
    page, off = slot // case["page"], slot % case["page"]
    for name, x in (("k_pool", ready["k"]), ("v_pool", s["v"].double())):
        if case["token_major"]:
            pool[name][page, off] = x[kept]
        else:
            pool[name][page, :, off] = x[kept]
    return {"q": ready["q"], "k": pool["k_pool"], "v": pool["v_pool"]}
