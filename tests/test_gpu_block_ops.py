"""The paged cache, rotary append, one-token attention and residual norm on the
GPU against their float64 definitions (``oracle/block_ops.py``).

Tolerances.  u = 2^-24 is half a 32-bit step, h = 2^-9 half a bf16 step
(relative).  A bf16 output may be off by its own rounding, h |ref|, and by one
step more where the 32-bit value lies at a rounding boundary: 2 h |ref| in all.
  * attention: 32-bit sums of D products put a score off by at most (D + 2) u
    reach (reach = scale sum |q_i k_i|), a weight by twice that, the sums over L
    tokens and the exponentials by (L + 16) u, all times mass = sum p |v|; with
    a 16-bit cache the weights may also be rounded to bf16: h mass twice (the
    weights and their sum); an 8-bit cache may round the query relative to its
    largest element by 2^-20, which is inside the 16-bit allowance.
  * rotary: two products and a sum, 3 u of |a| + |b|.
  * norms: sums of d squares (d + 8) u relative, for either norm.
"""
import numpy as np
import pytest

from oracle import block_ops as OB

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, HB = 2.0 ** -24, 2.0 ** -9
PAGES = 10     # SCUTE_ERR_PAGES


@pytest.fixture(scope="module")
def scute(gpu_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return gpu_lib


@pytest.fixture(scope="module")
def contexts(scute):
    c = {k: scute.Context(dtype=k, max_tokens=64, max_adapters=4, max_layers=1) for k in ("bf16", "fp32")}
    yield c
    for x in c.values():
        x.close()


def ctx_of(contexts, kind):
    return contexts["fp32" if kind == "fp32" else "bf16"]


DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def make_cache(scute, g, lens, H, D, page, kind, token_major, spare=3, scales=False):
    """(KvCache, keys and values of every request in 64 bits)."""
    lens = np.asarray(lens)
    need = -(-lens // page)
    total = int(need.sum()) + spare
    order = g.permutation(total)
    cols = max(1, int(need.max(initial=0)))
    table = np.full((len(lens), cols), -1, np.int32)
    k, v = (torch.from_numpy(g.standard_normal((total, page, H, D), dtype=np.float32)) for _ in range(2))
    at = 0
    for r, c in enumerate(need):
        table[r, :c] = order[at:at + c]
        at += c
        if lens[r] % page:       # what lies behind the last token is no number
            k[table[r, c - 1], lens[r] % page:] = float("nan")
            v[table[r, c - 1], lens[r] % page:] = float("nan")
    for p in order[at:]:
        k[p] = float("nan")
        v[p] = float("inf")
    ks = vs = None
    if scales:
        ks, vs = (torch.from_numpy((0.5 + g.random(H)).astype(np.float32)).cuda() for _ in range(2))
    k, v = k.to(DT[kind]), v.to(DT[kind])
    kk, vv = f64(k), f64(v)
    if scales:
        kk, vv = kk * f64(ks)[None, None, :, None], vv * f64(vs)[None, None, :, None]
    tokens = [(kk[table[r, :need[r]]].reshape(-1, H, D)[:lens[r]], vv[table[r, :need[r]]].reshape(-1, H, D)[:lens[r]])
              for r in range(len(lens))]
    if not token_major:
        k, v = (x.view(torch.uint8) if kind == "fp8" else x for x in (k, v))
        k, v = (x.permute(0, 2, 1, 3).contiguous().view(DT[kind]) for x in (k, v))
    cache = scute.KvCache(k.cuda(), v.cuda(), i32(table), token_major=token_major, k_scale=ks, v_scale=vs)
    return cache, tokens


def check_attend(out, lse, q, tokens, kind, group, window=0, softcap=0.0, scale=None):
    n, heads, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, lse, q = f64(out).reshape(n, heads, D), f64(lse), f64(q)
    for r in range(n):
        k, v = tokens[r]
        first = max(0, len(k) - window) if window else 0
        for h in range(heads // group):
            rows = slice(h * group, (h + 1) * group)
            ref, ref_lse, mass, reach = OB.attend(q[r, rows], k[first:, h], v[first:, h], scale, softcap)
            soft = U * (2 * reach[:, None] * (D + 2) + len(k) + 16)
            tol = mass * (soft + (0 if kind == "fp32" else 2 * HB)) + (0 if kind == "fp32" else 2 * HB) * np.abs(ref)
            err = np.abs(out[r, rows] - ref)
            assert np.all(err <= tol + 1e-30), (r, h, float((err / (tol + 1e-30)).max()))
            if len(k) - first == 0:
                assert np.all(out[r, rows] == 0) and np.all(lse[r, rows] == -np.inf)
            else:
                more = 0 if kind != "fp8" else 2.0 ** -19 * reach
                tol = U * (reach * (D + 2) + np.abs(ref_lse) + len(k) + 16) + more
                assert np.all(np.abs(lse[r, rows] - ref_lse) <= tol), (r, h)


EDGES = [0, 1, 2, 7, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500]


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("H,group,D,page,token_major", [
    (2, 4, 128, 16, False), (2, 4, 128, 16, True), (1, 1, 64, 1, False), (3, 2, 80, 24, True), (2, 7, 96, 8, False),
    (1, 8, 128, 64, True), (2, 9, 128, 33, False), (1, 16, 64, 16, False), (1, 19, 128, 16, False),
    (2, 5, 256, 16, False), (1, 12, 256, 40, True), (2, 3, 192, 32, False), (1, 2, 16, 5, False),
    (1, 40, 48, 16, True)])
def test_attention_heads_pages_and_lengths(scute, contexts, kind, H, group, D, page, token_major):
    g = np.random.default_rng(H * 1000 + group * 10 + D)
    cache, tokens = make_cache(scute, g, EDGES, H, D, page, kind, token_major, scales=kind == "fp8")
    q = torch.from_numpy(g.standard_normal((len(EDGES), H * group, D), dtype=np.float32) * 1.5)
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32(EDGES), out, lse=lse)
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, tokens, kind, group)
    again, lse2 = torch.empty_like(out), torch.empty_like(lse)
    ctx.paged_attention(cache, q, i32(EDGES), again, lse=lse2)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # the same bits


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("window,softcap,scale", [(1, 0.0, 0.0), (20, 0.0, 0.1), (64, 5.0, 0.0), (0, 30.0, -0.2),
                                                  (100000, 0.0, 0.0)])
def test_attention_window_softcap_scale(scute, contexts, kind, window, softcap, scale):
    g = np.random.default_rng(5)
    cache, tokens = make_cache(scute, g, EDGES, 2, 64, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((len(EDGES), 6, 64), dtype=np.float32) * 2)
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32(EDGES), out, lse=lse, window=window, softcap=softcap, scale=scale)
    check_attend(out, lse, q, tokens, kind, 3, window, softcap, scale or None)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("lens", [[20000], [5000, 3, 0, 9001], [64] * 300, [0] * 40, [1]])
def test_attention_split_over_the_gpu(scute, contexts, kind, lens):
    """One long request, uneven ones, more requests than SMs, none at all."""
    g = np.random.default_rng(len(lens))
    cache, tokens = make_cache(scute, g, lens, 2, 128, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((len(lens), 8, 128), dtype=np.float32))
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    for _ in range(3):       # counters are back at zero after each call
        out.fill_(float("nan"))
        ctx.paged_attention(cache, q, i32(lens), out, lse=lse)
        check_attend(out, lse, q, tokens, kind, 4)
    assert ctx.sync_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
def test_attention_most_requests(scute, contexts, kind):
    """As many requests as a call takes (fewer CTAs fit an SM then), mostly short or empty."""
    g = np.random.default_rng(16384)
    lens = g.integers(0, 4, 16384)
    lens[[0, 5000, 16383]] = 900, 3000, 40
    cache, tokens = make_cache(scute, g, lens, 1, 64, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((len(lens), 2, 64), dtype=np.float32))
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32(lens), out, lse=lse)
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, tokens, kind, 2)


def test_attention_large_scores_and_one_token_dominates(scute, contexts):
    """Scores of +-2000 (nothing overflows, the maximum moves from tile to tile)
    and values whose weights all vanish but one."""
    g = np.random.default_rng(3)
    cache, tokens = make_cache(scute, g, [700], 1, 64, 16, "bf16", False)
    q = torch.from_numpy(g.standard_normal((1, 4, 64), dtype=np.float32) * 600).cuda().bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    contexts["bf16"].paged_attention(cache, q, i32([700]), out, lse=lse)
    check_attend(out, lse, q, tokens, "bf16", 4)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
def test_attention_long_tail_of_small_weights(scute, contexts, kind):
    """One token 2^26 times as heavy as each of 20000 others, whose sum still counts
    (many requests on the same pages, so that a warp takes most of a row)."""
    n, L, D = 700, 20000, 64
    k, v = torch.zeros(L // 16, 1, 16, D), torch.ones(L // 16, 1, 16, D)
    k[0, 0, 0], v[0, 0, 0] = 1.5, 0.0
    cache = scute.KvCache(k.to(DT[kind]).cuda(), v.to(DT[kind]).cuda(), i32(np.tile(np.arange(L // 16), (n, 1))))
    q = torch.full((n, 1, D), 1.5, device="cuda").to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty(n, 1, device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32([L] * n), out, lse=lse)
    assert ctx.sync_status() == 0
    one = f64(k).reshape(-1, 1, D), f64(v).reshape(-1, 1, D)
    check_attend(out, lse, q, [one] * n, kind, 1)


def test_attention_strided_in_place_on_another_stream_without_lse(scute, contexts):
    g = np.random.default_rng(11)
    lens = [40, 0, 333]
    cache, tokens = make_cache(scute, g, lens, 2, 128, 16, "bf16", False)
    wide = torch.from_numpy(g.standard_normal((3, 12 + 8 + 2, 128), dtype=np.float32)).cuda().bfloat16()
    q = wide[:, 4:12]                       # a slice of wider rows, and also the output
    q0, rest = q.clone(), wide.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kv_len = i32(lens)
    with torch.cuda.stream(s):
        contexts["bf16"].paged_attention(cache, q, kv_len, q)
    s.synchronize()
    lse = torch.empty(3, 8, device="cuda")
    contexts["bf16"].paged_attention(cache, q0, kv_len, torch.empty_like(q0), lse=lse)
    check_attend(q, lse, q0, tokens, "bf16", 4)
    rest[:, 4:12] = q
    assert torch.equal(rest, wide)


def test_attention_graph_replay_with_other_lengths(scute, contexts):
    g = np.random.default_rng(12)
    full = [300, 900, 64, 5]
    cache, tokens = make_cache(scute, g, full, 2, 128, 16, "bf16", False)
    q = torch.from_numpy(g.standard_normal((4, 8, 128), dtype=np.float32)).cuda().bfloat16()
    out, lse, kv_len = torch.empty_like(q), torch.empty(4, 8, device="cuda"), i32(full)
    ctx = contexts["bf16"]
    ctx.paged_attention(cache, q, kv_len, out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.paged_attention(cache, q, kv_len, out, lse=lse)
    for lens in ([300, 900, 64, 5], [1, 0, 33, 5], [299, 17, 0, 1]):
        kv_len.copy_(i32(lens))
        graph.replay()
        check_attend(out, lse, q, [(k[:n], v[:n]) for (k, v), n in zip(tokens, lens)], "bf16", 4)
    torch.cuda.synchronize()
    assert ctx.sync_status() == 0


def test_attention_pages_and_lengths_out_of_range_are_recorded(scute, contexts):
    """A length beyond the table counts as the table's; tokens of a page outside
    the pool are left out; the status word says so once."""
    g = np.random.default_rng(13)
    lens = [64, 48]
    cache, tokens = make_cache(scute, g, lens, 1, 64, 16, "bf16", False)
    table = cache.tensors[2]
    table[1, 1] = 10 ** 6
    table[1, 3] = 0
    q = torch.from_numpy(g.standard_normal((2, 4, 64), dtype=np.float32)).cuda().bfloat16()
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    ctx = contexts["bf16"]
    ctx.paged_attention(cache, q, i32([10 ** 9, 48]), out, lse=lse)
    assert ctx.sync_status() == PAGES and ctx.sync_status() == 0
    k, v = tokens[1]
    left = [tokens[0], (np.delete(k, slice(16, 32), 0), np.delete(v, slice(16, 32), 0))]
    check_attend(out, lse, q, left, "bf16", 4)
    ctx.paged_attention(cache, q, i32([-5, 0]), out, lse=lse)
    assert ctx.sync_status() == PAGES
    assert not out.any() and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_attention_offsets_beyond_32_bits(scute, contexts, kind):
    """Pages whose elements lie beyond 2^31 (and bytes beyond 2^32)."""
    g = np.random.default_rng(14)
    page, H, D = 16, 8, 128
    far = (5 << 30) // (page * H * D * (2 if kind == "bf16" else 1))
    k, v = (torch.zeros((far + 3, H, page, D), dtype=torch.uint8 if kind == "fp8" else DT[kind], device="cuda")
            .view(DT[kind]) for _ in range(2))
    ids = [far + 2, 0, far]
    for pool in (k, v):
        for p in ids:
            pool[p].copy_(torch.from_numpy(g.standard_normal((H, page, D), dtype=np.float32)).cuda())
    tokens = [tuple(f64(torch.cat([x[p].float().permute(1, 0, 2) for p in ids]))[:41] for x in (k, v))]
    cache = scute.KvCache(k, v, i32([ids]))
    q = torch.from_numpy(g.standard_normal((1, 32, D), dtype=np.float32)).cuda().bfloat16()
    out, lse = torch.empty_like(q), torch.empty(1, 32, device="cuda")
    contexts["bf16"].paged_attention(cache, q, i32([41]), out, lse=lse)
    check_attend(out, lse, q, tokens, kind, 4)


# ---------------------------------------------------------------- pages and slots
def run_resize(ctx, len_in, len_new, table, page, free, max_new, in_place=False, n_free_max=None):
    n = len(len_in)
    pool = np.full(n_free_max if n_free_max is not None else table.size + len(free) + 8, -7, np.int32)
    pool[:len(free)] = free
    t = {"len_in": i32(len_in), "len_new": i32(len_new), "table": i32(table), "free": i32(pool),
         "free_in": i32([len(free)]), "cu": i32(np.full(n + 1, -9)), "slot": i32(np.full(max_new, -9)),
         "pos": i32(np.full(max_new, -9)), "req": i32(np.full(max_new, -9))}
    len_out = t["len_in"] if in_place else i32(np.full(n, -9))
    free_out = t["free_in"] if in_place else i32([-9])
    ctx.kv_resize(t["len_in"], t["len_new"], t["table"], page, t["free"], t["free_in"], free_out, len_out, t["cu"],
                  t["slot"], t["pos"], t["req"])
    status = ctx.sync_status()
    c = lambda x: x.cpu().numpy()  # noqa: E731
    return {"table": c(t["table"]), "free": list(c(t["free"])[:int(free_out.item())]), "len_out": c(len_out),
            "cu_new": c(t["cu"]), "slot_map": c(t["slot"]), "positions": c(t["pos"]), "token_req": c(t["req"]),
            "above": c(t["free"])[int(free_out.item()):], "status": status}


def same_resize(got, ref):
    for k in ("len_out", "cu_new", "slot_map", "positions", "token_req", "table"):
        assert np.array_equal(got[k], ref[k]), k
    assert got["free"] == ref["free"]
    assert got["status"] == (0 if ref["ok"] else PAGES)


def draw_resize(g, n, hi, page, spare, grow=40):
    old = g.integers(0, hi + 1, n)
    new = np.where(g.random(n) < 0.3, g.integers(0, hi + 1, n), np.minimum(old + g.integers(0, grow, n), hi))
    new[g.random(n) < 0.15] = 0
    cols = max(1, -(-hi // page))
    need = -(-old // page)
    order = g.permutation(int(need.sum()) + spare)
    table = np.full((n, cols), -1, np.int32)
    table[np.arange(cols)[None, :] < need[:, None]] = order[:int(need.sum())]
    return old, new, table, list(order[int(need.sum()):])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,hi,page,spare,room", [
    (1, 1, 1, 1, 4), (1, 100, 16, 10, 128), (7, 64, 16, 50, 400), (64, 300, 16, 2000, 20000), (64, 300, 16, 20, 20000),
    (33, 50, 7, 0, 900), (200, 90, 8, 60, 300), (513, 40, 16, 900, 30000), (3000, 30, 4, 9000, 100000),
    (5000, 12, 4, 4000, 40000)])
def test_resize_matches_the_definition(scute, contexts, n, hi, page, spare, room, in_place):
    g = np.random.default_rng(n + page)
    for _ in range(2):
        old, new, table, free = draw_resize(g, n, hi, page, spare)
        ref = OB.resize(old, new, table, page, free, room)
        same_resize(run_resize(contexts["bf16"], old, new, table, page, free, room, in_place), ref)


def test_resize_edges(scute, contexts):
    ctx = contexts["bf16"]
    table = np.full((3, 4), -1, np.int32)
    table[0, :2] = [5, 9]
    # nothing asked; no rows; no requests
    same_resize(run_resize(ctx, [20, 0, 0], [20, 0, 0], table, 16, [1, 2], 5), OB.resize([20, 0, 0], [20, 0, 0], table, 16, [1, 2], 5))
    same_resize(run_resize(ctx, [20, 0, 0], [0, 0, 0], table, 16, [], 0), OB.resize([20, 0, 0], [0, 0, 0], table, 16, [], 0))
    got = run_resize(ctx, [], [], np.zeros((0, 4), np.int32), 16, [3, 4], 3)
    assert got["free"] == [3, 4] and list(got["cu_new"]) == [0] and list(got["slot_map"]) == [-1] * 3
    # growth to the very end of the row, and a page handed from one request to another
    for new in ([64, 0, 0], [0, 33, 0], [0, 64, 64], [20, 16, 16]):
        ref = OB.resize([20, 0, 0], new, table, 16, [1, 2], 200)
        same_resize(run_resize(ctx, [20, 0, 0], new, table, 16, [1, 2], 200), ref)
    # what stood above the count stays
    got = run_resize(ctx, [20, 0, 0], [33, 0, 0], table, 16, [1, 2], 20)
    assert list(got["above"][:2]) == [2, -7]


def test_resize_refusals_in_order(scute, contexts):
    """Too few pages: the second grower is refused, the third too although one
    page would do for it, the fourth grows inside its last page.  Too few rows:
    the first that passes them and the ones after it."""
    ctx, page = contexts["bf16"], 16
    table = np.full((5, 4), -1, np.int32)
    table[3, 0] = 40
    old, new = [0, 0, 0, 3, 0], [16, 33, 1, 9, 0]
    ref = OB.resize(old, new, table, page, [7, 8], 100)
    assert list(ref["len_out"]) == [16, 0, 0, 9, 0] and not ref["ok"]
    same_resize(run_resize(ctx, old, new, table, page, [7, 8], 100), ref)
    ref = OB.resize(old, new, table, page, list(range(20)), 50)
    assert list(ref["len_out"]) == [16, 33, 1, 3, 0]
    same_resize(run_resize(ctx, old, new, table, page, list(range(20)), 50), ref)
    # lengths outside the row
    old, new = [100, -3, 0, 3, 5], [10, 5, 65, -1, 5]
    table[0] = [1, 2, 3, 4]
    table[4, 0] = 9
    same_resize(run_resize(ctx, old, new, table, page, [7, 8], 100), OB.resize(old, new, table, page, [7, 8], 100))


def test_resize_free_list_too_short_is_recorded(scute, contexts):
    table = np.array([[5, 9]], np.int32)
    got = run_resize(contexts["bf16"], [32], [0], table, 16, [1], 1, n_free_max=2)
    assert got["status"] == PAGES and got["free"] == [1, 5]


def test_resize_decode_loop_in_a_graph(scute, contexts):
    """A captured step (lengths + 1, in place) replayed: positions move on and
    every request's pages stay its own."""
    ctx, n, page, cols = contexts["bf16"], 6, 4, 8
    t = {k: i32(v) for k, v in dict(len=[0] * n, want=[1] * n, table=np.full((n, cols), -1), free=np.arange(n * cols),
                                    count=[n * cols], cu=[0] * (n + 1), slot=[0] * n, pos=[0] * n, req=[0] * n).items()}

    def step():
        torch.add(t["len"], 1, out=t["want"])
        ctx.kv_resize(t["len"], t["want"], t["table"], page, t["free"], t["count"], t["count"], t["len"], t["cu"],
                      t["slot"], t["pos"], t["req"])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = set(t["slot"].tolist())
    for i in range(1, page * cols):
        graph.replay()
        slots = t["slot"].tolist()
        assert t["pos"].tolist() == [i] * n and t["req"].tolist() == list(range(n))
        assert len(set(slots)) == n and not seen & set(slots)
        seen |= set(slots)
    assert t["count"].item() == 0 and ctx.sync_status() == 0
    graph.replay()                               # rows are full: nothing grows
    assert ctx.sync_status() == PAGES and t["len"].tolist() == [page * cols] * n


# ---------------------------------------------------------------- rotary positions and the cache write
def rope_inputs(g, n, places, rot, axes):
    inv = 10000.0 ** (-np.arange(0, rot, 2) / rot)
    ang = np.arange(places)[:, None] * inv[None]
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    pos = g.integers(0, places, (axes, n))
    cut = sorted(g.integers(0, rot // 2 + 1, axes - 1))
    sections = np.diff([0] + cut + [rot // 2]).tolist()
    return table, pos, sections


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("n,H,qh,D,page,rot,axes,inter,token_major,skew", [
    (1, 1, 1, 16, 1, 16, 1, False, False, 0), (5, 2, 8, 128, 16, 128, 1, False, False, 0),
    (33, 2, 6, 128, 16, 64, 2, False, True, 0), (64, 8, 32, 128, 16, 128, 3, False, False, 0),
    (17, 1, 7, 80, 24, 80, 1, True, True, 0), (9, 3, 3, 96, 8, 30, 2, False, False, 0),
    (9, 3, 3, 96, 8, 34, 4, True, False, 0), (20, 2, 4, 64, 16, 64, 1, False, False, 1),
    (20, 2, 4, 256, 16, 256, 3, True, False, 3), (300, 2, 4, 128, 64, 126, 1, False, True, 0),
    (4, 2, 2, 48, 16, 2, 1, False, False, 0)])
def test_append_turns_and_writes(scute, contexts, kind, n, H, qh, D, page, rot, axes, inter, token_major, skew):
    g = np.random.default_rng(n * 7 + D)
    io = DT["fp32" if kind == "fp32" else "bf16"]
    pages = -(-n // page) + 2
    slots = g.permutation(pages * page)[:n]
    if n > 4:
        slots[[1, n - 1]] = -1
    shape = (pages, page, H, D) if token_major else (pages, H, page, D)
    pools = [torch.full(shape, 3.0, device="cuda").to(DT[kind]) for _ in range(2)]
    scale = [torch.from_numpy((0.2 + g.random(H)).astype(np.float32)).cuda() if kind == "fp8" else None for _ in range(2)]
    cache = scute.KvCache(*pools, token_major=token_major, k_scale=scale[0], v_scale=scale[1])
    # rows of one wider buffer; with skew they are not 16-byte aligned
    wide = torch.from_numpy(g.standard_normal((n, (qh + 2 * H) * D + skew), dtype=np.float32)).cuda().to(io)
    q, k, v = (wide[:, skew + a * D:skew + b * D] for a, b in ((0, qh), (qh, qh + H), (qh + H, qh + 2 * H)))
    table, pos, sections = rope_inputs(g, n, 4000, rot, axes)
    rope = scute.Rope(table, i32(pos[0] if axes == 1 else pos), sections=sections, interleaved=inter)
    q_out = torch.full((n, qh * D), float("nan"), device="cuda").to(io)
    ctx = ctx_of(contexts, kind)
    ctx.kv_append(cache, i32(slots), k, v, q=q, q_out=q_out, rope=rope)
    assert ctx.sync_status() == 0
    tab, axis = f64(table), np.repeat(np.arange(axes), sections)
    got = [f64(x) if token_major else f64(x).transpose(0, 2, 1, 3) for x in pools]
    got = [x.reshape(pages * page, H, D) for x in got]
    touched = np.zeros(pages * page, bool)
    rel = 0 if kind == "fp32" else 2 * HB
    for t in range(n):
        c = np.array([tab[pos[axis[i], t], i] for i in range(rot // 2)])
        s = np.array([tab[pos[axis[i], t], rot // 2 + i] for i in range(rot // 2)])

        def turn(x):
            a, b = (x[:, 0:rot:2], x[:, 1:rot:2]) if inter else (x[:, :rot // 2], x[:, rot // 2:rot])
            y, mag = x.copy(), np.abs(x)
            pairs = (a * c - b * s, b * c + a * s)
            for dst, val in ((y, pairs), (mag, (np.abs(a) + np.abs(b),) * 2)):
                if inter:
                    dst[:, 0:rot:2], dst[:, 1:rot:2] = val
                else:
                    dst[:, :rot // 2], dst[:, rot // 2:rot] = val
            return y, mag

        y, mag = turn(f64(q[t]).reshape(qh, D))
        assert np.all(np.abs(f64(q_out[t]).reshape(qh, D) - y) <= 3 * U * mag + rel * np.abs(y))
        if slots[t] < 0:
            continue
        touched[slots[t]] = True
        for i, (ref, mag) in enumerate((turn(f64(k[t]).reshape(H, D)), (f64(v[t]).reshape(H, D),) * 2)):
            have = got[i][slots[t]]
            if kind == "fp8":       # half a step of e4m3 (2^-4 relative, 2^-10 below 2^-6), either side of a boundary
                sc = f64(scale[i])[:, None]
                ref, mag = np.clip(ref / sc, -448, 448), mag / sc
                assert np.all(np.abs(have - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, 2.0 ** -10) * 1.001 + 4 * U * np.abs(mag))
            elif i == 1:
                assert np.array_equal(have, ref)
            else:
                assert np.all(np.abs(have - ref) <= 3 * U * mag + rel * np.abs(ref))
    for x in got:
        assert np.all(x[~touched] == 3.0)


def test_append_without_queries_or_positions_and_in_place(scute, contexts):
    g = np.random.default_rng(2)
    ctx = contexts["bf16"]
    k, v = (torch.from_numpy(g.standard_normal((6, 2, 64), dtype=np.float32)).cuda().bfloat16() for _ in range(2))
    pools = [torch.zeros(3, 2, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    cache = scute.KvCache(*pools)
    slots = [0, 3, 4, 11, -1, 7]
    ctx.kv_append(cache, i32(slots), k, v)
    for x, pool in ((k, pools[0]), (v, pools[1])):
        flat = pool.permute(0, 2, 1, 3).reshape(12, 2, 64)
        for t, s in enumerate(slots):
            if s >= 0:
                assert torch.equal(flat[s], x[t])
    table, pos, _ = rope_inputs(g, 6, 50, 64, 1)
    rope = scute.Rope(table, i32(pos[0]))
    q = torch.from_numpy(g.standard_normal((6, 4, 64), dtype=np.float32)).cuda().bfloat16()
    q_out = torch.empty_like(q)
    ctx.kv_append(cache, i32(slots), k, v, q=q, q_out=q_out, rope=rope)
    ctx.kv_append(cache, i32(slots), k, v, q=q, q_out=q, rope=rope)
    assert torch.equal(q, q_out)
    ctx.kv_append(cache, i32([]), k[:0], v[:0], q=q[:0], q_out=q[:0], rope=rope)
    assert ctx.sync_status() == 0


def test_append_slots_and_positions_out_of_range_are_recorded(scute, contexts):
    g = np.random.default_rng(4)
    ctx = contexts["bf16"]
    x = torch.from_numpy(g.standard_normal((3, 2, 64), dtype=np.float32)).cuda().bfloat16()
    pools = [torch.zeros(2, 2, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    cache = scute.KvCache(*pools)
    ctx.kv_append(cache, i32([8, 1, -2]), x, x)
    assert ctx.sync_status() == PAGES
    assert torch.equal(pools[1][0, :, 1], x[1]) and pools[1].ne(0).sum() <= 128
    table, _, _ = rope_inputs(g, 3, 10, 64, 1)
    q, near = torch.empty_like(x), torch.empty_like(x)
    ctx.kv_append(cache, i32([0, 1, 2]), x, x, q=x, q_out=q, rope=scute.Rope(table, i32([-4, 10, 5])))
    assert ctx.sync_status() == PAGES
    ctx.kv_append(cache, i32([0, 1, 2]), x, x, q=x, q_out=near, rope=scute.Rope(table, i32([0, 9, 5])))
    assert ctx.sync_status() == 0 and torch.equal(q, near)


def test_append_saturates_an_8_bit_cache(scute, contexts):
    x = torch.tensor([1e4, -1e4, 448.0, 500.0], device="cuda").repeat(16).view(1, 1, 64).bfloat16()
    pools = [torch.zeros(1, 1, 4, 64, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
    contexts["bf16"].kv_append(scute.KvCache(*pools), i32([2]), x, x)
    assert pools[0].float()[0, 0, 2, :4].tolist() == [448.0, -448.0, 448.0, 448.0]


def test_rope_table(scute, contexts):
    for rot, places, theta in ((2, 3, 10000.0), (126, 1000, 500000.0), (128, 70001, 10000.0)):
        out = torch.empty(places, rot, device="cuda")
        contexts["bf16"].rope_table(out, theta)
        ang = np.arange(places)[:, None] * (theta ** (-np.arange(0, rot, 2) / rot))[None]
        # the power's last bits times the largest position, then one rounding to 32 bits
        assert np.max(np.abs(f64(out) - np.concatenate([np.cos(ang), np.sin(ang)], 1))) <= U + places * 2.0 ** -50
    inv = torch.tensor([1.0, 0.25, 0.001], dtype=torch.float64, device="cuda")
    out = torch.empty(9, 6, device="cuda")
    contexts["fp32"].rope_table(out, inv_freq=inv)
    ang = np.arange(9)[:, None] * inv.cpu().numpy()[None]
    assert np.max(np.abs(f64(out) - np.concatenate([np.cos(ang), np.sin(ang)], 1))) <= U


# ---------------------------------------------------------------- norms
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d,post,pre,gate,layer,bias,res,res_out,skew", [
    (1, 1, True, True, None, False, False, True, True, 0), (3, 7, True, True, "vec", False, False, True, True, 0),
    (64, 4096, True, True, None, False, False, True, True, 0), (5, 4096, False, True, "rows", False, False, True, True, 0),
    (5, 1000, True, True, "vec", True, True, True, True, 0), (9, 2880, True, False, "rows", False, False, True, True, 0),
    (2, 14336, True, True, None, True, True, False, True, 0), (700, 256, False, True, None, False, False, True, False, 0),
    (3, 32768, True, True, "vec", False, False, True, True, 0), (4, 20000, True, True, None, True, True, True, True, 0),
    (33, 512, True, True, "rows", False, False, True, True, 1), (6, 8192, False, True, None, False, False, False, False, 3),
    (4, 257, False, True, None, True, False, True, True, 0), (300, 64, True, True, None, False, False, True, True, 0)])
def test_residual_norm(scute, contexts, kind, n, d, post, pre, gate, layer, bias, res, res_out, skew):
    g = np.random.default_rng(n + d)
    io = DT[kind]

    def rows(std=1.0):
        return torch.from_numpy(g.standard_normal((n, d + skew), dtype=np.float32) * np.float32(std)).cuda().to(io)[:, skew:]

    def vec(mean):
        return torch.from_numpy((mean + 0.2 * g.standard_normal(d)).astype(np.float32)).cuda()

    y, r = rows(0.7), rows(3.0) if res else None
    pw, pb = (vec(1.0), vec(0.0) if bias else None) if post else (None, None)
    nw, nb = (vec(1.0), vec(0.0) if bias else None) if pre else (None, None)
    gt = {None: None, "vec": vec(0.5), "rows": rows(0.5)}[gate]
    out = torch.full((n, d), float("nan"), device="cuda").to(io) if pre else None
    ro = torch.full((n, d), float("nan"), device="cuda").to(io) if res_out else None
    ctx = ctx_of(contexts, kind)
    ctx.residual_norm(y, out, residual=r, residual_out=ro, pre_w=nw, pre_b=nb, post_w=pw, post_b=pb, gate=gt,
                      scale=0.6, eps=1e-5, layer=layer)
    assert ctx.sync_status() == 0
    n64 = lambda t: None if t is None else f64(t)  # noqa: E731
    h, o = OB.residual_norm(f64(y), n64(r), (n64(pw), n64(pb)) if post else None, (n64(nw), n64(nb)) if pre else None,
                            n64(gt), 0.6, 1e-5, layer)
    rel = 0 if kind == "fp32" else 2 * HB
    t = np.abs(h) + np.abs(h - (0 if r is None else f64(r)))
    soft = U * (d + 8) * 2 + 8 * U
    # a layer norm's mean is off by d u of the values' size, which moves the centred value
    step = soft * (t + (np.abs(f64(y)).max(1, keepdims=True) * 4 if layer else 0))
    if ro is not None:
        assert np.all(np.abs(f64(ro) - h) <= step + rel * np.abs(h) + 1e-30)
    if pre:
        size = np.sqrt((h * h).mean(1, keepdims=True)) if not layer else h.std(1, keepdims=True)
        w = np.abs(n64(nw))
        tol = soft * np.abs(o) + w * (step + soft * np.abs(h)) / np.maximum(size, 1e-3) + (soft if layer else 0)
        assert np.all(np.abs(f64(out) - o) <= tol + rel * np.abs(o) + 1e-30)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("n,d,post,pre,gate,layer,bias", [
    (700, 480, True, True, "vec", False, False), (331, 2048, True, True, "rows", False, False),
    (1300, 4096, True, True, None, False, False), (1250, 4096, False, True, "vec", True, True),
    (1300, 5120, True, True, None, True, True), (2000, 1000, True, True, "rows", True, True),
    (320, 14336, True, True, "vec", False, False)])
def test_residual_norm_many_rows(scute, contexts, kind, n, d, post, pre, gate, layer, bias):
    """Several rows to a CTA: rows fetched ahead, factors held from row to row."""
    test_residual_norm(scute, contexts, kind, n, d, post, pre, gate, layer, bias, True, True, 0)


def test_residual_norm_in_place_strided_and_zero_rows(scute, contexts):
    g = np.random.default_rng(8)
    ctx = contexts["bf16"]
    wide = torch.from_numpy(g.standard_normal((5, 3, 128), dtype=np.float32)).cuda().bfloat16()
    wide[2] = 0
    y, r, keep = wide[:, 1], wide[:, 2], wide.clone()
    out, ro = torch.empty(5, 128, device="cuda", dtype=torch.bfloat16), torch.empty(5, 128, device="cuda", dtype=torch.bfloat16)
    ctx.residual_norm(y, out, residual=r, residual_out=ro)
    assert torch.isfinite(out.float()).all() and not out[2].any()
    ctx.residual_norm(y, y, residual=r, residual_out=r)             # over the inputs
    assert torch.equal(y, out) and torch.equal(r, ro) and torch.equal(wide[:, 0], keep[:, 0])
    ctx.residual_norm(y[:0], out[:0], residual=r[:0])


# ---------------------------------------------------------------- refusals
def refused(scute, code, f):
    with pytest.raises(scute.ScuteError) as e:
        f()
    assert e.value.code == code, e.value


def test_refusals(scute, contexts):
    """Every argument the host can see is refused before anything is launched."""
    ctx, f32 = contexts["bf16"], contexts["fp32"]
    before = ctx.launch_count()
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=torch.float32, device="cuda").to(t)  # noqa: E731
    cache = scute.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64), i32([[0, 1]]))
    q, lens = z(1, 4, 64), i32([3])
    out = torch.empty_like(q)
    A = lambda **kw: scute.scute_paged_attention(ctx.handle, **{**dict(  # noqa: E731
        cache=cache, q=q, q_stride=256, out=out, out_stride=256, lse=None, kv_len=lens, n_req=1, q_heads=4), **kw})
    for code, kw in [(1, dict(q=None)), (1, dict(out=None)), (1, dict(kv_len=None)), (1, dict(n_req=-1)),
                     (1, dict(n_req=16385)), (2, dict(q_heads=3)), (2, dict(q_heads=0)), (2, dict(q_stride=255)),
                     (2, dict(out_stride=260)), (1, dict(scale=float("nan"))), (1, dict(softcap=-1.0)),
                     (1, dict(softcap=float("inf"))), (1, dict(window=-1)), (1, dict(q=q.data_ptr() + 2)),
                     (1, dict(cache=scute.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64))))]:
        if "cache" in kw:
            kw["cache"].struct.table_cols = kw["cache"].struct.table_stride = 2
        refused(scute, code, lambda: A(**kw))

    def with_cache(**kw):
        c = scute.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64), i32([[0, 1]]))
        for k, v in kw.items():
            setattr(c.struct, k, v)
        return c

    for code, kw in [(1, dict(k=None)), (1, dict(v=None)), (3, dict(dtype=1)), (3, dict(dtype=7)), (2, dict(n_pages=0)),
                     (2, dict(page_size=0)), (2, dict(kv_heads=0)), (2, dict(n_pages=1 << 30)), (2, dict(head_dim=24)),
                     (2, dict(head_dim=272)), (2, dict(head_dim=0)), (2, dict(token_stride=63)),
                     (2, dict(token_stride=68)), (2, dict(page_stride=-64)), (2, dict(table_cols=0)),
                     (2, dict(table_stride=1)), (1, dict(block_table=None))]:
        refused(scute, code, lambda: A(cache=with_cache(**kw)))
    refused(scute, 1, lambda: A(cache=with_cache(k=cache.tensors[0].data_ptr() + 8)))
    refused(scute, 3, lambda: f32.paged_attention(cache, z(1, 4, 64, t=torch.float32), lens, z(1, 4, 64, t=torch.float32)))
    for bad in (lambda: ctx.paged_attention(cache, z(2, 4, 64), lens, z(2, 4, 64)),
                lambda: ctx.paged_attention(cache, q, lens, z(1, 2, 64)),
                lambda: ctx.paged_attention(cache, q, i32([1, 2]), out),
                lambda: ctx.paged_attention(cache, z(1, 64, 4).transpose(1, 2), lens, out),
                lambda: scute.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64, t=torch.float32)),
                lambda: scute.KvCache(z(4, 2, 16, 64, t=torch.float16), z(4, 2, 16, 64, t=torch.float16))):
        with pytest.raises(ValueError):
            bad()

    k = z(3, 2, 64)
    rope = scute.Rope(z(10, 64, t=torch.float32), i32([0, 1, 2]))
    P = lambda **kw: scute.scute_kv_append(ctx.handle, **{**dict(  # noqa: E731
        cache=cache, slot_map=i32([0, 1, 2]), n=3, k=k, k_stride=128, v=k, v_stride=128), **kw})
    Q = dict(q=k, q_stride=128, q_heads=2, q_out=k, q_out_stride=128, rope=rope)
    for code, kw in [(1, dict(n=-1)), (1, dict(n=(1 << 24) + 1)), (1, dict(slot_map=None)), (1, dict(k=None)),
                     (1, dict(v=None)), (2, dict(k_stride=127)), (2, dict(v_stride=0)), (1, {**Q, "rope": None}),
                     (1, {**Q, "q_out": None}), (2, {**Q, "q_heads": 0}), (2, {**Q, "q_stride": 64}),
                     (2, {**Q, "q_out_stride": 64}), (1, dict(k=k.data_ptr() + 1))]:
        refused(scute, code, lambda: P(**kw))
    for code, kw in [(2, dict(rotary_dim=0)), (2, dict(rotary_dim=65)), (2, dict(rotary_dim=128)), (2, dict(n_pos=0)),
                     (2, dict(n_axes=0)), (2, dict(n_axes=5)), (2, dict(n_axes=2)), (2, dict(axis_stride=-1)),
                     (1, dict(cos_sin=None)), (1, dict(positions=None))]:
        r = scute.Rope(z(10, 64, t=torch.float32), i32([0, 1, 2]))
        for name, val in kw.items():
            setattr(r.struct, name, val)
        refused(scute, code, lambda: P(**{**Q, "rope": r}))

    one = i32([0, 0])
    R = lambda **kw: scute.scute_kv_resize(ctx.handle, **{**dict(  # noqa: E731
        len_in=one, len_new=one, n_req=2, block_table=one, table_stride=1, table_cols=1, page_size=16, free_pages=one,
        n_free_max=2, free_in=one, free_out=one, len_out=one, cu_new=one, slot_map=one, positions=one, token_req=one,
        max_new=2), **kw})
    for code, kw in [(1, {x: None}) for x in ("len_in", "len_new", "block_table", "free_pages", "free_in", "free_out",
                                              "len_out", "cu_new", "slot_map", "positions", "token_req")] + [
            (1, dict(n_req=-1)), (1, dict(n_req=16385)), (1, dict(max_new=-1)), (1, dict(max_new=(1 << 30) + 1)),
            (1, dict(n_free_max=-1)), (2, dict(page_size=0)), (2, dict(table_cols=0)), (2, dict(table_stride=0)),
            (2, dict(table_cols=1 << 30, table_stride=1 << 30)), (2, dict(page_size=1 << 30, table_cols=2, table_stride=2))]:
        refused(scute, code, lambda: R(**kw))

    y = z(2, 64)
    w = torch.ones(64, device="cuda")
    N = lambda **kw: scute.scute_residual_norm(ctx.handle, **{**dict(  # noqa: E731
        n=2, d=64, y=y, y_stride=64, out=y, out_stride=64), **kw})
    for code, kw in [(1, dict(y=None)), (1, dict(n=-1)), (2, dict(d=0)), (2, dict(d=32769, y_stride=40000)),
                     (2, dict(y_stride=63)), (2, dict(out_stride=63)), (2, dict(residual=y, residual_stride=1)),
                     (2, dict(residual_out=y, residual_out_stride=1)), (2, dict(gate_rows=y, gate_stride=1)),
                     (1, dict(gate_rows=y, gate_stride=64, gate_vec=w)), (1, dict(post_b=w)), (1, dict(out=None)),
                     (1, dict(out=None, residual_out=y, residual_out_stride=64, pre_w=w)), (1, dict(eps=-1.0)),
                     (1, dict(eps=float("nan"))), (1, dict(scale=float("inf"))), (1, dict(y=y.data_ptr() + 1))]:
        refused(scute, code, lambda: N(**kw))
    T = lambda **kw: scute.scute_rope_table(ctx.handle, **{**dict(  # noqa: E731
        cos_sin=w, n_pos=1, rotary_dim=64, theta=1e4), **kw})
    for code, kw in [(1, dict(cos_sin=None)), (2, dict(n_pos=0)), (2, dict(rotary_dim=3)), (2, dict(rotary_dim=258)),
                     (1, dict(theta=0.0)), (1, dict(theta=float("nan")))]:
        refused(scute, code, lambda: T(**kw))
    assert ctx.launch_count() == before and ctx.sync_status() == 0


def test_wrong_sizes_types_and_strides_are_refused(scute, contexts):
    """What the tensors themselves show: a kernel would read past them, or other values."""
    ctx, f32 = contexts["bf16"], contexts["fp32"]
    before = ctx.launch_count()
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, device="cuda", dtype=t)  # noqa: E731
    whole = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.int32)  # noqa: E731
    cache = scute.KvCache(z(4, 2, 16, 64), z(4, 2, 16, 64), whole(2, 2))
    q, out, w = z(2, 4, 64), z(2, 4, 64), z(64, t=torch.float32)
    rope = scute.Rope(z(10, 64, t=torch.float32), whole(3))
    k, slots, y = z(3, 2, 64), whole(3), z(2, 64)
    steps = dict(len_in=whole(2), len_new=whole(2), block_table=whole(2, 2), page_size=16, free_pages=whole(4),
                 free_in=whole(1), free_out=whole(1), len_out=whole(2), cu_new=whole(3), slot_map=whole(2),
                 positions=whole(2), token_req=whole(2))
    bad = [lambda: ctx.paged_attention(cache, q, whole(4)[::2], out), lambda: ctx.paged_attention(cache, q, whole(2).long(), out),
           lambda: ctx.paged_attention(cache, q.float(), whole(2), out),
           lambda: ctx.paged_attention(cache, q, whole(2), out, lse=z(2, 4)),
           lambda: ctx.paged_attention(cache, q, whole(2), out, lse=z(2, 8, t=torch.float32)[:, ::2]),
           lambda: ctx.kv_append(cache, whole(6)[::2], k, k), lambda: ctx.kv_append(cache, slots.long(), k, k),
           lambda: ctx.kv_append(cache, slots, k.float(), k), lambda: ctx.kv_append(cache, slots, k, k[:2]),
           lambda: ctx.kv_append(cache, slots, k, k, q=k, q_out=k.float(), rope=rope),
           lambda: ctx.residual_norm(y, y, pre_w=w[:63]), lambda: ctx.residual_norm(y, y, pre_w=w.bfloat16()),
           lambda: ctx.residual_norm(y, y, gate=w.bfloat16()), lambda: ctx.residual_norm(y, y, residual=y.float()),
           lambda: f32.residual_norm(y, y), lambda: ctx.residual_norm(y, y[:1])]
    bad += [lambda kw=kw: ctx.kv_resize(**{**steps, **kw}) for kw in (
        dict(len_new=whole(1)), dict(len_in=whole(4)[::2]), dict(len_out=whole(2).long()), dict(cu_new=whole(2)),
        dict(positions=whole(1)), dict(token_req=whole(3)), dict(slot_map=whole(4)[::2]), dict(free_in=whole(1).long()),
        dict(free_out=whole(0)), dict(free_pages=whole(8)[::2]), dict(block_table=whole(1, 2)))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert ctx.launch_count() == before
