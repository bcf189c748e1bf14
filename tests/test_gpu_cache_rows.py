"""Rows that share cache pages (kv_fork, kv_copy), the append with normed heads and
attention with first tokens that stay visible, on the GPU against their float64
definitions (``oracle/block_ops.py``).

Tolerances, with u = 2^-24 (half a 32-bit step) and 2^-8 (half a bf16 step, of the value):
  * fork and copy: whole numbers and bits, equal;
  * a normed head of D elements: the sum of squares is off by (D + 2) u relative, its
    root by half that and the division, the root and the mean by 3 u more; the mean
    of a layer norm by (D + 2) u of the mean of |x|, which the weight and the factor
    carry on; the turning by 3 u of |a| + |b|; then the output's own rounding;
  * attention: as in the tests of the one-token attention (``check_attend``).
"""
import numpy as np
import pytest

from oracle import block_ops as OB
from test_gpu_block_ops import DT, EDGES, PAGES, U, check_attend, ctx_of, f64, i32, make_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


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


# ---------------------------------------------------------------- fork
class Fork:
    """A random state of a paged cache whose rows share pages, and a step on it."""

    def __init__(self, g, n_in, n_out, page, cols, spare=None, ends=0.2, wild=False):
        self.page, self.cols = page, cols
        cap = cols * page
        self.len_in = g.integers(0, cap + 1, n_in)
        self.len_in[g.random(n_in) < 0.2] = 0
        need = -(-self.len_in // page)
        spare = int(g.integers(0, n_out + 3)) if spare is None else spare
        total = int(need.sum()) + spare + 5
        order, at = g.permutation(total), 0
        self.table = np.full((n_in, cols), -1, np.int64)
        self.extra = np.zeros(total, np.int64)
        for r in range(n_in):
            k = 0
            if r and g.random() < 0.6:            # shares the full pages of an earlier row's beginning
                s = int(g.integers(0, r))
                k = int(g.integers(0, min(self.len_in[r], self.len_in[s]) // page + 1))
                self.table[r, :k] = self.table[s, :k]
                self.extra[self.table[r, :k]] += 1
            self.table[r, k:need[r]] = order[at:at + need[r] - k]
            at += need[r] - k
        for p in order[total - spare - 5:total - spare]:      # pages that others hold, one of them twice
            self.extra[p] = g.integers(0, 2)
        self.free = list(order[total - spare:]) if spare else []
        self.n_pages = total
        self.source = g.integers(0, n_in, n_out) if n_in else np.full(n_out, -1)
        if n_in == n_out and g.random() < 0.4:
            keep = g.random(n_out) < 0.6
            self.source[keep] = np.arange(n_out)[keep]
        self.source[g.random(n_out) < ends] = -1
        have = np.where(self.source >= 0, self.len_in[self.source] if n_in else 0, 0)
        self.len_new = np.where(g.random(n_out) < 0.5, have, (have * g.random(n_out)).astype(np.int64))
        if wild:                                   # out of range: clipped, left out, recorded
            self.source[0], self.len_new[-1] = n_in + 3, 10 ** 6
            self.len_in[0] = cap + 7
            self.table[0] = self.table[0].clip(0)
            self.table[1, 0] = total + 9

    def run(self, ctx, len_new=True, cols_out=None):
        dev = lambda x: i32(np.asarray(x, np.int64))  # noqa: E731
        n_out = len(self.source)
        wide = torch.full((max(n_out, 1), self.cols + 3), -7, dtype=torch.int32, device="cuda")
        table_out = wide[:, :self.cols]
        extra, free = dev(self.extra), torch.full((self.n_pages,), -9, dtype=torch.int32, device="cuda")
        free[:len(self.free)] = dev(self.free)
        kept = free.clone()
        count = dev([len(self.free)])
        out = [torch.full((n_out,), -5, dtype=torch.int32, device="cuda") for _ in range(4)]
        table_in, len_in = dev(self.table), dev(self.len_in)
        ctx.kv_fork(table_in, len_in, dev(self.source), table_out, out[0], self.page, extra, free, count, count, *out[1:],
                    len_new=dev(self.len_new) if len_new else None)
        status = ctx.sync_status()
        ref = OB.fork(self.table, self.len_in, self.source, self.len_new if len_new else None,
                      np.full((n_out, self.cols), -7), self.page, self.extra, self.free)
        assert status == (0 if ref["ok"] else PAGES)
        for name, got in zip(("len_out", "copy_from", "copy_to", "copy_tokens"), out):
            assert np.array_equal(got.cpu().numpy(), ref[name]), name
        assert np.array_equal(table_out[:n_out].cpu().numpy(), ref["table"])
        assert torch.all(wide[:, self.cols:] == -7)
        assert np.array_equal(extra.cpu().numpy(), ref["extra"])
        n = len(ref["free"])
        assert int(count) == n and free[:n].cpu().tolist() == ref["free"]
        assert torch.equal(free[n:], kept[n:])               # above the count the list keeps what it held
        assert torch.equal(table_in, dev(self.table)) and torch.equal(len_in, dev(self.len_in))
        return ref, table_out, out, extra, free, count


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("n_in,n_out,page,cols", [
    (1, 1, 16, 3), (1, 64, 16, 40), (4, 4, 1, 30), (5, 3, 24, 7), (64, 64, 16, 33), (7, 300, 8, 5), (300, 7, 5, 9),
    (1030, 1030, 16, 12), (33, 40, 64, 300), (3, 2, 16, 700), (2, 0, 16, 4), (0, 3, 16, 4)])
def test_fork_rows(scute, contexts, n_in, n_out, page, cols, seed):
    g = np.random.default_rng([seed, n_in, n_out, page])
    Fork(g, n_in, n_out, page, cols).run(contexts["bf16"], len_new=seed != 1)


@pytest.mark.parametrize("spare", [0, 1, 5])
def test_fork_when_pages_run_out(scute, contexts, spare):
    g = np.random.default_rng(spare)
    f = Fork(g, 20, 60, 16, 6, spare=spare, ends=0.0)
    ref = f.run(contexts["fp32"])[0]
    assert not ref["ok"]


def test_fork_clips_what_is_out_of_range(scute, contexts):
    g = np.random.default_rng(9)
    assert not Fork(g, 6, 9, 16, 5, wild=True).run(contexts["bf16"])[0]["ok"]


def test_fork_most_rows(scute, contexts):
    g = np.random.default_rng(16384)
    Fork(g, 16384, 16384, 16, 4).run(contexts["bf16"])


def test_fork_steps_keep_every_page_once(scute, contexts):
    """Fifty steps of forks, ends and growth: each page is free, or held by as many rows
    as its count says, and no row's last page in part is another's."""
    ctx, g = contexts["bf16"], np.random.default_rng(77)
    n, page, cols, total = 24, 8, 12, 400
    whole = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    table, length = [whole(n, cols) - 1, whole(n, cols) - 1], [whole(n), whole(n)]
    extra, free, count = whole(total), torch.arange(total, dtype=torch.int32, device="cuda"), whole(1) + total
    cf, ct, cn, cu, rows = whole(n), whole(n), whole(n), whole(n + 1), n * 9
    for step in range(50):
        a, b = step % 2, 1 - step % 2
        have = length[a].cpu().numpy()
        want = np.minimum(have + g.integers(0, 9, n), cols * page)
        ctx.kv_resize(length[a], i32(want), table[a], page, free, count, count, length[a], cu, whole(rows), whole(rows), whole(rows))
        source = g.integers(-1, n, n)
        cut = np.where(g.random(n) < 0.3, want[source] * g.random(n), want[source]).astype(np.int64)
        cut[source < 0] = 0
        ctx.kv_fork(table[a], length[a], i32(source), table[b], length[b], page, extra, free, count, count, cf, ct, cn,
                    len_new=i32(cut))
        assert ctx.sync_status() == 0
        tab, lens, ex = table[b].cpu().numpy(), length[b].cpu().numpy(), extra.cpu().numpy()
        holders = np.zeros(total, np.int64)
        for r in range(n):
            pages = tab[r, :-(-lens[r] // page)]
            holders[pages] += 1
            assert len(set(pages)) == len(pages)
        for r in range(n):
            if lens[r] % page:
                assert holders[tab[r, lens[r] // page]] == 1
        listed = free[:int(count)].cpu().numpy()
        assert len(set(listed)) == len(listed) and np.all(holders[listed] == 0)
        assert len(listed) + np.count_nonzero(holders) == total
        assert np.array_equal(ex, np.maximum(holders - 1, 0)) and np.array_equal(lens, cut)


# ---------------------------------------------------------------- copy
@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("H,D,page,token_major,layers", [(2, 128, 16, False, 1), (3, 80, 24, True, 3), (1, 16, 1, False, 2),
                                                         (8, 256, 5, False, 65)])
def test_copy_pages(scute, contexts, kind, H, D, page, token_major, layers):
    g = np.random.default_rng(H + D)
    n, pages = 9, 40
    shape = (pages, page, H, D) if token_major else (pages, H, page, D)
    tt = {"bf16": torch.int16, "fp32": torch.int32, "fp8": torch.uint8}[kind]
    draw = lambda: torch.from_numpy(g.integers(0, 100, shape)).to(tt).cuda()  # noqa: E731
    pools = [(draw(), draw()) for _ in range(layers)]
    order = g.permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    src[4] = src[5]                                      # two copies of one page
    tokens = g.integers(0, page + 1, n)
    dst[2] = -1
    want = [tuple(x.clone() for x in kv) for kv in pools]
    for use in (tokens, None):
        for kv in want:
            for x in kv:
                for i in range(n):
                    t = page if use is None else int(use[i])
                    if dst[i] >= 0 and token_major:
                        x[dst[i], :t] = x[src[i], :t]
                    elif dst[i] >= 0:
                        x[dst[i], :, :t] = x[src[i], :, :t]
        caches = scute.KvCaches([scute.KvCache(k.view(DT[kind]), v.view(DT[kind]), token_major=token_major) for k, v in pools])
        ctx = ctx_of(contexts, kind)
        ctx.kv_copy(caches, i32(src), i32(dst), None if use is None else i32(use))
        assert ctx.sync_status() == 0
        for got, ref in zip(pools, want):
            assert all(torch.equal(x, y) for x, y in zip(got, ref))


def test_copy_leaves_out_what_is_out_of_range(scute, contexts):
    pool = torch.arange(6 * 4 * 16 * 16, device="cuda").remainder(251).to(torch.bfloat16).view(6, 4, 16, 16)
    k, v = pool.clone(), pool.clone() + 1
    ctx = contexts["bf16"]
    caches = scute.KvCaches([scute.KvCache(k, v)])
    ctx.kv_copy(caches, i32([0, 6, 2, -1]), i32([1, 3, 6, 4]), i32([16, 16, 16, 16]))
    assert ctx.sync_status() == PAGES
    pool[1] = pool[0]
    assert torch.equal(k, pool) and torch.equal(v[1], v[0]) and torch.equal(v[3:], pool[3:] + 1)
    ctx.kv_copy(caches, i32([0]), i32([5]), i32([99]))
    assert ctx.sync_status() == PAGES
    pool[5] = pool[0]
    assert torch.equal(k, pool)


# ---------------------------------------------------------------- append with normed heads
@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("H,group,D,rot,interleaved,layer,each,shift,axes", [
    (8, 4, 128, 128, False, False, False, 0, 1), (2, 1, 128, 64, True, True, True, 0, 1), (1, 7, 80, 80, False, False, True, 0, 1),
    (2, 3, 96, 48, False, True, False, 0, 3), (3, 2, 256, 256, False, False, False, 0, 1), (1, 2, 256, 256, True, True, False, 0, 1),
    (2, 2, 64, 30, False, False, False, 0, 2), (1, 5, 16, 2, True, False, True, 0, 1), (2, 4, 128, 128, False, True, True, 1, 1),
    (2, 2, 256, 0, False, False, False, 0, 1), (1, 1, 256, 0, False, True, False, 1, 1), (4, 8, 128, 128, False, False, False, 0, 1)])
@pytest.mark.parametrize("n", [1, 37, 700])
def test_append_normed_heads(scute, contexts, kind, H, group, D, rot, interleaved, layer, each, shift, axes, n):
    g = np.random.default_rng([H, group, D, rot, n])
    dt, page, eps = DT["fp32" if kind == "fp32" else "bf16"], 16, 1e-5
    qh = H * group
    wide = torch.from_numpy(g.standard_normal((n, (qh + 2 * H) * D + 8), dtype=np.float32) * 2 + 0.3).to(dt).cuda()
    q, k, v = (wide[:, shift + a * D:shift + b * D] for a, b in ((0, qh), (qh, qh + H), (qh + H, qh + 2 * H)))
    total = -(-n // page) + 2
    slots = g.permutation(total * page)[:n]
    slots[g.random(n) < 0.1] = -1
    pools = [torch.zeros(total, H, page, D, dtype=dt, device="cuda").to(DT[kind]) for _ in range(2)]
    ks = vs = None
    if kind == "fp8":
        ks, vs = (torch.from_numpy((0.02 + 0.03 * g.random(H)).astype(np.float32)).cuda() for _ in range(2))
    cache = scute.KvCache(*pools, k_scale=ks, v_scale=vs)
    weight = lambda h: torch.from_numpy(1 + 0.3 * g.standard_normal((h, D) if each else D, dtype=np.float32)).cuda()  # noqa: E731
    qw, kw = weight(qh), weight(H)
    rope = angle = None
    if rot:
        pos = g.integers(0, 500, (axes, n))
        cs = torch.empty(500, rot, device="cuda")
        ctx_of(contexts, kind).rope_table(cs, 10000.0)
        pairs = rot // 2
        sections = [pairs - (axes - 1) * (pairs // 4)] + [pairs // 4] * (axes - 1)
        rope = scute.Rope(cs, i32(pos if axes > 1 else pos[0]), sections=sections, interleaved=interleaved)
        angle = pos[np.repeat(np.arange(axes), sections)].T * (10000.0 ** (-np.arange(pairs) / pairs))     # [n, pairs]
    out = torch.full((n, qh * D), float("nan"), dtype=dt, device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.kv_append(cache, i32(slots), k, v, q=q, q_out=out, rope=rope, norm=scute.HeadNorm(qw, kw, eps=eps, layer=layer))
    assert ctx.sync_status() == 0

    def ready(x, heads, w):
        x, w = f64(x).reshape(n, heads, D), f64(w)
        y = OB.head_norm(x, w, eps, layer)
        mean = x.mean(-1, keepdims=True) if layer else 0.0
        f = np.abs(w) / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
        # the factor off by (D / 2 + 6) u; a layer norm's mean by (D + 2) u of mean |x|,
        # which also moves the sum of squares by twice that times mean |x - mean| (0 but for rounding)
        err = U * (D / 2 + 8) * np.abs(y) + (U * (D + 4) * np.abs(x).mean(-1, keepdims=True) * f if layer else 0.0)
        if rot:
            z = np.stack([OB.rope(y[r], angle[r], rot, interleaved) for r in range(n)])
            part = np.stack([OB.rope(np.abs(y[r]), 0 * angle[r], rot, interleaved) for r in range(n)])
            pair = (lambda m: m[..., :rot].reshape(n, heads, rot // 2, 2)[..., ::-1].reshape(n, heads, rot)) if interleaved else \
                   (lambda m: np.concatenate([m[..., rot // 2:rot], m[..., :rot // 2]], -1))
            other, other_err = pair(part), pair(err)
            err = err.copy()
            # the partner's error joins; cosines and sines in 32 bits, two products and a sum
            err[..., :rot] = err[..., :rot] + other_err + 5 * U * (part[..., :rot] + other)
            return z, err
        return y, err

    def close(got, ref, err, half_step):
        err = err + half_step * 1.001 * np.abs(ref) + half_step * err + 1e-30
        assert np.all(np.abs(got - ref) <= err), float((np.abs(got - ref) / err).max())

    own = U if kind == "fp32" else 2.0 ** -8
    zq, eq = ready(q, qh, qw)
    close(f64(out).reshape(n, qh, D), zq, eq, own)
    zk, ek = ready(k, H, kw)
    zv = f64(v).reshape(n, H, D)
    kept = np.nonzero(slots >= 0)[0]
    at = slots[kept]
    gk, gv = (f64(p)[at // page, :, at % page] for p in pools)
    if kind == "fp8":
        sk, sv = f64(ks)[None, :, None], f64(vs)[None, :, None]
        for got, ref, err in ((gk, zk[kept] / sk, ek[kept] / sk), (gv, zv[kept] / sv, 0 * zv[kept])):
            ref = np.clip(ref, -448, 448)
            # e4m3: half a step is 2^-4 of the value, or 2^-10 below 2^-6
            assert np.all(np.abs(got - ref) <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10) * 1.001 + err * 1.1 + U * np.abs(ref))
    else:
        close(gk, zk[kept], ek[kept], own)
        assert np.array_equal(gv, zv[kept])
    rest = np.ones(total * page, bool)
    rest[at] = False
    left = np.nonzero(rest)[0]
    assert not f64(pools[0])[left // page, :, left % page].any() and not f64(pools[1])[left // page, :, left % page].any()


def test_append_norms_keys_or_queries_alone_and_in_place(scute, contexts):
    """q's weights alone leave k as kv_append writes it, and the other way round; q_out may be q."""
    g = np.random.default_rng(4)
    ctx, n, H, D = contexts["bf16"], 50, 2, 64
    draw = lambda h: torch.from_numpy(g.standard_normal((n, h, D), dtype=np.float32)).bfloat16().cuda()  # noqa: E731
    q, k, v, slots = draw(6), draw(H), draw(H), i32(np.arange(n))
    cs = torch.empty(99, D, device="cuda")
    ctx.rope_table(cs, 10000.0)
    rope = scute.Rope(cs, i32(g.integers(0, 99, n)))
    w = torch.rand(D, device="cuda") + 0.5

    def run(norm, q=q, out=None, rope=rope):
        pools = [torch.zeros(4, H, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out = torch.empty_like(q) if out is None else out
        ctx.kv_append(scute.KvCache(*pools), slots, k, v, q=q, q_out=out, rope=rope, norm=norm)
        return out, pools[0], pools[1]

    plain, both = run(None), run(scute.HeadNorm(w, w))
    only_q, only_k = run(scute.HeadNorm(q_w=w)), run(scute.HeadNorm(k_w=w))
    assert torch.equal(only_q[0], both[0]) and torch.equal(only_q[1], plain[1])
    assert torch.equal(only_k[0], plain[0]) and torch.equal(only_k[1], both[1])
    assert all(torch.equal(x[2], plain[2]) for x in (both, only_q, only_k))
    mine = q.clone()
    run(scute.HeadNorm(w, w), q=mine, out=mine)
    assert torch.equal(mine, both[0])
    # keys and values alone
    pools = [torch.zeros(4, H, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ctx.kv_append(scute.KvCache(*pools), slots, k, v, rope=rope, norm=scute.HeadNorm(w, w))
    assert torch.equal(pools[0], both[1])
    assert ctx.sync_status() == 0


# ---------------------------------------------------------------- first tokens that stay visible
@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (16, 4), (20, 17), (64, 33), (100, 400), (100000, 5), (0, 7), (31, 1)])
@pytest.mark.parametrize("H,group,D,page,token_major", [(2, 4, 128, 16, False), (1, 3, 80, 24, True), (2, 12, 64, 1, False)])
def test_attention_window_and_first_tokens(scute, contexts, kind, window, sinks, H, group, D, page, token_major):
    g = np.random.default_rng([window, sinks, D])
    cache, tokens = make_cache(scute, g, EDGES, H, D, page, kind, token_major, scales=kind == "fp8")
    q = torch.from_numpy(g.standard_normal((len(EDGES), H * group, D), dtype=np.float32) * 1.5)
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    for _ in range(2):
        ctx.paged_attention(cache, q, i32(EDGES), out, lse=lse, window=window, sinks=sinks)
        assert ctx.sync_status() == 0
        kept = [[x[OB.seen(len(x), window, sinks)] for x in kv] for kv in tokens]
        check_attend(out, lse, q, kept, kind, group)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
def test_attention_between_first_tokens_and_window_nothing_is_read(scute, contexts, kind):
    """Long requests whose middle holds no numbers, split over the GPU, capped scores."""
    g = np.random.default_rng(8)
    lens, window, sinks = [9000, 40, 2047, 5000, 0, 1030], 1000, 20
    cache, tokens = make_cache(scute, g, lens, 2, 64, 16, kind, False)
    k, v, table = cache.tensors[:3]
    tab = table.cpu().numpy()
    for r, n in enumerate(lens):
        gone = tab[r, -(-sinks // 16):max(0, n - window) // 16]
        for x in (k, v):
            (x.view(torch.uint8) if kind == "fp8" else x)[torch.from_numpy(gone.astype(np.int64)).cuda()] = 127 if kind == "fp8" else float("nan")
    q = torch.from_numpy(g.standard_normal((len(lens), 8, 64), dtype=np.float32)).cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32(lens), out, lse=lse, window=window, sinks=sinks, softcap=20.0)
    assert ctx.sync_status() == 0
    kept = [[x[OB.seen(len(x), window, sinks)] for x in kv] for kv in tokens]
    check_attend(out, lse, q, kept, kind, 4, softcap=20.0)


# ---------------------------------------------------------------- graphs, streams, alignment
def test_fork_and_copy_in_a_graph_on_another_stream(scute, contexts):
    """A captured fork and copy, replayed on other sources and lengths."""
    ctx, g = contexts["bf16"], np.random.default_rng(21)
    f = Fork(g, 30, 30, 16, 12, spare=40)
    dev = lambda x: i32(np.asarray(x, np.int64))  # noqa: E731
    table, lens, source, new = dev(f.table), dev(f.len_in), dev(f.source), dev(f.len_new)
    extra0, free0 = dev(f.extra), torch.zeros(f.n_pages, dtype=torch.int32, device="cuda")
    free0[:len(f.free)] = dev(f.free)
    extra, free, count = extra0.clone(), free0.clone(), dev([0])
    out = torch.zeros(30, 12, dtype=torch.int32, device="cuda")
    vec = [torch.zeros(30, dtype=torch.int32, device="cuda") for _ in range(4)]
    k0 = torch.randn(f.n_pages, 2, 16, 32, device="cuda").bfloat16()
    k, v = k0.clone(), k0 + 1
    v0 = v.clone()
    caches = scute.KvCaches([scute.KvCache(k, v)])
    s = torch.cuda.Stream()

    def step():
        extra.copy_(extra0), free.copy_(free0), count.fill_(len(f.free)), k.copy_(k0), v.copy_(v0)
        ctx.kv_fork(table, lens, source, out, vec[0], 16, extra, free, count, count, *vec[1:], len_new=new)
        ctx.kv_copy(caches, *vec[1:])

    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        src = g.integers(-1, 30, 30)
        want = np.where(src >= 0, (f.len_in[src] * g.random(30)).astype(np.int64), 0)
        source.copy_(dev(src)), new.copy_(dev(want))
        graph.replay()
        ok = ctx.sync_status()
        ref = OB.fork(f.table, f.len_in, src, want, out.cpu().numpy(), 16, f.extra, f.free)
        assert ok == (0 if ref["ok"] else PAGES)
        for t, name in zip(vec, ("len_out", "copy_from", "copy_to", "copy_tokens")):
            assert np.array_equal(t.cpu().numpy(), ref[name])
        assert np.array_equal(out.cpu().numpy(), ref["table"]) and np.array_equal(extra.cpu().numpy(), ref["extra"])
        assert free[:int(count)].cpu().tolist() == ref["free"]
        kk = k0.clone()
        for a, b, n in zip(ref["copy_from"], ref["copy_to"], ref["copy_tokens"]):
            if b >= 0:
                kk[b, :, :n] = k0[a, :, :n]
        assert torch.equal(k, kk) and torch.equal(v[:, :, :, 0], torch.where(kk != k0, kk + 1, v0)[:, :, :, 0])


def test_append_norm_weights_of_any_alignment_and_positions_out_of_range(scute, contexts):
    """Weights that begin at any element, and strided ones, give what aligned ones give;
    slots and positions outside are left out and recorded."""
    ctx, g = contexts["bf16"], np.random.default_rng(8)
    n, H, D = 33, 2, 64
    draw = lambda h: torch.from_numpy(g.standard_normal((n, h, D), dtype=np.float32)).bfloat16().cuda()  # noqa: E731
    q, k, v = draw(4), draw(H), draw(H)
    cs = torch.empty(50, D, device="cuda")
    ctx.rope_table(cs, 10000.0)
    slots, pos = np.arange(n), g.integers(0, 50, n)
    w, each = torch.rand(D, device="cuda") + 0.5, torch.rand(4, D, device="cuda") + 0.5
    odd = torch.zeros(D + 1, device="cuda")[1:].copy_(w)
    wide = torch.zeros(4, D + 3, device="cuda")[:, :D].copy_(each)

    def run(norm, slots=slots, pos=pos):
        pools = [torch.zeros(3, H, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out = torch.empty_like(q)
        ctx.kv_append(scute.KvCache(*pools), i32(slots), k, v, q=q, q_out=out, rope=scute.Rope(cs, i32(pos)), norm=norm)
        return out, pools[0], pools[1], ctx.sync_status()

    for a, b in ((scute.HeadNorm(w, w), scute.HeadNorm(odd, odd)), (scute.HeadNorm(each, w), scute.HeadNorm(wide, odd))):
        x, y = run(a), run(b)
        assert x[3] == y[3] == 0 and torch.equal(x[2], y[2])
        # the two kernels add squares in another order, so that their 32-bit results, 2^-21 of a
        # pair's elements (below 8) apart, may round to neighbouring bf16 numbers: those are
        # 2^-7 of the smaller one's power of two apart, up to 2^-7 of the value
        for s, t in zip(x[:2], y[:2]):
            far = (s.float() - t.float()).abs() > 2.0 ** -7 * torch.maximum(s.float().abs(), t.float().abs()) + 2.0 ** -18
            assert not far.any()
    bad_slots, bad_pos = slots.copy(), pos.copy()
    bad_slots[3], bad_pos[5], bad_pos[6] = 3 * 16, 50, -1
    clipped = pos.copy()
    clipped[5], clipped[6] = 49, 0
    without = slots.copy()
    without[3] = -1
    for norm in (scute.HeadNorm(w, w), scute.HeadNorm(odd, odd)):
        x, y = run(norm, bad_slots, bad_pos), run(norm, without, clipped)
        assert x[3] == PAGES and y[3] == 0
        assert all(torch.equal(s, t) for s, t in zip(x[:3], y[:3]))


def test_append_norm_zero_heads_and_infinities_stay_in_their_heads(scute, contexts):
    """A head of zeros stays zero; one with an infinity or no number leaves the others as they were."""
    ctx = contexts["fp32"]
    n, H, D = 3, 4, 32
    q = torch.randn(n, H, D, device="cuda")
    q[0, 1] = 0.0
    bad = q.clone()
    bad[1, 2, 5], bad[2, 0, 0] = float("inf"), float("nan")
    w = torch.ones(D, device="cuda")
    out = []
    for x in (q, bad):
        pools = [torch.zeros(1, H, 16, D, device="cuda") for _ in range(2)]
        y = torch.empty_like(x)
        ctx.kv_append(scute.KvCache(*pools), i32([0, 1, 2]), x, x, q=x, q_out=y, norm=scute.HeadNorm(w, w))
        out.append(y)
    assert ctx.sync_status() == 0 and not out[0][0, 1].any()
    same = torch.ones(n, H, dtype=torch.bool)
    same[1, 2] = same[2, 0] = False
    assert torch.equal(out[0][same], out[1][same])


# ---------------------------------------------------------------- refusals
def test_refusals_of_forks_copies_norms_and_sinks(scute, contexts):
    ctx = contexts["bf16"]
    whole = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(table_in=whole(2, 4), len_in=whole(2), source=whole(3), table_out=whole(3, 4), len_out=whole(3), page_size=16,
                extra=whole(9), free_pages=whole(9), free_in=whole(1), free_out=whole(1), copy_from=whole(3), copy_to=whole(3),
                copy_tokens=whole(3), len_new=whole(3))
    ctx.kv_fork(**good)
    both = whole(6)
    bad = [dict(page_size=0), dict(page_size=1 << 30), dict(table_out=whole(3, 5)), dict(table_out=whole(2, 4)), dict(table_in=whole(1, 4)),
           dict(len_out=good["len_in"]), dict(len_out=good["len_new"]), dict(copy_from=good["source"]), dict(copy_to=good["copy_from"]),
           dict(table_out=good["table_in"].expand(2, 4)), dict(len_out=whole(2)), dict(copy_tokens=whole(4)), dict(len_new=whole(2)),
           dict(free_out=whole(2)), dict(free_in=good["free_pages"][:1], free_out=good["free_pages"][:1]),
           dict(extra=good["free_pages"]), dict(len_in=whole(2).float()), dict(source=whole(3).long()), dict(extra=whole(18)[::2]),
           dict(table_in=whole(4, 2).t()), dict(table_out=whole(1, 4).expand(3, 4)), dict(len_out=both[:3], copy_from=both[2:5])]
    for i, kw in enumerate(bad):
        with pytest.raises((ValueError, scute.ScuteError)):
            ctx.kv_fork(**{**good, **kw})
            raise AssertionError(i)
    pool = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    cache = lambda *s, **kw: scute.KvCache(pool(*s), pool(*s), **kw)  # noqa: E731
    one = cache(4, 2, 16, 64)
    ctx.kv_copy(scute.KvCaches([one, cache(4, 2, 16, 64)]), whole(2) + 1, whole(2) - 1)
    bad = [lambda: scute.KvCaches([]), lambda: scute.KvCaches([pool(4, 2, 16, 64)]),
           lambda: ctx.kv_copy(scute.KvCaches([one, cache(5, 2, 16, 64)]), whole(2), whole(2)),
           lambda: ctx.kv_copy(scute.KvCaches([one, cache(4, 2, 16, 64, token_major=True)]), whole(2), whole(2)),
           lambda: ctx.kv_copy(scute.KvCaches([scute.KvCache(*[pool(4, 2, 16, 64, t=torch.float32)] * 2)]), whole(2), whole(2)),
           lambda: ctx.kv_copy(scute.KvCaches([one]), whole(2), whole(3)), lambda: ctx.kv_copy(scute.KvCaches([one]), whole(2).long(), whole(2)),
           lambda: ctx.kv_copy(scute.KvCaches([one]), whole(2), whole(2), whole(1)),
           lambda: ctx.kv_copy(scute.KvCaches([one] * 1025), whole(2), whole(2))]
    w, k, q = torch.ones(64, device="cuda"), pool(3, 2, 64), pool(3, 4, 64)
    append = lambda norm, **kw: ctx.kv_append(one, whole(3), k, k, norm=norm, **kw)  # noqa: E731
    append(scute.HeadNorm(w, w), q=q, q_out=q)
    bad += [lambda: scute.HeadNorm(), lambda: scute.HeadNorm(w.double()), lambda: scute.HeadNorm(w.bfloat16()), lambda: scute.HeadNorm(w.view(1, 1, 64)),
            lambda: scute.HeadNorm(torch.ones(128, device="cuda")[::2]), lambda: scute.HeadNorm(w.view(1, 64).expand(4, 64)),
            lambda: append(scute.HeadNorm(torch.ones(32, device="cuda")), q=q, q_out=q),
            lambda: append(scute.HeadNorm(torch.ones(2, 64, device="cuda")), q=q, q_out=q),
            lambda: append(scute.HeadNorm(k_w=torch.ones(4, 64, device="cuda"))), lambda: append(scute.HeadNorm(w, w, eps=-1.0)),
            lambda: append(scute.HeadNorm(w, w, eps=float("nan"))), lambda: append(scute.HeadNorm(w), q=q)]
    lens, table = whole(3), scute.KvCache(pool(4, 2, 16, 64), pool(4, 2, 16, 64), whole(3, 2))
    ctx.paged_attention(table, q, lens, q, window=3, sinks=1 << 30)
    bad += [lambda: ctx.paged_attention(table, q, lens, q, window=3, sinks=-1),
            lambda: ctx.paged_attention(table, q, lens, q, window=3, sinks=(1 << 30) + 1)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, scute.ScuteError)):
            call()
            raise AssertionError(i)
    for null in (lambda: scute.load().scute_kv_fork(ctx.handle, None, None), lambda: scute.load().scute_kv_copy(ctx.handle, None, 1, None, None, None, 1, None),
                 lambda: scute.load().scute_paged_attention_shared(ctx.handle, table.ref, None, None, None),
                 lambda: scute.load().scute_kv_fork(None, None, None)):
        assert null() == 1                    # SCUTE_ERR_ARG
    assert ctx.sync_status() == 0


def test_fork_of_counts_that_are_no_counts(scute, contexts):
    """Counts far below any that rows can leave (a buffer that was never set) are recorded,
    and nothing is written beside the tables."""
    for n_in, n_out, page, cols in [(5, 40, 16, 6), (300, 300, 8, 5), (1030, 1030, 16, 12)]:
        g = np.random.default_rng(n_in)
        f = Fork(g, n_in, n_out, page, cols, spare=3)
        wild = np.array([-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 7, -2 ** 30 - 1, -2 ** 30, -9, 2 ** 31 - 1, 0])
        extra = i32(wild[g.integers(0, len(wild), f.n_pages)])
        wide = torch.full((n_out, cols + 3), -7, dtype=torch.int32, device="cuda")
        free, count = i32(np.pad(f.free, (0, f.n_pages - len(f.free)))), i32([len(f.free)])
        out = [torch.full((n_out,), -5, dtype=torch.int32, device="cuda") for _ in range(4)]
        contexts["bf16"].kv_fork(i32(f.table), i32(f.len_in), i32(f.source), wide[:, :cols], out[0], page, extra, free, count, count,
                                 *out[1:], len_new=i32(f.len_new))
        assert contexts["bf16"].sync_status() == PAGES
        assert torch.all(wide[:, cols:] == -7) and int(wide[:, :cols].max()) < f.n_pages
        assert 0 <= int(count) <= f.n_pages and torch.all(free[:int(count)] < f.n_pages)
        assert -1 <= int(out[2].min()) and int(out[2].max()) < f.n_pages


def test_fork_refuses_outputs_over_the_list_s_count(scute, contexts):
    whole = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    both = whole(3)
    for name in ("len_out", "copy_to", "extra", "free_pages"):
        good = dict(table_in=whole(2, 4), len_in=whole(2), source=whole(3), table_out=whole(3, 4), len_out=whole(3), page_size=16,
                    extra=whole(3), free_pages=whole(3), free_in=both[1:2], free_out=whole(1), copy_from=whole(3),
                    copy_to=whole(3), copy_tokens=whole(3))
        contexts["bf16"].kv_fork(**good)
        with pytest.raises(scute.ScuteError):
            contexts["bf16"].kv_fork(**{**good, name: both})


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (20, 17), (100, 400), (300, 5)])
@pytest.mark.parametrize("n,H,group,D,page,token_major", [
    (160, 2, 4, 128, 16, False), (160, 2, 3, 80, 24, True), (160, 2, 12, 64, 1, False), (90, 4, 1, 64, 7, True), (80, 2, 40, 128, 16, False),
    (3, 400, 1, 16, 16, False), (1, 2600, 1, 16, 16, True)])
def test_attention_window_and_first_tokens_of_many_rows(scute, contexts, kind, window, sinks, n, H, group, D, page, token_major):
    """Rows enough for warps on their own: several requests in a warp's range, ranges that
    end in a request, heads that have more ranges than one or fewer warps than heads."""
    g = np.random.default_rng([window, n, H, D])
    lens = [int(x) for x in np.where(g.random(n) < 0.2, 0, g.integers(1, 500, n))]
    lens[-1] = 700
    cache, tokens = make_cache(scute, g, lens, H, D, page, kind, token_major, scales=kind == "fp8")
    q = torch.from_numpy(g.standard_normal((n, H * group, D), dtype=np.float32) * 1.5).cuda().bfloat16()
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx, was = contexts["bf16"], None
    before = ctx.launch_count()
    for _ in range(2):
        ctx.paged_attention(cache, q, i32(lens), out, lse=lse, window=window, sinks=sinks)
        assert ctx.sync_status() == 0
        assert was is None or (torch.equal(out, was[0]) and torch.equal(lse, was[1]))
        was = out.clone(), lse.clone()
    assert ctx.launch_count() - before == 4                  # the rows' kernel and the join of its parts
    check_attend(out, lse, q, [[x[OB.seen(len(x), window, sinks)] for x in kv] for kv in tokens], kind, group)
    # more tokens than the rule lets, with up to eight heads to a key: the other kernel
    ctx.paged_attention(cache, q, i32(lens), out, lse=lse, window=1 << 20, sinks=sinks)
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, tokens, kind, group)


def counted_short():
    """Old tables with more rows of a page than its count allows: (table, len_in, source, len_new, extra, whether
    the step can go on without giving a held page away), pages of 16 tokens."""
    two, whole, part = [[0], [0]], [16, 16], [5, 5]
    return [(two, whole, [0], None, [0], False),              # kept whole by one: given up all the same
            (two, whole, [1], None, [0], False), (two, whole, [-1, 1], None, [0], False),
            (two, whole, [-1, -1, 0], None, [0], False),      # the same, counted down and up
            (two, part, [0], None, [0], False),               # below nobody, and claimed
            (two, part, [1, 0, 1], None, [0], False),
            (two, whole, [0, 1], [16, 5], [0], False),        # one's whole, another ends in it
            (two, whole, [0], [5], [0], False),
            (two, whole, [-1], None, [0], False),             # nobody's, below nobody
            ([[0, 1], [0, 2], [0, 3]], [32, 20, 16], [0], None, [1, 0, 0, 0], False),
            (two, whole, [0], None, [1], True), (two, part, [0], None, [1], True), (two, whole, [0, 1], [16, 5], [1], True),
            (two, whole, [-1], None, [1], True), ([[0], [0]], whole, [-1], None, [2], True),
            ([[0, 1], [0, 2], [0, 3]], [32, 20, 16], [0, 1], None, [2, 0, 0, 0], True)]


@pytest.mark.parametrize("case", range(len(counted_short())))
@pytest.mark.parametrize("beside", [0, 1030])
def test_fork_records_pages_of_more_rows_than_their_count(scute, contexts, case, beside):
    """A page that a row still names is not given up, or to a row that ends in it, without a word; alone
    (one cluster) and beside many healthy rows (four launches)."""
    table, len_in, source, len_new, extra, fine = counted_short()[case]
    f = Fork(np.random.default_rng(case), beside, beside, 16, 2, spare=beside + 4)
    n, at = beside, f.n_pages
    f.table = np.concatenate([f.table, np.full((len(table), 2), -1)])
    for r, row in enumerate(table):
        f.table[n + r, :len(row)] = np.array(row) + at
    f.len_in = np.concatenate([f.len_in, len_in]).astype(np.int64)
    f.extra, f.n_pages = np.concatenate([f.extra, extra]), at + len(extra)
    new = [16 * 2 if s < 0 else len_in[s] for s in source] if len_new is None else len_new
    f.len_new = np.concatenate([f.len_new, [0 if s < 0 else x for s, x in zip(source, new)]]).astype(np.int64)
    f.source = np.concatenate([f.source, [s if s < 0 else s + n for s in source]]).astype(np.int64)
    assert f.run(contexts["bf16"])[0]["ok"] == fine


@pytest.mark.parametrize("n", [3, 1030])
@pytest.mark.parametrize("outside", [0, -1, 2 ** 31 - 1])
def test_fork_records_pages_of_the_list_that_are_none(scute, contexts, n, outside):
    """A number outside the pool that the free list hands to a row that copies; one that stays in the list is
    nobody's yet."""
    f = object.__new__(Fork)
    f.page, f.cols, f.n_pages = 16, 3, 2 * n + 5           # every old row ends in its page, and two new ones in it
    f.table = np.full((n, 3), -1)
    f.table[:, 0] = np.arange(n)
    f.len_in, f.extra = np.full(n, 5), np.zeros(f.n_pages, np.int64)
    f.source, f.len_new = np.repeat(np.arange(n), 2), np.full(2 * n, 4)
    outside = outside or f.n_pages
    for place, fine in ((-1, False), (5, False), (4, True)):     # five entries are left
        f.free = list(range(n, 2 * n + 5))
        f.free[place] = outside
        ref = f.run(contexts["bf16"])[0]
        assert ref["ok"] == fine and np.count_nonzero(ref["copy_from"] >= 0) == n


@pytest.mark.parametrize("kind", ["bf16", "fp32", "fp8"])
@pytest.mark.parametrize("window,sinks", [(1, 1), (20, 17), (64, 33), (100, 400), (100000, 5)])
@pytest.mark.parametrize("H,group,D,page,token_major", [(2, 4, 256, 16, False), (1, 3, 192, 24, True), (1, 9, 144, 8, False)])
def test_attention_window_and_first_tokens_of_wide_heads(scute, contexts, kind, window, sinks, H, group, D, page, token_major):
    g = np.random.default_rng([window, sinks, D])
    lens = EDGES + [5000]
    cache, tokens = make_cache(scute, g, lens, H, D, page, kind, token_major, scales=kind == "fp8")
    q = torch.from_numpy(g.standard_normal((len(lens), H * group, D), dtype=np.float32) * 1.5)
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx, was = ctx_of(contexts, kind), None
    for _ in range(2):
        ctx.paged_attention(cache, q, i32(lens), out, lse=lse, window=window, sinks=sinks)
        assert ctx.sync_status() == 0
        assert was is None or (torch.equal(out, was[0]) and torch.equal(lse, was[1]))
        was = out.clone(), lse.clone()
    check_attend(out, lse, q, [[x[OB.seen(len(x), window, sinks)] for x in kv] for kv in tokens], kind, group)


@pytest.mark.parametrize("kind,group,D", [("fp8", 2, 64), ("bf16", 2, 64), ("bf16", 4, 128), ("fp8", 1, 32)])
def test_attention_window_and_first_tokens_of_most_requests(scute, contexts, kind, group, D):
    """The most requests a call takes, read by warps on their own, with whatever rings the list leaves them; or by
    CTAs, where their parts are more than the context's workspace holds."""
    g = np.random.default_rng([16384, D])
    lens = [int(x) for x in g.integers(0, 60, 16384)]
    cache, tokens = make_cache(scute, g, lens, 1, D, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((16384, group, D), dtype=np.float32) * 1.5).cuda().bfloat16()
    out, lse = torch.full_like(q, float("nan")), torch.empty(q.shape[:2], device="cuda")
    ctx = contexts["bf16"]
    ctx.paged_attention(cache, q, i32(lens), out, lse=lse, window=20, sinks=5)
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, [[x[OB.seen(len(x), 20, 5)] for x in kv] for kv in tokens], kind, group)


def test_append_norm_refuses_rows_that_32_bits_do_not_count(scute, contexts):
    ctx, heads, D = contexts["bf16"], 1 << 22, 256
    pool, w, n = torch.zeros(2, 1, 16, D, dtype=torch.bfloat16, device="cuda"), torch.ones(D, device="cuda"), 1
    cache, norm = scute.KvCache(pool, pool), scute.HeadNorm(w, w)
    slots, k = i32([-1]), torch.zeros(D, dtype=torch.bfloat16, device="cuda")
    cache.struct.kv_heads = heads
    for q_heads in (0, 8):
        q = k if q_heads else None
        with pytest.raises(scute.ScuteError, match="elements"):
            scute.scute_kv_append_norm(ctx.handle, cache, slots, n, k, heads * D, k, heads * D, q, q_heads * D, q_heads, q, q_heads * D, norm=norm)
    assert ctx.sync_status() == 0


def test_fork_of_the_widest_table(scute, contexts):
    """A row of as many entries as a table may have, few of them pages."""
    cols, n, m, pages = 2 ** 31 - 1, 5000, 4099, 6000
    g = np.random.default_rng(31)
    order = g.permutation(pages)
    ref = OB.fork(order[None, :n], [n], [0], [m], np.full((1, n), -1), 1, [0] * pages, order[n:].tolist())
    whole = lambda x: i32(np.asarray(x, np.int64))  # noqa: E731
    table, out = (torch.empty(1, cols, dtype=torch.int32, device="cuda") for _ in range(2))
    table[0, :n], out[0, :n + 9] = whole(order[:n]), -1
    extra, free, count = whole([0] * pages), whole([0] * pages), whole([pages - n])
    free[:pages - n] = whole(order[n:])
    vec = [whole([7]) for _ in range(4)]
    contexts["bf16"].kv_fork(table, whole([n]), whole([0]), out, vec[0], 1, extra, free, count, count, *vec[1:], len_new=whole([m]))
    assert contexts["bf16"].sync_status() == 0
    assert [int(x) for x in vec] == [m, -1, -1, 0] and ref["ok"] and not extra.any()
    assert out[0, :n].cpu().tolist() == ref["table"][0].tolist() and torch.all(out[0, n:n + 9] == -1)
    assert free[:int(count)].cpu().tolist() == ref["free"] and torch.equal(table[0, :n], whole(order[:n]))


@pytest.mark.parametrize("n,cols", [(60, 2000), (600, 300), (2, 40000)])
def test_fork_looks_at_every_page_that_rows_take_whole(scute, contexts, n, cols):
    """A page of more rows than its count allows, at any place of a long row."""
    f = object.__new__(Fork)
    f.page, f.cols, f.n_pages, f.free = 1, cols, n * cols + 2, [n * cols, n * cols + 1]
    own = np.random.default_rng(n).permutation(n * cols).reshape(n, cols)
    f.extra, f.source, f.len_new = np.zeros(f.n_pages, np.int64), np.arange(n), np.full(n, cols)
    for r, j in ((n // 2, None), (0, 0), (n - 1, cols - 1), (n // 2, 255), (1, 256), (n - 1, cols // 2 + 1)):
        f.table = np.concatenate([own, np.full((1, cols), -1)])
        f.len_in = np.append(np.full(n, cols), 0 if j is None else 1)
        if j is not None:
            f.table[n, 0] = own[r, j]                       # the last old row, which nobody continues
        assert f.run(contexts["bf16"])[0]["ok"] == (j is None)


@pytest.mark.parametrize("n", [5, 700])
def test_fork_of_lists_too_short_for_what_comes_back(scute, contexts, n):
    """Pages beyond the list's room are lost and recorded; rows that copy take them before."""
    whole = lambda x: i32(np.asarray(x, np.int64))  # noqa: E731
    for room, copies in ((0, 0), (3, 0), (n - 1, 2), (n, 0), (n + 2, 2), (2 * n + 2, 0)):
        # old rows of two pages, the second in part; a third of them goes on, the first `copies` twice
        table, extra, free = np.arange(2 * n).reshape(n, 2), [0] * (2 * n + 2), [2 * n, 2 * n + 1][:room]
        source = list(range(n // 3)) + list(range(copies))
        ref = OB.fork(table, [20] * n, source, None, np.full((len(source), 2), -1), 16, extra, free, room)
        got, counts, count = torch.full((len(source), 2), -1, dtype=torch.int32, device="cuda"), whole(extra), whole([len(free)])
        slots = torch.full((room + 4,), -9, dtype=torch.int32, device="cuda")
        slots[:len(free)] = whole(free)
        vec = [torch.zeros(len(source), dtype=torch.int32, device="cuda") for _ in range(4)]
        contexts["bf16"].kv_fork(whole(table), whole([20] * n), whole(source), got, vec[0], 16, counts, slots[:room], count, count, *vec[1:])
        assert contexts["bf16"].sync_status() == (0 if ref["ok"] else PAGES)
        assert int(count) == len(ref["free"]) and slots[:int(count)].cpu().tolist() == ref["free"] and torch.all(slots[room:] == -9)
        assert np.array_equal(got.cpu().numpy(), ref["table"]) and np.array_equal(counts.cpu().numpy(), ref["extra"])
        for t, name in zip(vec, ("len_out", "copy_from", "copy_to", "copy_tokens")):
            assert np.array_equal(t.cpu().numpy(), ref[name])


def test_fork_of_no_rows_and_no_pages(scute, contexts):
    none, one = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    out = torch.full((1,), 7, dtype=torch.int32, device="cuda")
    ctx = contexts["bf16"]
    ctx.kv_fork(table, none, none, table, none, 16, none, none, one, out, none, none, none)
    assert ctx.sync_status() == 0 and int(out) == 0
    # all rows let go, none taken; rows without tokens of rows without tokens
    extra, free, count = torch.zeros(9, dtype=torch.int32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda"), one.clone()
    ctx.kv_fork(i32([[3, 1], [8, -1]]), i32([17, 16]), none, table[:, :2], none, 16, extra, free, count, count, none, none, none)
    assert ctx.sync_status() == 0 and int(count) == 3 and free[:3].tolist() == [1, 3, 8] and not extra.any()
    vec = [torch.full((2,), 7, dtype=torch.int32, device="cuda") for _ in range(4)]
    wide = torch.full((2, 2), -7, dtype=torch.int32, device="cuda")
    ctx.kv_fork(i32([[-1, -1]]), i32([0]), i32([0, -1]), wide, vec[0], 16, extra, free, count, count, *vec[1:])
    assert ctx.sync_status() == 0 and int(count) == 3 and torch.all(wide == -7)
    assert [x.tolist() for x in vec] == [[0, 0], [-1, -1], [-1, -1], [0, 0]]
