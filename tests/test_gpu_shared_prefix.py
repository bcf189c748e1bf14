"""One-token attention of groups of requests that share the beginnings of their
contexts, on the GPU against the float64 definition of each request's attention over
all of its tokens (``oracle/block_ops.py``).  Tolerances are those of the one-token
attention (``check_attend``): a score's sum over D products, the sums over L tokens and the
roundings of weights and outputs are the same, however the tokens are shared out."""
import time

import numpy as np
import pytest

from oracle import block_ops as OB
from test_gpu_block_ops import DT, PAGES, U, check_attend, ctx_of, f64, i32

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


class Batch:
    """groups: (requests, shared tokens, request lengths or a function of the index); a
    request of at least the shared tokens names its group's pages, a shorter one its own."""

    def __init__(self, scute, g, groups, H, group, D, page, kind, token_major=False, scales=False, before=0, behind=0, spread=1.5):
        self.kind, self.group, self.scute = kind, group, scute
        rows, start, shared = [], [before], []           # rows: (length, group or -1)
        rows += [(int(x), -1) for x in g.integers(0, 90, before)]
        for i, (n, T, lens) in enumerate(groups):
            rows += [(int(lens(j)), i) for j in range(n)]
            start.append(start[-1] + n)
            shared.append(T)
        rows += [(int(x), -1) for x in g.integers(0, 90, behind)]
        self.lens, self.start, self.shared = [x for x, _ in rows], start, shared
        # whole pages are shared; a page that the shared tokens end in is everybody's with the same beginning
        need = [-(-x // page) for x in self.lens]
        cols = max(1, max(need, default=1))
        table, at = np.full((len(rows), cols), -1, np.int64), 0
        first_of = {}
        src = {}                                          # page: page whose first tokens it repeats
        for r, (n, i) in enumerate(rows):
            k = 0
            if i >= 0 and n >= shared[i] and shared[i]:
                whole = shared[i] // page
                if i in first_of:
                    table[r, :whole] = table[first_of[i], :whole]
                    k = whole
                    if shared[i] % page:
                        src[at] = (table[first_of[i], whole], shared[i] % page)
                else:
                    first_of[i] = r
            table[r, k:need[r]] = np.arange(at, at + need[r] - k)
            at += need[r] - k
        total = at + 3
        order = g.permutation(total)
        k, v = (g.standard_normal((total, page, H, D), dtype=np.float32) for _ in range(2))
        for p, (q, t) in src.items():
            k[p, :t], v[p, :t] = k[q, :t], v[q, :t]
        for r, n in enumerate(self.lens):
            if n % page and not (rows[r][1] >= 0 and n // page < shared[rows[r][1]] // page and n >= shared[rows[r][1]]):
                k[table[r, n // page], n % page:] = np.nan
                v[table[r, n // page], n % page:] = np.nan
        k[at:], v[at:] = np.nan, np.inf
        ks = vs = None
        if scales:
            ks, vs = (torch.from_numpy((0.5 + g.random(H)).astype(np.float32)).cuda() for _ in range(2))
        k, v = torch.from_numpy(k).to(DT[kind]), torch.from_numpy(v).to(DT[kind])
        kk, vv = f64(k), f64(v)
        if scales:
            kk, vv = kk * f64(ks)[None, None, :, None], vv * f64(vs)[None, None, :, None]
        self.tokens = [(kk[table[r, :need[r]]].reshape(-1, H, D)[:n], vv[table[r, :need[r]]].reshape(-1, H, D)[:n])
                       for r, n in enumerate(self.lens)]
        # the pages at random places of the pool
        inv = torch.from_numpy(np.argsort(order).astype(np.int64))
        as_bits = (lambda x: x.view(torch.uint8)) if kind == "fp8" else (lambda x: x)
        k, v = (as_bits(x)[inv].view(DT[kind]) for x in (k, v))
        table = np.where(table >= 0, order[table], -1)
        if not token_major:
            k, v = (as_bits(x).permute(0, 2, 1, 3).contiguous().view(DT[kind]) for x in (k, v))
        self.table = i32(table)
        self.cache = scute.KvCache(k.cuda(), v.cuda(), self.table, token_major=token_major, k_scale=ks, v_scale=vs)
        q = torch.from_numpy(g.standard_normal((len(rows), H * group, D), dtype=np.float32) * spread)
        self.q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])

    def run(self, ctx, times=2, always=True, **kw):
        n, heads = self.q.shape[:2]
        work = ctx.shared_work(self.cache, n, heads)
        work.fill_(255)                                   # not a number, whatever is read of it
        sh = self.scute.Shared(i32(self.start), i32(self.shared), work, always=always)
        out, lse = torch.full_like(self.q, float("nan")), torch.empty(n, heads, device="cuda")
        lens, was = i32(self.lens), None
        for _ in range(times):
            ctx.paged_attention(self.cache, self.q, lens, out, lse=lse, shared=sh, **kw)
            if was is not None:
                assert torch.equal(out, was[0]) and torch.equal(lse, was[1])      # the same bits
            was = out.clone(), lse.clone()
        assert ctx.sync_status() == 0
        scale, softcap = kw.get("scale") or None, kw.get("softcap", 0.0)
        check_attend(out, lse, self.q, self.tokens, self.kind, self.group, 0, softcap, scale)
        return out, lse


SOME = [0, 1, 2, 5, 16, 17, 40, 100]
GROUPS = {
    "one": [(3, 300, lambda j: 300 + SOME[j])],
    "page": [(2, 16, lambda j: 16 + 3 * j), (5, 128, lambda j: 128 + SOME[j]), (4, 129, lambda j: 129 + SOME[j])],
    "rows": [(40, 500, lambda j: 500 + j % 7), (70, 260, lambda j: 260 + j % 40), (1, 700, lambda j: 720)],
    "idle": [(6, 200, lambda j: [0, 210, 150, 200, 333, 1][j]), (3, 100, lambda j: 0), (4, 0, lambda j: 30 * j), (2, 90, lambda j: 10 + 90 * j)],
}


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("groups", sorted(GROUPS))
@pytest.mark.parametrize("H,group,D,page,token_major", [
    (2, 4, 128, 16, False), (1, 1, 64, 1, False), (2, 3, 80, 24, True), (1, 7, 96, 8, False), (1, 16, 128, 64, True),
    (2, 2, 16, 5, False), (1, 40, 64, 16, True), (1, 128, 64, 16, False), (1, 130, 32, 16, False), (1, 4, 256, 16, False)])
def test_shared_groups_heads_and_pages(scute, contexts, kind, groups, H, group, D, page, token_major):
    g = np.random.default_rng([H, group, D, page])
    b = Batch(scute, g, GROUPS[groups], H, group, D, page, kind, token_major, scales=kind == "fp8", before=2, behind=3)
    b.run(ctx_of(contexts, kind))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("H,group,D,n,T", [(8, 4, 128, 3, 30011), (8, 4, 128, 50, 20480), (4, 2, 64, 5, 50000), (2, 9, 128, 40, 9000)])
def test_shared_long_beginnings(scute, contexts, kind, H, group, D, n, T):
    """Many tiles to a CTA, work rows that several CTAs share, both ways of the streams."""
    g = np.random.default_rng([H, n, T])
    Batch(scute, g, [(n, T, lambda j: T + j % 5), (2, 700, lambda j: 710)], H, group, D, 16, kind, scales=kind == "fp8").run(ctx_of(contexts, kind))


@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("softcap,scale", [(5.0, 0.0), (0.0, -0.2), (30.0, -0.1), (0.0, 0.02)])
def test_shared_softcap_and_scale(scute, contexts, kind, softcap, scale):
    g = np.random.default_rng(7)
    b = Batch(scute, g, [(5, 400, lambda j: 400 + 9 * j), (40, 130, lambda j: 130 + j)], 2, 4, 64, 16, kind, spread=2.0)
    b.run(ctx_of(contexts, kind), softcap=softcap, scale=scale)


def test_shared_large_scores(scute, contexts):
    """Scores of +-2000: the maximum moves from tile to tile, from part to part."""
    g = np.random.default_rng(3)
    Batch(scute, g, [(3, 3000, lambda j: 3000 + 7 * j), (70, 500, lambda j: 500 + j)], 1, 4, 64, 16, "bf16", spread=600.0).run(contexts["bf16"])


def test_shared_many_groups(scute, contexts):
    """As many groups as a call takes, of one to three requests, some sharing nothing."""
    g = np.random.default_rng(1024)
    sizes, common = g.integers(0, 4, 1024), g.integers(0, 200, 1024)
    groups = [(int(n), int(t), (lambda t: lambda j: t + j % 3)(int(t))) for n, t in zip(sizes, common)]
    Batch(scute, g, groups, 1, 2, 64, 16, "bf16", behind=4).run(contexts["bf16"])


def test_shared_most_requests(scute, contexts):
    g = np.random.default_rng(16384)
    Batch(scute, g, [(16000, 50, lambda j: 50 + j % 3), (300, 20, lambda j: 20)], 1, 2, 64, 16, "bf16", behind=84).run(contexts["bf16"])


def test_shared_nothing(scute, contexts):
    """No groups, no requests, groups without requests, lengths of zero."""
    ctx, g = contexts["bf16"], np.random.default_rng(0)
    b = Batch(scute, g, [(4, 0, lambda j: 30 + j)], 2, 4, 64, 16, "bf16", before=3)
    b.run(ctx)
    b.start, b.shared = [3], []
    b.run(ctx)
    b.start, b.shared = [0, 0, 7, 7], [50, 0, 12]
    b.run(ctx)
    empty = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda")
    ctx.paged_attention(b.cache, empty, i32([]), empty, shared=scute.Shared(i32([0, 0]), i32([5]), ctx.shared_work(b.cache, 0, 8), always=True))
    assert ctx.sync_status() == 0


def test_shared_strided_in_place_on_another_stream_without_lse(scute, contexts):
    ctx, g = contexts["bf16"], np.random.default_rng(11)
    b = Batch(scute, g, [(5, 300, lambda j: 300 + 11 * j)], 2, 4, 128, 16, "bf16", behind=1)
    out, lse = b.run(ctx)
    n = b.q.shape[0]
    wide = torch.randn(n, 8 + 8 + 4, 128, device="cuda").bfloat16()
    rest = wide.clone()
    q = wide[:, 8:16]
    q.copy_(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens, sh = i32(b.lens), scute.Shared(i32(b.start), i32(b.shared), ctx.shared_work(b.cache, n, 8), always=True)
    with torch.cuda.stream(s):
        ctx.paged_attention(b.cache, q, lens, q, shared=sh)
    s.synchronize()
    assert torch.equal(q, out)
    rest[:, 8:16] = out
    assert torch.equal(wide, rest)


def test_shared_graph_replay_with_other_lengths_and_groups(scute, contexts):
    ctx, g = contexts["bf16"], np.random.default_rng(12)
    b = Batch(scute, g, [(4, 320, lambda j: 320 + 40 * j), (3, 160, lambda j: 200 + j)], 2, 4, 128, 16, "bf16")
    n, full = 7, list(b.lens)
    lens, start, common = i32(full), i32(b.start), i32(b.shared)
    sh = scute.Shared(start, common, ctx.shared_work(b.cache, n, 8), always=True)
    out, lse = torch.empty_like(b.q), torch.empty(n, 8, device="cuda")
    ctx.paged_attention(b.cache, b.q, lens, out, lse=lse, shared=sh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ctx.paged_attention(b.cache, b.q, lens, out, lse=lse, shared=sh)
    for now, at, t in ((full, b.start, b.shared), ([320, 0, 350, 16, 160, 201, 0], b.start, [96, 160]),
                       (full, [1, 4, 4], [320, 9]), ([5] * 7, b.start, [320, 160])):
        lens.copy_(i32(now))
        start.copy_(i32(at))
        common.copy_(i32(t))
        out.fill_(float("nan"))
        graph.replay()
        assert ctx.sync_status() == 0
        check_attend(out, lse, b.q, [(k[:x], v[:x]) for (k, v), x in zip(b.tokens, now)], "bf16", 4)


def test_shared_out_of_range_is_recorded(scute, contexts):
    """Starts, lengths and pages outside: nothing is read out of range, the status says
    so, and what lies outside counts as the nearest inside."""
    ctx, g = contexts["bf16"], np.random.default_rng(5)
    b = Batch(scute, g, [(4, 320, lambda j: 320 + 40 * j)], 2, 4, 64, 16, "bf16", behind=2)
    n, cap = 6, b.table.shape[1] * 16
    out, lse, lens = torch.empty_like(b.q), torch.empty(n, 8, device="cuda"), i32(b.lens)

    def run(start, common, cache=b.cache, lens=lens):
        sh = scute.Shared(i32(start), i32(common), ctx.shared_work(cache, n, 8), always=True)
        ctx.paged_attention(cache, b.q, lens, out, lse=lse, shared=sh)
        return ctx.sync_status()

    assert run([-3, 4], [320]) == PAGES
    check_attend(out, lse, b.q, b.tokens, "bf16", 4)
    assert run([0, 4, 99], [320, -5]) == PAGES
    check_attend(out, lse, b.q, b.tokens, "bf16", 4)
    assert run([0, 4], [cap + 1000]) == PAGES            # nobody has so many: attended alone
    check_attend(out, lse, b.q, b.tokens, "bf16", 4)
    for falling in ([4, 0], [0, 5, 2], [6, 6, 0, 6]):
        assert run(falling, [320] * (len(falling) - 1)) == PAGES
    # a page of the shared tokens outside the pool: its tokens are left out, for all
    table = b.table.clone()
    table[:4, 3] = 10 ** 6
    assert run([0, 4], [320], scute.KvCache(*b.cache.tensors[:2], table)) == PAGES
    left = [(np.delete(k, slice(48, 64), 0), np.delete(v, slice(48, 64), 0)) for k, v in b.tokens[:4]] + b.tokens[4:]
    check_attend(out, lse, b.q, left, "bf16", 4)
    # a length beyond the table
    long = i32([cap + 5] + b.lens[1:])
    assert run([1, 4], [320], lens=long) == PAGES
    check_attend(out[1:], lse[1:], b.q[1:], b.tokens[1:], "bf16", 4)
    assert run([0, 4], [320]) == 0
    check_attend(out, lse, b.q, b.tokens, "bf16", 4)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_shared_offsets_beyond_32_bits(scute, contexts, kind):
    """Pages whose elements lie beyond 2^32 in the pool."""
    ctx, g = ctx_of(contexts, kind), np.random.default_rng(6)
    H, page, D, pages = 1, 16, 64, 9
    stride = (1 << 29) + 1024
    dt = DT[kind]
    tok = torch.from_numpy(g.standard_normal((2, pages, H, page, D), dtype=np.float32)).to(dt)
    flat = [torch.zeros(stride * (pages - 1) + H * page * D, dtype=torch.uint8 if kind == "fp8" else dt, device="cuda") for _ in range(2)]
    pools = [f.view(dt).as_strided((pages, H, page, D), (stride, page * D, D, 1)) for f in flat]
    for p, t in zip(pools, tok):
        (p.view(torch.uint8) if kind == "fp8" else p).copy_((t.view(torch.uint8) if kind == "fp8" else t).cuda())
    table = i32([[8, 7, 6, 5, 4], [8, 7, 6, 5, 3]])
    cache, lens = scute.KvCache(*pools, table), i32([70, 80])
    q = torch.from_numpy(g.standard_normal((2, 4, D), dtype=np.float32)).cuda().bfloat16()
    out, lse = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    ctx.paged_attention(cache, q, lens, out, lse=lse, shared=scute.Shared(i32([0, 2]), i32([64]), ctx.shared_work(cache, 2, 4), always=True))
    assert ctx.sync_status() == 0
    kk, vv = f64(tok[0]), f64(tok[1])
    tokens = [(np.concatenate([kk[p].transpose(1, 0, 2) for p in row])[:n], np.concatenate([vv[p].transpose(1, 0, 2) for p in row])[:n])
              for row, n in zip(table.cpu().tolist(), (70, 80))]
    check_attend(out, lse, q, tokens, kind, 4)
    # a page of each pool copied there and back
    caches = scute.KvCaches([scute.KvCache(*pools)])
    ctx.kv_copy(caches, i32([8, 0]), i32([1, 2]))
    assert ctx.sync_status() == 0
    for p in pools:
        p = p.view(torch.uint8) if kind == "fp8" else p
        assert torch.equal(p[1], p[8]) and torch.equal(p[2], p[0])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("D,group", [(64, 1), (64, 16), (128, 4)])
def test_shared_keeps_the_bits_of_its_weights(scute, contexts, kind, D, group):
    """As in the one-token attention's test: two tokens of values +1 and -1 with scores s
    and 0, both shared, or one of them the request's own.  What is left beside the output's
    rounding: 2^-20 of exponent, exponential, sums and division, and 2^-17 of a weight's
    two bf16 parts (with an e4m3 cache too: its keys and values become bf16 ones here)."""
    g = np.random.default_rng(D + group)
    n, ctx = 40, contexts["bf16"]
    k, v = torch.zeros(2, 1, 1, D), torch.zeros(2, 1, 1, D)
    k[0, 0, 0, D // 2], v[0], v[1] = 1.0, 1.0, -1.0
    cache = scute.KvCache(k.to(DT[kind]).cuda(), v.to(DT[kind]).cuda(), i32(np.tile([0, 1], (n, 1))))
    s = (2.0 ** g.uniform(-11, -8, (n, group)) * g.choice([-1.0, 1.0], (n, group))).astype(np.float32)
    q = torch.zeros(n, group, D)
    q[:, :, D // 2] = torch.from_numpy(s)
    q = q.bfloat16().cuda()
    ref = np.tanh(f64(q)[:, :, D // 2] / 2)[:, :, None]
    for common in (2, 1):
        out = torch.empty_like(q)
        ctx.paged_attention(cache, q, i32([2] * n), out, scale=1.0,
                            shared=scute.Shared(i32([0, n]), i32([common]), ctx.shared_work(cache, n, group), always=True))
        assert ctx.sync_status() == 0
        err = np.abs(f64(out) - ref)
        assert np.all(err <= 2.0 ** -20 + 2.0 ** -17 + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_shared_long_tail_of_small_weights(scute, contexts, kind):
    """One token 2^26 times as heavy as each of 20000 others, whose sum still counts."""
    n, L, D, ctx = 70, 20000, 64, contexts["bf16"]
    k, v = torch.zeros(L // 16, 1, 16, D), torch.ones(L // 16, 1, 16, D)
    k[0, 0, 0], v[0, 0, 0] = 1.5, 0.0
    cache = scute.KvCache(k.to(DT[kind]).cuda(), v.to(DT[kind]).cuda(), i32(np.tile(np.arange(L // 16), (n, 1))))
    q = torch.full((n, 1, D), 1.5, device="cuda").bfloat16()
    out, lse = torch.empty_like(q), torch.empty(n, 1, device="cuda")
    ctx.paged_attention(cache, q, i32([L] * n), out, lse=lse, shared=scute.Shared(i32([0, n]), i32([L - 8]), ctx.shared_work(cache, n, 1), always=True))
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, [(f64(k).reshape(-1, 1, D), f64(v).reshape(-1, 1, D))] * n, kind, 1)


@pytest.mark.parametrize("kind,D,n", [("bf16", 128, 3), ("bf16", 64, 50), ("fp8", 128, 40)])
def test_shared_whose_waits_run_out_reports_and_recovers(scute, contexts, kind, D, n):
    """A call whose slots of keys are never given back (test hook): its waits end after
    2 s, the status says so, and the next call is right."""
    ctx, g = contexts["bf16"], np.random.default_rng(D)
    b = Batch(scute, g, [(n, 150000 if D == 64 else 80000, lambda j: (150000 if D == 64 else 80000) + j)], 2, 4, D, 16, kind)
    work = ctx.shared_work(b.cache, n, 8)
    sh = scute.Shared(i32(b.start), i32(b.shared), work, always=True)
    out, lens = torch.empty_like(b.q), i32(b.lens)
    scute.scute_debug_inject(ctx.handle, scute.INJECT_STALL_ATTENTION)
    t0 = time.time()
    ctx.paged_attention(b.cache, b.q, lens, out, shared=sh)
    assert ctx.sync_status() == 7                  # SCUTE_ERR_TIMEOUT
    assert 0.5 < time.time() - t0 < 60.0
    a, lse = torch.empty_like(out), torch.empty(n, 8, device="cuda")
    ctx.paged_attention(b.cache, b.q, lens, a, lse=lse, shared=sh)
    assert ctx.sync_status() == 0
    check_attend(a[:3], lse[:3], b.q[:3], b.tokens[:3], kind, 4)


def test_shared_refusals(scute, contexts):
    ctx, g = contexts["bf16"], np.random.default_rng(0)
    b = Batch(scute, g, [(3, 32, lambda j: 40)], 2, 4, 64, 16, "bf16")
    work = ctx.shared_work(b.cache, 3, 8)
    lens, out = i32(b.lens), torch.empty_like(b.q)
    good = scute.Shared(i32(b.start), i32(b.shared), work, always=True)
    ctx.paged_attention(b.cache, b.q, lens, out, shared=good)
    bad = [lambda: ctx.paged_attention(b.cache, b.q, lens, out, shared=good, window=8),
           lambda: ctx.paged_attention(b.cache, b.q, lens, out, shared=good, sinks=3),
           lambda: ctx.paged_attention(b.cache, b.q, lens, out, shared=scute.Shared(i32(b.start), i32(b.shared), work[:-32], always=True)),
           lambda: ctx.paged_attention(b.cache, b.q, lens, out, shared=scute.Shared(i32(b.start), i32(b.shared), work[8:], always=True)),
           lambda: ctx.paged_attention(b.cache, b.q, lens, out, shared=scute.Shared(i32([0] * 1026), i32([0] * 1025), work, always=True)),
           lambda: scute.Shared(i32(b.start), i32([1, 2]), work, always=True), lambda: scute.Shared(i32(b.start).float(), i32(b.shared), work, always=True),
           lambda: scute.Shared(i32(b.start), i32(b.shared).long(), work, always=True), lambda: scute.Shared(i32([0, 1, 2, 3])[::3], i32([1]), work, always=True),
           lambda: scute.Shared(i32(b.start), i32(b.shared), work[::2], always=True),
           lambda: ctx.shared_work(b.cache, 16385, 8), lambda: ctx.shared_work(b.cache, -1, 8), lambda: ctx.shared_work(b.cache, 3, 7)]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, scute.ScuteError)):
            call()
            raise AssertionError(i)
    ctx.paged_attention(b.cache, b.q, lens, out, shared=good)
    assert ctx.sync_status() == 0


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("all_shared", [True, False])
def test_shared_as_many_tokens_as_a_row_may_have(scute, contexts, kind, all_shared):
    """A row of almost 2^30 tokens, all of one page of 127 tokens, shared or the request's own.
    Every score is 0 and every value of an element the same power of two, so that a CTA's
    or warp's sums are whole multiples of it (fewer than 2^24) and exact; the at most 2500
    parts add up in 32 bits, 2500 x 2^-24 < 2^-12 off at most, and the quotient, that far
    from a power of two, rounds to it (2^-9 or more)."""
    page, D = 127, 16
    cols = 2 ** 30 // page
    n = page * cols
    as_kv = lambda x: x.expand(1, 1, page, D).contiguous().to(DT[kind])  # noqa: E731
    v = 2.0 ** (torch.arange(D, device="cuda") % 5 - 2)
    cache = scute.KvCache(as_kv(torch.zeros(D, device="cuda")), as_kv(v), torch.zeros(1, cols, dtype=torch.int32, device="cuda"))
    ctx = contexts["bf16"]
    q, lse = torch.ones(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 2, device="cuda")
    out = torch.full_like(q, float("nan"))
    sh = scute.Shared(i32([0, 1]), i32([n if all_shared else 0]), ctx.shared_work(cache, 1, 2), always=True)
    ctx.paged_attention(cache, q, i32([n]), out, lse=lse, shared=sh)
    assert ctx.sync_status() == 0
    assert torch.equal(out, v.bfloat16().expand(1, 2, D))
    assert np.allclose(lse.cpu().numpy(), np.log(n), rtol=0, atol=1e-4)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H", [(3, 400), (1, 2600)])
def test_shared_many_heads(scute, contexts, kind, n, H):
    """More key/value heads than the requests' own tokens have warps for."""
    g = np.random.default_rng([n, H])
    Batch(scute, g, [(n, 40, lambda j: 300 + 50 * j)], H, 1, 16, 16, kind, scales=kind == "fp8").run(contexts["bf16"])


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_shared_only_where_it_saves(scute, contexts, kind):
    """Groups on both sides of what is read together: by tokens, by requests, by both."""
    g = np.random.default_rng(4)
    sizes = [(9, 127), (9, 128), (8, 146), (8, 147), (2, 1023), (2, 1024), (1, 3000), (12, 255), (12, 256), (11, 255), (11, 256), (4, 2047),
             (4, 2048), (3, 5000), (30, 400)]
    b = Batch(scute, g, [(n, t, (lambda t: lambda j: t + 7 * j - (j == 2))(t)) for n, t in sizes], 1, 4, 64, 16, kind, before=1, behind=2)
    for always in (False, True):
        b.run(contexts["bf16"], always=always)


@pytest.mark.parametrize("kind,H,group,D", [("fp32", 2, 4, 64), ("bf16", 1, 2, 256), ("fp8", 2, 2, 192), ("bf16", 1, 130, 32)])
def test_shared_out_of_range_is_recorded_whatever_reads_the_cache(scute, contexts, kind, H, group, D):
    """Starts and lengths outside are recorded for caches whose requests are read one by one, too."""
    ctx, g = ctx_of(contexts, kind), np.random.default_rng(5)
    b = Batch(scute, g, [(4, 320, lambda j: 320 + 40 * j)], H, group, D, 16, kind, behind=2)
    n, cap, lens = 6, b.table.shape[1] * 16, i32(b.lens)
    out, lse = torch.empty_like(b.q), torch.empty(n, H * group, device="cuda")
    work = ctx.shared_work(b.cache, n, H * group)

    def run(start, common, always=True):
        ctx.paged_attention(b.cache, b.q, lens, out, lse=lse, shared=scute.Shared(i32(start), i32(common), work, always=always))
        return ctx.sync_status()

    many = [0] + [4] * 300
    for start, common in (([-3, 4], [320]), ([0, 4, 99], [320, 5]), ([0, 4], [-5]), ([0, 4], [cap + 1]), ([4, 0], [320]), ([0, 5, 2], [320, 1]),
                          ([6, 6, 0, 6], [1, 1, 1]), (many, [320] * 299 + [cap + 1]), (many[:-1] + [3], [320] * 300), ([7], [])):
        for always in (True, False):
            assert run(start, common, always) == (PAGES if common else 0)      # (no groups: nothing is read of them)
            check_attend(out, lse, b.q, b.tokens, kind, group)
    for start, common in (([0, 4], [320]), ([0, 6], [cap]), ([2, 2, 4], [0, 9]), (many, [320] * 300), ([6, 6], [cap])):
        assert run(start, common) == 0
    check_attend(out, lse, b.q, b.tokens, kind, group)
    # the numbers are those of the call's place on the stream, changed before and after it
    start, common = i32([0, 4]), i32([cap + 7])
    sh = scute.Shared(start, common, work)
    for _ in range(20):
        common.fill_(320)
        ctx.paged_attention(b.cache, b.q, lens, out, lse=lse, shared=sh)
        common.fill_(cap + 7)
    assert ctx.sync_status() == 0
    ctx.paged_attention(b.cache, b.q, lens, out, lse=lse, shared=sh)
    common.fill_(320)
    assert ctx.sync_status() == PAGES


@pytest.mark.parametrize("kind,group,D", [("fp8", 2, 64), ("bf16", 4, 128), ("fp8", 9, 128)])
def test_shared_most_requests_of_wide_heads(scute, contexts, kind, group, D):
    """The list of the most requests beside the rings of wide heads: one CTA on an SM with rings of five tiles,
    and (e4m3, heads of 64) two with rings of two."""
    g = np.random.default_rng([16384, D])
    Batch(scute, g, [(16000, 30, lambda j: 30 + j % 3), (300, 20, lambda j: 20)], 1, group, D, 16, kind, behind=84).run(contexts["bf16"])
