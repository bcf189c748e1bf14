"""The cache's operators together, as a server that branches uses them: prompts written
with normed heads, samples forked off them, beams chosen again and again, requests that
end, each step's attention over what the rows of a prompt share, and the same contexts
read through a window with first tokens.  Graded step by step against a float64 model
that keeps every sequence's keys and values whole."""
import numpy as np
import pytest

from oracle import block_ops as OB
from test_gpu_block_ops import check_attend, f64, i32

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def scute(gpu_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return gpu_lib


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_prompts_samples_and_beams(scute, kind):
    g = np.random.default_rng(2)
    prompts, width, H, group, D, page, layers, steps = [150, 31, 64, 7], 5, 2, 4, 64, 16, 2, 12
    n, heads, io = len(prompts) * width, H * group, torch.bfloat16 if kind == "bf16" else torch.float32
    total, cols = 220, 20
    ctx = scute.Context(dtype=kind, max_tokens=64, max_adapters=1, max_layers=1)
    whole = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = [[torch.full((total, H, page, D), float("nan"), dtype=io, device="cuda") for _ in range(2)] for _ in range(layers)]
    tables = [whole(n, cols) - 1, whole(n, cols) - 1]
    views = [[scute.KvCache(*p, t) for p in pools] for t in tables]
    all_layers = scute.KvCaches(views[0])
    length = [whole(n), whole(n)]
    extra, free, count = whole(total), torch.arange(total, dtype=torch.int32, device="cuda"), whole(1) + total
    cf, ct, cn, cu = whole(n), whole(n), whole(n), whole(n + 1)
    cs = torch.empty(512, D, device="cuda")
    ctx.rope_table(cs, 10000.0)
    freq = 10000.0 ** (-np.arange(D // 2) / (D // 2))
    qw, kw = (torch.from_numpy(1 + 0.2 * g.standard_normal(D, dtype=np.float32)).cuda() for _ in range(2))
    norm = scute.HeadNorm(qw, kw, eps=1e-6)
    seqs = [[([], []) for _ in range(layers)] for _ in range(n)]        # of each row and layer: keys, values

    def draw(*s):
        return torch.from_numpy(g.standard_normal(s, dtype=np.float32)).to(io).cuda()

    def write(at, rows, want):
        """Tokens for the rows whose length grows to `want`; their queries (last layer's)."""
        slots, pos, req = whole(rows), whole(rows), whole(rows)
        ctx.kv_resize(length[at], i32(want), tables[at], page, free, count, count, length[at], cu, slots, pos, req)
        out = []
        for i in range(layers):
            q, k, v = draw(rows, heads, D), draw(rows, H, D), draw(rows, H, D)
            qr = torch.empty_like(q)
            ctx.kv_append(views[at][i], slots, k, v, q=q, q_out=qr, rope=scute.Rope(cs, pos), norm=norm)
            kk = OB.head_norm(f64(k), f64(kw), 1e-6, False)
            for row, (p, r) in enumerate(zip(pos.tolist(), req.tolist())):
                if r >= 0:
                    seqs[r][i][0].append(OB.rope(kk[row], p * freq, D, False))
                    seqs[r][i][1].append(f64(v[row]))
            out.append(qr)
        assert ctx.sync_status() == 0
        return out, req.tolist()

    # the cached keys are rounded: the model takes what the cache holds, after checking it
    def held(at, r, i):
        row, m = tables[at][r].cpu().numpy(), len(seqs[r][i][0])
        got = [np.concatenate([f64(p[int(b)]).transpose(1, 0, 2) for b in row[:-(-m // page)]])[:m] if m else np.zeros((0, H, D))
               for p in pools[i]]
        if m:
            k, v = np.stack(seqs[r][i][0]), np.stack(seqs[r][i][1])
            half = 2.0 ** -8 if kind == "bf16" else 2.0 ** -24
            # a normed and turned key: (D / 2 + 8) u of the factor, 5 u of turning, on elements up to the pair's size
            size = np.abs(k) + np.abs(np.concatenate([k[..., D // 2:], k[..., :D // 2]], -1))
            assert np.all(np.abs(got[0] - k) <= half * np.abs(k) * 1.01 + 2.0 ** -24 * (D + 20) * size)
            assert np.array_equal(got[1], v)
        return got

    def attend(at, q, i, groups):
        """One query of every row over its context: groups of (first row, rows, shared tokens)."""
        start = [0] + [a + m for a, m, _ in groups]
        sh = scute.Shared(i32(start), i32([t for _, _, t in groups]), ctx.shared_work(views[at][i], n, heads), always=True)
        out, lse = torch.full_like(q, float("nan")), torch.empty(n, heads, device="cuda")
        ctx.paged_attention(views[at][i], q, length[at], out, lse=lse, shared=sh)
        tokens = [held(at, r, i) for r in range(n)]
        check_attend(out, lse, q, tokens, kind, group)
        ctx.paged_attention(views[at][i], q, length[at], out, lse=lse, window=40, sinks=5)
        check_attend(out, lse, q, [[x[OB.seen(len(x), 40, 5)] for x in kv] for kv in tokens], kind, group)
        assert ctx.sync_status() == 0

    def branch(at, source, new):
        """Rows of the other table that continue these; the model's likewise."""
        to = 1 - at
        ctx.kv_fork(tables[at], length[at], i32(source), tables[to], length[to], page, extra, free, count, count, cf, ct, cn,
                    len_new=i32(new))
        ctx.kv_copy(all_layers, cf, ct, cn)
        assert ctx.sync_status() == 0 and length[to].tolist() == list(new)
        seqs[:] = [[([*k[:m]], [*v[:m]]) for k, v in (seqs[s] if s >= 0 else [((), ())] * layers)] for s, m in zip(source, new)]
        return to

    # prompts in the rows 0, width, 2 width, ..., then every row a sample of its prompt
    want = np.zeros(n, np.int64)
    want[::width] = prompts
    write(0, sum(prompts) + 3, want)
    source = np.repeat(np.arange(len(prompts)) * width, width)
    at = branch(0, source, np.repeat(prompts, width))
    alive = np.ones(len(prompts), bool)
    for step in range(steps):
        have = np.array(length[at].tolist())
        groups = [(p * width, width, prompts[p] // page * page) for p in range(len(prompts))]
        q, _ = write(at, n, have + np.repeat(alive, width))
        rows = np.full((n,), -1)
        rows[np.repeat(alive, width)] = np.arange(alive.sum() * width)
        qq = draw(n, heads, D)
        qq[torch.from_numpy(rows >= 0)] = q[-1][torch.from_numpy(rows[rows >= 0])]
        attend(at, qq, layers - 1, groups)
        if step == 5:
            alive[1] = False                              # a prompt's samples end
        have = np.array(length[at].tolist())
        source = np.repeat(np.arange(len(prompts)) * width, width) + g.integers(0, width, n)
        source[~np.repeat(alive, width)] = -1
        new = np.where(source >= 0, have[source], 0)
        if step % 4 == 3:                                 # and some give their last tokens back
            new[::3] = np.maximum(new[::3] - 2, 0)
        at = branch(at, source, new)
    # everything is let go: every page is free again, once
    at = branch(at, np.full(n, -1), np.zeros(n, np.int64))
    assert int(count) == total and sorted(free.tolist()) == list(range(total)) and not extra.any()
    ctx.close()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_captured_steps_of_two_contexts_at_once(scute, kind):
    """A step of beams (fork, copy, growth, normed append, shared and windowed attention) captured as a graph for
    each of two contexts, both replayed on streams of their own at the same time, on other choices and lengths
    each time: the bits of the same steps run one after the other without a graph."""
    g = np.random.default_rng(6)
    prompts, width, H, group, D, page, cols, total, steps = [500, 77, 16, 901], 5, 2, 4, 64, 16, 80, 700, 6
    n, heads = len(prompts) * width, H * group
    whole = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    cs = torch.empty(2048, D, device="cuda")
    # prompts in whole pages: every row's table begins with them
    table0, length0, extra0, at = np.full((n, cols), -1), np.repeat(prompts, width), np.zeros(total, np.int64), 0
    for p, m in enumerate(prompts):
        k = m // page
        table0[p * width:(p + 1) * width, :k] = np.arange(at, at + k)
        extra0[at:at + k], at = width - 1, at + k
        if m % page:
            for r in range(p * width, (p + 1) * width):
                table0[r, k], at = at, at + 1
    free0 = np.pad(np.arange(at, total), (0, at))
    pool0 = [torch.randn(total, H, page, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).bfloat16() for i in range(2)]
    choices = [(np.repeat(np.arange(len(prompts)) * width, width) + g.integers(0, width, n)).astype(np.int64) for _ in range(steps)]
    start = i32(np.arange(len(prompts) + 1) * width)
    common = i32([m // page * page for m in prompts])
    w = torch.rand(D, device="cuda") + 0.5

    class Server:
        def __init__(self, seed):
            self.ctx = scute.Context(dtype="bf16", max_tokens=64, max_adapters=1, max_layers=1)
            self.ctx.rope_table(cs, 10000.0)
            self.pools = [x.clone() if kind == "bf16" else x.to(torch.float8_e4m3fn) for x in pool0]
            self.tables, self.length = [i32(table0), whole(n, cols) - 1], [i32(length0), whole(n)]
            self.extra, self.free, self.count = i32(extra0), i32(free0), i32([total - at])
            self.cache = [scute.KvCache(*self.pools, t) for t in self.tables]
            self.both = scute.KvCaches([self.cache[0]])
            self.vec, self.cu, self.one = [whole(n) for _ in range(7)], whole(n + 1), whole(n) + 1
            gen = torch.Generator(device="cuda").manual_seed(seed)
            self.q, self.k, self.v = (torch.randn(n, h, D, device="cuda", generator=gen).bfloat16() for h in (heads, H, H))
            self.qr, self.out, self.win = (torch.zeros(n, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
            self.lse = torch.zeros(n, heads, device="cuda")
            self.source, self.want = whole(n), whole(n)
            self.shared = [scute.Shared(start, common, self.ctx.shared_work(c, n, heads), always=True) for c in self.cache]
            self.rope, self.norm = scute.Rope(cs, self.vec[5]), scute.HeadNorm(w, w)

        def half(self, a):
            b, ctx, (cf, ct, cn, slots, new, pos, req) = 1 - a, self.ctx, self.vec
            ctx.kv_fork(self.tables[a], self.length[a], self.source, self.tables[b], self.length[b], page, self.extra, self.free, self.count,
                        self.count, cf, ct, cn)
            ctx.kv_copy(self.both, cf, ct, cn)
            torch.add(self.length[b], self.one, out=self.want)
            ctx.kv_resize(self.length[b], self.want, self.tables[b], page, self.free, self.count, self.count, self.length[b], self.cu, slots,
                          pos, req)
            ctx.kv_append(self.cache[b], slots, self.k, self.v, q=self.q, q_out=self.qr, rope=self.rope, norm=self.norm)
            ctx.paged_attention(self.cache[b], self.qr, self.length[b], self.out, lse=self.lse, shared=self.shared[b])
            ctx.paged_attention(self.cache[b], self.qr, self.length[b], self.win, window=60, sinks=5)

        def seen(self):
            return [x.clone() for x in (self.out, self.lse, self.win, *self.length, self.extra, self.count, *(p.view(torch.uint8) for p in self.pools))]

    def advance(s, i):
        s.source.copy_(i32(choices[i]))

    plain = [Server(s) for s in (1, 2)]
    want = [[], []]
    for i in range(steps):
        for j, s in enumerate(plain):
            advance(s, i)
            s.half(i % 2)
            want[j].append(s.seen())
            assert s.ctx.sync_status() == 0
    servers, streams = [Server(s) for s in (1, 2)], [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for s in servers:
        pair = []
        for a in (0, 1):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.half(a)
            pair.append(graph)
        graphs.append(pair)
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(steps):
        for s in servers:
            advance(s, i)
        torch.cuda.synchronize()
        for s, pair, stream in zip(servers, graphs, streams):
            with torch.cuda.stream(stream):
                pair[i % 2].replay()
        torch.cuda.synchronize()
        for j, s in enumerate(servers):
            got[j].append(s.seen())
            assert s.ctx.sync_status() == 0
    for j in range(2):
        for x, y in zip(got[j], want[j]):
            assert all(torch.equal(p, q) for p, q in zip(x, y))
    assert not torch.equal(got[0][-1][0], got[1][-1][0])
    for s in plain + servers:
        s.ctx.close()
