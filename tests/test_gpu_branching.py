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
