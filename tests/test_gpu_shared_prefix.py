"""One-token attention of groups of requests that share the beginnings of their
contexts, on the GPU against the float64 definition of each request's attention over
all of its tokens (``oracle/block_ops.py``).  Tolerances are those of the one-token
attention (``check_attend``): a score's sum over D products, the sums over L tokens and the
roundings of weights and outputs are the same, however the tokens are shared out."""
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

    def run(self, ctx, times=2, **kw):
        n, heads = self.q.shape[:2]
        work = ctx.shared_work(self.cache, n, heads)
        work.fill_(255)                                   # not a number, whatever is read of it
        sh = self.scute.Shared(i32(self.start), i32(self.shared), work)
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
