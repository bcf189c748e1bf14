"""The decoder block's operators where they can go wrong without a large error:
cache slots that a page number cannot form, joins whose grouping must not depend
on which CTA comes last, weights rounded to fewer bits, waits that run out.
Definitions and bounds as in ``test_gpu_block_ops.py``."""
import time

import numpy as np
import pytest

from test_gpu_block_ops import DT, HB, PAGES, U, check_attend, ctx_of, f64, i32, make_cache

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TIMEOUT = 7      # SCUTE_ERR_TIMEOUT


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


# ---------------------------------------------------------------- slots
NO_SLOT = -2 ** 31      # where a page number forms no slot


@pytest.mark.parametrize("page,old,new,entries,free,want", [
    # the last token of a page that the table has as -1: -1 * 16 + 15 is the mark of "no slot"
    (16, 15, 16, [-1], [], [NO_SLOT]),
    (1, 2, 3, [4, 5], [-1], [NO_SLOT]),
    # a product beyond 32 bits wraps to another request's slot
    (16, 14, 17, [1 << 28], [7], [NO_SLOT, NO_SLOT, 7 * 16]),
    (16, 0, 2, [], [(1 << 28) + 1], [NO_SLOT, NO_SLOT]),
    (7, 6, 8, [-3], [613566757], [NO_SLOT, NO_SLOT]),
    # the largest slots there are
    (16, 15, 17, [(1 << 27) - 1], [0], [2 ** 31 - 1, 0]),
    (1, 0, 1, [], [2 ** 31 - 1], [2 ** 31 - 1])])
def test_resize_pages_that_form_no_slot_are_recorded(scute, contexts, page, old, new, entries, free, want):
    """Beside two sound requests, whose slots stay what they were."""
    ctx, cols = contexts["bf16"], 20
    table = np.full((3, cols), -1, np.int32)
    table[0, 0], table[2, 0] = 2, 3
    table[1, :len(entries)] = entries
    first = 1 if page > 1 else 0            # the sound ones grow inside their page, or keep still
    lens = [first, old, first]
    more = [1 if page > 1 else 0, new - old, 1 if page > 1 else 0]
    t = {k: i32(v) for k, v in dict(old=lens, new=np.add(lens, more), table=table, free=free + [0] * 4, free_in=[len(free)],
                                    free_out=[0], out=[0] * 3, cu=[0] * 4, slot=[-9] * 8, pos=[0] * 8, req=[0] * 8).items()}
    ctx.kv_resize(t["old"], t["new"], t["table"], page, t["free"], t["free_in"], t["free_out"], t["out"], t["cu"],
                  t["slot"], t["pos"], t["req"])
    status = ctx.sync_status()
    sound = [[2 * page + 1], [3 * page + 1]] if page > 1 else [[], []]
    rows = sound[0] + want + sound[1]
    assert t["slot"].tolist() == rows + [-1] * (8 - len(rows))
    assert t["out"].tolist() == np.add(lens, more).tolist()
    assert status == (PAGES if NO_SLOT in want else 0)


def test_append_skips_and_records_what_forms_no_slot(scute, contexts):
    ctx = contexts["bf16"]
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    pools = [torch.zeros(2, 2, 4, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    ctx.kv_append(scute.KvCache(*pools), i32([NO_SLOT, 5]), x, x)
    assert ctx.sync_status() == PAGES
    for p in pools:
        assert p[1, :, 1].eq(1).all() and p.sum() == 128


# ---------------------------------------------------------------- joins
@pytest.mark.parametrize("kind,D,group,H", [("fp32", 128, 12, 4), ("fp32", 128, 9, 4), ("bf16", 256, 12, 2), ("bf16", 128, 20, 2),
                                            ("fp8", 128, 20, 2), ("bf16", 128, 4, 4)])
def test_shared_rows_of_unequal_head_chunks_give_the_same_bits(scute, contexts, kind, D, group, H):
    """A group that is no multiple of the heads taken at a time has rows of two
    sizes.  Rows of about 13 parts do not fit the join's memory at once in the
    larger size: how their parts are grouped may depend on the row alone, not on
    which CTA happened to be last for it and what else that one had to join."""
    g = np.random.default_rng(group + D)
    lens = [4003, 4511, 5000, 5520, 6007, 4750]
    cache, tokens = make_cache(scute, g, lens, H, D, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((len(lens), H * group, D), dtype=np.float32) * 2)
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    ctx, at = ctx_of(contexts, kind), i32(lens)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx.paged_attention(cache, q, at, out, lse=lse)
    assert ctx.sync_status() == 0
    check_attend(out, lse, q, tokens, kind, group)
    outs, lses = [torch.empty_like(out) for _ in range(200)], [torch.empty_like(lse) for _ in range(200)]
    side = torch.zeros(1 << 26, device="cuda")
    for i, (o, s) in enumerate(zip(outs, lses)):
        if i % 2:
            side.add_(1.0)             # another state of the L2, another order of arrival
        ctx.paged_attention(cache, q, at, o, lse=s)
    for o, s in zip(outs, lses):
        assert torch.equal(o, out) and torch.equal(s, lse)


# ---------------------------------------------------------------- waits
@pytest.mark.parametrize("kind,D,group", [("bf16", 128, 4), ("bf16", 128, 16), ("fp8", 64, 4), ("fp32", 128, 4), ("bf16", 256, 8)])
def test_attention_whose_waits_run_out_reports_and_recovers(scute, contexts, kind, D, group):
    """A launch whose stages are never given back (test hook): the fetching warps'
    waits and the computing warps' run out together, after 2 s.  The launch ends,
    the status says so, and the next call on the context is right."""
    g = np.random.default_rng(D)
    lens = [120000, 0, 5, 80000] if kind == "fp8" else [30000, 0, 5, 20000]     # beyond every ring
    cache, tokens = make_cache(scute, g, lens, 2, D, 16, kind, False)
    q = torch.from_numpy(g.standard_normal((len(lens), 2 * group, D), dtype=np.float32))
    q = q.cuda().to(DT["fp32" if kind == "fp32" else "bf16"])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    ctx = ctx_of(contexts, kind)
    scute.scute_debug_inject(ctx.handle, scute.INJECT_STALL_ATTENTION)
    t0 = time.time()
    ctx.paged_attention(cache, q, i32(lens), out, lse=lse)
    assert ctx.sync_status() == TIMEOUT
    assert 0.5 < time.time() - t0 < 60.0
    for _ in range(2):             # the hook was for that launch; counters are back at zero
        out.fill_(float("nan"))
        ctx.paged_attention(cache, q, i32(lens), out, lse=lse)
        assert ctx.sync_status() == 0
        check_attend(out, lse, q, tokens, kind, group)


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("kind", ["bf16", "fp8", "fp32"])
@pytest.mark.parametrize("D,group,page", [(64, 1, 16), (64, 16, 16), (128, 4, 16), (128, 16, 16), (128, 8, 1), (256, 8, 16)])
def test_attention_keeps_the_bits_of_its_weights(scute, contexts, kind, D, group, page):
    """Two tokens with values of +1 and -1 and scores s and 0: the output is
    tanh(s / 2), next to nothing for the s of 2^-11 to 2^-8 here, beside weights
    of a half each.  Queries and keys have one element that is not zero, so that
    the scores are exact but for one rounding each.  What is left:
      * the output's rounding, 2 h |ref| (none in fp32, 2 u |ref|);
      * a weight: its exponent (below 8) rounded to 2^-22 and hence ln 2 2^-22 of
        it, the exponential 2^-22, sums and the division 3 u, 2^-20 in all;
      * with a bf16 cache its two bf16 parts, 2^-17 (2^-9 had it one part; an
        e4m3 cache's two fp16 parts 2^-22 are inside the 2^-20, one part 2^-12 is not)."""
    g = np.random.default_rng(D + group)
    n = 40
    k, v = torch.zeros(2 if page == 1 else 1, 1, page, D), torch.zeros(2 if page == 1 else 1, 1, page, D)
    first, second = ((0, 0, 0), (1, 0, 0)) if page == 1 else ((0, 0, 0), (0, 0, 1))
    k[first][D // 2] = 1.0
    v[first], v[second] = 1.0, -1.0
    table = i32(np.tile(np.arange(k.shape[0]), (n, 1)))
    cache = scute.KvCache(k.to(DT[kind]).cuda(), v.to(DT[kind]).cuda(), table)
    io = DT["fp32" if kind == "fp32" else "bf16"]
    q = torch.zeros(n, group, D)
    s = (2.0 ** g.uniform(-11, -8, (n, group)) * g.choice([-1.0, 1.0], (n, group))).astype(np.float32)
    q[:, :, D // 2] = torch.from_numpy(s)
    q = q.to(io).cuda()
    out, lse = torch.empty_like(q), torch.empty(n, group, device="cuda")
    ctx = ctx_of(contexts, kind)
    ctx.paged_attention(cache, q, i32([2] * n), out, lse=lse, scale=1.0)
    assert ctx.sync_status() == 0
    ref = np.tanh(f64(q)[:, :, D // 2] / 2)[:, :, None]
    tol = 2.0 ** -20 + (2.0 ** -17 if kind == "bf16" else 0) + (2 * U if kind == "fp32" else 2 * HB) * np.abs(ref)
    err = np.abs(f64(out) - ref)
    assert np.all(err <= tol), float((err / tol).max())
