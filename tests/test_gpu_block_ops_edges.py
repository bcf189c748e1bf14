"""The decoder block's operators where they can go wrong without a large error:
cache slots that a page number cannot form, joins whose grouping must not depend
on which CTA comes last, weights rounded to fewer bits, waits that run out.
Definitions and bounds as in ``test_gpu_block_ops.py``."""
import numpy as np
import pytest

from test_gpu_block_ops import PAGES, i32

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
