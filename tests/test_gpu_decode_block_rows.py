"""The example decoder's step when some requests take no token: they idle, have
ended, or are refused for want of pages.  ``kv_resize`` packs the step's rows, so
row i is then not request i's; every request's keys must still land in its own
pages.  Oracle and tolerance as in ``test_gpu_decode_block.py`` (fp32)."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_decode_block import SIZE, OracleDecoder  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block as DB  # noqa: E402

PAGES = 10     # SCUTE_ERR_PAGES


class Batch:
    """The oracle's requests, of which some take a token in a step."""

    def __init__(self, w, norms, n):
        self.ref, self.length = OracleDecoder(w, norms, SIZE), np.zeros(n, int)

    def step(self, x, takes):
        kept = {key: tuple(list(part) for part in pair) for key, pair in self.ref.cache.items()}
        out = self.ref.step(x, self.length)
        for (layer, r), pair in kept.items():
            if not takes[r]:
                self.ref.cache[layer, r] = pair
        self.length[takes] += 1
        return out


def close(got, want, t):
    rms = np.sqrt((want * want).mean())
    assert np.max(np.abs(got - want)) <= 1.7e-3 * 3 * rms, t
    assert np.sqrt(((got - want) ** 2).mean()) <= 1.7e-3 * rms, t


@pytest.mark.parametrize("graph", [False, True])
def test_idle_and_ended_requests_leave_the_others_right(gpu_lib, graph):
    n, page = 7, 4
    dec, w, norms = DB.build("fp32", requests=n, max_len=16, page_size=page, rank=8, rv=32, **SIZE)
    batch, g, run = Batch(w, norms, n), np.random.default_rng(3), None
    for t in range(11):
        x = g.standard_normal((n, SIZE["hidden"])).astype(np.float32)
        dec.x.copy_(torch.from_numpy(x).cuda())
        takes = g.random(n) < (1.0 if t == 0 else 0.6)
        if t == 4:
            takes[:] = False                           # a step in which no request takes one
        ends = ~takes & (g.random(n) < 0.3)
        dec.want.copy_(torch.from_numpy(np.where(ends, 0, batch.length + takes).astype(np.int32)).cuda())
        if graph and t == 2:
            before = [b.clone() for b in (dec.length, dec.table, dec.free, dec.free_count)]
            want = dec.want.clone()
            dec.want.copy_(dec.length)
            dec.step()                                 # warmed up: nothing grows
            torch.cuda.synchronize()
            run = torch.cuda.CUDAGraph()
            with torch.cuda.graph(run):
                dec.step()
            for b, old in zip((dec.length, dec.table, dec.free, dec.free_count), before):
                assert torch.equal(b, old)
            dec.want.copy_(want)
        if run is None:
            dec.step()
        else:
            run.replay()
        ref = batch.step(x.astype(np.float64), takes)
        batch.length[ends] = 0
        assert dec.length.tolist() == batch.length.tolist()
        if takes.any():
            close(dec.a.cpu().numpy().astype(np.float64)[takes], ref[takes], t)
    assert dec.ctx.sync_status() == 0
    dec.ctx.close()


def test_a_request_without_pages_leaves_the_others_right(gpu_lib):
    """Seven requests on six pages of two tokens: one is refused at every third
    length until another ends."""
    n, page = 7, 2
    dec, w, norms = DB.build("fp32", requests=n, max_len=16, page_size=page, rank=8, rv=32, **SIZE)
    dec.free_count.fill_(6)
    batch, g, refusals = Batch(w, norms, n), np.random.default_rng(4), 0
    for t in range(6):
        x = g.standard_normal((n, SIZE["hidden"])).astype(np.float32)
        dec.x.copy_(torch.from_numpy(x).cuda())
        want = batch.length + 1
        want[[1, 4]] = batch.length[[1, 4]] + (t not in (1, 4))    # these idle at times
        if t == 3:
            want[[0, 3]] = 0
        dec.want.copy_(torch.from_numpy(want.astype(np.int32)).cuda())
        dec.step()
        length = np.array(dec.length.tolist())
        takes = (length == batch.length + 1) & (want == batch.length + 1)
        refused = (want == batch.length + 1) & ~takes
        assert np.array_equal(length[~takes & ~refused], want[~takes & ~refused])
        assert np.array_equal(length[refused], batch.length[refused])
        refusals += int(refused.sum())
        assert dec.ctx.sync_status() == (PAGES if refused.any() else 0)
        ref = batch.step(x.astype(np.float64), takes)
        batch.length[want == 0] = 0
        if takes.any():
            close(dec.a.cpu().numpy().astype(np.float64)[takes], ref[takes], t)
    assert refusals > 0
    dec.ctx.close()
