"""The operators together, as a decoder step runs them: a two-layer decoder with
mixed adapters and a paged cache, token by token, against the float64 oracle
(adapted layers from their definitions, attention, norms and rotary positions
from ``oracle/block_ops.py``) over whole sequences.

Tolerance.  In an fp32 context a linear layer is within 2.3e-4 of its output's
rms (the split-precision product's measured bound under the stricter floor of
``tests/metrics.py``), and a norm, attention or gated product passes relative
errors on with a factor of at most about 2; the residual stream keeps the rest.
Seven layers deep twice, errors of independent sign: 2 * sqrt(14) * 2.3e-4 =
1.7e-3 of the output's rms."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import batch as BT  # noqa: E402
from oracle import block_ops as OB  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decode_block as DB  # noqa: E402

SIZE = dict(hidden=128, heads=4, kv_heads=2, dim=32, ffn=256, layers=2)


class OracleDecoder:
    def __init__(self, w, norms, size, theta=500000.0, eps=1e-5):
        self.w, self.norms, self.size, self.eps = w, [v.astype(np.float64) for v in norms], size, eps
        self.inv = theta ** (-np.arange(0, size["dim"], 2) / size["dim"])
        self.cache = {}

    def lin(self, name, x):
        return BT.linear(self.w, name, x=x)

    def step(self, x, positions):
        s, n = self.size, len(x)
        h, heads, kvh, dim = x.copy(), s["heads"], s["kv_heads"], s["dim"]
        a = OB.norm(h, self.norms[0], None, self.eps, False)
        for i in range(s["layers"]):
            q, k, v = (self.lin(f"{i}.{p}", a) for p in "qkv")
            att = np.zeros((n, heads * dim))
            for r in range(n):
                ang = positions[r] * self.inv
                qr = OB.rope(q[r].reshape(heads, dim), ang, dim, False)
                kr = OB.rope(k[r].reshape(kvh, dim), ang, dim, False)
                ks, vs = self.cache.setdefault((i, r), ([], []))
                del ks[positions[r]:], vs[positions[r]:]
                ks.append(kr)
                vs.append(v[r].reshape(kvh, dim))
                kk, vv = np.stack(ks), np.stack(vs)
                for g in range(kvh):
                    rows = slice(g * heads // kvh, (g + 1) * heads // kvh)
                    att[r].reshape(heads, dim)[rows] = OB.attend(qr[rows], kk[:, g], vv[:, g], dim ** -0.5)[0]
            h, b = OB.residual_norm(self.lin(f"{i}.o", att), h, None, (self.norms[2 * i + 1], None), None, 1.0, self.eps, False)
            gate, up = self.lin(f"{i}.gate", b), self.lin(f"{i}.up", b)
            down = self.lin(f"{i}.down", gate / (1 + np.exp(-gate)) * up)
            h, a = OB.residual_norm(down, h, None, (self.norms[2 * i + 2], None), None, 1.0, self.eps, False)
        return a


@pytest.mark.parametrize("graph", [False, True])
def test_decoder_steps_match_the_oracle(gpu_lib, graph):
    n, steps, page = 7, 9, 4
    dec, w, norms = DB.build("fp32", requests=n, max_len=16, page_size=page, rank=8, rv=32, **SIZE)
    ref = OracleDecoder(w, norms, SIZE)
    g = np.random.default_rng(0)
    run = None
    for t in range(steps):
        x = g.standard_normal((n, SIZE["hidden"])).astype(np.float32)
        dec.x.copy_(torch.from_numpy(x).cuda())
        lengths = dec.length.cpu().numpy()
        if t == 5:          # two requests end and begin anew: their pages go back and come again
            dec.want.copy_(dec.length)
            dec.want[2] = dec.want[5] = 0
            c = dec.ctx
            c.kv_resize(dec.length, dec.want, dec.table, page, dec.free, dec.free_count, dec.free_count, dec.length,
                        dec.cu, dec.slots, dec.positions, dec.req)
            lengths = dec.length.cpu().numpy()
            assert lengths[2] == lengths[5] == 0 and lengths[0] == 5
        torch.add(dec.length, 1, out=dec.want)
        if graph and t == 2:
            torch.cuda.synchronize()
            run = torch.cuda.CUDAGraph()
            with torch.cuda.graph(run):
                dec.step()
        if run is not None:
            run.replay()
            out = dec.a
        else:
            out = dec.step()
        got = out.cpu().numpy().astype(np.float64)
        want = ref.step(x.astype(np.float64), lengths)
        rms = np.sqrt((want * want).mean())
        assert np.max(np.abs(got - want)) <= 1.7e-3 * 3 * rms, t     # the largest of a few hundred: three deviations
        assert np.sqrt(((got - want) ** 2).mean()) <= 1.7e-3 * rms, t
    assert dec.ctx.sync_status() == 0
    kinds = set(dec.ctx.timing_kinds())
    assert not kinds
    dec.ctx.timing(True)
    torch.add(dec.length, 1, out=dec.want)
    dec.step()
    torch.cuda.synchronize()
    assert {"kv_resize", "kv_append", "attention", "norm"} <= set(dec.ctx.timing_kinds())
    dec.ctx.close()


def test_bf16_decoder_follows_the_fp32_one(gpu_lib):
    """The bf16 step (one launch per projection group, a 16-bit cache): every
    linear layer rounds its output to bf16 (2^-9 relative), as do the cache, the
    rotated queries, the attention and the norms: about 30 roundings of 2^-9 /
    sqrt(3) in a two-layer step, independent, each passed on at most doubled:
    2 * sqrt(30) * 2^-9 / sqrt(3) = 1.2 % of the output's rms."""
    n = 12
    dec, w, norms = DB.build("bf16", requests=n, max_len=16, page_size=4, rank=8, rv=32, **SIZE)
    ref = OracleDecoder(w, norms, SIZE)
    g = np.random.default_rng(1)
    for t in range(6):
        dec.x.copy_(torch.from_numpy(g.standard_normal((n, SIZE["hidden"])).astype(np.float32)).cuda())
        lengths = dec.length.cpu().numpy()
        torch.add(dec.length, 1, out=dec.want)
        got = dec.step().float().cpu().numpy().astype(np.float64)
        want = ref.step(dec.x.float().cpu().numpy().astype(np.float64), lengths)
        assert np.sqrt(((got - want) ** 2).mean()) <= 1.2e-2 * np.sqrt((want * want).mean()), t
    assert dec.ctx.sync_status() == 0
    dec.ctx.close()
