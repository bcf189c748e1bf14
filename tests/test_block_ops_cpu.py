"""CPU checks of the operators between the projections: the oracle's own
definitions pinned by identities and brute force, the binding's structures
against the C header's layout, and null contexts refused."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import block_ops as OB

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import lora_normal_form_gb300 as scute
    if not os.path.exists(scute.LIB_PATH):
        from lora_normal_form_gb300 import build as B
        B.build()
    return scute


# ---------------------------------------------------------------- the oracle's definitions
def test_attend_pins():
    g = np.random.default_rng(0)
    q, k, v = g.standard_normal((3, 8)), g.standard_normal((5, 8)), g.standard_normal((5, 8))
    out, lse, mass, reach = OB.attend(q, k, v, 0.3)
    for h in range(3):          # brute force
        e = [np.exp(0.3 * float(q[h] @ k[t])) for t in range(5)]
        assert np.allclose(out[h], sum(w * v[t] for t, w in enumerate(e)) / sum(e), rtol=1e-13)
        assert np.isclose(lse[h], np.log(sum(e)), rtol=1e-13)
    assert np.all(mass >= np.abs(out) - 1e-15) and np.all(reach >= np.abs(0.3 * q @ k.T).max(1) - 1e-15)
    # equal keys: the mean; one token: its value; order does not matter; a shift of all scores neither
    assert np.allclose(OB.attend(q, np.repeat(k[:1], 5, 0), v, 1.0)[0], v.mean(0))
    assert np.allclose(OB.attend(q, k[:1], v[:1], 1.0)[0], v[0])
    p = g.permutation(5)
    assert np.allclose(OB.attend(q, k[p], v[p], 0.3)[0], out)
    u = q[0] / (q[0] @ q[0])
    assert np.allclose(OB.attend(q[:1], k + 7.0 * u, v, 0.3)[0], out[:1])
    # parts joined by their lse are the whole; a huge cap changes nothing, a tiny one flattens
    a, la, _, _ = OB.attend(q, k[:2], v[:2], 0.3)
    b, lb, _, _ = OB.attend(q, k[2:], v[2:], 0.3)
    w = np.exp(la - np.logaddexp(la, lb))[:, None]
    assert np.allclose(w * a + (1 - w) * b, out)
    assert np.allclose(OB.attend(q, k, v, 0.3, 1e9)[0], out)
    assert np.allclose(OB.attend(q, k, v, 0.3, 1e-12)[0], v.mean(0))
    out, lse, _, _ = OB.attend(q, k[:0], v[:0], 1.0)
    assert not out.any() and np.all(lse == -np.inf)


def test_rope_pins():
    g = np.random.default_rng(1)
    x, y = g.standard_normal((2, 12)), g.standard_normal((2, 12))
    ang = g.standard_normal(4)
    for inter in (False, True):
        assert np.allclose(OB.rope(x, 0 * ang, 8, inter), x)
        r = OB.rope(x, ang, 8, inter)
        assert np.allclose(np.linalg.norm(r, axis=1), np.linalg.norm(x, axis=1)) and np.array_equal(r[:, 8:], x[:, 8:])
        assert np.allclose(OB.rope(r, -ang, 8, inter), x)
        # products depend on the difference of positions alone
        a = (OB.rope(x, 5 * ang, 8, inter) * OB.rope(y, 3 * ang, 8, inter)).sum(1)
        assert np.allclose(a, (OB.rope(x, 2 * ang, 8, inter) * y).sum(1))
    quarter = OB.rope(np.arange(4.0)[None], np.array([np.pi / 2, 0.0]), 4, False)
    assert np.allclose(quarter, [[-2.0, 1.0, 0.0, 3.0]])
    assert np.allclose(OB.rope(np.arange(4.0)[None], np.array([np.pi / 2, 0.0]), 4, True), [[-1.0, 0.0, 2.0, 3.0]])


def test_norm_pins():
    g = np.random.default_rng(2)
    x = g.standard_normal((4, 50)) * 3 + 1
    assert np.allclose((OB.norm(x, None, None, 0.0, False) ** 2).mean(1), 1)
    n = OB.norm(x, None, None, 0.0, True)
    assert np.allclose(n.mean(1), 0, atol=1e-14) and np.allclose(n.std(1), 1)
    assert np.allclose(OB.norm(7 * x, None, None, 0.0, False), OB.norm(x, None, None, 0.0, False))
    assert np.allclose(OB.norm(x + 9, None, None, 0.0, True), n)
    h, o = OB.residual_norm(x, 2 * x, None, None, None, 0.5, 1e-5, False)
    assert np.allclose(h, 2.5 * x) and o is None


def test_resize_keeps_every_page_once():
    g = np.random.default_rng(3)
    page, cols, n, pages = 4, 6, 9, 40
    table, free = np.full((n, cols), -1), list(range(pages))
    length = np.zeros(n, int)
    for _ in range(200):
        want = np.where(g.random(n) < 0.2, 0, np.minimum(length + g.integers(0, 9, n), cols * page))
        r = OB.resize(length, want, table, page, free, 30)
        table, free, length = r["table"], r["free"], r["len_out"]
        held = [int(table[i, b]) for i in range(n) for b in range(OB.ceil_div(length[i], page))]
        assert sorted(held + free) == list(range(pages))
        rows = r["slot_map"][:r["cu_new"][-1]]
        assert len(set(rows)) == len(rows) and np.all(r["slot_map"][r["cu_new"][-1]:] == -1)
        for i, slot in enumerate(rows):
            q, pos = r["token_req"][i], r["positions"][i]
            assert slot == table[q, pos // page] * page + pos % page and pos < length[q]


# ---------------------------------------------------------------- the binding
STRUCTS = {"scute_kv_cache": "_KvCacheStruct", "scute_rope": "_RopeStruct", "scute_attention": "_AttentionStruct",
           "scute_norm": "_NormStruct"}


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_structures_have_the_header_s_layout(lib, tmp_path):
    lines = []
    for c, py in STRUCTS.items():
        lines.append(f'printf("{c} %zu", sizeof({c}));')
        lines += [f'printf(" %zu", offsetof({c}, {f[0]}));' for f in getattr(lib, py)._fields_]
        lines.append('printf("\\n");')
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include "scute.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0;\n}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "l")], check=True)
    got = {x.split()[0]: [int(v) for v in x.split()[1:]] for x in
           subprocess.run([str(tmp_path / "l")], check=True, capture_output=True, text=True).stdout.splitlines()}
    for c, py in STRUCTS.items():
        cls = getattr(lib, py)
        assert got[c] == [ctypes.sizeof(cls)] + [getattr(cls, f[0]).offset for f in cls._fields_], c


def test_null_contexts_are_refused(lib):
    L = lib.load()
    assert L.scute_kv_resize(None, None, None, 0, None, 1, 1, 16, None, 0, None, None, None, None, None, None, None, 0, None) == 1
    assert L.scute_rope_table(None, None, 1, 2, 1e4, None, None) == 1
    assert L.scute_kv_append(None, None, None, 0, None, 0, None, 0, None, 0, 0, None, 0, None, None) == 1
    assert L.scute_paged_attention(None, None, None, None) == 1
    assert L.scute_residual_norm(None, None, 0, 1, None) == 1


def test_binding_refuses_what_a_call_could_not_mean(lib):
    torch = pytest.importorskip("torch")
    pool = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    table = torch.zeros(3, 2, dtype=torch.int32)
    for args in ((pool, pool[:3]), (pool, pool.float()), (pool.half(), pool.half()), (pool[0], pool[0]),
                 (pool.transpose(2, 3), pool.transpose(2, 3)), (pool, pool, table.long()), (pool, pool, table[0]),
                 (pool, pool, None, False, torch.ones(3)), (pool, pool, None, False, torch.ones(2, dtype=torch.float64))):
        with pytest.raises(ValueError):
            lib.KvCache(*args)
    c = lib.KvCache(pool, pool, table)
    assert (c.struct.n_pages, c.struct.page_size, c.struct.kv_heads, c.struct.head_dim) == (4, 16, 2, 64)
    assert (c.struct.page_stride, c.struct.head_stride, c.struct.token_stride) == (2048, 1024, 64)
    t = lib.KvCache(pool, pool, token_major=True)
    assert (t.struct.page_size, t.struct.kv_heads, t.struct.token_stride, t.struct.head_stride) == (2, 16, 1024, 64)
    one = lib.KvCache(pool[:1, :1, :1].expand(1, 1, 1, 64), pool[:1, :1, :1])
    assert min(one.struct.page_stride, one.struct.head_stride, one.struct.token_stride) >= 64
    cs = torch.zeros(10, 64)
    for args in ((cs, torch.zeros(3, dtype=torch.int64)), (cs, torch.zeros(2, 3, dtype=torch.int32)), (cs.double(), torch.zeros(3, dtype=torch.int32)),
                 (cs.t(), torch.zeros(3, dtype=torch.int32)), (cs, torch.zeros(5, 3, dtype=torch.int32), [1] * 5)):
        with pytest.raises(ValueError):
            lib.Rope(*args)
    assert lib._rows(torch.zeros(5, 8), 5, 8) == 8 and lib._rows(torch.zeros(5, 12)[:, 2:10], 5, 8) == 12
    assert lib._rows(torch.zeros(5, 6, 4)[:, 1:3], 5, 8) == 24 and lib._rows(torch.zeros(1, 8)[:, :8], 1, 8) >= 8
    for bad in (torch.zeros(5, 9), torch.zeros(4, 8), torch.zeros(8, 5).t(), torch.zeros(5, 4, 2).transpose(1, 2)):
        with pytest.raises(ValueError):
            lib._rows(bad, 5, 8)
