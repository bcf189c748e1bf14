"""CPU checks of the operators for rows that share cache pages: the oracle's definitions
pinned by what they must keep, the binding's structures against the C header, and what the
binding takes and refuses.  Contexts without a handle, as in the other binding's tests:
arguments that pass reach the library, which refuses the null context."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import block_ops as OB

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    import lora_normal_form_gb300 as scute
    if not os.path.exists(scute.LIB_PATH):
        from lora_normal_form_gb300 import build as B
        B.build()
    return scute


# ---------------------------------------------------------------- the oracle's definitions
def test_fork_keeps_every_page_and_every_token():
    """Whatever is forked, cut and let go: pages are free or held as often as their count
    says, no row's last page in part is another's, and every row reads the tokens that its
    source had (a page's contents are simulated as the tokens written to it)."""
    g = np.random.default_rng(3)
    page, cols, n, pages = 4, 6, 9, 70
    table, free, extra = np.full((n, cols), -1), list(range(pages)), [0] * pages
    length, cells, rows, clock = np.zeros(n, int), np.full((pages, page), -1), [[] for _ in range(n)], 0
    for _ in range(300):
        want = np.minimum(length + g.integers(0, 6, n), cols * page)
        r = OB.resize(length, want, table, page, free, n * 6)
        table, free, length = r["table"], r["free"], r["len_out"]
        for slot, req in zip(r["slot_map"], r["token_req"]):
            if req >= 0:
                clock += 1
                cells[slot // page, slot % page] = clock
                rows[req].append(clock)
        source = g.integers(-1, n, n)
        cut = np.where(source >= 0, np.where(g.random(n) < 0.3, length[source] * g.random(n), length[source]), 0).astype(int)
        f = OB.fork(table, length, source, cut, np.full((n, cols), -1), page, extra, free)
        assert f["ok"] == np.all(f["len_out"] == cut)
        for a, b, t in zip(f["copy_from"], f["copy_to"], f["copy_tokens"]):
            if b >= 0:
                cells[b, :t] = cells[a, :t]
        rows = [list(rows[s][:m]) if s >= 0 else [] for s, m in zip(source, f["len_out"])]
        table, free, length, extra = f["table"], f["free"], f["len_out"], f["extra"]
        held = np.zeros(pages, int)
        for i in range(n):
            own = table[i, :OB.ceil_div(length[i], page)]
            held[own] += 1
            assert [int(cells[own[t // page], t % page]) for t in range(length[i])] == rows[i]
        assert all(held[table[i, length[i] // page]] == 1 for i in range(n) if length[i] % page)
        assert sorted(set(free)) == sorted(free) and not held[free].any()
        assert np.array_equal(extra, np.maximum(held - 1, 0)) and len(free) + np.count_nonzero(held) == pages


def test_fork_by_hand():
    table = np.array([[5, 6, -1], [5, 7, 8]])
    # row 0 has 5 5 5 5 | 6 6, row 1 has 5 5 5 5 | 7 7 7 7 | 8: pages of four tokens, 5 shared
    out = OB.fork(table, [6, 9], [1, 1, 0, -1], None, np.full((4, 3), -1), 4, [0, 0, 0, 0, 0, 1, 0, 0, 0], [1, 2])
    assert out["table"].tolist() == [[5, 7, 8], [5, 7, 2], [5, 6, -1], [-1, -1, -1]]
    assert out["len_out"].tolist() == [9, 9, 6, 0] and out["free"] == [1]
    assert out["copy_from"].tolist() == [-1, 8, -1, -1] and out["copy_to"].tolist() == [-1, 2, -1, -1]
    assert out["copy_tokens"].tolist() == [0, 1, 0, 0]
    assert out["extra"].tolist() == [0, 0, 0, 0, 0, 2, 0, 1, 0]
    # nobody goes on with row 0: its own page is free again, by number; no page is left for the copy of 8
    out = OB.fork(table, [6, 9], [1, 1, 1], [9, 8, 9], np.full((3, 3), -1), 4, [0] * 5 + [1, 0, 0, 0], [])
    assert out["table"].tolist() == [[5, 7, 8], [5, 7, -1], [5, 7, 6]] and out["free"] == [] and out["ok"]
    out = OB.fork(table, [6, 9], [0, 1, 1], [6, 9, 9], np.full((3, 3), -1), 4, [0] * 5 + [1, 0, 0, 0], [])
    assert not out["ok"] and out["len_out"].tolist() == [6, 9, 8] and out["table"][2].tolist() == [5, 7, -1]


def test_head_norm_and_seen_pins():
    g = np.random.default_rng(1)
    x, w = g.standard_normal((3, 2, 40)) * 4 + 1, g.standard_normal((2, 40))
    y = OB.head_norm(x, 1.0, 0.0, False)
    assert np.allclose((y ** 2).mean(-1), 1) and np.allclose(OB.head_norm(3 * x, w, 0.0, False), OB.head_norm(x, w, 0.0, False))
    z = OB.head_norm(x, 1.0, 0.0, True)
    assert np.allclose(z.mean(-1), 0) and np.allclose(z.std(-1), 1) and np.allclose(OB.head_norm(x + 5, w, 1e-3, True), OB.head_norm(x, w, 1e-3, True))
    for r in range(3):
        for h in range(2):
            assert np.allclose(OB.head_norm(x, w, 1e-5, False)[r, h], OB.norm(x[r, h][None], w[h], None, 1e-5, False)[0])
    assert OB.seen(5) == [0, 1, 2, 3, 4] and OB.seen(9, 3, 2) == [0, 1, 6, 7, 8] and OB.seen(4, 3, 2) == [0, 1, 2, 3]
    assert OB.seen(9, 3, 100) == list(range(9)) and OB.seen(0, 3, 2) == [] and OB.seen(9, 0, 2) == list(range(9))


def test_fork_counts_rows_by_themselves():
    """More rows of a page than its count allows: noticed where the page is given up, or to another
    row, though a row has it, and where its count falls below nobody; and only there."""
    two = np.array([[0], [0]])
    go = lambda lens, source, extra, new=None: OB.fork(two, lens, source, new, np.full((len(source), 1), -1), 16, [extra], [])  # noqa: E731
    out = go([16, 16], [0], 0)
    assert not out["ok"] and out["table"].tolist() == [[0]] and out["free"] == [0]
    assert not go([5, 5], [0], 0)["ok"] and not go([16, 16], [0, 1], 0, [16, 5])["ok"] and not go([16, 16], [-1], 0)["ok"]
    assert not go([16, 16], [1], 0)["ok"] and not go([16, 16], [0], 0, [5])["ok"]
    for lens, source, new in (([16, 16], [0], None), ([16, 16], [0, 1], [16, 0]), ([16, 16], [-1], None)):
        assert go(lens, source, 1, new)["ok"]
    assert go([16, 16], [0, 1], 0)["ok"]               # nobody lets go: nothing is given away


# ---------------------------------------------------------------- the binding
STRUCTS = {"scute_head_norm": "_HeadNormStruct", "scute_fork": "_ForkStruct", "scute_shared": "_SharedStruct"}


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


def test_packed_fork_is_the_structure(lib):
    values = [8 * (i + 1) for i in range(len(lib._ForkStruct._fields_))]
    assert lib._FORK.pack(*values) == bytes(lib._ForkStruct(*values))


def test_null_contexts_are_refused(lib):
    L = lib.load()
    assert L.scute_kv_append_norm(None, None, None, 0, None, 0, None, 0, None, 0, 0, None, 0, None, None, None) == 1
    assert L.scute_kv_fork(None, None, None) == 1 and L.scute_kv_copy(None, None, 0, None, None, None, 0, None) == 1
    assert L.scute_paged_attention_sinks(None, None, None, 1, None) == 1
    assert L.scute_paged_attention_shared(None, None, None, None, None) == 1
    assert L.scute_shared_bytes(None, 1, 1, 1, 64) == -1


def no_handle(lib, dtype="bf16"):
    c = object.__new__(lib.Context)
    c.dtype, c.handle, c.device = dtype, None, 0
    return c


def whole(*s):
    return torch.zeros(*s, dtype=torch.int32)


def test_what_the_binding_takes_and_refuses(lib):
    ctx, half = no_handle(lib), lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    pool = half(4, 2, 16, 64)
    cache, k, q, lens = lib.KvCache(pool, pool, whole(3, 2)), half(3, 2, 64), half(3, 4, 64), whole(3)
    w, work = torch.ones(64), torch.zeros(4096, dtype=torch.uint8)
    norm, shared = lib.HeadNorm(w, torch.ones(2, 64)), lib.Shared(whole(2), whole(1), work)
    fork = dict(table_in=whole(2, 4), len_in=whole(2), source=whole(3), table_out=whole(3, 4), len_out=whole(3), page_size=16,
                extra=whole(9), free_pages=whole(9), free_in=whole(1), free_out=whole(1), copy_from=whole(3), copy_to=whole(3),
                copy_tokens=whole(3), len_new=whole(3))
    append = lambda norm=norm, **kw: ctx.kv_append(cache, lens, k, k, norm=norm, **kw)  # noqa: E731
    attend = lambda **kw: ctx.paged_attention(cache, q, lens, q, **kw)  # noqa: E731
    good = [append, lambda: append(q=q, q_out=q), lambda: append(lib.HeadNorm(q_w=torch.ones(4, 64)), q=q, q_out=q),
            lambda: append(lib.HeadNorm(torch.ones(7, 64)[:1], w)), lambda: append(lib.HeadNorm(torch.ones(4, 80)[:, :64]), q=q, q_out=q),
            lambda: ctx.kv_fork(**fork), lambda: ctx.kv_fork(**{**fork, "len_new": None}),
            lambda: ctx.kv_fork(**{**fork, "table_in": whole(2, 9)[:, 2:6], "table_out": whole(5, 7)[:, :4]}),
            lambda: ctx.kv_fork(**{**fork, "table_in": whole(1, 4), "len_in": whole(1)}),
            lambda: ctx.kv_copy(lib.KvCaches([cache, cache]), lens, lens, lens), lambda: ctx.kv_copy(lib.KvCaches([cache]), lens, lens),
            lambda: attend(sinks=4), lambda: attend(shared=shared)]
    for call in good:
        with pytest.raises(lib.ScuteError):
            call()
    bad = [lambda: append(lib.HeadNorm(torch.ones(32)), q=q, q_out=q), lambda: append(lib.HeadNorm(k_w=torch.ones(3, 64))),
           lambda: append(lib.HeadNorm(torch.ones(2, 64)), q=q, q_out=q), lambda: lib.HeadNorm(), lambda: lib.HeadNorm(half(64)),
           lambda: lib.HeadNorm(torch.ones(2, 2, 64)), lambda: lib.HeadNorm(torch.ones(64, 2).t()), lambda: lib.HeadNorm(torch.ones(0, 64)),
           lambda: lib.HeadNorm(w.expand(2, 64)), lambda: lib.KvCaches([]), lambda: lib.KvCaches([pool]),
           lambda: ctx.kv_copy(lib.KvCaches([cache]), lens, whole(2)), lambda: ctx.kv_copy(lib.KvCaches([cache]), lens, lens, lens.float()),
           lambda: attend(shared=shared, sinks=2), lambda: lib.Shared(whole(3), whole(1), work), lambda: lib.Shared(whole(2).float(), whole(1), work),
           lambda: lib.Shared(whole(2), whole(1).long(), work), lambda: lib.Shared(whole(4)[::2], whole(1), work), lambda: lib.Shared(whole(2), whole(1), work[::2])]
    wrong = dict(len_in=whole(3), len_out=whole(2), copy_from=whole(4), copy_to=whole(2), copy_tokens=whole(2), len_new=whole(2),
                 free_in=whole(2), free_out=whole(0), table_in=whole(2, 5), table_out=whole(2, 4))
    bad += [lambda n=n: ctx.kv_fork(**{**fork, n: wrong[n]}) for n in wrong]
    bad += [lambda n=n: ctx.kv_fork(**{**fork, n: fork[n].float()}) for n in fork if n != "page_size"]
    bad += [lambda n=n: ctx.kv_fork(**{**fork, n: whole(2 * fork[n].numel())[::2]}) for n in ("len_in", "source", "len_new", "len_out", "extra", "free_pages",
                                                                                             "copy_from", "copy_to", "copy_tokens")]
    bad += [lambda: ctx.kv_fork(**{**fork, "table_out": whole(1, 4).expand(3, 4)}), lambda: ctx.kv_fork(**{**fork, "table_in": whole(4, 2).t()})]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
