"""CPU checks of what the Python binding of the decoder block's operators takes
and refuses.  The contexts here have no handle: arguments that pass the
binding's checks reach the library, which refuses the null context
(``ScuteError``); those that the binding refuses raise ``ValueError`` first."""
import os

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    import lora_normal_form_gb300 as scute
    if not os.path.exists(scute.LIB_PATH):
        from lora_normal_form_gb300 import build as B
        B.build()
    return scute


def no_handle(lib, dtype="bf16"):
    c = object.__new__(lib.Context)
    c.dtype, c.handle, c.device = dtype, None, 0
    return c


def whole(*s):
    return torch.zeros(*s, dtype=torch.int32)


def half(*s, t=torch.bfloat16):
    return torch.zeros(*s, dtype=t)


def refused_by_library(lib, call):
    with pytest.raises(lib.ScuteError):
        call()


# ---------------------------------------------------------------- block tables
def test_cache_refuses_tables_whose_rows_overlap(lib):
    """A row pitch below the row's length cannot be told to the library: read
    with a longer one, the rows would lie behind the table's end."""
    pool = half(4, 2, 16, 64)
    for bad in (torch.arange(3, dtype=torch.int32).view(1, 3).expand(8, 3), whole(20).as_strided((6, 4), (2, 1)),
                whole(8).as_strided((4, 3), (1, 1))):
        with pytest.raises(ValueError):
            lib.KvCache(pool, pool, bad)
    wide = lib.KvCache(pool, pool, whole(8, 5)[:, :3])
    assert (wide.struct.table_stride, wide.struct.table_cols, wide.requests) == (5, 3, 8)
    # one row has no pitch: any is as good
    for one in (whole(1, 3), whole(3).as_strided((1, 3), (1, 1)), whole(1, 3).expand(1, 3)):
        c = lib.KvCache(pool, pool, one)
        assert (c.struct.table_stride, c.struct.table_cols, c.requests) == (3, 3, 1)
    for rows, cols in ((8, 1), (0, 4)):
        c = lib.KvCache(pool, pool, whole(rows, cols))
        assert (c.struct.table_stride, c.struct.table_cols, c.requests) == (cols, cols, rows)
    with pytest.raises(ValueError):
        lib.KvCache(pool, pool, whole(1, 1).expand(8, 1))


# ---------------------------------------------------------------- the rotary table
def test_rope_table_refuses_what_it_would_read_or_write_wrongly(lib):
    """Frequencies are 64-bit: 32-bit ones of the right number would be read to
    twice their length."""
    ctx, out, inv = no_handle(lib), half(9, 6, t=torch.float32), half(3, t=torch.float64)
    refused_by_library(lib, lambda: ctx.rope_table(out, 10000.0))
    refused_by_library(lib, lambda: ctx.rope_table(out, inv_freq=inv))
    for bad in (inv.float(), inv[:2], half(4, t=torch.float64), half(6, t=torch.float64)[::2], half(3, 1, t=torch.float64)[:2]):
        with pytest.raises(ValueError):
            ctx.rope_table(out, inv_freq=bad)
    for bad in (out.double(), out.bfloat16(), whole(9, 6), out.t(), out[:, :4], out[::2], out.view(9, 2, 3), out.view(-1)):
        with pytest.raises(ValueError):
            ctx.rope_table(bad, inv_freq=None)


# ---------------------------------------------------------------- types of the right size
def test_other_types_of_the_same_size_are_refused(lib):
    """float16 is no bf16, and neither float32 nor an unsigned or int32 tensor the
    other: the kernels would read the bits as another type's numbers."""
    ctx, f32 = no_handle(lib), no_handle(lib, "fp32")
    f16, real = lambda *s: half(*s, t=torch.float16), lambda *s: half(*s, t=torch.float32)  # noqa: E731
    pool = half(4, 2, 16, 64)
    cache = lib.KvCache(pool, pool, whole(2, 2))
    for kw in (dict(block_table=real(2, 2)), dict(k_scale=whole(2)), dict(v_scale=whole(2))):
        with pytest.raises(ValueError):
            lib.KvCache(pool, pool, **kw)
    for args in ((real(10, 64), real(3)), (whole(10, 64), whole(3))):
        with pytest.raises(ValueError):
            lib.Rope(*args)
    rope, k, q, y, w = lib.Rope(real(10, 64), whole(3)), half(3, 2, 64), half(2, 4, 64), half(2, 64), real(64)
    lens, slots = whole(2), whole(3)
    attend = lambda q=q, lens=lens, out=q, **kw: ctx.paged_attention(cache, q, lens, out, **kw)  # noqa: E731
    append = lambda slots=slots, k=k, v=k, q=k, q_out=k: ctx.kv_append(cache, slots, k, v, q=q, q_out=q_out, rope=rope)  # noqa: E731
    norm = lambda y=y, out=y, **kw: ctx.residual_norm(y, out, **kw)  # noqa: E731
    steps = dict(len_in=whole(2), len_new=whole(2), block_table=whole(2, 2), page_size=16, free_pages=whole(4),
                 free_in=whole(1), free_out=whole(1), len_out=whole(2), cu_new=whole(3), slot_map=whole(2),
                 positions=whole(2), token_req=whole(2))
    good = [attend, lambda: attend(lse=real(2, 4)), append, norm, lambda: norm(pre_w=w, gate=y, residual=y, residual_out=y),
            lambda: norm(gate=w), lambda: ctx.kv_resize(**steps), lambda: f32.residual_norm(real(2, 64), real(2, 64))]
    bad = [lambda: attend(q=f16(2, 4, 64)), lambda: attend(out=f16(2, 4, 64)), lambda: attend(q=q.view(torch.int16)),
           lambda: attend(lens=real(2)), lambda: attend(lse=whole(2, 4)),
           lambda: append(slots=real(3)), lambda: append(k=f16(3, 2, 64)), lambda: append(v=f16(3, 2, 64)),
           lambda: append(q=f16(3, 2, 64)), lambda: append(q_out=f16(3, 2, 64)),
           lambda: norm(y=f16(2, 64)), lambda: norm(out=f16(2, 64)), lambda: norm(residual=f16(2, 64)),
           lambda: norm(residual_out=f16(2, 64)), lambda: norm(gate=f16(2, 64)), lambda: norm(gate=whole(64)),
           lambda: f32.residual_norm(whole(2, 64), real(2, 64)), lambda: f32.residual_norm(real(2, 64), whole(2, 64))]
    bad += [lambda n=n: norm(out=y, **{n: whole(64)}) for n in ("pre_w", "pre_b", "post_w", "post_b")]
    bad += [lambda n=n: ctx.kv_resize(**{**steps, n: real(*steps[n].shape)}) for n in steps if n != "page_size"]
    for call in good:
        refused_by_library(lib, call)
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)


# ---------------------------------------------------------------- dimensions of one element
def test_strides_of_dimensions_of_one_element_do_not_count(lib):
    """One row, page, head or token may carry any stride: the library gets one
    that passes (rows' and pools' strides are multiples of 16 bytes there)."""
    row = half(1, 1031)[:, :512]
    assert row.stride(0) == 1031 and lib._rows(row, 1, 512, torch.bfloat16) == 512
    assert lib._rows(half(1, 1031)[:, :512].view(1, 8, 64), 1, 512) == 512
    pool = torch.zeros(4 * 16 * 64 + 72, dtype=torch.bfloat16)
    for shape, strides in (((4, 1, 16, 64), (1024, 1031, 64, 1)), ((1, 2, 16, 64), (2061, 1024, 64, 1)),
                           ((2, 2, 1, 64), (128, 64, 67, 1))):
        k = pool.as_strided(shape, strides)
        c = lib.KvCache(k, k)
        assert all(s >= 64 and s % 8 == 0 for s in (c.struct.page_stride, c.struct.head_stride, c.struct.token_stride))
    at = whole(12).as_strided((2, 1), (5, 3))
    assert lib.Rope(half(10, 64, t=torch.float32), at, sections=[16, 16]).struct.axis_stride == 5
    with pytest.raises(ValueError):
        lib.Rope(half(10, 64, t=torch.float32), whole(12).as_strided((2, 2), (5, 3)), sections=[16, 16])


# ---------------------------------------------------------------- addresses
def test_addresses_are_taken_without_exceptions(lib):
    """An integer, an array and a tensor: none by way of an exception raised and
    caught (eight times an integer's own cost, on every call that passes one)."""
    import sys

    import numpy as np

    a, t, raised = np.arange(3.0), half(3), []

    def watch(frame, event, arg):
        if event == "exception":
            raised.append(frame.f_code.co_name)
        return watch

    before = sys.gettrace()
    sys.settrace(watch)
    try:
        got = [lib.ptr(x) for x in (None, 4096, True, a, t)]
    finally:
        sys.settrace(before)
    assert got == [None, 4096, True, a.ctypes.data, t.data_ptr()] and not raised
    for bad in (a[::2], "x", 1.5):
        with pytest.raises((ValueError, TypeError)):
            lib.ptr(bad)
