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
    c.dtype, c.esz, c.handle, c.device = dtype, 2 if dtype == "bf16" else 4, None, 0
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
