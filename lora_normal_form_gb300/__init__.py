"""Python binding of libscute.so: the adapted linear layer in normal form.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  The functions below carry the C ABI's names (``include/scute.h``) and
take torch tensors (device pointers), numpy arrays (host pointers) or ints.
Loading fails loudly when ``libscute.so`` is missing; there is no fallback.

Citations name sections of the article "Scute: Exact Batched Serving for PEFT
Adapters Beyond LoRA" (paper-daily.com).
"""
from __future__ import annotations

import ctypes
import os
import struct
import sys
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libscute.so")

LORA, DORA, IA3, VERA, OFT, NF = range(6)
METHOD_ID = {"lora": LORA, "dora": DORA, "ia3": IA3, "vera": VERA, "oft": OFT, "nf": NF}
BF16, FP32 = 0, 1
STATUS = {0: "OK", 1: "ERR_ARG", 2: "ERR_SHAPE", 3: "ERR_DTYPE", 4: "ERR_OOM", 5: "ERR_BAD_ADAPTER",
          6: "ERR_CUDA", 7: "ERR_TIMEOUT", 8: "ERR_UNSUPPORTED", 9: "ERR_NO_DEVICE", 10: "ERR_PAGES"}
MAX_TOKENS = 16384
TIMING_SLOTS = 256
BM_MAX_KERNELS = 64


class ScuteError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class LayerTensors(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_int), ("rank", ctypes.c_int), ("c", ctypes.c_float),
                ("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("d", ctypes.c_void_p),
                ("e", ctypes.c_void_p), ("s", ctypes.c_void_p), ("b", ctypes.c_void_p),
                ("R", ctypes.c_void_p), ("magnitude", ctypes.c_void_p), ("l", ctypes.c_void_p)]


class ByteReport(ctypes.Structure):
    _fields_ = [("n_kernels", ctypes.c_int), ("name", (ctypes.c_char * 24) * BM_MAX_KERNELS),
                ("bytes", ctypes.c_int64 * BM_MAX_KERNELS), ("flops", ctypes.c_int64 * BM_MAX_KERNELS),
                ("algorithmic_bytes", ctypes.c_int64), ("adapter_bytes", ctypes.c_int64),
                ("base_weight_bytes", ctypes.c_int64), ("distinct_adapters", ctypes.c_int32)]

    def as_dict(self) -> dict:
        k = self.n_kernels
        return {"kernels": [(self.name[i].value.decode(), int(self.bytes[i]), int(self.flops[i]))
                            for i in range(k)],
                "algorithmic_bytes": int(self.algorithmic_bytes),
                "adapter_bytes": int(self.adapter_bytes),
                "base_weight_bytes": int(self.base_weight_bytes),
                "distinct_adapters": int(self.distinct_adapters)}


class BmAdapter(ctypes.Structure):
    _fields_ = [("method", ctypes.c_int), ("rank", ctypes.c_int), ("has_s", ctypes.c_int),
                ("has_b", ctypes.c_int), ("has_R", ctypes.c_int), ("has_vera", ctypes.c_int),
                ("has_vera_e", ctypes.c_int)]


class BmLayer(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("d_in", ctypes.c_int),
                ("d_out", ctypes.c_int), ("shared_rank", ctypes.c_int),
                ("lowrank_launched", ctypes.c_int), ("vera_launched", ctypes.c_int),
                ("max_adapters", ctypes.c_int), ("adapters", ctypes.POINTER(BmAdapter)), ("variant", ctypes.c_int)]


class Call(ctypes.Structure):
    """One entry of a batched call (scute_call)."""
    _fields_ = [("x", ctypes.c_void_p), ("layer", ctypes.c_int), ("out", ctypes.c_void_p)]


MAX_CALLS = 8

# ------------------------------------------------------------------ paged cache and block operators
KV_BF16, KV_FP32, KV_E4M3 = 0, 1, 2
_KV_DTYPE = {"torch.bfloat16": KV_BF16, "torch.float32": KV_FP32, "torch.float8_e4m3fn": KV_E4M3}
MAX_REQUESTS, MAX_HEAD_DIM, MAX_NORM_DIM = 16384, 256, 32768


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("table_cols", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _RopeStruct(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("n_pos", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("section", ctypes.c_int32 * 4),
                ("positions", ctypes.c_void_p), ("axis_stride", ctypes.c_int64)]


class _AttentionStruct(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_stride", ctypes.c_int64), ("lse", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("n_req", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("scale", ctypes.c_float),
                ("softcap", ctypes.c_float), ("window", ctypes.c_int32)]


class _NormStruct(ctypes.Structure):
    _fields_ = [("y", ctypes.c_void_p), ("y_stride", ctypes.c_int64), ("residual", ctypes.c_void_p),
                ("residual_stride", ctypes.c_int64), ("residual_out", ctypes.c_void_p),
                ("residual_out_stride", ctypes.c_int64), ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("post_w", ctypes.c_void_p), ("post_b", ctypes.c_void_p), ("pre_w", ctypes.c_void_p),
                ("pre_b", ctypes.c_void_p), ("gate_vec", ctypes.c_void_p), ("gate_rows", ctypes.c_void_p),
                ("gate_stride", ctypes.c_int64), ("scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("layer", ctypes.c_int32)]


class _HeadNormStruct(ctypes.Structure):
    _fields_ = [("q_w", ctypes.c_void_p), ("k_w", ctypes.c_void_p), ("q_w_stride", ctypes.c_int64),
                ("k_w_stride", ctypes.c_int64), ("eps", ctypes.c_float), ("layer", ctypes.c_int32)]


class _SharedStruct(ctypes.Structure):
    _fields_ = [("start", ctypes.c_void_p), ("len", ctypes.c_void_p), ("work", ctypes.c_void_p),
                ("work_bytes", ctypes.c_int64), ("n_groups", ctypes.c_int32), ("always", ctypes.c_int32)]


class _ForkStruct(ctypes.Structure):
    _fields_ = [("table_in", ctypes.c_void_p), ("len_in", ctypes.c_void_p), ("table_in_stride", ctypes.c_int64),
                ("source", ctypes.c_void_p), ("len_new", ctypes.c_void_p), ("table_out", ctypes.c_void_p),
                ("len_out", ctypes.c_void_p), ("table_out_stride", ctypes.c_int64), ("n_in", ctypes.c_int32),
                ("n_out", ctypes.c_int32), ("table_cols", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int32), ("extra", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("n_free_max", ctypes.c_int64), ("free_in", ctypes.c_void_p), ("free_out", ctypes.c_void_p),
                ("copy_from", ctypes.c_void_p), ("copy_to", ctypes.c_void_p), ("copy_tokens", ctypes.c_void_p)]


def _packer(cls):
    """``struct`` form of a structure, whose fields take less time to fill."""
    codes = {ctypes.c_void_p: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f"}
    form = "@" + "".join(codes[t] for _, t in cls._fields_)
    return struct.Struct(f"{form}{ctypes.sizeof(cls) - struct.calcsize(form)}x")


_ATTENTION, _NORM, _FORK = _packer(_AttentionStruct), _packer(_NormStruct), _packer(_ForkStruct)


class KvCache:
    """A paged key/value cache over the caller's tensors (scute_kv_cache).

    ``k``, ``v``: device pools [n_pages, kv_heads, page_size, head_dim], or
    [n_pages, page_size, kv_heads, head_dim] with ``token_major``; the strides
    are taken from ``k`` and ``v`` must have the same.  ``block_table``: device
    int32 [n_req, pages of a request] (attention only), a row of its own for each
    request (not one row expanded).  ``k_scale``,
    ``v_scale``: device float32 [kv_heads] or None.  Holds references to the
    tensors, copies nothing."""

    def __init__(self, k, v, block_table=None, token_major=False, k_scale=None, v_scale=None):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-D pools of one shape, layout and type")
        if str(k.dtype) not in _KV_DTYPE or k.stride(3) != 1:
            raise ValueError("cache pools are bf16, fp32 or float8_e4m3fn with consecutive elements")
        tok, head = (1, 2) if token_major else (2, 1)
        self.tensors = (k, v, block_table, k_scale, v_scale)
        self.page_size, self.kv_heads, self.head_dim = k.shape[tok], k.shape[head], k.shape[3]
        self.kv_row, self.requests = self.kv_heads * self.head_dim, 0
        # a dimension of one element may carry any stride, which is never used: give it one that passes
        def stride(dim):
            return k.stride(dim) if k.shape[dim] > 1 else self.head_dim
        self.struct = _KvCacheStruct(k.data_ptr(), v.data_ptr(), _KV_DTYPE[str(k.dtype)], k.shape[0], self.page_size,
                                     self.kv_heads, self.head_dim, stride(0), stride(tok), stride(head), None, 0, 0,
                                     ptr(k_scale), ptr(v_scale))
        for s in (k_scale, v_scale):
            if s is not None and (s.numel() != self.kv_heads or not s.is_contiguous() or s.dtype is not _torch().float32):
                raise ValueError("scales are float32, one for each key/value head")
        if block_table is not None:
            _check_table(block_table)
            requests, cols = block_table.shape
            # the pitch of one row or none is never used
            pitch = block_table.stride(0) if requests > 1 else cols
            if pitch < cols:
                raise ValueError(f"a block table's rows may not overlap: {cols} entries, {pitch} apart")
            self.struct.block_table = block_table.data_ptr()
            self.struct.table_stride, self.struct.table_cols, self.requests = pitch, cols, requests
        self.ref = ctypes.byref(self.struct)


class Rope:
    """Rotary positions of a step's token rows (scute_rope).  ``cos_sin``: device
    float32 [n_pos, rotary_dim]; ``positions``: device int32 [n] or [axes, n];
    ``sections``: pairs of each axis (several axes)."""

    def __init__(self, cos_sin, positions, sections=None, interleaved=False):
        axes = 1 if positions.dim() == 1 else positions.shape[0]
        if positions.dtype is not _torch().int32 or (positions.stride(-1) != 1 and positions.shape[-1] > 1) or not 1 <= axes <= 4:
            raise ValueError("positions are int32, [n] or [axes, n] with at most 4 axes")
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.dtype is not _torch().float32:
            raise ValueError("cos_sin is a contiguous float32 table")
        if axes > 1 and (sections is None or len(sections) != axes):
            raise ValueError("several axes need a section each")
        self.tensors = (cos_sin, positions)
        self.n = positions.shape[-1]
        sec = (ctypes.c_int32 * 4)(*(list(sections)[:4] if axes > 1 else []))
        self.struct = _RopeStruct(cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1], 1 if interleaved else 0, axes,
                                  sec, positions.data_ptr(), positions.stride(0) if axes > 1 else 0)
        self.ref = ctypes.byref(self.struct)


class KvCaches:
    """The caches of a model's layers, of one type, size and layout, as
    ``kv_copy`` takes them (the tensors stay those of the ``KvCache`` objects)."""

    def __init__(self, caches):
        self.caches = tuple(caches)
        if not self.caches or not all(isinstance(c, KvCache) for c in self.caches):
            raise ValueError("KvCaches takes one KvCache or more")
        self.struct = (_KvCacheStruct * len(self.caches))(*(c.struct for c in self.caches))


class HeadNorm:
    """Norms of every head's queries and keys (scute_head_norm): ``q_w``, ``k_w``
    device float32 [head_dim], or [heads, head_dim] with weights for each head;
    None: not normed (one of them at least).  ``layer``: the mean is taken off
    first."""

    def __init__(self, q_w=None, k_w=None, eps: float = 1e-6, layer: bool = False):
        if q_w is None and k_w is None:
            raise ValueError("no weights to norm with")
        strides = []
        for w in (q_w, k_w):
            if w is not None and (w.dtype is not _torch().float32 or w.dim() not in (1, 2) or w.numel() == 0
                                  or (w.stride(-1) != 1 and w.shape[-1] > 1)
                                  or (w.dim() == 2 and w.shape[0] > 1 and w.stride(0) < w.shape[1])):
                raise ValueError("norm weights are float32 [head_dim] or [heads, head_dim] with consecutive rows")
            # one head's weights are everybody's
            strides.append(0 if w is None or w.dim() == 1 or w.shape[0] == 1 else w.stride(0))
        self.tensors = (q_w, k_w)
        self.struct = _HeadNormStruct(ptr(q_w), ptr(k_w), strides[0], strides[1], eps, 1 if layer else 0)
        self.ref = ctypes.byref(self.struct)

    def check(self, head_dim: int, q_heads: int, kv_heads: int):
        for w, heads in zip(self.tensors, (q_heads, kv_heads)):
            if w is not None and heads and (w.shape[-1] != head_dim or (w.dim() == 2 and w.shape[0] != heads)):
                raise ValueError(f"norm weights of {heads} heads of {head_dim} are [{head_dim}] or [{heads}, {head_dim}], "
                                 f"got {tuple(w.shape)}")


class Shared:
    """Groups of a batch whose requests share the beginnings of their contexts
    (scute_shared): requests ``start[g]`` .. ``start[g + 1] - 1`` the first ``length[g]``
    tokens (device int32 [groups + 1] and [groups]).  ``work``: a tensor of
    ``Context.shared_work``, for one call at a time.  ``always``: beginnings too short, or
    of too few requests, to gain from it are read for the group too."""

    def __init__(self, start, length, work, always: bool = False):
        _flat(_torch().int32, length.numel() + 1, start)
        _flat(_torch().int32, length.numel(), length)
        if not work.is_contiguous():
            raise ValueError("the workspace is consecutive bytes")
        self.tensors = (start, length, work)
        self.struct = _SharedStruct(ptr(start), ptr(length), ptr(work), work.nbytes, length.numel(), 1 if always else 0)
        self.ref = ctypes.byref(self.struct)


def _torch():
    """torch, which has been imported where there is a tensor to check."""
    return sys.modules["torch"]


def _check_table(t):
    if t.dim() != 2 or t.dtype is not _torch().int32 or (t.stride(1) != 1 and t.shape[1] > 1 and t.numel() > 1):
        raise ValueError("a block table is int32 [n_req, pages] with consecutive rows")


def _flat(dtype, count, *tensors):
    """Check that each is None or ``count`` consecutive elements of a type."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.numel() != count or not t.is_contiguous()):
            raise ValueError(f"expected {count} consecutive elements of {dtype}, got shape {tuple(t.shape)}, strides "
                             f"{t.stride()}, {t.dtype}")


def _rows(t, n, cols, dtype=None):
    """Elements between the rows of ``t``: [n, cols], or [n, heads, dim] with
    consecutive heads; elements of a type."""
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"expected elements of {dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if shape == (n, cols):
        ok = st[1] == 1 or cols == 1
    elif len(shape) == 3:
        ok = shape[0] == n and shape[1] * shape[2] == cols and st[2] == 1 and (st[1] == shape[2] or shape[1] == 1)
    else:
        ok = False
    if not ok and n:
        raise ValueError(f"expected {n} rows of {cols} consecutive elements, got shape {tuple(shape)}, strides {st}")
    return st[0] if n > 1 else cols          # one row's pitch is never used


_lib: Optional[ctypes.CDLL] = None

_SIGS = {
    "scute_version": (ctypes.c_int, []),
    "scute_create": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "scute_destroy": (None, [ctypes.c_void_p]),
    "scute_last_error": (ctypes.c_char_p, [ctypes.c_void_p]),
    "scute_add_layer": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_void_p]),
    "scute_set_shared": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "scute_register_adapter": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(LayerTensors),
                                              ctypes.c_int, ctypes.POINTER(ctypes.c_int32)]),
    "scute_unregister_adapter": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32]),
    "scute_linear": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                    ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "scute_linear_host": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "scute_linear_batch": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(Call), ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]),
    "scute_linear_batch_host": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(Call), ctypes.c_int,
                                               ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]),
    "scute_sync_status": (ctypes.c_int, [ctypes.c_void_p]),
    "scute_debug_index": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64] +
                          [ctypes.c_void_p] * 5 + [ctypes.c_void_p]),
    "scute_index_tokens_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p,
                                                  ctypes.c_int64] + [ctypes.c_void_p] * 7),
    "scute_byte_model": (ctypes.c_int, [ctypes.POINTER(BmLayer), ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(ByteReport)]),
    "scute_predict_bytes": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                           ctypes.c_int, ctypes.POINTER(ByteReport)]),
    "scute_byte_model_batch": (ctypes.c_int, [ctypes.POINTER(BmLayer), ctypes.c_int, ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.POINTER(ByteReport)]),
    "scute_predict_batch": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(Call), ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_int, ctypes.POINTER(ByteReport)]),
    "scute_predict_time": (ctypes.c_int, [ctypes.POINTER(ByteReport), ctypes.c_double, ctypes.c_double,
                                          ctypes.c_double, ctypes.POINTER(ctypes.c_double)]),
    "scute_kv_resize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_int64] + [ctypes.c_void_p] * 7 +
                        [ctypes.c_int64, ctypes.c_void_p]),
    "scute_rope_table": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_double, ctypes.c_void_p, ctypes.c_void_p]),
    "scute_kv_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "scute_kv_append_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "scute_kv_fork": (ctypes.c_int, [ctypes.c_void_p] * 3),
    "scute_kv_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
    "scute_paged_attention": (ctypes.c_int, [ctypes.c_void_p] * 4),
    "scute_paged_attention_shared": (ctypes.c_int, [ctypes.c_void_p] * 5),
    "scute_shared_bytes": (ctypes.c_int64, [ctypes.c_void_p] + [ctypes.c_int] * 4),
    "scute_paged_attention_sinks": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int32, ctypes.c_void_p]),
    "scute_residual_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                           ctypes.c_void_p]),
    "scute_launch_count": (ctypes.c_int64, [ctypes.c_void_p]),
    "scute_timing_enable": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "scute_timing_reset": (ctypes.c_int, [ctypes.c_void_p]),
    "scute_debug_inject": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "scute_debug_fail_alloc": (None, [ctypes.c_int]),
    "scute_set_variant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "scute_debug_step_plan": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_int)]),
    "scute_timing_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_float), ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int)]),
    "scute_timing_kinds": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int), ctypes.c_int,
                                          ctypes.POINTER(ctypes.c_int)]),
}


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libscute.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; "
                           "g.build()'` (the CUDA library is required; there is no fallback)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


_tensor = None          # torch.Tensor, once one has been given


def ptr(x) -> Optional[int]:
    """Address of a torch tensor, numpy array, int or None."""
    global _tensor
    if type(x) is _tensor:          # most calls' arguments
        return x.data_ptr()
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if type(x) is getattr(sys.modules.get("torch"), "Tensor", None):
            _tensor = type(x)
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("numpy array must be C-contiguous")
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream_handle(stream) -> Optional[int]:
    """The cudaStream_t to pass: an int as given, a torch stream's handle, or,
    for None, torch's current stream on the current device (so that calls
    made under ``torch.cuda.stream(s)`` are ordered with that stream's work)."""
    if stream is None:
        torch = sys.modules.get("torch")
        if torch is not None and torch.cuda.is_initialized():
            c = torch._C
            if hasattr(c, "_cuda_getCurrentRawStream"):     # the same handle without a Stream object
                return c._cuda_getCurrentRawStream(c._cuda_getDevice())
            return torch.cuda.current_stream().cuda_stream
        return None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(ctx, code: int):
    if code != 0:
        msg = _lib.scute_last_error(ctx).decode() if ctx else ""
        raise ScuteError(code, msg)


# ------------------------------------------------------------------ C ABI names
def scute_version() -> int:
    return load().scute_version()


def scute_create(device: int, dtype: int, max_tokens: int, max_adapters: int, max_layers: int) -> int:
    lib = load()
    h = ctypes.c_void_p()
    code = lib.scute_create(ctypes.byref(h), device, dtype, max_tokens, max_adapters, max_layers)
    if code != 0:
        raise ScuteError(code, "scute_create failed")
    return h.value


def scute_destroy(ctx: int) -> None:
    load().scute_destroy(ctx)


def scute_add_layer(ctx, layer, d_in, d_out, W):
    _check(ctx, load().scute_add_layer(ctx, layer, d_in, d_out, ptr(W)))


def scute_set_shared(ctx, layer, rank, A_sh, B_sh):
    _check(ctx, load().scute_set_shared(ctx, layer, rank, ptr(A_sh), ptr(B_sh)))


def scute_register_adapter(ctx, method: int, tensors: list) -> int:
    """tensors: list of dicts with keys layer, rank, c, A, B, d, e, s, b, R, magnitude, l."""
    arr = (LayerTensors * len(tensors))()
    for i, t in enumerate(tensors):
        arr[i].layer = t["layer"]
        arr[i].rank = int(t.get("rank", 0))
        arr[i].c = float(t.get("c", 1.0))
        for k in ("A", "B", "d", "e", "s", "b", "R", "magnitude", "l"):
            setattr(arr[i], k, ptr(t.get(k)))
    out = ctypes.c_int32()
    _check(ctx, load().scute_register_adapter(ctx, method, arr, len(tensors), ctypes.byref(out)))
    return out.value


def scute_unregister_adapter(ctx, adapter_id: int):
    _check(ctx, load().scute_unregister_adapter(ctx, adapter_id))


def scute_linear(ctx, x, adapter_ids, n, layer, out, out_dtype, stream=None):
    _check(ctx, load().scute_linear(ctx, ptr(x), ptr(adapter_ids), n, layer, ptr(out), out_dtype,
                                    _stream_handle(stream)))


def scute_linear_host(ctx, x_host, ids_host, n, layer, out_host, out_dtype, stream=None):
    _check(ctx, load().scute_linear_host(ctx, ptr(x_host), ptr(ids_host), n, layer, ptr(out_host),
                                         out_dtype, _stream_handle(stream)))


def _calls(calls):
    arr = (Call * max(1, len(calls)))()
    for i, (x, layer, out) in enumerate(calls):
        arr[i].x = ptr(x)
        arr[i].layer = layer
        arr[i].out = ptr(out)
    return arr


def scute_linear_batch(ctx, calls, adapter_ids, n, out_dtype, stream=None):
    """``calls``: sequence of (x, layer, out) with device tensors."""
    _check(ctx, load().scute_linear_batch(ctx, _calls(calls), len(calls), ptr(adapter_ids), n, out_dtype,
                                          _stream_handle(stream)))


def scute_linear_batch_host(ctx, calls, ids_host, n, out_dtype, stream=None):
    """``calls``: sequence of (x_host, layer, out_host) with host arrays."""
    _check(ctx, load().scute_linear_batch_host(ctx, _calls(calls), len(calls), ptr(ids_host), n, out_dtype,
                                               _stream_handle(stream)))


def scute_sync_status(ctx) -> int:
    return load().scute_sync_status(ctx)


def scute_debug_index(ctx, ids, n, perm, aid_sorted, seg_start, seg_aid, counts, stream=None):
    _check(ctx, load().scute_debug_index(ctx, ptr(ids), n, ptr(perm), ptr(aid_sorted), ptr(seg_start),
                                         ptr(seg_aid), ptr(counts), _stream_handle(stream)))


NOALLOC_MAX_ADAPTERS = 8192


def scute_index_tokens_noalloc(method_of_adapter, ids, n, perm, aid_sorted, seg_start, seg_aid, counts,
                               flags=None, stream=None):
    """Context-free indexing on the current device; ``method_of_adapter`` is a
    host int8 numpy array (method code per adapter id, -1 = none)."""
    import numpy as np
    tab = np.ascontiguousarray(method_of_adapter, dtype=np.int8)
    code = load().scute_index_tokens_noalloc(ptr(tab), int(tab.size), ptr(ids), n, ptr(perm), ptr(aid_sorted),
                                             ptr(seg_start), ptr(seg_aid), ptr(counts), ptr(flags),
                                             _stream_handle(stream))
    if code != 0:
        why = {1: "null output, n < 0, no adapters or a method code outside -1..5",
               8: f"n above {MAX_TOKENS} tokens or more than {NOALLOC_MAX_ADAPTERS} adapters "
                  "(size of the static method table)",
               9: "the current device is not sm_103", 6: "a CUDA call failed"}.get(code, "")
        raise ScuteError(code, why)


def scute_kv_resize(ctx, len_in, len_new, n_req, block_table, table_stride, table_cols, page_size, free_pages,
                    n_free_max, free_in, free_out, len_out, cu_new, slot_map, positions, token_req, max_new,
                    stream=None):
    _check(ctx, load().scute_kv_resize(ctx, ptr(len_in), ptr(len_new), n_req, ptr(block_table), table_stride,
                                       table_cols, page_size, ptr(free_pages), n_free_max, ptr(free_in),
                                       ptr(free_out), ptr(len_out), ptr(cu_new), ptr(slot_map), ptr(positions),
                                       ptr(token_req), max_new, _stream_handle(stream)))


def scute_rope_table(ctx, cos_sin, n_pos, rotary_dim, theta, inv_freq=None, stream=None):
    _check(ctx, load().scute_rope_table(ctx, ptr(cos_sin), n_pos, rotary_dim, theta, ptr(inv_freq),
                                        _stream_handle(stream)))


def scute_kv_append(ctx, cache: KvCache, slot_map, n, k, k_stride, v, v_stride, q=None, q_stride=0, q_heads=0,
                    q_out=None, q_out_stride=0, rope: Optional[Rope] = None, stream=None):
    _check(ctx, load().scute_kv_append(ctx, cache.ref, ptr(slot_map), n, ptr(k), k_stride, ptr(v), v_stride, ptr(q),
                                       q_stride, q_heads, ptr(q_out), q_out_stride,
                                       None if rope is None else rope.ref, _stream_handle(stream)))


def scute_kv_append_norm(ctx, cache: KvCache, slot_map, n, k, k_stride, v, v_stride, q=None, q_stride=0, q_heads=0,
                         q_out=None, q_out_stride=0, rope: Optional[Rope] = None, norm: Optional[HeadNorm] = None,
                         stream=None):
    _check(ctx, load().scute_kv_append_norm(ctx, cache.ref, ptr(slot_map), n, ptr(k), k_stride, ptr(v), v_stride,
                                            ptr(q), q_stride, q_heads, ptr(q_out), q_out_stride,
                                            None if rope is None else rope.ref, None if norm is None else norm.ref,
                                            _stream_handle(stream)))


def scute_kv_fork(ctx, table_in, len_in, table_in_stride, source, len_new, table_out, len_out, table_out_stride, n_in,
                  n_out, table_cols, page_size, n_pages, extra, free_pages, n_free_max, free_in, free_out, copy_from,
                  copy_to, copy_tokens, stream=None):
    at = lambda x: ptr(x) or 0  # noqa: E731
    f = _FORK.pack(at(table_in), at(len_in), table_in_stride, at(source), at(len_new), at(table_out), at(len_out),
                   table_out_stride, n_in, n_out, table_cols, page_size, n_pages, at(extra), at(free_pages), n_free_max,
                   at(free_in), at(free_out), at(copy_from), at(copy_to), at(copy_tokens))
    _check(ctx, load().scute_kv_fork(ctx, f, _stream_handle(stream)))


def scute_kv_copy(ctx, caches: KvCaches, copy_from, copy_to, tokens, n, stream=None):
    _check(ctx, load().scute_kv_copy(ctx, caches.struct, len(caches.caches), ptr(copy_from), ptr(copy_to), ptr(tokens), n,
                                     _stream_handle(stream)))


def scute_paged_attention(ctx, cache: KvCache, q, q_stride, out, out_stride, lse, kv_len, n_req, q_heads,
                          scale=0.0, softcap=0.0, window=0, stream=None, sinks=0, shared: Optional[Shared] = None):
    """``sinks``, ``shared``: scute_paged_attention_sinks, scute_paged_attention_shared where given."""
    a = _ATTENTION.pack(ptr(q) or 0, q_stride, ptr(out) or 0, out_stride, ptr(lse) or 0, ptr(kv_len) or 0, n_req,
                        q_heads, scale, softcap, window)
    if shared is not None:
        if sinks:
            raise ValueError("shared beginnings with a window's first tokens")
        _check(ctx, load().scute_paged_attention_shared(ctx, cache.ref, a, shared.ref, _stream_handle(stream)))
    elif sinks:
        _check(ctx, load().scute_paged_attention_sinks(ctx, cache.ref, a, sinks, _stream_handle(stream)))
    else:
        _check(ctx, load().scute_paged_attention(ctx, cache.ref, a, _stream_handle(stream)))


def scute_shared_bytes(ctx, n_req, q_heads, kv_heads, head_dim) -> int:
    n = load().scute_shared_bytes(ctx, n_req, q_heads, kv_heads, head_dim)
    if n < 0:
        raise ScuteError(2, f"no workspace for {n_req} requests of {q_heads} heads on {kv_heads} of {head_dim}")
    return n


def scute_residual_norm(ctx, n, d, y, y_stride, residual=None, residual_stride=0, residual_out=None,
                        residual_out_stride=0, out=None, out_stride=0, post_w=None, post_b=None, pre_w=None,
                        pre_b=None, gate_vec=None, gate_rows=None, gate_stride=0, scale=1.0, eps=1e-5, layer=False,
                        stream=None):
    a = _NORM.pack(ptr(y) or 0, y_stride, ptr(residual) or 0, residual_stride, ptr(residual_out) or 0,
                   residual_out_stride, ptr(out) or 0, out_stride, ptr(post_w) or 0, ptr(post_b) or 0, ptr(pre_w) or 0,
                   ptr(pre_b) or 0, ptr(gate_vec) or 0, ptr(gate_rows) or 0, gate_stride, scale, eps, 1 if layer else 0)
    _check(ctx, load().scute_residual_norm(ctx, a, n, d, _stream_handle(stream)))


def scute_byte_model(layer: BmLayer, ids_host, n) -> dict:
    rep = ByteReport()
    code = load().scute_byte_model(ctypes.byref(layer), ptr(ids_host), n, ctypes.byref(rep))
    if code != 0:
        raise ScuteError(code, "scute_byte_model failed")
    return rep.as_dict()


def scute_predict_bytes(ctx, ids_host, n, layer, out_dtype) -> dict:
    rep = ByteReport()
    _check(ctx, load().scute_predict_bytes(ctx, ptr(ids_host), n, layer, out_dtype, ctypes.byref(rep)))
    return rep.as_dict()


def scute_byte_model_batch(layers, ids_host, n) -> dict:
    """``layers``: sequence of BmLayer (one per call of the batch)."""
    arr = (BmLayer * max(1, len(layers)))(*layers)
    rep = ByteReport()
    code = load().scute_byte_model_batch(arr, len(layers), ptr(ids_host), n, ctypes.byref(rep))
    if code != 0:
        raise ScuteError(code, "scute_byte_model_batch failed")
    return rep.as_dict()


def scute_predict_batch(ctx, layers, ids_host, n, out_dtype) -> dict:
    """Launch list of a batched call over the given layer ids."""
    arr = (Call * max(1, len(layers)))()
    for i, layer in enumerate(layers):
        arr[i].layer = layer
    rep = ByteReport()
    _check(ctx, load().scute_predict_batch(ctx, arr, len(layers), ptr(ids_host), n, out_dtype, ctypes.byref(rep)))
    return rep.as_dict()


def scute_predict_time(report: dict, hbm_gbs: float, tensor_tflops: float, launch_us: float) -> float:
    """Predicted microseconds of a launch list (a report dict as returned above)."""
    rep = ByteReport()
    ks = report["kernels"]
    if len(ks) > BM_MAX_KERNELS:
        raise ValueError("too many launches")
    rep.n_kernels = len(ks)
    for i, (name, b, f) in enumerate(ks):
        rep.name[i].value = name.encode()[:23]
        rep.bytes[i] = int(b)
        rep.flops[i] = int(f)
    us = ctypes.c_double()
    code = load().scute_predict_time(ctypes.byref(rep), float(hbm_gbs), float(tensor_tflops), float(launch_us),
                                     ctypes.byref(us))
    if code != 0:
        raise ScuteError(code, "scute_predict_time failed")
    return us.value


def scute_launch_count(ctx) -> int:
    return load().scute_launch_count(ctx)


def scute_timing_enable(ctx, enable: bool):
    _check(ctx, load().scute_timing_enable(ctx, 1 if enable else 0))


def scute_timing_reset(ctx):
    _check(ctx, load().scute_timing_reset(ctx))


INJECT_STALL, INJECT_STALL_ATTENTION = 1, 2


def scute_debug_inject(ctx, what: int) -> None:
    _check(ctx, load().scute_debug_inject(ctx, what))


VARIANT_OFT_PASS, VARIANT_S_PASS = 1, 2


def scute_set_variant(ctx, flags: int) -> None:
    """Place OFT's rotation (1) and / or DoRA's and (IA)^3's s (2) in launches
    of their own around the decode step (byte-model validation)."""
    _check(ctx, load().scute_set_variant(ctx, int(flags)))


PLAN_HEAD, PLAN_CALL_FIELDS = 19, 18


def scute_debug_step_plan(ctx) -> list:
    """The last decode-step launch's plan as a list of ints (layout in scute.h)."""
    n = ctypes.c_int()
    _check(ctx, load().scute_debug_step_plan(ctx, None, 0, ctypes.byref(n)))
    buf = (ctypes.c_int64 * max(n.value, 1))()
    _check(ctx, load().scute_debug_step_plan(ctx, buf, n.value, ctypes.byref(n)))
    return [int(buf[i]) for i in range(n.value)]


def scute_debug_fail_alloc(k: int) -> None:
    """Make the k-th device allocation of the library from now fail as out of
    memory (test hook; k <= 0 switches it off)."""
    load().scute_debug_fail_alloc(int(k))


def scute_timing_read(ctx, max_slots: int = TIMING_SLOTS) -> list:
    buf = (ctypes.c_float * max_slots)()
    n = ctypes.c_int()
    _check(ctx, load().scute_timing_read(ctx, buf, max_slots, ctypes.byref(n)))
    return [float(buf[i]) for i in range(n.value)]


KIND_NAMES = ("step", "index", "rotate", "base_gemm", "lowrank", "vera_shrink", "vera_expand", "oft_pass", "s_pass",
              "kv_resize", "kv_append", "attention", "norm", "kv_fork", "kv_copy")


def scute_timing_kinds(ctx, max_slots: int = TIMING_SLOTS) -> list:
    buf = (ctypes.c_int * max_slots)()
    n = ctypes.c_int()
    _check(ctx, load().scute_timing_kinds(ctx, buf, max_slots, ctypes.byref(n)))
    return [KIND_NAMES[buf[i]] for i in range(n.value)]


from .context import Context  # noqa: E402,F401
