"""A small owner object around a scute context handle (marshalling only)."""
from __future__ import annotations

import numpy as np

from . import (BF16, FP32, METHOD_ID, KvCache, Rope, _check_table, _flat, _rows, _torch, scute_add_layer, scute_create, scute_debug_index, scute_destroy,
               scute_kv_append, scute_kv_resize, scute_launch_count, scute_linear, scute_linear_batch, scute_linear_batch_host,
               scute_linear_host, scute_paged_attention, scute_predict_batch, scute_predict_bytes,
               scute_register_adapter, scute_residual_norm, scute_rope_table, scute_set_shared, scute_set_variant, scute_sync_status,
               scute_timing_enable,
               scute_timing_kinds, scute_timing_read, scute_timing_reset, scute_unregister_adapter)


class Context:
    """Owns one scute context; every method is one C ABI call."""

    def __init__(self, dtype: str = "bf16", max_tokens: int = 1024, max_adapters: int = 64,
                 max_layers: int = 16, device: int = 0):
        self.dtype = dtype
        self.device = device
        self.max_tokens = max_tokens
        self.handle = scute_create(device, BF16 if dtype == "bf16" else FP32, max_tokens, max_adapters,
                                   max_layers)
        self.layer_ids = {}          # layer name -> id
        self.layer_dims = {}         # id -> (d_in, d_out)

    def close(self):
        if self.handle:
            scute_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ---------------------------------------------------------------- setup
    def add_layer(self, layer: int, d_in: int, d_out: int, W):
        scute_add_layer(self.handle, layer, d_in, d_out, W)
        self.layer_dims[layer] = (d_in, d_out)

    def set_shared(self, layer: int, rank: int, A_sh, B_sh):
        scute_set_shared(self.handle, layer, rank, A_sh, B_sh)

    def register(self, method: str, tensors: list) -> int:
        return scute_register_adapter(self.handle, METHOD_ID[method], tensors)

    def unregister(self, adapter_id: int):
        scute_unregister_adapter(self.handle, adapter_id)

    def load_workload(self, w, layer_names=None, drop_host: bool = False):
        """Register the layers, shared pairs and adapters of a synthetic workload
        (``workloads.Workload``) in order, so that adapter ids match."""
        names = [L.name for L in w.layers] if layer_names is None else list(layer_names)
        for L in w.layers:
            if L.name not in names:
                continue
            lid = len(self.layer_ids)
            self.layer_ids[L.name] = lid
            self.add_layer(lid, L.d_in, L.d_out, np.ascontiguousarray(L.get("W")))
            if L.shared_rank:
                self.set_shared(lid, L.shared_rank, np.ascontiguousarray(L.get("A_sh")),
                                np.ascontiguousarray(L.get("B_sh")))
            if drop_host:
                L._cache.pop("W", None)
                L._cache.pop("A_sh", None)
                L._cache.pop("B_sh", None)
        for a in sorted(w.adapters, key=lambda a: a.id):
            tens = []
            for lname in a.layers:
                if lname not in self.layer_ids:
                    continue
                t = {"layer": self.layer_ids[lname], "rank": a.rank, "c": a.c}
                for slot in a.slots(lname):
                    key = {"m": "magnitude"}.get(slot, slot)
                    t[key] = np.ascontiguousarray(a.get(lname, slot))
                tens.append(t)
            # an adapter with no tensors on the chosen layers has identity slots there
            aid = self.register(a.method, tens)
            if aid != a.id:
                raise RuntimeError(f"adapter id mismatch: library gave {aid}, workload has {a.id}")
            if drop_host:
                a.drop()

    # ---------------------------------------------------------------- hot path
    def linear(self, x, ids, layer: int, out, out_dtype: str = "bf16", stream=None, n=None):
        n = int(ids.shape[0]) if n is None else n
        scute_linear(self.handle, x, ids, n, layer, out, BF16 if out_dtype == "bf16" else FP32, stream)

    def linear_host(self, x_host, ids_host, layer: int, out_host, out_dtype: str = "bf16", stream=None):
        scute_linear_host(self.handle, x_host, ids_host, int(ids_host.shape[0]), layer, out_host,
                          BF16 if out_dtype == "bf16" else FP32, stream)

    def linear_batch(self, calls, ids, out_dtype: str = "bf16", stream=None, n=None):
        """``calls``: sequence of (x, layer id, out); every layer sees the same ids."""
        n = int(ids.shape[0]) if n is None else n
        scute_linear_batch(self.handle, list(calls), ids, n, BF16 if out_dtype == "bf16" else FP32, stream)

    def linear_batch_host(self, calls, ids_host, out_dtype: str = "bf16", stream=None):
        scute_linear_batch_host(self.handle, list(calls), ids_host, int(ids_host.shape[0]),
                                BF16 if out_dtype == "bf16" else FP32, stream)

    # ---------------------------------------------------------------- between the projections
    _types = None

    def _dtypes(self):
        """torch's types of rows, of whole numbers and of vectors, looked up at the first call."""
        if self._types is None:
            t = _torch()
            self._types = t.bfloat16 if self.dtype == "bf16" else t.float32, t.int32, t.float32
        return self._types

    def kv_resize(self, len_in, len_new, block_table, page_size: int, free_pages, free_in, free_out, len_out, cu_new,
                  slot_map, positions, token_req, stream=None):
        """Pages for every request's new length, slots for its new tokens (device
        int32 tensors; scute.h has the layout).  The step has ``slot_map.numel()``
        token rows."""
        _check_table(block_table)
        n, (requests, cols) = len_in.numel(), block_table.shape
        rows, n_free = slot_map.numel(), free_pages.numel()
        if not (len_in.dtype is len_new.dtype is len_out.dtype is cu_new.dtype is free_in.dtype is free_out.dtype
                is slot_map.dtype is positions.dtype is token_req.dtype is free_pages.dtype is self._dtypes()[1]
                and requests >= n and len_new.nbytes == len_out.nbytes == 4 * n
                and cu_new.nbytes == 4 * n + 4 and free_in.nbytes == free_out.nbytes == 4
                and positions.nbytes == token_req.nbytes == 4 * rows
                and len_in.is_contiguous() and len_new.is_contiguous() and len_out.is_contiguous()
                and cu_new.is_contiguous() and slot_map.is_contiguous() and positions.is_contiguous()
                and token_req.is_contiguous() and free_pages.is_contiguous()):
            raise ValueError("kv_resize takes consecutive int32 elements: lengths of the requests, a count of free "
                             "pages, cu_new one longer, token rows of one number, and a table row for each request")
        scute_kv_resize(self.handle, len_in, len_new, n, block_table,
                        block_table.stride(0) if requests > 1 else max(cols, block_table.stride(0)), cols,
                        page_size, free_pages, n_free, free_in, free_out, len_out, cu_new, slot_map,
                        positions, token_req, rows, stream)

    def rope_table(self, cos_sin, theta: float = 10000.0, inv_freq=None, stream=None):
        """Fill the float32 table ``cos_sin`` [n_pos, rotary_dim]; ``inv_freq``:
        float64 [rotary_dim / 2]."""
        if cos_sin.dim() != 2 or not cos_sin.is_contiguous() or cos_sin.dtype is not _torch().float32:
            raise ValueError("cos_sin is a contiguous float32 table")
        if inv_freq is not None and (inv_freq.dtype is not _torch().float64 or not inv_freq.is_contiguous()
                                     or 2 * inv_freq.numel() != cos_sin.shape[1]):
            raise ValueError("inv_freq is consecutive float64, one for each pair")
        scute_rope_table(self.handle, cos_sin, cos_sin.shape[0], cos_sin.shape[1], theta, inv_freq, stream)

    def kv_append(self, cache: KvCache, slot_map, k, v, q=None, q_out=None, rope: Rope = None, stream=None):
        """Write k and v [n, kv_heads, dim] (or [n, kv_heads * dim]) into the cache;
        keys, and queries into ``q_out``, turned by ``rope``."""
        n, row, (io, int32, _) = slot_map.shape[0], cache.kv_row, self._dtypes()
        _flat(int32, n, slot_map)
        q_heads = q_stride = q_out_stride = 0
        if q is not None:
            q_row = q.numel() // n if n else cache.head_dim
            q_heads = q_row // cache.head_dim
            if q_out is None or q_heads * cache.head_dim != q_row:
                raise ValueError("q rows are heads * head_dim elements, and need q_out")
            q_stride, q_out_stride = _rows(q, n, q_row, io), _rows(q_out, n, q_row, io)
        if rope is not None and rope.n < n:
            raise ValueError("fewer positions than rows")
        scute_kv_append(self.handle, cache, slot_map, n, k, _rows(k, n, row, io), v, _rows(v, n, row, io), q, q_stride,
                        q_heads, q_out, q_out_stride, rope, stream)

    def paged_attention(self, cache: KvCache, q, kv_len, out, scale: float = 0.0, softcap: float = 0.0,
                        window: int = 0, lse=None, stream=None):
        """One new token of each request over its cached tokens: q and out
        [n_req, q_heads, dim] (or [n_req, q_heads * dim])."""
        n, dim, (io, int32, float32) = kv_len.shape[0], cache.head_dim, self._dtypes()
        row = q.numel() // n if n else cache.kv_row
        if row % dim or cache.requests < n:
            raise ValueError("q rows are heads * head_dim elements, and the block table has a row for each request")
        _flat(int32, n, kv_len)
        _flat(float32, n * row // dim, lse)
        scute_paged_attention(self.handle, cache, q, _rows(q, n, row, io), out, _rows(out, n, row, io), lse, kv_len, n,
                              row // dim, scale, softcap, window, stream)

    def residual_norm(self, y, out=None, residual=None, residual_out=None, pre_w=None, pre_b=None, post_w=None,
                      post_b=None, gate=None, scale: float = 1.0, eps: float = 1e-5, layer: bool = False, stream=None):
        """h = residual + scale * gate * post(y), out = pre(h), for rows [n, d].
        ``gate``: float32 [d], or the context's dtype [n, d]."""
        (n, d), (io, _, float32) = y.shape, self._dtypes()
        gate_vec, gate_rows = (None, gate) if gate is not None and gate.dim() == 2 else (gate, None)
        _flat(float32, d, post_w, post_b, pre_w, pre_b, gate_vec)
        scute_residual_norm(self.handle, n, d, y, _rows(y, n, d, io),
                            residual, 0 if residual is None else _rows(residual, n, d, io),
                            residual_out, 0 if residual_out is None else _rows(residual_out, n, d, io),
                            out, 0 if out is None else _rows(out, n, d, io), post_w, post_b, pre_w, pre_b, gate_vec,
                            gate_rows, 0 if gate_rows is None else _rows(gate_rows, n, d, io), scale, eps, layer, stream)

    def sync_status(self) -> int:
        return scute_sync_status(self.handle)

    def debug_index(self, ids, n, perm, aid_sorted, seg_start, seg_aid, counts, stream=None):
        scute_debug_index(self.handle, ids, n, perm, aid_sorted, seg_start, seg_aid, counts, stream)

    def predict_bytes(self, ids_host, layer: int, out_dtype: str = "bf16") -> dict:
        ids_host = np.ascontiguousarray(ids_host, dtype=np.int32)
        return scute_predict_bytes(self.handle, ids_host, int(ids_host.size), layer,
                                   BF16 if out_dtype == "bf16" else FP32)

    def predict_batch(self, layers, ids_host, out_dtype: str = "bf16") -> dict:
        ids_host = np.ascontiguousarray(ids_host, dtype=np.int32)
        return scute_predict_batch(self.handle, list(layers), ids_host, int(ids_host.size),
                                   BF16 if out_dtype == "bf16" else FP32)

    def set_variant(self, flags: int):
        scute_set_variant(self.handle, flags)

    def launch_count(self) -> int:
        return scute_launch_count(self.handle)

    def timing(self, enable: bool):
        scute_timing_enable(self.handle, enable)

    def timing_reset(self):
        scute_timing_reset(self.handle)

    def timing_read(self) -> list:
        return scute_timing_read(self.handle)

    def timing_kinds(self) -> list:
        return scute_timing_kinds(self.handle)
