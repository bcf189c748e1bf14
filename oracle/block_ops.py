"""Float64 definitions of the operators between the adapted projections: pages
and slots of a paged key/value cache, rotary positions and the cache write,
attention of one new token, and the residual norm.  Plain loops over requests
and rows; shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def ceil_div(a: int, b: int) -> int:
    return -(-a // b)


def resize(len_in, len_new, table, page_size, free, max_new):
    """One step's pages and slots.  ``free``: list of free pages, the top last.
    Returns a dict (table, free, len_out, cu_new, slot_map, positions,
    token_req, ok); ``ok`` is False when something was refused or out of range."""
    n, cols = table.shape
    cap = cols * page_size
    table, free, ok = table.copy(), list(free), True
    span = []
    for r in range(n):
        o, w = int(len_in[r]), int(len_new[r])
        if not 0 <= o <= cap:
            ok, o = False, min(max(o, 0), cap)
        if not 0 <= w <= cap:
            ok, w = False, o
        span.append((o, w))
    for r, (o, w) in enumerate(span):
        for b in range(ceil_div(w, page_size), ceil_div(o, page_size)):
            free.append(int(table[r, b]))
    budget, asked, rows, asked_rows = len(free), 0, [], 0
    len_out, cu = [], [0]
    for r, (o, w) in enumerate(span):
        if w <= o:
            len_out.append(w)
            cu.append(len(rows))
            continue
        have, want = ceil_div(o, page_size), ceil_div(w, page_size)
        asked += want - have
        fits = want == have or asked <= budget
        if fits:
            asked_rows += w - o
            fits = asked_rows <= max_new
        if not fits:
            ok = False
            len_out.append(o)
            cu.append(len(rows))
            continue
        for b in range(have, want):
            table[r, b] = free.pop()
        for pos in range(o, w):
            rows.append((int(table[r, pos // page_size]) * page_size + pos % page_size, pos, r))
        len_out.append(w)
        cu.append(len(rows))
    rows += [(-1, 0, -1)] * (max_new - len(rows))
    at = np.array(rows, np.int64).reshape(-1, 3)
    return {"table": table, "free": free, "len_out": np.array(len_out, np.int64), "cu_new": np.array(cu, np.int64),
            "slot_map": at[:, 0], "positions": at[:, 1], "token_req": at[:, 2], "ok": ok}


def rope(x, angle, rotary_dim, interleaved):
    """x [heads, dim], angle [rotary_dim / 2]: pairs turned by their angles."""
    y = x.astype(np.float64).copy()
    for i in range(rotary_dim // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
        c, s = math.cos(angle[i]), math.sin(angle[i])
        y[:, a] = x[:, a] * c - x[:, b] * s
        y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def attend(q, k, v, scale, softcap=0.0):
    """q [heads, dim] over k, v [tokens, dim] of their one key/value head.
    Returns (out, lse, mass, reach): mass = sum p |v| and reach = the largest
    scale * sum |q_i k_i|, which bound what rounding can do."""
    heads, dim = q.shape
    if len(k) == 0:
        return np.zeros((heads, dim)), np.full(heads, -np.inf), np.zeros((heads, dim)), np.zeros(heads)
    s = scale * (q @ k.T)
    reach = abs(scale) * (np.abs(q) @ np.abs(k).T).max(1)
    if softcap:
        s = softcap * np.tanh(s / softcap)
    top = s.max(1, keepdims=True)
    p = np.exp(s - top)
    total = p.sum(1, keepdims=True)
    p /= total
    return p @ v, (top + np.log(total))[:, 0], p @ np.abs(v), reach


def norm(x, w, b, eps, layer):
    if layer:
        x = x - x.mean(1, keepdims=True)
    x = x / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    if w is not None:
        x = x * w
    return x if b is None else x + b


def residual_norm(y, residual, post, pre, gate, scale, eps, layer):
    """(h, out); post and pre are (w, b) or None."""
    t = y if post is None else norm(y, post[0], post[1], eps, layer)
    if gate is not None:
        t = t * gate
    h = scale * t + (0.0 if residual is None else residual)
    return h, None if pre is None else norm(h, pre[0], pre[1], eps, layer)
