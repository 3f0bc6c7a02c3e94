"""64-bit references of the paged-cache calls (append, one-token attention,
compaction, page copies), written from their definitions; test infrastructure
only.  Arrays are numpy; pools are float64 ``[num_pages, 2, h_kv, 16, d]``."""
from __future__ import annotations

import numpy as np

PAGE = 16


def kv_length(page_indptr, length_info, b):
    n = int(page_indptr[b + 1]) - int(page_indptr[b])
    return (n - 1) * PAGE + int(length_info[b]) if n > 0 else 0


def slots(page_indptr, page_values, length_info, b):
    """(page, slot) of every kv row of sequence b."""
    n = kv_length(page_indptr, length_info, b)
    r = np.arange(n)
    return np.asarray(page_values)[int(page_indptr[b]) + r // PAGE].astype(np.int64), r % PAGE


def decode(q, pages, page_indptr, page_values, length_info, sm_scale):
    """out, base-2 lse, and two sums that bound a kernel's rounding: for every
    output the weights times |v|, for every row the largest sum of |q k|
    (scaled, base 2).  A page outside the pool reads zeros."""
    B, h_q, d = q.shape
    h_kv = pages.shape[2]
    g = h_q // h_kv
    out = np.zeros((B, h_q, d))
    mag = np.zeros((B, h_q, d))
    lse = np.full((B, h_q), -np.inf)
    smag = np.zeros((B, h_q))
    for b in range(B):
        pid, sl = slots(page_indptr, page_values, length_info, b)
        if not len(pid):
            continue
        inside = (pid >= 0) & (pid < pages.shape[0])
        kv = pages[np.where(inside, pid, 0), :, :, sl]           # [rows, 2, h_kv, d]
        kv = np.where(inside[:, None, None, None], kv, 0.0)
        for h in range(h_q):
            k, v = kv[:, 0, h // g], kv[:, 1, h // g]
            x = (k @ q[b, h]) * sm_scale
            m = x.max()
            w = np.exp(x - m)
            out[b, h] = w @ v / w.sum()
            mag[b, h] = w @ np.abs(v) / w.sum()
            lse[b, h] = (m + np.log(w.sum())) / np.log(2.0)
            smag[b, h] = (np.abs(k) @ np.abs(q[b, h])).max() * abs(sm_scale) / np.log(2.0)
    return out, lse, mag, smag


def norm(x, weight, eps):
    """Root-mean-square norm of every head row."""
    if weight is None:
        return x
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * weight


def rotate(x, positions, layout, rotary_dim, freq, magnitude=1.0):
    """Rotation of x [tokens, heads, d] by positions * freq [rotary_dim / 2]."""
    if layout is None:
        return x
    h = rotary_dim // 2
    lo = slice(0, h) if layout == "half" else slice(0, rotary_dim, 2)
    hi = slice(h, rotary_dim) if layout == "half" else slice(1, rotary_dim, 2)
    z = (x[..., lo] + 1j * x[..., hi]) * magnitude
    z = z * np.exp(1j * (np.asarray(positions, dtype=np.float64)[:, None] * freq))[:, None]
    y = x.copy()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def append(pool, k, v, append_indptr, page_indptr, page_values, length_info):
    """The pool with the new rows in the last slots of their sequences."""
    pool = pool.copy()
    for b in range(len(length_info)):
        a, e = int(append_indptr[b]), int(append_indptr[b + 1])
        pid, sl = slots(page_indptr, page_values, length_info, b)
        for i in range(e - a):
            r = len(pid) - (e - a) + i
            pool[pid[r], 0, :, sl[r]] = k[a + i]
            pool[pid[r], 1, :, sl[r]] = v[a + i]
    return pool


def compact(pool, page_indptr, page_values, length_info, mn_indptr, accept_indptr, accept_nodes):
    """pool, page_indptr, page_values, length_info after it, and the freed pages."""
    old, pool = pool, pool.copy()
    new_values, new_indptr, new_len, freed = [], [0], [], []
    for b in range(len(length_info)):
        pid, sl = slots(page_indptr, page_values, length_info, b)
        t0 = len(pid) - int(mn_indptr[b + 1] - mn_indptr[b])
        path = accept_nodes[int(accept_indptr[b]):int(accept_indptr[b + 1])]
        for j, node in enumerate(path):
            pool[pid[t0 + j], :, :, sl[t0 + j]] = old[pid[t0 + node], :, :, sl[t0 + node]]
        rows = t0 + len(path)
        keep = -(-rows // PAGE)
        mine = list(page_values[int(page_indptr[b]):int(page_indptr[b + 1])])
        new_values += mine[:keep]
        freed += mine[keep:]
        new_indptr.append(new_indptr[-1] + keep)
        new_len.append(rows - (keep - 1) * PAGE if keep else 0)
    return pool, new_indptr, new_values, new_len, freed
