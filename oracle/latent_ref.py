"""64-bit references of the latent-attention calls, written from their
definitions; test infrastructure only.  Tensors are torch float64 on any device,
tables anything that indexes to integers; pools are ``[num_pages, 16, W]``."""
from __future__ import annotations

import math

import torch

from .paged_cache_ref import kv_length

PAGE = 16


def slots(page_indptr, page_values, length_info, b, device="cpu"):
    """(page, slot) of every row of sequence b."""
    r = torch.arange(kv_length(page_indptr, length_info, b), device=device)
    values = torch.as_tensor(page_values, device=device)
    return values[int(page_indptr[b]) + r // PAGE].long(), r % PAGE


def rows_of(pool, table, b):
    """The rows of sequence b; a page outside the pool reads zeros."""
    pid, sl = slots(*table, b, device=pool.device)
    inside = (pid >= 0) & (pid < pool.shape[0])
    rows = pool[torch.where(inside, pid, 0), sl]
    return torch.where(inside[:, None], rows, 0.0)


def visible(parent, qo, kv):
    """Which of a sequence's rows the last ``qo`` nodes of its tree see: those in
    front of the tree, themselves and their ancestors."""
    n = len(parent)
    seen = torch.zeros((n, kv), dtype=torch.bool)
    seen[:, :kv - n] = True
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, kv - n + j] = True
            j = int(parent[j])
    return seen[n - qo:]


def softmax_attention(q, k, v, seen, sm_scale):
    """q [h, rows, W], k [h or 1, kv, W], v [h or 1, kv, d], seen [rows, kv]: out
    [h, rows, d], base-2 lse [h, rows], and what bounds a kernel's rounding: the
    weights times |v| per output, the largest sum of |q k| per row (scaled, base
    2).  What is not seen has no part in any of them; nor has a row whose score
    is -inf."""
    h, n = q.shape[:2]
    out = torch.zeros((h, n, v.shape[-1]), dtype=torch.float64, device=q.device)
    mag, lse, smag = torch.zeros_like(out), torch.full_like(out[..., 0], -math.inf), \
        torch.zeros_like(out[..., 0])
    if k.shape[1] == 0 or n == 0:
        return out, lse, mag, smag
    seen = seen.to(q.device)
    x = (q @ k.transpose(1, 2) * sm_scale).masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m) & (m < 0), 0.0, m)
    w = torch.exp(x - m)
    z = w.sum(-1, keepdim=True)
    any_ = z[..., 0] != 0
    z = torch.where(z == 0, 1.0, z)
    clean = torch.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)
    # values that are not finite count where their weight is not zero
    odd = torch.where(torch.isfinite(v), 0.0, v)
    out = w @ clean / z
    for j in torch.nonzero((odd != 0).any(-1).any(0))[:, 0].tolist():
        out += torch.where((w[..., j:j + 1] != 0) & (odd[:, j:j + 1] != 0),
                           w[..., j:j + 1] * odd[:, j:j + 1], 0.0)
    mag = w @ clean.abs() / z
    lse = torch.where(any_, (m + torch.log(z))[..., 0] / math.log(2.0), -math.inf)
    s = (q.abs() @ torch.nan_to_num(k, nan=0.0, posinf=0.0, neginf=0.0).abs().transpose(1, 2))
    smag = s.masked_fill(~seen, 0.0).amax(-1) * abs(sm_scale) / math.log(2.0)
    return out, lse, mag, smag


def absorbed(q, pool, table, rank, sm_scale, q_rows=None, parents=None):
    """Attention over a latent cache: q [rows, h, W]; per sequence q_rows[b] of
    them, the last nodes of the tree with ``parents[b]`` (None: one row each that
    sees every row).  Returns out, lse, mag, smag as rows of heads."""
    parts, at = [], 0
    for b in range(len(table[2])):
        rows = rows_of(pool, table, b)
        n = 1 if q_rows is None else q_rows[b]
        seen = (torch.ones((1, len(rows)), dtype=torch.bool) if q_rows is None
                else visible(parents[b], n, len(rows)))
        r = softmax_attention(q[at:at + n].transpose(0, 1), rows[None], rows[None, :, :rank], seen,
                              sm_scale)
        parts.append([t.transpose(0, 1) for t in r])
        at += n
    return [torch.cat(t) for t in zip(*parts)]


def expanded(q, k, k_rope, v, q_rows, kv_rows, sm_scale):
    """Causal attention: q [rows, h, d + r], k, v [kv, h, d], k_rope [kv, r]."""
    parts, a, c = [], 0, 0
    h = q.shape[1]
    for n, m in zip(q_rows, kv_rows):
        shared = k_rope[c:c + m][:, None].expand(m, h, k_rope.shape[1])
        keys = torch.cat([k[c:c + m], shared], -1).transpose(0, 1)
        seen = torch.arange(m) <= torch.arange(m - n, m)[:, None]
        r = softmax_attention(q[a:a + n].transpose(0, 1), keys, v[c:c + m].transpose(0, 1), seen,
                              sm_scale)
        parts.append([t.transpose(0, 1) for t in r])
        a, c = a + n, c + m
    return [torch.cat(t) for t in zip(*parts)]


def norm(x, weight, eps):
    if weight is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight


def rotate(x, positions, layout, freq, magnitude=1.0):
    """Rotation of x [tokens, .., n] by positions * freq [n / 2]."""
    if layout is None:
        return x
    h = x.shape[-1] // 2
    lo = slice(0, h) if layout == "half" else slice(0, None, 2)
    hi = slice(h, None) if layout == "half" else slice(1, None, 2)
    turn = positions.double()[:, None] * freq
    turn = turn.view(turn.shape[0], *[1] * (x.dim() - 2), h)
    c, s = torch.cos(turn) * magnitude, torch.sin(turn) * magnitude
    y = x.clone()
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y
