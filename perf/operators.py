"""Cases for the paged-cache operators: appending tokens to the cache (with the
norm and rotation of queries and keys), attention of one new token per sequence
over it, compaction after a draft tree was verified, and copies of pages.

``run`` computes each operator in elementary torch operations, or, with ``own``,
through ``tree_attention_gb300.PagedCache``.  ``exact`` gives the same outputs
in 64 bits from the definitions.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _decode(name, batch, lo, hi, h_q, h_kv, d, dtype, shape):
    return {"name": name, "op": "decode", "batch": batch, "lo": lo, "hi": hi, "h_q": h_q,
            "h_kv": h_kv, "d": d, "dtype": dtype, "shape": shape}


def _append(name, batch, lo, hi, ctx, h_q, h_kv, d, dtype, norm, layout, rotary_dim, theta, scale,
            shape):
    return {"name": name, "op": "append", "batch": batch, "lo": lo, "hi": hi, "ctx": ctx,
            "h_q": h_q, "h_kv": h_kv, "d": d, "dtype": dtype, "norm": norm, "layout": layout,
            "rotary_dim": rotary_dim, "theta": theta, "scale": scale, "shape": shape}


def _compact(name, batch, nodes, depth, ctx, h_kv, d, dtype, shape):
    return {"name": name, "op": "compact", "batch": batch, "nodes": nodes, "depth": depth,
            "ctx": ctx, "h_kv": h_kv, "d": d, "dtype": dtype, "shape": shape}


def _copy(name, n, h_kv, d, dtype):
    return {"name": name, "op": "copy", "n": n, "h_kv": h_kv, "d": d, "dtype": dtype}


def listed():
    return [
        # the smallest call: two short chats, the sizes of the "tiny" workload; launch latency
        _decode("decode-tiny", 2, 7, 12, 4, 2, 64, "fp16", 1),
        # one user's chat, keys and values of every head (the "degenerate" workload's heads)
        _decode("decode-one", 1, 4096, 4096, 16, 16, 128, "fp16", 2),
        # a small server: 32 chats of about a thousand tokens (the "spec-decode" workload's heads)
        _decode("decode-chats", 32, 500, 1500, 32, 8, 128, "bf16", 3),
        # four long documents (the "long-prefix" workload): the cache's length has to be split
        _decode("decode-long", 4, 32000, 33600, 32, 8, 128, "bf16", 4),
        # a full server: ragged lengths from a page to 16k tokens (the "ragged-large" heads)
        _decode("decode-server", 64, 16, 16384, 64, 8, 128, "bf16", 5),
        # one new token for each of 32 chats far into long contexts, with norms of q and k
        _append("append-token", 32, 1, 1, 60000, 32, 8, 128, "bf16", True, "half", 128, 5e5, 1.0, 6),
        # a draft tree of 64 nodes for each of 32 chats, before its verification
        _append("append-tree", 32, 64, 64, 1000, 32, 8, 128, "bf16", False, "half", 128, 1e4, 1.0, 7),
        # prompts of 16 to 512 tokens for 64 chats; interleaved pairs on half of the head, positions
        # scaled for a longer context
        _append("append-prompt", 64, 16, 512, 0, 64, 8, 128, "fp16", True, "interleaved", 64, 1e4,
                0.25, 8),
        # after the verification of 32 draft trees of 64 nodes
        _compact("compact-draft", 32, 64, 8, 1000, 8, 128, "bf16", 9),
        # the same for 512 sequences, with long accepted paths
        _compact("compact-wide", 512, 64, 24, 2000, 8, 128, "bf16", 10),
        # 32 chats forked: the partly filled last page of each
        _copy("copy-fork", 32, 8, 128, "bf16"),
        # a prefix of 64k tokens moved to other pages
        _copy("copy-prefix", 4096, 8, 128, "bf16"),
    ]


HEADS = {128: [(4, 2), (32, 8), (64, 8), (16, 16), (8, 1), (18, 2), (40, 8), (32, 1)],
         64: [(4, 2), (64, 8), (8, 1), (18, 2), (40, 8), (12, 4)]}


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "compact", "copy"])
    d = rng.choice([128, 128, 64])
    dtype = rng.choice(["bf16", "fp16"])
    h_q, h_kv = rng.choice(HEADS[d])
    shape = rng.randrange(1 << 30)
    if op == "decode":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(40000, 2000000 // (batch * h_kv))))
        lo = 0 if batch > 4 and rng.random() < 0.3 else rng.randint(1, hi)
        c = _decode("", batch, lo, hi, h_q, h_kv, d, dtype, shape)
    elif op == "append":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, 12000 // batch))
        layout = rng.choice(["half", "interleaved", "none"])
        c = _append("", batch, rng.randint(1, hi), hi, _log(rng, 1, 4000), h_q, h_kv, d, dtype,
                    rng.random() < 0.5, layout, rng.choice([16, d // 2, d]),
                    rng.choice([1e4, 5e5]), rng.choice([1.0, 0.25, 0.125]), shape)
    elif op == "compact":
        nodes = _log(rng, 1, 200)
        c = _compact("", _log(rng, 1, 400), nodes, rng.randint(1, nodes), _log(rng, 1, 2000), h_kv,
                     d, dtype, shape)
    else:
        c = _copy("", _log(rng, 1, 4000), h_kv, d, dtype)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _between(case, key_lo, key_hi, salt):
    """``batch`` sizes of the case's range: log-uniform, the first the largest."""
    r = random.Random(case["shape"] * 7 + salt)
    lo, hi = case[key_lo], case[key_hi]
    n = [int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))))) - 1
         for _ in range(case["batch"])]
    n[0] = hi
    return [min(hi, max(lo, x)) for x in n]


def _sizes(case):
    """Host sizes of a case: kv lengths, new tokens, accepted nodes."""
    r = random.Random(case.get("shape", 0) * 7 + 3)
    if case["op"] == "decode":
        return {"kv": _between(case, "lo", "hi", 1)}
    if case["op"] == "append":
        new = _between(case, "lo", "hi", 1)
        # the cache holds a part of the context's rows; the positions count all of it
        ctx = [r.randint(case["ctx"] // 2, case["ctx"]) for _ in new]
        held = [min(c, 2000) for c in ctx]
        return {"new": new, "ctx": ctx, "kv": [h + n for h, n in zip(held, new)]}
    if case["op"] == "compact":
        ctx = [r.randint(case["ctx"] // 2, case["ctx"]) for _ in range(case["batch"])]
        acc = [r.randint(1, case["depth"]) for _ in ctx]
        return {"kv": [c + case["nodes"] for c in ctx], "acc": acc}
    return {}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _table(case, kv, seed, gen):
    """A page pool with a scattered page table for kv lengths ``kv``."""
    kv = np.asarray(kv, dtype=np.int64)
    n_pages = (kv + PAGE - 1) // PAGE
    nnz = int(n_pages.sum())
    pool = nnz + 5
    perm = np.random.default_rng(seed).permutation(pool)[:nnz]
    indptr = np.concatenate([[0], np.cumsum(n_pages)])
    last = np.where(n_pages > 0, kv - (n_pages - 1) * PAGE, 0)
    pages = _randn(gen, (pool, 2, case["h_kv"], PAGE, case["d"]), DTYPES[case["dtype"]])
    return {"pages": pages, "page_indptr": _i32(indptr), "page_values": _i32(perm),
            "length_info": _i32(last), "max_pages": int(n_pages.max())}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    h_kv, d = case["h_kv"], case["d"]
    size = _sizes(case)
    s = {"case": case}
    if case["op"] == "copy":
        n = case["n"]
        perm = np.random.default_rng(seed).permutation(2 * n + 3)
        s["pages"] = _randn(gen, (2 * n + 3, 2, h_kv, PAGE, d), dt)
        s["src"], s["dst"] = _i32(perm[:n]), _i32(perm[n:2 * n])
        s["h_q"] = h_kv
        s["page_indptr"], s["page_values"], s["length_info"] = _i32([0, 1]), _i32([0]), _i32([PAGE])
    else:
        s.update(_table(case, size["kv"], seed, gen))
        s["h_q"] = case.get("h_q", h_kv)
    if case["op"] == "decode":
        s["q"] = _randn(gen, (case["batch"], case["h_q"], d), dt)
        s["sm_scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    elif case["op"] == "append":
        h_q, n = case["h_q"], sum(size["new"])
        qkv = _randn(gen, (n, h_q + 2 * h_kv, d), dt)      # one fused projection's output
        s["q"], s["k"], s["v"] = qkv[:, :h_q], qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:]
        s["append_indptr"] = _i32(np.concatenate([[0], np.cumsum(size["new"])]))
        s["positions"] = _i32(np.concatenate([np.arange(c, c + m)
                                              for c, m in zip(size["ctx"], size["new"])]))
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * _randn(gen, (d,), torch.float32)).to(dt)
            s["k_weight"] = (1 + 0.1 * _randn(gen, (d,), torch.float32)).to(dt)
        s["eps"] = 1e-6
        s["q_out"] = torch.empty((n, h_q, d), dtype=dt, device=DEV)
    elif case["op"] == "compact":
        rng = np.random.default_rng(seed)
        nodes = case["nodes"]
        # an accepted path: the root, then ever later nodes
        path = [np.concatenate([[0], 1 + np.sort(rng.permutation(nodes - 1)[:a - 1])])
                for a in size["acc"]]
        s["tree_indptr"] = _i32(np.arange(case["batch"] + 1) * nodes)
        s["accept_indptr"] = _i32(np.concatenate([[0], np.cumsum(size["acc"])]))
        s["accept_nodes"] = _i32(np.concatenate(path))
        nnz = s["page_values"].numel()
        s["new_indptr"] = torch.full_like(s["page_indptr"], -1)
        s["new_values"] = torch.full((nnz,), -1, dtype=torch.int32, device=DEV)
        s["new_length"] = torch.full_like(s["length_info"], -1)
        s["freed"] = torch.full((nnz,), -1, dtype=torch.int32, device=DEV)
        s["num_freed"] = torch.full((1,), -1, dtype=torch.int32, device=DEV)
    if own:
        import tree_attention_gb300 as ta
        s["cache"] = ta.PagedCache(s["pages"], s["page_indptr"], s["page_values"],
                                   s["length_info"], h_q=s["h_q"])
        if case["op"] == "append" and case["layout"] != "none":
            s["rope"] = ta.Rope(case["layout"], case["rotary_dim"], theta=case["theta"],
                                scale=case["scale"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        c = s["cache"]
        if op == "decode":
            c.decode(s["q"], s["sm_scale"], out=s["out"], lse=s["lse"])
            return s["out"], s["lse"]
        if op == "append":
            c.append(s["q"], s["k"], s["v"], s["append_indptr"], s["positions"],
                     rope=s.get("rope"), q_weight=s["q_weight"], k_weight=s["k_weight"],
                     norm_eps=s["eps"], q_out=s["q_out"])
            return s["q_out"], s["pages"]
        if op == "compact":
            c.compact(s["tree_indptr"], s["accept_indptr"], s["accept_nodes"],
                      new_page_indptr=s["new_indptr"], new_page_values=s["new_values"],
                      new_length_info=s["new_length"], freed_pages=s["freed"],
                      num_freed=s["num_freed"])
            return (s["pages"], s["new_indptr"], s["new_values"], s["new_length"], s["freed"],
                    s["num_freed"])
        c.copy_pages(s["src"], s["dst"])
        return s["pages"]
    return {"decode": _plain_decode, "append": _plain_append, "compact": _plain_compact,
            "copy": _plain_copy}[op](s)


def _kv_lengths(s):
    n = s["page_indptr"][1:].long() - s["page_indptr"][:-1].long()
    return n, torch.where(n > 0, (n - 1) * PAGE + s["length_info"].long(), 0)


def _slots(s, seq, row):
    """Physical page and slot of kv row ``row`` of sequence ``seq``."""
    return s["page_values"][s["page_indptr"][seq].long() + row // PAGE].long(), row % PAGE


def _sequence_of(indptr, n):
    """The sequence that each of the ``n`` entries of a CSR list belongs to."""
    return torch.searchsorted(indptr[1:].long(), torch.arange(n, device=DEV), right=True)


def _plain_decode(s):
    c = s["case"]
    b, h_kv, d, g = c["batch"], c["h_kv"], c["d"], c["h_q"] // c["h_kv"]
    n_pages, kv = _kv_lengths(s)
    cols = torch.arange(max(1, s["max_pages"]), device=DEV)
    at = s["page_indptr"][:-1].long()[:, None] + cols
    pid = s["page_values"][at.clamp(max=s["page_values"].numel() - 1)].long()
    got = s["pages"][pid]                                  # [b, pages, 2, h_kv, 16, d]
    k = got[:, :, 0].permute(0, 2, 1, 3, 4).reshape(b, h_kv, -1, d).float()
    v = got[:, :, 1].permute(0, 2, 1, 3, 4).reshape(b, h_kv, -1, d).float()
    x = s["q"].float().view(b, h_kv, g, d) @ k.transpose(2, 3) * s["sm_scale"]
    seen = torch.arange(k.shape[2], device=DEV) < kv[:, None]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    out = (p @ v) / z.clamp(min=1e-30)
    lse = (m + torch.log(z)) / math.log(2.0)
    lse = torch.where(z > 0, lse, -math.inf)
    return out.view(b, -1, d).to(s["q"].dtype), lse.view(b, -1)


def _plain_norm(x, w, eps):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.float()


def _plain_rotate(x, cos, sin, layout, rd):
    if layout == "none":
        return x
    r, rest = x[..., :rd], x[..., rd:]
    if layout == "half":
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)
    a, b = r[..., 0::2], r[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)


def _plain_append(s):
    c = s["case"]
    rd, n = c["rotary_dim"], s["q"].shape[0]
    # far positions: the angle in 64 bits
    freq = c["scale"] * torch.exp(torch.arange(rd // 2, device=DEV, dtype=torch.float64)
                                  * (-2.0 / rd * math.log(c["theta"])))
    angle = s["positions"].double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_rotate(_plain_norm(s["q"].float(), s["q_weight"], s["eps"]), cos, sin, c["layout"], rd)
    k = _plain_rotate(_plain_norm(s["k"].float(), s["k_weight"], s["eps"]), cos, sin, c["layout"], rd)
    _, kv = _kv_lengths(s)
    seq = _sequence_of(s["append_indptr"], n)
    # the new tokens are the last rows of their sequence
    row = kv[seq] - s["append_indptr"][seq + 1].long() + torch.arange(n, device=DEV)
    page, slot = _slots(s, seq, row)
    s["pages"][page, 0, :, slot] = k.to(s["pages"].dtype)
    s["pages"][page, 1, :, slot] = s["v"]
    return q.to(s["q"].dtype), s["pages"]


def _plain_compact(s):
    n_pages, kv = _kv_lengths(s)
    n, nnz = s["accept_nodes"].numel(), s["page_values"].numel()
    trees = (s["tree_indptr"][1:] - s["tree_indptr"][:-1]).long()
    acc = (s["accept_indptr"][1:] - s["accept_indptr"][:-1]).long()
    seq = _sequence_of(s["accept_indptr"], n)
    start = (kv - trees)[seq]
    page, slot = _slots(s, seq, start + s["accept_nodes"].long())
    rows = s["pages"][page, :, :, slot]
    page, slot = _slots(s, seq, start + torch.arange(n, device=DEV) - s["accept_indptr"][seq].long())
    s["pages"][page, :, :, slot] = rows
    # the table: the first pages of each sequence stay, the others are freed, in order
    new_kv = kv - trees + acc
    keep = (new_kv + PAGE - 1) // PAGE
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    indptr = torch.cat([zero, keep.cumsum(0)])
    s["new_indptr"].copy_(indptr)
    s["new_length"].copy_(torch.where(keep > 0, new_kv - (keep - 1) * PAGE, 0))
    seq = _sequence_of(s["page_indptr"], nnz)
    off = torch.arange(nnz, device=DEV) - s["page_indptr"][seq].long()
    kept = off < keep[seq]
    gone = torch.cat([zero, (n_pages - keep).cumsum(0)])
    spare = torch.full((2, nnz + 1), -1, dtype=torch.int32, device=DEV)
    spare[0].scatter_(0, torch.where(kept, indptr[seq] + off, nnz), s["page_values"])
    spare[1].scatter_(0, torch.where(kept, nnz, gone[seq] + off - keep[seq]), s["page_values"])
    s["new_values"].copy_(spare[0, :nnz])
    s["freed"].copy_(spare[1, :nnz])
    s["num_freed"].copy_(gone[-1:])
    return (s["pages"], s["new_indptr"], s["new_values"], s["new_length"], s["freed"],
            s["num_freed"])


def _plain_copy(s):
    s["pages"][s["dst"].long()] = s["pages"][s["src"].long()]
    return s["pages"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size, h_kv, d = _sizes(case), case["h_kv"], case["d"]
    if case["op"] == "copy":
        return {"bytes": 2.0 * case["n"] * 2 * h_kv * PAGE * d * 2 + 8.0 * case["n"], "flops": 0.0}
    rows = sum(size["kv"])
    table = 4.0 * sum(-(-x // PAGE) for x in size["kv"]) + 8.0 * case["batch"]
    if case["op"] == "decode":
        h_q = case["h_q"]
        return {"bytes": 2.0 * rows * h_kv * d * 2 + 2.0 * case["batch"] * h_q * d * 2
                + 4.0 * case["batch"] * h_q + table, "flops": 4.0 * rows * h_q * d}
    if case["op"] == "append":
        n, h_q = sum(size["new"]), case["h_q"]
        b = 2.0 * n * (h_q + 2 * h_kv) * d * 2 + 4.0 * n + 12.0 * case["batch"] + 4.0 * n / PAGE
        per = (4.0 if case["norm"] else 0.0) * d
        per += 3.0 * case["rotary_dim"] if case["layout"] != "none" else 0.0
        return {"bytes": b, "flops": per * n * (h_q + h_kv)}
    # the first node never moves; of the others all but a few do
    moved = sum(a - 1 for a in size["acc"])
    return {"bytes": 2.0 * moved * 2 * h_kv * d * 2 + 2.0 * table + 4.0 * sum(size["acc"]),
            "flops": 0.0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------

def _rows(s, b):
    """The (page, slot) of every kv row of sequence b, in order."""
    p0, p1 = int(s["page_indptr"][b]), int(s["page_indptr"][b + 1])
    if p0 == p1:
        return torch.zeros((0, 2), dtype=torch.long, device=DEV)
    n = (p1 - p0 - 1) * PAGE + int(s["length_info"][b])
    pid = s["page_values"][p0:p1].long().repeat_interleave(PAGE)[:n]
    return torch.stack([pid, torch.arange(n, device=DEV) % PAGE], 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "copy":
        pool = s["pages"].double()
        for i, j in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[j] = pool[i]
        return pool
    if case["op"] == "decode":
        h_kv, g = case["h_kv"], case["h_q"] // case["h_kv"]
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        for b in range(case["batch"]):
            at = _rows(s, b)
            if not len(at):
                continue
            kv = s["pages"][at[:, 0], :, :, at[:, 1]].double()        # [rows, 2, h_kv, d]
            q = s["q"][b].double().reshape(h_kv, g, -1)
            x = torch.einsum("hgd,rhd->hgr", q, kv[:, 0]) * s["sm_scale"]
            z = torch.logsumexp(x, -1)
            out[b] = torch.einsum("hgr,rhd->hgd", torch.exp(x - z[..., None]),
                                  kv[:, 1]).reshape(out[b].shape)
            lse[b] = (z / math.log(2.0)).reshape(-1)
        return out, lse
    pool = s["pages"].double()
    if case["op"] == "compact":
        for b in range(case["batch"]):
            at = _rows(s, b)
            t0 = len(at) - int(s["tree_indptr"][b + 1] - s["tree_indptr"][b])
            path = s["accept_nodes"][int(s["accept_indptr"][b]):int(s["accept_indptr"][b + 1])]
            src, dst = at[t0 + path.long()], at[t0:t0 + len(path)]
            pool[dst[:, 0], :, :, dst[:, 1]] = pool[src[:, 0], :, :, src[:, 1]]
        return pool, None, None, None, None, None
    rd, half = case["rotary_dim"], case["rotary_dim"] // 2
    i = torch.arange(half, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.ones(len(s["positions"]), half, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * case["scale"]
                       / torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=DEV),
                                   2 * i / rd))[:, None]
    new = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        x = x.clone()
        if case["layout"] != "none":
            pair = x[..., :rd].unflatten(-1, (2, half)).transpose(-1, -2) \
                if case["layout"] == "half" else x[..., :rd].unflatten(-1, (half, 2))
            z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            x[..., :rd] = (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)
        new.append(x)
    for b in range(case["batch"]):
        t0, t1 = int(s["append_indptr"][b]), int(s["append_indptr"][b + 1])
        at = _rows(s, b)
        at = at[len(at) - (t1 - t0):]
        pool[at[:, 0], 0, :, at[:, 1]] = new[1][t0:t1]
        pool[at[:, 0], 1, :, at[:, 1]] = s["v"][t0:t1].double()
    return new[0], pool
