"""Cases for attention whose keys and values come from one shared latent vector
a token (latent attention): appending latents to a paged latent cache (with the
norm of the latent and the rotation of the shared key and of the queries'
rotary part), attention of one new token per sequence and of draft trees over
that cache (absorbed form: all heads read the same row), and attention of
prompts with keys and values per head (expanded form).

``run`` computes each operator in elementary torch operations, or, with ``own``,
through ``tree_attention_gb300``.  ``exact`` gives the same outputs in 64 bits
from the definitions.
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

def _append(name, batch, lo, hi, ctx, h, rank, rope, dtype, norm, layout, theta, scale, rows, shape):
    return {"name": name, "op": "append", "batch": batch, "lo": lo, "hi": hi, "ctx": ctx, "h": h,
            "rank": rank, "rope": rope, "dtype": dtype, "norm": norm, "layout": layout,
            "theta": theta, "scale": scale, "rows": rows, "shape": shape}


def _decode(name, batch, lo, hi, h, rank, rope, dtype, shape):
    return {"name": name, "op": "decode", "batch": batch, "lo": lo, "hi": hi, "h": h,
            "rank": rank, "rope": rope, "dtype": dtype, "shape": shape}


def _tree(name, batch, nodes_lo, nodes, lo, hi, h, rank, rope, dtype, shape):
    return {"name": name, "op": "tree", "batch": batch, "nodes_lo": nodes_lo, "nodes": nodes,
            "lo": lo, "hi": hi, "h": h, "rank": rank, "rope": rope, "dtype": dtype, "shape": shape}


def _expand(name, batch, lo, hi, held, h, d, rope, dtype, shape):
    return {"name": name, "op": "expand", "batch": batch, "lo": lo, "hi": hi, "held": held, "h": h,
            "d": d, "rope": rope, "dtype": dtype, "shape": shape}


def listed():
    return [
        # one new token for each of 32 chats far into long contexts
        _append("append-token", 32, 1, 1, 60000, 128, 512, 64, "bf16", True, "interleaved", 5e5, 1.0,
                False, 1),
        # prompts of 16 to 512 tokens for 64 chats; the rows are wanted for the expanded form too
        _append("append-prompt", 64, 16, 512, 0, 64, 512, 64, "bf16", True, "half", 1e4, 0.25, True, 2),
        # the smallest call: two short chats, the sizes of the "tiny" workload; launch latency
        _decode("decode-tiny", 2, 7, 12, 4, 256, 32, "fp16", 3),
        # one user's chat on a model of few heads
        _decode("decode-one", 1, 4096, 4096, 16, 512, 64, "fp16", 4),
        # a small server: 32 chats of about a thousand tokens, the most heads
        _decode("decode-chats", 32, 500, 1500, 128, 512, 64, "bf16", 5),
        # four long documents (the "long-prefix" workload): the cache's length has to be split
        _decode("decode-long", 4, 32000, 33600, 128, 512, 64, "bf16", 6),
        # a full server: ragged lengths from a page to 16k tokens (the "ragged-large" heads)
        _decode("decode-server", 64, 16, 16384, 64, 512, 64, "bf16", 7),
        # two small draft trees without a prefix, the "tiny" workload
        _tree("tree-tiny", 2, 7, 12, 0, 0, 4, 256, 32, "fp16", 8),
        # draft trees of 64 nodes for 32 chats (the "spec-decode" workload with its prefix)
        _tree("tree-draft", 32, 64, 64, 500, 1500, 32, 512, 64, "bf16", 9),
        # the same behind four long documents (the "long-prefix" workload)
        _tree("tree-long", 4, 64, 64, 32768, 32768, 32, 512, 64, "bf16", 10),
        # ragged prompts of 16 to 512 tokens for 64 chats (the "ragged-large" heads)
        _expand("expand-prompts", 64, 16, 512, 0, 64, 128, 64, "bf16", 11),
        # a 2,000-token part of two prompts, 14,000 tokens of which are there already
        _expand("expand-chunk", 2, 2000, 2000, 14000, 32, 128, 64, "fp16", 12),
    ]


HEADS = {512: [1, 4, 5, 8, 16, 20, 32, 40, 64, 128], 256: [1, 3, 4, 8, 16, 18, 32, 64, 80, 128]}
EXPAND_HEADS = [1, 3, 4, 8, 10, 20, 32, 40, 64]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "tree", "expand"])
    dtype = rng.choice(["bf16", "fp16"])
    rank = rng.choice([512, 512, 256])
    rope = rng.choice([64, 64, 32, 16])
    h = rng.choice(HEADS[rank])
    shape = rng.randrange(1 << 30)
    if op == "append":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, 10000 // batch))
        c = _append("", batch, rng.randint(1, hi), hi, _log(rng, 1, 60000), h, rank, rope, dtype,
                    rng.random() < 0.7, rng.choice(["half", "interleaved", "none"]),
                    rng.choice([1e4, 5e5]), rng.choice([1.0, 0.25]), rng.random() < 0.5, shape)
    elif op == "decode":
        batch = _log(rng, 1, 256)
        hi = _log(rng, 1, max(2, min(40000, 200000 // batch)))
        lo = 0 if batch > 4 and rng.random() < 0.3 else rng.randint(1, hi)
        c = _decode("", batch, lo, hi, h, rank, rope, dtype, shape)
    elif op == "tree":
        batch = _log(rng, 1, 64)
        nodes = _log(rng, 1, 200)
        # rows of queries times kv rows stays below the longest listed case's
        hi = _log(rng, 1, max(2, min(40000, int(2e8 / (batch * nodes * h)))))
        c = _tree("", batch, rng.randint(1, nodes), nodes, rng.randint(0, hi), hi, h, rank, rope, dtype,
                  shape)
    else:
        h = rng.choice(EXPAND_HEADS)
        batch = _log(rng, 1, 64)
        hi = _log(rng, 1, max(2, min(4000, 500000 // (batch * h))))
        held = 0 if rng.random() < 0.5 else _log(rng, 1, max(2, min(8000, 500000 // (batch * h))))
        c = _expand("", batch, rng.randint(1, hi), hi, held, h, rng.choice([128, 128, 64]), rope, dtype,
                    shape)
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


def _parents(n, r):
    """A draft tree: most nodes continue one of the last few, none is deeper than 12."""
    parent, depth = [-1], [0]
    for i in range(1, n):
        p = r.randint(max(0, i - 6), i - 1)
        while depth[p] >= 12:
            p = parent[p]
        parent.append(p)
        depth.append(depth[p] + 1)
    return parent, depth


def _intervals(parent):
    """(enter, exit) of each node of a depth-first walk, children in order."""
    n = len(parent)
    size = [1] * n
    for i in range(n - 1, 0, -1):
        size[parent[i]] += size[i]
    enter, nxt = [0] * n, [1] * n
    for i in range(1, n):
        enter[i] = nxt[parent[i]]
        nxt[parent[i]] += size[i]
        nxt[i] = enter[i] + 1
    return [(enter[i], enter[i] + size[i]) for i in range(n)]


def _sizes(case):
    """Host sizes of a case: kv lengths, and new tokens, or trees, or query rows."""
    r = random.Random(case["shape"] * 7 + 3)
    if case["op"] == "decode":
        return {"kv": _between(case, "lo", "hi", 1)}
    if case["op"] == "append":
        new = _between(case, "lo", "hi", 1)
        # the cache holds a part of the context's rows; the positions count all of it
        ctx = [r.randint(case["ctx"] // 2, case["ctx"]) for _ in new]
        held = [min(c, 2000) for c in ctx]
        return {"new": new, "ctx": ctx, "kv": [h + n for h, n in zip(held, new)]}
    if case["op"] == "tree":
        nodes = _between(case, "nodes_lo", "nodes", 2)
        trees = [_parents(n, r) for n in nodes]
        ctx = _between(case, "lo", "hi", 1)
        return {"nodes": nodes, "trees": trees, "kv": [c + n for c, n in zip(ctx, nodes)]}
    new = _between(case, "lo", "hi", 1)
    held = [r.randint(case["held"] // 2, case["held"]) for _ in new]
    return {"new": new, "kv": [h + n for h, n in zip(held, new)]}


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _indptr(n):
    return np.concatenate([[0], np.cumsum(np.asarray(n, dtype=np.int64))])


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=dtype)


def _table(case, kv, seed, gen):
    """A page pool with a scattered page table for kv lengths ``kv``."""
    kv = np.asarray(kv, dtype=np.int64)
    n_pages = (kv + PAGE - 1) // PAGE
    nnz = int(n_pages.sum())
    pool = nnz + 5
    perm = np.random.default_rng(seed).permutation(pool)[:nnz]
    last = np.where(n_pages > 0, kv - (n_pages - 1) * PAGE, 0)
    pages = _randn(gen, (pool, PAGE, case["rank"] + case["rope"]), DTYPES[case["dtype"]])
    return {"pages": pages, "page_indptr": _i32(_indptr(n_pages)), "page_values": _i32(perm),
            "length_info": _i32(last), "kv": kv.tolist()}


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    dt, h, op, rope = DTYPES[case["dtype"]], case["h"], case["op"], case["rope"]
    size = _sizes(case)
    s = {"case": case}
    if op == "expand":
        d, nq, nk = case["d"], sum(size["new"]), sum(size["kv"])
        s["q"] = _randn(gen, (nq, h, d + rope), dt)
        kv = _randn(gen, (nk, h, 2 * d), dt)               # one projection of the latents
        rows = _randn(gen, (nk, 4 * d + rope), dt)         # the latents and their rotated keys
        s["k"], s["v"], s["k_rope"] = kv[:, :, :d], kv[:, :, d:], rows[:, 4 * d:]
        s["q_indptr"], s["kv_indptr"] = _i32(_indptr(size["new"])), _i32(_indptr(size["kv"]))
        s["new"], s["kv"] = size["new"], size["kv"]
        s["sm_scale"] = 1.0 / math.sqrt(d + rope)
        s["out"] = torch.empty((nq, h, d), dtype=dt, device=DEV)
        s["lse"] = torch.empty((nq, h), dtype=torch.float32, device=DEV)
        if own:
            import tree_attention_gb300 as ta
            dims = ta.make_expanded_dims(s["q"], s["k"], s["q_indptr"])
            s["workspace"] = torch.zeros(ta.expanded_workspace_size(dims), dtype=torch.uint8, device=DEV)
        return s
    rank = case["rank"]
    s.update(_table(case, size["kv"], seed, gen))
    # queries of 128 elements and the rotary ones, before the former were absorbed
    s["sm_scale"] = 1.0 / math.sqrt(128 + rope)
    if op == "append":
        n = sum(size["new"])
        down = _randn(gen, (n, rank + rope), dt)           # one down projection's output
        up = _randn(gen, (n, h, 128 + rope), dt)           # the queries' projection
        s["latent"], s["k_rope"], s["q_rope"] = down[:, :rank], down[:, rank:], up[:, :, 128:]
        s["append_indptr"] = _i32(_indptr(size["new"]))
        s["positions"] = _i32(np.concatenate([np.arange(c, c + m)
                                              for c, m in zip(size["ctx"], size["new"])]))
        s["weight"] = None
        if case["norm"]:
            s["weight"] = (1 + 0.1 * _randn(gen, (rank,), torch.float32)).to(dt)
        s["eps"] = 1e-6
        # the absorbed queries, whose last elements the call fills
        s["q_out"] = torch.zeros((n, h, rank + rope), dtype=dt, device=DEV)[:, :, rank:]
        s["rows_out"] = torch.empty((n, rank + rope), dtype=dt, device=DEV) if case["rows"] else None
    else:
        rows = case["batch"] if op == "decode" else sum(size["nodes"])
        s["q"] = _randn(gen, (rows, h, rank + rope), dt)
        s["out"] = torch.empty((rows, h, rank), dtype=dt, device=DEV)
        s["lse"] = torch.empty((rows, h), dtype=torch.float32, device=DEV)
        if op == "tree":
            s["nodes"] = size["nodes"]
            s["mn_indptr"] = _i32(_indptr(size["nodes"]))
            s["tree_order"] = _i32([iv for p, _ in size["trees"] for iv in _intervals(p)])
    if own:
        import tree_attention_gb300 as ta
        s["cache"] = ta.LatentCache(s["pages"], s["page_indptr"], s["page_values"], s["length_info"],
                                    h_q=h, rank=rank)
        if op == "append" and case["layout"] != "none":
            s["rotation"] = ta.Rope(case["layout"], rope, theta=case["theta"], scale=case["scale"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        if op == "expand":
            import tree_attention_gb300 as ta
            ta.tree_attn_expanded(s["q"], s["q_indptr"], s["k"], s["k_rope"], s["v"], s["kv_indptr"],
                                  s["out"], s["lse"], s["sm_scale"], s["workspace"])
            return s["out"], s["lse"]
        c = s["cache"]
        if op == "append":
            c.append(s["latent"], s["k_rope"], s["append_indptr"], s["positions"], q_rope=s["q_rope"],
                     rope=s.get("rotation"), weight=s["weight"], norm_eps=s["eps"], q_out=s["q_out"],
                     rows_out=s["rows_out"])
            return (s["q_out"], s["pages"]) if s["rows_out"] is None else (s["q_out"], s["pages"],
                                                                           s["rows_out"])
        if op == "decode":
            c.decode(s["q"], s["sm_scale"], out=s["out"], lse=s["lse"])
        else:
            c.tree_attn(s["q"], s["mn_indptr"], s["mn_indptr"], s["tree_order"], s["sm_scale"],
                        out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    return {"append": _plain_append, "decode": _plain_decode, "tree": _plain_tree,
            "expand": _plain_expand}[op](s)


def _attend(q, k, v, seen, sm_scale):
    """Softmax attention of q [.., rows, W] over k, v [.., kv, ..]; seen: which columns count."""
    x = (q @ k.transpose(-1, -2) * sm_scale).masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    lse = torch.where(z > 0, (m + torch.log(z)) / math.log(2.0), -math.inf)
    return (p @ v) / z.clamp(min=1e-30), lse[..., 0]


def _gathered(s, b0, b1):
    """The cache rows of sequences b0 .. b1 - 1 in float32, padded to the longest's pages, and their
    lengths."""
    indptr = s["page_indptr"].long()
    n = indptr[b0 + 1:b1 + 1] - indptr[b0:b1]
    kv = torch.where(n > 0, (n - 1) * PAGE + s["length_info"][b0:b1].long(), 0)
    most = max(1, -(-max(s["kv"][b0:b1]) // PAGE))
    at = indptr[b0:b1, None] + torch.arange(most, device=DEV)
    if not s["page_values"].numel():
        return torch.zeros((b1 - b0, PAGE, s["pages"].shape[2]), device=DEV), kv
    pid = s["page_values"][at.clamp(max=s["page_values"].numel() - 1)].long()
    return s["pages"][pid].float().flatten(1, 2), kv


def _plain_decode(s):
    rank = s["case"]["rank"]
    rows, kv = _gathered(s, 0, s["case"]["batch"])
    seen = torch.arange(rows.shape[1], device=DEV) < kv[:, None]
    out, lse = _attend(s["q"].float(), rows, rows[:, :, :rank], seen[:, None], s["sm_scale"])
    return out.to(s["q"].dtype), lse


def _plain_tree(s):
    c, h = s["case"], s["case"]["h"]
    outs, lses, t0 = [], [], 0
    for b, n in enumerate(s["nodes"]):
        rows, _ = _gathered(s, b, b + 1)
        rows = rows[0, :s["kv"][b]]
        iv = s["tree_order"][t0:t0 + n].view(n, 2)
        seen = torch.ones((n, rows.shape[0]), dtype=torch.bool, device=DEV)
        seen[:, rows.shape[0] - n:] = (iv[None, :, 0] <= iv[:, None, 0]) & (iv[:, None, 0] < iv[None, :, 1])
        q = s["q"][t0:t0 + n].float().flatten(0, 1)
        out, lse = _attend(q, rows, rows[:, :c["rank"]], seen.repeat_interleave(h, 0), s["sm_scale"])
        outs.append(out.view(n, h, -1))
        lses.append(lse.view(n, h))
        t0 += n
    return torch.cat(outs).to(s["q"].dtype), torch.cat(lses)


def _plain_expand(s):
    c, h = s["case"], s["case"]["h"]
    outs, lses, q0, k0 = [], [], 0, 0
    for nq, nk in zip(s["new"], s["kv"]):
        q = s["q"][q0:q0 + nq].float().transpose(0, 1)
        k = torch.cat([s["k"][k0:k0 + nk].float(),
                       s["k_rope"][k0:k0 + nk].float()[:, None].expand(nk, h, c["rope"])], -1)
        v = s["v"][k0:k0 + nk].float().transpose(0, 1)
        # a query is one of the last rows and sees those up to its own
        seen = torch.arange(nk, device=DEV) <= torch.arange(nk - nq, nk, device=DEV)[:, None]
        out, lse = _attend(q, k.transpose(0, 1), v, seen, s["sm_scale"])
        outs.append(out.transpose(0, 1))
        lses.append(lse.transpose(0, 1))
        q0, k0 = q0 + nq, k0 + nk
    return torch.cat(outs).to(s["q"].dtype), torch.cat(lses).contiguous()


def _plain_rotate(x, cos, sin, layout):
    if layout == "none":
        return x
    half = x.shape[-1] // 2
    if layout == "half":
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)


def _plain_append(s):
    c = s["case"]
    rd, n = c["rope"], s["latent"].shape[0]
    # far positions: the angle in 64 bits
    freq = c["scale"] * torch.exp(torch.arange(rd // 2, device=DEV, dtype=torch.float64)
                                  * (-2.0 / rd * math.log(c["theta"])))
    angle = s["positions"].double()[:, None] * freq
    cos, sin = angle.cos().float(), angle.sin().float()
    latent = s["latent"].float()
    if s["weight"] is not None:
        latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + s["eps"]) \
            * s["weight"].float()
    k = _plain_rotate(s["k_rope"].float(), cos, sin, c["layout"])
    q = _plain_rotate(s["q_rope"].float(), cos[:, None], sin[:, None], c["layout"])
    rows = torch.cat([latent, k], -1).to(s["pages"].dtype)
    # the new tokens are the last rows of their sequence
    seq = torch.searchsorted(s["append_indptr"][1:].long(), torch.arange(n, device=DEV), right=True)
    pages = (s["page_indptr"][1:] - s["page_indptr"][:-1]).long()
    kv = (pages - 1) * PAGE + s["length_info"].long()
    row = kv[seq] - s["append_indptr"][seq + 1].long() + torch.arange(n, device=DEV)
    page = s["page_values"][s["page_indptr"][seq].long() + row // PAGE].long()
    s["pages"][page, row % PAGE] = rows
    s["q_out"].copy_(q)
    if s["rows_out"] is None:
        return s["q_out"], s["pages"]
    s["rows_out"].copy_(rows)
    return s["q_out"], s["pages"], s["rows_out"]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    size, h, rope = _sizes(case), case["h"], case["rope"]
    if case["op"] == "expand":
        d = case["d"]
        pairs = sum(n * (k - n) + n * (n + 1) / 2 for n, k in zip(size["new"], size["kv"]))
        nq, nk = sum(size["new"]), sum(size["kv"])
        return {"bytes": 2.0 * nq * h * (2 * d + rope) + 4.0 * nq * h + 2.0 * nk * (h * 2 * d + rope)
                + 8.0 * case["batch"], "flops": 2.0 * pairs * h * (2 * d + rope)}
    rank = case["rank"]
    w = rank + rope
    table = 4.0 * sum(-(-x // PAGE) for x in size["kv"]) + 8.0 * case["batch"]
    if case["op"] == "append":
        n = sum(size["new"])
        b = 2.0 * n * 2 * w + 2.0 * n * 2 * h * rope + (2.0 * n * w if case["rows"] else 0.0)
        per = (4.0 * rank if case["norm"] else 0.0) + (3.0 * rope * (h + 1)
                                                       if case["layout"] != "none" else 0.0)
        return {"bytes": b + 4.0 * n + 12.0 * case["batch"] + 4.0 * n / PAGE, "flops": per * n}
    if case["op"] == "decode":
        rows, pairs, own_tables = case["batch"], float(sum(size["kv"])), 0.0
    else:
        rows, own_tables = sum(size["nodes"]), 8.0 * sum(size["nodes"])
        pairs = 0.0
        for n, k, (_, depth) in zip(size["nodes"], size["kv"], size["trees"]):
            pairs += float(n) * (k - n) + sum(depth) + n
    return {"bytes": 2.0 * sum(size["kv"]) * w + 2.0 * rows * h * (w + rank) + 4.0 * rows * h + table
            + own_tables, "flops": 2.0 * pairs * h * (w + rank)}


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


def _softmax64(x, v):
    z = torch.logsumexp(x, -1)
    return torch.exp(x - z[..., None]) @ v, z / math.log(2.0)


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    op, h = case["op"], case["h"]
    if op in ("decode", "tree"):
        size, rank = _sizes(case), case["rank"]
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
        t0 = 0
        for b in range(case["batch"]):
            at = _rows(s, b)
            n = 1 if op == "decode" else size["nodes"][b]
            if len(at):
                rows = s["pages"][at[:, 0], at[:, 1]].double()
                hide = torch.zeros((n, len(at)), dtype=torch.float64)
                if op == "tree":
                    # a node sees itself and the nodes on its way to the root
                    hide[:, len(at) - n:] = -math.inf
                    for i in range(n):
                        j = i
                        while j >= 0:
                            hide[i, len(at) - n + j] = 0.0
                            j = size["trees"][b][0][j]
                hide = hide.to(DEV)
                for i in range(h):
                    x = (s["q"][t0:t0 + n, i].double() @ rows.T) * s["sm_scale"] + hide
                    out[t0:t0 + n, i], lse[t0:t0 + n, i] = _softmax64(x, rows[:, :rank])
            t0 += n
        return out, lse
    if op == "expand":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
        d, q0, k0 = case["d"], 0, 0
        for nq, nk in zip(s["new"], s["kv"]):
            hide = torch.full((nq, nk), -math.inf, dtype=torch.float64, device=DEV).triu(nk - nq + 1)
            hide = torch.where(hide == 0, 0.0, hide)
            shared = s["k_rope"][k0:k0 + nk].double()
            for i in range(h):
                q = s["q"][q0:q0 + nq, i].double()
                x = (q[:, :d] @ s["k"][k0:k0 + nk, i].double().T + q[:, d:] @ shared.T) * s["sm_scale"]
                out[q0:q0 + nq, i], lse[q0:q0 + nq, i] = _softmax64(x + hide,
                                                                    s["v"][k0:k0 + nk, i].double())
            q0, k0 = q0 + nq, k0 + nk
        return out, lse
    pool, rd = s["pages"].double(), case["rope"]
    half = rd // 2
    i = torch.arange(half, dtype=torch.float64, device=DEV)
    turn = torch.polar(torch.ones(len(s["positions"]), half, dtype=torch.float64, device=DEV),
                       s["positions"].double()[:, None] * case["scale"]
                       / torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device=DEV),
                                   2 * i / rd))[:, None]

    def rotated(x):
        if case["layout"] == "none":
            return x
        pair = x.unflatten(-1, (2, half)).transpose(-1, -2) if case["layout"] == "half" \
            else x.unflatten(-1, (half, 2))
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        return (z.transpose(-1, -2) if case["layout"] == "half" else z).flatten(-2)

    latent = s["latent"].double()
    if s["weight"] is not None:
        latent = latent / torch.sqrt((latent * latent).sum(-1, keepdim=True) / case["rank"] + s["eps"]) \
            * s["weight"].double()
    rows = torch.cat([latent, rotated(s["k_rope"].double()[:, None])[:, 0]], -1)
    for b in range(case["batch"]):
        t0, t1 = int(s["append_indptr"][b]), int(s["append_indptr"][b + 1])
        at = _rows(s, b)
        at = at[len(at) - (t1 - t0):]
        pool[at[:, 0], at[:, 1]] = rows[t0:t1]
    out = (rotated(s["q_rope"].double()), pool)
    return out if s["rows_out"] is None else out + (rows,)
