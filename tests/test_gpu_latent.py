"""GPU tests of the latent-attention calls against the 64-bit references.

Tolerances.  Rounding to a 16-bit type is off by at most ``half = eps / 2`` of the
value.  A weight is rounded to 16 bits before it meets the values and the result
divided by the sum of the rounded weights: the weighted mean is off by ``2 half`` of ``sum w |v|``
(numerator and denominator), and is itself rounded once.  fp16 weights below
2^-14 are off by 2^-25 instead; the largest weight is 2^7 at least, so this is
2^-32 of the largest |v| per row.  A score is a float32 sum of W products, off by
at most ``(W + 4) 2^-23`` (truncating adds) of the sum of its products' sizes in
base-2 units; a weight is off by that times ln 2, relative, twice, and the lse
by it once.  Exponentials, the weighted sum's additions (a few dozen float32
terms one after the other per 128 rows, of equal size) and the factors of moved
references and merged parts: 2^-16 of ``sum w |v|`` together for up to 40,000
rows.  lse: its sum is of the float32 weights, 2^-19, and 2^-22 of its value.  append: a rotated element is a sum of two products of
float32 factors, a normed one a product of three behind a sum of 512 squares:
2^-19 of the pair's length, or of the element.  Compaction and copies move bits.
"""
import math

import numpy as np
import pytest
import torch

import tree_attention_gb300 as ta
import workloads as wl
from oracle import latent_ref as ref
from oracle import paged_cache_ref as paged

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tree_attention_gb300 import build
    build.build()
    ta.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def indptr(n):
    return np.concatenate([[0], np.cumsum(np.asarray(n, dtype=np.int64))])


class Setup:
    """A latent pool with a scattered table for lengths ``kv``; slots nobody owns
    hold NaN.  The table's arrays have spare capacity at the end."""

    def __init__(self, kv, h, rank=512, rope=64, dtype="bf16", seed=0, spare=3, fill=NAN):
        rng = np.random.default_rng(seed)
        self.kv = np.asarray(kv, dtype=np.int64)
        n = -(-self.kv // 16)
        self.indptr = indptr(n)
        nnz = int(n.sum())
        self.values = np.concatenate([rng.permutation(nnz + spare)[:nnz], [-7] * 2]).astype(int)
        self.last = np.where(n > 0, self.kv - (n - 1) * 16, 0)
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.dtype, self.h, self.rank, self.rope, self.w = DT[dtype], h, rank, rope, rank + rope
        self.pool = torch.full((nnz + spare, 16, self.w), fill, dtype=self.dtype, device="cuda")
        for b in range(len(kv)):
            pid, sl = self.slots(b)
            self.pool[pid, sl] = self.randn(len(pid), self.w)
        self.cache = self.handle()

    def handle(self, **kw):
        a = {"page_indptr": self.indptr, "page_values": self.values, "length_info": self.last}
        a.update(kw)
        return ta.LatentCache(self.pool, *[i32(a[k]) for k in a], h_q=self.h, rank=self.rank)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(self.dtype)

    def slots(self, b):
        return ref.slots(*self.table, b, device="cuda")

    @property
    def table(self):
        return self.indptr, self.values, self.last


def check(dtype, width, rows, vmax, out, lse, want):
    ro, rl, mag, smag = want
    half = torch.finfo(dtype).eps / 2
    serr = (width + 4) * 2.0 ** -23 * smag
    tol = half * ro.abs() + (2 * half + 2.0 ** -16 + 2 * serr[..., None]) * mag \
        + torch.finfo(dtype).smallest_normal * half * 2
    if dtype == torch.float16:
        tol = tol + rows * 2.0 ** -32 * vmax
    out, lse = out.double(), lse.double()
    assert torch.isfinite(out).all()
    far = ((out - ro).abs() / tol)
    assert (far <= 1).all(), far.max()
    fin = torch.isfinite(rl)
    assert torch.equal(fin, torch.isfinite(lse)) and (lse[~fin] == -INF).all()
    ltol = serr + 2.0 ** -19 + 2.0 ** -22 * rl.abs()
    assert ((lse - rl).abs() <= ltol)[fin].all(), ((lse - rl).abs() / ltol)[fin].max()


def check_absorbed(s, q, out, lse, sm, q_rows=None, parents=None):
    want = ref.absorbed(q.double(), s.pool.double(), s.table, s.rank, sm, q_rows, parents)
    clean = torch.nan_to_num(s.pool.double(), nan=0.0, posinf=0.0, neginf=0.0)
    check(s.dtype, s.w, int(max(s.kv.max(), 1)), float(clean.abs().max()), out, lse, want)


# --------------------------------------------------------------------------
# one token per sequence
# --------------------------------------------------------------------------

DECODE = {
    # kv lengths, heads, rank, rope, dtype
    "one_row": ([1], 8, 512, 64, "bf16"),
    "page_edges": ([1, 15, 16, 17, 31, 32, 33], 16, 512, 64, "fp16"),
    "tile_edges": ([127, 128, 129, 255, 256, 257, 64, 65], 4, 512, 64, "bf16"),
    "empty_rows": ([0, 5, 0, 0, 40, 0], 4, 256, 32, "bf16"),
    "all_empty": ([0, 0, 0], 4, 512, 64, "bf16"),
    "one_head": ([200, 3], 1, 512, 64, "bf16"),
    "five_heads": ([77, 130], 5, 256, 48, "fp16"),
    "heads_63": ([300, 31], 63, 512, 16, "bf16"),
    "heads_64": ([300, 31], 64, 512, 64, "fp16"),
    "heads_65": ([150, 2], 65, 512, 64, "bf16"),
    "heads_127": ([90, 518], 127, 256, 64, "fp16"),
    "heads_128": ([1000, 18, 700], 128, 512, 64, "bf16"),
    "heads_128_small": ([1000, 18, 700], 128, 256, 32, "fp16"),
    "one_long": ([9000], 32, 512, 64, "bf16"),
    "one_long_fp16": ([20000], 8, 256, 64, "fp16"),
    "ragged": ([int(x) for x in np.random.default_rng(4).integers(0, 700, 40)], 12, 512, 64, "bf16"),
    "many_short": ([1 + i % 37 for i in range(300)], 4, 256, 16, "fp16"),
    "long_and_short": ([6000, 1, 2, 3, 17, 0, 900], 20, 512, 32, "fp16"),
    "many_tiles": ([2500] * 9 + [100] * 30, 40, 512, 64, "bf16"),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name):
    kv, h, rank, rope, dtype = DECODE[name]
    s = Setup(kv, h, rank, rope, dtype, seed=len(kv))
    q = s.randn(len(kv), h, s.w)
    for sm in (192 ** -0.5, 0.3):
        out, lse = s.cache.decode(q, sm)
        assert s.cache.device_status() == ta.TA_OK
        check_absorbed(s, q, out, lse, sm)


def test_decode_largest_batch():
    rng = np.random.default_rng(9)
    s = Setup([1], 2, 256, 16, seed=10)
    kv = rng.integers(0, 21, 16384)
    n = -(-kv // 16)
    pool = s.randn(int(n.sum()), 16, s.w)
    s.kv, s.indptr, s.values = kv, indptr(n), np.arange(n.sum())
    s.last, s.pool = np.where(n > 0, kv - (n - 1) * 16, 0), pool
    s.cache = s.handle()
    q = s.randn(16384, 2, s.w)
    out, lse = s.cache.decode(q, 0.1)
    assert s.cache.device_status() == ta.TA_OK
    check_absorbed(s, q, out, lse, 0.1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_merges_in_large_units_of_the_small_rank(dtype):
    """Enough sequences that several pairs of SMs share for the merge's large units
    (32 rows by 128 columns: two CTAs' worth of them per SM and more)."""
    kv = [int(x) for x in np.random.default_rng(28).integers(400, 2200, 70)]
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    tiles = np.cumsum([0] + [-(-n // 128) for n in kv])
    per, extra = divmod(int(tiles[-1]), pairs)
    starts = {i * per + min(i, extra) for i in range(pairs)}
    cut = sum(any(u in starts for u in range(a + 1, b)) for a, b in zip(tiles[:-1], tiles[1:]))
    assert cut * 4 * 2 * 2 >= 4 * 2 * pairs
    s = Setup(kv, 128, 256, 64, dtype, seed=29)
    q = s.randn(len(kv), 128, s.w)
    out, lse = s.cache.decode(q, 0.07)
    assert s.cache.device_status() == ta.TA_OK
    check_absorbed(s, q, out, lse, 0.07)


def test_decode_without_any_page():
    pool = torch.full((2, 16, 576), NAN, dtype=torch.bfloat16, device="cuda")
    c = ta.LatentCache(pool, i32([0, 0, 0]), i32([]), i32([0, 0]), h_q=4, rank=512)
    out, lse = c.decode(torch.ones((2, 4, 576), dtype=torch.bfloat16, device="cuda"), 0.1)
    assert c.device_status() == ta.TA_OK
    assert (out == 0).all() and (lse == -INF).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h", [4, 100])
def test_decode_scores_that_rise_and_fall(dtype, h):
    """The running reference has to move on every tile, and must not let a large
    early score be forgotten."""
    s = Setup([1200, 1200], h, 256, 64, dtype, seed=8)
    ramp = torch.linspace(-6, 6, 1200, device="cuda").to(s.dtype)
    for b, r in ((0, ramp), (1, ramp.flip(0))):
        pid, sl = s.slots(b)
        s.pool[pid, sl, 256:] = r[:, None].expand(1200, 64)
    q = s.randn(2, h, s.w)
    q[:, :, 256:] = 1
    q[:, 1, 256:] = -1
    out, lse = s.cache.decode(q, 0.5)
    check_absorbed(s, q, out, lse, 0.5)


def test_decode_many_equal_small_weights():
    """One large score and 20,000 far smaller ones that still hold half of the mass."""
    for dtype in ("bf16", "fp16"):
        s = Setup([20001], 4, 256, 16, dtype, seed=2, fill=0.0)
        pid, sl = s.slots(0)
        s.pool[pid, sl, 256:] = 0
        s.pool[pid, sl, :16] = 0
        s.pool[pid[0], sl[0], 256] = math.log(20000)
        q = torch.zeros((1, 4, s.w), dtype=s.dtype, device="cuda")
        q[:, :, 256] = 1
        out, lse = s.cache.decode(q, 1.0)
        check_absorbed(s, q, out, lse, 1.0)


def test_decode_page_outside_the_pool_reads_zeros():
    s = Setup([50, 20], 4, seed=3)
    s.values[1], s.values[4] = 10 ** 6, -1
    s.cache = s.handle()
    q = s.randn(2, 4, s.w)
    out, lse = s.cache.decode(q, 0.1)
    check_absorbed(s, q, out, lse, 0.1)
    assert s.cache.device_status() == ta.TA_OK


@pytest.mark.parametrize("h,dtype", [(8, "bf16"), (100, "fp16")])
def test_decode_scores_that_are_not_finite(h, dtype):
    """A NaN query reaches its head, a NaN row its sequence; a row whose score is
    -inf counts as if it were not there, +inf makes NaN."""
    kv = [40, 2000, 17, 600, 300]
    s = Setup(kv, h, dtype=dtype, seed=20)
    q = s.randn(len(kv), h, s.w)
    q[:, :, 0] = q[:, :, 0].abs() + 0.1
    base = [t.clone() for t in s.cache.decode(q, 0.07)]
    nan = torch.zeros((len(kv), h), dtype=torch.bool, device="cuda")
    q[1, 3, 7] = NAN
    nan[1, 3] = True
    pid, sl = s.slots(0)
    s.pool[pid[39], sl[39], 5] = NAN
    nan[0] = True
    pid, sl = s.slots(4)
    s.pool[pid[7], sl[7], 0] = INF
    nan[4] = True
    pid, sl = s.slots(3)
    s.pool[pid[500:], sl[500:], 0] = -INF
    out, lse = s.cache.decode(q, 0.07)
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
    assert torch.equal(torch.isnan(lse), nan)
    same = ~nan
    same[3] = False
    assert torch.equal(out[same], base[0][same]) and torch.equal(lse[same], base[1][same])
    keep = ~nan
    want = [t[keep] for t in ref.absorbed(torch.nan_to_num(q.double()), s.pool.double(), s.table, s.rank,
                                          0.07)]
    check(s.dtype, s.w, 2000, 6.0, out[keep], lse[keep], want)


def test_offsets_past_32_bits():
    """A pool of 2^31 elements and more, the pages at its end in use."""
    n = 240_000
    s = Setup([1], 16, seed=4)
    s.pool = torch.empty((n, 16, s.w), dtype=s.dtype, device="cuda")
    s.kv, s.indptr, s.last = np.array([300, 40]), np.array([0, 19, 22]), np.array([12, 8])
    s.values = np.array(list(range(n - 19, n)) + [0, n // 2, n - 25])
    assert (n - 25) * 16 * s.w > 2 ** 31
    for b in (0, 1):
        pid, sl = s.slots(b)
        s.pool[pid, sl] = s.randn(len(pid), s.w)
    s.cache = s.handle()
    q = s.randn(2, 16, s.w)
    out, lse = s.cache.decode(q, 0.07)
    assert s.cache.device_status() == ta.TA_OK
    small = s.pool[torch.from_numpy(s.values).cuda()].double()
    want = ref.absorbed(q.double(), small, (s.indptr, np.arange(22), s.last), 512, 0.07)
    check(s.dtype, s.w, 300, 6.0, out, lse, want)
    x = s.randn(2, 576)
    s.cache.append(x[:, :512], x[:, 512:], i32([0, 1, 2]))
    for b in (0, 1):
        pid, sl = s.slots(b)
        assert torch.equal(s.pool[pid[-1], sl[-1]], x[b])


# --------------------------------------------------------------------------
# trees
# --------------------------------------------------------------------------

def _tree(kind, n, rng):
    return {"chain": wl.chain_tree, "star": wl.star_tree, "binary": wl.binary_tree,
            "random": lambda m: wl.random_tree(m, rng)}[kind](n)


TREE = {
    # (prefix, nodes, q rows, kind) per sequence, heads, rank, rope, dtype
    "one_node": ([(0, 1, 1, "chain")], 4, 512, 64, "bf16"),
    "tiny": ([(0, 7, 7, "random"), (0, 12, 12, "binary")], 4, 256, 32, "fp16"),
    "prefixes": ([(40, 9, 9, "star"), (0, 20, 20, "random"), (300, 5, 5, "chain")], 8, 512, 64, "bf16"),
    "some_rows": ([(40, 30, 3, "random"), (17, 50, 50, "binary"), (5, 9, 0, "star")], 5, 512, 48, "fp16"),
    "no_rows_between": ([(0, 0, 0, "chain"), (130, 64, 64, "random"), (0, 0, 0, "chain"),
                         (16, 4, 4, "chain")], 32, 512, 64, "bf16"),
    "tile_edges": ([(64, 64, 64, "random"), (63, 65, 65, "random"), (128, 1, 1, "chain"),
                    (127, 2, 2, "star")], 16, 256, 64, "bf16"),
    "wide_heads": ([(100, 33, 33, "random"), (200, 7, 7, "binary")], 128, 512, 64, "bf16"),
    "odd_heads": ([(100, 33, 33, "random"), (200, 7, 7, "binary")], 37, 256, 16, "fp16"),
    "large_tree": ([(50, 400, 400, "random"), (0, 300, 257, "binary")], 6, 512, 64, "bf16"),
    "long": ([(9000, 64, 64, "random"), (17, 3, 3, "chain")], 16, 512, 64, "bf16"),
    "long_fp16": ([(5000, 20, 20, "binary")], 128, 256, 32, "fp16"),
}


class Trees:
    def __init__(self, spec, h, rank, rope, dtype, seed=0):
        rng = np.random.default_rng(seed)
        self.parents = [_tree(k, n, rng) if n else np.zeros(0, int) for _, n, _, k in spec]
        self.nodes, self.rows = [n for _, n, _, _ in spec], [r for _, _, r, _ in spec]
        self.s = Setup([p + n for p, n, _, _ in spec], h, rank, rope, dtype, seed=seed + 1)
        iv = [wl.tree_intervals(p) for p in self.parents if len(p)]
        self.order = i32(np.concatenate(iv)) if iv else i32(np.zeros((0, 2)))
        self.q = self.s.randn(sum(self.rows), h, self.s.w)

    def run(self, sm, **kw):
        return self.s.cache.tree_attn(self.q, i32(indptr(self.rows)), i32(indptr(self.nodes)), self.order,
                                      sm, **kw)

    def check(self, out, lse, sm):
        check_absorbed(self.s, self.q, out, lse, sm, self.rows, self.parents)


@pytest.mark.parametrize("name", list(TREE))
def test_tree(name):
    spec, h, rank, rope, dtype = TREE[name]
    t = Trees(spec, h, rank, rope, dtype, seed=len(name))
    for sm in (192 ** -0.5, 0.3):
        out, lse = t.run(sm)
        assert t.s.cache.device_status() == ta.TA_OK
        t.check(out, lse, sm)


@pytest.mark.parametrize("h,dtype", [(8, "bf16"), (64, "fp16")])
def test_tree_rows_that_others_see_may_hold_anything(h, dtype):
    """NaN and infinite rows of one branch leave the other branches' nodes alone."""
    spec = [(100, 21, 21, "star"), (900, 64, 64, "random"), (10, 12, 12, "binary")]
    t = Trees(spec, h, 512, 64, dtype, seed=5)
    base = [x.clone() for x in t.run(0.07)]
    touched = torch.zeros(97, dtype=torch.bool, device="cuda")
    at = 0
    for b, (prefix, n, _, _) in enumerate(spec):
        pid, sl = t.s.slots(b)
        for i, x in ((n - 1, NAN), (n - 2, INF), (n // 2, NAN)):
            t.s.pool[pid[prefix + i], sl[prefix + i], 3 * i:3 * i + 40] = x
            for j in range(n):
                k = j
                while k > i:
                    k = int(t.parents[b][k])
                touched[at + j] |= k == i
        at += n
    out, lse = t.run(0.07)
    assert t.s.cache.device_status() == ta.TA_OK
    assert torch.isnan(out[touched]).any(-1).all()
    free = ~touched
    ro, rl, mag, smag = ref.absorbed(t.q.double(), t.s.pool.double(), t.s.table, 512, 0.07, t.rows,
                                     t.parents)
    check(t.s.dtype, t.s.w, 1000, 6.0, out[free], lse[free],
          [x[free] for x in (ro, rl, mag, smag)])
    assert free.sum() > 60 and base is not None


def milliseconds(f, n=5):
    """The median of ``n`` calls, timed on the GPU."""
    e = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(n)]
    f()
    for a, b in e:
        a.record()
        f()
        b.record()
    torch.cuda.synchronize()
    return sorted(a.elapsed_time(b) for a, b in e)[n // 2]


@pytest.mark.parametrize("h,rank,dtype", [(1, 512, "bf16"), (8, 512, "fp16"), (24, 256, "bf16")])
def test_rows_not_seen_have_no_part_behind_long_prefixes(h, rank, dtype):
    """Draft rows that are not finite, in columns of either SM's half, behind 40,000
    rows: for the nodes that do not see them not a bit differs from a call without
    them, nor does the call take longer by more than a look at some tiles' values
    (a second pass over 40,000 rows would)."""
    spec = [(40000, 64, 64, "star"), (33000, 40, 40, "random")]
    t = Trees(spec, h, rank, 64, dtype, seed=6)
    base = [x.clone() for x in t.run(0.07)]
    quick = milliseconds(lambda: t.run(0.07))
    touched = torch.zeros(104, dtype=torch.bool, device="cuda")
    at = 0
    for b, (prefix, n, _, _) in enumerate(spec):
        pid, sl = t.s.slots(b)
        for i, c, x in ((n - 1, 5, NAN), (n - 2, rank - 1, INF), (n // 2, rank // 2 + 3, -INF),
                        (n // 3, rank + 9, NAN), (n // 4, slice(None), NAN)):
            t.s.pool[pid[prefix + i], sl[prefix + i], c] = x
            for j in range(n):
                k = j
                while k > i:
                    k = int(t.parents[b][k])
                touched[at + j] |= k == i
        at += n
    out, lse = t.run(0.07)
    assert t.s.cache.device_status() == ta.TA_OK
    free = ~touched
    assert free.sum() > 60
    assert torch.equal(out[free], base[0][free]) and torch.equal(lse[free], base[1][free])
    assert milliseconds(lambda: t.run(0.07)) < 2 * quick
    # of the others, those whose scores are -inf there (a column of one sign) are as
    # if the row were not there, all else is NaN
    want = ref.absorbed(t.q.double(), t.s.pool.double(), t.s.table, rank, 0.07, t.rows, t.parents)
    nan = torch.isnan(want[0]).any(-1)
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(out).any(-1), nan)
    assert torch.equal(torch.isnan(lse), nan)
    check(t.s.dtype, t.s.w, 40000, 6.0, out[~nan], lse[~nan], [x[~nan] for x in want])


def test_tree_is_decode_for_single_nodes():
    kv = [5, 130, 1, 2000, 16]
    s = Setup(kv, 24, 512, 64, seed=6)
    q = s.randn(5, 24, s.w)
    out, lse = s.cache.decode(q, 0.1)
    one = i32(np.arange(6))
    o2, l2 = s.cache.tree_attn(q, one, one, i32([[0, 1]] * 5), 0.1)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

APPEND = {
    # tokens held, new tokens, heads, rank, rope, dtype, layout, norm, rows_out
    "token": ([5, 16, 31, 0], [1, 1, 1, 1], 16, 512, 64, "bf16", "half", True, False),
    "prompt": ([0, 3], [37, 130], 128, 512, 64, "fp16", "interleaved", True, True),
    "plain": ([15, 1], [2, 20], 3, 256, 32, "bf16", None, False, True),
    "no_norm": ([15, 1], [2, 20], 5, 256, 48, "bf16", "half", False, False),
    "norm_only": ([15, 1], [2, 20], 5, 512, 16, "fp16", None, True, True),
    "small_rope": ([0], [70], 40, 256, 16, "bf16", "interleaved", True, True),
    "no_queries": ([9, 0, 4], [3, 0, 60], 0, 512, 64, "bf16", "half", True, True),
    "gaps": ([3, 0, 0, 700], [0, 5, 0, 9], 1, 512, 48, "fp16", "half", True, False),
}


@pytest.mark.parametrize("name", list(APPEND))
def test_append(name):
    held, new, h, rank, rope, dtype, layout, normed, with_rows = APPEND[name]
    queries, h = h > 0, max(h, 1)
    s = Setup([a + b for a, b in zip(held, new)], h, rank, rope, dtype, seed=len(name))
    n, half = sum(new), torch.finfo(s.dtype).eps / 2
    down, up = s.randn(n, rank + rope + 8), s.randn(n, h, rope + 128)
    latent, k = down[:, :rank], down[:, rank:rank + rope]
    q = up[:, :, 128:] if queries else None
    weight = (1 + 0.2 * s.randn(rank).float()).to(s.dtype) if normed else None
    rng = np.random.default_rng(0)
    pos = np.concatenate([np.arange(c, c + m) for c, m in zip(rng.integers(0, 1 << 30, len(new)), new)])
    r = ta.Rope(layout, rope, theta=5e5, scale=0.25, magnitude=1.25) if layout else None
    q_out = torch.full((n, h, s.w), 7.0, dtype=s.dtype, device="cuda") if queries else None
    rows = torch.empty((n, s.w), dtype=s.dtype, device="cuda") if with_rows else None
    before = s.pool.clone()
    got = s.cache.append(latent, k, i32(indptr(new)), i32(pos), q_rope=q, rope=r, weight=weight,
                         norm_eps=1e-5, q_out=None if q is None else q_out[:, :, rank:], rows_out=rows)
    assert s.cache.device_status() == ta.TA_OK
    freq = 0.25 * 5e5 ** (-torch.arange(rope // 2, dtype=torch.float64, device="cuda") * 2 / rope)
    mag = 1.25 if layout else 1.0
    p = torch.from_numpy(pos).cuda()
    want_k = ref.rotate(k.double(), p, layout, freq, mag)
    want_l = ref.norm(latent.double(), None if weight is None else weight.double(), 1e-5)

    # below the smallest normal number steps no longer shrink with the value: half
    # a step is smallest_normal * half there (2^-25 in fp16)
    least = torch.finfo(s.dtype).smallest_normal * half

    def close(a, b, length):
        far = (a.double() - b).abs() - (half * b.abs() + 2.0 ** -19 * length + least)
        assert (far <= 0).all(), far.max()

    def pair(x):     # a bound of every pair's length
        return x.double().abs().amax(-1, keepdim=True) * 1.5 * mag

    at = 0
    touched = torch.zeros(s.pool.shape[:2], dtype=torch.bool, device="cuda")
    for b, m in enumerate(new):
        pid, sl = s.slots(b)
        pid, sl = pid[len(pid) - m:], sl[len(sl) - m:]
        touched[pid, sl] = True
        row, t = s.pool[pid, sl], slice(at, at + m)
        if weight is None:
            assert torch.equal(row[:, :rank], latent[t])
        else:
            close(row[:, :rank], want_l[t], want_l[t].abs())
        if layout is None:
            assert torch.equal(row[:, rank:], k[t])
        else:
            close(row[:, rank:], want_k[t], pair(k[t]))
        if rows is not None:
            assert torch.equal(rows[t], row)
        at += m
    keep = ~touched
    assert torch.equal(s.pool[keep].view(torch.int16), before[keep].view(torch.int16))
    if queries:
        assert got.data_ptr() == q_out[:, :, rank:].data_ptr() and (q_out[:, :, :rank] == 7).all()
        if layout is None:
            assert torch.equal(got, q)
        else:
            close(got, ref.rotate(q.double(), p, layout, freq, mag), pair(q))
        # in place, and into a new tensor
        new_q = s.cache.append(latent, k, i32(indptr(new)), i32(pos), q_rope=q, rope=r, weight=weight,
                               norm_eps=1e-5)
        assert torch.equal(new_q, got)
        s.cache.append(latent, k, i32(indptr(new)), i32(pos), q_rope=q, rope=r, weight=weight,
                       norm_eps=1e-5, q_out=q)
        assert torch.equal(q, got)
    else:
        assert got is None


def test_append_heads_outside_tokens():
    """Queries laid out head by head."""
    s = Setup([9, 4], 6, 512, 64, seed=2)
    x, q = s.randn(7, 576), s.randn(6, 7, 64).transpose(0, 1)
    r, pos, ptr = ta.Rope("half", 64), i32(range(7)), i32([0, 4, 7])
    a = s.cache.append(x[:, :512], x[:, 512:], ptr, pos, q_rope=q, rope=r)
    b = s.cache.append(x[:, :512], x[:, 512:], ptr, pos, q_rope=q.contiguous(), rope=r)
    assert torch.equal(a, b)


def test_append_of_a_bad_table_writes_nothing():
    s = Setup([40, 20], 2, 256, 32, seed=3, fill=0.0)
    x, before = s.randn(4, 288), s.pool.clone()
    for kw in (dict(page_indptr=[0, 3, 2]), dict(length_info=[8, 17]), dict(length_info=[8, 0]),
               dict(page_values=[0, 1, 2, 3, 99])):
        c = s.handle(**kw)
        c.append(x[:, :256], x[:, 256:], i32([0, 0, 4]))
        assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
        assert torch.equal(s.pool, before)


# --------------------------------------------------------------------------
# bad tables, compaction, copies
# --------------------------------------------------------------------------

def test_bad_tables_compute_nothing():
    s = Setup([40, 20, 7], 8, 256, 32, seed=7)
    q = s.randn(3, 8, s.w)
    bad = [dict(page_indptr=[0, 3, 2, 6]), dict(page_indptr=[1, 3, 5, 6]), dict(length_info=[8, 17, 7]),
           dict(length_info=[0, 4, 7]), dict(page_indptr=[0, 3, 5, 99])]
    order = i32([[0, 1]] * 3)
    for kw in bad:
        c = s.handle(**kw)
        out, lse = torch.full((3, 8, 256), 5.0, dtype=s.dtype, device="cuda"), \
            torch.full((3, 8), 5.0, device="cuda")
        c.decode(q, 0.1, out=out, lse=lse)
        assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
        c.tree_attn(q, i32(range(4)), i32(range(4)), order, 0.1, out=out, lse=lse)
        assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
        assert (out == 5).all() and (lse == 5).all()
    c = s.handle()
    for qi, mi in (([0, 2, 1, 3], [0, 1, 2, 3]), ([0, 1, 2, 3], [0, 2, 1, 3]), ([0, 1, 2, 4], [0, 1, 2, 3]),
                   ([0, 1, 1, 3], [0, 1, 2, 3]), ([1, 1, 2, 3], [0, 1, 2, 3])):
        c.tree_attn(q, i32(qi), i32(mi), order, 0.1, out=out, lse=lse)
        assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
        assert (out == 5).all() and (lse == 5).all()
    # a tree longer than its sequence
    big = i32([[0, 1]] * 12)
    c.tree_attn(q, i32([0, 1, 2, 3]), i32([0, 2, 4, 12]), big, 0.1, out=out, lse=lse)
    assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT and (out == 5).all()


@pytest.mark.parametrize("rank,rope,dtype", [(512, 64, "bf16"), (256, 16, "fp16"), (256, 48, "bf16")])
def test_compact_and_copies(rank, rope, dtype):
    s = Setup([45, 100, 7, 16], 4, rank, rope, dtype, seed=11, fill=0.0)
    trees, paths = [20, 64, 7, 5], [[0, 3, 7, 19], [1, 2, 40, 41, 63], [], [0, 1, 2]]
    mn, ai, an = indptr(trees), indptr([len(p) for p in paths]), sum(paths, [])
    five = s.pool.double().cpu().numpy()[:, None, None]
    want = paged.compact(five, *s.table, mn, ai, an)
    got = s.cache.compact(i32(mn), i32(ai), i32(an))
    assert s.cache.device_status() == ta.TA_OK
    assert np.array_equal(s.pool.double().cpu().numpy(), want[0][:, 0, 0])
    n = want[1][-1]
    assert got[0].tolist() == want[1] and got[1][:n].tolist() == want[2] and got[2].tolist() == want[3]
    assert got[3][:int(got[4])].tolist() == want[4]
    c = s.cache.with_table(got[0], got[1], got[2])
    assert c.workspace is s.cache.workspace and c.rank == rank
    pool = s.pool.clone()
    c.copy_pages(i32([1, 0, 5]), i32([3, 2, 5]))
    pool[3], pool[2] = pool[1].clone(), pool[0].clone()
    assert c.device_status() == ta.TA_OK and torch.equal(s.pool, pool)
    c.copy_pages(i32([1, 4]), i32([4, 6]))        # 4 is a source too
    assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    pool[6] = pool[4]
    assert torch.equal(s.pool, pool)


def test_many_copies():
    """Enough pages for the marked form, their last line short."""
    pool = torch.randn((9000, 16, 272), device="cuda").to(torch.bfloat16)
    c = ta.LatentCache(pool, i32([0, 1]), i32([0]), i32([3]), h_q=1, rank=256)
    perm = torch.randperm(9000, device="cuda").int()
    src, dst = perm[:4000].contiguous(), perm[4000:8000].contiguous()
    want = pool.clone()
    want[dst.long()] = want[src.long()]
    for _ in range(2):
        c.copy_pages(src, dst)
        assert c.device_status() == ta.TA_OK and torch.equal(pool, want)


# --------------------------------------------------------------------------
# expanded form
# --------------------------------------------------------------------------

EXPANDED = {
    # new rows, kv rows per sequence, heads, d, rope, dtype
    "one": ([1], [1], 2, 128, 64, "bf16"),
    "prompts": ([7, 130, 64], [7, 130, 64], 4, 128, 64, "bf16"),
    "edges": ([127, 128, 129, 1, 256, 257], [127, 128, 129, 1, 256, 257], 2, 64, 32, "fp16"),
    "chunks": ([5, 100, 33], [300, 129, 2000], 3, 128, 48, "bf16"),
    "one_token_each": ([1, 1, 1, 1], [1, 128, 129, 700], 8, 128, 64, "fp16"),
    "empties": ([0, 9, 0, 0, 70], [5, 9, 0, 12, 70], 4, 64, 16, "bf16"),
    "one_head_long": ([600], [2500], 1, 128, 64, "bf16"),
    "many_short": ([1 + i % 13 for i in range(90)], [1 + i % 13 + (i % 5) * 31 for i in range(90)], 5, 64, 64,
                   "fp16"),
    "many_heads": ([40, 3], [40, 70], 200, 64, 16, "bf16"),
}


class Expanded:
    def __init__(self, new, kv, h, d, rope, dtype, seed=0, packed=False, spare=0):
        g = torch.Generator("cuda").manual_seed(seed)
        self.dtype, self.new, self.kv, self.d, self.h, self.rope = DT[dtype], new, kv, d, h, rope
        self.randn = lambda *x: torch.randn(x, generator=g, device="cuda").to(self.dtype)
        nq, nk = sum(new), sum(kv)
        self.q, both, rows = self.randn(nq, h, d + rope), self.randn(nk, h, 2 * d), self.randn(nk, 64 + rope)
        self.k, self.v, self.kr = both[:, :, :d], both[:, :, d:], rows[:, 64:]
        if packed:
            self.k, self.v, self.kr = [x.contiguous() for x in (self.k, self.v, self.kr)]
        self.out = torch.full((nq, h, d), 5.0, dtype=self.dtype, device="cuda")
        self.lse = torch.full((nq, h), 5.0, device="cuda")
        self.qi, self.ki = i32(indptr(new)), i32(indptr(kv))
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")

    def run(self, sm, **kw):
        a = dict(q=self.q, q_indptr=self.qi, k=self.k, k_rope=self.kr, v=self.v, kv_indptr=self.ki,
                 out=self.out, lse=self.lse)
        a.update(kw)
        ta.tree_attn_expanded(*a.values(), sm, self.ws)
        return a["out"], a["lse"]

    def check(self, out, lse, sm):
        want = ref.expanded(self.q.double(), self.k.double(), self.kr.double(), self.v.double(), self.new,
                            self.kv, sm)
        check(self.dtype, self.d + self.rope, max(self.kv), 6.0, out, lse, want)


@pytest.mark.parametrize("name", list(EXPANDED))
@pytest.mark.parametrize("packed", [False, True])
def test_expanded(name, packed):
    e = Expanded(*EXPANDED[name], seed=len(name), packed=packed)
    for sm in ((e.d + e.rope) ** -0.5, 0.4):
        out, lse = e.run(sm)
        assert ta.device_status(e.ws) == ta.TA_OK
        e.check(out, lse, sm)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_expanded_rows_not_seen_may_hold_anything(dtype):
    """Later rows of the sequence, other sequences' and those behind the last."""
    e = Expanded([70, 300, 40], [70, 700, 40], 3, 128, 64, dtype, seed=3)
    for j in (50, 69, 70 + 690, 770):                   # rows of k and v; the last is sequence 2's first
        e.k[j, 1, 5], e.v[j, 2, 9], e.kr[j, 3] = NAN, INF, NAN
        e.v[j, 0] = NAN
    out, lse = e.run(0.07)
    assert ta.device_status(e.ws) == ta.TA_OK
    free = torch.ones(410, dtype=torch.bool, device="cuda")
    free[50:70], free[70 + 290:] = False, False
    want = [t[free] for t in ref.expanded(e.q.double(), e.k.double(), e.kr.double(), e.v.double(), e.new,
                                          e.kv, 0.07)]
    check(e.dtype, 192, 700, 6.0, out[free], lse[free], want)
    assert torch.isnan(out[~free]).any(-1).all()


def check_expanded_with_odd_values(e, out, lse, sm):
    """Element by element: NaN and infinities where the reference has them, its
    numbers elsewhere."""
    want = ref.expanded(e.q.double(), e.k.double(), e.kr.double(), e.v.double(), e.new, e.kv, sm)
    fin = torch.isfinite(want[0])
    assert torch.equal(torch.isfinite(out), fin)
    assert torch.equal(torch.nan_to_num(out[~fin].double(), nan=7.0, posinf=8.0, neginf=9.0),
                       torch.nan_to_num(want[0][~fin], nan=7.0, posinf=8.0, neginf=9.0))
    zero = lambda x: torch.where(fin, x, 0.0)
    check(e.dtype, e.d + e.rope, max(e.kv), 6.0, zero(out.double()), lse, [zero(want[0]), *want[1:]])
    return fin


@pytest.mark.parametrize("h,d,rope,dtype", [(3, 128, 64, "bf16"), (5, 64, 32, "fp16")])
def test_expanded_rows_not_seen_have_no_part_behind_long_prefixes(h, d, rope, dtype):
    """Values that are not finite among the last rows of long sequences: for the q
    rows that do not see them not a bit differs from a call without them; a second
    look at all units is the most that they cost."""
    new, kv = [300, 64, 150, 20], [40300, 33064, 150, 90]
    e = Expanded(new, kv, h, d, rope, dtype, seed=30)
    base = [x.clone() for x in e.run(0.07)]
    quick = milliseconds(lambda: e.run(0.07))
    first, seen_from = 0, torch.full((sum(new),), -1, device="cuda")
    at = 0
    for n, m in zip(new, kv):
        odd = [(m - 1, slice(None), NAN), (m - 5, d - 1, INF), (m - 17, 0, -INF), (m - n // 2, 7, NAN)]
        for j, c, x in odd:
            e.v[first + j, :, c] = x
        seen_from[at:at + n] = min(j for j, _, _ in odd) - (m - n)
        first, at = first + m, at + n
    own = torch.cat([torch.arange(n, device="cuda") for n in new])
    free = own < seen_from
    out, lse = e.run(0.07, out=torch.zeros_like(e.out), lse=torch.zeros_like(e.lse))
    assert ta.device_status(e.ws) == ta.TA_OK
    assert free.sum() > 200
    assert torch.equal(out[free], base[0][free]) and torch.equal(lse, base[1])
    assert milliseconds(lambda: e.run(0.07)) < 4 * quick
    fin = check_expanded_with_odd_values(e, out, lse, 0.07)
    assert (~fin).any() and torch.equal(out[fin], base[0][fin])


@pytest.mark.parametrize("name", ["edges", "chunks", "empties", "many_short", "one_head_long"])
def test_expanded_values_that_are_not_finite(name):
    """Infinities and NaN all over the values, seen and not; with keys whose score is
    -inf, whose rows count as if they were not there."""
    e = Expanded(*EXPANDED[name], seed=31)
    g = torch.Generator("cuda").manual_seed(5)
    nk = sum(e.kv)
    pick = lambda share: torch.rand(e.v.shape, generator=g, device="cuda") < share
    e.v[pick(0.0007)] = NAN
    e.v[pick(0.0007)] = INF
    e.v[pick(0.0007)] = -INF
    e.q[:, :, 1] = e.q[:, :, 1].abs() + 0.1
    gone = torch.rand(nk, generator=g, device="cuda") < 0.1
    e.k[gone, :, 1] = -INF
    e.v[gone, :, :3] = NAN
    out, lse = e.run(0.07)
    assert ta.device_status(e.ws) == ta.TA_OK
    check_expanded_with_odd_values(e, out, lse, 0.07)
    again = e.run(0.07, out=torch.zeros_like(out), lse=torch.zeros_like(lse))
    assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(again[0], nan=7.0))
    # all of them, for one sequence after the other
    e.v[:] = NAN
    out, lse = e.run(0.07)
    assert ta.device_status(e.ws) == ta.TA_OK
    check_expanded_with_odd_values(e, out, lse, 0.07)


def test_expanded_spare_rows_are_left_alone():
    """Buffers longer than the batch: behind the last sequence nothing is read or
    written.  (The totals are the batch's, the tensors views.)"""
    e = Expanded([20, 100], [20, 150], 4, 64, 32, "bf16", seed=4)
    pad = lambda x: torch.cat([x, torch.full_like(x[:50], NAN)])
    out, lse = pad(e.out), pad(e.lse)
    e.q, e.k, e.v, e.kr = [pad(x)[:x.shape[0]] for x in (e.q, e.k, e.v, e.kr)]
    e.run(0.1, out=out[:120], lse=lse[:120])
    e.check(out[:120], lse[:120], 0.1)
    assert torch.isnan(out[120:]).all() and torch.isnan(lse[120:]).all()


def test_expanded_bad_arrays_compute_nothing():
    e = Expanded([4, 6], [5, 9], 2, 64, 16, "bf16", seed=5)
    for qi, ki in (([0, 4, 9], [0, 5, 14]), ([0, 11, 10], [0, 5, 14]), ([1, 4, 10], [0, 5, 14]),
                   ([0, 4, 10], [0, 3, 14]), ([0, 4, 10], [0, 5, 15]), ([0, 4, 10], [0, -5, 14])):
        out, lse = e.run(0.1, q_indptr=i32(qi), kv_indptr=i32(ki))
        assert ta.device_status(e.ws) == ta.TA_ERR_INVALID_ARGUMENT
        assert (out == 5).all() and (lse == 5).all()


def test_expanded_refusals():
    e = Expanded([4], [5], 2, 64, 16, "bf16")
    for kw in (dict(q=e.q.cpu()), dict(k=e.k.half()), dict(v=e.v[:, :1]), dict(k_rope=e.kr[:4]),
               dict(out=e.out.float()), dict(lse=e.lse.half()), dict(kv_indptr=e.ki.long()),
               dict(kv_indptr=e.ki[:1]), dict(q=e.q.transpose(0, 2)), dict(out=e.out[:3])):
        with pytest.raises(ValueError):
            e.run(0.1, **kw)
    with pytest.raises(ta.TreeAttnError):
        e.run(math.nan)


def test_python_refusals():
    s = Setup([5, 40], 4, 512, 64, seed=1)
    c, q = s.cache, s.randn(2, 4, 576)
    x, ptr = s.randn(3, 576), i32([0, 1, 3])
    lat, k = x[:, :512], x[:, 512:]
    for f in (lambda: c.decode(q[:1], 0.1), lambda: c.decode(q.float(), 0.1),
              lambda: c.decode(q.cpu(), 0.1), lambda: c.decode(q, 0.1, out=q),
              lambda: c.tree_attn(q, ptr[:2], ptr, i32([[0, 1]] * 3), 0.1),
              lambda: c.tree_attn(q, ptr, ptr, i32([0, 1]), 0.1),
              lambda: c.append(lat, k[:2], ptr), lambda: c.append(lat.float(), k, ptr),
              lambda: c.append(lat, k, ptr, rope=ta.Rope("half", 64)),
              lambda: c.append(lat, k, ptr, q_out=s.randn(3, 4, 64)),
              lambda: c.append(lat, k, ptr, q_rope=s.randn(3, 4, 32)),
              lambda: c.append(lat, k, ptr, q_rope=s.randn(3, 4, 128)[..., ::2]),
              lambda: c.append(lat, k, ptr, rows_out=x.t()),
              lambda: ta.LatentCache(s.pool, i32([0, 1]), i32([0]), i32([1, 1]), h_q=4, rank=512)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: c.append(lat, k, ptr, i32([0, 1, 2]), rope=ta.Rope("half", 32)),
              lambda: c.decode(q, math.inf),
              lambda: ta.LatentCache(s.pool, i32([0, 1]), i32([0]), i32([1]), h_q=200, rank=512),
              lambda: ta.LatentCache(s.pool, i32([0, 1]), i32([0]), i32([1]), h_q=4, rank=500)):
        with pytest.raises(ta.TreeAttnError):
            f()


# --------------------------------------------------------------------------
# used together
# --------------------------------------------------------------------------

def test_absorbed_and_expanded_agree():
    """A prompt through the cache and through keys and values per head.  The two
    differ by the rounding of the absorbed queries, of keys and values to 16
    bits: half a step of each product's parts, a few times the forms' own."""
    g = torch.Generator("cuda").manual_seed(3)
    h, d, n = 4, 128, 200
    s = Setup([n], h, 512, 64, "fp16", seed=5)
    pid, sl = s.slots(0)
    rows = s.pool[pid, sl]
    wk, wv = (torch.randn((2, h, 512, d), generator=g, device="cuda") / 512 ** 0.5)
    q = s.randn(n, h, d + 64)
    qa = torch.cat([torch.einsum("nhd,hrd->nhr", q[..., :d].float(), wk), q[..., d:].float()], -1).half()
    sm = (d + 64) ** -0.5
    out, lse = s.cache.tree_attn(qa, i32([0, n]), i32([0, n]), i32(wl.tree_intervals(wl.chain_tree(n))), sm)
    k = torch.einsum("tr,hrd->thd", rows[:, :512].float(), wk).half()
    v = torch.einsum("tr,hrd->thd", rows[:, :512].float(), wv).half()
    o2, l2 = torch.empty((n, h, d), dtype=torch.half, device="cuda"), torch.empty((n, h), device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ta.tree_attn_expanded(q, i32([0, n]), k, rows[:, 512:], v, i32([0, n]), o2, l2, sm, ws)
    assert ta.device_status(ws) == ta.TA_OK
    o1 = torch.einsum("nhr,hrd->nhd", out.float(), wv)
    # scores: 2^-11 of |q| |k| per product, random signs; bounded by their sum over sqrt(elements)
    assert (lse - l2).abs().max() < 2.0 ** -6
    assert (o1 - o2.float()).abs().max() < 2.0 ** -5


@pytest.mark.parametrize("captured", [False, True])
def test_decoding_loop(captured):
    """append a draft tree, verify it, keep the accepted path, append a token and
    attend it, with the references in step; also from a captured graph, replayed."""
    h, rank, rope = 16, 512, 64
    ctx, nodes = [37, 500, 0, 129], 20
    paths = [[0, 2], [0], [0, 1, 3, 9], []]
    rng = np.random.default_rng(1)
    parents = [wl.random_tree(nodes, rng) for _ in ctx]
    kv = [c + nodes for c in ctx]
    s = Setup(kv, h, rank, rope, "bf16", seed=3, fill=0.0)
    start = s.pool.clone()
    n, r = nodes * len(ctx), ta.Rope("half", rope)
    x, q, q2 = s.randn(n, 576), s.randn(n, h, s.w), s.randn(4, h, s.w)
    q_in = q.clone()
    pos = i32(np.concatenate([[c + d for d in wl.tree_depths(p)] for c, p in zip(ctx, parents)]))
    mn, order = i32(indptr([nodes] * 4)), i32(np.concatenate([wl.tree_intervals(p) for p in parents]))
    ai, an = i32(indptr([len(p) for p in paths])), i32(sum(paths, []))
    bufs = [torch.empty_like(t) for t in (s.cache.page_indptr, s.cache.page_values, s.cache.length_info)]

    def step():
        s.pool.copy_(start)
        q.copy_(q_in)
        s.cache.append(x[:, :rank], x[:, rank:], mn, pos, q_rope=q[:, :, rank:], rope=r,
                       q_out=q[:, :, rank:])
        a = s.cache.tree_attn(q, mn, mn, order, 0.07)
        verified = s.pool.clone()
        t = s.cache.compact(mn, ai, an, new_page_indptr=bufs[0], new_page_values=bufs[1],
                            new_length_info=bufs[2])
        c = s.cache.with_table(*t[:3])
        return a, verified, c.decode(q2, 0.07), c

    step()
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        for _ in range(3):
            for t in (*res[0], *res[2]):
                t.fill_(3)
            g.replay()
    else:
        res = step()
    (out, lse), verified, (o2, l2), c = res
    assert c.device_status() == ta.TA_OK
    now, s.pool = s.pool, verified
    check_absorbed(s, q, out, lse, 0.07, [nodes] * 4, parents)
    want, ni, nv, nl, _ = paged.compact(verified.double().cpu().numpy()[:, None, None], *s.table,
                                        mn.tolist(), ai.tolist(), an.tolist())
    assert np.array_equal(now.double().cpu().numpy(), want[:, 0, 0])
    s.pool, s.indptr, s.values, s.last = now, np.array(ni), np.array(nv + [0]), np.array(nl)
    s.kv = np.array([c + len(p) for c, p in zip(ctx, paths)])
    check_absorbed(s, q2, o2, l2, 0.07)


def test_streams_and_repetition():
    """Two handles on two streams at once; results do not depend on timing."""
    a, b = Setup([3000, 40, 900], 64, seed=1), Setup([50] * 40 + [5000], 16, 256, 32, "fp16", seed=2)
    qa, qb = a.randn(3, 64, a.w), b.randn(41, 16, b.w)
    wa, wb = a.cache.decode(qa, 0.07), b.cache.decode(qb, 0.07)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [(a.cache.decode(qa, 0.07, stream=s1), b.cache.decode(qb, 0.07, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x[0], wa[0]) and torch.equal(x[1], wa[1])
        assert torch.equal(y[0], wb[0]) and torch.equal(y[1], wb[1])
    check_absorbed(a, qa, *wa, 0.07)
    check_absorbed(b, qb, *wb, 0.07)


def test_one_workspace_for_several_caches():
    """Handles of other heads, ranks and pools take turns on one workspace."""
    a = Setup([1700, 3], 128, 512, 64, seed=1)   # the larger pool, so the larger workspace
    b = Setup([900, 70, 5], 4, 256, 16, "fp16", seed=2)
    shared = ta.LatentCache(b.pool, *[i32(t) for t in b.table], h_q=4, rank=256,
                            workspace=a.cache.workspace)
    assert shared.workspace is a.cache.workspace
    qa, qb = a.randn(2, 128, a.w), b.randn(3, 4, b.w)
    for _ in range(3):
        oa, ob = a.cache.decode(qa, 0.07), shared.decode(qb, 0.07)
        shared.copy_pages(i32([0]), i32([0]))
    check_absorbed(a, qa, *oa, 0.07)
    check_absorbed(b, qb, *ob, 0.07)
    assert shared.device_status() == ta.TA_OK


def test_workspaces_of_the_two_kinds_of_cache_are_kept_apart():
    """What one keeps at zero lies where the other has its partial states."""
    s = Setup([900, 3], 4, 256, 16)
    table = [i32(x) for x in s.table]
    pool = torch.zeros(s.pool.shape[0], 2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="kind of cache"):
        ta.PagedCache(pool, *table, h_q=4, workspace=s.cache.workspace)
    other = ta.PagedCache(pool, *table, h_q=4)
    with pytest.raises(ValueError, match="kind of cache"):
        ta.LatentCache(s.pool, *table, h_q=4, rank=256, workspace=other.workspace)


def test_a_reset_workspace_serves_the_other_kind():
    """Views are refused like the tensor itself; after a reset every call of the
    other kind is as on a workspace of its own, copies by marks among them."""
    s = Setup([3000, 40, 900], 64, 256, 16, seed=26)
    table = [i32(x) for x in s.table]
    q = s.randn(3, 64, s.w)
    want = [t.clone() for t in s.cache.decode(q, 0.07)]
    g = torch.Generator("cuda").manual_seed(27)
    pool = torch.randn((6000, 2, 2, 16, 64), generator=g, device="cuda").bfloat16()
    small = ta.PagedCache(pool, *table, h_q=4)
    for ws in (s.cache.workspace[:], s.cache.workspace.view(torch.int32), s.cache.workspace[256:]):
        with pytest.raises(ValueError, match="kind of cache"):
            ta.PagedCache(pool, *table, h_q=4, workspace=ws)
    with pytest.raises(ValueError, match="kind of cache"):
        ta.LatentCache(s.pool, *table, h_q=64, rank=256, workspace=small.workspace[:])
    ws = torch.zeros(max(s.cache.workspace.numel(), small.workspace.numel()), dtype=torch.uint8, device="cuda")
    latent = ta.LatentCache(s.pool, *table, h_q=64, rank=256, workspace=ws)
    latent.decode(q, 0.07)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ta.reset_workspace(ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    shared = ta.PagedCache(pool, *table, h_q=4, workspace=ws)
    assert shared.workspace is ws
    perm = torch.randperm(6000, generator=torch.Generator().manual_seed(1)).int().cuda()
    src, dst = perm[:3000].contiguous(), perm[3000:].contiguous()
    qp = torch.randn((3, 4, 64), generator=g, device="cuda").bfloat16()
    for _ in range(2):
        assert all(torch.equal(x, y) for x, y in zip(shared.decode(qp, 0.1), small.decode(qp, 0.1)))
        after = pool.clone()
        after[dst.long()] = after[src.long()]
        shared.copy_pages(src, dst)
        assert shared.device_status() == ta.TA_OK and torch.equal(pool, after)
    ta.reset_workspace(ws, stream=torch.cuda.current_stream().cuda_stream)
    latent = ta.LatentCache(s.pool, *table, h_q=64, rank=256, workspace=ws)
    got = latent.decode(q, 0.07)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_copies_by_marks_between_attention_on_one_workspace():
    """Handles of other pools and ranks: what one call leaves in a workspace is not
    in the way of another's marks."""
    a = Setup([1700, 3, 900], 128, 512, 64, seed=1)
    g = torch.Generator("cuda").manual_seed(2)
    pool = torch.randn((7000, 16, 272), generator=g, device="cuda").bfloat16()
    b = ta.LatentCache(pool, i32([0, 1]), i32([0]), i32([3]), h_q=1, rank=256)
    a.cache = ta.LatentCache(a.pool, *[i32(x) for x in a.table], h_q=128, rank=512, workspace=b.workspace)
    assert a.cache.workspace is b.workspace
    q = a.randn(3, 128, a.w)
    perm = torch.randperm(7000, generator=torch.Generator().manual_seed(3)).int().cuda()
    src, dst = perm[:3500].contiguous(), perm[3500:].contiguous()
    for _ in range(3):
        out, lse = a.cache.decode(q, 0.07)
        after = pool.clone()
        after[dst.long()] = after[src.long()]
        b.copy_pages(src, dst)
        assert b.device_status() == ta.TA_OK and torch.equal(pool, after)
        check_absorbed(a, q, out, lse, 0.07)
        src, dst = dst, src


# --------------------------------------------------------------------------
# the ends of what is allowed
# --------------------------------------------------------------------------

@pytest.mark.parametrize("sm", [0.0, -0.07])
def test_scales_of_zero_and_below(sm):
    s = Setup([700, 3, 130], 20, 512, 64, seed=12)
    q = s.randn(3, 20, s.w)
    out, lse = s.cache.decode(q, sm)
    check_absorbed(s, q, out, lse, sm)
    e = Expanded([70, 300], [90, 300], 3, 128, 64, "bf16", seed=13)
    out, lse = e.run(sm)
    assert ta.device_status(e.ws) == ta.TA_OK
    e.check(out, lse, sm)


def test_a_scale_of_zero_weighs_large_rows_as_any_other():
    """Products near the end of float32's range times zero are zero; an infinite one
    is NaN, for the rows that see it."""
    s = Setup([200, 40, 30], 5, 256, 64, seed=24)
    q = s.randn(3, 5, s.w)
    q[:, :, 256] = 1.5e19
    pid, sl = s.slots(0)
    s.pool[pid, sl, 256] = torch.where(torch.arange(200, device="cuda") % 2 == 0, 1.5e19, 0.0).to(s.dtype)
    pid, sl = s.slots(1)
    s.pool[pid[17], sl[17], 256] = -INF
    out, lse = s.cache.decode(q, 0.0)
    nan = torch.zeros((3, 5), dtype=torch.bool, device="cuda")
    nan[1] = True
    assert torch.equal(torch.isnan(out).all(-1), nan) and torch.equal(torch.isnan(lse), nan)
    want = [t[~nan] for t in ref.absorbed(q.double(), s.pool.double(), s.table, 256, 0.0)]
    assert (want[1] - torch.log2(torch.tensor([200.0, 30.0], device="cuda")).repeat_interleave(5)).abs().max() < 1e-6
    check(s.dtype, s.w, 200, 6.0, out[~nan], lse[~nan], want)
    # a tree's nodes do not see one another's branches at any scale
    t = Trees([(20, 12, 12, "star")], 5, 256, 64, "bf16", seed=25)
    pid, sl = t.s.slots(0)
    t.s.pool[pid[30], sl[30], 7] = INF
    out, lse = t.run(0.0)
    keep = torch.arange(12, device="cuda") != 10
    assert torch.isnan(out[10]).all() and torch.isnan(lse[10]).all()
    want = ref.absorbed(t.q.double(), t.s.pool.double(), t.s.table, 256, 0.0, t.rows, t.parents)
    check(t.s.dtype, t.s.w, 32, 6.0, out[keep], lse[keep], [x[keep] for x in want])


def test_expanded_rows_head_by_head():
    """Queries, keys and values laid out with the heads outside the tokens."""
    e = Expanded([70, 130], [200, 130], 5, 128, 48, "fp16", seed=14)
    far = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)
    want = [t.clone() for t in e.run(0.07)]
    got = e.run(0.07, q=far(e.q), k=far(e.k), v=far(e.v), out=torch.zeros_like(e.out),
                lse=torch.zeros_like(e.lse))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    e.check(*want, 0.07)


def test_expanded_repeats_and_captures():
    """A captured call replayed, and another beside it on the same workspace."""
    e = Expanded([200, 3, 900], [200, 50, 1500], 4, 128, 64, "bf16", seed=15)
    want = [t.clone() for t in e.run(0.07)]
    e.check(*want, 0.07)
    out, lse = torch.zeros_like(e.out), torch.zeros_like(e.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.run(0.07, out=out, lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        g.replay()
        with torch.cuda.stream(side):
            o2, l2 = e.run(0.07, out=torch.empty_like(out), lse=torch.empty_like(lse))
    torch.cuda.synchronize()
    for o, x in ((out, want[0]), (o2, want[0]), (lse, want[1]), (l2, want[1])):
        assert torch.equal(o, x)
    assert ta.device_status(e.ws) == ta.TA_OK


def test_expanded_largest_batch():
    rng = np.random.default_rng(16)
    kv = rng.integers(0, 6, 16384)
    new = np.minimum(rng.integers(0, 4, 16384), kv)
    e = Expanded([int(x) for x in new], [int(x) for x in kv], 2, 64, 16, "bf16", seed=16)
    out, lse = e.run(0.1)
    assert ta.device_status(e.ws) == ta.TA_OK
    e.check(out, lse, 0.1)
    with pytest.raises(ta.TreeAttnError):
        e.run(0.1, q_indptr=i32(np.zeros(16386)), kv_indptr=i32(np.zeros(16386)))


def test_expanded_long_prompt():
    e = Expanded([12000], [20000], 2, 128, 64, "bf16", seed=17)
    out, lse = e.run(0.07)
    assert ta.device_status(e.ws) == ta.TA_OK
    e.check(out, lse, 0.07)


def test_tree_and_append_of_the_largest_batch():
    """16,384 sequences of 1 to 40 rows, each ending in a tree of one node."""
    rng = np.random.default_rng(18)
    kv = rng.integers(1, 41, 16384)
    n = -(-kv // 16)
    s = Setup([1], 3, 256, 16, seed=18)
    s.kv, s.indptr, s.values = kv, indptr(n), np.arange(n.sum())
    s.last, s.pool = kv - (n - 1) * 16, s.randn(int(n.sum()), 16, s.w)
    s.cache = s.handle()
    one, q = i32(np.arange(16385)), s.randn(16384, 3, s.w)
    x = s.randn(16384, s.w)
    s.cache.append(x[:, :256], x[:, 256:], one)
    pid = torch.from_numpy(s.indptr[1:] - 1).cuda()
    assert torch.equal(s.pool[pid, torch.from_numpy(s.last - 1).cuda()], x)
    out, lse = s.cache.tree_attn(q, one, one, i32([[0, 1]] * 16384), 0.1)
    assert s.cache.device_status() == ta.TA_OK
    check_absorbed(s, q, out, lse, 0.1)


def test_streams_given_by_address():
    s = Setup([300, 40], 16, 512, 64, seed=19)
    q, st = s.randn(2, 16, s.w), torch.cuda.Stream()
    want = s.cache.decode(q, 0.07)
    torch.cuda.synchronize()
    got = s.cache.decode(q, 0.07, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_longest_sequence():
    """2^31 - 16 rows, one page over and over: its 16 rows' attention.  A pair of SMs
    adds its 220,753 tiles one after the other; every addition may lose 2^-23 of the
    sum, one a tile for the sums of the weights, eight (of 16 rows) for the output."""
    n = (1 << 27) - 1
    g = torch.Generator("cuda").manual_seed(30)
    pool = torch.randn((2, 16, 272), generator=g, device="cuda").bfloat16()
    pool[1] = NAN
    values = torch.zeros(n, dtype=torch.int32, device="cuda")
    c = ta.LatentCache(pool, i32([0, n]), values, i32([16]), h_q=1, rank=256)
    q = torch.randn((1, 1, 272), generator=g, device="cuda").bfloat16()
    out, lse = c.decode(q, 0.07, out=torch.full((1, 1, 256), NAN, dtype=torch.bfloat16, device="cuda"))
    assert c.device_status() == ta.TA_OK
    ro, rl, mag, _ = ref.absorbed(q.double(), pool.double(), ([0, 1], [0], [16]), 256, 0.07)
    lost = -(-n // 8 // 76) * 2.0 ** -23
    assert ((out.double() - ro).abs() <= 9 * lost * mag + 2.0 ** -7 * mag).all()
    assert (lse.double() - rl - math.log2(n)).abs().max() <= -math.log2(1 - lost) + 2.0 ** -10


# --------------------------------------------------------------------------
# a wait that runs out
# --------------------------------------------------------------------------

def test_waits_that_run_out_are_reported():
    """The products' warp waits on a barrier that nothing arrives on: every wait
    ends, the status says so, nothing is written, and the next call is as ever."""
    s = Setup([2000, 30], 64, 512, 64, seed=21)
    q = s.randn(2, 64, s.w)
    want = [t.clone() for t in s.cache.decode(q, 0.07)]
    e = Expanded([200, 3], [200, 50], 4, 128, 64, "bf16", seed=22)
    ewant = [t.clone() for t in e.run(0.07)]
    torch.cuda.synchronize()
    out, lse = torch.full_like(want[0], 5), torch.full_like(want[1], 5)
    eout, else_ = torch.full_like(e.out, 5), torch.full_like(e.lse, 5)
    ta.set_wait_hooks(20_000_000, True)
    try:
        s.cache.decode(q, 0.07, out=out, lse=lse)
        assert s.cache.device_status() == ta.TA_ERR_DEVICE_TIMEOUT
        e.run(0.07, out=eout, lse=else_)
        assert ta.device_status(e.ws) == ta.TA_ERR_DEVICE_TIMEOUT
    finally:
        ta.set_wait_hooks(0, False)
    assert (out == 5).all() and (lse == 5).all() and (eout == 5).all() and (else_ == 5).all()
    for _ in range(2):
        got, egot = s.cache.decode(q, 0.07), e.run(0.07)
        assert s.cache.device_status() == ta.TA_OK and ta.device_status(e.ws) == ta.TA_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(egot[0], ewant[0]) and torch.equal(egot[1], ewant[1])


def test_parts_of_an_earlier_call_are_not_joined():
    """One pair of SMs gives up: a sequence with a part of its is left as it was,
    not joined from the part that the call before left in the workspace; the
    others' results are those of any call."""
    # one tile of 128 rows for almost every pair, in order: pair 20 works on the
    # first sequence, pair 60 on the second
    s = Setup([4500, 4500], 16, 512, 64, seed=23)
    q, before = s.randn(2, 16, s.w), s.randn(2, 16, s.w)
    want = [t.clone() for t in s.cache.decode(q, 0.07)]
    for pair, left in ((60, 1), (20, 0)):
        s.cache.decode(before, 0.07)
        out, lse = torch.full_like(want[0], 5), torch.full_like(want[1], 5)
        ta.set_wait_hooks(20_000_000, -1 - pair)
        try:
            s.cache.decode(q, 0.07, out=out, lse=lse)
            assert s.cache.device_status() == ta.TA_ERR_DEVICE_TIMEOUT
        finally:
            ta.set_wait_hooks(0, False)
        assert (out[left] == 5).all() and (lse[left] == 5).all()
        assert torch.equal(out[1 - left], want[0][1 - left]) and torch.equal(lse[1 - left], want[1][1 - left])
        got = s.cache.decode(q, 0.07)
        assert s.cache.device_status() == ta.TA_OK
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_waits_are_limited_from_the_last_progress():
    """Some warps wait for a whole unit of work: with a limit far below what one
    takes, but far above what one of its tiles takes, nothing runs out."""
    e = Expanded([1, 3], [200001, 150003], 1, 64, 16, "bf16", seed=40)
    want = [t.clone() for t in e.run(0.1)]
    # 12 or 13 items of 128 packed rows for a pair of SMs, 400 tiles of kv rows each
    trees = Trees([(51000, 64, 64, "star")] * 30, 64, 256, 16, "bf16", seed=41)
    twant = [t.clone() for t in trees.run(0.1)]
    assert milliseconds(lambda: e.run(0.1), 1) > 2 and milliseconds(lambda: trees.run(0.1), 1) > 2
    ta.set_wait_hooks(150_000, False)
    try:
        out, lse = e.run(0.1, out=torch.zeros_like(want[0]), lse=torch.zeros_like(want[1]))
        assert ta.device_status(e.ws) == ta.TA_OK
        tout, tlse = trees.run(0.1)
        assert trees.s.cache.device_status() == ta.TA_OK
    finally:
        ta.set_wait_hooks(0, False)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(tout, twant[0]) and torch.equal(tlse, twant[1])
