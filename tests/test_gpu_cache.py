"""GPU tests of the paged-cache calls (``PagedCache``) against the 64-bit
references.

Tolerances.  A value rounded to a 16-bit type is off by at most half a step,
``eps / 2`` of it.  decode: the output is rounded once; a weight passes as its
rounding and the rounding of the rest, which leaves ``(eps / 2)^2`` of it, and
the weighted sums add up to a few dozen float32 terms one after the other
(2^-23 each, truncated), 2^-18 of ``sum w |v|`` together.  A score is a float32 sum of d products: it is off by at most
``(d + 4) * 2^-23`` (truncating adds) of the sum of its products' sizes, S, in
base-2 units; a weight is then off by that times ln 2, relative, twice (in the
weight and in the sum), and the lse by it once, plus the float32 rounding of
the exponentials, the sum and the logarithm (2^-20, and 2^-22 of the lse).
append: a rotated element is a sum of two products of float32 factors, each
good to a few 2^-24 (norm: a sum of d squares, a square root, three products),
2^-19 of the pair's length in all.  compact and copies move bits.
"""
import numpy as np
import pytest
import torch

import tree_attention_gb300 as ta
import workloads as wl
from oracle import paged_cache_ref as ref

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from tree_attention_gb300 import build
    build.build()
    ta.lib()


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


class Setup:
    """A pool with a scattered table for kv lengths ``kv``; slots nobody owns
    hold NaN.  The table's arrays have spare capacity at the end."""

    def __init__(self, kv, h_q, h_kv, d, dtype="bf16", seed=0, spare=3, fill=float("nan")):
        rng = np.random.default_rng(seed)
        self.kv = np.asarray(kv, dtype=np.int64)
        n = -(-self.kv // 16)
        self.indptr = np.concatenate([[0], np.cumsum(n)])
        nnz = int(n.sum())
        self.values = np.concatenate([rng.permutation(nnz + spare)[:nnz], [-7] * 2]).astype(int)
        self.last = np.where(n > 0, self.kv - (n - 1) * 16, 0)
        g = torch.Generator().manual_seed(seed)
        pool = torch.full((nnz + spare, 2, h_kv, 16, d), fill)
        for b in range(len(kv)):
            pid, sl = ref.slots(self.indptr, self.values, self.last, b)
            pool[pid, :, :, sl] = torch.randn((len(pid), 2, h_kv, d), generator=g)
        self.dtype = DT[dtype]
        self.pool = pool.to(self.dtype).cuda()
        self.h_q, self.h_kv, self.d, self.g = h_q, h_kv, d, g
        self.cache = self.handle()

    def handle(self, **kw):
        a = {"page_indptr": self.indptr, "page_values": self.values, "length_info": self.last}
        a.update(kw)
        return ta.PagedCache(self.pool, *[i32(a[k]) for k in a], h_q=self.h_q)

    def randn(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype).cuda()

    @property
    def table(self):
        return self.indptr, self.values, self.last


def check_decode(s, q, out, lse, sm_scale):
    # a reference over the slots that belong to a sequence; NaN elsewhere would show
    ro, rl, mag, smag = ref.decode(f64(q), f64(s.pool), *s.table, sm_scale)
    out, lse = f64(out), f64(lse)
    half = torch.finfo(s.dtype).eps / 2
    serr = (s.d + 4) * 2.0 ** -23 * smag
    tol = half * np.abs(ro) + (half ** 2 + 2.0 ** -18) * mag + 2 * serr[..., None] * mag \
        + torch.finfo(s.dtype).smallest_normal * half * 2
    assert np.isfinite(out).all()
    bad = np.abs(out - ro) > tol
    assert not bad.any(), (np.abs(out - ro) / np.maximum(tol, 1e-30)).max()
    fin = np.isfinite(rl)
    assert np.array_equal(fin, np.isfinite(lse)) and (lse[~fin] == -np.inf).all()
    lse, rl, serr = lse[fin], rl[fin], serr[fin]
    assert (np.abs(lse - rl) <= serr + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl)).all()


DECODE = {
    # kv lengths, h_q, h_kv, d, dtype
    "one_token": ([1], 8, 2, 128, "bf16"),
    "page_edges": ([1, 15, 16, 17, 31, 32, 33], 8, 2, 128, "fp16"),
    "empty_rows": ([0, 5, 0, 0, 40, 0], 4, 4, 64, "bf16"),
    "all_empty": ([0, 0, 0], 4, 2, 128, "bf16"),
    "group_1": ([200, 3], 4, 4, 128, "bf16"),
    "group_3": ([77, 130], 6, 2, 64, "fp16"),
    "group_4": ([1000, 19, 250], 32, 8, 128, "bf16"),
    "group_8": ([333, 64], 16, 2, 128, "fp16"),
    "group_9": ([100, 47], 18, 2, 128, "bf16"),
    "group_16": ([300, 31], 16, 1, 64, "bf16"),
    "group_20": ([150, 2], 20, 1, 128, "fp16"),
    "group_128": ([90, 18], 128, 1, 128, "bf16"),
    "group_12_long": ([7000, 33, 2500], 24, 2, 64, "fp16"),
    "group_40_long": ([4000, 1, 900], 40, 1, 128, "bf16"),
    "group_128_long": ([3500], 128, 1, 64, "bf16"),
    "many_kv_heads": ([260, 0, 31], 80, 80, 64, "bf16"),
    "one_long": ([9000], 4, 1, 128, "bf16"),
    "ragged": ([int(x) for x in np.random.default_rng(4).integers(0, 700, 40)], 8, 2, 64, "bf16"),
    "many_short": ([1 + i % 37 for i in range(300)], 4, 2, 128, "fp16"),
    "long_and_short": ([6000, 1, 2, 3, 17, 0, 900], 10, 2, 128, "fp16"),
}


@pytest.mark.parametrize("name", list(DECODE))
def test_decode(name):
    kv, h_q, h_kv, d, dtype = DECODE[name]
    s = Setup(kv, h_q, h_kv, d, dtype, seed=len(kv))
    q = s.randn(len(kv), h_q, d)
    for sm in (d ** -0.5, 0.6):
        out, lse = s.cache.decode(q, sm)
        assert s.cache.device_status() == ta.TA_OK
        check_decode(s, q, out, lse, sm)


def test_decode_largest_batch():
    """16,384 sequences of 0 to 20 rows."""
    rng = np.random.default_rng(9)
    s = Setup(rng.integers(0, 21, 16384), 2, 1, 64, "bf16", seed=10)
    q = s.randn(16384, 2, 64)
    out, lse = s.cache.decode(q, 0.125)
    assert s.cache.device_status() == ta.TA_OK
    check_decode(s, q, out, lse, 0.125)
    with pytest.raises(ta.TreeAttnError):
        ta.PagedCache(s.pool, i32(np.zeros(16386)), i32([0]), i32(np.zeros(16385)), h_q=2)


def test_decode_many_pages_per_warp():
    """A range of 70 pages per warp: page indices are fetched 32 at a time.  The
    reference is torch in float64 on the GPU; a weighted sum adds up to 70 pages
    one after the other, 2^-23 each."""
    n, h = 170_000, 16
    s = Setup([1], h, h, 64, "bf16", seed=15)
    pages = -(-n // 16)
    g = torch.Generator("cuda").manual_seed(3)
    pool = torch.randn((pages + 4, 2, h, 16, 64), generator=g, device="cuda", dtype=s.dtype)
    perm = torch.randperm(pages + 4, generator=g, device="cuda")[:pages]
    c = ta.PagedCache(pool, i32([0, pages]), perm.int(), i32([n - (pages - 1) * 16]), h_q=h)
    q = s.randn(1, h, 64)
    out, lse = c.decode(q, 0.125)
    assert c.device_status() == ta.TA_OK
    kv = pool[perm].permute(1, 2, 0, 3, 4).reshape(2, h, -1, 64)[:, :, :n]
    for i in range(h):
        k, v, x = kv[0, i].double(), kv[1, i].double(), q[0, i].double()
        sc = (k * x).sum(1) * 0.125
        w = torch.softmax(sc, 0)[:, None]
        want, mag = (w * v).sum(0), (w * v.abs()).sum(0)
        serr = 68 * 2.0 ** -23 * ((k * x).abs().sum(1).max() * 0.125 / np.log(2))
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -16 + 80 * 2.0 ** -23 + 2 * serr) * mag
        assert ((out[0, i].double() - want).abs() <= tol).all()
        rl = torch.logsumexp(sc, 0) / np.log(2)
        assert (lse[0, i].double() - rl).abs() <= serr + 2.0 ** -20 + 2.0 ** -22 * rl.abs()


def test_decode_without_any_page():
    pool = torch.full((2, 2, 2, 16, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    c = ta.PagedCache(pool, i32([0, 0, 0]), i32([]), i32([0, 0]), h_q=4)
    q = torch.ones((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = c.decode(q, 0.1)
    assert c.device_status() == ta.TA_OK
    assert (out == 0).all() and (lse == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_decode_scores_that_rise_and_fall(dtype):
    """The running reference has to move on every page, and must not let a
    large early score be forgotten."""
    s = Setup([400, 400], 4, 1, 128, dtype, seed=8)
    pid, sl = ref.slots(*s.table, 0)
    ramp = torch.linspace(-6, 6, 400)
    s.pool[pid, 0, 0, sl] = ramp[:, None].to(s.dtype).expand(400, 128).cuda()
    pid, sl = ref.slots(*s.table, 1)
    s.pool[pid, 0, 0, sl] = ramp.flip(0)[:, None].to(s.dtype).expand(400, 128).cuda()
    q = torch.ones((2, 4, 128), dtype=s.dtype, device="cuda")
    q[:, 1] *= -1
    q[:, 2] *= 0.01
    out, lse = s.cache.decode(q, 0.25)
    check_decode(s, q, out, lse, 0.25)


def test_decode_many_equal_small_weights():
    """One large score and 20,000 far smaller ones that still hold a tenth of
    the sum: weights below the 16-bit type's normal range must count."""
    n = 20000
    s = Setup([n], 1, 1, 64, "fp16", seed=2)
    pid, sl = ref.slots(*s.table, 0)
    k = torch.zeros(n, 64)
    k[0, 0] = 12.0
    s.pool[pid, 0, 0, sl] = k.half().cuda()
    q = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    q[0, 0, 0] = 1.0
    out, lse = s.cache.decode(q, 1.0)
    check_decode(s, q, out, lse, 1.0)


@pytest.mark.parametrize("ramp", [False, True])
@pytest.mark.parametrize("h_q,h_kv,d,dtype", [(8, 2, 128, "bf16"), (8, 2, 64, "fp16"),
                                              (32, 2, 128, "fp16"), (40, 1, 64, "bf16")])
def test_decode_values_that_are_not_finite(h_q, h_kv, d, dtype, ramp):
    """Weights are positive: an element whose column of values has an infinity
    is that infinity, NaN with a NaN or infinities of both signs, for every
    head; all others, and the lse, are those of the values without them.  With
    ramp, scores rise or fall by 550 powers of two along a sequence."""
    kv = [40, 3, 5000, 700, 2600]
    s = Setup(kv, h_q, h_kv, d, dtype, seed=18)
    if ramp:
        for b in (0, 2, 3, 4):
            pid, sl = ref.slots(*s.table, b)
            r = torch.linspace(-6, 6, kv[b]) * (128 / d) * (-1 if b in (2, 3) else 1)
            s.pool[pid, 0, :, sl] = r[:, None, None].to(s.dtype).expand(kv[b], h_kv, d).cuda()
    q = s.randn(len(kv), h_q, d) if not ramp else torch.ones((len(kv), h_q, d), dtype=s.dtype,
                                                             device="cuda")
    sm = 0.25 if ramp else d ** -0.5
    clean = s.pool.clone()
    inf, nan = float("inf"), float("nan")
    want = {}
    # sequence, row, kv head, element, value
    for b, r, h, e, x in [(0, 0, 0, 5, inf), (0, 39, 0, 6, -inf), (0, 17, h_kv - 1, d - 1, nan),
                          (0, 2, 0, 9, inf), (0, 36, 0, 9, -inf),
                          (1, 2, 0, 0, -inf), (1, 1, 0, 1, inf), (1, 0, 0, 1, inf),
                          (2, 0, 0, 3, inf), (2, 4999, 0, 4, -inf), (2, 2500, 0, 63, inf),
                          (2, 10, h_kv - 1, 40, inf), (2, 4000, h_kv - 1, 40, nan),
                          (3, 699, 0, 8, inf), (3, 0, 0, 11, -inf), (4, 1300, 0, 20, -inf),
                          (4, 0, 0, 21, inf), (4, 2599, 0, 22, inf)]:
        pid, sl = ref.slots(*s.table, b)
        s.pool[pid[r], 1, h, sl[r], e] = x
        clean[pid[r], 1, h, sl[r], e] = 0
        want[b, h, e] = x if want.get((b, h, e), x) == x else nan
    out, lse = s.cache.decode(q, sm)
    dirty, s.pool = s.pool, clean
    s.cache = s.handle()
    base, base_lse = s.cache.decode(q, sm)
    check_decode(s, q, base, base_lse, sm)
    assert torch.equal(lse, base_lse)
    g, expect = h_q // h_kv, base.clone()
    for (b, h, e), x in want.items():
        expect[b, h * g:(h + 1) * g, e] = x
    assert torch.equal(torch.isnan(out), torch.isnan(expect))
    assert torch.equal(out.nan_to_num(7, inf, -inf), expect.nan_to_num(7, inf, -inf))


@pytest.mark.parametrize("h_q,h_kv,d,dtype", [(8, 2, 128, "bf16"), (36, 2, 64, "fp16")])
def test_decode_scores_that_are_not_finite(h_q, h_kv, d, dtype):
    """NaN queries and keys reach their heads and kv heads only; a row whose
    score is -inf counts as if it were not there."""
    kv = [40, 2000, 17, 600]
    s = Setup(kv, h_q, h_kv, d, dtype, seed=20, fill=0.0)
    q = s.randn(len(kv), h_q, d)
    q[3] = q[3].abs()
    base = [t.clone() for t in s.cache.decode(q, d ** -0.5)]
    g, nan = h_q // h_kv, torch.zeros((len(kv), h_q), dtype=torch.bool)
    bad_q = q.clone()
    bad_q[1, 3, 7] = float("nan")
    nan[1, 3] = True
    for b, r, h in ((0, 39, 1), (1, 999, 1)):
        pid, sl = ref.slots(*s.table, b)
        s.pool[pid[r], 0, h, sl[r], 5] = float("nan")
        nan[b, h * g:(h + 1) * g] = True
    # the last 100 rows of sequence 3, kv head 0; the same sequence without them
    pid, sl = ref.slots(*s.table, 3)
    cut = Setup([500], h_q, h_kv, d, dtype, seed=21, fill=0.0)
    to, tl = ref.slots(*cut.table, 0)
    cut.pool[to, :, :, tl] = s.pool[pid[:500], :, :, sl[:500]]
    s.pool[pid[500:], 0, 0, sl[500:], 3] = -float("inf")
    out, lse = s.cache.decode(bad_q, d ** -0.5)
    nan = nan.cuda()
    assert torch.equal(torch.isnan(lse), nan) and torch.equal(torch.isnan(out).all(-1), nan)
    same = ~nan
    same[3, :g] = False
    assert torch.equal(out[same], base[0][same]) and torch.equal(lse[same], base[1][same])
    ro, rl, mag, smag = ref.decode(f64(q[3:]), f64(cut.pool), *cut.table, d ** -0.5)
    half = torch.finfo(s.dtype).eps / 2
    serr = (d + 4) * 2.0 ** -23 * smag
    tol = half * np.abs(ro) + (half ** 2 + 2.0 ** -18 + 2 * serr[..., None]) * mag \
        + torch.finfo(s.dtype).smallest_normal * half * 2
    assert (np.abs(f64(out[3:]) - ro) <= tol)[:, :g].all()
    assert (np.abs(f64(lse[3:]) - rl) <= serr + 2.0 ** -20 + 2.0 ** -22 * np.abs(rl))[:, :g].all()


def test_decode_page_outside_the_pool_reads_zeros():
    s = Setup([50, 20], 4, 2, 128, seed=3)
    s.values[1], s.values[4] = 10 ** 6, -1
    s.cache = s.handle()
    q = s.randn(2, 4, 128)
    out, lse = s.cache.decode(q, 0.1)
    check_decode(s, q, out, lse, 0.1)
    assert s.cache.device_status() == ta.TA_OK


def test_decode_is_repeatable_and_leaves_its_workspace_ready():
    s = Setup([5000, 30, 0, 700], 8, 2, 128, seed=5)
    q = s.randn(4, 8, 128)
    a = [t.clone() for t in s.cache.decode(q, 0.1)]
    ws = s.cache.workspace.clone()
    for _ in range(5):
        b = s.cache.decode(q, 0.1)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert s.cache.workspace[:256].eq(ws[:256]).all()


@pytest.mark.parametrize("kv,h_q,h_kv,d", [([32768], 32, 8, 128), ([16384, 16384], 32, 8, 128),
                                           ([9000], 8, 2, 128), ([20000, 9000], 8, 4, 64)])
def test_decode_does_not_depend_on_which_cta_ends_last(kv, h_q, h_kv, d):
    """Sequences over dozens of CTAs, whose borders with the next sequence or kv
    head lie within a CTA: it may be the last of one of its two or of both."""
    s = Setup(kv, h_q, h_kv, d, seed=17, fill=0.0)
    q = s.randn(len(kv), h_q, d)
    out, lse = [t.clone() for t in s.cache.decode(q, d ** -0.5)]
    differ = 0
    for _ in range(300):
        a, b = s.cache.decode(q, d ** -0.5)
        differ += (a != out).any().long() + (b != lse).any().long()
    assert int(differ) == 0
    check_decode(s, q, out, lse, d ** -0.5)


def test_decode_follows_a_changed_table():
    """One handle, lengths that change in place between calls (a decoding loop),
    also under a captured graph."""
    s = Setup([160, 160, 160], 8, 2, 64, "fp16", seed=6)
    q = s.randn(3, 8, 64)
    out, lse = s.cache.decode(q, 0.125)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.cache.decode(q, 0.125, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.cache.decode(q, 0.125, out=out, lse=lse)
    for lens in ([16, 1, 9], [3, 16, 16]):
        s.last = np.asarray(lens)
        s.cache.length_info.copy_(i32(s.last))
        out.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        check_decode(s, q, out, lse, 0.125)


BAD_TABLES = {
    "falling_indptr": dict(page_indptr=[0, 5, 3, 7]),
    "indptr_start": dict(page_indptr=[1, 3, 4, 7]),
    "past_capacity": dict(page_indptr=[0, 3, 4, 99]),
    "negative": dict(page_indptr=[0, -3, 4, 7]),
    "length_0": dict(length_info=[2, 0, 4]),
    "length_17": dict(length_info=[2, 16, 17]),
}


@pytest.mark.parametrize("name", list(BAD_TABLES))
def test_decode_reports_bad_tables(name):
    s = Setup([34, 16, 36], 8, 2, 128, seed=7)
    c = s.handle(**BAD_TABLES[name])
    q = s.randn(3, 8, 128)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    c.decode(q, 0.1, out=out, lse=lse)
    assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    assert (out == 7).all() and (lse == 7).all()
    assert c.device_status() == ta.TA_OK                    # cleared
    good = ta.PagedCache(s.pool, *[i32(x) for x in s.table], h_q=8, workspace=c.workspace)
    check_decode(s, q, *good.decode(q, 0.1), 0.1)


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

APPEND = {
    # held rows, new rows, h_q, h_kv, d, dtype, norm (q, k), layout, rotary_dim, theta, fused
    "one": ([0], [1], 8, 2, 128, "bf16", (True, True), "half", 128, 1e4, True),
    "page_edges": ([0, 15, 16, 17, 3], [16, 1, 17, 0, 30], 4, 2, 64, "fp16", (True, True), "half",
                   64, 5e5, True),
    "interleaved": ([7, 100], [33, 2], 6, 3, 128, "bf16", (False, False), "interleaved", 128, 1e4,
                    True),
    "part_half": ([5, 0, 0], [9, 0, 40], 4, 4, 128, "bf16", (True, False), "half", 48, 1e4, False),
    "part_interleaved": ([5], [50], 5, 1, 64, "fp16", (False, True), "interleaved", 16, 1e4, True),
    "no_rotation": ([2, 30], [20, 3], 16, 2, 128, "fp16", (True, True), None, 128, 1e4, True),
    "copy_only": ([2, 30], [20, 3], 3, 1, 64, "bf16", (False, False), None, 64, 1e4, False),
    "many": ([3 + i for i in range(70)], [i % 5 for i in range(70)], 8, 1, 128, "bf16",
             (True, True), "half", 128, 1e4, True),
}


def append_inputs(s, new, fused):
    n = int(np.sum(new))
    if fused:
        x = s.randn(n, s.h_q + 2 * s.h_kv, s.d)
        return x[:, :s.h_q], x[:, s.h_q:s.h_q + s.h_kv], x[:, s.h_q + s.h_kv:]
    return s.randn(n, s.h_q, s.d), s.randn(n, s.h_kv, s.d), s.randn(n, s.h_kv, s.d)


def append_reference(s, q, k, pos, layout, rd, theta, scale, qw, kw, eps, magnitude=1.0):
    """Rounded-once values and what one of them may be off by."""
    freq = scale * theta ** (-2.0 * np.arange(rd // 2) / rd)
    half, got = torch.finfo(s.dtype).eps / 2, []
    for x, w in ((q, qw), (k, kw)):
        x = ref.norm(f64(x), None if w is None else f64(w), eps)
        y = ref.rotate(x, pos, layout, rd, freq, magnitude)
        # the length of each element's pair (itself, where it is not rotated)
        size = np.abs(x)
        if layout is not None:
            lo = slice(0, rd // 2) if layout == "half" else slice(0, rd, 2)
            hi = slice(rd // 2, rd) if layout == "half" else slice(1, rd, 2)
            size[..., lo] = size[..., hi] = abs(magnitude) * np.hypot(x[..., lo], x[..., hi])
        tol = half * np.abs(y) * (1 + 2.0 ** -10) + 2.0 ** -19 * size \
            + torch.finfo(s.dtype).smallest_normal * half
        got.append((y, tol))
    return got


@pytest.mark.parametrize("far", [0, 1_000_000, 2 ** 31 - 200])
@pytest.mark.parametrize("name", list(APPEND))
def test_append(name, far):
    held, new, h_q, h_kv, d, dtype, (nq, nk), layout, rd, theta, fused = APPEND[name]
    s = Setup(np.add(held, new), h_q, h_kv, d, dtype, seed=11)
    q, k, v = append_inputs(s, new, fused)
    ai = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([far + np.arange(h, h + n) for h, n in zip(held, new)])
    qw = (1 + 0.2 * s.randn(d)) if nq else None
    kw = (1 + 0.2 * s.randn(d)) if nk else None
    before = s.pool.clone()
    rope = None if layout is None else ta.Rope(layout, rd, theta=theta, scale=0.5)
    qo = s.cache.append(q, k, v, i32(ai), i32(pos), rope=rope, q_weight=qw, k_weight=kw,
                        norm_eps=1e-5)
    assert s.cache.device_status() == ta.TA_OK
    (yq, tq), (yk, tk) = append_reference(s, q, k, pos, layout, rd, theta, 0.5, qw, kw, 1e-5)
    assert (np.abs(f64(qo) - yq) <= tq).all()
    want = ref.append(f64(before), yk, f64(v), ai, *s.table)
    tol = ref.append(np.zeros(before.shape), tk, 0 * f64(v), ai, *s.table)
    got = f64(s.pool)
    same = np.isnan(want) & np.isnan(got)
    assert (same | (np.abs(got - want) <= tol)).all()        # zero tolerance off the new keys


def test_append_many_tokens_per_warp():
    """120,000 tokens of single heads: 40 tokens per warp, looked up 32 at a time."""
    new = [60001, 1, 0, 47, 59951]
    s = Setup(np.add(new, [3, 0, 7, 30, 0]), 1, 1, 64, "fp16", seed=16, fill=0.0)
    q, k, v = append_inputs(s, new, True)
    ai = np.concatenate([[0], np.cumsum(new)])
    pos = np.concatenate([np.arange(n) for n in new])
    before = s.pool.clone()
    qo = s.cache.append(q, k, v, i32(ai), i32(pos), rope=ta.Rope("half", 64))
    assert s.cache.device_status() == ta.TA_OK
    (yq, tq), (yk, tk) = append_reference(s, q, k, pos, "half", 64, 1e4, 1.0, None, None, 0.0)
    assert (np.abs(f64(qo) - yq) <= tq).all()
    want = ref.append(f64(before), yk, f64(v), ai, *s.table)
    tol = ref.append(np.zeros(before.shape), tk, 0 * f64(v), ai, *s.table)
    assert (np.abs(f64(s.pool) - want) <= tol).all()


def test_append_warps_over_several_sequences():
    """Single heads, three steps per token: a warp's dozen steps begin in the
    middle of a token and go over five, of as many sequences."""
    rng = np.random.default_rng(19)
    new = rng.integers(0, 6, 16000)
    s = Setup(new + rng.integers(0, 20, 16000), 1, 1, 64, "bf16", seed=19, fill=0.0)
    q, k, v = append_inputs(s, new, True)
    assert len(q) * 3 > 12 * 4 * 5 * torch.cuda.get_device_properties(0).multi_processor_count
    ai = np.concatenate([[0], np.cumsum(new)])
    pos = rng.integers(-2 ** 31, 2 ** 31, len(q))
    before = s.pool.clone()
    qo = s.cache.append(q, k, v, i32(ai), i32(pos), rope=ta.Rope("interleaved", 32))
    assert s.cache.device_status() == ta.TA_OK
    (yq, tq), (yk, tk) = append_reference(s, q, k, pos, "interleaved", 32, 1e4, 1.0, None, None, 0.0)
    assert (np.abs(f64(qo) - yq) <= tq).all()
    want = ref.append(f64(before), yk, f64(v), ai, *s.table)
    tol = ref.append(np.zeros(before.shape), tk, 0 * f64(v), ai, *s.table)
    assert (np.abs(f64(s.pool) - want) <= tol).all()


def test_append_in_place_and_magnitude_and_frequencies():
    """q_out may be q; a table of frequencies and a factor of cos and sin."""
    s = Setup([40], 4, 2, 64, "bf16", seed=12)
    q, k, v = append_inputs(s, [40], False)
    freq = [0.3 ** i for i in range(16)]
    rope = ta.Rope("half", 32, inv_freq=freq, scale=2.0, magnitude=1.25)
    pos = np.arange(-20, 20)
    other = s.cache.append(q, k, v, i32([0, 40]), i32(pos), rope=rope)
    x = f64(q)
    y = ref.rotate(x, pos, "half", 32, 2.0 * np.asarray(freq), 1.25)
    size = 1.25 * np.hypot(x[..., :16], x[..., 16:32])
    tol = 2.0 ** -8 * np.abs(y) * (1 + 2.0 ** -10)
    tol[..., :32] += 2.0 ** -19 * np.concatenate([size, size], -1)
    assert (np.abs(f64(other) - y) <= tol).all()
    res = s.cache.append(q, k, v, i32([0, 40]), i32(pos), rope=rope, q_out=q)
    assert res is q and torch.equal(q, other)


def test_append_of_zero_rows_and_of_zero_inputs():
    s = Setup([20, 0], 4, 2, 64, "bf16", seed=13)
    q, k, v = (torch.zeros((0, h, 64), dtype=s.dtype, device="cuda") for h in (4, 2, 2))
    before = s.pool.clone()
    s.cache.append(q, k, v, i32([0, 0, 0]))
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int16), s.pool.view(torch.int16))
    q, k, v = (torch.zeros((2, h, 64), dtype=s.dtype, device="cuda") for h in (4, 2, 2))
    w = torch.ones(64, dtype=s.dtype, device="cuda")
    out = s.cache.append(q, k, v, i32([0, 2, 2]), i32([5, 6]), rope=ta.Rope("half", 64),
                         q_weight=w, k_weight=w, norm_eps=1e-6)
    assert (out == 0).all() and s.cache.device_status() == ta.TA_OK


@pytest.mark.parametrize("kw,written", [
    # sequence 0: 20 rows in two pages, its new ones 17, 18, 19; sequence 1: 2 rows, both new
    (dict(append_indptr=[0, 3, 6]), [0]),              # more new tokens than rows
    (dict(page_values=[0, 99, 1, -1, 2]), [1]),        # sequence 0's second page: outside
    (dict(page_values=[0, 3, -1, -1, 2]), [0]),
    (dict(page_indptr=[0, 2, 1]), [0]),
    (dict(page_indptr=[0, 2, 99]), [0]),
    (dict(length_info=[4, 0]), [0]),
    (dict(length_info=[4, 17]), [0]),
    (dict(append_indptr=[0, 3, 3]), [0]),              # ends before the last token
])
def test_append_reports_bad_tables(kw, written):
    """The sound sequence is written; nothing of the other one is."""
    kw = dict(kw)
    ai = kw.pop("append_indptr", [0, 3, 5])
    s = Setup([20, 2], 4, 2, 64, "bf16", seed=14, fill=0.0)
    q, k, v = append_inputs(s, [max(5, ai[-1])], True)
    c = s.handle(**kw)
    want = s.pool.clone()
    values = kw.get("page_values", s.values)
    for t, (b, page, slot) in enumerate([(0, values[1], r) for r in (1, 2, 3)]
                                        + [(1, values[2], r) for r in (0, 1)]):
        if b in written:
            want[page, 0, :, slot], want[page, 1, :, slot] = k[t], v[t]
    c.append(q, k, v, i32(ai))
    assert c.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    assert (want == s.pool).all().item()


# --------------------------------------------------------------------------
# compact
# --------------------------------------------------------------------------

def run_compact(s, nodes, paths):
    mn = np.concatenate([[0], np.cumsum(nodes)])
    ai = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
    an = np.concatenate([np.asarray(p, dtype=int) for p in paths])
    before = s.pool.clone()
    new = s.cache.compact(i32(mn), i32(ai), i32(an))
    st = s.cache.device_status()
    return before, new, ref.compact(f64(before), *s.table, mn, ai, an), st


COMPACT = {
    "nothing_moves": ([20, 33], [4, 33], [[0, 1, 2], list(range(33))]),
    "paths": ([70, 40, 64], [64, 30, 17], [[0, 3, 9, 40, 63], [29], [0, 1, 15, 16]]),
    "nothing_kept": ([20, 0, 16, 5], [20, 0, 16, 0], [[], [], [], []]),
    "shift_by_one": ([400], [400], [list(range(1, 400))]),
    "long_paths": ([900, 700], [880, 700], [list(range(0, 880, 2)), list(range(100, 700))]),
    "one_node": ([1, 17], [1, 1], [[0], []]),
    "many": ([30 + i % 40 for i in range(90)], [1 + i % 30 for i in range(90)],
             [sorted({0, i % (1 + i % 30)}) for i in range(90)]),
}


@pytest.mark.parametrize("heads", [(4, 2, 64, "fp16"), (16, 16, 128, "bf16"), (3, 3, 128, "bf16")])
@pytest.mark.parametrize("name", list(COMPACT))
def test_compact(name, heads):
    kv, nodes, paths = COMPACT[name]
    s = Setup(kv, *heads, seed=21)
    _, (ni, nv, nl, fr, nf), (pool, ri, rv, rl, rf), st = run_compact(s, nodes, paths)
    assert st == ta.TA_OK
    np.testing.assert_array_equal(f64(s.pool), pool)         # NaN slots stay NaN
    assert ni.tolist() == ri and nl.tolist() == rl
    assert nv[:ri[-1]].tolist() == rv
    assert int(nf) == len(rf) and fr[:len(rf)].tolist() == rf


def test_compact_largest_batch():
    """16,384 sequences of 0 to 20 rows; trees and paths of any size."""
    rng = np.random.default_rng(25)
    kv = rng.integers(0, 21, 16384)
    nodes = [int(rng.integers(0, n + 1)) for n in kv]
    paths = [sorted(rng.permutation(n)[:rng.integers(0, n + 1)]) for n in nodes]
    s = Setup(kv, 1, 1, 64, seed=26)
    _, (ni, nv, nl, fr, nf), (pool, ri, rv, rl, rf), st = run_compact(s, nodes, paths)
    assert st == ta.TA_OK
    np.testing.assert_array_equal(f64(s.pool), pool)
    assert ni.tolist() == ri and nl.tolist() == rl
    assert nv[:ri[-1]].tolist() == rv
    assert int(nf) == len(rf) and fr[:len(rf)].tolist() == rf


def test_compact_leaves_the_arrays_tails():
    s = Setup([40, 20], 4, 2, 64, seed=22)
    nnz = len(s.values)
    nv = torch.full((nnz,), -9, dtype=torch.int32, device="cuda")
    fr = torch.full((nnz,), -9, dtype=torch.int32, device="cuda")
    s.cache.compact(i32([0, 30, 40]), i32([0, 1, 2]), i32([4, 2]), new_page_values=nv,
                    freed_pages=fr)
    assert (nv[2:] == -9).all() and (fr[3:] == -9).all()
    assert sorted(nv[:2].tolist() + fr[:3].tolist()) == sorted(s.values[:5].tolist())


@pytest.mark.parametrize("mn,ai,an", [
    ([0, 41, 61], [0, 1, 2], [0, 0]),            # more nodes than rows
    ([0, 30, 40], [0, 31, 32], list(range(32))),  # more accepted than nodes
    ([0, 30, 40], [0, 2, 1], [0, 1]),            # falling
    ([0, 30, 40], [0, 1, 1], [0, 1]),            # does not end at the list's length
])
def test_compact_reports_bad_counts_and_writes_nothing(mn, ai, an):
    s = Setup([40, 20], 4, 2, 64, seed=23)
    before = s.pool.clone()
    outs = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (3, len(s.values), 2,
                                                                            len(s.values), 1)]
    s.cache.compact(i32(mn), i32(ai), i32(an), new_page_indptr=outs[0], new_page_values=outs[1],
                    new_length_info=outs[2], freed_pages=outs[3], num_freed=outs[4])
    assert s.cache.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    assert torch.equal(before.view(torch.int16), s.pool.view(torch.int16))
    assert all((t == -9).all() for t in outs)


@pytest.mark.parametrize("path", [[3, 3], [5, 4], [-1, 2], [2, 30]])
def test_compact_keeps_the_rows_of_a_bad_path(path):
    s = Setup([40, 20], 4, 2, 64, seed=24)
    before = s.pool.clone()
    s.cache.compact(i32([0, 30, 40]), i32([0, 2, 3]), i32(path + [7]))
    assert s.cache.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    want = f64(before)
    pid, sl = ref.slots(*s.table, 1)
    want[pid[10], :, :, sl[10]] = want[pid[17], :, :, sl[17]]
    np.testing.assert_array_equal(f64(s.pool), want)


# --------------------------------------------------------------------------
# copies of pages
# --------------------------------------------------------------------------

@pytest.mark.parametrize("n,pages,heads", [(1, 2, (2, 64)), (7, 20, (3, 128)), (300, 700, (1, 64)),
                                           (1500, 3100, (8, 128)), (2040, 4100, (10, 128)),
                                           (5000, 10001, (1, 64))])
def test_copy_pages(n, pages, heads):
    s = Setup([16], heads[0], heads[0], heads[1], seed=31, spare=pages - 1)
    s.pool.copy_(torch.randn(s.pool.shape, device="cuda"))
    p = np.random.default_rng(n).permutation(pages)
    src, dst = p[:n].copy(), p[n:2 * n] if 2 * n <= pages else p[pages - n:]
    src[: n // 3] = src[0]                                   # one page to many
    want = s.pool.clone()
    want[torch.from_numpy(dst).cuda()] = want[torch.from_numpy(src).cuda()]
    s.cache.copy_pages(i32(src), i32(dst))
    assert s.cache.device_status() == ta.TA_OK
    assert torch.equal(s.pool, want)


def test_copy_pages_skips_conflicting_pairs():
    s = Setup([16], 2, 2, 64, seed=32, spare=30)
    s.pool.copy_(torch.randn(s.pool.shape, device="cuda"))
    before = s.pool.clone()
    #      ok   chain: 2 -> 3 -> 4   same destination twice   outside        itself   ok
    src = [0, 2, 3, 5, 6, 40, 9, -1, 12, 14]
    dst = [1, 3, 4, 7, 7, 8, 99, 10, 12, 15]
    s.cache.copy_pages(i32(src), i32(dst))
    assert s.cache.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    want = before.clone()
    for a, b in ((0, 1), (3, 4), (14, 15)):
        want[b] = before[a]
    assert torch.equal(s.pool, want)
    s.cache.copy_pages(i32([12]), i32([12]))
    assert s.cache.device_status() == ta.TA_OK and torch.equal(s.pool, want)


@pytest.mark.parametrize("n", [1900, 5000])
def test_copy_pages_finds_conflicts_anywhere_in_a_long_list(n):
    rng = np.random.default_rng(33)
    pages = 12000
    s = Setup([16], 1, 1, 64, seed=33, spare=pages - 1)
    s.pool.copy_(torch.randn(s.pool.shape, device="cuda"))
    p = rng.permutation(pages)
    src, dst = p[:n].copy(), p[n:2 * n].copy()
    for i, j in rng.integers(0, n, (20, 2)):                # a destination twice
        dst[i] = dst[j]
    for i, j in rng.integers(0, n, (20, 2)):                # a destination that is a source
        dst[i] = src[j]
    uses = {}
    for i in range(n):
        for page in {int(src[i]), int(dst[i])}:
            uses.setdefault(page, set()).add(i)
    good = [i for i in range(n) if src[i] != dst[i] and uses[int(dst[i])] == {i}]
    assert n - 60 <= len(good) < n
    want = s.pool.clone()
    want[torch.from_numpy(dst[good]).cuda()] = s.pool[torch.from_numpy(src[good]).cuda()]
    s.cache.copy_pages(i32(src), i32(dst))
    assert s.cache.device_status() == ta.TA_ERR_INVALID_ARGUMENT
    assert torch.equal(s.pool, want)
    # the next call, on the sound pairs alone, finds nothing of this one
    s.cache.copy_pages(i32(src[good]), i32(dst[good]))
    assert s.cache.device_status() == ta.TA_OK and torch.equal(s.pool, want)


# --------------------------------------------------------------------------
# the handle, and all of them together
# --------------------------------------------------------------------------

def test_offsets_past_32_bits():
    """Pages whose first element lies past 2^32 elements: every call gives there
    what it gives on the same pages of a small pool."""
    h_kv, d, far = 8, 128, 140000                            # 32768 elements per page
    s = Setup([100, 37], 16, h_kv, d, "bf16", seed=71, spare=6, fill=0.0)
    assert far * 2 * h_kv * 16 * d > 2 ** 32
    big = torch.empty((far + s.pool.shape[0], 2, h_kv, 16, d), dtype=s.dtype, device="cuda")
    big[far:] = s.pool
    table = [i32(s.indptr), i32(s.values + far), i32(s.last)]
    c = ta.PagedCache(big, *table, h_q=16)
    rope = ta.Rope("interleaved", 64)
    x = append_inputs(s, [20, 5], True)
    res = []
    for cache, off in ((s.cache, 0), (c, far)):
        q = cache.append(*x, i32([0, 20, 25]), i32(np.arange(25)), rope=rope)
        last = q[[19, 24]].contiguous()
        out, lse = cache.decode(last, 0.09)
        cache.copy_pages(i32(s.values[:2] + off), i32(np.array([p for p in range(14) if p not in
                                                                s.values[:10].tolist()][:2]) + off))
        new = cache.compact(i32([0, 20, 25]), i32([0, 3, 4]), i32([1, 5, 19, 2]))
        assert cache.device_status() == ta.TA_OK
        res.append([q, out, lse, new[0], new[1][:int(new[0][-1])] - off, new[2],
                    new[3][:int(new[4])] - off])
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert torch.equal(big[far:], s.pool)

def test_handle_refusals():
    s = Setup([20, 3], 4, 2, 64, seed=41)
    q = s.randn(2, 4, 64)
    for bad in (q.float(), q[:1], q.cpu(), q.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            s.cache.decode(bad, 0.1)
    k = s.randn(2, 2, 64)
    with pytest.raises(ValueError):
        s.cache.append(q, k, k[:1], i32([0, 1, 2]))
    with pytest.raises(ValueError):
        s.cache.append(q.transpose(1, 2).contiguous().transpose(1, 2), k, k, i32([0, 1, 2]))
    with pytest.raises(ValueError):
        s.cache.append(q, k, k, i32([0, 1, 2]), rope=ta.Rope("half", 64))
    with pytest.raises(ValueError):
        s.cache.copy_pages(i32([0, 1]), i32([2]))
    with pytest.raises(ta.TreeAttnError):
        s.cache.append(q, k, k, i32([0, 1, 2]), i32([0, 1]), rope=ta.Rope("half", 128))
    with pytest.raises(ta.TreeAttnError):
        ta.PagedCache(s.pool, *[i32(x) for x in s.table], h_q=5)


def test_a_workspace_shared_by_caches_of_other_heads():
    """A draft's and a target's cache: head counts, head_dim and pools differ.
    After a decode of either, the other's sequences over several CTAs are merged
    and its copies made."""
    kv = [6000] + [300 + 7 * i for i in range(31)]
    a = Setup(kv, 32, 2, 128, "bf16", seed=72, fill=0.0)
    others = [Setup(kv, 32, 8, 128, "bf16", seed=73, spare=2500, fill=0.0),
              Setup(kv, 8, 2, 64, "fp16", seed=74, spare=300, fill=0.0),
              Setup(kv, 128, 1, 64, "bf16", seed=75, spare=2500, fill=0.0)]
    big = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
    caches = [ta.PagedCache(s.pool, *[i32(x) for x in s.table], h_q=s.h_q, workspace=big)
              for s in [a] + others]
    assert all(c.workspace is big for c in caches)
    for i in (0, 1, 0, 2, 3, 0, 1, 3, 2):
        s, c = ([a] + others)[i], caches[i]
        q = s.randn(len(kv), s.h_q, s.d)
        out = torch.full_like(q, 7.0)
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        c.decode(q, s.d ** -0.5, out=out, lse=lse)
        check_decode(s, q, out, lse, s.d ** -0.5)
        for o, oc in zip(others, caches[1:]):       # enough pairs for marks in the workspace
            free = np.setdiff1d(np.arange(o.pool.shape[0]), o.values)
            src = np.resize(o.values[:-2], 2100)
            if len(free) < 2100:
                continue
            oc.copy_pages(i32(src), i32(free[:2100]))
            assert oc.device_status() == ta.TA_OK
            assert torch.equal(o.pool[free[:2100]], o.pool[src])
        assert c.device_status() == ta.TA_OK


def test_a_workspace_has_to_be_on_the_pools_device():
    s = Setup([20], 4, 2, 64, seed=76)
    with pytest.raises(ValueError, match="workspace"):
        s.cache.with_table(*[i32(x) for x in s.table], workspace=torch.zeros(8 << 20, dtype=torch.uint8))


def test_a_speculative_step_and_a_decoding_step():
    """Prompt, draft trees, their verification, compaction, a fork, one more
    token: the calls as a decoding loop makes them, on one stream without a
    host synchronisation between them, against the references and against the
    contiguous tree attention."""
    h_q, h_kv, d, rng = 8, 2, 128, np.random.default_rng(5)
    prompt, nodes = [37, 16, 90], [20, 33, 8]
    s = Setup(np.add(prompt, nodes), h_q, h_kv, d, "bf16", seed=51, spare=8, fill=0.0)
    s.pool.zero_()
    rope = ta.Rope("half", d, theta=1e4)
    w = (1 + 0.1 * s.randn(d))
    kw = dict(rope=rope, q_weight=w, k_weight=w)

    def table(kv):                    # the same pages, as far as kv rows need them
        n = -(-np.asarray(kv) // 16)
        ind = np.concatenate([[0], np.cumsum(n)])
        val = np.concatenate([s.values[s.indptr[b]:s.indptr[b] + n[b]] for b in range(len(n))])
        return [i32(ind), i32(val), i32(np.asarray(kv) - (n - 1) * 16)]

    # 1. the prompts
    xp = append_inputs(s, prompt, True)
    c0 = s.cache.with_table(*table(prompt))
    c0.append(*xp, i32(np.concatenate([[0], np.cumsum(prompt)])),
              i32(np.concatenate([np.arange(n) for n in prompt])), **kw)
    # 2. the draft trees: appended, then attended
    trees = [wl.random_tree(n, rng) for n in nodes]
    order = i32(np.concatenate([wl.tree_intervals(t) for t in trees]))
    mn = i32(np.concatenate([[0], np.cumsum(nodes)]))
    pos = np.concatenate([p + wl.tree_depths(t) for p, t in zip(prompt, trees)])
    xt = append_inputs(s, nodes, True)
    c1 = s.cache.with_table(*table(np.add(prompt, nodes)))
    qt = c1.append(*xt, mn, i32(pos), **kw)
    out = torch.empty_like(qt)
    lse = torch.empty(qt.shape[:2], dtype=torch.float32, device="cuda")
    dims = ta.make_paged_dims(qt, s.pool, mn, c1.page_values, order)
    ws = torch.zeros(ta.paged_workspace_size(dims), dtype=torch.uint8, device="cuda")
    ta.tree_attn_paged(qt, mn, s.pool, c1.page_indptr, c1.page_values, c1.length_info, mn, order,
                       out, lse, 0, d ** -0.5, ws)
    after_trees = s.pool.clone()
    # 3. the path to the last node is accepted
    paths = [sorted(wl.ancestors(t, len(t) - 1)) for t in trees]
    ai = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
    ni, nv, nl, fr, nf = c1.compact(mn, i32(ai), i32(np.concatenate(paths)))
    # 4. one more token each; its row fits the last page or takes a spare one
    kv = [p + len(a) + 1 for p, a in zip(prompt, paths)]
    c2 = s.cache.with_table(*table(kv))
    xd = append_inputs(s, [1, 1, 1], True)
    qd = c2.append(*xd, i32([0, 1, 2, 3]), i32(np.asarray(kv) - 1), **kw)
    od, ld = c2.decode(qd, d ** -0.5)
    # 5. the first sequence forks: whole pages shared, the last one copied
    t2 = [t.cpu().numpy() for t in table(kv)]
    n0 = int(t2[0][1])
    fresh = [p for p in range(s.pool.shape[0]) if p not in s.values.tolist()][0]
    c2.copy_pages(i32([t2[1][n0 - 1]]), i32([fresh]))
    fork = s.cache.with_table(i32([0, n0]), i32(list(t2[1][:n0 - 1]) + [fresh]), i32(t2[2][:1]))
    of, lf = fork.decode(qd[:1].contiguous(), d ** -0.5)
    for c in (c0, c1, c2, fork):
        assert c.device_status() == ta.TA_OK
    assert ta.device_status(ws) == ta.TA_OK
    assert torch.equal(of, od[:1]) and (lf - ld[:1]).abs().max() < 1e-5
    # the tree attention saw the appended rows: the contiguous call on the same keys agrees
    rows = [ref.slots(*[t.cpu().numpy() for t in (c1.page_indptr, c1.page_values, c1.length_info)],
                      b) for b in range(3)]
    k, v = (torch.cat([after_trees[p, i, :, sl] for p, sl in rows]).contiguous() for i in (0, 1))
    kvi = i32(np.concatenate([[0], np.cumsum(np.add(prompt, nodes))]))
    attn = ta.TreeAttention(qt, k, mn, order, 0, 1.0, 1e4, d ** -0.5)
    oc, lc = attn(qt, mn, k, v, kvi, None, mn, order)
    assert torch.equal(oc, out) and torch.equal(lc, lse)
    # compaction left the accepted rows, then the decoding step saw exactly them and its own
    n_kept = [int(x) for x in ni.tolist()]
    assert nl.tolist() == [(p + len(a) - 1) % 16 + 1 for p, a in zip(prompt, paths)]
    for b in range(3):
        pid, sl = rows[b]
        keep = list(range(prompt[b])) + [prompt[b] + i for i in paths[b]]
        vals = nv[n_kept[b]:n_kept[b + 1]].tolist()
        assert vals == s.values[s.indptr[b]:s.indptr[b] + len(vals)].tolist()
        got = torch.stack([s.pool[vals[r // 16], :, :, r % 16] for r in range(len(keep))])
        assert torch.equal(got, after_trees[pid[keep], :, :, sl[keep]])
    ref_s = s
    ref_s.indptr, ref_s.values, ref_s.last = t2
    check_decode(ref_s, qd, od, ld, d ** -0.5)


def test_two_streams_with_workspaces_of_their_own():
    """The same cache read by two handles at once: each has its own workspace."""
    s = Setup([7000, 3, 900, 0, 2500], 8, 2, 128, seed=62, fill=0.0)
    q = s.randn(5, 8, 128)
    want = [t.clone() for t in s.cache.decode(q, 0.1)]
    other = s.cache.with_table(*[i32(x) for x in s.table], workspace=None)
    assert other.workspace.data_ptr() != s.cache.workspace.data_ptr()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[(torch.empty_like(want[0]), torch.empty_like(want[1])) for _ in range(30)]
            for _ in streams]
    torch.cuda.synchronize()
    for i in range(30):
        for c, st, o in zip((s.cache, other), streams, outs):
            c.decode(q, 0.1, *o[i], stream=st)
    torch.cuda.synchronize()
    for o in outs:
        for out, lse in o:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert s.cache.device_status() == ta.TA_OK and other.device_status() == ta.TA_OK


def test_a_captured_decoding_step_follows_its_inputs():
    """append and decode captured once: tokens, positions and lengths change in
    place between replays, and each replay does what the eager calls do."""
    s = Setup([100, 40, 33], 8, 2, 64, "bf16", seed=63, fill=0.0)
    eager = Setup([100, 40, 33], 8, 2, 64, "bf16", seed=63, fill=0.0)
    x = s.randn(3, 12, 64)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    ai, pos, rope = i32([0, 1, 2, 3]), i32([0, 0, 0]), ta.Rope("half", 64)
    s.cache.length_info.copy_(i32([1, 1, 1]))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        s.cache.decode(s.cache.append(q, k, v, ai, pos, rope=rope), 0.125)
    torch.cuda.synchronize()
    s.pool.copy_(eager.pool)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo = s.cache.append(q, k, v, ai, pos, rope=rope)
        out, lse = s.cache.decode(qo, 0.125)
    for step in range(1, 5):
        lens = i32([3 + step, 7 + step, step])
        x.copy_(s.randn(3, 12, 64))
        pos.copy_(i32([99 + step, 1000 * step, 32 + step]))
        s.cache.length_info.copy_(lens)
        graph.replay()
        eager.cache.length_info.copy_(lens)
        e_qo = eager.cache.append(q, k, v, ai, pos, rope=rope)
        e_out, e_lse = eager.cache.decode(e_qo, 0.125)
        torch.cuda.synchronize()
        assert torch.equal(qo, e_qo) and torch.equal(out, e_out) and torch.equal(lse, e_lse)
        assert torch.equal(s.pool, eager.pool)
    assert s.cache.device_status() == ta.TA_OK


def test_calls_on_a_side_stream():
    """Work queued on another stream than torch's current one keeps its order."""
    s = Setup([500, 60], 8, 2, 128, seed=61, fill=0.0)
    side = torch.cuda.Stream()
    q, k, v = append_inputs(s, [1, 1], True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    s.cache.append(q, k, v, i32([0, 1, 2]), stream=side)
    torch.cuda.synchronize()
    out, lse = s.cache.decode(q.contiguous(), 0.1, stream=side)
    side.synchronize()
    check_decode(s, q.contiguous(), out, lse, 0.1)


STREAM_AS = {"object": lambda s: s, "address": lambda s: s.cuda_stream}


@pytest.mark.parametrize("form", list(STREAM_AS))
def test_calls_run_on_the_stream_they_are_given(form):
    """Inputs that a busy side stream is still to write: calls on any other
    stream would read what was there before."""
    s = Setup([500, 60], 8, 2, 128, seed=64, fill=0.0)
    side = torch.cuda.Stream()
    x = s.randn(2, 12, 128)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    new, ai, src, dst = s.randn(2, 12, 128), i32([0, 1, 2]), i32([0]), i32([0])
    free = np.setdiff1d(np.arange(s.pool.shape[0]), s.values)[:1]
    want = s.pool.clone()
    for b, t in ((0, 499), (1, 59)):
        pid, sl = ref.slots(*s.table, b)
        want[pid[t], 0, :, sl[t]], want[pid[t], 1, :, sl[t]] = new[b, 8:10], new[b, 10:]
    want[free] = want[s.values[:1]]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(new)
        src.fill_(int(s.values[0]))
        dst.fill_(int(free[0]))
    at = STREAM_AS[form](side)
    qo = s.cache.append(q, k, v, ai, stream=at)
    out, lse = s.cache.decode(qo, 0.1, stream=at)
    s.cache.copy_pages(src, dst, stream=at)
    tables = s.cache.compact(i32([0, 0, 0]), i32([0, 0, 0]), i32([]), stream=at)
    side.synchronize()
    assert torch.equal(qo, new[:, :8]) and torch.equal(s.pool, want)
    check_decode(s, qo, out, lse, 0.1)
    assert tables[0].tolist() == s.indptr.tolist() and s.cache.device_status(at) == ta.TA_OK


@pytest.mark.parametrize("form", list(STREAM_AS))
def test_outputs_come_from_the_pool_of_the_calls_stream(form):
    """Memory that the current stream still reads is not given to a call on
    another stream."""
    s = Setup([500, 60], 8, 2, 128, seed=65, fill=0.0)
    side = torch.cuda.Stream()
    q = s.randn(2, 8, 128)
    x = torch.full((2, 8, 128), 3.0, dtype=s.dtype, device="cuda")
    at = x.data_ptr()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    y = x * 2
    del x
    out, lse = s.cache.decode(q, 0.1, stream=STREAM_AS[form](side))
    assert out.data_ptr() != at
    side.synchronize()
    check_decode(s, q, out, lse, 0.1)
    assert (y == 6).all()


@pytest.mark.parametrize("address", [0, 1, 2])
def test_calls_on_the_default_streams_by_address(address):
    s = Setup([500, 60], 8, 2, 128, seed=66, fill=0.0)
    q = s.randn(2, 8, 128)
    torch.cuda.synchronize()
    out, lse = s.cache.decode(q, 0.1, stream=address)
    torch.cuda.synchronize()
    check_decode(s, q, out, lse, 0.1)


def test_a_dropped_handles_workspace_outlives_its_calls():
    """On a stream object and on the current stream: the handle's own workspace
    is not given to another tensor before the calls are done."""
    s = Setup([3000, 60], 8, 2, 128, seed=67, fill=0.0)
    q = s.randn(2, 8, 128)
    want = [t.clone() for t in s.cache.decode(q, 0.1)]
    for given in (True, False):
        side = torch.cuda.Stream()
        c = s.cache.with_table(*[i32(x) for x in s.table], workspace=None)
        at, n = c.workspace.data_ptr(), c.workspace.numel()
        out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            c.decode(q, 0.1, out=out, lse=lse, stream=side if given else None)
            if given:
                c.decode(q, 0.1, out=out, lse=lse, stream=side)
        del c
        other = torch.empty(n, dtype=torch.uint8, device="cuda")
        assert other.data_ptr() != at
        other.fill_(255)
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert (other == 255).all()


def test_a_handle_made_in_a_captured_graph():
    """Its workspace is in memory that another graph has left dirty.  Calls
    outside the graph, in another one, and in its own, before and after the
    replays of each."""
    s = Setup([6000, 60, 900], 8, 2, 128, seed=68, fill=0.0)
    q = s.randn(3, 8, 128)
    tables = [i32(x) for x in s.table]
    want = [t.clone() for t in s.cache.decode(q, 0.1)]
    outs = [(torch.empty_like(want[0]), torch.empty_like(want[1])) for _ in range(3)]
    torch.cuda.synchronize()
    dirty, first, second = (torch.cuda.CUDAGraph() for _ in range(3))
    with torch.cuda.graph(dirty):
        x = torch.full((64 << 20,), 127, dtype=torch.uint8, device="cuda")
    dirty.replay()
    torch.cuda.synchronize()
    pool = dirty.pool()
    del x
    with torch.cuda.graph(first, pool=pool):
        tmp = torch.full((64 << 20,), 126, dtype=torch.uint8, device="cuda")
        del tmp
        c = s.cache.with_table(*tables, workspace=None)
        c.decode(q, 0.1, *outs[0])
    with torch.cuda.graph(second):
        c.decode(q, 0.1, *outs[1])

    def check(*which):
        torch.cuda.synchronize()
        assert c.device_status() == ta.TA_OK
        for i in which:
            assert torch.equal(outs[i][0], want[0]) and torch.equal(outs[i][1], want[1])
            outs[i][0].fill_(7)
            outs[i][1].fill_(7)

    assert bool((c.workspace == 0).all())
    c.decode(q, 0.1, *outs[2])
    check(2)
    second.replay()
    check(1)
    first.replay()
    check(0)
    second.replay()
    check(1)
    c.decode(q, 0.1, *outs[2])
    first.replay()
    check(0, 2)


def test_captured_compaction_and_copies_follow_their_inputs():
    """Paths, node counts and page lists that change in place between replays;
    a list for either way of finding conflicts."""
    s = Setup([100, 64, 40], 8, 2, 64, seed=69, spare=6000, fill=0.0)
    s.pool.copy_(torch.randn(s.pool.shape, device="cuda"))
    mn, ai, an = i32([0, 30, 80, 90]), i32([0, 4, 6, 7]), i32([0, 3, 9, 20, 1, 40, 5])
    free = np.setdiff1d(np.arange(s.pool.shape[0]), s.values)
    lists = [(i32(free[:n]), i32(free[n:2 * n])) for n in (40, 2500)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for a, b in lists:
            s.cache.copy_pages(a, a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new = s.cache.compact(mn, ai, an)
        for a, b in lists:
            s.cache.copy_pages(a, b)
    for step in range(3):
        nodes = [[30, 50, 10], [1, 64, 0], [7, 16, 33]][step]
        paths = [[[0, 3, 9, 20], [1, 40], [5]], [[0], list(range(58, 64)), []],
                 [[1, 6], [0, 1, 2, 3], [32]]][step]
        ai_now = np.concatenate([[0], np.cumsum([len(p) for p in paths])])
        mn.copy_(i32(np.concatenate([[0], np.cumsum(nodes)])))
        ai.copy_(i32(ai_now))
        an.copy_(i32(np.concatenate([np.asarray(p, dtype=int) for p in paths])))
        rng = np.random.default_rng(step)
        for a, b in lists:
            p = rng.permutation(free)
            a.copy_(i32(p[:len(a)]))
            b.copy_(i32(p[len(a):2 * len(a)]))
        want, ri, rv, rl, rf = ref.compact(f64(s.pool), *s.table, f64(mn).astype(int), ai_now,
                                           f64(an).astype(int))
        for a, b in lists:
            want[f64(b).astype(int)] = want[f64(a).astype(int)]
        graph.replay()
        torch.cuda.synchronize()
        assert s.cache.device_status() == ta.TA_OK
        np.testing.assert_array_equal(f64(s.pool), want)
        assert new[0].tolist() == ri and new[2].tolist() == rl and int(new[4]) == len(rf)
        assert new[1][:ri[-1]].tolist() == rv and new[3][:len(rf)].tolist() == rf


def test_a_dropped_handles_table_outlives_its_calls():
    """A table whose last references go with the handle."""
    s = Setup([3000, 60], 8, 2, 128, seed=70, fill=0.0)
    q = s.randn(2, 8, 128)
    want = [t.clone() for t in s.cache.decode(q, 0.1)]
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    side = torch.cuda.Stream()
    c = s.cache.with_table(*[i32(x) for x in s.table])
    tables = [(t.data_ptr(), t.numel()) for t in (c.page_indptr, c.page_values, c.length_info)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    c.decode(q, 0.1, out=out, lse=lse, stream=side)
    del c
    others = [torch.full((n,), 99, dtype=torch.int32, device="cuda") for _ in range(8)
              for _, n in tables]
    assert not {o.data_ptr() for o in others} & {at for at, _ in tables}
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
