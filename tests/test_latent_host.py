"""CPU tests of the latent-attention calls: the references against other facts,
and the arguments that the C entry points refuse before they launch anything."""
import ctypes
import math

import numpy as np
import pytest
import torch

import tree_attention_gb300 as ta
import workloads as wl
from oracle import latent_ref as ref
from oracle import paged_cache_ref as paged
from tree_attention_gb300 import build as ta_build


@pytest.fixture(scope="module")
def lib():
    ta_build.build()
    return ta.lib()


# --------------------------------------------------------------------------
# the references
# --------------------------------------------------------------------------

def test_absorbed_and_expanded_forms_are_one_attention():
    """Queries with the key projection applied to them, over the latents, and the
    value projection behind, against keys and values per head: a chain as tree,
    which is causal."""
    g = torch.Generator().manual_seed(0)
    h, rank, rope, d, kv, n = 3, 32, 16, 8, 21, 5
    rows = torch.randn((kv, rank + rope), generator=g, dtype=torch.float64)
    wk, wv = torch.randn((2, h, rank, d), generator=g, dtype=torch.float64)
    q = torch.randn((n, h, d + rope), generator=g, dtype=torch.float64)
    pool = torch.zeros((2, 16, rank + rope), dtype=torch.float64)
    table = ([0, 2], [1, 0], [5])
    pid, sl = ref.slots(*table, 0)
    pool[pid, sl] = rows
    qa = torch.cat([torch.einsum("nhd,hrd->nhr", q[..., :d], wk), q[..., d:]], -1)
    out, lse, _, _ = ref.absorbed(qa, pool, table, rank, 0.2, [n], [wl.chain_tree(7)])
    k = torch.einsum("tr,hrd->thd", rows[:, :rank], wk)
    v = torch.einsum("tr,hrd->thd", rows[:, :rank], wv)
    o2, l2, _, _ = ref.expanded(q, k, rows[:, rank:], v, [n], [kv], 0.2)
    torch.testing.assert_close(torch.einsum("nhr,hrd->nhd", out, wv), o2)
    torch.testing.assert_close(lse, l2)


def test_one_token_reference_is_that_of_keys_and_values():
    g = torch.Generator().manual_seed(1)
    pool = torch.randn((5, 16, 24), generator=g, dtype=torch.float64)
    table = ([0, 2, 2, 3], [3, 0, 4], [7, 0, 16])
    q = torch.randn((3, 4, 24), generator=g, dtype=torch.float64)
    out, lse, mag, smag = ref.absorbed(q, pool, table, 24, 0.3)
    both = torch.stack([pool, pool], 1)[:, :, None].numpy()
    o2, l2, m2, s2 = paged.decode(q.numpy(), both, *table, 0.3)
    for a, b in ((out, o2), (lse, l2), (mag, m2), (smag, s2)):
        np.testing.assert_allclose(a.numpy(), b, atol=1e-12)


def test_rotation_reference_is_that_of_whole_heads():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 32))
    freq = 1e4 ** (-np.arange(16) / 16.0)
    pos = np.arange(5) + 70000
    for layout in ("half", "interleaved"):
        a = ref.rotate(torch.from_numpy(x), torch.from_numpy(pos), layout, torch.from_numpy(freq), 1.5)
        np.testing.assert_allclose(a.numpy(), paged.rotate(x, pos, layout, 32, freq, 1.5), atol=1e-9)


def test_visible_reference_is_the_interval_test():
    rng = np.random.default_rng(2)
    parent = wl.random_tree(30, rng)
    iv = wl.tree_intervals(parent)
    seen = ref.visible(parent, 30, 34).numpy()
    for i in range(30):
        for j in range(30):
            assert seen[i, 4 + j] == (iv[j][0] <= iv[i][0] < iv[j][1])
    assert seen[:, :4].all()


# --------------------------------------------------------------------------
# refusals (fake pointers: nothing is launched)
# --------------------------------------------------------------------------

F = 0x10000
ODD = ctypes.c_void_p(F + 8)
INV, UNS = ta.TA_ERR_INVALID_ARGUMENT, ta.TA_ERR_UNSUPPORTED


def _dims(**kw):
    d = dict(batch_size=3, h_q=8, rank=512, rope_dim=64, dtype=ta.TA_BF16, num_pages=12,
             nnz_pages=6)
    d.update(kw)
    return ta.LatentDims(**d)


def _rope(rd=64):
    return ctypes.byref(ta.Rope("half", rd).struct)


def _append(lib, dims=None, **kw):
    a = dict(x=F, xs=576, k=F, ks=576, q=F, qt=1536, qh=192, n=5, ai=F, pos=F, w=F, eps=1e-6,
             rope=_rope(), pages=F, pi=F, pv=F, li=F, qo=2 * F, ot=4608, oh=576, ro=F, ws=2 * F,
             wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_append_latent(
        a["x"], a["xs"], a["k"], a["ks"], a["q"], a["qt"], a["qh"], a["n"], a["ai"], a["pos"], a["w"],
        a["eps"], a["rope"], a["pages"], a["pi"], a["pv"], a["li"], a["qo"], a["ot"], a["oh"], a["ro"],
        ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


def _decode(lib, dims=None, **kw):
    a = dict(q=F, pages=F, pi=F, pv=F, li=F, out=F, lse=F, sm=0.1, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_decode_latent(a["q"], a["pages"], a["pi"], a["pv"], a["li"], a["out"], a["lse"],
                                       a["sm"], ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


def _tree(lib, dims=None, **kw):
    a = dict(q=F, qi=F, nq=9, pages=F, pi=F, pv=F, li=F, mn=F, to=F, nt=9, out=F, lse=F, sm=0.1,
             ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_latent(a["q"], a["qi"], a["nq"], a["pages"], a["pi"], a["pv"], a["li"], a["mn"],
                                a["to"], a["nt"], a["out"], a["lse"], a["sm"],
                                ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


def _compact(lib, dims=None, **kw):
    a = dict(pages=F, pi=F, pv=F, li=F, mn=F, ai=F, an=F, n=4, ni=3 * F, nv=3 * F, nl=3 * F, fr=4 * F,
             nf=F, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_compact_latent(a["pages"], a["pi"], a["pv"], a["li"], a["mn"], a["ai"], a["an"],
                                        a["n"], a["ni"], a["nv"], a["nl"], a["fr"], a["nf"],
                                        ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


def _copy(lib, dims=None, **kw):
    a = dict(pages=F, s=F, d=F, n=2, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_copy_pages_latent(a["pages"], a["s"], a["d"], a["n"],
                                           ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


CALLS = {"append": _append, "decode": _decode, "tree": _tree, "compact": _compact, "copy": _copy}


@pytest.mark.parametrize("name", list(CALLS))
def test_refusals_common(lib, name):
    call = CALLS[name]
    for kw in (dict(batch_size=0), dict(h_q=0), dict(rank=0), dict(rope_dim=0), dict(dtype=7),
               dict(num_pages=0), dict(nnz_pages=-1), dict(nnz_pages=1 << 28)):
        assert call(lib, _dims(**kw)) == INV, kw
    for kw in (dict(rank=384), dict(rank=1024), dict(rope_dim=8), dict(rope_dim=24), dict(rope_dim=80),
               dict(h_q=129), dict(batch_size=16385)):
        assert call(lib, _dims(**kw)) == UNS, kw
    for kw in (dict(pages=None), dict(pages=ODD), dict(ws=None), dict(ws=ctypes.c_void_p(F + 16)),
               dict(wsb=16)):
        assert call(lib, **kw) == INV, kw


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(eps=-1.0), dict(eps=math.nan), dict(rope=_rope(32)), dict(pi=None), dict(li=None),
    dict(pv=None), dict(x=None), dict(k=None), dict(ai=None), dict(pos=None), dict(q=None),
    dict(qo=None), dict(x=ODD), dict(k=ODD), dict(q=ODD), dict(qo=ODD), dict(ro=ODD), dict(w=ODD),
    dict(xs=504), dict(xs=580), dict(ks=56), dict(ks=68), dict(qt=1532), dict(qh=56), dict(qh=196),
    dict(qt=1400), dict(ot=560), dict(oh=60), dict(qo=F),
])
def test_refusals_append(lib, kw):
    assert _append(lib, **kw) == INV


def test_append_of_nothing(lib):
    assert _append(lib, n=0) == ta.TA_OK


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=ODD), dict(out=None), dict(out=ODD), dict(lse=None), dict(pi=None),
    dict(pv=None), dict(li=None), dict(sm=math.nan), dict(sm=math.inf),
])
def test_refusals_attention(lib, kw):
    assert _decode(lib, **kw) == INV
    assert _tree(lib, **kw) == INV


@pytest.mark.parametrize("kw", [
    dict(qi=None), dict(mn=None), dict(to=None), dict(nq=-1), dict(nt=-1),
    dict(to=ctypes.c_void_p(F + 4)),
])
def test_refusals_tree(lib, kw):
    assert _tree(lib, **kw) == INV


def test_tree_of_nothing_and_of_too_much(lib):
    assert _tree(lib, nq=0) == ta.TA_OK
    assert _tree(lib, nq=1 << 29) == UNS


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(mn=None), dict(ai=None), dict(an=None), dict(ni=None), dict(nl=None), dict(nf=None),
    dict(nv=None), dict(fr=None), dict(ni=F), dict(nl=F), dict(nv=F), dict(fr=F), dict(fr=3 * F),
])
def test_refusals_compact(lib, kw):
    assert _compact(lib, **kw) == INV


def test_refusals_copy(lib):
    for kw in (dict(n=-1), dict(s=None), dict(d=None)):
        assert _copy(lib, **kw) == INV
    assert _copy(lib, n=0) == ta.TA_OK


def test_workspace_sizes(lib):
    n = ta.latent_workspace_size(_dims())
    assert n > 0 and n % 256 == 0
    # room for any heads and ranks, so that handles may share one
    assert ta.latent_workspace_size(_dims(rank=256, h_q=128, rope_dim=16)) == n
    assert ta.latent_workspace_size(_dims(num_pages=10 ** 6)) > n
    assert ta.latent_workspace_size(_dims(rank=128)) == 0


def _edims(**kw):
    d = dict(batch_size=2, total_q=10, total_kv=12, heads=4, head_dim=128, rope_dim=64, dtype=ta.TA_BF16)
    d.update(kw)
    return ta.ExpandedDims(**d)


def _expanded(lib, dims=None, **kw):
    a = dict(q=F, qt=768, qh=192, qi=F, k=F, kt=1024, kh=256, kr=F, ks=576, v=F, vt=1024, vh=256, ki=F,
             out=F, lse=F, sm=0.1, ws=2 * F, wsb=256)
    a.update(kw)
    return lib.tree_attn_expanded(a["q"], a["qt"], a["qh"], a["qi"], a["k"], a["kt"], a["kh"], a["kr"],
                                  a["ks"], a["v"], a["vt"], a["vh"], a["ki"], a["out"], a["lse"],
                                  a["sm"], ctypes.byref(dims or _edims()), a["ws"], a["wsb"], None)


def test_refusals_expanded(lib):
    for kw in (dict(batch_size=0), dict(total_q=-1), dict(total_kv=-1), dict(heads=0), dict(head_dim=0),
               dict(rope_dim=0), dict(dtype=5), dict(total_kv=0)):
        assert _expanded(lib, _edims(**kw)) == INV, kw
    for kw in (dict(heads=1025), dict(head_dim=96), dict(rope_dim=40), dict(batch_size=16385),
               dict(total_q=1 << 30)):
        assert _expanded(lib, _edims(**kw)) == UNS, kw
    for kw in [{n: None} for n in ("q", "qi", "k", "kr", "v", "ki", "out", "lse", "ws")] + \
            [{n: ODD} for n in ("q", "k", "kr", "v", "out")] + \
            [dict(qt=764), dict(qt=184), dict(qh=128), dict(kt=120), dict(kh=132), dict(ks=56),
             dict(vt=64), dict(vh=12), dict(kt=1 << 36), dict(sm=math.inf), dict(wsb=128),
             dict(ws=ctypes.c_void_p(F + 16))]:
        assert _expanded(lib, **kw) == INV, kw
    assert _expanded(lib, _edims(total_q=0)) == ta.TA_OK
    assert ta.expanded_workspace_size(_edims()) == 256
    assert ta.expanded_workspace_size(_edims(rope_dim=8)) == 0


def test_python_refusals(lib):
    """What Python can refuse without a GPU."""
    z = torch.zeros
    pages, i = z((3, 16, 576), dtype=torch.bfloat16), z(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        ta.LatentCache(z((3, 2, 1, 16, 64)), i, i, i, h_q=2, rank=512)
    with pytest.raises(ValueError):
        ta.LatentCache(pages, i, i, i[:1], h_q=2, rank=512)      # not on a GPU
    q = z((4, 2, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ta.tree_attn_expanded(q, i, q[..., :128], z((4, 64)), q[..., :128], i, None, None, 0.1, None)
    with pytest.raises(ValueError):
        ta.tree_attn_expanded(q[0], i, q, q, q, i, None, None, 0.1, None)


# --------------------------------------------------------------------------
# workspaces of the two kinds of cache
# --------------------------------------------------------------------------

def test_claims_go_by_memory_until_reset():
    """A view of a workspace is that workspace; parts of one buffer are not."""
    a, b = "latent", "paged"
    buf = torch.full((1000,), 7, dtype=torch.uint8)
    ta._claim(buf[:400], a)
    for view in (buf, buf[:400], buf[399:500], buf.view(-1)[100:200], buf.view(torch.int32)[:2]):
        with pytest.raises(ValueError, match="kind of cache"):
            ta._claim(view, b)
        ta._claim(view, a, used=False)
    ta._claim(buf[400:], b)
    with pytest.raises(ValueError):
        ta._claim(buf[300:500], a)
    ta.reset_workspace(buf[:600])
    assert (buf[:600] == 0).all() and (buf[600:] == 7).all()
    ta._claim(buf[:600], a)
    with pytest.raises(ValueError):
        ta._claim(buf[599:601], a)            # the rest is still the other kind's
    ta.reset_workspace(buf)
    ta._claim(buf, b)
    ta._claim(torch.zeros(1000, dtype=torch.uint8), a)
    with pytest.raises(ValueError, match="contiguous"):
        ta.reset_workspace(buf[::2])
