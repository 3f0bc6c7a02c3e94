"""CPU tests of the paged-cache calls: the references against other facts, the
rotation table, and the arguments that the C entry points refuse before they
launch anything."""
import ctypes
import math

import numpy as np
import pytest

import oracle
import tree_attention_gb300 as ta
import workloads as wl
from oracle import paged_cache_ref as ref
from tree_attention_gb300 import build as ta_build


@pytest.fixture(scope="module")
def lib():
    ta_build.build()
    return ta.lib()


# --------------------------------------------------------------------------
# the references
# --------------------------------------------------------------------------

def test_decode_reference_is_tree_attention_of_single_nodes():
    """A tree of one node that ends its sequence sees every kv row."""
    rng = np.random.default_rng(3)
    w = wl.build_workload("t", [wl.chain_tree(1) for _ in range(4)], h_q=4, h_kv=2, head_dim=64,
                          dtype="bf16", tensor_seed=1, prefix_lens=[0, 15, 16, 60])
    pk = wl.paged_from(w, seed=9, fill=0.0)
    ro, rl = oracle.tree_attention_paged(w.q, w.q_indptr, pk.pages, pk.page_indptr,
                                         pk.page_values, pk.last_page_len, w.mn_indptr,
                                         w.tree_order, 0, w.sm_scale)
    out, lse, mag, smag = ref.decode(w.q.double().numpy(), pk.pages.double().numpy(),
                                     pk.page_indptr, pk.page_values, pk.last_page_len, w.sm_scale)
    np.testing.assert_allclose(out, ro, atol=1e-6)
    np.testing.assert_allclose(lse, rl, atol=1e-6)
    assert (np.abs(out) <= mag + 1e-12).all() and rng is not None


def test_rotation_reference():
    """Norms are kept, positions only count through their difference, and the
    two layouts are one rotation in another order of elements."""
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 5, 3, 64))
    freq = 1e4 ** (-np.arange(16) / 16.0)
    pos = np.arange(5) + 70000
    a = ref.rotate(x, pos, "half", 32, freq)
    np.testing.assert_allclose((a ** 2).sum(-1), (x ** 2).sum(-1))
    np.testing.assert_array_equal(a[..., 32:], x[..., 32:])
    dots = [(ref.rotate(x, pos + s, "half", 32, freq)
             * ref.rotate(y, pos[::-1] + s, "half", 32, freq)).sum(-1) for s in (0, 17)]
    np.testing.assert_allclose(dots[0], dots[1], atol=1e-9)
    order = np.arange(32).reshape(2, 16).T.reshape(-1)       # interleave the halves
    b = ref.rotate(x[..., :32][..., order], pos, "interleaved", 32, freq)
    np.testing.assert_allclose(b, a[..., :32][..., order], atol=1e-12)


def test_compact_reference_keeps_paths():
    rng = np.random.default_rng(1)
    pool = rng.normal(size=(6, 2, 1, 16, 4))
    indptr, values, last = [0, 3, 5], [4, 0, 2, 5, 1], [8, 3]
    # sequence 0: 40 rows, 30 of them nodes; sequence 1: 19 rows, 19 nodes, nothing kept
    p, ni, nv, nl, fr = ref.compact(pool, indptr, values, last, [0, 30, 49], [0, 3, 3], [0, 7, 29])
    rows = lambda q, v, i: np.stack([q[v[r // 16], :, :, r % 16] for r in i])
    np.testing.assert_array_equal(rows(p, values[:3], range(13)),
                                  rows(pool, values[:3], list(range(10)) + [10, 17, 39]))
    assert (ni, nv, nl, fr) == ([0, 1, 1], [4], [13, 0], [0, 2, 5, 1])


# --------------------------------------------------------------------------
# the rotation table
# --------------------------------------------------------------------------

@pytest.mark.parametrize("theta,scale,rd", [(1e4, 1.0, 128), (5e5, 0.25, 64), (1e4, -1.0, 16)])
def test_rope_table_turns(lib, theta, scale, rd):
    """turns / 2^64 is the frequency in turns; the table keeps at least 2^-53 of
    the value (the doubles it is made from) and 2^-64 of a turn."""
    r = ta.Rope("half", rd, theta=theta, scale=scale).struct
    for j in range(rd // 2):
        want = scale * theta ** (-2.0 * j / rd) / (2 * math.pi)
        got = r.turns[j] / 2 ** 64
        got -= 1.0 if want < 0 else 0.0
        assert abs(got - want) <= 4 * 2.0 ** -53 * abs(want) + 2.0 ** -53
    assert list(r.turns)[rd // 2:] == [0] * (64 - rd // 2)


def test_rope_table_takes_frequencies(lib):
    f = [0.5 ** i for i in range(8)]
    a = ta.Rope("interleaved", 16, inv_freq=f, theta=float("nan"))
    b = ta.Rope("interleaved", 16, theta=2.0 ** 8)
    assert list(a.struct.turns)[:8] == pytest.approx(list(b.struct.turns)[:8], rel=1e-14)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=144), dict(theta=0.0),
    dict(theta=float("inf")), dict(scale=float("nan")), dict(magnitude=float("inf")),
    dict(inv_freq=[float("inf")] * 32),
])
def test_rope_refusals(lib, kw):
    with pytest.raises(ta.TreeAttnError) as e:
        ta.Rope("half", **{"rotary_dim": 64, **kw})
    assert e.value.status == ta.TA_ERR_INVALID_ARGUMENT


def test_rope_refuses_unknown_layouts_and_short_tables(lib):
    with pytest.raises(ValueError):
        ta.Rope("quarter", 64)
    with pytest.raises(ValueError):
        ta.Rope("half", 64, inv_freq=[1.0])
    assert lib.tree_attn_rope_init(None, 1, 64, 1e4, 1.0, 1.0, None) == ta.TA_ERR_INVALID_ARGUMENT
    r = ta.Rope("half", 64).struct
    assert lib.tree_attn_rope_init(ctypes.byref(r), 3, 64, 1e4, 1.0, 1.0,
                                   None) == ta.TA_ERR_INVALID_ARGUMENT


# --------------------------------------------------------------------------
# refusals of the C entry points (fake pointers: nothing is launched)
# --------------------------------------------------------------------------

F = 0x10000
ODD = ctypes.c_void_p(F + 8)


def _dims(**kw):
    d = dict(batch_size=3, h_q=8, h_kv=2, head_dim=128, dtype=ta.TA_BF16, num_pages=12,
             nnz_pages=6)
    d.update(kw)
    return ta.CacheDims(**d)


def _append(lib, dims=None, **kw):
    a = dict(q=F, qs=1024, k=F, ks=256, v=F, vs=256, n=5, ai=F, pos=F, qw=F, kw=F, eps=1e-6,
             rope=ctypes.byref(ta.Rope("half", 128).struct), pages=F, pi=F, pv=F, li=F, qo=F,
             ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_append_paged(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["n"],
                                      a["ai"], a["pos"], a["qw"], a["kw"], a["eps"], a["rope"],
                                      a["pages"], a["pi"], a["pv"], a["li"], a["qo"],
                                      ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


def _decode(lib, dims=None, **kw):
    a = dict(q=F, pages=F, pi=F, pv=F, li=F, out=F, lse=F, sm=0.1, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_decode_paged(a["q"], a["pages"], a["pi"], a["pv"], a["li"], a["out"],
                                      a["lse"], a["sm"], ctypes.byref(dims or _dims()), a["ws"],
                                      a["wsb"], None)


def _compact(lib, dims=None, **kw):
    a = dict(pages=F, pi=F, pv=F, li=F, mn=F, ai=F, an=F, n=4, npi=3 * F, npv=4 * F, nli=5 * F,
             fr=6 * F, nf=7 * F, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_compact_paged(a["pages"], a["pi"], a["pv"], a["li"], a["mn"], a["ai"],
                                       a["an"], a["n"], a["npi"], a["npv"], a["nli"], a["fr"],
                                       a["nf"], ctypes.byref(dims or _dims()), a["ws"], a["wsb"],
                                       None)


def _copy(lib, dims=None, **kw):
    a = dict(pages=F, src=F, dst=F, n=4, ws=2 * F, wsb=1 << 30)
    a.update(kw)
    return lib.tree_attn_copy_pages(a["pages"], a["src"], a["dst"], a["n"],
                                    ctypes.byref(dims or _dims()), a["ws"], a["wsb"], None)


CALLS = {"append": _append, "decode": _decode, "compact": _compact, "copy": _copy}


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("dims,expect", [
    (dict(batch_size=0), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(h_q=7), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(h_kv=0), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(dtype=5), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(num_pages=0), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(nnz_pages=-1), ta.TA_ERR_INVALID_ARGUMENT),
    (dict(nnz_pages=1 << 27), ta.TA_ERR_INVALID_ARGUMENT),     # kv rows past int32
    (dict(head_dim=96), ta.TA_ERR_UNSUPPORTED),
    (dict(h_q=258, h_kv=2), ta.TA_ERR_UNSUPPORTED),            # 129 heads per kv head
    (dict(batch_size=16385), ta.TA_ERR_UNSUPPORTED),
])
def test_bad_dims(lib, call, dims, expect):
    assert CALLS[call](lib, _dims(**dims)) == expect
    assert ta.cache_workspace_size(_dims(**dims)) == 0


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("kw", [dict(pages=None), dict(pages=ODD), dict(ws=None),
                                dict(ws=ctypes.c_void_p(2 * F + 16)), dict(wsb=16)])
def test_bad_pool_or_workspace(lib, call, kw):
    assert CALLS[call](lib, **kw) == ta.TA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("call", ["append", "decode", "compact"])
@pytest.mark.parametrize("name", ["pi", "pv", "li"])
def test_missing_table(lib, call, name):
    assert CALLS[call](lib, **{name: None}) == ta.TA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(ai=None),
    dict(pos=None), dict(eps=-1.0), dict(eps=float("nan")), dict(q=ODD), dict(k=ODD), dict(v=ODD),
    dict(qo=ODD), dict(qw=ODD), dict(kw=ODD), dict(qs=1028), dict(qs=1016), dict(ks=248),
    dict(vs=0), dict(ks=-256),
])
def test_append_refusals(lib, kw):
    assert _append(lib, **kw) == ta.TA_ERR_INVALID_ARGUMENT


def test_append_refuses_a_rotation_wider_than_the_head(lib):
    assert _append(lib, _dims(head_dim=64)) == ta.TA_ERR_INVALID_ARGUMENT
    blank = ta._RopeStruct()
    assert _append(lib, rope=ctypes.byref(blank)) == ta.TA_ERR_INVALID_ARGUMENT


def test_append_of_nothing(lib):
    assert _append(lib, n=0, q=None, k=None, v=None, qo=None) == ta.TA_OK


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(lse=None), dict(q=ODD),
                                dict(out=ODD), dict(sm=float("inf"))])
def test_decode_refusals(lib, kw):
    assert _decode(lib, **kw) == ta.TA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(n=-1), dict(mn=None), dict(ai=None), dict(an=None), dict(npi=None), dict(npv=None),
    dict(nli=None), dict(fr=None), dict(nf=None),
    dict(npi=F), dict(npv=F), dict(nli=F), dict(fr=F), dict(fr=4 * F),     # over the old table
])
def test_compact_refusals(lib, kw):
    assert _compact(lib, **kw) == ta.TA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(n=-1), dict(src=None), dict(dst=None)])
def test_copy_refusals(lib, kw):
    assert _copy(lib, **kw) == ta.TA_ERR_INVALID_ARGUMENT


def test_copy_of_nothing(lib):
    assert _copy(lib, n=0, src=None, dst=None) == ta.TA_OK


def test_workspace_leaves_the_same_room_for_parts_whatever_the_heads(lib):
    """Handles that share a workspace differ in marks (4 bytes per page) and
    counters only, both zero between calls: what is left of the size, 256 bytes
    apart, is one number."""
    up = lambda n: -(-n // 256) * 256
    rest = set()
    for h_q, h_kv in ((8, 2), (32, 8), (32, 2), (18, 2), (128, 1), (40, 8), (256, 2)):
        for d in (64, 128):
            for pages, batch in ((12, 3), (5000, 700)):
                g = h_q // h_kv
                groups = 1 if g <= 8 else -(-g // 16)
                n = ta.cache_workspace_size(_dims(h_q=h_q, h_kv=h_kv, head_dim=d, num_pages=pages,
                                                  batch_size=batch))
                rest.add(n - up(4 * pages) - up(4 * batch * h_kv * groups))
    assert len(rest) == 1


# --------------------------------------------------------------------------
# the compiled argument checks of PagedCache (on CPU tensors: all refused)
# --------------------------------------------------------------------------

def _handle(d):
    import torch
    z = torch.zeros(4, dtype=torch.int32)
    pages = torch.zeros((12, 2, 2, 16, 128), dtype=torch.bfloat16)
    return ta._compiled().handle(ctypes.addressof(d), pages, z, torch.zeros(6, dtype=torch.int32),
                                 z[:3], torch.zeros(256, dtype=torch.uint8))


def test_binding_refuses_what_is_not_on_the_handles_device(lib):
    import torch
    b, d = ta._compiled(), _dims()
    h = _handle(d)
    q = torch.zeros((3, 8, 128), dtype=torch.bfloat16)
    lse = torch.zeros((3, 8))
    with pytest.raises(ValueError, match="q must be"):
        b.decode(h, q, 0.1, q, lse, None)
    kv = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="must be"):
        b.append(h, q, kv, kv, z, None, None, None, None, 1e-6, q, None)
    with pytest.raises(ValueError, match="must be"):
        b.compact(h, z, z, z, z, z, z, z, z, None)
    with pytest.raises(ValueError, match="must be"):
        b.copy_pages(h, z, z, None)


@pytest.mark.parametrize("call", [
    lambda b, h: b.decode(h, 1, 0.1, None, None, None),
    lambda b, h: b.copy_pages(h, None, None, None),
    lambda b, h: b.append(h, "q", None, None, None, None, None, None, None, 0.0, None, None),
    lambda b, h: b.decode(h),
    lambda b, h: b.compact(),
    lambda b, h: b.handle(1),
    lambda b, h: b.handle(1, 2, 3, 4, 5, 6),
    lambda b, h: b.decode(None, 1, 0.1, None, None, None),
])
def test_binding_refuses_what_is_no_tensor_or_no_handle(lib, call):
    with pytest.raises(ValueError):
        call(ta._compiled(), _handle(_dims()))


def test_binding_refuses_tensors_without_memory(lib):
    """torch throws on the address of a batched tensor: a Python error, not the
    end of the process."""
    import torch
    d, z = _dims(), torch.zeros(4, dtype=torch.int32)
    said = []

    def make(pages):
        with pytest.raises(RuntimeError) as e:
            ta._compiled().handle(ctypes.addressof(d), pages, z, z, z, z)
        said.append(str(e.value))
        return pages

    torch.func.vmap(make)(torch.zeros((2, 12, 2, 2, 16, 128), dtype=torch.bfloat16))
    assert len(said) == 1


# --------------------------------------------------------------------------
# building the extension module
# --------------------------------------------------------------------------

def test_module_is_rebuilt_for_another_torch(lib, monkeypatch):
    assert ta_build.binding_up_to_date() and ta_build.up_to_date()
    monkeypatch.setattr("torch.__version__", "0.0")
    assert not ta_build.binding_up_to_date() and not ta_build.up_to_date()


@pytest.mark.parametrize("fails", ["_compile_binding", "_link_binding"])
def test_library_is_linked_though_the_module_fails(lib, monkeypatch, tmp_path, fails):
    def fail(*a):
        raise RuntimeError("no headers")
    for name, file in (("LIB_PATH", "l.so"), ("BINDING_PATH", "b.so"), ("BINDING_STAMP", "b.txt"),
                       ("BUILD_DIR", "")):
        monkeypatch.setattr(ta_build, name, str(tmp_path / file))
    monkeypatch.setattr(ta_build, "SOURCES", ["ta_merge.cu"])     # the shortest
    monkeypatch.setattr(ta_build, "_compile_binding", lambda: "b.o")
    monkeypatch.setattr(ta_build, fails, fail)
    with pytest.raises(RuntimeError, match="no headers"):
        ta_build.build()
    assert (tmp_path / "l.so").exists() and not (tmp_path / "b.so").exists()
    monkeypatch.setattr(ta_build, "_compile_binding", lambda: "b.o")
    monkeypatch.setattr(ta_build, "_link_binding", lambda o: (tmp_path / "b.so").touch())
    monkeypatch.setattr(ta_build, "_link_library", fail)          # already there
    ta_build.build()


@pytest.mark.parametrize("there,says", [(True, "cannot be loaded"), (False, "is not built")])
def test_a_module_that_does_not_load_is_told_from_one_that_is_not_there(lib, monkeypatch, there,
                                                                        says):
    import importlib
    def fail(name):
        raise ImportError("undefined symbol")
    monkeypatch.setattr(ta, "_binding_module", None)
    monkeypatch.setattr(importlib, "import_module", fail)
    monkeypatch.setattr(ta.os.path, "exists", lambda p: there)
    with pytest.raises(RuntimeError, match=says + r" \(undefined symbol\)"):
        ta._compiled()
