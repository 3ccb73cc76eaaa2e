"""Refusals of the drafted-token calls: every bad argument returns before a CUDA call."""
import ctypes

import pytest

FAKE = 0x10000          # never dereferenced
ARG, CAP, UNSUP, WS = 1, 2, 3, 6


def kv(ds4a, **kw):
    a = dict(B=2, D=128, page=64, max_pages=100, n_pages=300, k=FAKE, v=FAKE, table=FAKE, len=FAKE)
    a.update(kw)
    return ctypes.byref(ds4a.PagedKVDesc(**a))


BAD_CACHE = [(dict(B=-1), ARG), (dict(B=65536), UNSUP), (dict(D=96), UNSUP), (dict(D=256), UNSUP), (dict(page=0), ARG),
             (dict(page=24), UNSUP), (dict(page=1 << 17), UNSUP), (dict(max_pages=0), ARG), (dict(n_pages=0), ARG),
             (dict(max_pages=1 << 25), UNSUP), (dict(n_pages=1 << 25), UNSUP), (dict(n_pages=1 << 62), UNSUP),
             (dict(k=None), ARG), (dict(v=None), ARG), (dict(table=None), ARG), (dict(len=None), ARG),
             (dict(k=FAKE + 8), ARG), (dict(v=FAKE + 2), ARG), (dict(table=FAKE + 2), ARG), (dict(len=FAKE + 4), ARG)]


def append(L, cache, **kw):
    a = dict(k=FAKE, v=FAKE, N=4, n=FAKE, parent=FAKE, inv=FAKE, rot=64, off=64, inter=1, q=FAKE, H=64, qo=FAKE)
    a.update(kw)
    return L.ds4a_paged_append(cache, a["k"], a["v"], a["N"], a["n"], a["parent"], a["inv"], a["rot"], a["off"],
                               a["inter"], a["q"], a["H"], a["qo"], None)


def compress(L, cache, **kw):
    a = dict(N=4, n=FAKE, parent=FAKE, w=FAKE, ratio=4, state=FAKE, ck=FAKE, cv=FAKE, cap=100)
    a.update(kw)
    return L.ds4a_compress_tree(cache, a["N"], a["n"], a["parent"], a["w"], a["ratio"], a["state"], a["ck"], a["cv"],
                                a["cap"], None)


def attn(L, cache, **kw):
    a = dict(q=FAKE, N=4, H=64, n=FAKE, parent=FAKE, window=128, ck=FAKE, cv=FAKE, cap=100, ratio=4, sel=None, n_sel=0,
             out=FAKE + (1 << 24), ws=FAKE, nb=None, scale=0.1)
    a.update(kw)
    nb = L.ds4a_attn_tree_workspace_bytes(2, 4, 64, 128) if a["nb"] is None else a["nb"]
    return L.ds4a_attn_tree(cache, a["q"], a["N"], a["H"], a["n"], a["parent"], a["window"], a["ck"], a["cv"], a["cap"],
                            a["ratio"], a["sel"], a["n_sel"], ctypes.c_float(a["scale"]), a["out"], a["ws"], nb, None)


def commit(L, cache, **kw):
    a = dict(N=4, n=FAKE, parent=FAKE, leaf=FAKE, lo=FAKE, w=FAKE, ratio=4, state=FAKE, so=FAKE, ck=FAKE, cv=FAKE,
             cap=100, ki=None, di=0)
    a.update(kw)
    return L.ds4a_commit_tree(cache, a["N"], a["n"], a["parent"], a["leaf"], a["lo"], a["w"], a["ratio"], a["state"],
                              a["so"], a["ck"], a["cv"], a["cap"], a["ki"], a["di"], None)


@pytest.mark.parametrize("call", [append, compress, attn, commit])
def test_bad_caches_are_refused(ds4a_lib, call):
    L = ds4a_lib.lib()
    assert call(L, None) == ARG
    for kw, code in BAD_CACHE:
        assert call(L, kv(ds4a_lib, **kw)) == code, kw
    # no sessions: nothing to do
    assert call(L, kv(ds4a_lib, B=0, k=None, v=None, table=None, len=None)) == 0


@pytest.mark.parametrize("call", [compress, attn, commit])
def test_bad_trees_are_refused(ds4a_lib, call):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    for kw, code in [(dict(N=0), ARG), (dict(N=-3), ARG), (dict(N=65), UNSUP), (dict(n=None), ARG), (dict(n=FAKE + 2), ARG),
                     (dict(parent=FAKE + 1), ARG), (dict(ratio=-1), ARG), (dict(ratio=1025), UNSUP), (dict(cap=-1), ARG),
                     (dict(cap=1 << 31), UNSUP), (dict(cap=3), CAP), (dict(ck=None), ARG), (dict(cv=None), ARG),
                     (dict(ck=FAKE + 8), ARG), (dict(cv=FAKE + 8), ARG)]:
        assert call(L, c, **kw) == code, kw


def test_append_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    for kw, code in [(dict(k=None), ARG), (dict(v=None), ARG), (dict(n=None), ARG), (dict(N=-1), ARG), (dict(N=65), UNSUP),
                     (dict(k=FAKE + 8), ARG), (dict(v=FAKE + 8), ARG), (dict(q=FAKE + 8), ARG), (dict(qo=FAKE + 8), ARG),
                     (dict(qo=None), ARG), (dict(q=None), ARG), (dict(H=12), UNSUP), (dict(H=72), UNSUP), (dict(H=0), UNSUP),
                     (dict(inv=None), ARG), (dict(inv=FAKE + 2), ARG), (dict(rot=-16), ARG), (dict(rot=24), UNSUP),
                     (dict(rot=144, off=0), UNSUP), (dict(off=72), UNSUP), (dict(off=-8), ARG), (dict(off=60), UNSUP),
                     (dict(n=FAKE + 2), ARG), (dict(parent=FAKE + 2), ARG),
                     # queries that overlap their output without being it
                     (dict(qo=FAKE + 16), ARG), (dict(q=FAKE + 16 * 1024), ARG)]:
        assert append(L, c, **kw) == code, kw
    assert append(L, c, N=0, k=None, v=None, n=None) == 0


def test_compress_and_commit_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    for kw, code in [(dict(ratio=0), ARG), (dict(w=None), ARG), (dict(state=None), ARG), (dict(state=FAKE + 2), ARG),
                     (dict(w=FAKE + 2), ARG)]:
        assert compress(L, c, **kw) == code, kw
    for kw, code in [(dict(leaf=None), ARG), (dict(leaf=FAKE + 2), ARG), (dict(lo=None), ARG), (dict(lo=FAKE + 4), ARG),
                     (dict(so=None), ARG), (dict(state=None), ARG), (dict(w=None), ARG), (dict(so=FAKE + 2), ARG),
                     (dict(ki=FAKE, di=12), UNSUP), (dict(ki=FAKE, di=264), UNSUP), (dict(ki=FAKE, di=0), UNSUP),
                     (dict(ki=FAKE + 8, di=128), ARG), (dict(ki=FAKE, di=128, ratio=0), ARG)]:
        assert commit(L, c, **kw) == code, kw


def test_attn_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    nb = L.ds4a_attn_tree_workspace_bytes(2, 4, 64, 128)
    assert nb > 0
    for kw, code in [(dict(q=None), ARG), (dict(out=None), ARG), (dict(q=FAKE + 8), ARG), (dict(out=FAKE + 8), ARG),
                     (dict(H=12), UNSUP), (dict(H=72), UNSUP), (dict(window=0), ARG), (dict(window=-1), ARG),
                     (dict(sel=FAKE, n_sel=0), ARG), (dict(sel=FAKE, n_sel=8, ratio=0), ARG), (dict(n_sel=-1), ARG),
                     (dict(sel=FAKE + 2, n_sel=8), ARG), (dict(sel=FAKE, n_sel=1 << 30), UNSUP),
                     (dict(cap=1 << 30), UNSUP), (dict(out=FAKE), ARG), (dict(out=FAKE + 16), ARG), (dict(scale=0.0), ARG), (dict(scale=-1.0), ARG), (dict(scale=float("nan")), ARG),
                     (dict(scale=float("inf")), ARG), (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(nb=nb - 1), WS)]:
        assert attn(L, c, **kw) == code, kw
    for bad in [(-1, 4, 64, 128), (2, 0, 64, 128), (2, 65, 64, 128), (2, 4, 12, 128), (2, 4, 64, 96)]:
        assert L.ds4a_attn_tree_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors_and_shapes(ds4a_lib):
    import torch
    pool = torch.zeros(4, 16, 64, dtype=torch.float16)
    tab, ln = torch.zeros(1, 3, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ds4a_lib.paged_kv_desc(pool, pool, tab, ln)
    with pytest.raises(ValueError, match="pools"):
        ds4a_lib.paged_kv_desc(pool[0], pool[0], tab, ln)
    with pytest.raises(ValueError, match="pools"):
        ds4a_lib.paged_kv_desc(pool, pool, tab, torch.zeros(2, dtype=torch.int64))
    desc = ds4a_lib.PagedKVDesc(B=1, D=64, page=16, max_pages=3, n_pages=4)
    desc.tensors, desc.device = (), 0
    q = torch.zeros(1, 4, 8, 64, dtype=torch.float16)
    n, par = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="attn_tree: q, out"):
        ds4a_lib.ds4a_attn_tree(desc, q[0], n, par, 128, None, None, 0, None, 0.1, q, q)
    with pytest.raises(ValueError, match="attn_tree: sel"):
        ds4a_lib.ds4a_attn_tree(desc, q, n, par, 128, None, None, 4, par, 0.1, q, q)
    with pytest.raises(ValueError, match="paged_append: k, v"):
        ds4a_lib.ds4a_paged_append(desc, pool[0], pool[0], n)
    with pytest.raises(ValueError, match="come together"):
        ds4a_lib.ds4a_paged_append(desc, q[:, :, 0], q[:, :, 0], n, q=q)
    with pytest.raises(ValueError, match="needs N"):
        ds4a_lib.ds4a_compress_tree(desc, n, None, n, 4, n, pool, pool)
    with pytest.raises(ValueError, match="commit_tree: leaf"):
        ds4a_lib.ds4a_commit_tree(desc, n, par, par, ln)
