"""Refusals of the calls on caches held to a budget: every bad argument returns before a CUDA call."""
import ctypes

import pytest

from test_tree_host import ARG, BAD_CACHE, FAKE, UNSUP, WS, kv

APART = 1 << 24         # farther than any array of these sizes


def append(L, cache, **kw):
    a = dict(k=FAKE, v=FAKE, N=4, n=FAKE, parent=FAKE, kw=FAKE, qw=FAKE, eps=1e-6, inv=FAKE, rot=64, off=64, inter=1, q=FAKE,
             H=64, qo=FAKE, pos0=FAKE, sp=FAKE, slots=100)
    a.update(kw)
    return L.ds4a_paged_append_norm(cache, a["k"], a["v"], a["N"], a["n"], a["parent"], a["kw"], a["qw"],
                                    ctypes.c_float(a["eps"]), a["inv"], a["rot"], a["off"], a["inter"], a["q"], a["H"], a["qo"],
                                    a["pos0"], a["sp"], a["slots"], None)


def weights(L, cache, **kw):
    a = dict(q=FAKE, N=4, H=64, n=FAKE, lse=FAKE, scale=0.1, decay=1.0, acc=FAKE, slots=100)
    a.update(kw)
    return L.ds4a_attn_weights(cache, a["q"], a["N"], a["H"], a["n"], a["lse"], ctypes.c_float(a["scale"]),
                               ctypes.c_float(a["decay"]), a["acc"], a["slots"], None)


def prefix(L, cache, **kw):
    a = dict(q=FAKE, N=4, H=64, n=FAKE, parent=FAKE, start=FAKE, shared=FAKE, G=3, scale=0.1, out=FAKE + APART, lse=FAKE, ws=FAKE,
             nb=None)
    a.update(kw)
    nb = L.ds4a_attn_prefix_workspace_bytes(2, 4, 64, 128, 3) if a["nb"] is None else a["nb"]
    return L.ds4a_attn_prefix(cache, a["q"], a["N"], a["H"], a["n"], a["parent"], a["start"], a["shared"], a["G"],
                              ctypes.c_float(a["scale"]), a["out"], a["lse"], a["ws"], nb, None)


def evict(L, cache, **kw):
    a = dict(acc=FAKE, pos=FAKE + APART, slots=100, next=FAKE, budget=50, sink=4, recent=8, ao=FAKE, po=FAKE + APART,
             lo=FAKE + 2 * APART, ws=FAKE, nb=None)
    a.update(kw)
    nb = L.ds4a_evict_workspace_bytes(2, 100, 50) if a["nb"] is None else a["nb"]
    return L.ds4a_evict(cache, a["acc"], a["pos"], a["slots"], a["next"], a["budget"], a["sink"], a["recent"], a["ao"], a["po"],
                        a["lo"], a["ws"], nb, None)


@pytest.mark.parametrize("call", [append, weights, evict, prefix])
def test_bad_caches_are_refused(ds4a_lib, call):
    L = ds4a_lib.lib()
    assert call(L, None) == ARG
    for kw, code in BAD_CACHE:
        assert call(L, kv(ds4a_lib, **kw)) == code, kw
    assert call(L, kv(ds4a_lib, B=0, k=None, v=None, table=None, len=None)) == 0


def test_append_norm_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    for kw, code in [(dict(k=None), ARG), (dict(v=None), ARG), (dict(n=None), ARG), (dict(N=-1), ARG), (dict(N=65), UNSUP),
                     (dict(k=FAKE + 8), ARG), (dict(q=FAKE + 8), ARG), (dict(qo=None), ARG), (dict(H=12), UNSUP),
                     (dict(inv=None), ARG), (dict(rot=24), UNSUP), (dict(off=72), UNSUP), (dict(qo=FAKE + 16), ARG),
                     (dict(eps=0.0), ARG), (dict(eps=-1e-6), ARG), (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG),
                     (dict(kw=FAKE + 2), ARG), (dict(qw=FAKE + 1), ARG), (dict(pos0=FAKE + 4), ARG), (dict(sp=FAKE + 2), ARG),
                     (dict(slots=0), ARG), (dict(slots=-1), ARG)]:
        assert append(L, c, **kw) == code, kw
    assert append(L, c, N=0, k=None, v=None, n=None) == 0


def test_weights_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    for kw, code in [(dict(q=None), ARG), (dict(lse=None), ARG), (dict(acc=None), ARG), (dict(n=None), ARG), (dict(N=0), ARG),
                     (dict(N=65), UNSUP), (dict(H=12), UNSUP), (dict(H=72), UNSUP), (dict(q=FAKE + 8), ARG), (dict(lse=FAKE + 2), ARG),
                     (dict(acc=FAKE + 2), ARG), (dict(slots=0), ARG), (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG),
                     (dict(scale=2.5e38), ARG), (dict(decay=-0.1), ARG), (dict(decay=1.5), ARG), (dict(decay=float("nan")), ARG)]:
        assert weights(L, c, **kw) == code, kw


def test_prefix_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    nb = L.ds4a_attn_prefix_workspace_bytes(2, 4, 64, 128, 3)
    assert nb > 0
    for kw, code in [(dict(q=None), ARG), (dict(out=None), ARG), (dict(n=None), ARG), (dict(N=0), ARG), (dict(N=65), UNSUP),
                     (dict(H=12), UNSUP), (dict(q=FAKE + 8), ARG), (dict(out=FAKE + APART + 8), ARG), (dict(parent=FAKE + 2), ARG),
                     (dict(start=None), ARG), (dict(shared=None), ARG), (dict(start=FAKE + 2), ARG), (dict(shared=FAKE + 4), ARG),
                     (dict(G=-1), ARG), (dict(G=65536), UNSUP), (dict(lse=FAKE + 2), ARG), (dict(out=FAKE), ARG), (dict(out=FAKE + 16), ARG),
                     (dict(scale=0.0), ARG), (dict(scale=float("nan")), ARG), (dict(scale=2.5e38), ARG), (dict(ws=None), WS),
                     (dict(ws=FAKE + 128), WS), (dict(nb=nb - 1), WS)]:
        assert prefix(L, c, **kw) == code, kw
    for bad in [(-1, 4, 64, 128, 1), (65536, 4, 64, 128, 1), (2, 0, 64, 128, 1), (2, 65, 64, 128, 1), (2, 4, 12, 128, 1),
                (2, 4, 64, 96, 1), (2, 4, 64, 128, -1), (2, 4, 64, 128, 65536)]:
        assert L.ds4a_attn_prefix_workspace_bytes(*bad) == 0


def test_evict_refusals(ds4a_lib):
    L, c = ds4a_lib.lib(), kv(ds4a_lib)
    nb = L.ds4a_evict_workspace_bytes(2, 100, 50)
    assert nb > 0
    for kw, code in [(dict(acc=None), ARG), (dict(pos=None), ARG), (dict(next=None), ARG), (dict(ao=None), ARG), (dict(po=None), ARG),
                     (dict(lo=None), ARG), (dict(slots=0), ARG), (dict(slots=(1 << 23) + 1), UNSUP), (dict(budget=0), ARG),
                     (dict(sink=-1), ARG), (dict(recent=-1), ARG), (dict(sink=43), ARG), (dict(recent=47), ARG),
                     (dict(sink=1 << 30, recent=(1 << 31) - 1), ARG), (dict(acc=FAKE + 2, ao=FAKE + 2), ARG),
                     (dict(next=FAKE + 4), ARG), (dict(lo=FAKE + 2 * APART + 4), ARG),
                     # one array in place and one apart, arrays that overlap in part or one another
                     (dict(ao=FAKE + 4 * APART), ARG), (dict(po=FAKE + 4 * APART), ARG),
                     (dict(ao=FAKE + 16, po=FAKE + 4 * APART), ARG), (dict(ao=FAKE + 4 * APART, po=FAKE + APART + 16), ARG),
                     (dict(pos=FAKE, po=FAKE), ARG), (dict(ao=FAKE + 4 * APART, po=FAKE + 4 * APART), ARG),
                     (dict(lo=FAKE + 8), ARG), (dict(ws=None), WS), (dict(ws=FAKE + 128), WS), (dict(nb=nb - 1), WS)]:
        assert evict(L, c, **kw) == code, kw
    for bad in [(-1, 100, 50), (2, 0, 50), (2, 100, 0), (2, (1 << 23) + 1, 50)]:
        assert L.ds4a_evict_workspace_bytes(*bad) == 0


def test_binding_refuses_shapes(ds4a_lib):
    import torch
    desc = ds4a_lib.PagedKVDesc(B=1, D=64, page=16, max_pages=3, n_pages=4)
    desc.tensors, desc.device = (), 0
    q = torch.zeros(1, 4, 8, 64, dtype=torch.float16)
    n, f = torch.zeros(1, dtype=torch.int32), torch.zeros(1, 40)
    with pytest.raises(ValueError, match="paged_append_norm: k, v"):
        ds4a_lib.ds4a_paged_append_norm(desc, q, q, n, None, None, 1e-6)
    with pytest.raises(ValueError, match="paged_append_norm: k_w"):
        ds4a_lib.ds4a_paged_append_norm(desc, q[:, :, 0], q[:, :, 0], n, f, None, 1e-6)
    with pytest.raises(ValueError, match="paged_append_norm: pos0"):
        ds4a_lib.ds4a_paged_append_norm(desc, q[:, :, 0], q[:, :, 0], n, None, None, 1e-6, pos0=f)
    with pytest.raises(ValueError, match="attn_prefix: q, out"):
        ds4a_lib.ds4a_attn_prefix(desc, q[0], n, None, None, None, 0.1, q, None, q)
    with pytest.raises(ValueError, match="come together"):
        ds4a_lib.ds4a_attn_prefix(desc, q, n, None, n, None, 0.1, q, None, q)
    with pytest.raises(ValueError, match="attn_prefix: start"):
        ds4a_lib.ds4a_attn_prefix(desc, q, n, None, n, n, 0.1, q, None, q)
    with pytest.raises(ValueError, match="attn_prefix: lse"):
        ds4a_lib.ds4a_attn_prefix(desc, q, n, None, None, None, 0.1, q, f, q)
    with pytest.raises(ValueError, match="attn_weights: q"):
        ds4a_lib.ds4a_attn_weights(desc, q[0], n, f, 0.1, 1.0, f)
    with pytest.raises(ValueError, match="attn_weights: lse"):
        ds4a_lib.ds4a_attn_weights(desc, q, n, f, 0.1, 1.0, f)
    with pytest.raises(ValueError, match="evict: acc, pos"):
        ds4a_lib.ds4a_evict(desc, f, n, n, 10, 0, 0, f, f, n, None)
    with pytest.raises(ValueError, match="evict: next_pos"):
        ds4a_lib.ds4a_evict(desc, f, f, f, 10, 0, 0, f, f, n, None)
