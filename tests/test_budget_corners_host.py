"""Refusals of the calls on caches held to a budget: arrays that one CTA would write while another reads them.  The
defaults overlap nothing, so only the checks on overlaps stand between them and a launch: no call here passes them."""
import ctypes

import numpy as np
import pytest
import torch

from test_tree_host import ARG, FAKE, kv

B, N, H, D, PAGE, MAX_PAGES, POOL, SLOTS, G = 2, 4, 64, 128, 64, 100, 300, 100, 3
STEP = 1 << 28              # farther than any array of these sizes
NAMES = ["pk", "pv", "table", "len", "k", "v", "n", "parent", "kw", "qw", "inv", "q", "qo", "pos0", "sp", "lse", "acc", "start",
         "shared", "out", "ws", "pos", "next", "ao", "po", "lo"]
AT = {name: (1 + i) * STEP for i, name in enumerate(NAMES)}
BYTES = dict(pk=POOL * PAGE * D * 2, pv=POOL * PAGE * D * 2, table=B * MAX_PAGES * 4, len=B * 8, k=B * N * D * 2, v=B * N * D * 2, n=B * 4,
             parent=B * N * 4, kw=D * 4, qw=D * 4, inv=32 * 4, q=B * N * H * D * 2, qo=B * N * H * D * 2, pos0=B * 8, sp=B * SLOTS * 4,
             lse=B * N * H * 4, acc=B * SLOTS * 4, start=(G + 1) * 4, shared=G * 8, out=B * N * H * D * 2, pos=B * SLOTS * 4, next=B * 8,
             ao=B * SLOTS * 4, po=B * SLOTS * 4, lo=B * 8)


def cache(ds4a, a):
    return kv(ds4a, B=B, D=D, page=PAGE, max_pages=MAX_PAGES, n_pages=POOL, k=a["pk"], v=a["pv"], table=a["table"], len=a["len"])


def refused(ds4a, call, pairs, **fixed):
    """Each pair (out, other): out's start at other's end, on its start, and out's end behind its start."""
    for out, other in pairs:
        for where in {max(0, BYTES[other] - 16) // 16 * 16, 0, min(0, 16 - BYTES[out]) // 16 * 16}:
            a = {**AT, **fixed}
            a[out] = a[other] + where
            assert call(ds4a, a) == ARG, (out, other, where)


def evict(ds4a, a):
    L = ds4a.lib()
    return L.ds4a_evict(cache(ds4a, a), a["acc"], a["pos"], SLOTS, a["next"], 50, 4, 8, a["ao"], a["po"], a["lo"], a["ws"],
                        L.ds4a_evict_workspace_bytes(B, SLOTS, 50), None)


def test_evict_outputs_overlap_nothing(ds4a_lib):
    BYTES["ws"] = ds4a_lib.lib().ds4a_evict_workspace_bytes(B, SLOTS, 50)
    outs = ["ao", "po", "lo"]
    rest = ["table", "next", "pk", "pv", "ws"]
    refused(ds4a_lib, evict, [(o, r) for o in outs for r in rest + [x for x in outs if x != o] + ["len", "acc", "pos"]
                              if (o, r) not in (("lo", "len"), ("ao", "acc"), ("po", "pos"))])
    # in place (acc, pos and the lengths are what is written)
    for x, y in (("lo", "acc"), ("lo", "pos"), ("acc", "table"), ("acc", "next"), ("acc", "len"), ("pos", "next"), ("pos", "len"),
                 ("pos", "table"), ("acc", "pk"), ("pos", "pv"), ("acc", "ws")):
        a = dict(AT)
        a[x] = a[y]
        a["ao"], a["po"] = a["acc"], a["pos"]
        assert evict(ds4a_lib, a) == ARG, (x, y)
    a = dict(AT, lo=AT["len"], next=AT["len"])          # the length in place is not the next position
    assert evict(ds4a_lib, a) == ARG


def prefix(ds4a, a):
    L = ds4a.lib()
    return L.ds4a_attn_prefix(cache(ds4a, a), a["q"], N, H, a["n"], a["parent"], a["start"], a["shared"], G, ctypes.c_float(0.1), a["out"],
                              a["lse"], a["ws"], L.ds4a_attn_prefix_workspace_bytes(B, N, H, D, G), None)


def test_prefix_outputs_overlap_nothing(ds4a_lib):
    BYTES["ws"] = ds4a_lib.lib().ds4a_attn_prefix_workspace_bytes(B, N, H, D, G)
    assert BYTES["ws"] < STEP
    refused(ds4a_lib, prefix, [(o, r) for o in ("out", "lse") for r in
                               ("q", "n", "parent", "start", "shared", "len", "table", "pk", "pv", "ws", "out" if o == "lse" else "lse")])
    for other in ("q", "n", "parent", "start", "shared", "len", "table", "pk", "pv"):
        assert prefix(ds4a_lib, dict(AT, ws=AT[other])) == ARG, other


def weights(ds4a, a):
    return ds4a.lib().ds4a_attn_weights(cache(ds4a, a), a["q"], N, H, a["n"], a["lse"], ctypes.c_float(0.1), ctypes.c_float(1.0), a["acc"],
                                        SLOTS, None)


def test_weights_sums_overlap_nothing(ds4a_lib):
    refused(ds4a_lib, weights, [("acc", r) for r in ("q", "lse", "n", "len", "table", "pk", "pv")])


def append(ds4a, a):
    return ds4a.lib().ds4a_paged_append_norm(cache(ds4a, a), a["k"], a["v"], N, a["n"], a["parent"], a["kw"], a["qw"], ctypes.c_float(1e-6),
                                             a["inv"], 64, 64, 1, a["q"], H, a["qo"], a["pos0"], a["sp"], SLOTS, None)


def test_append_norm_outputs_overlap_nothing(ds4a_lib):
    rest = ("k", "v", "n", "parent", "kw", "qw", "inv", "pos0", "len", "table", "pk", "pv")
    refused(ds4a_lib, append, [(o, r) for o in ("qo", "sp") for r in rest + ("sp" if o == "qo" else "qo",)] + [("sp", "q")])
    refused(ds4a_lib, append, [("sp", "q"), ("sp", "k")], qo=AT["q"])           # queries in place


@pytest.mark.parametrize("eps,code", [(float(np.finfo(np.float32).max), 0), (3.4014e38, 0), (float(np.float32(1e-45)), 0), (float("inf"), ARG),
                                      (float("nan"), ARG), (0.0, ARG)])
def test_append_norm_takes_every_finite_eps(ds4a_lib, eps, code):
    """Without sessions the call ends behind its checks."""
    none = kv(ds4a_lib, B=0, k=None, v=None, table=None, len=None)
    assert ds4a_lib.lib().ds4a_paged_append_norm(none, FAKE, FAKE, 1, FAKE, None, None, None, ctypes.c_float(eps), None, 0, 0, 1, None, 0, None,
                                                 None, None, 0, None) == code


@pytest.mark.parametrize("name", ["budget", "n_sink", "n_recent"])
@pytest.mark.parametrize("x", [(1 << 32) + 8, 1 << 31, -(1 << 31) - 1, 1 << 63])
def test_evict_counts_are_not_cut_to_32_bits(ds4a_lib, name, x):
    """A budget of 2^32 + 8 is not one of 8."""
    desc = ds4a_lib.PagedKVDesc(B=1, D=64, page=16, max_pages=3, n_pages=4)
    desc.tensors, desc.device = (), 0
    f, n = torch.zeros(1, 40), torch.zeros(1, dtype=torch.int64)
    counts = {**dict(budget=10, n_sink=0, n_recent=0), name: x}
    for call in (ds4a_lib.ds4a_evict, lambda *a: ds4a_lib.bind("ds4a_evict", *a)):
        with pytest.raises(ValueError, match=f"evict: {name} {x} does not fit"):
            call(desc, f, f, n, counts["budget"], counts["n_sink"], counts["n_recent"], f, f, n, None)
