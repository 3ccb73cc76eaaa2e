"""Caches held to a budget of tokens on the GPU: the normed append, attention weights and eviction,
each against its definition in 64 bits.  What a call must not read is NaN."""
import math

import numpy as np
import pytest
import torch

import budget_ref as E
import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_tree import Cache, dev, no_error

pytestmark = pytest.mark.gpu


def last_error():
    torch.cuda.synchronize()
    return ds4a.ds4a_last_device_error()


# ---- append with norms -------------------------------------------------------------------------

def check_append(rng, lens, n, N, H, D, page, rot, off, inter, tree, weights=True, ahead=True, in_place=False, mag=1.0,
                 eps=1e-6):
    c = Cache(rng, lens, n, D, page, N)
    B, S = c.B, c.mp * page + 3
    k = (mag * rng.standard_normal((B, N, D))).astype(np.float16)
    v = rng.standard_normal((B, N, D)).astype(np.float16)
    q = (mag * rng.standard_normal((B, N, H, D))).astype(np.float16) if H else None
    kw, qw = ((1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if weights else None for _ in range(2))
    par = R.random_parents(rng, B, N) if tree else None
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    pos0 = (np.array(lens) + rng.integers(0, 1 << 20, B)).astype(np.int64) if ahead else None
    kv = c.upload()
    dq = dev(q) if H else None
    dqo = (dq if in_place else torch.full_like(dq, 7.0)) if H else None
    sp = torch.full((B, S), -7, dtype=torch.int32, device="cuda")
    ds4a.ds4a_paged_append_norm(kv, dev(k), dev(v), c.dn, dev(kw) if weights else None, dev(qw) if weights else None, eps,
                                dev(par) if tree else None, dev(inv) if rot else None, off, inter, dq, dqo,
                                dev(pos0) if ahead else None, sp)
    no_error()
    gk, gv = c.dk.cpu().numpy().reshape(-1, D), c.dv.cpu().numpy().reshape(-1, D)
    ek, ev = c.k.astype(np.float64), c.v.copy()
    eq = (q.astype(np.float64) if in_place else np.full(q.shape, 7.0)) if H else None
    esp = np.full((B, S), -7, np.int32)
    for s in range(B):
        paths = R.paths_of(par[s], n[s]) if tree else None
        for i in range(n[s]):
            pos = (pos0[s] if ahead else lens[s]) + (len(paths[i]) - 1 if tree else i)
            r = c.rows(s, [lens[s] + i])[0]
            ek[r], ev[r] = R.rotate(E.norm(k[s, i].astype(np.float64), kw, eps), pos, inv, off, inter), v[s, i]
            esp[s, lens[s] + i] = pos
            if H:
                eq[s, i] = R.rotate(E.norm(q[s, i].astype(np.float64), qw, eps), pos, inv, off, inter)
    assert np.array_equal(gv, ev, equal_nan=True)
    assert np.array_equal(sp.cpu().numpy(), esp)
    # One rounding to 16 bits (2^-11 of the value, 2^-25 where it is tiny), and binary32 arithmetic on values of at most
    # amp: 22 roundings of the sum of squares halved by the root, the root's 2^-22 and two products (2^-19 in all); the
    # rotation as in the append without norms (the angle 2^-23, sine and cosine 2^-22, products and their sum) of
    # at most |x1| + |x2|.
    both = [ek] + ([eq] if H else [])
    amp = max(np.nanmax(np.abs(x)) for x in both)
    for got, want in zip((gk, dqo.cpu().numpy() if H else None), both):
        nan = np.isnan(want)
        assert np.array_equal(np.isnan(got), nan)
        err = np.abs(got.astype(np.float64) - want)[~nan]
        tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2 * amp * (2.0 ** -19 + 2.0 ** -20))[~nan]
        assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("lens,n,N,H,D,page,rot,off,inter,tree", [
    ([0], [1], 1, 8, 128, 16, 128, 0, True, False),
    ([5], [1], 1, 64, 128, 64, 64, 64, True, False),
    ([100, 0, 63, 17], [5, 0, 7, 1], 7, 8, 64, 48, 32, 16, False, True),
    ([3, 250], [64, 33], 64, 16, 128, 16, 16, 8, True, True),
    ([0, 9], [700, 331], 700, 0, 128, 128, 96, 32, False, False),
    ([1000], [300], 300, 24, 64, 80, 64, 0, True, False),
    ([31], [9], 9, 40, 128, 32, 0, 0, True, True),
])
def test_append_norms_rotates_and_places(lens, n, N, H, D, page, rot, off, inter, tree):
    check_append(np.random.default_rng(N), lens, n, N, H, D, page, rot, off, inter, tree)


@pytest.mark.parametrize("mag,eps", [(1e-3, 1e-6), (2000.0, 1e-5), (1e-6, 1e-12)])
def test_append_norm_of_small_and_large_rows(mag, eps):
    check_append(np.random.default_rng(2), [7, 40], [3, 5], 5, 8, 64, 16, 64, 0, False, False, mag=mag, eps=eps)


def test_append_norm_without_weights_in_place_at_slots():
    check_append(np.random.default_rng(3), [77, 12], [9, 4], 9, 64, 128, 16, 64, 64, True, True, weights=False, ahead=False,
                 in_place=True)


def test_append_norm_is_the_append_when_rows_are_of_norm_one():
    """Rows of +-1 have mean(x^2) = 1: with eps far below 2^-24 the norm changes nothing, and the bits are the append's."""
    rng = np.random.default_rng(4)
    c, d = (Cache(np.random.default_rng(5), [30, 7], [6, 3], 128, 16, 6) for _ in range(2))
    k, v = (rng.choice([-1.0, 1.0], (2, 6, 128)).astype(np.float16) for _ in range(2))
    q = rng.choice([-1.0, 1.0], (2, 6, 16, 128)).astype(np.float16)
    inv = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    qa, qb = torch.zeros(2, 6, 16, 128, dtype=torch.float16, device="cuda"), torch.zeros(2, 6, 16, 128, dtype=torch.float16, device="cuda")
    ds4a.ds4a_paged_append(c.upload(), dev(k), dev(v), c.dn, None, inv, 64, True, dev(q), qa)
    ds4a.ds4a_paged_append_norm(d.upload(), dev(k), dev(v), d.dn, None, None, 1e-20, None, inv, 64, True, dev(q), qb)
    no_error()
    assert torch.equal(qa, qb)
    assert torch.equal(c.dk.view(torch.int16), d.dk.view(torch.int16)) and torch.equal(c.dv.view(torch.int16), d.dv.view(torch.int16))


def test_append_norm_leaves_bad_sessions_alone():
    rng = np.random.default_rng(6)
    for what, code in (("pos0", 7), ("far", 7), ("slots", 2), ("page", 7)):
        c = Cache(rng, [20, 33], [4, 4], 64, 16, 4)
        if what == "page":
            c.table[0, 1] = c.n_pages
        kv = c.upload()
        k = dev(rng.standard_normal((2, 4, 64)).astype(np.float16))
        q = dev(rng.standard_normal((2, 4, 8, 64)).astype(np.float16))
        out = torch.full_like(q, 7.0)
        sp = torch.full((2, 23 if what == "slots" else 40), -7, dtype=torch.int32, device="cuda")
        pos0 = {"pos0": [-1, 50], "far": [(1 << 31) - 4, 50]}.get(what, [60, 50])
        before = c.dk.clone()
        ds4a.ds4a_paged_append_norm(kv, k, k, c.dn, None, None, 1e-6, None, None, 0, True, q, out,
                                    torch.tensor(pos0, device="cuda"), sp)
        assert last_error() == code, what
        r0, r1 = c.rows(0, [20, 21, 22, 23]) if what != "page" else None, c.rows(1, [33, 34, 35, 36])
        flat, old = c.dk.view(-1, 64).cpu(), before.view(-1, 64).cpu()
        if r0 is not None:
            assert torch.equal(flat[r0].view(torch.int16), old[r0].view(torch.int16)), what
        assert (sp[0] == -7).all(), what
        if what != "page":
            assert (out[0] == 7).all()
        if what == "slots":                 # 33 + 4 tokens pass 23 slots too
            assert (out == 7).all()
        else:
            assert torch.isfinite(flat[r1]).all() and sp[1, 33:37].tolist() == [50, 51, 52, 53]


# ---- attention weights --------------------------------------------------------------------------

def weights_setup(rng, lens, n, N, H, D, page, scale, slots_extra=5, mag=1.0):
    c = Cache(rng, lens, n, D, page, N)
    c.draft()
    B, S = c.B, c.mp * page + slots_extra
    q = (mag * rng.standard_normal((B, N, H, D))).astype(np.float16)
    lse = np.full((B, N, H), np.nan, np.float32)
    acc = np.full((B, S), np.nan, np.float32)
    for s in range(B):
        q[s, n[s]:] = np.nan
        acc[s, :lens[s]] = rng.random(lens[s]).astype(np.float32)
        T = lens[s] + n[s]
        if n[s]:
            see = np.arange(T) <= lens[s] + np.arange(n[s])[:, None]
            lse[s, :n[s]] = E.rows_lse(q[s, :n[s]], c.k[c.rows(s, range(T))], scale, see)[1]
    return c, q, lse, acc


def check_weights(c, q, lse, acc, got, scale, decay, lens, n):
    want, tol = acc.astype(np.float64), np.zeros(acc.shape)
    for s in range(c.B):
        T = lens[s] + n[s]
        if not n[s]:
            continue
        add, t = E.weights(q[s, :n[s]], c.k[c.rows(s, range(T))], scale, lse[s, :n[s]], lens[s])
        old = np.where(np.arange(T) < lens[s], decay * acc[s, :T].astype(np.float64), 0.0) if decay else np.zeros(T)
        want[s, :T], tol[s, :T] = old + add, t + 2.0 ** -23 * np.abs(old) + 2.0 ** -24 * np.abs(old + add)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    err = np.abs(got.astype(np.float64) - want)[~nan]
    assert (err <= tol[~nan]).all(), (err / np.maximum(tol[~nan], 1e-300)).max()


@pytest.mark.parametrize("lens,n,N,H,D,page,decay", [
    ([0], [1], 1, 8, 64, 16, 1.0),                                  # the token itself and nothing before
    ([127], [1], 1, 64, 128, 64, 1.0),                              # a tile to its last key
    ([128], [1], 1, 64, 128, 128, 0.5),                             # one key into the next
    ([100, 0, 640, 17], [3, 2, 1, 0], 3, 8, 128, 16, 1.0),          # a session without new tokens
    ([300, 5], [33, 20], 33, 24, 64, 48, 0.25),                     # many chunks, rows that end inside one
    ([200], [64], 64, 64, 128, 256, 1.0),                           # 4096 rows
    ([2000, 1], [1, 1], 1, 72 - 8, 128, 80, 0.0),
    ([5000], [2], 2, 40, 64, 32, 1.0),
    ([90 + 37 * i for i in range(45)], [1 + i % 2 for i in range(45)], 2, 16, 64, 16, 1.0),   # two walks of sessions
    ([40000], [1], 1, 8, 64, 1024, 1.0),                            # more than two tiles an SM
    ([3 + 17 * i % 601 for i in range(256)], [1 - i % 5 // 4 for i in range(256)], 1, 8, 64, 16, 1.0),   # as many as are looked up at once
    ([3 + 17 * i % 601 for i in range(300)], [i % 3 for i in range(300)], 2, 8, 64, 16, 1.0),            # and more
])
def test_weights(lens, n, N, H, D, page, decay):
    scale = 1 / math.sqrt(D)
    c, q, lse, acc = weights_setup(np.random.default_rng(N + len(lens)), lens, n, N, H, D, page, scale)
    kv = c.upload()
    da = dev(acc)
    ds4a.ds4a_attn_weights(kv, dev(q), c.dn, dev(lse), scale, decay, da)
    no_error()
    check_weights(c, q, lse, acc, da.cpu().numpy(), scale, decay, lens, n)


def test_weights_of_a_row_sum_to_one():
    """With exact sums every row gives 1 in all: heads x tokens over a session."""
    rng = np.random.default_rng(8)
    c, q, lse, acc = weights_setup(rng, [700], [5], 5, 64, 128, 64, 0.3)
    da = dev(np.zeros_like(acc))
    ds4a.ds4a_attn_weights(c.upload(), dev(q), c.dn, dev(lse), 0.3, 1.0, da)
    no_error()
    # each weight is off by E.weights' tolerance: scores up to 0.3 * 128 * 4 = 154 in mass
    assert abs(da.sum(dtype=torch.float64).item() - 320) < 320 * (2 * (256 * 154 + 6 * 60) * 2.0 ** -24 + 2.0 ** -20)


def test_weights_decay_zero_does_not_read_and_rows_without_keys_add_nothing():
    rng = np.random.default_rng(9)
    c, q, lse, acc = weights_setup(rng, [150], [3], 3, 8, 64, 16, 0.125)
    acc[:] = np.nan
    lse[0, 1, :] = -np.inf
    da = dev(acc)
    ds4a.ds4a_attn_weights(c.upload(), dev(q), c.dn, dev(lse), 0.125, 0.0, da)
    no_error()
    check_weights(c, q, lse, acc, da.cpu().numpy(), 0.125, 0.0, [150], [3])


def test_weights_same_bits_whatever_shares_the_call():
    """A session's sums do not depend on what else is in the call."""
    rng = np.random.default_rng(10)
    lens, n = [300, 1000, 77], [2, 3, 1]
    c, q, lse, acc = weights_setup(rng, lens, n, 3, 16, 128, 32, 0.1)
    kv = c.upload()
    both = dev(acc)
    ds4a.ds4a_attn_weights(kv, dev(q), c.dn, dev(lse), 0.1, 1.0, both)
    for s in range(3):
        one = dev(acc[s:s + 1])
        kv1 = ds4a.paged_kv_desc(c.dk, c.dv, c.dtab[s:s + 1].contiguous(), c.dlen[s:s + 1].contiguous())
        ds4a.ds4a_attn_weights(kv1, dev(q[s:s + 1]), c.dn[s:s + 1].contiguous(), dev(lse[s:s + 1]), 0.1, 1.0, one)
        no_error()
        assert torch.equal(one.view(torch.int32), both[s:s + 1].view(torch.int32))


def test_weights_bad_sessions_and_pages():
    rng = np.random.default_rng(11)
    lens, n = [100, 60, 50], [2, 2, 2]
    c, q, lse, acc = weights_setup(rng, lens, n, 2, 8, 64, 16, 0.125)
    good = acc.copy()
    c.table[0, 3] = -5                      # slots 48 .. 63 of session 0
    kv = c.upload()
    c.dn[1] = 3
    da = dev(acc)
    ds4a.ds4a_attn_weights(kv, dev(q), c.dn, dev(lse), 0.125, 1.0, da)
    assert last_error() == 7
    got = da.cpu().numpy()
    assert np.array_equal(got[1], acc[1], equal_nan=True)
    assert np.array_equal(got[0, 48:64], acc[0, 48:64])
    c.table[0, 3] = 0
    rest = np.r_[0:48, 64:102]
    add, t = E.weights(q[0, :2], c.k[c.rows(0, range(102))], 0.125, lse[0, :2], 100)
    want = np.where(np.arange(102) < 100, np.nan_to_num(good[0, :102]), 0) + add
    assert (np.abs(got[0, :102] - want)[rest] <= (t + 2.0 ** -22 * np.abs(want))[rest]).all()
    # more tokens than acc has entries for: left alone, the others not
    c, q, lse, acc = weights_setup(rng, lens, n, 2, 8, 64, 16, 0.125)
    short = dev(np.ascontiguousarray(acc[:, :101]))
    before = short.clone()
    ds4a.ds4a_attn_weights(c.upload(), dev(q), c.dn, dev(lse), 0.125, 1.0, short)
    assert last_error() == 2
    assert torch.equal(short[0].view(torch.int32), before[0].view(torch.int32))
    for s in (1, 2):
        assert not torch.equal(short[s, :lens[s]], before[s, :lens[s]])


# ---- eviction --------------------------------------------------------------------------------------

def check_evict(rng, lens, budget, sink, recent, D=64, page=16, acc=None, extra=0, in_place=False, pos=None):
    c = Cache(rng, lens, [0] * len(lens), D, page, 0)
    B, S = c.B, max(lens) + extra
    if acc is None:
        acc = np.exp(2 * rng.standard_normal((B, S))).astype(np.float32)
        acc[rng.random((B, S)) < 0.1] = 0
    acc = acc.copy()
    pos = np.stack([rng.permutation(S + 50)[:S] for _ in range(B)]).astype(np.int32) if pos is None else pos
    nxt = np.array([pos[s, :lens[s]].max() + 1 if lens[s] else 0 for s in range(B)], np.int64)
    for s in range(B):
        acc[s, lens[s]:], pos[s, lens[s]:] = np.nan, -9
    kv = c.upload()
    da, dp = dev(acc), dev(pos)
    ao, po = (da, dp) if in_place else (torch.full_like(da, 5.0), torch.full_like(dp, 6))
    lo = c.dlen if in_place else torch.full_like(c.dlen, -1)
    ws = torch.full((ds4a.ds4a_evict_workspace_bytes(B, S, budget),), 255, dtype=torch.uint8, device="cuda")
    ds4a.ds4a_evict(kv, da, dp, dev(nxt), budget, sink, recent, ao, po, lo, ws)
    no_error()
    ek, ev = c.k.copy(), c.v.copy()
    ea, ep = (acc.copy(), pos.copy()) if in_place else (np.full(acc.shape, 5, np.float32), np.full(pos.shape, 6, np.int32))
    for s in range(B):
        place, holes = E.evict(acc[s], pos[s], int(nxt[s]), lens[s], budget, sink, recent)
        ea[s, :len(place)], ep[s, :len(place)] = acc[s, place], pos[s, place]
        if len(holes):
            to, fr = c.rows(s, holes), c.rows(s, place[holes])
            ek[to], ev[to] = c.k[fr], c.v[fr]
    assert lo.tolist() == [min(n, budget) for n in lens]
    assert np.array_equal(po.cpu().numpy(), ep)
    assert np.array_equal(ao.cpu().numpy(), ea, equal_nan=True)
    for got, want in ((c.dk, ek), (c.dv, ev)):
        assert np.array_equal(got.cpu().numpy().reshape(-1, D).view(np.int16), want.view(np.int16))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget,sink,recent,D,page", [
    ([1], 1, 0, 0, 64, 16), ([2], 1, 0, 0, 128, 16), ([5, 0, 3, 4], 4, 1, 1, 64, 16), ([100, 64, 65, 30], 64, 4, 16, 128, 48),
    ([513, 511, 512], 200, 0, 0, 64, 32), ([4160], 4096, 4, 256, 128, 64), ([5000, 8000], 4097, 0, 4097, 64, 80),
    ([9000, 8193, 17, 4096], 3000, 3000, 0, 64, 16), ([20000], 777, 5, 50, 64, 16), ([40000, 39999], 35000, 4, 1000, 64, 128),
    ([70 + 13 * i for i in range(50)], 100, 2, 9, 64, 16),
])
def test_evict(lens, budget, sink, recent, D, page, in_place):
    check_evict(np.random.default_rng(budget), lens, budget, sink, recent, D, page, extra=len(lens) % 3, in_place=in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "special", "low bits", "negative"])
@pytest.mark.parametrize("ln", [300, 9001, 33000])
def test_evict_ties_and_special_sums(ln, kind):
    rng = np.random.default_rng(ln)
    a = np.ones((1, ln), np.float32)
    if kind == "zeros":
        a = rng.choice(np.array([0.0, -0.0], np.float32), (1, ln))
    if kind == "two":
        a = rng.choice(np.array([1.0, 2.0], np.float32), (1, ln))
    if kind == "special":
        a = rng.choice(np.array([np.nan, np.inf, -np.inf, 0, 1e-45, 3e38, -np.nan], np.float32), (1, ln))
    if kind == "low bits":                      # differ in the last ten bits alone
        a = (np.float32(1).view(np.uint32) + rng.integers(0, 700, (1, ln)).astype(np.uint32)).view(np.float32)
    if kind == "negative":
        a = rng.standard_normal((1, ln)).astype(np.float32)
    check_evict(rng, [ln], ln // 2, 3, 40, acc=a)


def test_evict_positions_that_repeat_keep_the_budget():
    """Positions that all count as always kept: the lower slots stay, exactly `budget` of them."""
    check_evict(np.random.default_rng(1), [300], 100, 100, 0, pos=np.zeros((1, 300), np.int32))


def test_evict_longer_than_shared_memory():
    check_evict(np.random.default_rng(2), [400001, 330000], 200000, 4, 1000, page=4096)


def test_evict_the_longest_that_shared_memory_holds():
    check_evict(np.random.default_rng(5), [327680, 300000], 250000, 64, 100, page=1024)


def test_evict_leaves_bad_sessions_alone():
    rng = np.random.default_rng(3)
    S, budget = 100, 40
    for what, code in (("len", 7), ("slots", 2), ("pages", 2), ("page", 7)):
        c = Cache(rng, [90, 80], [0, 0], 64, 16, 0)
        if what == "page":
            c.table[0, 4] = c.n_pages + 1
        kv = c.upload()
        if what in ("len", "slots", "pages"):
            c.dlen[0] = {"len": -1, "slots": S + 1, "pages": c.mp * 16 + 1}[what]
        acc, pos = dev(rng.random((2, S)).astype(np.float32)), torch.arange(S, device="cuda", dtype=torch.int32).repeat(2, 1).contiguous()
        ao, po, lo = torch.full_like(acc, 5), torch.full_like(pos, 6), torch.full_like(c.dlen, -4)
        ws = torch.zeros(ds4a.ds4a_evict_workspace_bytes(2, S, budget), dtype=torch.uint8, device="cuda")
        before = c.dk.clone()
        ds4a.ds4a_evict(kv, acc, pos, torch.tensor([90, 80], device="cuda"), budget, 2, 5, ao, po, lo, ws)
        assert last_error() == code, what
        assert lo.tolist() == [-4, budget] and (ao[0] == 5).all() and (po[0] == 6).all(), what
        r = np.unique(c.table[1])
        same = (c.dk.view(torch.int16) == before.view(torch.int16)).flatten(1).all(1).cpu().numpy()
        assert same[np.setdiff1d(np.arange(c.n_pages), r)].all() and not same[r].all(), what
