"""Attention of sessions that share prefixes, against its definition in 64 bits.  Page entries that a call
must not read are invalid, slots that it must not attend are NaN."""
import math

import numpy as np
import pytest
import torch

import budget_ref as E
import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_tree import Cache, dev, no_error

pytestmark = pytest.mark.gpu


class Shared(Cache):
    """Sessions whose groups share prefixes: a member's entries of whole prefix pages are invalid, and its copy of
    the page that the prefix ends in is NaN before its own first slot."""

    def __init__(self, rng, lens, n, start, shared, D, page, N, room=0):
        super().__init__(rng, lens, n, D, page, N + room)
        self.N = N
        self.draft()
        self.start, self.shared = np.array(start, np.int32), np.array(shared, np.int64)
        self.lead = {s: (a, m) for a, b, m in zip(start[:-1], start[1:], shared) for s in range(a + 1, b)}
        for s, (a, m) in self.lead.items():
            if m % page:
                r = self.rows(s, range(m - m % page, m))
                self.k[r] = self.v[r] = np.nan
            self.table[s, :m // page] = -1

    def key_rows(self, s, slots):
        a, m = self.lead.get(s, (s, 0))
        t = np.asarray(list(slots), np.int64)
        own, lead = self.table[s], self.table[a]
        pg = np.where(t < m, lead[t // self.page], own[t // self.page]).astype(np.int64)
        return pg * self.page + t % self.page


def reference(c, q, par, scale):
    B, N, H, D = q.shape
    out, tol = np.full(q.shape, 7.0), np.zeros(q.shape)
    lse, ltol = np.full((B, N, H), 7.0), np.zeros((B, N, H))
    for s in range(B):
        if not c.n[s]:
            continue
        base = c.key_rows(s, range(c.lens[s]))
        for i, path in enumerate(R.paths_of(par[s], c.n[s])):
            rows = np.concatenate([base, c.key_rows(s, [c.lens[s] + j for j in path])])
            k, v = c.k[rows].astype(np.float64), c.v[rows].astype(np.float64)
            out[s, i], tol[s, i] = R.attend(q[s, i], k, v, scale)
            lse[s, i] = E.rows_lse(q[s, i][None], k, scale, np.ones((1, len(rows)), bool))[1][0]
            # scores as in R.attend; a power of two 2^-22, the sum 256 * 2^-24, the reference, the logarithm and the
            # change of base 2^-21 of |lse| + 24 (a sum of up to 2^15 * 2^9 in powers of two)
            ds = (2 * D * 2.0 ** -24 * scale * (np.abs(q[s, i].astype(np.float64)) @ np.abs(k).T)).max(1)
            ltol[s, i] = 2 * ds + 2.0 ** -22 + 2.0 ** -16 + 2.0 ** -21 * (np.abs(lse[s, i]) + 24)
    return out, tol, lse, ltol


def run(c, q, par, scale, with_lse=True, groups=True):
    B, N, H, D = q.shape
    kv = c.upload()
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    lse = torch.full((B, N, H), 7.0, device="cuda") if with_lse else None
    G = len(c.shared)
    ws = torch.full((ds4a.ds4a_attn_prefix_workspace_bytes(B, N, H, D, G),), 255, dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_prefix(kv, dev(q), c.dn, None if par is None else dev(par), dev(c.start) if G else None,
                          dev(c.shared) if G else None, scale, out, lse, ws)
    torch.cuda.synchronize()
    return out.cpu().numpy(), lse.cpu().numpy() if with_lse else None


def check(rng, lens, n, N, H, D, page, start, shared, kind="tree", scale=None, room=0, mag=1.0):
    c = Shared(rng, lens, n, start, shared, D, page, N, room)
    q = (mag * rng.standard_normal((c.B, N, H, D))).astype(np.float16)
    for s in range(c.B):
        q[s, n[s]:] = np.nan
    par = R.random_parents(rng, c.B, N, kind)
    scale = scale or 1 / math.sqrt(D)
    out, lse = run(c, q, None if kind == "chain" else par, scale)
    no_error()
    want, tol, wl, lt = reference(c, q, par, scale)
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    err = np.abs(out.astype(np.float64) - want)
    assert (err <= tol).all(), (err - tol).max()
    err = np.abs(lse.astype(np.float64) - wl)
    assert (err <= lt).all(), (err - lt).max()


@pytest.mark.parametrize("lens,n,N,H,D,page,start,shared,kind", [
    ([301, 300, 310, 355], [1, 1, 1, 1], 1, 64, 128, 16, [0, 4], [300], "chain"),          # one token each over a prompt
    ([64, 64], [1, 1], 1, 8, 64, 16, [0, 2], [64], "chain"),                               # nothing of their own, whole pages
    ([7, 9, 5], [2, 1, 2], 2, 16, 64, 16, [0, 3], [5], "tree"),                            # a prefix inside one run
    ([500, 40, 430, 0, 460, 33], [3, 2, 3, 1, 0, 3], 3, 24, 128, 48, [2, 5, 5, 6], [0, 9, 33], "tree"),   # shared 0, empty group
    ([500, 40, 430, 433, 460, 33], [3, 2, 3, 1, 0, 3], 3, 24, 128, 48, [2, 2, 5], [100, 429], "tree"),   # sessions outside groups
    ([1000 + 13 * i for i in range(20)], [1] * 20, 1, 64, 64, 128, [0, 20], [1000], "chain"),   # 1280 rows share
    ([200 + i for i in range(45)], [1 + i % 2 for i in range(45)], 2, 8, 64, 16, [1, 7, 13, 44], [200, 203, 77], "tree"),
    ([130, 150, 140], [64, 33, 64], 64, 64, 64, 32, [0, 3], [129], "tree"),                # 64-node trees
    ([9000, 9100], [1, 2], 2, 8, 128, 64, [0, 2], [8999], "chain"),                        # few rows over many tiles
    ([5000, 5100, 5003, 5001, 5050, 5000, 5010, 5090], [8] * 8, 8, 64, 128, 64, [0, 8], [4990], "tree"),   # two row blocks
    ([300, 17], [5, 4], 5, 40, 64, 16, [0], [], "tree"),                                   # nothing shared
    ([4000], [1], 1, 64, 128, 80, [0, 1], [4000], "chain"),                                # a group of one
    ([60 + i % 50 for i in range(250)], [1 + i % 2 for i in range(250)], 2, 8, 64, 16, [0, 9, 9, 40, 100, 100, 249], [60, 7, 33, 1, 5, 48], "tree"),   # 256 entries
    ([60 + i % 50 for i in range(290)], [i % 3 for i in range(290)], 2, 8, 64, 16, [3, 9, 9, 40, 100, 280], [60, 7, 33, 59, 16], "tree"),   # and more
])
def test_prefix(lens, n, N, H, D, page, start, shared, kind):
    check(np.random.default_rng(len(lens) + N), lens, n, N, H, D, page, start, shared, kind)


def test_prefix_large_scores():
    """Scores up to some hundreds: references move, weights underflow."""
    check(np.random.default_rng(1), [600, 700, 650], [2, 3, 1], 3, 16, 64, 16, [0, 3], [590], mag=6.0, scale=0.5)


def test_prefix_without_lse_and_rows_behind_the_last_node():
    rng = np.random.default_rng(2)
    c = Shared(rng, [100, 90, 95], [3, 0, 2], [0, 3], [80], 64, 16, 4)
    q = rng.standard_normal((3, 4, 8, 64)).astype(np.float16)
    par = R.random_parents(rng, 3, 4)
    a, _ = run(c, q, par, 0.125, with_lse=False)
    b, lse = run(c, q, par, 0.125)
    no_error()
    assert np.array_equal(a, b)
    for s in range(3):
        assert (b[s, c.n[s]:] == 7).all() and (lse[s, c.n[s]:] == 7).all()


def test_prefix_is_the_tree_call_over_the_same_tokens():
    """Against ds4a_attn_tree with the whole prefix in every session's pages: both within tolerance of the exact one."""
    rng = np.random.default_rng(3)
    lens, n, N, H, D, page, scale = [700, 730, 690], [4, 3, 4], 4, 16, 128, 16, 0.1
    c = Shared(rng, lens, n, [0, 3], [680], D, page, N)
    q = rng.standard_normal((3, N, H, D)).astype(np.float16)
    par = R.random_parents(rng, 3, N)
    out, _ = run(c, q, par, scale)
    for s, (a, m) in c.lead.items():        # the prefix in the members' own pages too
        c.table[s, :m // page] = c.table[a, :m // page]
        c.k[c.rows(s, range(m - m % page, m))] = c.k[c.rows(a, range(m - m % page, m))]
        c.v[c.rows(s, range(m - m % page, m))] = c.v[c.rows(a, range(m - m % page, m))]
    kv = c.upload()
    other = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(3, N, H, D), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_tree(kv, dev(q), c.dn, dev(par), 1 << 40, None, None, 0, None, scale, other, ws)
    no_error()
    tol = reference(c, q, par, scale)[1]
    assert (np.abs(out.astype(np.float64) - other.cpu().numpy()) <= 2 * tol).all()


def test_prefix_values_that_are_not_finite():
    """An infinite value in the prefix reaches every row of the group and no other; a value of a draft's branch only
    that branch."""
    rng = np.random.default_rng(4)
    c = Shared(rng, [200, 210, 190], [3, 3, 3], [0, 2], [180], 64, 16, 3)
    par = np.tile(np.array([-1, 0, 0], np.int32), (3, 1))
    c.v[c.key_rows(1, [50]), 7] = np.inf
    c.v[c.rows(0, [201]), 9] = -np.inf            # node 1 of session 0
    q = rng.standard_normal((3, 3, 8, 64)).astype(np.float16)
    out, lse = run(c, q, par, 0.05)
    no_error()
    assert (out[:2, :, :, 7] == np.inf).all() and np.isfinite(out[2]).all() and np.isfinite(lse).all()
    assert (out[0, 1, :, 9] == -np.inf).all() and np.isfinite(out[0, [0, 2], :, 9]).all() and np.isfinite(out[1, :, :, 9]).all()


def test_prefix_ends_beside_another_sessions_tokens():
    """The first session's own tokens sit in the same page and run as the prefix's end; their NaN reach that session alone."""
    rng = np.random.default_rng(9)
    c = Shared(rng, [85, 84, 90], [1, 1, 1], [0, 3], [83], 64, 16, 1)
    r = c.rows(0, [83, 84, 85])
    c.k[r] = c.v[r] = np.nan
    q = rng.standard_normal((3, 1, 8, 64)).astype(np.float16)
    out, lse = run(c, q, None, 0.125)
    no_error()
    assert np.isnan(out[0]).all() and np.isnan(lse[0]).all()
    want, tol, wl, lt = reference(c, q, R.random_parents(rng, 3, 1), 0.125)
    for s in (1, 2):
        assert (np.abs(out[s].astype(np.float64) - want[s]) <= tol[s]).all() and (np.abs(lse[s] - wl[s]) <= lt[s]).all()


def test_prefix_scores_of_minus_infinity():
    rng = np.random.default_rng(5)
    c = Shared(rng, [40, 44], [1, 1], [0, 2], [40], 64, 16, 1)
    q = np.abs(rng.standard_normal((2, 1, 8, 64))).astype(np.float16) + np.float16(0.1)
    c.k[c.key_rows(0, range(40))] = -np.inf       # the whole prefix, and session 0's own token
    c.k[c.rows(0, [40])] = -np.inf
    out, lse = run(c, q, None, 0.125)
    no_error()
    assert np.isnan(out[0]).all() and (lse[0] == -np.inf).all()
    k, v = c.k[c.rows(1, range(40, 45))].astype(np.float64), c.v[c.rows(1, range(40, 45))].astype(np.float64)
    want, tol = R.attend(q[1, 0], k, v, 0.125)
    assert (np.abs(out[1, 0].astype(np.float64) - want) <= tol).all() and np.isfinite(lse[1]).all()


def error_of(c, q, par, scale):
    out, lse = run(c, q, par, scale)
    return ds4a.ds4a_last_device_error(), out, lse


def test_prefix_bad_groups_and_sessions():
    rng = np.random.default_rng(6)
    lens, n = [100, 120, 90, 80], [2, 2, 2, 2]
    q = rng.standard_normal((4, 2, 8, 64)).astype(np.float16)
    par = R.random_parents(rng, 4, 2)

    def fresh():
        return Shared(np.random.default_rng(7), lens, n, [0, 3], [85], 64, 16, 2)
    good, wl = run(fresh(), q, par, 0.125)
    no_error()
    many = Shared(rng, [20] * 300, [1] * 300, [0, 300], [18], 64, 16, 1)     # more entries than are looked up at once
    many.start = np.array([0, 301], np.int32)
    code, out, lse = error_of(many, rng.standard_normal((300, 1, 8, 64)).astype(np.float16), None, 0.125)
    assert code == 7 and (out == 7).all() and (lse == 7).all()
    for start in ([0, 5], [-1, 3], [2, 1]):
        c = fresh()
        c.start = np.array(start, np.int32)
        code, out, lse = error_of(c, q, par, 0.125)
        assert code == 7 and (out == 7).all() and (lse == 7).all(), start
    # a prefix that is longer than one session: that one alone; a negative one: the group
    for shared, left in ((95, [2]), (-1, [0, 1, 2])):
        c = fresh()
        c.shared = np.array([shared], np.int64)
        if shared < 0:
            c.lead = {}
        code, out, lse = error_of(c, q, par, 0.125)
        assert code == 7
        for s in range(4):
            assert ((out[s] == 7).all() and (lse[s] == 7).all()) == (s in left), (shared, s)
        assert np.array_equal(out[3], good[3])
    # a bad parent: that session
    c, bad = fresh(), par.copy()
    bad[1, 1] = 1
    code, out, lse = error_of(c, q, bad, 0.125)
    assert code == 7 and (out[1] == 7).all() and np.array_equal(out[[0, 2, 3]], good[[0, 2, 3]])
    # a page of the prefix outside the pool: its tokens are attended by nobody
    c = fresh()
    page0 = c.table[0, 1]
    c.table[0, 1] = c.n_pages
    code, out, lse = error_of(c, q, par, 0.125)
    assert code == 7
    c.table[0, 1] = page0
    for s in (0, 2):
        keys = [t for t in range(lens[s]) if not 16 <= t < 32]
        k, v = (x[c.key_rows(s, keys + [lens[s]])].astype(np.float64) for x in (c.k, c.v))
        want, tol = R.attend(q[s, 0], k, v, 0.125)
        assert (np.abs(out[s, 0].astype(np.float64) - want) <= tol).all()
    assert np.array_equal(out[3], good[3])


@pytest.mark.parametrize("B", [4, 60, 300])          # the walk, the table, more than the table holds
def test_prefix_and_weights_bad_counts(B):
    """Counts and lengths that do not fit leave their sessions alone, in both calls, and no other."""
    rng = np.random.default_rng(B)
    lens, n = [40 + i % 7 for i in range(B)], [1 + i % 2 for i in range(B)]
    q = rng.standard_normal((B, 2, 8, 64)).astype(np.float16)

    def call(spoil):
        c = Shared(np.random.default_rng(7), lens, n, [0, B - 1], [37], 64, 16, 2)
        for s, (first, m) in c.lead.items():    # the weights call reads the prefix through each session's own entries
            c.table[s, :m // 16] = c.table[first, :m // 16]
            c.k[c.rows(s, range(m - m % 16, m))] = c.k[c.rows(first, range(m - m % 16, m))]
            c.v[c.rows(s, range(m - m % 16, m))] = c.v[c.rows(first, range(m - m % 16, m))]
        kv = c.upload()
        spoil(c)
        out, lse = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda"), torch.full((B, 2, 8), 7.0, device="cuda")
        acc = torch.full((B, c.mp * 16), 3.0, device="cuda")
        ws = torch.zeros(ds4a.ds4a_attn_prefix_workspace_bytes(B, 2, 8, 64, 1), dtype=torch.uint8, device="cuda")
        ds4a.ds4a_attn_prefix(kv, dev(q), c.dn, None, dev(c.start), dev(c.shared), 0.125, out, lse, ws)
        torch.cuda.synchronize()
        code = ds4a.ds4a_last_device_error()
        ds4a.ds4a_attn_weights(kv, dev(q), c.dn, lse, 0.125, 1.0, acc)
        torch.cuda.synchronize()
        return code, ds4a.ds4a_last_device_error(), out.cpu(), lse.cpu(), acc.cpu()
    good = call(lambda c: None)
    assert good[:2] == (0, 0)

    def put(name, s, x):
        return lambda c: getattr(c, name).__setitem__(s, x)
    cap = Shared(np.random.default_rng(7), lens, n, [0, B - 1], [37], 64, 16, 2).mp * 16
    for what, s, code in ((put("dn", 1, -1), 1, 7), (put("dn", 2, 3), 2, 7), (put("dlen", B - 1, -5), B - 1, 7),
                          (put("dlen", 1, cap), 1, 2), (put("dlen", 2, (1 << 63) - 1), 2, 2)):
        got = call(what)
        assert got[:2] == (code, code)
        assert (got[2][s] == 7).all() and (got[3][s] == 7).all() and (got[4][s] == 3).all()
        keep = [i for i in range(B) if i != s]
        for x, y in zip(got[2:], good[2:]):
            assert torch.equal(x[keep], y[keep])


def test_prefix_captured_replays_with_other_groups():
    """A captured call with the groups, lengths and counts of another batch."""
    rng = np.random.default_rng(8)
    N, H, D, page = 2, 16, 64, 16
    batches = [Shared(rng, [300, 290, 310, 280], [2, 1, 2, 2], [0, 2, 4], [280, 270], D, page, N),
               Shared(rng, [296, 40, 200, 150], [1, 2, 0, 2], [1, 1, 4], [8, 30], D, page, N)]
    q = rng.standard_normal((4, N, H, D)).astype(np.float16)
    par = np.tile(np.array([-1, 0], np.int32), (4, 1))
    want = [run(c, q, None, 0.125) for c in batches]
    no_error()
    a, b = batches
    mp, pages = max(a.mp, b.mp), max(a.n_pages, b.n_pages)
    bufs = dict(k=torch.zeros(pages, page, D, dtype=torch.float16, device="cuda"), table=torch.full((4, mp), -1, dtype=torch.int32, device="cuda"),
                ln=torch.zeros(4, dtype=torch.int64, device="cuda"), n=torch.zeros(4, dtype=torch.int32, device="cuda"),
                start=torch.zeros(3, dtype=torch.int32, device="cuda"), shared=torch.zeros(2, dtype=torch.int64, device="cuda"))
    bufs["v"] = torch.zeros_like(bufs["k"])
    out = torch.zeros(4, N, H, D, dtype=torch.float16, device="cuda")
    lse = torch.zeros(4, N, H, device="cuda")
    dq = dev(q)
    ws = torch.zeros(ds4a.ds4a_attn_prefix_workspace_bytes(4, N, H, D, 2), dtype=torch.uint8, device="cuda")
    kv = ds4a.paged_kv_desc(bufs["k"], bufs["v"], bufs["table"], bufs["ln"])
    call = lambda: ds4a.ds4a_attn_prefix(kv, dq, bufs["n"], None, bufs["start"], bufs["shared"], 0.125, out, lse, ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for x in (0, 1, 0):
        c = batches[x]
        bufs["k"][:c.n_pages], bufs["v"][:c.n_pages] = c.dk, c.dv
        bufs["table"][:, :c.mp] = c.dtab
        for name, val in (("ln", c.dlen), ("n", c.dn), ("start", dev(c.start)), ("shared", dev(c.shared))):
            bufs[name].copy_(val)
        out.fill_(7)
        lse.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        no_error()
        assert np.array_equal(out.cpu().numpy(), want[x][0]) and np.array_equal(lse.cpu().numpy(), want[x][1])
