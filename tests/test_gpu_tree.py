"""The paged token cache and drafted-token trees on the GPU: each call against its
definition in 64 bits, and a draft checked and committed against token-by-token decode.

Everything that a call must not read is filled with NaN (pages of nobody, slots behind the
tokens, rows not complete), so a masked value that leaks shows."""
import math

import numpy as np
import pytest
import torch

import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a

pytestmark = pytest.mark.gpu

NAN16 = np.float16(np.nan)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Cache:
    """A paged cache of random tokens with NaN everywhere else."""

    def __init__(self, rng, lens, n, D=128, page=16, N=8, spare=3):
        self.rng, self.lens, self.n, self.D, self.page, self.N = rng, list(lens), list(n), D, page, N
        self.B = len(self.lens)
        self.mp = max((ln + N + page - 1) // page for ln in self.lens)
        self.n_pages = self.B * self.mp + spare
        self.table = rng.permutation(self.n_pages)[:self.B * self.mp].reshape(self.B, self.mp).astype(np.int32)
        self.k = np.full((self.n_pages * page, D), NAN16)
        self.v = np.full((self.n_pages * page, D), NAN16)
        for s in range(self.B):
            r = self.rows(s, range(self.lens[s]))
            self.k[r] = rng.standard_normal((len(r), D)).astype(np.float16)
            self.v[r] = rng.standard_normal((len(r), D)).astype(np.float16)

    def rows(self, s, slots):
        return R.slot_rows(self.table[s], self.page, list(slots))

    def draft(self):
        """Random drafted tokens into their slots."""
        for s in range(self.B):
            r = self.rows(s, range(self.lens[s], self.lens[s] + self.n[s]))
            self.k[r] = self.rng.standard_normal((len(r), self.D)).astype(np.float16)
            self.v[r] = self.rng.standard_normal((len(r), self.D)).astype(np.float16)

    def upload(self):
        self.dk, self.dv = dev(self.k.reshape(self.n_pages, self.page, self.D)), dev(self.v.reshape(self.n_pages, self.page, self.D))
        self.dlen, self.dn, self.dtab = dev(np.array(self.lens, np.int64)), dev(np.array(self.n, np.int32)), dev(self.table)
        return ds4a.paged_kv_desc(self.dk, self.dv, self.dtab, self.dlen)


def no_error():
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == 0


# ---- append ----------------------------------------------------------------------------------

def check_append(rng, lens, n, N, H, D, page, rot, off, inter, tree, in_place=False):
    c = Cache(rng, lens, n, D, page, N)
    B = c.B
    k, v = (rng.standard_normal((B, N, D)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((B, N, H, D)).astype(np.float16) if H else None
    par = R.random_parents(rng, B, N) if tree else None
    inv = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    kv = c.upload()
    dq = dev(q) if H else None
    dqo = (dq if in_place else torch.full_like(dq, 7.0)) if H else None
    ds4a.ds4a_paged_append(kv, dev(k), dev(v), c.dn, dev(par) if tree else None, dev(inv) if rot else None, off, inter,
                           dq, dqo)
    no_error()
    gk, gv = c.dk.cpu().numpy().reshape(-1, D), c.dv.cpu().numpy().reshape(-1, D)
    ek, ev = c.k.astype(np.float64), c.v.copy()
    eq = (q.astype(np.float64) if in_place else np.full(q.shape, 7.0)) if H else None
    for s in range(B):
        paths = R.paths_of(par[s], n[s]) if tree else None
        for i in range(n[s]):
            pos = lens[s] + (len(paths[i]) - 1 if tree else i)
            r = c.rows(s, [lens[s] + i])[0]
            ek[r], ev[r] = R.rotate(k[s, i].astype(np.float64), pos, inv, off, inter), v[s, i]
            if H:
                eq[s, i] = R.rotate(q[s, i].astype(np.float64), pos, inv, off, inter)
    assert np.array_equal(gv, ev, equal_nan=True)
    # one rounding to 16 bits (2^-11 of the value), and binary32 arithmetic: the angle (a half-turn fraction rounded to
    # 2^-25, 2^-23 radians), sine and cosine (2^-22) and two products and a sum, of at most |x1| + |x2|
    amp = 2 * np.abs(k).max() if not H else 2 * max(np.abs(k).max(), np.abs(q).max())
    for got, want in ((gk, ek),) + (((dqo.cpu().numpy(), eq),) if H else ()):
        ok = np.isnan(want)
        assert np.array_equal(np.isnan(got), ok)
        err = np.abs(got.astype(np.float64) - want)[~ok]
        tol = (2.0 ** -11 * np.abs(want) + 2.0 ** -25 + amp * 2.0 ** -20)[~ok]
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
def test_append_rotates_and_places(lens, n, N, H, D, page, rot, off, inter, tree):
    check_append(np.random.default_rng(N), lens, n, N, H, D, page, rot, off, inter, tree)


def test_append_in_place_queries():
    check_append(np.random.default_rng(3), [77, 12], [9, 4], 9, 64, 128, 16, 64, 64, True, True, in_place=True)


def test_append_far_position():
    """Positions past 2^24, where an angle in 32 bits is off by whole radians."""
    page, D, ln = 65536, 64, (1 << 24) + 12345
    mp = ln // page + 1
    table = torch.zeros(1, mp, dtype=torch.int32, device="cuda")    # every page is page 0: only one slot is written
    pk = torch.zeros(1, page, D, dtype=torch.float16, device="cuda")
    pv = torch.zeros_like(pk)
    kv = ds4a.paged_kv_desc(pk, pv, table, torch.tensor([ln], device="cuda"))
    rng = np.random.default_rng(0)
    k = rng.standard_normal((1, 1, D)).astype(np.float16)
    inv = np.array([1.0, 0.7, 3.5, 1e-3, 1e-6, 0.5, 0.25, 6.0], np.float32)
    ds4a.ds4a_paged_append(kv, dev(k), dev(k), torch.ones(1, dtype=torch.int32, device="cuda"), None, dev(inv), 16, True)
    no_error()
    want = R.rotate(k[0, 0].astype(np.float64), ln, inv, 16, True)
    got = pk[0, ln % page].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 8 * 2.0 ** -20).all()


@pytest.mark.parametrize("ln", [0, 1, (1 << 24) + 12345])
@pytest.mark.parametrize("inv", [
    [-3.5, -1.0, -1e-3, -100.25],       # turns backwards
    [0.0, -0.0, 1e-30, 1e-42],          # no turn at all: zeros, below 2^-64 of a turn, a denormal
    [100.25, 6.5, 2.0 ** -40, 1.0],     # more than a turn a token, and next to none
])
def test_append_unusual_frequencies(ln, inv):
    """The angle, in radians: two roundings of f / 2 pi <= 16 to 2^-53 each, times 2^24 positions
    (2^-21.3); what falls below 2^-64 and 2^-32 turns (2^-29); float(angle) (2^-23.3); the sine's
    own error (2^-23); the oracle's product (2^-22.4): below 2^-20.  The products and their sum add
    2^-23 of |x1| + |x2| < 8: in all below 8 * 2^-19, beside the rounding to 16 bits."""
    page, D = 65536, 64
    mp = ln // page + 1
    table = torch.zeros(1, mp, dtype=torch.int32, device="cuda")    # every page is page 0: only one slot is written
    pk = torch.zeros(1, page, D, dtype=torch.float16, device="cuda")
    kv = ds4a.paged_kv_desc(pk, torch.zeros_like(pk), table, torch.tensor([ln], device="cuda"))
    inv = np.array(inv * 2, np.float32)
    k = np.random.default_rng(1).uniform(-3, 3, (1, 1, D)).astype(np.float16)
    ds4a.ds4a_paged_append(kv, dev(k), dev(k), torch.ones(1, dtype=torch.int32, device="cuda"), None, dev(inv), 16, True)
    no_error()
    want = R.rotate(k[0, 0].astype(np.float64), ln, inv, 16, True)
    got = pk[0, ln % page].cpu().numpy().astype(np.float64)
    assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 8 * 2.0 ** -19).all()


# ---- rows completed in the draft, commit --------------------------------------------------------

def comp_setup(rng, c, ratio, D, room=2):
    """Compressed rows [B, cap, D] (NaN where nothing is committed) and the open blocks' states,
    made by the library's one-token compressor."""
    B, N = c.B, c.N
    cap = max(ln + N for ln in c.lens) // ratio + room + N
    w = (rng.standard_normal(D) * math.sqrt(1 / 128)).astype(np.float32)
    ck, cv = np.full((B, cap, D), NAN16), np.full((B, cap, D), NAN16)
    for s in range(B):
        m = c.lens[s] // ratio
        ck[s, :m], cv[s, :m] = (rng.standard_normal((m, D)).astype(np.float16) for _ in range(2))
    state = torch.full((B, 2 + 2 * D), math.nan, device="cuda")
    dck, dcv, dw = dev(ck), dev(cv), dev(w)
    for s in range(B):
        lo = c.lens[s] - c.lens[s] % ratio
        feed_path(c, s, range(lo, c.lens[s]), lo, dw, ratio, state[s], dck[s], dcv[s])
    torch.cuda.synchronize()
    return ck, cv, w, state, dck, dcv, dw


def feed_path(c, s, slots, pos, dw, ratio, state, ck, cv):
    """The library's compressor fed the tokens in `slots` one at a time."""
    for t in slots:
        r = c.rows(s, [t])
        ds4a.ds4a_compress_append(dev(c.k[r]), dev(c.v[r]), dw, ratio, pos, state, ck, cv)
        pos += 1


CASES = [([5], [1], 1, 128, 16, 1, "chain"), ([3, 8, 0, 250], [7, 5, 8, 1], 8, 128, 16, 4, "tree"),
         ([127, 120, 60, 0], [64, 20, 64, 64], 64, 64, 48, 128, "chain"),
         ([13, 14], [33, 64], 64, 128, 32, 3, "tree"), ([6, 1, 2], [9, 0, 9], 9, 64, 16, 4, "roots"),
         ([1023], [40], 40, 128, 64, 1024, "chain"), ([30, 31], [64, 63], 64, 128, 16, 7, "tree")]


@pytest.mark.parametrize("lens,n,N,D,page,ratio,kind", CASES)
def test_compress_tree_is_the_path_token_by_token(lens, n, N, D, page, ratio, kind):
    rng = np.random.default_rng(N + ratio)
    c = Cache(rng, lens, n, D, page, N)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D)
    par = R.random_parents(rng, c.B, N, kind)
    kv = c.upload()
    before = dck.clone(), dcv.clone(), state.clone()
    ds4a.ds4a_compress_tree(kv, c.dn, None if kind == "chain" else dev(par), dw, ratio, state, dck, dcv, N=N)
    no_error()
    assert torch.equal(state.view(torch.int32), before[2].view(torch.int32))
    cap = ck.shape[1]
    want_k, want_v = before[0].clone(), before[1].clone()
    for s in range(c.B):
        for i, path in enumerate(R.paths_of(par[s], n[s])):
            if (lens[s] + len(path)) % ratio:
                continue
            tmp_s, tk, tv = state[s].clone(), torch.zeros_like(dck[s]), torch.zeros_like(dcv[s])
            feed_path(c, s, [lens[s] + j for j in path], lens[s], dw, ratio, tmp_s, tk, tv)
            row = (lens[s] + len(path)) // ratio - 1
            want_k[s, cap - N + i], want_v[s, cap - N + i] = tk[row], tv[row]
            # and against the definition: binary32 sums over at most `ratio` tokens, rounded once to 16 bits
            first = max(lens[s], lens[s] + len(path) - ratio)
            rows = c.rows(s, [lens[s] + j for j in path[first - lens[s]:]])
            cont = first == lens[s] and lens[s] % ratio != 0
            kk, vv = c.k[rows].astype(np.float64), c.v[rows].astype(np.float64)
            _, l, a, b = R.pool_block(kk, vv, w.astype(np.float64), state[s].cpu().numpy().astype(np.float64) if cont else None)
            for got, num in ((dck[s, cap - N + i], a), (dcv[s, cap - N + i], b)):
                ref = num / l
                err = np.abs(got.cpu().numpy().astype(np.float64) - ref)
                # weights: exp of a score off by D 2^-23 of at most |w||k|, through up to ratio rescalings of 2^-22 each
                assert (err <= 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + (ratio * 2.0 ** -21 + 2.0 ** -12) * 6).all()
    assert torch.equal(dck.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(dcv.view(torch.int16), want_v.view(torch.int16))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,n,N,D,page,ratio,kind", CASES)
def test_commit_moves_the_path_and_continues_the_compressor(lens, n, N, D, page, ratio, kind, in_place):
    rng = np.random.default_rng(7 * N + ratio)
    c = Cache(rng, lens, n, D, page, N)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D)
    par = R.random_parents(rng, c.B, N, kind)
    B, cap, di = c.B, ck.shape[1], 40
    ki = rng.standard_normal((B, cap, di)).astype(np.float16)
    dki = dev(ki)
    leaf = np.array([rng.integers(-1, n[s]) if s else n[s] - 1 for s in range(B)], np.int32)
    kv = c.upload()
    dpar = dev(par)
    ds4a.ds4a_compress_tree(kv, c.dn, dpar, dw, ratio, state, dck, dcv)
    # the reference: the compressor fed the accepted tokens one at a time
    want_s, want_k, want_v = state.clone(), dck.clone(), dcv.clone()
    want_ki, want_pk, want_pv, want_len = ki.copy(), c.k.copy(), c.v.copy(), list(lens)
    for s in range(B):
        path = R.paths_of(par[s], n[s])[leaf[s]] if leaf[s] >= 0 else []
        feed_path(c, s, [lens[s] + j for j in path], lens[s], dw, ratio, want_s[s], want_k[s], want_v[s])
        for d, j in enumerate(path):
            to, fr = c.rows(s, [lens[s] + d]), c.rows(s, [lens[s] + j])
            want_pk[to], want_pv[to] = c.k[fr], c.v[fr]
            if (lens[s] + d + 1) % ratio == 0:
                want_ki[s, (lens[s] + d) // ratio] = ki[s, cap - N + j]
        want_len[s] += len(path)
        if want_len[s] % ratio == 0:
            want_s[s] = state[s]      # nothing open: not written
    state_out = state if in_place else torch.where(torch.isnan(state), state, state)
    if not in_place:
        state_out = state.clone()
    len_out = c.dlen if in_place else torch.full_like(c.dlen, -5)
    ds4a.ds4a_commit_tree(kv, c.dn, dpar, dev(leaf), len_out, dw, ratio, state, state_out, dck, dcv, dki)
    no_error()
    assert len_out.tolist() == want_len
    assert np.array_equal(c.dk.cpu().numpy().reshape(-1, D), want_pk, equal_nan=True)
    assert np.array_equal(c.dv.cpu().numpy().reshape(-1, D), want_pv, equal_nan=True)
    assert np.array_equal(dki.cpu().numpy(), want_ki)
    assert torch.equal(dck.view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(dcv.view(torch.int16), want_v.view(torch.int16))
    for s in range(B):
        if want_len[s] % ratio:
            assert torch.equal(state_out[s].view(torch.int32), want_s[s].view(torch.int32)), s


def test_append_compress_commit_leave_bad_sessions_alone():
    """A bad count, length, parent, leaf or page id: that session's arrays keep their bits, the
    others' are served, and the error word says so."""
    IDX, CAP = ds4a.DS4A_ERR_DEVICE_INDEX, ds4a.DS4A_ERR_CAPACITY
    N, ratio, D = 6, 2, 64

    def make(seed=3):
        rng = np.random.default_rng(seed)
        c = Cache(rng, [21, 34, 15], [6, 5, 4], D, 16, N)
        c.draft()
        x = comp_setup(rng, c, ratio, D)
        par = R.random_parents(rng, 3, N)
        return rng, c, x, par

    def run(call, c, x, par, leaf=(5, 4, 3)):
        ck, cv, w, state, dck, dcv, dw = x
        kv = c.upload()
        so, lo = state.clone(), torch.full((3,), -9, device="cuda")
        before = [t.clone() for t in (c.dk, c.dv, dck, dcv, so, lo)]
        kn = torch.ones(3, N, D, dtype=torch.float16, device="cuda")
        if call == "append":
            ds4a.ds4a_paged_append(kv, kn, kn, c.dn, dev(par))
        elif call == "compress":
            ds4a.ds4a_compress_tree(kv, c.dn, dev(par), dw, ratio, state, dck, dcv)
        else:
            ds4a.ds4a_commit_tree(kv, c.dn, dev(par), dev(np.array(leaf, np.int32)), lo, dw, ratio, state, so, dck, dcv)
        torch.cuda.synchronize()
        return ds4a.ds4a_last_device_error(), before, [c.dk, c.dv, dck, dcv, so, lo]

    def rows_of(c, t, s):
        return t.view(-1, D)[torch.from_numpy(c.rows(s, range(c.mp * c.page)).clip(0)).cuda()]
    for call in ("append", "compress", "commit"):
        for what in ("n_low", "n_high", "len", "cap", "parent", "leaf", "page"):
            if what == "leaf" and call != "commit":
                continue
            rng, c, x, par = make()
            good_table, code, leaf = c.table.copy(), IDX, (5, 4, 3)
            if what == "n_low":
                c.n[1] = -1
            elif what == "n_high":
                c.n[1] = N + 1
            elif what == "len":
                c.lens[1] = -4
            elif what == "cap":
                c.lens[1], code = c.mp * 16 - 2, CAP
            elif what == "parent":
                par[1, 3] = 3
            elif what == "leaf":
                leaf = (5, 5, 3)
            else:                                   # every drafted token of session 1 in a page that is none
                c.table[1, 34 // 16:] = 1 << 30
            err, before, after = run(call, c, x, par, leaf)
            assert err == code, (call, what)
            c.table = good_table
            for b, a in zip(before[:2], after[:2]):     # session 1's pages
                assert torch.equal(rows_of(c, b, 1).view(torch.int16), rows_of(c, a, 1).view(torch.int16)), (call, what)
            for b, a in zip(before[2:], after[2:]):
                assert torch.equal(b[1].view(torch.uint8) if b.dim() > 1 else b[1], a[1].view(torch.uint8) if a.dim() > 1 else a[1]), (call, what)
            # the others are served as without the fault
            rng2, c2, x2, par2 = make()
            err2, _, ok = run(call, c2, x2, par2)
            assert err2 == 0
            for s in (0, 2):
                for b, a in zip(ok[:2], after[:2]):
                    assert torch.equal(rows_of(c, b, s).view(torch.int16), rows_of(c, a, s).view(torch.int16)), (call, what, s)
                for b, a in zip(ok[2:5], after[2:5]):
                    assert torch.equal(b[s].view(torch.int16), a[s].view(torch.int16)), (call, what, s)
                assert ok[5][s] == after[5][s]


def test_commit_of_compressed_rows_past_the_capacity_is_refused():
    rng = np.random.default_rng(8)
    c = Cache(rng, [16, 4], [4, 4], 64, 16, 4)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, 4, 64)
    keep = 4 + 4                                     # committed rows 0 .. 3: session 0's next row has no place
    dck, dcv = dck[:, :keep].contiguous(), dcv[:, :keep].contiguous()
    kv = c.upload()
    lo = torch.full((2,), -9, device="cuda")
    leaf = torch.tensor([3, 3], dtype=torch.int32, device="cuda")
    ds4a.ds4a_commit_tree(kv, c.dn, None, leaf, lo, dw, 4, state, state, dck, dcv, N=4)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_CAPACITY
    assert lo.tolist() == [-9, 8]


def test_pools_past_32_bit_offsets():
    """Pages whose elements lie past 2^31: append, compress, attention and commit reach them."""
    D, page, n_pages, N, ln = 128, 4096, 4200, 5, 8190           # 2.2e9 values a pool
    pk = torch.empty(n_pages, page, D, dtype=torch.float16, device="cuda")
    pv = torch.empty_like(pk)
    ids = [n_pages - 1, n_pages - 3, n_pages - 2]
    for i in ids:
        pk[i].normal_()
        pv[i].normal_()
    table = torch.tensor([ids], dtype=torch.int32, device="cuda")
    length = torch.tensor([ln], device="cuda")
    kv = ds4a.paged_kv_desc(pk, pv, table, length)
    rng = np.random.default_rng(0)
    k, v = (rng.standard_normal((1, N, D)).astype(np.float16) for _ in range(2))
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    par = np.array([[-1, 0, 0, 1, 3]], np.int32)
    ds4a.ds4a_paged_append(kv, dev(k), dev(v), n, dev(par))
    q = rng.standard_normal((1, N, 8, D)).astype(np.float16)
    out = torch.zeros(1, N, 8, D, dtype=torch.float16, device="cuda")
    ws = torch.empty(ds4a.ds4a_attn_tree_workspace_bytes(1, N, 8, D), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_tree(kv, dev(q), n, dev(par), 1 << 20, None, None, 0, None, 0.08, out, ws)
    no_error()
    # the three pages as a small pool of their own
    small_k = pk[torch.tensor(ids).cuda()].cpu().numpy().reshape(-1, D)
    small_v = pv[torch.tensor(ids).cuda()].cpu().numpy().reshape(-1, D)
    assert np.array_equal(small_k[ln:ln + N], k[0]) and np.array_equal(small_v[ln:ln + N], v[0])
    for i, path in enumerate(R.paths_of(par[0], N)):
        kk, vv = R.node_keys(small_k, small_v, None, None, np.arange(3), page, ln, path, N, 1 << 20, 0, None)
        want, tol = R.attend(q[0, i], kk, vv, 0.08)
        assert (np.abs(out[0, i].cpu().numpy().astype(np.float64) - want) <= tol).all()
    leaf = torch.tensor([4], dtype=torch.int32, device="cuda")
    ds4a.ds4a_commit_tree(kv, n, dev(par), leaf, length)
    no_error()
    assert length.item() == ln + 4
    got = pk[torch.tensor(ids).cuda()].cpu().numpy().reshape(-1, D)
    assert np.array_equal(got[ln:ln + 4], k[0][[0, 1, 3, 4]])


# ---- attention -----------------------------------------------------------------------------------

def attn_setup(rng, lens, n, N, H, D, page, window, ratio, n_sel, kind):
    c = Cache(rng, lens, n, D, page, N)
    c.draft()
    B = c.B
    par = R.random_parents(rng, B, N, kind)
    q = np.full((B, N, H, D), NAN16)
    for s in range(B):
        q[s, :n[s]] = rng.standard_normal((n[s], H, D)).astype(np.float16)
    ck = cv = sel = None
    if ratio:
        cap = max(ln + N for ln in lens) // ratio + 1 + N
        ck, cv = np.full((B, cap, D), NAN16), np.full((B, cap, D), NAN16)
        for s in range(B):
            rows = list(range(lens[s] // ratio))
            for i, path in enumerate(R.paths_of(par[s], n[s])):
                if (lens[s] + len(path)) % ratio == 0:
                    rows.append(cap - N + i)
            ck[s, rows], cv[s, rows] = (rng.standard_normal((len(rows), D)).astype(np.float16) for _ in range(2))
        if n_sel:
            sel = np.full((B, N, n_sel), -1, np.int32)
            for s in range(B):
                for i, path in enumerate(R.paths_of(par[s], n[s])):
                    vis = (lens[s] + len(path)) // ratio
                    m = min(n_sel, vis)
                    sel[s, i, :m] = np.sort(rng.permutation(vis)[:m])
    return c, par, q, ck, cv, sel


def run_attn(c, par, q, ck, cv, sel, window, ratio, scale, out=None, ws=None, stream=None):
    B, N, H, D = q.shape
    kv = c.upload()
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda") if out is None else out
    if ws is None:
        ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(B, N, H, D), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_tree(kv, dev(q), c.dn, None if par is None else dev(par), window, None if ck is None else dev(ck),
                        None if cv is None else dev(cv), ratio, None if sel is None else dev(sel), scale, out, ws,
                        stream=stream)
    return out


def check_attn(c, par, q, ck, cv, sel, window, ratio, scale, out, skip=()):
    got = out.cpu().numpy().astype(np.float64)
    worst = 0.0
    for s in range(c.B):
        paths = R.paths_of(par[s], c.n[s])
        for i, path in enumerate(paths):
            if (s, i) in skip:
                continue
            k, v = R.node_keys(c.k, c.v, None if ck is None else ck[s], None if cv is None else cv[s], c.table[s], c.page,
                               c.lens[s], path, c.N, window, ratio, None if sel is None else sel[s, i])
            want, tol = R.attend(q[s, i], k, v, scale)
            err = np.abs(got[s, i] - want)
            assert (err <= tol).all(), (s, i, float((err / tol).max()))
            worst = max(worst, float((err / tol).max()))
        assert (got[s, c.n[s]:] == 7.0).all(), "rows behind the last node changed"
    return worst


ATTN = [
    # lens, n, N, H, D, page, window, ratio, n_sel, tree
    ([0], [1], 1, 8, 64, 16, 1, 0, 0, "chain"),
    ([0, 1, 2], [1, 2, 1], 2, 8, 128, 16, 128, 4, 0, "chain"),
    ([200], [4], 4, 64, 128, 64, 128, 0, 0, "tree"),
    ([127, 128, 129, 40], [8, 8, 3, 0], 8, 64, 128, 48, 128, 4, 0, "tree"),
    ([1000, 37], [13, 5], 13, 24, 64, 16, 100, 7, 0, "tree"),
    ([515, 300], [64, 64], 64, 8, 128, 16, 30, 16, 0, "tree"),
    ([1023, 5], [64, 64], 64, 64, 128, 128, 128, 128, 0, "chain"),
    ([700], [33], 33, 40, 128, 80, 1 << 40, 0, 0, "tree"),
    ([5000], [3], 3, 64, 128, 64, 1 << 30, 0, 0, "tree"),
    ([4097, 3000, 1], [2, 16, 7], 16, 16, 64, 32, 2000, 128, 0, "roots"),
    ([600, 90, 3], [9, 5, 9], 9, 64, 128, 16, 128, 4, 64, "tree"),
    ([600, 90, 3], [9, 5, 9], 9, 64, 128, 16, 128, 4, 61, "tree"),
    ([2500, 8], [16, 16], 16, 64, 128, 64, 128, 4, 512, "tree"),
    ([333], [20], 20, 8, 64, 48, 17, 1, 40, "tree"),
    ([100, 700], [64, 2], 64, 32, 128, 16, 300, 2, 130, "chain"),
    ([70000], [2], 2, 8, 64, 256, 1 << 30, 0, 0, "tree"),
    # more row tiles than SMs: several a CTA, of several sizes
    ([40 + 37 * s for s in range(44)], [8 - s % 5 for s in range(44)], 8, 8, 128, 16, 64, 4, 100, "tree"),
    ([1000 - 9 * s for s in range(60)], [10 - s % 9 for s in range(60)], 10, 64, 64, 16, 128, 8, 0, "tree"),
    ([300 + s for s in range(200)], [1 + s % 2 for s in range(200)], 2, 8, 128, 32, 100, 0, 0, "roots"),
    ([900, 901, 902, 903, 904], [5, 4, 3, 2, 1], 5, 48, 128, 112, 64, 64, 1, "tree"),
    # few row tiles over many keys: one line of key tiles over the SMs, sessions without nodes in it
    ([9000, 0, 4000, 77], [3, 2, 0, 3], 3, 64, 128, 64, 1 << 30, 0, 0, "tree"),
    ([12000], [1], 1, 8, 128, 64, 1 << 30, 4, 0, "chain"),
    ([7000 - 150 * s for s in range(40)], [s % 3 for s in range(40)], 2, 16, 64, 48, 1 << 30, 128, 0, "tree"),
    ([20000, 3], [40, 2], 40, 64, 128, 128, 1 << 30, 128, 0, "tree"),
    ([6000], [2], 2, 64, 128, 16, 128, 1, 2048, "chain"),
]


@pytest.mark.parametrize("lens,n,N,H,D,page,window,ratio,n_sel,kind", ATTN)
def test_attn_tree(lens, n, N, H, D, page, window, ratio, n_sel, kind):
    rng = np.random.default_rng(N * 31 + H)
    c, par, q, ck, cv, sel = attn_setup(rng, lens, n, N, H, D, page, window, ratio, n_sel, kind)
    out = run_attn(c, None if kind == "chain" else par, q, ck, cv, sel, window, ratio, 1 / math.sqrt(D))
    no_error()
    check_attn(c, par, q, ck, cv, sel, window, ratio, 1 / math.sqrt(D), out)


def test_attn_tree_scores_far_apart():
    """Scores that grow along the keys (the running maximum moves at every tile) and scores far
    below the maximum."""
    rng = np.random.default_rng(5)
    c, par, q, ck, cv, sel = attn_setup(rng, [1500, 800], [6, 6], 6, 16, 128, 16, 4096, 16, 0, "tree")
    for s in range(2):
        r = c.rows(s, range(c.lens[s] + 6))
        c.k[r] = (c.k[r] * np.linspace(0.05, 6.0, len(r))[:, None]).astype(np.float16)
    out = run_attn(c, par, q, ck, cv, sel, 4096, 16, 1 / math.sqrt(128))
    no_error()
    check_attn(c, par, q, ck, cv, sel, 4096, 16, 1 / math.sqrt(128), out)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("where", ["sibling", "window_edge", "draft_row"])
def test_attn_tree_keeps_other_nodes_values_out(bad, where):
    """A value that is not finite reaches the nodes that attend its token and no others, whose
    outputs keep their bits."""
    rng = np.random.default_rng(11)
    lens, n, N = [300], [12], 12
    c, par, q, ck, cv, sel = attn_setup(rng, lens, n, N, 64, 128, 16, 64, 4, 0, "tree")
    paths = R.paths_of(par[0], 12)
    depth = [len(p) - 1 for p in paths]
    clean = run_attn(c, par, q, ck, cv, sel, 64, 4, 0.09).clone()
    if where == "sibling":
        hit = {i for i in range(12) if 5 in paths[i]}
        c.v[c.rows(0, [305])[0], 3] = bad
        c.k[c.rows(0, [305])[0], 9] = bad if np.isnan(bad) else c.k[c.rows(0, [305])[0], 9]
    elif where == "window_edge":
        t = 300 - 64 + 1 + 1                       # attended up to depth 1
        hit = {i for i in range(12) if t > 300 + depth[i] - 64}
        c.v[c.rows(0, [t])[0], 3] = bad
    else:
        i0 = next(i for i in range(12) if (300 + depth[i] + 1) % 4 == 0)
        hit = {i for i in range(12) if i0 in paths[i]}
        cv[0, ck.shape[1] - N + i0, 3] = bad
    assert 0 < len(hit) < 12
    out = run_attn(c, par, q, ck, cv, sel, 64, 4, 0.09)
    no_error()
    for i in range(12):
        if i in hit:
            x = out[0, i, :, 3].float().cpu().numpy()
            if np.isinf(bad):
                assert (x == bad).all(), i
            else:
                assert np.isnan(x).all(), i
        else:
            assert torch.equal(out[0, i], clean[0, i]), i


@pytest.mark.parametrize("B,N,H,D,window,ratio,lens", [
    (40, 10, 64, 128, 96, 4, lambda s: 130 + 11 * s),        # two row blocks an item, more items than SMs
    (40, 10, 64, 64, 96, 4, lambda s: 130 + 11 * s),
    (90, 6, 16, 128, 60, 0, lambda s: 100 + s),              # one row block
    (3, 6, 64, 128, 1 << 30, 16, lambda s: 6000 - 900 * s),  # a line of key tiles, its pieces joined
])
def test_attn_tree_keeps_values_that_are_not_finite_to_their_nodes(B, N, H, D, window, ratio, lens):
    """The same over many items: every third session has drafted tokens (and, with a window, a token
    at its edge) with values that are not finite; nodes that do not attend them keep their bits,
    the others get them in those columns and keep the rest within the tolerance."""
    rng = np.random.default_rng(B + D)
    ln, n = [lens(s) for s in range(B)], [N - s % 3 for s in range(B)]
    c, par, q, ck, cv, _ = attn_setup(rng, ln, n, N, H, D, 16, window, ratio, 0, "tree")
    clean = run_attn(c, par, q, ck, cv, None, window, ratio, 0.09).clone()
    no_error()
    bad = {}                                          # (session, node) -> {column: value}
    for s in range(0, B, 3):
        paths = R.paths_of(par[s], n[s])
        marks = [(int(rng.integers(0, n[s])), int(rng.integers(0, D)), v) for v in (np.inf, -np.inf, np.nan)]
        for j, col, val in marks:
            r = c.rows(s, [ln[s] + j])[0]
            c.v[r, col] = val
            for i, path in enumerate(paths):
                if j in path and len(path) - path.index(j) <= window:
                    bad.setdefault((s, i), {}).setdefault(col, set()).add((j, str(val)))
        if window < 1 << 20:
            t, col = ln[s] - window + 2, int(rng.integers(0, D))   # attended up to depth 1
            c.v[c.rows(s, [t])[0], col] = np.inf
            for i, path in enumerate(paths):
                if t >= ln[s] + len(path) - 1 - window + 1:
                    bad.setdefault((s, i), {}).setdefault(col, set()).add((-1, "inf"))
    # a later mark in one place replaces an earlier one: what the arrays hold counts
    out = run_attn(c, par, q, ck, cv, None, window, ratio, 0.09)
    no_error()
    o, w = out.float().cpu().numpy(), clean.float().cpu().numpy()
    for s in range(B):
        paths = R.paths_of(par[s], n[s])
        for i, path in enumerate(paths):
            _, v = R.node_keys(c.k, c.v, None if ck is None else ck[s], None if cv is None else cv[s], c.table[s], 16, ln[s],
                               path, N, window, ratio, None)
            with np.errstate(invalid="ignore"):
                total = np.where(np.isfinite(v), 0.0, v).sum(0)
            odd = ~np.isfinite(v).all(0)
            if not odd.any():
                assert np.array_equal(o[s, i], w[s, i]), (s, i)
                continue
            assert (s, i) in bad
            assert np.array_equal(o[s, i][:, ~odd], w[s, i][:, ~odd]), (s, i)
            for col in np.flatnonzero(odd):
                got = o[s, i][:, col]
                if np.isnan(total[col]):
                    assert np.isnan(got).all(), (s, i, col)
                else:
                    assert (got == total[col]).all(), (s, i, col)


def test_attn_tree_two_streams_at_once():
    """Two calls on two streams, each with its own workspace, give the bits that they give alone."""
    rng = np.random.default_rng(13)
    sets = [(attn_setup(rng, [9000, 40], [7, 5], 7, 64, 128, 64, 1 << 30, 16, 0, "tree"), 1 << 30, 16),
            (attn_setup(rng, [900 - 5 * s for s in range(30)], [9] * 30, 9, 64, 128, 16, 128, 4, 0, "tree"), 128, 4)]
    alone = [run_attn(*x, w, r, 0.1).clone() for x, w, r in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = []
        for (x, w, r), st in zip(sets, streams):
            with torch.cuda.stream(st):
                outs.append(run_attn(*x, w, r, 0.1, stream=st))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, outs))
    no_error()


def test_attn_tree_same_row_twice_and_no_nodes():
    rng = np.random.default_rng(14)
    # a list that names rows twice attends them twice
    c, par, q, ck, cv, sel = attn_setup(rng, [300, 70], [5, 4], 5, 16, 64, 16, 40, 4, 12, "tree")
    sel[:, :, 7:] = sel[:, :, :5]
    out = run_attn(c, par, q, ck, cv, sel, 40, 4, 0.1)
    no_error()
    check_attn(c, par, q, ck, cv, sel, 40, 4, 0.1, out)
    # a list of nothing: the window alone
    sel[:] = -1
    out = run_attn(c, par, q, ck, cv, sel, 40, 4, 0.1)
    no_error()
    check_attn(c, par, q, ck, cv, sel, 40, 4, 0.1, out)
    # no session has a node, in each way of cutting the work
    for lens, window in (([30, 40], 16), ([9000], 1 << 30), ([20] * 200, 8)):
        c, par, q, ck, cv, sel = attn_setup(rng, lens, [0] * len(lens), 3, 64, 64, 16, window, 0, 0, "tree")
        out = run_attn(c, par, q, ck, cv, sel, window, 0, 0.1)
        no_error()
        assert (out == 7.0).all()


def test_binding_refuses_other_layouts_and_devices():
    c, par, q, ck, cv, sel = attn_setup(np.random.default_rng(0), [20], [2], 2, 8, 64, 16, 16, 0, 0, "chain")
    kv = c.upload()
    dq, dpar = dev(q), dev(par)
    ws = torch.empty(ds4a.ds4a_attn_tree_workspace_bytes(1, 2, 8, 64), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(dq)
    wide = torch.zeros(1, 2, 8, 128, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        ds4a.ds4a_attn_tree(kv, wide[..., ::2], c.dn, dpar, 16, None, None, 0, None, 0.1, out, ws)
    with pytest.raises(TypeError, match="float16"):
        ds4a.ds4a_attn_tree(kv, dq.float(), c.dn, dpar, 16, None, None, 0, None, 0.1, out, ws)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ds4a.ds4a_attn_tree(kv, dq, c.dn.cpu(), dpar, 16, None, None, 0, None, 0.1, out, ws)
    with pytest.raises(ds4a.Ds4aError, match="workspace"):
        ds4a.ds4a_attn_tree(kv, dq, c.dn, dpar, 16, None, None, 0, None, 0.1, out, ws[:-1])
    kv.device = 1                                    # as if the cache were on another device than the current one
    with pytest.raises(ValueError, match="current device"):
        ds4a.ds4a_attn_tree(kv, dq, c.dn, dpar, 16, None, None, 0, None, 0.1, out, ws)


def test_attn_tree_reports_bad_device_values():
    """Bad parents, counts, lengths, page ids and sel entries are skipped and recorded."""
    rng = np.random.default_rng(2)
    base = lambda: attn_setup(rng, [100, 60], [4, 4], 4, 8, 64, 16, 64, 4, 0, "tree")
    IDX, CAP = ds4a.DS4A_ERR_DEVICE_INDEX, ds4a.DS4A_ERR_CAPACITY

    def session0_alone(c, par, q, ck, cv, code, par_ok):
        out = run_attn(c, par, q, ck, cv, None, 64, 4, 0.1)
        torch.cuda.synchronize()
        assert ds4a.ds4a_last_device_error() == code
        assert (out[0] == 7.0).all()
        c.n[0] = 0
        check_attn(c, par_ok, q, ck, cv, None, 64, 4, 0.1, out)
    for bad in (2, 7, -2):
        c, par, q, ck, cv, _ = base()
        p2 = par.copy()
        p2[0, 2] = bad
        session0_alone(c, p2, q, ck, cv, IDX, par)
    for n0 in (-1, 5):
        c, par, q, ck, cv, _ = base()
        c.n[0] = n0
        session0_alone(c, par, q, ck, cv, IDX, par)
    c, par, q, ck, cv, _ = base()
    c.lens[0] = c.mp * 16 - 3
    session0_alone(c, par, q, ck, cv, CAP, par)
    c, par, q, ck, cv, _ = base()
    c.lens[0] = -1
    session0_alone(c, par, q, ck, cv, IDX, par)
    # a page outside the pool: its tokens are not attended
    for bad in (-1, 10 ** 6):
        c, par, q, ck, cv, _ = base()
        keep = c.table.copy()
        c.table[0, 100 // 16 - 1] = bad
        out = run_attn(c, par, q, ck, cv, None, 64, 4, 0.1)
        torch.cuda.synchronize()
        assert ds4a.ds4a_last_device_error() == IDX
        got = out[0].float().cpu().numpy()
        lost = 16 * (100 // 16 - 1)
        for i, path in enumerate(R.paths_of(par[0], 4)):
            p = 100 + len(path) - 1
            slots = [t if t < 100 else 100 + path[t - 100] for t in range(max(0, p - 63), p + 1)]
            slots = [t for t in slots if not lost <= t < lost + 16]
            js = [j if j < 25 else ck.shape[1] - 4 + path[(j + 1) * 4 - 101] for j in range((p + 1) // 4)]
            rows = R.slot_rows(keep[0], 16, slots)
            k = np.concatenate([c.k[rows], ck[0, js]]).astype(np.float64)
            v = np.concatenate([c.v[rows], cv[0, js]]).astype(np.float64)
            want, tol = R.attend(q[0, i], k, v, 0.1)
            assert (np.abs(got[i] - want) <= tol).all()
    # sel entries that are not complete, or far out of range
    c, par, q, ck, cv, sel = attn_setup(rng, [100, 60], [4, 4], 4, 8, 64, 16, 64, 4, 10, "tree")
    sel[0, 1, 3], sel[0, 2, 0], sel[1, 0, 9] = 2 ** 31 - 1, 27, -2 ** 31
    out = run_attn(c, par, q, ck, cv, sel, 64, 4, 0.1)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == IDX
    check_attn(c, par, q, ck, cv, sel, 64, 4, 0.1, out)


def test_attn_tree_reports_bad_sessions_among_many():
    """More row tiles than SMs: sessions with bad counts, lengths, parents or no nodes between others."""
    rng = np.random.default_rng(6)
    B, N = 70, 9
    lens, n = [50 + s for s in range(B)], [1 + s % N for s in range(B)]
    c, par, q, ck, cv, _ = attn_setup(rng, lens, n, N, 64, 64, 16, 40, 4, 0, "tree")
    good = list(n)
    for s, bad in ((0, 10), (33, -1), (69, 1 << 20), (40, 0)):
        c.n[s], good[s] = bad, 0
    c.lens[12], good[12] = -7, 0
    par[50, 1], good[50] = 1, 0
    c.n[50] = 3
    out = run_attn(c, par, q, ck, cv, None, 40, 4, 0.1)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_DEVICE_INDEX
    c.n, par[50, 1] = good, 0
    check_attn(c, par, q, ck, cv, None, 40, 4, 0.1, out)


def test_attn_tree_without_a_readable_row_gives_zeros():
    c, par, q, ck, cv, sel = attn_setup(np.random.default_rng(1), [20, 20], [2, 2], 2, 8, 64, 16, 64, 0, 0, "chain")
    c.table[0, :] = -1
    out = run_attn(c, par, q, ck, cv, sel, 64, 0, 0.1)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_DEVICE_INDEX
    assert (out[0] == 0).all()
    c.n[0] = 0
    out[0] = 7.0
    check_attn(c, par, q, ck, cv, sel, 64, 0, 0.1, out)


def test_attn_tree_repeats_its_bits_and_its_workspace():
    """Calls of different shapes in turn on one workspace: the same bits as on a fresh one."""
    rng = np.random.default_rng(9)
    sets = [(attn_setup(rng, [5000, 40], [7, 5], 7, 64, 128, 64, 4096, 16, 0, "tree"), 4096, 16),
            (attn_setup(rng, [9000], [1], 1, 64, 128, 16, 1 << 30, 0, 0, "chain"), 1 << 30, 0),
            (attn_setup(rng, [900, 33], [9, 4], 9, 8, 64, 16, 128, 4, 50, "tree"), 128, 4)]
    nb = max(ds4a.ds4a_attn_tree_workspace_bytes(*s[0][2].shape) for s in sets)
    ws = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    fresh = [run_attn(*s[0], s[1], s[2], 0.1).clone() for s in sets]
    for _ in range(3):
        for s, want in zip(sets, fresh):
            assert torch.equal(run_attn(*s[0], s[1], s[2], 0.1, ws=ws), want)
    no_error()


# ---- streams, graphs, the calls together ------------------------------------------------------------

def step_setup(seed, lens, n, N, H=64, D=128, page=16, ratio=4):
    """A whole step's tensors: cache, new tokens, tree, compressor."""
    rng = np.random.default_rng(seed)
    c = Cache(rng, lens, n, D, page, N)
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D, room=N)
    kv = c.upload()
    par = R.random_parents(rng, c.B, N)
    x = dict(c=c, kv=kv, par=par, dpar=dev(par), state=state, ck=dck, cv=dcv, w=dw, ratio=ratio, N=N)
    x["k"], x["v"] = (dev(rng.standard_normal((c.B, N, D)).astype(np.float16)) for _ in range(2))
    x["q"] = dev(rng.standard_normal((c.B, N, H, D)).astype(np.float16))
    x["leaf"] = dev(np.array([ni - 1 for ni in n], np.int32))
    x["out"] = torch.zeros_like(x["q"])
    x["qr"] = torch.zeros_like(x["q"])
    x["inv"] = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    x["ws"] = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(c.B, N, H, D), dtype=torch.uint8, device="cuda")
    return x


def step(x, commit=True, stream=None):
    ds4a.ds4a_paged_append(x["kv"], x["k"], x["v"], x["c"].dn, x["dpar"], x["inv"], 64, True, x["q"], x["qr"], stream=stream)
    ds4a.ds4a_compress_tree(x["kv"], x["c"].dn, x["dpar"], x["w"], x["ratio"], x["state"], x["ck"], x["cv"], stream=stream)
    ds4a.ds4a_attn_tree(x["kv"], x["qr"], x["c"].dn, x["dpar"], 128, x["ck"], x["cv"], x["ratio"], None, 0.088, x["out"],
                        x["ws"], stream=stream)
    if commit:
        ds4a.ds4a_commit_tree(x["kv"], x["c"].dn, x["dpar"], x["leaf"], x["c"].dlen, x["w"], x["ratio"], x["state"],
                              x["state"], x["ck"], x["cv"], stream=stream)


def bits(x):
    return [t.clone().view(torch.uint8) for t in (x["out"], x["c"].dk, x["c"].dv, x["c"].dlen, x["state"], x["ck"], x["cv"])]


@pytest.mark.parametrize("ratio", [4, 128])
def test_checked_draft_equals_token_by_token_decode(ratio):
    """Every node's output is what decoding its path gives (ds4a_attn_decode over the same
    window and compressed rows), and after the commit the next draft continues from there."""
    x = step_setup(1, [300, 125, 0], [11, 9, 6], 12, ratio=ratio)
    c = x["c"]
    for rnd in range(3):
        lens = c.dlen.tolist()
        state0, ck0, cv0 = x["state"].clone(), x["ck"].clone(), x["cv"].clone()
        step(x, commit=False)
        no_error()
        pk, pv = c.dk.view(-1, 128), c.dv.view(-1, 128)
        for s in range(3):
            for i, path in enumerate(R.paths_of(x["par"][s], c.n[s])):
                st, tk, tv = state0[s].clone(), ck0[s].clone(), cv0[s].clone()
                slots = [lens[s] + j for j in path]
                for d, t in enumerate(slots):
                    r = c.rows(s, [t])[0]
                    ds4a.ds4a_compress_append(pk[r:r + 1], pv[r:r + 1], x["w"], ratio, lens[s] + d, st, tk, tv)
                p = lens[s] + len(path) - 1
                win = [t if t < lens[s] else slots[t - lens[s]] for t in range(max(0, p - 127), p + 1)]
                at = torch.from_numpy(c.rows(s, win)).cuda()
                ref = torch.empty(64, 128, dtype=torch.float16, device="cuda")
                torch.cuda.synchronize()
                ds4a.ds4a_attn_decode(x["qr"][s, i], pk[at], pv[at], tk, tv, None, (p + 1) // ratio, 0.088, ref)
                torch.cuda.synchronize()
                # two 16-bit results of one value: both are within the repository's 2e-3 of it
                assert float((ref.float() - x["out"][s, i].float()).abs().max()) <= 4e-3, (s, i)
        ds4a.ds4a_commit_tree(x["kv"], c.dn, x["dpar"], x["leaf"], c.dlen, x["w"], ratio, x["state"], x["state"], x["ck"],
                              x["cv"])
        no_error()
        if max(c.dlen.tolist()) + 12 > c.mp * 16:
            break
        x["k"].copy_(torch.randn_like(x["k"], dtype=torch.float32).half())
    assert rnd >= 0


def test_step_on_another_stream_and_captured():
    a, b, g = (step_setup(4, [200, 90], [6, 4], 6) for _ in range(3))
    step(a)
    no_error()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    step(b, stream=st)
    st.synchronize()
    assert all(torch.equal(p, r) for p, r in zip(bits(a), bits(b)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(g)
    graph.replay()
    no_error()
    assert all(torch.equal(p, r) for p, r in zip(bits(a), bits(g)))


def test_captured_step_replays_with_new_lengths_and_trees():
    """Lengths, counts and parents are device memory: a captured attention follows them."""
    rng = np.random.default_rng(21)
    c, par, q, ck, cv, sel = attn_setup(rng, [700, 33], [7, 7], 7, 64, 128, 16, 128, 4, 0, "tree")
    kv = c.upload()
    dq, dpar, dck, dcv = dev(q), dev(par), dev(ck), dev(cv)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(*q.shape), dtype=torch.uint8, device="cuda")
    call = lambda: ds4a.ds4a_attn_tree(kv, dq, c.dn, dpar, 128, dck, dcv, 4, None, 0.1, out, ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, n in (([700, 33], [7, 7]), ([90, 30], [3, 7]), ([650, 2], [1, 0])):
        c2, par2, q2, ck2, cv2, _ = attn_setup(rng, lens, n, 7, 64, 128, 16, 128, 4, 0, "tree")
        # the new contents in the captured tensors
        for s in range(2):
            src, dst = c2.rows(s, range(lens[s] + n[s])), c.rows(s, range(lens[s] + n[s]))
            c.k[dst], c.v[dst] = c2.k[src], c2.v[src]
        cap, cap2 = ck.shape[1], ck2.shape[1]
        nk, nv = np.full_like(ck, NAN16), np.full_like(cv, NAN16)
        nk[:, :cap2 - 7], nv[:, :cap2 - 7], nk[:, cap - 7:], nv[:, cap - 7:] = ck2[:, :-7], cv2[:, :-7], ck2[:, -7:], cv2[:, -7:]
        c.lens, c.n = list(lens), list(n)
        for t, a in ((c.dk, c.k.reshape(c.dk.shape)), (c.dv, c.v.reshape(c.dv.shape)), (c.dlen, np.array(lens, np.int64)),
                     (c.dn, np.array(n, np.int32)), (dpar, par2), (dq, q2), (dck, nk), (dcv, nv)):
            t.copy_(dev(a))
        out.fill_(7.0)
        graph.replay()
        no_error()
        check_attn(c, par2, q2, nk, nv, None, 128, 4, 0.1, out)
