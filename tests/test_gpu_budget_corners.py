"""Calls on caches held to a budget that the other tests do not make."""
import math

import numpy as np
import pytest
import torch

import budget_ref as E
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_budget import check_evict, check_weights, last_error, weights_setup
from test_gpu_tree import Cache, dev, no_error

pytestmark = pytest.mark.gpu


# ---- eviction ----------------------------------------------------------------------------------

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("ln,other,budget,bad", [
    (30, 80, 40, 1),                # one CTA a session
    (3000, 3500, 3200, 187),        # a cluster: its last page
    (600 * 16, 9700, 9650, 514),    # more pages than a CTA has threads
])
def test_evict_uncut_session_with_a_bad_page_is_left_alone(ln, other, budget, bad, in_place):
    """A page id outside the pool among a session's tokens leaves it alone, whether it would be cut or not; a bad entry
    behind them does not matter."""
    rng = np.random.default_rng(ln)
    c = Cache(rng, [ln, other, ln], [0] * 3, 64, 16, 16)
    c.table[0, bad] = c.n_pages
    c.table[2, (ln - 1) // 16 + 1] = -1
    kv = c.upload()
    S = c.mp * 16
    acc, pos = rng.random((3, S)).astype(np.float32), np.tile(np.arange(S, dtype=np.int32), (3, 1))
    da, dp = dev(acc), dev(pos)
    ao, po = (da, dp) if in_place else (torch.full_like(da, 5), torch.full_like(dp, 6))
    lo = torch.full_like(c.dlen, -4)
    ws = torch.zeros(ds4a.ds4a_evict_workspace_bytes(3, S, budget), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_evict(kv, da, dp, torch.tensor([ln, other, ln], device="cuda"), budget, 2, 5, ao, po, lo, ws)
    assert last_error() == 7
    assert lo.tolist() == [-4, budget, ln]
    want_a, want_p = (acc[0], pos[0]) if in_place else (np.full(S, 5, np.float32), np.full(S, 6, np.int32))
    assert np.array_equal(ao[0].cpu().numpy(), want_a) and np.array_equal(po[0].cpu().numpy(), want_p)
    assert np.array_equal(ao[2, :ln].cpu().numpy(), acc[2, :ln])
    place, _ = E.evict(acc[1], pos[1], other, other, budget, 2, 5)
    assert np.array_equal(po[1, :budget].cpu().numpy(), pos[1, place])


@pytest.mark.parametrize("nxt,always", [(-(1 << 63), True), (3 - (1 << 63), True), (-1, True), (5, True), (6, False),
                                        ((1 << 63) - 1, False)])
def test_evict_next_positions_at_the_ends_of_their_range(nxt, always):
    """Kept: positions of next - 5 and above, in exact arithmetic.  All of them (the lower slots stay), or only position 0's."""
    rng = np.random.default_rng(3)
    c = Cache(rng, [50], [0], 64, 16, 0)
    acc = rng.permutation(50).astype(np.float32)[None]
    acc[0, 0] = -1                              # the least, at position 0
    pos = np.arange(50, dtype=np.int32)[None]
    if not always:
        pos[0, 1:] = 0                          # 0 >= 6 - 5 is false
    da, dp, lo = dev(acc), dev(pos), torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.zeros(ds4a.ds4a_evict_workspace_bytes(1, 50, 20), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_evict(c.upload(), da, dp, torch.tensor([nxt], device="cuda"), 20, 0, 5, da, dp, lo, ws)
    no_error()
    got = np.sort(da[0, :20].cpu().numpy())
    assert np.array_equal(got, np.sort(acc[0, :20] if always else np.sort(acc[0])[-20:]))


# ---- attention weights ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,n,N,H", [([150], [3], 3, 8), ([300, 77], [5, 2], 5, 64), ([200], [33], 33, 24)])
@pytest.mark.parametrize("what", ["rows", "keys"])
def test_weights_rows_of_lse_minus_infinity_add_nothing_whatever_their_scores(lens, n, N, H, what):
    """rows: a padded token among the new ones, whose queries are NaN or infinite and whose lse is -inf.  keys: all rows'
    lse are -inf and some keys NaN or infinite."""
    rng = np.random.default_rng(N)
    scale = 0.125
    c, q, lse, acc = weights_setup(rng, lens, n, N, H, 64, 16, scale)
    if what == "rows":
        q[0, 1, :, 5], q[0, n[0] - 1, ::2] = np.nan, np.inf
        lse[0, [1, n[0] - 1]] = -np.inf
    else:
        lse[0] = -np.inf
        c.k[c.rows(0, [3, 40])], c.k[c.rows(0, [lens[0]])] = np.nan, -np.inf
        c.k[c.rows(0, [lens[0] - 1]), ::2] = np.inf
    da = dev(acc)
    ds4a.ds4a_attn_weights(c.upload(), dev(q), c.dn, dev(lse), scale, 0.5, da)
    no_error()
    got = da.cpu().numpy().astype(np.float64)
    for s, ln in enumerate(lens):
        T = ln + n[s]
        k = c.k[c.rows(s, range(T))]
        dead = lse[s, :n[s], 0] == -np.inf
        add, tol = E.weights(np.where(dead[:, None, None], 0, q[s, :n[s]]), np.where(dead.all(), 0, k), scale, lse[s, :n[s]], ln)
        old = np.where(np.arange(T) < ln, 0.5 * acc[s, :T].astype(np.float64), 0)
        assert np.isfinite(got[s, :T]).all()
        assert (np.abs(got[s, :T] - old - add) <= tol + 2.0 ** -23 * old + 2.0 ** -24 * (old + add)).all()


def bits(t):
    return t.view(torch.int32)


@pytest.mark.parametrize("lens,n,N,H,D,page", [
    ([12001 + 371 * i for i in range(8)], [4, 1, 3, 2, 4, 4, 1, 3], 4, 64, 128, 64),             # 1 or 2 chunks, two or three blocks a CTA
    ([1900 + 17 * i for i in range(40)], [1 + i % 3 for i in range(40)], 3, 64, 64, 16),         # the table, pairs, sessions of 1 - 2 chunks
    ([1000 + 29 * i for i in range(30)] + [40, 3, 0], [20 - i % 7 for i in range(30)] + [20, 0, 20], 20, 24, 64, 48),   # 4 chunks
    ([30000, 10500], [64, 33], 64, 16, 128, 128),                                                 # 8 chunks, two sessions
])
def test_weights_of_many_rows_over_more_tiles_than_ctas(lens, n, N, H, D, page):
    """Query chunks are loaded again for every block of two tiles, over several pieces of a CTA; each session gets the bits that
    it gets alone."""
    scale = 1 / math.sqrt(D)
    c, q, lse, acc = weights_setup(np.random.default_rng(N), lens, n, N, H, D, page, scale)
    kv = c.upload()
    da, dq, dl = dev(acc), dev(q), dev(lse)
    ds4a.ds4a_attn_weights(kv, dq, c.dn, dl, scale, 0.75, da)
    no_error()
    check_weights(c, q, lse, acc, da.cpu().numpy(), scale, 0.75, lens, n)
    for s in (0, len(lens) // 2):
        one = dev(acc[s:s + 1])
        ds4a.ds4a_attn_weights(ds4a.paged_kv_desc(c.dk, c.dv, c.dtab[s:s + 1].contiguous(), c.dlen[s:s + 1].contiguous()),
                               dq[s:s + 1].contiguous(), c.dn[s:s + 1].contiguous(), dl[s:s + 1].contiguous(), scale, 0.75, one)
        no_error()
        assert torch.equal(bits(one), bits(da[s:s + 1]))


# ---- eviction: clusters of two, and slices whose keys are read again each round ---------------------

@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,budget,sink,recent,extra", [
    ([2600, 3000, 2100, 1400], 1500, 4, 100, 50),                                # two CTAs a session by its slots
    ([4000] * 3, 2100, 0, 0, 90),                                                # the same, moves by the second kernel
    ([8448 - 3 * i for i in range(64)], 8192, 4, 256, 0),                        # by the batch
    ([700 - i for i in range(76)] + [3], 250, 4, 60, 41000),                     # one, not in shared memory
    ([500 + i for i in range(40)], 400, 8, 0, 90000),                            # two, not in shared memory
])
def test_evict_two_ctas_a_session_and_long_rows(lens, budget, sink, recent, extra, in_place):
    check_evict(np.random.default_rng(budget), lens, budget, sink, recent, extra=extra, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("budget", [4000, 397000])
def test_evict_few_moves_in_sessions_longer_than_shared_memory(budget, in_place):
    """Eight CTAs that read their keys again each round, and carry out the moves themselves over what they read."""
    check_evict(np.random.default_rng(6), [400001, 399000, 17], budget, 4, 1000, page=4096, in_place=in_place)


# ---- shared prefixes ----------------------------------------------------------------------------------

@pytest.mark.parametrize("B,ln", [(2, 40), (3, 5000), (40, 300)])
def test_prefix_sessions_without_a_readable_page(B, ln):
    """Zeros and an lse of -inf, joined from one piece or from many; then the weights call adds nothing."""
    rng = np.random.default_rng(B)
    c = Cache(rng, [ln + i % 7 for i in range(B)], [1 + i % 2 for i in range(B)], 64, 16, 2)
    c.draft()
    c.table[:] = np.where(np.arange(c.mp) % 2, -1, c.n_pages)
    q = rng.standard_normal((B, 2, 8, 64)).astype(np.float16)
    kv, dq = c.upload(), dev(q)
    out, lse = torch.full_like(dq, 7), torch.full((B, 2, 8), 7.0, device="cuda")
    ws = torch.full((ds4a.ds4a_attn_prefix_workspace_bytes(B, 2, 8, 64, 1),), 255, dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_prefix(kv, dq, c.dn, None, dev(np.array([0, B - 1], np.int32)), torch.tensor([ln - 3], device="cuda"), 0.125, out, lse, ws)
    assert last_error() == 7
    for s in range(B):
        assert (out[s, :c.n[s]] == 0).all() and (lse[s, :c.n[s]] == -math.inf).all()
        assert (out[s, c.n[s]:] == 7).all() and (lse[s, c.n[s]:] == 7).all()
    c.table[:] = np.arange(B * c.mp).reshape(B, c.mp)       # readable again, over tokens that are NaN and numbers
    kv = c.upload()
    acc = torch.full((B, c.mp * 16), 2.0, device="cuda")
    ds4a.ds4a_attn_weights(kv, dq, c.dn, lse, 0.125, 0.5, acc)
    no_error()
    for s in range(B):
        assert (acc[s, :c.lens[s]] == 1).all() and (acc[s, c.lens[s]:c.lens[s] + c.n[s]] == 0).all() and (acc[s, c.lens[s] + c.n[s]:] == 2).all()
