"""Drafted-token calls at the ends of their ranges: lengths and positions near the largest,
capacities that are passed, values that are not finite, calls directly behind one another."""
import math

import numpy as np
import pytest
import torch

import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_tree import NAN16, Cache, attn_setup, check_attn, comp_setup, dev, no_error, run_attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("call", ["append", "compress", "attn", "commit"])
@pytest.mark.parametrize("ln", [(1 << 63) - 1, (1 << 63) - 4, 1 << 62])
def test_lengths_near_the_end_of_int64_are_refused(call, ln):
    """len + n does not fit 64 bits: the session is past its pages all the same, and is left alone."""
    rng = np.random.default_rng(1)
    N, ratio, D, H = 4, 2, 64, 8
    c, par, q, _, _, _ = attn_setup(rng, [21, 34, 15], [4, 4, 3], N, H, D, 16, 64, 0, 0, "tree")
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D)
    c.lens[1] = ln
    kv = c.upload()
    kn = torch.ones(3, N, D, dtype=torch.float16, device="cuda")
    lo, so = torch.full((3,), -9, device="cuda"), torch.full_like(state, 5.0)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(3, N, H, D), dtype=torch.uint8, device="cuda")
    own = torch.from_numpy(c.rows(1, range(c.mp * c.page))).cuda()       # session 1's pool rows
    mine = lambda: [c.dk.view(-1, D)[own], c.dv.view(-1, D)[own], dck[1], dcv[1], lo[1], so[1], out[1]]
    before = [t.clone() for t in mine()]
    if call == "append":
        ds4a.ds4a_paged_append(kv, kn, kn, c.dn, dev(par))
    elif call == "compress":
        ds4a.ds4a_compress_tree(kv, c.dn, dev(par), dw, ratio, state, dck, dcv)
    elif call == "attn":
        ds4a.ds4a_attn_tree(kv, dev(q), c.dn, dev(par), 64, None, None, 0, None, 0.1, out, ws)
    else:
        leaf = torch.tensor([3, 3, 2], dtype=torch.int32, device="cuda")
        ds4a.ds4a_commit_tree(kv, c.dn, dev(par), leaf, lo, dw, ratio, state, so, dck, dcv)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_CAPACITY
    for b, a in zip(before, mine()):
        assert torch.equal(b.view(-1).view(torch.uint8), a.contiguous().view(-1).view(torch.uint8))
    if call == "attn":
        c.n[1] = 0
        check_attn(c, par, q, None, None, None, 64, 0, 0.1, out)
    if call == "commit":
        assert lo.tolist() == [21 + len(R.paths_of(par[0], 4)[3]), -9, 15 + len(R.paths_of(par[2], 3)[2])]


def test_compress_tree_leaves_committed_rows_past_the_capacity_alone():
    """Session 0 has more committed rows than lie before the draft's: those rows keep their bits."""
    rng = np.random.default_rng(8)
    N, D = 4, 64
    c = Cache(rng, [6, 3], [4, 4], D, 16, N)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, 1, D)
    keep = 4 + N                                     # rows 0 .. 3 before the draft's; session 0 has six
    dck, dcv = dck[:, :keep].contiguous(), dcv[:, :keep].contiguous()
    before = dck.clone(), dcv.clone()
    ds4a.ds4a_compress_tree(c.upload(), c.dn, None, dw, 1, state, dck, dcv, N=N)
    torch.cuda.synchronize()
    assert ds4a.ds4a_last_device_error() == ds4a.DS4A_ERR_CAPACITY
    for b, a in zip(before, (dck, dcv)):
        assert torch.equal(b[0].view(torch.int16), a[0].view(torch.int16))
        assert torch.isfinite(a[1, 4:]).all()        # session 1's four rows (a row of one token is the token)
    at = c.rows(1, range(3, 7))
    assert np.array_equal(dck[1, 4:].cpu().numpy(), c.k[at]) and np.array_equal(dcv[1, 4:].cpu().numpy(), c.v[at])


# page * max_pages = 2^31 - 16, the most slots that pages of multiples of 16 can hold
FAR_PAGE, FAR_PAGES = 8176, 262657


@pytest.mark.parametrize("window,ln", [(128, 2147483600), (200, 2147483611), (128, 2147483628), (64, 2147483568)])
def test_attn_tree_at_the_last_positions(window, ln):
    """Slots up to 2^31 - 17: a node attends its own tokens, and what was never written or is another
    branch's (NaN there) stays out."""
    rng = np.random.default_rng(ln % 97)
    N, H, D = 4, 16, 64
    table = np.zeros((1, FAR_PAGES), np.int32)       # page 0: NaN, nobody reads it
    table[0, -1] = 1
    k, v = np.full((2 * FAR_PAGE, D), NAN16), np.full((2 * FAR_PAGE, D), NAN16)
    rows = R.slot_rows(table[0], FAR_PAGE, range(ln - window, ln + N))
    k[rows], v[rows] = (rng.standard_normal((len(rows), D)).astype(np.float16) for _ in range(2))
    par, n = np.array([[-1, 0, 0, 1]], np.int32), 4
    v[R.slot_rows(table[0], FAR_PAGE, [ln + 2])] = NAN16
    q = rng.standard_normal((1, N, H, D)).astype(np.float16)
    pool = lambda a: dev(a.reshape(2, FAR_PAGE, D))
    kv = ds4a.paged_kv_desc(pool(k), pool(v), dev(table), torch.tensor([ln], device="cuda"))
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(1, N, H, D), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_tree(kv, dev(q), torch.tensor([n], dtype=torch.int32, device="cuda"), dev(par), window, None, None, 0,
                        None, 0.125, out, ws)
    no_error()
    for i, path in enumerate(R.paths_of(par[0], n)):
        if i == 2:
            assert torch.isnan(out[0, i]).all()
            continue
        kk, vv = R.node_keys(k, v, None, None, table[0], FAR_PAGE, ln, path, N, window, 0, None)
        want, tol = R.attend(q[0, i], kk, vv, 0.125)
        assert (np.abs(out[0, i].cpu().numpy().astype(np.float64) - want) <= tol).all(), i


def test_append_and_commit_at_the_last_positions():
    """The angle, in radians, at positions below 2^31 with f <= 1: f / 2 pi is off by two roundings of
    2^-53 each, which is 2^-21 at 2^31 positions; what is dropped below 2^-64 and 2^-32 of a turn 2^-29;
    float(angle) 2^-23.3; the sine's own error 2^-23: below 2^-20.  The products and their sum add
    2^-23 of |x1| + |x2| < 8: in all below 8 * 2^-19, beside the rounding to 16 bits.  The oracle
    takes the angle modulo a turn in integers."""
    rng = np.random.default_rng(0)
    D, N, ln = 64, 4, (1 << 31) - 16 - 4
    turn = int("6283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234135")  # 2 pi * 10^99
    table = np.zeros((1, FAR_PAGES), np.int32)
    table[0, -1] = 1
    pk = torch.zeros(2, FAR_PAGE, D, dtype=torch.float16, device="cuda")
    pv, length = torch.zeros_like(pk), torch.tensor([ln], device="cuda")
    kv = ds4a.paged_kv_desc(pk, pv, dev(table), length)
    k = rng.uniform(-3, 3, (1, N, D)).astype(np.float16)
    inv = np.array([1.0, 0.7, 2.0 ** -20, 1e-3, 1e-6, 0.5, 0.25, 0.0], np.float32)
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    par = np.array([[-1, 0, 0, 2]], np.int32)
    ds4a.ds4a_paged_append(kv, dev(k), dev(k), n, dev(par), dev(inv), 16, True)
    no_error()
    at = R.slot_rows(table[0], FAR_PAGE, range(ln, ln + N))
    got = pk.view(-1, D).cpu().numpy()[at].astype(np.float64)
    for i, path in enumerate(R.paths_of(par[0], N)):
        pos = ln + len(path) - 1
        th = []
        for f in inv:
            num, den = float(f).as_integer_ratio()
            th.append((pos * num * 10 ** 99 // den) % turn / 10 ** 99)
        want = R.rotate(k[0, i].astype(np.float64), 1, np.array(th), 16, True)
        assert (np.abs(got[i] - want) <= 2.0 ** -11 * np.abs(want) + 8 * 2.0 ** -19).all(), i
    ds4a.ds4a_commit_tree(kv, n, dev(par), torch.tensor([3], dtype=torch.int32, device="cuda"), length)
    no_error()
    assert length.item() == ln + 3
    moved = pk.view(-1, D).cpu().numpy()[at].astype(np.float64)
    assert np.array_equal(moved[:3], got[[0, 2, 3]])


# ways of cutting the work: two row blocks, one (its sides joined), one line of key tiles (its pieces joined)
CUTS = [(40, 10, 64, 96, 4, lambda s: 130 + 11 * s), (3, 6, 16, 200, 0, lambda s: 300 + s),
        (2, 6, 64, 1 << 30, 16, lambda s: 6000 - 900 * s)]


@pytest.mark.parametrize("B,N,H,window,ratio,lens", CUTS)
@pytest.mark.parametrize("common,own", [(np.nan, np.inf), (-np.inf, np.inf), (np.inf, -np.inf), (np.nan, -np.inf),
                                        (np.inf, np.inf)])
def test_attn_tree_adds_values_that_are_not_finite(B, N, H, window, ratio, lens, common, own):
    """A token that every node attends and a drafted one that some do, both with a value that is not
    finite in one column: the nodes that attend both get their sum."""
    rng = np.random.default_rng(B + N)
    ln, n = [lens(s) for s in range(B)], [N - s % 2 for s in range(B)]
    c, par, q, ck, cv, _ = attn_setup(rng, ln, n, N, H, 128, 16, window, ratio, 0, "tree")
    for s in range(B):
        c.v[c.rows(s, [ln[s] - 30]), 5] = common
        c.v[c.rows(s, [ln[s] + 1]), 5] = own
    out = run_attn(c, par, q, ck, cv, None, window, ratio, 0.09)
    no_error()
    o = out.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        both = common + own
    for s in range(B):
        for i, path in enumerate(R.paths_of(par[s], n[s])):
            want = both if 1 in path else common
            got = o[s, i, :, 5]
            assert np.isnan(got).all() if np.isnan(want) else (got == want).all(), (s, i)
            assert np.isfinite(np.delete(o[s, i], 5, 1)).all()


def test_attn_tree_keeps_nan_of_far_smaller_weights():
    """One node over a long cache, cut into pieces: a NaN in V whose weight underflows beside the
    others' is still a term of the sum."""
    rng = np.random.default_rng(3)
    ln = 9000
    c, par, q, _, _, _ = attn_setup(rng, [ln], [1], 1, 8, 128, 64, 1 << 30, 0, 0, "chain")
    q[0, 0] = np.abs(q[0, 0]) + np.float16(0.5)
    c.k[c.rows(0, range(ln))] = np.float16(-2.0)     # scores below -64: 2^-160 beside the newest token's
    c.k[c.rows(0, [ln])] = np.float16(1.0)
    c.v[c.rows(0, [100]), 7] = NAN16
    out = run_attn(c, par, q, None, None, None, 1 << 30, 0, 1.0)
    no_error()
    assert torch.isnan(out[0, 0, :, 7]).all()
    rest = torch.cat([out[0, 0, :, :7], out[0, 0, :, 8:]], 1)
    v = dev(c.v[c.rows(0, [ln])])[0]
    assert torch.equal(rest, torch.cat([v[:7], v[8:]]).expand_as(rest))


@pytest.mark.parametrize("B,N,H,window,ratio,lens", CUTS)
def test_attn_tree_over_scores_that_are_all_minus_infinity(B, N, H, window, ratio, lens):
    """A softmax without a finite score is NaN, as by its definition; with one finite score it is
    that row's value."""
    rng = np.random.default_rng(7)
    ln, n = [lens(s) for s in range(B)], [N] * B
    c, par, q, ck, cv, _ = attn_setup(rng, ln, n, N, H, 128, 16, window, ratio, 0, "roots")
    q[..., 0] = np.float16(1.0)
    q[:, :, 1, 0] = np.float16(-1.0)                 # head 1: +inf scores, NaN in any case
    for s in range(B):
        c.k[c.rows(s, range(ln[s] + n[s])), 0] = np.float16(-np.inf)
    if ratio:
        ck[:, :, 0] = np.where(np.isnan(ck[:, :, 0]), NAN16, np.float16(-np.inf))
    k2 = [c.rows(s, [ln[s] + 2])[0] for s in range(B)]
    for s in range(0, B, 2):                         # even sessions: node 2 has a finite score for itself
        c.k[k2[s], 0] = np.float16(0.25)
    out = run_attn(c, par, q, ck, cv, None, window, ratio, 0.09)
    no_error()
    for s in range(B):
        for i in range(N):
            if s % 2 == 0 and i == 2:
                o = torch.cat([out[s, i, :1], out[s, i, 2:]])
                assert torch.equal(o, dev(c.v[k2[s]]).expand_as(o)), s
                assert torch.isnan(out[s, i, 1]).all()
            else:
                assert torch.isnan(out[s, i]).all(), (s, i)


def test_attn_tree_one_key_of_minus_infinity():
    """A window of one token, whose score is -inf."""
    rng = np.random.default_rng(2)
    c, par, q, _, _, _ = attn_setup(rng, [20], [2], 2, 8, 64, 16, 1, 0, 0, "roots")
    q[..., 3] = np.float16(2.0)
    c.k[c.rows(0, [20]), 3] = np.float16(-np.inf)
    out = run_attn(c, par, q, None, None, None, 1, 0, 0.1)
    no_error()
    assert torch.isnan(out[0, 0]).all()
    v = dev(c.v[c.rows(0, [21])])[0]
    assert torch.equal(out[0, 1], v.expand_as(out[0, 1]))


@pytest.mark.parametrize("first", [True, False])
def test_attn_tree_one_dominant_key_over_a_long_tail(first):
    """2^18 keys of weight e^-17 .. e^-21 and V = 1 beside one of weight 1 and V = 0: 1e-2 .. 2e-4 in all.

    A weight is rounded to 16 bits beside a reference of 2^7 or more, half a step being 2^-11 of it, or
    2^-25 below the smallest normal, 2^-32 of the largest weight: 2^-11 of the result and n 2^-32.  The
    scores have one product, exact; log2(e), its product with the score and the difference are off by
    2^-24 of at most 32 each, and 2^x by 2^-22: 2^-17 in a weight.  The sum: parts of 64 (64 2^-24) and
    at most 4096 of those (2^-12).  The accumulator, of binary32, holds only what these keys gave; each
    product may lose 2^-24 of it: for 2^17 keys a side, the accumulator half full on average, 2^-8.  The
    result's own rounding: 2^-11 of it, or 2^-25."""
    B = torch.cuda.get_device_properties(0).multi_processor_count     # a whole row tile a CTA
    N, H, D, page, ln = 2, 64, 128, 4096, 1 << 18
    pages = ln // page + 1
    k, v = np.zeros((pages, page, D), np.float16), np.ones((pages, page, D), np.float16)
    at = 5 if first else ln - 1
    k.reshape(-1, D)[at, 0] = 17.0
    v.reshape(-1, D)[at] = 0.0
    k.reshape(-1, D)[ln:ln + 2, 0] = -50.0           # the drafted tokens themselves: nothing
    q = np.zeros((B, N, H, D), np.float16)
    q[:, :, :, 0] = (1 + np.arange(H) / 256).astype(np.float16)
    table = np.tile(np.arange(pages, dtype=np.int32), (B, 1))         # the sessions share their pages
    kv = ds4a.paged_kv_desc(dev(k), dev(v), dev(table), torch.full((B,), ln, device="cuda"))
    n = torch.full((B,), N, dtype=torch.int32, device="cuda")
    out = torch.zeros(B, N, H, D, dtype=torch.float16, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(B, N, H, D), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_tree(kv, dev(q), n, None, 1 << 30, None, None, 0, None, 1.0, out, ws)
    no_error()
    got = out.cpu().numpy().astype(np.float64)
    gap = q[0, 0, :, 0].astype(np.float64) * 17.0
    tail = (ln - 1) * np.exp(-gap)
    want = (tail / (1 + tail))[:, None]
    tol = want * (2.0 ** -8 + 2 * 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16) + ln * 2.0 ** -32 + 2.0 ** -25
    err = np.abs(got - want)
    assert (err <= tol).all(), float((err / tol).max())


def captured(*calls):
    """The calls directly behind one another in a graph."""
    for call in calls:
        call()                                       # once on the stream: set-up is done
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    return graph


@pytest.mark.parametrize("N", [1, 700])
def test_decode_attention_directly_behind_an_append(N):
    """ds4a_attn_decode reads queries and window rows before its dependency wait: an append directly
    ahead of it that writes them has finished by then."""
    rng = np.random.default_rng(N)
    D, H, page, ln = 128, 64, 64, 40
    mp = (ln + N) // page + 1
    pk, pv = (torch.randn(mp, page, D, device="cuda").half() for _ in range(2))
    kv = ds4a.paged_kv_desc(pk, pv, torch.arange(mp, dtype=torch.int32, device="cuda")[None], torch.tensor([ln], device="cuda"))
    k, v = (dev(rng.standard_normal((1, N, D)).astype(np.float16)) for _ in range(2))
    q = dev(rng.standard_normal((1, N, H, D)).astype(np.float16))
    qo, n = torch.zeros_like(q), torch.tensor([N], dtype=torch.int32, device="cuda")
    inv = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    w0 = ln + N - 33                                 # the newest 33 tokens as the window
    fk, fv = pk.view(-1, D), pv.view(-1, D)
    out = torch.zeros(H, D, dtype=torch.float16, device="cuda")
    append = lambda: ds4a.ds4a_paged_append(kv, k, v, n, None, inv, 64, True, q, qo)
    decode = lambda: ds4a.ds4a_attn_decode(qo[0, N - 1], fk[w0:ln + N], fv[w0:ln + N], None, None, None, 0, 0.088, out)
    graph = captured(append, decode)
    torch.cuda.synchronize()
    append()
    torch.cuda.synchronize()
    decode()
    torch.cuda.synchronize()
    want = out.clone()
    for _ in range(50):
        qo.fill_(math.nan)
        fk[ln:ln + N] = math.nan
        fv[ln:ln + N] = math.nan
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        no_error()
        assert torch.equal(out, want)


def test_indexer_directly_behind_a_commit():
    """ds4a_indexer_topk reads key rows before its dependency wait: a commit directly ahead of it that
    moves them into place has finished by then."""
    rng = np.random.default_rng(4)
    D, N, ratio, ln, topk = 128, 64, 1, 70, 32
    c = Cache(rng, [ln], [N], D, 16, N)
    c.draft()
    ck, cv, w, state, dck, dcv, dw = comp_setup(rng, c, ratio, D)
    cap = ck.shape[1]
    kidx = torch.randn(1, cap, D, device="cuda").half()
    kidx[0, cap - N:] *= 4                           # the path's rows rank first
    kv, leaf, lo = c.upload(), torch.tensor([N - 1], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    qi = torch.randn(1, D, device="cuda").half()
    sel = torch.zeros(1, topk, dtype=torch.int32, device="cuda")
    ws = torch.zeros(ds4a.ds4a_indexer_workspace_bytes(1, cap, topk), dtype=torch.uint8, device="cuda")
    so = state.clone()
    commit = lambda: ds4a.ds4a_commit_tree(kv, c.dn, None, leaf, lo, dw, ratio, state, so, dck, dcv, kidx, N=N)
    rank = lambda: ds4a.ds4a_indexer_topk(qi, kidx[0], ln + N, ratio, topk, sel, None, ws, n_rows=ln + N)
    graph = captured(commit, rank)
    commit()
    torch.cuda.synchronize()
    rank()
    torch.cuda.synchronize()
    want = sel.clone()
    assert (want >= ln).sum() > topk // 2
    for _ in range(50):
        kidx[0, ln:ln + N] = 0
        sel.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        no_error()
        assert torch.equal(sel, want)


@pytest.mark.parametrize("ratio", [4, 128])
def test_three_drafts_one_after_the_other(ratio):
    """Drafts checked and committed three times over one cache: every node's output is what
    ds4a_attn_decode gives over its path, rows completed in a draft among what the next attends."""
    rng = np.random.default_rng(ratio)
    N, H, D, room = 12, 64, 128, 40
    c = Cache(rng, [300, 118, 0], [11, 9, 6], D, 16, N + room)
    c.N = N
    ck0, cv0, w, state, ck, cv, dw = comp_setup(rng, c, ratio, D, room=N + room)
    kv = c.upload()
    out = torch.zeros(3, N, H, D, dtype=torch.float16, device="cuda")
    qr = torch.zeros_like(out)
    inv = dev((10000.0 ** (-np.arange(32) / 32)).astype(np.float32))
    ws = torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(3, N, H, D), dtype=torch.uint8, device="cuda")
    pk, pv = c.dk.view(-1, D), c.dv.view(-1, D)
    drafts = 0
    for _ in range(3):
        lens = c.dlen.tolist()
        par = R.random_parents(rng, 3, N)
        dpar, leaf = dev(par), [n - 1 for n in c.n]
        k, v = (dev(rng.standard_normal((3, N, D)).astype(np.float16)) for _ in range(2))
        q = dev(rng.standard_normal((3, N, H, D)).astype(np.float16))
        ds4a.ds4a_paged_append(kv, k, v, c.dn, dpar, inv, 64, True, q, qr)
        ds4a.ds4a_compress_tree(kv, c.dn, dpar, dw, ratio, state, ck, cv)
        ds4a.ds4a_attn_tree(kv, qr, c.dn, dpar, 128, ck, cv, ratio, None, 0.088, out, ws)
        no_error()
        after = []
        for s in range(3):
            for i, path in enumerate(R.paths_of(par[s], c.n[s])):
                st, tk, tv = state[s].clone(), ck[s].clone(), cv[s].clone()
                slots = [lens[s] + j for j in path]
                for d, t in enumerate(slots):
                    r = c.rows(s, [t])[0]
                    ds4a.ds4a_compress_append(pk[r:r + 1], pv[r:r + 1], dw, ratio, lens[s] + d, st, tk, tv)
                p = lens[s] + len(path) - 1
                win = [t if t < lens[s] else slots[t - lens[s]] for t in range(max(0, p - 127), p + 1)]
                at = torch.from_numpy(c.rows(s, win)).cuda()
                ref = torch.empty(H, D, dtype=torch.float16, device="cuda")
                wk, wv = pk[at], pv[at]
                torch.cuda.synchronize()
                ds4a.ds4a_attn_decode(qr[s, i], wk, wv, tk, tv, None, (p + 1) // ratio, 0.088, ref)
                torch.cuda.synchronize()
                # two 16-bit results of one value: both are within the repository's 2e-3 of it
                assert float((ref.float() - out[s, i].float()).abs().max()) <= 4e-3, (drafts, s, i)
                if i == leaf[s]:
                    after.append((lens[s] + len(path), st, tk, tv))
        ds4a.ds4a_commit_tree(kv, c.dn, dpar, dev(np.array(leaf, np.int32)), c.dlen, dw, ratio, state, state, ck, cv)
        no_error()
        for s, (ln, st, tk, tv) in enumerate(after):
            assert c.dlen[s].item() == ln
            m = ln // ratio
            assert torch.equal(ck[s, :m].view(torch.int16), tk[:m].view(torch.int16))
            assert torch.equal(cv[s, :m].view(torch.int16), tv[:m].view(torch.int16))
            if ln % ratio:
                assert torch.equal(state[s].view(torch.int32), st.view(torch.int32))
        drafts += 1
    assert drafts == 3 and c.dlen.max().item() <= c.mp * c.page


def test_bound_calls_repeat_the_calls():
    """ds4a.bind marshals each of the four calls once: the same bits as the calls themselves."""
    def setup():
        rng = np.random.default_rng(6)
        N, H, D, ratio = 5, 16, 64, 3
        c, par, q, _, _, _ = attn_setup(rng, [50, 13], [5, 4], N, H, D, 16, 32, 0, 0, "tree")
        _, _, _, state, ck, cv, dw = comp_setup(rng, c, ratio, D)
        kv = c.upload()
        k, v = (dev(rng.standard_normal((2, N, D)).astype(np.float16)) for _ in range(2))
        t = dict(q=dev(q), qo=torch.zeros(2, N, H, D, dtype=torch.float16, device="cuda"), par=dev(par), lo=torch.zeros_like(c.dlen),
                 out=torch.zeros(2, N, H, D, dtype=torch.float16, device="cuda"), so=state.clone(), state=state, ck=ck, cv=cv,
                 leaf=torch.tensor([4, 2], dtype=torch.int32, device="cuda"), k=k, v=v, w=dw,
                 inv=dev((10000.0 ** (-np.arange(16) / 16)).astype(np.float32)),
                 ws=torch.zeros(ds4a.ds4a_attn_tree_workspace_bytes(2, N, H, D), dtype=torch.uint8, device="cuda"))
        calls = [("ds4a_paged_append", (kv, k, v, c.dn, t["par"], t["inv"], 16, False, t["q"], t["qo"])),
                 ("ds4a_compress_tree", (kv, c.dn, t["par"], dw, ratio, state, ck, cv)),
                 ("ds4a_attn_tree", (kv, t["qo"], c.dn, t["par"], 32, ck, cv, ratio, None, 0.125, t["out"], t["ws"])),
                 ("ds4a_commit_tree", (kv, c.dn, t["par"], t["leaf"], t["lo"], dw, ratio, state, t["so"], ck, cv))]
        return c, t, calls
    a, b = setup(), setup()
    for name, args in a[2]:
        getattr(ds4a, name)(*args)
    for call in [ds4a.bind(name, *args) for name, args in b[2]]:
        call()
    no_error()
    for x, y in zip((a[0].dk, a[0].dv) + tuple(a[1][n] for n in ("qo", "out", "lo", "so", "ck", "cv")),
                    (b[0].dk, b[0].dv) + tuple(b[1][n] for n in ("qo", "out", "lo", "so", "ck", "cv"))):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.isfinite(a[1]["out"][0].float()).all() and a[1]["lo"].tolist() == [50 + len(R.paths_of(a[1]["par"][0].tolist(), 5)[4]),
                                                                                  13 + len(R.paths_of(a[1]["par"][1].tolist(), 4)[2])]
