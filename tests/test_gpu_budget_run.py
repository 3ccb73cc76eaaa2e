"""The calls on shared prefixes and budgeted caches used together, captured, bound and side by side: sessions
that share a prompt decode token by token over a cache that is cut to its budget."""
import math

import numpy as np
import pytest
import torch

import budget_ref as E
import tree_ref as R
from compressed_sparse_mqa_gb300 import ds4a
from test_gpu_tree import dev, no_error

pytestmark = pytest.mark.gpu

B, H, D, PAGE, SHARED, EPS, SCALE = 3, 16, 64, 16, 37, 1e-5, 0.3
BUDGET, SINK, RECENT, SLOTS = 60, 40, 8, 80
INV = (10000.0 ** (-np.arange(16) / 16)).astype(np.float32)
ROT = dict(rot_off=16, interleaved=False)


class Server:
    """Three sessions over one prompt of 37 tokens (its whole pages shared), a cache of 60 tokens each."""

    def __init__(self, seed):
        rng = np.random.default_rng(seed)
        mp = SLOTS // PAGE
        table = np.arange(B * mp).reshape(B, mp).astype(np.int32)
        table[1:, :SHARED // PAGE] = table[0, :SHARED // PAGE]
        self.table = table
        self.pk = torch.zeros(B * mp, PAGE, D, dtype=torch.float16, device="cuda")
        self.pv = torch.zeros_like(self.pk)
        self.length = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.next = torch.zeros(B, dtype=torch.int64, device="cuda")
        self.kv = ds4a.paged_kv_desc(self.pk, self.pv, dev(table), self.length)
        self.kw, self.qw = (1 + 0.2 * rng.standard_normal(D)).astype(np.float32), (1 + 0.2 * rng.standard_normal(D)).astype(np.float32)
        self.dkw, self.dqw, self.inv = dev(self.kw), dev(self.qw), dev(INV)
        self.acc, self.pos = torch.zeros(B, SLOTS, device="cuda"), torch.full((B, SLOTS), -1, dtype=torch.int32, device="cuda")
        self.one = torch.ones(B, dtype=torch.int32, device="cuda")
        self.start, self.shared = dev(np.array([0, B], np.int32)), torch.tensor([SHARED], device="cuda")
        self.q = torch.zeros(B, 1, H, D, dtype=torch.float16, device="cuda")
        self.out, self.lse = torch.zeros_like(self.q), torch.zeros(B, 1, H, device="cuda")
        self.ws = torch.zeros(ds4a.ds4a_attn_prefix_workspace_bytes(B, 1, H, D, 1), dtype=torch.uint8, device="cuda")
        self.ews = torch.zeros(ds4a.ds4a_evict_workspace_bytes(B, SLOTS, BUDGET), dtype=torch.uint8, device="cuda")
        # the prompt: the first session's pages; the others copy the page that it ends in
        k, v = (rng.standard_normal((B, SHARED, D)).astype(np.float16) for _ in range(2))
        n = torch.tensor([SHARED, 0, 0], dtype=torch.int32, device="cuda")
        ds4a.ds4a_paged_append_norm(self.kv, dev(k), dev(v), n, self.dkw, self.dqw, EPS, None, self.inv, **ROT, pos0=self.next,
                                    slot_pos=self.pos)
        for s in range(1, B):
            self.pk[table[s, SHARED // PAGE]], self.pv[table[s, SHARED // PAGE]] = (x[table[0, SHARED // PAGE]] for x in (self.pk, self.pv))
            self.pos[s] = self.pos[0]
        self.length.fill_(SHARED)
        self.next.fill_(SHARED)
        self.prompt_k, self.prompt_v = k[0], v[0]

    def token(self, rng):
        return [dev(rng.standard_normal(shape).astype(np.float16)) for shape in ((B, 1, D), (B, 1, D), (B, 1, H, D))]

    def step(self, k, v, q, evict):
        ds4a.ds4a_paged_append_norm(self.kv, k, v, self.one, self.dkw, self.dqw, EPS, None, self.inv, **ROT, q=q, q_out=self.q,
                                    pos0=self.next, slot_pos=self.pos)
        ds4a.ds4a_attn_prefix(self.kv, self.q, self.one, None, self.start, self.shared, SCALE, self.out, self.lse, self.ws)
        ds4a.ds4a_attn_weights(self.kv, self.q, self.one, self.lse, SCALE, 0.875, self.acc)
        self.length.add_(1)
        self.next.add_(1)
        if evict:
            ds4a.ds4a_evict(self.kv, self.acc, self.pos, self.next, BUDGET, SINK, RECENT, self.acc, self.pos, self.length, self.ews)


def test_sessions_over_one_prompt_held_to_a_budget():
    rng = np.random.default_rng(11)
    srv = Server(12)
    no_error()
    keys = [{p: (srv.prompt_k[p], srv.prompt_v[p]) for p in range(SHARED)} for _ in range(B)]   # raw tokens by position
    sums = [{p: 0.0 for p in range(SHARED)} for _ in range(B)]
    slack = [{p: 0.0 for p in range(SHARED)} for _ in range(B)]
    evictions = 0
    for step in range(40):
        k, v, q = srv.token(rng)
        before = [srv.pos[s, :int(srv.length[s])].tolist() for s in range(B)]
        nxt = srv.next.tolist()
        evict = step % 6 == 5
        srv.step(k, v, q, False)
        no_error()
        acc, pos, ln = srv.acc.cpu().numpy(), srv.pos.cpu().numpy(), srv.length.tolist()
        flat = srv.pk.cpu().numpy().reshape(-1, D), srv.pv.cpu().numpy().reshape(-1, D)
        qg, out, lse = srv.q.cpu().numpy(), srv.out.cpu().numpy(), srv.lse.cpu().numpy()
        for s in range(B):
            keys[s][nxt[s]] = (k[s, 0].cpu().numpy(), v[s, 0].cpu().numpy())
            order = before[s] + [nxt[s]]
            assert pos[s, :ln[s]].tolist() == order and len(set(order)) == len(order)
            rows = R.slot_rows(srv.table[s], PAGE, range(ln[s]))
            # what is cached is each position's token: values to the bit, keys normed and rotated to their own position
            assert np.array_equal(flat[1][rows], np.stack([keys[s][p][1] for p in order]))
            want = np.stack([R.rotate(E.norm(keys[s][p][0].astype(np.float64), srv.kw, EPS), p, INV, 16, False) for p in order])
            tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2 * np.abs(want).max() * 2.0 ** -18     # as in the append's test
            assert (np.abs(flat[0][rows].astype(np.float64) - want) <= tol).all()
            # attention over what is cached, and the running sums
            kk, vv = flat[0][rows].astype(np.float64), flat[1][rows].astype(np.float64)
            ref, tol = R.attend(qg[s, 0], kk, vv, SCALE)
            assert (np.abs(out[s, 0].astype(np.float64) - ref) <= tol).all()
            add, t = E.weights(qg[s], flat[0][rows], SCALE, lse[s], ln[s] - 1)
            for i, p in enumerate(order):
                old, off = (sums[s][p], slack[s][p]) if p != nxt[s] else (0.0, 0.0)
                sums[s][p] = 0.875 * old + add[i]
                slack[s][p] = 0.875 * off + t[i] + 2.0 ** -22 * sums[s][p]
                assert abs(acc[s, i] - sums[s][p]) <= slack[s][p]
        if evict:
            evictions += max(ln) > BUDGET
            ds4a.ds4a_evict(srv.kv, srv.acc, srv.pos, srv.next, BUDGET, SINK, RECENT, srv.acc, srv.pos, srv.length, srv.ews)
            no_error()
            got, left = srv.pos.cpu().numpy(), srv.length.tolist()
            for s in range(B):
                place, _ = E.evict(acc[s], pos[s], srv.next[s].item(), ln[s], BUDGET, SINK, RECENT)
                assert left[s] == len(place) and np.array_equal(got[s, :left[s]], pos[s, place])
                assert np.array_equal(srv.acc[s, :left[s]].cpu().numpy(), acc[s, place])
                assert set(range(SINK)) <= set(got[s, :left[s]])      # the shared prompt stays whole
    assert evictions >= 2


def test_the_same_steps_captured():
    """A captured step (with its eviction) replayed gives the bits of the calls."""
    rng = np.random.default_rng(13)
    a, b = Server(14), Server(14)
    tokens = [a.token(rng) for _ in range(45)]
    buf = [torch.zeros_like(t) for t in tokens[0]]
    g, warm = torch.cuda.CUDAGraph(), Server(14)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step(*buf, True)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        b.step(*buf, True)
    for t in tokens:
        for x, y in zip(buf, t):
            x.copy_(y)
        a.step(*t, True)
        g.replay()
        no_error()
        for x, y in ((a.out, b.out), (a.lse, b.lse), (a.acc, b.acc), (a.pk, b.pk), (a.pv, b.pv)):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(a.pos, b.pos) and torch.equal(a.length, b.length)


def test_bound_calls_give_the_bits_of_the_calls():
    rng = np.random.default_rng(15)
    a, b = Server(16), Server(16)
    k, v, q = a.token(rng)
    calls = [ds4a.bind("ds4a_paged_append_norm", b.kv, k, v, b.one, b.dkw, b.dqw, EPS, None, b.inv, **ROT, q=q, q_out=b.q,
                       pos0=b.next, slot_pos=b.pos),
             ds4a.bind("ds4a_attn_prefix", b.kv, b.q, b.one, None, b.start, b.shared, SCALE, b.out, b.lse, b.ws),
             ds4a.bind("ds4a_attn_weights", b.kv, b.q, b.one, b.lse, SCALE, 0.875, b.acc),
             ds4a.bind("ds4a_evict", b.kv, b.acc, b.pos, b.next, BUDGET, SINK, RECENT, b.acc, b.pos, b.length, b.ews)]
    for _ in range(30):
        a.step(k, v, q, True)
        for c in calls[:3]:
            c()
        b.length.add_(1)
        b.next.add_(1)
        calls[3]()
        no_error()
        for x, y in ((a.out, b.out), (a.lse, b.lse), (a.acc, b.acc), (a.pk, b.pk), (a.pv, b.pv)):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(a.pos, b.pos) and torch.equal(a.length, b.length)


def test_a_call_without_tokens_does_not_let_the_next_one_start():
    """Sessions without new tokens have no rows to join; what follows waits for the attention all the same: eviction
    behind it in a captured graph, over many replays, gives the bits of the calls one by one."""
    rng = np.random.default_rng(21)
    a, b = Server(22), Server(22)
    for _ in range(30):                                   # past the budget
        t = a.token(rng)
        a.step(*t, False)
        b.step(*t, False)
    none = torch.zeros(B, dtype=torch.int32, device="cuda")
    for srv in (a, b):
        srv.out.fill_(5)
        srv.lse.fill_(6)

    def attend_none(srv):
        ds4a.ds4a_attn_prefix(srv.kv, srv.q, none, None, srv.start, srv.shared, SCALE, srv.out, srv.lse, srv.ws)
        ds4a.ds4a_attn_weights(srv.kv, srv.q, none, srv.lse, SCALE, 0.875, srv.acc)

    def cut(srv):
        ds4a.ds4a_evict(srv.kv, srv.acc, srv.pos, srv.next, BUDGET, SINK, RECENT, srv.acc, srv.pos, srv.length, srv.ews)
    before = [x.clone() for x in (b.acc, b.pos, b.length, b.pk, b.pv)]
    attend_none(a)
    torch.cuda.synchronize()
    assert (a.out == 5).all() and (a.lse == 6).all() and torch.equal(a.acc, before[0])
    cut(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attend_none(b)
        cut(b)
    for _ in range(20):
        for x, y in zip((b.acc, b.pos, b.length, b.pk, b.pv), before):
            x.copy_(y)
        g.replay()
        no_error()
        assert (b.out == 5).all() and torch.equal(a.pos, b.pos) and torch.equal(a.acc, b.acc)
        assert torch.equal(a.pk.view(torch.int16), b.pk.view(torch.int16)) and b.length.tolist() == a.length.tolist()


def test_two_streams_at_once():
    """Two servers on two streams, each with workspaces of its own, give what they give alone."""
    rng = np.random.default_rng(17)
    ref, pair = Server(18), [Server(18), Server(18)]
    tokens = [ref.token(rng) for _ in range(30)]
    for t in tokens:
        ref.step(*t, True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    for t in tokens:
        for srv, st in zip(pair, streams):
            with torch.cuda.stream(st):
                srv.step(*t, True)
    no_error()
    for srv in pair:
        for x, y in ((ref.out, srv.out), (ref.acc, srv.acc), (ref.pk, srv.pk)):
            assert torch.equal(x.view(torch.int16), y.view(torch.int16))
        assert torch.equal(ref.pos, srv.pos)


# ---- arrays past 4 GB ------------------------------------------------------------------------------

def test_pages_past_32_bits():
    """Pools of 9 GB each: tokens appended to, attended in and moved between the last pages."""
    rng = np.random.default_rng(19)
    page, d, n_pages, ln = 512, 128, 70000, 700
    pk = torch.empty(n_pages, page, d, dtype=torch.float16, device="cuda")
    pv = torch.empty_like(pk)
    table = np.array([[n_pages - 1, 3], [n_pages - 1, n_pages - 2]], np.int32)     # the first page is shared
    length = torch.tensor([512, 512], device="cuda")
    kv = ds4a.paged_kv_desc(pk, pv, dev(table), length)
    k, v = (rng.standard_normal((2, 188, d)).astype(np.float16) for _ in range(2))
    first = [rng.standard_normal((512, d)).astype(np.float16) for _ in range(2)]
    pk[n_pages - 1], pv[n_pages - 1] = dev(first[0]), dev(first[1])
    q = rng.standard_normal((2, 188, 8, d)).astype(np.float16)
    dq = dev(q)
    qo = torch.zeros_like(dq)
    pos = torch.arange(1024, dtype=torch.int32, device="cuda").repeat(2, 1).contiguous()
    n = torch.full((2,), 188, dtype=torch.int32, device="cuda")
    ds4a.ds4a_paged_append_norm(kv, dev(k), dev(v), n, None, None, EPS, None, None, 0, True, dq, qo, None, pos)
    no_error()
    for s, p in ((0, 3), (1, n_pages - 2)):
        want = E.norm(k[s].astype(np.float64), None, EPS)
        got = pk[p, :188].cpu().numpy().astype(np.float64)
        assert (np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25 + 2 * np.abs(want).max() * 2.0 ** -18).all()
        assert np.array_equal(pv[p, :188].cpu().numpy(), v[s])
    length.fill_(ln - 1)
    keys = [np.concatenate([first[0], pk[p, :188].cpu().numpy()]) for p in (3, n_pages - 2)]
    vals = [np.concatenate([first[1], v[s]]) for s in range(2)]
    q1 = qo[:, -1:].contiguous()
    out, lse = torch.zeros_like(q1), torch.zeros(2, 1, 8, device="cuda")
    one = torch.ones(2, dtype=torch.int32, device="cuda")
    ws = torch.zeros(ds4a.ds4a_attn_prefix_workspace_bytes(2, 1, 8, d, 1), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_prefix(kv, q1, one, None, dev(np.array([0, 2], np.int32)), torch.tensor([512], device="cuda"), 0.1, out, lse, ws)
    acc = torch.zeros(2, 1024, device="cuda")
    ds4a.ds4a_attn_weights(kv, q1, one, lse, 0.1, 1.0, acc)
    no_error()
    for s in range(2):
        want, tol = R.attend(q1[s, 0].cpu().numpy(), keys[s].astype(np.float64), vals[s].astype(np.float64), 0.1)
        assert (np.abs(out[s, 0].cpu().numpy().astype(np.float64) - want) <= tol).all()
        add, t = E.weights(q1[s].cpu().numpy(), keys[s], 0.1, lse[s].cpu().numpy(), ln - 1)
        assert (np.abs(acc[s, :ln].cpu().numpy() - add) <= t).all()
    # the second session alone drops tokens (its first page its own again)
    own = table[1:].copy()
    own[0, 0] = 5
    pk[5], pv[5] = pk[n_pages - 1], pv[n_pages - 1]
    one_len = torch.tensor([ln], device="cuda")
    kv1 = ds4a.paged_kv_desc(pk, pv, dev(own), one_len)
    a1, p1 = acc[1:].contiguous(), pos[1:].contiguous()
    a0, p0 = a1.cpu().numpy()[0], p1.cpu().numpy()[0]
    ews = torch.zeros(ds4a.ds4a_evict_workspace_bytes(1, 1024, 300), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_evict(kv1, a1, p1, torch.tensor([ln], device="cuda"), 300, 4, 100, a1, p1, one_len, ews)
    no_error()
    place, holes = E.evict(a0, p0, ln, ln, 300, 4, 100)
    assert len(holes) and (place[holes] >= 512).any() and one_len.item() == 300
    assert np.array_equal(pk[5, :300].cpu().numpy(), keys[1][place]) and np.array_equal(pv[5, :300].cpu().numpy(), vals[1][place])


def test_queries_past_32_bits():
    """Queries and outputs of 4.4 GB: the last sessions of 4200 are the only ones with tokens."""
    rng = np.random.default_rng(20)
    b, n, h, d, page, shared = 4200, 64, 64, 128, 16, 20
    q = torch.zeros(b, n, h, d, dtype=torch.float16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((b, n, h), 7.0, device="cuda")
    q[-2:, :2] = dev(rng.standard_normal((2, 2, h, d)).astype(np.float16))
    table = torch.full((b, 3), -1, dtype=torch.int32, device="cuda")
    table[-2:] = torch.tensor([[0, 1, 2], [0, 4, 5]], dtype=torch.int32)
    pools = rng.standard_normal((2, 6 * page, d)).astype(np.float16)
    pools[:, 4 * page:4 * page + 4] = pools[:, page:page + 4]          # the page that the prefix ends in
    pk, pv = (dev(x.reshape(6, page, d)) for x in pools)
    length, n_tok = torch.zeros(b, dtype=torch.int64, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    length[-2:] = torch.tensor([30, 25])
    n_tok[-2:] = torch.tensor([2, 1], dtype=torch.int32)
    kv = ds4a.paged_kv_desc(pk, pv, table, length)
    ws = torch.empty(ds4a.ds4a_attn_prefix_workspace_bytes(b, n, h, d, 1), dtype=torch.uint8, device="cuda")
    ds4a.ds4a_attn_prefix(kv, q, n_tok, None, torch.tensor([b - 2, b], dtype=torch.int32, device="cuda"),
                          torch.tensor([shared], device="cuda"), 0.1, out, lse, ws)
    acc = torch.zeros(b, 48, device="cuda")
    ds4a.ds4a_attn_weights(kv, q, n_tok, lse, 0.1, 1.0, acc)
    no_error()
    assert (out[:-2] == 7).all() and (lse[:-2] == 7).all() and (acc[:-2] == 0).all()
    tab = table[-2:].cpu().numpy()
    for s, (ln, m) in enumerate(((30, 2), (25, 1))):
        rows = R.slot_rows(tab[s], page, range(ln + m))
        for i in range(m):
            want, tol = R.attend(q[s - 2, i].cpu().numpy(), pools[0][rows[:ln + i + 1]].astype(np.float64),
                                 pools[1][rows[:ln + i + 1]].astype(np.float64), 0.1)
            assert (np.abs(out[s - 2, i].cpu().numpy().astype(np.float64) - want) <= tol).all()
        assert (out[s - 2, m:] == 7).all()
        add, t = E.weights(q[s - 2, :m].cpu().numpy(), pools[0][rows], 0.1, lse[s - 2, :m].cpu().numpy(), ln)
        assert (np.abs(acc[s - 2, :ln + m].cpu().numpy() - add) <= t).all()


# ---- calls that read early, directly behind ---------------------------------------------------------------

def replayed(first, then, spoil, out):
    """`then` directly behind `first` in a graph gives, over 50 replays, what it gives behind a wait."""
    first()
    then()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first()
        then()
    spoil()
    torch.cuda.synchronize()
    first()
    torch.cuda.synchronize()
    then()
    torch.cuda.synchronize()
    want = out.clone()
    assert torch.isfinite(want).all()
    for _ in range(50):
        spoil()
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        no_error()
        assert torch.equal(out, want)


@pytest.mark.parametrize("n", [1, 700])
def test_decode_attention_directly_behind_a_normed_append(n):
    """ds4a_attn_decode reads queries and window rows before its dependency wait."""
    rng = np.random.default_rng(n)
    d, h, page, ln = 128, 64, 64, 40
    mp = (ln + n) // page + 1
    pk, pv = (dev(rng.standard_normal((mp, page, d)).astype(np.float16)) for _ in range(2))
    kv = ds4a.paged_kv_desc(pk, pv, torch.arange(mp, dtype=torch.int32, device="cuda")[None], torch.tensor([ln], device="cuda"))
    k, v = (dev(rng.standard_normal((1, n, d)).astype(np.float16)) for _ in range(2))
    q = dev(rng.standard_normal((1, n, h, d)).astype(np.float16))
    qo, count = torch.zeros_like(q), torch.tensor([n], dtype=torch.int32, device="cuda")
    fk, fv, w0 = pk.view(-1, d), pv.view(-1, d), ln + n - 33
    out = torch.zeros(h, d, dtype=torch.float16, device="cuda")

    def spoil():
        qo.fill_(math.nan)
        fk[ln:ln + n] = math.nan
        fv[ln:ln + n] = math.nan
    replayed(lambda: ds4a.ds4a_paged_append_norm(kv, k, v, count, None, None, EPS, None, None, 0, True, q, qo),
             lambda: ds4a.ds4a_attn_decode(qo[0, n - 1], fk[w0:ln + n], fv[w0:ln + n], None, None, None, 0, 0.088, out), spoil, out)


@pytest.mark.parametrize("slots,budget", [(200, 100), (20000, 9000)])          # moves in the clusters, and by the second kernel
def test_decode_attention_directly_behind_an_eviction(slots, budget):
    rng = np.random.default_rng(slots)
    d, h, page = 128, 64, 16
    mp = slots // page + 1
    pk, pv = (dev(rng.standard_normal((mp, page, d)).astype(np.float16)) for _ in range(2))
    kv = ds4a.paged_kv_desc(pk, pv, torch.arange(mp, dtype=torch.int32, device="cuda")[None], torch.tensor([slots], device="cuda"))
    acc = dev(rng.permutation(slots).astype(np.float32)[None])
    acc[0, :33] = -1.0                                                        # the first 33 are dropped, and filled
    pos = torch.arange(slots, dtype=torch.int32, device="cuda")[None].contiguous()
    ao, po, lo = torch.zeros_like(acc), torch.zeros_like(pos), torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.zeros(ds4a.ds4a_evict_workspace_bytes(1, slots, budget), dtype=torch.uint8, device="cuda")
    q = dev(rng.standard_normal((h, d)).astype(np.float16))
    fk, fv = pk.view(-1, d), pv.view(-1, d)
    nxt = torch.tensor([slots], device="cuda")
    out = torch.zeros(h, d, dtype=torch.float16, device="cuda")

    def spoil():
        fk[:33] = math.nan
        fv[:33] = math.nan
    replayed(lambda: ds4a.ds4a_evict(kv, acc, pos, nxt, budget, 0, 0, ao, po, lo, ws),
             lambda: ds4a.ds4a_attn_decode(q, fk[:33], fv[:33], None, None, None, 0, 0.088, out), spoil, out)
