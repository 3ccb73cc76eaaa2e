"""Workloads of sessions that share a prefix and of caches held to a budget of tokens.

Four operators over the paged token cache, each in a plain form (elementary torch operations in
32 bits) and, with `own` set, through the library's calls:

  append   tokens appended with the RMS norm of each key and query head and the rotation of their
           positions in one pass; positions may run ahead of slots (a cache that dropped tokens)
  prefix   attention of a batch whose sessions share long prefixes, group by group: the shared keys
           serve all of a group's rows at once, each session's own tokens its rows alone
  weights  every cached token's attention weight, summed over heads and queries, added to a running
           sum that decays
  evict    a cache cut to its budget: the first and newest tokens and the largest running sums stay;
           kept tokens behind the budget move into the places of dropped ones

A session has `len` cached tokens in slots 0 .. len-1; new token i sits in slot len + i.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------------------

def _case(name, op, B, N, ctx, H=64, D=128, page=64, rot=64, rot_off=64, interleaved=True, q=True, tree="chain", groups=0,
          shared=0, alone=0, decay=1.0, budget=0, sink=0, recent=0):
    return dict(name=name, op=op, B=B, N=N, ctx=ctx, H=H, D=D, page=page, rot=rot, rot_off=rot_off, interleaved=interleaved,
                q=q, tree=tree, groups=groups, shared=shared, alone=alone, decay=decay, budget=budget, sink=sink,
                recent=recent)


def listed():
    return [
        # one session's next token: the launch-bound end of the range
        _case("anorm_1x1", "append", 1, 1, 32768),
        # a ragged batch of small drafted trees, 8 heads of 64, whole-head rotation in halves, pages that are no power of two
        _case("anorm_16x13_d64", "append", 16, 13, 5000, H=8, D=64, page=48, rot=64, rot_off=0, interleaved=False, tree="tree"),
        # a prefill chunk after a 30720-token prefix, keys and 64 query heads
        _case("anorm_2048", "append", 1, 2048, 30720),
        # four answers sampled from one 2048-token prompt, next token each: latency
        _case("prefix_4x1", "prefix", 4, 1, 60, groups=1, shared=2048),
        # three system prompts, drafted trees, 8 heads of 64, some sessions without a prefix, odd lengths
        _case("prefix_29x5_d64", "prefix", 29, 5, 700, H=8, D=64, page=48, tree="tree", groups=3, shared=9001, alone=3),
        # a loaded server: 64 sessions over one 32768-token document, up to 512 tokens of their own
        _case("prefix_64x1", "prefix", 64, 1, 512, groups=1, shared=32768),
        # one session's next token over a budget of 4096: latency
        _case("weights_1x1", "weights", 1, 1, 4096),
        # prompts scored in chunks of up to 33 tokens, 24 heads of 64, older weights fade
        _case("weights_5x33_d64", "weights", 5, 33, 5000, H=24, D=64, page=48, decay=0.96875),
        # a loaded server's next tokens over 32768 cached tokens each
        _case("weights_64x1", "weights", 64, 1, 32768),
        # a session that outgrew its budget by 64 tokens
        _case("evict_1x4096", "evict", 1, 0, 4160, budget=4096, sink=4, recent=256),
        # prompts cut to a third of their tokens, ragged
        _case("evict_24x4000", "evict", 24, 0, 12001, page=48, budget=4000, sink=1, recent=37),
        # a loaded server: 64 sessions, each 256 tokens over its budget
        _case("evict_64x8192", "evict", 64, 0, 8448, budget=8192, sink=4, recent=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "prefix", "prefix", "weights", "weights", "evict", "evict"])
    D = rng.choice([64, 128, 128])
    H = 8 * rng.randint(1, 8)
    page = 16 * rng.randint(1, 16)
    base = dict(H=H, D=D, page=page)
    if op == "append":
        rot = 16 * rng.randint(0, D // 16)
        base.update(rot=rot, rot_off=8 * rng.randint(0, (D - rot) // 8), interleaved=rng.random() < 0.5)
        if rng.random() < 0.5:          # prompts and chunks
            B = _log(rng, 1, 8)
            return _case("", op, B, _log(rng, 1, 2048 // B), _log(rng, 1, 32768), q=rng.random() < 0.8, **base)
        return _case("", op, _log(rng, 1, 64), _log(rng, 1, 24), _log(rng, 1, 8192), q=rng.random() < 0.8,
                     tree=rng.choice(["chain", "tree"]), **base)
    if op == "prefix":
        N = _log(rng, 1, 64)
        B = _log(rng, 1, max(1, 64 // N))
        groups = min(B, _log(rng, 1, 6))
        return _case("", op, B, N, _log(rng, 1, 1024), tree=rng.choice(["chain", "tree"]), groups=groups,
                     shared=_log(rng, 16, 32768), alone=rng.randint(0, B - groups) // 2, **base)
    if op == "weights":
        N = _log(rng, 1, 64)
        B = _log(rng, 1, max(1, 64 // N))
        return _case("", op, B, N, _log(rng, 1, 32768), decay=rng.choice([1.0, 1.0, 0.5, 0.99]), **base)
    ctx = _log(rng, 64, 32768)
    budget = max(1, min(ctx, int(ctx * rng.uniform(0.2, 1.1))))
    sink = min(budget, _log(rng, 1, 64) - 1)
    return _case("", op, _log(rng, 1, max(1, min(64, 540000 // ctx))), 0, ctx, budget=budget, sink=sink,
                 recent=int((budget - sink) * rng.uniform(0, 0.5)), **base)


# ---- inputs ----------------------------------------------------------------------------------

def _groups(c):
    """(start [G + 1], shared [G]): sessions start[g] .. start[g+1]-1 share their first shared[g] tokens."""
    G = c["groups"]
    w = 1 + (np.arange(G) * 7) % 3
    start = np.concatenate([[0], np.cumsum(w)]) * (c["B"] - c["alone"]) // max(1, w.sum())
    shared = c["shared"] - (np.arange(G) * 977) % (c["shared"] // 8 + 1)
    return start.astype(np.int64), shared.astype(np.int64)


def _lengths(c):
    """Cached tokens, new tokens and shared tokens of each session: ragged, the first session full."""
    s = np.arange(c["B"])
    ln = c["ctx"] - (s * 977) % (c["ctx"] // 8 + 1)
    n = c["N"] - (s * 5) % (c["N"] // 2 + 1)
    sh = np.zeros(c["B"], np.int64)
    if c["op"] == "prefix":             # ctx: a session's own tokens
        start, shared = _groups(c)
        for g in range(c["groups"]):
            sh[start[g]:start[g + 1]] = shared[g]
        ln = ln + sh
    return ln.astype(np.int64), n.astype(np.int32), sh


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    B, N, H, D, page = c["B"], c["N"], c["H"], c["D"], c["page"]
    ln, n, sh = _lengths(c)
    top = int((ln + N).max())
    mp = (top + page - 1) // page

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).half()
    x = dict(case=c, ln=ln, nn=n, slots=(mp * page + 3) // 4 * 4)
    x["len"] = torch.from_numpy(ln).to(DEV)
    x["n"] = torch.from_numpy(n).to(DEV)
    # every session's pages scattered over a shared pool with some pages of nobody; the pages that lie
    # inside a shared prefix are one session's, and a page that a prefix ends in is each session's copy
    n_pages = B * mp + 3
    table = r.permutation(n_pages)[:B * mp].reshape(B, mp).astype(np.int32)
    spare = np.setdiff1d(np.arange(n_pages), table)[0]
    x["pool_k"] = normal(n_pages, page, D)
    x["pool_v"] = normal(n_pages, page, D)
    if c["op"] == "prefix":
        start, shared = _groups(c)
        for a, b, m in zip(start[:-1], start[1:], shared):
            for s in range(a + 1, b):
                table[s, :m // page] = table[a, :m // page]
                if m % page:
                    for pool in (x["pool_k"], x["pool_v"]):
                        pool[table[s, m // page], :m % page] = pool[table[a, m // page], :m % page]
        x["start"] = torch.from_numpy(start.astype(np.int32)).to(DEV)
        x["shared"] = torch.from_numpy(shared).to(DEV)
    x["spare"] = int(spare) * page
    x["table"] = torch.from_numpy(table).to(DEV)
    par = np.full((B, max(1, N)), -1, np.int32)
    if c["tree"] == "tree":
        for i in range(1, N):           # a tree that grows mostly downwards, with some branches
            par[:, i] = i - 1 - np.minimum(r.geometric(0.6, B) - 1, i)
    else:
        par[:] = np.arange(max(1, N)) - 1
    x["parent"] = torch.from_numpy(par).to(DEV)
    if c["op"] == "append":
        x["k"], x["v"] = 3.0 * normal(B, N, D), normal(B, N, D)
        x["k_w"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        x["q_w"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=DEV)
        x["inv_freq"] = None
        if c["rot"]:
            inv = 10000.0 ** (-np.arange(c["rot"] // 2) / (c["rot"] // 2))
            x["inv_freq"] = torch.from_numpy(inv.astype(np.float32)).to(DEV)
        x["pos0"] = x["len"] + torch.from_numpy((np.arange(B) * 613 % 5000).astype(np.int64)).to(DEV)
        x["slot_pos"] = torch.full((B, x["slots"]), -1, dtype=torch.int32, device=DEV)
        if c["q"]:
            x["q"] = 3.0 * normal(B, N, H, D)
            x["q_out"] = torch.zeros_like(x["q"])
    if c["op"] == "prefix":
        x["q"] = normal(B, N, H, D)
        x["out"] = torch.zeros_like(x["q"])
        x["lse"] = torch.zeros(B, N, H, device=DEV)
    if c["op"] == "weights":
        x["q"] = normal(B, N, H, D)
        x["acc"] = torch.rand(B, x["slots"], generator=g, device=DEV)
        x["lse"] = torch.zeros(B, N, H, device=DEV)
        for s in range(B):              # the sums that the attention call leaves: log of the sum of exp
            m = int(n[s])
            kk = x["pool_k"].view(-1, D)[_rows(x, s, np.arange(ln[s] + m))].float()
            sc = (x["q"][s, :m].float().view(m * H, D) @ kk.T / math.sqrt(D)).view(m, H, -1)
            sc.masked_fill_(torch.arange(sc.shape[2], device=DEV) > int(ln[s]) + torch.arange(m, device=DEV)[:, None, None],
                            -math.inf)
            x["lse"][s, :m] = torch.logsumexp(sc.double() if sc.numel() < 1 << 26 else sc, 2).float()
    if c["op"] == "evict":
        # running sums with a long tail, some tokens never attended; positions with gaps, some out of order
        a = torch.exp(2.0 * torch.randn(B, x["slots"], generator=g, device=DEV) - 3.0)
        x["acc"] = torch.where(torch.rand(B, x["slots"], generator=g, device=DEV) < 0.05, 0.0, a)
        pos = np.zeros((B, x["slots"]), np.int32)
        nxt = np.zeros(B, np.int64)
        for s in range(B):
            m = int(ln[s])
            p = np.cumsum(r.integers(1, 3, m)) - 1
            swap = r.permutation(m)[:m // 10]
            p[np.sort(swap)] = p[swap]
            pos[s, :m] = p
            nxt[s] = p.max() + 1
        x["pos"] = torch.from_numpy(pos).to(DEV)
        x["next"] = torch.from_numpy(nxt).to(DEV)
        x["acc_out"], x["pos_out"], x["len_out"] = torch.zeros_like(x["acc"]), torch.zeros_like(x["pos"]), x["len"].clone()
    return x


def _rows(x, s, t):
    """Pool rows of slots t of session s (host page table lookups would cost more: t is a numpy range)."""
    page = x["case"]["page"]
    t = torch.from_numpy(np.asarray(t, np.int64)).to(DEV)
    return x["table"][s].long()[t // page] * page + t % page


def prepare(case, seed):
    x = _inputs(case, seed)
    if own:
        from compressed_sparse_mqa_gb300 import ds4a
        c = case
        x["kv"] = ds4a.paged_kv_desc(x["pool_k"], x["pool_v"], x["table"], x["len"])
        nb = 0
        if c["op"] == "prefix":
            nb = ds4a.ds4a_attn_prefix_workspace_bytes(c["B"], c["N"], c["H"], c["D"], c["groups"])
        if c["op"] == "evict":
            nb = ds4a.ds4a_evict_workspace_bytes(c["B"], x["slots"], c["budget"])
        x["ws"] = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    return x


# ---- one pass --------------------------------------------------------------------------------

def run(x):
    return (_run_own if own else _run_plain)(x)


OUTPUTS = {"append": ("pool_k", "pool_v", "slot_pos", "q_out"), "prefix": ("out", "lse"), "weights": ("acc",),
           "evict": ("pool_k", "pool_v", "acc_out", "pos_out", "len_out")}


def _outs(x):
    return {k: x[k] for k in OUTPUTS[x["case"]["op"]] if k in x}


def _run_own(x):
    from compressed_sparse_mqa_gb300 import ds4a
    c = x["case"]
    parent = x["parent"] if c["tree"] == "tree" else None
    if c["op"] == "append":
        ds4a.ds4a_paged_append_norm(x["kv"], x["k"], x["v"], x["n"], x["k_w"], x["q_w"], EPS, parent, x["inv_freq"],
                                    c["rot_off"], c["interleaved"], x.get("q"), x.get("q_out"), x["pos0"], x["slot_pos"])
    elif c["op"] == "prefix":
        ds4a.ds4a_attn_prefix(x["kv"], x["q"], x["n"], parent, x["start"], x["shared"], 1.0 / math.sqrt(c["D"]), x["out"],
                              x["lse"], x["ws"])
    elif c["op"] == "weights":
        ds4a.ds4a_attn_weights(x["kv"], x["q"], x["n"], x["lse"], 1.0 / math.sqrt(c["D"]), c["decay"], x["acc"])
    else:
        ds4a.ds4a_evict(x["kv"], x["acc"], x["pos"], x["next"], c["budget"], c["sink"], c["recent"], x["acc_out"],
                        x["pos_out"], x["len_out"], x["ws"])
    return _outs(x)


def _run_plain(x):
    {"append": _append_plain, "prefix": _prefix_plain, "weights": _weights_plain, "evict": _evict_plain}[x["case"]["op"]](x)
    return _outs(x)


def _all_rows(x, t):
    """Pool row of slot t [B, n] of every session."""
    page = x["case"]["page"]
    pg = torch.gather(x["table"].long(), 1, torch.div(t, page, rounding_mode="floor"))
    return pg * page + t % page


def _ancestors(x):
    """(anc [B, N, N] truth values including the node itself, depth [B, N])."""
    N = x["case"]["N"]
    node = torch.arange(N, device=DEV)
    anc = (x["parent"][:, :, None] == node) | (node[:, None] == node)
    span = 1
    while span < N:
        f = anc.float()
        anc = (f @ f) > 0
        span *= 2
    return anc, anc.sum(2) - 1


def _append_plain(x):
    c = x["case"]
    N, D, rot, off = c["N"], c["D"], c["rot"], c["rot_off"]
    node = torch.arange(N, device=DEV)
    slot = x["len"][:, None] + node
    pos = x["pos0"][:, None] + (_ancestors(x)[1] if c["tree"] == "tree" else node)
    ok = node < x["n"][:, None]

    def encode(t, w):                   # t [B, N, heads, D]
        f = t.float()
        f = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
        if rot:
            ang = pos.double()[..., None] * x["inv_freq"].double()
            cs, sn = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
            part = f[..., off:off + rot]
            if c["interleaved"]:
                a, b = part[..., 0::2], part[..., 1::2]
                new = torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)
            else:
                a, b = part[..., :rot // 2], part[..., rot // 2:]
                new = torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
            f = torch.cat([f[..., :off], new, f[..., off + rot:]], -1)
        return f.half()
    row = _all_rows(x, slot)
    for pool, new in ((x["pool_k"], encode(x["k"][:, :, None], x["k_w"])[:, :, 0]), (x["pool_v"], x["v"])):
        flat = pool.view(-1, D)
        flat[row] = torch.where(ok[..., None], new, flat[row])
    x["slot_pos"].scatter_(1, slot, torch.where(ok, pos.int(), x["slot_pos"].gather(1, slot)))
    if "q_out" in x:
        x["q_out"].copy_(torch.where(ok[..., None, None], encode(x["q"], x["q_w"]), x["q_out"]))


def _prefix_plain(x):
    c = x["case"]
    B, N, H, D, page = c["B"], c["N"], c["H"], c["D"], c["page"]
    scale = 1.0 / math.sqrt(D)
    qf = x["q"].float().view(B, N * H, D)
    fk, fv = x["pool_k"].view(-1, D), x["pool_v"].view(-1, D)
    start, shared = _groups(c)
    m1 = torch.full((B, N * H, 1), -math.inf, device=DEV)
    l1 = torch.zeros(B, N * H, 1, device=DEV)
    o1 = torch.zeros(B, N * H, D, device=DEV)
    for a, b, m in zip(start[:-1], start[1:], shared):
        if a == b:
            continue
        t = torch.arange(int(m), device=DEV)
        row = x["table"][a].long()[t // page] * page + t % page
        s = (qf[a:b].reshape(-1, D) @ fk[row].float().T) * scale
        top = s.max(1, keepdim=True).values
        e = torch.exp(s - top)
        m1[a:b], l1[a:b] = top.view(b - a, -1, 1), e.sum(1).view(b - a, -1, 1)
        o1[a:b] = (e @ fv[row].float()).view(b - a, -1, D)
    # the sessions' own tokens: from their prefix's end to their last new token
    sh = x["len"].new_zeros(B)
    for g in range(c["groups"]):
        sh[start[g]:start[g + 1]] = int(shared[g])
    anc, _ = _ancestors(x)
    t = sh[:, None] + torch.arange(c["ctx"] + N, device=DEV)
    i = t - x["len"][:, None]           # a new token's number, or negative
    row = _all_rows(x, torch.where(i < N, t, 0))
    seen = torch.gather(anc, 2, i.clamp(0, N - 1)[:, None].expand(B, N, -1))
    mask = (i < 0)[:, None] | (seen & (i < x["n"][:, None])[:, None])
    k, v = fk[row].float(), fv[row].float()
    s = torch.where(mask[:, :, None], (qf @ k.transpose(1, 2)).view(B, N, H, -1) * scale, -math.inf).view(B, N * H, -1)
    top = torch.maximum(s.max(2, keepdim=True).values, m1)
    e = torch.exp(s - top)
    f = torch.exp(m1 - top)
    total = e.sum(2, keepdim=True) + f * l1
    o = (e @ v + f * o1) / total
    ok = torch.arange(N, device=DEV) < x["n"][:, None]
    x["out"].copy_(torch.where(ok[..., None, None], o.view(B, N, H, D).half(), x["out"]))
    x["lse"].copy_(torch.where(ok[..., None], (top + torch.log(total)).view(B, N, H), x["lse"]))


def _weights_plain(x):
    c = x["case"]
    B, N, H, D = c["B"], c["N"], c["H"], c["D"]
    t = torch.arange(int((x["ln"] + x["nn"]).max()), device=DEV)
    i = t - x["len"][:, None]
    have = i < x["n"][:, None]
    k = x["pool_k"].view(-1, D)[_all_rows(x, torch.where(have, t, 0))].float()
    s = (x["q"].float().view(B, N * H, D) @ k.transpose(1, 2)).view(B, N, H, -1) * (1.0 / math.sqrt(D))
    node = torch.arange(N, device=DEV)
    see = (i[:, None] <= node[:, None]) & (node < x["n"][:, None])[:, :, None]
    p = torch.where(see[:, :, None], torch.exp(s - x["lse"][..., None]), 0.0)
    old = torch.where(i < 0, c["decay"] * x["acc"][:, :t.numel()], 0.0)
    x["acc"][:, :t.numel()] = torch.where(have, old + p.sum((1, 2)), x["acc"][:, :t.numel()])


def _evict_plain(x):
    c = x["case"]
    D, S, budget = c["D"], x["slots"], c["budget"]
    slot = torch.arange(S, device=DEV)
    have = slot < x["len"][:, None]
    kept_always = (x["pos"] < c["sink"]) | (x["pos"] >= x["next"][:, None] - c["recent"])
    key = torch.where(kept_always, math.inf, x["acc"])
    key = torch.where(have, key, -math.inf)
    order = torch.sort(key, dim=1, descending=True, stable=True).indices
    kept = torch.zeros_like(have).scatter_(1, order[:, :budget], True) & have
    most = max(1, min(budget, S - budget))
    hole = torch.sort(torch.where(have & ~kept & (slot < budget), slot, S), 1).values[:, :most]
    mover = torch.sort(torch.where(kept & (slot >= budget), slot, S), 1).values[:, :most]
    real = mover < S
    to, fr = torch.where(real, hole, 0), torch.where(real, mover, 0)
    row_to = torch.where(real, _all_rows(x, to), x["spare"])
    row_fr = torch.where(real, _all_rows(x, fr), x["spare"])
    for pool in (x["pool_k"], x["pool_v"]):
        flat = pool.view(-1, D)
        flat[row_to] = flat[row_fr]
    x["len_out"].copy_(x["len"].clamp(max=budget))
    stays = slot < x["len_out"][:, None]
    for a, b in ((x["acc"], x["acc_out"]), (x["pos"], x["pos_out"])):
        new = torch.cat([a, a[:, :1]], 1)
        new.scatter_(1, torch.where(real, hole, S), a.gather(1, fr))
        b.copy_(torch.where(stays, new[:, :S], b))


# ---- work ------------------------------------------------------------------------------------

def work(case):
    c = case
    H, D = c["H"], c["D"]
    ln, n, sh = _lengths(c)
    tok = int(n.sum())
    if c["op"] == "append":
        return {"bytes": tok * (8 * D + 4 + (4 * H * D if c["q"] else 0)),
                "flops": tok * (1 + (H if c["q"] else 0)) * (4 * D + 3 * c["rot"])}
    if c["op"] == "evict":
        cut = ln[ln > c["budget"]]
        moved = int(((cut - c["budget"]) * c["budget"] // np.maximum(1, cut)).sum())
        left = int(np.minimum(ln, c["budget"]).sum())
        return {"bytes": int(ln.sum()) * 8 + left * 8 + moved * 8 * D, "flops": int(ln.sum())}
    if c["op"] == "weights":
        keys = int((ln + n).sum())
        return {"bytes": keys * (2 * D + 8) + tok * H * (2 * D + 4),
                "flops": int((2 * D + 3) * H * (n * (ln + 1)).sum())}
    start, shared = _groups(c)
    keys = int((ln - sh + n).sum()) + int(shared[start[1:] > start[:-1]].sum())
    return {"bytes": keys * 4 * D + tok * H * (4 * D + 4), "flops": int(4 * D * H * (n * (ln + 1)).sum())}


# ---- the definitions in 64 bits --------------------------------------------------------------

def _paths(par, n):
    ps = []
    for i in range(n):
        ps.append((ps[par[i]] if par[i] >= 0 else []) + [i])
    return ps


def exact(case, seed):
    x = _inputs(case, seed)
    c = case
    B, H, D, page = c["B"], c["H"], c["D"], c["page"]
    ln, n = x["ln"], x["nn"]
    par, tab = x["parent"].cpu().numpy(), x["table"].cpu().numpy()
    if c["op"] == "evict":
        return _exact_evict(x, tab)

    def place(s, t):
        t = np.asarray(t, np.int64)
        return torch.from_numpy(tab[s][t // page].astype(np.int64) * page + t % page).to(DEV)
    pk, pv = x["pool_k"].view(-1, D).double(), x["pool_v"].view(-1, D).double()
    if c["op"] == "append":
        half = c["rot"] // 2
        j = torch.arange(half, device=DEV)
        i1 = c["rot_off"] + (2 * j if c["interleaved"] else j)
        i2 = i1 + (1 if c["interleaved"] else half)

        def enc(t, w, pos):             # t [m, ..., D] at positions [m]
            t = t.double()
            t = t / torch.sqrt(torch.linalg.vector_norm(t, dim=-1, keepdim=True) ** 2 / D + EPS) * w.double()
            if not half:
                return t
            th = torch.from_numpy(np.asarray(pos, np.float64)).to(DEV)[:, None] * x["inv_freq"].double()
            z = torch.polar(torch.ones_like(th), th).view(th.shape[0], *([1] * (t.dim() - 2)), half)
            y = torch.complex(t[..., i1], t[..., i2]) * z
            r = t.clone()
            r[..., i1], r[..., i2] = y.real, y.imag
            return r
        sp = x["slot_pos"].cpu()
        pos0 = x["pos0"].cpu().numpy()
        qo = x["q_out"].double() if "q_out" in x else None
        for s in range(B):
            m = int(n[s])
            pos = pos0[s] + np.array([len(p) - 1 for p in _paths(par[s], m)], np.int64)
            where = place(s, ln[s] + np.arange(m))
            pk[where] = enc(x["k"][s, :m], x["k_w"], pos)
            pv[where] = x["v"][s, :m].double()
            sp[s, ln[s]:ln[s] + m] = torch.from_numpy(pos.astype(np.int32))
            if qo is not None:
                qo[s, :m] = enc(x["q"][s, :m], x["q_w"], pos)
        o = {"pool_k": pk.view_as(x["pool_k"]), "pool_v": pv.view_as(x["pool_v"]), "slot_pos": sp}
        if qo is not None:
            o["q_out"] = qo
        return o
    if int((ln + n).sum()) * c["N"] * H * D > 1 << 38:
        return None
    out = x["out"].double() if c["op"] == "prefix" else None
    lse, acc = x["lse"].double(), x["acc"].double() if c["op"] == "weights" else None
    for s in range(B):
        m, a0 = int(n[s]), int(ln[s])
        rows = place(s, np.arange(a0 + m))
        see = np.zeros((m, m), bool)
        for i, p in enumerate(_paths(par[s], m)):
            see[i, p] = True
        sc = (x["q"][s, :m].double().view(m * H, D) @ pk[rows].T / math.sqrt(D)).view(m, H, a0 + m)
        sc[:, :, a0:] = sc[:, :, a0:].masked_fill(~torch.from_numpy(see).to(DEV)[:, None], -math.inf)
        if c["op"] == "weights":
            got = torch.exp(sc - lse[s, :m, :, None]).sum((0, 1))
            got[:a0] += c["decay"] * acc[s, :a0]
            acc[s, :a0 + m] = got
        else:
            out[s, :m] = torch.softmax(sc, 2) @ pv[rows]
            lse[s, :m] = torch.logsumexp(sc, 2)
    return {"acc": acc} if c["op"] == "weights" else {"out": out, "lse": lse}


def _exact_evict(x, tab):
    c, D = x["case"], x["case"]["D"]
    page, budget = c["page"], c["budget"]
    pk, pv = x["pool_k"].view(-1, D).clone(), x["pool_v"].view(-1, D).clone()
    acc, pos, nxt = x["acc"].cpu().numpy(), x["pos"].cpu().numpy(), x["next"].cpu().numpy()
    ao, po, lo = x["acc_out"].cpu().numpy(), x["pos_out"].cpu().numpy(), x["len_out"].cpu().numpy()
    for s in range(c["B"]):
        m = int(x["ln"][s])
        kept = np.ones(m, bool)
        if m > budget:
            safe = (pos[s, :m] < c["sink"]) | (pos[s, :m] >= nxt[s] - c["recent"])
            rank = np.lexsort((np.arange(m), -acc[s, :m], ~safe))
            kept[rank[budget:]] = False
        left = min(m, budget)
        lo[s] = left
        src = np.arange(left)
        hole, mover = np.nonzero(~kept[:left])[0], left + np.nonzero(kept[left:])[0]
        src[hole] = mover
        ao[s, :left], po[s, :left] = acc[s, src], pos[s, src]

        def place(t):
            return torch.from_numpy(tab[s][t // page].astype(np.int64) * page + t % page).to(DEV)
        if len(hole):
            a, b = place(hole), place(mover)
            pk[a], pv[a] = pk[b], pv[b]
    return {"pool_k": pk.view_as(x["pool_k"]), "pool_v": pv.view_as(x["pool_v"]), "acc_out": torch.from_numpy(ao),
            "pos_out": torch.from_numpy(po), "len_out": torch.from_numpy(lo)}
