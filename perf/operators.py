"""Workloads of the paged token cache and of drafted-token verification.

Four operators, each in a plain form (elementary torch operations in 32 bits) and, with
`own` set, through the library's calls:

  append    tokens appended to a paged K/V cache, keys and queries rotated to their positions
  compress  the compressed rows that drafted tokens complete along their own paths
  attn      attention of a tree of drafted tokens over the window, the compressed rows and the tree
  commit    drafted tokens appended (keys as the model encoded them), then the accepted path moved to its place

A session has `len` committed tokens.  Drafted node i has a parent (an earlier node, or -1),
sits in slot len + i of its session's pages and at position len + depth(i).
"""
import math

import numpy as np
import torch

own = False

SIGMA_W = math.sqrt(1.0 / 128.0)      # spread of a layer's compressor score weights
DEV = "cuda"


# ---- cases -----------------------------------------------------------------------------------

def _case(name, op, B, N, ctx, H=64, D=128, page=64, window=128, ratio=0, sel=0, q=True, rot=64, rot_off=64,
          interleaved=True, tree="tree"):
    return dict(name=name, op=op, B=B, N=N, ctx=ctx, H=H, D=D, page=page, window=window, ratio=ratio, sel=sel, q=q,
                rot=rot, rot_off=rot_off, interleaved=interleaved, tree=tree)


def listed():
    return [
        # one session's next token: the launch-bound end of the range
        _case("append_1x1", "append", 1, 1, 32768, tree="none"),
        # a ragged batch of small trees, 8 heads of 64, whole-head rotation in halves, pages that are no power of two
        _case("append_16x13_d64", "append", 16, 13, 5000, H=8, D=64, page=48, rot=64, rot_off=0, interleaved=False),
        # a prefill chunk after a 30720-token prefix, keys and 64 query heads
        _case("append_2048", "append", 1, 2048, 30720, tree="none"),
        # a window-only layer checking four drafted tokens: latency
        _case("attn_window_1x4", "attn", 1, 4, 32768),
        # a ratio-128 layer at context 131072 (1024 compressed rows), one session, 16 drafted tokens
        _case("attn_r128_1x16", "attn", 1, 16, 131072, ratio=128),
        # a ratio-4 layer: every node attends its own 512 kept rows, 16 sessions of up to 16 nodes
        _case("attn_sel_16x16", "attn", 16, 16, 32768, ratio=4, sel=512),
        # a loaded server: 64 sessions around context 65536 with up to 32 nodes each
        _case("attn_r128_64x32", "attn", 64, 32, 65536, ratio=128),
        # a layer without a window limit over long caches, full 64-node trees
        _case("attn_full_4x64", "attn", 4, 64, 32768, window=1 << 30),
        # rows completed inside the drafts of a batch: every fourth position
        _case("compress_r4_16x16", "compress", 16, 16, 32768, ratio=4),
        # the same on a ratio-128 layer of a loaded server (few rows complete, long blocks)
        _case("compress_r128_64x64", "compress", 64, 64, 65536, ratio=128),
        # a few sessions with odd sizes
        _case("commit_3x13_d64", "commit", 3, 13, 777, H=8, D=64, page=16, ratio=7),
        # a loaded server's accepted paths on a ratio-4 layer with indexer keys
        _case("commit_64x32", "commit", 64, 32, 32768, ratio=4),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "attn", "attn", "attn", "compress", "commit"])
    D = rng.choice([64, 128, 128])
    H = 8 * rng.randint(1, 8)
    page = 16 * rng.randint(1, 16)
    rot = 16 * rng.randint(1, D // 16)
    rot_off = 8 * rng.randint(0, (D - rot) // 8)
    inter = rng.random() < 0.5
    B = _log(rng, 1, 64)
    N = _log(rng, 1, 64)
    ctx = _log(rng, 1, 65536)
    base = dict(H=H, D=D, page=page, rot=rot, rot_off=rot_off, interleaved=inter)
    if op == "append":
        if rng.random() < 0.5:          # prompts and chunks: no tree, longer
            B = _log(rng, 1, 8)
            return dict(_case("", op, B, _log(rng, 1, 2048 // B), ctx, q=rng.random() < 0.7, tree="none", **base))
        return dict(_case("", op, B, N, min(ctx, 16384), q=rng.random() < 0.7, **base))
    if op == "compress" or op == "commit":
        ratio = rng.choice([1, 4, 4, 128, rng.randint(2, 200)])
        ctx = min(ctx, 16384)
        return dict(_case("", op, B, N, ctx, ratio=ratio, **base))
    kind = rng.choice(["window", "rows", "sel", "full"])
    if kind == "window":
        return dict(_case("", op, B, N, min(ctx, 16384), window=_log(rng, 1, 4096), **base))
    if kind == "rows":
        ratio = rng.choice([64, 128, rng.randint(16, 300)])
        return dict(_case("", op, B, N, ctx, window=_log(rng, 16, 512), ratio=ratio, **base))
    if kind == "sel":
        B, N = _log(rng, 1, 16), _log(rng, 1, 16)
        return dict(_case("", op, B, N, min(ctx, 32768), window=_log(rng, 16, 256), ratio=rng.choice([4, 4, 16]),
                          sel=_log(rng, 1, 512), **base))
    B = _log(rng, 1, 4)
    return dict(_case("", op, B, N, min(ctx, 32768), window=1 << 30, **base))


# ---- inputs ----------------------------------------------------------------------------------

def _lengths(c):
    """Committed tokens and drafted tokens of each session: ragged, the first session full."""
    s = np.arange(c["B"])
    ln = c["ctx"] - (s * 977) % (c["ctx"] // 8 + 1)
    n = c["N"] - (s * 5) % (c["N"] // 2 + 1)
    return ln.astype(np.int64), n.astype(np.int32)


def _rows_cap(c):
    """Compressed rows per session: the committed ones, what a draft can add, the draft's own N."""
    return (c["ctx"] + c["N"]) // c["ratio"] + c["N"] if c["ratio"] else 0


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = np.random.default_rng(seed)
    B, N, H, D, page = c["B"], c["N"], c["H"], c["D"], c["page"]
    ln, n = _lengths(c)
    mp = (c["ctx"] + N + page - 1) // page

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32).half()
    x = dict(case=c)
    x["len"] = torch.from_numpy(ln).to(DEV)
    x["n"] = torch.from_numpy(n).to(DEV)
    # every session's pages scattered over a shared pool with some pages of nobody
    n_pages = B * mp + 3
    x["table"] = torch.from_numpy(r.permutation(n_pages)[:B * mp].reshape(B, mp).astype(np.int32)).to(DEV)
    x["pool_k"] = normal(n_pages, page, D)
    x["pool_v"] = normal(n_pages, page, D)
    par = np.full((B, N), -1, np.int32)
    if c["tree"] == "tree":
        for i in range(1, N):           # a tree that grows mostly downwards, with some branches
            back = 1 + np.minimum(r.geometric(0.6, B) - 1, i)
            par[:, i] = i - back
    else:
        par[:] = np.arange(N) - 1
    x["parent"] = torch.from_numpy(par).to(DEV)
    if c["op"] in ("append", "commit"):
        x["k"], x["v"] = normal(B, N, D), normal(B, N, D)
    if c["op"] == "append":
        inv = 10000.0 ** (-np.arange(c["rot"] // 2) / (c["rot"] // 2))
        x["inv_freq"] = torch.from_numpy(inv.astype(np.float32)).to(DEV)
    if c["op"] == "append" and c["q"]:
        x["q"] = normal(B, N, H, D)
        x["q_out"] = torch.zeros_like(x["q"])
    if c["ratio"]:
        cap = _rows_cap(c)
        x["comp_k"], x["comp_v"] = normal(B, cap, D), normal(B, cap, D)
        x["w"] = torch.randn(D, generator=g, device=DEV) * SIGMA_W
    if c["op"] in ("compress", "commit"):
        # the open block's running state: (max score, sum, weighted K, weighted V) of its committed tokens
        cnt = x["len"] % c["ratio"]
        t = (x["len"] - cnt)[:, None] + torch.arange(c["ratio"], device=DEV)
        ok = t < x["len"][:, None]
        row = _rows(x, torch.where(ok, t, 0))
        kk, vv = x["pool_k"].view(-1, D)[row].double(), x["pool_v"].view(-1, D)[row].double()
        s = torch.where(ok, kk @ x["w"].double(), -math.inf)
        m = s.max(1, keepdim=True).values
        m = torch.where(torch.isfinite(m), m, 0.0)
        e = torch.exp(s - m)
        x["state"] = torch.cat([m, e.sum(1, keepdim=True), (e[:, None] @ kk)[:, 0], (e[:, None] @ vv)[:, 0]],
                               1).float()
    if c["op"] == "commit":
        x["state_out"] = x["state"].clone()
        x["len_out"] = x["len"].clone()
        x["leaf"] = torch.from_numpy((r.integers(0, 1 << 30, B) % (n + 1) - 1).astype(np.int32)).to(DEV)
        if c["ratio"] == 4:
            x["k_idx"] = normal(B, _rows_cap(c), D)
    if c["op"] == "attn":
        x["q"] = normal(B, N, H, D)
        x["out"] = torch.zeros_like(x["q"])
        if c["sel"]:
            # each node's kept rows: random visible ones in ascending order, -1 behind them
            depth = _depths_np(par)
            vis = torch.from_numpy((ln[:, None] + depth + 1) // c["ratio"]).to(DEV)
            m = max(int((c["ctx"] + N) // c["ratio"]), c["sel"])
            u = torch.rand(B, N, m, generator=g, device=DEV)
            u[torch.arange(m, device=DEV) >= vis[..., None]] = 2.0
            pick = u.topk(c["sel"], dim=2, largest=False)
            idx = torch.where(pick.values < 2.0, pick.indices, 1 << 30).sort(2).values
            x["sel"] = torch.where(idx < (1 << 30), idx, -1).int().contiguous()
    return x


def _depths_np(par):
    d = np.zeros(par.shape, np.int64)
    for i in range(par.shape[1]):
        up = np.take_along_axis(d, np.maximum(par[:, i:i + 1], 0).astype(np.int64), 1)[:, 0]
        d[:, i] = np.where(par[:, i] >= 0, up + 1, 0)
    return d


def _rows(x, t):
    """Pool row of slot t [B, n] of every session."""
    page = x["case"]["page"]
    pg = torch.gather(x["table"].long(), 1, torch.div(t, page, rounding_mode="floor"))
    return pg * page + t % page


def prepare(case, seed):
    x = _inputs(case, seed)
    if own:
        from compressed_sparse_mqa_gb300 import ds4a
        x["kv"] = ds4a.paged_kv_desc(x["pool_k"], x["pool_v"], x["table"], x["len"])
        if case["op"] == "attn":
            nb = ds4a.ds4a_attn_tree_workspace_bytes(case["B"], case["N"], case["H"], case["D"])
            x["ws"] = torch.zeros(nb, dtype=torch.uint8, device=DEV)
    return x


# ---- one pass --------------------------------------------------------------------------------

def run(x):
    return (_run_own if own else _run_plain)(x)


def _run_own(x):
    from compressed_sparse_mqa_gb300 import ds4a
    c = x["case"]
    parent = x["parent"] if c["tree"] == "tree" else None
    if c["op"] == "append":
        ds4a.ds4a_paged_append(x["kv"], x["k"], x["v"], x["n"], parent, x["inv_freq"], c["rot_off"], c["interleaved"],
                               x.get("q"), x.get("q_out"))
        return _outs_append(x)
    if c["op"] == "compress":
        ds4a.ds4a_compress_tree(x["kv"], x["n"], x["parent"], x["w"], c["ratio"], x["state"], x["comp_k"],
                                x["comp_v"])
        return {"comp_k": x["comp_k"], "comp_v": x["comp_v"]}
    if c["op"] == "attn":
        ds4a.ds4a_attn_tree(x["kv"], x["q"], x["n"], x["parent"], c["window"], x.get("comp_k"), x.get("comp_v"),
                            c["ratio"], x.get("sel"), 1.0 / math.sqrt(c["D"]), x["out"], x["ws"])
        return {"out": x["out"]}
    ds4a.ds4a_paged_append(x["kv"], x["k"], x["v"], x["n"])
    ds4a.ds4a_commit_tree(x["kv"], x["n"], x["parent"], x["leaf"], x["len_out"], x["w"], c["ratio"], x["state"],
                          x["state_out"], x["comp_k"], x["comp_v"], x.get("k_idx"))
    return _outs_commit(x)


def _outs_append(x):
    o = {"pool_k": x["pool_k"], "pool_v": x["pool_v"]}
    if "q_out" in x:
        o["q_out"] = x["q_out"]
    return o


def _outs_commit(x):
    o = {k: x[k] for k in ("pool_k", "pool_v", "len_out", "state_out", "comp_k", "comp_v")}
    if "k_idx" in x:
        o["k_idx"] = x["k_idx"]
    return o


def _ancestors(x):
    """(anc [B, N, N] truth values including the node itself, depth [B, N])."""
    c = x["case"]
    N = c["N"]
    node = torch.arange(N, device=DEV)
    anc = (x["parent"][:, :, None] == node) | (node[:, None] == node)
    span = 1
    while span < N:
        f = anc.float()
        anc = (f @ f) > 0
        span *= 2
    return anc, anc.sum(2) - 1


def _rotate(c, t, pos, inv_freq):
    """t [B, N, heads, D] rotated to pos [B, N]."""
    rot, off = c["rot"], c["rot_off"]
    ang = pos.double()[..., None] * inv_freq.double()
    cs, sn = torch.cos(ang).float()[:, :, None], torch.sin(ang).float()[:, :, None]
    f = t.float()
    part = f[..., off:off + rot]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack([a * cs - b * sn, a * sn + b * cs], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        new = torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
    return torch.cat([f[..., :off], new, f[..., off + rot:]], -1).half()


def _append_plain(x):
    c = x["case"]
    N, D = c["N"], c["D"]
    slot = x["len"][:, None] + torch.arange(N, device=DEV)
    pos = slot
    if c["tree"] == "tree" and "inv_freq" in x:
        pos = x["len"][:, None] + _ancestors(x)[1]
    ok = torch.arange(N, device=DEV) < x["n"][:, None]
    row = _rows(x, slot)
    k = _rotate(c, x["k"][:, :, None], pos, x["inv_freq"])[:, :, 0] if "inv_freq" in x else x["k"]
    for pool, new in ((x["pool_k"], k), (x["pool_v"], x["v"])):
        flat = pool.view(-1, D)
        flat[row] = torch.where(ok[..., None], new, flat[row])
    if "q_out" in x:
        x["q_out"].copy_(torch.where(ok[..., None, None], _rotate(c, x["q"], pos, x["inv_freq"]), x["q_out"]))


def _run_plain(x):
    c = x["case"]
    B, N, H, D, ratio = c["B"], c["N"], c["H"], c["D"], c["ratio"]
    if c["op"] == "append":
        _append_plain(x)
        return _outs_append(x)
    if c["op"] == "commit":
        _append_plain(x)
    anc, depth = _ancestors(x)
    pos = x["len"][:, None] + depth
    node = torch.arange(N, device=DEV)
    ok = node < x["n"][:, None]
    drow = _rows(x, x["len"][:, None] + node)
    dk, dv = x["pool_k"].view(-1, D)[drow].float(), x["pool_v"].view(-1, D)[drow].float()
    if c["op"] == "compress":
        done = ok & ((pos + 1) % ratio == 0)
        blk = torch.div(pos, ratio, rounding_mode="floor")
        s = dk @ x["w"]
        member = anc & (blk[:, :, None] == blk[:, None, :])
        has = (blk == torch.div(x["len"], ratio, rounding_mode="floor")[:, None]) & (x["len"] % ratio > 0)[:, None]
        sm = torch.where(member, s[:, None, :], -math.inf)
        so = torch.where(has, x["state"][:, :1], -math.inf)
        m = torch.maximum(sm.max(2).values, so)
        e, eo = torch.exp(sm - m[..., None]), torch.exp(so - m)
        total = e.sum(2) + eo * x["state"][:, 1:2]
        cap = x["comp_k"].shape[1]
        for dst, tok, acc in ((x["comp_k"], dk, x["state"][:, 2:2 + D]), (x["comp_v"], dv, x["state"][:, 2 + D:])):
            acc = torch.where(has[..., None], acc[:, None], torch.zeros((), device=DEV))
            row = (e @ tok + eo[..., None] * acc) / total[..., None]
            dst[:, cap - N:] = torch.where(done[..., None], row.half(), dst[:, cap - N:])
        return {"comp_k": x["comp_k"], "comp_v": x["comp_v"]}
    if c["op"] == "attn":
        return _attn_plain(x, anc, depth, pos, ok, dk, dv)
    return _commit_plain(x, anc, depth, pos, dk, dv)


def _attn_plain(x, anc, depth, pos, ok, dk, dv):
    c = x["case"]
    B, N, H, D, ratio = c["B"], c["N"], c["H"], c["D"], c["ratio"]
    scale = 1.0 / math.sqrt(D)
    ln = x["len"][:, None]
    wn = min(c["window"], c["ctx"])
    t = ln - wn + torch.arange(wn, device=DEV)
    row = _rows(x, t.clamp(min=0))
    ks, vs = [x["pool_k"].view(-1, D)[row].float(), dk], [x["pool_v"].view(-1, D)[row].float(), dv]
    masks = [(t >= 0)[:, None] & (t[:, None] > pos[..., None] - c["window"]),
             anc & (pos[:, None, :] > pos[..., None] - c["window"])]
    qf = x["q"].float()
    if ratio and not c["sel"]:
        cap = x["comp_k"].shape[1]
        ks.append(x["comp_k"].float())
        vs.append(x["comp_v"].float())
        j = torch.arange(cap - N, device=DEV)
        n_vis = torch.div(ln, ratio, rounding_mode="floor")
        masks.append((j < n_vis)[:, None].expand(B, N, cap - N))
        masks.append(anc & ((pos + 1) % ratio == 0)[:, None, :])
    k, v, mask = torch.cat(ks, 1), torch.cat(vs, 1), torch.cat(masks, 2)
    s = (qf.view(B, N * H, D) @ k.transpose(1, 2)).view(B, N, H, -1) * scale
    s = torch.where(mask[:, :, None], s, -math.inf)
    if c["sel"]:
        cap = x["comp_k"].shape[1]
        j = x["sel"].long()
        n_vis = torch.div(ln, ratio, rounding_mode="floor")[..., None]
        # a row past the committed ones is the one that the ancestor at its last position completed
        want = (j + 1) * ratio - 1 - ln[..., None]
        hit = anc[:, :, None, :] & (depth[:, None, None, :] == want[..., None])
        rowi = torch.where(j < n_vis, j, cap - N + hit.float().argmax(3)).clamp(min=0)
        b = torch.arange(B, device=DEV)[:, None, None]
        ck, cv = x["comp_k"][b, rowi].float(), x["comp_v"][b, rowi].float()
        s2 = (qf @ ck.transpose(2, 3)) * scale
        s = torch.cat([s, torch.where((j >= 0)[:, :, None], s2, -math.inf)], 3)
    p = torch.exp(s - s.max(3, keepdim=True).values)
    p = p / p.sum(3, keepdim=True)
    m = k.shape[1]
    o = (p[..., :m].reshape(B, N * H, m) @ v).view(B, N, H, D)
    if c["sel"]:
        o = o + p[..., m:] @ cv
    x["out"].copy_(torch.where(ok[..., None, None], o.half(), x["out"]))
    return {"out": x["out"]}


def _commit_plain(x, anc, depth, pos, dk, dv):
    c = x["case"]
    B, N, D, ratio = c["B"], c["N"], c["D"], c["ratio"]
    node = torch.arange(N, device=DEV)
    b = torch.arange(B, device=DEV)
    leaf = x["leaf"].long()
    on = anc[b, leaf.clamp(min=0)] & (leaf >= 0)[:, None]               # nodes of the accepted path
    cnt = on.sum(1)
    x["len_out"].copy_(x["len"] + cnt)
    # path[d]: the path's node at depth d (the node itself behind the path's end)
    hit = on[:, None, :] & (depth[:, None, :] == node[:, None])
    inside = node < cnt[:, None]
    path = torch.where(inside, hit.float().argmax(2), node)
    dst = _rows(x, x["len"][:, None] + node)
    src = _rows(x, x["len"][:, None] + path)
    for pool in (x["pool_k"], x["pool_v"]):
        flat = pool.view(-1, D)
        flat[dst] = flat[src]
    # compressed rows completed on the path
    cap = x["comp_k"].shape[1]
    done = inside & ((x["len"][:, None] + node + 1) % ratio == 0)
    row = torch.div(x["len"][:, None] + node, ratio, rounding_mode="floor")
    draft = cap - N + path
    to = torch.where(done, row, cap - N + node)                         # the others write their own row back
    fr = torch.where(done, draft, cap - N + node)
    arrays = [x["comp_k"], x["comp_v"]] + ([x["k_idx"]] if "k_idx" in x else [])
    for a in arrays:
        a[b[:, None], to] = a[b[:, None], fr]
    # the block left open
    end = x["len"] + cnt
    blk = torch.div(end, ratio, rounding_mode="floor")
    member = on & (torch.div(pos, ratio, rounding_mode="floor") == blk[:, None])
    has = (blk == torch.div(x["len"], ratio, rounding_mode="floor")) & (x["len"] % ratio > 0)
    s = torch.where(member, dk @ x["w"], -math.inf)
    so = torch.where(has, x["state"][:, 0], -math.inf)
    m = torch.maximum(s.max(1).values, so)
    e, eo = torch.exp(s - m[:, None]), torch.where(has, torch.exp(so - m), 0.0)
    l = e.sum(1) + eo * x["state"][:, 1]
    ak = (e[:, None] @ dk)[:, 0] + eo[:, None] * x["state"][:, 2:2 + D]
    av = (e[:, None] @ dv)[:, 0] + eo[:, None] * x["state"][:, 2 + D:]
    new = torch.cat([m[:, None], l[:, None], ak, av], 1)
    x["state_out"].copy_(torch.where((end % ratio > 0)[:, None], new, x["state_out"]))
    return _outs_commit(x)


# ---- work ------------------------------------------------------------------------------------

def work(case):
    c = case
    N, H, D, ratio = c["N"], c["H"], c["D"], c["ratio"]
    ln, n = _lengths(c)
    tok = int(n.sum())
    if c["op"] == "append":
        by = tok * (8 * D + (4 * H * D if c["q"] else 0))
        return {"bytes": by, "flops": tok * (1 + (H if c["q"] else 0)) * 3 * c["rot"]}
    if c["op"] == "compress":
        rows = sum(max(1, int(k) // ratio) for k in n)
        return {"bytes": 4 * tok * D + 4 * rows * D + c["B"] * 4 * (2 + 2 * D), "flops": 8 * tok * D}
    if c["op"] == "commit":
        acc = tok // 4
        by = tok * 8 * D + acc * 8 * D + c["B"] * 8 * (2 + 2 * D)
        return {"bytes": by, "flops": acc * 6 * D}
    by, fl = 0, 0
    for a, k in zip(ln, n):
        a, k = int(a), int(k)
        raw = min(c["window"], a)
        rows = min(c["sel"], a // ratio) if c["sel"] else (a // ratio if ratio else 0)
        read = min(a // ratio, rows * k) if c["sel"] else rows
        by += 4 * k * H * D + 4 * D * (raw + k + read) + (4 * c["sel"] * k if c["sel"] else 0)
        fl += 4 * D * H * k * (raw + rows + 1)
    return {"bytes": by, "flops": fl}


# ---- the definitions in 64 bits --------------------------------------------------------------

def exact(case, seed):
    x = _inputs(case, seed)
    c = case
    B, N, D, page, ratio = c["B"], c["N"], c["D"], c["page"], c["ratio"]
    ln, n, par, tab = (x[k].cpu().numpy() for k in ("len", "n", "parent", "table"))
    pk, pv = x["pool_k"].view(-1, D).double(), x["pool_v"].view(-1, D).double()

    def place(s, t):
        t = np.asarray(t, np.int64)
        return torch.from_numpy(tab[s][t // page].astype(np.int64) * page + t % page).to(DEV)
    paths = []                          # root-to-node lists
    for s in range(B):
        ps = []
        for i in range(int(n[s])):
            up = int(par[s, i])
            ps.append((ps[up] if up >= 0 else []) + [i])
        paths.append(ps)
    if c["op"] == "commit":
        for s in range(B):
            where = place(s, ln[s] + np.arange(int(n[s])))
            pk[where], pv[where] = x["k"][s, :n[s]].double(), x["v"][s, :n[s]].double()
    if c["op"] == "append":
        half = c["rot"] // 2
        if c["interleaved"]:
            i1 = c["rot_off"] + 2 * torch.arange(half, device=DEV)
            i2 = i1 + 1
        else:
            i1 = c["rot_off"] + torch.arange(half, device=DEV)
            i2 = i1 + half

        def turn(t, pos):               # t [m, ..., D] by positions [m]
            th = torch.from_numpy(np.asarray(pos, np.float64)).to(DEV)[:, None] * x["inv_freq"].double()
            th = th.view(th.shape[0], *([1] * (t.dim() - 2)), half)
            r = t.clone()
            r[..., i1] = t[..., i1] * torch.cos(th) - t[..., i2] * torch.sin(th)
            r[..., i2] = t[..., i1] * torch.sin(th) + t[..., i2] * torch.cos(th)
            return r
        qo = x["q_out"].double() if "q_out" in x else None
        for s in range(B):
            m = int(n[s])
            pos = [int(ln[s]) + (len(paths[s][i]) - 1 if c["tree"] == "tree" else i) for i in range(m)]
            where = place(s, ln[s] + np.arange(m))
            pk[where] = turn(x["k"][s, :m].double(), pos)
            pv[where] = x["v"][s, :m].double()
            if qo is not None:
                qo[s, :m] = turn(x["q"][s, :m].double(), pos)
        o = {"pool_k": pk.view_as(x["pool_k"]), "pool_v": pv.view_as(x["pool_v"])}
        if qo is not None:
            o["q_out"] = qo
        return o
    if c["op"] == "attn":
        return {"out": _exact_attn(x, ln, n, paths, place, pk, pv)}

    def pooled(s, toks, p0):
        """(max, sum, K, V) over the open block's state (if p0, the first token's position, is inside one) and
        drafted tokens toks."""
        rows = place(s, int(ln[s]) + np.array(toks))
        k, v = pk[rows], pv[rows]
        sc = k @ x["w"].double()
        m = sc.max()
        st = x["state"][s].double()
        cont = p0 == int(ln[s]) and p0 % ratio != 0
        if cont:
            m = torch.maximum(m, st[0])
        e = torch.exp(sc - m)
        l, a, b = e.sum(), e @ k, e @ v
        if cont:
            f = torch.exp(st[0] - m)
            l, a, b = l + f * st[1], a + f * st[2:2 + D], b + f * st[2 + D:]
        return m, l, a, b

    cap = x["comp_k"].shape[1]
    ck, cv = x["comp_k"].double(), x["comp_v"].double()
    if c["op"] == "compress":
        for s in range(B):
            for i, path in enumerate(paths[s]):
                end = int(ln[s]) + len(path)
                if end % ratio:
                    continue
                first = max(int(ln[s]), end - ratio)
                _, l, a, b = pooled(s, path[first - int(ln[s]):], first)
                ck[s, cap - N + i], cv[s, cap - N + i] = a / l, b / l
        return {"comp_k": ck, "comp_v": cv}
    leaf = x["leaf"].cpu().numpy()
    len_out, state = x["len"].clone(), x["state_out"].double()
    ki = x["k_idx"].double() if "k_idx" in x else None
    nk, nv = pk.clone(), pv.clone()
    for s in range(B):
        path = paths[s][int(leaf[s])] if leaf[s] >= 0 else []
        a0 = int(ln[s])
        end = a0 + len(path)
        len_out[s] = end
        for d, i in enumerate(path):
            to, fr = place(s, [a0 + d]), place(s, [a0 + i])
            nk[to], nv[to] = pk[fr], pv[fr]
            if (a0 + d + 1) % ratio == 0:
                r = (a0 + d) // ratio
                for arr in (ck, cv) + ((ki,) if ki is not None else ()):
                    arr[s, r] = arr[s, cap - N + i]
        first = max(a0, end - end % ratio)
        if end % ratio and first < end:
            m, l, a, b = pooled(s, path[first - a0:], first)
            state[s] = torch.cat([m[None], l[None], a, b])
    o = {"pool_k": nk.view_as(x["pool_k"]), "pool_v": nv.view_as(x["pool_v"]), "len_out": len_out, "state_out": state,
         "comp_k": ck, "comp_v": cv}
    if ki is not None:
        o["k_idx"] = ki
    return o


def _exact_attn(x, ln, n, paths, place, pk, pv):
    c = x["case"]
    B, N, D, ratio = c["B"], c["N"], c["D"], c["ratio"]
    out = x["out"].double()
    cap = x["comp_k"].shape[1] if ratio else 0
    sel = x["sel"].cpu().numpy() if c["sel"] else None
    for s in range(B):
        a0 = int(ln[s])
        lo = max(0, a0 - c["window"] + 1)
        base = place(s, np.arange(lo, a0))
        kb, vb = pk[base], pv[base]
        n_vis = a0 // ratio if ratio else 0
        if ratio:
            ck, cv = x["comp_k"][s].double(), x["comp_v"][s].double()
        for i, path in enumerate(paths[s]):
            p = a0 + len(path) - 1
            first = max(0, p - c["window"] + 1)
            skip = min(max(0, first - lo), a0 - lo)
            near = [j for d, j in enumerate(path) if a0 + d >= first]
            rows = place(s, a0 + np.array(near))
            ks, vs = [kb[skip:], pk[rows]], [vb[skip:], pv[rows]]
            if ratio:
                by_row = {(a0 + d) // ratio: cap - N + j for d, j in enumerate(path) if (a0 + d + 1) % ratio == 0}
                if sel is None:
                    idx = list(range(n_vis)) + list(by_row.values())
                else:
                    idx = [int(j) if j < n_vis else by_row[int(j)] for j in sel[s, i] if j >= 0]
                at = torch.tensor(idx, dtype=torch.long, device=DEV)
                ks.append(ck[at])
                vs.append(cv[at])
            k, v = torch.cat(ks), torch.cat(vs)
            w = torch.softmax(x["q"][s, i].double() @ k.T / math.sqrt(D), 1)
            out[s, i] = w @ v
    return out
