"""Drafted-token trees in 64 bits, one node at a time (numpy): what the calls on the paged
cache are compared with."""
import numpy as np


def paths_of(parent, n):
    """Root-to-node index lists of nodes 0 .. n-1."""
    out = []
    for i in range(n):
        out.append((out[parent[i]] if parent[i] >= 0 else []) + [i])
    return out


def random_parents(rng, B, N, kind="tree"):
    par = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        if kind == "chain":
            par[:, i] = i - 1
        elif kind == "tree":
            par[:, i] = rng.integers(max(-1, i - 4), i, B)
        # "roots": every node continues the last committed token
    return par


def slot_rows(table_row, page, slots):
    slots = np.asarray(slots, np.int64)
    return table_row[slots // page].astype(np.int64) * page + slots % page


def rotate(x, pos, inv_freq, off, interleaved):
    """x [..., D] float64 rotated to position pos."""
    half = len(inv_freq)
    th = float(pos) * inv_freq.astype(np.float64)
    i1 = off + (2 * np.arange(half) if interleaved else np.arange(half))
    i2 = i1 + 1 if interleaved else i1 + half
    y = x.copy()
    y[..., i1] = x[..., i1] * np.cos(th) - x[..., i2] * np.sin(th)
    y[..., i2] = x[..., i1] * np.sin(th) + x[..., i2] * np.cos(th)
    return y


def node_keys(pool_k, pool_v, comp_k, comp_v, table_row, page, ln, path, N, window, ratio, sel):
    """(K, V) rows that the last node of `path` attends; pools [rows, D], comp [cap, D]."""
    p = ln + len(path) - 1
    first = max(0, p - window + 1)
    slots = [t if t < ln else ln + path[t - ln] for t in range(first, p + 1)]
    rows = slot_rows(table_row, page, slots)
    ks, vs = [pool_k[rows]], [pool_v[rows]]
    if ratio:
        cap = comp_k.shape[0]
        js = range((p + 1) // ratio) if sel is None else [j for j in sel if 0 <= j < (p + 1) // ratio]
        at = [j if j < ln // ratio else cap - N + path[(j + 1) * ratio - 1 - ln] for j in js]
        ks.append(comp_k[at])
        vs.append(comp_v[at])
    return np.concatenate(ks).astype(np.float64), np.concatenate(vs).astype(np.float64)


def attend(q, k, v, scale):
    """(out [H, D], tolerance [H, D]) of one node.  The kernel rounds each weight to 16 bits
    (half a step: 2^-11 of it, or 2^-25 below the smallest normal, the largest weight being
    at least 1) in the products with V and possibly in their sum, and the result once more; its
    scores carry binary32 sums of D products, off by at most 2 D 2^-24 of the sum of |q k|, which
    moves a weight by that much relatively, and so does the sum of n weights (n 2^-24, taken in
    parts of 128)."""
    q = q.astype(np.float64)
    s = q @ k.T * scale
    w = np.exp(s - s.max(1, keepdims=True))
    l = w.sum(1, keepdims=True)
    out = w @ v / l
    d = q.shape[1]
    ds = (2 * d * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(k).T)).max(1, keepdims=True)
    wabs = w @ np.abs(v) / l
    mean = (w.sum(1, keepdims=True) + 0 * out) / l
    rel = 2 * 2.0 ** -11 + 2 * ds + 256 * 2.0 ** -24
    tol = rel * (wabs + np.abs(out) * mean) + 2.0 ** -25 * np.abs(v).sum(0) / l + 2.0 ** -11 * np.abs(out) + 2.0 ** -25
    return out, tol


def pool_block(k, v, w, state=None):
    """(max, sum, K sum, V sum) of the tokens k, v [m, D], continuing `state`."""
    s = k @ w
    m = s.max() if len(s) else -np.inf
    D = k.shape[1]
    if state is not None:
        m = max(m, float(state[0]))
    e = np.exp(s - m)
    l, a, b = e.sum(), e @ k, e @ v
    if state is not None:
        f = np.exp(float(state[0]) - m)
        l, a, b = l + f * state[1], a + f * state[2:2 + D], b + f * state[2 + D:]
    return m, l, a, b
