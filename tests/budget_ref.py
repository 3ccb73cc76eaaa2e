"""Caches held to a budget, in 64 bits (numpy): normed rows, attention weights, eviction."""
import numpy as np


def norm(x, w, eps):
    """x [..., D] float64 through the RMS norm with weights w (None: ones)."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if w is None else y * w.astype(np.float64)


def rows_lse(q, k, scale, see):
    """(scaled scores [n, H, T], log of the sum of exp [n, H]) of queries q [n, H, D] over keys k [T, D],
    see [n, T]: which keys a token attends."""
    s = np.einsum("nhd,td->nht", q.astype(np.float64), k.astype(np.float64)) * scale
    s = np.where(see[:, None], s, -np.inf)
    m = s.max(2, keepdims=True)
    return s, np.where(np.isfinite(m), m + np.log(np.exp(s - np.where(np.isfinite(m), m, 0)).sum(2, keepdims=True)), m)[..., 0]


def weights(q, k, scale, lse32, ln):
    """(weight that each of the len + n slots gets, tolerance) from the tokens q [n, H, D] over k [len + n, D],
    lse32 [n, H] as given.  The score's products are exact in binary32 and their sum of D is off by at most
    2 D 2^-24 of the sum of |q k|; its factor (scale times log2 e, each rounded: 3 * 2^-24), the scaled lse
    (2 * 2^-24) and the exponent (2^-24 of at most |s| + |lse|) add 6 * 2^-24 of |s| + |lse|; a power of two is
    off by 2^-22 of itself, and a sum of m weights by m 2^-24 of the sum."""
    n, H, D = q.shape
    T = k.shape[0]
    see = np.arange(T) <= ln + np.arange(n)[:, None]
    q, k = q.astype(np.float64), k.astype(np.float64)
    s = np.einsum("nhd,td->nht", q, k) * scale
    mass = np.einsum("nhd,td->nht", np.abs(q), np.abs(k)) * scale
    lse = lse32.astype(np.float64)[..., None]
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.where(see[:, None] & (lse != -np.inf), np.exp(s - lse), 0.0)
    off = 2 * D * 2.0 ** -24 * mass + 6 * 2.0 ** -24 * (np.abs(s) + np.abs(np.where(np.isfinite(lse), lse, 0))) + 2.0 ** -22
    total = p.sum((0, 1))
    return total, (p * 2 * off).sum((0, 1)) + n * H * 2.0 ** -24 * total + 2.0 ** -126


def evict(acc, pos, nxt, ln, budget, sink, recent):
    """(kept tokens' slots in their new places [min(len, budget)], dropped slots below the budget)."""
    if ln <= budget:
        return np.arange(ln), np.zeros(0, np.int64)
    a = acc[:ln].astype(np.float64)
    always = (pos[:ln] < sink) | (pos[:ln].astype(np.int64) >= nxt - recent)
    number = np.where(np.isnan(a) & ~always, 0, 1)
    a = np.where(np.isnan(a) | always, 0, a)            # more that are always kept than the budget has place for: by slot
    rank = np.lexsort((np.arange(ln), -a, -number, ~always))
    kept = np.zeros(ln, bool)
    kept[rank[:budget]] = True
    place = np.arange(budget)
    holes = np.nonzero(~kept[:budget])[0]
    place[holes] = budget + np.nonzero(kept[budget:])[0]
    return place, holes
