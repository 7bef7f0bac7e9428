"""Plain fp64 CPU oracle of the attention operators around the reuse path.

TEST INFRASTRUCTURE ONLY, like the rest of this directory: numpy float64, no code
shared with the library.  Inputs are upcast exactly; loops are plain, one head or one
query at a time.  Pinned in tests/test_attention_host.py to torch's
scaled_dot_product_attention, to complex multiplication, to hand-worked rows and to
brute force over all subsets.
"""
from __future__ import annotations

import numpy as np

NEG = -np.inf


def visible(p: int, n: int, window: int, sinks: int) -> np.ndarray:
    """Keys 0..n-1 that a query at position p sees."""
    j = np.arange(n)
    v = j <= p
    if window > 0:
        v &= (j > p - window) | (j < sinks)
    return v


def attend(q, K, V, scale, seen):
    """One query over the keys `seen`: (o [d], lse, weights [n], terms [d], bound).

    terms = sum_j w_j |v_j| and bound = max_j |scale| sum_e |q_e k_je| are what
    tolerances are derived from.  Masked rows of K and V are never touched."""
    n, d = K.shape
    w = np.zeros(n)
    idx = np.flatnonzero(seen)
    if idx.size == 0:
        return np.zeros(d), NEG, w, np.zeros(d), 0.0
    with np.errstate(invalid="ignore"):
        s = scale * (K[idx] @ q)
        bound = float(np.max(abs(scale) * (np.abs(K[idx]) @ np.abs(q))))
        m = s.max()
        e = np.exp(s - m)
        l = e.sum()
        w[idx] = e / l
        o = w[idx] @ V[idx]
        return o, m + np.log(l), w, w[idx] @ np.abs(V[idx]), bound


def attention(Q, K, V, scale, window=0, sinks=0):
    """Q [H][M][d], K [Hk][N][d], V [N][Hk][d]: dict of O [M][H][d], lse [H][M], the
    per-key mass [Hk][N], and the tolerance terms A [M][H][d], bound [H][M]."""
    Q, K, V, scale = (np.asarray(x, dtype=np.float64) for x in (Q, K, V, scale))
    H, M, d = Q.shape
    Hk, N, _ = K.shape
    O, A = np.zeros((M, H, d)), np.zeros((M, H, d))
    lse, bound = np.zeros((H, M)), np.zeros((H, M))
    mass = np.zeros((Hk, N))
    for i in range(M):
        seen = visible(N - M + i, N, window, sinks)
        for h in range(H):
            g = h // (H // Hk)
            O[i, h], lse[h, i], w, A[i, h], bound[h, i] = attend(Q[h, i], K[g], V[:, g], scale[h],
                                                                 seen)
            mass[g] += w
    return dict(O=O, lse=lse, mass=mass, A=A, bound=bound)


def cache_rows(pool, table, n, page):
    """[Hk][n][d] rows of one sequence and which of them lie on a page of the pool."""
    P, Hk, _, d = pool.shape
    rows, ok = np.zeros((Hk, n, d)), np.zeros(n, dtype=bool)
    for j in range(n):
        pg = int(table[j // page])
        if 0 <= pg < P:
            rows[:, j] = pool[pg, :, j % page]
            ok[j] = True
    return rows, ok


def decode(Q, K, V, lens, table, scale, window=0, sinks=0):
    """Q [S][H][d], pools [P][Hk][page][d], table [S][max_pages]: dict of O, lse [S][H],
    mass (list of [Hk][n]), A, bound."""
    Q, K, V, scale = (np.asarray(x, dtype=np.float64) for x in (Q, K, V, scale))
    S, H, d = Q.shape
    Hk, page = K.shape[1], K.shape[2]
    O, A = np.zeros((S, H, d)), np.zeros((S, H, d))
    lse, bound, mass = np.zeros((S, H)), np.zeros((S, H)), []
    for s in range(S):
        n = int(lens[s])
        Ks, ok = cache_rows(K, table[s], n, page)
        Vs, _ = cache_rows(V, table[s], n, page)
        seen = ok & visible(n - 1, n, window, sinks)
        ms = np.zeros((Hk, n))
        for h in range(H):
            g = h // (H // Hk)
            O[s, h], lse[s, h], w, A[s, h], bound[s, h] = attend(Q[s, h], Ks[g], Vs[g], scale[h],
                                                                 seen)
            ms[g] += w
        mass.append(ms)
    return dict(O=O, lse=lse, mass=mass, A=A, bound=bound)


def norm_rope(x, w, eps, freq, positions, layout, factor):
    """x [N][H][d] -> the normed and rotated rows (w None: no norm)."""
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    y = x.copy()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + len(freq))
        t = np.asarray(positions, dtype=np.float64) * f
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        y[..., a] = (x[..., a] * c - x[..., b] * s) * factor
        y[..., b] = (x[..., b] * c + x[..., a] * s) * factor
    return y


def evict_rows(mass, n, budget, sinks, recent):
    """Kept rows of one head, ascending: the first `sinks`, the last `recent`, and the
    heaviest others, equal masses lowest row first, NaN as -infinity."""
    if n <= budget:
        return list(range(n))
    forced = set(range(sinks)) | set(range(n - recent, n))
    rest = [j for j in range(n) if j not in forced]
    key = [(-(NEG if np.isnan(mass[j]) else float(mass[j])), j) for j in rest]
    take = [j for _, j in sorted(key)[:budget - len(forced)]]
    return sorted(forced | set(take))
