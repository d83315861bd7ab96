"""Plain 64-bit forms of the quantised cache's and the trees' operators, for the tests."""
import math

import numpy as np

from _kv_ref import U32, UBF, ceil_div

LOWEST = -100


def quantise(x):
    """Codes' values and exponents of rows [..., D] (float64): the smallest 2^e, e >= -100, with max |x| <= 448 * 2^e; the
    nearest of e4m3's values to x / 2^e, ties to the even one. Rows with values that are not finite: zeros and None's place, 128."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    x = np.where(bad[..., None], 0.0, x)
    top = np.abs(x).max(-1)
    e = np.full(top.shape, LOWEST, dtype=np.int64)
    while True:
        low = top > np.ldexp(448.0, e)
        if not low.any():
            break
        e += low
    y = np.ldexp(x, -e[..., None])
    step = np.ldexp(1.0, np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6))).astype(np.int64) - 3)
    return np.round(y / step) * step, np.where(bad, 128, e)


def restored(codes, scales):
    """Numbers of codes' values [..., D] and scale bytes [...]."""
    s = np.asarray(scales, dtype=np.int64)
    return np.where((s == 255)[..., None], np.nan, np.ldexp(np.asarray(codes, dtype=np.float64), (s - 127)[..., None]))


def ancestors(parent, window=0):
    """[n, n] truth values: node i sees node j (itself or an ancestor less than `window` above it); depths."""
    n = len(parent)
    seen, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int64)
    for i in range(n):
        j, up = i, 0
        while j >= 0:
            if not window or up < window:
                seen[i, j] = True
            j, up = parent[j], up + 1
        depth[i] = up - 1
    return seen, depth


def words(seen, W):
    """Rows of truth values as W int32 words, the lowest bit first."""
    n, m = seen.shape
    out = np.zeros((n, W), dtype=np.int64)
    for i, j in zip(*np.nonzero(seen)):
        out[i, j // 32] |= 1 << int(j % 32)
    return out.astype(np.uint32).view(np.int32)


def tree_seen(mask, depth, n, kv, window):
    """[n, kv]: what the rows of a tree see; mask [n, n] truth values."""
    first = kv - n
    seen = np.zeros((n, kv), dtype=bool)
    j = np.arange(kv)
    for i in range(n):
        p = first + (0 if depth is None else max(0, int(depth[i])))
        seen[i] = (j < first) & ((j > p - window) if window else True)
        for t in range(n):
            if mask[i, t] and first + t >= 0:
                seen[i, first + t] = True
    return seen


def attend(q, k_pool, v_pool, table, kv_len, q_start, seen_of, scale, bf16):
    """out, lse and the bounds of their absolute errors, as in _kv_ref.attend, with `seen_of(b)` [rows, kv_len[b]] for
    what a request's rows see. Pages that no row sees are not looked at."""
    T, H, D = q.shape
    Hk, S = k_pool.shape[2], k_pool.shape[1]
    G = H // Hk
    out, lse = np.zeros((T, H, D)), np.full((T, H), -np.inf)
    out_tol, lse_tol = np.zeros((T, H, D)), np.zeros((T, H))
    for b in range(len(kv_len)):
        n, q0 = int(kv_len[b]), int(q_start[b])
        rows = int(q_start[b + 1]) - q0
        if rows == 0 or n == 0:
            continue
        seen = seen_of(b)
        visible = seen.any(0)
        k = np.zeros((ceil_div(n, S) * S, Hk, D))
        v = np.zeros_like(k)
        for page in range(ceil_div(n, S)):
            if visible[page * S:(page + 1) * S].any():
                k[page * S:(page + 1) * S] = k_pool[table[b, page]]
                v[page * S:(page + 1) * S] = v_pool[table[b, page]]
        for h in range(H):
            kk = np.where(visible[:, None], k[:n, h // G], 0.0)
            vv = np.where(visible[:, None], v[:n, h // G], 0.0)
            x = q[q0:q0 + rows, h].astype(np.float64)
            s = np.where(seen, scale * (x @ kk.T), -np.inf)
            mass = np.where(seen, scale * (np.abs(x) @ np.abs(kk).T), 0.0).max(1)
            m = s.max(1)
            some = np.isfinite(m)
            e = np.where(seen, np.exp(s - np.where(some, m, 0.0)[:, None]), 0.0)
            l = e.sum(1)
            p = e / np.where(l > 0, l, 1.0)[:, None]
            out[q0:q0 + rows, h] = p @ vv
            with np.errstate(divide="ignore"):
                lse[q0:q0 + rows, h] = np.where(some, m, 0.0) + np.log(l)
            J = seen.sum(1)
            ds = (D + 4) * U32 * mass + 4 * U32 * np.abs(np.where(some, m, 0.0))
            rel = 2 * ds + (J + 32) * U32 + (2 * 1.25 * UBF if bf16 else 0.0)
            out_tol[q0:q0 + rows, h] = rel[:, None] * (p @ np.abs(vv)) + 1e-30
            lse_tol[q0:q0 + rows, h] = ds + (J + 16) * U32 + 4 * U32 * np.abs(np.where(some, lse[q0:q0 + rows, h], 0.0))
    return out, lse, out_tol, lse_tol


def causal_seen(n, kv, causal=True, window=0):
    pos = kv - n + np.arange(n)
    j = np.arange(kv)
    hi = np.minimum(pos + 1, kv) if causal else np.full(n, kv)
    lo = np.maximum(0, pos - window + 1) if window else np.zeros(n, dtype=int)
    return (j[None] < hi[:, None]) & (j[None] >= lo[:, None])


def keep(rows, path, n, kv):
    """Where a request's row at each position comes from after its path is kept, and its length; None: refused.
    rows: positions of the request's tokens before."""
    m = next((i for i, x in enumerate(path) if x < 0), len(path))
    path = list(path[:m])
    first = kv - n
    if first < 0 or any(x >= n for x in path) or any(a >= z for a, z in zip(path, path[1:])):
        return None
    out = list(rows)
    for i, x in enumerate(path):
        out[first + i] = rows[first + x]
    return out, first + m


def random_tree(rng, n, roots=0.2, chain=0.0):
    """Parents of n nodes; `roots` of them hang on the context, `chain` of them on the node before."""
    parent = np.full(n, -1, dtype=np.int64)
    for i in range(1, n):
        u = rng.rand()
        parent[i] = -1 if u < roots else i - 1 if u < roots + chain else rng.randint(0, i)
    return parent


def default_scale(D):
    return 1.0 / math.sqrt(D)
