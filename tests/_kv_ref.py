"""Plain 64-bit forms of the paged cache's operators, for the tests.

Attention on numpy arrays, one request and head at a time, with the error bound
of each output; the pages' bookkeeping on Python lists, one request at a time."""
import math

import numpy as np

U32 = 2.0 ** -24          # unit roundoff of float32
UBF = 2.0 ** -8           # of bfloat16: 8 significand bits, so half a unit in the last place is 2^-8 of the value


def ceil_div(a, b):
    return -(-a // b)


def gather(pool, pages, n):
    """Tokens 0..n-1 of a request: [n, heads, D] float64 (pool [pages, S, heads, D])."""
    if n == 0:
        return np.zeros((0,) + pool.shape[2:])
    return pool[pages].reshape((-1,) + pool.shape[2:])[:n].astype(np.float64)


def attend(q, k_pool, v_pool, table, kv_len, q_start, causal, window, scale, bf16):
    """out, lse and the bounds of their absolute errors, all float64.

    With a = scale * max_j sum_d |q_d k_jd|: a score's error is at most (D + 4) U32 a (D products and
    sums, the scale), the factors exp(s - r) follow with that and a few U32 of their own, and the sums
    over J keys with J U32; each weight rounded to bfloat16 and the result rounded once more cost UBF
    each, all of them relative to sum_j p_j |v_j|. A margin of 1.25 on the bfloat16 roundings covers
    their second-order terms."""
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
        pos = n - rows + np.arange(rows)
        hi = np.minimum(pos + 1, n) if causal else np.full(rows, n)
        lo = np.maximum(0, pos - window + 1) if window else np.zeros(rows, dtype=int)
        first = int(min(max(0, lo.min()), n))
        # only what some row sees is read: pages before that need no entry
        need = np.arange(first // S, ceil_div(n, S))
        k = np.zeros((ceil_div(n, S) * S, Hk, D))
        v = np.zeros_like(k)
        for page in need:
            k[page * S:(page + 1) * S] = k_pool[table[b, page]]
            v[page * S:(page + 1) * S] = v_pool[table[b, page]]
        j = np.arange(n)
        seen = (j[None] < hi[:, None]) & (j[None] >= lo[:, None])
        visible = seen.any(0)
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


def update(table, kv_len, ref, new_len, parent, S, N):
    """(table, kv_len, ref, copies) afterwards; copies: {request: (from page, to page, tokens)}. None: no room."""
    B, M = len(table), len(table[0])
    ref = list(ref)
    parent = list(range(B)) if parent is None else parent
    for b in range(B):
        for p in table[b][:ceil_div(kv_len[b], S)]:
            ref[p] -= 1
    keep = [min(kv_len[p], new_len[b]) if p >= 0 else 0 for b, p in enumerate(parent)]
    rows = [list(table[p][:ceil_div(k, S)]) if k else [] for k, p in zip(keep, parent)]
    for r in rows:
        for p in r:
            ref[p] += 1
    writers = {}
    for b in range(B):
        if keep[b] % S and new_len[b] > keep[b]:
            writers.setdefault(rows[b][-1], []).append(b)
    copies = {}
    for page, who in writers.items():
        if ref[page] > 1:
            for b in (who[1:] if len(who) == ref[page] else who):
                copies[b] = page
    free = [p for p in range(N) if ref[p] == 0]
    wanted = sum(ceil_div(new_len[b], S) - len(rows[b]) + (b in copies) for b in range(B))
    if wanted > len(free):
        return None
    done = {}
    for b in range(B):
        if b in copies:
            page = free.pop(0)
            ref[copies[b]] -= 1
            ref[page] = 1
            done[b] = (copies[b], page, keep[b] % S)
            rows[b][-1] = page
        while len(rows[b]) < ceil_div(new_len[b], S):
            page = free.pop(0)
            ref[page] = 1
            rows[b].append(page)
    return [r + [-1] * (M - len(r)) for r in rows], list(new_len), ref, done


def compact(table, ref):
    """(table, ref, page_map, used, moves) afterwards; moves: [(from, to)]."""
    held = [p for p, n in enumerate(ref) if n > 0]
    used = len(held)
    moves = list(zip([p for p in held if p >= used], [p for p in range(used) if ref[p] == 0]))
    to = {p: p for p in held}
    to.update(moves)
    out = list(ref)
    for a, z in moves:
        out[z], out[a] = ref[a], 0
    return ([[to.get(p, -1) if p >= 0 else -1 for p in row] for row in table], out,
            [to.get(p, -1) for p in range(len(ref))], used, moves)


def default_scale(D):
    return 1.0 / math.sqrt(D)
