"""The paged KV cache's operators as they are measured: cases, inputs, plain forms and exact values.

Four operators of the verify cycle (speculative_decoding_draft_block_gb300.kv_cache):
  attend    attention of ragged new tokens over a paged cache: single tokens, K + 1 verify tokens, draft blocks, prompts
  append    the new tokens' keys and values into their pages
  update    every request's next state: grow, roll back, free, fork (copy on write)
  compact   held pages moved to the front of the pool

`run` computes them in elementary torch operations (32-bit arithmetic, rounded once at the end), or, with `own`, calls the
library. Sizes follow the framework's workloads (B = 1, 32, 128, 512 requests; K = 4, 8, 16 drafted tokens; hidden sizes
256, 2560 and 4096 as heads of 64 or 128), with generic context lengths.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAX_SCORES = 2.2e9        # padded query rows x keys of the plain form's score matrix
MAX_KEYS = 1.1e9          # padded key elements of its gathered cache


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # one request answering alone: the latency of a single token over a short context
        dict(name="attend_token_B1", op="attend", dtype="bf16", B=1, heads=32, kv_heads=8, D=128, S=16, layout="nhd",
             q_lo=1, q_hi=1, kv_lo=517, kv_hi=517, causal=True, window=0),
        # a decode step of 128 requests: the cache is read once, nothing is reused
        dict(name="attend_token_B128", op="attend", dtype="bf16", B=128, heads=32, kv_heads=8, D=128, S=64, layout="nhd",
             q_lo=1, q_hi=1, kv_lo=300, kv_hi=8000, causal=True, window=0),
        # the verify pass of the headline workload: 128 requests, up to K + 1 = 17 scheduled tokens each
        dict(name="attend_verify_B128", op="attend", dtype="bf16", B=128, heads=32, kv_heads=8, D=128, S=32, layout="nhd",
             q_lo=1, q_hi=17, kv_lo=500, kv_hi=6000, causal=True, window=0),
        # the draft backbone's block of K = 8 positions: bidirectional within the block, sliding window, 5 heads a KV head
        dict(name="attend_draft_B32", op="attend", dtype="bf16", B=32, heads=20, kv_heads=4, D=128, S=16, layout="hnd",
             q_lo=8, q_hi=8, kv_lo=60, kv_hi=4001, causal=False, window=128),
        # prompts in chunks against what is cached of them: bound by the tensor cores
        dict(name="attend_prompt_B2", op="attend", dtype="bf16", B=2, heads=32, kv_heads=8, D=128, S=256, layout="nhd",
             q_lo=1777, q_hi=2048, kv_lo=9001, kv_hi=16384, causal=True, window=0),
        # float32 cache of a small model (hidden size 256), K + 1 = 5 tokens
        dict(name="attend_f32_B4", op="attend", dtype="f32", B=4, heads=4, kv_heads=2, D=64, S=16, layout="hnd",
             q_lo=5, q_hi=5, kv_lo=33, kv_hi=1000, causal=True, window=0),
        # a verify cycle's new tokens into the cache
        dict(name="append_verify_B128", op="append", dtype="bf16", B=128, kv_heads=8, D=128, S=32, layout="nhd",
             q_lo=1, q_hi=17, kv_lo=500, kv_hi=6000),
        # prompts into the cache, heads outside the page's tokens
        dict(name="append_prompt_B16", op="append", dtype="bf16", B=16, kv_heads=8, D=128, S=64, layout="hnd",
             q_lo=1023, q_hi=8192, kv_lo=1023, kv_hi=8192),
        # a cycle's bookkeeping: most requests grow by K + 1 or fall back, some end, some begin
        dict(name="update_cycle_B128", op="update", dtype="bf16", B=128, width=1, kv_heads=8, D=128, S=16, layout="nhd",
             L=2, N=16384, kv_lo=300, kv_hi=6000, step=17),
        # 64 searches of 8 beams each take their next parents: pages shared, the partly filled ones copied
        dict(name="update_beams_B512", op="update", dtype="bf16", B=512, width=8, kv_heads=8, D=128, S=16, layout="nhd",
             L=4, N=16384, kv_lo=200, kv_hi=1500, step=1),
        # a small pool after its requests ended in mixed order
        dict(name="compact_N512", op="compact", dtype="bf16", B=16, kv_heads=2, D=64, S=16, layout="hnd", L=2, N=512,
             held=0.5),
        # a serving pool shrunk to what is held
        dict(name="compact_N16384", op="compact", dtype="bf16", B=128, kv_heads=8, D=128, S=16, layout="nhd", L=4,
             N=16384, held=0.6),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "update", "compact"])
    dtype = "f32" if rng.random() < 0.25 else "bf16"
    D, kv_heads = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
    base = dict(op=op, dtype=dtype, D=D, kv_heads=kv_heads, layout=rng.choice(["nhd", "hnd"]))
    while True:
        if op == "attend":
            S, group = rng.choice([16, 32, 64, 128, 256]), rng.choice([1, 2, 4, 5, 7, 8, 16])
            form = rng.choice(["token", "verify", "prompt"])
            kv_hi = _log(rng, 17, 16384)
            kv_lo = _log(rng, 1, kv_hi)
            q_hi = {"token": 1, "verify": rng.randint(2, 33), "prompt": _log(rng, 64, 2048)}[form]
            q_lo = 1 if form == "token" else rng.randint(1, q_hi)
            c = dict(base, B=_log(rng, 1, 512 if form != "prompt" else 8), heads=kv_heads * group, S=S, q_lo=q_lo, q_hi=q_hi,
                     kv_lo=kv_lo, kv_hi=kv_hi, causal=rng.random() < 0.75, window=0 if rng.random() < 0.7 else _log(rng, 32, 2048))
            cap = 8.0e11 if dtype == "bf16" else 4e10
            if (work(c)["flops"] <= cap and c["B"] * c["heads"] * q_hi * kv_hi <= MAX_SCORES
                    and c["B"] * (kv_hi + S) * kv_heads * D <= MAX_KEYS):
                return c
        elif op == "append":
            q_hi = _log(rng, 1, 8192)
            kv_hi = q_hi + _log(rng, 1, 4096) - 1
            c = dict(base, B=_log(rng, 1, 512), S=rng.choice([16, 32, 64, 128, 256]), q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                     kv_lo=rng.randint(1, kv_hi), kv_hi=kv_hi)
            if work(c)["bytes"] <= 1.2e9 and c["B"] * (kv_hi + 256) * kv_heads * D <= 2e9:
                return c
        elif op == "update":
            width = rng.choice([1, 1, 2, 4, 8])
            B = width * _log(rng, 1, 512 // width)
            kv_hi = _log(rng, 20, 8000)
            c = dict(base, B=B, width=width, S=rng.choice([16, 32, 64]), L=rng.randint(1, 4), N=0, kv_lo=rng.randint(1, kv_hi),
                     kv_hi=kv_hi, step=rng.choice([1, 5, 9, 17, 33]))
            c["N"] = _pages_wanted(c) + _log(rng, 1, 2000)
            if c["N"] * c["S"] * kv_heads * D * c["L"] <= 1e9 and c["N"] <= 65536:
                return c
        else:
            c = dict(base, B=_log(rng, 1, 256), S=rng.choice([16, 32, 64]), L=rng.randint(1, 4), N=_log(rng, 64, 65536),
                     held=rng.uniform(0.1, 0.9))
            if c["N"] * c["S"] * kv_heads * D * c["L"] <= 1e9:
                return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _lengths(case):
    """(new tokens, cached tokens with them) of the requests; some requests are shorter than their new rows only if the ranges say so."""
    q = _spread(case["B"], case["q_lo"], case["q_hi"])
    random.Random(1).shuffle(q)
    return list(zip(q, [max(a, b) for a, b in zip(q, _spread(case["B"], case["kv_lo"], case["kv_hi"]))]))


def _steps(case):
    """Lengths now and next of an update's requests (width 1: mixed; beams: every one grows)."""
    B, width, S, step = case["B"], case["width"], case["S"], case["step"]
    now = _spread(B // width, case["kv_lo"], case["kv_hi"])
    r = random.Random(2)
    r.shuffle(now)
    now = [n for n in now for _ in range(width)]
    if width > 1:
        return now, [n + step for n in now]
    nxt = []
    for i, n in enumerate(now):
        u = r.random()
        if u < 0.06:
            nxt.append(0)
        elif u < 0.12:
            now[i] = 0
            nxt.append(n)
        elif u < 0.5:
            nxt.append(max(1, n - r.randint(0, step)))
        else:
            nxt.append(n + step)
    return now, nxt


def _ceil(a, b):
    return -(-a // b)


def _pages_wanted(case):
    """Pages that hold an update's lengths before and after, however the parents fall."""
    now, nxt = _steps(case)
    S, width = case["S"], case["width"]
    if width == 1:
        return sum(_ceil(max(a, b), S) for a, b in zip(now, nxt))
    return sum(_ceil(a, S) + width * (1 + _ceil(b, S) - a // S + 1) + width * (a // S) // 2 for a, b in list(zip(now, nxt))[::width])


# ---- inputs -------------------------------------------------------------------------------------

def _dev():
    return torch.device("cuda")


def _randn(shape, dtype, g):
    x = torch.empty(shape, dtype=dtype, device=_dev())
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.shape, dtype=dtype if dtype is torch.float32 else torch.bfloat16, device=_dev(), generator=g))
    return x


def _pool(case, L, N, g):
    """One layer stack of pages as [L, N, S, kv_heads, D], in memory with tokens (nhd) or heads (hnd) outermost in a page."""
    S, Hk, D, dt = case["S"], case["kv_heads"], case["D"], DTYPES[case["dtype"]]
    if case["layout"] == "nhd":
        return tuple(_randn((L, N, S, Hk, D), dt, g) for _ in range(2))
    return tuple(_randn((L, N, Hk, S, D), dt, g).transpose(2, 3) for _ in range(2))


def _int(a):
    return torch.tensor(a, dtype=torch.int32, device=_dev())


def _tables(lens, S, M, N, rng):
    """Block tables of requests that hold pages of their own, scattered over the pool."""
    order = rng.permutation(N).tolist()
    table = np.full((len(lens), M), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(lens):
        p = _ceil(n, S)
        table[b, :p] = order[at:at + p]
        at += p
    return table


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed) & (2**62 - 1))
    rng = np.random.RandomState(int(seed) % (2**32))
    s = dict(case=case, status=torch.zeros(4, dtype=torch.int32, device=_dev()))
    {"attend": _prepare_rows, "append": _prepare_rows, "update": _prepare_update, "compact": _prepare_compact}[case["op"]](case, s, g, rng)
    if own:
        _prepare_calls(case, s)
    return s


def _prepare_rows(case, s, g, rng):
    S, Hk, D, dt = case["S"], case["kv_heads"], case["D"], DTYPES[case["dtype"]]
    pairs = [_lengths(case)[i] for i in rng.permutation(case["B"])]
    q_len, kv_len = [p[0] for p in pairs], [p[1] for p in pairs]
    M = max(_ceil(n, S) for n in kv_len)
    N = sum(_ceil(n, S) for n in kv_len) + 3
    s["k"], s["v"] = _pool(case, 1, N, g)
    s["table"] = _int(_tables(kv_len, S, M, N, rng))
    s["kv_len"] = _int(kv_len)
    s["q_start"] = _int(np.concatenate([[0], np.cumsum(q_len)]))
    s["max_q"] = max(q_len)
    T = sum(q_len)
    if case["op"] == "attend":
        s["q"] = _randn((T, case["heads"], D), dt, g)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, case["heads"]), dtype=torch.float32, device=_dev())
    else:
        s["k_new"], s["v_new"] = _randn((T, Hk, D), dt, g), _randn((T, Hk, D), dt, g)


def _prepare_update(case, s, g, rng):
    B, S, N, width = case["B"], case["S"], case["N"], case["width"]
    now, nxt = _steps(case)
    order = rng.permutation(B // width)
    now = [now[i * width + j] for i in order for j in range(width)]
    nxt = [nxt[i * width + j] for i in order for j in range(width)]
    M = max(max(_ceil(a, S), _ceil(b, S)) for a, b in zip(now, nxt)) + 1
    if width == 1:
        table, parent = _tables(now, S, M, N, rng), None
    else:
        # the beams of a search share its first pages (their common past) and own the rest
        pages, at, table, parent = rng.permutation(N), 0, np.full((B, M), -1, dtype=np.int32), np.empty(B, dtype=np.int32)
        for b0 in range(0, B, width):
            n = _ceil(now[b0], S)
            split = n - min(n, int(rng.randint(0, 3)))
            table[b0:b0 + width, :split] = pages[at:at + split]
            at += split
            for b in range(b0, b0 + width):
                table[b, split:n] = pages[at:at + n - split]
                at += n - split
                parent[b] = b0 + rng.randint(0, width)
        parent = _int(parent)
    s["k"], s["v"] = _pool(case, case["L"], N, g)
    s["ref"] = _int(np.bincount(table[table >= 0], minlength=N))
    s["table"], s["kv_len"], s["new_len"], s["parent"] = _int(table), _int(now), _int(nxt), parent
    s["table_out"], s["len_out"], s["ref_out"] = (torch.empty_like(s[k]) for k in ("table", "kv_len", "ref"))


def _prepare_compact(case, s, g, rng):
    N, B = case["N"], case["B"]
    held = max(1, int(round(case["held"] * N)))
    pages = rng.permutation(N)[:held]
    M = _ceil(held, B)
    table = np.full((B, M), -1, dtype=np.int32)
    for b in range(B):
        row = pages[b::B]
        table[b, :len(row)] = row
    s["k"], s["v"] = _pool(case, case["L"], N, g)
    s["table"], s["ref"] = _int(table), _int(np.bincount(table[table >= 0], minlength=N))
    s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
    s["page_map"], s["n_used"] = torch.empty_like(s["ref"]), torch.empty(1, dtype=torch.int32, device=_dev())


def _prepare_calls(case, s):
    """What a program keeps beside its buffers: the pool's description and a workspace."""
    from speculative_decoding_draft_block_gb300 import kv_cache
    s["pool"] = kv_cache.KvPool(s["k"], s["v"])
    B, N = s["table"].shape[0], s["k"].shape[1]
    n = {"attend": lambda: kv_cache.ds_paged_attention_workspace_bytes(s["pool"], case["heads"]),
         "append": lambda: 0,
         "update": lambda: kv_cache.ds_cache_update_workspace_bytes(B, N),
         "compact": lambda: kv_cache.ds_cache_compact_workspace_bytes(N)}[case["op"]]()
    s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device=_dev())


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if not own:
        return {"attend": _plain_attend, "append": _plain_append, "update": _plain_update, "compact": _plain_compact}[c["op"]](c, s)
    from speculative_decoding_draft_block_gb300 import kv_cache as kv
    if c["op"] == "attend":
        kv.check(kv.ds_paged_attention(s["pool"], 0, s["q"], s["q_start"], s["max_q"], s["table"], s["kv_len"], s["out"],
                                       s["workspace"], s["status"], lse=s["lse"], causal=c["causal"], window=c["window"]))
        return s["out"], s["lse"]
    if c["op"] == "append":
        kv.check(kv.ds_cache_append(s["pool"], 0, s["k_new"], s["v_new"], s["q_start"], s["table"], s["kv_len"], s["status"]))
        return s["k"], s["v"]
    if c["op"] == "update":
        kv.check(kv.ds_cache_update(s["pool"], s["table"], s["kv_len"], s["ref"], s["new_len"], s["table_out"], s["len_out"],
                                    s["ref_out"], s["workspace"], s["status"], parent=s["parent"]))
        return s["table_out"], s["len_out"], s["ref_out"], s["k"], s["v"]
    kv.check(kv.ds_cache_compact(s["pool"], s["table"], s["ref"], s["table_out"], s["ref_out"], s["page_map"], s["n_used"],
                                 s["workspace"], s["status"]))
    return s["table_out"], s["ref_out"], s["page_map"], s["n_used"], s["k"], s["v"]


def _rows(q_start, T):
    """Request and place within it of each of T ragged rows."""
    t = torch.arange(T, device=q_start.device)
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    return b, t - q_start[b]


def _plain_attend(c, s):
    q, table, kv_len, q_start, D = s["q"], s["table"], s["kv_len"].long(), s["q_start"].long(), c["D"]
    T, H, _ = q.shape
    B, Hk, Lq = c["B"], c["kv_heads"], s["max_q"]
    G = H // Hk
    n = q_start[1:] - q_start[:-1]
    i = torch.arange(Lq, device=q.device)
    at = (q_start[:-1, None] + i).clamp(max=T - 1)
    qp = q[at].float().view(B, Lq, Hk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hk, G * Lq, D)
    pages = table.clamp(min=0).long()
    k = s["k"][0][pages].float().reshape(B, -1, Hk, D).transpose(1, 2)
    v = s["v"][0][pages].float().reshape(B, -1, Hk, D).transpose(1, 2)
    J = k.shape[2]
    j = torch.arange(J, device=q.device)
    pos = (kv_len - n)[:, None] + i                                       # [B, Lq]
    seen = j < (torch.minimum(pos + 1, kv_len[:, None]) if c["causal"] else kv_len[:, None].expand(B, Lq))[..., None]
    if c["window"]:
        seen = seen & (j > pos[..., None] - c["window"])
    scores = torch.matmul(qp, k.transpose(2, 3)).view(B, Hk, G, Lq, J) * (1.0 / math.sqrt(D))
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    m = scores.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    e = torch.exp(scores - m0)
    l = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, Hk, G * Lq, J), v).view(B, Hk, G, Lq, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.log(l) + m0
    b, r = _rows(q_start, T)
    return o[b, :, :, r].reshape(T, H, D).to(q.dtype), lse[b, :, :, r].reshape(T, H)


def _plain_append(c, s):
    S, q_start, kv_len = c["S"], s["q_start"].long(), s["kv_len"].long()
    b, i = _rows(q_start, s["k_new"].shape[0])
    pos = kv_len[b] - (q_start[1:] - q_start[:-1])[b] + i
    page = s["table"][b, pos // S].long()
    s["k"][0][page, pos % S] = s["k_new"]
    s["v"][0][page, pos % S] = s["v_new"]
    return s["k"], s["v"]


def _plain_update(c, s):
    S, table, ref = c["S"], s["table"].long(), s["ref"].long()
    kv_len, new_len = s["kv_len"].long(), s["new_len"].long()
    (B, M), N = table.shape, ref.shape[0]
    dev = table.device
    req, j = torch.arange(B, device=dev), torch.arange(M, device=dev)
    parent = req if s["parent"] is None else s["parent"].long()
    keep = torch.where(parent >= 0, torch.minimum(kv_len[parent.clamp(min=0)], new_len), 0)
    kept, want = (keep + S - 1) // S, (new_len + S - 1) // S
    past = table[parent.clamp(min=0)]
    before, after = j < ((kv_len + S - 1) // S)[:, None], j < kept[:, None]
    count = ref.clone()
    count.index_add_(0, table.clamp(min=0).flatten(), -before.flatten().long())
    count.index_add_(0, past.clamp(min=0).flatten(), after.flatten().long())
    writes = (keep % S != 0) & (new_len > keep)
    last = past.gather(1, (kept - 1).clamp(min=0)[:, None])[:, 0].clamp(min=0)
    writers = torch.zeros_like(ref).index_add_(0, last, writes.long())
    first = torch.full_like(ref, B).scatter_reduce(0, last, torch.where(writes, req, B), "amin")
    copies = writes & (count[last] > 1) & ~((count[last] == writers[last]) & (first[last] == req))
    free = count == 0
    rank = torch.cumsum(free, 0) - 1
    free_list = torch.full((N + 1,), -1, dtype=torch.long, device=dev).scatter_(0, torch.where(free, rank, N), torch.arange(N, device=dev))
    shared = kept - copies.long()
    new = want - shared
    ends = torch.cumsum(new, 0)
    place = (ends - new)[:, None] + j - shared[:, None]
    table_out = torch.where(j < shared[:, None], past, torch.where(j < want[:, None], free_list[place.clamp(0, N)], -1))
    count.index_add_(0, last, -copies.long())
    ref_out = torch.where(free & (rank < ends[-1]), torch.ones_like(count), count)
    who = copies.nonzero()[:, 0]
    src, dst, tokens = last[who], table_out[who, shared[who]], (keep % S)[who]
    written = (torch.arange(S, device=dev) < tokens[:, None])[None, :, :, None, None]
    for x in (s["k"], s["v"]):
        x[:, dst] = torch.where(written, x[:, src], x[:, dst])
    return table_out.int(), new_len.int(), ref_out.int(), s["k"], s["v"]


def _plain_compact(c, s):
    table, ref = s["table"].long(), s["ref"]
    N = ref.shape[0]
    held, page = ref > 0, torch.arange(N, device=ref.device)
    used = held.sum()
    src, dst = (held & (page >= used)).nonzero()[:, 0], (~held & (page < used)).nonzero()[:, 0]
    page_map = torch.where(held, page, -1)
    page_map[src] = dst
    ref_out = ref.clone()
    ref_out[dst] = ref[src]
    ref_out[src] = 0
    table_out = torch.where(table >= 0, page_map[table.clamp(min=0)], -1)
    for x in (s["k"], s["v"]):
        x[:, dst] = x[:, src]
    return table_out.int(), ref_out, page_map.int(), used.int().view(1), s["k"], s["v"]


# ---- what a pass cannot do without ------------------------------------------------------------

def _visible(case, n, kv):
    """(visible pairs of a request's rows, cached tokens that some row sees)."""
    W, pairs, lowest = case["window"], 0, kv
    for i in range(n):
        p = kv - n + i
        hi = min(kv, p + 1) if case["causal"] else kv
        lo = max(0, p - W + 1) if W else 0
        pairs += max(0, hi - lo)
        lowest = min(lowest, lo)
    return pairs, kv - lowest


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    row = case["kv_heads"] * case["D"] * e
    if case["op"] == "attend":
        seen = [(n, kv) + _visible(case, n, kv) for n, kv in _lengths(case)]
        T = sum(x[0] for x in seen)
        tokens = sum(x[3] for x in seen)
        return {"bytes": 2 * tokens * row + T * case["heads"] * (2 * case["D"] * e + 4) + 4 * sum(_ceil(x[3], case["S"]) for x in seen),
                "flops": 4.0 * case["D"] * case["heads"] * sum(x[2] for x in seen)}
    if case["op"] == "append":
        T = sum(n for n, _ in _lengths(case))
        return {"bytes": 4 * T * row, "flops": 0}
    if case["op"] == "update":
        now, nxt = _steps(case)
        S, table = case["S"], 4 * sum(_ceil(a, case["S"]) + _ceil(b, case["S"]) for a, b in zip(*_steps(case)))
        copied = 0 if case["width"] == 1 else sum(a % S for a in now[::case["width"]]) * (case["width"] - 1) // 2
        return {"bytes": table + 8 * case["N"] + 4 * copied * row * case["L"], "flops": 0}
    N, held = case["N"], case["held"]
    return {"bytes": 4 * N * held * (1 - held) * case["S"] * row * case["L"] + 8 * N * held + 12 * N, "flops": 0}


# ---- the operators by their definitions, in 64 bits ---------------------------------------------

def exact(case, seed):
    s = _bare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "update": _exact_update, "compact": _exact_compact}[case["op"]](case, s)


def _bare(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _exact_attend(case, s):
    table, kv_len, q_start = s["table"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist()
    T, H, D = s["q"].shape
    S, G = case["S"], H // case["kv_heads"]
    out = torch.zeros((T, H, D), dtype=torch.float64, device=_dev())
    lse = torch.full((T, H), float("-inf"), dtype=torch.float64, device=_dev())
    if work(case)["flops"] > 6e12:
        return None
    for b in range(case["B"]):
        a, z, n = q_start[b], q_start[b + 1], kv_len[b]
        pages = torch.tensor(table[b][:_ceil(n, S)], device=_dev())
        first = n - (z - a)
        row, col = torch.arange(first, n, device=_dev())[:, None], torch.arange(n, device=_dev())[None]
        hidden = torch.zeros((z - a, n), dtype=torch.bool, device=_dev())
        if case["causal"]:
            hidden |= col > row
        if case["window"]:
            hidden |= row - col >= case["window"]
        for h in range(H):
            key = s["k"][0, pages, :, h // G].reshape(-1, D)[:n].double()
            val = s["v"][0, pages, :, h // G].reshape(-1, D)[:n].double()
            x = (s["q"][a:z, h].double() @ key.T) / math.sqrt(D)
            x[hidden] = float("-inf")
            lse[a:z, h] = torch.logsumexp(x, 1)
            out[a:z, h] = torch.nan_to_num(torch.exp(x - lse[a:z, h, None])) @ val
    return out, lse


def _exact_append(case, s):
    table, kv_len, q_start, S = s["table"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist(), case["S"]
    for b in range(case["B"]):
        p, t = kv_len[b] - (q_start[b + 1] - q_start[b]), q_start[b]
        while p < kv_len[b]:
            m = min(S - p % S, kv_len[b] - p)
            for pool, new in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
                pool[0, table[b][p // S], p % S:p % S + m] = new[t:t + m]
            p, t = p + m, t + m
    return s["k"], s["v"]


def _exact_update(case, s):
    S, N = case["S"], case["N"]
    table, now, nxt, ref = (s[k].tolist() for k in ("table", "kv_len", "new_len", "ref"))
    parent = list(range(len(now))) if s["parent"] is None else s["parent"].tolist()
    M = len(table[0])
    for b, n in enumerate(now):
        for p in table[b][:_ceil(n, S)]:
            ref[p] -= 1
    rows, keep = [], []
    for b, p in enumerate(parent):
        k = min(now[p], nxt[b]) if p >= 0 else 0
        keep.append(k)
        rows.append(table[p][:_ceil(k, S)] if k else [])
        for page in rows[-1]:
            ref[page] += 1
    writers = {}
    for b, k in enumerate(keep):
        if k % S and nxt[b] > k:
            writers.setdefault(rows[b][-1], []).append(b)
    copied = {}
    for page, who in writers.items():
        if ref[page] > 1:
            for b in who[1:] if ref[page] == len(who) else who:
                copied[b] = page
    free = iter([p for p in range(N) if ref[p] == 0])
    for b in range(len(rows)):
        if b in copied:
            rows[b] = rows[b][:-1]
        while len(rows[b]) < _ceil(nxt[b], S):
            page = next(free)
            if b in copied and len(rows[b]) == _ceil(keep[b], S) - 1:
                ref[copied[b]] -= 1
                for x in (s["k"], s["v"]):
                    x[:, page, :keep[b] % S] = x[:, copied[b], :keep[b] % S]
            ref[page] = 1
            rows[b] = rows[b] + [page]
    return _int([r + [-1] * (M - len(r)) for r in rows]), _int(nxt), _int(ref), s["k"], s["v"]


def _exact_compact(case, s):
    table, ref = s["table"].tolist(), s["ref"].tolist()
    held = [p for p, n in enumerate(ref) if n > 0]
    U = len(held)
    to = {p: p for p in held}
    holes = [p for p in range(U) if ref[p] == 0]
    for p, hole in zip([p for p in held if p >= U], holes):
        to[p] = hole
        ref[hole], ref[p] = ref[p], 0
        for x in (s["k"], s["v"]):
            x[:, hole] = x[:, p]
    rows = [[to[p] if p >= 0 else -1 for p in row] for row in table]
    return _int(rows), _int(ref), _int([to.get(p, -1) for p in range(case["N"])]), _int([U]), s["k"], s["v"]
