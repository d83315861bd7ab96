"""The quantised cache's and the draft trees' operators as they are measured: cases, inputs, plain forms and exact values.

Five operators beside the paged cache's first ones (speculative_decoding_draft_block_gb300.kv_cache):
  append   new keys and values into a cache of 8-bit floats (e4m3), each row of a head with a power of two as its scale
  attend   attention of ragged new tokens over such a cache
  tree     attention of a tree of drafted tokens over a cache: a node sees the cached context and its own ancestors
  keep     an accepted path of a tree: its rows move together behind the context, in all layers
  masks    a tree's masks and depths from its nodes' parents

`run` computes them in elementary torch operations (32-bit arithmetic, rounded once at the end), or, with `own`, calls the
library. What is held in 8 bits comes back as e4m3 and e8m0 tensors, that is, as numbers. Sizes follow the framework's
workloads (B = 1, 4, 32, 128 requests; K = 4, 8, 16 drafted tokens; hidden sizes 256, 2560 and 4096 as heads of 64 or 128),
with generic context lengths and tree sizes.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
LARGEST = 448.0           # of e4m3
LOWEST_SCALE = -100       # exponent of the smallest scale that a row is given
MAX_SCORES = 2.2e9        # padded query rows x keys of the plain form's score matrix
MAX_KEYS = 1.1e9          # padded key elements of its gathered cache


# ---- cases ------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's new tokens into the quantised cache: the latency of a small call
        dict(name="append_token_B64", op="append", dtype="e4m3", B=64, kv_heads=8, D=128, S=16, layout="nhd",
             q_lo=1, q_hi=1, kv_lo=100, kv_hi=3000),
        # prompts into the quantised cache, heads outside the page's tokens
        dict(name="append_prompt_B16", op="append", dtype="e4m3", B=16, kv_heads=8, D=128, S=64, layout="hnd",
             q_lo=1023, q_hi=8192, kv_lo=1023, kv_hi=8192),
        # one request answering alone over a quantised cache
        dict(name="attend_token_B1", op="attend", dtype="e4m3", B=1, heads=32, kv_heads=8, D=128, S=16, layout="nhd",
             q_lo=1, q_hi=1, kv_lo=517, kv_hi=517, window=0),
        # a decode step of 128 requests: the cache is read once, at half of bfloat16's bytes
        dict(name="attend_token_B128", op="attend", dtype="e4m3", B=128, heads=32, kv_heads=8, D=128, S=64, layout="nhd",
             q_lo=1, q_hi=1, kv_lo=300, kv_hi=8000, window=0),
        # prompts in chunks against what is cached of them: bound by the tensor cores
        dict(name="attend_prompt_B2", op="attend", dtype="e4m3", B=2, heads=32, kv_heads=8, D=128, S=256, layout="nhd",
             q_lo=1777, q_hi=2048, kv_lo=9001, kv_hi=16384, window=0),
        # a tree of 25 drafted tokens of one request
        dict(name="tree_B1", op="tree", dtype="bf16", B=1, heads=32, kv_heads=8, D=128, S=16, layout="nhd",
             q_lo=25, q_hi=25, kv_lo=742, kv_hi=742, window=0),
        # the verify pass of 128 requests with trees of 8 to 60 tokens over the quantised cache
        dict(name="tree_verify_B128", op="tree", dtype="e4m3", B=128, heads=32, kv_heads=8, D=128, S=32, layout="nhd",
             q_lo=8, q_hi=60, kv_lo=500, kv_hi=6000, window=0),
        # a small float32 model's trees, sliding window
        dict(name="tree_f32_B4", op="tree", dtype="f32", B=4, heads=4, kv_heads=2, D=64, S=16, layout="hnd",
             q_lo=9, q_hi=13, kv_lo=33, kv_hi=1000, window=300),
        # accepted paths of a few requests of a small model
        dict(name="keep_B4", op="keep", dtype="bf16", B=4, kv_heads=2, D=64, S=16, layout="hnd", L=2,
             q_lo=9, q_hi=13, kv_lo=33, kv_hi=300),
        # accepted paths of 128 requests in all layers of a quantised cache
        dict(name="keep_B128", op="keep", dtype="e4m3", B=128, kv_heads=8, D=128, S=16, layout="nhd", L=32,
             q_lo=8, q_hi=60, kv_lo=80, kv_hi=400),
        # one tree's masks
        dict(name="masks_B1", op="masks", B=1, q_lo=25, q_hi=25, window=0),
        # a batch's masks, large trees
        dict(name="masks_B256", op="masks", B=256, q_lo=40, q_hi=256, window=0),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "tree", "tree", "keep", "masks"])
    D, kv_heads, S = rng.choice([64, 128]), rng.choice([1, 2, 4, 8]), rng.choice([16, 32, 64, 128, 256])
    base = dict(op=op, dtype="e4m3", D=D, kv_heads=kv_heads, S=S, layout=rng.choice(["nhd", "hnd"]))
    while True:
        if op == "append":
            q_hi = _log(rng, 1, 8192)
            kv_hi = q_hi + _log(rng, 1, 4096) - 1
            c = dict(base, B=_log(rng, 1, 512), q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=rng.randint(1, kv_hi), kv_hi=kv_hi)
            if work(c)["bytes"] <= 3.5e8 and c["B"] * (kv_hi + 256) * kv_heads * D <= 1e9:
                return c
        elif op in ("attend", "tree"):
            group = rng.choice([1, 2, 4, 5, 7, 8, 16])
            form = rng.choice(["token", "verify", "prompt"]) if op == "attend" else rng.choice(["small", "small", "large"])
            kv_hi = _log(rng, 17, 16384)
            kv_lo = _log(rng, 1, kv_hi)
            q_hi = {"token": lambda: 1, "verify": lambda: rng.randint(2, 33), "prompt": lambda: _log(rng, 64, 2048),
                    "small": lambda: _log(rng, 1, 64), "large": lambda: _log(rng, 65, 512)}[form]()
            dtype = "e4m3" if op == "attend" else rng.choice(["e4m3", "e4m3", "bf16", "f32"])
            c = dict(base, dtype=dtype, B=_log(rng, 1, 8 if form == "prompt" else 32 if form == "large" else 256),
                     heads=kv_heads * group, q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=kv_lo, kv_hi=kv_hi,
                     window=0 if rng.random() < 0.75 else _log(rng, 32, 2048))
            cap = 8.0e11 if dtype != "f32" else 4e10
            if (work(c)["flops"] <= cap and c["B"] * c["heads"] * q_hi * max(kv_hi, q_hi) <= MAX_SCORES
                    and c["B"] * (max(kv_hi, q_hi) + S) * kv_heads * D <= MAX_KEYS):
                return c
        elif op == "keep":
            q_hi, kv_hi = _log(rng, 1, 256), _log(rng, 17, 2000)
            c = dict(base, dtype=rng.choice(["e4m3", "e4m3", "bf16", "f32"]), S=rng.choice([16, 32, 64]), L=rng.randint(1, 32),
                     B=_log(rng, 1, 256), q_lo=rng.randint(1, q_hi), q_hi=q_hi, kv_lo=rng.randint(1, kv_hi), kv_hi=kv_hi)
            if sum(n + 64 for _, n in _lengths(c)) * kv_heads * D * c["L"] * _size(c) <= 2.5e9 and work(c)["bytes"] <= 2e8:
                return c
        else:
            q_hi = _log(rng, 16, 512)
            c = dict(op=op, B=_log(rng, 1, 256), q_lo=rng.randint(1, q_hi), q_hi=q_hi,
                     window=0 if rng.random() < 0.75 else rng.randint(1, 16))
            if work(c)["bytes"] <= 4e6 and c["B"] * q_hi ** 2 <= 2e7:
                return c


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _lengths(case):
    """(new tokens, cached tokens with them) of the requests."""
    q = _spread(case["B"], case["q_lo"], case["q_hi"])
    random.Random(1).shuffle(q)
    if "kv_lo" not in case:
        return [(n, n) for n in q]
    return list(zip(q, [max(a, b) for a, b in zip(q, _spread(case["B"], case["kv_lo"], case["kv_hi"]))]))


def _ceil(a, b):
    return -(-a // b)


def _size(case):
    return {"e4m3": 1, "bf16": 2, "f32": 4}[case["dtype"]]


def _path_length(n):
    """Tokens of a tree of n that are accepted: a few, as many as the tree is deep in practice."""
    return max(1, min(n // 2, int(2 * math.log2(n + 1))))


# ---- inputs -------------------------------------------------------------------------------------

def _dev():
    return torch.device("cuda")


def _int(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device=_dev())


def _randn(shape, dtype, g):
    x = torch.empty(shape, dtype=dtype, device=_dev())
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 28):
        part = flat[at:at + (1 << 28)]
        part.copy_(torch.randn(part.shape, dtype=dtype, device=_dev(), generator=g))
    return x


def _quantise(x):
    """Codes and scales' exponents of rows [..., D]: the smallest power of two 2^e, e >= LOWEST_SCALE, with |x| <= 448 * 2^e."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))          # amax = m * 2^e, 1/2 <= m < 1; 448 = 7/8 * 2^9
    e = (e - 9 + (m > 0.875)).clamp(min=LOWEST_SCALE)
    e = torch.where(m == 0, LOWEST_SCALE, e)
    return torch.ldexp(x, -e.unsqueeze(-1)).to(torch.float8_e4m3fn), e


def _pool(case, L, N, g):
    """Layers of pages, K and V as [L, N, S, kv_heads, D], in memory with tokens (nhd) or heads (hnd) outermost in a page; scales
    of a quantised one as [L, N, 2, kv_heads, S] (K, V), a byte each: the exponent and 127. Its heads differ in size."""
    S, Hk, D = case["S"], case["kv_heads"], case["D"]
    nhd = case["layout"] == "nhd"
    shape = (L, N, S, Hk, D) if nhd else (L, N, Hk, S, D)
    if case["dtype"] != "e4m3":
        k, v = (_randn(shape, DTYPES[case["dtype"]], g) for _ in range(2))
        return (k, v, None) if nhd else (k.transpose(2, 3), v.transpose(2, 3), None)
    scales = torch.empty((L, N, 2, Hk, S), dtype=torch.uint8, device=_dev())
    kv = []
    size = torch.exp2(torch.linspace(-3, 4, Hk, device=_dev()))
    step = max(1, (1 << 27) // (S * Hk * D))
    for i in range(2):
        codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=_dev())
        for layer in range(L):
            for at in range(0, N, step):
                x = torch.randn((min(step, N - at),) + shape[2:], dtype=torch.bfloat16, device=_dev(), generator=g)
                # heads of all sizes (K of one, V of the other end), scores that stay those of unit rows through q
                f = (size if i == 0 else size.flip(0)).view((1, 1, Hk, 1) if nhd else (1, Hk, 1, 1))
                c, e = _quantise(x * f.to(torch.bfloat16))
                codes.view(torch.uint8)[layer, at:at + step] = c.view(torch.uint8)
                scales[layer, at:at + step, i] = ((e.transpose(1, 2) if nhd else e) + 127).to(torch.uint8)
        kv.append(codes if nhd else codes.transpose(2, 3))
    return kv[0], kv[1], scales


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


def _tree(n, rng):
    """Parents of a tree of n nodes, each before its children (-1: the context): wide at first, a few levels deep."""
    i = np.arange(n)
    return (np.minimum(i, (i + 1) * rng.uniform(0.1, 1.0, n) ** 1.5).astype(np.int64) - 1).astype(np.int32)


def _ancestors(parent):
    """Whether node i descends from node j or is it, and the nodes' depths."""
    n = len(parent)
    seen, depth = np.zeros((n, n), dtype=bool), np.zeros(n, dtype=np.int32)
    for i, p in enumerate(parent):
        if p >= 0:
            seen[i] = seen[p]
            depth[i] = depth[p] + 1
        seen[i, i] = True
    return seen, depth


def _words(seen, W):
    """Rows of truth values as W 32-bit words, the lowest bit first."""
    bits = np.zeros((seen.shape[0], 32 * W), dtype=bool)
    bits[:, :seen.shape[1]] = seen
    return np.packbits(bits, axis=1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def prepare(case, seed):
    g = torch.Generator(device=_dev()).manual_seed(int(seed) & (2**62 - 1))
    rng = np.random.RandomState(int(seed) % (2**32))
    s = dict(case=case, status=torch.zeros(4, dtype=torch.int32, device=_dev()))
    pairs = [_lengths(case)[i] for i in rng.permutation(case["B"])]
    q_len, kv_len = [p[0] for p in pairs], [p[1] for p in pairs]
    T = sum(q_len)
    s["q_start"] = _int(np.concatenate([[0], np.cumsum(q_len)]))
    s["max_q"] = max(q_len)
    W = _ceil(s["max_q"], 32)
    if case["op"] in ("tree", "masks"):
        s["parents"] = [_tree(n, rng) for n in q_len]
        s["parent"] = _int(np.concatenate(s["parents"]))
    if case["op"] == "masks":
        s["mask"] = torch.empty((T, W), dtype=torch.int32, device=_dev())
        s["depth"] = torch.empty(T, dtype=torch.int32, device=_dev())
        return s
    S, Hk, D = case["S"], case["kv_heads"], case["D"]
    M = max(_ceil(n, S) for n in kv_len)
    N = sum(_ceil(n, S) for n in kv_len) + 3
    s["k"], s["v"], s["scales"] = _pool(case, case.get("L", 1), N, g)
    s["table"], s["kv_len"] = _int(_tables(kv_len, S, M, N, rng)), _int(kv_len)
    rows = DTYPES["bf16" if case["dtype"] == "e4m3" else case["dtype"]]
    if case["op"] in ("attend", "tree"):
        s["q"] = _randn((T, case["heads"], D), rows, g)
        if case["dtype"] == "e4m3":
            s["q"] *= torch.exp2(-torch.linspace(-3, 4, Hk, device=_dev())).repeat_interleave(case["heads"] // Hk)[:, None].to(rows)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((T, case["heads"]), dtype=torch.float32, device=_dev())
    if case["op"] == "tree":
        trees = [_ancestors(p) for p in s["parents"]]
        near = [a & (d[:, None] - d[None] < case["window"]) if case["window"] else a for a, d in trees]
        s["mask"] = torch.as_tensor(np.concatenate([_words(a, W) for a in near]), device=_dev())
        s["depth"] = _int(np.concatenate([d for _, d in trees]))
    elif case["op"] == "append":
        s["k_new"], s["v_new"] = (_randn((T, Hk, D), rows, g) * torch.exp2(torch.linspace(-3, 4, Hk, device=_dev()))[:, None].to(rows) for _ in range(2))
    elif case["op"] == "keep":
        # the first nodes of a path stand where they are to go, the others behind the whole path
        most = max(_path_length(n) for n in q_len)
        path = np.full((case["B"], most), -1, dtype=np.int32)
        for b, n in enumerate(q_len):
            m = _path_length(n)
            stay = min(m, int(rng.randint(0, 3)))
            path[b, :m] = np.concatenate([np.arange(stay), np.sort(m + rng.permutation(n - m)[:m - stay])]) if n - m >= m - stay else np.arange(m)
        s["path"], s["new_len"] = _int(path), torch.empty(case["B"], dtype=torch.int32, device=_dev())
    if own:
        _prepare_calls(case, s)
    return s


def _prepare_calls(case, s):
    """What a program keeps beside its buffers: the pool's description and a workspace."""
    from speculative_decoding_draft_block_gb300 import kv_cache
    s["pool"] = kv_cache.KvPool(s["k"], s["v"], s["scales"])
    n = kv_cache.ds_paged_attention_workspace_bytes(s["pool"], case["heads"]) if "heads" in case else 0
    s["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device=_dev())
    s["held"] = _held(s)   # the same buffers as numbers, for what comes back: no part of a call


# ---- one pass ------------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _own(c, s)
    return {"append": _plain_append, "attend": _plain_attend, "tree": _plain_attend, "keep": _plain_keep, "masks": _plain_masks}[c["op"]](c, s)


def _own(c, s):
    from speculative_decoding_draft_block_gb300 import kv_cache as kv
    if c["op"] == "append":
        kv.check(kv.ds_cache_append(s["pool"], 0, s["k_new"], s["v_new"], s["q_start"], s["table"], s["kv_len"], s["status"]))
        return s["held"]
    if c["op"] == "attend":
        kv.check(kv.ds_paged_attention(s["pool"], 0, s["q"], s["q_start"], s["max_q"], s["table"], s["kv_len"], s["out"],
                                       s["workspace"], s["status"], lse=s["lse"], window=c["window"]))
        return s["out"], s["lse"]
    if c["op"] == "tree":
        kv.check(kv.ds_paged_attention(s["pool"], 0, s["q"], s["q_start"], s["max_q"], s["table"], s["kv_len"], s["out"],
                                       s["workspace"], s["status"], lse=s["lse"], window=c["window"], mask=s["mask"], depth=s["depth"]))
        return s["out"], s["lse"]
    if c["op"] == "keep":
        kv.check(kv.ds_cache_keep(s["pool"], s["path"], s["q_start"], s["table"], s["kv_len"], s["new_len"], s["status"]))
        return s["new_len"], s["held"]
    kv.check(kv.ds_tree_masks(s["parent"], s["q_start"], s["max_q"], s["mask"], s["depth"], s["status"], window=c["window"]))
    return s["mask"], s["depth"]


def _held(s):
    """The pool: 8-bit floats and scales are numbers, not whole ones."""
    return (s["k"], s["v"]) if s["scales"] is None else (s["k"], s["v"], s["scales"].view(torch.float8_e8m0fnu))


def _rows(q_start, T):
    """Request and place within it of each of T ragged rows."""
    t = torch.arange(T, device=q_start.device)
    b = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    return b, t - q_start[b]


def _bits(x):
    """A tensor that torch can index whatever its type."""
    return x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x


def _plain_append(c, s):
    S, q_start, kv_len = c["S"], s["q_start"].long(), s["kv_len"].long()
    b, i = _rows(q_start, s["k_new"].shape[0])
    pos = kv_len[b] - (q_start[1:] - q_start[:-1])[b] + i
    page = s["table"][b, pos // S].long()
    for n, (pool, new) in enumerate(((s["k"], s["k_new"]), (s["v"], s["v_new"]))):
        codes, e = _quantise(new)
        _bits(pool)[0][page, pos % S] = codes.view(torch.uint8)
        s["scales"][0, :, n].transpose(1, 2)[page, pos % S] = (e + 127).to(torch.uint8)
    return _held(s)


def _gather(s, x, n, pages):
    """A request's keys or values as floats, [B, J, kv_heads, D]."""
    y = _bits(x)[0][pages]
    if s["scales"] is not None:
        e = s["scales"][0, :, n][pages].transpose(2, 3).int() - 127
        y = torch.ldexp(y.view(torch.float8_e4m3fn).float(), e.unsqueeze(-1))
    return y.float().flatten(1, 2)


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
    k, v = (_gather(s, x, m, pages).transpose(1, 2) for m, x in enumerate((s["k"], s["v"])))
    J = k.shape[2]
    j = torch.arange(J, device=q.device)
    first = (kv_len - n)[:, None]                                          # tokens cached before the new ones
    if c["op"] == "tree":
        bit = (j - first)[:, None].clamp(0, 32 * s["mask"].shape[1] - 1)                       # [B, 1, J]
        word = s["mask"][at].gather(2, (bit >> 5).expand(B, Lq, J))
        seen = (j < first)[:, None] | ((word >> (bit & 31).int()) & 1).bool() & (j < kv_len[:, None])[:, None]
        pos = first + s["depth"][at]
        near = (j >= first)[:, None] | (j > pos[..., None] - c["window"])  # (the mask has the window among the nodes)
    else:
        pos = first + i
        seen = j < torch.minimum(pos + 1, kv_len[:, None])[..., None]
        near = j > pos[..., None] - c["window"]
    if c["window"]:
        seen = seen & near
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


def _plain_keep(c, s):
    S, path, kv_len, q_start = c["S"], s["path"].long(), s["kv_len"].long(), s["q_start"].long()
    first = kv_len - (q_start[1:] - q_start[:-1])
    i = torch.arange(path.shape[1], device=path.device)
    there = path >= 0
    src = first[:, None] + path.clamp(min=0)
    dst = torch.where(there, first[:, None] + i, src)
    pages = s["table"].long()
    sp, dp = pages.gather(1, src // S)[there], pages.gather(1, dst // S)[there]
    si, di = (src % S)[there], (dst % S)[there]
    for x in (s["k"], s["v"]):
        y = _bits(x)
        y[:, dp, di] = y[:, sp, si]
    if s["scales"] is not None:
        s["scales"][:, dp, :, :, di] = s["scales"][:, sp, :, :, si]
    return (first + there.sum(1)).int(), _held(s)


def _plain_masks(c, s):
    q_start, Lq = s["q_start"].long(), s["max_q"]
    T, W = s["mask"].shape
    n = q_start[1:] - q_start[:-1]
    i = torch.arange(Lq, device=n.device)
    parent = torch.where(i < n[:, None], s["parent"][(q_start[:-1, None] + i).clamp(max=T - 1)].long(), -1)
    # ancestors and the node itself: (1 + A)^(2^k), A a node's step to its parent
    r = ((parent[..., None] == i) | torch.eye(Lq, dtype=torch.bool, device=n.device)).float()
    for _ in range(max(1, (Lq - 1).bit_length())):
        r = torch.matmul(r, r).clamp(max=1)
    depth = r.sum(2).long() - 1
    seen = r > 0
    if c["window"]:
        seen &= depth[:, :, None] - depth[:, None] < c["window"]
    bits = torch.zeros((c["B"], Lq, 32 * W), dtype=torch.long, device=n.device)
    bits[..., :Lq] = seen
    words = (bits.view(c["B"], Lq, W, 32) << torch.arange(32, device=n.device)).sum(-1).to(torch.int32)
    b, k = _rows(q_start, T)
    return words[b, k], depth[b, k].int()


# ---- what a pass cannot do without ------------------------------------------------------------

def _visible(case, n, kv):
    """(visible pairs of a request's rows, cached tokens that some row sees); a tree counts log2 of its size as ancestors."""
    W, first = case["window"], kv - n
    if case["op"] == "tree":
        deep = math.log2(n + 1)
        return n * (min(first, W or first) + deep), n + min(first, W or first)
    pairs, lowest = 0, kv
    for p in range(first, kv):
        lo = max(0, p - W + 1) if W else 0
        pairs += p + 1 - lo
        lowest = min(lowest, lo)
    return pairs, kv - lowest


def work(case):
    if case["op"] == "masks":
        T, W = sum(n for n, _ in _lengths(case)), _ceil(case["q_hi"], 32)
        return {"bytes": T * (8 + 4 * W), "flops": 0}
    quantised = case["dtype"] == "e4m3"
    e = _size(case)
    row = case["kv_heads"] * (case["D"] * e + quantised)              # of K or V of a token, its scales counted
    wide = 2 if quantised else e
    lengths = _lengths(case)
    T = sum(n for n, _ in lengths)
    if case["op"] == "append":
        return {"bytes": 2 * T * (row + case["kv_heads"] * case["D"] * wide), "flops": 0}
    if case["op"] == "keep":
        return {"bytes": 4 * sum(_path_length(n) for n, _ in lengths) * row * case["L"], "flops": 0}
    seen = [_visible(case, n, kv) for n, kv in lengths]
    tokens = sum(x[1] for x in seen)
    masks = 4 * T * (1 + _ceil(case["q_hi"], 32)) if case["op"] == "tree" else 0
    return {"bytes": 2 * tokens * row + T * case["heads"] * (2 * case["D"] * wide + 4) + 4 * sum(_ceil(x[1], case["S"]) for x in seen) + masks,
            "flops": 4.0 * case["D"] * case["heads"] * sum(x[0] for x in seen)}


# ---- the operators by their definitions, in 64 bits ---------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _exact_append, "attend": _exact_attend, "tree": _exact_attend, "keep": _exact_keep, "masks": _exact_masks}[case["op"]](case, s)


def _exact_codes(x):
    """Nearest e4m3 values (ties to the even one) of x over its scale, and the scales' exponents, by arithmetic alone."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(top, float(LOWEST_SCALE))
    for _ in range(400):
        low = top > LARGEST * torch.exp2(e)
        if not bool(low.any()):
            break
        e += low
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # 3 bits behind the leading one
    return torch.round(y / step) * step, e.squeeze(-1)


def _exact_append(case, s):
    table, kv_len, q_start, S = s["table"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist(), case["S"]
    k, v, scales = s["k"].float(), s["v"].float(), torch.exp2(s["scales"].double() - 127)
    for n, (pool, new) in enumerate(((k, s["k_new"]), (v, s["v_new"]))):
        for b in range(case["B"]):
            p, t = kv_len[b] - (q_start[b + 1] - q_start[b]), q_start[b]
            y, e = _exact_codes(new[t:q_start[b + 1]])
            t = 0
            while p < kv_len[b]:
                m = min(S - p % S, kv_len[b] - p)
                pool[0, table[b][p // S], p % S:p % S + m] = y[t:t + m].float()
                scales[0, table[b][p // S], n, :, p % S:p % S + m] = torch.exp2(e[t:t + m]).T
                p, t = p + m, t + m
    return k, v, scales


def _exact_attend(case, s):
    if work(case)["flops"] > 6e12:
        return None
    table, kv_len, q_start = s["table"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist()
    T, H, D = s["q"].shape
    S, G = case["S"], H // case["kv_heads"]
    out = torch.zeros((T, H, D), dtype=torch.float64, device=_dev())
    lse = torch.full((T, H), float("-inf"), dtype=torch.float64, device=_dev())
    for b in range(case["B"]):
        a, z, n = q_start[b], q_start[b + 1], kv_len[b]
        pages = torch.tensor(table[b][:_ceil(n, S)], device=_dev())
        first = n - (z - a)
        col = torch.arange(n, device=_dev())[None]
        hidden = torch.zeros((z - a, n), dtype=torch.bool, device=_dev())
        if case["op"] == "tree":
            line = []                                    # each node's ancestors, from itself up
            for i, p in enumerate(s["parents"][b].tolist()):
                line.append([i] + (line[p] if p >= 0 else []))
            row = torch.tensor([first + len(x) - 1 for x in line], device=_dev())[:, None]
            own_nodes = np.ones((z - a, z - a), dtype=bool)
            for i, x in enumerate(line):
                own_nodes[i, x[:case["window"]] if case["window"] else x] = False
            hidden[:, first:] = torch.as_tensor(own_nodes, device=_dev())
            if case["window"]:
                hidden[:, :first] |= row - col[:, :first] >= case["window"]
        else:
            row = torch.arange(first, n, device=_dev())[:, None]
            hidden |= col > row
            if case["window"]:
                hidden |= row - col >= case["window"]
        for h in range(case["kv_heads"]):
            key, val = (x[0].view(torch.uint8)[pages][:, :, h].view(x.dtype) if x.dtype is torch.float8_e4m3fn else x[0, pages, :, h]
                        for x in (s["k"], s["v"]))
            key, val = key.double(), val.double()
            if s["scales"] is not None:
                two = torch.exp2(s["scales"][0, pages, :, h].double() - 127)[..., None]
                key, val = key * two[:, 0], val * two[:, 1]
            key, val = key.reshape(-1, D)[:n], val.reshape(-1, D)[:n]
            x = s["q"][a:z, h * G:h * G + G].double().transpose(0, 1) @ key.T / math.sqrt(D)
            x.masked_fill_(hidden, float("-inf"))
            y = torch.logsumexp(x, 2)
            lse[a:z, h * G:h * G + G] = y.T
            out[a:z, h * G:h * G + G] = (torch.nan_to_num(torch.exp(x - y[..., None])) @ val).transpose(0, 1)
    return out, lse


def _exact_keep(case, s):
    table, kv_len, q_start, S = s["table"].tolist(), s["kv_len"].tolist(), s["q_start"].tolist(), case["S"]
    lens = []
    pools = [_bits(s["k"]), _bits(s["v"])]
    for b, path in enumerate(s["path"].tolist()):
        first = kv_len[b] - (q_start[b + 1] - q_start[b])
        path = [p for p in path if p >= 0]
        for i, p in enumerate(path):
            (dp, di), (sp, si) = divmod(first + i, S), divmod(first + p, S)
            dp, sp = table[b][dp], table[b][sp]
            if i != p:
                for x in pools:
                    x[:, dp, di] = x[:, sp, si]
                if s["scales"] is not None:
                    s["scales"][:, dp, :, :, di] = s["scales"][:, sp, :, :, si]
        lens.append(first + len(path))
    held = (s["k"], s["v"]) if s["scales"] is None else (s["k"], s["v"], torch.exp2(s["scales"].double() - 127))
    return _int(lens), held


def _exact_masks(case, s):
    T, W = s["mask"].shape
    mask, depth, at = np.zeros((T, W), dtype=np.int64), np.zeros(T, dtype=np.int64), 0
    for parent in s["parents"]:
        for i in range(len(parent)):
            j, line = i, []
            while j >= 0:
                line.append(j)
                j = int(parent[j])
            depth[at + i] = len(line) - 1
            for j in line[:case["window"]] if case["window"] else line:
                mask[at + i, j // 32] |= 1 << (j % 32)
        at += len(parent)
    return _int(mask.astype(np.uint32).view(np.int32)), _int(depth)
