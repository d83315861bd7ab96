"""Quantised pools, trees of drafted tokens and accepted paths on the GPU against plain 64-bit forms (_tree_ref.py)."""
import os

import numpy as np
import pytest

import _tree_ref as ref
from _kv_ref import ceil_div

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_draft_block_gb300 import _lib, build, kv_cache
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    return kv_cache


DT = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BOUNDS = 6


def _i32(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _status():
    return torch.zeros(4, dtype=torch.int32, device="cuda")


def _pool_values(k, v, scales):
    """A layer's K and V in float64, [N, S, Hk, D]; NaN where a scale says so."""
    if scales is None:
        return _host(k), _host(v)
    s = scales.cpu().numpy().astype(np.int64).transpose(1, 0, 3, 2)      # [2, N, S, Hk]
    return tuple(ref.restored(_host(x), y) for x, y in zip((k, v), s))


def _empty_pool(dtype, L, N, S, Hk, D, layout):
    """Pools whose every place is NaN (quantised: by its scale, with codes of all kinds)."""
    shape = (L, N, S, Hk, D) if layout == "nhd" else (L, N, Hk, S, D)
    scales = None
    if dtype == "e4m3":
        g = torch.Generator(device="cuda").manual_seed(3)
        k, v = (torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g).view(DT[dtype]) for _ in range(2))
        scales = torch.full((L, N, 2, Hk, S), 255, dtype=torch.uint8, device="cuda")
    else:
        k, v = (torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
    return (k, v, scales) if layout == "nhd" else (k.transpose(2, 3), v.transpose(2, 3), scales)


def _bytes(x):
    return x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x


class Batch:
    """Ragged rows over a pool whose unseen places hold NaN; pages scattered; the table -1 where nothing is seen."""

    def __init__(self, dtype, D, S, Hk, G, lens, layout="nhd", window=0, causal=True, seed=0, spread=1.0, trees=None,
                 extra=5, W=None, depth=True, masks=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.RandomState(seed)
        self.dtype, self.D, self.S, self.causal, self.window = dtype, D, S, causal, window
        n_q, n_kv = [a for a, _ in lens], [b for _, b in lens]
        self.max_q = max(1, max(n_q))
        self.mask = self.depth = None
        T = sum(n_q)
        if trees is None:
            self.seen = [ref.causal_seen(n, m, causal, window) for n, m in lens]
        else:
            pairs = [ref.ancestors(t(rng, n), window) for t, n in zip(trees, n_q)]
            if masks is not None:
                pairs = [(masks(rng, n), d) for (_, d), n in zip(pairs, n_q)]
            W = W or ceil_div(self.max_q, 32)
            if not depth:
                pairs = [(a, None) for a, _ in pairs]
            self.mask = torch.as_tensor(np.concatenate([ref.words(a, W) for a, _ in pairs] + [np.zeros((0, W), np.int32)]), device="cuda")
            self.depth = _i32(np.concatenate([d for _, d in pairs])) if depth else None
            self.seen = [ref.tree_seen(a, d, n, m, window) for (a, d), (n, m) in zip(pairs, lens)]
        M = max(1, max(ceil_div(n, S) for n in n_kv))
        N = sum(ceil_div(n, S) for n in n_kv) + extra
        self.k, self.v, self.scales = _empty_pool(dtype, 1, N, S, Hk, D, layout)
        order = rng.permutation(N)
        table, at = np.full((len(lens), M), -1, dtype=np.int32), 0
        for b, n in enumerate(n_kv):
            rows = self.seen[b].any(0)
            # pages between the first and the last that some row may see need an entry
            lo = int(rows.argmax()) if rows.any() else n
            if trees is not None and n:
                first = n - n_q[b]
                lo = max(0, first - window + 1) if window else 0
            for p in range(ceil_div(n, S)):
                if n_q[b] == 0 or (p + 1) * S <= lo:
                    continue
                page = table[b, p] = order[at]
                at += 1
                a, z = max(lo, p * S) - p * S, min(n, (p + 1) * S) - p * S
                there = torch.as_tensor(np.nonzero(rows[p * S + a:p * S + z])[0] + a, device="cuda")
                if not len(there):
                    continue
                for i, x in enumerate((self.k, self.v)):
                    y = (torch.randn((len(there), Hk, D), device="cuda", generator=g) * spread).to(torch.bfloat16 if dtype == "e4m3" else DT[dtype])
                    if dtype == "e4m3":
                        c, e = ref.quantise(_host(y))
                        _bytes(x)[0, int(page), there] = torch.as_tensor(c, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
                        self.scales[0, int(page), i].T[there] = torch.as_tensor(e + 127, device="cuda").to(torch.uint8)
                    else:
                        x[0, int(page), there] = y
        H, rows_dt = G * Hk, torch.bfloat16 if dtype == "e4m3" else DT[dtype]
        self.q = torch.randn((T, H, D), device="cuda", generator=g).to(rows_dt) * spread
        self.out = torch.full((T, H, D), 7.0, dtype=rows_dt, device="cuda")
        self.lse = torch.full((T, H), 7.0, device="cuda")
        self.table, self.kv_len = _i32(table), _i32(n_kv)
        self.q_start = _i32(np.concatenate([[0], np.cumsum(n_q)]))
        self.status = _status()

    def call(self, kv, stream=None, scale=None):
        pool = kv.KvPool(self.k, self.v, self.scales)
        if not hasattr(self, "ws"):
            self.ws = torch.full((kv.ds_paged_attention_workspace_bytes(pool, self.q.shape[1]),), 0xA5, dtype=torch.uint8,
                                 device="cuda")
        return kv.ds_paged_attention(pool, 0, self.q, self.q_start, self.max_q, self.table, self.kv_len, self.out, self.ws,
                                     self.status, lse=self.lse, causal=self.causal, window=self.window, scale=scale,
                                     stream=stream, mask=self.mask, depth=self.depth)

    def compare(self, scale=None):
        assert int(self.status[0]) == 0
        k, v = _pool_values(self.k[0], self.v[0], None if self.scales is None else self.scales[0])
        want, lse, tol, lse_tol = ref.attend(_host(self.q), k, v, self.table.cpu().numpy(), self.kv_len.cpu().numpy(),
                                             self.q_start.cpu().numpy(), lambda b: self.seen[b],
                                             scale or ref.default_scale(self.D), self.dtype != "f32")
        got = _host(self.out)
        assert np.isfinite(got).all()
        off = np.abs(got - want) - tol
        assert off.size == 0 or off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape), np.abs(got - want).max())
        got = _host(self.lse)
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(got), empty)
        off = np.abs(got[~empty] - lse[~empty]) - lse_tol[~empty]
        assert off.size == 0 or off.max() <= 0, off.max()

    def verify(self, kv, **kw):
        assert self.call(kv, **kw) == 0
        self.compare(kw.get("scale"))


# ---- append to a quantised pool ----------------------------------------------------------

def _append_case(kv, D, S, Hk, layout, k_new, v_new, lens, seed=0):
    """Appends rows to a fresh pool: the pool as it was and is, and the rows' places."""
    rng = np.random.RandomState(seed)
    n_q, n_kv = [a for a, _ in lens], [b for _, b in lens]
    N = sum(ceil_div(n, S) for n in n_kv) + 3
    k, v, scales = _empty_pool("e4m3", 2, N, S, Hk, D, layout)
    before = [x.clone() for x in (_bytes(k), _bytes(v), scales)]
    order, at, places = rng.permutation(N), 0, []
    table = np.full((len(lens), max(1, max(ceil_div(n, S) for n in n_kv))), -1, dtype=np.int32)
    for b, (nq, n) in enumerate(lens):
        for p in range(ceil_div(n, S)):
            table[b, p] = order[at]
            at += 1
        places += [(table[b, p // S], p % S) if p >= 0 else None for p in range(n - nq, n)]
    st = _status()
    pool = kv.KvPool(k, v, scales)
    kv.check(kv.ds_cache_append(pool, 1, k_new, v_new, _i32(np.concatenate([[0], np.cumsum(n_q)])), _i32(table), _i32(n_kv), st))
    assert int(st[0]) == 0
    return (k, v, scales), before, places


def _check_append(pool, before, places, k_new, v_new):
    k, v, scales = pool
    want = [x.clone() for x in before]
    for i, new in enumerate((k_new, v_new)):
        codes, e = ref.quantise(_host(new))
        codes = torch.as_tensor(codes, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        e = torch.as_tensor(e + 127, device="cuda").to(torch.uint8)
        for t, where in enumerate(places):
            if where is not None:
                want[i][1, where[0], where[1]] = codes[t]
                want[2][1, where[0], i, :, where[1]] = e[t]
    # (codes as numbers: -0 is 0)
    for x, y in zip((k, v), want):
        assert torch.equal(x.float().nan_to_num(1e9), y.view(torch.float8_e4m3fn).float().nan_to_num(1e9))
    assert torch.equal(scales, want[2])


LENS = [(1, 1), (0, 37), (3, 3), (5, 2), (17, 200), (1, 129), (40, 300)]


@pytest.mark.parametrize("D,S,Hk,layout", [(128, 16, 8, "nhd"), (64, 32, 2, "hnd"), (16, 64, 1, "nhd"), (48, 16, 3, "hnd"),
                                           (256, 256, 2, "nhd"), (80, 128, 5, "nhd"), (112, 16, 1, "hnd")])
def test_append_quantises(kv, D, S, Hk, layout):
    T = sum(a for a, _ in LENS)
    g = torch.Generator(device="cuda").manual_seed(D + S)
    size = torch.exp2(torch.randint(-40, 40, (T, Hk, 1), device="cuda", generator=g).float())
    k_new, v_new = ((torch.randn((T, Hk, D), device="cuda", generator=g) * size).to(torch.bfloat16) for _ in range(2))
    _check_append(*_append_case(kv, D, S, Hk, layout, k_new, v_new, LENS), k_new, v_new)


def test_append_quantises_values_at_the_borders(kv):
    """Zeros, subnormals, the largest bfloat16, maxima at and about 448 * 2^e, ties of e4m3, values that are not finite."""
    D, big = 64, 3.3895313892515355e38
    rows = []
    for top in (0.0, -0.0, 448.0, 450.0, 446.0, 447.0, 449.0, 2.0 ** -133, 2.0 ** -126, 448.0 * 2.0 ** -100, 450.0 * 2.0 ** -100,
                2.0 ** -92, 2.0 ** -110, big, -big, 57344.0, 57600.0, 65536.0, 1.0, 1.75, 1.7578125, 0.875):
        x = np.zeros(D)
        x[3] = top
        rows.append(x)
    ties = np.array([(1 + (2 * i + 1) / 16) * 2.0 ** e for e in (-6, -1, 0, 7) for i in range(8)] +
                    [(2 * i + 1) * 2.0 ** -10 for i in range(8)] + [2.0 ** -10, -2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -11])
    for s in (0, 5, -90, 100):
        x = np.zeros(D)
        x[:len(ties)] = ties * 2.0 ** s
        x[len(ties):2 * len(ties)] = -ties[:D - len(ties)] * 2.0 ** s
        x[-1] = 448.0 * 2.0 ** s
        rows.append(x)
    for what in (np.nan, np.inf, -np.inf):
        for at in (0, 17, D - 1):
            x = np.linspace(-2, 3, D)
            x[at] = what
            rows.append(x)
    k_new = torch.as_tensor(np.stack(rows), device="cuda").to(torch.bfloat16)[:, None].contiguous()
    v_new = k_new.flip(0).contiguous()
    n = len(rows)
    pool, before, places = _append_case(kv, D, 16, 1, "nhd", k_new, v_new, [(n, n + 5)])
    _check_append(pool, before, places, k_new, v_new)
    # no value is further off than half a step: 2^-4 of it, or half of the smallest code
    codes, e = ref.quantise(_host(k_new))
    fine = np.isfinite(_host(k_new)).all(-1)
    got = np.ldexp(codes, e[..., None])[fine]
    want = _host(k_new)[fine]
    assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, np.ldexp(1.0, e[fine] - 10)[..., None])).all()


def test_append_quantises_the_last_binade(kv):
    """Above 1.75 * 2^127 the scale is 247. Up to 247 * 2^120 a finite row restores to finite bfloat16 values; from 248 * 2^120 on
    (half a step below 256) the nearest code stands for 2^128, which bfloat16 does not hold."""
    D, tops = 64, [224, 225, 232, 239, 240, 247, 248, 255]
    x = torch.zeros((2 * len(tops), 1, D), dtype=torch.float64)
    for i, top in enumerate(tops + [-t for t in tops]):
        x[i, 0, :4] = torch.tensor([top, 1.0, -top / 2, 3.0], dtype=torch.float64) * 2.0 ** 120
    new = x.to("cuda").to(torch.bfloat16)
    assert torch.equal(new.cpu().double(), x)
    n = len(new)
    pool, before, places = _append_case(kv, D, 16, 1, "nhd", new, new, [(n, n)])
    _check_append(pool, before, places, new, new)
    k, _, scales = pool
    at = [torch.as_tensor([p[i] for p in places], device="cuda") for i in range(2)]
    byte = scales[1, at[0], 0, 0, at[1]].int()
    assert byte.tolist() == [246] + [247] * 7 + [246] + [247] * 7
    got = (k[1, at[0], at[1], 0].double() * torch.exp2(byte.double() - 127)[:, None]).to(torch.bfloat16)
    finite = torch.isfinite(got.float()).all(1).tolist()
    assert finite == [t <= 247 for t in tops] * 2
    off = (got.double() - new[:, 0].double()).abs().cpu()[torch.tensor(finite)]
    assert (off <= (2.0 ** -4 * x[:, 0].abs())[torch.tensor(finite)]).all()


def test_append_quantises_strided_rows(kv):
    """Keys and values as slices of one wide projection."""
    D, Hk, n = 64, 2, 50
    wide = torch.randn((n, 2 * Hk + 1, 2 * D), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    k_new, v_new = wide[:, :Hk, D:], wide[:, Hk + 1:, :D]
    _check_append(*_append_case(kv, D, 16, Hk, "nhd", k_new, v_new, [(30, 100), (20, 20)]), k_new, v_new)


@pytest.mark.parametrize("Hk,D", [(8, 128), (1, 64)])
def test_append_quantised_reports_a_bad_page_and_writes_the_rest(kv, Hk, D):
    S, n = 16, 50
    k, v, scales = _empty_pool("e4m3", 1, 4, S, Hk, D, "nhd")
    new = torch.randn((n, Hk, D), device="cuda").to(torch.bfloat16)
    table = _i32([[2, 4, 0, 1]])     # page 4 is none of four
    st = _status()
    before = _bytes(k).clone()
    assert kv.ds_cache_append(kv.KvPool(k, v, scales), 0, new, new, _i32([0, n]), table, _i32([n]), st) == 0
    assert int(st[0]) == BOUNDS
    codes, e = ref.quantise(_host(new))
    for p in (0, 2, 3):
        page, rows = int(table[0, p]), range(p * S, min(n, (p + 1) * S))
        assert np.array_equal(_host(k[0, page])[:len(rows)], codes[p * S:p * S + len(rows)])
        assert np.array_equal(scales[0, page, 0, :, :len(rows)].cpu().numpy().T, e[p * S:p * S + len(rows)] + 127)
    assert torch.equal(_bytes(k)[0, 1, 2:], before[0, 1, 2:])
    assert (scales[0, 1, :, :, 2:] == 255).all()


# ---- attention over a quantised pool --------------------------------------------------------

MIXED = [(1, 1), (1, 0), (0, 37), (3, 3), (5, 2), (17, 200), (1, 129), (2, 128), (4, 127), (9, 33), (33, 40)]


@pytest.mark.parametrize("D,S,Hk,G,layout", [(128, 16, 2, 4, "nhd"), (64, 32, 1, 1, "hnd"), (128, 64, 2, 5, "hnd"),
                                             (64, 128, 3, 8, "nhd"), (128, 256, 1, 16, "nhd"), (64, 16, 1, 7, "nhd"),
                                             (128, 32, 1, 128, "hnd"), (64, 64, 2, 33, "nhd")])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20)])
def test_quantised_attention_of_mixed_requests(kv, D, S, Hk, G, layout, causal, window):
    Batch("e4m3", D, S, Hk, G, MIXED, layout, window, causal, seed=D + S + G).verify(kv)


@pytest.mark.parametrize("D,lens", [(128, [(1, 5000)]), (64, [(1, 4097), (17, 3000), (5, 1)]), (128, [(300, 700)]),
                                    (64, [(130, 1500), (1, 900)]), (128, [(257, 257), (64, 64)])])
def test_quantised_attention_of_long_contexts(kv, D, lens):
    Batch("e4m3", D, 32, 2, 4, lens, seed=len(lens)).verify(kv)


@pytest.mark.parametrize("D,S,Hk,G,lens", [(128, 64, 8, 1, [(1, 1700 + 61 * i) for i in range(24)]),
                                           (64, 128, 8, 2, [(5, 900 + 77 * i) for i in range(20)]),
                                           (128, 32, 6, 8, [(17, 400 + 83 * i) for i in range(20)]),
                                           (64, 16, 8, 4, [(40 + 13 * i, 700 + 50 * i) for i in range(10)])])
def test_quantised_attention_of_many_long_contexts(kv, D, S, Hk, G, lens):
    Batch("e4m3", D, S, Hk, G, lens, seed=D + G).verify(kv)


@pytest.mark.parametrize("D,G,n_q", [(128, 1, 1), (64, 3, 1), (128, 8, 1), (64, 2, 4), (64, 16, 1), (128, 17, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
def test_quantised_attention_of_few_rows(kv, D, G, n_q, causal, window):
    Batch("e4m3", D, 16, 2, G, [(n_q, n) for n in (1, 15, 16, 17, 127, 128, 129, 300, 1000) if n >= n_q], window=window,
          causal=causal, seed=G).verify(kv)


@pytest.mark.parametrize("D,Hk,G,n_q", [(64, 4, 2, 1), (64, 8, 1, 5), (64, 6, 4, 2), (128, 4, 8, 1), (128, 6, 3, 5), (64, 4, 5, 3), (128, 3, 4, 2)])
@pytest.mark.parametrize("S,layout", [(16, "nhd"), (64, "hnd"), (128, "nhd"), (256, "hnd")])
def test_quantised_attention_of_few_rows_and_many_heads(kv, D, Hk, G, n_q, S, layout):
    """Groups of one, two and four KV heads; pages below, at and above a tile's keys of a head."""
    Batch("e4m3", D, S, Hk, G, [(n_q, n) for n in (5, 31, 33, 64, 255, 700)] + [(0, 9), (1, 0)], layout=layout, seed=D + Hk).verify(kv)


@pytest.mark.parametrize("D,Hk,G,n_q", [(128, 1, 4, 2), (128, 2, 4, 1), (64, 4, 1, 1), (64, 2, 3, 4), (64, 1, 2, 1)])
def test_quantised_attention_of_requests_that_see_nothing_between_others(kv, D, Hk, G, n_q):
    """Shares of several units, some of which have no keys and so no meeting of their warps; the same bits every time.
    (More requests than threads, too: their shares are found in two passes.)"""
    lens = [(n_q, 0 if i % 3 == 1 else n_q + (7 * i) % 50) for i in range(1000)]
    b = Batch("e4m3", D, 16, Hk, G, lens, seed=D + Hk)
    b.verify(kv)
    out, lse = b.out.clone(), b.lse.clone()
    for _ in range(10):
        b.out.fill_(5)
        assert b.call(kv) == 0
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse)


@pytest.mark.parametrize("G,n_q", [(2, 1), (4, 4), (4, 30), (8, 40)])
def test_quantised_attention_of_large_keys_and_values(kv, G, n_q):
    """Keys of 2^110 and values of 2^100 (scores far past any exponent: one key has all the weight); nothing overflows."""
    b = Batch("e4m3", 128, 16, 2, G, [(n_q, 200)], seed=G)
    far = b.scales != 255
    far[:, :, 1] = False
    b.scales[far] = 230
    values = b.scales != 255
    values[:, :, 0] = False
    b.scales[values] = 220
    b.q *= 2.0 ** -60
    assert b.call(kv) == 0
    assert torch.isfinite(b.out.float()).all() and torch.isfinite(b.lse).all() and int(b.status[0]) == 0
    k, v = _pool_values(b.k[0], b.v[0], b.scales[0])
    pages = b.table[0].tolist()
    kk, vv = (x[pages].reshape(-1, 2, 128)[:200] for x in (k, v))
    for t in (0, n_q - 1):
        for h in range(2 * G):
            s = kk[:, h // G] @ _host(b.q[t, h])
            s[200 - n_q + t + 1:] = -np.inf
            first, second = np.sort(s)[::-1][:2]
            if (first - second) * ref.default_scale(128) > 30:      # the others' weights: below 1e-12
                got, want = _host(b.out[t, h]), vv[s.argmax(), h // G]
                assert (np.abs(got - want) <= 2.0 ** -7 * np.abs(want) + 1e-12 * np.abs(vv).max()).all()


@pytest.mark.parametrize("G,n_q", [(2, 3), (4, 4), (4, 30), (8, 40)])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_quantised_attention_of_a_query_that_is_not_finite(kv, G, n_q, what):
    """It has no effect on other rows."""
    lens = [(n_q, 300), (2, 50)]
    b = Batch("e4m3", 128, 16, 2, G, lens, seed=G)
    b.verify(kv)
    good = b.out.clone()
    b.q[1, 1, 5] = what
    assert b.call(kv) == 0
    b.out[1, 1], good[1, 1] = 0, 0
    assert torch.equal(b.out, good) and int(b.status[0]) == 0


@pytest.mark.parametrize("G,n_q", [(1, 4), (4, 4), (4, 40), (2, 100)])
def test_quantised_attention_of_a_key_that_some_do_not_see(kv, G, n_q):
    """A key of NaN (its scale says so) makes the rows that see it NaN, and no others."""
    n = 260
    b = Batch("e4m3", 64, 16, 1, G, [(n_q, n)], seed=n_q)
    at = n - n_q // 2
    page, place = int(b.table[0, at // 16]), at % 16
    b.scales[0, page, 0, 0, place] = 255
    assert b.call(kv) == 0
    first = at - (n - n_q)
    assert torch.isnan(b.out[first:].float()).all() and torch.isfinite(b.out[:first].float()).all()
    keep, keep_lse = b.out[:first].clone(), b.lse[:first].clone()
    b.scales[0, page, 0, 0, place] = 120
    assert b.call(kv) == 0
    b.out[:first], b.lse[:first] = keep, keep_lse
    b.compare()


@pytest.mark.parametrize("spread", [1e-4, 3.0])
def test_quantised_attention_of_small_and_peaked_scores(kv, spread):
    Batch("e4m3", 128, 16, 2, 4, [(3, 500), (20, 300)], spread=spread, seed=5).verify(kv)


@pytest.mark.parametrize("scale_byte", [3, 26, 134, 135, 140, 246])
def test_quantised_attention_of_scales_at_the_borders(kv, scale_byte):
    """Values of rows whose scale needs two factors, or is below what append writes: out is their mean, in bfloat16's range.
    (Keys of zero: every weight is 1 / n; n * 2^-8 bounds the sums' and the last rounding, twice.)"""
    D, n = 64, 40
    b = Batch("e4m3", D, 16, 1, 2, [(1, n)], seed=1)
    two = 2.0 ** (scale_byte - 127)
    codes = torch.randint(0, 127, (1, b.k.shape[1], 16, 1, D), device="cuda", dtype=torch.uint8)
    # (below 2^120, so that their sum stays in float32's range)
    if scale_byte == 246:
        codes = codes.remainder(8 * 9)      # up to 2^2 * 2^119
    codes[codes == 127] = 0
    b.v = codes.view(torch.float8_e4m3fn)
    b.k = torch.zeros_like(codes).view(torch.float8_e4m3fn)
    b.scales[:, :, 0] = 127
    b.scales[:, :, 1] = scale_byte
    assert b.call(kv) == 0
    pages = b.table[0].long()
    want = (b.v[0].double()[pages].reshape(-1, D)[:n] * two).mean(0).cpu().numpy()
    got = b.out.double().cpu().numpy()[0]
    assert int(b.status[0]) == 0
    assert (np.abs(got - want) <= 4 * 2.0 ** -8 * np.abs(want) + 2.0 ** -133).all()


@pytest.mark.parametrize("D,G,n_q", [(64, 4, 8), (128, 4, 8), (64, 4, 40), (128, 4, 40), (128, 24, 1)])
@pytest.mark.parametrize("scale_byte", [3, 26, 27, 134, 135, 140, 246])
def test_quantised_attention_of_scales_at_the_borders_with_many_rows(kv, D, G, n_q, scale_byte):
    """As above with more than 16 rows a KV head, whose tiles are restored as bfloat16 in one product or two. Keys of zero: out is
    the mean of what a row sees, with weights of exactly 1, so its error is the sums' (each of n terms 2^-24 of the values' mean
    size, and the factor 1 / l twice that) and bfloat16's 2^-8 once; 2^-133 is the smallest bfloat16."""
    n = 50
    b = Batch("e4m3", D, 16, 1, G, [(n_q, n)], seed=1)
    # sums below float32's range: 50 values of up to 3.75 * 2^119 with the largest scale
    codes = torch.randint(0, 72 if scale_byte == 246 else 127, (1, b.k.shape[1], 16, 1, D), device="cuda", dtype=torch.uint8)
    codes += 128 * torch.randint(0, 2, codes.shape, device="cuda", dtype=torch.uint8)
    b.v = codes.view(torch.float8_e4m3fn)
    b.k = torch.zeros_like(codes).view(torch.float8_e4m3fn)
    b.scales[:, :, 0] = 127
    b.scales[:, :, 1] = scale_byte
    assert b.call(kv) == 0 and int(b.status[0]) == 0
    v = (b.v[0].double()[b.table[0].long()].reshape(-1, D)[:n] * 2.0 ** (scale_byte - 127)).cpu().numpy()
    got = b.out.double().cpu().numpy()
    for t in range(n_q):
        m = n - n_q + t + 1
        want, size = v[:m].mean(0), np.abs(v[:m]).mean(0)
        assert (np.abs(got[t] - want) <= 2.0 ** -8 * np.abs(want) + (m + 2) * 2.0 ** -24 * size * (1 + 2.0 ** -8) + 2.0 ** -133).all()


@pytest.mark.parametrize("D,G,n_q", [(128, 2, 1), (64, 2, 1), (128, 4, 4), (128, 4, 30), (64, 4, 30), (128, 8, 40)])
@pytest.mark.parametrize("far", [100, -60])
def test_quantised_attention_of_large_and_small_rows_with_ordinary_scores(kv, D, G, n_q, far):
    """Keys times 2^far, queries and values times 2^-far: the scores, and so all weights, are those of ordinary rows."""
    b = Batch("e4m3", D, 16, 2, G, [(n_q, 300), (1, 90)], seed=G)
    rows = b.scales != 255
    keys = rows.clone()
    keys[:, :, 1] = False
    b.scales[keys] += far % 256
    b.scales[rows & ~keys] -= far % 256
    b.q *= 2.0 ** -far
    b.verify(kv)


@pytest.mark.parametrize("D,G,n_q", [(128, 1, 4), (64, 4, 2), (128, 24, 1), (128, 4, 70), (64, 2, 90)])
@pytest.mark.parametrize("window", [0, 30])
def test_quantised_attention_of_rows_that_some_do_not_see(kv, D, G, n_q, window):
    """A NaN row (its scale says so) has no effect on rows that do not see it, and is NaN for those that do."""
    n = 300
    b = Batch("e4m3", D, 16, 1, G, [(n_q, n)], window=window, seed=D + n_q)
    at = n - 1                                     # seen by the last row only
    page, place = int(b.table[0, at // 16]), at % 16
    b.scales[0, page, 1, 0, place] = 255
    assert b.call(kv) == 0
    last = _host(b.out[-1:])
    assert np.isnan(last).all()
    if n_q > 1:                                     # the others, as if the value were zero
        b.scales[0, page, 1, 0, place] = 127
        keep = b.out[:-1].clone()
        b.seen = [s.copy() for s in b.seen]
        assert b.call(kv) == 0
        b.out[:-1] = keep
        b.compare()


# ---- trees ----------------------------------------------------------------------------------

def _mixed(rng, n):
    return ref.random_tree(rng, n, 0.15, 0.3)


def _chain(rng, n):
    return np.arange(n) - 1


def _star(rng, n):
    return np.full(n, -1)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("D,S,Hk,G,layout", [(128, 16, 2, 4, "nhd"), (64, 32, 1, 1, "hnd"), (128, 64, 2, 5, "hnd"),
                                             (64, 128, 2, 8, "nhd"), (128, 256, 1, 16, "nhd"), (64, 16, 1, 33, "nhd")])
@pytest.mark.parametrize("window", [0, 3, 25])
def test_tree_attention_of_mixed_requests(kv, dtype, D, S, Hk, G, layout, window):
    """Empty requests and contexts, trees about the tiles' and words' ends, more nodes than places."""
    lens = [(1, 1), (1, 0), (0, 37), (3, 3), (5, 2), (17, 200), (31, 159), (32, 128), (33, 161), (1, 129), (4, 130), (64, 70)]
    trees = [_mixed, _chain, _star] * 4
    Batch(dtype, D, S, Hk, G, lens, layout, window, seed=D + G, trees=trees).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("D,Hk,G,lens", [(128, 2, 4, [(25, 742)]), (64, 2, 1, [(300, 1100), (7, 50)]), (128, 1, 3, [(130, 130), (129, 900)]),
                                         (64, 2, 2, [(8, 3000), (3, 2100)]), (128, 8, 1, [(12 + i, 900 + 100 * i) for i in range(12)])])
def test_tree_attention_of_long_contexts(kv, dtype, D, Hk, G, lens):
    """Work split over the context and joined; trees over several tiles, of few rows and of many."""
    Batch(dtype, D, 32, Hk, G, lens, seed=D + len(lens), trees=[_mixed] * len(lens)).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("G,n", [(1, 4), (2, 7), (4, 4), (3, 40), (8, 70)])
def test_tree_attention_of_any_mask(kv, dtype, G, n):
    """Masks that are no tree's: rows that do not see themselves, that see later ones, or, without a context, nothing at all."""
    def masks(rng, m):
        a = rng.rand(m, m) < 0.4
        a[m // 2] = False
        return a
    lens = [(n, n), (n, n + 100), (n - 1, n - 1), (n, n + 127)]
    Batch(dtype, 64, 16, 2, G, lens, seed=n, trees=[_mixed] * 4, masks=masks).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("n,G", [(6, 2), (50, 4)])
def test_tree_attention_without_depths_and_wide_masks(kv, dtype, n, G):
    """Without depths a window counts from the first new token; words past the request's tokens may hold anything."""
    b = Batch(dtype, 128, 16, 1, G, [(n, 400), (2, 90)], window=60, seed=n, trees=[_mixed] * 2, depth=False, W=9)
    for t, m in zip(range(n + 2), [n] * n + [2] * 2):
        b.mask[t, ceil_div(m, 32):] = -1
        if m % 32:
            b.mask[t, m // 32] |= -(1 << (m % 32))
    b.verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("n,G", [(4, 2), (30, 4)])
def test_tree_attention_of_depths_past_a_window_longer_than_the_table(kv, dtype, n, G):
    """Depths are the caller's: a row far below its context sees little of it, or nothing."""
    b = Batch(dtype, 64, 16, 2, G, [(n, n + 300), (2, 90)], window=5000, seed=n, trees=[_mixed] * 2)
    far = [0, 4800, 4990, 6000][:n] + [0] * (n - 4) + [2**31 - 1, 4950]
    b.depth += _i32(far)
    depth, seen = b.depth.cpu().numpy().astype(np.int64), []
    for at, (m, total), s in zip((0, n), [(n, n + 300), (2, 90)], b.seen):
        first = total - m
        low = first + depth[at:at + m, None] - 5000 + 1
        seen.append(np.concatenate([np.arange(first) >= low, s[:, first:]], axis=1))
    b.seen = seen
    b.verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("D,G,n", [(128, 1, 9), (64, 2, 8), (64, 4, 40), (128, 4, 70)])
@pytest.mark.parametrize("window", [0, 50])
def test_tree_attention_of_nan_in_other_branches(kv, dtype, D, G, n, window):
    """Values that are not finite, of nodes that some rows see and others do not."""
    kw = dict(window=window, seed=n, trees=[_star])
    b = Batch(dtype, D, 16, 1, G, [(n, n + 200)], **kw)
    at = n + 200 - n // 2                 # a node that no other row sees
    page, place = int(b.table[0, at // 16]), at % 16
    if dtype == "e4m3":
        b.scales[0, page, :, 0, place] = 255
    else:
        b.k[0, page, place] = float("inf")
        b.v[0, page, place] = float("nan")
    assert b.call(kv) == 0
    row = n - n // 2
    got = b.out.clone()
    assert torch.isnan(got[row].float()).all()
    c = Batch(dtype, D, 16, 1, G, [(n, n + 200)], **kw)
    assert c.call(kv) == 0
    others = [i for i in range(n) if i != row]
    # the same sums in another order: each within the bound of the exact ones
    c.out[others], c.lse[others] = b.out[others], b.lse[others]
    c.compare()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
@pytest.mark.parametrize("D,G,n", [(128, 1, 4), (64, 1, 8), (64, 2, 8), (128, 2, 12), (64, 4, 30), (128, 4, 70)])
@pytest.mark.parametrize("past", [0, 40, 300])
def test_tree_attention_of_nan_beside_depths_past_the_window(kv, dtype, D, G, n, past):
    """Hand-made depths that put the window's beginning behind new tokens: these are seen by the masks alone, also where a
    value that is not finite stands beside them, of a token that only the last row sees."""
    def masks(rng, m):
        a = np.tril(rng.rand(m, m) < 0.5)
        a[:, 1] = np.arange(m) == m - 1
        a[np.arange(2, m), np.arange(2, m)] = True
        return a
    window = 5
    kw = dict(window=window, seed=n + past, trees=[_mixed], masks=masks)
    b = Batch(dtype, D, 16, 1, G, [(n, n + past)], **kw)
    # rows with the window's beginning in the context, among the new tokens, behind them
    b.depth = _i32([i % 3 * (window + i) if i % 4 else 10000 for i in range(n)])
    depth = b.depth.cpu().numpy().astype(np.int64)
    mask = b.seen[0][:, past:]
    b.seen = [ref.tree_seen(mask, depth, n, n + past, window)]
    page, place = int(b.table[0, (past + 1) // 16]), (past + 1) % 16
    if dtype == "e4m3":
        was = b.scales[0, page, :, 0, place].clone()
        b.scales[0, page, :, 0, place] = 255
    else:
        was = b.k[0, page, place].clone(), b.v[0, page, place].clone()
        b.k[0, page, place] = float("inf")
        b.v[0, page, place] = float("nan")
    assert b.call(kv) == 0
    assert torch.isnan(b.out[-1].float()).all()
    out, lse = b.out.clone(), b.lse.clone()
    if dtype == "e4m3":
        b.scales[0, page, :, 0, place] = was
    else:
        b.k[0, page, place], b.v[0, page, place] = was
    assert b.call(kv) == 0
    b.compare()
    b.out[:-1], b.lse[:-1] = out[:-1], lse[:-1]
    b.compare()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_a_chain_is_causal_attention(kv, dtype):
    lens = [(1, 40), (16, 200), (40, 41), (7, 700)]
    a = Batch(dtype, 128, 16, 2, 4, lens, seed=9, trees=[_chain] * 4)
    assert a.call(kv) == 0
    tree_out = a.out.clone()
    a.mask = a.depth = None
    assert a.call(kv) == 0
    a.compare()
    a.out.copy_(tree_out)
    a.compare()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_tree_attention_same_bits_twice_in_a_graph_and_on_another_stream(kv, dtype):
    b = Batch(dtype, 64, 16, 2, 4, [(12, 500), (33, 90), (1, 77)], seed=2, trees=[_mixed] * 3)
    b.verify(kv)
    out, lse = b.out.clone(), b.lse.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.out.fill_(5)
    s.wait_stream(torch.cuda.current_stream())
    assert b.call(kv, stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(b.out, out) and torch.equal(b.lse, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert b.call(kv) == 0
    for _ in range(3):
        b.out.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out, out) and torch.equal(b.lse, lse)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
def test_tree_attention_of_trees_that_fill_most_of_a_row_tile(kv, dtype, D):
    """Two row tiles a unit, of which some requests have one."""
    Batch(dtype, D, 16, 2, 4, [(60, 400), (20, 700), (14, 14), (9, 130)], seed=D, trees=[_mixed] * 4).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "e4m3"])
def test_two_calls_at_once(kv, dtype):
    """Calls with workspaces of their own on two streams, interleaved."""
    a = Batch(dtype, 128, 16, 8, 4, [(1, 900), (3, 2000)], seed=4, trees=[_mixed] * 2)
    b = Batch(dtype, 128, 16, 8, 4, [(40, 900), (13, 1500)], seed=5, trees=[_mixed] * 2)
    a.call(kv), b.call(kv)   # (workspaces)
    torch.cuda.synchronize()
    a.out.fill_(7), b.out.fill_(7)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, s in zip((a, b), streams):
            assert x.call(kv, stream=s.cuda_stream) == 0
    torch.cuda.synchronize()
    a.compare()
    b.compare()


# ---- malformed device data, strides, many requests ----------------------------------------------

@pytest.mark.parametrize("dtype,tree", [("e4m3", False), ("e4m3", True), ("bf16", True), ("f32", True), ("bf16", False), ("f32", False)])
@pytest.mark.parametrize("n", [4, 40])
def test_attention_reports_what_is_out_of_bounds(kv, dtype, tree, n):
    """The status says so, nothing faults, the other requests' rows stand."""
    def fresh():
        return Batch(dtype, 64, 16, 2, 2, [(2, 100), (n, n + 50), (1, 70)], seed=11, trees=[_mixed] * 3 if tree else None)

    good = fresh()
    good.verify(kv)
    for what in (good.k.shape[1], -1, 2**31 - 1, -2**31, "kv_len", "negative kv_len", "q_start", "max_q", "q_end"):
        x = fresh()
        if what == "kv_len":
            x.kv_len[1] = x.table.shape[1] * 16 + 1
        elif what == "negative kv_len":
            x.kv_len[1] = -5
        elif what == "q_start":
            x.q_start[2] = 1
        elif what == "max_q":
            x.max_q = n - 1
        elif what == "q_end":
            x.q_start[3] = 1000
        else:
            x.table[1, 2] = what
        assert x.call(kv) == 0
        assert int(x.status[0]) == BOUNDS, what
        # (the work is cut by the whole batch's, so the sums' order may be another: each within the bound of the exact ones)
        good.out[:2], good.lse[:2] = x.out[:2], x.lse[:2]
        good.compare()


@pytest.mark.parametrize("dtype,tree", [("e4m3", False), ("e4m3", True), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("D,G,n", [(128, 4, 3), (64, 2, 5), (128, 4, 40), (64, 4, 70)])
def test_attention_of_strided_rows(kv, dtype, tree, D, G, n):
    """q as a slice of a joint projection, out as one of a wider tensor, beside which nothing is written."""
    b = Batch(dtype, D, 16, 2, G, [(n, 90), (1, 300), (n + 1, n + 2)], seed=n, trees=[_mixed] * 3 if tree else None)
    T, H, _ = b.q.shape
    q = torch.full((T, H + 4, 2 * D), float("nan"), dtype=b.q.dtype, device="cuda")
    q[:, 1:H + 1, :D] = b.q
    out = torch.zeros((T, H + 1, 2 * D), dtype=b.q.dtype, device="cuda")
    b.q, b.out = q[:, 1:H + 1, :D], out[:, :H, D:]
    b.verify(kv, scale=0.07)
    assert (out[:, -1] == 0).all() and (out[:, :, :D] == 0).all()


def _joint(kind, L, N, S, Hk, D, dtype):
    """K and V as views of one tensor, and a tensor of truth values: what of it is theirs."""
    dt = torch.uint8 if dtype == "e4m3" else DT[dtype]
    if kind == "token":          # K and V of a token side by side
        shape, cut = (L, N, S, 2, Hk, D), lambda x: (x[:, :, :, 0], x[:, :, :, 1])
    elif kind == "head":         # of a head, with a gap behind them
        shape, cut = (L, N, S, Hk, 2 * D + 16), lambda x: (x[..., :D], x[..., D:2 * D])
    else:                        # layers inside pages, heads outside a page's tokens, more heads than are used
        shape, cut = (N, 2, L, Hk + 1, S, D), lambda x: tuple(x[:, i, :, :Hk].permute(1, 0, 3, 2, 4) for i in range(2))
    buf, mine = torch.full(shape, 7, dtype=dt, device="cuda"), torch.zeros(shape, dtype=torch.bool, device="cuda")
    for x in cut(mine):
        x.fill_(True)
    views = cut(buf)
    return buf, mine, [x.view(DT[dtype]) for x in views] if dtype == "e4m3" else list(views)


@pytest.mark.parametrize("dtype,kind", [("e4m3", "token"), ("e4m3", "head"), ("e4m3", "layers"), ("bf16", "head"), ("f32", "layers")])
@pytest.mark.parametrize("S,Hk,D,G,n", [(16, 2, 128, 4, 3), (64, 3, 64, 1, 2), (128, 1, 128, 5, 40), (16, 4, 64, 2, 60)])
def test_trees_and_paths_over_interleaved_pools(kv, dtype, kind, S, Hk, D, G, n):
    """K and V in one tensor with strides that are not dense: the same bits as over dense pools from append, attention with and
    without masks, keep, copy on write and compaction; what lies between the rows stays as it was."""
    L, B, N, M = 2, 3, 40, 8
    g = torch.Generator(device="cuda").manual_seed(S + D + n)
    rng = np.random.RandomState(n)
    rows_dt = torch.bfloat16 if dtype == "e4m3" else DT[dtype]
    buf, mine, joint = _joint(kind, L, N, S, Hk, D, dtype)

    def scales():
        return torch.full((L, N, 2, Hk, S), 255, dtype=torch.uint8, device="cuda") if dtype == "e4m3" else None

    pools = [kv.KvPool(*joint, scales()), kv.KvPool(*(torch.full_like(x, 7).contiguous() for x in joint), scales())]
    for x in pools[1].k, pools[1].v:
        _bytes(x).fill_(7)
    ws = torch.empty(max(kv.ds_cache_update_workspace_bytes(B, N), kv.ds_cache_compact_workspace_bytes(N),
                         kv.ds_paged_attention_workspace_bytes(pools[0], G * Hk)), dtype=torch.uint8, device="cuda")
    status = _status()
    held = torch.zeros(N, dtype=torch.int32, device="cuda")
    held[::3] = 1                                       # somebody else's, so that pages lie apart
    states = [[_i32(np.full((B, M), -1)), _i32([0] * B), held.clone()] for _ in pools]

    def both(call):
        """The call over each pool with its own state; the results have to be equal."""
        x, y = (call(pool, state) for pool, state in zip(pools, states))
        assert all(torch.equal(a, z) for a, z in zip(x, y))
        assert all(torch.equal(a, z) for a, z in zip(*states))
        for a, z in ((pools[0].k, pools[1].k), (pools[0].v, pools[1].v)) + (((pools[0].scales, pools[1].scales),) if dtype == "e4m3" else ()):
            assert torch.equal(_bytes(a), _bytes(z))
        assert (buf[~mine] == 7).all() and int(status[0]) == 0
        return x

    def update(new, parent=None):
        def call(pool, state):
            out = [torch.empty_like(x) for x in state]
            kv.check(kv.ds_cache_update(pool, *state, _i32(new), *out, ws, status, parent=None if parent is None else _i32(parent)))
            state[:] = out
            return []
        both(call)

    def rows(sizes, masked):
        start = _i32(np.concatenate([[0], np.cumsum(sizes)]))
        T = sum(sizes)
        mask = depth = None
        if masked:
            pairs = [ref.ancestors(ref.random_tree(rng, m)) for m in sizes]
            mask = torch.as_tensor(np.concatenate([ref.words(a, ceil_div(max(sizes), 32)) for a, _ in pairs]), device="cuda")
            depth = _i32(np.concatenate([d for _, d in pairs]))
        for layer in range(L):
            k, v = (torch.randn((T, Hk, D), device="cuda", generator=g).to(rows_dt) for _ in range(2))
            q = torch.randn((T, G * Hk, D), device="cuda", generator=g).to(rows_dt)

            def call(pool, state):
                out, lse = torch.empty_like(q), torch.empty((T, G * Hk), device="cuda")
                kv.check(kv.ds_cache_append(pool, layer, k, v, start, state[0], state[1], status))
                kv.check(kv.ds_paged_attention(pool, layer, q, start, max(sizes), state[0], state[1], out, ws, status, lse=lse, mask=mask,
                                               depth=depth))
                return out, lse
            assert torch.isfinite(both(call)[0].float()).all()
        return start

    lens = [3 * S + 7, n, 5]
    update(lens)
    rows(lens, False)
    update([lens[0], lens[0], 5], [0, 0, 2])             # request 1 becomes a copy of request 0
    new = [4, n, 1]
    update([lens[0] + 4, lens[0] + n, 6])                # both write into the shared last page
    start = rows(new, True)
    path = np.full((B, 3), -1)
    path[0], path[1, :2], path[2, 0] = [0, 2, 3], [0, n - 1], 0

    def keep(pool, state):
        new_len = torch.empty(B, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_keep(pool, _i32(path), start, state[0], state[1], new_len, status))
        return [new_len]

    new_len = both(keep)[0].tolist()
    assert new_len == [lens[0] + 3, lens[0] + 2, 6]
    update(new_len)

    def compact(pool, state):
        state[2] = state[2] - (torch.arange(N, device="cuda") % 3 == 0).int()
        out, page_map, used = (torch.empty_like(state[0]), torch.empty_like(state[2])), torch.empty_like(state[2]), _i32([0])
        kv.check(kv.ds_cache_compact(pool, state[0], state[2], *out, page_map, used, ws, status))
        state[0], state[2] = out
        return [used]

    assert int(both(compact)[0]) == int((states[0][2] > 0).sum())
    update([x + n for x in new_len])
    rows([n] * B, True)


@pytest.mark.parametrize("dtype,tree", [("e4m3", False), ("e4m3", True), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("G,most", [(2, 5), (4, 12)])
def test_attention_of_more_requests_than_threads(kv, dtype, tree, G, most):
    """Shares are found in two passes over the requests."""
    rng = np.random.RandomState(most)
    lens = [(int(a), int(a + c)) for a, c in zip(rng.randint(0, most + 1, 700), rng.randint(0, 60, 700))]
    Batch(dtype, 64, 16, 1, G, lens, seed=most, trees=[_mixed] * 700 if tree else None).verify(kv)


# ---- masks ----------------------------------------------------------------------------------

@pytest.mark.parametrize("window", [0, 1, 3])
@pytest.mark.parametrize("sizes", [[1], [25], [0, 1, 2, 31, 32, 33, 64, 65, 0], [300, 5], [1, 1, 1, 700]])
def test_tree_masks(kv, sizes, window):
    rng = np.random.RandomState(len(sizes))
    makers = [_mixed, _chain, _star]
    trees = [makers[i % 3](rng, n) for i, n in enumerate(sizes)]
    T, most = sum(sizes), max(sizes)
    for W in (ceil_div(most, 32), ceil_div(most, 32) + 2):
        mask = torch.full((T + 1, W), 77, dtype=torch.int32, device="cuda")
        depth = torch.full((T + 1,), 77, dtype=torch.int32, device="cuda")
        st = _status()
        parent = _i32(np.concatenate(trees))
        start = _i32(np.concatenate([[0], np.cumsum(sizes)]))
        kv.check(kv.ds_tree_masks(parent, start, most, mask[:T], depth[:T], st, window=window))
        pairs = [ref.ancestors(t, window) for t in trees]
        assert int(st[0]) == 0
        assert np.array_equal(mask[:T].cpu().numpy(), np.concatenate([ref.words(a, W) for a, _ in pairs]))
        assert np.array_equal(depth[:T].cpu().numpy(), np.concatenate([d for _, d in pairs]))
        assert (mask[T] == 77).all() and depth[T] == 77
        kv.check(kv.ds_tree_masks(parent, start, most, mask[:T], None, st, window=window))


def test_tree_masks_of_the_longest_chain(kv):
    n = 4096
    mask, depth, st = torch.empty((n, 128), dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"), _status()
    kv.check(kv.ds_tree_masks(_i32(np.arange(n) - 1), _i32([0, n]), n, mask, depth, st))
    assert int(st[0]) == 0 and torch.equal(depth, torch.arange(n, dtype=torch.int32, device="cuda"))
    i, w = torch.arange(n, device="cuda")[:, None], torch.arange(128, device="cuda")[None]
    bits = (i + 1 - 32 * w).clamp(0, 32)
    want = torch.where(bits == 32, -1, ((1 << bits.clamp(max=31)) - 1)).int()
    assert torch.equal(mask, want)


def test_tree_masks_reports_bad_parents_and_requests(kv):
    T = 8
    for parent, start, rows in (([-1, 1, 0, -2, 9, -1, 5, 6], [0, 5, 8], range(8)), ([-1] * 8, [0, 9], []), ([-1] * 8, [3, 2, 8], range(2, 8)),
                                ([-1] * 8, [-1, 2, 8], range(2, 8))):
        mask, depth, st = torch.full((T, 1), 77, dtype=torch.int32, device="cuda"), torch.full((T,), 77, dtype=torch.int32, device="cuda"), _status()
        kv.check(kv.ds_tree_masks(_i32(parent), _i32(start), 8, mask, depth, st))
        assert int(st[0]) == BOUNDS
        left = [i for i in range(T) if i not in rows]
        assert (depth[left] == 77).all() and (mask[left] == 77).all()
        if len(rows) == 8:   # bad parents count as none
            a = [ref.ancestors([-1, -1, 0, -1, -1])[0], ref.ancestors([-1, -1, -1])[0]]
            assert np.array_equal(mask.cpu().numpy(), np.concatenate([ref.words(x, 1) for x in a]))


# ---- accepted paths -------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,D,S,Hk,L,layout", [("bf16", 64, 16, 2, 3, "nhd"), ("f32", 8, 32, 1, 2, "hnd"), ("e4m3", 128, 16, 8, 4, "nhd"),
                                                   ("e4m3", 48, 64, 3, 1, "hnd"), ("bf16", 128, 256, 8, 9, "hnd")])
def test_keep_against_the_plain_form(kv, dtype, D, S, Hk, L, layout):
    """Paths that stay, that move onto their own later places, over pages' ends; requests that are refused stay as they are."""
    rng = np.random.RandomState(D + L)
    lens = [(5, 5), (9, 30), (0, 17), (33, 40), (60, 300), (4, 16), (12, 100), (3, 2), (7, 50), (6, 31), (1, 1), (300, 400)]
    P = 270
    paths = [[0, 1, 2], [1, 2, 3, 4], [], list(range(1, 33)), sorted(rng.permutation(60)[:20]), [0, 3], [11], [0], [2, 2, 3], [1, 6],
             [0], sorted(rng.permutation(300)[:270])]
    path = np.full((len(lens), P), -1, dtype=np.int32)
    for b, x in enumerate(paths):
        path[b, :len(x)] = x
    path[0, 5] = 4                     # behind the end: not looked at
    n_q, n_kv = [a for a, _ in lens], [b for _, b in lens]
    M = max(ceil_div(n, S) for n in n_kv)
    N = sum(ceil_div(n, S) for n in n_kv) + 2
    k, v, scales = _empty_pool(dtype, L, N, S, Hk, D, layout)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in (k, v):
        if dtype == "e4m3":
            _bytes(x).copy_(torch.randint(0, 127, x.shape, dtype=torch.uint8, device="cuda", generator=g))
        else:
            x.copy_(torch.randn(x.shape, device="cuda", generator=g).to(DT[dtype]))
    if scales is not None:
        scales.copy_(torch.randint(0, 256, scales.shape, device="cuda", generator=g).to(torch.uint8))
    order, at, table = rng.permutation(N), 0, np.full((len(lens), M), -1, dtype=np.int32)
    for b, n in enumerate(n_kv):
        table[b, :ceil_div(n, S)] = order[at:at + ceil_div(n, S)]
        at += ceil_div(n, S)
    want = [_bytes(k).clone(), _bytes(v).clone()] + ([scales.clone()] if scales is not None else [])
    was = [x.clone() for x in want]
    lengths = []
    for b, (n, m) in enumerate(lens):
        got = ref.keep(range(m), path[b].tolist(), n, m)
        lengths.append(m if got is None else got[1])
        for to, src in enumerate(got[0] if got else []):
            if to != src:
                a, z = (int(table[b, to // S]), to % S), (int(table[b, src // S]), src % S)
                for i in range(2):
                    want[i][:, a[0], a[1]] = was[i][:, z[0], z[1]]
                if scales is not None:
                    want[2][:, a[0], :, :, a[1]] = was[2][:, z[0], :, :, z[1]]
    st, new_len = _status(), torch.full((len(lens),), 99, dtype=torch.int32, device="cuda")
    kv.check(kv.ds_cache_keep(kv.KvPool(k, v, scales), _i32(path), _i32(np.concatenate([[0], np.cumsum(n_q)])), _i32(table), _i32(n_kv),
                              new_len, st))
    assert int(st[0]) == BOUNDS        # requests 7 (longer than its length), 8 (not ascending), 9 (past its rows)
    assert new_len.tolist() == lengths
    for x, y in zip([_bytes(k), _bytes(v)] + ([scales] if scales is not None else []), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,D", [("e4m3", 128), ("bf16", 64)])
def test_keep_of_many_requests(kv, dtype, D):
    """More requests than blocks of two waves: a block takes several pieces of its request's rows."""
    B, n, S, Hk, L = 700, 6, 16, 8, 8
    k, v, scales = _empty_pool(dtype, L, B, S, Hk, D, "nhd")
    g = torch.Generator(device="cuda").manual_seed(3)
    pool = [_bytes(k), _bytes(v)] + ([scales] if scales is not None else [])
    for x in pool:
        x.copy_(torch.randint(0, 127, x.shape, device="cuda", generator=g).to(x.dtype))
    rng = np.random.RandomState(3)
    kv_len, page = rng.randint(n, S + 1, B), rng.permutation(B)
    path = np.full((B, 4), -1, dtype=np.int32)
    want = [x.clone() for x in pool]
    for b in range(B):
        path[b, :b % 5] = np.sort(rng.permutation(n)[:b % 5])
    for i in range(4):
        b = np.nonzero(path[:, i] >= 0)[0]
        to, src = kv_len[b] - n + i, kv_len[b] - n + path[b, i]
        for x, y in zip(want[:2], pool[:2]):
            x[:, page[b], to] = y[:, page[b], src]
        if scales is not None:
            # (the layers and K, V come behind the indexes)
            w, t = want[2].permute(1, 4, 0, 2, 3), scales.permute(1, 4, 0, 2, 3)
            w[page[b], to] = t[page[b], src]
    st, new_len = _status(), torch.zeros(B, dtype=torch.int32, device="cuda")
    kv.check(kv.ds_cache_keep(kv.KvPool(k, v, scales), _i32(path), _i32(np.arange(B + 1) * n), _i32(page[:, None]), _i32(kv_len),
                              new_len, st))
    assert int(st[0]) == 0
    assert np.array_equal(new_len.cpu().numpy(), kv_len - n + (path >= 0).sum(1))
    for x, y in zip(pool, want):
        assert torch.equal(x, y)


def test_keep_refuses_a_page_out_of_range(kv):
    k, v, _ = _empty_pool("bf16", 1, 4, 16, 1, 64, "nhd")
    k.copy_(torch.randn(k.shape, device="cuda").to(torch.bfloat16))
    for page in (-1, 4):
        before, st, new_len = k.clone(), _status(), torch.zeros(2, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_keep(kv.KvPool(k, v), _i32([[3, 9], [0, 2]]), _i32([0, 10, 13]), _i32([[0, page], [2, -1]]), _i32([24, 13]),
                                  new_len, st))
        assert int(st[0]) == BOUNDS and new_len.tolist() == [24, 12]
        before[0, 2, 11] = before[0, 2, 12]
        assert torch.equal(k.nan_to_num(), before.nan_to_num())


# ---- the pages of a quantised pool -----------------------------------------------------------

@pytest.mark.parametrize("S,Hk,D,layout", [(16, 8, 128, "nhd"), (64, 1, 64, "hnd"), (32, 3, 48, "nhd")])
def test_update_and_compact_of_a_quantised_pool(kv, S, Hk, D, layout):
    """Pages that are copied on write, and those that move, take their scales along: of a partly filled one those of its
    tokens, no byte more."""
    L, N, B, M = 3, 40, 6, 5
    k, v, scales = _empty_pool("e4m3", L, N, S, Hk, D, layout)
    g = torch.Generator(device="cuda").manual_seed(1)
    scales.copy_(torch.randint(0, 256, scales.shape, device="cuda", generator=g).to(torch.uint8))
    pool, st = kv.KvPool(k, v, scales), _status()
    now = [2 * S + 5, 2 * S + 5, 3, S, 0, 0]
    table = np.full((B, M), -1)
    table[0, :3] = table[1, :3] = [30, 7, 22]
    table[2, :1], table[3, :1] = [11], [39]
    count = np.bincount(table[table >= 0], minlength=N)
    nxt, parent = [2 * S + 9, 2 * S + 6, 4, S + 1, 2 * S + 6, 5], [0, 1, 2, 3, 0, 2]
    t2, n2, r2 = torch.empty((B, M), dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"), torch.empty(N, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(kv.ds_cache_update_workspace_bytes(B, N), kv.ds_cache_compact_workspace_bytes(N)), dtype=torch.uint8, device="cuda")
    was = [_bytes(k).clone(), _bytes(v).clone(), scales.clone()]
    kv.check(kv.ds_cache_update(pool, _i32(table), _i32(now), _i32(count), _i32(nxt), t2, n2, r2, ws, st, parent=_i32(parent)))
    assert int(st[0]) == 0
    want = [x.clone() for x in was]
    for b, (src, at, tokens) in {1: (22, 2, 5), 4: (22, 2, 5), 0: (22, 2, 5), 5: (11, 0, 3), 2: (11, 0, 3)}.items():
        page = int(t2[b, at])
        if page != src:
            for i in range(2):
                want[i][:, page, :tokens] = was[i][:, src, :tokens]
            want[2][:, page, :, :, :tokens] = was[2][:, src, :, :, :tokens]
    for x, y in zip((_bytes(k), _bytes(v), scales), want):
        assert torch.equal(x, y)
    t3, r3, pm, used = torch.empty_like(t2), torch.empty_like(r2), torch.empty_like(r2), torch.empty(4, dtype=torch.int32, device="cuda")[:1]
    was = [_bytes(k).clone(), _bytes(v).clone(), scales.clone()]
    kv.check(kv.ds_cache_compact(pool, t2, r2, t3, r3, pm, used, ws, st))
    assert int(st[0]) == 0
    for p in (r2 > 0).nonzero()[:, 0].tolist():
        q = int(pm[p])
        assert q < int(used) and int(r3[q]) == int(r2[p])
        for x, y in zip((_bytes(k), _bytes(v), scales), was):
            assert torch.equal(x[:, q], y[:, p])


def test_quantised_places_past_32_bits(kv):
    """Pages more than 2^32 bytes into a quantised pool: written, read by few rows and by many, kept, copied on write, moved."""
    N, S, Hk, D, G = 270000, 16, 8, 128, 2
    g = torch.Generator(device="cuda").manual_seed(12)
    c = kv.PagedCache(1, N, S, Hk, D, 3, 400, dtype=torch.float8_e4m3fn)
    c.ref[:N - 60] = 1                    # somebody else's: new pages are the last ones
    c.update(_i32([70, 300, 0]))
    assert int(c.block_table[0, 0]) == N - 60
    kn, vn = (torch.randn((370, Hk, D), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    c.append(0, kn, vn, _i32([0, 70, 370, 370]))
    held = [np.ldexp(x, e[..., None]) for x, e in (ref.quantise(_host(y)) for y in (kn, vn))]
    past = [np.stack([x[:70] for x in held]), np.stack([x[70:] for x in held]), np.stack([x[:70] for x in held])]

    def check(n, pages):
        q = torch.randn((sum(n), Hk * G, D), device="cuda", generator=g).to(torch.bfloat16)
        start = np.concatenate([[0], np.cumsum(n)])
        out = c.attend(0, q, _i32(start), max(n))
        c.check_status()
        lens = [x.shape[1] for x in past]
        assert c.kv_len.tolist() == lens
        kp, vp = (np.zeros((3, max(lens), Hk, D)) for _ in range(2))
        for b in range(3):
            kp[b, :lens[b]], vp[b, :lens[b]] = past[b]
        want, _, tol, _ = ref.attend(_host(q), kp, vp, np.arange(3)[:, None], lens, start, lambda b: ref.causal_seen(n[b], lens[b]),
                                     ref.default_scale(D), True)
        assert (np.abs(_host(out) - want) <= tol).all()
        table = c.block_table[c.block_table >= 0]
        assert pages(int(table.min()), int(table.max()))

    c.update(_i32([70, 300, 70]), parent=_i32([0, 1, 0]))
    check([3, 1, 4], lambda lo, hi: lo >= N - 60)
    check([3, 9, 40], lambda lo, hi: lo >= N - 60)
    c.update(_i32([75, 300, 73]))         # both write into the shared last page: one copy
    new = [torch.randn((8, Hk, D), device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
    c.append(0, new[0], new[1], _i32([0, 5, 5, 8]))
    x = np.stack([np.ldexp(y, e[..., None]) for y, e in (ref.quantise(_host(z)) for z in new)])
    c.keep(_i32([[1, 2, 4], [-1, -1, -1], [0, 2, -1]]), _i32([0, 5, 5, 8]))
    past = [np.concatenate([past[0], x[:, [1, 2, 4]]], 1), past[1], np.concatenate([past[2], x[:, [5, 7]]], 1)]
    check([2, 1, 1], lambda lo, hi: lo >= N - 60)
    c.ref[:N - 60] = 0
    c.compact()
    check([20, 1, 7], lambda lo, hi: hi < 60)


# ---- together ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,window", [("e4m3", 0), ("bf16", 0), ("f32", 0), ("e4m3", 40)])
def test_cycles_of_trees_over_a_cache(kv, dtype, window):
    """Prompts, then cycles of tree, attention, path and pages, against a plain list of every request's rows: after each
    cycle the cache holds the rows of the accepted paths, and attention over it is that over the list."""
    L, S, Hk, G, D, B = 2, 16, 2, 2, 64, 4
    rng = np.random.RandomState(4)
    rows_dt = torch.bfloat16 if dtype == "e4m3" else DT[dtype]
    cache = kv.PagedCache(L, 64, S, Hk, D, B, 256, dtype=DT[dtype])
    g = torch.Generator(device="cuda").manual_seed(8)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(rows_dt)

    def held(x):   # what the cache makes of rows
        x = _host(x)
        return np.ldexp(*(lambda c, e: (c, e[..., None]))(*ref.quantise(x))) if dtype == "e4m3" else x

    past = [[np.zeros((2, 0, Hk, D)) for _ in range(B)] for _ in range(L)]

    def write(sizes):
        start = _i32(np.concatenate([[0], np.cumsum(sizes)]))
        new = [(randn(sum(sizes), Hk, D), randn(sum(sizes), Hk, D)) for _ in range(L)]
        for layer, (k, v) in enumerate(new):
            cache.append(layer, k, v, start)
            at = 0
            for b, n in enumerate(sizes):
                past[layer][b] = np.concatenate([past[layer][b], np.stack([held(x[at:at + n]) for x in (k, v)])], 1)
                at += n
        return start

    prompts = [1, 40, 17, 33]
    cache.update(_i32(prompts))
    write(prompts)
    for cycle in range(5):
        sizes = [int(x) for x in rng.randint(1, 40, B)]
        trees = [ref.random_tree(rng, n) for n in sizes]
        T, most = sum(sizes), max(sizes)
        cache.update(cache.kv_len + _i32(sizes))
        start = write(sizes)
        mask = torch.empty((T, ceil_div(most, 32)), dtype=torch.int32, device="cuda")
        depth = torch.empty(T, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_tree_masks(_i32(np.concatenate(trees)), start, most, mask, depth, cache.status, window=window))
        path = np.full((B, most), -1, dtype=np.int32)
        pairs = [ref.ancestors(t, window) for t in trees]
        for b, t in enumerate(trees):
            x, line = int(rng.randint(0, sizes[b])), []
            while x >= 0:
                line.append(x)
                x = int(t[x])
            path[b, :len(line)] = line[::-1]
        for layer in range(L):
            q, lse = randn(T, G * Hk, D), torch.empty((T, G * Hk), device="cuda")
            out = cache.attend(layer, q, start, most, lse=lse, window=window, mask=mask, depth=depth)
            cache.check_status()
            at = 0
            for b, n in enumerate(sizes):
                kk, vv = past[layer][b]
                m = kk.shape[0]
                seen = ref.tree_seen(pairs[b][0], pairs[b][1], n, m, window)
                want, wl, tol, lt = ref.attend(_host(q[at:at + n]), kk[None], vv[None], np.zeros((1, 1), int), [m], [0, n],
                                               lambda _: seen, ref.default_scale(D), dtype != "f32")
                assert (np.abs(_host(out[at:at + n]) - want) <= tol).all() and (np.abs(_host(lse[at:at + n]) - wl) <= lt).all()
                at += n
        cache.keep(_i32(path), start)
        for layer in range(L):
            for b, n in enumerate(sizes):
                x = past[layer][b]
                first = x.shape[1] - n
                line = [p for p in path[b] if p >= 0]
                past[layer][b] = np.concatenate([x[:, :first], x[:, [first + p for p in line]]], 1)
        assert cache.kv_len.tolist() == [x.shape[1] for x in past[0]]
        if cycle == 2:
            cache.compact()
    cache.check_status()
    k, v = cache.pool.k, cache.pool.v
    for layer in range(L):
        kk, vv = _pool_values(k[layer], v[layer], None if cache.pool.scales is None else cache.pool.scales[layer])
        for b in range(B):
            n = past[layer][b].shape[1]
            pages = cache.block_table[b, :ceil_div(n, S)].tolist()
            for x, y in zip((kk, vv), past[layer][b]):
                assert np.array_equal(x[pages].reshape(-1, Hk, D)[:n], y)


def test_a_cycle_of_a_quantised_cache_in_a_graph(kv):
    """Append, attention of a tree and path, captured once and replayed on other rows."""
    S, Hk, G, D, n = 16, 2, 4, 128, 11
    cache = kv.PagedCache(1, 32, S, Hk, D, 2, 128, dtype=torch.float8_e4m3fn)
    g = torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)

    cache.update(_i32([20, 50]))
    cache.append(0, randn(70, Hk, D), randn(70, Hk, D), _i32([0, 20, 70]))
    cache.update(_i32([20 + n, 50 + n]))
    start = _i32([0, n, 2 * n])
    rng = np.random.RandomState(0)
    trees = [ref.random_tree(rng, n) for _ in range(2)]
    parent, mask, depth = _i32(np.concatenate(trees)), torch.empty((2 * n, 1), dtype=torch.int32, device="cuda"), torch.empty(2 * n, dtype=torch.int32, device="cuda")
    path, new_len = _i32([[0, 3, 7], [2, -1, -1]]), torch.empty(2, dtype=torch.int32, device="cuda")
    k, v, q = randn(2 * n, Hk, D), randn(2 * n, Hk, D), randn(2 * n, G * Hk, D)
    out = torch.empty_like(q)

    def cycle():
        kv.check(kv.ds_tree_masks(parent, start, n, mask, depth, cache.status))
        cache.append(0, k, v, start)
        cache.attend(0, q, start, n, out=out, mask=mask, depth=depth)
        kv.check(kv.ds_cache_keep(cache.pool, path, start, cache.block_table, cache.kv_len, new_len, cache.status))

    cycle()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cycle()
    for _ in range(3):
        for x in (k, v, q):
            x.copy_(randn(*x.shape))
        graph.replay()
        torch.cuda.synchronize()
        first = [x.clone() for x in (out, _bytes(cache.pool.k), cache.pool.scales)]
        cycle()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, (out, _bytes(cache.pool.k), cache.pool.scales)))
        assert new_len.tolist() == [23, 51]
    cache.check_status()
