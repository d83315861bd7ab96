"""The paged cache on the GPU against its plain 64-bit forms (_kv_ref.py)."""
import os

import numpy as np
import pytest

import _kv_ref as ref

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


DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Batch:
    """Ragged rows over a pool whose unseen places hold NaN; pages scattered; the table -1 where nothing is needed."""

    def __init__(self, dtype, D, S, Hk, G, lens, layout="nhd", window=0, causal=True, seed=0, spread=1.0, extra=5,
                 strided=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.RandomState(seed)
        self.dtype, self.D, self.S, self.causal, self.window = dtype, D, S, causal, window
        n_q, n_kv = [a for a, _ in lens], [b for _, b in lens]
        M = max(1, max(ref.ceil_div(n, S) for n in n_kv))
        N = sum(ref.ceil_div(n, S) for n in n_kv) + extra
        shape = (1, N, S, Hk, D) if layout == "nhd" else (1, N, Hk, S, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=DT[dtype], device="cuda") for _ in range(2))
        if layout != "nhd":
            self.k, self.v = self.k.transpose(2, 3), self.v.transpose(2, 3)
        order = rng.permutation(N)
        table, at = np.full((len(lens), M), -1, dtype=np.int32), 0
        for b, (nq, n) in enumerate(lens):
            lo = max(0, n - nq - window + 1) if window else 0   # nothing before this is seen
            for p in range(ref.ceil_div(n, S)):
                if (p + 1) * S <= lo:
                    continue
                table[b, p] = order[at]
                at += 1
                a, z = max(lo, p * S) - p * S, min(n, (p + 1) * S) - p * S
                for x in (self.k, self.v):
                    x[0, int(table[b, p]), a:z] = (torch.randn((z - a, Hk, D), device="cuda", generator=g) * spread).to(DT[dtype])
        T = sum(n_q)
        H = G * Hk
        if strided:   # a slice of a wider projection, heads 2 * D apart
            wide = torch.randn((T, H + 2, 2 * D), device="cuda", generator=g).to(DT[dtype])
            self.q = wide[:, 1:H + 1, :D]
            self.out = torch.zeros((T, H + 1, 2 * D), dtype=DT[dtype], device="cuda")[:, :H, D:]
        else:
            self.q = torch.randn((T, H, D), device="cuda", generator=g).to(DT[dtype]) * spread
            self.out = torch.full((T, H, D), 7.0, dtype=DT[dtype], device="cuda")
        self.lse = torch.full((T, H), 7.0, device="cuda")
        self.table, self.kv_len = _i32(table), _i32(n_kv)
        self.q_start = _i32(np.concatenate([[0], np.cumsum(n_q)]))
        self.max_q = max(1, max(n_q))
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")

    def call(self, kv, stream=None, scale=None, lse=True):
        pool = kv.KvPool(self.k, self.v)
        ws = torch.full((kv.ds_paged_attention_workspace_bytes(pool, self.q.shape[1]),), 0xA5, dtype=torch.uint8,
                        device="cuda")
        self.ws = ws
        return kv.ds_paged_attention(pool, 0, self.q, self.q_start, self.max_q, self.table, self.kv_len, self.out, ws,
                                     self.status, lse=self.lse if lse else None, causal=self.causal, window=self.window,
                                     scale=scale, stream=stream)

    def verify(self, kv, **kw):
        assert self.call(kv, **kw) == 0
        assert int(self.status[0]) == 0
        scale = kw.get("scale") or ref.default_scale(self.D)
        k, v = _host(self.k[0]), _host(self.v[0])
        want, lse, tol, lse_tol = ref.attend(_host(self.q), k, v, self.table.cpu().numpy(), self.kv_len.cpu().numpy(),
                                             self.q_start.cpu().numpy(), self.causal, self.window, scale,
                                             self.dtype == "bf16")
        got = _host(self.out)
        assert np.isfinite(got).all()
        off = np.abs(got - want) - tol
        assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape), np.abs(got - want).max())
        if kw.get("lse", True):
            got = _host(self.lse)
            empty = np.isneginf(lse)
            assert np.array_equal(np.isneginf(got), empty)
            off = np.abs(got[~empty] - lse[~empty]) - lse_tol[~empty]
            assert off.size == 0 or off.max() <= 0, off.max()


MIXED = [(1, 1), (1, 0), (0, 37), (3, 3), (5, 2), (17, 200), (1, 129), (2, 128), (4, 127), (9, 33), (33, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,S,Hk,G,layout", [(128, 16, 2, 4, "nhd"), (64, 32, 1, 1, "hnd"), (128, 64, 2, 5, "hnd"),
                                             (64, 128, 3, 8, "nhd"), (128, 256, 1, 16, "nhd"), (64, 16, 1, 7, "nhd"),
                                             (128, 32, 1, 128, "hnd"), (64, 64, 2, 33, "nhd")])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20), (False, 1)])
def test_attention_of_mixed_requests(kv, dtype, D, S, Hk, G, layout, causal, window):
    """Empty requests, empty contexts, more rows than tokens, lengths about the pages' and tiles' ends."""
    Batch(dtype, D, S, Hk, G, MIXED, layout, window, causal, seed=D + S + G).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 5000)], [(1, 4097), (17, 3000), (5, 1)], [(300, 700)], [(130, 1500), (1, 900)],
                                  [(257, 257), (64, 64)]])
def test_attention_of_long_contexts(kv, dtype, lens):
    """Work split over the context and joined; prompts of several tiles."""
    Batch(dtype, 128, 32, 2, 4, lens, seed=len(lens)).verify(kv)


@pytest.mark.parametrize("D,S,Hk,G,lens", [(128, 64, 8, 1, [(1, 1700 + 61 * i) for i in range(24)]),
                                           (64, 128, 8, 2, [(5, 900 + 77 * i) for i in range(20)]),
                                           (128, 32, 6, 8, [(17, 400 + 83 * i) for i in range(20)]),
                                           (64, 16, 8, 4, [(40 + 13 * i, 700 + 50 * i) for i in range(10)])])
def test_attention_of_many_long_contexts(kv, D, S, Hk, G, lens):
    """Many key tiles and several units for every SM, of one row tile and of two."""
    Batch("bf16", D, S, Hk, G, lens, seed=D + G).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,n_q", [(128, 1, 1), (64, 3, 1), (128, 1, 4), (64, 5, 1), (128, 8, 1), (64, 2, 4), (128, 3, 3),
                                     (64, 16, 1), (128, 17, 1)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 70)])
def test_attention_of_few_rows(kv, dtype, D, G, n_q, causal, window):
    """1 to 17 rows a KV head: each form of the kernels for few rows, whole units and cut ones, empty ones between."""
    lens = [(1, 1), (n_q, 0), (n_q, 63), (0, 10), (n_q, 64), (max(1, n_q - 1), 65), (n_q, 900), (1, 3000), (n_q, n_q)]
    Batch(dtype, D, 16, 2, G, lens, window=window, causal=causal, seed=D + G + n_q).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 128, 129, 500])
def test_attention_windows_on_long_contexts(kv, dtype, window):
    """Pages before the window hold NaN or have no entry."""
    Batch(dtype, 64, 16, 2, 3, [(40, 2000), (1, 1025), (7, 600), (200, 450)], window=window, seed=window).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_many_small_requests(kv, dtype):
    rng = np.random.RandomState(3)
    lens = [(int(a), int(a + c)) for a, c in zip(rng.randint(0, 4, 700), rng.randint(0, 90, 700))]
    Batch(dtype, 64, 16, 1, 2, lens, seed=9).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_of_peaked_scores(kv, dtype):
    """Scores that span hundreds: the running maximum rises many times."""
    Batch(dtype, 128, 64, 2, 4, [(9, 1100), (1, 777), (140, 300)], seed=4, spread=4.0).verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_rising_scores(kv, dtype):
    """Keys that grow along the context: the maximum rises in every tile."""
    x = Batch(dtype, 64, 32, 1, 4, [(1, 3000), (30, 1000)], seed=5)
    scale = torch.linspace(0.0, 6.0, 3000, device="cuda")
    table = x.table.cpu().numpy()
    for b, n in ((0, 3000), (1, 1000)):
        for p in range(ref.ceil_div(n, 32)):
            z = min(32, n - 32 * p)
            x.k[0, int(table[b, p]), :z] = (x.k[0, int(table[b, p]), :z].float()
                                            * scale[32 * p:32 * p + z, None, None]).to(DT[dtype])
    x.verify(kv)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,window", [(128, 4, 0), (64, 1, 0), (128, 2, 40), (64, 8, 20)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_attention_of_values_that_some_rows_do_not_see(kv, dtype, D, G, window, what):
    """A later token's value, or one before a row's window, that is not finite: rows that do not see it are as
    without it, rows that do are not finite in its columns."""
    check_unseen_values(kv, dtype, D, G, window, what, [(9, 300), (70, 200), (40, 40), (20, 1400), (5, 130)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,n_q,window", [(128, 1, 4, 0), (64, 2, 4, 0), (128, 2, 3, 40), (64, 4, 4, 20)])
def test_attention_of_values_that_some_of_few_rows_do_not_see(kv, dtype, D, G, n_q, window):
    check_unseen_values(kv, dtype, D, G, window, float("nan"), [(n_q, 300), (3, 70), (n_q, 2100), (n_q, n_q)])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,G,n_q", [(128, 1, 1), (64, 4, 2), (64, 16, 1), (128, 24, 1), (128, 4, 70)])
def test_attention_of_an_infinite_value(kv, dtype, D, G, n_q):
    """An infinite value that every row of a request sees is their sum in its column; other columns are as without it."""
    lens = [(n_q, 300), (n_q, n_q + 3), (n_q, 2500), (n_q, 5000)]
    x = Batch(dtype, D, 16, 2, G, lens, seed=17)
    x.verify(kv)
    clean = x.out.clone()
    table, row = x.table.cpu().numpy(), 0
    for b, (nq, n) in enumerate(lens):
        j = (n - nq) // 2
        x.v[0, int(table[b, j // 16]), j % 16, 1, 3] = float("inf") if b % 2 else -float("inf")
    assert x.call(kv) == 0 and int(x.status[0]) == 0
    got, want = _host(x.out), _host(clean)
    for b, (nq, n) in enumerate(lens):
        rows, row = slice(row, row + nq), row + nq
        assert (got[rows, G:, 3] == (np.inf if b % 2 else -np.inf)).all(), b
        got[rows, G:, 3] = want[rows, G:, 3]
    assert (np.abs(got - want) <= 2 ** -7 * np.abs(want).max()).all()


def check_unseen_values(kv, dtype, D, G, window, what, lens):
    x = Batch(dtype, D, 16, 2, G, lens, window=window, seed=31)
    x.verify(kv)
    clean = x.out.clone()
    table, spots = x.table.cpu().numpy(), []
    for b, (nq, n) in enumerate(lens):
        spots.append((b, n - 1 - nq // 3))                       # a new token that the first rows do not see
        if window:
            spots.append((b, max(0, n - nq - window + 1) + 2))   # at the window's edge: the last rows do not see it
    for b, j in spots:
        x.v[0, int(table[b, j // 16]), j % 16, 1, 3] = what
    assert x.call(kv) == 0 and int(x.status[0]) == 0
    got, want = _host(x.out), _host(clean)
    _, _, tol, _ = ref.attend(_host(x.q), np.nan_to_num(_host(x.k[0])), np.nan_to_num(_host(x.v[0]), posinf=0, neginf=0), table,
                              x.kv_len.cpu().numpy(), x.q_start.cpu().numpy(), True, window, ref.default_scale(D), dtype == "bf16")
    row = 0
    for b, (nq, n) in enumerate(lens):
        for i in range(nq):
            p = n - nq + i
            sees = [j for c, j in spots if c == b and j <= p and (not window or j > p - window)]
            bad = np.zeros(got.shape[1:], dtype=bool)
            if sees:
                bad[G:, 3] = True                                # the second KV head's column 3
            assert np.isfinite(got[row][~bad]).all(), (b, i)
            assert not np.isfinite(got[row][bad]).any(), (b, i)
            assert (np.abs(got[row] - want[row])[~bad] <= 2 * tol[row][~bad] + 1e-6).all(), (b, i)
            row += 1


@pytest.mark.parametrize("G,n_q,B", [(3, 70, 304), (4, 8, 608), (4, 4, 608)])
def test_attention_waits_for_a_long_recomputation(kv, G, n_q, B):
    """A NaN in the last new token's value and two whole units of 100,000 keys for every share: up to 32 rows a warp are
    computed again over 100,000 keys while the next unit waits (seconds, if a key and a row at a time). All requests
    hold the same pages. Values grow along the context, so that keys left out or counted twice show."""
    n, S, D = 100000, 256, 64
    g = torch.Generator(device="cuda").manual_seed(G)
    pages = ref.ceil_div(n, S)
    k = torch.randn((1, pages, S, 1, D), device="cuda", generator=g).to(torch.bfloat16)
    ramp = torch.arange(pages * S, device="cuda").view(1, pages, S, 1, 1) / n
    v = (torch.rand(k.shape, device="cuda", generator=g) + 3 * ramp).to(torch.bfloat16)
    q = torch.randn((B * n_q, G, D), device="cuda", generator=g).to(torch.bfloat16)
    pool, status = kv.KvPool(k, v), torch.zeros(4, dtype=torch.int32, device="cuda")
    table, q_start = _i32(np.tile(np.arange(pages), (B, 1))), _i32(np.arange(B + 1) * n_q)
    ws = torch.empty(kv.ds_paged_attention_workspace_bytes(pool, G), dtype=torch.uint8, device="cuda")

    def call():
        out, lse = torch.full_like(q, 7.0), torch.full((B * n_q, G), 7.0, device="cuda")
        kv.check(kv.ds_paged_attention(pool, 0, q, q_start, n_q, table, _i32([n] * B), out, ws, status, lse=lse))
        assert int(status[0]) == 0
        return out.float().view(B, n_q, G, D), lse

    clean, lse = call()
    last = divmod(n - 1, S)
    v[0, last[0], last[1], 0, 3] = float("nan")
    got, lse_got = call()
    assert torch.equal(lse, lse_got)
    assert got[:, -1, :, 3].isnan().all()
    got[:, -1, :, 3] = clean[:, -1, :, 3]
    # Values are positive, so both are within their bound of the exact sum relative to themselves: J + 32 roundings of
    # float32 and, at most, two of bfloat16 (and a quarter); scores of size 5 add (D + 4) 5 * 2^-24 twice.
    bound = 2 * ((n + 32 + 10 * (D + 4)) * ref.U32 + 2.5 * ref.UBF)
    assert ((got - clean).abs() <= bound * clean).all()
    # float64, a few requests
    kk, vv = (x[0].reshape(-1, D)[:n].double() for x in (k, v))
    vv[-1, 3] = 0
    for b in (0, B // 2, B - 1):
        s = torch.einsum("igd,jd->igj", q[b * n_q:(b + 1) * n_q].double(), kk) * D ** -0.5
        s = s.masked_fill((torch.arange(n, device="cuda") > torch.arange(n - n_q, n, device="cuda")[:, None])[:, None], -np.inf)
        want = torch.softmax(s, -1) @ vv
        assert ((got[b][:-1] - want[:-1]).abs() <= bound / 2 * want[:-1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_strided_rows_and_scale(kv, dtype):
    x = Batch(dtype, 128, 16, 2, 4, [(5, 90), (1, 300), (40, 41)], strided=True, seed=6)
    base = x.out._base if x.out._base is not None else x.out
    x.verify(kv, scale=0.03)
    assert (base[:, -1] == 0).all() and (base[:, :, :128] == 0).all()      # nothing beside the rows is written
    x.verify(kv, lse=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_same_bits_twice_and_on_another_stream(kv, dtype):
    x = Batch(dtype, 128, 16, 2, 4, [(1, 2500), (17, 1300), (60, 61)], seed=7)
    x.verify(kv)
    first = x.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            x.out.fill_(3.0)
            assert x.call(kv) == 0
    s.synchronize()
    assert torch.equal(first.view(torch.int16 if dtype == "bf16" else torch.int32),
                       x.out.view(torch.int16 if dtype == "bf16" else torch.int32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_in_a_graph(kv, dtype):
    x = Batch(dtype, 64, 64, 2, 4, [(1, 600), (9, 300)], seed=8)
    pool = kv.KvPool(x.k, x.v)
    ws = torch.empty(kv.ds_paged_attention_workspace_bytes(pool, 8), dtype=torch.uint8, device="cuda")

    def step():
        kv.check(kv.ds_paged_attention(pool, 0, x.q, x.q_start, x.max_q, x.table, x.kv_len, x.out, ws, x.status, lse=x.lse))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    x.kv_len.copy_(_i32([433, 300]))                # a shorter context at replay: lengths are read on the device
    # the request's row stands at its last token now
    x.out.fill_(1.0)
    g.replay()
    torch.cuda.synchronize()
    got = x.out.clone()
    x.verify(kv)
    assert torch.equal(got, x.out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_reports_what_is_out_of_bounds(kv, dtype):
    """Malformed device data: the status says so, nothing faults, the other requests' rows stand."""
    def fresh():
        return Batch(dtype, 64, 16, 1, 2, [(2, 100), (3, 50), (1, 70)], seed=11)

    good = fresh()
    good.verify(kv)
    for what in ("page", "negative page", "kv_len", "negative kv_len", "q_start", "max_q", "q_end"):
        x = fresh()
        if what == "page":
            x.table[1, 0] = x.k.shape[1]
        elif what == "negative page":
            x.table[1, 2] = -1
        elif what == "kv_len":
            x.kv_len[1] = x.table.shape[1] * 16 + 1
        elif what == "negative kv_len":
            x.kv_len[1] = -5
        elif what == "q_start":
            x.q_start[2] = 1
        elif what == "max_q":
            x.max_q = 2
        else:
            x.q_start[3] = 1000
        assert x.call(kv) == 0
        assert int(x.status[0]) == 6, what
        assert torch.equal(x.out[:2], good.out[:2]), what


def test_append_places_rows(kv):
    for dtype, D, S, Hk, layout in (("bf16", 128, 16, 2, "nhd"), ("f32", 64, 32, 3, "hnd"), ("bf16", 8, 256, 1, "nhd"),
                                    ("f32", 200, 64, 5, "hnd"), ("bf16", 72, 128, 4, "nhd")):
        lens = [(1, 1), (0, 20), (3, 3), (5, 2), (40, 300), (1, S + 1), (S, S), (2, 0)] + [(1, 7)] * 300
        rng = np.random.RandomState(S)
        M = max(ref.ceil_div(n, S) for _, n in lens)
        N = sum(ref.ceil_div(n, S) for _, n in lens) + 2
        shape = (3, N, S, Hk, D) if layout == "nhd" else (3, N, Hk, S, D)
        k, v = (torch.zeros(shape, dtype=DT[dtype], device="cuda") for _ in range(2))
        if layout == "hnd":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        table, at, order = np.full((len(lens), M), -1, np.int32), 0, rng.permutation(N)
        for b, (_, n) in enumerate(lens):
            p = ref.ceil_div(n, S)
            table[b, :p] = order[at:at + p]
            at += p
        q_start = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
        T = int(q_start[-1])
        g = torch.Generator(device="cuda").manual_seed(1)
        wide = torch.randn((T, 2 * Hk, D), device="cuda", generator=g).to(DT[dtype])    # K and V of one projection
        kn, vn = wide[:, :Hk], torch.randn((T, Hk, D), device="cuda", generator=g).to(DT[dtype])
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        want_k, want_v = k.clone(), v.clone()
        for b, (a, n) in enumerate(lens):
            for i in range(a):
                p = n - a + i
                if p >= 0:
                    want_k[1, int(table[b, p // S]), p % S] = kn[q_start[b] + i]
                    want_v[1, int(table[b, p // S]), p % S] = vn[q_start[b] + i]
        pool = kv.KvPool(k, v)
        kv.check(kv.ds_cache_append(pool, 1, kn, vn, _i32(q_start), _i32(table), _i32([n for _, n in lens]), status))
        assert int(status[0]) == 0
        assert torch.equal(k, want_k) and torch.equal(v, want_v)
        # a page out of range: reported, the rest written, nothing else touched
        k.zero_(), v.zero_()
        bad = table.copy()
        bad[4, 18 if S == 16 else 0] = N
        kv.check(kv.ds_cache_append(pool, 1, kn, vn, _i32(q_start), _i32(bad), _i32([n for _, n in lens]), status))
        lost = 300 - 40 < (19 * 16 if S == 16 else S)
        assert int(status[0]) == (6 if lost else 0)


@pytest.mark.parametrize("dtype,D,S,Hk", [("bf16", 128, 16, 2), ("f32", 64, 32, 3), ("bf16", 8, 256, 1), ("f32", 200, 64, 5),
                                          ("bf16", 72, 128, 4)])
@pytest.mark.parametrize("which", ["first", "last"])
def test_append_reports_a_bad_page_and_writes_the_rest(kv, dtype, D, S, Hk, which):
    """The page of a request's first (last) new token is none: reported, that page's rows are lost, every other row is
    written, nothing else is touched, in this layer or another."""
    lens, bad, layer = [(3, 3), (0, 20), (40, 300), (S, S + 1), (1, 7)], 2, 1
    n_new, n = lens[bad]
    rng = np.random.RandomState(S + D)
    M, N = max(ref.ceil_div(x, S) for _, x in lens), sum(ref.ceil_div(x, S) for _, x in lens) + 2
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.randn((3, N, S, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    table, at, order = np.full((len(lens), M), -1, np.int32), 0, rng.permutation(N)
    for b, (_, x) in enumerate(lens):
        table[b, :ref.ceil_div(x, S)] = order[at:at + ref.ceil_div(x, S)]
        at += ref.ceil_div(x, S)
    gone = (n - n_new if which == "first" else n - 1) // S
    table[bad, gone] = N if which == "first" else -3
    q_start = np.concatenate([[0], np.cumsum([a for a, _ in lens])])
    kn, vn = (torch.randn((int(q_start[-1]), Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    want_k, want_v = k.clone(), v.clone()
    lost = 0
    for b, (a, x) in enumerate(lens):
        for i in range(a):
            p = x - a + i
            if b == bad and p // S == gone:
                lost += 1
                continue
            want_k[layer, int(table[b, p // S]), p % S] = kn[q_start[b] + i]
            want_v[layer, int(table[b, p // S]), p % S] = vn[q_start[b] + i]
    assert lost > 0
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv.check(kv.ds_cache_append(kv.KvPool(k, v), layer, kn, vn, _i32(q_start), _i32(table), _i32([x for _, x in lens]), status))
    assert int(status[0]) == 6
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def _interleaved(kind, L, N, S, Hk, D, dtype):
    """K and V as views of one tensor: (buffer, k, v) of shape [L, N, S, Hk, D]."""
    if kind == "token":          # K and V of a token side by side
        buf = torch.zeros((L, N, S, 2, Hk, D), dtype=dtype, device="cuda")
        return buf, buf[:, :, :, 0], buf[:, :, :, 1]
    if kind == "head":           # of a head, with a gap behind them
        buf = torch.zeros((L, N, S, Hk, 2 * D + 8), dtype=dtype, device="cuda")
        return buf, buf[..., :D], buf[..., D:2 * D]
    if kind == "page":           # of a page, heads outside its tokens
        buf = torch.zeros((L, N, 2, Hk, S, D), dtype=dtype, device="cuda")
        return buf, buf[:, :, 0].transpose(2, 3), buf[:, :, 1].transpose(2, 3)
    # layers inside pages, tokens of several layers side by side, more heads than are used
    buf = torch.zeros((N, S, L, 2, Hk + 1, D), dtype=dtype, device="cuda")
    k, v = (buf[:, :, :, i, :Hk].permute(2, 0, 1, 3, 4) for i in range(2))
    return buf, k, v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["token", "head", "page", "layers"])
@pytest.mark.parametrize("S,Hk,D,G,n", [(16, 2, 128, 4, 5), (64, 3, 64, 1, 2), (128, 1, 128, 5, 40), (16, 4, 64, 2, 90)])
def test_interleaved_pools(kv, dtype, kind, S, Hk, D, G, n):
    """K and V in one tensor, with strides that are not dense: append, attention, copy on write and compaction through
    the calls, against dense arrays; what lies between the rows stays as it was."""
    L, B, N, lens = 2, 3, 64, [3 * S + 7, n, 5]
    g = torch.Generator(device="cuda").manual_seed(S + D + n)
    buf, k, v = _interleaved(kind, L, N, S, Hk, D, DT[dtype])
    mine = torch.zeros_like(buf)
    for x in _views(kind, mine, Hk, D):
        x.fill_(1)
    pool, status = kv.KvPool(k, v), torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(kv.ds_cache_update_workspace_bytes(B, N), kv.ds_cache_compact_workspace_bytes(N),
                         kv.ds_paged_attention_workspace_bytes(pool, G * Hk)), dtype=torch.uint8, device="cuda")
    M = 10
    held = torch.zeros(N, dtype=torch.int32, device="cuda")
    held[::3] = 1                                       # somebody else's, so that pages lie apart
    state = [_i32(np.full((B, M), -1)), _i32([0] * B), held]

    def update(new, parent=None):
        out = [torch.empty_like(x) for x in state]
        kv.check(kv.ds_cache_update(pool, *state, _i32(new), *out, ws, status, parent=None if parent is None else _i32(parent)))
        state[:] = out

    past = [[torch.zeros((2, 0, Hk, D), dtype=DT[dtype], device="cuda") for _ in range(B)] for _ in range(L)]

    def add(rows):
        start = _i32(np.concatenate([[0], np.cumsum(rows)]))
        for layer in range(L):
            new = torch.randn((2, sum(rows), Hk, D), device="cuda", generator=g).to(DT[dtype])
            kv.check(kv.ds_cache_append(pool, layer, new[0], new[1], start, state[0], state[1], status))
            past[layer] = [torch.cat([x, y], 1) for x, y in zip(past[layer], new.split(rows, 1))]

    def check(rows):
        start = np.concatenate([[0], np.cumsum(rows)])
        held_len = [x.shape[1] for x in past[0]]
        assert state[1].tolist() == held_len
        for layer in range(L):
            q = torch.randn((sum(rows), G * Hk, D), device="cuda", generator=g).to(DT[dtype])
            out = torch.empty_like(q)
            kv.check(kv.ds_paged_attention(pool, layer, q, _i32(start), max(rows), state[0], state[1], out, ws, status))
            dense = np.zeros((2, B, max(held_len), Hk, D))
            for b in range(B):
                dense[:, b, :held_len[b]] = _host(past[layer][b])
            want, _, tol, _ = ref.attend(_host(q), dense[0], dense[1], np.arange(B)[:, None], held_len, start, True, 0,
                                         ref.default_scale(D), dtype == "bf16")
            assert (np.abs(_host(out) - want) <= tol).all()
        assert int(status[0]) == 0
        assert (buf[mine == 0] == 0).all()

    update(lens)
    add(lens)
    check([n, n, 5])
    update([lens[0], lens[0], 5], [0, 0, 2])            # request 1 becomes a copy of request 0
    for layer in range(L):
        past[layer][1] = past[layer][0]
    update([lens[0] + 3, lens[0] + n, 6])               # both write into the shared last page
    add([3, n, 1])
    check([3, n, 1])
    state[2] -= (torch.arange(N, device="cuda") % 3 == 0).int()
    out = torch.empty_like(state[0]), torch.empty_like(state[2])
    page_map, used = torch.empty_like(state[2]), _i32([0])
    kv.check(kv.ds_cache_compact(pool, state[0], state[2], *out, page_map, used, ws, status))
    state[0], state[2] = out
    assert int(used[0]) == int((state[2] > 0).sum()) and int(state[0].max()) < int(used[0])
    check([4, n, 2])


def _views(kind, buf, Hk, D):
    """K's and V's parts of a buffer of _interleaved."""
    if kind == "token":
        return buf[:, :, :, 0], buf[:, :, :, 1]
    if kind == "head":
        return buf[..., :D], buf[..., D:2 * D]
    if kind == "page":
        return buf[:, :, 0], buf[:, :, 1]
    return buf[:, :, :, 0, :Hk], buf[:, :, :, 1, :Hk]


@pytest.mark.parametrize("dtype,Hk", [("bf16", 8), ("f32", 1)])
@pytest.mark.parametrize("q_start,kv_len", [([0, 20, 3, 4], [30, 32, 32]), ([0, 100, 1, 2], [30, 32, 32]),
                                            ([0, 4, 8, 25], [30, 31, 32]), ([-1, 4, 8, 20], [32, 9, 32]),
                                            ([0, 20, 12, 20], [32, 32, 32]), ([-1, -1, -1, -1], [32, 32, 32]),
                                            ([0, 4, 8, 20], [30, 33, 32]), ([0, 4, 8, 20], [4, -1, 12]),
                                            ([21, 21, 21, 21], [8, 8, 8]), ([5, 3, 0, 2], [32, 32, 32])])
def test_append_refuses_malformed_requests(kv, dtype, Hk, q_start, kv_len):
    """Row starts that decrease or leave the rows, lengths out of range: reported, and only rows of a well-formed request
    are written, each to its own place. Behind the table stand words that would pass for pages."""
    S, M, N, T, D = 16, 2, 90, 20, 64
    B = len(kv_len)
    ok = [0 <= q_start[b] <= q_start[b + 1] <= T and 0 <= kv_len[b] <= M * S for b in range(B)]
    g = torch.Generator(device="cuda").manual_seed(2)
    words = _i32(np.arange(B * M + 64))
    table = words[:B * M].view(B, M)
    k, v = (torch.randn((1, N, S, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    kn, vn = (torch.randn((T, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    old_k, old_v = k.clone(), v.clone()
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    kv.check(kv.ds_cache_append(kv.KvPool(k, v), 0, kn, vn, _i32(q_start), table, _i32(kv_len), status))
    assert int(status[0]) == 6
    free = torch.ones((N, S), dtype=torch.bool, device="cuda")
    for b in range(B):
        n = q_start[b + 1] - q_start[b]
        for i in range(n if ok[b] else 0):
            p, t = kv_len[b] - n + i, q_start[b] + i
            if p < 0:
                continue
            page, at = b * M + p // S, p % S
            free[page, at] = False
            for x, new, old in ((k, kn, old_k), (v, vn, old_v)):
                assert torch.equal(x[0, page, at], new[t]) or torch.equal(x[0, page, at], old[0, page, at])
    assert torch.equal(k[0][free], old_k[0][free]) and torch.equal(v[0][free], old_v[0][free])
    if q_start == sorted(q_start) and 0 <= q_start[0] and q_start[-1] <= T:      # the rows of the others stand
        for b in range(B):
            n = q_start[b + 1] - q_start[b]
            for i in range(n if ok[b] else 0):
                p = kv_len[b] - n + i
                assert p < 0 or torch.equal(k[0, b * M + p // S, p % S], kn[q_start[b] + i])


def _state(rng, B, S, N, width, M, pins):
    """Requests in groups that share their first pages; some empty; some pages pinned from outside."""
    pages = list(rng.permutation(N))
    table, lens = [[-1] * M for _ in range(B)], [0] * B
    for b0 in range(0, B, width):
        common = int(rng.randint(0, max(1, M * S - 2 * S)))
        row = [pages.pop() for _ in range(min(ref.ceil_div(common, S), len(pages)))]
        common = min(common, len(row) * S)
        for b in range(b0, min(B, b0 + width)):
            if rng.rand() < 0.1:
                continue
            if rng.rand() < 0.5 or not pages:
                table[b][:len(row)], lens[b] = row, common
            else:
                n = common // S
                extra = min(int(rng.randint(1, 3)), len(pages), M - n)
                mine = row[:n] + [pages.pop() for _ in range(extra)]
                table[b][:len(mine)] = mine
                lens[b] = n * S + (int(rng.randint(1, extra * S + 1)) if extra else 0)
    table = [[int(p) for p in r] for r in table]
    lens = [int(n) for n in lens]
    held = [0] * N
    for b in range(B):
        for p in table[b][:ref.ceil_div(lens[b], S)]:
            held[p] += 1
    for _ in range(pins):
        held[int(rng.randint(N))] += 1
    return table, lens, held


@pytest.mark.parametrize("B,S,N,width,M,pins", [(1, 16, 9, 1, 6, 0), (7, 16, 64, 3, 6, 0), (64, 32, 900, 8, 9, 20),
                                                (300, 16, 5000, 4, 11, 100), (33, 64, 70, 33, 5, 1), (5, 256, 11, 2, 3, 0),
                                                (2000, 16, 30000, 2, 7, 50)])
@pytest.mark.parametrize("kind", ["grow", "mixed", "beams"])
def test_update_against_the_plain_form(kv, B, S, N, width, M, pins, kind):
    for seed in range(4):
        rng = np.random.RandomState(100 * seed + B)
        table, lens, held = _state(rng, B, S, N, width, M, pins)
        parent = None
        if kind == "grow":
            new = [min(M * S, n + int(rng.randint(0, S))) for n in lens]
        elif kind == "mixed":
            new = [int(rng.choice([0, n, max(0, n - int(rng.randint(0, 2 * S))), min(M * S, n + 1)])) for n in lens]
        else:
            parent = [int(rng.randint(-1, B)) if rng.rand() < 0.2 else min(B - 1, b // width * width + int(rng.randint(width)))
                      for b in range(B)]
            new = [min(M * S, (lens[p] if p >= 0 else 0) + int(rng.randint(0, 3))) for p in parent]
        want = ref.update(table, lens, held, new, parent, S, N)
        k = torch.arange(2 * N * S * 1 * 8, device="cuda").reshape(2, N, S, 1, 8).to(torch.float32)
        v = -k
        want_k, want_v = k.clone(), v.clone()
        pool = kv.KvPool(k, v)
        state = _i32(table), _i32(lens), _i32(held)
        out = tuple(torch.full_like(x, -77) for x in state)
        ws = torch.full((kv.ds_cache_update_workspace_bytes(B, N),), 0xA5, dtype=torch.uint8, device="cuda")
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_update(pool, *state, _i32(new), *out, ws, status, parent=None if parent is None else _i32(parent)))
        if want is None:
            assert int(status[0]) == 8
            want = [[table[b][j] for j in range(M)] for b in range(B)], lens, held, {}
        else:
            assert int(status[0]) == 0
        assert out[0].tolist() == want[0] and out[1].tolist() == want[1] and out[2].tolist() == want[2]
        for a, z, n in want[3].values():
            for x in (want_k, want_v):
                x[:, z, :n] = x[:, a, :n]
        assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_update_copies_every_layout(kv):
    for dtype, layout, Hk, D, S in (("bf16", "nhd", 4, 128, 16), ("bf16", "hnd", 3, 72, 32), ("f32", "hnd", 2, 64, 64)):
        N, L = 12, 3
        shape = (L, N, S, Hk, D) if layout == "nhd" else (L, N, Hk, S, D)
        k, v = (torch.randn(shape, device="cuda").to(DT[dtype]) for _ in range(2))
        if layout == "hnd":
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        want_k, want_v = k.clone(), v.clone()
        table, lens = [[3, 5, -1], [3, 5, -1], [3, 5, -1]], [S + 7] * 3
        held = [0] * N
        held[3] = held[5] = 3
        new = [S + 8, S + 7, 2 * S + 1]
        want = ref.update(table, lens, held, new, None, S, N)
        assert sorted(want[3]) == [0, 2]
        state = _i32(table), _i32(lens), _i32(held)
        out = tuple(torch.empty_like(x) for x in state)
        ws = torch.empty(kv.ds_cache_update_workspace_bytes(3, N), dtype=torch.uint8, device="cuda")
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_update(kv.KvPool(k, v), *state, _i32(new), *out, ws, status))
        for a, z, n in want[3].values():
            for x in (want_k, want_v):
                x[:, z, :n] = x[:, a, :n]
        assert int(status[0]) == 0 and out[0].tolist() == want[0] and out[2].tolist() == want[2]
        assert torch.equal(k, want_k) and torch.equal(v, want_v)


@pytest.mark.parametrize("L", [1, 32767, 32768, 40000])
def test_update_and_compact_of_many_layers(kv, L):
    """More layers than a grid has rows of blocks: the copied page and the moved ones in every layer."""
    N, S = 4, 16
    k = torch.randn((L, N, S, 1, 8), device="cuda")
    v = torch.randn((L, N, S, 1, 8), device="cuda")
    want = [k.clone(), v.clone()]
    pool, status = kv.KvPool(k, v), torch.zeros(4, dtype=torch.int32, device="cuda")
    state = _i32([[2, -1], [2, -1]]), _i32([9, 9]), _i32([0, 0, 2, 1])
    out = tuple(torch.empty_like(x) for x in state)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    kv.check(kv.ds_cache_update(pool, *state, _i32([10, 11]), *out, ws, status))
    assert int(status[0]) == 0 and out[0].tolist() == [[2, -1], [0, -1]] and out[2].tolist() == [1, 0, 1, 1]
    for x, y in zip((k, v), want):
        y[:, 0, :9] = y[:, 2, :9]
        assert torch.equal(x, y)
    page_map, n_used = _i32([0] * N), _i32([0])
    moved = tuple(torch.empty_like(x) for x in (out[0], out[2]))
    kv.check(kv.ds_cache_compact(pool, out[0], out[2], *moved, page_map, n_used, ws, status))
    assert int(status[0]) == 0 and n_used.tolist() == [3] and page_map.tolist() == [0, -1, 2, 1]
    for x, y in zip((k, v), want):
        y[:, 1] = y[:, 3]
        assert torch.equal(x, y)


def test_update_refuses_bad_state_and_changes_nothing(kv):
    S, N, M, B = 16, 8, 3, 3
    k = torch.zeros((1, N, S, 1, 8), device="cuda")
    pool = kv.KvPool(k, k.clone())
    table, lens, held = [[0, 1, -1], [2, -1, -1], [-1, -1, -1]], [20, 5, 0], [1, 1, 1, 0, 0, 0, 0, 0]
    ok = [30, 6, 48]
    cases = [(dict(new=[49, 6, 1]), 6), (dict(new=[-1, 6, 1]), 6), (dict(parent=[0, 3, 2]), 6), (dict(parent=[0, -2, 2]), 6),
             (dict(lens=[20, 5, 49]), 6), (dict(lens=[-1, 5, 0]), 6), (dict(held=[1, 0, 1, 0, 0, 0, 0, 0], new=[0, 6, 1]), 6),
             (dict(table=[[0, 9, -1], [2, -1, -1], [-1, -1, -1]], new=[30, 6, 1]), 6),
             (dict(held=[1, 1, 1, 1, 1, 1, 0, 0]), 8), (dict(), 0)]
    for change, code in cases:
        t, n, h = change.get("table", table), change.get("lens", lens), change.get("held", held)
        parent = change.get("parent")
        state = _i32(t), _i32(n), _i32(h)
        out = tuple(torch.full_like(x, -77) for x in state)
        ws = torch.empty(kv.ds_cache_update_workspace_bytes(B, N), dtype=torch.uint8, device="cuda")
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_update(pool, *state, _i32(change.get("new", ok)), *out, ws, status,
                                    parent=None if parent is None else _i32(parent)))
        assert int(status[0]) == code, (change, int(status[0]))
        if code:
            assert all(torch.equal(a, b) for a, b in zip(state, out)), change


@pytest.mark.parametrize("B,own", [(1, False), (16, True), (40, False), (300, True), (300, False)])
def test_update_refuses_bad_pages_that_stay(kv, B, own):
    """A table entry that is no page, anywhere in what a request keeps from itself, whether it grows, stays, falls back or
    (its pages being given back) ends: the state out is the state in."""
    S, M = 16, 40
    N = B * M
    rng = np.random.RandomState(B)
    k = torch.zeros((1, N, S, 1, 8), device="cuda")
    pool = kv.KvPool(k, k.clone())
    ws = torch.empty(kv.ds_cache_update_workspace_bytes(B, N), dtype=torch.uint8, device="cuda")
    full = rng.permutation(N).reshape(B, M)
    lens = rng.randint(1, M * S, size=B)
    held = np.zeros(N, dtype=np.int32)
    for b in range(B):
        full[b, ref.ceil_div(int(lens[b]), S):] = -1
    held[full[full >= 0]] = 1
    parent = _i32(np.arange(B)) if own else None

    def update(table, new):
        state = _i32(table), _i32(lens), _i32(held)
        out = tuple(torch.full_like(x, -77) for x in state)
        status = torch.zeros(4, dtype=torch.int32, device="cuda")
        kv.check(kv.ds_cache_update(pool, *state, _i32(new), *out, ws, status, parent=parent))
        return state, out, int(status[0])

    for i in range(12):
        b = int(rng.choice([0, B - 1, rng.randint(B)]))
        new = np.minimum(M * S, lens + rng.randint(0, 3, size=B))
        new[b] = [new[b], lens[b], max(0, lens[b] - 20), 0][i % 4]
        _, out, code = update(full, new)
        assert code == 0 and out[1].tolist() == new.tolist()
        last = ref.ceil_div(int(lens[b]), S) - 1
        table = full.copy()
        table[b, int(rng.choice([0, last, rng.randint(last + 1)]))] = [N, -1, 1 << 30][i % 3]
        state, out, code = update(table, new)
        assert code == 6, (i, b)
        assert all(torch.equal(x, y) for x, y in zip(state, out)), (i, b)


@pytest.mark.parametrize("N,B,held", [(1, 1, 1.0), (5, 2, 0.0), (64, 3, 0.5), (1000, 9, 0.9), (20000, 40, 0.3), (4099, 7, 1.0)])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_compact_against_the_plain_form(kv, N, B, held, layout):
    rng = np.random.RandomState(N)
    S, Hk, D, L = 16, 2, 8, 2
    pages = rng.permutation(N)[:int(round(held * N))]
    M = max(1, ref.ceil_div(len(pages), B) + 1)
    table = [[int(p) for p in pages[b::B]] for b in range(B)]
    table = [r + [-1] * (M - len(r)) for r in table]
    cnt = [0] * N
    for p in pages:
        cnt[int(p)] = int(rng.randint(1, 4))
    shape = (L, N, S, Hk, D) if layout == "nhd" else (L, N, Hk, S, D)
    k = torch.randn(shape, device="cuda")
    v = torch.randn(shape, device="cuda")
    if layout == "hnd":
        k, v = k.transpose(2, 3), v.transpose(2, 3)
    want_k, want_v = k.clone(), v.clone()
    want = ref.compact(table, cnt)
    out_t, out_r, out_m = (torch.full((B, M), -77, dtype=torch.int32, device="cuda"),
                           torch.full((N,), -77, dtype=torch.int32, device="cuda"),
                           torch.full((N,), -77, dtype=torch.int32, device="cuda"))
    used, status = _i32([-1]), torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.full((kv.ds_cache_compact_workspace_bytes(N),), 0xA5, dtype=torch.uint8, device="cuda")
    kv.check(kv.ds_cache_compact(kv.KvPool(k, v), _i32(table), _i32(cnt), out_t, out_r, out_m, used, ws, status))
    assert int(status[0]) == 0
    assert out_t.tolist() == want[0] and out_r.tolist() == want[1] and out_m.tolist() == want[2]
    assert used.tolist() == [want[3]]
    for a, z in want[4]:
        for x in (want_k, want_v):
            x[:, z] = x[:, a]
    assert torch.equal(k, want_k) and torch.equal(v, want_v)


def test_compact_refuses_negative_counts(kv):
    N, B, M = 8, 1, 4
    k = torch.randn((1, N, 16, 1, 8), device="cuda")
    before = k.clone()
    table, cnt = _i32([[6, 7, 2, -1]]), _i32([0, -1, 1, 0, 0, 0, 1, 1])
    t, r, m = torch.empty_like(table), torch.empty_like(cnt), torch.empty_like(cnt)
    used, status = _i32([0]), torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.empty(kv.ds_cache_compact_workspace_bytes(N), dtype=torch.uint8, device="cuda")
    kv.check(kv.ds_cache_compact(kv.KvPool(k, k.clone()), table, cnt, t, r, m, used, ws, status))
    assert int(status[0]) == 6
    assert torch.equal(t, table) and torch.equal(r, cnt) and torch.equal(k, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_cycles_of_a_paged_cache(kv, dtype):
    """Verify cycles through PagedCache (grow, append, attend, fall back, fork, compact) against a contiguous copy."""
    rng = np.random.RandomState(5)
    g = torch.Generator(device="cuda").manual_seed(5)
    B, Hk, G, D, S, n = 6, 2, 2, 64, 16, 5
    c = kv.PagedCache(2, 90, S, Hk, D, B, 160, dtype=DT[dtype], heads_outside=True)
    past = [[(np.zeros((0, Hk, D)), np.zeros((0, Hk, D))) for _ in range(2)] for _ in range(B)]
    q_start = _i32([n * b for b in range(B + 1)])
    for cycle in range(8):
        lens = [past[b][0][0].shape[0] for b in range(B)]
        c.update(_i32([x + n for x in lens]))
        for layer in range(2):
            kn, vn = (torch.randn((B * n, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
            q = torch.randn((B * n, Hk * G, D), device="cuda", generator=g).to(DT[dtype])
            c.append(layer, kn, vn, q_start)
            out = c.attend(layer, q, q_start, n)
            for b in range(B):
                k0, v0 = past[b][layer]
                past[b][layer] = (np.concatenate([k0, _host(kn[b * n:(b + 1) * n])]),
                                  np.concatenate([v0, _host(vn[b * n:(b + 1) * n])]))
            kk = [past[b][layer][0] for b in range(B)]
            longest = max(x.shape[0] for x in kk)
            kp, vp = np.zeros((B, longest, Hk, D)), np.zeros((B, longest, Hk, D))
            for b in range(B):
                kp[b, :kk[b].shape[0]], vp[b, :kk[b].shape[0]] = past[b][layer]
            want, _, tol, _ = ref.attend(_host(q), kp, vp, np.arange(B)[:, None], [x.shape[0] for x in kk],
                                         list(range(0, B * n + 1, n)), True, 0, ref.default_scale(D), dtype == "bf16")
            assert (np.abs(_host(out) - want) <= tol).all()
        c.check_status()
        parent = list(range(B)) if cycle % 3 else [int(rng.randint(B)) for _ in range(B)]
        keep = [len(past[p][0][0]) - int(rng.randint(0, n)) for p in parent]
        c.update(_i32(keep), parent=_i32(parent))
        past = [[(past[p][layer][0][:m], past[p][layer][1][:m]) for layer in range(2)] for p, m in zip(parent, keep)]
        if cycle % 2:
            c.compact()
            assert int(c.n_used[0]) == int((c.ref > 0).sum())
            assert (c.ref[:int(c.n_used[0])] > 0).all()
    c.check_status()


def test_attend_on_another_stream_has_that_streams_memory(kv):
    """Without `out`, a call on another stream does not write into a block that the current stream has freed and may still read."""
    H, Hk, D, n = 4, 2, 64, 50
    g = torch.Generator(device="cuda").manual_seed(21)
    c = kv.PagedCache(1, 16, 16, Hk, D, 2, 100)
    start = _i32([0, n, 2 * n])
    q, k, v = (torch.randn((2 * n, h, D), device="cuda", generator=g).to(torch.bfloat16) for h in (H, Hk, Hk))
    c.update(_i32([n, n]))
    c.append(0, k, v, start)
    want = c.attend(0, q, start, n)
    torch.cuda.synchronize()
    for how in (lambda s: s, lambda s: s.cuda_stream):
        s = torch.cuda.Stream()
        block = torch.ones_like(q)
        at = block.data_ptr()
        torch.cuda._sleep(20_000_000)
        total = block.sum()
        del block
        out = c.attend(0, q, start, n, stream=how(s))
        assert out.data_ptr() != at
        torch.cuda.synchronize()
        assert total.item() == q.numel() and torch.equal(out, want)
    c.check_status()


@pytest.mark.parametrize("dtype,outside", [("bf16", False), ("bf16", True), ("f32", False)])
def test_places_past_32_bits(kv, dtype, outside):
    """Pages more than 2^32 bytes (and 2^31 elements) into a layer: written, read, copied on write and moved."""
    N, S, Hk, D, G = 140000, 16, 8, 128, 2
    g = torch.Generator(device="cuda").manual_seed(12)
    c = kv.PagedCache(1, N, S, Hk, D, 3, 400, dtype=DT[dtype], heads_outside=outside)
    c.ref[:N - 60] = 1                    # somebody else's: new pages are the last ones
    lens = [70, 300, 0]
    c.update(_i32(lens))
    assert int(c.block_table[0, 0]) == N - 60
    T = sum(lens)
    kn, vn = (torch.randn((T, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    c.append(0, kn, vn, _i32([0, 70, 370, 370]))
    k = [kn[:70], kn[70:], kn[:70]]
    v = [vn[:70], vn[70:], vn[:70]]

    def check(n, pages):
        q = torch.randn((2 * sum(n), Hk * G, D), device="cuda", generator=g).to(DT[dtype])[::2]
        start = _i32([0, n[0], n[0] + n[1], sum(n)])
        out = c.attend(0, q, start, max(n), out=torch.empty((sum(n), Hk * G, D), dtype=DT[dtype], device="cuda"))
        c.check_status()
        held = [x.shape[0] for x in k]
        kp, vp = (np.zeros((3, max(held), Hk, D)) for _ in range(2))
        for b in range(3):
            kp[b, :held[b]], vp[b, :held[b]] = _host(k[b]), _host(v[b])
        assert c.kv_len.tolist() == held
        want, _, tol, _ = ref.attend(_host(q), kp, vp, np.arange(3)[:, None], held, start.cpu().numpy(), True, 0,
                                     ref.default_scale(D), dtype == "bf16")
        assert (np.abs(_host(out) - want) <= tol).all()
        table = c.block_table[c.block_table >= 0]
        assert pages(int(table.min()), int(table.max()))

    c.update(_i32([70, 300, 70]), parent=_i32([0, 1, 0]))
    check([3, 9, 40], lambda lo, hi: lo >= N - 60)
    c.update(_i32([75, 300, 73]))         # both write into the shared last page: one copy
    new = [torch.randn((8, Hk, D), device="cuda", generator=g).to(DT[dtype]) for _ in range(2)]
    c.append(0, new[0], new[1], _i32([0, 5, 5, 8]))
    k, v = ([torch.cat([a[0], x[:5]]), a[1], torch.cat([a[2], x[5:]])] for a, x in ((k, new[0]), (v, new[1])))
    check([1, 1, 1], lambda lo, hi: lo >= N - 60)
    c.ref[:N - 60] = 0
    c.compact()
    check([20, 1, 7], lambda lo, hi: hi < 60)
