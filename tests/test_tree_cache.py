"""Quantised pools, trees and accepted paths on the host: refusals, and the tests' own plain forms (no GPU needed)."""
import ctypes
import os

import numpy as np
import pytest

import _tree_ref as ref
from test_kv_cache import FAKE, INVALID, UNSUPPORTED, WORKSPACE, _append, _attend, _compact, _pool, _Tensor, _update

E4M3 = 2


@pytest.fixture(scope="module")
def kv():
    from speculative_decoding_draft_block_gb300 import _lib, build, kv_cache
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    kv_cache.load()
    return kv_cache


def _call(kv, name, args, scales=FAKE, tree=None):
    f = getattr(kv.load(), name)
    if name == "ds_paged_attention_tree":
        return f(ctypes.byref(args), scales, None if tree is None else ctypes.byref(tree), None)
    return f(ctypes.byref(args), scales, None) if name.endswith("_scaled") else f(ctypes.byref(args), None)


SCALED = (("ds_cache_append_scaled", _append), ("ds_paged_attention_tree", _attend), ("ds_cache_update_scaled", _update),
          ("ds_cache_compact_scaled", _compact))


@pytest.mark.parametrize("bad,scales", [(dict(), None), (dict(), FAKE + 8), (dict(dtype=1), FAKE), (dict(dtype=0), FAKE), (dict(dtype=3), FAKE),
                                        (dict(head_dim=24, head_stride=32), FAKE), (dict(head_dim=8), FAKE), (dict(token_stride=264), FAKE),
                                        (dict(head_stride=136), FAKE), (dict(k=FAKE + 8), FAKE), (dict(page_size=8), FAKE)], ids=str)
def test_bad_quantised_pools_are_refused(kv, bad, scales):
    pool = _pool(kv, **dict(dict(dtype=E4M3), **bad))
    for name, make in SCALED:
        assert _call(kv, name, make(kv, pool), scales) == INVALID
    assert _call(kv, "ds_cache_keep", _keep(kv, pool, scales=scales)) == INVALID


def test_quantised_calls_on_the_host(kv):
    lib = kv.load()
    pool = _pool(kv, dtype=E4M3)
    for name, _ in SCALED[:1] + SCALED[2:]:
        assert getattr(lib, name)(None, FAKE, None) == INVALID
    assert lib.ds_paged_attention_tree(None, FAKE, None, None) == INVALID
    for D in (64, 128):
        assert lib.ds_paged_attention_workspace_bytes(E4M3, D) == lib.ds_paged_attention_workspace_bytes(1, D)
    # no rows: nothing to do
    assert _call(kv, "ds_cache_append_scaled", _append(kv, pool, T=0)) == 0
    assert _call(kv, "ds_paged_attention_tree", _attend(kv, pool, T=0)) == 0
    # rows' strides are those of bfloat16, the pool's those of bytes
    assert _call(kv, "ds_paged_attention_tree", _attend(kv, pool, q_token_stride=1028)) == INVALID
    assert _call(kv, "ds_cache_append_scaled", _append(kv, pool, k_head_stride=132)) == INVALID
    assert _call(kv, "ds_paged_attention_tree", _attend(kv, _pool(kv, dtype=E4M3, head_dim=96, token_stride=192, head_stride=96))) == UNSUPPORTED
    assert _call(kv, "ds_paged_attention_tree", _attend(kv, pool, workspace_bytes=10)) == WORKSPACE
    # as the calls without the suffix refuse them
    for name, make in SCALED:
        assert _call(kv, name, make(kv, _pool(kv, dtype=E4M3)), None) == INVALID
        assert getattr(lib, name.replace("_scaled", "").replace("_tree", ""))(ctypes.byref(make(kv, pool)), None) == INVALID


@pytest.mark.parametrize("heads,group", [(256, 1), (255, 2), (254, 16), (256, 128)])
@pytest.mark.parametrize("max_q", [1, 300])
def test_the_longest_tables_of_many_heads_are_taken(kv, heads, group, max_q):
    """The work over a quantised pool is counted in 32 bits for any table and number of heads."""
    pool = _pool(kv, dtype=E4M3, n_kv_heads=heads, token_stride=heads * 128, page_stride=heads * 128 * 16)
    args = _attend(kv, pool, T=0, n_heads=heads * group, max_q=max_q, max_pages=(1 << 30) // pool.page_size)
    assert _call(kv, "ds_paged_attention_tree", args) == 0


@pytest.mark.parametrize("bad,args", [(dict(mask=None), {}), (dict(mask=FAKE + 2), {}), (dict(depth=FAKE + 1), {}), (dict(mask_words=0), {}),
                                      (dict(mask_words=(1 << 18) + 1), {}), (dict(mask_words=1), dict(max_q=33, T=40)), ({}, dict(causal=0))], ids=str)
def test_bad_trees_are_refused(kv, bad, args):
    for dtype, scales in ((1, None), (0, None), (E4M3, FAKE)):
        tree = kv.Tree(**dict(dict(mask=FAKE, mask_words=2, depth=FAKE), **bad))
        f = dict(q_token_stride=1024, q_head_stride=128)
        f.update(args)
        assert _call(kv, "ds_paged_attention_tree", _attend(kv, _pool(kv, dtype=dtype), **f), scales, tree) == INVALID


def test_masks_of_fewer_rows_than_max_q(kv):
    """Words are asked for the longest request that T rows can hold."""
    tree = kv.Tree(mask=FAKE, mask_words=1, depth=None)
    assert _call(kv, "ds_paged_attention_tree", _attend(kv, max_q=1000, T=0, q=None, out=None), None, tree) == 0
    assert _call(kv, "ds_tree_masks", _masks(kv, max_q=1000, T=0, mask_words=1)) == 0


def _masks(kv, **kw):
    f = dict(B=2, T=8, max_q=6, mask_words=1, window=0, parent=FAKE, q_start=FAKE + 4096, mask=FAKE + 8192, depth=FAKE + 16384, status=FAKE + 1024)
    f.update(kw)
    return kv.TreeArgs(**f)


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=65536), dict(T=-1), dict(T=(1 << 23) + 1), dict(max_q=0), dict(max_q=4097), dict(mask_words=0),
                                 dict(window=-1), dict(parent=None), dict(parent=FAKE + 2), dict(q_start=None), dict(q_start=FAKE + 4),
                                 dict(mask=None), dict(mask=FAKE + 1), dict(depth=FAKE + 3), dict(status=None), dict(status=FAKE + 8),
                                 dict(T=80, max_q=64, mask_words=1), dict(mask=FAKE + 16), dict(depth=FAKE + 28), dict(mask=FAKE + 4096 - 28),
                                 dict(depth=FAKE + 4096), dict(depth=FAKE + 8192 + 28)], ids=str)
def test_bad_mask_calls_are_refused(kv, bad):
    assert kv.load().ds_tree_masks(None, None) == INVALID
    assert _call(kv, "ds_tree_masks", _masks(kv, **bad)) == INVALID


def _keep(kv, pool=None, **kw):
    f = dict(B=4, T=8, max_pages=10, path_len=5, path=FAKE, q_start=FAKE + 4096, block_table=FAKE + 8192, kv_len=FAKE + 12288,
             new_len=FAKE + 16384, scales=None, status=FAKE + 20480)
    f.update(kw)
    return kv.KeepArgs(pool=pool or _pool(kv), **f)


@pytest.mark.parametrize("bad", [dict(B=0), dict(T=-1), dict(max_pages=0), dict(path_len=0), dict(path_len=4097), dict(path=None),
                                 dict(q_start=FAKE + 8), dict(block_table=None), dict(kv_len=None), dict(new_len=None), dict(status=None),
                                 dict(new_len=FAKE + 64), dict(new_len=FAKE + 12288), dict(new_len=FAKE + 4096 + 16),
                                 dict(new_len=FAKE + 8192 + 144), dict(scales=FAKE)], ids=str)
def test_bad_keep_calls_are_refused(kv, bad):
    assert kv.load().ds_cache_keep(None, None) == INVALID
    assert _call(kv, "ds_cache_keep", _keep(kv, **bad)) == INVALID


def test_quantised_pools_of_the_binding(kv):
    torch = pytest.importorskip("torch")
    e = torch.zeros((1, 4, 16, 2, 64), dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        kv.KvPool(e, e, torch.zeros((1, 4, 2, 2, 16), dtype=torch.uint8))         # not CUDA tensors

    def t(shape, dtype, device=0):
        return _Tensor(torch, shape, dtype, device)

    class Pool(_Tensor):
        @property
        def device(self):
            return torch.device("cuda", self.device_index)

    def k(dtype):
        return Pool(torch, (1, 4, 16, 2, 64), dtype, 0)

    def s(shape=(1, 4, 2, 2, 16), dtype=torch.uint8, device=0):
        return Pool(torch, shape, dtype, device)

    pool = kv.KvPool(k(torch.float8_e4m3fn), k(torch.float8_e4m3fn), s())
    assert pool.dtype is torch.bfloat16 and pool.desc.dtype == E4M3
    for args in ((k(torch.float8_e4m3fn), k(torch.float8_e4m3fn)), (k(torch.bfloat16), k(torch.bfloat16), s()),
                 (k(torch.float8_e4m3fn), k(torch.float8_e4m3fn), s((1, 4, 2, 16, 2))),
                 (k(torch.float8_e4m3fn), k(torch.float8_e4m3fn), s(dtype=torch.int8)),
                 (k(torch.float8_e4m3fn), k(torch.float8_e4m3fn), s(device=1))):
        with pytest.raises(ValueError):
            kv.KvPool(*args)


def test_binding_chooses_the_call_and_refuses_bad_arguments(kv, monkeypatch):
    """Which C call a pool and a mask lead to, and what is refused before any."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    B, M, N, T, H, Hk, D = 2, 3, 8, 5, 4, 2, 64
    called = []
    monkeypatch.setattr(kv, "_entry", lambda name: lambda *args: called.append((name, len(args))) or 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)

    def t(shape, dtype=torch.int32, device=0):
        return _Tensor(torch, shape, dtype, device)

    def pool(scales):
        return SimpleNamespace(packed=bytes(ctypes.sizeof(kv.PoolDesc)), device_index=0, dtype=torch.bfloat16, n_pages=N,
                               n_kv_heads=Hk, head_dim=D, scales=t((1, N, 2, Hk, 16), torch.uint8) if scales else None)

    bf = torch.bfloat16
    w = dict(q_start=t((B + 1,)), block_table=t((B, M)), kv_len=t((B,)), status=t((4,)))

    def attend(p, **kw):
        return kv.ds_paged_attention(p, 0, t((T, H, D), bf), max_q=3, out=t((T, H, D), bf), workspace=t((64,), torch.uint8), **w, **kw)

    def keep(p, **kw):
        return kv.ds_cache_keep(p, **dict(dict(path=t((B, 4)), new_len=t((B,)), **w), **kw))

    def masks(**kw):
        f = dict(dict(parent=t((T,)), q_start=t((B + 1,)), max_q=3, mask=t((T, 1)), depth=t((T,)), status=t((4,))), **kw)
        return kv.ds_tree_masks(f.pop("parent"), f.pop("q_start"), f.pop("max_q"), f.pop("mask"), f.pop("depth"), f.pop("status"), **f)

    for q in (False, True):
        p = pool(q)
        kv.ds_cache_append(p, 0, t((T, Hk, D), bf), t((T, Hk, D), bf), **w)
        attend(p)
        attend(p, mask=t((T, 1)), depth=t((T,)))
        kv.ds_cache_update(p, w["block_table"], w["kv_len"], t((N,)), t((B,)), t((B, M)), t((B,)), t((N,)), t((64,), torch.uint8), w["status"])
        kv.ds_cache_compact(p, w["block_table"], t((N,)), t((B, M)), t((N,)), t((N,)), t((1,)), t((64,), torch.uint8), w["status"])
        keep(p)
        masks()
    plain = [("ds_cache_append", 2), ("ds_paged_attention", 2), ("ds_paged_attention_tree", 4), ("ds_cache_update", 2), ("ds_cache_compact", 2),
             ("ds_cache_keep", 2), ("ds_tree_masks", 2)]
    scaled = [("ds_cache_append_scaled", 3), ("ds_paged_attention_tree", 4), ("ds_paged_attention_tree", 4), ("ds_cache_update_scaled", 3),
              ("ds_cache_compact_scaled", 3), ("ds_cache_keep", 2), ("ds_tree_masks", 2)]
    assert called == plain + scaled
    for bad in (dict(mask=t((T,))), dict(mask=t((T + 1, 1))), dict(mask=t((T, 1), torch.int64)), dict(mask=t((T, 1), device=1)),
                dict(depth=t((T,))), dict(mask=t((T, 1)), depth=t((T + 1,))), dict(mask=t((T, 1)), depth=t((T,), torch.int64))):
        with pytest.raises(ValueError):
            attend(pool(False), **bad)
    for bad in (dict(path=t((B + 1, 4))), dict(path=t((B,))), dict(path=t((B, 4), torch.int64)), dict(new_len=t((B + 1,))), dict(kv_len=t((B,), device=1))):
        with pytest.raises(ValueError):
            keep(pool(False), **bad)
    for bad in (dict(parent=t((T, 1))), dict(parent=t((T,), device=-1)), dict(mask=t((T + 1, 1))), dict(mask=t((T, 1), device=1)), dict(depth=t((T + 1,))),
                dict(q_start=t((1,))), dict(status=t((4,), torch.int64))):
        with pytest.raises(ValueError):
            masks(**bad)
    with pytest.raises(ValueError, match="current device"):
        masks(parent=t((T,), device=1), q_start=t((B + 1,), device=1), mask=t((T, 1), device=1), depth=None, status=t((4,), device=1))
    assert len(called) == 14


def test_plain_forms_agree_with_hand_made_states():
    """The tests' own reference on states small enough to check by hand."""
    torch = pytest.importorskip("torch")
    # every e4m3 number is its own code; half-way values go to the even neighbour, as torch's conversion does
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    codes = codes[torch.isfinite(codes)]
    x = torch.cat([codes, (codes[1:126] + codes[:125]) / 2, torch.tensor([448.0])])
    y, e = ref.quantise(x.numpy())
    assert e == 0 and np.array_equal(y, x.float().to(torch.float8_e4m3fn).double().numpy())
    _, e = ref.quantise(np.array([[448.0], [449.0], [224.0], [0.0], [2.0 ** -100 * 448], [2.0 ** -100], [np.inf], [np.nan]]))
    assert e.tolist() == [0, 1, -1, -100, -100, -100, 128, 128]
    assert ref.restored(np.array([[1.5, -2.0]]), [130]).tolist() == [[12.0, -16.0]] and np.isnan(ref.restored(np.zeros((1, 2)), [255])).all()
    a, d = ref.ancestors([-1, 0, 0, 2, -1])
    assert d.tolist() == [0, 1, 1, 2, 0]
    assert a.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 0, 1, 1, 0], [0, 0, 0, 0, 1]]
    assert ref.ancestors([-1, 0, 0, 2, -1], 2)[0][3].astype(int).tolist() == [0, 0, 1, 1, 0]
    assert ref.words(a, 1).tolist() == [[1], [3], [5], [13], [16]]
    assert ref.tree_seen(a, d, 5, 7, 0)[3].astype(int).tolist() == [1, 1, 1, 0, 1, 1, 0]
    assert ref.tree_seen(ref.ancestors([-1, 0, 0, 2, -1], 3)[0], d, 5, 7, 3)[3].astype(int).tolist() == [0, 0, 1, 0, 1, 1, 0]
    assert ref.keep(list("abcde"), [1, 2, -1, 0], 3, 5) == (["a", "b", "d", "e", "e"], 4)
    assert ref.keep(list("abcde"), [1, 1], 3, 5) is None and ref.keep(list("ab"), [0], 3, 2) is None
    assert ref.keep(list("abc"), [0, 3], 3, 3) is None
    assert (ref.causal_seen(2, 4, True, 2) == np.array([[0, 1, 1, 0], [0, 0, 1, 1]], bool)).all()
