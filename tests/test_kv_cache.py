"""The paged cache's C ABI on the host: exports, sizes and refusals (no GPU needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20          # an aligned address that is never read
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def kv():
    from speculative_decoding_draft_block_gb300 import _lib, build, kv_cache
    if not os.path.exists(_lib.LIB_PATH):
        build.build()
    kv_cache.load()
    return kv_cache


def test_header_declares_the_binding_exports(kv):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ds_cache.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(ds_[a-z0-9_]+)\s*\(", src))) == sorted(kv.EXPORTS)
    for name in kv.EXPORTS:
        assert hasattr(kv.load(), name)


def _pool(kv, **kw):
    f = dict(dtype=1, n_layers=2, n_pages=100, page_size=16, n_kv_heads=2, head_dim=128, k=FAKE, v=FAKE,
             layer_stride=100 * 16 * 256, page_stride=16 * 256, token_stride=256, head_stride=128)
    f.update(kw)
    return kv.PoolDesc(**f)


def _attend(kv, pool=None, **kw):
    f = dict(layer=0, B=4, T=8, max_pages=10, max_q=2, n_heads=8, causal=1, window=0, scale=0.1, q=FAKE,
             q_token_stride=1024, q_head_stride=128, q_start=FAKE, block_table=FAKE, kv_len=FAKE, out=FAKE,
             out_token_stride=1024, out_head_stride=128, lse=None, workspace=FAKE, workspace_bytes=1 << 40, status=FAKE)
    f.update(kw)
    return kv.AttentionArgs(pool=pool or _pool(kv), **f)


def _append(kv, pool=None, **kw):
    f = dict(layer=0, B=4, T=8, max_pages=10, k_new=FAKE, v_new=FAKE, k_token_stride=256, k_head_stride=128,
             v_token_stride=256, v_head_stride=128, q_start=FAKE, block_table=FAKE, kv_len=FAKE, status=FAKE)
    f.update(kw)
    return kv.AppendArgs(pool=pool or _pool(kv), **f)


def _update(kv, pool=None, **kw):
    f = dict(B=4, max_pages=10, block_table=FAKE, kv_len=FAKE + 4096, ref=FAKE + 8192, parent=None, new_len=FAKE + 12288,
             table_out=FAKE + 16384, len_out=FAKE + 20480, ref_out=FAKE + 24576, workspace=FAKE, workspace_bytes=1 << 40,
             status=FAKE)
    f.update(kw)
    return kv.UpdateArgs(pool=pool or _pool(kv), **f)


def _compact(kv, pool=None, **kw):
    f = dict(B=4, max_pages=10, block_table=FAKE, ref=FAKE + 4096, table_out=FAKE + 8192, ref_out=FAKE + 12288,
             page_map=FAKE + 16384, n_used=FAKE + 20480, workspace=FAKE, workspace_bytes=1 << 40, status=FAKE)
    f.update(kw)
    return kv.CompactArgs(pool=pool or _pool(kv), **f)


BAD_POOLS = [dict(dtype=2), dict(n_layers=0), dict(n_pages=0), dict(n_pages=(1 << 28) + 1), dict(page_size=8),
             dict(page_size=48), dict(page_size=512), dict(n_kv_heads=0), dict(n_kv_heads=257), dict(head_dim=4),
             dict(head_dim=12), dict(head_dim=264), dict(k=None), dict(v=FAKE + 8), dict(page_stride=100), dict(page_stride=-8),
             dict(token_stride=130), dict(token_stride=64), dict(head_stride=0), dict(layer_stride=12), dict(layer_stride=-1024)]


@pytest.mark.parametrize("bad", BAD_POOLS, ids=str)
def test_bad_pools_are_refused(kv, bad):
    lib = kv.load()
    pool = _pool(kv, **bad)
    for fn, make in ((lib.ds_cache_append, _append), (lib.ds_paged_attention, _attend), (lib.ds_cache_update, _update),
                     (lib.ds_cache_compact, _compact)):
        assert fn(ctypes.byref(make(kv, pool)), None) == INVALID


@pytest.mark.parametrize("bad,code", [
    (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(B=0), INVALID), (dict(B=65536), INVALID), (dict(T=-1), INVALID),
    (dict(max_pages=0), INVALID), (dict(max_pages=1 << 28), INVALID), (dict(max_q=0), INVALID), (dict(n_heads=0), INVALID),
    (dict(n_heads=3), INVALID), (dict(n_heads=258), INVALID), (dict(causal=2), INVALID), (dict(window=-1), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(q=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(out=None), INVALID),
    (dict(q_token_stride=1028), INVALID), (dict(out_head_stride=0), INVALID), (dict(q_start=None), INVALID),
    (dict(block_table=FAKE + 4), INVALID), (dict(kv_len=None), INVALID), (dict(lse=FAKE + 2), INVALID),
    (dict(status=None), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace=FAKE + 8), WORKSPACE),
    (dict(workspace_bytes=100), WORKSPACE)], ids=str)
def test_bad_attention_calls_are_refused(kv, bad, code):
    assert kv.load().ds_paged_attention(ctypes.byref(_attend(kv, **bad)), None) == code


def test_attention_head_dims(kv):
    lib = kv.load()
    assert lib.ds_paged_attention(None, None) == INVALID
    for D in (8, 96, 256):
        assert lib.ds_paged_attention(ctypes.byref(_attend(kv, _pool(kv, head_dim=D, head_stride=256, token_stride=512))), None) == UNSUPPORTED
        assert lib.ds_paged_attention_workspace_bytes(1, D) == 0
    assert lib.ds_paged_attention_workspace_bytes(7, 128) == 0
    for dtype in (0, 1):
        for D in (64, 128):
            assert lib.ds_paged_attention_workspace_bytes(dtype, D) > 0
    # no rows: nothing to do, nothing launched (also without a device)
    assert lib.ds_paged_attention(ctypes.byref(_attend(kv, T=0, q=None, out=None)), None) == 0


def test_layers_of_a_pool(kv):
    """2^28 layers at most (twice their number is counted in 32 bits)."""
    lib = kv.load()
    for L, code in ((1 << 28, 0), ((1 << 28) + 1, INVALID), (2 ** 31 - 1, INVALID)):
        pool = _pool(kv, n_layers=L)
        assert lib.ds_cache_append(ctypes.byref(_append(kv, pool, T=0)), None) == code
        assert lib.ds_paged_attention(ctypes.byref(_attend(kv, pool, T=0)), None) == code
        if code:
            assert lib.ds_cache_update(ctypes.byref(_update(kv, pool)), None) == code
            assert lib.ds_cache_compact(ctypes.byref(_compact(kv, pool)), None) == code


def test_attention_work_that_passes_32_bits(kv):
    """Tiles of a block of rows times KV heads: 2^24 + 1 tiles of 64 keys and 256 heads are 2^32 + 256. (No rows: what
    is not refused launches nothing.)"""
    call = kv.load().ds_paged_attention
    for dtype, heads, tokens, code in ((0, 256, 1 << 30, UNSUPPORTED), (0, 255, 1 << 30, 0), (0, 256, (1 << 30) - 128, 0),
                                       (0, 256, (1 << 30) - 16, UNSUPPORTED), (1, 256, 1 << 30, 0)):
        pool = _pool(kv, dtype=dtype, n_kv_heads=heads, head_dim=64)
        args = _attend(kv, pool, n_heads=heads, max_pages=tokens // 16, T=0, q=None, out=None)
        assert call(ctypes.byref(args), None) == code, (dtype, heads, tokens)


@pytest.mark.parametrize("bad", [dict(layer=2), dict(B=0), dict(T=-1), dict(max_pages=0), dict(k_new=None), dict(v_new=FAKE + 4),
                                 dict(k_token_stride=129), dict(v_head_stride=0), dict(q_start=None), dict(block_table=None),
                                 dict(kv_len=FAKE + 8), dict(status=None)], ids=str)
def test_bad_appends_are_refused(kv, bad):
    assert kv.load().ds_cache_append(ctypes.byref(_append(kv, **bad)), None) == INVALID


def test_append_of_nothing(kv):
    assert kv.load().ds_cache_append(None, None) == INVALID
    assert kv.load().ds_cache_append(ctypes.byref(_append(kv, T=0, k_new=None, v_new=None)), None) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), INVALID), (dict(max_pages=0), INVALID), (dict(block_table=None), INVALID), (dict(new_len=None), INVALID),
    (dict(parent=FAKE + 8), INVALID), (dict(table_out=None), INVALID), (dict(table_out=FAKE), INVALID),
    (dict(len_out=FAKE + 4096), INVALID), (dict(ref_out=FAKE + 8192 + 16), INVALID), (dict(len_out=FAKE + 12288), INVALID),
    (dict(len_out=FAKE + 16384), INVALID), (dict(parent=FAKE + 24576), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=64), WORKSPACE), (dict(status=FAKE + 4), INVALID)], ids=str)
def test_bad_updates_are_refused(kv, bad, code):
    assert kv.load().ds_cache_update(None, None) == INVALID
    assert kv.load().ds_cache_update(ctypes.byref(_update(kv, **bad)), None) == code


@pytest.mark.parametrize("bad,code", [
    (dict(B=0), INVALID), (dict(block_table=None), INVALID), (dict(ref=None), INVALID), (dict(table_out=FAKE + 16), INVALID),
    (dict(ref_out=FAKE + 4096), INVALID), (dict(page_map=FAKE + 12288), INVALID), (dict(n_used=None), INVALID),
    (dict(n_used=FAKE + 16384), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE)], ids=str)
def test_bad_compactions_are_refused(kv, bad, code):
    assert kv.load().ds_cache_compact(None, None) == INVALID
    assert kv.load().ds_cache_compact(ctypes.byref(_compact(kv, **bad)), None) == code


def test_status_texts_name_the_cache(kv):
    text = kv._lib.ds_status_string
    assert "page" in text(6) and "token" in text(6) and "page" in text(8)


def test_workspace_sizes(kv):
    lib = kv.load()
    assert lib.ds_cache_update_workspace_bytes(128, 1000) >= 4 * (4 * 1000 + 2 * 128)
    assert lib.ds_cache_update_workspace_bytes(0, 10) == 0
    assert lib.ds_cache_update_workspace_bytes(65536, 10) == 0
    assert lib.ds_cache_update_workspace_bytes(1, 0) == 0
    assert lib.ds_cache_compact_workspace_bytes(1000) >= 4 * 2 * 500
    assert lib.ds_cache_compact_workspace_bytes(0) == 0


def test_binding_refuses_what_is_no_device_tensor(kv):
    torch = pytest.importorskip("torch")
    k = torch.zeros((1, 4, 16, 2, 64))
    with pytest.raises(ValueError):
        kv.KvPool(k, k.clone())                               # host memory
    with pytest.raises(ValueError):
        kv.KvPool(k, torch.zeros((1, 4, 16, 2, 32)))          # shapes differ
    with pytest.raises(ValueError):
        kv._words(torch.zeros(3), "lengths")                  # not int32


class _Tensor:
    """What the binding asks of a tensor, on a device of choice (its address is never read)."""
    is_cuda = True

    def __init__(self, torch, shape, dtype, device):
        self.meta, self.dtype, self.shape, self.device_index = torch.empty(shape, device="meta"), dtype, torch.Size(shape), device

    def __getattr__(self, name):
        return getattr(self.meta, name)

    def get_device(self):
        return self.device_index

    def data_ptr(self):
        return FAKE


def test_binding_refuses_other_devices(kv, monkeypatch):
    """A pool beside the current device, or an argument beside the pool's device, is refused before anything is called."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    B, M, N, T, H, Hk, D = 2, 3, 8, 5, 4, 2, 64

    def calls(pool_device, odd=None):
        def t(name, shape, dtype=torch.int32):
            return _Tensor(torch, shape, dtype, 1 - pool_device if name == odd else pool_device)

        pool = SimpleNamespace(packed=bytes(kv.ctypes.sizeof(kv.PoolDesc)), device_index=pool_device, dtype=torch.bfloat16, n_pages=N,
                               n_kv_heads=Hk, head_dim=D)
        bf = torch.bfloat16
        w = dict(q_start=t("q_start", (B + 1,)), block_table=t("block_table", (B, M)), kv_len=t("kv_len", (B,)))
        status, ws = t("status", (4,)), t("workspace", (64,), torch.uint8)
        table_out, ref = t("table_out", (B, M)), t("ref", (N,))
        return {"append": lambda: kv.ds_cache_append(pool, 0, t("k_new", (T, Hk, D), bf), t("v_new", (T, Hk, D), bf), status=status, **w),
                "attention": lambda: kv.ds_paged_attention(pool, 0, t("q", (T, H, D), bf), max_q=3, out=t("out", (T, H, D), bf), status=status,
                                                           workspace=ws, lse=t("lse", (T, H), torch.float32), **w),
                "update": lambda: kv.ds_cache_update(pool, w["block_table"], w["kv_len"], ref, t("new_len", (B,)), table_out,
                                                     t("len_out", (B,)), t("ref_out", (N,)), ws, status, parent=t("parent", (B,))),
                "compact": lambda: kv.ds_cache_compact(pool, w["block_table"], ref, table_out, t("ref_out", (N,)), t("page_map", (N,)),
                                                       t("n_used", (1,)), ws, status)}

    called = []
    monkeypatch.setattr(kv, "_entry", lambda name: lambda args, stream: called.append(name) or 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    for f in calls(0).values():
        assert f() == 0
    assert len(called) == 4
    for f in calls(1).values():                                # the pool is on another device than the current one
        with pytest.raises(ValueError, match="current device"):
            f()
    odd = {"append": ("k_new", "v_new"), "attention": ("q", "out", "lse", "workspace"),
           "update": ("new_len", "parent", "table_out", "len_out", "ref", "ref_out", "workspace"),
           "compact": ("ref", "table_out", "ref_out", "page_map", "n_used", "workspace")}
    for call, names in odd.items():
        for name in names + ("block_table", "status") + (("q_start", "kv_len") if call in ("append", "attention") else ()):
            with pytest.raises(ValueError, match=name):
                calls(0, name)[call]()
    assert len(called) == 4


def test_plain_forms_agree_with_hand_made_states():
    """The tests' own reference on states small enough to check by hand."""
    import _kv_ref as ref
    # two requests share pages 0 and 1 (page 1 partly filled); both grow: the lower one keeps page 1
    t, n, r, c = ref.update([[0, 1, -1], [0, 1, -1]], [20, 20], [2, 2, 0, 0], [21, 33], None, 16, 4)
    assert t == [[0, 1, -1], [0, 2, 3]] and n == [21, 33] and r == [2, 1, 1, 1] and c == {1: (1, 2, 4)}
    # a holder that does not write makes every writer copy
    t, n, r, c = ref.update([[0], [0]], [5, 5], [2, 0, 0], [6, 5], None, 16, 3)
    assert t == [[1], [0]] and r == [1, 1, 0] and c == {0: (0, 1, 5)}
    # the end of request 0 frees what request 1 takes; fork from it first
    t, n, r, c = ref.update([[2], [-1]], [16, 0], [0, 0, 1], [0, 16], [-1, 0], 16, 3)
    assert t == [[-1], [2]] and r == [0, 0, 1] and c == {}
    assert ref.update([[0], [-1]], [16, 0], [1, 0], [16, 32], None, 16, 2) is None
    assert ref.compact([[4, 1], [-1, -1]], [0, 2, 0, 0, 1]) == ([[0, 1], [-1, -1]], [1, 2, 0, 0, 0], [-1, 1, -1, -1, 0], 2, [(4, 0)])
