"""Host-side checks of the page operators, which return before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    return ck


def _struct(ck, **kw):
    base = dict(kind=ck.LAYER_CSA, m=4, n_win=128, d_qk=576, d_v=512, d_idx=128, page_size=64, kv_dtype=ck.BF16,
                idx_dtype=ck.BF16, gate_cols=576, gate_cols_idx=128, n_seqs=8, max_pages_per_seq=64, n_pages=512)
    base.update(kw)
    s = ck.Layer(**base).struct
    # addresses that no call below follows
    for i, f in enumerate(("page_table", "kv_pool", "idx_pool", "ring_x", "ring_z", "ring_xi", "ring_zi")):
        setattr(s, f, (i + 1) << 40)
    return s


def _b():
    from compressed_sparse_kv_02_b200 import _binding as b
    return b


FAKE = 1 << 46


def test_null_and_short_structs(ck):
    L, b = ck.lib(), _b()
    for f in (L.cskv_cache_fork, L.cskv_cache_free):
        assert f(None, None) == ck.ERR_INVALID_ARG
    for f in (L.cskv_cache_reserve, L.cskv_cache_compact):
        assert f(None, None, 0, None) == ck.ERR_INVALID_ARG
    s = _struct(ck)
    p = ctypes.pointer(s)
    for a, f in ((b.ForkArgs(0, p, FAKE, 1, FAKE, FAKE, FAKE, None), L.cskv_cache_fork),
                 (b.FreeArgs(0, p, FAKE, 1, FAKE, FAKE, None), L.cskv_cache_free)):
        for size in (0, ctypes.sizeof(a) - 8):
            a.struct_size = size
            assert f(ctypes.byref(a), None) == ck.ERR_INVALID_ARG
    a = b.ReserveArgs(ctypes.sizeof(b.ReserveArgs) - 8, p, FAKE, 1, FAKE, FAKE, FAKE, 1, None)
    assert L.cskv_cache_reserve(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG


def test_missing_buffers(ck):
    L, b = ck.lib(), _b()
    p = ctypes.pointer(_struct(ck))
    size = ctypes.sizeof
    for i in range(4):
        v = [FAKE] * 4
        v[i] = None
        a = b.ForkArgs(size(b.ForkArgs), p, v[0], 1, v[1], v[2], v[3], None)
        assert L.cskv_cache_fork(ctypes.byref(a), None) == ck.ERR_INVALID_ARG
        a = b.ReserveArgs(size(b.ReserveArgs), p, v[0], 1, v[1], v[2], v[3], 1, None)
        assert L.cskv_cache_reserve(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG
    for i in range(3):
        v = [FAKE] * 3
        v[i] = None
        a = b.FreeArgs(size(b.FreeArgs), p, v[0], 1, v[1], v[2], None)
        assert L.cskv_cache_free(ctypes.byref(a), None) == ck.ERR_INVALID_ARG
    for f in ("page_table", "kv_pool", "idx_pool"):
        s = _struct(ck)
        setattr(s, f, None)
        a = b.ReserveArgs(size(b.ReserveArgs), ctypes.pointer(s), FAKE, 1, FAKE, FAKE, FAKE, 1, None)
        assert L.cskv_cache_reserve(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG
    # unaligned counts and pools
    a = b.ReserveArgs(size(b.ReserveArgs), p, FAKE + 4, 1, FAKE, FAKE, FAKE, 1, None)
    assert L.cskv_cache_reserve(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG
    s = _struct(ck)
    s.idx_pool += 8
    a = b.ForkArgs(size(b.ForkArgs), ctypes.pointer(s), FAKE, 1, FAKE, FAKE, FAKE, None)
    assert L.cskv_cache_fork(ctypes.byref(a), None) == ck.ERR_INVALID_ARG


def test_counts_and_workspaces(ck):
    L, b = ck.lib(), _b()
    layer = ck.Layer(kind=ck.LAYER_HCA, m=128, n_win=128, d_qk=128, d_v=128, d_idx=0, page_size=64, kv_dtype=ck.BF16,
                     idx_dtype=ck.BF16, gate_cols=128, gate_cols_idx=1, n_seqs=8, max_pages_per_seq=64, n_pages=512)
    small, large = ck.cskv_reserve_ws_bytes(layer, 1, 1), ck.cskv_reserve_ws_bytes(layer, 8, 64 * 64)
    assert 0 < small <= large
    for n, most in ((-1, 1), (1, -1), (4097, 1), (1, 1 << 60)):
        with pytest.raises(ck.CskvError):
            ck.cskv_reserve_ws_bytes(layer, n, most)
    s = _struct(ck)
    a = b.ReserveArgs(ctypes.sizeof(b.ReserveArgs), ctypes.pointer(s), FAKE, 4, FAKE, FAKE, FAKE, 100, None)
    n = ctypes.c_size_t()
    assert L.cskv_reserve_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.OK
    for ws, size in ((None, n.value), (FAKE, n.value - 1), (FAKE + 8, n.value)):
        assert L.cskv_cache_reserve(ctypes.byref(a), ws, size, None) == ck.ERR_WORKSPACE
    for n_list in (-1, 4097):
        f = b.ForkArgs(ctypes.sizeof(b.ForkArgs), ctypes.pointer(s), FAKE, n_list, FAKE, FAKE, FAKE, None)
        assert L.cskv_cache_fork(ctypes.byref(f), None) in (ck.ERR_INVALID_ARG, ck.ERR_UNSUPPORTED)
        f = b.FreeArgs(ctypes.sizeof(b.FreeArgs), ctypes.pointer(s), FAKE, n_list, FAKE, FAKE, None)
        assert L.cskv_cache_free(ctypes.byref(f), None) in (ck.ERR_INVALID_ARG, ck.ERR_UNSUPPORTED)


def test_empty_lists_are_nothing_to_do(ck):
    L, b = ck.lib(), _b()
    p = ctypes.pointer(_struct(ck))
    a = b.ForkArgs(ctypes.sizeof(b.ForkArgs), p, FAKE, 0, None, None, None, None)
    assert L.cskv_cache_fork(ctypes.byref(a), None) == ck.OK
    a = b.FreeArgs(ctypes.sizeof(b.FreeArgs), p, FAKE, 0, None, None, None)
    assert L.cskv_cache_free(ctypes.byref(a), None) == ck.OK
    a = b.ReserveArgs(ctypes.sizeof(b.ReserveArgs), p, FAKE, 0, None, None, None, 1, None)
    assert L.cskv_cache_reserve(ctypes.byref(a), None, 0, None) == ck.OK


@pytest.mark.parametrize("other", [dict(page_size=32), dict(d_qk=592), dict(kv_dtype=2), dict(idx_dtype=3),
                                   dict(d_idx=64, gate_cols_idx=64), dict(n_seqs=7), dict(max_pages_per_seq=63),
                                   dict(kind=1)])
def test_compact_layers_must_agree(ck, other):
    L, b = ck.lib(), _b()
    x, y = _struct(ck), _struct(ck, **(dict(gate_cols=other["d_qk"], **other) if "d_qk" in other else other))
    a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), FAKE, FAKE * 2, None)
    n = ctypes.c_size_t()
    assert L.cskv_compact_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.ERR_INVALID_ARG
    assert L.cskv_cache_compact(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG


def test_compact_refuses_shared_buffers(ck):
    L, b = ck.lib(), _b()
    far = 1 << 44

    def pair(**same):
        x, y = _struct(ck), _struct(ck, n_pages=400)
        for f in ("page_table", "kv_pool", "idx_pool"):
            if f not in same:
                setattr(y, f, getattr(y, f) + far)
            else:
                setattr(y, f, getattr(x, f) + same[f])
        return x, y

    for same, refs in ((dict(page_table=0), FAKE * 2), (dict(kv_pool=512 * 64 * 576 * 2 - 16), FAKE * 2),
                       (dict(idx_pool=16), FAKE * 2), (dict(), FAKE)):
        x, y = pair(**same)
        a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), FAKE, refs, None)
        assert L.cskv_cache_compact(ctypes.byref(a), FAKE * 4, 1 << 30, None) == ck.ERR_INVALID_ARG
    x, y = pair()
    a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), FAKE, FAKE * 2, None)
    assert L.cskv_cache_compact(ctypes.byref(a), None, 1 << 30, None) == ck.ERR_WORKSPACE
    assert L.cskv_cache_compact(ctypes.byref(a), FAKE * 4, 8, None) == ck.ERR_WORKSPACE
