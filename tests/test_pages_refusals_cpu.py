"""Host-side refusals of cskv_cache_compact, which return before any CUDA call."""
import ctypes

import pytest

from test_pages_cpu import FAKE, _b, _struct


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    return ck


@pytest.mark.parametrize("other", [dict(m=8), dict(n_win=64), dict(d_v=496), dict(gate_cols=1), dict(gate_cols_idx=1),
                                   dict(overlap=4)])
def test_compact_layers_agree_in_every_field(ck, other):
    """Everything but the page counts, as the header says: a layer with another fold or window is another cache."""
    L, b = ck.lib(), _b()
    for swap in (False, True):
        x, y = _struct(ck), _struct(ck, **other)
        if swap:
            x, y = y, x
        a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), FAKE, FAKE * 2, None)
        n = ctypes.c_size_t()
        assert L.cskv_compact_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.ERR_INVALID_ARG
        assert L.cskv_cache_compact(ctypes.byref(a), FAKE, 1 << 30, None) == ck.ERR_INVALID_ARG


@pytest.mark.parametrize("field,value", [("d_idx", 64), ("idx_dtype", 3), ("gate_cols_idx", 7)])
def test_compact_ignores_what_an_hca_layer_does_not_use(ck, field, value):
    b, L = _b(), ck.lib()
    hca = dict(kind=ck.LAYER_HCA, m=128, d_idx=0, gate_cols_idx=1)
    x, y = _struct(ck, **hca), _struct(ck, **dict(hca, **{field: value}))
    a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), FAKE, FAKE * 2, None)
    n = ctypes.c_size_t()
    assert L.cskv_compact_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.OK


@pytest.mark.parametrize("mine,others", [("kv_pool", "idx_pool"), ("idx_pool", "kv_pool"), ("kv_pool", "page_table"),
                                         ("page_table", "kv_pool"), ("page_table", "refs"), ("refs", "idx_pool")])
def test_compact_refuses_any_shared_buffer(ck, mine, others):
    """A buffer of dst inside another one of src."""
    L, b = ck.lib(), _b()
    for shared in (True, False):
        x, y = _struct(ck), _struct(ck, n_pages=400)
        for f in ("page_table", "kv_pool", "idx_pool"):
            setattr(y, f, getattr(y, f) + (1 << 44))
        refs = {"x": FAKE, "y": FAKE * 2}
        if shared:
            at = (refs["x"] if others == "refs" else getattr(x, others)) + 32
            if mine == "refs":
                refs["y"] = at
            else:
                setattr(y, mine, at)
        a = b.CompactArgs(ctypes.sizeof(b.CompactArgs), ctypes.pointer(x), ctypes.pointer(y), refs["x"], refs["y"], None)
        want = ck.ERR_INVALID_ARG if shared else ck.ERR_WORKSPACE  # without a workspace nothing is launched
        assert L.cskv_cache_compact(ctypes.byref(a), None, 1 << 30, None) == want
