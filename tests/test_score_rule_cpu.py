"""Host-side checks of the score rule's arguments, which return before any CUDA call."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    return ck


def _args(ck, **kw):
    from compressed_sparse_kv_02_b200 import _binding as b
    layer = ck.Layer(kind=ck.LAYER_HCA, m=128, n_win=128, d_qk=576, d_v=512, d_idx=0, page_size=64, kv_dtype=ck.BF16,
                     idx_dtype=ck.BF16, gate_cols=1, gate_cols_idx=1, n_seqs=8, max_pages_per_seq=64, n_pages=512)
    return b._attend_args(layer, None, None, 1000, None, None, None, 0, None, None, None, None, 0, None, n_q=4,
                          n_heads=64, **kw)


@pytest.mark.parametrize("cap", [-1.0, -1e-30, math.nan, math.inf, -math.inf, 3e38, 2.0 ** 101, 2.0 ** -101, 1e-45])
def test_bad_caps_are_refused(ck, cap):
    a = _args(ck, score_cap=cap)
    n = ctypes.c_size_t()
    assert ck.lib().cskv_attend_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.ERR_INVALID_ARG
    assert ck.lib().hca_attend(ctypes.byref(a), None, 0, None) == ck.ERR_INVALID_ARG


def test_callers_without_the_fields(ck):
    """A struct that ends before the rule gets none, whatever lies behind it."""
    from compressed_sparse_kv_02_b200 import _binding as b
    n = ctypes.c_size_t()
    a = _args(ck, score_cap=-1.0)
    a.struct_size = b.AttendArgs.score_cap.offset
    assert ck.lib().cskv_attend_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.OK
    plain = n.value
    a = _args(ck, score_cap=20.0)
    assert ck.lib().cskv_attend_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.OK
    assert n.value == plain  # the query covers both forms


def test_workspace_covers_the_split_kernel_behind_the_tensor_core_kernel(ck):
    """Where the two forms take different kernels, the query gives the larger need, and grows with the queries."""
    layer = ck.Layer(kind=ck.LAYER_HCA, m=128, n_win=128, d_qk=576, d_v=512, d_idx=0, page_size=64,
                     kv_dtype=ck.FP8_E4M3, idx_dtype=ck.BF16, gate_cols=1, gate_cols_idx=1, n_seqs=8,
                     max_pages_per_seq=64, n_pages=512)
    sizes = [ck.cskv_attend_ws_bytes(layer, n, 64, 4000) for n in (100, 111, 112, 150, 175, 176, 300)]
    assert all(s > 0 for s in sizes)


@pytest.mark.parametrize("sm_scale,cap", [(2.0 ** -30, 2.0 ** 100), (2.0 ** 40, 2.0 ** -90), (2.0 ** -121, 1.0), (3e38, 1.0)])
def test_scales_beyond_the_cap_are_refused(ck, sm_scale, cap):
    """sm_scale / score_cap outside 2^-120 .. 2^120."""
    a = _args(ck, score_cap=cap)
    a.sm_scale = sm_scale
    n = ctypes.c_size_t()
    assert ck.lib().cskv_attend_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.ERR_INVALID_ARG
    assert ck.lib().hca_attend(ctypes.byref(a), None, 0, None) == ck.ERR_INVALID_ARG
    a.score_cap = 0.0
    assert ck.lib().cskv_attend_ws_bytes(ctypes.byref(a), ctypes.byref(n)) == ck.OK
