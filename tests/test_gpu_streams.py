"""GPU tests of calls given another stream than the current one: the temporary workspace of a call without one stays
its own until that stream has run the call."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ck


def _attend(ck):
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, 128, 128, 1, 40, 40, gate_cols=1)
    L.set_pages(0, torch.arange(40))
    L.kv_pool.copy_(torch.randn(L.kv_pool.shape, device="cuda"))
    n, t = 4, 128 * 64 * 39
    q = torch.randn(n, 32, 128, device="cuda").to(torch.bfloat16)
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), t, dtype=torch.int64, device="cuda")
    out = torch.zeros(n, 32, 128, dtype=torch.bfloat16, device="cuda")
    return (lambda **kw: ck.hca_attend(L, seq, pos, t, q, out, score_cap=30.0, **kw)), out, \
        ck.cskv_attend_ws_bytes(L, n, 32, t)


def _select(ck):
    L = ck.Layer.allocate(ck.LAYER_CSA, 4, 128, 128, 1, 40, 40, d_idx=64, gate_cols=1, gate_cols_idx=1)
    L.set_pages(0, torch.arange(40))
    L.idx_pool.copy_(torch.randn(L.idx_pool.shape, device="cuda"))
    n, t = 4, 4 * 64 * 39
    w, qi = torch.randn(n, 4, device="cuda"), torch.randn(n, 4, 64, device="cuda").to(torch.bfloat16)
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), t, dtype=torch.int64, device="cuda")
    idx = torch.zeros(n, 64, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(n, dtype=torch.int32, device="cuda")
    return (lambda **kw: ck.csa_index_score_topk(L, seq, pos, t, qi, w, 64, idx, cnt, **kw)), idx, \
        ck.csa_index_ws_bytes(L, n, 4, t, 64)


def _reserve(ck):
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, 128, 128, 64, 4096, 64, gate_cols=1)
    L.track_pages()
    seqs = torch.arange(64, dtype=torch.int32, device="cuda")
    first, count = (torch.full((64,), v, dtype=torch.int64, device="cuda") for v in (0, 60 * 64))

    def call(**kw):
        L.page_table.fill_(-1)
        L.page_refs.zero_()
        torch.cuda.current_stream().synchronize()
        ck.cskv_cache_reserve(L, seqs, first, count, 60 * 64, **kw)

    return call, L.page_table, ck.cskv_reserve_ws_bytes(L, 64, 60 * 64)


def _compact(ck):
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, 128, 128, 2, 4096, 2000, gate_cols=1)
    L.set_pages(0, torch.randperm(4096)[:2000])
    L.track_pages()
    D = ck.Layer.allocate(ck.LAYER_HCA, 128, 128, 128, 2, 2100, 2000, gate_cols=1)
    D.track_pages()
    return (lambda **kw: ck.cskv_cache_compact(L, D, **kw)), D.page_table, ck.cskv_compact_ws_bytes(L, D)


@pytest.mark.parametrize("make", [_attend, _select, _reserve, _compact])
@pytest.mark.parametrize("handle", [False, True])
def test_a_temporary_workspace_outlives_its_call(ck, make, handle):
    call, out, size = make(ck)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    out.fill_(0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # the call runs some 50 ms from now
    call(stream=side.cuda_stream if handle else side)
    others = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(4)]  # on the current stream, now
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in others)
    assert torch.equal(out, want)
