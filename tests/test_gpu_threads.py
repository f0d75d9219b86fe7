"""GPU test of calls from several host threads."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ck


def _attend_call(ck, d_qk, d_v, H, n, chunk=False, **kw):
    """hca_attend of n queries at position 700, as a function without arguments, and its output."""
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, d_qk, d_v, 1, 8, 8, gate_cols=1)
    L.set_pages(0, torch.arange(8))
    g = torch.Generator(device="cuda").manual_seed(n)
    L.kv_pool.copy_(torch.randn(L.kv_pool.shape, generator=g, device="cuda"))
    L.ring_x.copy_(torch.randn(L.ring_x.shape, generator=g, device="cuda"))
    q = torch.randn(n, H, d_qk, generator=g, device="cuda").to(torch.bfloat16)
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), 700, dtype=torch.int64, device="cuda")
    out = torch.zeros(n, H, d_v, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(ck.cskv_attend_ws_bytes(L, n, H, 700), dtype=torch.uint8, device="cuda")
    if chunk:
        kw.update(x_chunk=torch.randn(1, d_qk, generator=g, device="cuda").to(torch.bfloat16), chunk_pos0=700)
    return lambda: ck.hca_attend(L, seq, pos, 700, q, out, workspace=ws, **kw), out


def _select_call(ck, n):
    L = ck.Layer.allocate(ck.LAYER_CSA, 4, 128, 128, 1, 8, 8, d_idx=64, gate_cols=1, gate_cols_idx=1)
    L.set_pages(0, torch.arange(8))
    g = torch.Generator(device="cuda").manual_seed(n)
    L.idx_pool.copy_(torch.randn(L.idx_pool.shape, generator=g, device="cuda"))
    w = torch.randn(n, 4, generator=g, device="cuda")
    qi = torch.randn(n, 4, 64, generator=g, device="cuda").to(torch.bfloat16)
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.full((n,), 1500, dtype=torch.int64, device="cuda")
    idx = torch.zeros(n, 64, dtype=torch.int32, device="cuda")
    cnt = torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(ck.csa_index_ws_bytes(L, n, 4, 1500, 64), dtype=torch.uint8, device="cuda")
    return lambda: ck.csa_index_score_topk(L, seq, pos, 1500, qi, w, 64, idx, cnt, workspace=ws), idx


@pytest.mark.parametrize("make", [
    lambda ck: _attend_call(ck, 128, 128, 32, 3, score_cap=30.0), lambda ck: _attend_call(ck, 576, 512, 64, 3),
    lambda ck: _attend_call(ck, 576, 512, 64, 3, score_cap=30.0), lambda ck: _attend_call(ck, 128, 128, 64, 600),
    lambda ck: _attend_call(ck, 128, 128, 64, 600, score_cap=30.0),
    lambda ck: _attend_call(ck, 128, 128, 64, 600, chunk=True, score_cap=30.0), lambda ck: _select_call(ck, 3),
    lambda ck: _select_call(ck, 70), lambda ck: _select_call(ck, 900)],
    ids=["split", "latent", "latent rule", "pair", "pair rule", "chunk", "scan", "scan group", "scan tc"])
def test_first_call_of_a_thread(ck, make):
    """A host thread may begin with any entry point: nothing has made a CUDA context current for it yet."""
    call, out = make(ck)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            bad.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not bad, bad
    assert torch.equal(out, want)
