"""GPU tests of calls from several host threads: a thread's first call, and calls of two sizes at once."""
import ctypes
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


def _raw_reserve(ck, n, stream):
    """cskv_cache_reserve of n sequences without new pages, through the C ABI: as little Python between calls as possible."""
    from compressed_sparse_kv_02_b200 import _binding as b
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, 16, 16, 4096, 64, 4, page_size=16, gate_cols=1)
    L.track_pages()
    seqs, zero = torch.arange(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    ws, s = torch.empty(ck.cskv_reserve_ws_bytes(L, n, 1), dtype=torch.uint8, device="cuda"), L.struct
    a = b.ReserveArgs(ctypes.sizeof(b.ReserveArgs), ctypes.pointer(s), L.page_refs.data_ptr(), n, seqs.data_ptr(),
                      zero.data_ptr(), zero.data_ptr(), 1, None)
    return ck.lib().cskv_cache_reserve, a, ws, stream, (L, seqs, zero, s)


def _raw_attend(ck, n, stream, d_qk, d_v, H, cap):
    from compressed_sparse_kv_02_b200 import _binding as b
    L = ck.Layer.allocate(ck.LAYER_HCA, 128, d_qk, d_v, 1, 8, 8, gate_cols=1)
    L.set_pages(0, torch.arange(8))
    q, out = (torch.zeros(n, H, d, dtype=torch.bfloat16, device="cuda") for d in (d_qk, d_v))
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
    ws = torch.empty(ck.cskv_attend_ws_bytes(L, n, H, 700), dtype=torch.uint8, device="cuda")
    a = b._attend_args(L, seq, pos, 700, q, None, None, 0, None, out, None, None, 0, None, score_cap=cap)
    return ck.lib().hca_attend, a, ws, stream, (L, q, out, seq, pos)


def _raw_select(ck, n, stream):
    from compressed_sparse_kv_02_b200 import _binding as b
    L = ck.Layer.allocate(ck.LAYER_CSA, 4, 128, 128, 1, 8, 8, d_idx=64, gate_cols=1, gate_cols_idx=1)
    L.set_pages(0, torch.arange(8))
    w, qi = torch.zeros(n, 4, device="cuda"), torch.zeros(n, 4, 64, dtype=torch.bfloat16, device="cuda")
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.full((n,), 500, dtype=torch.int64, device="cuda")
    idx, cnt = torch.zeros(n, 64, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(ck.csa_index_ws_bytes(L, n, 4, 500, 64), dtype=torch.uint8, device="cuda")
    a = b._index_args(L, seq, pos, 500, qi, w, 64, idx, cnt, None, None, None)
    return ck.lib().csa_index_score_topk, a, ws, stream, (L, w, qi, seq, pos, idx, cnt)


@pytest.mark.parametrize("make,sizes,times", [
    (_raw_reserve, (3400, 4096), 500),
    (lambda ck, n, s: _raw_attend(ck, n, s, 128, 128, 32, 0.0), (1, 400), 8000),
    (lambda ck, n, s: _raw_attend(ck, n, s, 128, 128, 32, 30.0), (1, 400), 8000),
    (lambda ck, n, s: _raw_attend(ck, n, s, 576, 512, 64, 0.0), (1, 170), 8000),
    (lambda ck, n, s: _raw_attend(ck, n, s, 576, 512, 64, 30.0), (1, 170), 8000),
    (lambda ck, n, s: _raw_attend(ck, n, s, 576, 512, 64, 30.0), (300, 900), 4000),
    (_raw_select, (1, 10), 4000), (_raw_select, (40, 63), 4000), (_raw_select, (700, 900), 4000)],
    ids=["reserve", "split", "split rule", "latent", "latent rule", "latent split", "scan", "scan group", "scan tc"])
def test_calls_of_two_sizes_at_once(ck, make, sizes, times):
    """Two threads on streams and buffers of their own: a kernel's limit on dynamic shared memory is the process's, so a
    smaller call may not lower it between the other's setting it and its launch."""
    streams = [torch.cuda.Stream() for _ in sizes]
    made = [make(ck, n, s) for n, s in zip(sizes, streams)]
    torch.cuda.synchronize()
    gate, failed = threading.Barrier(len(sizes)), [0] * len(sizes)

    def work(i):
        f, a, ws, stream, _ = made[i]
        p, w, n, st = ctypes.byref(a), ws.data_ptr(), ws.numel(), ctypes.c_void_p(stream.cuda_stream)
        gate.wait(60)
        for k in range(times):
            failed[i] += f(p, w, n, st) != ck.OK
            if k % 500 == 499:
                stream.synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(sizes)
