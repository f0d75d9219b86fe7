"""GPU tests of csa_attend / hca_attend at the edges of what the header allows: buffers at any 16-byte boundary.

Where a result is compared with the 64-bit formula, the bound is that of test_gpu_score_rule.
"""
import pytest
import torch

from test_gpu_score_rule import N_WIN, Setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ck


def _at_16(t):
    """The same values at an address that is 16 bytes past a 32-byte boundary."""
    n = 16 // t.element_size()
    buf = torch.empty(t.numel() + n, dtype=t.dtype, device=t.device)
    assert buf.data_ptr() % 32 == 0
    view = buf[n:].view(t.shape)
    view.copy_(t)
    return view


# the split kernel, the latent kernel (bf16, FP8), the query-pair kernel (selection; inverse RoPE) and the chunk form
FORMS = [("hca", 128, 128, 32, 3, False, 0), ("csa", 128, 128, 16, 5, True, 0), ("hca", 576, 512, 64, 3, False, 0),
         ("csa", 576, 512, 128, 5, True, 0), ("csa", 128, 128, 64, 640, False, 0), ("hca", 128, 128, 64, 640, False, 32),
         ("hca", 128, 128, 64, 700, False, 0), ("hca", 128, 128, 16, 700, False, 0)]


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q,fp8,rope", FORMS)
@pytest.mark.parametrize("cap,bias", [(30.0, True), (70.0, False), (0.0, True), (0.0, False)])
def test_buffers_need_16_byte_alignment_only(ck, kind, d_qk, d_v, H, n_q, fp8, rope, cap, bias):
    """Outputs and inputs at addresses 16 bytes past a 32-byte boundary: the same bits."""
    pos = list(range(1500, 1500 + n_q))
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=64 if kind == "csa" else 0, fp8=fp8, seed=H + n_q,
              chunk={0: (0, 1500, n_q)})
    slopes = s.slopes if bias else None
    good, good_lse = s.run(cap, slopes, rope_dims=rope)
    s.q, s.x_chunk = _at_16(s.q), _at_16(s.x_chunk)
    s.L.ring_x, s.L.kv_pool = _at_16(s.L.ring_x), _at_16(s.L.kv_pool)
    out, lse = _at_16(torch.full_like(good, 7.0)), torch.full_like(good_lse, 7.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(x_chunk=s.x_chunk, chunk_pos0=1500, status=st, score_cap=cap, slopes=slopes, rope_dims=rope)
    if s.k:
        ck.csa_attend(s.L, s.q_seq, s.q_pos, max(pos), s.q, s.sel, s.cnt, out, lse, **kw)
    else:
        ck.hca_attend(s.L, s.q_seq, s.q_pos, max(pos), s.q, out, lse, **kw)
    assert ck.cskv_get_status(st) == ck.OK
    assert torch.equal(out, good) and torch.equal(lse, good_lse)


# which queries of 4096 (64 heads: four queries share 256 rows; 16 heads: sixteen) have no keys
EMPTY = {
    "tail": lambda i, n: i >= n * 9 // 16,           # a padded batch
    "head": lambda i, n: i < n * 7 // 16,
    "blocks": lambda i, n: (i // 600) % 2 == 1,      # runs far longer than a block's rows
    "one left": lambda i, n: i != n // 2,
    "scattered": lambda i, n: (i * 2654435761 >> 7) % 19 < 18,
    "all": lambda i, n: True,
}


@pytest.mark.parametrize("empty", list(EMPTY))
@pytest.mark.parametrize("H,several", [(64, False), (16, False), (64, True), (16, True)])
@pytest.mark.parametrize("cap,bias", [(30.0, True), (70.0, True), (0.0, True)])
def test_chunk_with_many_queries_without_keys(ck, empty, H, several, cap, bias):
    """Whole blocks of invalid positions in a chunk (padding): zeros and -inf for them, the others' answers, no other
    report. Some blocks of rows then have no key at all, several in a row for one CTA."""
    n, pos0 = 4096, 700
    seqs, pos, chunk = [0] * n, list(range(pos0, pos0 + n)), {0: (0, pos0, n)}
    if several:  # two sequences, described by chunk_desc
        seqs = [0] * (n // 2) + [1] * (n - n // 2)
        pos = list(range(pos0, pos0 + n // 2)) * 2
        chunk = {0: (0, pos0, n // 2), 1: (n // 2, pos0, n // 2)}
    s = Setup(ck, "hca", 128, 128, H, seqs, pos, seed=H, chunk=chunk)
    gone = torch.tensor([EMPTY[empty](i, n) for i in range(n)], device="cuda")
    s.q_pos = torch.where(gone, -1, s.q_pos)
    out, lse = s.run(cap, s.slopes, want=ck.ERR_INVALID_ARG)
    assert not bool(out[gone].any()) and bool((lse[gone] == -float("inf")).all())
    live = (~gone).nonzero().flatten().tolist()
    s.check(out, lse, cap, s.slopes, sorted(set(live[:3] + live[-3:] + live[:: max(1, len(live) // 12)])))


def test_chunk_of_queries_of_unknown_sequences(ck):
    """The same with sequence ids outside the layer, and without lse."""
    n, pos0 = 2000, 300
    s = Setup(ck, "hca", 128, 128, 64, [0] * n, list(range(pos0, pos0 + n)), seed=3, chunk={0: (0, pos0, n)})
    s.q_seq[40:1960] = 7
    out, _ = s.run(20.0, s.slopes, want=ck.ERR_OUT_OF_RANGE, lse=False)
    assert not bool(out[40:1960].any())
    s.check(out, None, 20.0, s.slopes, [0, 39, 1960, 1999])


def _small(s, std):
    """Keys of the given standard deviation (Setup's have 2): values that leave a sum's overflow alone."""
    for t in (s.L.kv_pool, s.L.ring_x, s.x_chunk):
        t.mul_(std / 2)


@pytest.mark.parametrize("cap", [20.0, 50.0, 55.0])
@pytest.mark.parametrize("lo,hi", [(-1.0, -5.0), (-1.3, -1.7), (-2.4, -2.6), (-2.9, -3.1), (-0.01, -1.0)])
def test_steep_negative_slopes_near_the_first_entry(ck, cap, lo, hi):
    """Far keys lead, and at positions 128 to 190 the window's first token is farther than the middle of entry 0."""
    H, pos = 64, list(range(100, 321))
    for seed in range(4):
        s = Setup(ck, "hca", 128, 128, H, [0] * len(pos), pos, seed=seed, chunk={0: (0, 100, len(pos))}, q_std=1.0)
        _small(s, 128 ** -0.5)
        slopes = torch.linspace(lo, hi, H, device="cuda")
        out, lse = s.run(cap, slopes)
        s.check(out, lse, cap, slopes)


def _mask_entries(s, lo, hi):
    """The 64-bit formula's keys without entries lo .. hi - 1 (whose page is missing)."""
    rows = s.rows

    def kept(i):
        r, p = rows(i)
        j = (p - (s.m - 1) / 2) / s.m
        n_w = min(s.positions[i] + 1, N_WIN)
        keep = torch.ones(p.numel(), dtype=torch.bool, device="cuda")
        keep[n_w:] = (j[n_w:] < lo) | (j[n_w:] >= hi)
        return r[keep], p[keep]

    s.rows = kept


@pytest.mark.parametrize("cap", [20.0, 55.0, 70.0, 0.0])
@pytest.mark.parametrize("H,n_q", [(64, 300), (32, 5)])
def test_a_missing_first_page_under_a_negative_slope(ck, cap, H, n_q):
    """The key that leads has no row (reported): the others' answer, as with any missing page."""
    pos0 = 128 * 40
    s = Setup(ck, "hca", 128, 128, H, [0] * n_q, list(range(pos0, pos0 + n_q)), seed=5, chunk={0: (0, pos0, n_q)},
              page_size=16, q_std=1.0)
    _small(s, 128 ** -0.5)
    slopes = -torch.exp2(torch.linspace(-9, 1, H, device="cuda"))
    _mask_entries(s, 0, 16)
    page = int(s.L.page_table[0, 0])
    s.L.page_table[0, 0] = -1
    out, lse = s.run(cap, slopes, want=ck.ERR_OUT_OF_RANGE)
    s.L.page_table[0, 0] = page
    s.check(out, lse, cap, slopes, range(0, n_q, max(1, n_q // 20)))


# every kernel: split (HCA in pieces, CSA, FP8), latent (bf16, FP8, one piece and several), query pairs, chunk
FAR = [("hca", 128, 128, 32, 3, False, 0), ("csa", 128, 128, 16, 3, False, 0), ("csa", 128, 128, 32, 2, True, 0),
       ("hca", 576, 512, 64, 3, False, 0), ("csa", 576, 512, 128, 3, False, 0), ("csa", 576, 512, 64, 3, True, 0),
       ("csa", 576, 512, 64, 160, False, 0), ("csa", 128, 128, 64, 600, False, 0), ("hca", 128, 128, 64, 600, False, 32),
       ("hca", 128, 128, 64, 600, False, 0), ("hca", 128, 128, 48, 600, False, 0)]


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q,fp8,rope", FAR)
@pytest.mark.parametrize("cap", [0.0, 50.0, 400.0])
def test_negative_slopes_over_long_distances(ck, kind, d_qk, d_v, H, n_q, fp8, rope, cap):
    """Far keys lead by biases of up to 5e5, whose fp32 step alone would be several percent of a weight: the logits that
    count are small beside each other. (The bound allows for biases up to 100 below the leading key's.)"""
    pos = [(1 << 20) - 1 - i for i in range(n_q)][::-1]
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=96 if kind == "csa" else 0, fp8=fp8, seed=H + n_q,
              chunk={0: (0, pos[0], n_q)} if n_q > 160 else None, q_std=2.0 if kind == "csa" else 16.0)
    if s.k:  # neighbours among the far entries, so that several of them have a weight
        s.sel[:, :64] = torch.arange(3, 67, device="cuda")
        s.sel[:, 64:] = s.sel[:, 64:].clamp(min=1000).sort(1).values
    slopes = -torch.exp2(torch.linspace(-9, -1, H, device="cuda"))
    slopes[1::5] = 2.0 ** -8  # some heads look near
    out, lse = s.run(cap, slopes, rope_dims=rope)
    some = sorted({0, 1, n_q // 2, n_q - 1})
    s.check(out, lse, cap, slopes, some, rope=rope)


BIG = (1 << 63) - 1


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q,fp8", [("hca", 128, 128, 32, 4, False), ("csa", 576, 512, 64, 5, True),
                                                      ("hca", 576, 512, 64, 5, False), ("csa", 128, 128, 64, 640, False),
                                                      ("hca", 128, 128, 64, 700, False)])
@pytest.mark.parametrize("desc,outside", [((BIG, 1500, 1), True), ((1, 1500, BIG), True), ((-1, 1500, 2), True),
                                          ((0, 1500, -1), True), ((BIG - 5, 1500, 6), True), ((4, 1500, 100000), True),
                                          ((0, BIG, 2), False), ((0, -BIG - 1, 2), False), ((0, -BIG - 1 + 1500, 1), False)])
@pytest.mark.parametrize("cap", [30.0, 70.0])
def test_descriptors_of_any_value(ck, kind, d_qk, d_v, H, n_q, fp8, desc, outside, cap):
    """A chunk descriptor outside x_chunk, its sums past 63 bits among them, is reported and its rows come from the ring;
    positions far from every query's name none of them."""
    pos = list(range(1500, 1500 + n_q))
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=64 if kind == "csa" else 0, fp8=fp8, seed=2, chunk={1: (0, 0, n_q)})
    from compressed_sparse_kv_02_b200 import _binding as b
    import ctypes
    out = torch.full((n_q, H, d_v), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n_q, H), 7.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.zeros(s.L.n_seqs, 3, dtype=torch.int64)
    d[0] = torch.tensor(desc)
    d = d.cuda()
    ws = torch.empty(ck.cskv_attend_ws_bytes(s.L, n_q, H, max(pos), s.k), dtype=torch.uint8, device="cuda")
    a = b._attend_args(s.L, s.q_seq, s.q_pos, max(pos), s.q, s.sel if s.k else None, s.cnt if s.k else None, s.k, None,
                       out, lse, s.x_chunk, 0, st, chunk_desc=d, score_cap=cap, slopes=s.slopes)
    f = ck.lib().csa_attend if s.k else ck.lib().hca_attend
    assert f(ctypes.byref(a), ws.data_ptr(), ws.numel(), b._stream(None)) == ck.OK
    assert ck.cskv_get_status(st) == (ck.ERR_OUT_OF_RANGE if outside else ck.OK)
    s.chunk = None  # every window row is the ring's
    s.check(out, lse, cap, s.slopes, sorted({0, n_q // 2, n_q - 1}))


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q", [("hca", 128, 128, 32, 4), ("csa", 576, 512, 64, 5),
                                                 ("csa", 128, 128, 64, 640), ("hca", 128, 128, 64, 700)])
@pytest.mark.parametrize("power,cap", [(60, 2.0 ** 20), (60, 2.0 ** 30), (-22, 190.0), (-30, 30.0), (30, 30.0)])
def test_scales_far_from_one(ck, kind, d_qk, d_v, H, n_q, power, cap):
    """Queries times 2^power with sm_scale times 2^-power: the same scores, from products far from one."""
    pos = list(range(2000, 2000 + n_q))
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=64 if kind == "csa" else 0, seed=4, chunk={0: (0, 2000, n_q)})
    q = s.q
    s.q = q * 2.0 ** power
    out, lse = s.run(cap, s.slopes, sm_scale=2.0 ** -power / d_qk ** 0.5)
    s.q = q
    s.check(out, lse, cap, s.slopes, sorted({0, n_q // 2, n_q - 1}))


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q", [("hca", 128, 128, 32, 4), ("csa", 576, 512, 64, 5),
                                                 ("csa", 128, 128, 64, 640), ("hca", 128, 128, 64, 700)])
@pytest.mark.parametrize("cap", [300.0, 1000.0, 3000.0, 20000.0])
def test_large_caps_within_reach(ck, kind, d_qk, d_v, H, n_q, cap):
    """Scores of up to several times a large cap, and below it."""
    pos = list(range(2000, 2000 + n_q))
    for reach in (0.1, 0.5, 2.0):
        s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=64 if kind == "csa" else 0, seed=6, chunk={0: (0, 2000, n_q)},
                  q_std=cap * reach / 4)
        out, lse = s.run(cap, None)
        s.check(out, lse, cap, None, sorted({0, n_q // 2, n_q - 1}))


@pytest.mark.parametrize("empty", list(EMPTY))
@pytest.mark.parametrize("kind,d_qk,d_v,H,n,rope", [("csa", 128, 128, 64, 1300, 0), ("hca", 128, 128, 64, 1300, 32),
                                                    ("csa", 128, 128, 16, 900, 0), ("hca", 576, 512, 64, 170, 0),
                                                    ("csa", 576, 512, 64, 500, 0)])
def test_many_queries_without_keys_in_the_other_forms(ck, empty, kind, d_qk, d_v, H, n, rope):
    """Padding in calls that the query-pair, split and latent kernels take, with the rule and without."""
    pos = list(range(600, 600 + n))
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n, pos, k=64 if kind == "csa" else 0, seed=n, chunk={0: (0, 600, n)})
    gone = torch.tensor([EMPTY[empty](i, n) for i in range(n)], device="cuda")
    s.q_pos = torch.where(gone, 1 << 40, s.q_pos)
    live = (~gone).nonzero().flatten().tolist()
    for cap, slopes in ((30.0, s.slopes), (0.0, None)):
        out, lse = s.run(cap, slopes, want=ck.ERR_INVALID_ARG if bool(gone.any()) else 0, rope_dims=rope)
        assert not bool(out[gone].any()) and bool((lse[gone] == -float("inf")).all())
        s.check(out, lse, cap, slopes, sorted(set(live[:2] + live[-2:] + live[:: max(1, len(live) // 8)])), rope=rope)
