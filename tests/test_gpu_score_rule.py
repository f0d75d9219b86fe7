"""GPU tests of csa_attend / hca_attend with a score rule (cap, distance bias) against the formula in 64 bits, in
every kernel: the split kernel, the 576 / 512 tensor-core kernel (bf16 and FP8), the query-pair kernel and the chunk
form.

Bound of an output element, per (query, head), from the roundings the kernels make:
  - a logit's absolute error D: the fp32 dot product, d_qk 2^-24 sm_scale sum |q||k| at worst; the rule's own fp32
    arithmetic, 2^-20 of the capped logit (tanh to 4e-7 and three roundings) and 2^-22 of the bias; weights whose
    bias is below -100 are 0 on both sides, so the bias counts up to 100;
  - a weight exp(s - max) then has a relative error of at most 2 D, its rounding to bf16 adds 2^-8 (half a step), so
    the weighted sum is off by (2 D + 2^-8) sum w |v|, and so is its denominator, without the bf16 rounding: 2 D |o|;
  - the output's own rounding, 2^-8 |o|; the fp32 sums and the merge of the splits, 2^-16 sum w |v|.
log-sum-exp: D, and 2^-20 of its size (exp2, log2 and fp32 sums).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

N_WIN = 128


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ck


def visible(t, m):
    return max(0, -(-(t + 1 - N_WIN) // m))


class Setup:
    """A layer with random entries and rings; queries at `positions` of sequences `seqs`."""

    def __init__(self, ck, kind, d_qk, d_v, H, seqs, positions, k=0, fp8=False, seed=0, chunk=None, page_size=64,
                 q_std=2.0):
        self.ck, self.kind, self.d_v, self.H = ck, kind, d_v, H
        self.m = m = 4 if kind == "csa" else 128
        n_seqs, top = max(seqs) + 1, max(positions)
        per = -(-(top // m + 2) // page_size)
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        L = self.L = ck.Layer.allocate(ck.LAYER_CSA if kind == "csa" else ck.LAYER_HCA, m, d_qk, d_v, n_seqs,
                                       n_seqs * per + 2, per, page_size=page_size, d_idx=64 if kind == "csa" else 0,
                                       kv_dtype=ck.FP8_E4M3 if fp8 else ck.BF16, gate_cols=1, gate_cols_idx=1)
        perm = torch.randperm(n_seqs * per + 2, generator=torch.Generator().manual_seed(seed))
        for s in range(n_seqs):
            L.set_pages(s, perm[s * per:(s + 1) * per])
        if fp8:
            L.kv_pool.copy_((torch.randn(L.kv_pool.shape, generator=g, device="cuda") * 100).clamp(-448, 448)
                            .to(torch.float8_e4m3fn).view(torch.uint8))
            L.kv_scale.copy_((torch.rand(L.kv_scale.shape, generator=g, device="cuda") + 0.5) / 50)
        else:
            L.kv_pool.copy_(torch.randn(L.kv_pool.shape, generator=g, device="cuda") * 2)
        L.ring_x.copy_(torch.randn(L.ring_x.shape, generator=g, device="cuda") * 2)
        n = len(positions)
        self.seqs, self.positions = seqs, positions
        self.q_seq = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        self.q_pos = torch.tensor(positions, dtype=torch.int64, device="cuda")
        self.q = (torch.randn(n, H, d_qk, generator=g, device="cuda") * q_std).to(torch.bfloat16)
        self.slopes = torch.exp2(-1 - 15 * torch.rand(H, generator=g, device="cuda"))
        self.chunk = chunk  # {seq: (first row, first position, length)} of x_chunk
        if chunk:
            self.x_chunk = (torch.randn(max(r + l for r, _, l in chunk.values()), d_qk, generator=g, device="cuda") * 2
                            ).to(torch.bfloat16)
        self.k = k
        if k:
            sel = torch.full((n, k), -1, dtype=torch.int32)
            cnt = torch.zeros(n, dtype=torch.int32)
            cg = torch.Generator().manual_seed(seed + 1)
            for i, t in enumerate(positions):
                v = visible(t, m)
                c = min(k, v)
                sel[i, :c] = torch.randperm(v, generator=cg)[:c].sort().values.int()
                cnt[i] = c
            self.sel, self.cnt = sel.cuda(), cnt.cuda()

    def run(self, cap=0.0, slopes=None, want=0, lse=True, **kw):
        from compressed_sparse_kv_02_b200 import _binding as b
        import ctypes
        ck, n = self.ck, len(self.positions)
        out = torch.full((n, self.H, self.d_v), 7.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((n, self.H), 7.0, device="cuda") if lse else None
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        top = max(self.positions)
        if self.chunk and len(self.chunk) == 1 and 0 in self.chunk:
            kw.update(x_chunk=self.x_chunk, chunk_pos0=self.chunk[0][1])
        if self.chunk and "x_chunk" not in kw:  # several sequences: the descriptor form of the C ABI
            desc = torch.zeros(self.L.n_seqs, 3, dtype=torch.int64)
            for s, d in self.chunk.items():
                desc[s] = torch.tensor(d)
            desc = desc.cuda()
            ws = torch.empty(ck.cskv_attend_ws_bytes(self.L, n, self.H, top, self.k), dtype=torch.uint8, device="cuda")
            a = b._attend_args(self.L, self.q_seq, self.q_pos, top, self.q, self.sel if self.k else None,
                               self.cnt if self.k else None, self.k, None, out, ls, self.x_chunk, 0, st,
                               chunk_desc=desc, score_cap=cap, slopes=slopes)
            f = ck.lib().csa_attend if self.k else ck.lib().hca_attend
            assert f(ctypes.byref(a), ws.data_ptr(), ws.numel(), b._stream(None)) == ck.OK
        elif self.k:
            ck.csa_attend(self.L, self.q_seq, self.q_pos, top, self.q, self.sel, self.cnt, out, ls, status=st,
                          score_cap=cap, slopes=slopes, **kw)
        else:
            ck.hca_attend(self.L, self.q_seq, self.q_pos, top, self.q, out, ls, status=st, score_cap=cap,
                          slopes=slopes, **kw)
        assert ck.cskv_get_status(st) == want
        return out, ls

    def rows(self, i):
        """(rows, positions) of query i's keys, in 64 bits."""
        s, t = self.seqs[i], self.positions[i]
        p = torch.arange(max(0, t - N_WIN + 1), t + 1, device="cuda")
        raw = self.L.ring_x[s][p % N_WIN].double()
        if self.chunk and s in self.chunk:
            r0, p0, n = self.chunk[s]
            new = (p >= p0) & (p < p0 + n)
            raw[new] = self.x_chunk[r0 + p[new] - p0].double()
        j = torch.arange(visible(t, self.m), device="cuda")
        if self.k:
            j = self.sel[i, : int(self.cnt[i])].long()
        if j.numel():
            e = self.L.read_entries(s, int(j.max()) + 1)
            ent = e["kv"][j]
            ent = ent.double() if "kv_scale" not in e else (ent.view(torch.float8_e4m3fn).double() *
                                                            e["kv_scale"][j].double()[:, None])
        else:
            ent = raw[:0]
        return torch.cat([raw, ent]), torch.cat([p.double(), j.double() * self.m + (self.m - 1) / 2])

    def check(self, out, lse, cap, slopes, queries=None, rope=0):
        for i in range(len(self.positions)) if queries is None else queries:
            rows, pos = self.rows(i)
            q = self.q[i].double()
            sm = 1 / math.sqrt(q.shape[1])
            s = q @ rows.t() * sm
            bias = torch.zeros_like(s)
            if cap:
                s = cap * torch.tanh(s / cap)
            if slopes is not None:
                bias = slopes.double()[:, None] * (self.positions[i] - pos)[None]
            z = s - bias
            l = torch.logsumexp(z, 1)
            w = torch.exp(z - l[:, None])
            v = rows[:, : self.d_v]
            o = w @ v
            D = q.shape[1] * 2.0 ** -24 * sm * (q.abs() @ rows.abs().t()).amax(1)
            D = D + 2.0 ** -20 * s.abs().amax(1) + 2.0 ** -22 * bias.abs().clamp(max=100).amax(1)
            wv = w @ v.abs()
            tol = (2 * D[:, None] + 2.0 ** -8 + 2.0 ** -16) * wv + 2 * D[:, None] * o.abs()
            if rope:  # pairs of the last channels rotated by -t theta: so are their bounds, and cos, sin in fp32
                c0 = self.d_v - rope
                k = torch.arange(rope // 2, device="cuda", dtype=torch.float64)
                ang = self.positions[i] * 10000.0 ** (-2 * k / rope)
                c, n = torch.cos(ang), torch.sin(ang)
                a, b = o[:, c0::2].clone(), o[:, c0 + 1::2].clone()
                ta, tb = tol[:, c0::2] + 2.0 ** -20 * a.abs(), tol[:, c0 + 1::2] + 2.0 ** -20 * b.abs()
                o[:, c0::2], o[:, c0 + 1::2] = a * c + b * n, b * c - a * n
                tol[:, c0::2], tol[:, c0 + 1::2] = ta * c.abs() + tb * n.abs(), tb * c.abs() + ta * n.abs()
            tol = tol + 2.0 ** -8 * o.abs()
            err = (out[i].double() - o).abs()
            assert bool((err <= tol).all()), "query %d (t = %d): off by %.3g of its bound" % (
                i, self.positions[i], float((err / tol).max()))
            if lse is not None:
                el = (lse[i].double() - l).abs()
                assert bool((el <= D + 2.0 ** -20 * (l.abs() + 1)).all()), (i, float(el.max()), float(D.max()))


RULES = [(30.0, True), (20.0, False), (0.0, True), (70.0, True)]  # 70: above what bounds the chunk form's logits


def _both(s, rules=RULES, queries=None):
    for cap, bias in rules:
        slopes = s.slopes if bias else None
        out, lse = s.run(cap, slopes)
        s.check(out, lse, cap, slopes, queries)


EDGE = [0, 1, 5, 126, 127, 128, 129, 300, 128 * 9 + 1, 128 * 40 + 77]


@pytest.mark.parametrize("H", [16, 32, 64])
@pytest.mark.parametrize("fp8", [False, True])
def test_hca_split_kernel(ck, H, fp8):
    _both(Setup(ck, "hca", 128, 128, H, list(range(10)), EDGE, fp8=fp8, seed=H))


@pytest.mark.parametrize("H,k", [(16, 1), (32, 300), (64, 64)])
@pytest.mark.parametrize("fp8", [False, True])
def test_csa_split_kernel(ck, H, k, fp8):
    _both(Setup(ck, "csa", 128, 128, H, list(range(10)), EDGE, k=k, fp8=fp8, seed=H + 1))


@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("fp8", [False, True])
def test_latent_576(ck, H, fp8):
    _both(Setup(ck, "hca", 576, 512, H, list(range(10)), EDGE, fp8=fp8, seed=H + 2))
    _both(Setup(ck, "csa", 576, 512, H, list(range(4)), [0, 127, 131, 5000], k=512, fp8=fp8, seed=H + 3))


def test_long_contexts(ck):
    """Positions up to 1M: distances far beyond what the slopes leave, and ones they keep."""
    _both(Setup(ck, "hca", 576, 512, 128, [0, 1], [(1 << 20) - 1, 777777], seed=4))
    _both(Setup(ck, "csa", 128, 128, 32, [0, 1], [(1 << 20) - 1, 777777], k=512, seed=5))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_q", [110, 113, 180])
def test_many_decode_queries_576(ck, n_q, fp8):
    """The tensor-core kernel's limit on queries per call, and the split kernel behind it."""
    pos = [(37 * i) % 2000 for i in range(n_q)]
    _both(Setup(ck, "hca", 576, 512, 64, [i % 5 for i in range(n_q)], pos, fp8=fp8, seed=n_q), rules=RULES[:1],
          queries=range(0, n_q, 11))


@pytest.mark.parametrize("kind", ["hca", "csa"])
@pytest.mark.parametrize("n_q,pos0", [(1, 0), (1, 700), (5, 0), (97, 31), (601, 0), (777, 1009), (2051, 128 * 70 + 5)])
@pytest.mark.parametrize("H", [16, 64])
def test_chunk(ck, kind, n_q, pos0, H):
    """Chunks of one sequence: from one token to thousands, from an empty cache and behind a long one."""
    pos = list(range(pos0, pos0 + n_q))
    s = Setup(ck, kind, 128, 128, H, [0] * n_q, pos, k=300 if kind == "csa" else 0, seed=n_q + H,
              chunk={0: (0, pos0, n_q)})
    some = sorted({0, min(1, n_q - 1), n_q // 2, n_q - 1, min(n_q - 1, 127), min(n_q - 1, 128)} | set(range(0, n_q, 61)))
    _both(s, queries=some)


@pytest.mark.parametrize("kind", ["hca", "csa"])
@pytest.mark.parametrize("H", [32, 64])
def test_ragged_chunks_of_several_sequences(ck, kind, H):
    """Varlen: chunks of several sequences back to back, lengths 1 to 500, one sequence without a chunk."""
    chunk, seqs, pos, at = {}, [], [], 0
    for s, (p0, n) in enumerate([(0, 301), (5000, 1), (127, 2), (900, 333), (64, 64), (3000, 500)]):
        chunk[s] = (at, p0, n)
        seqs += [s] * n
        pos += list(range(p0, p0 + n))
        at += n
    seqs.append(6)
    pos.append(2222)
    _both(Setup(ck, kind, 128, 128, H, seqs, pos, k=128 if kind == "csa" else 0, seed=9, chunk=chunk),
          queries=[0, 1, 2, 299, 300, 301, 302, 303, 304, 400, 636, 637, 700, 701, 1000, 1199, 1200, 1201])


def test_chunk_queries_in_any_order(ck):
    """The queries of a call need not be consecutive: shuffled, repeated and far apart."""
    n, pos0 = 700, 4000
    g = torch.Generator().manual_seed(3)
    pos = (torch.randint(0, n, (n,), generator=g) + pos0).tolist()
    _both(Setup(ck, "hca", 128, 128, 64, [0] * n, pos, seed=8, chunk={0: (0, pos0, n)}), rules=RULES[:1],
          queries=range(0, n, 37))


@pytest.mark.parametrize("kind,d_qk,d_v,H,n_q", [("hca", 128, 128, 32, 3), ("hca", 576, 512, 64, 3),
                                                  ("csa", 128, 128, 64, 3), ("hca", 128, 128, 64, 700)])
def test_rule_off_and_extreme_caps(ck, kind, d_qk, d_v, H, n_q):
    """Zero slopes and no cap, or a cap far above every logit, answer as the plain form within the bounds; a tiny cap
    makes the scores equal; a negative slope looks far."""
    pos = [2000 + i for i in range(n_q)]
    s = Setup(ck, kind, d_qk, d_v, H, [0] * n_q, pos, k=64 if kind == "csa" else 0, seed=12, chunk={0: (0, 2000, n_q)})
    some = sorted({0, n_q // 2, n_q - 1})
    zero = torch.zeros_like(s.slopes)
    for cap, slopes in ((0.0, zero), (1e30, None), (2.0 ** 100, zero), (1e-3, None), (0.0, -s.slopes / 64), (1e-30, None),
                        (20.0, -s.slopes / 64), (55.0, s.slopes)):
        out, lse = s.run(cap, slopes)
        s.check(out, lse, cap, slopes, some)


@pytest.mark.parametrize("cap", [20.0, 55.0, 70.0])
def test_chunk_with_far_logits(ck, cap):
    """Logits at the cap on both sides, rows whose keys all sit at the lower one, and biases that bury all but the
    nearest keys: sums from 2^-80 to 2^80 around the reference."""
    n, pos0, H = 700, 3000, 64
    s = Setup(ck, "hca", 128, 128, H, [0] * n, list(range(pos0, pos0 + n)), seed=18, chunk={0: (0, pos0, n)}, q_std=40.0)
    s.q[:, 1::4] = s.q[:, 1::4].abs()
    s.x_chunk[: n // 2] = -s.x_chunk[: n // 2].abs()  # heads 1, 5, ..: every near key far below
    steep = s.slopes.clone()
    steep[::2] = 3.0
    some = [0, 1, 127, 128, 200, 349, 350, 351, 480, 699]
    for slopes in (None, steep, -s.slopes / 64):
        out, lse = s.run(cap, slopes)
        s.check(out, lse, cap, slopes, some)


def test_inverse_rope_and_no_lse(ck):
    """The output's rotation follows the softmax of the ruled scores; lse may be left out."""
    for d_qk, d_v, H, n_q in ((128, 128, 32, 2), (576, 512, 64, 2), (128, 128, 64, 640)):
        pos = [3000 + i for i in range(n_q)]
        s = Setup(ck, "hca", d_qk, d_v, H, [0] * n_q, pos, seed=13, chunk={0: (0, 3000, n_q)})
        out, _ = s.run(30.0, s.slopes, lse=False, rope_dims=32)
        s.check(out, None, 30.0, s.slopes, sorted({0, n_q // 2, n_q - 1}), rope=32)


def test_masked_keys_keep_out(ck):
    """Selected ids outside the visible entries, pages without an id and NaN in entries no query may see: reported
    where the call says so, and without effect on the answer."""
    for d_qk, d_v, H, n_q in ((128, 128, 32, 4), (576, 512, 64, 4), (128, 128, 64, 640)):
        pos = [1500 + i for i in range(n_q)]
        s = Setup(ck, "csa", d_qk, d_v, H, [0] * n_q, pos, k=64, seed=14)
        v = visible(max(pos), 4)  # entries from here on are in the pool, and no query sees them
        rows = s.L.rows_of(0, v, 3)
        s.L.kv_pool[rows] = float("nan")
        out, lse = s.run(20.0, s.slopes)
        keep = s.sel.clone()
        s.sel[:, 0] = v + 1
        s.sel[:, 5] = -3
        bad, _ = s.run(20.0, s.slopes, want=ck.ERR_OUT_OF_RANGE)
        s.sel = keep
        assert bool(torch.isfinite(bad.float()).all()) and not torch.equal(bad, out)
        drop = torch.ones(64, dtype=torch.bool, device="cuda")
        drop[0] = drop[5] = False
        s.sel = torch.cat([keep[:, drop], torch.full((n_q, 2), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
        s.cnt = s.cnt - 2
        s.check(bad, None, 20.0, s.slopes, sorted({0, n_q // 2, n_q - 1}))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_chunk_nan_stays_with_the_queries_that_see_it(ck, value):
    """A bad token and a bad entry in the middle of a chunk: queries that do not see them answer as before, those that
    do give NaN (their softmax has a NaN logit, or a NaN or infinite value with a weight)."""
    n, pos0, H = 1300, 1000, 64
    chunk = {0: (0, pos0, n // 2), 1: (n // 2, 70, n // 2)}
    seqs = [0] * (n // 2) + [1] * (n // 2)
    pos = list(range(pos0, pos0 + n // 2)) + list(range(70, 70 + n // 2))
    s = Setup(ck, "hca", 128, 128, H, seqs, pos, seed=17, chunk=chunk)
    good, lse = s.run(30.0, s.slopes)
    token, entry = pos0 + 301, 9  # entry 9 of sequence 0: visible from t = 9 * 128 + 127 on
    s.x_chunk[token - pos0, 5] = value
    s.L.kv_pool[s.L.rows_of(0, entry, 1), 7] = value
    bad, bad_lse = s.run(30.0, s.slopes)
    t = s.q_pos
    sees = (s.q_seq == 0) & (((t >= token) & (t < token + N_WIN)) | (entry * 128 < t + 1 - N_WIN))
    clean = ~sees
    # the clean rows: the same keys, at most another order of the same sums (a row taken again on its own)
    diff = (bad[clean].float() - good[clean].float()).abs()
    assert bool((diff <= 2.0 ** -7 * (good[clean].float().abs() + 2.0)).all())
    assert bool(((bad_lse[clean] - lse[clean]).abs() <= 1e-3).all())
    assert not bool(torch.isfinite(bad[sees].float()).all(-1).any())
    s.check(bad, bad_lse, 30.0, s.slopes, [i for i in range(0, n, 53) if not bool(sees[i])])


def test_rows_without_keys(ck):
    """A position past the caller's bound or a sequence outside the layer: zeros, -inf, and the report."""
    for d_qk, d_v, H, n_q in ((128, 128, 32, 3), (576, 512, 64, 3), (128, 128, 64, 640)):
        pos = [200 + i for i in range(n_q)]
        s = Setup(ck, "hca", d_qk, d_v, H, [0] * n_q, pos, seed=15)
        good, _ = s.run(20.0, s.slopes)
        s.q_pos[1] = -1
        out, lse = s.run(20.0, s.slopes, want=ck.ERR_INVALID_ARG)
        assert not bool(out[1].any()) and bool((lse[1] == -math.inf).all())
        assert torch.equal(out[0], good[0])
        s.q_pos[1] = pos[1]
        s.q_seq[2] = 5
        out, lse = s.run(20.0, s.slopes, want=ck.ERR_OUT_OF_RANGE)
        assert not bool(out[2].any()) and bool((lse[2] == -math.inf).all())
        assert torch.equal(out[:2], good[:2])


def test_calls_repeat_bit_for_bit_and_replay(ck):
    """The same call twice, and replayed from a graph with other work between, gives the same bits."""
    for d_qk, d_v, H, n_q in ((128, 128, 16, 7), (576, 512, 128, 2), (128, 128, 64, 650)):
        pos = [5000 + i for i in range(n_q)]
        s = Setup(ck, "hca", d_qk, d_v, H, [0] * n_q, pos, seed=16, chunk={0: (0, 5000, n_q)})
        a, la = s.run(30.0, s.slopes)
        b, lb = s.run(30.0, s.slopes)
        assert torch.equal(a, b) and torch.equal(la, lb)
        out, lse = torch.zeros_like(a), torch.zeros_like(la)
        ws = torch.empty(ck.cskv_attend_ws_bytes(s.L, n_q, H, max(pos)), dtype=torch.uint8, device="cuda")
        args = dict(workspace=ws, x_chunk=s.x_chunk, chunk_pos0=5000, score_cap=30.0, slopes=s.slopes)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ck.hca_attend(s.L, s.q_seq, s.q_pos, max(pos), s.q, out, lse, **args)
        for _ in range(2):
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, a) and torch.equal(lse, la)
        del graph


@pytest.mark.parametrize("H", [48, 80, 96, 128])
def test_chunk_head_counts(ck, H):
    """Head counts that do not divide the chunk form's tiles, and ones above its rows per query."""
    n, pos0 = 403, 1700
    pos = list(range(pos0, pos0 + n))
    s = Setup(ck, "hca", 128, 128, H, [0] * n, pos, seed=H, chunk={0: (0, pos0, n)})
    _both(s, rules=RULES[:2], queries=[0, 1, 2, 3, 5, 7, 100, 127, 128, 200, 401, 402])


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_pair_form_keeps_a_bad_row_to_its_queries(ck, value):
    """With inverse RoPE a chunk takes the query-pair form: the pair of a query that sees a bad token answers as before."""
    n, pos0 = 640, 3000
    s = Setup(ck, "hca", 128, 128, 64, [0] * n, list(range(pos0, pos0 + n)), seed=18, chunk={0: (0, pos0, n)})
    token = pos0 + 301  # odd: the second query of its pair is the first to see it
    s.x_chunk[token - pos0, 5] = value
    out, _ = s.run(30.0, s.slopes, lse=False, rope_dims=32)
    s.check(out, None, 30.0, s.slopes, [0, 1, 299, 300, 301 + N_WIN, 302 + N_WIN, n - 1], rope=32)


def test_fp8_codes_of_every_value(ck):
    """Entries of all finite E4M3 codes (subnormal ones and zeros of both signs included), and a NaN code that one query
    has selected: the others answer as before."""
    seqs, pos = [0, 1, 2, 0, 1, 2, 0], [3000, 2500, 1111, 2999, 700, 131, 40]
    s = Setup(ck, "csa", 576, 512, 128, seqs, pos, k=200, fp8=True, seed=19)
    codes = torch.randint(0, 254, s.L.kv_pool.shape, generator=s.g, device="cuda")
    s.L.kv_pool.copy_((codes + (codes >= 127).int()).to(torch.uint8))  # 0x7f and 0xff are NaN
    s.L.kv_scale.mul_(1 / 8)
    _both(s, rules=RULES[:2])
    row = s.L.rows_of(1, int(s.sel[1, 17]), 1)
    s.L.kv_pool[row, 33] = 0x7F
    out, lse = s.run(20.0, s.slopes)
    hit = [i for i in range(len(pos)) if seqs[i] == 1 and int(s.sel[1, 17]) in s.sel[i, : int(s.cnt[i])].tolist()]
    assert 1 in hit
    s.check(out, lse, 20.0, s.slopes, [i for i in range(len(pos)) if i not in hit])


@pytest.mark.parametrize("kind,fp8", [("csa", True), ("hca", True), ("csa", False)])
def test_latent_576_chunk(ck, kind, fp8):
    """A chunk's rows in the wide latent's window: tiles of several sources, FP8 entries among them."""
    n, pos0 = 37, 1501
    s = Setup(ck, kind, 576, 512, 64, [0] * n, list(range(pos0, pos0 + n)), k=100 if kind == "csa" else 0, fp8=fp8,
              seed=20, chunk={0: (0, pos0, n)})
    _both(s, rules=RULES[:2], queries=[0, 1, 17, 36])


@pytest.mark.parametrize("d_qk,d_v,H,fp8", [(576, 512, 128, False), (576, 512, 64, True), (128, 128, 32, False)])
def test_lengths_far_apart(ck, d_qk, d_v, H, fp8):
    """One call's sequences from one token to 300,000: the keys are cut by the real lengths, and a query in one piece, or
    with inverse RoPE through the merge, answers the same."""
    pos = [5, 299999, 130, 90001, 0, 3000, 128 * 64, 40000]
    s = Setup(ck, "hca", d_qk, d_v, H, list(range(8)), pos, fp8=fp8, seed=21)
    _both(s, rules=RULES[:2])
    out, lse = s.run(30.0, s.slopes, rope_dims=64)
    s.check(out, lse, 30.0, s.slopes, rope=64)


@pytest.mark.parametrize("H", [16, 48, 64])
def test_single_tokens_beside_a_chunk(ck, H):
    """Decode tokens of many sequences in one call with a chunk: next to each other, they share no key."""
    chunk, seqs, pos = {0: (0, 900, 330)}, [0] * 330, list(range(900, 1230))
    for s in range(1, 41):
        seqs.append(s)
        pos.append((s * 977) % 6000)
        if s % 3:  # its token in the chunk's rows; the others' in the ring
            chunk[s] = (329 + s, pos[-1], 1)
    order = list(range(0, 330, 2)) + list(range(330, 370)) + list(range(1, 330, 2))  # the chunk's tokens on both sides
    s = Setup(ck, "hca", 128, 128, H, [seqs[i] for i in order], [pos[i] for i in order], seed=H + 22, chunk=chunk)
    s.q_pos[180] = -1  # one of the single tokens is invalid: zeros, and its neighbours as ever
    for cap, bias in RULES[:3]:
        slopes = s.slopes if bias else None
        out, lse = s.run(cap, slopes, want=ck.ERR_INVALID_ARG)
        assert not bool(out[180].any()) and bool((lse[180] == -math.inf).all())
        s.check(out, lse, cap, slopes, [0, 1, 77, 164] + [i for i in range(165, 205) if i != 180] + [205, 206, 300, 369])
