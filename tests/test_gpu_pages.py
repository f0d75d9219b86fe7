"""GPU tests of the page operators (fork, free, reserve, compact) against a plain sequential model: tables,
counts, pools and rings are compared bit for bit after every call of random call sequences, and refusals leave
everything as it was."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

POOLS = ("kv_pool", "kv_scale", "idx_pool", "idx_scale")
RINGS = ("ring_x", "ring_z", "ring_xi", "ring_zi")


@pytest.fixture(scope="module")
def ck(cskv_built):
    import compressed_sparse_kv_02_b200 as ck
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ck


def _bytes(t):
    return t.detach().contiguous().view(torch.uint8).cpu().numpy().copy()


def make(ck, kind="csa", m=4, d=128, d_v=128, d_idx=64, page_size=64, n_seqs=6, n_pages=40, max_pages=8, n_win=128,
         fp8=False, fp4=False, gate=None, seed=0, fill=True):
    L = ck.Layer.allocate(ck.LAYER_CSA if kind == "csa" else ck.LAYER_HCA, m, d, d_v, n_seqs, n_pages, max_pages,
                          page_size=page_size, n_win=n_win, d_idx=d_idx if kind == "csa" else 0,
                          kv_dtype=ck.FP8_E4M3 if fp8 else ck.BF16, idx_dtype=ck.FP4_E2M1 if fp4 else ck.BF16,
                          gate_cols=gate, gate_cols_idx=gate)
    if fill:
        g = torch.Generator(device="cuda").manual_seed(seed)
        for name in POOLS + RINGS:
            t = getattr(L, name)
            if t is not None:
                v = t.view(torch.uint8)
                v.copy_(torch.randint(0, 256, v.shape, generator=g, device="cuda", dtype=torch.uint8))
    L.track_pages()
    return L


class Model:
    """The operators' definition, one step at a time, on host copies."""

    def __init__(self, L):
        self.P, self.n_pages, self.width = L.page_size, L.n_pages, L.max_pages_per_seq
        self.table = L.page_table.cpu().numpy().copy()
        self.refs = L.page_refs.cpu().numpy().copy()
        self.pools = {n: _bytes(getattr(L, n)).reshape(L.n_pages, -1) for n in POOLS if getattr(L, n) is not None}
        self.rings = {n: _bytes(getattr(L, n)).reshape(L.n_seqs, -1) for n in RINGS if getattr(L, n) is not None}

    def free(self, seqs, keep):
        for s, n in zip(seqs, keep):
            for k in range(-(-n // self.P), self.width):
                if self.table[s, k] >= 0:
                    self.refs[self.table[s, k]] -= 1
                    self.table[s, k] = -1

    def fork(self, src, dst, n):
        for s, d, e in zip(src, dst, n):
            self.free([d], [0])
            for k in range(-(-e // self.P)):
                self.table[d, k] = self.table[s, k]
                self.refs[self.table[s, k]] += 1
            for r in self.rings.values():
                r[d] = r[s]

    def reserve(self, seqs, first, count):
        before = self.refs.copy()
        asked = []
        for s, f, c in zip(seqs, first, count):
            if c:
                for k in range(f // self.P, (f + c - 1) // self.P + 1):
                    p = self.table[s, k]
                    if p < 0 or before[p] > 1:
                        asked.append((s, k, p))
        free = np.flatnonzero(before == 0)
        if len(asked) > len(free):
            return False
        for (s, k, p), new in zip(asked, free):
            if p >= 0:
                self.refs[p] -= 1
                for a in self.pools.values():
                    a[new] = a[p]
            self.table[s, k] = new
            self.refs[new] = 1
        return True

    def check(self, L, what=""):
        assert np.array_equal(L.page_table.cpu().numpy(), self.table), what
        assert np.array_equal(L.page_refs.cpu().numpy(), self.refs), what
        for n, a in self.pools.items():
            assert np.array_equal(_bytes(getattr(L, n)).reshape(L.n_pages, -1), a), (what, n)
        for n, a in self.rings.items():
            assert np.array_equal(_bytes(getattr(L, n)).reshape(L.n_seqs, -1), a), (what, n)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def i64(v):
    return torch.tensor(v, dtype=torch.int64, device="cuda")


class Both:
    """Runs every call on the GPU and on the model, and compares."""

    def __init__(self, ck, L):
        self.ck, self.L, self.m = ck, L, Model(L)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _end(self, want, what):
        assert self.ck.cskv_get_status(self.status) == want, what
        self.m.check(self.L, what)

    def fork(self, src, dst, n):
        self.ck.cskv_cache_fork(self.L, i32(src), i32(dst), i64(n), status=self.status)
        self.m.fork(src, dst, n)
        self._end(self.ck.OK, "fork")

    def free(self, seqs, keep):
        self.ck.cskv_cache_free(self.L, i32(seqs), i64(keep), status=self.status)
        self.m.free(seqs, keep)
        self._end(self.ck.OK, "free")

    def reserve(self, seqs, first, count, most=None):
        self.ck.cskv_cache_reserve(self.L, i32(seqs), i64(first), i64(count), max(count) if most is None else most,
                                   status=self.status)
        ok = self.m.reserve(seqs, first, count)
        self._end(self.ck.OK if ok else self.ck.ERR_NO_PAGES, "reserve")
        return ok


SHAPES = [
    dict(),
    dict(kind="hca", m=128, d=576, d_v=512, page_size=16),
    dict(d=576, d_v=512, d_idx=128, fp8=True, fp4=True, page_size=48),
    dict(d=144, d_v=16, d_idx=32, gate=1, n_win=33, page_size=64, fp4=True),  # rings of 66 bytes: no 16-byte copies
]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_random_calls(ck, shape):
    L = make(ck, seed=shape, n_seqs=9, n_pages=47, max_pages=8, **SHAPES[shape])
    b = Both(ck, L)
    P, cap = L.page_size, 8 * L.page_size
    rng = np.random.default_rng(shape)
    length = [0] * 9  # entries each sequence has room for
    full = 0
    for step in range(60):
        op = rng.integers(0, 4)
        if op == 0:
            src = int(rng.integers(0, 9))
            dst = [int(d) for d in rng.permutation(9) if d != src][: int(rng.integers(1, 4))]
            n = [int(rng.integers(0, length[src] + 1)) for _ in dst]
            b.fork([src] * len(dst), dst, n)
            for d, e in zip(dst, n):
                length[d] = e
        elif op == 1:
            seqs = [int(s) for s in rng.permutation(9)[: int(rng.integers(1, 4))]]
            keep = [int(rng.integers(0, cap + 1)) for _ in seqs]
            b.free(seqs, keep)
            for s, k in zip(seqs, keep):
                length[s] = min(length[s], k)
        else:
            seqs = [int(s) for s in rng.permutation(9)[: int(rng.integers(1, 6))]]
            first = [int(rng.integers(0, length[s] + 1)) for s in seqs]
            count = [int(min(cap - f, rng.integers(0, 2 * P + 2))) for f in first]
            if b.reserve(seqs, first, count, most=2 * P + 2):
                for s, f, c in zip(seqs, first, count):
                    length[s] = max(length[s], f + c)
            else:
                full += 1
    assert full < 40


def test_page_edges(ck):
    """Counts of 0, 1, a whole page and one more; first at, before and after a page's end; the whole table row."""
    L = make(ck, n_seqs=5, n_pages=21, max_pages=4)
    b = Both(ck, L)
    b.reserve([0, 1, 2, 3], [0, 0, 0, 0], [0, 1, 64, 65], most=256)
    b.reserve([0, 1, 2, 3], [0, 1, 64, 65], [256, 63, 1, 63], most=256)
    b.reserve([1, 2], [64, 65], [192, 191], most=192)
    b.free([0, 0, 3], [200, 64, 0])  # the same sequence twice keeps the smaller part
    b.fork([1, 1, 2], [0, 3, 4], [256, 0, 63])
    b.reserve([0, 3, 4], [255, 0, 63], [1, 1, 1])


def test_every_holder_reserves(ck):
    """All holders of a shared page reserve it in one call: each gets a copy and the page becomes free."""
    L = make(ck, n_seqs=4, n_pages=12, max_pages=2)
    b = Both(ck, L)
    b.reserve([0], [0], [70])
    b.fork([0, 0], [1, 2], [70, 70])
    b.reserve([0, 1, 2], [70, 70, 70], [1, 1, 1])
    assert sorted(np.flatnonzero(b.m.refs == 0).tolist())[:1] == [1]


def test_many_pages_and_sequences(ck):
    """Ranks over several 4096-count chunks, rows wider than a block, hundreds of sequences in one call."""
    L = make(ck, kind="hca", m=128, d=16, d_v=16, gate=1, n_win=128, page_size=16, n_seqs=700, n_pages=21001,
             max_pages=1100, seed=5)
    b = Both(ck, L)
    rng = np.random.default_rng(1)
    seqs = rng.permutation(700).tolist()
    b.reserve(seqs, [0] * 700, rng.integers(0, 16 * 29, 700).tolist(), most=16 * 29)
    b.free(seqs[::3], rng.integers(0, 16 * 29, len(seqs[::3])).tolist())
    b.reserve([seqs[0]], [0], [16 * 1100])
    b.fork([seqs[0]] * 3, seqs[1:4], [16 * 1100, 17000, 5])
    b.reserve(seqs[:4], [17500, 0, 16999, 5], [100, 16 * 40, 16, 11], most=16 * 40)


def test_the_longest_list(ck):
    """4096 sequences in one call, and one of them listed twice."""
    L = make(ck, kind="hca", m=128, d=16, d_v=16, gate=1, n_win=128, page_size=16, n_seqs=4097, n_pages=4200, max_pages=2)
    b = Both(ck, L)
    seqs = np.random.default_rng(2).permutation(4097)[:4096].tolist()
    b.reserve(seqs, [0] * 4096, [1] * 4096)
    b.free(seqs, [0] * 4096)
    seqs[4095] = seqs[17]
    _refused(ck, b, ck.ERR_INVALID_ARG,
             lambda: ck.cskv_cache_reserve(L, i32(seqs), i64([0] * 4096), i64([1] * 4096), 1, status=b.status))


def test_no_pages_changes_nothing(ck):
    L = make(ck, n_seqs=4, n_pages=5, max_pages=4)
    b = Both(ck, L)
    assert b.reserve([0, 1], [0, 0], [129, 64])
    assert not b.reserve([2, 3], [0, 0], [65, 1])
    assert b.reserve([2], [0], [64])
    b.free([0], [64])
    assert b.reserve([2, 3], [64, 0], [1, 1])


def _refused(ck, b, code, call):
    call()
    assert ck.cskv_get_status(b.status) == code
    b.m.check(b.L)


def test_refused_requests_change_nothing(ck):
    L = make(ck, n_seqs=4, n_pages=12, max_pages=4)
    b = Both(ck, L)
    b.reserve([0, 1], [0, 0], [130, 10])
    st, end = b.status, 4 * 64
    R, BAD, OUT = ck.cskv_cache_reserve, ck.ERR_INVALID_ARG, ck.ERR_OUT_OF_RANGE
    for seqs, first, count, code in (([2, 2], [0, 0], [1, 1], BAD), ([2, 4], [0, 0], [1, 1], OUT),
                                     ([2, -1], [0, 0], [1, 1], OUT), ([2, 3], [0, -1], [1, 1], BAD),
                                     ([2, 3], [0, 0], [1, -1], BAD), ([2, 3], [0, 0], [1, 101], BAD),
                                     ([2, 3], [0, end], [1, 1], BAD), ([2, 3], [0, 1 << 62], [1, 1], BAD)):
        _refused(ck, b, code, lambda: R(L, i32(seqs), i64(first), i64(count), 100, status=st))
    F = ck.cskv_cache_fork
    for src, dst, n, code in (([0], [0], [1], BAD), ([0, 1], [1, 2], [1, 1], BAD), ([0, 1], [2, 2], [1, 1], BAD),
                              ([0], [4], [1], OUT), ([-1], [2], [1], OUT), ([0], [2], [-1], BAD),
                              ([0], [2], [end + 1], BAD)):
        def call():
            F(L, i32(src), i32(dst), i64(n), status=st)
            if src == [0, 1] and dst == [1, 2]:  # the good entry of the list is carried out
                b.m.fork([1], [2], [1])
        _refused(ck, b, code, call)
    for seqs, keep, code in (([4], [0], OUT), ([-1], [0], OUT), ([0], [-1], BAD), ([0], [end + 1], BAD)):
        _refused(ck, b, code, lambda: ck.cskv_cache_free(L, i32(seqs), i64(keep), status=st))


def test_bad_table_slots_are_reported(ck):
    """A slot that names a page outside the pool or a free page: reported, never followed."""
    L = make(ck, n_seqs=4, n_pages=6, max_pages=2)
    b = Both(ck, L)
    b.reserve([0], [0], [70])
    for bad in (6, 1 << 30, 5):  # past the pool, far past it, free
        L.page_table[1, 0] = bad
        b.m.table[1, 0] = bad
        _refused(ck, b, ck.ERR_OUT_OF_RANGE,
                 lambda: ck.cskv_cache_reserve(L, i32([1]), i64([0]), i64([1]), 1, status=b.status))
        ck.cskv_cache_fork(L, i32([1]), i32([2]), i64([1]), status=b.status)
        for r in b.m.rings.values():
            r[2] = r[1]
        assert ck.cskv_get_status(b.status) == ck.ERR_OUT_OF_RANGE
        b.m.check(L)  # the branch's slot stays -1
        ck.cskv_cache_free(L, i32([1]), i64([0]), status=b.status)
        assert ck.cskv_get_status(b.status) == ck.ERR_OUT_OF_RANGE
        b.m.table[1, 0] = -1
        b.m.check(L)


@pytest.mark.parametrize("shape", range(3))
def test_compact(ck, shape):
    kw = SHAPES[shape]
    L = make(ck, seed=shape, n_seqs=6, n_pages=50, max_pages=9, **kw)
    b = Both(ck, L)
    P = L.page_size
    b.reserve([0, 1, 2, 3], [0] * 4, [9 * P, 5 * P, 1, 7 * P], most=9 * P)
    b.free([0, 1], [3 * P, 0])
    b.fork([3], [4], [6 * P + 1])
    live = np.flatnonzero(b.m.refs > 0)
    for n_pages, width in ((live.size, 9), (live.size + 7, 12), (live.size - 1, 9)):
        D = make(ck, seed=77, n_seqs=6, n_pages=n_pages, max_pages=width, **kw)
        old = Model(D)
        D.page_refs.fill_(3)
        D.page_table.fill_(5)
        ck.cskv_cache_compact(L, D, status=b.status)
        if n_pages < live.size:
            assert ck.cskv_get_status(b.status) == ck.ERR_NO_PAGES
            old.refs[:], old.table[:] = 3, 5
            old.check(D)
            continue
        assert ck.cskv_get_status(b.status) == ck.OK
        to = np.full(L.n_pages, -1)
        to[live] = np.arange(live.size)
        want = np.full((6, width), -1)
        want[:, :9] = np.where(b.m.table >= 0, to[b.m.table], -1)
        old.table, old.refs = want, np.concatenate([b.m.refs[live], np.zeros(n_pages - live.size, np.int32)])
        for n, a in old.pools.items():
            a[: live.size] = b.m.pools[n][live]
        old.check(D)
        b.m.check(L)  # the source is left as it was


def test_compact_empty_and_bad_slot(ck):
    L = make(ck, n_seqs=2, n_pages=9000, max_pages=3, kind="hca", d=16, d_v=16, gate=1, page_size=16)
    D = make(ck, n_seqs=2, n_pages=1, max_pages=3, kind="hca", d=16, d_v=16, gate=1, page_size=16)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ck.cskv_cache_compact(L, D, status=st)
    assert ck.cskv_get_status(st) == ck.OK and int(D.page_refs[0]) == 0 and int(D.page_table.max()) == -1
    L.page_table[0, 0], L.page_refs[8999] = 8999, 1
    L.page_table[1, 1], L.page_table[1, 2] = 17, 9000  # a free page, a page outside the pool
    ck.cskv_cache_compact(L, D, status=st)
    assert ck.cskv_get_status(st) == ck.ERR_OUT_OF_RANGE
    assert D.page_table.tolist() == [[0, -1, -1], [-1, -1, -1]]
    assert np.array_equal(_bytes(D.kv_pool), _bytes(L.kv_pool[-16:]))


def test_captured_calls_replay(ck):
    """fork + reserve + free captured in one graph, replayed on a changed list: counts come back each time."""
    L = make(ck, n_seqs=5, n_pages=30, max_pages=4)
    b = Both(ck, L)
    b.reserve([0, 1], [0, 0], [100, 20], most=100)
    src, dst, n, c = i32([0, 0]), i32([2, 3]), i64([100, 70]), i64([40, 1])
    zero = i64([0, 0])
    ws = torch.empty(ck.cskv_reserve_ws_bytes(L, 2, 40), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ck.cskv_cache_free(L, dst, zero, status=b.status)
        ck.cskv_cache_fork(L, src, dst, n, status=b.status)
        ck.cskv_cache_reserve(L, dst, n, c, 40, workspace=ws, status=b.status)
    for s, lens in (([0, 0], [100, 70]), ([1, 0], [20, 64]), ([0, 0], [100, 70])):
        src.copy_(i32(s))
        n.copy_(i64(lens))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.m.free([2, 3], [0, 0])
        b.m.fork(s, [2, 3], lens)
        assert b.m.reserve([2, 3], lens, [40, 1])
        b._end(ck.OK, "replay")
    del graph


def test_branches_decode_as_their_sources(ck):
    """A run of the operators as a server uses them: a prompt, three branches of it, a token appended to each,
    attention over every branch, the pool compacted, attention again. Branches with the same token answer alike,
    the source's own entries stay untouched by its branches, and compaction changes no bit of any answer."""
    m, d, H, P = 4, 128, 16, 16
    L = make(ck, m=m, d=d, d_v=d, d_idx=64, page_size=P, n_seqs=4, n_pages=60, max_pages=20, fill=False)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    n = 1000  # prompt tokens: 250 entries, the last page partly filled
    one = i32([0])
    x, z, xi, zi = rand(1, n, d), rand(1, n, d), rand(1, n, 64), rand(1, n, 64)
    ck.cskv_cache_reserve(L, one, i64([0]), i64([n // m]), n // m, status=st)
    ck.csa_compress_kv(L, one, 0, x, z, xi, zi, status=st)
    tail = [v[:, n - 128:].contiguous() for v in (x, z, xi, zi)]
    ck.cskv_cache_append(L, one, i64([n - 128]), *tail, ring_only=True, status=st)
    ck.cskv_cache_fork(L, i32([0, 0, 0]), i32([1, 2, 3]), i64([n // m] * 3), status=st)
    before = L.read_entries(0, n // m)["kv"].clone()
    seqs = i32([0, 1, 2, 3])
    new = [rand(1, 4, w).repeat(4, 1, 1) for w in (d, d, 64, 64)]
    for v in new:
        v[3] = rand(*v[3].shape)  # the last branch takes another continuation
    pos = i64([n] * 4)
    ck.cskv_cache_reserve(L, seqs, i64([n // m] * 4), i64([1] * 4), 1, status=st)
    ck.cskv_cache_append(L, seqs, pos, *new, status=st)
    assert ck.cskv_get_status(st) == ck.OK
    assert torch.equal(L.read_entries(0, n // m)["kv"], before)
    for s in (1, 2, 3):
        assert torch.equal(L.read_entries(s, n // m)["kv"], before)
    t = n + 3
    q = rand(1, H, d).repeat(4, 1, 1)
    qi, w = rand(1, 4, 64).repeat(4, 1, 1), torch.rand(1, 4, generator=g, device="cuda").repeat(4, 1)

    def answer(layer):
        idx, cnt = torch.zeros(4, 64, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
        out = torch.zeros(4, H, d, dtype=torch.bfloat16, device="cuda")
        ck.csa_index_score_topk(layer, seqs, i64([t] * 4), t, qi, w, 64, idx, cnt, status=st)
        ck.csa_attend(layer, seqs, i64([t] * 4), t, q, idx, cnt, out, status=st)
        assert ck.cskv_get_status(st) == ck.OK
        return out

    a = answer(L)
    assert torch.equal(a[0], a[1]) and torch.equal(a[0], a[2]) and not torch.equal(a[0], a[3])
    live = int((L.page_refs > 0).sum())
    D = make(ck, m=m, d=d, d_v=d, d_idx=64, page_size=P, n_seqs=4, n_pages=live, max_pages=20, fill=False)
    D.ring_x, D.ring_z, D.ring_xi, D.ring_zi = L.ring_x, L.ring_z, L.ring_xi, L.ring_zi
    ck.cskv_cache_compact(L, D, status=st)
    assert ck.cskv_get_status(st) == ck.OK
    assert torch.equal(answer(D), a)
    ck.cskv_cache_free(D, seqs, i64([0] * 4), status=st)
    assert ck.cskv_get_status(st) == ck.OK
    assert int(D.page_refs.abs().max()) == 0 and int(D.page_table.max()) == -1
