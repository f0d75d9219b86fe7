"""What is measured of the page operators (fork, free, reserve, compact) and of the attention with capped
scores and a distance bias, decode and chunk: the cases, their inputs, their plain forms and their calls.

Plain forms are elementary torch operations in 32 bits; `exact` computes the floating outputs in 64 bits
from the definition. With `own` set, `run` makes the library's calls.

Layouts are those of the library's paged cache: pool row = page * page_size + slot, rings of n_win raw rows.
"""
import math

import torch

own = False

DEV = "cuda"
N_WIN = 128
PAGE = 64

# Latent widths and storage of the repository's configurations: (d_qk, d_v, d_idx, kv, idx)
SHAPES = {
    "flash": (128, 128, 64, "bf16", "bf16"),    # the narrow latent (tiny, flash and prefill workloads)
    "pro": (576, 512, 128, "bf16", "bf16"),     # the 512 + 64 channel latent
    "mixed": (576, 512, 128, "fp8", "fp4"),     # the same with FP8 entries and FP4 indexer keys
}


def listed():
    return [
        # one sequence of the tiny workload's length gets one branch (a retry of one answer): latency
        dict(name="branch tiny", op="branch", shape="flash", kind="csa", sources=1, branches=1, ctx=8185, count=2),
        # eight prompts of 128K tokens, seven sampled answers each, on the wide latent
        dict(name="branch beams", op="branch", shape="pro", kind="csa", sources=8, branches=7, ctx=131071, count=3),
        # one sequence drops a rejected draft and makes room for the next: latency
        dict(name="regrow one", op="regrow", shape="flash", kind="hca", seqs=1, ctx=4099, drop=1, count=40),
        # the mixed workload's 64 sequences: each gives back a draft and reserves a prefill chunk's room
        dict(name="regrow mixed", op="regrow", shape="mixed", kind="csa", seqs=64, ctx=65536, drop=1500, count=4100),
        # a small pool of the narrow latent after a few sequences have ended
        dict(name="compact small", op="compact", shape="flash", kind="hca", seqs=5, pages=37, spare=3),
        # a pool of the wide latent, half of it free, moved into a smaller one
        dict(name="compact pool", op="compact", shape="pro", kind="csa", seqs=24, pages=12000, spare=16),
        # one token of the tiny workload: latency
        dict(name="hca token", op="attend", shape="flash", kind="hca", heads=16, seqs=1, ctx=8185, chunk=0, k=0, cap=30.0,
             bias=True),
        # one token of each of the flash workload's 32 sequences, lengths from 4K to 128K
        dict(name="csa flash", op="attend", shape="flash", kind="csa", heads=32, seqs=32, ctx=131072, chunk=0, k=512,
             cap=50.0, bias=True),
        # one token of each of the pro workload's 8 sequences, the longest at 1M tokens
        dict(name="hca pro", op="attend", shape="pro", kind="hca", heads=128, seqs=8, ctx=1048576, chunk=0, k=0, cap=50.0,
             bias=False),
        # the mixed workload's 64 sequences, FP8 entries
        dict(name="csa mixed", op="attend", shape="mixed", kind="csa", heads=128, seqs=64, ctx=262144, chunk=0, k=1024,
             cap=0.0, bias=True),
        # a block of the prefill workload: 4096 new tokens on 61,440 cached ones
        dict(name="hca chunk", op="attend", shape="flash", kind="hca", heads=64, seqs=1, ctx=65536, chunk=4096, k=0,
             cap=50.0, bias=True),
        # a ragged chunk through the selection
        dict(name="csa chunk", op="attend", shape="flash", kind="csa", heads=64, seqs=1, ctx=30011, chunk=1001, k=512,
             cap=30.0, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["branch", "regrow", "compact", "decode", "decode", "chunk", "chunk"])
    kind = rng.choice(["csa", "hca"])
    if op == "branch":
        return dict(op=op, shape=rng.choice(["flash", "pro", "mixed"]), kind=kind, sources=rng.randint(1, 8),
                    branches=rng.randint(1, 7), ctx=_log_int(rng, 130, 131071), count=rng.randint(1, 100))
    if op == "regrow":
        return dict(op=op, shape=rng.choice(["flash", "pro", "mixed"]), kind=kind, seqs=rng.randint(1, 64),
                    ctx=_log_int(rng, 1000, 65536), drop=rng.randint(0, 2000), count=_log_int(rng, 1, 4100))
    if op == "compact":
        return dict(op=op, shape=rng.choice(["flash", "pro", "mixed"]), kind=kind, seqs=rng.randint(1, 24),
                    pages=_log_int(rng, 8, 12000), spare=rng.randint(0, 64))
    cap = rng.choice([0.0, 20.0, 30.0, 50.0])
    bias = True if cap == 0.0 else rng.choice([True, False])
    k = 0 if kind == "hca" else rng.choice([64, 300, 512])
    if op == "chunk":
        n = _log_int(rng, 5, 4096)
        return dict(op="attend", shape="flash", kind=kind, heads=rng.choice([16, 32, 64, 64]), seqs=1,
                    ctx=n + _log_int(rng, 1, 61440), chunk=n, k=k, cap=cap, bias=bias)
    if rng.random() < 0.5:
        return dict(op="attend", shape="flash", kind=kind, heads=rng.choice([16, 32, 64]), seqs=rng.randint(1, 48),
                    ctx=_log_int(rng, 1, 262144), chunk=0, k=k, cap=cap, bias=bias)
    return dict(op="attend", shape=rng.choice(["pro", "mixed"]), kind=kind, heads=rng.choice([32, 64, 128]),
                seqs=rng.randint(1, 16), ctx=_log_int(rng, 1, 524288), chunk=0, k=0 if kind == "hca" else 1024, cap=cap,
                bias=bias)


# ------------------------------------------------------------------------------------------- sizes
def _m(case):
    return 4 if case["kind"] == "csa" else 128


def _pages(entries):
    return -(-entries // PAGE)


def _lens(case):
    """Sequence lengths: the first is ctx, the others spread down to ctx / 32 (at least 1)."""
    n, ctx = case["seqs"], case["ctx"]
    return [max(1, int(round(ctx * 32.0 ** (-b / max(1, n - 1))))) for b in range(n)]


def _visible(t, m):
    lim = t + 1 - N_WIN
    return 0 if lim <= 0 else -(-lim // m)


def _page_bytes(case):
    d_qk, _, d_idx, kv, idx = SHAPES[case["shape"]]
    b = d_qk * 2 if kv == "bf16" else d_qk + 4
    if case["kind"] == "csa":
        b += d_idx * 2 if idx == "bf16" else d_idx // 2 + d_idx // 16
    return PAGE * b


def _ring_bytes(case):
    d_qk, _, d_idx, _, _ = SHAPES[case["shape"]]
    return N_WIN * 2 * (2 * d_qk + (2 * d_idx if case["kind"] == "csa" else 0))


def _branch_sizes(case):
    e = case["ctx"] // _m(case)
    have, most = _pages(e), _pages(e + case["count"])
    n = case["sources"] * case["branches"]
    return e, have, most, n, case["sources"] * have + n * (most - have + 1) + 5


def _regrow_sizes(case):
    es = [c // _m(case) for c in _lens(case)]
    keep = [max(0, e - case["drop"]) for e in es]
    return es, keep, [_pages(k + case["count"]) for k in keep]


def _compact_sizes(case):
    """Pages of each sequence: shares of `pages`, every odd one beginning with half of its neighbour's pages."""
    n = case["seqs"]
    each = [max(1, case["pages"] * (i + 1) * 2 // (n * (n + 1))) for i in range(n)]
    shared = [each[i - 1] // 2 if i % 2 and each[i] > each[i - 1] // 2 else 0 for i in range(n)]
    return each, shared, sum(e - s for e, s in zip(each, shared))


def work(case):
    if case["op"] == "branch":
        e, have, most, n, pool = _branch_sizes(case)
        copied = 1 if e % PAGE else 0
        return dict(bytes=(case["sources"] + n) * _ring_bytes(case) + copied * (case["sources"] + n) * _page_bytes(case) +
                    (case["sources"] * have + 2 * n * most + pool) * 4, flops=0)
    if case["op"] == "regrow":
        es, keep, grown = _regrow_sizes(case)
        return dict(bytes=(sum(grown) * 2 + sum(grown) + 8) * 4, flops=0)
    if case["op"] == "compact":
        each, _, live = _compact_sizes(case)
        return dict(bytes=2 * live * _page_bytes(case) + (3 * live + 2 * sum(each)) * 4, flops=0)
    d_qk, d_v, _, kv, _ = SHAPES[case["shape"]]
    row = d_qk * 2 if kv == "bf16" else d_qk + 4
    m, h = _m(case), case["heads"]
    if case["chunk"]:
        n_q = case["chunk"]
        ts = range(case["ctx"] - n_q, case["ctx"])
        vis = _visible(case["ctx"] - 1, m)
        read = (min(case["ctx"], n_q + N_WIN - 1)) * d_qk * 2
        read += (min(vis, sum(min(_visible(t, m), case["k"]) for t in ts)) if case["k"] else vis) * row
    else:
        n_q = case["seqs"]
        ts = [c - 1 for c in _lens(case)]
        read = sum(min(t + 1, N_WIN) * d_qk * 2 + (min(_visible(t, m), case["k"]) if case["k"] else _visible(t, m)) * row
                   for t in ts)
    keys = sum(min(t + 1, N_WIN) + (min(_visible(t, m), case["k"]) if case["k"] else _visible(t, m)) for t in ts)
    return dict(bytes=read + n_q * h * ((d_qk + d_v) * 2 + 4) + n_q * 4 * case["k"], flops=2 * h * (d_qk + d_v) * keys)


# ------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape, std=1.0, dtype=torch.bfloat16):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV, dtype=torch.bfloat16) * std)
    return out


def _pool(g, case, n_pages, std=1.0, keys=False):
    """Pools of n_pages pages with stored entries: bf16, or FP8 codes with a scale per entry; indexer keys (CSA)."""
    d_qk, _, d_idx, kv, idx = SHAPES[case["shape"]]
    rows = n_pages * PAGE
    p = {}
    if kv == "bf16":
        p["kv_pool"] = _randn(g, rows, d_qk, std=std)
    else:
        p["kv_pool"] = _randn(g, rows, d_qk, std=100.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        p["kv_scale"] = (torch.rand(rows, generator=g, device=DEV) + 0.5) * (std / 100.0)
    if case["kind"] == "csa" and keys:
        if idx == "bf16":
            p["idx_pool"] = _randn(g, rows, d_idx)
        else:
            p["idx_pool"] = torch.randint(0, 256, (rows, d_idx // 2), generator=g, device=DEV, dtype=torch.uint8)
            p["idx_scale"] = torch.randint(40, 72, (rows, d_idx // 16), generator=g, device=DEV, dtype=torch.uint8)
    return p


def _rings(g, case, n_seqs, std=1.0):
    d_qk, _, d_idx, _, _ = SHAPES[case["shape"]]
    r = dict(ring_x=_randn(g, n_seqs, N_WIN, d_qk, std=std), ring_z=_randn(g, n_seqs, N_WIN, d_qk))
    if case["kind"] == "csa":
        r["ring_xi"] = _randn(g, n_seqs, N_WIN, d_idx)
        r["ring_zi"] = _randn(g, n_seqs, N_WIN, d_idx)
    return r


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


def _table(g, counts, width, n_pages, shared=None):
    """A page table whose rows own `counts` pages of a random permutation, and the pages' reference counts."""
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, c in enumerate(counts):
        s = shared[i] if shared else 0
        if s:
            table[i, :s] = table[i - 1, :s]
        table[i, s:c] = perm[at:at + c - s]
        at += c - s
    flat = table.view(-1)
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device=DEV)
    refs.scatter_add_(0, torch.where(flat >= 0, flat, n_pages).long(), torch.ones_like(flat))
    return table, refs[:n_pages].clone()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    st = dict(case=case)
    if case["op"] == "branch":
        e, have, most, n, pool = _branch_sizes(case)
        src = case["sources"]
        st["page_table"], st["page_refs"] = _table(g, [have] * src + [0] * n, most, pool)
        st.update(_pool(g, case, pool, keys=True))
        st.update(_rings(g, case, src + n))
        st["src"] = _i32([i // case["branches"] for i in range(n)])
        st["dst"] = _i32([src + i for i in range(n)])
        st["n_entries"] = _i64([e] * n)
        st["count"] = _i64([case["count"]] * n)
    elif case["op"] == "regrow":
        es, keep, grown = _regrow_sizes(case)
        most = [max(_pages(e), p) for e, p in zip(es, grown)]
        st["page_table"], st["page_refs"] = _table(g, [_pages(e) for e in es], max(most), sum(most) + 8)
        st.update(_pool(g, case, sum(most) + 8, keys=True))
        st.update(_rings(g, case, case["seqs"]))
        st["seq"] = _i32(list(range(case["seqs"])))
        st["keep"] = _i64(keep)
        st["count"] = _i64([case["count"]] * case["seqs"])
    elif case["op"] == "compact":
        each, shared, live = _compact_sizes(case)
        st["page_table"], st["page_refs"] = _table(g, each, max(each) + 1, 2 * live, shared)
        st.update(_pool(g, case, 2 * live, keys=True))
        st.update(_rings(g, case, case["seqs"]))
        st["dst"] = {k: torch.zeros(((live + case["spare"]) * PAGE,) + tuple(v.shape[1:]), dtype=v.dtype, device=DEV)
                     for k, v in st.items() if k in ("kv_pool", "kv_scale", "idx_pool", "idx_scale")}
        st["dst"]["page_table"] = torch.zeros_like(st["page_table"])
        st["dst"]["page_refs"] = torch.zeros(live + case["spare"], dtype=torch.int32, device=DEV)
    else:
        d_qk, d_v, _, _, _ = SHAPES[case["shape"]]
        m, h = _m(case), case["heads"]
        lens = _lens(case)
        counts = [_pages(c // m) + 1 for c in lens]
        st["page_table"], st["page_refs"] = _table(g, counts, max(counts), sum(counts) + 3)
        # queries ~ N(0, 1) on keys of standard deviation 2: logits of a few units, as after training
        st.update(_pool(g, case, sum(counts) + 3, std=2.0))
        st["ring_x"] = _randn(g, case["seqs"], N_WIN, d_qk, std=2.0)
        if case["chunk"]:
            n_q, pos0 = case["chunk"], case["ctx"] - case["chunk"]
            st["q_seq"], st["q_pos"] = _i32([0] * n_q), torch.arange(pos0, case["ctx"], device=DEV)
            st["x_chunk"], st["pos0"] = _randn(g, n_q, d_qk, std=2.0), pos0
        else:
            n_q = case["seqs"]
            st["q_seq"], st["q_pos"] = _i32(list(range(n_q))), _i64([c - 1 for c in lens])
        st["max_pos"] = max(lens) - 1
        st["q"] = _randn(g, n_q, h, d_qk, std=2.0)
        st["sm_scale"] = 1.0 / math.sqrt(d_qk)
        st["slopes"] = None
        if case["bias"]:  # from 1/2 down to 2^-16: some heads look near, some across the whole context
            st["slopes"] = torch.exp2(-1.0 - torch.arange(h, device=DEV, dtype=torch.float32) * (15.0 / (h - 1)))
        if case["k"]:
            vis = torch.tensor([_visible(t, m) for t in st["q_pos"].tolist()], device=DEV)
            wide = max(int(vis.max()), case["k"])
            j = torch.arange(wide, device=DEV)
            key = torch.rand(n_q, wide, generator=g, device=DEV).masked_fill_(j[None] >= vis[:, None], -1.0)
            top = key.topk(case["k"], dim=1).indices
            top = torch.where(top < vis[:, None], top, wide).sort(dim=1).values
            st["sel_idx"] = torch.where(top < wide, top, -1).to(torch.int32)
            st["sel_cnt"] = vis.clamp(max=case["k"]).to(torch.int32)
        st["out"] = torch.empty(n_q, h, d_v, dtype=torch.bfloat16, device=DEV)
        st["lse"] = torch.empty(n_q, h, dtype=torch.float32, device=DEV)
    return st


# ------------------------------------------------------------------------------------------- plain forms
POOLS = ("kv_pool", "kv_scale", "idx_pool", "idx_scale")
RINGS = ("ring_x", "ring_z", "ring_xi", "ring_zi")


def _plain_release(table, refs, seqs, gone):
    """Give back the pages of rows `seqs` where `gone` [n, width] says so."""
    rows = table[seqs.long()]
    gone = gone & (rows >= 0)
    refs.scatter_add_(0, rows.clamp(min=0).long().view(-1), -gone.view(-1).to(torch.int32))
    table[seqs.long()] = torch.where(gone, -1, rows)


def _plain_fork(st):
    table, refs = st["page_table"], st["page_refs"]
    slot = torch.arange(table.shape[1], device=DEV)
    _plain_release(table, refs, st["dst"], slot[None] >= 0)
    used = slot[None] < ((st["n_entries"] + PAGE - 1) // PAGE)[:, None]
    rows = torch.where(used, table[st["src"].long()], -1)
    refs.scatter_add_(0, rows.clamp(min=0).long().view(-1), (rows >= 0).view(-1).to(torch.int32))
    table[st["dst"].long()] = rows
    for r in RINGS:
        if r in st:
            st[r][st["dst"].long()] = st[r][st["src"].long()]


def _plain_reserve(st, seqs, first, count, most):
    table, refs = st["page_table"], st["page_refs"]
    slot = first[:, None] // PAGE + torch.arange(_pages(most) + 1, device=DEV)[None]
    touched = slot * PAGE < (first + count)[:, None]
    at = torch.where(touched, slot, table.shape[1])  # a column of its own takes what is not touched
    rows = torch.cat([table[seqs.long()], torch.full_like(table[:1, :1], -1).expand(seqs.numel(), 1)], 1)
    page = rows.gather(1, at).long()
    shared = touched & (page >= 0) & (refs[page.clamp(min=0)] > 1)
    need = touched & ((page < 0) | shared)
    ids = torch.arange(refs.numel(), device=DEV)
    free = torch.where(refs == 0, ids, ids + refs.numel()).sort().values  # the free pages, lowest first
    rank = need.view(-1).cumsum(0) - 1
    new = torch.where(need, free[rank.clamp(min=0)].view(need.shape) % refs.numel(), page)
    refs.scatter_add_(0, page.clamp(min=0).view(-1), -shared.view(-1).to(torch.int32))
    refs.scatter_add_(0, new.clamp(min=0).view(-1), need.view(-1).to(torch.int32))
    table[seqs.long()] = rows.scatter(1, at, new.to(torch.int32))[:, :-1]
    # only the first pages can be shared; a second one that is not touched repeats the first
    new, page = (torch.where(touched[:, :2], x[:, :2], x[:, :1]) for x in (new, torch.where(shared, page, new)))
    to, of = new.reshape(-1), page.reshape(-1)
    for r in POOLS:
        if r in st:
            v = st[r].view((refs.numel(), PAGE) + tuple(st[r].shape[1:]))
            v[to] = v[of]


def _plain_compact(st):
    d, refs = st["dst"], st["page_refs"]
    live = refs > 0
    rank = live.cumsum(0) - 1
    n_dst = d["page_refs"].numel()
    to = torch.where(live, rank, n_dst)  # row n_dst takes what is not live
    of = torch.empty(n_dst + 1, dtype=torch.int64, device=DEV).fill_(-1).scatter_(0, to, torch.arange(refs.numel(), device=DEV))[:n_dst]
    d["page_refs"].copy_(torch.where(of >= 0, refs[of.clamp(min=0)], 0))
    t = st["page_table"]
    d["page_table"].copy_(torch.where(t >= 0, rank[t.clamp(min=0).long()].to(torch.int32), -1))
    for r in POOLS:
        if r in st:
            v = st[r].view((refs.numel(), PAGE) + tuple(st[r].shape[1:]))
            w = d[r].view((n_dst, PAGE) + tuple(st[r].shape[1:]))
            keep = (of >= 0).view([-1] + [1] * (w.dim() - 1))
            w.copy_(torch.where(keep, v[of.clamp(min=0)], w))


def _key_rows(st, real):
    """Rows [n_q, keys, d_qk] of every query's keys in `real`, their positions, and which of them it sees."""
    case, m = st["case"], _m(st["case"])
    t, seq = st["q_pos"], st["q_seq"].long()
    pos = t[:, None] - (N_WIN - 1) + torch.arange(N_WIN, device=DEV)[None]
    win = st["ring_x"][seq[:, None], pos % N_WIN]
    if case["chunk"]:
        at = (pos - st["pos0"]).clamp(min=0)
        win = torch.where((pos >= st["pos0"])[:, :, None], st["x_chunk"][at], win)
    lim = t + 1 - N_WIN
    vis = torch.where(lim > 0, (lim + m - 1) // m, 0)
    if case["k"]:
        j = st["sel_idx"].long()
        see = torch.arange(case["k"], device=DEV)[None] < st["sel_cnt"][:, None]
    else:
        j = torch.arange(_visible(st["max_pos"], m), device=DEV)[None].expand(t.numel(), -1)
        see = j < vis[:, None]
    j = torch.where(see, j, 0)
    row = st["page_table"][seq[:, None], j // PAGE].long().clamp(min=0) * PAGE + j % PAGE
    if "kv_scale" in st:
        ent = st["kv_pool"].view(torch.float8_e4m3fn)[row].to(real) * st["kv_scale"][row].to(real)[:, :, None]
    else:
        ent = st["kv_pool"][row].to(real)
    rows = torch.cat([win.to(real), ent], 1)
    where = torch.cat([pos.to(real), (j * m).to(real) + (m - 1) / 2.0], 1)
    return rows, where, torch.cat([pos >= 0, see], 1)


def _plain_attend(st):
    case = st["case"]
    rows, where, see = _key_rows(st, torch.float32)
    s = torch.einsum("qhd,qkd->qhk", st["q"].float(), rows) * st["sm_scale"]
    if case["cap"] > 0:
        s = torch.tanh(s / case["cap"]) * case["cap"]
    if st["slopes"] is not None:
        s = s - st["slopes"][None, :, None] * (st["q_pos"].float()[:, None] - where)[:, None, :]
    s = s.masked_fill(~see[:, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    tot = p.sum(-1, keepdim=True)
    out = torch.einsum("qhk,qkd->qhd", p / tot, rows[:, :, : st["out"].shape[2]])
    return out.to(torch.bfloat16), (top + torch.log(tot)).squeeze(-1)


# ------------------------------------------------------------------------------------------- calls
def _layer(st, part=None):
    """The library's view of the state's caches, built on the first pass and kept with them."""
    key = "layer" if part is None else "layer_" + part
    if key not in st:
        import compressed_sparse_kv_02_b200 as ck
        case, src = st["case"], st if part is None else st[part]
        d_qk, d_v, d_idx, kv, idx = SHAPES[case["shape"]]
        csa = case["kind"] == "csa"
        table = src["page_table"]
        rings = {r: st[r] for r in RINGS if r in st}
        if case["op"] == "attend":  # attention reads neither gate logits nor indexer keys: the smallest the layer takes
            d_idx, idx = (32 if csa else 0), "bf16"
            rings["ring_z"] = torch.empty(table.shape[0], N_WIN, 1, dtype=torch.bfloat16, device=DEV)
            if csa:
                rings["ring_xi"] = torch.empty(table.shape[0], N_WIN, 32, dtype=torch.bfloat16, device=DEV)
                rings["ring_zi"] = torch.empty(table.shape[0], N_WIN, 1, dtype=torch.bfloat16, device=DEV)
                st["idx_pool"] = torch.empty(src["kv_pool"].shape[0], 32, dtype=torch.bfloat16, device=DEV)
        st[key] = ck.Layer(
            kind=ck.LAYER_CSA if csa else ck.LAYER_HCA, m=_m(case), n_win=N_WIN, d_qk=d_qk, d_v=d_v,
            d_idx=d_idx if csa else 0, page_size=PAGE, kv_dtype=ck.BF16 if kv == "bf16" else ck.FP8_E4M3,
            idx_dtype=ck.BF16 if idx == "bf16" or not csa else ck.FP4_E2M1, gate_cols=rings["ring_z"].shape[2],
            gate_cols_idx=rings["ring_zi"].shape[2] if csa else 1, n_seqs=table.shape[0], max_pages_per_seq=table.shape[1],
            n_pages=src["kv_pool"].shape[0] // PAGE, page_table=table, kv_pool=src["kv_pool"], kv_scale=src.get("kv_scale"),
            idx_pool=src.get("idx_pool", st.get("idx_pool")), idx_scale=src.get("idx_scale"), page_refs=src["page_refs"],
            **rings)
        st["ck"], st["status"] = ck, torch.zeros(1, dtype=torch.int32, device=DEV)
    return st[key]


def _workspace(st, size):
    if "ws" not in st:
        st["ws"] = torch.empty(max(16, size()), dtype=torch.uint8, device=DEV)
    return st["ws"]


def _own_pages(st):
    case, L = st["case"], _layer(st)
    ck = st["ck"]
    if case["op"] == "branch":
        n = st["dst"].numel()
        ws = _workspace(st, lambda: ck.cskv_reserve_ws_bytes(L, n, case["count"]))
        ck.cskv_cache_fork(L, st["src"], st["dst"], st["n_entries"], status=st["status"])
        ck.cskv_cache_reserve(L, st["dst"], st["n_entries"], st["count"], case["count"], workspace=ws, status=st["status"])
    elif case["op"] == "regrow":
        n = st["seq"].numel()
        ws = _workspace(st, lambda: ck.cskv_reserve_ws_bytes(L, n, case["count"]))
        ck.cskv_cache_free(L, st["seq"], st["keep"], status=st["status"])
        ck.cskv_cache_reserve(L, st["seq"], st["keep"], st["count"], case["count"], workspace=ws, status=st["status"])
    else:
        D = _layer(st, "dst")
        ck.cskv_cache_compact(L, D, workspace=_workspace(st, lambda: ck.cskv_compact_ws_bytes(L, D)), status=st["status"])


def _own_attend(st):
    case, L = st["case"], _layer(st)
    ck = st["ck"]
    ws = _workspace(st, lambda: ck.cskv_attend_ws_bytes(L, st["q"].shape[0], case["heads"], st["max_pos"], case["k"]))
    more = dict(sm_scale=st["sm_scale"], workspace=ws, x_chunk=st.get("x_chunk"), chunk_pos0=st.get("pos0", 0),
                status=st["status"], score_cap=case["cap"], slopes=st["slopes"])
    if case["k"]:
        ck.csa_attend(L, st["q_seq"], st["q_pos"], st["max_pos"], st["q"], st["sel_idx"], st["sel_cnt"], st["out"],
                      st["lse"], **more)
    else:
        ck.hca_attend(L, st["q_seq"], st["q_pos"], st["max_pos"], st["q"], st["out"], st["lse"], **more)
    return st["out"], st["lse"]


def _page_outputs(st):
    of = st["dst"] if st["case"]["op"] == "compact" else st
    out = {r: of[r] for r in POOLS + ("page_table", "page_refs") if r in of}
    if st["case"]["op"] == "branch":
        out.update({r: st[r] for r in RINGS if r in st})
    if "kv_scale" in out:
        out["kv_pool"] = out["kv_pool"].view(torch.float8_e4m3fn)
    return out


def run(st):
    case = st["case"]
    if case["op"] == "attend":
        return _own_attend(st) if own else _plain_attend(st)
    if own:
        _own_pages(st)
    elif case["op"] == "branch":
        _plain_fork(st)
        _plain_reserve(st, st["dst"], st["n_entries"], st["count"], case["count"])
    elif case["op"] == "regrow":
        slot = torch.arange(st["page_table"].shape[1], device=DEV)
        _plain_release(st["page_table"], st["page_refs"], st["seq"],
                       slot[None] >= ((st["keep"] + PAGE - 1) // PAGE)[:, None])
        _plain_reserve(st, st["seq"], st["keep"], st["count"], case["count"])
    else:
        _plain_compact(st)
    return _page_outputs(st)


# ------------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """Attention in 64 bits, one block of queries at a time; the page operators move bits and have no such value."""
    if case["op"] != "attend":
        return None
    st = prepare(case, seed)
    d_v, m, h = st["out"].shape[2], _m(case), case["heads"]
    pool = st["kv_pool"].view(torch.float8_e4m3fn) if "kv_scale" in st else st["kv_pool"]
    outs, lses = [], []
    for b in range(st["q"].shape[0]) if not case["chunk"] else range(0, st["q"].shape[0], 256):
        ts = st["q_pos"][b:b + (256 if case["chunk"] else 1)]
        seq, t_lo, t_hi = int(st["q_seq"][b]), int(ts[0]), int(ts[-1])
        # the raw tokens any of these queries sees, then every entry up to the last one's
        p = torch.arange(max(0, t_lo - N_WIN + 1), t_hi + 1, device=DEV)
        raw = st["ring_x"][seq][p % N_WIN].double()
        if case["chunk"]:
            new = p >= st["pos0"]
            raw[new] = st["x_chunk"][p[new] - st["pos0"]].double()
        n_e = _visible(t_hi, m)
        j = torch.arange(n_e, device=DEV)
        row = st["page_table"][seq][j // PAGE].long() * PAGE + j % PAGE
        ent = pool[row].double()
        if "kv_scale" in st:
            ent = ent * st["kv_scale"][row].double()[:, None]
        see = torch.cat([(p[None] <= ts[:, None]) & (p[None] > ts[:, None] - N_WIN), j[None] * m < ts[:, None] + 1 - N_WIN], 1)
        if case["k"]:
            chosen = torch.zeros(ts.numel(), n_e + 1, dtype=torch.bool, device=DEV)
            sel = st["sel_idx"][b:b + ts.numel()].long()
            live = torch.arange(case["k"], device=DEV)[None] < st["sel_cnt"][b:b + ts.numel(), None]
            chosen.scatter_(1, torch.where(live, sel, n_e), True)
            see[:, p.numel():] &= chosen[:, :n_e]
        keys = torch.cat([raw, ent])
        where = torch.cat([p.double(), j.double() * m + (m - 1) / 2])
        q = st["q"][b:b + ts.numel()].double()
        z = (q.reshape(-1, q.shape[2]) @ keys.t()).view(ts.numel(), h, -1) / math.sqrt(q.shape[2])
        if case["cap"] > 0:
            z = case["cap"] * torch.tanh(z / case["cap"])
        if st["slopes"] is not None:
            z = z - st["slopes"].double()[None, :, None] * (ts.double()[:, None] - where[None])[:, None]
        z = torch.where(see[:, None], z, -math.inf)
        lse = torch.logsumexp(z, -1)
        outs.append((torch.exp(z - lse[..., None]).reshape(ts.numel() * h, -1) @ keys[:, :d_v]).view(ts.numel(), h, d_v))
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
