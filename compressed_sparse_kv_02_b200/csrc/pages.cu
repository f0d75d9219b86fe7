// pages.cu -- page operators of the paged compressed cache: fork, free, reserve
// (growth and copy on write) and compaction (10100.com article, section 5: paged
// KV with prefix reuse).
//
// Every page carries a count of the page-table slots that hold it; a page with
// count 0 is free. Forking shares pages, so only the rings (the raw tokens a
// branch will overwrite) and, at the branch's first write, one partly filled page
// are copied. What the operators need besides atomics on the counts is a rank:
// the k-th free page (reserve) or the k-th live page (compact), in page order, so
// that page choices repeat from call to call. rank_chunk computes it without an
// inter-CTA wait: each CTA takes kChunk counts and counts the matches in all the
// chunks before its own by itself. That reads n^2 / (2 kChunk) counts in all, from
// L2: 8 CTAs and 0.5 MB at 32,768 pages, 64 CTAs and 33 MB at 262,144.
//
// Bounds: fork, reserve and compaction move bytes (rings and pages, each read and
// written once, 16 bytes per access, four in flight per thread); free and the
// table work are a few dependent loads, so latency. Measured: compaction of 12,000
// pages of the wide latent (1.64 GB) 276-280 us, 0.90-0.91 of the copy rate; 56
// branches of 128K tokens forked and their next page reserved (29 MB) 15.0 us; one
// sequence's fork and reserve 9.5 us, three launches.
#include "cskv_device.cuh"
#include "cskv_internal.h"

namespace cskv {
namespace {

constexpr int kCopyThreads = 256;
constexpr int kSlice = kCopyThreads * 16 * 4;  // bytes one CTA moves at a time: four 16-byte accesses per thread
constexpr int kRankThreads = 1024;
constexpr int kChunk = kRankThreads * 4;       // counts per rank CTA (one int4 per thread)

// Copy `n` bytes (n <= kSlice when both addresses and n are multiples of 16: then every access is in flight
// at once); any other alignment of 2-byte elements goes element by element.
__device__ __forceinline__ void copy_slice(uint8_t* dst, const uint8_t* src, int n) {
  const int tid = threadIdx.x;
  if (((reinterpret_cast<uintptr_t>(dst) | reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(n)) & 15u) == 0) {
    uint4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = (j * kCopyThreads + tid) * 16;
      if (o < n) v[j] = *reinterpret_cast<const uint4*>(src + o);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int o = (j * kCopyThreads + tid) * 16;
      if (o < n) *reinterpret_cast<uint4*>(dst + o) = v[j];
    }
  } else {
    for (int o = 2 * tid; o < n; o += 2 * kCopyThreads)
      *reinterpret_cast<uint16_t*>(dst + o) = *reinterpret_cast<const uint16_t*>(src + o);
  }
}

__host__ __device__ __forceinline__ int slices_of(const PagePool& p) {
  return p.bytes ? static_cast<int>((p.bytes + kSlice - 1) / kSlice) : 0;
}
__host__ __device__ __forceinline__ int slices_of(const PagePool (&p)[4]) {
  return slices_of(p[0]) + slices_of(p[1]) + slices_of(p[2]) + slices_of(p[3]);
}

// Slice u of page `from` of pools a to page `to` of pools b.
__device__ __forceinline__ void copy_page_slice(const PagePool (&a)[4], int64_t from, const PagePool (&b)[4], int64_t to,
                                                int u) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int s = slices_of(a[i]);
    if (u >= 0 && u < s) {
      const int64_t o = (int64_t)u * kSlice;
      const int64_t left = a[i].bytes - o;
      copy_slice(b[i].base + to * b[i].bytes + o, a[i].base + from * a[i].bytes + o,
                 static_cast<int>(left < kSlice ? left : kSlice));
    }
    u -= s;
  }
}

__device__ __forceinline__ bool live_page(const PageParams& p, int32_t page) {
  return page >= 0 && page < p.n_pages && p.refs[page] > 0;
}

// One slot gives back its page. A slot that holds no live page is reported.
__device__ __forceinline__ void release(const PageParams& p, int32_t page) {
  if (page < 0) return;
  if (page >= p.n_pages) {
    report(p.status, CSKV_ERR_OUT_OF_RANGE);
    return;
  }
  if (atomicSub(&p.refs[page], 1) <= 0) {
    atomicAdd(&p.refs[page], 1);
    report(p.status, CSKV_ERR_OUT_OF_RANGE);
  }
}

__device__ __forceinline__ int64_t pages_of(const PageParams& p, int64_t entries) {
  return (entries + p.page_size - 1) / p.page_size;
}

// ---------------------------------------------------------------- fork
// grid (list entry, part): every CTA of an entry checks the entry, then takes its share of the slots and of the
// ring slices. No src row is written by any entry (an entry whose dst is a src is refused), so the parts need no
// order among them.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(PageParams p) {
  grid_dependency_wait();
  const int i = blockIdx.x, tid = threadIdx.x;
  const int src = p.src[i], dst = p.seq[i];
  const int64_t n = p.first[i];
  int bad = 0;
  for (int j = tid; j < p.n; j += kCopyThreads) bad |= p.src[j] == dst || (j != i && p.seq[j] == dst);
  bad = __syncthreads_or(bad);
  const bool out = src < 0 || src >= p.n_seqs || dst < 0 || dst >= p.n_seqs;
  if (out || bad || n < 0 || n > (int64_t)p.max_pages * p.page_size) {
    if (tid == 0 && blockIdx.y == 0) report(p.status, out ? CSKV_ERR_OUT_OF_RANGE : CSKV_ERR_INVALID_ARG);
    return;
  }
  const int used = static_cast<int>(pages_of(p, n));
  const int32_t* from = p.table + (int64_t)src * p.max_pages;
  int32_t* to = p.table + (int64_t)dst * p.max_pages;
  for (int64_t k = (int64_t)blockIdx.y * kCopyThreads + tid; k < p.max_pages; k += (int64_t)gridDim.y * kCopyThreads) {
    const int32_t old = to[k];
    int32_t page = k < used ? from[k] : -1;
    if (k < used && !live_page(p, page)) {
      report(p.status, CSKV_ERR_OUT_OF_RANGE);
      page = -1;
    }
    if (old == page) continue;
    if (page >= 0) atomicAdd(&p.refs[page], 1);
    release(p, old);
    to[k] = page;
  }
  const int units = slices_of(p.ring);
  for (int u = blockIdx.y; u < units; u += gridDim.y) copy_page_slice(p.ring, src, p.ring, dst, u);
}

// ---------------------------------------------------------------- free
// A slot is taken by an exchange, so a sequence listed twice gives each page back once.
__global__ void __launch_bounds__(kCopyThreads) free_kernel(PageParams p) {
  grid_dependency_wait();
  const int i = blockIdx.x;
  const int seq = p.seq[i];
  const int64_t keep = p.first[i];
  const bool out = seq < 0 || seq >= p.n_seqs;
  if (out || keep < 0 || keep > (int64_t)p.max_pages * p.page_size) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(p.status, out ? CSKV_ERR_OUT_OF_RANGE : CSKV_ERR_INVALID_ARG);
    return;
  }
  int32_t* row = p.table + (int64_t)seq * p.max_pages;
  for (int64_t k = pages_of(p, keep) + (int64_t)blockIdx.y * kCopyThreads + threadIdx.x; k < p.max_pages;
       k += (int64_t)gridDim.y * kCopyThreads)
    if (row[k] >= 0) release(p, atomicExch(&row[k], -1));
}

// ---------------------------------------------------------------- ranks
// The matches (free or live pages) before this thread's four counts, over the whole pool; match[j] says which of the
// four match, `sum` is the matches up to and including this chunk.
template <bool LIVE>
__device__ __forceinline__ int rank_chunk(const int32_t* refs, int64_t n, int chunk, bool (&match)[4], int& sum,
                                          int* warp_sums) {
  const int tid = threadIdx.x;
  int before = 0;
  const int4* r4 = reinterpret_cast<const int4*>(refs);
#pragma unroll 4
  for (int c = 0; c < chunk; ++c) {
    const int4 v = r4[(int64_t)c * kRankThreads + tid];
    before += ((v.x > 0) == LIVE) + ((v.y > 0) == LIVE) + ((v.z > 0) == LIVE) + ((v.w > 0) == LIVE);
  }
  const int64_t at = (int64_t)chunk * kChunk + 4 * tid;
  int mine = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    match[j] = at + j < n && (refs[at + j] > 0) == LIVE;
    mine += match[j];
  }
  int total, own;
  block_exclusive_scan<kRankThreads>(before, warp_sums, total);
  const int ex = block_exclusive_scan<kRankThreads>(mine, warp_sums, own);
  sum = total + own;
  return total + ex;
}

// ---------------------------------------------------------------- reserve
struct ReserveWs {
  int32_t* head;  // new pages asked for | free pages | shared pages to copy | error code
  int4* slot;     // [cap] (sequence, slot, shared page or -1, -) of the r-th new page
  int32_t* list;  // [cap] the r-th free page
  int32_t* cow;   // [cap] the new pages (indices r) that copy a shared one
  int64_t cap;
};
constexpr int kHeadBytes = 64;

__host__ __device__ __forceinline__ int64_t reserve_cap(const PageParams& p) {
  const int64_t most = (int64_t)p.n * (p.max_count / p.page_size + 2);
  return most < p.n_pages ? most : p.n_pages;
}
ReserveWs reserve_ws(const PageParams& p, void* ws) {
  ReserveWs w;
  w.cap = reserve_cap(p);
  w.head = static_cast<int32_t*>(ws);
  w.slot = reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + kHeadBytes);
  w.list = reinterpret_cast<int32_t*>(w.slot + w.cap);
  w.cow = w.list + w.cap;
  return w;
}

// Block 0 checks the requests and numbers the new pages they need, in request order; the other blocks list the free
// pages. Nothing but the workspace is written: the counts must not change while other CTAs rank them.
__global__ void __launch_bounds__(kRankThreads) reserve_plan_kernel(PageParams p, ReserveWs w) {
  __shared__ int s_warp[32];
  extern __shared__ int s_req[];  // [n] sequences | [n] first slots | [n + 1] touched slots before each request
  grid_dependency_wait();
  grid_dependents_launch();
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    bool match[4];
    int sum;
    const int chunk = blockIdx.x - 1;
    int r = rank_chunk<false>(p.refs, p.n_pages, chunk, match, sum, s_warp);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (match[j]) {
        if (r < w.cap) w.list[r] = chunk * kChunk + 4 * tid + j;
        ++r;
      }
    if (blockIdx.x == gridDim.x - 1 && tid == 0) w.head[1] = sum;
    return;
  }
  int* s_seq = s_req;
  int* s_slot = s_seq + p.n;  // a request's first slot minus the touched slots before it
  int* s_pre = s_slot + p.n;
  int code = 0, run = 0;
  for (int base = 0; base < p.n; base += kRankThreads) {
    const int i = base + tid;
    int touched = 0, k0 = 0;
    if (i < p.n) {
      const int seq = p.seq[i];
      const int64_t first = p.first[i], count = p.count[i], end = (int64_t)p.max_pages * p.page_size;
      if (seq < 0 || seq >= p.n_seqs) {
        code = CSKV_ERR_OUT_OF_RANGE;
      } else if (first < 0 || count < 0 || count > p.max_count || first > end || first + count > end) {
        code = CSKV_ERR_INVALID_ARG;
      } else if (count > 0) {
        k0 = static_cast<int>(first / p.page_size);
        touched = static_cast<int>((first + count - 1) / p.page_size) - k0 + 1;
      }
      s_seq[i] = seq;
    }
    int tot;
    const int ex = block_exclusive_scan<kRankThreads>(touched, s_warp, tot);
    if (i < p.n) {
      s_pre[i] = run + ex;
      s_slot[i] = k0 - (run + ex);
    }
    run += tot;
  }
  __syncthreads();
  for (int f = tid; f < p.n * p.n; f += kRankThreads) {
    const int i = f / p.n, j = f % p.n;
    if (j < i && s_seq[j] == s_seq[i]) code = CSKV_ERR_INVALID_ARG;  // listed twice
  }
  if (tid == 0) s_pre[p.n] = run;
  int need = 0, n_cow = 0;
  if (!__syncthreads_or(code != 0)) {
    for (int64_t base = 0; base < run; base += kChunk) {
      // four slots per thread; the loads of all four are issued before any is used
      int seq[4], k[4];
      int32_t page[4], refs[4];
      int lo = 0, hi = p.n - 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int f = static_cast<int>(base + 4 * tid + j < run ? base + 4 * tid + j : run - 1);
        while (j == 0 && lo < hi) {  // the request of the thread's first slot; the others follow on
          const int mid = (lo + hi + 1) >> 1;
          if (s_pre[mid] <= f) lo = mid; else hi = mid - 1;
        }
        while (s_pre[lo + 1] <= f) ++lo;
        seq[j] = s_seq[lo];
        k[j] = f + s_slot[lo];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) page[j] = p.table[(int64_t)seq[j] * p.max_pages + k[j]];
#pragma unroll
      for (int j = 0; j < 4; ++j) refs[j] = page[j] >= 0 && page[j] < p.n_pages ? p.refs[page[j]] : 0;
      int flags = 0;  // needs a new page in the low half, copies one in the high half
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (base + 4 * tid + j >= run || (page[j] >= 0 && refs[j] == 1)) {
          seq[j] = -1;  // nothing to do
        } else if (page[j] >= 0 && refs[j] <= 0) {
          seq[j] = -1;
          code = CSKV_ERR_OUT_OF_RANGE;
        } else {
          flags += page[j] >= 0 ? 1 + (1 << 16) : 1;
        }
      }
      int tot;
      const int ex = block_exclusive_scan<kRankThreads>(flags, s_warp, tot);
      int r = need + (ex & 0xffff), c = n_cow + (ex >> 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (seq[j] >= 0) {
          if (r < w.cap) {
            w.slot[r] = make_int4(seq[j], k[j], page[j] >= 0 ? page[j] : -1, 0);
            if (page[j] >= 0) w.cow[c] = r;
          }
          c += page[j] >= 0;
          ++r;
        }
      need += tot & 0xffff;
      n_cow += tot >> 16;
    }
  }
  // one code for the call: the first thread that has one names it
  __syncthreads();
  if (tid == 0) s_warp[0] = 0;
  __syncthreads();
  if (code) atomicCAS(&s_warp[0], 0, code);
  __syncthreads();
  if (tid == 0) {
    w.head[0] = need;
    w.head[2] = n_cow;
    w.head[3] = s_warp[0];
  }
}

__global__ void __launch_bounds__(kCopyThreads) reserve_apply_kernel(PageParams p, ReserveWs w) {
  grid_dependency_wait();
  const int need = w.head[0], n_free = w.head[1], n_cow = w.head[2];
  int code = w.head[3];
  if (!code && need > n_free) code = CSKV_ERR_NO_PAGES;
  if (code) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, code);
    return;
  }
  for (int r = blockIdx.x * kCopyThreads + threadIdx.x; r < need; r += gridDim.x * kCopyThreads) {
    const int4 s = w.slot[r];
    const int32_t page = w.list[r];
    p.table[(int64_t)s.x * p.max_pages + s.y] = page;
    p.refs[page] = 1;
    if (s.z >= 0) atomicSub(&p.refs[s.z], 1);
  }
  const int per = slices_of(p.pool);
  const int64_t units = (int64_t)n_cow * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int r = w.cow[u / per];
    copy_page_slice(p.pool, w.slot[r].z, p.pool, w.list[r], static_cast<int>(u % per));
  }
}

// ---------------------------------------------------------------- compact
struct CompactWs {
  int32_t* head;   // live pages
  int32_t* to;     // [n_pages] new id of a live page, -1 of a free one
  int32_t* order;  // [n_pages] the r-th live page
};
CompactWs compact_ws(const PageParams& p, void* ws) {
  CompactWs w;
  w.head = static_cast<int32_t*>(ws);
  w.to = w.head + kHeadBytes / 4;
  w.order = w.to + p.n_pages;
  return w;
}

__global__ void __launch_bounds__(kRankThreads) compact_rank_kernel(PageParams p, CompactWs w) {
  __shared__ int s_warp[32];
  grid_dependency_wait();
  grid_dependents_launch();
  bool match[4];
  int sum;
  int r = rank_chunk<true>(p.refs, p.n_pages, blockIdx.x, match, sum, s_warp);
  const int64_t at = (int64_t)blockIdx.x * kChunk + 4 * threadIdx.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (at + j >= p.n_pages) break;
    w.to[at + j] = match[j] ? r : -1;
    if (match[j]) w.order[r++] = static_cast<int32_t>(at + j);
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) w.head[0] = sum;
}

__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(PageParams p, PageParams d, CompactWs w) {
  grid_dependency_wait();
  const int live = w.head[0];
  if (live > d.n_pages) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report(p.status, CSKV_ERR_NO_PAGES);
    return;
  }
  const int64_t step = (int64_t)gridDim.x * kCopyThreads, me = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  for (int64_t r = me; r < d.n_pages; r += step) d.refs[r] = r < live ? p.refs[w.order[r]] : 0;
  for (int64_t f = me; f < (int64_t)d.n_seqs * d.max_pages; f += step) {
    const int64_t s = f / d.max_pages, k = f % d.max_pages;
    int32_t page = k < p.max_pages ? p.table[s * p.max_pages + k] : -1;
    if (page >= 0) {
      page = page < p.n_pages ? w.to[page] : -1;
      if (page < 0) report(p.status, CSKV_ERR_OUT_OF_RANGE);
    }
    d.table[f] = page < 0 ? -1 : page;
  }
  const int per = slices_of(p.pool);
  const int64_t units = (int64_t)live * per;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t r = u / per;
    copy_page_slice(p.pool, w.order[r], d.pool, r, static_cast<int>(u % per));
  }
}

int rank_ctas(int64_t n_pages) { return static_cast<int>((n_pages + kChunk - 1) / kChunk); }

}  // namespace

cudaError_t launch_fork(const PageParams& p, int n_sm, cudaStream_t st) {
  // parts per entry: a ring slice or a row of slots each, up to eight CTAs per SM in all
  int64_t parts = slices_of(p.ring);
  const int64_t rows = (p.max_pages + kCopyThreads - 1) / kCopyThreads;
  if (parts < rows) parts = rows;
  const int64_t most = ((int64_t)8 * n_sm + p.n - 1) / p.n;
  if (parts > most) parts = most;
  return launch_pdl(fork_kernel, dim3(p.n, static_cast<unsigned>(parts)), dim3(kCopyThreads), 0, st, p);
}

cudaError_t launch_free(const PageParams& p, int n_sm, cudaStream_t st) {
  int64_t parts = (p.max_pages + kCopyThreads - 1) / kCopyThreads;
  const int64_t most = ((int64_t)8 * n_sm + p.n - 1) / p.n;
  if (parts > most) parts = most;
  return launch_pdl(free_kernel, dim3(p.n, static_cast<unsigned>(parts)), dim3(kCopyThreads), 0, st, p);
}

size_t reserve_ws_bytes(const PageParams& p) { return kHeadBytes + static_cast<size_t>(reserve_cap(p)) * 24; }

cudaError_t launch_reserve(const PageParams& p, void* ws, int n_sm, cudaStream_t st) {
  const ReserveWs w = reserve_ws(p, ws);
  const size_t smem = sizeof(int) * (3 * (size_t)p.n + 1);
  cudaError_t e = cudaSuccess;
  if (smem > 40000)  // the static default is 48 KB, the kernel's own arrays included
    e = allow_smem(reserve_plan_kernel, smem, 32 * sizeof(int));
  if (e != cudaSuccess) return e;
  e = launch_pdl(reserve_plan_kernel, dim3(1 + rank_ctas(p.n_pages)), dim3(kRankThreads), smem, st, p, w);
  if (e != cudaSuccess) return e;
  int64_t grid = w.cap * slices_of(p.pool);
  if (grid > 4 * n_sm) grid = 4 * n_sm;
  return launch_pdl(reserve_apply_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0, st, p, w);
}

size_t compact_ws_bytes(const PageParams& p) { return kHeadBytes + static_cast<size_t>(p.n_pages) * 8; }

cudaError_t launch_compact(const PageParams& p, const PageParams& d, void* ws, int n_sm, cudaStream_t st) {
  const CompactWs w = compact_ws(p, ws);
  cudaError_t e = launch_pdl(compact_rank_kernel, dim3(rank_ctas(p.n_pages)), dim3(kRankThreads), 0, st, p, w);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_move_kernel, dim3(8 * n_sm), dim3(kCopyThreads), 0, st, p, d, w);
}

}  // namespace cskv
