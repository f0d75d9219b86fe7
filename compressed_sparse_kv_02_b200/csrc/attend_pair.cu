// attend_pair.cu -- CSA / HCA core attention on the tensor cores (tcgen05) for
// calls with many queries on the narrow latent: d_qk = d_v = 128, 64 query
// heads (DeepSeek-V4 report digest, section 3: one softmax over the window and
// the selected / all compressed entries; DeepSeek-V4-book ch.1, section 4: every
// head reads the one shared latent row).
//
// A prefill block holds thousands of query positions, so no key split is
// needed: a work item is a PAIR of queries (2i, 2i + 1), each with its own key
// list (window rows, then its selection or every visible entry), run to the end
// by one CTA, which writes the normalised bf16 output itself (no merge pass).
// The 64 heads of one query are an M = 64 tcgen05 tile; the accumulator of such
// a tile fills lanes 0-15 of each 32-lane quarter of tensor memory, and the
// second query's tile sits at lane offset 16, so the two queries' S (and O)
// share the 128 lanes and one softmax warpgroup serves both: thread (warp w,
// lane l) owns head 16 w + (l & 15) of query l >> 4.
//   loaders (warps 5-8): per tile, the source rows of 64 keys of each query,
//     then cp.async of the 2 x 64 rows (16 threads per 256-byte row) into a
//     128-byte-swizzled stage (four stages: the loaders run up to three tiles
//     ahead, so the hand-offs of consecutive tiles overlap); Q of the pair by TMA;
//   MMA (warp 4, one lane issues): S(t) = Q K^T (2 x 8 MMAs, M = 64, N = 64, K = 16)
//     into S buffer t & 1; then O += P(t - 1) V (2 x 4 MMAs, N = d_v = 128, V read
//     MN-major from the same stage: V is the first d_v channels of each key);
//   softmax (warps 0-3): max pass over S(t) in tensor memory, lazy O rescale,
//     exp pass writing bf16 P(t) into shared buffer t & 1 (the A operand).
// O is rescaled only when a row's running max rises by more than 2^8, so most
// tiles skip it (the probabilities stay below 256 in bf16).
//
// RULE is the form with a cap or a distance bias on the logits: the loaders write each key's distance beside its row,
// and the softmax, on eight warps with two threads per head row, applies the rule once and keeps the ruled logits in
// registers for its exponentials (the plain form reads S twice instead). Its loader warps have 32 rows of a tile each and
// go their own way: TMA gathers the rows, four per copy, or, where four rows have several sources (ring and pool),
// cp.async. With one thread per row and cp.async alone 1001 queries of 640 keys took 121 us, with both 100; a tile then
// takes 3,700 cycles, 2,700 of them one softmax pass (a chain of dependent steps: issue slots 39% used, tensor 17%).
//
// Shared memory (1024-aligned): Q 32 KB | key stages 4 x 32 KB | P 2 x 16 KB |
// source-row codes | barriers | valid-key bits. Tensor memory: O 128 | S 2 x 64
// columns. A key without a valid source row (an index outside the
// visible entries) is masked out of the softmax and reported.
#include "cskv_device.cuh"
#include "cskv_internal.h"
#include "score_rule.cuh"
#include "tc_issue.cuh"

namespace cskv {
namespace {

constexpr int kD = 128;             // d_qk = d_v
constexpr int kH = 64;              // heads of one query (the M of its tile)
constexpr int kNk = 64;             // keys per tile and query
constexpr int kNS = 4;              // key stages: the loaders run up to three tiles ahead
constexpr int kSlotBytes = kNk * kD * 2;        // 16384: one query's key tile (two 64-channel halves)
constexpr int kHalfBytes = kNk * 128;           // 8192: one 64-channel half of it
constexpr int kStageBytes = 2 * kSlotBytes;     // 32768
constexpr int kQBytes = 2 * kH * kD * 2;        // 32768: Q of both queries
constexpr int kPBytes = 2 * kH * kNk * 2;       // 16384: P of both queries (one buffer)
constexpr int kRows = 2 * kNk;                  // key rows of a tile (both queries)
constexpr int kLoadThread0 = 160;   // warps 0-3 softmax, warp 4 MMA, warps 5-8 loads, RULE: warps 9-12 softmax too
constexpr int kLoaders = 128;
constexpr int kSecondWarp0 = (kLoadThread0 + kLoaders) / 32;  // 9
template <bool RULE>
struct Block {
  static constexpr int kThreads = kLoadThread0 + kLoaders + (RULE ? 128 : 0);
  static constexpr int kSoftmax = RULE ? 256 : 128;  // softmax threads: one per row, RULE two
};
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0, kColS = 128;       // O | S buffer 0 | S buffer 1 (64 columns each)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;        // log2 units

struct Smem {
  static constexpr int Q = 0;
  static constexpr int K = Q + kQBytes;
  static constexpr int P = K + kNS * kStageBytes;
  static constexpr int ROWS = P + 2 * kPBytes;    // [2] source-row codes of the tile being issued, and the last one's
  static constexpr int DIST = ROWS + 2 * kRows * 4;  // RULE: minus the distances [stage][query][64 keys]
  static constexpr int BIAS = DIST + kNS * 2 * kNk * 4;  // RULE: [256 softmax threads] slope and reference of a row
  static constexpr int BAR = BIAS + 256 * 8;
  static constexpr int TMEM = BAR + (2 * kNS + 9) * 8;
  static constexpr int FLAGS = TMEM + 4;
  static constexpr int MASK = FLAGS + 8;          // valid-key bits: [stage][query][2 words]
  static constexpr int SIDE = MASK + kNS * 2 * 2 * 4;   // RULE: [2][2 halves][128 rows] what the halves of a row exchange
  static constexpr int END = SIDE + 2 * 2 * 128 * 4;
  static constexpr size_t bytes() { return 1024 + END; }
};
static_assert(Smem::bytes() <= 232448, "shared memory budget");
static_assert(Smem::DIST % 16 == 0 && Smem::BAR % 8 == 0 && Smem::MASK % 4 == 0 && Smem::BIAS % 8 == 0, "alignment");

// source-row code: kind in bits [31:30] (0 none, 1 pool entry, 2 ring row, 3 chunk row), row below
constexpr uint32_t kRowBits = 30;
constexpr uint32_t kRowMask = (1u << kRowBits) - 1u;

struct Keys {
  int64_t t, ws;
  int n_w;
  int n;  // window + compressed keys (0 for an invalid position)
  int64_t n_vis;  // entries visible at t
};

__device__ __forceinline__ Keys keys_of(const AttendParams& p, int b) {
  Keys r;
  r.t = p.q_pos[b];
  r.ws = 0;
  r.n_w = 0;
  r.n = 0;
  r.n_vis = 0;
  if (r.t < 0 || r.t > p.max_pos) return r;
  r.ws = window_start(r.t, p.n_win);
  r.n_w = static_cast<int>(r.t - r.ws + 1);
  int64_t n_c = r.n_vis = visible_entries(r.t, p.m, p.n_win);
  if (p.is_csa) {
    const int64_t c = p.sel_cnt[b];
    n_c = c < 0 ? 0 : (c > p.k ? p.k : c);
  }
  r.n = static_cast<int>(r.n_w + n_c);
  return r;
}

// The source row of one key, found in three steps a tile apart, so that no step waits for the loads of the one before
// it: which key (its entry, through the selection), which page, which row.
// Window keys come first (ring-slot order when every window row is in the ring, position order when a prefill chunk
// supplies some), then the compressed entries. A code of 0 is an invalid row.
struct Lookup {
  uint32_t code;  // of a window row
  int entry;      // else the entry, -1: none
  int32_t page;   // and its page
  int32_t slot;   // and its place there
  float dist;     // the key's distance from position k.t in tokens (RULE)
};
// key u (< k.n) of query b
__device__ __forceinline__ void look_key(const AttendParams& p, int b, int seq, const Keys& k, int u, Lookup& l) {
  l.code = 0;
  l.entry = -1;
  l.dist = 0.f;
  if (u < k.n_w) {
    if (!p.x_chunk) {
      l.dist = static_cast<float>((k.t - u) % p.n_win);  // slot u holds the latest position up to t that is u mod n_win
      l.code = (2u << kRowBits) | static_cast<uint32_t>(seq * p.n_win + u);
      return;
    }
    const int64_t pos = k.ws + u;
    l.dist = static_cast<float>(k.t - pos);
    const int64_t cr = chunk_row(p, seq, pos);
    l.code = cr >= 0 ? (3u << kRowBits) | static_cast<uint32_t>(cr)
                     : (2u << kRowBits) | static_cast<uint32_t>(seq * p.n_win + pos % p.n_win);
    return;
  }
  l.entry = p.is_csa ? p.sel_idx[(int64_t)b * p.k + (u - k.n_w)] : u - k.n_w;
}
__device__ __forceinline__ void look_page(const AttendParams& p, int seq, const Keys& k, Lookup& l) {
  l.page = -1;
  const int64_t j = l.entry;
  if (j < 0 || j >= k.n_vis) return;
  l.dist = entry_distance(k.t, j, p.m);
  const int32_t pi = l.entry / p.page_size;
  l.slot = l.entry - pi * p.page_size;
  if (pi < p.max_pages_per_seq) l.page = p.page_table[(int64_t)seq * p.max_pages_per_seq + pi];
}
__device__ __forceinline__ uint32_t look_row(const AttendParams& p, const Lookup& l) {
  if (l.code) return l.code;
  if (l.page < 0 || l.page >= p.n_pages) return 0;
  return (1u << kRowBits) | static_cast<uint32_t>((int64_t)l.page * p.page_size + l.slot);
}

__device__ __forceinline__ const uint16_t* code_row(const AttendParams& p, uint32_t c) {
  const uint32_t kind = c >> kRowBits, row = c & kRowMask;
  if (kind == 1) return static_cast<const uint16_t*>(p.kv_pool) + (size_t)row * kD;
  if (kind == 2) return p.ring_x + (size_t)row * kD;
  if (kind == 3) return p.x_chunk + (size_t)row * kD;
  return nullptr;
}


// S of both queries: 8 MMAs each (K = 16 channels) over the two 64-channel halves (N = 64 keys). The two chains are
// issued alternately: an MMA that accumulates into the tile of the one before it waits for it.
__device__ __forceinline__ void issue_s(uint32_t issuer, uint32_t d, uint32_t q, uint32_t k0, uint32_t k1, uint32_t idesc) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks) {
    const uint32_t off = (ks & 3) * 32u;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      umma_ss_if(issuer, d + (j ? 16u << 16 : 0u),
                 umma_desc_sw128(q + j * (kQBytes / 2) + (ks >> 2) * (kH * 128) + off, 16, 1024),
                 umma_desc_sw128((j ? k1 : k0) + (ks >> 2) * kHalfBytes + off, 16, 1024), idesc, ks > 0 ? 1u : 0u);
  }
}
// O += P V of both queries, alternately: 4 MMAs each (K = 16 keys; P is one 64-key swizzle atom); V MN-major
// (its two 64-channel halves kHalfBytes apart, 8-key groups 1024 bytes apart)
__device__ __forceinline__ void issue_pv(uint32_t issuer, uint32_t d, uint32_t pm, uint32_t v0, uint32_t v1,
                                         uint32_t idesc, bool acc) {
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      umma_ss_if(issuer, d + (j ? 16u << 16 : 0u), umma_desc_sw128(pm + j * (kPBytes / 2) + ks * 32, 16, 1024),
                 umma_desc_sw128((j ? v1 : v0) + ks * 16 * 128, kHalfBytes, 1024), idesc, (acc || ks > 0) ? 1u : 0u);
}

// Pipeline (tiles numbered gt across the CTA's items; stage gt % 4, S buffer gt & 1,
// P buffer gt & 1):
//   loaders : wait kempty[stage] (P V of tile gt - 4 done) -> cp.async -> kfull of the tile before, once landed
//   MMA     : wait kfull -> S(gt) -> commit sfull[gt & 1] (and qempty after an item's last S);
//             wait pfull[(gt - 1) & 1] -> P V(gt - 1) -> commit kempty, obar[(gt - 1) & 1]
//   softmax : wait sfull, kfull (valid-key bits) -> row max -> wait obar (P V of tile gt - 2
//             done: P buffer free)
//             -> rescale O if needed (after P V of gt - 1) -> P(gt) -> arrive pfull
template <bool RULE>
__global__ void __launch_bounds__(Block<RULE>::kThreads, 1)
    attend_pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_pool,
                       const __grid_constant__ CUtensorMap tm_ring, const __grid_constant__ CUtensorMap tm_chunk,
                       const AttendParams p, const __grid_constant__ Rule rule) {
  constexpr int kThreads = Block<RULE>::kThreads, kSoftmax = Block<RULE>::kSoftmax;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm + Smem::Q;
  uint8_t* sK = sm + Smem::K;
  uint8_t* sP = sm + Smem::P;
  uint32_t* sRow = reinterpret_cast<uint32_t*>(sm + Smem::ROWS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Smem::BAR);
  uint64_t* kfull = bars;               // [kNS] loaders (128) -> MMA and softmax
  uint64_t* kempty = bars + kNS;        // [kNS] MMA -> loaders (commit after the tile's P V)
  uint64_t* sfull = bars + 2 * kNS;     // [2] MMA -> softmax
  uint64_t* pfull = sfull + 2;          // [2] softmax -> MMA (128 arrivals)
  uint64_t* obar = pfull + 2;           // [2] MMA -> softmax (P V of that P buffer done)
  uint64_t* qfull = obar + 2;           //     Q of the item landed (TMA)
  uint64_t* qempty = qfull + 1;         //     the item's S products are done with Q
  uint64_t* dbar = qempty + 1;          //     the item's last P V is done
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + Smem::TMEM);
  volatile int* sAbort = reinterpret_cast<int*>(sm + Smem::FLAGS);
  uint32_t* sMask = reinterpret_cast<uint32_t*>(sm + Smem::MASK);
  float* sDist = reinterpret_cast<float*>(sm + Smem::DIST);
  float* sSide = reinterpret_cast<float*>(sm + Smem::SIDE);
  float2* sBias = reinterpret_cast<float2*>(sm + Smem::BIAS);

  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&kfull[i], kLoaders);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], kSoftmax);
      mbar_init(&obar[i], 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(dbar, 1);
    fence_barrier_init();
    *sAbort = 0;
  }
  if (tid == kLoadThread0) {
    prefetch_tensormap(&tm_q);
    if (RULE) {
      prefetch_tensormap(&tm_pool);
      prefetch_tensormap(&tm_ring);
      prefetch_tensormap(&tm_chunk);
    }
  }
  if (warp == 4) {
    tmem_alloc(sTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *sTmem, 0);
  // the set-up above overlaps the tail of the kernel ahead of this one; its outputs
  // (the selection, new cache rows) are read only from here on
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.n_q; b += kThreads)
      if (p.q_pos[b] < 0 || p.q_pos[b] > p.max_pos) report(p.status, CSKV_ERR_INVALID_ARG);

  if (RULE && (warp < 4 || warp >= kSecondWarp0)) {
    // A softmax thread's slope and what its row's logits are relative to: the bias of the farthest key, where the slope
    // is negative. In shared memory, each thread its own, they cost no register in the loops.
    const int qd = warp & 3, hf = warp >= kSecondWarp0;
    sBias[hf * 128 + qd * 32 + lane] = make_float2(p.slopes ? p.slopes[qd * 16 + (lane & 15)] * kLog2e : 0.f, 0.f);
  }

  const int n_items = (p.n_q + 1) >> 1;
  uint32_t g = 0;       // tiles of this CTA before the current item
  uint32_t n_item = 0;  // items with keys of this CTA before the current one
  for (int item = blockIdx.x; item < n_items && !__shfl_sync(kFull, *sAbort, 0); item += gridDim.x) {
    const int b0 = 2 * item, b1 = b0 + 1 < p.n_q ? b0 + 1 : -1;
    const Keys k0 = keys_of(p, b0);
    Keys k1;
    k1.n = 0;
    k1.n_w = 0;
    k1.t = 0;
    k1.ws = 0;
    k1.n_vis = 0;
    if (b1 >= 0) k1 = keys_of(p, b1);
    const int s0 = p.q_seq[b0], s1 = b1 >= 0 ? p.q_seq[b1] : 0;
    const bool ok0 = s0 >= 0 && s0 < p.n_seqs_layer, ok1 = b1 >= 0 && s1 >= 0 && s1 < p.n_seqs_layer;
    const int n0 = ok0 ? k0.n : 0, n1 = ok1 ? k1.n : 0;
    // a sequence id outside the layer: the query's keys are all masked (zero output), as in the
    // other attention kernels, and the status word says why
    if (tid == 0 && ((!ok0 && k0.n > 0) || (b1 >= 0 && !ok1 && k1.n > 0))) report(p.status, CSKV_ERR_OUT_OF_RANGE);
    // HCA rows of a prefill chunk: consecutive positions t, t + 1 of one sequence see the same
    // entries up to the last one of t + 1 and windows that differ by one row, so the pair shares
    // one key list (window rows ws(t) .. t + 1, then the entries of t + 1) and every tile is loaded
    // once for both; the valid-key bits tell each query which of the keys it sees. (Not with a rule: a
    // masked key's P = 0 times a NaN in its row would be NaN, so each query has its own rows only.)
    const bool shared = !RULE && !p.is_csa && p.x_chunk && ok0 && ok1 && s0 == s1 && k0.n > 0 && k1.n > 0 &&
                        k1.t == k0.t + 1;
    Keys ksh;  // the shared list (window start of t, last position t + 1)
    ksh.t = k1.t;
    ksh.ws = k0.ws;
    ksh.n_w = static_cast<int>(k1.t - k0.ws + 1);
    ksh.n = ksh.n_w + (k1.n - k1.n_w);
    ksh.n_vis = k1.n_vis;
    const int nmax = shared ? ksh.n : (n0 > n1 ? n0 : n1);
    const int ntiles = (nmax + kNk - 1) / kNk;
    if (ntiles == 0) {
      // Neither query has keys (padding): zeros and -inf. The item takes no part in the pipeline: with no tile to wait for,
      // the MMA warp would run more than one phase of dbar ahead of the softmax, which would then wait for the wrong one.
      const int n_out = b1 >= 0 ? 2 : 1;  // consecutive rows
      uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)b0 * kH * kD);
      for (int i = tid; i < n_out * kH * (kD / 8); i += kThreads) out[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int i = tid; i < n_out * kH; i += kThreads) p.lse[(int64_t)b0 * kH + i] = -INFINITY;
      continue;
    }

    if (tid >= kLoadThread0 && tid < kLoadThread0 + kLoaders) {
      // ---------------------------------------------------------------- loaders
      const int lt = tid - kLoadThread0, lw = lt >> 5, ll = lt & 31;
      // Q of both queries, by the first loader warp, once the last item's S products are done with the buffer: it looks
      // at each tile and waits at the third, so that the first tiles of an item are on their way before (the wait does
      // not depend on this item).
      bool q_sent = false;
      auto load_q = [&](bool wait) {
        if (lw != 0 || q_sent || !(wait || n_item == 0 || mbar_done(qempty, (n_item - 1) & 1u))) return;
        q_sent = true;
        const bool okq = __all_sync(kFull, n_item == 0 || mbar_wait(qempty, (n_item - 1) & 1u, p.status));
        if (ll == 0) {
          if (okq) {
            mbar_arrive_expect_tx(qfull, kQBytes);
            const int qb1 = b1 >= 0 ? b1 : b0;  // a lone last query: its slot repeats it (never read out)
            for (int h = 0; h < 2; ++h) {
              tma_load_2d(sQ + h * (kH * 128), &tm_q, h * 64, b0 * kH, qfull);
              tma_load_2d(sQ + kQBytes / 2 + h * (kH * 128), &tm_q, h * 64, qb1 * kH, qfull);
            }
          } else {
            *sAbort = 1;
          }
        }
        __syncwarp();
      };
      // this thread's part of every tile: the source row of key (lt & 63) of query lt >> 6, and
      // chunk (lt & 15) of rows (lt >> 4) + 8 q. The steps of a lookup run ahead of the tile they are for (the key
      // three tiles, its page two), and a tile is signalled, by every loader thread, when its copies have
      // landed, while the next tile's fly.
      const int chunk = lt & 15, half = chunk >> 3, c8 = chunk & 7;
      const int my_slot = lt >> 6, my_key = lt & (kNk - 1);
      const bool second = shared || my_slot;  // a shared list is that of query b1's last position
      const Keys kl = shared ? ksh : my_slot ? k1 : k0;
      const int bl = second ? b1 : b0, sl = second ? s1 : s0;
      const int nl = shared ? (lt < kNk ? ksh.n : 0) : (my_slot ? n1 : n0);
      auto key_at = [&](int it, Lookup& l) {
        l.code = 0;
        l.entry = -1;
        const int u = it * kNk + (shared ? lt : my_key);
        if (it < ntiles && u < nl) look_key(p, bl, sl, kl, u, l);
      };
      Lookup l0, l1, l2;  // of the tiles it, it + 1 (pages found) and it + 2 (keys found)
      key_at(0, l0);
      key_at(1, l1);
      key_at(2, l2);
      look_page(p, sl, kl, l0);
      look_page(p, sl, kl, l1);
      bool tma_before = false;  // the tile before this one was copied by TMA, which signals it
      for (int it = 0; it < ntiles; ++it) {
        const uint32_t gt = g + it;
        const int st = gt % kNS;
        load_q(it == 2);
        const uint32_t c = look_row(p, l0);
        const float di = l0.dist;
        if (it * kNk + (shared ? lt : my_key) < nl && !c) report(p.status, CSKV_ERR_OUT_OF_RANGE);
        const bool free =
            __all_sync(kFull, gt < (uint32_t)kNS || mbar_wait(&kempty[st], ((gt / kNS) - 1) & 1u, p.status));
        bool tma = false;
        if constexpr (RULE) {
          // Every loader warp has 32 rows of its own and goes through the tiles alone.
          if (!__all_sync(kFull, free && !*sAbort)) {
            *sAbort = 1;
            cp_async_wait<0>();  // the copies in flight may not outlive the block
            if (it > 0 && !tma_before) mbar_arrive(&kfull[(gt - 1) % kNS]);
            for (uint32_t d = 1; d <= (uint32_t)kNS && d <= gt; ++d)
              mbar_wait(&kfull[(gt - d) % kNS], ((gt - d) / kNS) & 1u, nullptr);
            break;
          }
          sDist[st * kRows + lt] = -di;
          const unsigned mw = __ballot_sync(kFull, c != 0);  // valid-key bits: keys 32 (lw & 1) .. + 31 of query lw >> 1
          if (ll == 0) sMask[st * 4 + lw] = mw;
          // four consecutive rows that come from one source (or have none) are one copy
          const uint32_t kind = c >> kRowBits;
          const unsigned m1 = __ballot_sync(kFull, kind == 1), m2 = __ballot_sync(kFull, kind == 2),
                         m3 = __ballot_sync(kFull, kind == 3);
          auto any4 = [](unsigned m) { return (m | m >> 1 | m >> 2 | m >> 3) & 0x11111111u; };
          const unsigned a1 = any4(m1), a2 = any4(m2), a3 = any4(m3);
          tma = ((a1 & a2) | (a1 & a3) | (a2 & a3)) == 0;
          uint8_t* slot0 = sK + st * kStageBytes + (lw >> 1) * kSlotBytes + (lw & 1) * (32 * 128);
          if (tma) {
            // 16 gathers of four rows' 64 channels (issued one by one); a missing row reads row -1, outside the map: zeros
            int y[4];
            uint32_t from = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t cd = __shfl_sync(kFull, c, (ll & 7) * 4 + e);
              y[e] = cd ? static_cast<int>(cd & kRowMask) : -1;
              from |= cd >> kRowBits;
            }
            if (ll < 16) {
              mbar_arrive_expect_tx(&kfull[st], 4 * 128);
              tma_gather4(slot0 + (ll >> 3) * kHalfBytes + (ll & 7) * (4 * 128),
                          from == 2 ? &tm_ring : from == 3 ? &tm_chunk : &tm_pool, (ll >> 3) * 64, y[0], y[1], y[2], y[3],
                          &kfull[st]);
            } else {
              mbar_arrive(&kfull[st]);
            }
            __syncwarp();
          } else {
#pragma unroll 4
            for (int q = 0; q < 16; ++q) {
              const int row = 2 * q + (ll >> 4);
              const uint16_t* src = code_row(p, __shfl_sync(kFull, c, row));
              cp_async16(slot0 + half * kHalfBytes + row * 128 + ((c8 ^ (row & 7)) << 4),
                         src ? static_cast<const void*>(src + half * 64 + c8 * 8) : static_cast<const void*>(p.q),
                         src ? 16 : 0);
            }
          }
          cp_async_commit();
        } else {
          uint32_t* row_of = sRow + (gt & 1u) * kRows;
          row_of[lt] = c;
          if (shared) {  // loader warps 0 and 1 hold keys 32 w .. + 31 of the shared list
            const int u = it * kNk + lt;
            const bool win = u < ksh.n_w;
            // t sees the window rows up to t (all but the last) and its own entries; t + 1 the rows
            // from its window start and every entry of the list
            const bool v0 = c != 0 && (win ? u < ksh.n_w - 1 : u - ksh.n_w < k0.n - k0.n_w);
            const bool v1 = c != 0 && (!win || k0.ws + u >= k1.ws);
            const unsigned m0 = __ballot_sync(kFull, v0), m1 = __ballot_sync(kFull, v1);
            if (ll == 0 && lw < 2) {
              sMask[st * 4 + lw] = m0;
              sMask[st * 4 + 2 + lw] = m1;
            }
          } else {  // valid-key bits of the tile (the softmax reads them after kfull[st]): warp w of
                    // the loaders holds keys 32 (w & 1) .. + 31 of query w >> 1
            const unsigned mw = __ballot_sync(kFull, c != 0);
            if ((lt & 31) == 0) sMask[st * 4 + (lt >> 5)] = mw;
          }
          // the tile's rows are visible to every loader, or some wait gave up (the same answer for all)
          if (named_sync_or(3, kLoaders, !free || *sAbort)) {
            *sAbort = 1;
            break;
          }
          uint8_t* dst = sK + st * kStageBytes + half * kHalfBytes;
          const int n_q8 = shared ? kNk / 8 : kRows / 8;  // 8-row steps: one list or two
#pragma unroll 4
          for (int q = 0; q < n_q8; ++q) {
            const int row = (lt >> 4) + 8 * q;  // query row / kNk, key row % kNk
            const int key = row & (kNk - 1);
            const uint16_t* src = code_row(p, row_of[row]);
            cp_async16(dst + (row / kNk) * kSlotBytes + key * 128 + ((c8 ^ (key & 7)) << 4),
                       src ? static_cast<const void*>(src + half * 64 + c8 * 8) : static_cast<const void*>(p.q),
                       src ? 16 : 0);
          }
          cp_async_commit();
        }
        l0 = l1;
        l1 = l2;
        look_page(p, sl, kl, l1);
        key_at(it + 3, l2);
        if (it > 0 && !tma_before) {  // the tile before this one has landed
          cp_async_wait<1>();
          fence_proxy_async_smem();
          mbar_arrive(&kfull[(gt - 1) % kNS]);
        }
        tma_before = tma;
      }
      load_q(true);
      cp_async_wait<0>();
      if (!*sAbort && !tma_before) {
        fence_proxy_async_smem();
        mbar_arrive(&kfull[(g + ntiles - 1) % kNS]);
      }
    } else if (warp == 4) {
      // ---------------------------------------------------------------- MMA issue
      // The whole warp takes every wait (it never diverges around a barrier); one elected lane issues
      // the MMAs and their commits.
      const uint32_t issuer = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(kH, kNk, false);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(kH, kD, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sPa = smem_u32(sP);
      const uint32_t slot1 = __shfl_sync(kFull, shared ? 0 : kSlotBytes, 0);  // the second query's key tile
      bool ok = __all_sync(kFull, mbar_wait(qfull, n_item & 1u, p.status));
      tc_fence_after();
      const int nt = __shfl_sync(kFull, ntiles, 0);
      for (int it = 0; it <= nt && ok; ++it) {
        if (__shfl_sync(kFull, *sAbort, 0)) break;
        if (it < nt) {
          const uint32_t gt = __shfl_sync(kFull, g + it, 0);
          const int st = gt % kNS;
          if (!(ok = __all_sync(kFull, mbar_wait(&kfull[st], (gt / kNS) & 1u, p.status)))) break;
          tc_fence_after();
          const uint32_t d = tmem + kColS + (gt & 1u) * kNk;
          const uint32_t kb = sKa + st * kStageBytes;
          issue_s(issuer, d, sQa, kb, kb + slot1, idesc_s);
          commit_if(issuer, &sfull[gt & 1u]);
          if (it == nt - 1) commit_if(issuer, qempty);
          __syncwarp();
        }
        if (it >= 1) {
          const uint32_t gp = __shfl_sync(kFull, g + it - 1, 0);
          const int pb = gp & 1u, sp = gp % kNS;
          if (!(ok = __all_sync(kFull, mbar_wait(&pfull[pb], (gp >> 1) & 1u, p.status)))) break;
          tc_fence_after();
          const uint32_t vb = sKa + sp * kStageBytes, pm = sPa + pb * kPBytes;
          issue_pv(issuer, tmem + kColO, pm, vb, vb + slot1, idesc_pv, it > 1);
          commit_if(issuer, &kempty[sp]);
          commit_if(issuer, &obar[pb]);
          __syncwarp();
        }
      }
      commit_if(issuer, dbar);  // one completion per item, also after an abort
      if (lane == 0 && !ok) *sAbort = 1;
      __syncwarp();
    } else if constexpr (RULE) {
      // ---------------------------------------------------------------- softmax with a rule (two threads per head row)
      // A thread has half of the row's keys (hf: 0-31 or 32-63 of each tile) in registers from the rule to the
      // exponentials, and half of its channels when O is rescaled or written. The two of a row, on two warps, agree on
      // the row's maximum through shared memory, so every decision is the same in both.
      const int qd = warp & 3, hf = warp >= kSecondWarp0;  // quarter of tensor memory (a warp reads that of its number)
      const int slot = lane >> 4, h = qd * 16 + (lane & 15), row = qd * 32 + lane;
      const int b_mine = slot ? b1 : b0;
      float2* bias = sBias + hf * 128 + row;
      if (bias->x < 0.f) {  // far keys lead
        const Keys km = slot ? k1 : k0;
        const int64_t j = km.n == km.n_w ? -1 : p.is_csa ? static_cast<int64_t>(p.sel_idx[(int64_t)b_mine * p.k]) : 0;
        bias->y = bias->x * far_distance(km.t, km.ws, j, p.m, p.n_win);
      }
      const uint32_t trow = tmem + (static_cast<uint32_t>(qd * 32) << 16);
      uint8_t* prow = sP + slot * (kPBytes / 2) + h * 128;
      const int sw = h & 7;
      float m_used = -INFINITY, l_run = 0.f;
      // a wait that gave up is told at the next barrier, which every warp of the row reaches
      bool ok = true, good = true;
      for (int it = 0; it < ntiles; ++it) {
        const uint32_t gt = g + it;
        const int st = gt % kNS;
        // kfull: the stage's valid-key bits and distances (that phase cannot move on before this thread's pfull arrival)
        good = good && __all_sync(kFull, mbar_wait(&sfull[gt & 1u], (gt >> 1) & 1u, p.status)) &&
                    __all_sync(kFull, mbar_wait(&kfull[st], (gt / kNS) & 1u, p.status));
        uint32_t s[32];
        float mt = -INFINITY;
        if (good) {
          tc_fence_after();
          tmem_ld32(trow + kColS + (gt & 1u) * kNk + 32 * hf, s);
          tmem_ld_wait();
          const float4* pos = reinterpret_cast<const float4*>(sDist + st * kRows + slot * kNk + 32 * hf);
          const float2 sb = *bias;
          if (rule.cap2.x > 0.f)
            apply_rule<true>(s, pos, rule, sb.x, sb.y);
          else
            apply_rule<false>(s, pos, rule, sb.x, sb.y);
          const uint32_t vm = sMask[st * 4 + slot * 2 + hf];
          if (!__all_sync(kFull, vm == kFull)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((vm >> j) & 1u)) s[j] = 0xff800000u;  // -inf
          }
          float m1 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            mt = max3(mt, __uint_as_float(s[j]), __uint_as_float(s[j + 1]));
            m1 = max3(m1, __uint_as_float(s[j + 2]), __uint_as_float(s[j + 3]));
          }
          mt = fmaxf(mt, m1);
        }
        float* side = sSide + (gt & 1u) * 256;  // two buffers: a thread writes the next tile's before its partner reads this
        side[hf * 128 + row] = mt;
        ok = !named_sync_or(4 + qd, 64, !good || *sAbort);
        if (!ok) {
          *sAbort = 1;
          break;
        }
        mt = fmaxf(mt, side[(1 - hf) * 128 + row]);
        float corr = 1.f;
        bool rescale = false;
        if (mt > m_used + kRescaleThreshold || (m_used == -INFINITY && mt != -INFINITY)) {
          corr = ex2(m_used - mt);  // 0 when m_used is -inf
          rescale = it > 0;
          l_run *= corr;
          m_used = mt;
        }
        const float msub = m_used == -INFINITY ? 0.f : m_used;
        float l0 = 0.f, l1 = 0.f;
        uint32_t pp[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float e0 = ex2(__uint_as_float(s[2 * j]) - msub), e1 = ex2(__uint_as_float(s[2 * j + 1]) - msub);
          l0 += e0;
          l1 += e1;
          pp[j] = pack_bf16(e0, e1);
        }
        l_run += l0 + l1;
        // P buffer gt & 1 was read by the P V of tile gt - 2; O takes a rescale once that of tile gt - 1 has landed
        if (gt >= 2) good = __all_sync(kFull, mbar_wait(&obar[gt & 1u], ((gt >> 1) - 1) & 1u, p.status));
        if (good && __any_sync(kFull, rescale)) {
          const uint32_t gq = gt - 1;
          good = __all_sync(kFull, mbar_wait(&obar[gq & 1u], (gq >> 1) & 1u, p.status));
          if (good) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 64 * hf; c < 64 * hf + 64; c += 32) {
              uint32_t o[32];
              tmem_ld32(trow + kColO + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
              tmem_st32(trow + kColO + c, o);
            }
            tmem_st_wait();
          }
        }
        if (!good) continue;
        // keys 32 hf + 8 i .. + 7: 16-byte chunk 4 hf + i of the row (one 64-key atom)
        uint8_t* pbuf = prow + (gt & 1u) * kPBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(pbuf + (((4 * hf + i) ^ sw) << 4)) =
              make_uint4(pp[4 * i], pp[4 * i + 1], pp[4 * i + 2], pp[4 * i + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&pfull[gt & 1u]);
      }
      // epilogue: O / l in bf16, and the log-sum-exp; the halves' sums go through the buffer the last tile did not use
      ok = __all_sync(kFull, mbar_wait(dbar, n_item & 1u, p.status)) && ok;
      float* side = sSide + ((g + ntiles) & 1u) * 256;
      side[hf * 128 + row] = l_run;
      ok = !named_sync_or(4 + qd, 64, !ok || !good);
      if (!ok) *sAbort = 1;
      l_run += side[(1 - hf) * 128 + row];
      named_sync_or(4 + qd, 64, false);  // read by both before the next item writes there
      tc_fence_after();
      // a row without keys (or after an abort) writes zeros without reading O
      const bool has = ok && l_run > 0.f;
      const float inv = has ? 1.f / l_run : 0.f;
      const bool write = b_mine >= 0;
      uint16_t* orow = write ? p.out + ((int64_t)b_mine * p.n_heads + h) * kD : nullptr;
      const int64_t tq = write ? p.q_pos[b_mine] : 0;
#pragma unroll 1
      for (int c = 64 * hf; c < 64 * hf + 64; c += 32) {
        uint32_t o[32];
        if (ok) {  // warp-uniform: every lane takes part in the tensor-memory load
          tmem_ld32(trow + kColO + c, o);
          tmem_ld_wait();
        }
        if (!write) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = has ? __uint_as_float(o[8 * i + e]) * inv : 0.f;
          if (p.rope_dims > 0 && has) {  // inverse RoPE of the output's last rope_dims channels
            float a4[4] = {f[0], f[1], f[2], f[3]}, b4[4] = {f[4], f[5], f[6], f[7]};
            inverse_rope4(a4, c + 8 * i, kD, p.rope_dims, p.rope_base, tq);
            inverse_rope4(b4, c + 8 * i + 4, kD, p.rope_dims, p.rope_base, tq);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = a4[e];
              f[4 + e] = b4[e];
            }
          }
          *reinterpret_cast<uint4*>(orow + c + 8 * i) =
              make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
      }
      if (hf == 0 && write && p.lse)
        p.lse[(int64_t)b_mine * p.n_heads + h] = has ? (m_used + log2f(l_run)) * kLn2 - bias->y * kLn2 : -INFINITY;
      tc_fence_before();  // the next item's first P V overwrites O: this thread's reads of it are complete
    } else if constexpr (!RULE) {
      // ---------------------------------------------------------------- softmax (one head row per thread)
      const int slot = lane >> 4, h = warp * 16 + (lane & 15);
      const int b_mine = slot ? b1 : b0;
      const float sl2 = p.sm_scale * kLog2e;
      const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      uint8_t* prow = sP + slot * (kPBytes / 2) + h * 128;
      const int sw = h & 7;
      float m_used = -INFINITY, l_run = 0.f;
      bool ok = true;
      for (int it = 0; it < ntiles && ok; ++it) {
        const uint32_t gt = g + it;
        const uint32_t sb = trow + kColS + (gt & 1u) * kNk;
        if (!__all_sync(kFull, mbar_wait(&sfull[gt & 1u], (gt >> 1) & 1u, p.status))) {
          *sAbort = 1;
          ok = false;
          break;
        }
        // the stage's valid-key bits (written before the loaders' kfull arrival; that phase
        // cannot move on before this thread's pfull arrival for the tile)
        if (!__all_sync(kFull, mbar_wait(&kfull[gt % kNS], (gt / kNS) & 1u, p.status))) {
          *sAbort = 1;
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t* valid = sMask + (gt % kNS) * 4 + slot * 2;
        // the tile's 64 logits of this row (two loads, one wait); the row max in four chains
        const uint64_t vm = static_cast<uint64_t>(valid[0]) | (static_cast<uint64_t>(valid[1]) << 32);
        float mt;
        {
          uint32_t s[kNk];
          tmem_ld32(sb, *reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_ld32(sb + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
          tmem_ld_wait();
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int j = 0; j < kNk; j += 4) {
            if ((vm >> j) & 1u) m0 = fmaxf(m0, __uint_as_float(s[j]) * sl2);
            if ((vm >> (j + 1)) & 1u) m1 = fmaxf(m1, __uint_as_float(s[j + 1]) * sl2);
            if ((vm >> (j + 2)) & 1u) m2 = fmaxf(m2, __uint_as_float(s[j + 2]) * sl2);
            if ((vm >> (j + 3)) & 1u) m3 = fmaxf(m3, __uint_as_float(s[j + 3]) * sl2);
          }
          mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
        }
        float corr = 1.f;
        bool rescale = false;
        if (mt > m_used + kRescaleThreshold || (m_used == -INFINITY && mt != -INFINITY)) {
          corr = exp2f(m_used - mt);  // 0 when m_used is -inf
          rescale = it > 0;
          l_run *= corr;
          m_used = mt;
        }
        const float msub = m_used == -INFINITY ? 0.f : m_used;
        // P buffer gt & 1 was read by the P V of tile gt - 2
        if (gt >= 2 && !__all_sync(kFull, mbar_wait(&obar[gt & 1u], ((gt >> 1) - 1) & 1u, p.status))) {
          *sAbort = 1;
          ok = false;
          break;
        }
        if (__any_sync(kFull, rescale)) {
          // O takes the rescale once the P V of tile gt - 1 (and so every earlier one) has landed
          const uint32_t gq = gt - 1;
          if (!__all_sync(kFull, mbar_wait(&obar[gq & 1u], (gq >> 1) & 1u, p.status))) {
            *sAbort = 1;
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kD; c += 32) {
            uint32_t o[32];
            tmem_ld32(trow + kColO + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
            tmem_st32(trow + kColO + c, o);
          }
          tmem_st_wait();
        }
        uint8_t* pbuf = prow + (gt & 1u) * kPBytes;
        {  // the logits again (two loads, one wait), their exponentials, the row sum in two chains
          float l0 = 0.f, l1 = 0.f;
          uint32_t pp[kNk / 2];
          {
            uint32_t s[kNk];
            tmem_ld32(sb, *reinterpret_cast<uint32_t(*)[32]>(s));
            tmem_ld32(sb + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kNk / 2; ++j) {
              const float e0 = (vm >> (2 * j)) & 1u ? exp2f(__uint_as_float(s[2 * j]) * sl2 - msub) : 0.f;
              const float e1 = (vm >> (2 * j + 1)) & 1u ? exp2f(__uint_as_float(s[2 * j + 1]) * sl2 - msub) : 0.f;
              l0 += e0;
              l1 += e1;
              pp[j] = pack_bf16(e0, e1);
            }
          }
          l_run += l0 + l1;
          // keys 8 i .. 8 i + 7: 16-byte chunk i of the row (one 64-key atom)
#pragma unroll
          for (int i = 0; i < kNk / 8; ++i)
            *reinterpret_cast<uint4*>(pbuf + ((i ^ sw) << 4)) =
                make_uint4(pp[4 * i], pp[4 * i + 1], pp[4 * i + 2], pp[4 * i + 3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&pfull[gt & 1u]);
      }
      // epilogue: O / l in bf16, and the log-sum-exp
      ok = __all_sync(kFull, mbar_wait(dbar, n_item & 1u, p.status)) && ok;
      if (!ok) *sAbort = 1;
      tc_fence_after();
      // a row without keys (or after an abort) writes zeros without reading O
      const bool has = ok && l_run > 0.f;
      const float inv = has ? 1.f / l_run : 0.f;
      const bool write = b_mine >= 0;
      uint16_t* orow = write ? p.out + ((int64_t)b_mine * p.n_heads + h) * kD : nullptr;
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (ok) {  // warp-uniform: every lane takes part in the tensor-memory load
          tmem_ld32(trow + kColO + c, o);
          tmem_ld_wait();
        }
        if (write) {
          const int64_t tq = p.q_pos[b_mine];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = has ? __uint_as_float(o[8 * i + e]) * inv : 0.f;
            if (p.rope_dims > 0 && has) {  // inverse RoPE of the output's last rope_dims channels
              float a4[4] = {f[0], f[1], f[2], f[3]}, b4[4] = {f[4], f[5], f[6], f[7]};
              inverse_rope4(a4, c + 8 * i, kD, p.rope_dims, p.rope_base, tq);
              inverse_rope4(b4, c + 8 * i + 4, kD, p.rope_dims, p.rope_base, tq);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                f[e] = a4[e];
                f[4 + e] = b4[e];
              }
            }
            uint4 v;
            v.x = pack_bf16(f[0], f[1]);
            v.y = pack_bf16(f[2], f[3]);
            v.z = pack_bf16(f[4], f[5]);
            v.w = pack_bf16(f[6], f[7]);
            *reinterpret_cast<uint4*>(orow + c + 8 * i) = v;
          }
        }
      }
      if (write && p.lse) p.lse[(int64_t)b_mine * p.n_heads + h] = has ? (m_used + log2f(l_run)) * kLn2 : -INFINITY;
      // the next item's first P V overwrites O: this thread's reads of it are complete
      tc_fence_before();
    }
    g += ntiles;
    ++n_item;
  }
  // after an abort, give tensor-core work and copies in flight a bounded chance to land (each
  // warp decides on lane 0's reading of the flag, so it stays converged)
  if (warp == 4 && __shfl_sync(kFull, *sAbort, 0)) {
    commit_if(elect_one(), dbar);
    __syncwarp();
    mbar_wait(dbar, n_item & 1u, nullptr);
  }
  if (warp == kLoadThread0 / 32 && __shfl_sync(kFull, *sAbort, 0)) mbar_wait(qfull, n_item & 1u, nullptr);
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, kTmemCols);
}

// rows of 128 channels in 64-channel boxes of box_rows rows, 128-byte swizzle
bool encode_rows(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool attend_pair_supported(const AttendParams& p, int n_sm) {
  const uint64_t pool_rows = static_cast<uint64_t>(p.n_pages) * p.page_size;
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  return p.d_qk == kD && p.d_v == kD && p.n_heads == kH && p.kv_dtype == CSKV_BF16 &&
         p.n_q >= 4 * n_sm &&  // enough pairs for every SM without splitting keys
         pool_rows <= kRowMask && ring_rows <= kRowMask && static_cast<uint64_t>(p.chunk_len) <= kRowMask;
}

cudaError_t launch_attend_pair(AttendParams& p, int n_sm, cudaStream_t st) {
  CUtensorMap tm_q, tm_pool, tm_ring, tm_chunk;
  const bool rule = has_score_rule(p);
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  if (!encode_rows(&tm_q, p.q, static_cast<uint64_t>(p.n_q) * kH, kH) ||
      !encode_rows(&tm_pool, p.kv_pool, static_cast<uint64_t>(p.n_pages) * p.page_size, 1) ||
      !encode_rows(&tm_ring, p.ring_x, ring_rows, 1) ||
      !(p.x_chunk && p.chunk_len > 0 ? encode_rows(&tm_chunk, p.x_chunk, static_cast<uint64_t>(p.chunk_len), 1)
                                     : encode_rows(&tm_chunk, p.ring_x, ring_rows, 1)))
    return cudaErrorNotSupported;
  const size_t smem = Smem::bytes();
  auto kern = rule ? attend_pair_kernel<true> : attend_pair_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int items = (p.n_q + 1) / 2;
  const int grid = items < n_sm ? items : n_sm;
  return launch_pdl(kern, dim3(static_cast<unsigned>(grid)),
                    dim3(rule ? Block<true>::kThreads : Block<false>::kThreads), smem, st, tm_q, tm_pool, tm_ring, tm_chunk, p,
                    make_rule(p.sm_scale, p.score_cap));
}

}  // namespace cskv
