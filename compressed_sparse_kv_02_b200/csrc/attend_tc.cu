// attend_tc.cu -- CSA / HCA core attention on the 5th-generation tensor cores
// (tcgen05) for the wide shared latent: d_qk = 576 (512 latent + 64 RoPE
// channels), d_v = 512, query heads in groups of 64 (DeepSeek-V4 report
// digest, section 3: one softmax over the window and the selected / all
// compressed entries; DeepSeek-V4-book ch.1, section 4: the MLA latent shared
// by every head).
//
// With 128 heads on one 576-wide latent every key carries 2 x 128 x 1088
// flops against 1152 bytes, at the B200's ridge point. O for 128 heads x 512
// channels in fp32 would fill a whole SM's tensor memory, so a work item =
// (query, 64-head group, key split): the two head groups of a split run on two
// CTAs that read the same key tiles (the second read is served by L2) and never
// talk to each other. Per CTA, everything is local:
//   - S = Q K^T with the 64 heads as M and a 64-key tile as N, Q (64 x 576) and
//     the key tile (64 x 576) in shared memory; the channel blocks alternate
//     between two accumulators (a tcgen05.mma that accumulates into the tile of
//     the one before it waits for it, ~90 cycles per step, while two chains run
//     at the operand rate), the even blocks at tensor-memory lane offset 0 and
//     the odd ones at lane offset 16 of the same columns (an M = 64 accumulator
//     fills lanes 0-15 of each 32-lane quarter);
//   - O = P V in two halves of 256 channels, O[:, 0:256] at lane offset 0 and
//     O[:, 256:512] at lane offset 16 of columns 0-255, P (bf16) in shared
//     memory as the A operand, V read MN-major from the key tile (V = the first
//     d_v channels of every key);
//   - thread (warp w, lane l) of the softmax warpgroup owns head row 16 w +
//     (l & 15) and keys 32 (l >> 4) .. + 31 of each tile: it reads its lane's
//     accumulator, swaps 32 values with lane l ^ 16 to form the full S of its
//     keys, and the row max is one more swap; the two lanes of a row keep the
//     same running max, and the rare O rescale touches exactly the O rows of
//     every lane (both halves);
//   - one warp issues S and P V, so the next tile's S runs while this tile's
//     exponentials are taken;
//   - loaders look up each tile's source rows one tile ahead, while the tile
//     before it is copied (its page-table reads included): TMA when a
//     tile's rows are contiguous (window rows of the ring, HCA entries of one
//     page), TMA gather of single rows for a bf16 tile of pool rows (the CSA
//     selection), cp.async through the looked-up rows otherwise; the codes of an
//     FP8 tile of pool rows are gathered and widened exactly to bf16, in place, by
//     warps of their own.
// O is rescaled only when a row's running max rises by more than 2^8 (the
// probabilities stay below 256 in bf16), so most tiles skip it. Window keys are
// taken in ring-slot order (the softmax does not depend on the order of its
// keys), which makes a window tile 64 consecutive ring rows. Each item writes
// its normalised partial output and log-sum-exp; attend_merge_t_kernel combines
// the splits.
//
// Measured: a tile's way through its stage (lookup, copy, S, softmax, P V) is a
// chain of ~8,400 cycles for bf16 entries and ~16,800 for FP8 (gather 2,700,
// widening 4,000, S 1,700, softmax 3,700, P V 2,000), with two stages in flight;
// neither memory nor the tensor cores (16-19% active) set the pace. With a rule,
// 8 queries up to 1M tokens (HCA, 128 heads) take 36.7 us; 64 FP8 queries of 1152
// keys (CSA, 128 heads) 99-100 us, 201 before the codes came by TMA, 159 with loader
// warps that also widened them.
//
// RULE is the form with a cap or a distance bias on the logits: the loaders write
// each key's distance beside its source row, and the softmax applies the rule to
// the fp32 logits before the running max.
#include "attend_plan.cuh"
#include "cskv_device.cuh"
#include "cskv_internal.h"
#include "score_rule.cuh"
#include "tc_issue.cuh"

namespace cskv {
namespace {

constexpr int kDqk = 576, kDv = 512, kH = 64, kNk = 64;
constexpr int kNb = kDqk / 64;                  // 9 channel blocks of a key row
constexpr int kBlkBytes = kNk * 128;            // 8192: one channel block of a 64-row tile
constexpr int kStageBytes = kNb * kBlkBytes;    // 73728: a key tile (also the Q block set)
constexpr int kNS = 2;                          // key-tile stages
constexpr int kPBytes = kH * kNk * 2;           // 8192: P of the tile (bf16)
constexpr int kLoadThread0 = 160;               // warps 0-3 softmax, warp 4 MMA, 5-7 loaders, FP8: 8-15 wideners
// Three loader warps. FP8 entries have eight more that copy the codes of a tile and widen them to bf16, eight keys each,
// while the loaders look up the next one.
constexpr int kLoaders = 96;
constexpr int kWidenThread0 = 256, kWideners = 256;
template <bool FP8>
struct Block {
  static constexpr int kThreads = FP8 ? kWidenThread0 + kWideners : 256;
};
constexpr int kChunks = kNk * kNb * 8;          // 16-byte chunks of a bf16 tile (4608)
// an FP8 tile's codes: pieces of 128 channels behind the stage's first four blocks
constexpr int kPieces = (kDqk + 127) / 128, kCodes0 = 4 * kBlkBytes;
static_assert(kCodes0 + kPieces * kBlkBytes == kStageBytes, "code pieces");
constexpr uint32_t kTmemCols = 512;
// O[:, 0:256] lanes +0 and O[:, 256:512] lanes +16 of columns 0-255; S buffer k at columns
// 256 + 64 k (even channel blocks at lanes +0, odd ones at lanes +16)
constexpr uint32_t kColO = 0, kColS = 256;
constexpr uint32_t kLane16 = 16u << 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;       // log2 units
constexpr int kMaxSplitKeys = 1024;             // keys of one HCA work item at most (16 tiles)

template <bool FP8, bool RULE>
struct Smem {
  // FP8 entries with a rule have both a scale and a distance per key; the tiles' source-row codes, which only the
  // loaders read, then keep one buffer (every read of it is done when the loaders meet for the next tile)
  static constexpr int kCodes = FP8 && RULE ? 1 : kNS;
  static constexpr int Q = 0;                          // 9 blocks of 64 heads x 128 B
  static constexpr int K = Q + kStageBytes;            // kNS key tiles
  static constexpr int P = K + kNS * kStageBytes;      // P of the tile (64 rows x 128 B)
  static constexpr int CODE = P + kPBytes;             // [kCodes][kNk] source-row codes of a stage's keys
  static constexpr int SCALE = CODE + kCodes * kNk * 4;  // [kNS][kNk] FP8 scale of each key (1 for bf16 rows)
  static constexpr int DIST = SCALE + (FP8 ? kNS * kNk * 4 : 0);  // RULE: [kNS][kNk] minus the distance of each key
  static constexpr int MASK = DIST + (RULE || !FP8 ? kNS * kNk * 4 : 0);  // [kNS][2] valid-key bits
  static constexpr int BAR = MASK + 32;                // mbarriers
  static constexpr int TMEM = BAR + 16 * 8;            // allocated tensor-memory address | FP8: tile kinds
  static constexpr int FLAGS = TMEM + 16;
  static constexpr int PREF = FLAGS + 16;              // [n_q + 1] items per query, exclusive prefix
  static size_t bytes(int n_q) { return 1024 + PREF + sizeof(int) * (size_t)(n_q + 1); }
};

static_assert(Smem<false, true>::DIST % 16 == 0 && Smem<true, true>::DIST % 16 == 0 && Smem<true, true>::SCALE % 16 == 0 &&
                  Smem<true, false>::SCALE % 16 == 0,
              "alignment");

// source-row code: kind in bits [31:30] (0 none, 1 pool entry, 2 ring row, 3 chunk row), row below
constexpr uint32_t kRowBits = 30;
constexpr uint32_t kRowMask = (1u << kRowBits) - 1u;

struct Keys {
  int64_t t, ws;
  int n_w;
  int64_t n;
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
  r.n = r.n_w + n_c;
  return r;
}

// The source row of one key, found in three steps a tile apart, so that no step waits for the loads of the one before
// it: which key (its entry, through the selection), which page, which row (and scale).
// Window keys come first, in ring-slot order (slot u) when every window row is in the ring, in position order when a
// prefill chunk supplies some of them; then the compressed entries. A code of 0 is an invalid row.
struct Lookup {
  uint32_t code;  // of a window row
  int32_t page;   // of an entry's
  int32_t slot;   // its place in the page
  int64_t entry;  // the entry, -1: none
  float dist;     // the key's distance from the query in tokens (RULE)
};
__device__ __forceinline__ void look_key(const AttendParams& p, int b, int seq, const Keys& k, int64_t u, Lookup& l) {
  l.code = 0;
  l.entry = -1;
  l.dist = 0.f;
  if (u < k.n_w) {
    if (!p.x_chunk) {
      l.dist = static_cast<float>((k.t - u) % p.n_win);  // slot u holds the latest position up to t that is u mod n_win
      l.code = (2u << kRowBits) | static_cast<uint32_t>((int64_t)seq * p.n_win + u);
      return;
    }
    const int64_t pos = k.ws + u;
    l.dist = static_cast<float>(k.t - pos);
    const int64_t cr = chunk_row(p, seq, pos);
    l.code = cr >= 0 ? (3u << kRowBits) | static_cast<uint32_t>(cr)
                     : (2u << kRowBits) | static_cast<uint32_t>((int64_t)seq * p.n_win + pos % p.n_win);
    return;
  }
  const int64_t jj = u - k.n_w;
  l.entry = p.is_csa ? static_cast<int64_t>(p.sel_idx[(int64_t)b * p.k + jj]) : jj;
}
__device__ __forceinline__ void look_page(const AttendParams& p, int seq, const Keys& k, Lookup& l) {
  l.page = -1;
  const int64_t j = l.entry;
  if (j < 0 || j >= k.n_vis) return;
  l.dist = entry_distance(k.t, j, p.m);
  const int64_t pi = j < 0x7fffffff ? static_cast<uint32_t>(j) / static_cast<uint32_t>(p.page_size) : j / p.page_size;
  l.slot = static_cast<int32_t>(j - pi * p.page_size);
  if (pi < p.max_pages_per_seq) l.page = p.page_table[(int64_t)seq * p.max_pages_per_seq + pi];
}
__device__ __forceinline__ uint32_t look_row(const AttendParams& p, const Lookup& l) {
  if (l.code) return l.code;
  if (l.page < 0 || l.page >= p.n_pages) return 0;
  return (1u << kRowBits) | static_cast<uint32_t>((int64_t)l.page * p.page_size + l.slot);
}

// the bf16 row of a code (an FP8 pool row is read as codes by the loaders)
__device__ __forceinline__ const uint16_t* code_row(const AttendParams& p, uint32_t c) {
  const uint32_t kind = c >> kRowBits, row = c & kRowMask;
  if (kind == 1) return static_cast<const uint16_t*>(p.kv_pool) + (size_t)row * kDqk;
  if (kind == 2) return p.ring_x + (size_t)row * kDqk;
  if (kind == 3) return p.x_chunk + (size_t)row * kDqk;
  return nullptr;
}

// 4 E4M3 codes -> 4 bf16, exact: every E4M3 value is a bf16 value. A code's four exponent and three mantissa bits, put
// at the bottom of the exponent and the top of the mantissa of a bf16, stand for the value times 2^-120 (subnormals
// included), so one packed product per two codes is left. The two codes that are NaN (all seven bits set) have no such
// product: nan_codes finds them and set_nan writes them.
__device__ __forceinline__ uint2 code_bits(uint32_t w) {
  const uint32_t lo = (w << 4) & 0xf0f0f0f0u, hi = ((w >> 4) & 0x07070707u) | (w & 0x80808080u);  // the halves' bytes
  return make_uint2(__byte_perm(lo, hi, 0x5140u), __byte_perm(lo, hi, 0x7362u));
}
__device__ __forceinline__ uint32_t unscale(uint32_t v) {
  const uint32_t scale = 0x7b807b80u;  // 2^120 twice
  const __nv_bfloat162 f = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&scale));
  return *reinterpret_cast<const uint32_t*>(&f);
}
__device__ __forceinline__ uint4 widen8(uint2 c) {
  const uint2 a = code_bits(c.x), b = code_bits(c.y);
  return make_uint4(unscale(a.x), unscale(a.y), unscale(b.x), unscale(b.y));
}
__device__ __forceinline__ uint32_t nan_bits(uint32_t w) { return (w & 0x7f7f7f7fu) + 0x01010101u; }
// bit 7 of a byte: some code there is NaN
__device__ __forceinline__ uint32_t nan_codes(uint2 c) { return (nan_bits(c.x) | nan_bits(c.y)) & 0x80808080u; }
__device__ __forceinline__ uint4 set_nan(uint4 v, uint2 c) {
  const uint2 a = code_bits(c.x), b = code_bits(c.y);
  auto nan = [](uint32_t h) { return ((((h & 0x07f007f0u) + 0x00100010u) >> 11) & 0x00010001u) * 0x7fffu; };
  return make_uint4(v.x | nan(a.x), v.y | nan(a.y), v.z | nan(b.x), v.w | nan(b.y));
}
__device__ __forceinline__ uint4 e4m3x8_to_bf16x8(uint2 c) {
  const uint4 v = widen8(c);
  return nan_codes(c) ? set_nan(v, c) : v;
}

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(n) : "memory");
}
// S of one key tile: 9 channel blocks x 4 K-steps (M = 64 heads, N = 64 keys); even blocks
// accumulate at d (lanes +0), odd blocks at d + 16 lanes, the two chains issued alternately.
// The stage is a uniform value, not a branch: every copy of this code is fetched cold once a block.
__device__ __forceinline__ void issue_s(uint32_t issuer, uint32_t d, uint32_t q, uint32_t k, uint32_t idesc) {
  const uint64_t qd = umma_desc_sw128(q, 16, 1024), kd = umma_desc_sw128(k, 16, 1024);
#pragma unroll
  for (int ia = 0; ia < kNb; ia += 2) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {  // a descriptor counts addresses in 16 bytes
      const int o = ia * (kBlkBytes / 16) + 2 * ks;
      umma_ss_if(issuer, d, qd + o, kd + o, idesc, o > 0 ? 1u : 0u);
      if (ia + 1 < kNb)
        umma_ss_if(issuer, d + kLane16, qd + kBlkBytes / 16 + o, kd + kBlkBytes / 16 + o, idesc, o > 0 ? 1u : 0u);
    }
  }
}

// Pipeline (per CTA; tiles numbered gt across its items; stage and S buffer gt & 1):
//   loaders : look up the tile's source rows -> wait kempty (P V of tile gt - 2 done) ->
//             TMA, or cp.async / widened FP8 stores, into the stage -> kfull
//   MMA warp: kfull, sfree (softmax has read S(gt - 2)) -> S(gt) -> commit sfull;
//             pfull -> P V(gt) -> commit kempty, obar
//   softmax : wait sfull -> read S, swap halves with lane ^ 16, arrive sfree -> P(gt) ->
//             wait obar (P V of gt - 1 done: P buffer free, O settled; rare rescale) ->
//             store P -> pfull
// FP8: the pool holds E4M3 entries with an fp32 scale each (a separate
// instantiation keeps the bf16 kernel's code small)
template <bool FP8, bool RULE>
__global__ void __launch_bounds__(Block<FP8>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_ring,
                     const __grid_constant__ CUtensorMap tm_kv, const __grid_constant__ CUtensorMap tm_kvg,
                     const AttendParams p, const __grid_constant__ Rule rule) {
  using Sm = Smem<FP8, RULE>;
  constexpr int kThreads = Block<FP8>::kThreads;
  constexpr int kPasses = FP8 ? 6 : 2, kPer = kChunks / (kPasses * kLoaders);
  static_assert(kPer * kPasses * kLoaders == kChunks, "chunks per pass");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm + Sm::Q;
  uint8_t* sK = sm + Sm::K;
  uint8_t* sP = sm + Sm::P;
  uint32_t* sCodes = reinterpret_cast<uint32_t*>(sm + Sm::CODE);
  float* sScale = reinterpret_cast<float*>(sm + Sm::SCALE);
  float* sDist = reinterpret_cast<float*>(sm + Sm::DIST);
  uint32_t* sMask = reinterpret_cast<uint32_t*>(sm + Sm::MASK);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sm::BAR);
  uint64_t* kfull = bars;             // [2] loaders (and wideners) -> MMA warp (and the softmax, for the stage's key bits)
  uint64_t* kempty = bars + 2;        // [2] P V of the stage's tile done (commit)
  uint64_t* sfull = bars + 4;         // [2] S of the buffer's tile done (commit)
  uint64_t* sfree = bars + 6;         // [2] softmax has read the buffer (128 arrivals)
  uint64_t* obar = bars + 8;          //     a tile's P V done (commit)
  uint64_t* qbar = bars + 9;          //     Q of the item landed (TMA)
  uint64_t* dbar = bars + 10;         //     the item's last P V done (commit)
  uint64_t* rdy = bars + 11;          // [2] FP8, loaders -> wideners: the tile's kind and source rows are known
  uint64_t* cfree = bars + 13;        //     FP8, wideners -> loaders: they have read the tile's source rows
  uint64_t* cbar = bars + 14;         //     FP8: a tile's codes landed (TMA)
  uint64_t* pfull = bars + 15;        //     softmax -> MMA warp: P of a tile is stored (128 arrivals)
  constexpr bool fp8 = FP8;
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + Sm::TMEM);
  volatile int* sAbort = reinterpret_cast<int*>(sm + Sm::FLAGS);
  volatile int* sLdOk = reinterpret_cast<int*>(sm + Sm::FLAGS) + 1;
  volatile int* sPool = reinterpret_cast<int*>(sm + Sm::FLAGS) + 2;  // [2] per code warp: the tile is gatherable
  volatile int* sKind = reinterpret_cast<int*>(sm + Sm::TMEM) + 1;  // [2] FP8: the stage's tile is one of codes
  int* sPref = reinterpret_cast<int*>(sm + Sm::PREF);
  __shared__ int s_wsum[32];

  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  const int groups = p.n_heads / kH;
  int kps = p.keys_per_split;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&kfull[i], FP8 ? 1 + kWideners / 32 : 1);
      mbar_init(&kempty[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 128);
      mbar_init(&rdy[i], 1);
    }
    mbar_init(obar, 1);
    mbar_init(qbar, 1);
    mbar_init(dbar, 1);
    mbar_init(pfull, 128);
    mbar_init(cfree, kWideners / 32);
    mbar_init(cbar, kWideners / 32);
    fence_barrier_init();
    *sAbort = 0;
  }
  if (tid == kLoadThread0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_ring);
    prefetch_tensormap(&tm_kv);
    prefetch_tensormap(&tm_kvg);
  }
  if (warp == 4) {
    tmem_alloc(sTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *sTmem, 0);
  // the set-up above overlaps the tail of the kernel launched before this one; its
  // outputs (the selection, new cache rows) are read only from here on
  grid_dependency_wait();
  grid_dependents_launch();
  if constexpr (RULE) kps = plan_split(p, kNk, p.slots, lane, [&](int b) { return keys_of(p, b).n; });
  {  // items per query: splits x head groups
    int run = 0;
    for (int base = 0; base < p.n_q; base += kThreads) {
      const int b = base + tid;
      int v = 0;
      if (b < p.n_q) {
        const Keys k = keys_of(p, b);
        v = static_cast<int>((k.n + kps - 1) / kps) * groups;
      }
      int tot;
      const int ex = block_exclusive_scan<kThreads>(v, s_wsum, tot);
      if (b < p.n_q) sPref[b] = run + ex;
      run += tot;
    }
    if (tid == 0) sPref[p.n_q] = run;
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.n_q; b += kThreads)
      if (p.q_pos[b] < 0 || p.q_pos[b] > p.max_pos) report(p.status, CSKV_ERR_INVALID_ARG);
  if (RULE && blockIdx.x == 0) {
    if (tid == 0) p.plan[0] = kps;
    for (int b = tid; b <= p.n_q; b += kThreads) p.plan[1 + b] = sPref[b] / groups;
  }
  const int total = sPref[p.n_q];
  uint32_t g = 0;       // tiles processed by this CTA before the current item
  uint32_t n_item = 0;  // items processed before the current one (qbar / dbar phase)
  uint32_t n_gather = 0;  // FP8 tiles of codes before the current one (cbar phase)

  // consecutive items are the head groups of one split, so the CTAs reading the same keys run together
  for (int item = blockIdx.x; item < total; item += gridDim.x, ++n_item) {
    int lo = 0, hi = p.n_q - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sPref[mid] <= item) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const int r = item - sPref[b];
    const int grp = r % groups;
    const int split = r / groups;
    // where the piece's partial output goes
    const int64_t slot = RULE ? sPref[b] / groups + split : (int64_t)b * p.max_splits + split;
    const Keys kk = keys_of(p, b);
    const int seq = p.q_seq[b];
    const bool seq_ok = seq >= 0 && seq < p.n_seqs_layer;
    const int64_t u0 = (int64_t)split * kps;
    const int nk = static_cast<int>(kk.n - u0 < kps ? kk.n - u0 : kps);
    const int ntiles = (nk + kNk - 1) / kNk;
    if (tid == 0 && grp == 0 && !seq_ok && kk.n > 0) report(p.status, CSKV_ERR_OUT_OF_RANGE);

    if (tid >= kLoadThread0 && tid < kWidenThread0) {
      // ------------------------------------------------------------ loaders
      const int lt = tid - kLoadThread0, lw = lt >> 5, ll = lt & 31;
      if (lw == 2) {  // Q of the head group: 9 boxes of 64 rows x 64 channels (by the warp without lookups)
        if (ll == 0) {
          mbar_arrive_expect_tx(qbar, kStageBytes);
          const int qrow = b * p.n_heads + grp * kH;
          for (int j = 0; j < kNb; ++j) tma_load_2d(sQ + j * kBlkBytes, &tm_q, j * 64, qrow, qbar);
        }
        __syncwarp();
      }
      // TMA source of tile it: 0 = ring rows, 1 = pool rows (row0 set), -1 = looked-up rows
      auto tile_src = [&](int it, int& row0) -> int {
        const int64_t a = u0 + (int64_t)it * kNk;
        if (!seq_ok || (it + 1) * kNk > nk) return -1;  // a partial tile: rows past its end are not zero
        if (!p.x_chunk && a + kNk <= kk.n_w) {
          row0 = static_cast<int>((int64_t)seq * p.n_win + a);
          return 0;
        }
        if (!p.is_csa && !fp8 && a >= kk.n_w) {
          const int64_t j0 = a - kk.n_w;
          const int64_t pi = j0 / p.page_size;
          if (j0 % p.page_size + kNk > p.page_size || pi >= p.max_pages_per_seq) return -1;
          const int32_t page = p.page_table[(int64_t)seq * p.max_pages_per_seq + pi];
          if (page < 0 || page >= p.n_pages) return -1;
          row0 = static_cast<int>((int64_t)page * p.page_size + j0 % p.page_size);
          return 1;
        }
        return -1;
      };
      // key lt of tile it (threads 0 .. kNk - 1)
      auto key_at = [&](int it, Lookup& l) {
        l.code = 0;
        l.entry = -1;
        l.dist = 0.f;
        const int i = it * kNk + lt;
        if (lt < kNk && i < nk && seq_ok) look_key(p, b, seq, kk, u0 + i, l);
      };
      // the bf16 row into L2 ahead of its copy, line by line (a bulk prefetch is issued for one lane at a time: ~70
      // cycles a row, 4,500 a tile)
      auto prefetch = [&](uint32_t c) {
        if (!c) return;
        const uint8_t* row = reinterpret_cast<const uint8_t*>(code_row(p, c));
        for (int o = 0; o < 2 * kDqk; o += 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(row + o));
      };
      // the next tile's source is found before its stage frees; its key two tiles, its page one tile before that
      float nsc = 0.f, ndist = 0.f;
      uint32_t ncode = 0u;
      int nrow0 = 0, nmode = -1;
      Lookup l1, l2;  // of the tiles it + 1 (page found) and it + 2 (key found), seen from tile it
      auto next = [&](int it) {  // the source of tile it + 1, and the lookups of the two after it a step further
        ncode = look_row(p, l1);
        ndist = l1.dist;
        if (!ncode && lt < kNk && (it + 1) * kNk + lt < nk && seq_ok && grp == 0) report(p.status, CSKV_ERR_OUT_OF_RANGE);
        nsc = !ncode ? 0.f : (fp8 && (ncode >> kRowBits) == 1u) ? p.kv_scale[ncode & kRowMask] : 1.f;
        nmode = tile_src(it + 1, nrow0);
        if (nmode < 0 && !fp8) prefetch(ncode);  // a line of FP8 rows is gathered well before it is needed
        l1 = l2;
        look_page(p, seq, kk, l1);
        key_at(it + 3, l2);
      };
      key_at(0, l1);
      key_at(1, l2);
      look_page(p, seq, kk, l1);
      if (ntiles > 0) next(-1);
      for (int it = 0; it < ntiles; ++it) {
        const uint32_t gt = g + it;
        const int st = gt & 1;
        uint32_t* sCode = sCodes + (Sm::kCodes == 1 ? 0 : st * kNk);
        const uint32_t code = ncode;
        const float scale = nsc, dist = ndist;
        // the first loader warp takes the stage wait (all lanes; lane 0 records the result)
        if (lw == 0) {
          bool okw = __shfl_sync(kFull, *sAbort, 0) == 0;
          if (okw && gt >= 2u) okw = __all_sync(kFull, mbar_wait(&kempty[st], ((gt >> 1) - 1) & 1u, p.status));
          if (FP8 && okw && gt >= 1u) okw = __all_sync(kFull, mbar_wait(cfree, (gt - 1) & 1u, p.status));
          if (ll == 0) *sLdOk = okw;
        }
        named_sync(3, kLoaders);
        if (!*sLdOk) {
          *sAbort = 1;
          break;
        }
        if (lt < kNk) {
          sCode[lt] = code;
          if (FP8) sScale[st * kNk + lt] = code ? scale : 0.f;  // finite for every key of the tile
          if (RULE) sDist[st * kNk + lt] = -dist;
        }
        if (lw < 2) {
          const unsigned bits = __ballot_sync(kFull, code != 0u);
          // a bf16 tile whose rows are all pool rows (or none) is gathered by TMA
          const bool pool = __all_sync(kFull, code == 0u || (code >> kRowBits) == 1u);
          if (ll == 0) {
            sMask[st * 2 + lw] = bits;
            sPool[lw] = pool ? 1 : 0;
          }
        }
        named_sync(3, kLoaders);
        uint8_t* dst = sK + st * kStageBytes;
        const bool pool = sPool[0] && sPool[1];
        if (FP8 && lt == 0) {
          sKind[st] = nmode < 0 && pool;
          mbar_arrive(&rdy[st]);
        }
        const int row0 = nrow0;
        const int mode = nmode;
        if (mode >= 0) {
          if (lt == 0) {
            mbar_arrive_expect_tx(&kfull[st], kStageBytes);
            const CUtensorMap* map = mode == 0 ? &tm_ring : &tm_kv;
            for (int j = 0; j < kNb; ++j) tma_load_2d(dst + j * kBlkBytes, map, j * 64, row0, &kfull[st]);
          }
          if (it + 1 < ntiles) next(it);
        } else if (!fp8 && pool) {
          // the tile's rows by TMA gather, four rows of one 64-channel block per copy; a key without
          // a row reads row -1, outside the map: zeros, as the copies below would write
          if (lt == 0) mbar_arrive_expect_tx(&kfull[st], kStageBytes);
          named_sync(3, kLoaders);  // the stage's byte count is set before any of its copies lands
          for (int q = lt; q < kNb * (kNk / 4); q += kLoaders) {
            const int j = q / (kNk / 4), r4 = (q % (kNk / 4)) * 4;
            int y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t cd = sCode[r4 + e];
              y[e] = (cd >> kRowBits) == 1u ? static_cast<int>(cd & kRowMask) : -1;
            }
            tma_gather4(dst + j * kBlkBytes + r4 * 128, &tm_kvg, j * 64, y[0], y[1], y[2], y[3], &kfull[st]);
          }
          if (it + 1 < ntiles) next(it);
        } else if (fp8 && pool) {  // the wideners'
          if (lt == 0) mbar_arrive(&kfull[st]);
          if (it + 1 < ntiles) next(it);
        } else {
          // consecutive threads take consecutive 16-byte chunks of a row (coalesced): chunk c of key
          // kr is 16-byte piece c & 7 of channel block c >> 3; FP8 entries are read as 8 codes and
          // widened, in passes that bound the registers they hold
#pragma unroll
          for (int half = 0; half < kPasses; ++half) {
            uint2 codes8[kPer];
#pragma unroll
            for (int q = 0; q < kPer; ++q) {
              const int id = lt + (half * kPer + q) * kLoaders;
              codes8[q] = make_uint2(0u, 0u);
              {
                const int kr = id / (kNb * 8), c = id % (kNb * 8);
                const uint32_t cd = sCode[kr];
                if (fp8 && (cd >> kRowBits) == 1u) {
                  codes8[q] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.kv_pool) +
                                                                   (size_t)(cd & kRowMask) * kDqk + c * 8));
                } else {
                  const uint16_t* src = code_row(p, cd);
                  cp_async16(dst + (c >> 3) * kBlkBytes + kr * 128 + (((c & 7) ^ (kr & 7)) << 4),
                             src ? static_cast<const void*>(src + c * 8) : static_cast<const void*>(p.q),
                             src ? 16 : 0);
                }
              }
            }
            if (fp8) {
#pragma unroll
              for (int q = 0; q < kPer; ++q) {
                const int id = lt + (half * kPer + q) * kLoaders;
                if (id < kChunks) {
                  const int kr = id / (kNb * 8), c = id % (kNb * 8);
                  if ((sCode[kr] >> kRowBits) == 1u)
                    *reinterpret_cast<uint4*>(dst + (c >> 3) * kBlkBytes + kr * 128 + (((c & 7) ^ (kr & 7)) << 4)) =
                        e4m3x8_to_bf16x8(codes8[q]);
                }
              }
            }
          }
          cp_async_commit();
          if (it + 1 < ntiles) next(it);  // the next tile's rows are looked up while this tile's copies fly
          cp_async_wait<0>();
          fence_proxy_async_smem();
          named_sync(3, kLoaders);
          if (lt == 0) mbar_arrive(&kfull[st]);
        }
      }
    } else if (FP8 && tid >= kWidenThread0) {
      // ------------------------------------------------------------ wideners
      // A tile of FP8 pool rows: TMA gathers its E4M3 codes, four rows of 128 channels per copy (a missing row reads
      // zeros), into five pieces of 64 swizzled 128-byte rows over the stage's last 40 KB; the rows are spread over
      // the whole pool, and copies by the threads (cp.async) stood in line for their translations (4,400 cycles a
      // tile). The codes are then widened to bf16 in place. Row kr of block 4 + i lies where row kr of piece i was,
      // which holds blocks 2i and 2i + 1, and a warp has its eight keys' rows to itself: it goes through the blocks in
      // order, two at a time, each pair read a step ahead, and no other warp has to wait for it. Lane l has the 16
      // codes of key l % 8 in quarter l / 8 of every block: the swizzled pieces of a quarter warp's eight keys lie in
      // different banks, in the loads and in the stores.
      const int ww = warp - kWidenThread0 / 32, h = lane >> 3, kr = ww * 8 + (lane & 7);
      const uint32_t from0 = kCodes0 + kr * 128 + ((h ^ (kr & 7)) << 4), from1 = from0 ^ 64u;  // even and odd blocks
      const uint32_t to0 = kr * 128 + (((2 * h) ^ (kr & 7)) << 4), to1 = to0 ^ 16u;
      for (int it = 0; it < ntiles; ++it) {
        const uint32_t gt = g + it;
        const int st = gt & 1;
        bool okw = __shfl_sync(kFull, *sAbort, 0) == 0;
        if (okw) okw = __all_sync(kFull, mbar_wait(&rdy[st], (gt >> 1) & 1u, p.status));
        if (!okw) {
          *sAbort = 1;
          break;
        }
        uint8_t* dst = sK + st * kStageBytes;
        const bool codes = __shfl_sync(kFull, sKind[st], 0) != 0;
        if (codes) {
          const uint32_t* sCode = sCodes + (Sm::kCodes == 1 ? 0 : st * kNk);
          if (lane == 0) mbar_arrive_expect_tx(cbar, kPieces * 8 * 128);
          __syncwarp();
          if (lane < 2 * kPieces) {
            const int j = lane >> 1, r4 = ww * 8 + (lane & 1) * 4;
            int y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t cd = sCode[r4 + e];
              y[e] = (cd >> kRowBits) == 1u ? static_cast<int>(cd & kRowMask) : -1;
            }
            tma_gather4(dst + kCodes0 + j * kBlkBytes + r4 * 128, &tm_kvg, j * 128, y[0], y[1], y[2], y[3], cbar);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(cfree);
        if (codes) {
          if (!__all_sync(kFull, mbar_wait(cbar, n_gather & 1u, p.status))) {
            *sAbort = 1;
            mbar_wait(cbar, n_gather & 1u, nullptr);  // once more: the copies may not outlive the block
            break;
          }
          ++n_gather;
          uint4 v = *reinterpret_cast<const uint4*>(dst + from0), w = *reinterpret_cast<const uint4*>(dst + from1);
#pragma unroll 1
          for (int s = 0; s < kPieces; ++s) {  // blocks 2s and 2s + 1 (the last pair has one block)
            uint4 nv = make_uint4(0u, 0u, 0u, 0u), nw = nv;
            if (s + 1 < kPieces) {
              nv = *reinterpret_cast<const uint4*>(dst + from0 + (s + 1) * kBlkBytes);
              if (2 * s + 3 < kNb) nw = *reinterpret_cast<const uint4*>(dst + from1 + (s + 1) * kBlkBytes);
            }
            const uint2 c[4] = {make_uint2(v.x, v.y), make_uint2(v.z, v.w), make_uint2(w.x, w.y), make_uint2(w.z, w.w)};
            uint4 o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = widen8(c[i]);
            if (nan_codes(c[0]) | nan_codes(c[1]) | nan_codes(c[2]) | nan_codes(c[3])) {
#pragma unroll
              for (int i = 0; i < 4; ++i) o[i] = set_nan(o[i], c[i]);
            }
            __syncwarp();  // blocks 4 to 8 overwrite codes that the warp has read by now
            uint8_t* to = dst + 2 * s * kBlkBytes;
            *reinterpret_cast<uint4*>(to + to0) = o[0];
            *reinterpret_cast<uint4*>(to + to1) = o[1];
            if (2 * s + 1 < kNb) {
              *reinterpret_cast<uint4*>(to + kBlkBytes + to0) = o[2];
              *reinterpret_cast<uint4*>(to + kBlkBytes + to1) = o[3];
            }
            v = nv;
            w = nw;
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&kfull[st]);
      }
    } else if (warp == 4) {
      // ------------------------------------------------------------ MMA issue
      // One warp issues S of a tile and P V of the one before in the order in which they become possible. (P V from a
      // softmax warp stood in the tensor cores' queue behind the next S: 2,200 cycles of every tile's softmax.)
      const uint32_t issuer = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(kH, kNk, false), idesc_pv = umma_idesc_bf16(kH, 256, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK), sPa = smem_u32(sP);
      bool ok = __all_sync(kFull, mbar_wait(qbar, n_item & 1u, p.status));
      tc_fence_after();
      int is = 0, ip = 0;  // tiles whose S, whose P V have been issued
      uint32_t polls = 0;
      while (ip < ntiles && ok) {
        const uint32_t gp = __shfl_sync(kFull, g + ip, 0), gs = __shfl_sync(kFull, g + is, 0);
        const int kp = gp & 1, k = gs & 1;
        if (ip < is && mbar_done(pfull, gp & 1u)) {
          tc_fence_after();
          // channel blocks 0..7 of the tile: V
          const uint64_t pd = umma_desc_sw128(sPa, 16, 1024), vd = umma_desc_sw128(sKa + kp * kStageBytes, kBlkBytes, 1024);
#pragma unroll
          for (int ks = 0; ks < kNk / 16; ++ks) {
            const uint32_t acc = (ip > 0 || ks > 0) ? 1u : 0u;
            umma_ss_if(issuer, tmem + kColO, pd + 2 * ks, vd + ks * 16 * 8, idesc_pv, acc);
            umma_ss_if(issuer, tmem + kColO + kLane16, pd + 2 * ks, vd + 4 * kBlkBytes / 16 + ks * 16 * 8, idesc_pv, acc);
          }
          commit_if(issuer, &kempty[kp]);
          commit_if(issuer, obar);
          __syncwarp();
          ++ip;
          polls = 0;
        } else if (is < ntiles && mbar_done(&kfull[k], (gs >> 1) & 1u) &&
                   (gs < 2 || mbar_done(&sfree[k], ((gs >> 1) - 1) & 1u))) {
          // the stage is shared memory written by TMA or fenced cp.async / stores: the mbarrier
          // orders it; S buffer k is free once the softmax has read S(gs - 2)
          tc_fence_after();
          const uint32_t ks = __shfl_sync(kFull, k, 0);
          issue_s(issuer, tmem + kColS + ks * kNk, sQa, sKa + ks * kStageBytes, idesc_s);
          commit_if(issuer, &sfull[k]);
          __syncwarp();
          ++is;
          polls = 0;
        } else if ((++polls & 255u) == 0u) {  // bounded like every wait
          ok = __shfl_sync(kFull, *sAbort, 0) == 0 && polls < kSpinLimit;
          if (!ok && polls >= kSpinLimit) report(p.status, CSKV_ERR_TIMEOUT);
        }
      }
      commit_if(issuer, dbar);  // one completion per item, also after an abort
      if (!ok && lane == 0) *sAbort = 1;
      __syncwarp();
    } else if (warp < 4) {
      // ------------------------------------------------------------ softmax
      // thread (warp, lane): head row hr = 16 warp + (lane & 15), keys 32 kh .. + 31 of each tile
      const float sl2 = p.sm_scale * kLog2e;
      const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
      const int hr = warp * 16 + (lane & 15), kh = lane >> 4;
      const float slope2 = RULE && p.slopes ? p.slopes[grp * kH + hr] * kLog2e : 0.f;
      // a negative slope's logits are relative to the bias of the row's farthest key (no branch on the slope: its load
      // is waited for at the first softmax)
      float negref = 0.f;
      if (RULE && p.slopes) {
        const int64_t j = kk.n == kk.n_w ? -1 : p.is_csa ? static_cast<int64_t>(p.sel_idx[(int64_t)b * p.k]) : 0;
        negref = fminf(slope2, 0.f) * far_distance(kk.t, kk.ws, j, p.m, p.n_win);
      }
      uint8_t* prow = sP + hr * 128;
      float m_used = -INFINITY, l_run = 0.f;
      bool ok = true;
      for (int it = 0; it < ntiles && ok; ++it) {
        const uint32_t gt = g + it;
        const int k = gt & 1;
        bool good = __all_sync(kFull, mbar_wait(&sfull[k], (gt >> 1) & 1u, p.status));
        float s[32];
        if (good) {
          tc_fence_after();
          // this lane's accumulator row (all 64 keys); keep my 32 keys, swap the other 32 with lane ^ 16
          uint32_t a[32], o[32];
          tmem_ld32(tmem + lane_base + kColS + k * kNk, a);
          tmem_ld32(tmem + lane_base + kColS + k * kNk + 32, o);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float mine = __uint_as_float(kh ? o[j] : a[j]);
            const float give = __uint_as_float(kh ? a[j] : o[j]);
            s[j] = mine + __shfl_xor_sync(kFull, give, 16);
          }
        }
        tc_fence_before();
        mbar_arrive(&sfree[k]);
        // the stage's key bits and scales (written before the loaders' kfull arrival; that phase
        // cannot move on before this tile's P V, which waits for this thread's P)
        if (good) good = __all_sync(kFull, mbar_wait(&kfull[k], (gt >> 1) & 1u, p.status));
        bool rescale = false;
        float corr = 1.f;
        uint32_t pp[16];
        if (good) {
          const uint32_t vm = sMask[k * 2 + kh];
          const float4* scl = reinterpret_cast<const float4*>(sScale + k * kNk + 32 * kh);
          if (fp8) {  // an FP8 entry's logit and value carry its scale
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 c = scl[j / 4];
              s[j] *= c.x;
              s[j + 1] *= c.y;
              s[j + 2] *= c.z;
              s[j + 3] *= c.w;
            }
          }
          if constexpr (RULE) {
            const float4* pos = reinterpret_cast<const float4*>(sDist + k * kNk + 32 * kh);
            uint32_t u[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(s[j]);
            if (rule.cap2.x > 0.f)
              apply_rule<true>(u, pos, rule, slope2, negref);
            else
              apply_rule<false>(u, pos, rule, slope2, negref);
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = __uint_as_float(u[j]);
          }
          const float post = RULE ? 1.f : sl2;  // the rule has scaled its logits
          float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            s[j] = ((vm >> j) & 1u) ? s[j] * post : -INFINITY;  // keys past nk have no row
            s[j + 1] = ((vm >> (j + 1)) & 1u) ? s[j + 1] * post : -INFINITY;
            s[j + 2] = ((vm >> (j + 2)) & 1u) ? s[j + 2] * post : -INFINITY;
            s[j + 3] = ((vm >> (j + 3)) & 1u) ? s[j + 3] * post : -INFINITY;
            m0 = fmaxf(m0, s[j]);
            m1 = fmaxf(m1, s[j + 1]);
            m2 = fmaxf(m2, s[j + 2]);
            m3 = fmaxf(m3, s[j + 3]);
          }
          float mt = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
          mt = fmaxf(mt, __shfl_xor_sync(kFull, mt, 16));  // the row's max over the tile's 64 keys
          if (mt > m_used + kRescaleThreshold || (m_used == -INFINITY && mt != -INFINITY)) {
            corr = exp2f(m_used - mt);  // 0 when m_used is -inf
            rescale = it > 0;
            l_run *= corr;
            m_used = mt;
          }
          const float msub = m_used == -INFINITY ? 0.f : m_used;
          float l0 = 0.f, l1 = 0.f;
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = RULE ? ex2(s[2 * j + i] - msub) : exp2f(s[2 * j + i] - msub);
            l0 += e[0];
            l1 += e[1];
            l0 += e[2];
            l1 += e[3];
            if (fp8) {
              const float4 c = scl[j / 2];
              e[0] *= c.x;
              e[1] *= c.y;
              e[2] *= c.z;
              e[3] *= c.w;
            }
            pp[j] = pack_bf16(e[0], e[1]);
            pp[j + 1] = pack_bf16(e[2], e[3]);
          }
          l_run += l0 + l1;
          // the P buffer was read by the P V of tile gt - 1, which also finished O
          if (gt >= 1) good = __all_sync(kFull, mbar_wait(obar, (gt - 1) & 1u, p.status));
        }
        if (good) {
          tc_fence_after();
          if (__any_sync(kFull, rescale)) {
            // lanes +0 hold O[:, 0:256], lanes +16 O[:, 256:512] of the same head rows, and both lanes
            // of a row carry the same corr
#pragma unroll 1
            for (int c = 0; c < 256; c += 32) {
              uint32_t orow[32];
              tmem_ld32(tmem + lane_base + kColO + c, orow);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) orow[j] = __float_as_uint(__uint_as_float(orow[j]) * corr);
              tmem_st32(tmem + lane_base + kColO + c, orow);
            }
            tmem_st_wait();
          }
          // keys 32 kh + 8 i .. + 7: 16-byte chunk 4 kh + i of the row (one 64-key swizzle atom)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(prow + (((4 * kh + i) ^ (hr & 7)) << 4)) =
                make_uint4(pp[4 * i], pp[4 * i + 1], pp[4 * i + 2], pp[4 * i + 3]);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        if (!good || __shfl_sync(kFull, *sAbort, 0)) {
          *sAbort = 1;
          ok = false;
          break;
        }
        mbar_arrive(pfull);
      }
      // epilogue: normalised partial output of this split and head group, and its log-sum-exp
      ok = __all_sync(kFull, mbar_wait(dbar, n_item & 1u, p.status)) && ok;
      if (!ok) *sAbort = 1;
      tc_fence_after();
      const float l_row = l_run + __shfl_xor_sync(kFull, l_run, 16);
      const int head = grp * kH + hr;
      const float inv = l_row > 0.f ? 1.f / l_row : 0.f;
      // RULE: a query in one piece has its answer here, and the merge passes over it
      const bool whole = RULE && p.rope_dims == 0 && sPref[b + 1] - sPref[b] == groups;
      uint16_t* out = p.out + ((int64_t)b * p.n_heads + head) * kDv + kh * 256;
      // part_o is head-minor ([query x split][d_v / 4][heads][4]): the 16 lanes of a half-warp
      // write 16 consecutive heads, 256 contiguous bytes
      float4* po = reinterpret_cast<float4*>(p.part_o) +
                   (slot * (kDv / 4) + kh * 64) * p.n_heads + head;
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t orow[32];
        if (ok) {  // warp-uniform
          tmem_ld32(tmem + lane_base + kColO + c, orow);
          tmem_ld_wait();
        }
        if (whole) {
#pragma unroll
          for (int q = 0; q < 32; q += 16) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              v[i] = ok && l_row > 0.f ? pack_bf16(__uint_as_float(orow[q + 2 * i]) * inv, __uint_as_float(orow[q + 2 * i + 1]) * inv)
                                       : 0u;
            *reinterpret_cast<uint4*>(out + c + q) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(out + c + q + 8) = make_uint4(v[4], v[5], v[6], v[7]);
          }
          continue;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 v = ok ? make_float4(__uint_as_float(orow[4 * q]) * inv, __uint_as_float(orow[4 * q + 1]) * inv,
                                            __uint_as_float(orow[4 * q + 2]) * inv, __uint_as_float(orow[4 * q + 3]) * inv)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
          po[(int64_t)(c / 4 + q) * p.n_heads] = v;
        }
      }
      if (kh == 0) {
        const float lse = l_row > 0.f ? (m_used + log2f(l_row)) * kLn2 : -INFINITY;
        if (!whole) p.part_lse[slot * p.n_heads + head] = lse;
        // pieces are relative: the first leaves the reference where the merge looks for it
        if (RULE && p.lse && (whole || (split == 0 && p.slopes)))
          p.lse[(int64_t)b * p.n_heads + head] = whole ? lse - negref * kLn2 : -negref * kLn2;
      }
    }
    g += ntiles;
    tc_fence_before();
    __syncthreads();  // shared and tensor memory are reused by the next item
    tc_fence_after();
    if (*sAbort) break;
  }
  // after an abort, give tensor-core work in flight a bounded chance to land before freeing
  if (*sAbort && warp == 0) mbar_wait(dbar, n_item & 1u, nullptr);
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, kTmemCols);
}

bool encode_rows(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kDqk), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kDqk) * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of E4M3 codes in one-row boxes of 128 channels (the last box reaches past the row: zeros)
bool encode_codes(CUtensorMap* map, const void* base, uint64_t rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kDqk), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kDqk)};
  const cuuint32_t box[2] = {128, 1};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

static size_t smem_bytes(bool fp8, bool rule, int n_q) {
  return fp8 ? (rule ? Smem<true, true>::bytes(n_q) : Smem<true, false>::bytes(n_q))
             : (rule ? Smem<false, true>::bytes(n_q) : Smem<false, false>::bytes(n_q));
}

bool attend_tc_supported(int d_qk, int d_v, int n_heads, int kv_dtype, int n_q, bool rule) {
  return d_qk == kDqk && d_v == kDv && n_heads % kH == 0 && (kv_dtype == CSKV_BF16 || kv_dtype == CSKV_FP8_E4M3) &&
         smem_bytes(kv_dtype == CSKV_FP8_E4M3, rule, n_q) + 128 <= 232448;  // the per-query prefix table shares shared memory with the tiles
}

// keys per split: queries x head groups x splits ~ one CTA per SM
void attend_tc_plan(AttendParams& p, int n_sm) {
  const int64_t groups = p.n_heads / kH;
  const int64_t n_max = (int64_t)p.n_win + (p.is_csa ? p.k : visible_entries(p.max_pos, p.m, p.n_win));
  int64_t splits = n_sm / ((int64_t)p.n_q * groups);
  if (splits < 1) splits = 1;
  int64_t kps = (n_max + splits - 1) / splits;
  kps = (kps + kNk - 1) / kNk * kNk;
  if (kps < kNk) kps = kNk;
  // HCA key counts grow with the context (n / 128 + 128): with many queries of mixed lengths one split
  // per query would leave the longest ones on one CTA, so no HCA item takes more than kMaxSplitKeys
  // keys (a CSA query has at most n_win + k keys, all of similar count)
  if (!p.is_csa && kps > kMaxSplitKeys) kps = kMaxSplitKeys;
  p.keys_per_split = static_cast<int>(kps);
  p.max_splits = static_cast<int>((n_max + kps - 1) / kps);
  if (p.max_splits < 1) p.max_splits = 1;
}

cudaError_t launch_attend_tc(AttendParams& p, int n_sm, cudaStream_t st) {
  CUtensorMap tm_q, tm_ring, tm_kv, tm_kvg;
  const uint64_t kv_rows = static_cast<uint64_t>(p.n_pages) * p.page_size;
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  if (kv_rows > kRowMask || ring_rows > kRowMask || static_cast<uint64_t>(p.chunk_len) > kRowMask)
    return cudaErrorNotSupported;
  if (!encode_rows(&tm_q, p.q, static_cast<uint64_t>(p.n_q) * p.n_heads, kH) ||
      !encode_rows(&tm_ring, p.ring_x, ring_rows, kNk) ||
      // FP8 entries are gathered as codes, never copied as bf16 rows
      !encode_rows(&tm_kv, p.kv_dtype == CSKV_FP8_E4M3 ? static_cast<const void*>(p.ring_x) : p.kv_pool,
                   p.kv_dtype == CSKV_FP8_E4M3 ? ring_rows : kv_rows, kNk) ||
      // one-row boxes of the pool for the gathered tiles (the selection's rows, every FP8 entry)
      !(p.kv_dtype == CSKV_FP8_E4M3 ? encode_codes(&tm_kvg, p.kv_pool, kv_rows)
                                    : encode_rows(&tm_kvg, p.kv_pool, kv_rows, 1)))
    return cudaErrorNotSupported;
  const bool fp8 = p.kv_dtype == CSKV_FP8_E4M3, rule = has_score_rule(p);
  const size_t smem = smem_bytes(fp8, rule, p.n_q);
  auto kern = rule ? (fp8 ? attend_tc_kernel<true, true> : attend_tc_kernel<false, true>)
                   : (fp8 ? attend_tc_kernel<true, false> : attend_tc_kernel<false, false>);
  cudaError_t e = allow_smem(kern, smem, 32 * sizeof(int));  // s_wsum
  if (e != cudaSuccess) return e;
  const int64_t groups = p.n_heads / kH;
  const int64_t items = (int64_t)p.n_q * p.max_splits * groups;
  p.slots = static_cast<int>(n_sm / groups < (int64_t)p.n_q * p.max_splits ? n_sm / groups : (int64_t)p.n_q * p.max_splits);
  const int grid = static_cast<int>(items < n_sm ? items : n_sm);
  p.part_t = 1;
  e = launch_pdl(kern, dim3(static_cast<unsigned>(grid < 1 ? 1 : grid)), dim3(fp8 ? Block<true>::kThreads : Block<false>::kThreads), smem, st, tm_q, tm_ring,
                 tm_kv, tm_kvg, p, make_rule(p.sm_scale, p.score_cap));
  if (e != cudaSuccess) return e;
  return launch_attend_merge(p, st);
}

}  // namespace cskv
