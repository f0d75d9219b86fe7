// attend_chunk.cu -- HCA attention of a chunk of new tokens on the tensor cores
// (tcgen05), with a rule on the logits (cap, distance bias), for the narrow latent
// d_qk = d_v = 128 (DeepSeek-V4 report digest, section 3: one softmax over the last
// n_win raw tokens and every visible entry; DeepSeek-V4-book ch.1, section 4: every
// head reads the one shared latent row).
//
// Consecutive queries of a chunk see the same entries and windows that differ by a
// row each, and every head reads the same keys, so (query, head) rows of several
// queries share each key tile: a work item is 256 consecutive rows of q seen as
// [n_q n_heads, 128] (4 queries of 64 heads, 16 queries of 16), two M = 128 tiles
// that read every 128-key tile from shared memory once. Per tile and key tile
//     S = Q K^T (8 MMAs, M = N = 128),  P = 2^(s - m),  O += P V (8 MMAs)
// with P written as bf16 over S in tensor memory (the A operand of P V) and V read
// MN-major from the key tile. The two tiles alternate on the tensor cores: while
// one's softmax runs, the other's P V and next S do.
//   warps 0-15: softmax, two threads per row: warps 8 w + 4 h .. + 3 take keys
//     64 h .. + 63 of tile w. (One thread per row, with two softmax warps on a
//     scheduler, waited for its own instructions most of the time: 198 us where two
//     took 181.) With a running maximum the two agree on the row's reference at a
//     barrier, and it moves only when a logit exceeds it by more than 2^8; O is
//     rescaled then, half of its channels by each;
//   warp 16: issues the MMAs;
//   warps 17, 18: look up the keys' rows, four keys per lane, and have TMA copy the
//     two 64-channel halves of each tile: 16 consecutive rows per copy where a run
//     of 16 keys has them, else gathers of four rows. A copy costs its warp ~150
//     cycles whatever its size: 64 gathers by one warp took 10,000 cycles per tile,
//     and 96 threads copying by cp.async 5,700.
//
// Bound: the softmax's arithmetic, not the tensor cores. A pair of 128 x 128 tiles
// is 4 x 512 cycles of MMA and 32,768 logits. Where a logit of a tile reaches the cap
// each takes 15 fp32 operations (128 per clock and SM; packed pairs halve the issue
// slots, not the pipe time) and 1.5 special-function operations (16 per clock: its
// exponential and half a reciprocal, which two tanh share): 3840 cycles a pair of the
// first kind; below the cap 10 and 1, 2560 and 2048; without one 3 and 1, 770 and 2048.
// Measured: ~6,500 a pair, with 15 instructions a logit at half of the issue slots;
// 4096 queries of 64 heads on 61,440 cached tokens take 165 us.
//
//   warp 19: describes the items;
//   warps 20-23: write O / l, a row per thread and a 32-byte sector per store, while
//     the softmax warps are at the next item (as a part of their work it took a
//     third of an item's time).
// A row's segment is the run of consecutive queries of one sequence it stands in
// (positions at most kMaxStep apart, so that a segment's windows overlap), and an
// item is the 256 rows with one of their segments: the key
// list of a segment is its queries' window positions wlo .. thi, padded to a
// multiple of four, then the entries visible at thi, and each row's mask keeps its
// own window and entries. Rows of
// another segment are masked out.
//
// Masked keys are multiplied by P = 0, which a NaN or an infinity in a masked key's
// row would turn into NaN. A row whose sum or output is not finite is therefore taken
// again by its warp from its own keys only (slow_row), so that no key outside a
// query's own set can reach its answer.
#include "cskv_device.cuh"
#include "cskv_internal.h"
#include "score_rule.cuh"
#include "tc_issue.cuh"

namespace cskv {
namespace {

constexpr int kD = 128;                      // d_qk = d_v
constexpr int kTileRows = 128;               // rows of one M tile
constexpr int kItemRows = 2 * kTileRows;
constexpr int kNk = 128;                     // keys per tile
constexpr int kNS = 3;                       // key stages
constexpr int kHalfBytes = kNk * 128;        // 16384: one 64-channel half of 128 rows
constexpr int kStageBytes = 2 * kHalfBytes;  // 32768 (also one Q tile)
constexpr int kThreads = 768;
constexpr int kMmaWarp = 16, kLoadWarp0 = 17, kItemWarp = 19;  // 20 .. 23 write the outputs
constexpr int kTileThreads = 256;            // softmax threads of one tile
constexpr int kMaxStep = 32;                 // largest step between positions of one segment's queries
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // S of tile w at 128 w (P of each 64 keys over theirs), O at 256 + 128 w
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;    // log2 units

// source-row code: kind in bits [31:30] (0 none, 1 pool entry, 2 ring row, 3 chunk row), row below
constexpr uint32_t kRowBits = 30;
constexpr uint32_t kRowMask = (1u << kRowBits) - 1u;

__device__ __forceinline__ const uint16_t* code_row(const AttendParams& p, uint32_t c) {
  const uint32_t kind = c >> kRowBits, row = c & kRowMask;
  if (kind == 1) return static_cast<const uint16_t*>(p.kv_pool) + (size_t)row * kD;
  if (kind == 2) return p.ring_x + (size_t)row * kD;
  if (kind == 3) return p.x_chunk + (size_t)row * kD;
  return nullptr;
}
__device__ __forceinline__ uint32_t window_code(const AttendParams& p, int seq, int pos) {
  const int64_t cr = chunk_row(p, seq, pos);
  if (cr >= 0) return (3u << kRowBits) | static_cast<uint32_t>(cr);
  return (2u << kRowBits) | static_cast<uint32_t>((int64_t)seq * p.n_win + pos % p.n_win);
}
__device__ __forceinline__ uint32_t entry_code(const AttendParams& p, int seq, int j) {
  const int pi = j / p.page_size;
  if (pi >= p.max_pages_per_seq) return 0;
  const int32_t page = p.page_table[(int64_t)seq * p.max_pages_per_seq + pi];
  if (page < 0 || page >= p.n_pages) return 0;
  return (1u << kRowBits) | static_cast<uint32_t>((int64_t)page * p.page_size + j % p.page_size);
}
// visible_entries and window_start for positions below 2^31 and m = 2^lm
__device__ __forceinline__ int visible32(const AttendParams& p, int t, int lm) {
  const int lim = t + 1 - p.n_win;
  return lim <= 0 ? 0 : static_cast<int>((static_cast<unsigned>(lim) + (1u << lm) - 1u) >> lm);
}
__device__ __forceinline__ int start32(const AttendParams& p, int t) { return max(t - p.n_win + 1, 0); }

// An item as one warp describes it to the others: its queries (at most 17: 16 heads or more, rows that need
// not begin with a query) and one segment of them. The rows of its other segments are other items: on their way through
// the grid the 256 rows come up once per segment they may have (pass), on another CTA each time, so that 16 single tokens
// with long contexts of their own, which share no key, are 16 CTAs' work (64 such tokens at 1M beside a chunk of 1024, 16
// heads: 250 us, one CTA for all segments of 256 rows 3,211, the other kernels 341). Rows without keys are part of the
// item of the first segment; 256 rows without any key are none (write_empty).
struct Segment {
  int s, e;         // queries s .. e - 1 of the item
  int n_w, ntiles;  // window places of the key list, key tiles
  int wlo, thi;     // its window positions
  int seq, n;       // sequence, keys of the list
};
struct ItemDesc {
  int row0;  // first row (-1: no more items)
  int h0;    // its head
  int ntot;  // key tiles (0 with the end)
  int pad[5];
  uint8_t own[32];  // a bit per row: the item writes it (its segment's rows, and in the first pass those without keys)
  int t[20];        // each query's position, -1 without keys
  Segment seg;
};
constexpr int kItems = 4;  // descriptors in flight
static_assert(sizeof(ItemDesc) % 16 == 0 && sizeof(Segment) == 32, "descriptor layout");

// as many passes over the items as 256 rows have queries at most
__host__ __device__ __forceinline__ int item_passes(int n_heads) {
  return kItemRows % n_heads == 0 ? kItemRows / n_heads : (kItemRows - 2 + n_heads) / n_heads + 1;
}

// The queries of the 256 rows from `row0` = head h0 of query q0 on, one per lane: its position (-1: without keys) and
// sequence; returns the lanes where a segment begins.
__device__ __forceinline__ unsigned find_segments(const AttendParams& p, int row0, int q0, int h0, int rows, int lane, int& t,
                                                  int& seq) {
  t = seq = -1;
  if (lane * p.n_heads < min(kItemRows, rows - row0) + h0) {
    const int64_t pos = p.q_pos[q0 + lane];
    seq = p.q_seq[q0 + lane];
    if (pos >= 0 && pos <= p.max_pos && seq >= 0 && seq < p.n_seqs_layer) t = static_cast<int>(pos);
  }
  const int tp = __shfl_up_sync(kFull, t, 1);
  const int sp = __shfl_up_sync(kFull, seq, 1);
  const bool cont = lane > 0 && tp >= 0 && sp == seq && abs(t - tp) <= kMaxStep;
  return __ballot_sync(kFull, t >= 0 && !cont);
}

// Rows of which none has a key, by one warp: zeros and -inf. They are no item: the MMA warp looks for the next item's
// descriptor before it has finished its own, so every published one has key tiles to work on.
__device__ __forceinline__ void write_empty(const AttendParams& p, int row0, int rows, int lane) {
  const int n = min(kItemRows, rows - row0);
  uint4* out = reinterpret_cast<uint4*>(p.out + (int64_t)row0 * kD);
  for (int i = lane; i < n * (kD / 8); i += 32) out[i] = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse)
    for (int i = lane; i < n; i += 32) p.lse[(int64_t)row0 + i] = -INFINITY;
}

// Describes segment `pass` of them.
__device__ __forceinline__ void describe(const AttendParams& p, ItemDesc& d, int row0, int h0, int rows, unsigned starts, int pass,
                                         int t, int seq, int lm, int lane) {
  const unsigned runs = __ballot_sync(kFull, t >= 0);
  if (lane < 20) d.t[lane] = t;
  unsigned m = starts;
  for (int i = 0; i < pass; ++i) m &= m - 1;
  Segment g;
  g.s = __ffs(m) - 1;
  const unsigned stop = (starts | ~runs) & ~((2u << g.s) - 1u);  // the first lane past s that begins another or none
  g.e = stop ? __ffs(stop) - 1 : 32;
  g.seq = __shfl_sync(kFull, seq, g.s);
  const int ts = __shfl_sync(kFull, t, g.s);
  const int mine = lane >= g.s && lane < g.e ? t : ts;
  g.thi = __reduce_max_sync(kFull, mine);
  g.wlo = start32(p, __reduce_min_sync(kFull, mine));
  g.n_w = (g.thi - g.wlo + 4) & ~3;
  g.n = g.n_w + visible32(p, g.thi, lm);
  g.ntiles = (g.n + kNk - 1) / kNk;
  uint32_t own = 0;  // of rows 8 lane .. + 7
  for (int i = 0, at = h0 + 8 * lane; i < 8; ++i, ++at) {
    const int qi = at / p.n_heads, tq = __shfl_sync(kFull, t, qi);
    own |= (row0 + 8 * lane + i < rows && ((qi >= g.s && qi < g.e) || (pass == 0 && tq < 0)) ? 1u : 0u) << i;
  }
  d.own[lane] = static_cast<uint8_t>(own);
  if (lane == 0) {
    d.row0 = row0;
    d.h0 = h0;
    d.ntot = g.ntiles;
    d.seg = g;
  }
}

struct Smem {
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * kStageBytes;
  static constexpr int POS = K + kNS * kStageBytes;   // [kNS][kNk] key positions relative to the segment's last query
  static constexpr int ROWS = POS + kNS * kNk * 4;    // [2][kNk] source-row codes (a tile copied by cp.async)
  static constexpr int MASK = ROWS + 2 * kNk * 4;         // [kNS][4] valid-key bits
  static constexpr int SIDE = MASK + kNS * 16;        // [2 tiles][2 halves][128 rows] maxima the halves exchange
  static constexpr int SUM = SIDE + 4 * kTileRows * 4;   // [2 tiles][2 halves][128 rows] an item's sums
  static constexpr int BASE = SUM + 4 * kTileRows * 4;  // [2 tiles][128 rows] what a row's sum stands on
  static constexpr int ITEM = BASE + 2 * kTileRows * 4;  // [kItems] item descriptors
  static constexpr int BAR = ITEM + kItems * sizeof(ItemDesc);
  static constexpr int TMEM = BAR + 36 * 8;
  static constexpr int FLAGS = TMEM + 8;
  static constexpr int END = FLAGS + 8;
  static constexpr size_t bytes() { return 1024 + END; }
};
static_assert(Smem::bytes() <= 232448, "shared memory budget");
static_assert(Smem::POS % 16 == 0 && Smem::ROWS % 16 == 0 && Smem::ITEM % 16 == 0 && Smem::BAR % 8 == 0, "alignment");

// bits of lo <= u < hi for the 32 keys u = a .. a + 31
__device__ __forceinline__ uint32_t range_bits(int a, int lo, int hi) {
  const int l = min(max(lo - a, 0), 32), h = min(max(hi - a, 0), 32);
  return h > l ? (0xffffffffu >> (32 - (h - l))) << l : 0u;
}

// 32 bytes per thread: a whole sector in one store where the rows are 32-byte aligned (163 us for 4096 queries on 61,440
// cached tokens; two take 165), else two: callers align their buffers to 16 bytes only
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&v)[8], bool sector) {
  if (sector) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(dst), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<uint4*>(dst + 8) = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// The three forms of the kernel. kBounded: a cap of at most kMaxStatic (in log2 units) bounds every logit of a row by
// ref + cap2, for a reference known beforehand, and the row's own token, or with a negative slope its
// farthest key, is at ref - cap2 at least, so 2^(s - ref) neither overflows fp32 nor vanishes, and the softmax needs no
// running maximum: no pass for it, no agreement between the halves of a row, no rescaling (181 us -> 176 us
// when it came). Where that farthest key's page is missing the others may vanish: a sum below kMinSum, which the key
// alone would exceed, has its row taken again (slow_row). Above it a term that 2^-126 flushes to zero is at most 2^-36 of it.
enum Mode { kPlainMax, kCappedMax, kBounded };
constexpr float kMaxStatic = 80.f, kMinSum = 0x1p-90f;

// One row from its own keys only, by one warp (lane = 4 channels): scores in fp32, an online softmax, fp32 P.
template <bool CAP>
__device__ __forceinline__ void slow_row(const AttendParams& p, int64_t row, float sl2, float cap2, float slope2, float (&o)[4],
                                      float& m, float& l, float& far, int lane) {
  const int b = static_cast<int>(row / p.n_heads);
  const int t = static_cast<int>(p.q_pos[b]), ws = start32(p, t);
  const int seq = p.q_seq[b];
  const int n_w = t - ws + 1, n = n_w + visible32(p, t, __ffs(p.m) - 1);
  far = slope2 < 0.f ? far_distance(t, ws, 0, p.m, p.n_win) : 0.f;  // m is relative to its bias
  const uint2 qv = *reinterpret_cast<const uint2*>(p.q + row * kD + 4 * lane);
  const __nv_bfloat162* q2 = reinterpret_cast<const __nv_bfloat162*>(&qv);
  const float2 qa = __bfloat1622float2(q2[0]), qb = __bfloat1622float2(q2[1]);
  o[0] = o[1] = o[2] = o[3] = 0.f;
  m = -INFINITY;
  l = 0.f;
  for (int u = 0; u < n; ++u) {
    const uint32_t c = u < n_w ? window_code(p, seq, ws + u) : entry_code(p, seq, u - n_w);
    const uint16_t* src = code_row(p, c);
    if (!src) continue;
    const uint2 kv = *reinterpret_cast<const uint2*>(src + 4 * lane);
    const __nv_bfloat162* k2 = reinterpret_cast<const __nv_bfloat162*>(&kv);
    const float2 ka = __bfloat1622float2(k2[0]), kb = __bfloat1622float2(k2[1]);
    float s = qa.x * ka.x + qa.y * ka.y + qb.x * kb.x + qb.y * kb.y;
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(kFull, s, w);
    const float dist = u < n_w ? static_cast<float>(t - ws - u) : entry_distance(t, u - n_w, p.m);
    s = ruled_score<CAP>(s, sl2, cap2, slope2, dist - far);
    const float mn = fmaxf(m, s), corr = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float e = s == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * corr + e;
    o[0] = o[0] * corr + e * ka.x;
    o[1] = o[1] * corr + e * ka.y;
    o[2] = o[2] * corr + e * kb.x;
    o[3] = o[3] * corr + e * kb.y;
    m = mn;
  }
}

// Pipeline (key tiles numbered g over the CTA's items; stage g % kNS, kNS = 3):
//   loader  : look up rows -> wait kempty (P V of tile g - 3) -> TMA copies -> kfull
//   MMA     : S0(0) S1(0), then per key tile (kBounded: per part of it): wait pfull0 -> P V 0(g), S0(g + 1) -> sfull0 (or odone0);
//             wait pfull1 -> P V 1(g) -> kempty, S1(g + 1) -> sfull1 (or odone1); the last S1 of an item -> qempty
//   softmax : wait sfull (S here, and every earlier P V of this tile done: O may be rescaled) -> P -> pfull;
//             after the item's last tile: its rows' sums -> lready
//   outputs : wait lready, odone -> read O -> oread, which the next item's first P V waits for
template <int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_pool,
                        const __grid_constant__ CUtensorMap tm_ring, const __grid_constant__ CUtensorMap tm_chunk,
                        const __grid_constant__ CUtensorMap tm_pool16, const __grid_constant__ CUtensorMap tm_ring16,
                        const __grid_constant__ CUtensorMap tm_chunk16,
                        const __grid_constant__ AttendParams p, const __grid_constant__ Rule r) {
  constexpr bool CAP = MODE != kPlainMax;
  // Parts of a key tile that go through S, softmax and P V one after another. Without a running maximum a part of 64 keys
  // waits for nothing of the other: while the softmax is at one, P V and the next S of the other run, and its warps go
  // from part to part (a whole tile's warps waited 2,400 of 6,500 cycles for it: 164.7 us, in parts 161.3; the rest is issue: 49% of the
  // slots and 15 instructions a logit).
  constexpr int kParts = MODE == kBounded ? 2 : 1, kPartKeys = kNk / kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm + Smem::Q;
  uint8_t* sK = sm + Smem::K;
  float* sPos = reinterpret_cast<float*>(sm + Smem::POS);
  uint32_t* sRow = reinterpret_cast<uint32_t*>(sm + Smem::ROWS);
  uint32_t* sMask = reinterpret_cast<uint32_t*>(sm + Smem::MASK);
  float* sSide = reinterpret_cast<float*>(sm + Smem::SIDE);
  float* sSum = reinterpret_cast<float*>(sm + Smem::SUM);
  float* sBase = reinterpret_cast<float*>(sm + Smem::BASE);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + Smem::BAR);  // [3] loaders (2) -> MMA, softmax
  uint64_t* kempty = kfull + kNS;                                 // [3] MMA -> loaders
  uint64_t* sfull = kempty + kNS;                                 // [2 tiles][kParts] MMA -> softmax
  uint64_t* pfull = sfull + 4;                                    // [2 tiles][kParts] softmax (8 warps) -> MMA
  uint64_t* odone = pfull + 4;                                    // [2] MMA -> output warps
  uint64_t* oread = odone + 2;                                    // [2] output warps (4) -> MMA
  uint64_t* qfull = oread + 2;                                    // [2] Q of the tile landed (TMA)
  uint64_t* qempty = qfull + 2;                                   // [2] the item's S products of the tile are done
  uint64_t* lready = qempty + 2;                                  // [2] softmax (8 warps): an item's sums -> output warps
  uint64_t* lfree = lready + 2;                                   // [2] output warps (4) have read them
  uint64_t* ifull = lfree + 2;                                   // [kItems] descriptor written -> everyone
  uint64_t* ifree = ifull + kItems;                               // [kItems] everyone (23 warps) -> item warp
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + Smem::TMEM);
  volatile int* sAbort = reinterpret_cast<int*>(sm + Smem::FLAGS);

  // a shuffle from a constant lane is what the compiler takes as the same value in every lane
  const int tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&kfull[i], 2);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ifull[i], 1);
      mbar_init(&ifree[i], 23);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&odone[i], 1);
      mbar_init(&oread[i], 4);
      mbar_init(&lready[i], 8);
      mbar_init(&lfree[i], 4);
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], 1);
    }
    fence_barrier_init();
    *sAbort = 0;
  }
  if (tid == 32 * kLoadWarp0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_pool16);
    prefetch_tensormap(&tm_chunk16);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(kFull, *sTmem, 0);
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x == 0)
    for (int b = tid; b < p.n_q; b += kThreads) {
      const int64_t t = p.q_pos[b];
      if (t < 0 || t > p.max_pos)
        report(p.status, CSKV_ERR_INVALID_ARG);
      else if (p.q_seq[b] < 0 || p.q_seq[b] >= p.n_seqs_layer)
        report(p.status, CSKV_ERR_OUT_OF_RANGE);
    }
  const int rows = p.n_q * p.n_heads;
  const int lm = __ffs(p.m) - 1;  // m is a power of two
  ItemDesc* items = reinterpret_cast<ItemDesc*>(sm + Smem::ITEM);
  uint32_t n_item = 0;  // items before the current one
  // the current item's descriptor, and giving it back (whole warps)
  auto item_wait = [&](uint32_t n) {
    return __all_sync(kFull, mbar_wait(&ifull[n % kItems], (n / kItems) & 1u, p.status));
  };
  auto item_done = [&](uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ifree[n % kItems]);
  };
  uint32_t g = 0;      // key tiles before the current item

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;\n");
    if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issue (lane 0; the warp waits together)
      const uint32_t issuer = elect_one();
      constexpr uint32_t idesc_s = umma_idesc_bf16(kTileRows, kPartKeys, false);
      constexpr uint32_t idesc_pv = umma_idesc_bf16(kTileRows, kD, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait(bar, parity, p.status)); };
      auto s_of = [&](int w, int h, int st) {  // S of part h of tile w from stage st: 8 K-steps over the two channel halves
        const uint32_t q = sQa + w * kStageBytes, k = sKa + st * kStageBytes + h * (kPartKeys * 128);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32u;
          umma_ss_if(issuer, tmem + kColS + w * kNk + h * kPartKeys, umma_desc_sw128(q + off, 16, 1024),
                     umma_desc_sw128(k + off, 16, 1024), idesc_s, ks > 0 ? 1u : 0u);
        }
      };
      // O += P V of a part: K-steps of 16 keys. P of a thread's kPartKeys / 2 keys lies over the first half of their S.
      auto pv_of = [&](int w, int h, int st, uint32_t acc) {
        const uint32_t v = sKa + st * kStageBytes + h * (kPartKeys * 128);
        constexpr int kSteps = kPartKeys / 16;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
          umma_ts_if(issuer, tmem + kColO + w * kD,
                     tmem + kColS + w * kNk + h * kPartKeys + (ks / (kSteps / 2)) * (kPartKeys / 2) + (ks % (kSteps / 2)) * 8,
                     umma_desc_sw128(v + ks * 16 * 128, kHalfBytes, 1024), idesc_pv, ks > 0 ? 1u : acc);
      };
      // the stage as a constant in each branch, so that the descriptors are
      auto issue_s = [&](int w, int h, uint32_t gt) {
        const uint32_t st = gt % kNS;
        if (st == 0) s_of(w, h, 0);
        else if (st == 1) s_of(w, h, 1);
        else s_of(w, h, 2);
        commit_if(issuer, &sfull[w * kParts + h]);
      };
      auto issue_pv = [&](int w, int h, uint32_t gt, bool acc) {
        const uint32_t st = gt % kNS;
        if (st == 0) pv_of(w, h, 0, acc);
        else if (st == 1) pv_of(w, h, 1, acc);
        else pv_of(w, h, 2, acc);
      };
      static_assert(kNS == 3, "the stage branches");
      // The items, found one ahead: S of the next item's first key tile is issued behind P V of this item's last one, so
      // the softmax of a tile goes from item to item without a pause. (The wait for the next descriptor does not depend
      // on this item: its slot came free with the item kItems before it.)
      bool ok = true;
      uint32_t n_act = 0;  // items done (n_item: items found)
      auto next_tiles = [&]() {  // key tiles of the next item, 0 at the end (one exit: another spills)
        ok = item_wait(n_item);
        const int n = __shfl_sync(kFull, items[n_item % kItems].ntot, 0);
        item_done(n_item++);
        return ok ? n : 0;
      };
      int ntot = next_tiles();
      if (ntot && ok) {
#pragma unroll
        for (int i = 0; i < 2 * kParts; ++i) {
          const int h = i >> 1, w = i & 1;
          ok = ok && wait(&qfull[w], 0) && wait(&kfull[0], 0);
          if (!ok) break;
          tc_fence_after();
          issue_s(w, h, 0);
          if (ntot == 1 && h == kParts - 1) commit_if(issuer, &qempty[w]);
        }
      }
      while (ntot && ok) {
        const int nnext = next_tiles();
        if (!ok) break;
        for (int it = 0; it < ntot && ok; ++it) {
          if (__shfl_sync(kFull, *sAbort, 0)) {
            ok = false;
            break;
          }
          const uint32_t gt = g + it, gn = gt + 1;
          const bool last = it + 1 == ntot, more = !last || nnext > 0;
          const bool qlast = last ? nnext == 1 : it + 2 == ntot;  // the next S is the last one of its item
#pragma unroll
          for (int i = 0; i < 2 * kParts; ++i) {
            const int h = i >> 1, w = i & 1;
            ok = wait(&pfull[w * kParts + h], gt & 1u) &&
                 (h > 0 || it > 0 || n_act == 0 || wait(&oread[w], (n_act - 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            issue_pv(w, h, gt, h > 0 || it > 0);
            if (i == 2 * kParts - 1) commit_if(issuer, &kempty[gt % kNS]);
            if (last && h == kParts - 1) commit_if(issuer, &odone[w]);
            if (more) {
              ok = (!last || wait(&qfull[w], (n_act + 1) & 1u)) && wait(&kfull[gn % kNS], (gn / kNS) & 1u);
              if (!ok) break;
              tc_fence_after();
              issue_s(w, h, gn);
              if (qlast && h == kParts - 1) commit_if(issuer, &qempty[w]);
            }
            __syncwarp();
          }
        }
        if (!ok) break;
        g += ntot;
        ++n_act;
        ntot = nnext;
      }
      if (!ok) {
        *sAbort = 1;
        // what was issued gets a bounded chance to land before the tensor memory is freed
        commit_if(issuer, &odone[0]);
        __syncwarp();
        mbar_wait(&odone[0], n_act & 1u, nullptr);
      }
    } else if (warp < kLoadWarp0 + 2) {
      // ---------------------------------------------------------------- loaders (a warp per channel half and Q tile)
      const int half = warp - kLoadWarp0;
      bool ok = true;
      uint32_t issued = 0, q_issued = 0;  // key tiles and Q loads given to TMA
      for (; ok; ++n_item) {
        if (!(ok = item_wait(n_item))) break;
        const ItemDesc& d = items[n_item % kItems];
        const int row0 = d.row0, ntot = d.ntot;
        if (row0 < 0) break;
        ok = __all_sync(kFull, n_item == 0 || mbar_wait(&qempty[half], (n_item - 1) & 1u, p.status));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&qfull[half], kStageBytes);
          for (int h = 0; h < 2; ++h)
            tma_load_2d(sQ + half * kStageBytes + h * kHalfBytes, &tm_q, h * 64, row0 + half * kTileRows,
                        &qfull[half]);
        }
        __syncwarp();
        ++q_issued;
        uint32_t gt = g;
        {
          const Segment sg = d.seg;
          for (int it = 0; it < sg.ntiles; ++it, ++gt) {
            const int st = gt % kNS;
            // keys u .. u + 3 of the list: all window places, or all entries (of one page)
            const int u = it * kNk + 4 * lane;
            uint32_t code[4] = {0u, 0u, 0u, 0u};
            float pos[4];
            if (u < sg.n_w) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int at = sg.wlo + u + e;
                if (at <= sg.thi) code[e] = window_code(p, sg.seq, at);
                pos[e] = static_cast<float>(at - sg.thi);
              }
            } else {
              const int j = u - sg.n_w, left = sg.n - u;
              const uint32_t c = left > 0 ? entry_code(p, sg.seq, j) : 0u;
              if (half == 0 && left > 0 && !c) report(p.status, CSKV_ERR_OUT_OF_RANGE);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (c && e < left) code[e] = c + e;
                pos[e] = -entry_distance(sg.thi, j + e, p.m);
              }
            }
            // one source per group, so that TMA can gather it (a group that straddles the ring and the chunk cannot)
            const uint32_t kind = max(max(code[0], code[1]), max(code[2], code[3])) >> kRowBits;
            bool one = true;
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              one = one && (code[e] == 0u || (code[e] >> kRowBits) == kind);
              bits |= (code[e] ? 1u : 0u) << (4 * (lane & 7) + e);
            }
            const bool gather = __all_sync(kFull, one);
            // runs of 16 keys (4 lanes) in 16 consecutive rows of one source
            const uint32_t c0 = __shfl_sync(kFull, code[0], lane & ~3);
            bool run = code[0] != 0u && code[0] == c0 + 4 * (lane & 3);
#pragma unroll
            for (int e = 1; e < 4; ++e) run = run && code[e] == code[0] + e;
            run = ((__ballot_sync(kFull, run) >> (lane & ~3)) & 15u) == 15u;
            bits |= __shfl_xor_sync(kFull, bits, 1);
            bits |= __shfl_xor_sync(kFull, bits, 2);
            bits |= __shfl_xor_sync(kFull, bits, 4);
            ok = __all_sync(kFull, gt < kNS || mbar_wait(&kempty[st], ((gt / kNS) - 1) & 1u, p.status)) &&
                 !__any_sync(kFull, *sAbort != 0);
            if (!ok) break;
            if (half == 0) {
              reinterpret_cast<float4*>(sPos + st * kNk)[lane] = make_float4(pos[0], pos[1], pos[2], pos[3]);
              if ((lane & 7) == 0) sMask[st * 4 + (lane >> 3)] = bits;
            }
            uint8_t* dst = sK + st * kStageBytes + half * kHalfBytes;
            __syncwarp();
            if (gather) {
              if (lane == 0) mbar_arrive_expect_tx(&kfull[st], kHalfBytes);
              __syncwarp();
              if (run) {
                const CUtensorMap* map = kind == 3u ? &tm_chunk16 : kind == 2u ? &tm_ring16 : &tm_pool16;
                if ((lane & 3) == 0)
                  tma_load_2d(dst + lane * 512, map, half * 64, static_cast<int>(code[0] & kRowMask), &kfull[st]);
              } else {
                const CUtensorMap* map = kind == 3u ? &tm_chunk : kind == 2u ? &tm_ring : &tm_pool;
                int y[4];  // a key without a row reads row -1, outside the map: zeros
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = code[e] ? static_cast<int>(code[e] & kRowMask) : -1;
                tma_gather4(dst + lane * 512, map, half * 64, y[0], y[1], y[2], y[3], &kfull[st]);
              }
              __syncwarp();
            } else {
              reinterpret_cast<uint4*>(sRow + half * kNk)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
              __syncwarp();
#pragma unroll 4
              for (int id = lane; id < kNk * 8; id += 32) {  // 8 consecutive lanes copy half a row
                const int key = id >> 3, c = id & 7;
                const uint16_t* src = code_row(p, sRow[half * kNk + key]);
                cp_async16(dst + key * 128 + ((c ^ (key & 7)) << 4),
                           src ? static_cast<const void*>(src + half * 64 + c * 8) : static_cast<const void*>(p.q),
                           src ? 16 : 0);
              }
              cp_async_commit();
              cp_async_wait<0>();
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&kfull[st]);
            }
            issued = gt + 1;
          }
        }
        item_done(n_item);
        g += ntot;
      }
      if (!ok) {  // the copies in flight get a bounded chance to land before the block leaves
        *sAbort = 1;
        for (uint32_t i = issued > kNS ? issued - kNS : 0; i < issued; ++i)
          mbar_wait(&kfull[i % kNS], (i / kNS) & 1u, nullptr);
        if (q_issued > 0) mbar_wait(&qfull[half], (q_issued - 1) & 1u, nullptr);
      }
    }
    else if (warp == kItemWarp) {
      // ---------------------------------------------------------------- items
      // Several sequences: each pass begins at another CTA. One sequence: its queries mostly follow each other, and the
      // CTA of the rows takes all their segments (the look at every item in each pass took 9 of 177 us).
      const int passes = p.chunk_desc ? item_passes(p.n_heads) : 1;
      const int shift = max(static_cast<int>(gridDim.x) / passes, 1), n_items = (rows + kItemRows - 1) / kItemRows;
      bool ok = true;
      auto slot = [&]() {  // the next descriptor, once everyone has given it back
        ok = __all_sync(kFull, n_item < kItems || mbar_wait(&ifree[n_item % kItems], ((n_item / kItems) - 1) & 1u, p.status));
        return ok;
      };
      auto publish = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ifull[n_item % kItems]);
        ++n_item;
      };
      for (int pass = 0; pass < passes && ok; ++pass) {
        for (int idx = (blockIdx.x + pass * shift) % gridDim.x; idx < n_items; idx += gridDim.x) {
          const int row0 = idx * kItemRows, q0 = row0 / p.n_heads, h0 = row0 % p.n_heads;
          int t, seq;
          const unsigned starts = find_segments(p, row0, q0, h0, rows, lane, t, seq);
          if (starts == 0 && pass == 0) write_empty(p, row0, rows, lane);
          const int n_seg = __popc(starts), stop = passes > 1 ? min(pass + 1, n_seg) : n_seg;
          for (int i = pass; i < stop && slot(); ++i) {
            describe(p, items[n_item % kItems], row0, h0, rows, starts, i, t, seq, lm, lane);
            publish();
          }
          if (!ok) break;
        }
      }
      if (ok && slot()) {
        if (lane == 0) {
          items[n_item % kItems].row0 = -1;
          items[n_item % kItems].ntot = 0;
        }
        publish();
      }
      if (!ok) *sAbort = 1;
    } else {
      // ---------------------------------------------------------------- outputs: O / l in bf16, and the log-sum-exp
      const int tr = (warp & 3) * 32 + lane;  // row of the tile
      const uint32_t otile = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + kColO;
      const bool sector = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;  // every row's offset is a multiple of 256
      bool ok = true;
      for (; ok; ++n_item) {
        if (!(ok = item_wait(n_item))) break;
        const ItemDesc& d = items[n_item % kItems];
        if (d.row0 < 0) break;
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
          const int row = d.row0 + w * kTileRows + tr;
          const bool in = (d.own[(w * kTileRows + tr) >> 3] >> (tr & 7)) & 1u;
          ok = __all_sync(kFull, mbar_wait(&lready[w], n_item & 1u, p.status));
          if (!ok) break;
          const float l = sSum[2 * w * kTileRows + tr] + sSum[(2 * w + 1) * kTileRows + tr];
          const float base = sBase[w * kTileRows + tr];
          __syncwarp();
          if (lane == 0) mbar_arrive(&lfree[w]);
          if (!(ok = __all_sync(kFull, mbar_wait(&odone[w], n_item & 1u, p.status)))) break;
          tc_fence_after();
          const bool has = in && l > 0.f;
          const float inv = has ? 1.f / l : 0.f;
          float odd = 0.f;  // NaN once an output is not finite
#pragma unroll 1
          for (int c = 0; c < kD; c += 16) {
            uint32_t o[16], v[8];
            tmem_ld16(otile + w * kD + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              o[e] = has ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
              odd = fmaf(__uint_as_float(o[e]), 0.f, odd);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            if (in) store32(p.out + (int64_t)row * kD + c, v, sector);
          }
          // the next item's first P V overwrites O: this warp's reads of it are complete
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&oread[w]);
          float lse = has ? (base + log2f(l)) * kLn2 : -INFINITY;
          bool again = in && (!(l <= FLT_MAX) || !(odd == 0.f));
          if (MODE == kBounded && in && l < kMinSum) again = d.t[(d.h0 + w * kTileRows + tr) / p.n_heads] >= 0;
          const unsigned redo = __ballot_sync(kFull, again);
          if (redo) __syncwarp();
          for (unsigned left = redo; left; left &= left - 1) {
            const int b = __ffs(left) - 1;  // one row at a time, by the whole warp, over what its thread stored
            const int rr = __shfl_sync(kFull, row, b);
            const float slope2 = p.slopes ? p.slopes[rr % p.n_heads] * kLog2e : 0.f;
            float o4[4], m, lr, far;
            slow_row<CAP>(p, rr, r.pre.x, r.cap2.x, slope2, o4, m, lr, far, lane);
            const float iv = 1.f / lr;
#pragma unroll
            for (int e = 0; e < 4; ++e) o4[e] *= iv;
            *reinterpret_cast<uint2*>(p.out + (int64_t)rr * kD + 4 * lane) =
                make_uint2(pack_bf16(o4[0], o4[1]), pack_bf16(o4[2], o4[3]));
            if (lane == b) lse = (m + log2f(lr)) * kLn2 - slope2 * far * kLn2;
          }
          if (in && p.lse) p.lse[row] = lse;
        }
        if (!ok) break;
        item_done(n_item);
      }
      if (!ok) *sAbort = 1;
    }
  } else {
    // ------------------------------------------------------------------ softmax (half a row per thread)
    // Every softmax warp of a tile reaches the tile's barriers; a bounded wait that gave up only marks the tile bad,
    // and a barrier's OR decides for all of them.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 96;\n");
    const int w = warp >> 3, hf = (warp >> 2) & 1, tr = (warp & 3) * 32 + lane;  // tile, key half, row of the tile
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    // S of my keys (their P goes over its first 32 columns)
    const uint32_t sb = trow + kColS + w * kNk + 64 * hf;  // (kBounded: by parts)
    const uint32_t ob = trow + kColO + w * kD + 64 * hf;  // O of my channels (rescaling)
    float* side = sSide + (2 * w + hf) * kTileRows + tr;
    float* other = sSide + (2 * w + (hf ^ 1)) * kTileRows + tr;
    const float inv_heads = 1.f / static_cast<float>(p.n_heads);
    bool ok = true;
    for (; ok; ++n_item) {
      if (MODE == kBounded)
        ok = item_wait(n_item);
      else  // a barrier's OR, so that the warps of a tile leave together
        ok = !named_sync_or(1 + w, kTileThreads, !item_wait(n_item));
      if (!ok) break;
      const ItemDesc& d = items[n_item % kItems];
      const int row = d.row0 + w * kTileRows + tr;
      if (d.row0 < 0) break;
      const bool in = row < rows;
      // this row's query within the item and its head: small whole numbers, so the rounded quotient is exact
      const int at = d.h0 + w * kTileRows + tr;
      const int qi = static_cast<int>((static_cast<float>(at) + 0.5f) * inv_heads);
      const float slope2 = p.slopes && in ? p.slopes[at - qi * p.n_heads] * kLog2e : 0.f;
      const int t = in ? d.t[qi] : -1;
      float l_run = 0.f;
      bool fresh = true;  // before the row's first key
      int shift = 0;  // the row's logits are taken at distance 0 of its segment's last query
      int it = 0;
      bool fail = false;  // kBounded: a wait gave up (the item's barrier tells the others)
      float2 l_a = make_float2(0.f, 0.f), l_b = l_a;
      // What the row's distances are relative to: 0 where near keys lead, the farthest key's where far ones do.
      const float far = slope2 < 0.f && t >= 0 ? far_distance(t, start32(p, t), 0, p.m, p.n_win) : 0.f;
      const float ref = -slope2 * far;  // kBounded: the reference
      float negref = 0.f;  // otherwise what is added to the row's logits: their reference so far, with the other sign
      {
        const Segment& sg = d.seg;
        // this row's keys in the segment's list: window lo .. hi - 1, entries n_w .. end - 1
        const int n_w = sg.n_w, ntiles = sg.ntiles;
        int lo = 0, hi = 0, end = 0;
        if (t >= 0 && qi >= sg.s && qi < sg.e) {
          lo = start32(p, t) - sg.wlo;
          hi = t - sg.wlo + 1;
          end = n_w + visible32(p, t, lm);
          shift = t - sg.thi;
          if (MODE != kBounded && slope2 < 0.f) negref = slope2 * (far - static_cast<float>(shift));
        }
        for (int k = 0; k < ntiles; ++k, ++it) {
          const uint32_t gt = g + it;
          const int st = gt % kNS;
          // the stage's positions and key bits were written before kfull; that phase cannot move on before this
          // thread's P has been used
          bool good = __all_sync(kFull, mbar_wait(&sfull[w * kParts], gt & 1u, p.status)) &&
                      __all_sync(kFull, mbar_wait(&kfull[st], (gt / kNS) & 1u, p.status));
          tc_fence_after();
          if constexpr (MODE == kBounded) {
            const float nr = -slope2 * static_cast<float>(shift) - ref;
#pragma unroll 1
            for (int h = 0; h < kParts; ++h) {
              if (h > 0) good = __all_sync(kFull, mbar_wait(&sfull[w * kParts + h], gt & 1u, p.status));
              if (!good) {
                fail = true;
                break;
              }
              tc_fence_after();
              const int at = 64 * h + 32 * hf;  // this thread's keys of the part
              uint32_t s[32];
              tmem_ld32(trow + kColS + w * kNk + at, s);
              tmem_ld_wait();
              apply_rule<true>(s, reinterpret_cast<const float4*>(sPos + st * kNk + at), r, slope2, nr);
              const int a = k * kNk + at;
              const uint32_t vm = sMask[st * 4 + 2 * h + hf] & (range_bits(a, lo, hi) | range_bits(a, n_w, end));
              if (__any_sync(kFull, vm != kFull)) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((vm >> j) & 1u)) s[j] = 0xff800000u;  // -inf
              }
              uint32_t pp[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 e = make_float2(ex2(__uint_as_float(s[2 * j])), ex2(__uint_as_float(s[2 * j + 1])));
                if (j & 1) l_b = __fadd2_rn(l_b, e);
                else l_a = __fadd2_rn(l_a, e);
                pp[j] = pack_bf16(e.x, e.y);
              }
              tmem_st16(trow + kColS + w * kNk + at, pp);
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&pfull[w * kParts + h]);
            }
            if (fail) break;
            continue;
          }
          uint32_t s[64];
          tmem_ld32(sb, *reinterpret_cast<uint32_t(*)[32]>(s));
          tmem_ld32(sb + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
          tmem_ld_wait();
          apply_rule<CAP>(s, reinterpret_cast<const float4*>(sPos + st * kNk + 64 * hf), r, slope2, negref);
          float mt = -INFINITY;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int a = k * kNk + 64 * hf + 32 * c;
            const uint32_t vm = sMask[st * 4 + 2 * hf + c] & (range_bits(a, lo, hi) | range_bits(a, n_w, end));
            if (__any_sync(kFull, vm != kFull)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((vm >> j) & 1u)) s[32 * c + j] = 0xff800000u;  // -inf
            }
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              m0 = max3(m0, __uint_as_float(s[32 * c + j]), __uint_as_float(s[32 * c + j + 1]));
              m1 = max3(m1, __uint_as_float(s[32 * c + j + 2]), __uint_as_float(s[32 * c + j + 3]));
            }
            mt = max3(mt, m0, m1);
          }
          // The logits stand on the old maximum (the farthest key's bias, or 0, before the row's first key).
          const bool bad = !good || *sAbort != 0;
          if (named_sync_or(1 + w, kTileThreads, bad || mt > kRescaleThreshold || (fresh && mt != -INFINITY))) {
            *side = mt;
            if (named_sync_or(1 + w, kTileThreads, bad)) {
              ok = false;
              break;
            }
            mt = fmaxf(mt, *other);
            const bool up = mt > kRescaleThreshold || (fresh && mt != -INFINITY);
            // the step that negref takes, which may be a coarse one, not mt itself: every logit gets the same
            const float delta = up ? negref - (negref - mt) : 0.f;
            const float corr = up ? (fresh ? 0.f : ex2(-delta)) : 1.f;
            l_run *= corr;
            if (up) {
              negref -= mt;
              fresh = false;
            }
#pragma unroll
            for (int j = 0; j < 64; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) - delta);
            if (it > 0) {
#pragma unroll 1
              for (int c = 0; c < 64; c += 16) {
                uint32_t o[16];
                tmem_ld16(ob + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
                tmem_st16(ob + c, o);
              }
            }
          }
          float2 la = make_float2(0.f, 0.f), lb = la;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pp[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float e0 = ex2(__uint_as_float(s[32 * c + 2 * j])), e1 = ex2(__uint_as_float(s[32 * c + 2 * j + 1]));
              if (j & 1) lb = __fadd2_rn(lb, make_float2(e0, e1));
              else la = __fadd2_rn(la, make_float2(e0, e1));
              pp[j] = pack_bf16(e0, e1);
            }
            tmem_st16(sb + 16 * c, pp);
          }
          la = __fadd2_rn(la, lb);
          l_run += la.x + la.y;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[w]);
        }
      }
      if (!ok) break;
      // the row's sum and what it stands on, once the output warps have read the last item's
      if constexpr (MODE == kBounded) {
        l_a = __fadd2_rn(l_a, l_b);
        l_run = l_a.x + l_a.y;
      }
      ok = !fail && __all_sync(kFull, n_item == 0 || mbar_wait(&lfree[w], (n_item - 1) & 1u, p.status));
      if (MODE != kBounded) ok = !named_sync_or(1 + w, kTileThreads, !ok);
      if (!ok) break;
      sSum[(2 * w + hf) * kTileRows + tr] = l_run;
      if (hf == 0) sBase[w * kTileRows + tr] = MODE == kBounded ? ref : -negref - slope2 * static_cast<float>(shift);
      __syncwarp();
      if (lane == 0) mbar_arrive(&lready[w]);
      item_done(n_item);
      g += it;
    }
    if (!ok) *sAbort = 1;
  }
  cp_async_wait<0>();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
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

// The plain form (no rule) keeps the kernels it has always run on, and so its results. Inverse RoPE stays with the
// query-pair and split kernels: its fp64 sine and cosine do not fit the output warps' registers.
//
// Fewer than 32 rows per SM are better off with their keys split over the SMs, which this kernel does not do: it takes
// 19 us for 2000 cached tokens, 29 us for 60,000 and 230 us for 1M whatever the rows up to 256 per SM, where the others
// take 12, 17 and 67 us at 8 rows per SM (64 heads), 19, 30 and 237 us at 32, and 26, 49 and 466 us at 64. (With 16 heads
// they fall behind at 16 rows per SM already: 19, 31 and 267 us.)
bool attend_chunk_supported(const AttendParams& p, int n_sm) {
  const uint64_t pool_rows = static_cast<uint64_t>(p.n_pages) * p.page_size;
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  return !p.is_csa && has_score_rule(p) && p.x_chunk && p.rope_dims == 0 && p.d_qk == kD && p.d_v == kD && p.n_heads >= 16 &&
         p.kv_dtype == CSKV_BF16 && rows >= (int64_t)32 * n_sm && rows <= 0x7fffffff - (int64_t)kItemRows * (n_sm + 1) &&
         p.max_pos < (1 << 30) && p.n_win < (1 << 30) && p.chunk_len > 0 &&
         pool_rows <= kRowMask && ring_rows <= kRowMask && static_cast<uint64_t>(p.chunk_len) <= kRowMask;
}

cudaError_t launch_attend_chunk(AttendParams& p, int n_sm, cudaStream_t st) {
  CUtensorMap tm_q, tm_pool, tm_ring, tm_chunk, tm_pool16, tm_ring16, tm_chunk16;
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  const uint64_t pool_rows = static_cast<uint64_t>(p.n_pages) * p.page_size;
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  const uint64_t chunk_rows = static_cast<uint64_t>(p.chunk_len);
  if (!encode_rows(&tm_q, p.q, rows, kTileRows) ||
      !encode_rows(&tm_pool, p.kv_pool, pool_rows, 1) || !encode_rows(&tm_pool16, p.kv_pool, pool_rows, 16) ||
      !encode_rows(&tm_ring, p.ring_x, ring_rows, 1) || !encode_rows(&tm_ring16, p.ring_x, ring_rows, 16) ||
      !encode_rows(&tm_chunk, p.x_chunk, chunk_rows, 1) || !encode_rows(&tm_chunk16, p.x_chunk, chunk_rows, 16))
    return cudaErrorNotSupported;
  const size_t smem = Smem::bytes();
  auto kern = p.score_cap <= 0.f ? attend_chunk_kernel<kPlainMax>
              : p.score_cap * kLog2e <= kMaxStatic ? attend_chunk_kernel<kBounded> : attend_chunk_kernel<kCappedMax>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t items = (rows + kItemRows - 1) / kItemRows * (p.chunk_desc ? item_passes(p.n_heads) : 1);
  return launch_pdl(kern, dim3(static_cast<unsigned>(items < n_sm ? items : n_sm)), dim3(kThreads), smem, st, tm_q,
                    tm_pool, tm_ring, tm_chunk, tm_pool16, tm_ring16, tm_chunk16, p, make_rule(p.sm_scale, p.score_cap));
}

}  // namespace cskv
