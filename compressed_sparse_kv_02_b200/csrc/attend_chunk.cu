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
//   warps 0-3, 4-7: softmax of tile 0 / 1, one row per thread (all 128 logits of a
//     tile in registers: the rule is applied once, then the row max, then the
//     exponentials; O is rescaled only when the max rises by more than 2^8);
//   warp 8: issues the MMAs;  warps 9-11: look up the keys' rows and copy them
//     (cp.async) into four 128-byte-swizzled stages; Q by TMA.
//
// Bound: the softmax's arithmetic, not the tensor cores. A pair of 128 x 128 tiles
// is 4 x 512 cycles of MMA and 32,768 logits. With the cap a logit takes 1.5
// special-function operations (its exponential and half a reciprocal: two tanh share
// one) and about 12.5 issue slots (packed f32x2 arithmetic), 3072 and 3200 cycles a
// pair; without it 1 and 4.5, 2048 and 1150.
//
// A row's segment is the run of consecutive queries of one sequence it stands in
// (positions at most kMaxStep apart, so that a segment's windows overlap): the key
// list of a segment is its queries' window positions wlo .. thi, then the entries
// visible at thi, and each row's mask keeps its own window and entries. Rows that
// belong to another segment of the item are masked out of the whole segment.
//
// Masked keys are multiplied by P = 0, which a NaN or an infinity in a masked key's
// row would turn into NaN. A row whose output is not finite is therefore taken again
// by its warp from its own keys only (slow_row), so that no key outside a query's
// own set can reach its answer.
#include "cskv_device.cuh"
#include "cskv_internal.h"
#include "score_rule.cuh"

namespace cskv {
namespace {

constexpr int kD = 128;                      // d_qk = d_v
constexpr int kTileRows = 128;               // rows of one M tile
constexpr int kItemRows = 2 * kTileRows;
constexpr int kNk = 128;                     // keys per tile
constexpr int kNS = 4;                       // key stages
constexpr int kHalfBytes = kNk * 128;        // 16384: one 64-channel half of 128 rows
constexpr int kStageBytes = 2 * kHalfBytes;  // 32768 (also one Q tile)
constexpr int kThreads = 384;
constexpr int kLoadThread0 = 288;
constexpr int kLoaders = kThreads - kLoadThread0;  // 96
constexpr int kMaxStep = 32;                 // largest step between positions of one segment's queries
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // S of tile w at 128 w (P over its first 64 columns), O at 256 + 128 w
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;    // log2 units

struct Smem {
  static constexpr int Q = 0;
  static constexpr int K = Q + 2 * kStageBytes;
  static constexpr int POS = K + kNS * kStageBytes;   // [kNS][kNk] key positions relative to the segment's last query
  static constexpr int ROWS = POS + kNS * kNk * 4;    // [2][kNk] source-row codes
  static constexpr int MASK = ROWS + 2 * kNk * 4;     // [kNS][4] valid-key bits
  static constexpr int BAR = MASK + kNS * 16;
  static constexpr int TMEM = BAR + 24 * 8;
  static constexpr int FLAGS = TMEM + 8;
  static constexpr int END = FLAGS + 8;
  static constexpr size_t bytes() { return 1024 + END; }
};
static_assert(Smem::bytes() <= 232448, "shared memory budget");

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
__device__ __forceinline__ uint32_t window_code(const AttendParams& p, int seq, int64_t pos) {
  const int64_t cr = chunk_row(p, seq, pos);
  if (cr >= 0) return (3u << kRowBits) | static_cast<uint32_t>(cr);
  return (2u << kRowBits) | static_cast<uint32_t>((int64_t)seq * p.n_win + pos % p.n_win);
}
__device__ __forceinline__ uint32_t entry_code(const AttendParams& p, int seq, int64_t j) {
  const int64_t pi = j / p.page_size;
  if (pi >= p.max_pages_per_seq) return 0;
  const int32_t page = p.page_table[(int64_t)seq * p.max_pages_per_seq + pi];
  if (page < 0 || page >= p.n_pages) return 0;
  return (1u << kRowBits) | static_cast<uint32_t>((int64_t)page * p.page_size + j % p.page_size);
}

// The queries of an item (at most 17: 16 heads or more, rows that need not begin with a query), one per lane: position (-1: no keys) and sequence.
struct Queries {
  int q0, n;    // first query, queries the item touches
  int64_t t;    // this lane's
  int seq;
  unsigned starts;  // lanes where a segment begins
  unsigned runs;    // lanes that belong to one
};
__device__ __forceinline__ Queries load_queries(const AttendParams& p, int item, int lane) {
  Queries r;
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  const int64_t a = (int64_t)item * kItemRows, b = a + kItemRows < rows ? a + kItemRows : rows;
  r.q0 = static_cast<int>(a / p.n_heads);
  r.n = a < rows ? static_cast<int>((b - 1) / p.n_heads) - r.q0 + 1 : 0;
  r.t = -1;
  r.seq = -1;
  if (lane < r.n) {
    r.t = p.q_pos[r.q0 + lane];
    r.seq = p.q_seq[r.q0 + lane];
    if (r.t > p.max_pos || r.seq < 0 || r.seq >= p.n_seqs_layer) r.t = -1;
  }
  const bool ok = r.t >= 0;
  const int64_t tp = __shfl_up_sync(kFull, r.t, 1);
  const int sp = __shfl_up_sync(kFull, r.seq, 1);
  const int64_t step = r.t - tp;
  const bool cont = lane > 0 && tp >= 0 && sp == r.seq && step <= kMaxStep && step >= -kMaxStep;
  r.starts = __ballot_sync(kFull, ok && !cont);
  r.runs = __ballot_sync(kFull, ok);
  return r;
}

// One segment: lanes s .. e - 1, its key list (n_w window positions wlo .. thi, then nv entries).
struct Segment {
  int s, e, seq, n_w, n, ntiles;
  int64_t wlo, thi;
};
__device__ __forceinline__ Segment segment_at(const AttendParams& p, const Queries& q, int s, int lane) {
  Segment g;
  g.s = s;
  const unsigned after = ~((2u << s) - 1u);  // lanes past s
  const unsigned stop = (q.starts | ~q.runs) & after;
  g.e = stop ? __ffs(stop) - 1 : 32;
  g.seq = __shfl_sync(kFull, q.seq, s);
  const int64_t t0 = __shfl_sync(kFull, q.t, s);
  const int d = lane >= s && lane < g.e ? static_cast<int>(q.t - t0) : 0;  // a segment spans at most 16 kMaxStep
  const int64_t tlo = t0 + __reduce_min_sync(kFull, d);
  g.thi = t0 + __reduce_max_sync(kFull, d);
  g.wlo = window_start(tlo, p.n_win);
  g.n_w = static_cast<int>(g.thi - g.wlo + 1);
  g.n = g.n_w + static_cast<int>(visible_entries(g.thi, p.m, p.n_win));
  g.ntiles = (g.n + kNk - 1) / kNk;
  return g;
}
__device__ __forceinline__ int item_tiles(const AttendParams& p, const Queries& q, int lane) {
  int n = 0;
  for (unsigned m = q.starts; m; m &= m - 1) n += segment_at(p, q, __ffs(m) - 1, lane).ntiles;
  return n;
}

// bits of lo <= u < hi for the 32 keys u = a .. a + 31
__device__ __forceinline__ uint32_t range_bits(int a, int lo, int hi) {
  const int l = min(max(lo - a, 0), 32), h = min(max(hi - a, 0), 32);
  return h > l ? (0xffffffffu >> (32 - (h - l))) << l : 0u;
}

// named barrier over n threads that also returns the OR of `v` over them (the same in every thread)
__device__ __forceinline__ bool named_sync_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred q, p;\n setp.ne.u32 q, %1, 0;\n bar.red.or.pred p, %2, %3, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// ---------------------------------------------------------------- packed fp32 pairs
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(x));
  return r;
}
// cap2 tanh(s pre) + bias of two logits; the two quotients share one reciprocal of d0 d1 (each at most 2^7.3)
__device__ __forceinline__ uint64_t capped2(uint64_t s, uint64_t pre, float cap2, uint64_t bias) {
  uint64_t u = mul2(s, pre);
  float u0, u1, d0, d1;
  unpack2(u, u0, u1);
  u0 = tanh_clamp(u0);
  u1 = tanh_clamp(u1);
  u = pack2(u0, u1);
  const uint64_t x = mul2(u, u);
  uint64_t n = pack2(tanh_n(3), tanh_n(3)), d = pack2(tanh_d(4), tanh_d(4));
#pragma unroll
  for (int i = 2; i >= 0; --i) n = fma2(n, x, pack2(tanh_n(i), tanh_n(i)));
#pragma unroll
  for (int i = 3; i >= 0; --i) d = fma2(d, x, pack2(tanh_d(i), tanh_d(i)));
  unpack2(d, d0, d1);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(d0 * d1));
  r *= cap2;
  return fma2(mul2(mul2(u, n), pack2(d1, d0)), pack2(r, r), bias);
}

// One row from its own keys only, by one warp (lane = 4 channels): scores in fp32, an online softmax, fp32 P.
template <bool CAP>
__device__ __noinline__ void slow_row(const AttendParams& p, int64_t row, float sl2, float cap2, float slope2, float (&o)[4],
                                      float& m, float& l, int lane) {
  const int b = static_cast<int>(row / p.n_heads);
  const int64_t t = p.q_pos[b], ws = window_start(t, p.n_win);
  const int seq = p.q_seq[b];
  const int64_t n_w = t - ws + 1, n = n_w + visible_entries(t, p.m, p.n_win);
  const uint2 qv = *reinterpret_cast<const uint2*>(p.q + row * kD + 4 * lane);
  const __nv_bfloat162* q2 = reinterpret_cast<const __nv_bfloat162*>(&qv);
  const float2 qa = __bfloat1622float2(q2[0]), qb = __bfloat1622float2(q2[1]);
  o[0] = o[1] = o[2] = o[3] = 0.f;
  m = -INFINITY;
  l = 0.f;
  for (int64_t u = 0; u < n; ++u) {
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
    s = ruled_score<CAP>(s, sl2, cap2, slope2, dist);
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

// Pipeline (key tiles numbered g over the CTA's items; stage g % 4):
//   loaders : look up rows -> wait kempty (P V of tile g - 4) -> cp.async -> kfull (one tile later, once landed)
//   MMA     : S0(0) S1(0), then per key tile: wait pfull0 -> P V 0(g), S0(g + 1) -> sfull0 (or odone0);
//             wait pfull1 -> P V 1(g) -> kempty, S1(g + 1) -> sfull1 (or odone1); the last S1 of an item -> qempty
//   softmax : wait sfull (S here, and every earlier P V of this tile done: O may be rescaled) -> P -> pfull;
//             after the item's last tile: wait odone -> read O -> oread, which the next item's first P V waits for
template <bool CAP>
__global__ void __launch_bounds__(kThreads, 1)
    attend_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = sm + Smem::Q;
  uint8_t* sK = sm + Smem::K;
  float* sPos = reinterpret_cast<float*>(sm + Smem::POS);
  uint32_t* sRow = reinterpret_cast<uint32_t*>(sm + Smem::ROWS);
  uint32_t* sMask = reinterpret_cast<uint32_t*>(sm + Smem::MASK);
  uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + Smem::BAR);  // [4] loaders (96) -> MMA, softmax
  uint64_t* kempty = kfull + kNS;                                 // [4] MMA -> loaders
  uint64_t* sfull = kempty + kNS;                                 // [2] MMA -> softmax
  uint64_t* pfull = sfull + 2;                                    // [2] softmax (4 warps) -> MMA
  uint64_t* odone = pfull + 2;                                    // [2] MMA -> softmax
  uint64_t* oread = odone + 2;                                    // [2] softmax (4 warps) -> MMA
  uint64_t* qfull = oread + 2;                                    //     Q landed (TMA)
  uint64_t* qempty = qfull + 1;                                   //     the item's S products are done
  uint32_t* sTmem = reinterpret_cast<uint32_t*>(sm + Smem::TMEM);
  volatile int* sAbort = reinterpret_cast<int*>(sm + Smem::FLAGS);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&kfull[i], kLoaders);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&odone[i], 1);
      mbar_init(&oread[i], 4);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    fence_barrier_init();
    *sAbort = 0;
  }
  if (tid == kLoadThread0) prefetch_tensormap(&tm_q);
  if (warp == 8) {
    tmem_alloc(sTmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sTmem;
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
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  const int n_items = static_cast<int>((rows + kItemRows - 1) / kItemRows);
  const float cap2 = CAP ? p.score_cap * kLog2e : 0.f;
  const float sl2 = CAP ? p.sm_scale / p.score_cap : p.sm_scale * kLog2e;
  uint32_t g = 0;      // key tiles before the current item
  uint32_t n_act = 0;  // items with keys before the current one

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
    if (warp == 8) {
      // ---------------------------------------------------------------- MMA issue (lane 0; the warp waits together)
      const bool issuer = lane == 0;
      const uint32_t idesc_s = umma_idesc_bf16(kTileRows, kNk, false);
      const uint32_t idesc_pv = umma_idesc_bf16(kTileRows, kD, true);
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
      auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(kFull, mbar_wait(bar, parity, p.status)); };
      auto issue_s = [&](int w, uint32_t gt) {  // S of tile w: 8 K-steps over the two 64-channel halves
        if (issuer) {
          const uint32_t q = sQa + w * kStageBytes, k = sKa + (gt % kNS) * kStageBytes;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t off = (ks >> 2) * kHalfBytes + (ks & 3) * 32u;
            umma_ss(tmem + kColS + w * kNk, umma_desc_sw128(q + off, 16, 1024), umma_desc_sw128(k + off, 16, 1024),
                    idesc_s, ks > 0 ? 1u : 0u);
          }
          umma_commit(&sfull[w]);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int w, uint32_t gt, bool acc) {  // O += P V of tile w: 8 K-steps of 16 keys
        if (issuer) {
          const uint32_t v = sKa + (gt % kNS) * kStageBytes;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            umma_ts(tmem + kColO + w * kD, tmem + kColS + w * kNk + ks * 8,
                    umma_desc_sw128(v + ks * 16 * 128, kHalfBytes, 1024), idesc_pv, (acc || ks > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      bool ok = true;
      for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
        const int ntot = item_tiles(p, load_queries(p, item, lane), lane);
        if (ntot == 0) continue;
        if (!(ok = wait(qfull, n_act & 1u) && wait(&kfull[g % kNS], (g / kNS) & 1u))) break;
        tc_fence_after();
        issue_s(0, g);
        issue_s(1, g);
        if (ntot == 1 && issuer) umma_commit(qempty);
        for (int it = 0; it < ntot && ok; ++it) {
          if (__shfl_sync(kFull, *sAbort, 0)) {
            ok = false;
            break;
          }
          const uint32_t gt = g + it, gn = gt + 1;
          const bool more = it + 1 < ntot;
          ok = wait(&pfull[0], gt & 1u) && (it > 0 || n_act == 0 || wait(&oread[0], (n_act - 1) & 1u));
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, gt, it > 0);
          if (more) {
            if (!(ok = wait(&kfull[gn % kNS], (gn / kNS) & 1u))) break;
            tc_fence_after();
            issue_s(0, gn);
          } else if (issuer) {
            umma_commit(&odone[0]);
          }
          ok = wait(&pfull[1], gt & 1u) && (it > 0 || n_act == 0 || wait(&oread[1], (n_act - 1) & 1u));
          if (!ok) break;
          tc_fence_after();
          issue_pv(1, gt, it > 0);
          if (issuer) umma_commit(&kempty[gt % kNS]);
          if (more) {
            issue_s(1, gn);
            if (it + 2 == ntot && issuer) umma_commit(qempty);
          } else if (issuer) {
            umma_commit(&odone[1]);
          }
          __syncwarp();
        }
        g += ntot;
        ++n_act;
      }
      if (!ok) {
        *sAbort = 1;
        // what was issued gets a bounded chance to land before the tensor memory is freed
        if (issuer) umma_commit(&odone[0]);
        __syncwarp();
        mbar_wait(&odone[0], n_act & 1u, nullptr);
      }
    } else {
      // ---------------------------------------------------------------- loaders
      const int lt = tid - kLoadThread0, lw = lt >> 5;
      bool ok = true;
      for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
        const Queries q = load_queries(p, item, lane);
        const int ntot = item_tiles(p, q, lane);
        if (ntot == 0) continue;
        if (lw == 0) {  // Q once the last item's S products are done with it
          const bool free = __all_sync(kFull, n_act == 0 || mbar_wait(qempty, (n_act - 1) & 1u, p.status));
          if (!free) {
            *sAbort = 1;
          } else if (lane == 0) {
            mbar_arrive_expect_tx(qfull, 2 * kStageBytes);
            const int row0 = item * kItemRows;
            for (int w = 0; w < 2; ++w)
              for (int h = 0; h < 2; ++h)
                tma_load_2d(sQ + w * kStageBytes + h * kHalfBytes, &tm_q, h * 64, row0 + w * kTileRows, qfull);
          }
          __syncwarp();
        }
        uint32_t gt = g;
        for (unsigned ms = q.starts; ms && ok; ms &= ms - 1) {
          const Segment sg = segment_at(p, q, __ffs(ms) - 1, lane);
          for (int it = 0; it < sg.ntiles; ++it, ++gt) {
            const int st = gt % kNS;
            // keys lt and (threads 0-31) 96 + lt of the tile: source row and position
            uint32_t code[2] = {0u, 0u};
            float pos[2] = {0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int u = it * kNk + h * kLoaders + lt;
              if ((h == 0 || lw == 0) && u < sg.n) {
                if (u < sg.n_w) {
                  code[h] = window_code(p, sg.seq, sg.wlo + u);
                  pos[h] = static_cast<float>(sg.wlo + u - sg.thi);
                } else {
                  code[h] = entry_code(p, sg.seq, u - sg.n_w);
                  pos[h] = -entry_distance(sg.thi, u - sg.n_w, p.m);
                }
                if (!code[h]) report(p.status, CSKV_ERR_OUT_OF_RANGE);
              }
            }
            const bool free = gt < kNS || mbar_wait(&kempty[st], ((gt / kNS) - 1) & 1u, p.status);
            uint32_t* row = sRow + (gt & 1) * kNk;
            row[lt] = code[0];
            sPos[st * kNk + lt] = pos[0];
            const unsigned b0 = __ballot_sync(kFull, code[0] != 0u), b1 = __ballot_sync(kFull, code[1] != 0u);
            if (lw == 0) {
              row[kLoaders + lt] = code[1];
              sPos[st * kNk + kLoaders + lt] = pos[1];
            }
            if (lane == 0) {
              sMask[st * 4 + lw] = b0;
              if (lw == 0) sMask[st * 4 + 3] = b1;
            }
            if (named_sync_or(3, kLoaders, !free || *sAbort)) {
              *sAbort = 1;
              ok = false;
              break;
            }
            uint8_t* dst = sK + st * kStageBytes;
#pragma unroll 4
            for (int id = lt; id < kNk * 16; id += kLoaders) {  // 16 consecutive threads copy one 256-byte row
              const int key = id >> 4, c = id & 15;
              const uint16_t* src = code_row(p, row[key]);
              cp_async16(dst + (c >> 3) * kHalfBytes + key * 128 + (((c & 7) ^ (key & 7)) << 4),
                         src ? static_cast<const void*>(src + c * 8) : static_cast<const void*>(p.q), src ? 16 : 0);
            }
            cp_async_commit();
            if (gt > g) {  // the tile before this one has landed
              cp_async_wait<1>();
              fence_proxy_async_smem();
              mbar_arrive(&kfull[(gt - 1) % kNS]);
            }
          }
        }
        cp_async_wait<0>();
        if (!ok) break;
        fence_proxy_async_smem();
        mbar_arrive(&kfull[(gt - 1) % kNS]);
        g += ntot;
        ++n_act;
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax (one row per thread)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
    const int w = warp >> 2;
    const uint32_t trow = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t sb = trow + kColS + w * kNk, ob = trow + kColO + w * kD;
    bool ok = true;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      const Queries q = load_queries(p, item, lane);
      const int64_t row = (int64_t)item * kItemRows + w * kTileRows + (warp & 3) * 32 + lane;
      const bool in = row < rows;
      const int qi = in ? static_cast<int>(row / p.n_heads) - q.q0 : 0;  // this row's query lane
      const int h = in ? static_cast<int>(row % p.n_heads) : 0;
      const int64_t t = __shfl_sync(kFull, q.t, qi);
      const float slope2 = p.slopes ? p.slopes[h] * kLog2e : 0.f;
      const int ntot = item_tiles(p, q, lane);
      float m_used = -INFINITY, l_run = 0.f;
      int64_t shift = 0;  // the row's logits are taken at distance 0 of its segment's last query
      int it = 0;
      for (unsigned ms = q.starts; ms && ok; ms &= ms - 1) {
        const Segment sg = segment_at(p, q, __ffs(ms) - 1, lane);
        // this row's keys in the segment's list: window lo .. hi - 1, entries n_w .. end - 1
        int lo = 0, hi = 0, end = 0;
        if (in && t >= 0 && qi >= sg.s && qi < sg.e) {
          lo = static_cast<int>(window_start(t, p.n_win) - sg.wlo);
          hi = static_cast<int>(t - sg.wlo) + 1;
          end = sg.n_w + static_cast<int>(visible_entries(t, p.m, p.n_win));
          shift = t - sg.thi;
        }
        for (int k = 0; k < sg.ntiles; ++k, ++it) {
          const uint32_t gt = g + it;
          const int st = gt % kNS;
          // the stage's positions and key bits were written before kfull; that phase cannot move on before this
          // thread's P has been used
          ok = __all_sync(kFull, mbar_wait(&sfull[w], gt & 1u, p.status)) &&
               __all_sync(kFull, mbar_wait(&kfull[st], (gt / kNS) & 1u, p.status)) && !__any_sync(kFull, *sAbort != 0);
          if (!ok) break;
          tc_fence_after();
          uint32_t s[kNk];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(sb + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
          tmem_ld_wait();
          const float4* pos4 = reinterpret_cast<const float4*>(sPos + st * kNk);
          const uint64_t sl = pack2(slope2, slope2), pre = pack2(sl2, sl2);
#pragma unroll
          for (int j = 0; j < kNk; j += 4) {
            const float4 d = pos4[j / 4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const uint64_t bias = mul2(sl, e ? pack2(d.z, d.w) : pack2(d.x, d.y));
              const uint64_t x = pack2(__uint_as_float(s[j + e]), __uint_as_float(s[j + e + 1]));
              const uint64_t v = CAP ? capped2(x, pre, cap2, bias) : fma2(x, pre, bias);
              float a, b;
              unpack2(v, a, b);
              s[j + e] = __float_as_uint(a);
              s[j + e + 1] = __float_as_uint(b);
            }
          }
          const int a = k * kNk;
          float mt = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t vm = sMask[st * 4 + c] & (range_bits(a + 32 * c, lo, hi) | range_bits(a + 32 * c, sg.n_w, end));
            if (__any_sync(kFull, vm != kFull)) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((vm >> j) & 1u)) s[32 * c + j] = 0xff800000u;  // -inf
            }
            float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              m0 = fmaxf(m0, __uint_as_float(s[32 * c + j]));
              m1 = fmaxf(m1, __uint_as_float(s[32 * c + j + 1]));
            }
            mt = fmaxf(mt, fmaxf(m0, m1));
          }
          float corr = 1.f;
          bool rescale = false;
          if (mt > m_used + kRescaleThreshold || (m_used == -INFINITY && mt != -INFINITY)) {
            corr = ex2(m_used - mt);  // 0 when m_used is -inf
            rescale = it > 0;
            l_run *= corr;
            m_used = mt;
          }
          const float msub = m_used == -INFINITY ? 0.f : -m_used;
          if (__any_sync(kFull, rescale)) {
#pragma unroll 1
            for (int c = 0; c < kD; c += 16) {
              uint32_t o[16];
              tmem_ld16(ob + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
              tmem_st16(ob + c, o);
            }
          }
          const uint64_t sub = pack2(msub, msub);
          uint64_t l2 = pack2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t pp[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float e0, e1;
              unpack2(add2(pack2(__uint_as_float(s[32 * c + 2 * j]), __uint_as_float(s[32 * c + 2 * j + 1])), sub), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              l2 = add2(l2, pack2(e0, e1));
              pp[j] = pack_bf16(e0, e1);
            }
            tmem_st16(sb + 16 * c, pp);
          }
          float la, lb;
          unpack2(l2, la, lb);
          l_run += la + lb;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[w]);
        }
      }
      if (!ok) break;
      // epilogue: O / l in bf16, and the log-sum-exp
      if (ntot > 0) {
        if (!(ok = __all_sync(kFull, mbar_wait(&odone[w], n_act & 1u, p.status)))) break;
        tc_fence_after();
      }
      const bool has = in && l_run > 0.f;
      const float inv = has ? 1.f / l_run : 0.f;
      float odd = 0.f;  // NaN once an output is not finite
      auto put = [&](int c, const uint32_t (&o)[32]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float f[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] = has ? __uint_as_float(o[8 * i + e]) * inv : 0.f;
            odd = fmaf(f[e], 0.f, odd);
          }
          if (p.rope_dims > 0 && has) {  // inverse RoPE of the output's last rope_dims channels
            float a4[4] = {f[0], f[1], f[2], f[3]}, b4[4] = {f[4], f[5], f[6], f[7]};
            inverse_rope4(a4, c + 8 * i, kD, p.rope_dims, p.rope_base, t);
            inverse_rope4(b4, c + 8 * i + 4, kD, p.rope_dims, p.rope_base, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              f[e] = a4[e];
              f[4 + e] = b4[e];
            }
          }
          if (in)
            *reinterpret_cast<uint4*>(p.out + row * kD + c + 8 * i) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
      };
#pragma unroll 1
      for (int c = 0; c < kD; c += 32) {
        uint32_t o[32];
        if (ntot > 0) {
          tmem_ld32(ob + c, o);
          tmem_ld_wait();
        }
        put(c, o);
      }
      // the next item's first P V overwrites O: this warp's reads of it are complete
      tc_fence_before();
      __syncwarp();
      if (ntot > 0 && lane == 0) mbar_arrive(&oread[w]);
      float lse = has ? (m_used + log2f(l_run) - slope2 * static_cast<float>(shift)) * kLn2 : -INFINITY;
      for (unsigned bad = __ballot_sync(kFull, in && (l_run != l_run || !(odd == 0.f))); bad; bad &= bad - 1) {
        const int r = __ffs(bad) - 1;  // rows whose output is not finite, one at a time by the whole warp
        const int64_t rr = __shfl_sync(kFull, row, r);
        const int64_t tr = __shfl_sync(kFull, t, r);
        float o4[4], m, l;
        slow_row<CAP>(p, rr, sl2, cap2, __shfl_sync(kFull, slope2, r), o4, m, l, lane);
        const float iv = 1.f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e) o4[e] *= iv;
        inverse_rope4(o4, 4 * lane, kD, p.rope_dims, p.rope_base, tr);
        *reinterpret_cast<uint2*>(p.out + rr * kD + 4 * lane) = make_uint2(pack_bf16(o4[0], o4[1]), pack_bf16(o4[2], o4[3]));
        if (lane == r) lse = (m + log2f(l)) * kLn2;
      }
      if (in && p.lse) p.lse[row] = lse;
      g += ntot;
      if (ntot > 0) ++n_act;
    }
    if (!ok) *sAbort = 1;
  }
  cp_async_wait<0>();
  // after an abort, a Q copy in flight gets a bounded chance to land
  if (warp == 9 && __shfl_sync(kFull, *sAbort, 0)) mbar_wait(qfull, n_act & 1u, nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, kTmemCols);
}

bool encode_q(CUtensorMap* map, const void* base, uint64_t rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kTileRows)};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// The plain form (no rule) keeps the kernels it has always run on, and so its results.
bool attend_chunk_supported(const AttendParams& p, int n_sm) {
  const uint64_t pool_rows = static_cast<uint64_t>(p.n_pages) * p.page_size;
  const uint64_t ring_rows = static_cast<uint64_t>(p.n_seqs_layer) * p.n_win;
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  return !p.is_csa && has_score_rule(p) && p.x_chunk && p.d_qk == kD && p.d_v == kD && p.n_heads >= 16 &&
         p.kv_dtype == CSKV_BF16 && rows >= (int64_t)kItemRows * n_sm / 2 && rows <= 0x7fffffff - kItemRows &&
         visible_entries(p.max_pos, p.m, p.n_win) < (1 << 29) && p.n_win < (1 << 29) &&
         pool_rows <= kRowMask && ring_rows <= kRowMask && static_cast<uint64_t>(p.chunk_len) <= kRowMask;
}

cudaError_t launch_attend_chunk(AttendParams& p, int n_sm, cudaStream_t st) {
  CUtensorMap tm_q;
  const int64_t rows = (int64_t)p.n_q * p.n_heads;
  if (!encode_q(&tm_q, p.q, static_cast<uint64_t>(rows))) return cudaErrorNotSupported;
  const size_t smem = Smem::bytes();
  auto kern = p.score_cap > 0.f ? attend_chunk_kernel<true> : attend_chunk_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t items = (rows + kItemRows - 1) / kItemRows;
  return launch_pdl(kern, dim3(static_cast<unsigned>(items < n_sm ? items : n_sm)), dim3(kThreads), smem, st, tm_q, p);
}

}  // namespace cskv
