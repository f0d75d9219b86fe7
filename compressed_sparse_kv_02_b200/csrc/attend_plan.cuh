// attend_plan.cuh -- the key split of a call whose queries have key lists of very different lengths.
//
// The host knows the longest possible list only. Cutting by it gives the longest query its share of the GPU and every
// shorter one fewer pieces: with lengths from 32K to 1M tokens, 54 of 148 CTAs worked, on 15 key tiles each. The
// kernels with a score rule therefore find their split on the device, where the lengths are: the smallest piece (in
// units of the kernel's key tile) for which all queries' pieces fit the given number of slots, by bisection, once per
// CTA and warp. Pieces are numbered without gaps, query after query, in the partial outputs' buffer; the numbering is
// left in the workspace (plan) for the merge.
#pragma once

#include "cskv_device.cuh"
#include "cskv_internal.h"

namespace cskv {

// Keys per piece, called by whole warps: keys_of(b) is query b's number of keys, `unit` the key tile, `slots` the
// pieces wanted; never more than the host's keys_per_split (a multiple of unit), for which n_q * max_splits slots do.
template <typename F>
__device__ __forceinline__ int plan_split(const AttendParams& p, int unit, int slots, int lane, F keys_of) {
  const int most = p.keys_per_split / unit;
  if (p.n_q >= slots) return most * unit;
  auto tiles_of = [&](int b) { return static_cast<int>((keys_of(b) + unit - 1) / unit); };
  constexpr int kHeld = 3;  // the first 96 queries' tiles stay in registers: counting them takes loads and wide divisions
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = lane + 32 * i < p.n_q ? tiles_of(lane + 32 * i) : 0;
  auto pieces = [&](int per) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) n += (held[i] + per - 1) / per;
    for (int b = lane + 32 * kHeld; b < p.n_q; b += 32) n += (tiles_of(b) + per - 1) / per;
    return static_cast<int>(__reduce_add_sync(kFull, n));
  };
  int lo = (pieces(1) + slots - 1) / slots, hi = most;
  if (lo < 1) lo = 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pieces(mid) <= slots)
      hi = mid;
    else
      lo = mid + 1;
  }
  return (lo < most ? lo : most) * unit;
}

}  // namespace cskv
