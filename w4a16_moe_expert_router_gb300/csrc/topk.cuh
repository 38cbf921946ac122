// topk.cuh -- the router's choice of one token by one warp.
#pragma once

#include <cstdint>

#include "internal.h"

namespace moe {

// Router order as one unsigned key: a larger logit gives a larger key, -0 and
// +0 give the same key (they compare equal as fp32 values); NaN ranks below
// every number.  Equal keys go to the lower expert index.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 1u;
  if (v == 0.f) v = 0.f;
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Compare-exchange of two candidates of a lane: afterwards slot a holds the one
// that ranks first (larger key, then lower slot, i.e. lower expert index).
__device__ __forceinline__ void cx(uint32_t& ka, int& ja, float& va, uint32_t& kb, int& jb, float& vb) {
  const bool swap = kb > ka || (kb == ka && jb < ja);
  if (swap) {
    const uint32_t tk = ka;
    const int tj = ja;
    const float tv = va;
    ka = kb;
    ja = jb;
    va = vb;
    kb = tk;
    jb = tj;
    vb = tv;
  }
}

// Top-k of one token's E logits by one warp, then the softmax over the k selected
// logits, summed in rank order.  Lane l holds experts l + 32 j (j < NS, NS = 4 for
// E <= 128, else 8) and sorts them once by (key descending, index ascending) with a
// sorting network (5 or 19 compare-exchanges), so its head is its best remaining
// candidate.  Each round takes the largest head key over the warp (one reduction);
// if one lane holds it (one ballot) that lane wins, otherwise the lowest expert
// index among the tied heads does (a second reduction); the winning lane drops its
// head.
template <int NS>
__device__ __forceinline__ void topk_softmax_warp(const float* row, int E, int k, int lane, int32_t* idx_out,
                                                  float* w_out, int* sel_out) {
  float v[NS];
  uint32_t key[NS];
  int js[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int e = lane + 32 * j;
    v[j] = 0.f;
    key[j] = 0u;  // below every real key (order_key >= 1)
    js[j] = j;
    if (e < E) {
      v[j] = __ldcg(row + e);  // from L2: a launch that starts early finds nothing old
      key[j] = order_key(v[j]);
    }
  }
  if constexpr (NS == 4) {
    constexpr int net[5][2] = {{0, 1}, {2, 3}, {0, 2}, {1, 3}, {1, 2}};
#pragma unroll
    for (int c = 0; c < 5; ++c) {
      const int a = net[c][0], b = net[c][1];
      cx(key[a], js[a], v[a], key[b], js[b], v[b]);
    }
  } else {
    constexpr int net[19][2] = {{0, 2}, {1, 3}, {4, 6}, {5, 7}, {0, 4}, {1, 5}, {2, 6}, {3, 7}, {0, 1}, {2, 3},
                                {4, 5}, {6, 7}, {2, 4}, {3, 5}, {1, 4}, {3, 6}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int c = 0; c < 19; ++c) {
      const int a = net[c][0], b = net[c][1];
      cx(key[a], js[a], v[a], key[b], js[b], v[b]);
    }
  }
  float sel_v[kMaxTopK];
  int sel_e[kMaxTopK];
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r) {
    sel_v[r] = 0.f;
    sel_e[r] = 0;
    if (r < k) {
      const uint32_t kmax = __reduce_max_sync(0xffffffffu, key[0]);
      const bool mine = key[0] == kmax;
      const unsigned tied = __ballot_sync(0xffffffffu, mine);
      int wl;  // winning lane
      if ((tied & (tied - 1u)) == 0u) {
        wl = __ffs(tied) - 1;
      } else {
        const uint32_t cand = mine ? static_cast<uint32_t>(lane + 32 * js[0]) : 0xffffffffu;
        wl = static_cast<int>(__reduce_min_sync(0xffffffffu, cand) & 31u);
      }
      sel_e[r] = __shfl_sync(0xffffffffu, lane + 32 * js[0], wl);
      sel_v[r] = __shfl_sync(0xffffffffu, v[0], wl);
      if (lane == wl) {
#pragma unroll
        for (int j = 0; j + 1 < NS; ++j) {
          key[j] = key[j + 1];
          js[j] = js[j + 1];
          v[j] = v[j + 1];
        }
        key[NS - 1] = 0u;
      }
    }
  }
  const float m = sel_v[0];
  float den = 0.f;
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r)
    if (r < k) den += expf(sel_v[r] - m);
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r)
    if (r < k && r == lane) {
      idx_out[r] = sel_e[r];
      w_out[r] = expf(sel_v[r] - m) / den;
      sel_out[r] = sel_e[r];
    }
}

}  // namespace moe
