// few.cu -- the whole W4A16 layer for a few tokens (at most kFewTokens), from the router's logits
// to the output, in two launches: gate_up with the activation, then down with the weighted sum.
//
//   a = Wgu x,  h = gelu(a_gate) a_up,  out[t] = residual[t] + sum over the token's experts of w (Wd h)
//
// A few tokens meet almost as many experts as they have choices, and an expert's weights are used
// for one or two of them: the time is the way of the chosen experts' weights from memory (19 MB for
// one token of top-8, d 2048, f 704: 2.9 us), and, for one token, what is not hidden behind it. So
//  - every CTA forms the routing itself (a warp per token), instead of a launch for it;
//  - the down launch starts while the gate_up launch runs, forms the routing too and requests its
//    first weights before it waits for h;
//  - work is cut finely: 16 (8 gate and 8 up, twice) rows of weights by one CTA, whose warps share
//    the contraction; each warp streams its own stages with cp.async, several ahead, also across
//    work items, and needs no other warp until the item's sums meet in shared memory.
//
// The weights stay integers: a group's codes are multiplied as they are (exact products in the fp32
// accumulators), then scale and zero-point are applied to the group's sum,
//   sum_k w_k x_k = s sum_k q_k x_k + c sum_k x_k,   c = -s z (affine: the bias),
// the sum of x coming from one more matrix instruction with ones. h is kept as two 16-bit values, h =
// hi + lo, which take two columns of one instruction (four tokens per instruction, not eight): 22 bits
// of h for fp16, 16 for bf16. A warp multiplies its stages in ascending order, the warps' sums
// meet in their order, and a token's experts are added in ascending order within each half of them
// (even and odd numbers): the result does not depend on the other tokens and is the same in every run.
#include "activation.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs16 = kFewTokens * kMaxTopK;  // pairs at most, and items
static_assert(kMaxPairs16 <= kThreads && kMaxExperts <= kThreads, "a thread per pair and per expert");
constexpr int kUpTokens = 8, kDownTokens = 4;       // tokens of an item
constexpr int kDepth = 4;                           // pieces of a warp in flight
constexpr int kXRow = kStageCols * 2 + 16;          // bytes of a token's stage in shared memory: rows shifted by a bank group
constexpr int kHBytes = 2048;                       // a stage's h fragments: 4 tokens x (hi, lo) x 128 columns
constexpr int kRedStride = 33;

struct Args {
  const void* x;
  const float* logits;
  const uint8_t* w;       // this launch's projection
  const void* residual;
  int32_t* topk_idx;
  float* topk_w;
  void* out;
  uint16_t* h;            // [pairs][2][f], in the order of the down launch's fragments
  int T, d, f, E, k, act, affine;
  int K;                  // contraction: d or f
  int64_t expert_bytes, block_bytes;
  int stage_warps;        // warps that share an item's contraction
  int slot_bytes;         // a piece in shared memory
};

// Routing and items, formed by every CTA.
template <int kTokens>
struct Routing {
  int32_t sel[kMaxPairs16];
  int32_t spare[kMaxPairs16];
  float w[kMaxPairs16];
  uint32_t mask[kMaxExperts];          // tokens of an expert
  int32_t base[kMaxExperts];           // first item of an expert
  int32_t expert[kMaxPairs16];         // expert of an item
  int16_t pair[kMaxPairs16][kTokens];  // pairs of an item, -1 behind them
  int32_t warp_tot[kWarps];
  int32_t items, half;                 // items; those of even experts (split lists)
};

// Lists the items by expert ascending; kSplit: those of the even experts first.
template <int kTokens, bool kSplit>
__device__ __forceinline__ void form_routing(Routing<kTokens>& r, const Args& a) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  r.mask[tid] = 0u;
  for (int i = tid; i < kMaxPairs16 * kTokens; i += kThreads) (&r.pair[0][0])[i] = -1;
  for (int t = warp; t < a.T; t += kWarps) {
    const float* row = a.logits + static_cast<size_t>(t) * a.E;
    if (a.E <= 128)
      topk_softmax_warp<4>(row, a.E, a.k, lane, r.sel + t * a.k, r.w + t * a.k, r.spare + t * a.k);
    else
      topk_softmax_warp<8>(row, a.E, a.k, lane, r.sel + t * a.k, r.w + t * a.k, r.spare + t * a.k);
  }
  __syncthreads();
  const int t = tid / a.k, e = tid < a.T * a.k ? r.sel[tid] : 0;
  if (tid < a.T * a.k) atomicOr(&r.mask[e], 1u << t);
  __syncthreads();
  // thread i takes expert i, or with kSplit the i-th of the evens followed by the odds
  const int evens = (a.E + 1) / 2;
  const int mine = !kSplit ? tid : tid < evens ? 2 * tid : 2 * (tid - evens) + 1;
  const int n = tid < a.E ? (__popc(r.mask[mine]) + kTokens - 1) / kTokens : 0;
  int incl = n;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) r.warp_tot[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? r.warp_tot[w] : 0;
    total += r.warp_tot[w];
  }
  if (tid < a.E) {
    r.base[mine] = before + incl - n;
    if (tid == evens - 1) r.half = before + incl;
  }
  if (tid == 0) r.items = total;
  __syncthreads();
  if (tid < a.T * a.k) {
    const int nth = __popc(r.mask[e] & ((1u << t) - 1u)), item = r.base[e] + nth / kTokens;
    r.pair[item][nth % kTokens] = static_cast<int16_t>(tid);
    if (nth % kTokens == 0) r.expert[item] = e;
  }
  __syncthreads();
}

// One word of codes -> an m16n8k16 A fragment of codes. fp16: masks alone, the codes as
// subnormals (2^-24 for rows g, 2^-20 for rows g + 8, whose nibbles sit four bits higher). bf16, whose
// subnormals would fall out of fp32's range: 128 + q from exponent bits, less 128 (exact).
template <bool kBf16>
__device__ __forceinline__ void codes(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (!kBf16) {
    const uint32_t w8 = w >> 8;
    a[0] = w & 0x000f000fu;
    a[1] = w & 0x00f000f0u;
    a[2] = w8 & 0x000f000fu;
    a[3] = w8 & 0x00f000f0u;
  } else {
    const uint32_t k128 = 0x43004300u;
    const __nv_bfloat162 minus = *reinterpret_cast<const __nv_bfloat162*>(&k128);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = and_or(w >> (4 * i), 0x000f000fu, k128);
      const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), minus);
      a[i] = *reinterpret_cast<const uint32_t*>(&q);
    }
  }
}
template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    mma_bf16_16816(d, a, b0, b1);
  else
    mma_f16_16816(d, a, b0, b1);
}
template <bool kBf16>
constexpr uint32_t kOnes = kBf16 ? 0x3f803f80u : 0x3c003c00u;

// A group's sums into the totals: tot += s part + c sum, for rows g (first two) and g + 8.
template <bool kBf16>
__device__ __forceinline__ void apply_group(float (&tot)[4], const float (&part)[4], const float (&sum)[4], uint2 sz,
                                            int affine) {
  const float2 lo = __half22float2(bits_h2(sz.x)), hi = __half22float2(bits_h2(sz.y));
  const float s_lo = kBf16 ? lo.x : lo.x * 0x1p24f, s_hi = kBf16 ? hi.x : hi.x * 0x1p20f;
  const float c_lo = affine ? lo.y : -lo.x * lo.y, c_hi = affine ? hi.y : -hi.x * hi.y;
  tot[0] = fmaf(s_lo, part[0], fmaf(c_lo, sum[0], tot[0]));
  tot[1] = fmaf(s_lo, part[1], fmaf(c_lo, sum[1], tot[1]));
  tot[2] = fmaf(s_hi, part[2], fmaf(c_hi, sum[2], tot[2]));
  tot[3] = fmaf(s_hi, part[3], fmaf(c_hi, sum[3], tot[3]));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// The warp copies `bytes` (a multiple of 16) to its slot.
__device__ __forceinline__ void copy_warp(uint32_t dst, const uint8_t* src, int bytes, int lane) {
  for (int i = lane * 16; i < bytes; i += 512) cp_async_16(dst + i, src + i);
}

// The place of column c (0..63 of 64) in h's fragment order: [tq][step][value], value
// 0..3 the columns 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 of a 16-column step.
__device__ __forceinline__ int h_place(int c) {
  const int step = c >> 4, r = c & 15;
  return ((r & 7) >> 1) * 16 + step * 4 + (r & 1) + 2 * (r >> 3);
}

// ------------------------------------------------------------------ gate_up
//
// A unit is an item and kWarps / stage_warps pairs of strips; warp w takes pair w / stage_warps
// and the stages w % stage_warps, + stage_warps, ..
template <bool kBf16, int G>
__global__ void __launch_bounds__(kThreads) few_gate_up_kernel(const Args a) {
  constexpr int NG = kStageCols / G, kSteps = G / 16, kStripBytes = 1024 + 64 * NG;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Routing<kUpTokens> r;
  __shared__ float red[2][kWarps][2][4][kRedStride];
  grid_dependency_wait();    // the logits, x, and h, which the call before may still read
  grid_dependents_launch();  // only now: the down launch reads logits and weights before it waits
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  form_routing<kUpTokens, false>(r, a);
  if (blockIdx.x == 0)
    for (int i = tid; i < a.T * a.k; i += kThreads) {
      if (a.topk_idx) a.topk_idx[i] = r.sel[i];
      if (a.topk_w) a.topk_w[i] = r.w[i];
    }
  const int W = a.stage_warps, P = kWarps / W, my_pair = warp / W, my_stage = warp % W;
  const int S = a.K / kStageCols, per_item = a.f / 16 / P, units = r.items * per_item;
  const uint32_t ring = smem_addr(smem) + warp * kDepth * a.slot_bytes;
  const int xrows = min(a.T, kUpTokens);

  int pu = blockIdx.x, ps = my_stage, pslot = 0;  // the piece to request next
  const auto request = [&] {
    if (pu < units && ps < S) {
      const int item = pu / per_item, pr = (pu - item * per_item) * P + my_pair;
      const uint32_t dst = ring + pslot * a.slot_bytes;
      const uint8_t* src = a.w + r.expert[item] * a.expert_bytes + (pr >> 2) * a.block_bytes +
                           static_cast<int64_t>(ps) * (8 * kStripBytes) + (pr & 3) * (2 * kStripBytes);
      copy_warp(dst, src, 2 * kStripBytes, lane);
      for (int i = lane; i < xrows * 16; i += 32) {
        const int p = r.pair[item][i >> 4];
        if (p >= 0)
          cp_async_16(dst + 2 * kStripBytes + (i >> 4) * kXRow + (i & 15) * 16,
                      static_cast<const uint8_t*>(a.x) +
                          (static_cast<size_t>(p / a.k) * a.d + ps * kStageCols) * 2 + (i & 15) * 16);
      }
      ps += W;
      if (ps >= S) {
        ps = my_stage;
        pu += gridDim.x;
      }
      if (++pslot == kDepth) pslot = 0;
    }
    cp_async_commit();
  };
  for (int i = 0; i < kDepth - 1; ++i) request();
  // fragment of step kk: rows of eight tokens (those behind the last one repeat it; their columns are not used)
  const uint32_t xoff = 2 * kStripBytes + min(lane & 7, xrows - 1) * kXRow + (lane >> 3) * 16;
  int slot = 0, buf = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    float tot[2][4] = {};
    for (int s = my_stage; s < S; s += W) {
      cp_async_wait<kDepth - 2>();
      __syncwarp();
      request();
      const uint32_t at = ring + slot * a.slot_bytes;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        float part[2][4] = {}, sum[4] = {};
#pragma unroll
        for (int q = 0; q < kSteps; q += 2) {
          const int kk = j * kSteps + q;  // even
          uint32_t b[4];
          ldmatrix_x4(at + xoff + kk * 32, b[0], b[1], b[2], b[3]);
          uint2 word[2];
#pragma unroll
          for (int h = 0; h < 2; ++h)
            word[h] = lds64(at + h * kStripBytes + 64 * NG + (kk / 4) * 512 + lane * 16 + (kk % 4) * 4);
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const uint32_t ones[4] = {kOnes<kBf16>, kOnes<kBf16>, kOnes<kBf16>, kOnes<kBf16>};
            mma<kBf16>(sum, ones, b[2 * v], b[2 * v + 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t af[4];
              codes<kBf16>(v ? word[h].y : word[h].x, af);
              mma<kBf16>(part[h], af, b[2 * v], b[2 * v + 1]);
            }
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          apply_group<kBf16>(tot[h], part[h], sum, lds64(at + h * kStripBytes + (lane >> 2) * (8 * NG) + j * 8),
                             a.affine);
      }
      __syncwarp();  // the slot is read before it is requested again
      if (++slot == kDepth) slot = 0;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[buf][warp][h][i][lane] = tot[h][i];
    __syncthreads();
    // h of strip row j (8 of a strip) and token n: the warps' sums of its gate and up row in order
    const int item = u / per_item, pr0 = (u - item * per_item) * P;
    for (int o = tid; o < P * 128; o += kThreads) {
      const int n = o & 7, j = (o >> 3) & 7, h = (o >> 6) & 1, pr = o >> 7;
      const int p = r.pair[item][n];
      if (p < 0) continue;
      float gate = 0.f, up = 0.f;
      for (int w = pr * W; w < (pr + 1) * W; ++w) {
        gate += red[buf][w][h][n & 1][j * 4 + (n >> 1)];
        up += red[buf][w][h][2 + (n & 1)][j * 4 + (n >> 1)];
      }
      const float v = activate(gate, a.act) * up;
      const int c = 16 * (pr0 + pr) + 8 * h + j;
      constexpr int kType = kBf16 ? 1 : 0;
      const uint16_t hi = to16<kType>(v), lo = to16<kType>(v - from16<kType>(hi));
      uint16_t* dst = a.h + static_cast<size_t>(p) * 2 * a.f + (c & ~63) + h_place(c & 63);
      dst[0] = hi;
      dst[a.f] = lo;
    }
    buf ^= 1;
  }
  cp_async_wait<0>();
}

// --------------------------------------------------------------------- down
//
// A CTA takes one strip of 16 rows of every item. Its warps are two sets, for the even and the odd
// experts; warp w of a set takes the stages w, w + stage_warps, .. of the set's items.
template <bool kBf16, int G>
__global__ void __launch_bounds__(kThreads) few_down_kernel(const Args a) {
  constexpr int kMaxNg = kStageCols / G;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Routing<kDownTokens> r;
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  form_routing<kDownTokens, true>(r, a);
  const int W = a.stage_warps, sets = 2, set = warp / W, my_stage = warp - set * W;
  const int S = (a.K + kStageCols - 1) / kStageCols;
  const int i0 = set == 0 ? 0 : r.half, i1 = set >= sets ? i0 : set == 0 ? r.half : r.items;
  const int strip = blockIdx.x;
  const uint32_t ring = smem_addr(smem) + warp * kDepth * a.slot_bytes;
  float* const acc = reinterpret_cast<float*>(smem + kWarps * kDepth * a.slot_bytes) + warp * a.T * 17;
  for (int i = lane; i < a.T * 17; i += 32) acc[i] = 0.f;
  const int steps_of_last = (a.K % kStageCols) ? 4 : 8;

  const auto request_weights = [&](int item, int s, int slot) {
    const int kk = s == S - 1 ? steps_of_last : 8, strip_bytes = kk * 128 + 64 * (kk * 16 / min(G, kk * 16));
    const uint8_t* src = a.w + r.expert[item] * a.expert_bytes + (strip >> 3) * a.block_bytes +
                         static_cast<int64_t>(s) * (8 * (1024 + 64 * kMaxNg)) + (strip & 7) * strip_bytes;
    copy_warp(ring + slot * a.slot_bytes + kHBytes, src, strip_bytes, lane);
  };
  const auto request_h = [&](int item, int s, int slot) {  // every lane copies what it will read
    const int p = r.pair[item][lane >> 3], part = (lane >> 2) & 1, chunks = s == S - 1 ? steps_of_last / 4 : 2;
    if (p < 0) return;
    const uint16_t* src = a.h + (static_cast<size_t>(p) * 2 + part) * a.f + s * kStageCols + (lane & 3) * 16;
    for (int c = 0; c < chunks; ++c)
#pragma unroll
      for (int v = 0; v < 2; ++v)
        cp_async_16(ring + slot * a.slot_bytes + (2 * c + v) * 512 + lane * 16, src + c * 64 + v * 8);
  };
  const auto advance = [&](int& item, int& s, int& slot) {
    s += W;
    if (s >= S) {
      s = my_stage;
      ++item;
    }
    if (++slot == kDepth) slot = 0;
  };
  // groups in flight: the weights of the first pieces, then their h, then both per piece
  int pi = i0, ps = my_stage, pslot = 0;
  if (my_stage >= S) pi = i1;
  {
    int item = pi, s = ps, slot = pslot;
    for (int i = 0; i < kDepth - 1 && item < i1; ++i) {
      request_weights(item, s, slot);
      advance(item, s, slot);
    }
    cp_async_commit();
    grid_dependency_wait();  // h
    for (int i = 0; i < kDepth - 1; ++i) {
      if (pi < i1) {
        request_h(pi, ps, pslot);
        advance(pi, ps, pslot);
      }
      cp_async_commit();
    }
  }
  int slot = 0;
  for (int item = i0; item < i1 && my_stage < S; ++item) {
    float tot[4] = {};
    for (int s = my_stage; s < S; s += W) {
      cp_async_wait<kDepth - 2>();
      __syncwarp();
      if (pi < i1) {
        request_weights(pi, ps, pslot);
        request_h(pi, ps, pslot);
        advance(pi, ps, pslot);
      }
      cp_async_commit();
      const int kk_n = s == S - 1 ? steps_of_last : 8, ng = kk_n * 16 / min(G, kk_n * 16), per = kk_n / ng;
      const uint32_t at = ring + slot * a.slot_bytes, wat = at + kHBytes;
      for (int j = 0; j < ng; ++j) {
        float part[4] = {}, sum[4] = {};
        for (int q = 0; q < per; q += 2) {
          const int kk = j * per + q;
          const uint4 b = lds128(at + (kk / 2) * 512 + lane * 16);
          const uint2 word = lds64(wat + 64 * ng + (kk / 4) * 512 + lane * 16 + (kk % 4) * 4);
          const uint32_t ones[4] = {kOnes<kBf16>, kOnes<kBf16>, kOnes<kBf16>, kOnes<kBf16>};
          uint32_t af[4];
          mma<kBf16>(sum, ones, b.x, b.y);
          codes<kBf16>(word.x, af);
          mma<kBf16>(part, af, b.x, b.y);
          mma<kBf16>(sum, ones, b.z, b.w);
          codes<kBf16>(word.y, af);
          mma<kBf16>(part, af, b.z, b.w);
        }
        apply_group<kBf16>(tot, part, sum, lds64(wat + (lane >> 2) * (8 * ng) + j * 8), a.affine);
      }
      __syncwarp();
      if (++slot == kDepth) slot = 0;
    }
    // columns 2 n and 2 n + 1 are token n's hi and lo
    const int p = r.pair[item][lane & 3];
    if (p >= 0) {
      float* const dst = acc + (p / a.k) * 17 + (lane >> 2);
      dst[0] = fmaf(r.w[p], tot[0] + tot[1], dst[0]);
      dst[8] = fmaf(r.w[p], tot[2] + tot[3], dst[8]);
    }
    __syncwarp();
  }
  cp_async_wait<0>();
  __syncthreads();
  constexpr int kType = kBf16 ? 1 : 0;
  const float* const all = reinterpret_cast<const float*>(smem + kWarps * kDepth * a.slot_bytes);
  for (int o = tid; o < a.T * 16; o += kThreads) {
    const int t = o >> 4, i = o & 15;
    float v = 0.f;
    for (int w = 0; w < sets * W; ++w) v += all[(w * a.T + t) * 17 + i];
    const size_t at = static_cast<size_t>(t) * a.d + strip * 16 + i;
    if (a.residual) v += from16<kType>(static_cast<const uint16_t*>(a.residual)[at]);
    static_cast<uint16_t*>(a.out)[at] = to16<kType>(v);
  }
}

constexpr int kSmemLimit = 160 * 1024;  // of dynamic shared memory: both kernels at their largest

using Kernel = void (*)(Args);
Kernel gate_up_of(int type, int g) {
  if (type == 1)
    return g == 32 ? few_gate_up_kernel<true, 32> : g == 64 ? few_gate_up_kernel<true, 64> : few_gate_up_kernel<true, 128>;
  return g == 32 ? few_gate_up_kernel<false, 32> : g == 64 ? few_gate_up_kernel<false, 64>
                                                           : few_gate_up_kernel<false, 128>;
}
Kernel down_of(int type, int g) {
  if (type == 1)
    return g == 32 ? few_down_kernel<true, 32> : g == 64 ? few_down_kernel<true, 64> : few_down_kernel<true, 128>;
  return g == 32 ? few_down_kernel<false, 32> : g == 64 ? few_down_kernel<false, 64> : few_down_kernel<false, 128>;
}

}  // namespace

size_t few_ws_bytes(const Dims& s) { return s.T ? size_t(s.pairs()) * 2 * s.f * 2 : 16; }

cudaError_t init_few_kernels() {
  for (int type = 0; type < 2; ++type)
    for (int g : {32, 64, 128})
      for (Kernel k : {gate_up_of(type, g), down_of(type, g)}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
        if (e != cudaSuccess) return e;
      }
  return cudaSuccess;
}

cudaError_t launch_few(const Dims& s, int type, const void* x, const float* logits, const uint8_t* w_gate_up,
                       const uint8_t* w_down, const void* residual, int32_t* topk_idx, float* topk_w, void* out,
                       void* workspace, int num_sms, cudaStream_t st) {
  Args a{};
  a.x = x;
  a.logits = logits;
  a.residual = residual;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.out = out;
  a.h = static_cast<uint16_t*>(workspace);
  a.T = s.T;
  a.d = s.d;
  a.f = s.f;
  a.E = s.E;
  a.k = s.k;
  a.act = s.act;
  a.affine = s.fmt == 1;
  // gate_up
  a.w = w_gate_up;
  a.K = s.d;
  a.block_bytes = int64_t(kBlockRows) * (s.d / 2 + s.d / s.g1 * 4);
  a.expert_bytes = a.block_bytes * (s.f / 64);
  const int stages = s.d / kStageCols;
  a.stage_warps = stages >= 8 ? 8 : stages >= 4 ? 4 : 2;
  a.slot_bytes = 2 * (1024 + 64 * (kStageCols / s.g1)) + (s.T < kUpTokens ? s.T : kUpTokens) * kXRow;
  const int units = int(s.pairs()) * (s.f / 16 / (kWarps / a.stage_warps));
  cudaError_t err = launch_pdl(gate_up_of(type, s.g1), dim3(units < num_sms ? units : num_sms), dim3(kThreads),
                               size_t(kWarps) * kDepth * a.slot_bytes, st, a);
  if (err != cudaSuccess) return err;
  // down
  a.w = w_down;
  a.K = s.f;
  a.block_bytes = int64_t(kBlockRows) * (s.f / 2 + s.f / s.g2 * 4);
  a.expert_bytes = a.block_bytes * (s.d / kBlockRows);
  a.stage_warps = kWarps / 2;
  a.slot_bytes = 1024 + 64 * (kStageCols / s.g2) + kHBytes;
  return launch_pdl(down_of(type, s.g2), dim3(s.d / 16), dim3(kThreads),
                    size_t(kWarps) * (kDepth * a.slot_bytes + s.T * 17 * 4), st, a);
}

}  // namespace moe
