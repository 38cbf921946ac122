// few.cu -- the whole W4A16 layer for a few tokens (at most kFewTokens), from the router's logits
// to the output, in two launches: gate_up with the activation, then down with the weighted sum.
//
//   a = Wgu x,  h = gelu(a_gate) a_up,  out[t] = residual[t] + sum over the token's experts of w (Wd h)
//
// A few tokens meet almost as many experts as they have choices, and an expert's weights are used
// for one or two of them: the time is the way of the chosen experts' weights from memory (19 MB for
// one token of top-8, d 2048, f 704: 2.9 us), and, for one token, what is not hidden behind it. So
//  - every CTA forms the routing itself, instead of a launch for it;
//  - with few items (an expert and at most four of its tokens) the down launch starts while the gate_up launch
//    runs, forms the routing too and requests its first weights before it waits for h (with more its shared
//    memory does not fit beside the other's, or its warps there are too few; it gets the lists then);
//  - the contraction is shared by the warps of a CTA (gate_up) or by the CTAs of a cluster (down);
//    each warp streams its own stages with cp.async, some ahead, also across work items.
// Measured in a replayed graph over the weights of as many layers as exceed L2: 1 token 14.1 us (1.4 TB/s), 4 tokens of
// bf16 34.2 (2.0), 16 tokens 62.1 (3.2); one layer's again and again, from L2, 13.7, 32.1 and 62.7.
// One token is bound by the chain routing 2.0 us, first weights 2.3, products 2, the way to the down
// launch 0.9, its h, products and sums 3.5. Sixteen are bound by the latency of the chain from a stage's arrival over its
// loads from shared memory, the unpacking and the matrix instructions to the groups' scales, which four warps a scheduler
// do not hide (issue slots 42 and 39 %, memory at half its rate), and by the parts in which no weights move: routing 3.8,
// the lists' way 1.5, both ends' sums 4.
//
// The weights stay integers: a group's codes are multiplied as they are (exact products, summed in the fp32
// accumulators to 2^-23 of a group's sum), then scale and zero-point are applied to the group's sum,
//   sum_k w_k x_k = s sum_k q_k x_k + c sum_k x_k,   c = -s z (affine: the bias).
// The sums of x come from one more matrix instruction with ones for two or four strips, the sums of h
// from the gate_up launch. h is kept as two 16-bit values, h = hi + lo, which take two columns of
// one instruction (four tokens per instruction, not eight): 22 bits of h for fp16 (or 2^-25), 16 for bf16. Every
// sum has an order of its own (stages, then warps or CTAs in their order; a token's experts in rank
// order), so the result does not depend on the other tokens and is the same in every run.
#include <algorithm>
#include <cmath>

#include "activation.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"
#include "tcgen05.cuh"
#include "topk.cuh"

namespace moe {
namespace {

constexpr int kMaxItems = kFewTokens * kMaxTopK;  // as many as pairs
constexpr int kItemTokens = 4;                    // tokens of an item
constexpr int kUpThreads = 512, kUpWarps = kUpThreads / 32;
constexpr int kDownWarps = 24;                    // down: warps of a CTA at most, and where one of gate_up is beside it
constexpr int kDownBeside = 12;
constexpr int kDownMaxPairs = 4;                  // down: pairs of strips of a CTA
constexpr int kPairBytes = 512;                   // a pair's h of one stage: (hi, lo) x 128 columns
constexpr int kRowWords = 33;                     // down: a pair's 32 rows of two strips, and one word between pairs

struct Args {
  const void* x;
  const float* logits;
  const uint8_t* w;       // this launch's projection
  const void* residual;
  int32_t* topk_idx;
  float* topk_w;
  void* out;
  uint8_t* h;             // [stages][pairs][kPairBytes], as the down launch holds it
  float* hsum;            // [stages][pairs][16]: sums of eight columns of h, in the partial sums' units
  void* routing;          // the lists, for a down launch that does not form them
  int listed;
  int T, d, f, E, k, act, affine;
  int K;                  // contraction: d or f
  uint32_t expert16;      // 16-byte pieces of an expert's weights
  uint32_t block16;       // and of a block of 128 rows
  int stage_warps;        // gate_up: warps of a group, which share a unit's contraction
  int per_item;           // gate_up: units of an item
  float per_item_inv;
  int step_items[2], step_rest[2];  // and how far the units of all groups are, of small groups and of large ones
  float turn_inv;         // gate_up: one over the units of all small groups
  int tail;               // gate_up: turns of large groups that take less than one of small ones
  int strips, cluster;    // down: strips of a CTA, CTAs that share the contraction and the items
  int stage_ranks, parts; // of them: for the stages, and for each the items
  int down_warps;         // down: warps per pair of strips, which take the items in turn
  int depth;              // down: pieces of a warp in its ring
};

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Routing and items, formed by every CTA.
struct alignas(16) Routing {
  int32_t sel[kMaxItems];
  float w[kMaxItems];                     // a pair's value, then its weight
  uint32_t mask[kMaxExperts];             // tokens of an expert
  int32_t base[kMaxExperts];              // first item of an expert
  int16_t pair[kMaxItems][kItemTokens];   // pairs of an item and their tokens; pair and token 0 behind them
  uint8_t token[kMaxItems][kItemTokens];
  uint8_t expert[kMaxItems];              // expert of an item
  uint8_t count[kMaxItems];               // its tokens
  uint8_t item[kMaxItems];                // item of a pair
  int32_t items;
};

__device__ __forceinline__ float key_value(uint32_t key) {  // the value of an order_key
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The choice of one token by one warp, as topk_softmax_warp makes it: the largest logits, ties to the
// lower expert; w gets their values. Lane l holds experts l + 32 j. Without kTies every lane that holds the
// largest key takes it for its own, which saves the vote on who does; false where two did.
template <int NS, bool kTies>
__device__ __forceinline__ bool choose(const float* row, int E, int k, int lane, int32_t* sel, float* w) {
  uint32_t key[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) key[j] = lane + 32 * j < E ? order_key(__ldcg(row + lane + 32 * j)) : 0u;
  int taken = 0;
#pragma unroll 1
  for (int r = 0; r < k; ++r) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < NS; ++j) best = max(best, key[j]);
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    int first = 0;  // the lane's first expert of that key
#pragma unroll
    for (int j = NS - 1; j >= 0; --j)
      if (key[j] == top) first = j;
    const int e = lane + 32 * first;
    bool mine = best == top;
    if (kTies) mine = __reduce_min_sync(0xffffffffu, mine ? static_cast<uint32_t>(e) : ~0u) == static_cast<uint32_t>(e);
    if (mine) {
      sel[r] = e;
      w[r] = key_value(top);
      ++taken;
    }
#pragma unroll
    for (int j = 0; j < NS; ++j)
      if (mine && j == first) key[j] = 0u;
  }
  __syncwarp();
  return kTies || __reduce_add_sync(0xffffffffu, taken) == k;
}
template <int NS>
__device__ __forceinline__ void choose(const float* row, int E, int k, int lane, int32_t* sel, float* w) {
  if (!choose<NS, false>(row, E, k, lane, sel, w)) choose<NS, true>(row, E, k, lane, sel, w);
}

// The softmax over the k chosen values of a token, summed in rank order, by one warp.
__device__ __forceinline__ void weigh(float* w, int k, int lane) {
  __syncwarp();
  const float v = lane < k ? expf(w[lane] - w[0]) : 0.f;
  __syncwarp();
  if (lane < k) w[lane] = v;
  __syncwarp();
  float den = 0.f;
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r)
    if (r < k) den += w[r];
  __syncwarp();
  if (lane < k) w[lane] = v / den;
  __syncwarp();
}

// The choice of a single token by the CTA: an expert's rank is the number of keys that are not below its own,
// counted by the threads of the expert, each over a part of the keys (1.0 us, where eight rounds of a
// warp take 1.8; a layer of top-8 of 128 takes 9.0 us by rounds and 8.7 so, one of top-2 of 16 7.4 and 8.0; the work
// grows with the square of the experts, and two to four tokens lose 1 us to it).
// Tied keys leave a rank open: false. keys: two words per expert, padded to 128 or 256.
__device__ __forceinline__ bool choose_by_rank(Routing& r, const Args& a, uint32_t* keys) {
  const int tid = threadIdx.x, n = blockDim.x, shift = a.E > 128 ? 8 : 7, E = 1 << shift;
  uint32_t* const rank = keys + E;
  for (int e = tid; e < E; e += n) {
    keys[e] = e < a.E ? order_key(__ldcg(a.logits + e)) : 0u;  // below every real key
    rank[e] = 0u;
  }
  if (tid < kMaxTopK) r.sel[tid] = -1;
  __syncthreads();
  const int parts = n >> shift, part = tid >> shift, e = tid & (E - 1);
  const int chunk = ((E + parts - 1) / parts + 3) & ~3, j0 = part * chunk, j1 = min(E, j0 + chunk);
  if (part < parts) {
    const uint32_t mine = keys[e];
    int count = 0;
#pragma unroll 8
    for (int j = j0; j < j1; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + j);
      count += (v.x >= mine) + (v.y >= mine) + (v.z >= mine) + (v.w >= mine);
    }
    atomicAdd(rank + e, static_cast<uint32_t>(count));
  }
  __syncthreads();
  for (int i = tid; i < a.E; i += n) {
    const int at = static_cast<int>(rank[i]) - 1;
    if (at < a.k) {
      r.sel[at] = i;
      r.w[at] = key_value(keys[i]);
    }
  }
  __syncthreads();
  const int lane = tid & 31;
  const bool open = __any_sync(0xffffffffu, lane < a.k && r.sel[lane] < 0);
  if (open) __syncthreads();  // all warps have found it open before one of them makes the choice anew
  return !open;               // the same in every warp
}

// Lists the items (in any order that the choices alone decide); a pair's w is its value (weigh() follows).
// What a warp reads of it afterwards is there (each wrote it, or a barrier came last). scratch: kScratchBytes of
// free shared memory.
constexpr int kScratchBytes = 2 * kMaxExperts * 4;
__device__ __forceinline__ void form_routing(Routing& r, const Args& a, uint8_t* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = blockDim.x, pairs = a.T * a.k;
  if (a.T == 1) {
    if (a.k < 5 || n < (a.E > 128 ? 256 : 128) || !choose_by_rank(r, a, reinterpret_cast<uint32_t*>(scratch))) {
      if (warp == 0 && a.E <= 128) choose<4>(a.logits, a.E, a.k, lane, r.sel, r.w);
      if (warp == 0 && a.E > 128) choose<8>(a.logits, a.E, a.k, lane, r.sel, r.w);
      __syncthreads();
    }
    // every choice is an item; its place is the number of those that come before it (the same in every warp)
    const int e = lane < a.k ? r.sel[lane] : 0;
    int at = 0;
#pragma unroll
    for (int q = 0; q < kMaxTopK; ++q)
      if (q < a.k) at += r.sel[q] < e;
    if (lane < a.k) {
      r.item[lane] = static_cast<uint8_t>(at);
      *reinterpret_cast<uint2*>(r.pair[at]) = make_uint2(lane, 0u);
      *reinterpret_cast<uint32_t*>(r.token[at]) = 0u;
      r.expert[at] = static_cast<uint8_t>(e);
      r.count[at] = 1;
    }
    r.items = a.k;
    __syncthreads();
    return;
  }
  const auto choose_all = [&] {
#pragma unroll 1
    for (int t = warp; t < a.T; t += n >> 5) {
      const float* const row = a.logits + static_cast<size_t>(t) * a.E;
      if (a.E <= 128)
        choose<4>(row, a.E, a.k, lane, r.sel + t * a.k, r.w + t * a.k);
      else
        choose<8>(row, a.E, a.k, lane, r.sel + t * a.k, r.w + t * a.k);
      __syncwarp();
      if (a.T > kItemTokens && lane < a.k) atomicOr(&r.mask[r.sel[t * a.k + lane]], 1u << t);
    }
    __syncthreads();
  };
  if (a.T <= kItemTokens) {
    // An expert is an item, in the order of its first pair; a pair per lane, the same in every warp.
    static_assert(kItemTokens * kMaxTopK <= 32, "a pair per lane");
    choose_all();
    const int e = lane < pairs ? r.sel[lane] : -1 - lane;
    const unsigned peers = __match_any_sync(0xffffffffu, e), earlier = (1u << lane) - 1u;
    const unsigned firsts = __ballot_sync(0xffffffffu, lane < pairs && (peers & earlier) == 0u);
    const int leader = __ffs(peers) - 1, item = __popc(firsts & ((1u << leader) - 1u));
    if (lane < pairs) r.item[lane] = static_cast<uint8_t>(item);
    if (lane < pairs && lane == leader) {
      r.expert[item] = static_cast<uint8_t>(e);
      r.count[item] = static_cast<uint8_t>(__popc(peers));
    }
#pragma unroll
    for (int j = 0; j < kItemTokens; ++j) {  // pair and token 0 behind the last one
      const int nth = __popc(peers & earlier);
      if (lane < pairs && (nth == j || (lane == leader && __popc(peers) <= j))) {
        r.pair[item][j] = nth == j ? static_cast<int16_t>(lane) : int16_t(0);
        r.token[item][j] = nth == j ? static_cast<uint8_t>(lane / a.k) : uint8_t(0);
      }
    }
    if (lane == 0) r.items = __popc(firsts);
    __syncwarp();
    return;
  }
#pragma unroll 1
  for (int i = tid; i < kMaxExperts; i += n) r.mask[i] = 0u;
#pragma unroll 1
  for (int i = tid; i < pairs; i += n) {
    reinterpret_cast<uint2*>(r.pair)[i] = make_uint2(0u, 0u);
    reinterpret_cast<uint32_t*>(r.token)[i] = 0u;
  }
  __syncthreads();
  choose_all();
  // every warp forms the same list
  constexpr int kPer = kMaxExperts / 32;  // lane l takes experts kPer l .. kPer l + 7
  int own[kPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = lane * kPer + j;
    own[j] = e < a.E ? (__popc(r.mask[e]) + kItemTokens - 1) / kItemTokens : 0;
    sum += own[j];
  }
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  int at = incl - sum;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (lane * kPer + j < a.E) r.base[lane * kPer + j] = at;
    at += own[j];
  }
  if (lane == 31) r.items = incl;
  __syncwarp();
#pragma unroll 1
  for (int p = tid; p < pairs; p += n) {
    const int t = p / a.k, e = r.sel[p];
    const uint32_t m = r.mask[e];
    const int nth = __popc(m & ((1u << t) - 1u)), item = r.base[e] + nth / kItemTokens;
    r.item[p] = static_cast<uint8_t>(item);
    r.pair[item][nth % kItemTokens] = static_cast<int16_t>(p);
    r.token[item][nth % kItemTokens] = static_cast<uint8_t>(t);
    if (nth % kItemTokens == 0) {
      r.expert[item] = static_cast<uint8_t>(e);
      r.count[item] = static_cast<uint8_t>(min(__popc(m) - nth, kItemTokens));
    }
  }
  __syncthreads();
}

// One word of codes -> an m16n8k16 A fragment of codes. A sum in the matrix pipe keeps some 24 bits below its largest
// product's exponent, which counts a subnormal's leading zeros too; what a bias takes up is lost as well. So the codes sit
// as high as their shifts allow. fp16: as subnormals, by two shifts and masks (2^-22 for rows g, 2^-18 for rows g + 8, whose
// nibbles sit four bits higher); a group's sum is off by 2^-23 of it, without the two bits by 2^-20 (one shift; 16 tokens
// 60.7 us, now 62.6). bf16, whose subnormals would fall out of fp32's range: kBias + q, the code at the mantissa's top, with
// the bias taken off the group's sum, off by 2^-23 of it; with 128 + q, at its bottom, by up to 2^-19 (a shift in four
// less; 4 tokens 31.4 us, now 31.9). A subtraction per pair of codes was a sixth of all instructions.
template <bool kBf16>
constexpr float kBias = kBf16 ? 16.f : 0.f;
template <bool kBf16>
__device__ __forceinline__ void codes(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (!kBf16) {
    const uint32_t low = w << 2, high = w >> 6;
    a[0] = low & 0x003c003cu;
    a[1] = low & 0x03c003c0u;
    a[2] = high & 0x003c003cu;
    a[3] = high & 0x03c003c0u;
  } else {
    a[0] = and_or(w << 3, 0x00780078u, 0x41804180u);
#pragma unroll
    for (int i = 1; i < 4; ++i) a[i] = and_or(w >> (4 * i - 3), 0x00780078u, 0x41804180u);
  }
}
template <bool kBf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kBf16)
    mma_bf16_16816(d, a, b0, b1);
  else
    mma_f16_16816(d, a, b0, b1);
}
// Totals and the sums of x and h are kept in the units of rows g's partial sums.
template <bool kBf16>
constexpr float kUnit = kBf16 ? 1.f : 0x1p-22f;
template <bool kBf16>
constexpr uint32_t kOne = kBf16 ? 0x3f803f80u : 0x3c003c00u;  // two of them

// A group's sums into the totals: tot += s part + (c - bias s) sum, for rows g (first two) and g + 8.
template <bool kBf16>
__device__ __forceinline__ void apply_group(float (&tot)[4], const float (&part)[4], float sum0, float sum1, uint2 sz,
                                            int affine) {
  const float2 lo = __half22float2(bits_h2(sz.x)), hi = __half22float2(bits_h2(sz.y));
  const float s_hi = kBf16 ? hi.x : hi.x * 0.0625f;
  float c_lo = affine ? lo.y : -lo.x * lo.y, c_hi = affine ? hi.y : -hi.x * hi.y;
  if (kBf16) {
    c_lo = fmaf(-kBias<kBf16>, lo.x, c_lo);
    c_hi = fmaf(-kBias<kBf16>, hi.x, c_hi);
  }
  tot[0] = fmaf(lo.x, part[0], fmaf(c_lo, sum0, tot[0]));
  tot[1] = fmaf(lo.x, part[1], fmaf(c_lo, sum1, tot[1]));
  tot[2] = fmaf(s_hi, part[2], fmaf(c_hi, sum0, tot[2]));
  tot[3] = fmaf(s_hi, part[3], fmaf(c_hi, sum1, tot[3]));
}

__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {  // of a CTA of the cluster
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(addr, rank)) : "memory");
  return v;
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
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// The warp copies kBytes (a multiple of 16) to its slot.
template <int kBytes>
__device__ __forceinline__ void copy_warp(uint32_t dst, const uint8_t* src, int lane) {
#pragma unroll
  for (int i = 0; i < kBytes; i += 512)
    if (i + 512 <= kBytes || lane * 16 < kBytes - i) cp_async_16(dst + i + lane * 16, src + i + lane * 16);
}
// Waits until at most depth - 1 of the thread's groups of copies are pending: the oldest piece is there.
constexpr int kMaxDepth = 4;
__device__ __forceinline__ void wait_piece(int depth) {
  if (depth == 4)
    cp_async_wait<3>();
  else if (depth == 3)
    cp_async_wait<2>();
  else
    cp_async_wait<1>();
}

// A stage of KK steps of two strips (`pitch` bytes apart): b holds the other operand's fragments. The chains of
// products of both strips' groups take turns (one strip after the other: 16 tokens 60.0 us, now 58.2).
template <bool kBf16, int G, int KK>
__device__ __forceinline__ void strips_stage(float (&tot)[2][4], uint32_t at, uint32_t pitch,
                                             const uint32_t (&b)[KK][2], const float (&sum)[KK * 16 / G][2], int lane,
                                             int affine) {
  constexpr int NG = KK * 16 / G, kSteps = KK / NG;
  uint4 word[2][KK / 4];
#pragma unroll
  for (int v = 0; v < KK / 4; ++v)
#pragma unroll
    for (int h = 0; h < 2; ++h) word[h][v] = lds128(at + h * pitch + 64 * NG + v * 512 + lane * 16);
  float part[2][NG][4] = {};
#pragma unroll
  for (int q = 0; q < kSteps; ++q)
#pragma unroll
    for (int j = 0; j < NG; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kk = j * kSteps + q;
        uint32_t af[4];
        codes<kBf16>(word_of(word[h][kk / 4], kk % 4), af);
        mma<kBf16>(part[h][j], af, b[kk][0], b[kk][1]);
      }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < NG; ++j)
      apply_group<kBf16>(tot[h], part[h][j], sum[j][0], sum[j][1],
                         lds64(at + h * pitch + (lane >> 2) * (8 * NG) + j * 8), affine);
}

// The byte of column c (0..127 of a stage) of a pair's h, `part` 0 hi and 1 lo: [part][chunk of 64][tq][half][step of
// two][value], value 0..3 the columns 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 of a 16-column step. The two halves
// of lo change places: a warp's reads of hi and lo then meet different banks.
__device__ __forceinline__ int h_place(int c, int part) {
  const int step = (c >> 4) & 3, r = c & 15;
  const int piece = (c >> 6) * 8 + ((r & 7) >> 1) * 2 + (step >> 1);
  return part * 256 + (piece ^ part) * 16 + (step & 1) * 8 + (r & 1) * 2 + (r >> 3) * 4;
}

// ------------------------------------------------------------------ gate_up
//
// A unit is an item and kPairs pairs of strips (16 gate and 16 up rows each). A group of 4 or 16 warps takes a
// unit, its warp w the stages w, w + 4 (16), ..; the units are dealt to all groups in turn. Sixteen warps have
// a unit soonest, four need their barriers and the epilogue less often. Their sums meet in shared
// memory, of several units before the warps finish them together (after every unit, two or four of
// sixteen warps would have work, and the others wait). Both group sizes add a strip's stages in the same
// order: stages q, q + 4, .. one after the other for q = 0..3, then the four sums in a tree.
// The fragments of x come from L1; a single token's are the same for all units and loaded once.
constexpr int kRoundStrips = 8;  // strips of a warp in a round of a group of 16; half of it for 4
// words of a warp's sums: [strip][value][token / 2][row], shifted by eight banks from warp to warp
constexpr int kRedWarp = kRoundStrips * 4 * 16 + 8;

// Fragments of x of a stage, and its sums over the groups: a product with ones, into the units of the totals (ones in
// the units of the codes, subnormals, lost ten bits of the sum, which the zero-point multiplies). With
// one pair of strips all columns are loaded (the ragged layer 17.5 -> 17.0 us), with two the ones behind an item's
// tokens are zeros (16 tokens 62.6 -> 60.0: their rows' lines cost more than the selection).
__device__ __forceinline__ void load_x(const uint32_t* row, bool on, uint32_t (&b)[8][2]) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
#pragma unroll
    for (int v = 0; v < 2; ++v) b[kk][v] = on ? row[kk * 8 + v * 4] : 0u;
}
template <bool kBf16, int NG>
__device__ __forceinline__ void sum_x(const uint32_t (&b)[8][2], float (&sum)[NG][2]) {
  const uint32_t ones[4] = {kOne<kBf16>, kOne<kBf16>, kOne<kBf16>, kOne<kBf16>};
#pragma unroll
  for (int j = 0; j < NG; ++j) {
    float part[4] = {};
#pragma unroll
    for (int q = 0; q < 8 / NG; ++q) mma<kBf16>(part, ones, b[j * (8 / NG) + q][0], b[j * (8 / NG) + q][1]);
    sum[j][0] = part[0] * kUnit<kBf16>;
    sum[j][1] = part[1] * kUnit<kBf16>;
  }
}

// Pieces of a warp in its ring: what an SM's shared memory holds.
template <int kPairs>
constexpr int kUpDepth = kPairs == 1 ? 3 : 2;

// kBeside: with half of an SM's registers, so that a CTA of the down launch fits beside it.
template <bool kBf16, int G, int kPairs, bool kBeside>
__global__ void __launch_bounds__(kUpThreads, kBeside ? 2 : 1) few_gate_up_kernel(const Args a) {
  constexpr int NG = kStageCols / G, kStripBytes = 1024 + 64 * NG, kStrips = 2 * kPairs, kSlot = kStrips * kStripBytes;
  constexpr int kType = kBf16 ? 1 : 0, kDepth = kUpDepth<kPairs>;
  extern __shared__ __align__(16) uint8_t smem[];  // rings
  __shared__ Routing r;
  __shared__ float red[kUpWarps * kRedWarp];
  // the way to the logits and x (their pages' addresses) is found while the launch before runs
  for (int i = threadIdx.x; i * 32 < a.T * a.E; i += kUpThreads) prefetch_l2(a.logits + i * 32);
  for (int i = threadIdx.x; i * 64 < a.T * a.d; i += kUpThreads)
    prefetch_l2(static_cast<const uint16_t*>(a.x) + i * 64);
  grid_dependency_wait();    // the logits, x, and h, which the call before may still read
  grid_dependents_launch();  // only now: the down launch reads logits and weights before it waits
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int S = a.K / kStageCols;
  const uint32_t ring = smem_addr(smem) + warp * kDepth * kSlot;
  const auto* const x = static_cast<const uint32_t*>(a.x) + (lane & 3);
  uint32_t b[8][2], next[8][2];  // fragments of x, loaded a piece ahead where registers allow
  float sum[NG][2];
  const bool fixed = a.T == 1 && S <= a.stage_warps;  // a warp has one stage, in groups of both sizes
  if (fixed && (warp & (a.stage_warps - 1)) < S) {
    load_x(x + (warp & (a.stage_warps - 1)) * 64, true, b);
    sum_x<kBf16, NG>(b, sum);
  }
  const auto load = [&](int i, int stage, uint32_t (&f)[8][2]) {  // columns behind the item's tokens are not used
    load_x(x + r.token[i][(lane >> 2) & 3] * (a.d / 2) + stage * 64, kPairs == 1 || (lane >> 2) < r.count[i], f);
  };
  form_routing(r, a, smem);
  const int pairs = a.T * a.k, all_units = r.items * a.per_item;
  // Small groups take whole turns of units; what is left over goes to large groups where those finish it sooner.
  int narrow = all_units;
  if (a.stage_warps == kUpWarps) {
    narrow = 0;
  } else {
    const int turns = static_cast<int>((all_units + 0.5f) * a.turn_inv);
    const int whole = turns * static_cast<int>(gridDim.x) * 4;
    if (all_units - whole <= a.tail * static_cast<int>(gridDim.x)) narrow = whole;
  }
  int slot = 0, pslot = 0;
  bool first_piece = true;
  float tot[kStrips][4] = {};
#pragma unroll 1
  for (int large = narrow == 0; large < 2; ++large) {
    const bool wide = large;  // one group of 16, else four of 4
    const int W = wide ? kUpWarps : kUpWarps / 4, my_stage = warp & (W - 1), team = wide ? 0 : warp >> 2;
    const int round = (wide ? kRoundStrips : kRoundStrips / 2) / kStrips;
    const int unit0 = blockIdx.x + (wide ? narrow : team * static_cast<int>(gridDim.x));
    const int units = wide ? all_units : narrow;
    const auto team_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(wide ? 0 : 1 + team), "r"(W * 32) : "memory"); };

    // the piece to request next: unit pu, which is unit pg of item pi
    struct Place {
      int unit, item, group;
    };
    Place put{unit0, static_cast<int>((unit0 + 0.5f) * a.per_item_inv), 0}, got;  // exact: at most 2^8 items of 2^10 units
    put.group = unit0 - put.item * a.per_item;
    got = put;
    const auto step = [&](Place& p) {
      p.unit += static_cast<int>(gridDim.x) * (wide ? 1 : 4);
      p.item += a.step_items[large];
      p.group += a.step_rest[large];
      if (p.group >= a.per_item) {
        p.group -= a.per_item;
        ++p.item;
      }
    };
    int ps = my_stage, s = my_stage, ahead = kDepth - 1, in_round = 0;
    bool first_x = true;
    Place round_place = got;
#pragma unroll 1
    while (true) {
      if (put.unit < units && ps < S) {
        const uint32_t pair = put.group * kPairs;
        const uint32_t off = r.expert[put.item] * a.expert16 + (pair >> 2) * a.block16 +
                             static_cast<uint32_t>(ps) * (8 * kStripBytes / 16) + (pair & 3) * (2 * kStripBytes / 16);
        copy_warp<kSlot>(ring + pslot * kSlot, a.w + static_cast<size_t>(off) * 16, lane);
        ps += W;
        if (ps >= S) {
          ps = my_stage;
          step(put);
        }
        if (++pslot == kDepth) pslot = 0;
      }
      cp_async_commit();
      if (ahead > 0) {
        --ahead;
        continue;
      }
      if (first_piece) {  // what others want of the routing, while the first pieces arrive
        first_piece = false;
        if (a.listed && blockIdx.x == gridDim.x - 1)
#pragma unroll 1
          for (int i = tid; i < static_cast<int>(sizeof(Routing) / 16); i += kUpThreads)
            reinterpret_cast<uint4*>(a.routing)[i] = reinterpret_cast<const uint4*>(&r)[i];
      }
      if (got.unit < units) {
        if (s < S) {  // (a warp without a stage takes part in the sums alone)
          if (!fixed) {
            if (kBeside) load(got.item, s, b);
            if (!kBeside) {
              if (first_x) load(got.item, s, next);
              first_x = false;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
#pragma unroll
                for (int v = 0; v < 2; ++v) b[kk][v] = next[kk][v];
              Place p = got;
              int st = s + W;
              if (st >= S) {
                st = my_stage;
                step(p);
              }
              if (p.unit < units) load(p.item, st, next);
            }
            sum_x<kBf16, NG>(b, sum);
          }
          cp_async_wait<kDepth - 1>();
          __syncwarp();
          const uint32_t at = ring + slot * kSlot;
#pragma unroll
          for (int h = 0; h < kStrips; h += 2) {
            float t[2][4] = {};
            strips_stage<kBf16, G, 8>(t, at + h * kStripBytes, kStripBytes, b, sum, lane, a.affine);
#pragma unroll
            for (int i = 0; i < 8; ++i) tot[h + i / 4][i % 4] += t[i / 4][i % 4];
          }
          __syncwarp();  // the slot is read before it is requested again
          if (++slot == kDepth) slot = 0;
          s += W;
          if (s < S) continue;
        }
        s = my_stage;
        if (in_round == 0) team_sync();  // the round before has been finished
        if ((lane & 3) < 2)
#pragma unroll
          for (int h = 0; h < kStrips; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              red[warp * kRedWarp + ((in_round * kStrips + h) * 4 + i) * 16 + (lane & 3) * 8 + (lane >> 2)] = tot[h][i];
#pragma unroll
        for (int h = 0; h < kStrips; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[h][i] = 0.f;
        step(got);
        ++in_round;
        if (in_round < round && got.unit < units) continue;
      } else if (in_round == 0) {
        break;
      }
      team_sync();
      // A warp takes a strip of a unit of the round, a lane a column of h for a token: the sums of the warps with
      // stages q, q + 4, .. one after the other, then over q in a tree.
      const int local = warp & (W - 1), mine = local / kStrips, h = local & (kStrips - 1);
      if (mine < in_round) {
        Place p = round_place;
#pragma unroll 1
        for (int j = 0; j < mine; ++j) step(p);
        const int i = p.item, c = lane & 7, n = lane >> 3;
        const float* const from =
            red + (warp - local) * kRedWarp + ((mine * kStrips + h) * 4 + (n & 1)) * 16 + (n >> 1) * 8 + c;
        float gate[4], up[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          gate[q] = from[q * kRedWarp];
          up[q] = from[q * kRedWarp + 32];
        }
        if (wide)
#pragma unroll
          for (int w = 4; w < kUpWarps; ++w) {
            gate[w & 3] += from[w * kRedWarp];
            up[w & 3] += from[w * kRedWarp + 32];
          }
        constexpr float kBack = 1.f / kUnit<kBf16>;
        const float g = (gate[0] + gate[1]) + (gate[2] + gate[3]), u = (up[0] + up[1]) + (up[2] + up[3]);
        const float v = activate(g * kBack, a.act) * (u * kBack);
        const uint16_t hi = to16<kType>(v), lo = to16<kType>(v - from16<kType>(hi));
        float sums = from16<kType>(hi) + from16<kType>(lo);
#pragma unroll
        for (int off = 1; off < 8; off <<= 1) sums += __shfl_xor_sync(0xffffffffu, sums, off);
        if (n < r.count[i]) {
          const int col = 16 * (p.group * kPairs) + 8 * h + c;
          const size_t at = static_cast<size_t>(col >> 7) * pairs + r.pair[i][n];
          uint8_t* const dst = a.h + at * kPairBytes;
          *reinterpret_cast<uint16_t*>(dst + h_place(col & 127, 0)) = hi;
          *reinterpret_cast<uint16_t*>(dst + h_place(col & 127, 1)) = lo;
          if (c == 0) a.hsum[at * 16 + ((col & 127) >> 3)] = sums * kUnit<kBf16>;
        }
      }
      in_round = 0;
      round_place = got;
      if (got.unit >= units) break;
    }
  }
  cp_async_wait<0>();
}

// --------------------------------------------------------------------- down
//
// A CTA takes up to 2 kDownMaxPairs strips of 16 rows and one stage of 128 columns of every item (the
// stages rank, + ranks, .. of its cluster) or, where that leaves SMs without work, of a part of the items
// (22 tokens of 512 columns, for which 32 CTAs took 8 us: 27.5 -> 24.1 us in all); down_warps warps per pair of
// strips take the items in turn. h of the stage is held for all pairs, and so are the products' rows: a
// token's are then added in its experts' rank order, whichever warp or CTA made them. At the end the cluster's
// CTAs add up their sums, each for a part of the outputs.
template <bool kBf16, int G>
__global__ void __launch_bounds__(kDownWarps * 32, 1) few_down_kernel(const Args a) {
  constexpr int kMaxNg = kStageCols / G, kStrip = 1024 + 64 * kMaxNg, kSlot = 2 * kStrip, kType = kBf16 ? 1 : 0;
  constexpr int kHalfNg = G < 64 ? 2 : 1, kHalfStrip = 512 + 64 * kHalfNg;  // a last stage of 64 columns
  // h [pairs][512] | rings | sums of h [pairs][groups of a stage] | rows [pairs of strips][pairs][33]
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Routing r;
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
  const int C = a.cluster, rank = static_cast<int>(cluster_rank()), tile = static_cast<int>(blockIdx.x) / C;
  const int S = (a.K + kStageCols - 1) / kStageCols, pairs = a.T * a.k;
  const int stage_rank = rank % a.stage_ranks, part = rank / a.stage_ranks;
  const int turn = (warp % a.down_warps) * a.parts + part, item_step = a.down_warps * a.parts;
  const int strip_pair = warp / a.down_warps, strip = tile * a.strips + strip_pair * 2;
  const uint32_t hs = smem_addr(smem), ring = hs + pairs * kPairBytes + warp * a.depth * kSlot;
  float* const hsum = reinterpret_cast<float*>(smem + pairs * kPairBytes + warps * a.depth * kSlot);
  float* const all = hsum + pairs * kMaxNg;
  float* const rows = all + strip_pair * pairs * kRowWords + (lane >> 2);
  if (a.listed) {  // it could not start beside the gate_up launch: the lists are there
    grid_dependency_wait();
#pragma unroll 1
    for (int i = tid; i < static_cast<int>(sizeof(Routing) / 16); i += threads)
      reinterpret_cast<uint4*>(&r)[i] = __ldcg(reinterpret_cast<const uint4*>(a.routing) + i);
    __syncthreads();
  } else {
    form_routing(r, a, smem);
  }
  const int items = strip * 16 >= a.d ? 0 : r.items;  // no items for strips behind the last one
  bool weighed = false;
  const auto weigh_all = [&] {  // while something is on its way
    if (!weighed)
#pragma unroll 1
      for (int t = warp; t < a.T; t += warps) {
        weigh(r.w + t * a.k, a.k, lane);
        if (blockIdx.x == 0 && lane < a.k) {
          if (a.topk_idx) a.topk_idx[t * a.k + lane] = r.sel[t * a.k + lane];
          if (a.topk_w) a.topk_w[t * a.k + lane] = r.w[t * a.k + lane];
        }
      }
    weighed = true;
  };
#pragma unroll 1
  for (int s = stage_rank; s < S; s += a.stage_ranks) {
    const bool whole = (s + 1) * kStageCols <= a.K;
    const uint8_t* const src = a.w + (static_cast<size_t>(strip >> 3) * a.block16 + s * (8 * kStrip / 16) +
                                      (strip & 7) * ((whole ? kStrip : kHalfStrip) / 16)) * 16;
    int put = turn, pslot = 0, slot = 0, item = turn, ahead = a.depth - 1;
#pragma unroll 1
    while (true) {
      if (put < items) {
        const uint8_t* const from = src + static_cast<size_t>(r.expert[put] * a.expert16) * 16;
        if (whole)
          copy_warp<kSlot>(ring + pslot * kSlot, from, lane);
        else
          copy_warp<2 * kHalfStrip>(ring + pslot * kSlot, from, lane);
        put += item_step;
        if (++pslot == a.depth) pslot = 0;
      }
      cp_async_commit();
      if (ahead > 0) {
        if (--ahead > 0) continue;
        if (!a.listed) weigh_all();
        if (s == stage_rank)
          grid_dependency_wait();  // h
        else
          __syncthreads();  // h of the stage before has been read
        const uint8_t* const h = a.h + static_cast<size_t>(s) * pairs * kPairBytes;
#pragma unroll 4
        for (int i = tid; i < pairs * (kPairBytes / 16); i += threads) cp_async_16(hs + i * 16, h + i * 16);
        cp_async_commit();
        const int ng = whole ? kMaxNg : kHalfNg, eights = (whole ? kStageCols / kMaxNg : 64 / kHalfNg) / 8;
#pragma unroll 1
        for (int i = tid; i < pairs * ng; i += threads) {
          const int p = whole ? i / kMaxNg : i / kHalfNg, j = i - p * ng;
          const float* const part = a.hsum + (static_cast<size_t>(s) * pairs + p) * 16 + j * eights;
          float v = 0.f;
#pragma unroll 4
          for (int q = 0; q < eights; q += 4) {
            const float4 f = __ldcg(reinterpret_cast<const float4*>(part + q));
            v += (f.x + f.y) + (f.z + f.w);
          }
          hsum[p * kMaxNg + j] = v;
        }
        weigh_all();
        cp_async_wait<0>();
        __syncthreads();
        continue;
      }
      if (item >= items) break;
      const int mine = r.pair[item][lane >> 3], p = r.pair[item][lane & 3];
      const uint32_t hat = hs + mine * kPairBytes + ((lane >> 2) & 1) * 256 + (lane & 3) * 32;
      uint32_t b[8][2];
#pragma unroll
      for (int kk = 0; kk < 8; kk += 2) {
        const uint4 v = lds128(hat + (kk / 4) * 128 + ((((kk / 2) & 1) ^ ((lane >> 2) & 1)) << 4));
        b[kk][0] = v.x;
        b[kk][1] = v.y;
        b[kk + 1][0] = v.z;
        b[kk + 1][1] = v.w;
      }
      float sum[kMaxNg][2];
#pragma unroll
      for (int j = 0; j < kMaxNg; ++j) {
        sum[j][0] = hsum[p * kMaxNg + j];
        sum[j][1] = 0.f;
      }
      wait_piece(a.depth);
      __syncwarp();
      const uint32_t at = ring + slot * kSlot;
      const bool on = (lane & 3) < r.count[item];
      float* const dst = rows + p * kRowWords;
      // columns 2 n and 2 n + 1 are token n's hi and lo: their sum counts, and the sum of h once
      float t[2][4] = {};
      if (whole) {
        strips_stage<kBf16, G, 8>(t, at, kStrip, b, sum, lane, a.affine);
      } else if constexpr (G <= 64) {
        const uint32_t half[4][2] = {{b[0][0], b[0][1]}, {b[1][0], b[1][1]}, {b[2][0], b[2][1]}, {b[3][0], b[3][1]}};
        float part[64 / G][2];
#pragma unroll
        for (int j = 0; j < 64 / G; ++j) {
          part[j][0] = sum[j][0];
          part[j][1] = 0.f;
        }
        strips_stage<kBf16, G, 4>(t, at, kHalfStrip, half, part, lane, a.affine);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (on) {  // (stages of the CTA after its first are added to it)
          const float lo = t[h][0] + t[h][1], hi = t[h][2] + t[h][3];
          dst[16 * h] = s == stage_rank ? lo : dst[16 * h] + lo;
          dst[16 * h + 8] = s == stage_rank ? hi : dst[16 * h + 8] + hi;
        }
      }
      __syncwarp();
      if (++slot == a.depth) slot = 0;
      item += item_step;
    }
    cp_async_wait<0>();
  }
  __syncthreads();
  // a token's rows over its experts in rank order, into its first pair's place: 32 columns by a warp
  const int strip_pairs = a.strips / 2;
#pragma unroll 1
  for (int o = warp; o < a.T * strip_pairs && a.parts == 1; o += warps) {
    const int t = o / strip_pairs, g = o - t * strip_pairs;
    float* const at = all + (g * pairs + t * a.k) * kRowWords + lane;
    float part[kMaxTopK], v = 0.f;
#pragma unroll
    for (int q = 0; q < kMaxTopK; ++q) part[q] = q < a.k ? at[q * kRowWords] : 0.f;
#pragma unroll
    for (int q = 0; q < kMaxTopK; ++q)
      if (q < a.k) v = fmaf(r.w[t * a.k + q], part[q], v);
    at[0] = v;
  }
  if (C > 1)
    cluster_sync();
  else
    __syncthreads();
  // (token, pair of strips) by a warp of the cluster
  const int cols = a.strips * 16;
#pragma unroll 1
  for (int o = rank * warps + warp; o < a.T * strip_pairs; o += C * warps) {
    const int t = o / strip_pairs, g = o - t * strip_pairs, col = tile * cols + g * 32 + lane;
    if (col >= a.d) continue;
    const uint32_t at = smem_addr(all + (g * pairs + t * a.k) * kRowWords + lane);
    float sum[8];  // of the stages of a rank
    if (a.parts == 1) {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        sum[q] = 0.f;
        if (q < C) sum[q] = ld_cluster(at, q);
      }
    } else {  // the same sums, from the CTAs that have a pair's item
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[c] = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < a.stage_ranks) {
          float part[kMaxTopK];
#pragma unroll
          for (int q = 0; q < kMaxTopK; ++q)
            if (q < a.k)
              part[q] = ld_cluster(at + q * kRowWords * 4, c + r.item[t * a.k + q] % a.parts * a.stage_ranks);
#pragma unroll
          for (int q = 0; q < kMaxTopK; ++q)
            if (q < a.k) sum[c] = fmaf(r.w[t * a.k + q], part[q], sum[c]);
        }
    }
    float v = sum[0];
#pragma unroll
    for (int q = 1; q < 8; ++q)
      if (q < a.stage_ranks) v += sum[q];
    v *= 1.f / kUnit<kBf16>;
    const size_t dst = static_cast<size_t>(t) * a.d + col;
    if (a.residual) v += from16<kType>(static_cast<const uint16_t*>(a.residual)[dst]);
    static_cast<uint16_t*>(a.out)[dst] = to16<kType>(v);
  }
  if (C > 1) cluster_sync();  // the sums are read before their CTA leaves
}

constexpr int kSmemLimit = 226 * 1024;  // of a CTA, static and dynamic
constexpr int kUpStatic = sizeof(Routing) + kUpWarps * kRedWarp * 4 + 64;
constexpr int kDownStatic = sizeof(Routing) + 64;
static_assert(kUpDepth<2> * 2 * kUpWarps * 2 * (1024 + 64 * 4) <= kSmemLimit - kUpStatic, "groups of 32");
static_assert(kScratchBytes <= 2 * 2 * 1088, "the smallest rings hold what the choice of one token takes");

using Kernel = void (*)(Args);
template <bool kBf16, int kPairs, bool kBeside>
Kernel gate_up_of(int g) {
  if (g == 32) return few_gate_up_kernel<kBf16, 32, kPairs, kBeside>;
  return g == 64 ? few_gate_up_kernel<kBf16, 64, kPairs, kBeside> : few_gate_up_kernel<kBf16, 128, kPairs, kBeside>;
}
template <bool kBf16>
Kernel gate_up_of(int g, int pairs, bool beside) {
  if (beside) return gate_up_of<kBf16, 1, true>(g);
  return pairs == 1 ? gate_up_of<kBf16, 1, false>(g) : gate_up_of<kBf16, 2, false>(g);
}
Kernel gate_up_of(int type, int g, int pairs, bool beside) {
  return type == 1 ? gate_up_of<true>(g, pairs, beside) : gate_up_of<false>(g, pairs, beside);
}
Kernel down_of(int type, int g) {
  if (type == 1)
    return g == 32 ? few_down_kernel<true, 32> : g == 64 ? few_down_kernel<true, 64> : few_down_kernel<true, 128>;
  return g == 32 ? few_down_kernel<false, 32> : g == 64 ? few_down_kernel<false, 64> : few_down_kernel<false, 128>;
}

struct DownLaunch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  DownLaunch(int tiles, int cluster, int threads, size_t smem, cudaStream_t st) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(tiles * cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

}  // namespace

// Workspace: routing lists | h | sums of h.
static int down_stages(const Dims& s) { return (s.f + kStageCols - 1) / kStageCols; }
size_t few_ws_bytes(const Dims& s) { return sizeof(Routing) + size_t(down_stages(s)) * s.pairs() * (kPairBytes + 64); }

// Room for the kernel's shared memory, and an SM divided for as much of it as there is: a CTA of the down launch
// that finds it divided otherwise waits until the SM is empty.
static cudaError_t set_up(Kernel k, int smem) {
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  return e;
}

cudaError_t init_few_kernels(FewClusters& clusters) {
  cudaError_t e = cudaSuccess;
  for (int type = 0; type < 2; ++type)
    for (int g : {32, 64, 128}) {
      for (Kernel k : {gate_up_of(type, g, 1, true), gate_up_of(type, g, 1, false), gate_up_of(type, g, 2, false)})
        if (e == cudaSuccess) e = set_up(k, kSmemLimit - kUpStatic);
      if (e == cudaSuccess)
        e = set_up(down_of(type, g), kSmemLimit - kDownStatic);
    }
  for (int c = 1; c <= 8 && e == cudaSuccess; ++c) {
    const DownLaunch l(1, c, 18 * 32, 128 * 1024, nullptr);
    e = cudaOccupancyMaxActiveClusters(&clusters[c], down_of(0, 64), &l.cfg);
  }
  return e;
}

cudaError_t launch_few(const Dims& s, int type, const void* x, const float* logits, const uint8_t* w_gate_up,
                       const uint8_t* w_down, const void* residual, int32_t* topk_idx, float* topk_w, void* out,
                       void* workspace, int num_sms, const FewClusters& clusters, cudaStream_t st) {
  const int pairs = int(s.pairs());
  Args a{};
  a.x = x;
  a.logits = logits;
  a.residual = residual;
  a.topk_idx = topk_idx;
  a.topk_w = topk_w;
  a.out = out;
  a.routing = workspace;
  a.h = static_cast<uint8_t*>(workspace) + sizeof(Routing);
  a.hsum = reinterpret_cast<float*>(a.h + size_t(down_stages(s)) * pairs * kPairBytes);
  a.T = s.T;
  a.d = s.d;
  a.f = s.f;
  a.E = s.E;
  a.k = s.k;
  a.act = s.act;
  a.affine = s.fmt == 1;
  // The down launch: CTAs for the stages and strips of each so that it takes least, counted in stages of two strips,
  // with 1.5 for h and 1 for the start of a wave of clusters. (10 tokens of 2048 x 1408: 79 us with a CTA per stage, of
  // which one cluster had to wait for the others, now 51.5.) The number of tokens has no part in it, so a sum's
  // order does not depend on it.
  const int strips = s.d / 16, down_count = down_stages(s);
  int rounds = 1;
  double least = 1e30;
  for (int c = 1; c <= std::min(down_count, 8); ++c) {
    const int at_a_time = std::max(clusters[c], 1), r = (down_count + c - 1) / c;
    int n = 2;
    while (n < 2 * kDownMaxPairs && (strips + n - 1) / n > at_a_time) n += 2;
    const int tiles = (strips + n - 1) / n;
    const double time = (tiles + at_a_time - 1) / at_a_time * (r * (n / 2 + 1.5) + 1);
    if (time < least) {
      least = time;
      a.stage_ranks = c;
      a.strips = n;
      rounds = r;
    }
  }
  // Where few strips and stages leave SMs without work, more CTAs share the items, as long as each of their warps has
  // one (8 tokens of top-3 lose 1.3 us to a larger cluster). Which experts meet is not known here; their number is
  // about that of evenly chosen ones. (Where they have more than four tokens, there are more items than that.)
  const double items = s.E * (1.0 - std::pow(1.0 - double(s.k) / s.E, s.T));
  a.parts = 1;
  for (int p = 2; a.strips == 2 && p <= 8 / a.stage_ranks && items >= kDownWarps * p; ++p)
    if ((strips + 1) / 2 <= clusters[a.stage_ranks * p]) a.parts = p;
  a.cluster = a.stage_ranks * a.parts;
  const int slot = 2 * (1024 + 64 * (kStageCols / s.g2)), fixed = pairs * (kPairBytes + kStageCols / s.g2 * 4);
  const auto room = [&](int limit, int warps) {  // pieces of a warp that fit
    return (limit - kDownStatic - fixed - a.strips / 2 * pairs * kRowWords * 4) / (a.strips / 2 * warps * slot);
  };
  // With few items it runs beside the gate_up launch, which hides its start; where it does not fit there, or its fewer
  // warps would have more than three pieces each, it gets the lists from the gate_up launch (2 tokens of top-8,
  // 768 x 1856: 33.0 us beside it, 24.4 after it).
  const int stages = s.d / kStageCols, piece = kUpWarps * 2 * (1024 + 64 * (kStageCols / s.g1));
  const int beside = kSmemLimit - kUpStatic - 3 * piece;
  a.listed = room(beside, 4) < 2 || items * rounds > 3 * (kDownBeside / (a.strips / 2));
  const int least_warps = kDownWarps / kDownMaxPairs, limit = a.listed ? kSmemLimit : beside;
  while (a.listed && a.strips > 2 && room(kSmemLimit, least_warps) < 2) a.strips -= 2;
  // as many warps as there are items for
  const int most = (a.listed ? kDownWarps : kDownBeside) / (a.strips / 2);
  a.down_warps = std::max(std::min(most, (pairs + a.parts - 1) / a.parts), 1);
  while (a.down_warps > 1 && room(limit, a.down_warps) < 2) --a.down_warps;
  const int down_depth = std::min(room(limit, a.down_warps), kMaxDepth);
  // gate_up: the group size and the pairs of strips per unit that take the least time, counted in pieces of one
  // pair: two pairs at once take 1.6, a unit's barriers and epilogue 1 of a small group and 0.5 of a
  // large one.
  const auto cost = [&](int w, int p) { return (stages + w - 1) / w * (p == 2 ? 1.6 : 1.0) + (w == 4 ? 1.0 : 0.5); };
  least = 1e30;
  int per_warp = 1;
  a.stage_warps = kUpWarps;
  for (int w : {kUpWarps, 4})
    for (int p : {1, 2}) {
      if ((w == 4 && stages > kUpWarps) || (p == 2 && !a.listed)) continue;  // (the sums' order; registers)
      const double turns = std::ceil(items * (s.f / 16 / p) / (num_sms * (kUpWarps / w)));
      const double time = turns * cost(w, p);
      if (time < least) {
        least = time;
        per_warp = p;
        a.stage_warps = w;
      }
    }
  a.w = w_gate_up;
  a.K = s.d;
  a.block16 = uint32_t(kBlockRows) * (s.d / 2 + s.d / s.g1 * 4) / 16;
  a.expert16 = a.block16 * (s.f / 64);
  a.per_item = s.f / 16 / per_warp;
  a.per_item_inv = 1.f / a.per_item;
  const int units = pairs * a.per_item;
  const int grid = std::min(units, num_sms);
  for (int large = 0; large < 2; ++large) {
    a.step_items[large] = grid * (large ? 1 : 4) / a.per_item;
    a.step_rest[large] = grid * (large ? 1 : 4) % a.per_item;
  }
  a.turn_inv = 1.f / (4 * grid);
  // (0.5: the gap between the two)
  a.tail = stages <= kUpWarps ? int((cost(4, per_warp) - 0.5) / cost(kUpWarps, per_warp)) : 0;
  cudaError_t err = launch_pdl(gate_up_of(type, s.g1, per_warp, !a.listed), dim3(grid), dim3(kUpThreads),
                               size_t(per_warp == 1 ? kUpDepth<1> : 2 * kUpDepth<2>) * piece, st, a);
  if (err != cudaSuccess) return err;
  a.w = w_down;
  a.K = s.f;
  a.block16 = uint32_t(kBlockRows) * (s.f / 2 + s.f / s.g2 * 4) / 16;
  a.expert16 = a.block16 * (s.d / kBlockRows);
  a.depth = down_depth;
  const int warps = a.strips / 2 * a.down_warps;
  const DownLaunch l((strips + a.strips - 1) / a.strips, a.cluster, warps * 32,
                     size_t(fixed) + warps * a.depth * slot + a.strips / 2 * pairs * kRowWords * 4, st);
  return cudaLaunchKernelEx(&l.cfg, down_of(type, s.g2), a);
}

}  // namespace moe
