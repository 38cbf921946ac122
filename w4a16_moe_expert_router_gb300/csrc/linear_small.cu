// linear_small.cu -- the forward product for a handful of rows (single tokens and small
// batches of them).
//
// With at most kSmallRows rows the weights' way from memory is all that counts (2 bytes
// per weight for 2 R operations), and tiles of 256 outputs would leave most SMs without
// one (16 rows, 2048 x 4096: 8.0 us by tiles, 6.8 us here, 2.5 us at the copy rate).  An item
// of work is 16 rows of the weight (of a gated one 8 of the gate and the 8 of the up product
// with the same outputs).  One thread of a CTA streams its items by TMA through a ring of
// chunks in shared memory, up to 192 KB per SM; eight warps deal a chunk's blocks of 32
// columns among them and multiply with m16n8k16 instructions (leaving the products out
// changes nothing).  The instructions' order of k is free as long as both operands share it,
// so eight contiguous values of a lane are its four pairs of two instructions.  x comes from
// L2 into registers a chunk ahead; at 16 rows it is as many bytes as the weights, which is
// why more rows go by tiles (and 16 of a large weight: is_small_linear).  The warps' fp32
// sums meet in shared memory in order.  With experts an item's rows are one expert's.
//
// Two CTAs per SM walk the items, the next item's chunks on their way while one ends (1 row,
// 4096 x 8192: 15.3 -> 13.5 us; 16 rows of 128 experts, 2048 x 704 gated: 21.9 -> 19.4, each
// an item of its own before).  Fewer items with long rows are shared by the CTAs of a cluster,
// a part of the columns each, whose sums go to the first one and are added in order (1 row,
// 4096 x 128: 3.9 -> 2.5 us; 8192 x 2048: 10.3 -> 8.7).
#include <algorithm>

#include "activation.cuh"
#include "internal.h"
#include "row_vec.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kChunk = 1024;                      // columns per chunk
constexpr int kBox = 256;                          // columns per TMA box
constexpr int kRowBytes = kBox * 2;
constexpr int kChunkBytes = 16 * kChunk * 2;
constexpr int kStages = 3;
constexpr int kBlocks = kChunk / 32 / kWarps;     // blocks of 32 columns per warp and chunk
constexpr int kMaxSplit = 8;                      // CTAs that share an item
static_assert(kMaxExperts <= kThreads, "one thread per expert");

// Shared memory behind the ring.
template <int kTiles>
struct Tail {
  static constexpr int values = 8 * kTiles * 16;  // of an item
  float sums[kWarps][8 * kTiles][17];             // the warps'
  float parts[kMaxSplit - 1][values];             // the other CTAs' of a cluster
  float total[values];
  uint64_t full[kStages], got;
  int expert[kSmallRows], first[kSmallRows], end[kSmallRows], counts[kWarps];  // experts with rows
};
template <int kTiles>
constexpr int kSmem = kStages * kChunkBytes + static_cast<int>(sizeof(Tail<kTiles>));  // two CTAs per SM

// D += A B, A 16 x 16, B 16 x 8, fp32 sums.
template <int kType>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (kType == 0)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kTiles: tiles of 8 rows of x.  split: CTAs of a cluster that share an item.
template <int kType, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) linear_small_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                   const int32_t* offsets, const uint4* x,
                                                                   const float* bias,
                                                                   const uint16_t* residual, uint16_t* out,
                                                                   uint16_t* preact, int32_t* err, int R, int E, int K,
                                                                   int N, int gated, int act, int split) {
  extern __shared__ __align__(128) uint8_t ring[];
  auto& sm = *reinterpret_cast<Tail<kTiles>*>(ring + kStages * kChunkBytes);
  const uint32_t full = smem_addr(sm.full), got = smem_addr(&sm.got);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int part = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  grid_dependents_launch();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, 1);
    mbar_init(got, 1);
    if (split > 1) mbar_arrive_expect_tx(got, (split - 1) * sizeof(sm.total));
    fence_barrier_init();
  }
  const int Nw = gated ? 2 * N : N, nvec = K / 8, chunks = (K + kChunk - 1) / kChunk;
  const int per_item = gated ? 8 : 16, blocks = (N + per_item - 1) / per_item;  // N is a multiple of 8
  int item = blockIdx.x, step = gridDim.x, chunk0 = 0, len = chunks, e = 0, r0 = 0, rows = R;
  if (split > 1) {
    item /= split;
    step /= split;
    chunk0 = part * chunks / split;
    len = (part + 1) * chunks / split - chunk0;
  }
  __syncthreads();
  if (split > 1) cluster_sync();  // the first CTA's barrier is initialised
  grid_dependency_wait();
  int experts = 0;
  if (offsets) {
    // the same list in every CTA, in the order of the experts
    const int lo = tid < E ? offsets[tid] : 0, hi = tid < E ? min(offsets[tid + 1], R) : 0;
    const bool some = lo >= 0 && lo < hi;
    const unsigned those = __ballot_sync(0xffffffffu, some);
    if (lane == 0) sm.counts[warp] = __popc(those);
    __syncthreads();
    int k = __popc(those & ((1u << lane) - 1u));
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) k += sm.counts[w];
      experts += sm.counts[w];
    }
    if (some && k < kSmallRows) {
      sm.expert[k] = tid;
      sm.first[k] = lo;
      sm.end[k] = hi;
    }
    experts = min(experts, kSmallRows);
    __syncthreads();
  }
  const int items = offsets ? experts * blocks : blocks;
  // the next chunk to fetch, by one thread; zeros past the last column and row
  int fetch_item = item, fetch_chunk = 0, fetched = 0;
  const auto fetch = [&] {
    if (fetch_item >= items) return;
    const int s = fetched++ % kStages, k = offsets ? fetch_item / blocks : 0, n0 = (fetch_item - k * blocks) * per_item;
    mbar_arrive_expect_tx(full + 8 * s, kChunkBytes);
#pragma unroll
    for (int c = 0; c < kChunk / kBox; ++c)
      tma_load_5d_single(smem_addr(ring + s * kChunkBytes) + c * 16 * kRowBytes, &map_w,
                         (chunk0 + fetch_chunk) * kChunk + c * kBox, 0, 0, n0 >> 3, offsets ? sm.expert[k] : 0,
                         full + 8 * s);
    if (++fetch_chunk == len) {
      fetch_chunk = 0;
      fetch_item += step;
    }
  };
  const bool fetcher = warp == 0 && elect_one();
  if (fetcher)
    for (int i = 0; i < kStages; ++i) fetch();
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 vx[kBlocks][kTiles], vy[kBlocks][kTiles];  // a chunk's x, loaded a chunk ahead
  const auto load_x = [&](int i, uint4(&v)[kBlocks][kTiles]) {
    const uint4* const xr = x + static_cast<size_t>(r0) * nvec;
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int c = (chunk0 + i) * (kChunk / 8) + 4 * (warp + u * kWarps) + q;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int r = 8 * t + g;
        v[u][t] = r < rows && c < nvec ? xr[static_cast<size_t>(r) * nvec + c] : zero;
      }
    }
  };
  float acc[kTiles][4];
  int used = 0;  // chunks so far
  // the next chunk on its x `v`; false when a wait ran out
  const auto chunk = [&](const uint4(&v)[kBlocks][kTiles]) {
    const int s = used % kStages;
    const bool ok = stage_wait_warp(full + 8 * s, (used / kStages) & 1, err);
    ++used;
    const uint8_t* const stage = ring + s * kChunkBytes;
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int c = 4 * (warp + u * kWarps) + q;  // 16-byte pieces of the chunk, 32 to a box
      const uint8_t* const p = stage + (c >> 5) * 16 * kRowBytes + g * kRowBytes + (c & 31) * 16;
      const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 8 * kRowBytes);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        mma_16816<kType>(acc[t], a.x, b.x, a.y, b.y, v[u][t].x, v[u][t].y);
        mma_16816<kType>(acc[t], a.z, b.z, a.w, b.w, v[u][t].z, v[u][t].w);
      }
    }
    if (!__syncthreads_and(ok)) {  // (the chunk is read)
      // a wait ran out and is recorded: the copies in flight land, that chunk's among them, and the
      // outputs are invalid
      if (fetcher)
        for (int k = used - 1; k < fetched; ++k) mbar_wait(full + 8 * (k % kStages), (k / kStages) & 1, err);
      if (split > 1 && part == 0) mbar_wait(got, 0, err);
      return false;
    }
    if (fetcher) fetch();
    return true;
  };
  const auto rows_of = [&](int item) {
    if (!offsets) return;
    const int k = item / blocks;
    e = sm.expert[k];
    r0 = sm.first[k];
    rows = sm.end[k] - r0;
  };
  if (item < items) {
    rows_of(item);
    load_x(0, vx);
  }
  for (; item < items; item += step) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
    for (int i = 0; i < len; i += 2) {  // the two arrays in turn: a copy would wait for the loads
      if (i + 1 < len) load_x(i + 1, vy);
      if (!chunk(vx)) return;
      if (i + 1 >= len) break;
      if (i + 2 < len) load_x(i + 2, vx);
      if (!chunk(vy)) return;
    }
    const int n0 = (offsets ? item % blocks : item) * per_item, at_e = e, at_r0 = r0, at_rows = rows;
    if (item + step < items) {
      rows_of(item + step);
      load_x(0, vx);
    }
    // a thread holds rows g and g + 8 of the weight at rows 8 t + 2 q and 8 t + 2 q + 1 of x
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) sm.sums[warp][8 * t + 2 * q + (i & 1)][g + 8 * (i >> 1)] = acc[t][i];
    __syncthreads();
    const auto warps = [&](int r, int m) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += sm.sums[k][r][m];
      return v;
    };
    if (split > 1) {  // (one item to a cluster)
      if (tid < Tail<kTiles>::values) {
        float v = warps(tid >> 4, tid & 15);
        if (part > 0) {
          store_async_4(cluster_addr(smem_addr(&sm.parts[part - 1][tid]), 0), v, cluster_addr(got, 0));
        } else {
          // a wait that ran out is recorded; sums that are still on their way land before the CTA goes
          if (!mbar_wait<true>(got, 0, err)) mbar_wait<true>(got, 0, err);
          for (int k = 0; k < split - 1; ++k) v += sm.parts[k][tid];
          sm.total[tid] = v;
        }
      }
      if (part > 0) return;
      __syncthreads();
    }
    const int width = per_item;
    for (int i = tid; i < 8 * kTiles * width; i += kThreads) {
      const int r = gated ? i >> 3 : i >> 4, m = i & (width - 1), n = n0 + m;
      if (r >= at_rows || n >= N) continue;
      const auto total = [&](int at, int col) {
        const float v = split > 1 ? sm.total[r * 16 + at] : warps(r, at);
        return v + (bias ? bias[static_cast<size_t>(at_e) * Nw + col] : 0.f);
      };
      const size_t row = static_cast<size_t>(at_r0 + r);
      const float z = total(m, n);
      float y = activate(z, act);
      if (preact) preact[row * Nw + n] = to16<kType>(z);
      if (gated) {
        const float u = total(m + 8, N + n);
        if (preact) preact[row * Nw + N + n] = to16<kType>(u);
        y *= u;
      }
      if (residual) y += from16<kType>(residual[row * N + n]);
      out[row * N + n] = to16<kType>(y);
    }
  }
}

template <int kType>
cudaError_t launch_type(const LinearDims& s, const int32_t* offsets, const void* x, const void* w, const float* bias,
                        const void* residual, void* out, void* preact, int32_t* err, int num_sms, cudaStream_t st) {
  const int per_item = s.gated ? 8 : 16, chunks = (s.K + kChunk - 1) / kChunk;
  const int64_t items = int64_t((s.N + per_item - 1) / per_item) * (offsets ? s.R : 1);
  // CTAs share an item where all of them run at a time
  int split = 1;
  while (2 * split <= kMaxSplit && 2 * split <= chunks && 2 * split * items <= 2 * num_sms) split *= 2;
  const int ctas = static_cast<int>(std::min<int64_t>(items, 2 * num_sms / split)) * split;
  // rows in blocks of 8, a gated weight's gate and up blocks in turn
  const int64_t K = s.K, dims[5] = {K, 8, s.gated ? 2 : 1, s.N / 8, s.E}, strides[4] = {K, s.N * K, 8 * K, s.Nw() * K};
  const int box[5] = {kBox, 8, s.gated ? 2 : 1, s.gated ? 1 : 2, 1};
  CUtensorMap map;
  if (!make_map(&map, kType == 1, w, 5, dims, strides, box, false)) return cudaErrorInvalidValue;
  const auto go = [&](auto kernel, int smem) {
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, map, offsets, static_cast<const uint4*>(x), bias,
                              static_cast<const uint16_t*>(residual), static_cast<uint16_t*>(out),
                              static_cast<uint16_t*>(preact), err, s.R, s.E, s.K, s.N, s.gated, s.act, split);
  };
  static_assert(kSmallRows == 16, "two tiles of 8 rows at most");
  return s.R <= 8 ? go(linear_small_kernel<kType, 1>, kSmem<1>) : go(linear_small_kernel<kType, 2>, kSmem<2>);
}

template <int kType>
cudaError_t init_type() {
  const cudaError_t err = cudaFuncSetAttribute(linear_small_kernel<kType, 1>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<1>);
  return err != cudaSuccess ? err
                            : cudaFuncSetAttribute(linear_small_kernel<kType, 2>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<2>);
}

}  // namespace

cudaError_t init_linear_small_kernels() {
  const cudaError_t err = init_type<0>();
  return err == cudaSuccess ? init_type<1>() : err;
}

// Rows that go by this kernel.  A weight of 32 MB or more with 2^16 outputs in all goes by tiles, which
// read x less often (16 rows, 4096 x 4096: 10.8 us here, 10.3 by tiles; 8 rows, 4096 x 8192: 15.6 and
// 15.0; 16 rows, 8192 x 2048: 10.9 and 11.7).
bool is_small_linear(const LinearDims& s) {
  return s.R <= kSmallRows &&
         (s.grouped || int64_t(s.R) * s.N < (1 << 16) || int64_t(s.K) * s.Nw() < (1 << 24));
}

cudaError_t launch_linear_small(const LinearDims& s, const int32_t* offsets, const void* x, const void* w,
                                const float* bias, const void* residual, void* out, void* preact, int32_t* err,
                                int num_sms, cudaStream_t st) {
  return s.type == 1 ? launch_type<1>(s, offsets, x, w, bias, residual, out, preact, err, num_sms, st)
                     : launch_type<0>(s, offsets, x, w, bias, residual, out, preact, err, num_sms, st);
}

}  // namespace moe
