// linear_small.cu -- the forward product for a handful of rows (single tokens and small
// batches of them).
//
// With at most kSmallRows rows the weights' way from memory is all that counts (2 bytes
// per weight for 2 R operations), and tiles of 256 outputs would leave most SMs without
// one (16 rows, 2048 x 4096: 9.0 us by tiles, 6.9 us here, 2.5 us at the copy rate).  A CTA
// owns 16 rows of the weight (of a gated one 8 of the gate and the 8 of the up product with
// the same outputs).  One thread streams them by TMA through a ring of chunks in shared
// memory, up to 192 KB per SM; eight warps deal a chunk's blocks of 32 columns among them
// and multiply with m16n8k16 instructions (leaving the products out changes nothing).  The
// instructions' order of k is free as long as both operands share it, so eight contiguous
// values of a lane are its four pairs of two instructions.  x comes from L2 into registers a
// chunk ahead; at 16 rows it is as many bytes as the weights (16 rows, 8192 x 2048: 14.4 us,
// 10.7 without them), which is why more rows go by tiles.  The warps' fp32 sums meet in
// shared memory in order.  With experts a CTA column serves the rows of one expert: that of
// row blockIdx.y, if it is the expert's first.
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
constexpr int kSmem = kStages * kChunkBytes + 64;  // two CTAs per SM
static_assert(kMaxExperts <= kThreads, "one thread per expert");
static_assert(kWarps * 32 * 17 * 4 <= kStages * kChunkBytes, "the warps' sums take the ring's place");

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

// kTiles: tiles of 8 rows of x.
template <int kType, int kTiles>
__global__ void __launch_bounds__(kThreads, 2) linear_small_kernel(const __grid_constant__ CUtensorMap map_w,
                                                                   const int32_t* offsets, const uint4* x,
                                                                   const float* bias,
                                                                   const uint16_t* residual, uint16_t* out,
                                                                   uint16_t* preact, int32_t* err, int R, int E, int K,
                                                                   int N, int gated, int act) {
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int found[2];
  const uint32_t full = smem_addr(ring + kStages * kChunkBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  grid_dependents_launch();
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + 8 * s, 1);
    fence_barrier_init();
    found[0] = -1;
  }
  __syncthreads();
  grid_dependency_wait();
  int e = 0, r0 = 0, rows = R;
  if (offsets) {
    const int y = blockIdx.y;
    if (tid < E) {
      const int lo = offsets[tid], hi = offsets[tid + 1];
      if (lo == y && y < hi) {  // y is its first row
        found[0] = tid;
        found[1] = hi;
      }
    }
    __syncthreads();
    e = found[0];
    if (e < 0) return;
    r0 = y;
    rows = min(found[1], R) - y;
  }
  const int Nw = gated ? 2 * N : N, nvec = K / 8, chunks = (K + kChunk - 1) / kChunk;
  const int n0 = blockIdx.x * (gated ? 8 : 16);  // N is a multiple of 8
  const auto fetch = [&](int i) {  // chunk i, by one thread; zeros past the last column and row
    const int s = i % kStages;
    mbar_arrive_expect_tx(full + 8 * s, kChunkBytes);
#pragma unroll
    for (int c = 0; c < kChunk / kBox; ++c)
      tma_load_5d_single(smem_addr(ring + s * kChunkBytes) + c * 16 * kRowBytes, &map_w, i * kChunk + c * kBox, 0, 0,
                         n0 >> 3, e, full + 8 * s);
  };
  const bool fetcher = warp == 0 && elect_one();
  if (fetcher)
    for (int i = 0; i < kStages && i < chunks; ++i) fetch(i);
  const uint4* const xr = x + static_cast<size_t>(r0) * nvec;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float acc[kTiles][4];
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
  uint4 vx[kBlocks][kTiles], vy[kBlocks][kTiles];  // a chunk's x, loaded a chunk ahead
  const auto load_x = [&](int i, uint4(&v)[kBlocks][kTiles]) {
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int c = i * (kChunk / 8) + 4 * (warp + u * kWarps) + q;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int r = 8 * t + g;
        v[u][t] = r < rows && c < nvec ? xr[static_cast<size_t>(r) * nvec + c] : zero;
      }
    }
  };
  // chunk i on its x `v`; false when a wait ran out
  const auto chunk = [&](int i, const uint4(&v)[kBlocks][kTiles]) {
    const int s = i % kStages;
    const bool ok = stage_wait_warp(full + 8 * s, (i / kStages) & 1, err);
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
      // a wait ran out and is recorded: the other copies in flight land, and the outputs are invalid
      if (fetcher)
        for (int k = i + 1; k < chunks && k < i + kStages; ++k)
          mbar_wait(full + 8 * (k % kStages), (k / kStages) & 1, err);
      return false;
    }
    if (fetcher && i + kStages < chunks) fetch(i + kStages);
    return true;
  };
  load_x(0, vx);
  for (int i = 0; i < chunks; i += 2) {  // the two arrays in turn: a copy would wait for the loads
    if (i + 1 < chunks) load_x(i + 1, vy);
    if (!chunk(i, vx) || i + 1 >= chunks) break;
    if (i + 2 < chunks) load_x(i + 2, vx);
    if (!chunk(i + 1, vy)) break;
  }
  __syncthreads();
  auto* const sums = reinterpret_cast<float(*)[8 * kTiles][17]>(ring);
  // a thread holds rows g and g + 8 of the weight at rows 8 t + 2 q and 8 t + 2 q + 1 of x
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][8 * t + 2 * q + (i & 1)][g + 8 * (i >> 1)] = acc[t][i];
  __syncthreads();
  const int width = gated ? 8 : 16;
  for (int i = tid; i < 8 * kTiles * width; i += kThreads) {
    const int r = i / width, m = i - r * width, n = n0 + m;
    if (r >= rows || n >= N) continue;
    const auto total = [&](int at, int col) {
      float s = bias ? bias[static_cast<size_t>(e) * Nw + col] : 0.f;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) v += sums[k][r][at];
      return v + s;
    };
    const size_t row = static_cast<size_t>(r0 + r);
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

template <int kType>
cudaError_t launch_type(const LinearDims& s, const int32_t* offsets, const void* x, const void* w, const float* bias,
                        const void* residual, void* out, void* preact, int32_t* err, cudaStream_t st) {
  const int per_cta = s.gated ? 8 : 16;
  const dim3 grid((s.N + per_cta - 1) / per_cta, offsets ? s.R : 1);
  // rows in blocks of 8, a gated weight's gate and up blocks in turn
  const int64_t K = s.K, dims[5] = {K, 8, s.gated ? 2 : 1, s.N / 8, s.E}, strides[4] = {K, s.N * K, 8 * K, s.Nw() * K};
  const int box[5] = {kBox, 8, s.gated ? 2 : 1, s.gated ? 1 : 2, 1};
  CUtensorMap map;
  if (!make_map(&map, kType == 1, w, 5, dims, strides, box, false)) return cudaErrorInvalidValue;
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), kSmem, st, map, offsets, static_cast<const uint4*>(x), bias,
                      static_cast<const uint16_t*>(residual),
                      static_cast<uint16_t*>(out), static_cast<uint16_t*>(preact), err, s.R, s.E, s.K, s.N, s.gated,
                      s.act);
  };
  static_assert(kSmallRows == 16, "two tiles of 8 rows at most");
  return s.R <= 8 ? go(linear_small_kernel<kType, 1>) : go(linear_small_kernel<kType, 2>);
}

template <int kType>
cudaError_t init_type() {
  for (const void* fn : {reinterpret_cast<const void*>(linear_small_kernel<kType, 1>),
                         reinterpret_cast<const void*>(linear_small_kernel<kType, 2>)}) {
    const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t init_linear_small_kernels() {
  const cudaError_t err = init_type<0>();
  return err == cudaSuccess ? init_type<1>() : err;
}

cudaError_t launch_linear_small(const LinearDims& s, const int32_t* offsets, const void* x, const void* w,
                                const float* bias, const void* residual, void* out, void* preact, int32_t* err,
                                cudaStream_t st) {
  return s.type == 1 ? launch_type<1>(s, offsets, x, w, bias, residual, out, preact, err, st)
                     : launch_type<0>(s, offsets, x, w, bias, residual, out, preact, err, st);
}

}  // namespace moe
