// linear_small.cu -- the forward product for a handful of rows (single tokens).
//
// With at most kSmallRows rows the weights' way from memory is all that counts (2 bytes
// per weight for 2 R operations), and a tensor-core tile would spend its time on setting
// up.  A warp owns two outputs (of a gated product one output: its gate and its up row)
// and reads their weight rows with 16-byte loads, several in flight per lane, each used
// for every row; the lanes' fp32 sums meet in a butterfly.  With experts a CTA column
// serves the rows of one expert: that of row blockIdx.y, if it is the expert's first.
#include "activation.cuh"
#include "internal.h"
#include "row_vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = kSmallRows;

template <int kType, int kRows>
__global__ void __launch_bounds__(kThreads) linear_small_kernel(const int32_t* offsets, const uint4* x, const uint4* w,
                                                                const float* bias, const uint16_t* residual,
                                                                uint16_t* out, uint16_t* preact, int R, int E, int K,
                                                                int N, int gated, int act) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int e = 0, r0 = 0, rows = R;
  if (offsets) {
    // the expert of row y: the only one with off[e] <= y < off[e + 1]
    __shared__ int found[2];
    const int y = blockIdx.y;
    if (threadIdx.x == 0) found[0] = -1;
    __syncthreads();
    const int i = threadIdx.x;
    if (i < E) {
      const int lo = offsets[i], hi = offsets[i + 1];
      if (lo == y && y < hi) {  // y is its first row
        found[0] = i;
        found[1] = hi;
      }
    }
    __syncthreads();
    e = found[0];
    if (e < 0) return;
    r0 = y;
    rows = min(found[1], R) - y;
  }
  const int Nw = gated ? 2 * N : N, nvec = K / 8;
  const int per_warp = gated ? 1 : 2;
  const int n0 = (blockIdx.x * (kThreads / 32) + warp) * per_warp;
  if (n0 >= N) return;  // N is even
  const int n1 = gated ? n0 + N : n0 + 1;
  const uint4* w0 = w + (static_cast<size_t>(e) * Nw + n0) * nvec;
  const uint4* w1 = w + (static_cast<size_t>(e) * Nw + n1) * nvec;
  const uint4* xr = x + static_cast<size_t>(r0) * nvec;
  float acc[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) acc[r][0] = acc[r][1] = 0.f;
#pragma unroll 4
  for (int c = lane; c < nvec; c += 32) {
    const uint4 v0 = __ldcs(w0 + c), v1 = __ldcs(w1 + c);
    float a[8], b[8];
    Vec<kType>::load(v0, a);
    Vec<kType>::load(v1, b);
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < rows) {
        float f[8];
        Vec<kType>::load(xr[static_cast<size_t>(r) * nvec + c], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc[r][0] = fmaf(a[i], f[i], acc[r][0]);
          acc[r][1] = fmaf(b[i], f[i], acc[r][1]);
        }
      }
  }
  const float b0 = bias ? bias[static_cast<size_t>(e) * Nw + n0] : 0.f;
  const float b1 = bias ? bias[static_cast<size_t>(e) * Nw + n1] : 0.f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      acc[r][0] += __shfl_xor_sync(0xffffffffu, acc[r][0], off);
      acc[r][1] += __shfl_xor_sync(0xffffffffu, acc[r][1], off);
    }
    if (r < rows && lane == 0) {
      const size_t row = static_cast<size_t>(r0 + r);
      const float z0 = acc[r][0] + b0, z1 = acc[r][1] + b1;
      if (preact) {
        preact[row * Nw + n0] = to16<kType>(z0);
        preact[row * Nw + n1] = to16<kType>(z1);
      }
      const size_t o = row * N + n0;
      if (gated) {
        float y = activate(z0, act) * z1;
        if (residual) y += from16<kType>(residual[o]);
        out[o] = to16<kType>(y);
      } else {
        float y0 = activate(z0, act), y1 = activate(z1, act);
        if (residual) {
          y0 += from16<kType>(residual[o]);
          y1 += from16<kType>(residual[o + 1]);
        }
        out[o] = to16<kType>(y0);
        out[o + 1] = to16<kType>(y1);
      }
    }
  }
}

template <int kType>
cudaError_t launch_type(const LinearDims& s, const int32_t* offsets, const void* x, const void* w, const float* bias,
                        const void* residual, void* out, void* preact, cudaStream_t st) {
  const int per_cta = kThreads / 32 * (s.gated ? 1 : 2);
  const dim3 grid((s.N + per_cta - 1) / per_cta, offsets ? s.R : 1);
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, offsets, static_cast<const uint4*>(x),
                      static_cast<const uint4*>(w), bias, static_cast<const uint16_t*>(residual),
                      static_cast<uint16_t*>(out), static_cast<uint16_t*>(preact), s.R, s.E, s.K, s.N, s.gated, s.act);
  };
  if (s.R == 1) return go(linear_small_kernel<kType, 1>);
  if (s.R == 2) return go(linear_small_kernel<kType, 2>);
  if (s.R <= 4) return go(linear_small_kernel<kType, 4>);
  return go(linear_small_kernel<kType, kMaxRows>);
}

}  // namespace

cudaError_t launch_linear_small(const LinearDims& s, const int32_t* offsets, const void* x, const void* w,
                                const float* bias, const void* residual, void* out, void* preact, cudaStream_t st) {
  return s.type == 1 ? launch_type<1>(s, offsets, x, w, bias, residual, out, preact, st)
                     : launch_type<0>(s, offsets, x, w, bias, residual, out, preact, st);
}

}  // namespace moe
