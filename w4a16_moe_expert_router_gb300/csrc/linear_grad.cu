// linear_grad.cu -- the element-wise front of a product's gradient and its bias gradient.
//
//   dz = dout act'(z)                       (gated: dz_g = dout z_u act'(z_g), dz_u = dout act(z_g))
//   db[e][n] = sum over the rows of expert e of dz[r][n]
//
// One pass over z and dout writes dz in the rows' type, the operand of the two products
// that follow: a rounding of half a step per element, independent from element to
// element, so a sum over dz is off by about what its own rounding to the type costs.
// The bias gradient takes the fp32 values: a CTA sums up to linear_block_rows rows of one
// expert (64, or 256 of more than 2^21) for 256 columns (an eighth of the rows per thread,
// then eight threads in order) into a partial, and an expert's partials are added, eight
// strided sums per column in order, by an idle warp of the weight gradient that follows or,
// without one, by a launch of its own: no atomics.  Bound by memory: z and dout read once,
// dz written once; each thread requests two rows before it uses the first.
#include "activation.cuh"
#include "internal.h"
#include "row_vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 32;                 // 16-byte pieces (256 columns) per CTA
constexpr int kLanes = kThreads / kPieces;  // threads per column
constexpr int kBatch = 2;  // rows per thread at a time (four: too many registers, 79 against 70 us at 8192 x 8192)

// The row range of block b: experts own ceil(rows / per) blocks each, in order.
// Whole CTA; false when there is no such block.
__device__ __forceinline__ bool find_block(const int32_t* offsets, int E, int R, int per, int b, int* sh, int& e,
                                           int& r0, int& r1) {
  if (!offsets) {
    e = 0;
    r0 = b * per;
    r1 = min(R, r0 + per);
    return r0 < R;
  }
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int lo = 0, hi = 0;
  if (i < E) {
    lo = min(max(offsets[i], 0), R);
    hi = max(min(offsets[i + 1], R), lo);
  }
  const int n = (hi - lo + per - 1) / per;
  int incl = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) sh[warp] = incl;
  if (i == 0) sh[8] = -1;
  __syncthreads();
  int before = incl - n;
  for (int w = 0; w < warp; ++w) before += sh[w];
  if (n > 0 && b >= before && b < before + n) {
    sh[8] = i;
    sh[9] = lo + (b - before) * per;
    sh[10] = hi;
  }
  __syncthreads();
  e = sh[8];
  r0 = sh[9];
  r1 = min(sh[10], r0 + per);
  return e >= 0;
}

// g becomes act(g), o its derivative.
__device__ __forceinline__ void derivatives(float (&g)[8], int act, float (&o)[8]) {
  const auto all = [&](int kind) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y;
      activate_grad(g[i], kind, y, o[i]);
      g[i] = y;
    }
  };
  switch (act) {  // outside of the loop over the elements
    case kGeluTanh: all(kGeluTanh); break;
    case kGeluErf: all(kGeluErf); break;
    case kSilu: all(kSilu); break;
    default: all(kIdentity); break;
  }
}

// grid (column blocks of N, row blocks).  z NULL: dz is dout itself and only the bias is wanted.
template <int kType, bool kGated>
__global__ void __launch_bounds__(kThreads) linear_dz_kernel(const int32_t* offsets, const uint4* z, const uint4* dout,
                                                             uint4* dz, float* partial, int R, int E, int N, int act,
                                                             int per) {
  __shared__ int sh[12];
  __shared__ float sum[kGated ? 2 : 1][kLanes][kPieces * 8];
  grid_dependents_launch();
  grid_dependency_wait();
  int e, r0, r1;
  if (!find_block(offsets, E, R, per, blockIdx.y, sh, e, r0, r1)) return;
  const int piece = threadIdx.x % kPieces, rl = threadIdx.x / kPieces;
  const int nvec = N / 8, zvec = kGated ? 2 * nvec : nvec;
  const int col = blockIdx.x * kPieces + piece;
  float sg[8], su[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sg[i] = su[i] = 0.f;
  if (col < nvec) {
    for (int base = r0 + rl; base < r1; base += kLanes * kBatch) {
      uint4 vd[kBatch], vg[kBatch], vu[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = base + k * kLanes;
        if (r < r1) {
          vd[k] = dout[static_cast<size_t>(r) * nvec + col];
          if (z) {
            const size_t at = static_cast<size_t>(r) * zvec + col;
            vg[k] = z[at];
            if (kGated) vu[k] = z[at + nvec];
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int r = base + k * kLanes;
        if (r >= r1) break;
        float d[8];
        Vec<kType>::load(vd[k], d);
        if (z) {
          const size_t at = static_cast<size_t>(r) * zvec + col;
          float g[8];
          Vec<kType>::load(vg[k], g);
          float u[8], o[8];
          if (kGated) Vec<kType>::load(vu[k], u);
          derivatives(g, act, o);  // g becomes act(g), o its derivative
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float ou = d[i] * g[i];
            d[i] = kGated ? d[i] * u[i] * o[i] : d[i] * o[i];
            if (kGated) {
              u[i] = ou;
              su[i] += ou;
            }
          }
          dz[at] = Vec<kType>::store(d);
          if (kGated) dz[at + nvec] = Vec<kType>::store(u);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sg[i] += d[i];
      }
    }
  }
  if (!partial) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sum[0][rl][piece * 8 + i] = sg[i];
    if (kGated) sum[kGated ? 1 : 0][rl][piece * 8 + i] = su[i];
  }
  __syncthreads();
  const int n = blockIdx.x * kPieces * 8 + threadIdx.x;
  if (n >= N) return;
  constexpr int halves = kGated ? 2 : 1;
#pragma unroll
  for (int h = 0; h < halves; ++h) {
    float s = 0.f;
#pragma unroll
    for (int l = 0; l < kLanes; ++l) s += sum[h][l][threadIdx.x];
    partial[static_cast<size_t>(blockIdx.y) * halves * N + h * N + n] = s;
  }
}

// db[e][n]: the partials of expert e's blocks; grid (column blocks of 32, experts), warp l
// takes every eighth partial (the order in which the weight gradient's warp adds them too).
__global__ void __launch_bounds__(kThreads) linear_dbias_kernel(const int32_t* offsets, const float* partial, float* db,
                                                                int R, int E, int Nw, int per) {
  __shared__ int sh[9];
  __shared__ float sum[8][32];
  grid_dependents_launch();
  grid_dependency_wait();
  const int e = blockIdx.y, i = threadIdx.x, lane = i & 31, warp = i >> 5;
  int first = 0, count = (R + per - 1) / per;
  if (offsets) {
    int n = 0;
    if (i < E) {
      const int lo = min(max(offsets[i], 0), R), hi = max(min(offsets[i + 1], R), lo);
      n = (hi - lo + per - 1) / per;
    }
    if (i == e) sh[8] = n;
    int before = i < e ? n : 0;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
    if (lane == 0) sh[warp] = before;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; ++w) first += sh[w];
    count = sh[8];
  }
  const int n = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (n < Nw) {
    const float* p = partial + static_cast<size_t>(first) * Nw + n;
#pragma unroll 4
    for (int b = warp; b < count; b += 8) s += p[static_cast<size_t>(b) * Nw];
  }
  sum[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && n < Nw) {
    s = 0.f;
#pragma unroll
    for (int l = 0; l < 8; ++l) s += sum[l][lane];
    db[static_cast<size_t>(e) * Nw + n] = s;
  }
}

}  // namespace

int linear_row_blocks(const LinearDims& s) {
  const int per = linear_block_rows(s.R), blocks = (s.R + per - 1) / per;
  return s.grouped ? blocks + (s.E < s.R ? s.E : s.R) : blocks;
}

cudaError_t launch_linear_dz(const LinearDims& s, const int32_t* offsets, const void* z, const void* dout, void* dz,
                             float* partial, cudaStream_t st) {
  const dim3 grid((s.N + kPieces * 8 - 1) / (kPieces * 8), linear_row_blocks(s));
  const auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(kThreads), 0, st, offsets, static_cast<const uint4*>(z),
                      static_cast<const uint4*>(dout), static_cast<uint4*>(dz), partial, s.R, s.E, s.N, s.act,
                      linear_block_rows(s.R));
  };
  if (s.type == 1) return s.gated ? go(linear_dz_kernel<1, true>) : go(linear_dz_kernel<1, false>);
  return s.gated ? go(linear_dz_kernel<0, true>) : go(linear_dz_kernel<0, false>);
}

cudaError_t launch_linear_dbias(const LinearDims& s, const int32_t* offsets, const float* partial, float* dbias,
                                cudaStream_t st) {
  return launch_pdl(linear_dbias_kernel, dim3((s.Nw() + 31) / 32, s.E), dim3(kThreads), 0, st, offsets, partial, dbias,
                    s.R, s.E, s.Nw(), linear_block_rows(s.R));
}

}  // namespace moe
