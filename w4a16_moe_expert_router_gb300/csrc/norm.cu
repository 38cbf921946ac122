// norm.cu -- the RMS norms before and after a block, fused with the gate and the residual
// between them, and their gradient (fp16, bf16 or fp32 rows, fp32 weights).
//
//   v   = gamma_post y r1,  r1 = 1 / sqrt(mean y^2 + eps)   (without gamma_post: v = y)
//   out = scale x + gate v
//   u   = gamma_pre out r2,  r2 = 1 / sqrt(mean out^2 + eps)
// and backwards, with n = out r2, m = y r1 and means over a row's columns,
//   g  = dout + r2 (gamma_pre du - n mean(n gamma_pre du))        dx = scale g
//   dv = gate g       dy = r1 (gamma_post dv - m mean(m gamma_post dv))
//   dgamma_pre = sum du n,  dgamma_post = sum dv m,  dgate = sum g v  (over the rows they are shared by)
//
// Both directions read every row once and hold it in registers until its sums are known, so they
// move 4 and 6 rows per row and are bound by memory; the arithmetic is a dozen operations an element.
// Everything between load and store is fp32; u is the norm of the unrounded out.
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"

namespace moe {
namespace {

struct Args {
  const uint4 *x, *y;
  const float *gamma_post, *gate, *gamma_pre;
  uint4 *out, *u;
  int R, d, nvec, gate_rows;
  float scale, eps;
};

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = *reinterpret_cast<const float4*>(p + i);
    f[i] = v.x;
    f[i + 1] = v.y;
    f[i + 2] = v.z;
    f[i + 3] = v.w;
  }
}

template <int N>
__device__ __forceinline__ void store_floats(float* p, const float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// ----------------------------------------------------------------- forward
//
// A row by one warp (eight rows per CTA) or by one CTA; a thread holds kPieces 16-byte pieces of it.
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if constexpr (kWarp) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += part[w];
  return s;
}

constexpr int kForwardThreads = 256;  // of a CTA whose warps take a row each

template <int kType, int kPieces, bool kWarp>
__global__ void __launch_bounds__(kWarp ? kForwardThreads : 512) norm_kernel(const Args a) {
  constexpr int N = Vec<kType>::n;
  __shared__ float part[2][16];
  grid_dependents_launch();
  grid_dependency_wait();
  const int step = kWarp ? 32 : blockDim.x, at = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int row = kWarp ? blockIdx.x * (kForwardThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && row >= a.R) return;
  const size_t base = static_cast<size_t>(row) * a.nvec;
  uint4 xv[kPieces], yv[kPieces];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = at + p * step;
    xv[p] = yv[p] = make_uint4(0u, 0u, 0u, 0u);
    if (c < a.nvec) {
      if (a.y) yv[p] = a.y[base + c];
      if (a.x) xv[p] = a.x[base + c];
    }
  }
  float r1 = 1.f;
  if (a.gamma_post) {
    float ss = 0.f;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      float f[N], s = 0.f;
      Vec<kType>::load(yv[p], f);
#pragma unroll
      for (int i = 0; i < N; ++i) s = fmaf(f[i], f[i], s);
      ss += s;
    }
    r1 = __frsqrt_rn(row_sum<kWarp>(ss, part[0]) / a.d + a.eps);
  }
  const float* gate = a.gate ? a.gate + static_cast<size_t>(row / a.gate_rows) * a.d : nullptr;
  float o[kPieces][N], ss = 0.f;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = at + p * step;
    float f[N], s = 0.f;
    Vec<kType>::load(xv[p], o[p]);
#pragma unroll
    for (int i = 0; i < N; ++i) o[p][i] *= a.scale;
    if (c < a.nvec) {
      if (a.y) {
        float w[N];
        Vec<kType>::load(yv[p], f);
        if (a.gamma_post) {
          load_floats(a.gamma_post + c * N, w);
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = f[i] * r1 * w[i];
        }
        if (gate) {
          load_floats(gate + c * N, w);
#pragma unroll
          for (int i = 0; i < N; ++i) o[p][i] = fmaf(w[i], f[i], o[p][i]);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) o[p][i] += f[i];
        }
      }
      if (a.out) a.out[base + c] = Vec<kType>::store(o[p]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(o[p][i], o[p][i], s);
    ss += s;
  }
  if (!a.u) return;
  const float r2 = __frsqrt_rn(row_sum<kWarp>(ss, part[1]) / a.d + a.eps);
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = at + p * step;
    if (c < a.nvec) {
      float w[N];
      load_floats(a.gamma_pre + c * N, w);
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] *= o[p][i] * r2;
      a.u[base + c] = Vec<kType>::store(w);
    }
  }
}

// ---------------------------------------------------------------- backward
//
// A group of threads, a multiple of 32 that covers a row with kPieces pieces each, takes a
// contiguous run of rows ("unit"), so a thread's columns stay the same and the weights' gradients
// are summed in its registers. The sums over the units follow in a second launch, in the order of
// the units: no atomics, the same bits in every run. A gate row whose rows lie in one unit is
// written at once; the others leave a partial sum per unit (the unit's first gate row in slot
// 2 u, its last one in 2 u + 1).
struct GradArgs {
  const uint4 *y, *out, *dout, *du;
  const float *gamma_post, *gate, *gamma_pre;
  uint4 *dx, *dy;
  float *part_post, *part_pre;  // [CTAs][d], or NULL where not wanted
  float *dgate, *slots;         // [groups][d] or NULL; [2 units][d]
  int R, d, nvec, gate_rows, group, units;
  float scale, eps;
};

__host__ __device__ inline int unit_first(int u, int R, int units) {
  return static_cast<int>(static_cast<int64_t>(u) * R / units);
}
__host__ __device__ inline int unit_of(int row, int R, int units) {
  return static_cast<int>(((static_cast<int64_t>(row) + 1) * units - 1) / R);
}

// Sums of kCount values over the group, the same in all its threads. `part` alternates between
// two places from row to row: a thread that is a barrier ahead does not write what others still read.
template <int kCount>
__device__ __forceinline__ void group_sum(float (&v)[kCount], int group, int which, float (*part)[kCount]) {
#pragma unroll
  for (int i = 0; i < kCount; ++i) v[i] = warp_sum(v[i]);
  if (group == 32) return;
  const int warp = threadIdx.x >> 5, warps = group >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kCount; ++i) part[warp][i] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "r"(group) : "memory");
#pragma unroll
  for (int i = 0; i < kCount; ++i) {
    v[i] = 0.f;
    for (int w = 0; w < warps; ++w) v[i] += part[which * warps + w][i];
  }
}

template <int kType, int kPieces>
struct Held {
  uint4 y[kPieces], out[kPieces], dout[kPieces], du[kPieces];
};

template <int kType, int kPieces>
__device__ __forceinline__ void load_row(const GradArgs& a, int row, int at, Held<kType, kPieces>& h) {
  const size_t base = static_cast<size_t>(row) * a.nvec;
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = at + p * a.group;
    h.y[p] = h.out[p] = h.dout[p] = h.du[p] = make_uint4(0u, 0u, 0u, 0u);
    if (c < a.nvec) {
      if (a.du) {
        h.out[p] = a.out[base + c];
        h.du[p] = a.du[base + c];
      }
      if (a.y) h.y[p] = a.y[base + c];
      if (a.dout) h.dout[p] = a.dout[base + c];
    }
  }
}

template <int kType, int kPieces>
__global__ void __launch_bounds__(512) norm_backward_kernel(const GradArgs a) {
  constexpr int N = Vec<kType>::n;
  constexpr bool kAhead = kPieces == 1;  // the next row's loads on their way while one is summed
  extern __shared__ float gammas[];      // [2][d], where a CTA has several groups
  __shared__ float part_a[2][16][3], part_b[2][16][1];
  grid_dependents_launch();
  grid_dependency_wait();
  const int which = threadIdx.x / a.group, at = threadIdx.x - which * a.group;
  const int groups = blockDim.x / a.group, unit = blockIdx.x * groups + which;
  float acc_post[kPieces][N], acc_pre[kPieces][N], acc_gate[kPieces][N];
#pragma unroll
  for (int p = 0; p < kPieces; ++p)
#pragma unroll
    for (int i = 0; i < N; ++i) acc_post[p][i] = acc_pre[p][i] = acc_gate[p][i] = 0.f;
  const int r0 = unit < a.units ? unit_first(unit, a.R, a.units) : 0;
  const int r1 = unit < a.units ? unit_first(unit + 1, a.R, a.units) : 0;
  const int first_gate = a.gate ? r0 / a.gate_rows : 0;
  int gate_row = first_gate, gate_end = a.gate ? (first_gate + 1) * a.gate_rows : r1;
  Held<kType, kPieces> h, next;
  if (kAhead && r0 < r1) load_row(a, r0, at, h);
  for (int row = r0; row < r1; ++row) {
    if (kAhead) {
      if (row + 1 < r1) load_row(a, row + 1, at, next);
    } else {
      load_row(a, row, at, h);
    }
    // sums of out^2, of gamma_pre du out and of y^2
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = at + p * a.group;
      float o[N], f[N], w[N];
      if (a.du && c < a.nvec) {
        Vec<kType>::load(h.out[p], o);
        Vec<kType>::load(h.du[p], f);
        load_floats(a.gamma_pre + c * N, w);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          s[0] = fmaf(o[i], o[i], s[0]);
          s[1] = fmaf(w[i] * f[i], o[i], s[1]);
        }
      }
      Vec<kType>::load(h.y[p], f);
#pragma unroll
      for (int i = 0; i < N; ++i) s[2] = fmaf(f[i], f[i], s[2]);
    }
    group_sum(s, a.group, which, part_a[row & 1]);
    const float ra = __frsqrt_rn(s[0] / a.d + a.eps), mean_a = ra * s[1] / a.d;
    const float rb = a.gamma_post ? __frsqrt_rn(s[2] / a.d + a.eps) : 1.f;
    const float* gate = a.gate ? a.gate + static_cast<size_t>(gate_row) * a.d : nullptr;
    float g[kPieces][N], t[1] = {0.f};
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = at + p * a.group;
      float o[N], f[N], w[N];
      Vec<kType>::load(h.dout[p], g[p]);
      if (c < a.nvec) {
        if (a.du) {
          Vec<kType>::load(h.out[p], o);
          Vec<kType>::load(h.du[p], f);
          load_floats(a.gamma_pre + c * N, w);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float n = o[i] * ra;
            acc_pre[p][i] = fmaf(f[i], n, acc_pre[p][i]);
            g[p][i] = fmaf(ra, fmaf(-n, mean_a, w[i] * f[i]), g[p][i]);
          }
        }
        if (a.dx) {
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = a.scale * g[p][i];
          a.dx[static_cast<size_t>(row) * a.nvec + c] = Vec<kType>::store(f);
        }
        if (a.gamma_post) {
          Vec<kType>::load(h.y[p], f);
          load_floats(a.gamma_post + c * N, w);
          if (gate) {
            load_floats(gate + c * N, o);
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] *= o[i];
          }
#pragma unroll
          for (int i = 0; i < N; ++i) t[0] = fmaf(w[i] * g[p][i], f[i], t[0]);
        }
      }
    }
    float mean_b = 0.f;
    if (a.gamma_post) {
      group_sum(t, a.group, which, part_b[row & 1]);
      mean_b = rb * t[0] / a.d;
    }
    if (a.y || a.dy) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int c = at + p * a.group;
        if (c >= a.nvec) continue;
        float f[N], w[N], q[N];
        Vec<kType>::load(h.y[p], f);
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = q[i] = 1.f;
        if (a.gamma_post) load_floats(a.gamma_post + c * N, w);
        if (gate) load_floats(gate + c * N, q);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float m = f[i] * rb, dv = q[i] * g[p][i];
          acc_post[p][i] = fmaf(dv, m, acc_post[p][i]);
          acc_gate[p][i] = fmaf(g[p][i] * w[i], m, acc_gate[p][i]);
          f[i] = a.gamma_post ? rb * fmaf(-m, mean_b, w[i] * dv) : dv;
        }
        if (a.dy) a.dy[static_cast<size_t>(row) * a.nvec + c] = Vec<kType>::store(f);
      }
    }
    if (a.dgate && (row + 1 == gate_end || row + 1 == r1)) {
      const int last = min(gate_end, a.R) - 1;
      const bool whole = unit_of(gate_row * a.gate_rows, a.R, a.units) == unit && last < r1;
      float* dst = whole ? a.dgate + static_cast<size_t>(gate_row) * a.d
                         : a.slots + (static_cast<size_t>(2 * unit) + (gate_row != first_gate)) * a.d;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int c = at + p * a.group;
        if (c < a.nvec) store_floats(dst + c * N, acc_gate[p]);
#pragma unroll
        for (int i = 0; i < N; ++i) acc_gate[p][i] = 0.f;
      }
    }
    if (row + 1 == gate_end) {
      ++gate_row;
      gate_end += a.gate_rows;
    }
    if (kAhead) h = next;
  }
  if (groups == 1) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = at + p * a.group;
      if (c >= a.nvec) continue;
      if (a.part_post) store_floats(a.part_post + static_cast<size_t>(blockIdx.x) * a.d + c * N, acc_post[p]);
      if (a.part_pre) store_floats(a.part_pre + static_cast<size_t>(blockIdx.x) * a.d + c * N, acc_pre[p]);
    }
    return;
  }
  for (int q = 0; q < groups; ++q) {  // the groups' sums in order
    if (q == which)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int c = at + p * a.group;
        if (c >= a.nvec) continue;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float* const post = gammas + c * N + i;
          float* const pre = post + a.d;
          *post = (q ? *post : 0.f) + acc_post[p][i];
          *pre = (q ? *pre : 0.f) + acc_pre[p][i];
        }
      }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    if (a.part_post) a.part_post[static_cast<size_t>(blockIdx.x) * a.d + c] = gammas[c];
    if (a.part_pre) a.part_pre[static_cast<size_t>(blockIdx.x) * a.d + c] = gammas[a.d + c];
  }
}

// The second launch: 32 columns per CTA (8 lanes of four), 32 slices of the partial sums, which
// meet in order. blockIdx.y 0 and 1: the gammas over the CTAs; from 2 on: gate rows with partial sums.
struct SumArgs {
  const float *part_post, *part_pre, *slots;
  float *dgamma_post, *dgamma_pre, *dgate;
  int R, d, gate_rows, ctas, units, gates;
};

__global__ void __launch_bounds__(256) norm_sum_kernel(const SumArgs a) {
  __shared__ float4 part[32][8];
  grid_dependents_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + lane * 4;
  const bool on = col < a.d;
  const int y = blockIdx.y;
  const bool gates = y >= 2;
  if (!gates && !(y == 0 ? a.dgamma_post : a.dgamma_pre)) return;
  for (int g = gates ? y - 2 : 0; g < (gates ? a.gates : 1); g += gates ? gridDim.y - 2 : 1) {
    int u0 = 0, u1 = a.ctas - 1;
    if (gates) {
      u0 = unit_of(g * a.gate_rows, a.R, a.units);
      u1 = unit_of(min((g + 1) * a.gate_rows, a.R) - 1, a.R, a.units);
      if (u0 == u1) continue;  // written by its unit
    }
    const float* src = gates ? a.slots : y == 0 ? a.part_post : a.part_pre;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on)
      for (int u = u0 + slice; u <= u1; u += 32) {
        size_t at = u;
        if (gates) at = 2 * at + (unit_first(u, a.R, a.units) / a.gate_rows != g);
        const float4 v = *reinterpret_cast<const float4*>(src + at * a.d + col);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    part[slice][lane] = s;
    __syncthreads();
    if (slice == 0 && on) {
      for (int k = 1; k < 32; ++k) {
        const float4 v = part[k][lane];
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      float* dst = gates ? a.dgate + static_cast<size_t>(g) * a.d : y == 0 ? a.dgamma_post : a.dgamma_pre;
      *reinterpret_cast<float4*>(dst + col) = s;
    }
    __syncthreads();
  }
}

template <int kType, int kPieces, bool kWarp>
cudaError_t launch_forward(const Args& a, int threads, cudaStream_t st) {
  const int per = kWarp ? kForwardThreads / 32 : 1;
  return launch_pdl(norm_kernel<kType, kPieces, kWarp>, dim3((a.R + per - 1) / per), dim3(threads), 0, st, a);
}

// A warp per row needs no barrier, but with few rows the pieces are spread over more threads:
// latency counts then.
template <int kType>
cudaError_t forward(const Args& a, cudaStream_t st) {
  const auto threads = [&](int pieces) { return (a.nvec + 32 * pieces - 1) / (32 * pieces) * 32; };
  if (a.R >= 152 * 8 && a.nvec <= 256) {
    if (a.nvec <= 32) return launch_forward<kType, 1, true>(a, kForwardThreads, st);
    if (a.nvec <= 64) return launch_forward<kType, 2, true>(a, kForwardThreads, st);
    if (a.nvec <= 128) return launch_forward<kType, 4, true>(a, kForwardThreads, st);
    return launch_forward<kType, 8, true>(a, kForwardThreads, st);
  }
  if (a.nvec <= 512 && a.R < 152 * 4) return launch_forward<kType, 1, false>(a, threads(1), st);
  return launch_forward<kType, 4, false>(a, threads(4), st);
}

// Threads of a group and groups of a CTA of the gradient's kernel.
struct GradShape {
  int pieces, group, groups, ctas, units;
};
GradShape grad_shape(const NormDims& s) {
  GradShape g;
  const int nvec = s.nvec();
  g.pieces = nvec <= 512 ? 1 : nvec <= 1024 ? 2 : 4;
  g.group = (nvec + 32 * g.pieces - 1) / (32 * g.pieces) * 32;
  g.groups = g.group >= 256 ? 1 : 256 / g.group;
  const int rows = s.R > 0 ? s.R : 1;
  g.ctas = (rows + g.groups - 1) / g.groups;
  if (g.ctas > kNormCtas) g.ctas = kNormCtas;
  g.units = g.ctas * g.groups;
  if (g.units > rows) g.units = rows;
  return g;
}

template <int kType, int kPieces>
cudaError_t backward(const GradArgs& a, const GradShape& g, cudaStream_t st) {
  return launch_pdl(norm_backward_kernel<kType, kPieces>, dim3(g.ctas), dim3(g.group * g.groups),
                    g.groups > 1 ? size_t(2) * a.d * 4 : 0, st, a);
}

}  // namespace

cudaError_t launch_norm(const NormDims& s, const void* x, const void* y, const float* gamma_post, const float* gate,
                        const float* gamma_pre, void* out, void* u, cudaStream_t st) {
  const Args a{static_cast<const uint4*>(x), static_cast<const uint4*>(y), gamma_post, gate, gamma_pre,
               static_cast<uint4*>(out), static_cast<uint4*>(u), s.R, s.d, s.nvec(), s.gate_rows, s.scale, s.eps};
  return s.type == 0 ? forward<0>(a, st) : s.type == 1 ? forward<1>(a, st) : forward<2>(a, st);
}

size_t norm_backward_ws_bytes(const NormDims& s) {
  const GradShape g = grad_shape(s);
  return (size_t(g.ctas) + g.units) * 2 * s.d * 4;
}

cudaError_t launch_norm_backward(const NormDims& s, const void* y, const float* gamma_post, const float* gate,
                                 const void* out, const float* gamma_pre, const void* dout, const void* du, void* dx,
                                 void* dy, float* dgamma_post, float* dgate, float* dgamma_pre, void* workspace,
                                 cudaStream_t st) {
  const GradShape g = grad_shape(s);
  auto* const ws = static_cast<float*>(workspace);
  float* const pre = ws + size_t(g.ctas) * s.d;
  float* const slots = pre + size_t(g.ctas) * s.d;
  GradArgs a{};
  const bool needs_y = (dy && gamma_post) || dgamma_post || dgate;
  a.y = needs_y ? static_cast<const uint4*>(y) : nullptr;
  a.out = static_cast<const uint4*>(out);
  a.dout = static_cast<const uint4*>(dout);
  a.du = static_cast<const uint4*>(du);
  a.gamma_post = needs_y ? gamma_post : nullptr;
  a.gate = gate;
  a.gamma_pre = gamma_pre;
  a.dx = static_cast<uint4*>(dx);
  a.dy = static_cast<uint4*>(dy);
  a.part_post = dgamma_post ? ws : nullptr;
  a.part_pre = dgamma_pre ? pre : nullptr;
  a.dgate = dgate;
  a.slots = slots;
  a.R = s.R;
  a.d = s.d;
  a.nvec = s.nvec();
  a.gate_rows = gate ? s.gate_rows : s.R;
  a.group = g.group;
  a.units = g.units;
  a.scale = s.scale;
  a.eps = s.eps;
  cudaError_t err;
  const auto run = [&](auto type) {
    constexpr int kType = decltype(type)::value;
    if (g.pieces == 1) return backward<kType, 1>(a, g, st);
    if (kType < 2 || g.pieces == 2) return backward<kType, 2>(a, g, st);  // 8192 16-bit columns at most
    return backward<2, 4>(a, g, st);
  };
  if (s.type == 0)
    err = run(std::integral_constant<int, 0>{});
  else if (s.type == 1)
    err = run(std::integral_constant<int, 1>{});
  else
    err = run(std::integral_constant<int, 2>{});
  if (err != cudaSuccess || (!dgamma_post && !dgamma_pre && !dgate)) return err;
  const int gates = dgate ? (s.R + s.gate_rows - 1) / s.gate_rows : 0;
  const SumArgs b{ws, pre, slots, dgamma_post, dgamma_pre, dgate, s.R, s.d, a.gate_rows, g.ctas, g.units, gates};
  const int extra = gates > 64 ? 64 : gates;
  return launch_pdl(norm_sum_kernel, dim3((s.d + 31) / 32, 2 + extra), dim3(256), 0, st, b);
}

}  // namespace moe
