// clip.cu -- the norm over a list of tensors (fp16, bf16, fp32, of any length and alignment), and
// the tensors scaled down to a bound on it.
//
//   norm = sqrt(sum over all tensors of g^2),   out = g min(1, max_norm / norm)
//
// Two passes over the data, each bound by memory: the sum of the squares, and the scaling, which is
// left out where it would change nothing. The tensors are cut into chunks, and every CTA takes a
// contiguous run of them, so it looks for its first tensor once. A launch carries its tensors'
// addresses as kernel parameters (up to kLarge of them), so nothing is kept on the device from call
// to call and a captured graph holds its own.
//
// Squares are summed in fp32 over the 64 to 128 bytes that a thread takes of a chunk, in fp64 from
// there on: an fp64 addition per element would be the bound (its rate is a hundredth of fp32's), one
// per chunk is not seen. Where such a sum leaves the range in which fp32 squares keep their digits,
// it is taken again in fp64. All orders are fixed: the same bits in every run.
// Measured: 554 million bf16 values from one place to another 509 us (3.3 GB in the two passes, 6.5 TB/s), in
// place 518; 400 tensors of 47 MB in all below the bound 13.9 us, above it in place 15.3; five small ones 5.2 us, of which
// a launch is the most.
#include <cfloat>
#include <climits>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLoads = 8;                              // 16-byte pieces of a chunk per thread
constexpr int kChunkBytes = kThreads * kLoads * 16;    // 32 KB
// Tensors per launch: 23 KB of parameters, or 2.3 KB for short lists (the parameters are copied a few
// times on their way to the device).
constexpr int kLarge = 640, kSmall = 64;
constexpr int kCtas = 608;                             // four on each of 152 SMs (at most 64 registers a thread)

struct Entry {
  const void* data;
  void* out;       // NULL: the tensor is not scaled
  int64_t count;   // elements
  int32_t type;
  int32_t shift;   // elements between the 16-byte boundary below `data` and `data`
};
template <int kTable>
struct Table {
  Entry e[kTable];
  int32_t first[kTable + 1];  // chunks before an entry
  int32_t n;
};
static_assert(sizeof(Table<kLarge>) <= 32000, "kernel parameters");
// the chunks of a full table fit an int32
static_assert(kClipMaxCount * 4 / kChunkBytes * kLarge + kLarge < INT32_MAX, "chunk numbers");

template <int kTable>
__device__ __forceinline__ int find(const Table<kTable>& t, int chunk) {
  int lo = 0, hi = t.n - 1;  // the last entry with first <= chunk
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The first chunk of CTA b.
__device__ __forceinline__ int share(int chunks, int b) {
  return static_cast<int>(static_cast<int64_t>(chunks) * b / gridDim.x);
}

// Element i of 16 bytes (eight of 16 bits, four of 32).
template <int kType>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  if constexpr (kType == 2) return static_cast<const float*>(p)[i];
  else return from16<kType>(static_cast<const uint16_t*>(p)[i]);
}
// max_norm / norm, in two parts where the quotient is below fp32's normal range (a bound of 1e-3 on a norm of 1e37): as a
// number of its own it would have lost digits, or be zero, where its products with the values are not.
struct Factor {
  float first, second;
  __device__ __forceinline__ bool one() const { return first == 1.f; }
  __device__ __forceinline__ float of(float v) const { return v * first * second; }
};
template <int kType>
__device__ __forceinline__ void put_scaled(const Entry& e, int64_t i, Factor factor) {
  if constexpr (kType == 2) {
    const float v = static_cast<const float*>(e.data)[i];
    static_cast<float*>(e.out)[i] = factor.one() ? v : factor.of(v);
  } else {
    const uint16_t v = static_cast<const uint16_t*>(e.data)[i];
    static_cast<uint16_t*>(e.out)[i] = factor.one() ? v : to16<kType>(factor.of(from16<kType>(v)));
  }
}

// A chunk of a tensor: pieces of 16 bytes from the boundary below the tensor on, of whose elements lo .. hi - 1 are
// the tensor's.
template <int kType>
struct Chunk {
  static constexpr int N = Vec<kType>::n, kElements = kThreads * kLoads * N;
  const uint4* pieces;
  int64_t first;  // the tensor's element at the chunk's element 0 (below zero where the tensor starts later)
  int lo, hi;

  __device__ __forceinline__ Chunk(const Entry& e, int chunk) {
    pieces = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(e.data) & ~uintptr_t(15)) +
             static_cast<int64_t>(chunk) * (kThreads * kLoads);
    first = static_cast<int64_t>(chunk) * kElements - e.shift;
    lo = first < 0 ? static_cast<int>(-first) : 0;
    hi = static_cast<int>(min(e.count - first, static_cast<int64_t>(kElements)));
  }
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == kElements; }
  // Whether the tensor fills the piece.
  __device__ __forceinline__ bool full(int piece) const { return piece * N >= lo && (piece + 1) * N <= hi; }
  // The element of the thread, or -1: those of the pieces at the tensor's ends that it fills in part are taken one
  // by one by the first threads of two warps.
  __device__ __forceinline__ int edge() const {
    const int head = lo / N, tail = hi / N, t = threadIdx.x;
    int i = -1;
    if (t < N && lo % N) i = head * N + t;
    if (t >= 32 && t < 32 + N && hi % N && !(lo % N && head == tail)) i = tail * N + t - 32;
    return i >= lo && i < hi ? i : -1;
  }
};

// Sum of the squares of a thread's share of a chunk.
template <int kType>
__device__ double chunk_square(const Entry& e, int chunk) {
  constexpr int N = Vec<kType>::n;
  const Chunk<kType> c(e, chunk);
  uint4 x[kLoads];
  if (c.whole()) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) x[l] = c.pieces[threadIdx.x + l * kThreads];
  } else {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      x[l] = make_uint4(0u, 0u, 0u, 0u);
      if (c.full(threadIdx.x + l * kThreads)) x[l] = c.pieces[threadIdx.x + l * kThreads];
    }
  }
  float s = 0.f;
  uint32_t any = 0u;
  int edge = -1;
  if (!c.whole() && (edge = c.edge()) >= 0) {
    const float f = value<kType>(e.data, c.first + edge);
    any = __float_as_uint(f);
    s = f * f;
  }
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    float f[N], q = 0.f;
    Vec<kType>::load(x[l], f);
    any |= (x[l].x | x[l].y) | (x[l].z | x[l].w);
#pragma unroll
    for (int i = 0; i < N; ++i) q = fmaf(f[i], f[i], q);
    s += q;
  }
  // squares below 2^-100 may have lost digits to fp32's smallest step, those above its range are
  // infinite: an fp64 sum (`any` of signs alone is no reason)
  if (s >= 0x1p-100f && s <= 0x1p127f) return s;
  if ((any & (kType == 2 ? 0x7fffffffu : 0x7fff7fffu)) == 0u) return 0.0;
  double d = 0.0;
  if (edge >= 0) {
    const double f = value<kType>(e.data, c.first + edge);
    d = f * f;
  }
#pragma unroll 1
  for (int l = 0; l < kLoads; ++l) {
    const int piece = threadIdx.x + l * kThreads;
    if (!c.full(piece)) continue;
#pragma unroll 1
    for (int i = 0; i < N; ++i) {
      const double f = value<kType>(e.data, c.first + piece * N + i);
      d = fma(f, f, d);
    }
  }
  return d;
}

// The sum over the CTA, in thread 0 alone: fp64 operations of all threads would take their time.
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += part[w];
  return s;
}

template <int kType>
__device__ void scale_chunk(const Entry& e, int chunk, Factor factor) {
  constexpr int N = Vec<kType>::n, kBatch = 4;
  const Chunk<kType> c(e, chunk);
  auto* const dst = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(e.out) & ~uintptr_t(15)) +
                    static_cast<int64_t>(chunk) * (kThreads * kLoads);
  const auto scaled = [&](uint4 x) {
    if (!factor.one()) {  // else the bits are copied, a NaN's too
      float f[N];
      Vec<kType>::load(x, f);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = factor.of(f[i]);
      x = Vec<kType>::store(f);
    }
    return x;
  };
  // the output's pieces lie as the input's do, or it is written by elements
  const bool alike = ((reinterpret_cast<uintptr_t>(e.data) ^ reinterpret_cast<uintptr_t>(e.out)) & 15u) == 0;
  if (alike && c.whole()) {
#pragma unroll 1
    for (int l0 = 0; l0 < kLoads; l0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int l = 0; l < kBatch; ++l) x[l] = c.pieces[threadIdx.x + (l0 + l) * kThreads];
#pragma unroll
      for (int l = 0; l < kBatch; ++l) dst[threadIdx.x + (l0 + l) * kThreads] = scaled(x[l]);
    }
    return;
  }
  const int edge = c.edge();
  if (edge >= 0) put_scaled<kType>(e, c.first + edge, factor);
  if (alike) {
#pragma unroll 1
    for (int l0 = 0; l0 < kLoads; l0 += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int l = 0; l < kBatch; ++l)
        if (c.full(threadIdx.x + (l0 + l) * kThreads)) x[l] = c.pieces[threadIdx.x + (l0 + l) * kThreads];
#pragma unroll
      for (int l = 0; l < kBatch; ++l)
        if (c.full(threadIdx.x + (l0 + l) * kThreads)) dst[threadIdx.x + (l0 + l) * kThreads] = scaled(x[l]);
    }
  } else {  // neighbouring threads take neighbouring elements
    const int from = (c.lo + N - 1) / N * N, to = c.hi / N * N;
#pragma unroll 4
    for (int i = from + static_cast<int>(threadIdx.x); i < to; i += kThreads) put_scaled<kType>(e, c.first + i, factor);
  }
}

// The square root in fp32 (fp64's takes a microsecond here): of the value between 1 and 4 that a power of four leaves.
__device__ __forceinline__ float root(double s) {
  if (!(s > 0.0 && s < INFINITY)) return static_cast<float>(s);
  const int64_t bits = __double_as_longlong(s);
  const int e = (static_cast<int>(bits >> 52) - 1023) >> 1;  // s = m 4^e (squares do not reach fp64's subnormals)
  const double m = __longlong_as_double(bits - static_cast<int64_t>(2 * e) * (int64_t(1) << 52));
  return ldexpf(sqrtf(static_cast<float>(m)), e);
}

// Sum of the squares of a CTA's run of chunks, in thread 0.
template <int kTable>
__device__ __forceinline__ double run_square(const Table<kTable>& t, int c0, int c1) {
  double s = 0.0;
  int i = c0 < c1 ? find(t, c0) : 0;
  for (int c = c0; c < c1; ++c) {
    while (t.first[i + 1] <= c) ++i;
    const Entry& e = t.e[i];
    const int k = c - t.first[i];
    s += e.type == 0 ? chunk_square<0>(e, k) : e.type == 1 ? chunk_square<1>(e, k) : chunk_square<2>(e, k);
  }
  return cta_sum(s);
}
// The run scaled, from its last chunk back: what the pass before read last is still in L2.
template <int kTable>
__device__ __forceinline__ void run_scale(const Table<kTable>& t, int c0, int c1, Factor factor) {
  int i = c0 < c1 ? find(t, c1 - 1) : 0;
  for (int c = c1 - 1; c >= c0; --c) {
    while (t.first[i] > c) --i;
    const Entry& e = t.e[i];
    if (!e.out || (factor.one() && e.out == e.data)) continue;
    const int k = c - t.first[i];
    if (e.type == 0)
      scale_chunk<0>(e, k, factor);
    else if (e.type == 1)
      scale_chunk<1>(e, k, factor);
    else
      scale_chunk<2>(e, k, factor);
  }
}
// The factor, from the sum of the squares; a norm that is no number, or infinite, leaves the values as they are.
__device__ __forceinline__ Factor factor_of(double square, float max_norm, float* norm) {
  const float v = root(square);
  if (norm) *norm = v;
  if (!(v > max_norm && v < INFINITY)) return Factor{1.f, 1.f};
  const float q = max_norm / v;
  return q < FLT_MIN ? Factor{max_norm * 0x1p126f / v, 0x1p-126f} : Factor{q, 1.f};  // (max_norm is below 4 then)
}

template <int kTable>
__global__ void __launch_bounds__(kThreads, 4)
    clip_square_kernel(const __grid_constant__ Table<kTable> t, double* partial) {
  grid_dependents_launch();
  grid_dependency_wait();
  const int chunks = t.first[t.n];
  const double s = run_square(t, share(chunks, blockIdx.x), share(chunks, blockIdx.x + 1));
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Partial sums of several launches into the first place.
__global__ void __launch_bounds__(kThreads) clip_total_kernel(double* partial, int n) {
  grid_dependents_launch();
  grid_dependency_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  s = cta_sum(s);  // its barrier: all have read before the first place is written
  if (threadIdx.x == 0) partial[0] = s;
}

// One warp of every CTA adds up the partial sums, all in the same order (eight of four CTAs keep an SM's fp64
// unit busy for 2 us). copies: a tensor is scaled to another place.
template <int kTable>
__global__ void __launch_bounds__(kThreads, 4)
    clip_scale_kernel(const __grid_constant__ Table<kTable> t, const double* partial, int n_partial, float max_norm,
                      bool copies, float* norm) {
  __shared__ Factor shared_factor;
  grid_dependents_launch();
  grid_dependency_wait();
  if (threadIdx.x < 32) {
    double s[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 5
    for (int i = threadIdx.x; i < n_partial; i += 128)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (i + 32 * q < n_partial) s[q] += __ldcg(partial + i + 32 * q);
    double sum = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (threadIdx.x == 0) shared_factor = factor_of(sum, max_norm, blockIdx.x == 0 ? norm : nullptr);
  }
  __syncthreads();
  const Factor factor = shared_factor;
  if (factor.one() && !copies) return;
  const int chunks = t.first[t.n];
  run_scale(t, share(chunks, blockIdx.x), share(chunks, blockIdx.x + 1), factor);
}

// Few chunks: one launch of one cluster, whose CTAs read each other's sums.
constexpr int kCluster = 8, kClusterChunks = 16;
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    clip_cluster_kernel(const __grid_constant__ Table<kSmall> t, float max_norm, float* norm) {
  __shared__ double sum;
  __shared__ Factor shared_factor;
  grid_dependents_launch();
  grid_dependency_wait();
  const int chunks = t.first[t.n], c0 = share(chunks, blockIdx.x), c1 = share(chunks, blockIdx.x + 1);
  const double s = run_square(t, c0, c1);
  if (threadIdx.x == 0) sum = s;
  cluster_sync();
  if (threadIdx.x == 0) {
    double part[kCluster];
#pragma unroll
    for (int q = 0; q < kCluster; ++q)
      asm volatile("ld.shared::cluster.f64 %0, [%1];"
                   : "=d"(part[q])
                   : "r"(cluster_addr(smem_addr(&sum), q))
                   : "memory");
    const double all = ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7]));
    shared_factor = factor_of(all, max_norm, blockIdx.x == 0 ? norm : nullptr);
  }
  cluster_sync();  // the sums are read before their CTA leaves, and the factor is there
  run_scale(t, c0, c1, shared_factor);
}

// The next tensors of a list, up to kTable; returns how many it took.
template <int kTable>
int fill(Table<kTable>& t, const moe_w4a16_tensor* tensors, int n) {
  int taken = 0;
  t.n = 0;
  t.first[0] = 0;
  for (; taken < n && t.n < kTable; ++taken) {
    const moe_w4a16_tensor& in = tensors[taken];
    if (in.count == 0) continue;
    const int size = in.type == 2 ? 4 : 2;
    const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(in.data) & 15u) / size);
    const int64_t per = kChunkBytes / size;
    t.e[t.n] = Entry{in.data, in.out, in.count, in.type, shift};
    t.first[t.n + 1] = t.first[t.n] + static_cast<int32_t>((in.count + shift + per - 1) / per);
    ++t.n;
  }
  return taken;
}

int ctas_of(int chunks) { return chunks < 1 ? 1 : chunks < kCtas ? chunks : kCtas; }

template <int kTable>
cudaError_t run(const moe_w4a16_tensor* tensors, int n, double max_norm, float* norm, double* partial,
                cudaStream_t st) {
  static thread_local Table<kTable> t;
  cudaError_t err = cudaSuccess;
  const float bound = max_norm > FLT_MAX ? INFINITY : static_cast<float>(max_norm);
  int sums = 0, launches = 0;
  for (int at = 0; at < n || launches == 0; ++launches) {
    at += fill(t, tensors + at, n - at);
    if constexpr (kTable == kSmall)
      if (t.first[t.n] <= kClusterChunks)
        return launch_pdl(clip_cluster_kernel, dim3(kCluster), dim3(kThreads), 0, st, t, bound, norm);
    const int ctas = ctas_of(t.first[t.n]);
    if ((err = launch_pdl(clip_square_kernel<kTable>, dim3(ctas), dim3(kThreads), 0, st, t, partial + sums)) !=
        cudaSuccess)
      return err;
    sums += ctas;
  }
  if (launches > 1) {
    if ((err = launch_pdl(clip_total_kernel, dim3(1), dim3(kThreads), 0, st, partial, sums)) != cudaSuccess) return err;
    sums = 1;
  }
  for (int at = 0, i = 0; i < launches; ++i) {
    if (launches > 1) at += fill(t, tensors + at, n - at);
    bool copies = false, scaled = max_norm < INFINITY;  // whether a value may have to be written
    for (int j = 0; j < t.n; ++j) copies |= t.e[j].out && t.e[j].out != t.e[j].data;
    scaled |= copies;
    if (i > 0 && !scaled) continue;
    if ((err = launch_pdl(clip_scale_kernel<kTable>, dim3(scaled ? ctas_of(t.first[t.n]) : 1), dim3(kThreads), 0, st, t,
                          static_cast<const double*>(partial), sums, bound, copies,
                          i == 0 ? norm : nullptr)) != cudaSuccess)
      return err;
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_ws_bytes(int n) {
  const size_t launches = n <= kLarge ? 1 : (n + kLarge - 1) / kLarge;
  return launches * kCtas * sizeof(double);
}

cudaError_t launch_clip(const moe_w4a16_tensor* tensors, int n, double max_norm, float* norm, void* workspace,
                        cudaStream_t st) {
  auto* const partial = static_cast<double*>(workspace);
  return n <= kSmall ? run<kSmall>(tensors, n, max_norm, norm, partial, st)
                     : run<kLarge>(tensors, n, max_norm, norm, partial, st);
}

}  // namespace moe
