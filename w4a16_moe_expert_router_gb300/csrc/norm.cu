// norm.cu -- the RMS norms before and after a block, fused with the gate and the residual
// between them, and their gradient (fp16, bf16 or fp32 rows, fp32 weights).
//
//   v   = gamma_post y r1,  r1 = 1 / sqrt(mean y^2 + eps)   (without gamma_post: v = y)
//   out = scale x + gate v
//   u   = gamma_pre out r2,  r2 = 1 / sqrt(mean out^2 + eps)
// and backwards, with n = out r2, m = y r1 and means over a row's columns,
//   g  = dout + r2 (gamma_pre du - n c),  c = mean(n gamma_pre du)        dx = scale g
//   dv = gate g       dy = r1 (gamma_post dv - m mean(m gamma_post dv))
//   dgamma_pre = sum du n,  dgamma_post = sum dv m,  dgate = sum g v  (over the rows they are shared by)
//
// Both directions read every row once, 4 and 6 rows of memory traffic per row, and are bound by memory.
// A group of threads, a multiple of 32 that covers a row with kPieces 16-byte pieces each, takes a
// contiguous run of rows (a "unit"): a thread's columns stay the same, and with them the weights in
// its registers. Rows arrive by cp.async in a ring, several ahead; a thread copies what it will
// read itself, so the ring needs no barrier. (Loads into registers a row ahead reached 4.9 TB/s: an SM
// needs some 60 KB in flight all the time.) Where every row has a gate row of its own, that comes by the ring
// as well (loaded when its row began: 4099 rows of 4000 fp32 columns 72.6 us, now 52.8; the gradient 113 and 92).
// The arithmetic is fp32 from load to store, on pairs (the gradient spent 53 instructions an element, 63 %
// of the issue slots, one value at a time); u is the norm of the unrounded out.
// Measured: 16384 rows of 2048 bf16 columns with both norms and a gate 48.9 us (5.5 TB/s), their gradient
// 72.9 us (5.5 TB/s, 46 instructions an element); one row 2.3 us.
#include <algorithm>
#include <atomic>
#include <climits>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;

// Two fp32 values in one operation each.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 16 bytes of a row as pairs, and back.
template <int kType>
struct Pairs {
  static constexpr int n = Vec<kType>::n / 2;
  static __device__ __forceinline__ void load(uint32_t addr, float2 (&p)[n]) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    float f[2 * n];
    Vec<kType>::load(v, f);
#pragma unroll
    for (int i = 0; i < n; ++i) p[i] = make_float2(f[2 * i], f[2 * i + 1]);
  }
  static __device__ __forceinline__ uint4 store(const float2 (&p)[n]) {
    float f[2 * n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
      f[2 * i] = p[i].x;
      f[2 * i + 1] = p[i].y;
    }
    return Vec<kType>::store(f);
  }
};
template <int n>
__device__ __forceinline__ void load_pairs(const float* p, float2 (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n; i += 2) {
    const float4 q = *reinterpret_cast<const float4*>(p + 2 * i);
    v[i] = make_float2(q.x, q.y);
    v[i + 1] = make_float2(q.z, q.w);
  }
}
template <int n>
__device__ __forceinline__ void store_pairs(float* p, const float2 (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n; i += 2)
    *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
}

// The rows of the units: the first `more` have base + 1, the others base.
struct Units {
  int count, base, more;
  // Rows of unit u: first(u) .. first(u + 1) - 1.
  __device__ __forceinline__ int first(int u) const { return u * base + min(u, more); }
  __device__ __forceinline__ int of(int row) const {
    const int longer = more * (base + 1);
    return row < longer ? row / (base + 1) : more + (row - longer) / base;
  }
};

// Sums of kCount (1 or 6) values over the group, the same in all its threads. With six each step of a
// warp's tree halves the values that a lane carries on (eight shuffles, not thirty). `part`
// alternates between two places from call to call: a thread that is a barrier ahead does not write what
// others still read.
template <int kCount>
__device__ __forceinline__ void group_sum(float (&v)[kCount], int group, int which, float (*part)[8]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = group >> 5;
  if constexpr (kCount == 1) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
    if (group == 32) return;
    if (lane == 0) part[warp][0] = v[0];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "r"(group) : "memory");
    float s = lane < warps ? part[which * warps + lane][0] : 0.f;  // 16 warps at most
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    v[0] = __shfl_sync(0xffffffffu, s, 0);
  } else {
    static_assert(kCount == 6, "one or six");
    float a[4];
    const bool up16 = lane & 16, up8 = lane & 8, up4 = lane & 4;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      a[i] = (up16 ? v[i + 3] : v[i]) + __shfl_xor_sync(0xffffffffu, up16 ? v[i] : v[i + 3], 16);
    a[0] = (up8 ? a[2] : a[0]) + __shfl_xor_sync(0xffffffffu, up8 ? a[0] : a[2], 8);
    a[1] += __shfl_xor_sync(0xffffffffu, a[1], 8);  // (of lanes & 8 it is not used)
    a[0] = (up4 ? a[1] : a[0]) + __shfl_xor_sync(0xffffffffu, up4 ? a[0] : a[1], 4);
    a[0] += __shfl_xor_sync(0xffffffffu, a[0], 2);
    a[0] += __shfl_xor_sync(0xffffffffu, a[0], 1);
    // lanes 4 j .. 4 j + 3 hold value 3 (j / 4) + 2 (j / 2 % 2) + j % 2; nothing where j % 4 is 3
    int step = 4;
    if (group > 32) {
      if ((lane & 3) == 0) part[warp][lane >> 2] = a[0];
      asm volatile("bar.sync %0, %1;" ::"r"(1 + which), "r"(group) : "memory");
      float s = 0.f;  // value lane % 8 of every fourth warp
      for (int w = lane >> 3; w < warps; w += 4) s += part[which * warps + w][lane & 7];
      s += __shfl_xor_sync(0xffffffffu, s, 8);
      s += __shfl_xor_sync(0xffffffffu, s, 16);
      a[0] = s;
      step = 1;
    }
#pragma unroll
    for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, a[0], (i < 3 ? i : i + 1) * step);
  }
}

// A thread's ring of rows: kDepth stages of kTensors tensors of kPieces pieces, and of a gate row of its
// own per row, where there is one, kGate 16-byte parts per piece (two where the rows have 16 bits).
template <int kTensors, int kPieces, int kDepth, int kGate>
struct Ring {
  uint32_t at;     // the thread's place in the first stage
  uint32_t pitch;  // bytes from piece to piece
  int slot = 0, free = 0;

  __device__ __forceinline__ Ring(uint8_t* smem) : at(smem_addr(smem) + threadIdx.x * 16), pitch(blockDim.x * 16) {
    for (int i = 0; i < kDepth * (kTensors + kGate) * kPieces; ++i)  // what is never copied counts as zeros
      asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at + i * pitch), "r"(0) : "memory");
    if (kGate > 1) __syncwarp();
  }
  __device__ __forceinline__ uint32_t piece(int stage, int tensor, int p) const {
    return at + ((stage * (kTensors + kGate) + tensor) * kPieces + p) * pitch;
  }
  // Part h of the gate beside piece p.
  __device__ __forceinline__ uint32_t gate(int stage, int p, int h) const {
    return piece(stage, kTensors, 0) + (p * kGate + h) * pitch;
  }
  // Requests a row of every tensor that is there, and its gate.
  __device__ __forceinline__ void request(const uint4* const (&t)[kTensors], const uint4* gates, size_t base,
                                          int column, int nvec, int group, bool more) {
    if (kGate > 1) __syncwarp();  // the row that was there has been read
    if (more) {
#pragma unroll
      for (int i = 0; i < kTensors; ++i)
        if (t[i])
#pragma unroll
          for (int p = 0; p < kPieces; ++p)
            if (column + p * group < nvec) cp_async_16(piece(free, i, p), t[i] + base + column + p * group);
      if (kGate > 0)
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int i = 0; i < kGate; ++i) {
            // of two parts, two neighbours copy first the one's and then the other's: whole sectors
            const int owner = kGate == 1 ? 0 : i - static_cast<int>(threadIdx.x & 1);
            const int part = kGate == 1 ? 0 : threadIdx.x & 1, c = column + p * group + owner;
            if (c < nvec) cp_async_16(gate(free, p, part) + owner * 16, gates + (base + c) * kGate + part);
          }
      if (++free == kDepth) free = 0;
    }
    cp_async_commit();
  }
  // Until the oldest row requested is there.
  __device__ __forceinline__ void wait() const {
    cp_async_wait<kDepth - 1>();
    if (kGate > 1) __syncwarp();
  }
  __device__ __forceinline__ void next() {
    if (++slot == kDepth) slot = 0;
  }
  // The gate of piece p of the oldest row, times w.
  template <int n>
  __device__ __forceinline__ void times_gate(int p, const float2 (&w)[n], float2 (&q)[n]) const {
    float2 f[2];
#pragma unroll
    for (int h = 0; h < kGate; ++h) {
      Pairs<2>::load(gate(slot, p, h), f);
      q[2 * h] = mul2(f[0], w[2 * h]);
      q[2 * h + 1] = mul2(f[1], w[2 * h + 1]);
    }
  }
};

// ----------------------------------------------------------------- forward

struct Args {
  const uint4 *x, *y;
  const float *gamma_post, *gate, *gamma_pre;
  uint4 *out, *u;
  int R, d, nvec, gate_rows, group;
  Units units;
  float scale, eps;
};

// The factor of a thread's columns of y: gamma_post (with kPost) times the gate (with kGate, where there is one).
template <int kPieces, int n, bool kPost, bool kGate, class A>
__device__ __forceinline__ void factors(const A& a, int gate_row, int at, float2 (&w)[kPieces][n]) {
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int c = at + p * a.group;
#pragma unroll
    for (int i = 0; i < n; ++i) w[p][i] = both(1.f);
    if (c >= a.nvec) continue;
    if (kPost) load_pairs(a.gamma_post + c * 2 * n, w[p]);
    if (kGate && a.gate) {
      float2 q[n];
      load_pairs(a.gate + static_cast<size_t>(gate_row) * a.d + c * 2 * n, q);
#pragma unroll
      for (int i = 0; i < n; ++i) w[p][i] = mul2(w[p][i], q[i]);
    }
  }
}

// kY: y is there; kU: u is wanted; kByRow: every row has a gate row of its own.
template <int kType, int kPieces, int kDepth, bool kY, bool kU, bool kByRow>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const Args a) {
  constexpr int n = Pairs<kType>::n;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][16][8];
  grid_dependents_launch();
  Ring<2, kPieces, kDepth, kByRow ? n / 2 : 0> ring(smem);
  const int which = threadIdx.x / a.group, at = threadIdx.x - which * a.group;
  const int unit = blockIdx.x * (blockDim.x / a.group) + which;
  grid_dependency_wait();
  if (unit >= a.units.count) return;
  const int r0 = a.units.first(unit), r1 = a.units.first(unit + 1);
  const uint4* const rows[2] = {a.x, kY ? a.y : nullptr};
  const auto* const gates = reinterpret_cast<const uint4*>(a.gate);
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i)
    ring.request(rows, gates, static_cast<size_t>(r0 + i) * a.nvec, at, a.nvec, a.group, r0 + i < r1);
  float2 w[kPieces][n], pre[kPieces][n];
  const bool gated = kY && !kByRow && a.gate;
  int gate_row = gated ? r0 / a.gate_rows : 0, gate_end = gated ? (gate_row + 1) * a.gate_rows : r1;
  const auto load_w = [&] {
    if (a.gamma_post)
      factors<kPieces, n, true, !kByRow>(a, gate_row, at, w);
    else
      factors<kPieces, n, false, !kByRow>(a, gate_row, at, w);
  };
  if (kY) load_w();
  if (kU)
#pragma unroll
    for (int p = 0; p < kPieces; ++p)
      if (at + p * a.group < a.nvec) load_pairs(a.gamma_pre + (at + p * a.group) * 2 * n, pre[p]);
  const float inv_d = 1.f / a.d;
  int call = 0;
#pragma unroll 1
  for (int row = r0; row < r1; ++row) {
    ring.request(rows, gates, static_cast<size_t>(row + kDepth - 1) * a.nvec, at, a.nvec, a.group,
                 row + kDepth - 1 < r1);
    ring.wait();
    float r = 1.f;
    if (kY && a.gamma_post) {
      float2 ss = both(0.f);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        float2 y[n];
        Pairs<kType>::load(ring.piece(ring.slot, 1, p), y);
#pragma unroll
        for (int i = 0; i < n; ++i) ss = fma2(y[i], y[i], ss);
      }
      float s[1] = {ss.x + ss.y};
      group_sum(s, a.group, which, part[call++ & 1]);
      r = __frsqrt_rn(s[0] * inv_d + a.eps);
    }
    float2 o[kPieces][n], ss = both(0.f);
    const size_t base = static_cast<size_t>(row) * a.nvec + at;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      Pairs<kType>::load(ring.piece(ring.slot, 0, p), o[p]);
#pragma unroll
      for (int i = 0; i < n; ++i) o[p][i] = mul2(o[p][i], both(a.scale));
      if (kY) {
        float2 y[n];
        Pairs<kType>::load(ring.piece(ring.slot, 1, p), y);
        float2 q[n];
        if constexpr (kByRow) ring.times_gate(p, w[p], q);
#pragma unroll
        for (int i = 0; i < n; ++i) o[p][i] = fma2(kByRow ? q[i] : w[p][i], mul2(y[i], both(r)), o[p][i]);
      }
      if (kU)
#pragma unroll
        for (int i = 0; i < n; ++i) ss = fma2(o[p][i], o[p][i], ss);
      if (a.out && at + p * a.group < a.nvec) a.out[base + p * a.group] = Pairs<kType>::store(o[p]);
    }
    if (kU) {
      float s[1] = {ss.x + ss.y};
      group_sum(s, a.group, which, part[call++ & 1]);
      const float r2 = __frsqrt_rn(s[0] * inv_d + a.eps);
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
#pragma unroll
        for (int i = 0; i < n; ++i) o[p][i] = mul2(pre[p][i], mul2(o[p][i], both(r2)));
        if (at + p * a.group < a.nvec) a.u[base + p * a.group] = Pairs<kType>::store(o[p]);
      }
    }
    ring.next();
    if (kY && !kByRow && row + 1 == gate_end && row + 1 < r1) {
      ++gate_row;
      gate_end += a.gate_rows;
      load_w();
    }
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------- backward
//
// What the gradient needs of a whole row is linear in sums that the loaded values give at once,
//   mean(m gamma_post dv) = r1 / d (sum w y dout + r2 sum w y (gamma_pre du) - (r2 c) (r2 sum w y out)),
//   w = gamma_post gate,
// so six sums of a row go through one reduction and one barrier. The gate's and gamma_post's gradients
// come from the same sum over the rows of a gate row, P = sum g m: dgate = gamma_post P, dgamma_post +=
// gate P, held in registers over a unit like gamma_pre's.
// The sums over the units follow in a second launch, in the order of the units: no atomics, the same
// bits in every run. With one gate row (or none) that launch gets the sums P; with several, a
// gate row whose rows lie in one unit is written at once, and the others leave a partial sum per unit
// (the unit's first gate row in slot 2 u, its last one in 2 u + 1).
struct GradArgs {
  const uint4 *y, *out, *dout, *du;
  const float *gamma_post, *gate, *gamma_pre;
  uint4 *dx, *dy;
  float *part_post, *part_pre;  // [CTAs][d], or NULL where not wanted (part_post: sums P with one gate row)
  float *dgate, *slots;         // [gate rows][d] or NULL; [2 units][d]
  int R, d, nvec, gate_rows, group;
  Units units;
  float scale, eps;
};

// kNext: du is there; kPost: y goes through its norm; kGates: one gate row or none, several, one per row, or no
// y at all. (What else is missing counts as zeros.)
enum { kOneGate, kSeveralGates, kGateByRow, kNoY };
// CTAs of 256 threads for which an SM has registers: three where 80 a thread do without spills (16384 rows
// of 2048 bf16 columns, the norm before a block alone: 51.6 us with two, 49.4 with three; the norm after it 57.7 and
// 51.9).
constexpr int grad_ctas(int type, int pieces, bool next, int gates) {
  if (pieces > 1) return 1;
  if (type == 2) return !next || gates == kOneGate || gates == kNoY ? 3 : 2;
  return (next && gates == kNoY) || (!next && gates == kOneGate) ? 3 : 2;
}
template <int kType, int kPieces, int kDepth, bool kNext, bool kPost, int kGates>
__global__ void __launch_bounds__(kPieces == 1 ? 256 : kMaxThreads, grad_ctas(kType, kPieces, kNext, kGates))
    norm_backward_kernel(const GradArgs a) {
  constexpr int n = Pairs<kType>::n, N = 2 * n;
  constexpr bool kByRow = kGates == kGateByRow, kY = kGates != kNoY;
  constexpr int kTensors = (kNext ? 3 : 1) + kY, kYAt = kNext ? 3 : 1;  // dout, out, du, y
  extern __shared__ __align__(16) uint8_t smem[];  // the ring; at the end [2][d] sums, where a CTA has several groups
  __shared__ float part[2][16][8];
  grid_dependents_launch();
  Ring<kTensors, kPieces, kDepth, kByRow ? n / 2 : 0> ring(smem);
  const int which = threadIdx.x / a.group, at = threadIdx.x - which * a.group;
  const int groups = blockDim.x / a.group, unit = blockIdx.x * groups + which;
  grid_dependency_wait();
  const int r0 = unit < a.units.count ? a.units.first(unit) : 0;
  const int r1 = unit < a.units.count ? a.units.first(unit + 1) : 0;
  const uint4* rows[kTensors];
  rows[0] = a.dout;
  if constexpr (kNext) {
    rows[1] = a.out;
    rows[2] = a.du;
  }
  if constexpr (kY) rows[kYAt] = a.y;
  const auto* const gates = reinterpret_cast<const uint4*>(a.gate);
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i)
    ring.request(rows, gates, static_cast<size_t>(r0 + i) * a.nvec, at, a.nvec, a.group, r0 + i < r1);
  // of the thread's columns: gamma_pre, gamma_post times the gate; sums of du n, of g m over a gate row, of dv m
  float2 pre[kPieces][n], w[kPieces][n], acc_pre[kPieces][n], acc[kPieces][n], acc_post[kPieces][n];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
#pragma unroll
    for (int i = 0; i < n; ++i) acc_pre[p][i] = acc[p][i] = acc_post[p][i] = pre[p][i] = both(0.f);
    if (kNext && at + p * a.group < a.nvec) load_pairs(a.gamma_pre + (at + p * a.group) * N, pre[p]);
  }
  const int first_gate = kGates == kSeveralGates ? r0 / a.gate_rows : 0;
  int gate_row = first_gate, gate_end = (first_gate + 1) * a.gate_rows;
  const float inv_d = 1.f / a.d;
  if (kY && r0 < r1) factors<kPieces, n, kPost, !kByRow>(a, gate_row, at, w);
#pragma unroll 1
  for (int row = r0; row < r1; ++row) {
    ring.request(rows, gates, static_cast<size_t>(row + kDepth - 1) * a.nvec, at, a.nvec, a.group,
                 row + kDepth - 1 < r1);
    ring.wait();
    const int slot = ring.slot;
    float2 g[kPieces][n], y[kPieces][n], o[kPieces][n], f[kPieces][n];
    const auto load = [&](int p) {
      Pairs<kType>::load(ring.piece(slot, 0, p), g[p]);
      if (kY) Pairs<kType>::load(ring.piece(slot, kYAt, p), y[p]);
      if (kNext) {
        Pairs<kType>::load(ring.piece(slot, 1, p), o[p]);
        Pairs<kType>::load(ring.piece(slot, 2, p), f[p]);
      }
    };
    // out^2, (gamma_pre du) out, y^2, and w y times dout, gamma_pre du and out
    float2 t[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) t[i] = both(0.f);
    if (kNext || kPost) {
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        load(p);
        float2 q[n];
        if constexpr (kByRow && kPost) ring.times_gate(p, w[p], q);
#pragma unroll
        for (int i = 0; i < n; ++i) {
          float2 wd;
          if (kNext) {
            wd = mul2(pre[p][i], f[p][i]);
            t[0] = fma2(o[p][i], o[p][i], t[0]);
            t[1] = fma2(wd, o[p][i], t[1]);
          }
          if (kPost) {
            const float2 wy = mul2(kByRow ? q[i] : w[p][i], y[p][i]);
            t[2] = fma2(y[p][i], y[p][i], t[2]);
            t[3] = fma2(wy, g[p][i], t[3]);
            if (kNext) {
              t[4] = fma2(wy, wd, t[4]);
              t[5] = fma2(wy, o[p][i], t[5]);
            }
          }
        }
      }
    }
    float s[6];
#pragma unroll
    for (int i = 0; i < 6; ++i) s[i] = t[i].x + t[i].y;
    if (kNext || kPost) group_sum(s, a.group, which, part[row & 1]);
    // ra c and rb mean(m w g), which meet n and m below: with the powers of the inverse roots taken together instead (r^3
    // times a row's sum, times the row) rows of 1e14 lost digits, and rows of 1e-14 without eps gave infinities. The
    // products with r are 1.2 % of the time (16384 rows of 2048 bf16 columns 71.5 -> 72.4 us).
    const float ra = kNext ? __frsqrt_rn(s[0] * inv_d + a.eps) : 0.f, ca = ra * (ra * (s[1] * inv_d));
    const float rb = kPost ? __frsqrt_rn(s[2] * inv_d + a.eps) : 1.f;
    const float cb = kPost ? rb * (rb * (fmaf(ra, s[4], fmaf(-ca, ra * s[5], s[3])) * inv_d)) : 0.f;
    const size_t base = static_cast<size_t>(row) * a.nvec + at;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      // one piece stays in registers from the sums above; several are read again
      if (kPieces > 1 || !(kNext || kPost)) load(p);
      const bool on = at + p * a.group < a.nvec;
      if (kNext) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float2 fr = mul2(f[p][i], both(ra));
          acc_pre[p][i] = fma2(fr, o[p][i], acc_pre[p][i]);
          g[p][i] = fma2(both(-ca), mul2(o[p][i], both(ra)), fma2(pre[p][i], fr, g[p][i]));
        }
      }
      if (a.dx && on) {
        float2 v[n];
#pragma unroll
        for (int i = 0; i < n; ++i) v[i] = mul2(g[p][i], both(a.scale));
        a.dx[base + p * a.group] = Pairs<kType>::store(v);
      }
      if constexpr (kByRow) {
        float2 one[n], q[n], dq[n];
#pragma unroll
        for (int i = 0; i < n; ++i) one[i] = both(1.f);
        ring.times_gate(p, one, q);
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float2 gr = mul2(g[p][i], both(rb)), gm = mul2(gr, y[p][i]);
          acc_post[p][i] = fma2(q[i], gm, acc_post[p][i]);
          dq[i] = kPost ? mul2(w[p][i], gm) : gm;
          const float2 wg = mul2(kPost ? mul2(q[i], w[p][i]) : q[i], gr);
          y[p][i] = kPost ? fma2(both(-cb), mul2(y[p][i], both(rb)), wg) : wg;
        }
        if (a.dgate && on) store_pairs(a.dgate + (base + p * a.group) * N, dq);
      } else if constexpr (kY) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float2 gr = mul2(g[p][i], both(rb));
          acc[p][i] = fma2(gr, y[p][i], acc[p][i]);
          const float2 wg = mul2(w[p][i], gr);
          y[p][i] = kPost ? fma2(both(-cb), mul2(y[p][i], both(rb)), wg) : wg;
        }
      }
      if (kY && a.dy && on) a.dy[base + p * a.group] = Pairs<kType>::store(y[p]);
    }
    ring.next();
    if (kGates == kSeveralGates && (row + 1 == gate_end || row + 1 == r1)) {  // a gate row ends, or its part of the unit
      const int last = min(gate_end, a.R) - 1;
      const bool whole = gate_row * a.gate_rows >= r0 && last < r1;
      float* const dst = !a.dgate ? nullptr
                         : whole  ? a.dgate + static_cast<size_t>(gate_row) * a.d
                                  : a.slots + (static_cast<size_t>(2 * unit) + (gate_row != first_gate)) * a.d;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int c = at + p * a.group;
        if (c < a.nvec) {
          float2 q[n];
          load_pairs(a.gate + static_cast<size_t>(gate_row) * a.d + c * N, q);
#pragma unroll
          for (int i = 0; i < n; ++i) acc_post[p][i] = fma2(q[i], acc[p][i], acc_post[p][i]);
          if (dst) {
            if (kPost) {
              load_pairs(a.gamma_post + c * N, q);
#pragma unroll
              for (int i = 0; i < n; ++i) acc[p][i] = mul2(acc[p][i], q[i]);
            }
            store_pairs(dst + c * N, acc[p]);
          }
        }
#pragma unroll
        for (int i = 0; i < n; ++i) acc[p][i] = both(0.f);
      }
      if (row + 1 < r1) {
        ++gate_row;
        gate_end += a.gate_rows;
        factors<kPieces, n, kPost, true>(a, gate_row, at, w);
      }
    }
  }
  cp_async_wait<0>();
  if (groups == 1) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int c = at + p * a.group;
      if (c >= a.nvec) continue;
      const size_t dst = static_cast<size_t>(blockIdx.x) * a.d + c * N;
      if (a.part_post) store_pairs(a.part_post + dst, kGates ? acc_post[p] : acc[p]);
      if (a.part_pre) store_pairs(a.part_pre + dst, acc_pre[p]);
    }
    return;
  }
  auto* const gammas = reinterpret_cast<float*>(smem);
  __syncthreads();  // the groups' rings are read
  for (int q = 0; q < groups; ++q) {  // the groups' sums in order
    if (q == which)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int c = at + p * a.group;
        if (c >= a.nvec) continue;
        float2 post[n], before[n];
#pragma unroll
        for (int i = 0; i < n; ++i) post[i] = before[i] = both(0.f);
        if (q) {
          load_pairs(gammas + c * N, post);
          load_pairs(gammas + a.d + c * N, before);
        }
#pragma unroll
        for (int i = 0; i < n; ++i) {
          post[i] = fma2(both(1.f), kGates ? acc_post[p][i] : acc[p][i], post[i]);
          before[i] = fma2(both(1.f), acc_pre[p][i], before[i]);
        }
        store_pairs(gammas + c * N, post);
        store_pairs(gammas + a.d + c * N, before);
      }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    if (a.part_post) a.part_post[static_cast<size_t>(blockIdx.x) * a.d + c] = gammas[c];
    if (a.part_pre) a.part_pre[static_cast<size_t>(blockIdx.x) * a.d + c] = gammas[a.d + c];
  }
}

// The second launch. First, by CTAs of 16 columns: the sums over the CTAs, for gamma_post (and the gate, where it
// has one row) and for gamma_pre, in 64 slices that meet in a fixed tree. Then the gate rows with partial
// sums: in the same way, where a gate row spreads over many units; else (`thin`) a CTA of 1024 columns for
// every unit whose last gate row goes on in the next one.
struct SumArgs {
  const float *part_post, *part_pre, *slots;
  const float *gamma_post, *gate;  // the factors of P with one gate row (NULL: one)
  float *dgamma_post, *dgamma_pre, *dgate;
  int R, d, gate_rows, ctas, columns;  // columns: CTAs of 16 columns
  Units units;
  bool thin;
};

__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x;
  a.y += b.y;
  a.z += b.z;
  a.w += b.w;
}

__global__ void __launch_bounds__(256) norm_sum_kernel(const SumArgs a) {
  __shared__ float4 part[8][4];
  grid_dependents_launch();
  grid_dependency_wait();
  const int kind = blockIdx.x / a.columns;  // 0, 1: gamma_post, gamma_pre; from 2 on: gate rows
  int u0 = 0, u1 = a.ctas - 1, g = kind - 2;
  bool earlier = false;  // whether the first unit began with an earlier gate row: its part is in the second slot then
  if (kind >= 2) {
    const int i = (blockIdx.x - 2 * a.columns) / ((a.d + 1023) / 1024);  // thin: the unit
    if (a.thin) g = a.units.first(i + 1) / a.gate_rows;
    const int begin = g * a.gate_rows;
    // nothing goes on, or an earlier unit's CTA has it
    if (a.thin && (begin == a.units.first(i + 1) || begin < a.units.first(i))) return;
    u0 = a.units.of(begin);
    u1 = a.units.of(min(begin + a.gate_rows, a.R) - 1);
    if (u0 == u1) return;  // written by its unit
    earlier = a.units.first(u0) < begin;
    if (a.thin) {
      const int col = (blockIdx.x - 2 * a.columns - i * ((a.d + 1023) / 1024)) * 1024 + threadIdx.x * 4;
      if (col >= a.d) return;
      float4 s = *reinterpret_cast<const float4*>(a.slots + static_cast<size_t>(2 * u0 + earlier) * a.d + col);
#pragma unroll 4
      for (int u = u0 + 1; u <= u1; ++u)
        add4(s, *reinterpret_cast<const float4*>(a.slots + static_cast<size_t>(2 * u) * a.d + col));
      *reinterpret_cast<float4*>(a.dgate + static_cast<size_t>(g) * a.d + col) = s;
      return;
    }
  }
  const int lane = threadIdx.x & 3, slice = threadIdx.x >> 2, warp = threadIdx.x >> 5;
  const int col = (blockIdx.x - kind * a.columns) * 16 + lane * 4;
  const bool on = col < a.d;
  const float* const src = kind >= 2 ? a.slots : kind == 0 ? a.part_post : a.part_pre;
  if (!src) return;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on)
#pragma unroll 5
    for (int u = u0 + slice; u <= u1; u += 64) {
      size_t at = u;
      if (kind >= 2) at = 2 * at + (u == u0 && earlier);
      add4(s, *reinterpret_cast<const float4*>(src + at * a.d + col));
    }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1)
    add4(s, make_float4(__shfl_xor_sync(0xffffffffu, s.x, off), __shfl_xor_sync(0xffffffffu, s.y, off),
                        __shfl_xor_sync(0xffffffffu, s.z, off), __shfl_xor_sync(0xffffffffu, s.w, off)));
  if ((threadIdx.x & 31) < 4) part[warp][lane] = s;
  __syncthreads();
  if (slice != 0 || !on) return;
  s = part[0][lane];
#pragma unroll
  for (int k = 1; k < 8; ++k) add4(s, part[k][lane]);
  const auto put = [&](float* dst, const float* factor) {
    float4 v = s;
    if (factor) {
      const float4 f = *reinterpret_cast<const float4*>(factor + col);
      v = make_float4(s.x * f.x, s.y * f.y, s.z * f.z, s.w * f.w);
    }
    *reinterpret_cast<float4*>(dst + col) = v;
  };
  if (kind >= 2)
    put(a.dgate + static_cast<size_t>(g) * a.d, nullptr);
  else if (kind == 1)
    put(a.dgamma_pre, nullptr);
  if (kind == 0 && a.dgamma_post) put(a.dgamma_post, a.gate);
  if (kind == 0 && a.dgate && a.gate_rows >= a.R) put(a.dgate, a.gamma_post);
}

// Threads of a group, groups of a CTA and CTAs.
struct GroupShape {
  int pieces, group, groups, ctas;
  Units units;
};
GroupShape group_shape(int rows, int nvec, int pieces, int max_ctas) {
  GroupShape g;
  g.pieces = pieces;
  g.group = (nvec + 32 * pieces - 1) / (32 * pieces) * 32;
  g.groups = g.group >= 256 ? 1 : 256 / g.group;
  if (g.groups > rows) g.groups = rows > 0 ? rows : 1;
  g.ctas = (rows + g.groups - 1) / g.groups;
  if (g.ctas < 1) g.ctas = 1;
  if (g.ctas > max_ctas) g.ctas = max_ctas;
  const int units = std::min(g.ctas * g.groups, rows > 0 ? rows : 1);
  g.units = Units{units, rows / units, rows % units};
  return g;
}

constexpr int kSmem = 200 * 1024;  // of dynamic shared memory at most

// `room` says on which devices the kernel has been given room for its shared memory.
template <class K, class A>
cudaError_t launch(K kernel, std::atomic<uint64_t>& room, const GroupShape& g, size_t smem, cudaStream_t st,
                   const A& a) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (!(room.load(std::memory_order_acquire) & bit)) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    room.fetch_or(bit, std::memory_order_release);
  }
  return launch_pdl(kernel, dim3(g.ctas), dim3(g.group * g.groups), smem, st, a);
}

// CTAs that an SM holds at a time: each of its four parts has registers for so many warps, and a group's barrier is
// chosen at run time, so a CTA has 16 of the SM's 64.
int fitting(int registers, int threads, size_t smem) {
  const int warps = 4 * std::min(512 / registers, 16);
  return std::max(std::min({warps / (threads / 32), 226 * 1024 / (int(smem) + 2048), 4}), 1);
}

// kGates: with a gate row per row, without, or either.
enum { kNeverByRow, kAlwaysByRow, kMaybeByRow };
template <int kType, int kPieces, int kDepth, int kGates>
cudaError_t forward(Args a, cudaStream_t st) {
  const bool by_row = kGates == kMaybeByRow ? a.gate && a.gate_rows == 1 : kGates == kAlwaysByRow;
  GroupShape g = group_shape(a.R, a.nvec, kPieces, INT32_MAX);
  const int threads = g.group * g.groups;
  const size_t smem = size_t(kDepth) * (2 + (by_row ? kType == 2 ? 1 : 2 : 0)) * kPieces * threads * 16;
  const int registers = kPieces == 4   ? 128
                        : kPieces == 2 ? (kType == 2 ? 72 : by_row ? 112 : 96)
                                       : (kType == 2 ? 48 : 72);
  g = group_shape(a.R, a.nvec, kPieces, kNormSms * fitting(registers, threads, smem));
  a.group = g.group;
  a.units = g.units;
  static std::atomic<uint64_t> room[6];
  if constexpr (kGates != kNeverByRow)
    if (by_row)
      return a.u ? launch(norm_kernel<kType, kPieces, kDepth, true, true, true>, room[0], g, smem, st, a)
                 : launch(norm_kernel<kType, kPieces, kDepth, true, false, true>, room[1], g, smem, st, a);
  if constexpr (kGates != kAlwaysByRow) {
    if (!a.y)
      return a.u ? launch(norm_kernel<kType, kPieces, kDepth, false, true, false>, room[2], g, smem, st, a)
                 : launch(norm_kernel<kType, kPieces, kDepth, false, false, false>, room[3], g, smem, st, a);
    return a.u ? launch(norm_kernel<kType, kPieces, kDepth, true, true, false>, room[4], g, smem, st, a)
               : launch(norm_kernel<kType, kPieces, kDepth, true, false, false>, room[5], g, smem, st, a);
  }
}
// Pieces per thread: four, where there are rows enough (a barrier less often), two where four would leave a fifth of
// the threads without columns (8000 rows of 1344 bf16 columns 15.8 -> 14.6 us), one where latency counts.
template <int kType>
cudaError_t forward(const Args& a, cudaStream_t st) {
  if (a.nvec <= 32 || (a.nvec <= 512 && a.R <= 4 * kNormSms)) return forward<kType, 1, 3, kMaybeByRow>(a, st);
  const bool by_row = a.gate && a.gate_rows == 1;  // the ring holds the gate too
  const bool full = 4 * ((a.nvec + 127) / 128 * 128) <= 5 * a.nvec;
  if ((a.nvec <= 256 && !full) || (by_row && a.nvec <= 1024)) return forward<kType, 2, 3, kMaybeByRow>(a, st);
  if constexpr (kType == 2)  // (rows of 16 bits have 1024 pieces at most)
    if (by_row) return forward<2, 4, 2, kAlwaysByRow>(a, st);
  return forward<kType, 4, 3, kNeverByRow>(a, st);
}

// Rows of a ring: with four tensors four rows of one piece, three of two (two with the gates) and one of four (a row of
// 8192 fp32 columns takes 128 KB); with fewer tensors, what fits in the same memory.
constexpr int grad_tensors(bool next, int gates) { return (next ? 3 : 1) + (gates != kNoY); }
constexpr int grad_parts(int type, bool next, int gates) {  // 16-byte parts of a piece
  return grad_tensors(next, gates) + (gates == kGateByRow ? type == 2 ? 1 : 2 : 0);
}
constexpr int grad_depth(int type, int pieces, bool next, int gates) {
  const int all = grad_parts(type, true, gates == kGateByRow ? kGateByRow : kOneGate);
  const int most = pieces == 1 ? 4 * all : pieces == 2 ? gates == kGateByRow ? 2 * all : 12 : all;
  return std::max(most / grad_parts(type, next, gates), 1);
}
size_t grad_ring(int type, int pieces, bool next, int gates, int threads) {
  return size_t(grad_depth(type, pieces, next, gates)) * grad_parts(type, next, gates) * pieces * threads * 16;
}
// As many CTAs as fit (7518 rows of 1344 fp32 columns 40.4 -> 32.7 us against one per SM). One piece per thread
// where the rows fill 128 or 256 threads; between them two, in smaller groups of which more fit (8000
// rows of 1200 fp16 columns 39.6 -> 31.2 us; at 2048 columns one is better by 6 % with several gate rows).
GroupShape grad_shape(const NormDims& s, bool next, int gates) {
  const int nvec = s.nvec(), pieces = nvec <= 128 || (nvec > 192 && nvec <= 256) ? 1 : nvec <= 1024 ? 2 : 4;
  const GroupShape g = group_shape(s.R, nvec, pieces, INT32_MAX);
  const int threads = g.group * g.groups;
  const int registers = grad_ctas(s.type, pieces, next, gates) == 3 ? 80 : s.type == 2 && pieces == 1 ? 96 : 128;
  const int fit = fitting(registers, threads, grad_ring(s.type, pieces, next, gates, threads));
  return group_shape(s.R, nvec, pieces, kNormSms * fit);
}

template <int kType, int kPieces, int kGates, bool kNext, bool kPost>
cudaError_t backward(const GradArgs& a, const GroupShape& g, cudaStream_t st) {
  constexpr int kDepth = grad_depth(kType, kPieces, kNext, kGates);
  static_assert(kDepth <= 16, "registers of the ring");
  static std::atomic<uint64_t> room;
  return launch(norm_backward_kernel<kType, kPieces, kDepth, kNext, kPost, kGates>, room, g,
                std::max(grad_ring(kType, kPieces, kNext, kGates, g.group * g.groups), size_t(8) * a.d), st, a);
}
template <int kType, int kPieces, int kGates>
cudaError_t backward(const GradArgs& a, const GroupShape& g, cudaStream_t st) {
  const bool next = a.du, post = a.gamma_post;
  return next ? post ? backward<kType, kPieces, kGates, true, true>(a, g, st)
                     : backward<kType, kPieces, kGates, true, false>(a, g, st)
              : post ? backward<kType, kPieces, kGates, false, true>(a, g, st)
                     : backward<kType, kPieces, kGates, false, false>(a, g, st);
}
template <int kType, int kPieces>
cudaError_t backward(const GradArgs& a, const GroupShape& g, int gates, cudaStream_t st) {
  if (gates == kNoY) return backward<kType, kPieces, kNoY, true, false>(a, g, st);
  return gates == kOneGate        ? backward<kType, kPieces, kOneGate>(a, g, st)
         : gates == kSeveralGates ? backward<kType, kPieces, kSeveralGates>(a, g, st)
                                  : backward<kType, kPieces, kGateByRow>(a, g, st);
}

}  // namespace

cudaError_t launch_norm(const NormDims& s, const void* x, const void* y, const float* gamma_post, const float* gate,
                        const float* gamma_pre, void* out, void* u, cudaStream_t st) {
  const Args a{static_cast<const uint4*>(x), static_cast<const uint4*>(y), gamma_post, gate, gamma_pre,
               static_cast<uint4*>(out), static_cast<uint4*>(u), s.R, s.d, s.nvec(), gate ? s.gate_rows : s.R, 0,
               Units{}, s.scale, s.eps};
  return s.type == 0 ? forward<0>(a, st) : s.type == 1 ? forward<1>(a, st) : forward<2>(a, st);
}

// Workspace: sums P (or of gamma_post) by CTA | of gamma_pre by CTA | gate slots by unit; of the call that has most.
size_t norm_backward_ws_bytes(const NormDims& s) {
  size_t most = 0;
  const auto take = [&](bool next, int gates) {
    const GroupShape g = grad_shape(s, next, gates);
    most = std::max(most, (size_t(g.ctas) + g.units.count) * 2 * s.d * 4);
  };
  take(false, kOneGate);
  take(true, kOneGate);
  take(true, kNoY);
  if (s.gate_rows < s.R)
    for (bool next : {false, true}) take(next, s.gate_rows > 1 ? kSeveralGates : kGateByRow);
  return most;
}

cudaError_t launch_norm_backward(const NormDims& s, const void* y, const float* gamma_post, const float* gate,
                                 const void* out, const float* gamma_pre, const void* dout, const void* du, void* dx,
                                 void* dy, float* dgamma_post, float* dgate, float* dgamma_pre, void* workspace,
                                 cudaStream_t st) {
  const bool several = gate && s.gate_rows < s.R;
  const bool needs_y = (dy && gamma_post) || dgamma_post || dgate;
  const int all = !several ? kOneGate : s.gate_rows > 1 ? kSeveralGates : kGateByRow;
  const int gates = du && !needs_y && !dy ? kNoY : all;
  // The inputs alone decide who takes which rows: an output has the same bits whichever others are wanted.
  const GroupShape g = grad_shape(s, du, du && !y && !gamma_post && !gate ? kNoY : all);
  auto* const ws = static_cast<float*>(workspace);
  float* const pre = ws + size_t(g.ctas) * s.d;
  float* const slots = pre + size_t(g.ctas) * s.d;
  GradArgs a{};
  a.y = needs_y ? static_cast<const uint4*>(y) : nullptr;
  a.out = static_cast<const uint4*>(out);
  a.dout = static_cast<const uint4*>(dout);
  a.du = static_cast<const uint4*>(du);
  a.gamma_post = needs_y ? gamma_post : nullptr;
  a.gate = gate;
  a.gamma_pre = gamma_pre;
  a.dx = static_cast<uint4*>(dx);
  a.dy = static_cast<uint4*>(dy);
  a.part_post = dgamma_post || (dgate && !several) ? ws : nullptr;
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
    if (g.pieces == 1) return backward<kType, 1>(a, g, gates, st);
    if (kType < 2 || g.pieces == 2) return backward<kType, 2>(a, g, gates, st);  // 8192 16-bit columns at most
    return backward<2, 4>(a, g, gates, st);
  };
  if (s.type == 0)
    err = run(std::integral_constant<int, 0>{});
  else if (s.type == 1)
    err = run(std::integral_constant<int, 1>{});
  else
    err = run(std::integral_constant<int, 2>{});
  if (err != cudaSuccess || (!dgamma_post && !dgamma_pre && !dgate)) return err;
  const int columns = (s.d + 15) / 16, gate_count = (s.R + a.gate_rows - 1) / a.gate_rows;
  const bool thin = int64_t(g.units.count) * a.gate_rows <= int64_t(8) * s.R;  // a gate row in some eight units at most
  const int shared = !dgate || !several || a.gate_rows == 1 ? 0  // (a gate row of one row is in one unit)
                     : thin ? (g.units.count - 1) * ((s.d + 1023) / 1024) : gate_count * columns;
  const SumArgs b{a.part_post, a.part_pre, slots, gamma_post, several ? nullptr : gate, dgamma_post, dgamma_pre, dgate,
                  s.R, s.d, a.gate_rows, g.ctas, columns, g.units, thin};
  return launch_pdl(norm_sum_kernel, dim3(2 * columns + shared), dim3(256), 0, st, b);
}

}  // namespace moe
