// linear.cu -- products of token rows with weights, on the tcgen05 tensor cores, with
// bias, activation, gate and residual in the epilogue, and the two products of the
// gradient.  Rows are sorted by expert (one weight per expert) or share one weight.
//
//   forward      out[r][n]   = act(sum_k W[n][k] x[r][k] + b[n]) (gated: times the up product) + residual[r][n]
//   input grad   dx[r][k]    = sum_n W[n][k] dz[r][n]
//   weight grad  dW[e][n][k] = sum_{r in e} x[r][k] dz[r][n]
//
// All three are one kernel, D[m][c] = sum_j A[m][j] B[c][j], with m the contiguous
// index of the output (n, k, k) on the 128 lanes of tensor memory and c its row
// (r, r, n) on the columns; A is W or x, B is x or dz, and an operand whose
// contraction index j is not its contiguous one is read as it lies (the matrix
// instructions take either order), so nothing is transposed in memory.  The rows are
// the short side for few tokens: a tile of 32 columns costs little more than the
// weights' way from memory, and a column past an expert's last row is computed from
// its neighbour's data and not stored.
//
// One persistent CTA (or pair of CTAs) per SM walks a list of tiles: a warp loads
// 64-element stages of A and B by TMA, one thread issues the matrix instructions into
// one of two accumulators in tensor memory, and eight warps empty the other one: 32
// columns at a time through shared memory, so that the outputs leave as 16-byte pieces
// of contiguous rows.  Accumulation, bias, activation and residual are in fp32,
// rounded once.
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "activation.cuh"
#include "internal.h"
#include "row_vec.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {

constexpr int kForward = 0, kInputGrad = 1, kWeightGrad = 2;
constexpr int kTileM = 128;            // lanes of tensor memory
constexpr int kDepth = 64;             // contraction elements per stage (128 bytes)
constexpr int kABytes = kTileM * 128;  // A per stage
constexpr int kEpiCols = 32;           // columns per epilogue step
constexpr int kEpiBytes = kEpiCols * kTileM * 4;
constexpr int kThreads = 384;          // TMA, MMA, tail and one idle warp, then 8 epilogue warps
constexpr int kSmemLimit = 227 * 1024;

struct Args {
  const int32_t* offsets;  // NULL: one weight for all rows
  const float* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* preact;
  int32_t* err;
  int mode, R, E, K, N, Nw, act, gated, bf16;
  int width;    // extent of m, and the row length of out
  int tile_m;   // outputs per CTA tile (64 of a gate and their ups, or 128)
  int tiles_m;  // tiles along m, of the CTA or pair
  int tiles_c;  // weight grad: tiles along c
  int depth;    // contraction length (weight grad: the expert's rows)
  uint32_t word;
};

template <int kCols, int kCtas>
struct Config {
  static constexpr int cols = kCols / kCtas;  // columns whose B rows this CTA loads
  static constexpr int b_bytes = cols * 128;
  static constexpr int stage = kABytes + b_bytes;
  static constexpr int fixed = 2 * kEpiBytes + (2 * (kMaxExperts + 1) + 2) * 4 + 256;
  static constexpr int fit = (kSmemLimit - fixed) / stage;
  static constexpr int stages = fit < 8 ? fit : 8;
  static constexpr int smem = stages * stage + fixed;
  static constexpr uint32_t tmem = 2 * kCols;  // two accumulators
};

struct Tile {
  int e, m0, c0, row0, row_end, first, len;  // len: contraction length, first: its first row (weight grad)
};

// The tile of index t.  start[e]: tiles before expert e; off[e]: its first row.
__device__ __forceinline__ Tile tile_at(const Args& a, const int* start, const int* off, int t, int& e, int cols,
                                        int ctas, int rank) {
  while (t >= start[e + 1]) ++e;  // t only grows
  const int i = t - start[e];
  const int m = i % a.tiles_m, c = i / a.tiles_m;
  Tile r;
  r.e = e;
  r.m0 = (m * ctas + rank) * a.tile_m;
  if (a.mode == kWeightGrad) {
    r.c0 = c * cols;
    r.row0 = e * a.Nw + r.c0;
    r.row_end = (e + 1) * a.Nw;
    r.first = off[e];
    r.len = off[e + 1] - off[e];
  } else {
    r.c0 = off[e] + c * cols;
    r.row0 = r.c0;
    r.row_end = off[e + 1];
    r.first = 0;
    r.len = a.depth;
  }
  return r;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8], int bf16) {
  return bf16 ? Vec<1>::store(f) : Vec<0>::store(f);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8], int bf16) {
  if (bf16)
    Vec<1>::load(v, f);
  else
    Vec<0>::load(v, f);
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// Barrier of a group of 128 threads that tells each whether `ok` held for all, so that a
// group whose bounded wait ran out for one thread leaves together.
__device__ __forceinline__ bool group_all(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(ok)), "r"(id)
      : "memory");
  return r != 0;
}

// One epilogue step: rows row0 .. row0+31 (those below row_end) of the tile's outputs
// from the accumulator step in buf [32][128].  A thread owns eight contiguous outputs
// m0 + f .. of one row in `per` passes, with their biases in registers.
__device__ __forceinline__ void store_step(const Args& a, const float* buf, int tid, int m0, int row0, int row_end,
                                           const float (&b)[8], const float (&bu)[8]) {
  const int groups = a.gated ? 8 : 16;  // threads per row
  const int f = (tid % groups) * 8, rows = 128 / groups;
  if (m0 + f >= a.width) return;
  for (int c = tid / groups; c < kEpiCols; c += rows) {
    const int row = row0 + c;
    if (row >= row_end) break;
    const size_t o = static_cast<size_t>(row) * a.width + m0 + f;
    uint4 res = make_uint4(0u, 0u, 0u, 0u);
    if (a.residual) res = *reinterpret_cast<const uint4*>(a.residual + o);
    const float4 p = *reinterpret_cast<const float4*>(buf + c * kTileM + f);
    const float4 q = *reinterpret_cast<const float4*>(buf + c * kTileM + f + 4);
    float z[8] = {p.x + b[0], p.y + b[1], p.z + b[2], p.w + b[3], q.x + b[4], q.y + b[5], q.z + b[6], q.w + b[7]};
    float y[8];
    if (a.preact) {
      const size_t zo = static_cast<size_t>(row) * a.Nw + m0 + f;
      *reinterpret_cast<uint4*>(a.preact + zo) = pack8(z, a.bf16);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = activate(z[i], a.act);
    if (a.gated) {
      const float4 r = *reinterpret_cast<const float4*>(buf + c * kTileM + 64 + f);
      const float4 s = *reinterpret_cast<const float4*>(buf + c * kTileM + 64 + f + 4);
      float u[8] = {r.x + bu[0], r.y + bu[1], r.z + bu[2], r.w + bu[3],
                    s.x + bu[4], s.y + bu[5], s.z + bu[6], s.w + bu[7]};
      if (a.preact)
        *reinterpret_cast<uint4*>(a.preact + static_cast<size_t>(row) * a.Nw + a.N + m0 + f) = pack8(u, a.bf16);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= u[i];
    }
    if (a.residual) {
      float g[8];
      unpack8(res, g, a.bf16);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] += g[i];
    }
    *reinterpret_cast<uint4*>(a.out + o) = pack8(y, a.bf16);
  }
}

template <int kCols, int kCtas>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ Args a,
                                                             const __grid_constant__ CUtensorMap map_a,
                                                             const __grid_constant__ CUtensorMap map_b) {
  using C = Config<kCols, kCtas>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const epi = smem + C::stages * C::stage;
  int* const start = reinterpret_cast<int*>(epi + 2 * kEpiBytes);  // [E + 1]
  int* const off = start + kMaxExperts + 1;                        // [E + 1]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(off + kMaxExperts + 1 + 2);
  const uint32_t bar0 = smem_addr(bars);
  const auto full = [&](int s) { return bar0 + 8u * s; };
  const auto empty = [&](int s) { return bar0 + 8u * (8 + s); };
  const auto acc_full = [&](int s) { return bar0 + 8u * (16 + s); };
  const auto acc_empty = [&](int s) { return bar0 + 8u * (18 + s); };
  const uint32_t tail_ready = bar0 + 8u * 20, tail_done = bar0 + 8u * 21, drained = bar0 + 8u * 22;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 23);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = kCtas == 2 ? static_cast<int>(cluster_rank()) : 0;
  grid_dependents_launch();
  if (warp == 1) tmem_alloc<kCtas>(smem_addr(tmem_slot), C::tmem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full(s), 1);
      mbar_init(acc_empty(s), 8 * kCtas);
    }
    mbar_init(tail_ready, 1);
    mbar_init(tail_done, 1);
    mbar_init(drained, 1);
    fence_barrier_init();
  }
  grid_dependency_wait();
  if (warp == 2) {
    // first rows of the experts (clamped to the rows there are) and their tiles: eight
    // experts per lane, then a scan over the lanes
    int o[9], n[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      const int e = lane * 8 + i;
      o[i] = a.offsets ? (e <= a.E ? min(max(a.offsets[e], 0), a.R) : a.R) : (e == 0 ? 0 : a.R);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      const int rows = max(o[i + 1] - o[i], 0);
      n[i] = e < a.E ? a.tiles_m * (a.mode == kWeightGrad ? a.tiles_c : (rows + kCols - 1) / kCols) : 0;
      sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int at = incl - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      if (e < a.E) {
        start[e] = at;
        off[e] = o[i];
        at += n[i];
        if (e == a.E - 1) {
          start[a.E] = at;
          off[a.E] = max(o[i + 1], o[i]);
        }
      }
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  if (kCtas == 2) cluster_sync();  // the peer's barriers are initialised
  tcgen05_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles = start[a.E];
  const int first_tile = blockIdx.x / kCtas, step = gridDim.x / kCtas;

  if (warp == 0) {
    if (lane == 0) {
      // ---- loads
      int e = 0, s = 0;
      uint32_t phase = 0;
      bool alive = true;
      int issued = 0;
      for (int t = first_tile; alive && t < tiles; t += step) {
        const Tile r = tile_at(a, start, off, t, e, kCols, kCtas, rank);
        const int bc = r.c0 + rank * C::cols;
        for (int j = 0; j < r.len; j += kDepth) {
          if (!mbar_wait(empty(s), phase ^ 1, a.err)) {
            alive = false;
            break;
          }
          const uint32_t sa = smem_addr(smem + s * C::stage), sb = sa + kABytes;
          const uint32_t bar = kCtas == 2 ? cluster_addr(full(s), 0) : full(s);
          if (rank == 0) mbar_arrive_expect_tx(full(s), C::stage * kCtas);
          if (a.mode == kForward) {
            tma_load_4d<kCtas>(sa, &map_a, j, r.m0, 0, r.e, bar);
            tma_load_2d<kCtas>(sb, &map_b, j, bc, bar);
          } else if (a.mode == kInputGrad) {
            tma_load_3d<kCtas>(sa, &map_a, r.m0, j, r.e, bar);
            tma_load_3d<kCtas>(sa + kABytes / 2, &map_a, r.m0 + 64, j, r.e, bar);
            tma_load_2d<kCtas>(sb, &map_b, j, bc, bar);
          } else {
            tma_load_2d<kCtas>(sa, &map_a, r.m0, r.first + j, bar);
            tma_load_2d<kCtas>(sa + kABytes / 2, &map_a, r.m0 + 64, r.first + j, bar);
#pragma unroll
            for (int x = 0; x < C::cols / 64; ++x)
              tma_load_2d<kCtas>(sb + x * 8192, &map_b, bc + 64 * x, r.first + j, bar);
          }
          if (issued < C::stages) ++issued;
          if (++s == C::stages) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      if (!alive && rank == 0) {
        // a wait ran out: the copies in flight land before the CTA's shared memory goes
        // (the first CTA of a pair sees the bytes of both)
        for (int i = 0; i < issued; ++i) {
          if (--s < 0) {
            s = C::stages - 1;
            phase ^= 1;
          }
          mbar_wait(full(s), phase, a.err);
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // ---- matrix instructions
      int e = 0, s = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0, tail_phase = 0;
      bool alive = true;
      const bool a_strided = a.mode != kForward, b_strided = a.mode == kWeightGrad;
      const uint32_t a_step = a_strided ? 2048 >> 4 : 32 >> 4, b_step = b_strided ? 2048 >> 4 : 32 >> 4;
      for (int t = first_tile; alive && t < tiles; t += step) {
        const Tile r = tile_at(a, start, off, t, e, kCols, kCtas, rank);
        if (r.len <= 0) continue;  // no rows: the epilogue writes zeros
        if (!mbar_wait(acc_empty(acc), acc_phase ^ 1, a.err)) break;
        tcgen05_fence_after();
        const uint32_t d = tmem + acc * kCols;
        for (int j = 0; j < r.len; j += kDepth) {
          int ks = kDepth / 16;
          if (!mbar_wait(full(s), phase, a.err)) {
            alive = false;
            break;
          }
          if (kCtas == 1 && a.mode == kWeightGrad && r.len - j < kDepth) {
            ks = (r.len - j + 15) / 16;
            mbar_arrive(tail_ready);
            if (!mbar_wait(tail_done, tail_phase, a.err)) {
              alive = false;
              break;
            }
            tail_phase ^= 1;
          }
          tcgen05_fence_after();
          const uint32_t sa = smem_addr(smem + s * C::stage);
          const uint64_t da = smem_operand(sa, a_strided ? kABytes / 2 : 16);
          const uint64_t db = smem_operand(sa + kABytes, b_strided ? 8192 : 16);
          for (int k = 0; k < ks; ++k)
            mma_f16<kCtas>(d, da + k * a_step, db + k * b_step, a.word, (j | k) != 0);
          mma_commit<kCtas>(empty(s));
          if (++s == C::stages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!alive) break;
        mma_commit<kCtas>(acc_full(acc));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (!alive) {  // a wait ran out: the instructions in flight end before tensor memory is given back
        mma_commit<1>(drained);
        mbar_wait(drained, 0, a.err);
      }
    }
  } else if (warp == 2) {
    // ---- weight grad by experts: the last stage of an expert holds rows of the next one
    // (or rows that nobody wrote): zeros, up to a multiple of 16 rows, before it is used.
    // One weight for all rows needs none of this: TMA fills rows past the end with zeros.
    if (kCtas == 1 && a.mode == kWeightGrad) {
      int e = 0, it = 0;
      uint32_t phase = 0;
      for (int t = first_tile; t < tiles; t += step) {
        const Tile r = tile_at(a, start, off, t, e, kCols, kCtas, rank);
        if (r.len <= 0) continue;
        it += (r.len + kDepth - 1) / kDepth;
        const int rest = r.len % kDepth;
        if (rest == 0) continue;
        const int s = (it - 1) % C::stages;
        // the stage is announced, not taken from its own barrier, whose phase repeats
        if (!mbar_wait(tail_ready, phase, a.err)) break;
        phase ^= 1;
        const int z0 = rest * 128, z1 = (rest + 15) / 16 * 16 * 128;
        uint8_t* const base = smem + s * C::stage;
        for (int box = 0; box < C::stage / 8192; ++box)
          for (int z = z0 + lane * 16; z < z1; z += 512)
            *reinterpret_cast<uint4*>(base + box * 8192 + z) = make_uint4(0u, 0u, 0u, 0u);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(tail_done);
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: two groups of four warps take the 32-column steps in turn
    const int group = (warp - 4) >> 2, tid = threadIdx.x & 127, quarter = warp & 3;
    float* const buf = reinterpret_cast<float*>(epi + group * kEpiBytes);
    int e = 0, acc = 0;
    uint32_t acc_phase = 0;
    for (int t = first_tile; t < tiles; t += step) {
      const Tile r = tile_at(a, start, off, t, e, kCols, kCtas, rank);
      float b[8], bu[8];
      const int f = r.m0 + (tid % (a.gated ? 8 : 16)) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] = a.bias && f < a.width ? a.bias[static_cast<size_t>(r.e) * a.Nw + f + i] : 0.f;
        bu[i] = a.bias && a.gated && f < a.width ? a.bias[static_cast<size_t>(r.e) * a.Nw + a.N + f + i] : 0.f;
      }
      if (r.len > 0) {
        const bool ok = mbar_wait(acc_full(acc), acc_phase, a.err);
        __syncwarp();
        if (!group_all(1 + group, ok)) break;
        tcgen05_fence_after();
      }
      for (int c = group * kEpiCols; c < kCols && r.row0 + c < r.row_end; c += 2 * kEpiCols) {
        uint32_t v[32];
        if (r.len > 0) {
          tmem_load_32(tmem + acc * kCols + c + (static_cast<uint32_t>(quarter * 32) << 16), v);
          tmem_load_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
#pragma unroll
        for (int j = 0; j < 32; ++j) buf[j * kTileM + quarter * 32 + lane] = __uint_as_float(v[j]);
        group_sync(1 + group);
        store_step(a, buf, tid, r.m0, r.row0 + c, r.row_end, b, bu);
        group_sync(1 + group);
      }
      if (r.len > 0) {
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 2)
            mbar_arrive_cluster(cluster_addr(acc_empty(acc), 0));
          else
            mbar_arrive(acc_empty(acc));
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (kCtas == 2) cluster_sync();  // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tcgen05_fence_after();
    tmem_dealloc<kCtas>(tmem, C::tmem);
  }
}

// ------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// Map of a row-major array of 16-bit elements: extents from the contiguous one outwards,
// boxes 64 elements wide, 128-byte swizzle, zeros outside.
bool make_map(CUtensorMap* map, bool bf16, const void* base, int rank, const int64_t* dims, const int* box) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  cuuint64_t d[4], st[3];
  cuuint32_t b[4], es[4];
  uint64_t bytes = 2;
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    es[i] = 1;
    bytes *= d[i];
    if (i + 1 < rank) st[i] = bytes;
  }
  return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                  const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int kCols, int kCtas>
cudaError_t launch_tiles(const Args& a, const CUtensorMap& ma, const CUtensorMap& mb, int64_t most_tiles, int num_sms,
                         cudaStream_t st) {
  const int units = num_sms / kCtas;
  const int grid = static_cast<int>(most_tiles < units ? most_tiles : units) * kCtas;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Config<kCols, kCtas>::smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = kCtas == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, linear_kernel<kCols, kCtas>, a, ma, mb);
}

template <int kCols, int kCtas>
cudaError_t init_tiles() {
  return cudaFuncSetAttribute(linear_kernel<kCols, kCtas>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Config<kCols, kCtas>::smem);
}

struct Shape {
  int cols, ctas;
};

Shape choose(const LinearDims& s, int mode, int num_sms) {
  (void)num_sms;
  if (mode == kWeightGrad) return s.Nw() <= 64 ? Shape{64, 1} : s.Nw() <= 128 ? Shape{128, 1} : Shape{256, 1};
  const int rows = s.grouped ? (s.R + s.E - 1) / s.E * 3 / 2 : s.R;
  if (rows <= 32) return {32, 1};
  if (rows <= 64) return {64, 1};
  if (rows <= 128) return {128, 1};
  return {256, 1};
}

cudaError_t run_mode(const LinearDims& s, int mode, const int32_t* offsets, const void* x, const void* w, const void* dz,
                     Args& a, int num_sms, cudaStream_t st) {
  const Shape sh = choose(s, mode, num_sms);
  const int cols = sh.cols / sh.ctas;
  a.offsets = offsets;
  a.mode = mode;
  a.R = s.R;
  a.E = s.E;
  a.K = s.K;
  a.N = s.N;
  a.Nw = s.Nw();
  a.bf16 = s.type;
  a.width = mode == kForward ? s.N : s.K;
  a.tile_m = a.gated ? 64 : 128;
  a.tiles_m = (a.width + a.tile_m * sh.ctas - 1) / (a.tile_m * sh.ctas);
  a.tiles_c = (a.Nw + sh.cols - 1) / sh.cols;
  a.depth = mode == kForward ? s.K : a.Nw;
  a.word = mma_word(s.type == 1, mode != kForward, mode == kWeightGrad, 128 * sh.ctas, sh.cols);
  CUtensorMap ma, mb;
  bool ok;
  const int64_t K = s.K, R = s.R, E = s.E, Nw = a.Nw;
  if (mode == kForward) {
    const int64_t da[4] = {K, s.N, s.gated ? 2 : 1, E}, db[2] = {K, R};
    const int ba[4] = {kDepth, a.tile_m, s.gated ? 2 : 1, 1}, bb[2] = {kDepth, cols};
    ok = make_map(&ma, s.type == 1, w, 4, da, ba) && make_map(&mb, s.type == 1, x, 2, db, bb);
  } else if (mode == kInputGrad) {
    const int64_t da[3] = {K, Nw, E}, db[2] = {Nw, R};
    const int ba[3] = {64, kDepth, 1}, bb[2] = {kDepth, cols};
    ok = make_map(&ma, s.type == 1, w, 3, da, ba) && make_map(&mb, s.type == 1, dz, 2, db, bb);
  } else {
    const int64_t da[2] = {K, R}, db[2] = {Nw, R};
    const int bx[2] = {64, kDepth};
    ok = make_map(&ma, s.type == 1, x, 2, da, bx) && make_map(&mb, s.type == 1, dz, 2, db, bx);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int64_t most = mode == kWeightGrad ? E * a.tiles_m * a.tiles_c
                                           : int64_t(a.tiles_m) * ((R + sh.cols - 1) / sh.cols + (offsets ? E : 0));
  if (sh.cols == 32) return launch_tiles<32, 1>(a, ma, mb, most, num_sms, st);
  if (sh.cols == 64) return launch_tiles<64, 1>(a, ma, mb, most, num_sms, st);
  if (sh.cols == 128) return launch_tiles<128, 1>(a, ma, mb, most, num_sms, st);
  return launch_tiles<256, 1>(a, ma, mb, most, num_sms, st);
}

}  // namespace

cudaError_t init_linear_kernels() {
  cudaError_t err = init_tiles<32, 1>();
  if (err == cudaSuccess) err = init_tiles<64, 1>();
  if (err == cudaSuccess) err = init_tiles<128, 1>();
  if (err == cudaSuccess) err = init_tiles<256, 1>();
  return err;
}

cudaError_t launch_linear(const LinearDims& s, const int32_t* offsets, const void* x, const void* w, const float* bias,
                          const void* residual, void* out, void* preact, int32_t* err, int num_sms, cudaStream_t st) {
  Args a = {};
  a.bias = bias;
  a.residual = static_cast<const uint16_t*>(residual);
  a.out = static_cast<uint16_t*>(out);
  a.preact = static_cast<uint16_t*>(preact);
  a.err = err;
  a.act = s.act;
  a.gated = s.gated;
  return run_mode(s, kForward, offsets, x, w, nullptr, a, num_sms, st);
}

cudaError_t launch_linear_input_grad(const LinearDims& s, const int32_t* offsets, const void* w, const void* dz, void* dx,
                                     int32_t* err, int num_sms, cudaStream_t st) {
  Args a = {};
  a.out = static_cast<uint16_t*>(dx);
  a.err = err;
  a.act = 3;
  return run_mode(s, kInputGrad, offsets, nullptr, w, dz, a, num_sms, st);
}

cudaError_t launch_linear_weight_grad(const LinearDims& s, const int32_t* offsets, const void* x, const void* dz,
                                      void* dw, int32_t* err, int num_sms, cudaStream_t st) {
  Args a = {};
  a.out = static_cast<uint16_t*>(dw);
  a.err = err;
  a.act = 3;
  return run_mode(s, kWeightGrad, offsets, x, nullptr, dz, a, num_sms, st);
}

}  // namespace moe
