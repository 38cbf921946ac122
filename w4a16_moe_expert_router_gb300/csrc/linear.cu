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
// Persistent pairs of CTAs (two SMs on one tile of 256 outputs x up to kCols rows, each
// holding its 128 outputs of A and half of B) walk a list of tiles (few tiles with a long
// contraction are shared by the pairs of a cluster, which add their sums through
// distributed shared memory): a thread of each loads stages of A and B by TMA, one thread of the pair issues the matrix
// instructions into one of two accumulators in tensor memory, and eight warps of each
// empty the other one: 32 columns at a time through shared memory, so that the outputs
// leave by TMA.  Accumulation, bias, activation and residual are in fp32, rounded once.
//
// Measured: 8192 x 2048 x 8192 bf16 in 146 us (1.88 PFLOP/s, cuBLAS 142) in short bursts, 164 (158)
// under the power cap; gate and up products of 128 experts on 2048 rows in 111 us (6.7 TB/s); the
// gradient's products of 128 experts on 16384 rows, 2048 x 1408, in 127 us (input, 6.7 TB/s) and
// 148 us (weights: 738 MB of them leave at 5 TB/s, a fill's rate is 4).
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <mutex>

#include <cudaTypedefs.h>

#include "activation.cuh"
#include "internal.h"
#include "row_vec.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;
}  // namespace

bool make_map(CUtensorMap* map, bool bf16, const void* base, int rank, const int64_t* dims, const int64_t* strides,
              const int* box, bool swizzled) {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(dims[i]);
    b[i] = static_cast<cuuint32_t>(box[i]);
    es[i] = 1;
    if (i > 0) st[i - 1] = static_cast<cuuint64_t>(strides[i - 1]) * 2;
  }
  return g_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                  const_cast<void*>(base), d, st, b, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzled ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kForward = 0, kInputGrad = 1, kWeightGrad = 2;
constexpr int kTileM = 128;            // lanes of tensor memory: outputs of one CTA's half of a tile
// Columns per epilogue step: 64 for the weight gradient, whose tiles are a few stages long by
// experts, so that the epilogue's fences, barriers and stores bound it (16384 rows over 128
// experts, 2048 x 1408: 161 -> 149 us).
template <int kMode, bool kSplit = false>
constexpr int step_cols = kMode == kWeightGrad && !kSplit ? 64 : 32;
constexpr int kThreads = 384;          // TMA, MMA, tail and bias warps, then 8 epilogue warps
// The forward product's epilogue takes registers from the other warps: with the launch's 168 a
// thread its step spills (down of 128 experts, 32768 rows: 96.5 -> 93.2 us; 777 x 1000 x 2056: 10.4
// -> 10.0).
constexpr int kFewRegisters = 56, kManyRegisters = 224;
static_assert(kFewRegisters + 2 * kManyRegisters == 3 * 168);
constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 227 * 1024;
constexpr int kMaxSplit = 4;              // pairs that share a tile: a cluster of eight CTAs
constexpr int kBlockBytes = 32 * kTileM * 4;  // fp32 sums of a step, sent from pair to pair

struct Args {
  const int32_t* offsets;  // NULL: one weight for all rows
  const float* bias;
  const uint16_t* residual;
  uint16_t* out;
  uint16_t* preact;
  int32_t* err;
  int R, E, N, Nw, act, gated, bf16;
  int width;    // extent of m, and the row length of out
  int tile_m;   // outputs per CTA and tile (64 of a gate and their ups, or 128)
  int tiles_m;  // tiles along m
  uint64_t per_m;  // ceil(2^40 / tiles_m): i / tiles_m = i per_m >> 40 for i < 2^30 (tiles_m <= 1024)
  int tile_c;   // columns of a tile, kCols at most
  int tiles_c;  // weight grad: tiles along c
  int stage_bytes;  // what a CTA loads for a stage
  int depth;    // contraction length (weight grad: the expert's rows)
  uint32_t word;  // instruction word without its N
  int split;      // pairs of CTAs that share a tile's contraction
  int one_store;  // the output's map takes a step in one store (see run_mode)
  const float* partial;  // weight grad: the bias gradient's sums over row blocks, and where it goes (or NULL)
  float* dbias;
  int block_rows;
};

// A stage holds 64 contraction elements of the largest tile and 128 of the smaller ones: a
// stage costs its barriers and two waiting threads about 0.24 us whatever it holds (measured:
// tiles of 32 columns 814 -> 514 us on 8192 x 2048 x 8192, of 128 columns 219 -> 171 us),
// which is below the matrix instructions' time at 256 columns only, and there six short
// stages hide latency better than three long ones (141 against 146 us).
template <int kMode, int kCols, bool kSplit = false>
struct Config {
  static constexpr int depth = kCols == 256 ? 64 : 128;
  static constexpr int cols = kCols / 2;  // columns whose B rows each CTA loads
  static constexpr int a_bytes = kTileM * depth * 2;
  static constexpr int b_bytes = cols * depth * 2;
  static constexpr int box_bytes = depth * 128;  // 64 elements of each of a stage's contraction rows
  static constexpr int stage = a_bytes + b_bytes;
  static constexpr int step_bytes = step_cols<kMode, kSplit> * kTileM * 2;
  static constexpr int epi_bytes = 2 * step_bytes;  // two steps per group of four epilogue warps
  static constexpr int fixed = 2 * epi_bytes + (2 * (kMaxExperts + 1) + 2) * 4 + (4 * kMaxStages + 8) * 8 + 16;
  static constexpr int fit = (kSmemLimit - fixed) / stage;
  static constexpr int stages = fit < kMaxStages ? fit : kMaxStages;
  static constexpr int smem = stages * stage + fixed;
  static constexpr uint32_t tmem = 2 * kCols;  // two accumulators
};

// cols: the columns that are multiplied, as many as the tile has rounded up to what the
// instructions take (a pair's N in steps of 32; 64 strided columns to a box of each CTA), so
// that an expert's last tile costs what it holds.  first, len: the contraction elements (the
// pair's share of them where pairs split a tile).
struct Tile {
  int e, m0, c0, cols, row0, row_end, first, len;
};

// The CTA's half of the tile of index t.  start[e]: tiles before expert e; off[e]: its first row.
// rank: of the CTA in its cluster, pair by pair.
template <int kMode, bool kSplit>
__device__ __forceinline__ Tile tile_at(const Args& a, const int* start, const int* off, int t, int& e, int rank) {
  while (t >= start[e + 1]) ++e;  // t only grows
  const int i = t - start[e];
  const int c = static_cast<int>(i * a.per_m >> 40), m = i - c * a.tiles_m;
  Tile r;
  r.e = e;
  r.m0 = (m * 2 + (rank & 1)) * a.tile_m;
  if (kMode == kWeightGrad) {
    r.c0 = c * a.tile_c;
    r.row0 = e * a.Nw + r.c0;
    r.row_end = (e + 1) * a.Nw;
    r.cols = min(a.tile_c, (a.Nw - r.c0 + 127) & ~127);
    r.first = off[e];
    r.len = off[e + 1] - off[e];
  } else {
    r.c0 = off[e] + c * a.tile_c;
    r.row0 = r.c0;
    r.row_end = off[e + 1];
    r.cols = min(a.tile_c, (r.row_end - r.c0 + 31) & ~31);
    r.first = 0;
    r.len = a.depth;
  }
  if (kSplit) {  // whole stages to each pair, the rest to the last one
    constexpr int depth = Config<kMode, 128>::depth;
    const int stages = (r.len + depth - 1) / depth, part = rank >> 1;
    const int from = part * stages / a.split * depth, to = (part + 1) * stages / a.split * depth;
    r.first = from;
    r.len = min(r.len, to) - from;
  }
  return r;
}

// Two 16-bit values, the first in the lower half.
__device__ __forceinline__ float2 unpack2(uint32_t v, int bf16) {
  return bf16 ? make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)) : __half22float2(bits_h2(v));
}

__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// kCount / 2 pairs of values, rounded.
template <int kCount>
__device__ __forceinline__ void pack_all(const float (&f)[kCount], uint32_t (&r)[kCount / 2], int bf16) {
  if (bf16) {
#pragma unroll
    for (int i = 0; i < kCount / 2; ++i) r[i] = Vec<1>::pack(f[2 * i], f[2 * i + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < kCount / 2; ++i) r[i] = h2_bits(__floats2half2_rn(f[2 * i], f[2 * i + 1]));
  }
}

template <int kCount>
__device__ __forceinline__ void activate_all(float (&z)[kCount], int act) {
  switch (act) {
    case kGeluTanh:
#pragma unroll
      for (int i = 0; i < kCount; ++i) z[i] = activate(z[i], kGeluTanh);
      break;
    case kGeluErf:
#pragma unroll
      for (int i = 0; i < kCount; ++i) z[i] = activate(z[i], kGeluErf);
      break;
    case kSilu:
#pragma unroll
      for (int i = 0; i < kCount; ++i) z[i] = activate(z[i], kSilu);
      break;
    default:
      break;
  }
}

// ---- one epilogue step: 32 columns c of the accumulator.
//
// A warp holds 32 lanes x 32 columns as blocks of 8 x 8: block i of half h (16 lanes) gives
// a thread the lanes 16 h + g and 16 h + g + 8 at columns 8 i + q and 8 i + q + 1 (g = lane
// / 4, q = 2 (lane % 4)).  Everything between the accumulator and the rounding happens in
// these registers; the rounded blocks go transposed to a step buffer [32 columns][outputs],
// swizzled so that neither the blocks nor the rows meet in a bank, and leave by TMA, or,
// where the step ends inside an expert's rows, as 16-byte pieces of the rows that are the
// expert's.  A gated tile's lanes alternate, 8 of the gate and the 8 of the up product with
// the same outputs, so a thread holds both.

// Place of chunk `chunk` of column c in a step buffer: 64 outputs (8 chunks) of the step's
// columns, then the other 64, each in the 128-byte swizzle of a TMA box.
template <int kStep>
__device__ __forceinline__ uint32_t chunk_at(int c, int chunk) {
  return static_cast<uint32_t>((chunk >> 3) * (kStep * 128) + c * 128 + ((chunk ^ c) & 7) * 16);
}

// The rows of a 32-column step between a step buffer and global memory: thread tid of 128 takes
// chunk tid % kChunks of every (128 / kChunks)-th column, four at most.  f: the chunk's first
// column in elements, valid while f < width; rows of stride `ld` from row0 on, those below
// row_end.
template <int kChunks, typename Do>
__device__ __forceinline__ void for_rows(int tid, int f, int width, int row0, int row_end, Do&& act) {
  constexpr int rows = 128 / kChunks, passes = 32 / rows;
  const int c0 = tid / kChunks;
  if (f >= width) return;
#pragma unroll
  for (int i = 0; i < passes; ++i)
    if (row0 + c0 + i * rows < row_end) act(i, c0 + i * rows);
}
template <int kChunks>
__device__ __forceinline__ void store_rows(const uint8_t* buf, uint16_t* p, int tid, int f, int width, int ld, int row0,
                                           int row_end) {
  uint4 v[4];
  for_rows<kChunks>(tid, f, width, row0, row_end, [&](int i, int c) {
    v[i] = *reinterpret_cast<const uint4*>(buf + chunk_at<32>(c, tid % kChunks));
  });
  for_rows<kChunks>(tid, f, width, row0, row_end, [&](int i, int c) {
    *reinterpret_cast<uint4*>(p + static_cast<size_t>(row0 + c) * ld + f) = v[i];
  });
}

// Where the rows of an epilogue step go.
struct StepRows {
  int m0, row0, row_end;
  bool whole;  // the rows all belong to the tile (the maps clip those past the end of the array)
  int y, z;    // the rows in the output's map: row y of plane z
};

// The group's step buffer `buf`, all blocks stored, to the output (kSaved: to the saved z).
// One thread stores for the group; the store before has read the other buffer by now, which
// the barrier tells the rest, so that the two buffers may be taken in turn.
template <int kForm, int kStep, bool kSaved>
__device__ __forceinline__ void send_step(const Args& a, const CUtensorMap* map, uint8_t* buf, int group, int tid,
                                          const StepRows& r) {
  const bool issuer = (tid >> 5) == 0 && elect_one();
  if (r.whole) fence_proxy_async();
  if (issuer) bulk_wait_read();
  group_sync(1 + group);
  if (r.whole) {
    if (issuer && r.m0 < a.width) {
      const uint32_t src = smem_addr(buf);
      constexpr int half = kStep * 128;
      if (!kSaved) {
        if (a.one_store) {
          tma_store_4d(map, src, 0, r.y, r.m0 >> 6, r.z);
        } else {
          tma_store_4d(map, src, r.m0, r.y, 0, r.z);
          if (kForm != 2 && r.m0 + 64 < a.width) tma_store_4d(map, src + half, r.m0 + 64, r.y, 0, r.z);
        }
      } else if (kForm == 2) {  // planes: gate, up
        tma_store_3d(map, src, r.m0, 0, r.y);
        tma_store_3d(map, src + half, r.m0, 1, r.y);
      } else {
        tma_store_3d(map, src, r.m0, 0, r.y);
        if (r.m0 + 64 < a.width) tma_store_3d(map, src + half, r.m0 + 64, 0, r.y);
      }
      bulk_commit();
    }
  } else if constexpr (kStep == 32) {
    if (kSaved) {
      const int chunk = tid % 16;
      store_rows<16>(buf, kForm == 2 && chunk >= 8 ? a.preact + a.N : a.preact, tid,
                     r.m0 + (kForm == 2 ? chunk & 7 : chunk) * 8, a.width, a.Nw, r.row0, r.row_end);
    } else {
      constexpr int chunks = kForm == 2 ? 8 : 16;
      store_rows<chunks>(buf, a.out, tid, r.m0 + tid % chunks * 8, a.width, a.width, r.row0, r.row_end);
    }
  }
}

// The other pairs' sums of a step, where pairs split a tile: `count` blocks, in each of which
// thread tid finds its 16-byte piece i (in the order of its accumulators) at 128 i + tid.
struct Partials {
  const float4* at;
  int count;
};
__device__ __forceinline__ void add_partials(uint32_t (*v)[16], const Partials& p, int tid) {
#pragma unroll 1
  for (int s = 0; s < p.count; ++s) {
    const float4* const at = p.at + s * (kBlockBytes / 16) + tid;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = at[(h * 4 + i) * 128];
        v[h][4 * i] = __float_as_uint(__uint_as_float(v[h][4 * i]) + f.x);
        v[h][4 * i + 1] = __float_as_uint(__uint_as_float(v[h][4 * i + 1]) + f.y);
        v[h][4 * i + 2] = __float_as_uint(__uint_as_float(v[h][4 * i + 2]) + f.z);
        v[h][4 * i + 3] = __float_as_uint(__uint_as_float(v[h][4 * i + 3]) + f.w);
      }
  }
}
// The step at `tmem` to such a block of another CTA, counted on its barrier (cluster addresses).
__device__ __forceinline__ void send_partials(uint32_t tmem, uint32_t dst, uint32_t bar, int tid) {
  uint32_t v[2][16];
  tmem_load_16x32(tmem, v[0]);
  tmem_load_16x32(tmem + (16u << 16), v[1]);
  tmem_load_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t* const p = &v[i >> 2][4 * (i & 3)];
    store_async_16(dst + i * 2048 + tid * 16, p[0], p[1], p[2], p[3], bar);
  }
}

// A step of the gradients' products: kStep columns from `tmem` on (zeros where the tile has no
// contraction), rounded.  buf: the group's two step buffers, the next one to take is `flip`.
template <int kStep>
__device__ __forceinline__ void gradient_step(const Args& a, const CUtensorMap* map_out, uint32_t tmem, bool any,
                                              const Partials& others, uint8_t* buf, int& flip, int group, int tid,
                                              const StepRows& rows) {
  const int lane = tid & 31, quarter = tid >> 5;
  const int sub = lane >> 3, j = lane & 7;  // the block and row whose address this lane gives
  uint32_t v[kStep / 16][16];  // [32 columns][half of the lanes]
  if (any) {
#pragma unroll
    for (int h = 0; h < kStep / 32; ++h) {
      tmem_load_16x32(tmem + 32 * h, v[2 * h]);
      tmem_load_16x32(tmem + 32 * h + (16u << 16), v[2 * h + 1]);
    }
    tmem_load_wait();
    add_partials(v, others, tid);
  } else {
#pragma unroll
    for (int h = 0; h < kStep / 16; ++h)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[h][i] = 0u;
  }
  uint8_t* const ybuf = buf + flip * (kStep * kTileM * 2);
  flip ^= 1;
  float f[kStep];
  uint32_t r[kStep / 2];
#pragma unroll
  for (int i = 0; i < kStep; ++i)  // block column i / 8: the four blocks of 8 lanes
    f[i] = __uint_as_float(v[2 * (i >> 5) + (i >> 2 & 1)][4 * (i >> 3 & 3) + (i & 3)]);
  pack_all(f, r, a.bf16);
#pragma unroll
  for (int i = 0; i < kStep / 8; ++i)
    store_blocks_transposed(smem_addr(ybuf) + chunk_at<kStep>(8 * i + j, quarter * 4 + sub), &r[4 * i]);
  send_step<0, kStep, false>(a, map_out, ybuf, group, tid, rows);
}

// The residual's pieces of a step, requested a step ahead of their use.
template <int kForm>
__device__ __forceinline__ void request_residual(const Args& a, uint4 (&res)[4], int tid, int m0, int row0,
                                                 int row_end) {
  constexpr int chunks = kForm == 2 ? 8 : 16;
  const int f = m0 + tid % chunks * 8;
  for_rows<chunks>(tid, f, a.width, row0, row_end, [&](int i, int c) {
    res[i] = *reinterpret_cast<const uint4*>(a.residual + static_cast<size_t>(row0 + c) * a.width + f);
  });
}

// The biases of the lanes g, g + 8, g + 16, g + 24 of a quarter (g = lane / 4).
__device__ __forceinline__ void load_bias(const Args& a, float (&b)[4], const Tile& r, int quarter, int lane) {
  const float* const bp = a.bias + static_cast<size_t>(r.e) * a.Nw;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = lane >> 2;
    const int f = a.gated ? r.m0 + quarter * 16 + (i >> 1) * 8 + g : r.m0 + quarter * 32 + i * 8 + g;
    if (f < a.width) b[i] = bp[a.gated && (i & 1) ? a.N + f : f];
  }
}

// A forward step of 32 columns.  kForm: 1 plain, 2 gated.  b: the biases of the thread's lanes
// g, g + 8, g + 16, g + 24 of its quarter.  res: the step's residual, then the one's at `next`.
template <int kForm>
__device__ __forceinline__ void forward_step(const Args& a, const CUtensorMap* map_out, const CUtensorMap* map_z,
                                             uint32_t tmem, const Partials& others, const float (&b)[4],
                                             uint4 (&res)[4], int next, uint8_t* buf, int& flip, int group, int tid,
                                             const StepRows& rows) {
  constexpr int chunks = kForm == 2 ? 8 : 16;  // 16-byte chunks of outputs per column
  const int lane = tid & 31, quarter = tid >> 5;
  const int sub = lane >> 3, j = lane & 7;
  uint32_t v[2][16];
  tmem_load_16x32(tmem, v[0]);
  tmem_load_16x32(tmem + (16u << 16), v[1]);
  tmem_load_wait();
  add_partials(v, others, tid);
  float z[2][16];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i) z[h][i] = __uint_as_float(v[h][i]) + b[2 * h + (i >> 1 & 1)];
  if (a.preact) {
    uint8_t* const zbuf = buf + flip * 32 * kTileM * 2;
    flip ^= 1;
    float f[32];
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 32; ++i) f[i] = z[i >> 2 & 1][4 * (i >> 3) + (i & 3)];
    pack_all(f, r, a.bf16);
    // gated: chunks 0 .. 7 of the gate, 8 .. 15 of the up product
    const int chunk = kForm == 2 ? (sub & 1) * 8 + quarter * 2 + (sub >> 1) : quarter * 4 + sub;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      store_blocks_transposed(smem_addr(zbuf) + chunk_at<32>(8 * i + j, chunk), &r[4 * i]);
    send_step<kForm, 32, true>(a, map_z, zbuf, group, tid, rows);
  }
  uint8_t* const ybuf = buf + flip * 32 * kTileM * 2;
  flip ^= 1;
  if (a.residual) {
    for_rows<chunks>(tid, rows.m0 + tid % chunks * 8, a.width, rows.row0, rows.row_end, [&](int i, int c) {
      *reinterpret_cast<uint4*>(ybuf + chunk_at<32>(c, tid % chunks)) = res[i];
    });
    group_sync(1 + group);
    request_residual<kForm>(a, res, tid, rows.m0, next, rows.row_end);
  }
  // 16 values at a time, so that activation and type are asked for once or twice (for every 4 it
  // costs a step 200 cycles of 1,600); r[4 i ..] are the blocks that one instruction stores, of block column
  // 2 p + i (gated: 2 i and 2 i + 1)
#pragma unroll
  for (int p = 0; p < (kForm == 2 ? 1 : 2); ++p) {
    float y[16];
    uint32_t r[8];
    if (kForm == 2) {
      float u[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int at = 4 * (i >> 2) + (i & 1), h = i >> 1 & 1;
        y[i] = z[h][at];
        u[i] = z[h][at + 2];
      }
      activate_all(y, a.act);
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] *= u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) y[i] = z[i >> 2 & 1][8 * p + 4 * (i >> 3) + (i & 3)];
      activate_all(y, a.act);
    }
    const auto place = [&](int i) {
      return smem_addr(ybuf) + (kForm == 2 ? chunk_at<32>(8 * (2 * i + (sub >> 1)) + j, quarter * 2 + (sub & 1))
                                           : chunk_at<32>(8 * (2 * p + i) + j, quarter * 4 + sub));
    };
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < 2; ++i) load_blocks_transposed(place(i), &r[4 * i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 g = unpack2(r[i], a.bf16);
        y[2 * i] += g.x;
        y[2 * i + 1] += g.y;
      }
    }
    pack_all(y, r, a.bf16);
#pragma unroll
    for (int i = 0; i < 2; ++i) store_blocks_transposed(place(i), &r[4 * i]);
  }
  send_step<kForm, 32, false>(a, map_out, ybuf, group, tid, rows);
}

// A step of either kind.
template <int kMode, int kStep>
__device__ __forceinline__ void step_of(const Args& a, const CUtensorMap* map_out, const CUtensorMap* map_z,
                                        uint32_t tmem, bool any, const Partials& others, const float (&b)[4],
                                        uint4 (&res)[4], int next, uint8_t* buf, int& flip, int group, int tid,
                                        const StepRows& rows) {
  if constexpr (kMode != kForward)
    gradient_step<kStep>(a, map_out, tmem, any, others, buf, flip, group, tid, rows);
  else if (a.gated)
    forward_step<2>(a, map_out, map_z, tmem, others, b, res, next, buf, flip, group, tid, rows);
  else
    forward_step<1>(a, map_out, map_z, tmem, others, b, res, next, buf, flip, group, tid, rows);
}

// kSplit: a cluster of a.split pairs on one tile, each with a share of the contraction.
template <int kMode, int kCols, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ Args a,
                                                             const __grid_constant__ CUtensorMap map_a,
                                                             const __grid_constant__ CUtensorMap map_b,
                                                             const __grid_constant__ CUtensorMap map_out,
                                                             const __grid_constant__ CUtensorMap map_z) {
  using C = Config<kMode, kCols, kSplit>;
  constexpr int kDepth = C::depth;
  static_assert(!kSplit || 4 * kBlockBytes <= C::stages * C::stage, "a CTA's blocks take the stages' place");
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* const epi = smem + C::stages * C::stage;
  int* const start = reinterpret_cast<int*>(epi + 2 * C::epi_bytes);  // [E + 1]
  int* const off = start + kMaxExperts + 1;                        // [E + 1]
  uint64_t* const bars = reinterpret_cast<uint64_t*>(off + kMaxExperts + 1 + 2);
  const uint32_t bar0 = smem_addr(bars);
  constexpr int S = C::stages;
  const uint32_t full = bar0, empty = full + 8 * S, tail_full = empty + 8 * S, tail_done = tail_full + 8 * S;
  const uint32_t acc_full = tail_done + 8 * S, acc_empty = acc_full + 16, drained = acc_empty + 16,
                 vacant = drained + 8, summed = vacant + 8;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 * S + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), lead = kSplit ? rank & ~1 : 0;  // lead: the pair's first CTA
  grid_dependents_launch();
  if (warp == 1) tmem_alloc(smem_addr(tmem_slot), C::tmem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::stages; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
      mbar_init(tail_full + 8 * s, 1);
      mbar_init(tail_done + 8 * s, 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 16);  // the epilogue warps of both CTAs
    }
    mbar_init(drained, 1);
    if (kSplit) {
      mbar_init(vacant, a.split);
      for (int g = 0; g < 2; ++g) {
        mbar_init(summed + 8 * g, 1);
        mbar_arrive_expect_tx(summed + 8 * g, (a.split - 1) * kBlockBytes);
      }
    }
    fence_barrier_init();
    prefetch_map(&map_a);
    prefetch_map(&map_b);
    prefetch_map(&map_out);
  }
  if (!a.offsets && threadIdx.x == 32) {
    start[0] = off[0] = 0;
    start[1] = a.tiles_m * (kMode == kWeightGrad ? a.tiles_c : (a.R + a.tile_c - 1) / a.tile_c);
    off[1] = a.R;
  }
  // the set-up overlaps the launch before; what it may still write is read after the wait, which
  // each warp that reads global memory or has it read does for itself, as near to that as can be
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised
  tcgen05_fence_after();
  if (a.offsets && warp == 2) {
    grid_dependency_wait();
    // first rows of the experts (clamped to the rows there are) and their tiles: eight
    // experts per lane, then a scan over the lanes
    int o[9], n[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      const int e = lane * 8 + i;
      o[i] = e <= a.E ? min(max(a.offsets[e], 0), a.R) : a.R;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      const int rows = max(o[i + 1] - o[i], 0);
      n[i] = e < a.E ? a.tiles_m * (kMode == kWeightGrad ? a.tiles_c : (rows + a.tile_c - 1) / a.tile_c) : 0;
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
  if (a.offsets) __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const int tiles = start[a.E];
  const int ctas = kSplit ? 2 * a.split : 2;
  const int first_tile = blockIdx.x / ctas, step = gridDim.x / ctas;

  bool failed = false, late = false;  // a wait ran out; it was that for a split tile's sums

  if (warp < 4) {
    if constexpr (kMode == kForward) registers_release<kFewRegisters>();
    if (warp == 0) {
      if (elect_one()) {
        // ---- loads
        const uint32_t lead_full = cluster_addr(full, lead), stage0 = smem_addr(smem);
        const uint32_t own_tail = cluster_addr(tail_full, rank);
        int e = 0, s = 0, issued = 0;
        uint32_t phase = 0, uses = 0, tails = 0, tail_uses = 0;  // one bit per stage, see below
        bool alive = true, waited = false;
        for (int t = first_tile; alive && t < tiles; t += step) {
          const Tile r = tile_at<kMode, kSplit>(a, start, off, t, e, rank);
          const int bc = r.c0 + (rank & 1) * (r.cols >> 1);
#pragma unroll 1
          for (int j = 0, f = r.first; j < r.len; j += kDepth, f += kDepth) {
            if (!stage_wait<true>(empty + 8 * s, phase ^ 1, a.err)) {
              alive = false;
              break;
            }
            if (!waited) {
              grid_dependency_wait();
              waited = true;
            }
            const uint32_t sa = stage0 + s * C::stage, sb = sa + C::a_bytes;
            uint32_t bar = lead_full + 8 * s;
            if (kMode == kWeightGrad && r.len - j < kDepth) {
              bar = own_tail + 8 * s;  // a tail is mended by its own CTA first
              mbar_arrive_expect_tx(tail_full + 8 * s, C::stage);
              tail_uses ^= 1u << s;
              tails |= 1u << s;
            } else {
              if (rank == lead) mbar_arrive_expect_tx(full + 8 * s, 2 * a.stage_bytes);
              uses ^= 1u << s;
              tails &= ~(1u << s);
            }
            if (kMode == kForward) {
              tma_load_5d(sa, &map_a, f, 0, 0, r.m0 >> 3, r.e, bar);
              tma_load_2d(sb, &map_b, f, bc, bar);
              if constexpr (kDepth == 128) {
                tma_load_5d(sa + C::a_bytes / 2, &map_a, f + 64, 0, 0, r.m0 >> 3, r.e, bar);
                tma_load_2d(sb + C::b_bytes / 2, &map_b, f + 64, bc, bar);
              }
            } else if (kMode == kInputGrad) {
              tma_load_3d(sa, &map_a, r.m0, f, r.e, bar);
              tma_load_3d(sa + C::a_bytes / 2, &map_a, r.m0 + 64, f, r.e, bar);
              tma_load_2d(sb, &map_b, f, bc, bar);
              if constexpr (kDepth == 128) tma_load_2d(sb + C::b_bytes / 2, &map_b, f + 64, bc, bar);
            } else {
              tma_load_2d(sa, &map_a, r.m0, f, bar);
              tma_load_2d(sa + C::a_bytes / 2, &map_a, r.m0 + 64, f, bar);
#pragma unroll
              for (int x = 0; x < C::cols / 64; ++x)
                tma_load_2d(sb + x * C::box_bytes, &map_b, bc + 64 * x, f, bar);
            }
            if (issued < C::stages) ++issued;
            if (++s == C::stages) {
              s = 0;
              phase ^= 1;
            }
          }
        }
        // the peer's instructions have told this CTA of every stage before it leaves
        for (int i = 0; alive && i < C::stages; ++i) {
          alive = stage_wait<true>(empty + 8 * s, phase ^ 1, a.err);
          if (++s == C::stages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!alive) {
          // a wait ran out: the copies in flight land before the CTAs' shared memory goes.  A
          // stage's last copies are counted on its tail barrier (bit in `tails`), or for both
          // CTAs on the first one's barrier; a bit of `uses` is the number of uses, so the
          // parity of the last phase is its complement.
          for (int i = 0; i < issued; ++i) {
            if (tails >> i & 1)
              mbar_wait(tail_full + 8 * i, (tail_uses >> i & 1) ^ 1, a.err);
            else if (rank == lead)
              mbar_wait(full + 8 * i, (uses >> i & 1) ^ 1, a.err);
          }
        }
      }
    } else if (warp == 1) {
      if (rank == lead && elect_one()) {
        // ---- matrix instructions
        const uint32_t both = 3u << lead;
        constexpr bool a_strided = kMode != kForward, b_strided = kMode == kWeightGrad;
        const uint32_t stage0 = smem_addr(smem);
        int e = 0, s = 0, acc = 0;
        uint32_t phases = 0, acc_phase = 0, tail_phases = 0;  // per stage: parity of its next use
        bool alive = true;
        grid_dependency_wait();  // the limit of a wait for a stage does not run while the launch before does
        for (int t = first_tile; alive && t < tiles; t += step) {
          const Tile r = tile_at<kMode, kSplit>(a, start, off, t, e, rank);
          if (r.len <= 0) continue;  // no rows: the epilogue writes zeros
          if (!stage_wait<true>(acc_empty + 8 * acc, acc_phase ^ 1, a.err)) {
            alive = false;
            break;
          }
          tcgen05_fence_after();
          const uint32_t d = tmem + acc * kCols, word = a.word | static_cast<uint32_t>(r.cols >> 3) << 17;
#pragma unroll 1
          for (int j = 0; j < r.len; j += kDepth) {
            if (kMode == kWeightGrad && r.len - j < kDepth) {
              alive = stage_wait<true>(tail_done + 8 * s, tail_phases >> s & 1, a.err);
              tail_phases ^= 1u << s;
            } else {
              alive = stage_wait<true>(full + 8 * s, phases >> s & 1, a.err);
              phases ^= 1u << s;
            }
            if (!alive) break;
            tcgen05_fence_after();
            const uint32_t sa = stage0 + s * C::stage;
            const uint64_t da = smem_operand(sa, a_strided ? C::box_bytes : 16);
            const uint64_t db = smem_operand(sa + C::a_bytes, b_strided ? C::box_bytes : 16);
            const auto issue = [&](int k) {  // contraction elements 16 k .. of the stage
              const uint64_t ka = a_strided ? k * (2048 >> 4) : (k >> 2) * (C::a_bytes >> 5) + (k & 3) * (32 >> 4);
              const uint64_t kb = b_strided ? k * (2048 >> 4) : (k >> 2) * (C::b_bytes >> 5) + (k & 3) * (32 >> 4);
              mma_f16(d, da + ka, db + kb, word, static_cast<uint32_t>(j | k));
            };
            if (r.len - j >= kDepth) {
#pragma unroll
              for (int k = 0; k < kDepth / 16; ++k) issue(k);
            } else {
#pragma unroll 1
              for (int k = 0; 16 * k < r.len - j; ++k) issue(k);
            }
            mma_commit(empty + 8 * s, both);
            if (++s == C::stages) s = 0;
          }
          if (!alive) break;
          mma_commit(acc_full + 8 * acc, both);
          if (kSplit) mma_commit(vacant, (1 << 2 * a.split) - 1);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
        for (int i = 0; !kSplit && alive && i < 2; ++i) {  // and the peer's epilogue has told this one of its tiles
          alive = stage_wait<true>(acc_empty + 8 * acc, acc_phase ^ 1, a.err);
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
        if (!alive) {  // a wait ran out: the instructions in flight end before tensor memory is given back
          mma_commit(drained, 1 << lead);
          mbar_wait(drained, 0, a.err);
        }
      }
    } else if (warp == 2) {
      // ---- weight grad: the last stage of an expert holds rows of the next one (or rows that
      // nobody wrote): zeros, up to a multiple of 16 rows, in each CTA's operands before they are
      // used.  Such a stage has barriers of its own, so a stage's phases stay in step with the
      // thread that waits for them.
      if (kMode == kWeightGrad) {
        const uint32_t lead_done = cluster_addr(tail_done, lead);
        int e = 0, it = 0;
        uint32_t phases = 0;
        grid_dependency_wait();  // as the thread above
        for (int t = first_tile; t < tiles; t += step) {
          const Tile r = tile_at<kMode, kSplit>(a, start, off, t, e, rank);
          if (r.len <= 0) continue;
          it += (r.len + kDepth - 1) / kDepth;
          const int rest = r.len % kDepth;
          if (rest == 0) continue;
          const int s = (it - 1) % C::stages;
          if (!stage_wait_warp(tail_full + 8 * s, phases >> s & 1, a.err)) break;
          phases ^= 1u << s;
          const int z0 = rest * 128, z1 = (rest + 15) / 16 * 16 * 128;
          uint8_t* const base = smem + s * C::stage;
          for (int box = 0; box < C::stage / C::box_bytes; ++box)
            for (int z = z0 + lane * 16; z < z1; z += 512)
              *reinterpret_cast<uint4*>(base + box * C::box_bytes + z) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_shared(lead_done + 8 * s);
        }
      }
    } else if (kMode == kWeightGrad && warp == 3) {
      // ---- weight grad: the bias gradient, for the columns of one tile along m (not always the
      // same one, so that the pairs share the work: a load takes microseconds while the tiles
      // stream).  Eight strided sums over the expert's row blocks, added in order.
      if (a.dbias && rank == 0) {
        grid_dependency_wait();
        int e = 0, counted = 0, before = 0;  // row blocks of the experts before `counted`
        for (int t = first_tile; t < tiles; t += step) {
          const Tile r = tile_at<kMode, kSplit>(a, start, off, t, e, rank);
          if (r.m0 / (2 * kTileM) != (r.c0 / kCols + r.e) % a.tiles_m) continue;
          const auto blocks = [&](int i) { return (max(off[i + 1] - off[i], 0) + a.block_rows - 1) / a.block_rows; };
          for (; counted < r.e; ++counted) before += blocks(counted);
          const int count = blocks(r.e);
          constexpr int kParts = kCols > 128 ? kCols / 128 : 1;  // columns c0 + 128 i + 4 lane ..
          const float* const p = a.partial + static_cast<size_t>(before) * a.Nw + r.c0 + 4 * lane;
          float4 s[kParts][8];
#pragma unroll
          for (int i = 0; i < kParts; ++i)
#pragma unroll
            for (int l = 0; l < 8; ++l) s[i][l] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int b = 0; b < count; b += 8) {
            float4 v[kParts][8];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
              for (int l = 0; l < 8; ++l) {
                v[i][l] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (b + l < count && r.c0 + 128 * i + 4 * lane < a.Nw)
                  v[i][l] = *reinterpret_cast<const float4*>(p + static_cast<size_t>(b + l) * a.Nw + 128 * i);
              }
#pragma unroll
            for (int i = 0; i < kParts; ++i)
#pragma unroll
              for (int l = 0; l < 8; ++l)
                s[i][l] = make_float4(s[i][l].x + v[i][l].x, s[i][l].y + v[i][l].y, s[i][l].z + v[i][l].z,
                                      s[i][l].w + v[i][l].w);
          }
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int l = 0; l < 8; ++l)
              d = make_float4(d.x + s[i][l].x, d.y + s[i][l].y, d.z + s[i][l].z, d.w + s[i][l].w);
            const int c = r.c0 + 128 * i + 4 * lane;
            if (c < a.Nw) *reinterpret_cast<float4*>(a.dbias + static_cast<size_t>(r.e) * a.Nw + c) = d;
          }
        }
      }
    }
  } else if (!kSplit) {
    if constexpr (kMode == kForward) registers_take<kManyRegisters>();
    // ---- epilogue: two groups of four warps take the steps in turn
    constexpr int kStep = step_cols<kMode>;
    const int group = (warp - 4) >> 2, tid = threadIdx.x & 127, quarter = warp & 3;
    uint8_t* const buf = epi + group * C::epi_bytes;
    const uint32_t lead_empty = cluster_addr(acc_empty, 0);
    int e = 0, acc = 0, flip = 0;
    uint32_t acc_phase = 0;
    bool alive = true;
    grid_dependency_wait();
    for (int t = first_tile; t < tiles; t += step) {
      const Tile r = tile_at<kMode, kSplit>(a, start, off, t, e, rank);
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (kMode == kForward && a.bias) load_bias(a, b, r, quarter, lane);
      uint4 res[4];
      const int tile_end = min(r.row_end, r.row0 + a.tile_c);  // the next tile's rows may be written meanwhile
      if (kMode == kForward && a.residual) {
        const int row0 = r.row0 + group * kStep;
        if (a.gated)
          request_residual<2>(a, res, tid, r.m0, row0, tile_end);
        else
          request_residual<1>(a, res, tid, r.m0, row0, tile_end);
      }
      if (r.len > 0) {
        // a warp whose wait ran out goes on without waiting: the group's barriers stay matched, and
        // the outputs are invalid as recorded
        alive = alive && stage_wait_warp<true>(acc_full + 8 * acc, acc_phase, a.err);
        tcgen05_fence_after();
      }
#pragma unroll 1
      for (int c = group * kStep; r.row0 + c < tile_end; c += 2 * kStep) {
        const uint32_t at = tmem + acc * kCols + c + (static_cast<uint32_t>(quarter * 32) << 16);
        const int row0 = r.row0 + c;
        const StepRows rows{r.m0, row0, tile_end, kMode == kWeightGrad || row0 + kStep <= tile_end,
                            kMode == kWeightGrad ? r.c0 + c : row0, kMode == kWeightGrad ? r.e : 0};
        step_of<kMode, kStep>(a, &map_out, &map_z, at, r.len > 0, Partials{nullptr, 0}, b, res, row0 + 2 * kStep, buf,
                              flip, group, tid, rows);
      }
      if (r.len > 0) {
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(lead_empty + 8 * acc);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
    failed = !alive;
    __syncwarp();
    if (quarter == 0 && elect_one()) bulk_wait();
  } else {
    if constexpr (kMode == kForward) registers_take<kManyRegisters>();
    // ---- epilogue of the one tile of a cluster whose pairs split it: step i of the columns is
    // pair i % split's, which gets the other pairs' sums of it in the shared memory of its stages
    // (once its instructions have read them) and adds them in the order of the pairs after it
    const int group = (warp - 4) >> 2, tid = threadIdx.x & 127, quarter = warp & 3, part = rank >> 1;
    const int others = a.split - 1, mine = part + group * a.split;  // the group's step
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    int e = 0, flip = 0;
    const Tile r = tile_at<kMode, kSplit>(a, start, off, first_tile, e, rank);
    const int row0 = r.row0 + mine * 32, tile_end = min(r.row_end, r.row0 + a.tile_c);
    float b[4] = {0.f, 0.f, 0.f, 0.f};
    uint4 res[4];
    grid_dependency_wait();
    if (kMode == kForward && row0 < tile_end) {
      if (a.bias) load_bias(a, b, r, quarter, lane);
      if (a.residual) {
        if (a.gated)
          request_residual<2>(a, res, tid, r.m0, row0, tile_end);
        else
          request_residual<1>(a, res, tid, r.m0, row0, tile_end);
      }
    }
    failed = !stage_wait_warp<true>(acc_full, 0, a.err) || !stage_wait_warp<true>(vacant, 0, a.err);
    tcgen05_fence_after();
    for (int i = group; !failed && r.row0 + i * 32 < tile_end; i += 2) {
      const int owner = i % a.split, to = owner * 2 + (rank & 1);
      if (owner == part) continue;
      const int block = i / a.split * others + (part - owner + a.split) % a.split - 1;
      send_partials(at + i * 32, cluster_addr(smem_addr(smem) + block * kBlockBytes, to),
                    cluster_addr(summed + 8 * (i / a.split), to), tid);
    }
    if (row0 < tile_end) {
      late = !stage_wait_warp<true>(summed + 8 * group, 0, a.err);
      const StepRows rows{r.m0, row0, tile_end, kMode == kWeightGrad || row0 + 32 <= tile_end, row0, 0};
      step_of<kMode, 32>(a, &map_out, &map_z, at + mine * 32, true,
                         Partials{reinterpret_cast<const float4*>(smem + group * others * kBlockBytes), others}, b, res,
                         tile_end, epi + group * C::epi_bytes, flip, group, tid, rows);
    }
    tcgen05_fence_before();
    __syncwarp();
    if (quarter == 0 && elect_one()) bulk_wait();
  }
  __syncwarp();
  __syncthreads();
  // no CTA leaves while another may still signal it: it has waited for all signals by now, and the
  // barrier need not order memory (500 cycles instead of 1,400) unless a wait ran out
  if (failed || late)
    cluster_sync();
  else
    cluster_sync_relaxed();
  // (sums that a wait did not see are in flight at most: they land before the shared memory goes)
  if (kSplit && late) mbar_wait(summed + 8 * ((warp - 4) >> 2), 0, a.err);
  if (warp == 1) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, C::tmem);
  }
}

// ------------------------------------------------------------------- host

std::atomic<int> g_clusters[kMaxSplit + 1];  // how many clusters of that many pairs run at a time

// The launch of `clusters` clusters of `pairs` pairs.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  Launch(int clusters, int pairs, int smem, cudaStream_t st) : attr(), cfg() {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2 * pairs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(clusters * 2 * pairs);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Launch(const Launch&) = delete;
};

template <int kMode, int kCols, bool kSplit = false>
cudaError_t launch_tiles(const Args& a, const CUtensorMap (&maps)[4], int64_t most_tiles, int num_sms,
                         cudaStream_t st) {
  const int pairs = num_sms / 2;
  const Launch l(static_cast<int>(kSplit || most_tiles < pairs ? most_tiles : pairs), a.split,
                 Config<kMode, kCols, kSplit>::smem, st);
  return cudaLaunchKernelEx(&l.cfg, linear_kernel<kMode, kCols, kSplit>, a, maps[0], maps[1], maps[2], maps[3]);
}

template <int kMode, int kCols, bool kSplit = false>
cudaError_t init_tiles() {
  if (kMode == kForward) {  // the epilogue would wait for registers that nobody has
    cudaFuncAttributes f;
    const cudaError_t err = cudaFuncGetAttributes(&f, linear_kernel<kMode, kCols, kSplit>);
    if (err != cudaSuccess) return err;
    if (f.numRegs * 3 < kFewRegisters + 2 * kManyRegisters) return cudaErrorInvalidConfiguration;
  }
  return cudaFuncSetAttribute(linear_kernel<kMode, kCols, kSplit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Config<kMode, kCols, kSplit>::smem);
}

// Columns of a tile, in steps of 32 (of 128 for the weight gradient).  Rows by experts, from an
// expert's average rows: 32 columns where they hold it with room for uneven loads (16 rows, gate
// and up of 128 experts: 111 us, 116 with 128 columns), then 128, and 256 where most experts would
// otherwise take a second tile and their weights come twice (128 rows: input gradient 126 us, 131
// with 128 columns; the forward product's epilogue prefers 128 columns there, 135 against 139 us;
// 256 rows: 93 against 105).  Otherwise the least time, in ns, of: waves of tiles over the pairs of
// SMs, times 64-element steps (0.13 us for what an SM loads, or what all pairs load at the 18.5 TB/s
// of L2; above 128 columns 0.25 to 0.32, where the matrix instructions bound a step), plus the last
// tile's epilogue (8192 x 2048 x 8192: 256 columns 181 us, 224 189; 4096 x 2048 x 2048: 23.5 each,
// 128 columns 28).  Where few tiles leave most SMs without one and their contraction is long, two
// to four pairs share each (as many as run at a time) for the time of the exchange, 0.15 us per
// further pair and 0.045 per pair in all: 128 x 4096 x 1024 12.4 -> 8.2 us, 300 x 8192 x 1024 21.8 ->
// 12.1, 64 x 2048 x 4096 8.1 -> 7.2, the weight gradient of 16384 x 2048 x 128 60 -> 19.5; 512 x 1024 x
// 2048 takes 6.4 without, 7.6 with.
int choose_tiles(const LinearDims& s, int mode, int tiles_m, int depth, int num_sms, int* split) {
  *split = 1;
  if (s.grouped && mode != kWeightGrad) {
    const int rows = (s.R + s.E - 1) / s.E;
    return rows <= 22 ? 32 : rows <= (mode == kInputGrad ? 96 : 176) ? 128 : 256;
  }
  const int64_t c = mode == kWeightGrad ? s.Nw() : s.R, groups = mode == kWeightGrad ? s.E : 1;
  const int64_t pairs = num_sms / 2, steps = (depth + 63) / 64;
  const int by = mode == kWeightGrad ? 128 : 32;
  int best = 256;
  int64_t least = INT64_MAX;
  for (int cols = 256; cols >= by; cols -= by) {
    const int64_t tiles = groups * tiles_m * ((c + cols - 1) / cols);
    const auto step = [&](int64_t busy) {
      if (cols > 128) return static_cast<int64_t>(128 + cols * 3 / 4);
      return std::max<int64_t>({122, 45 + cols * 2 / 3, std::min(busy, pairs) * (256 + cols) / 145});
    };
    const int64_t cost = (tiles + pairs - 1) / pairs * steps * step(tiles) + std::max(600, cols * 15 / 2);
    if (cost < least) {
      least = cost;
      best = cols;
      *split = 1;
    }
    for (int n = 2; n <= kMaxSplit && !s.grouped && cols <= 128; ++n) {
      if (tiles > g_clusters[n] || steps < 4 * n) continue;
      const int64_t shared = (steps + n - 1) / n * step(tiles * n) + 600 + 150 * n - 100 + 45 * tiles * n;
      if (shared < least) {
        least = shared;
        best = cols;
        *split = n;
      }
    }
  }
  return best;
}

cudaError_t run_mode(const LinearDims& s, int mode, const int32_t* offsets, const void* x, const void* w, const void* dz,
                     Args& a, int num_sms, cudaStream_t st) {
  a.offsets = offsets;
  a.R = s.R;
  a.E = s.E;
  a.N = s.N;
  a.Nw = s.Nw();
  a.bf16 = s.type;
  a.width = mode == kForward ? s.N : s.K;
  a.tile_m = a.gated ? 64 : kTileM;
  a.tiles_m = (a.width + 2 * a.tile_m - 1) / (2 * a.tile_m);
  a.per_m = ((uint64_t(1) << 40) + a.tiles_m - 1) / a.tiles_m;
  a.depth = mode == kForward ? s.K : a.Nw;
  a.tile_c = choose_tiles(s, mode, a.tiles_m, mode == kWeightGrad ? (s.R + s.E - 1) / s.E : a.depth, num_sms,
                          &a.split);
  const int cols = a.tile_c <= 32 && a.split == 1 ? 32 : a.tile_c <= 128 ? 128 : 256;  // the kernel's
  const int depth = cols == 256 ? Config<kForward, 256>::depth : Config<kForward, 128>::depth;
  a.tiles_c = (a.Nw + a.tile_c - 1) / a.tile_c;
  a.stage_bytes = (kTileM + a.tile_c / 2) * depth * 2;
  a.word = mma_word(s.type == 1, mode != kForward, mode == kWeightGrad, 2 * kTileM);
  CUtensorMap maps[4] = {};  // A, B, output, saved z
  bool ok;
  const bool bf16 = s.type == 1;
  const int64_t K = s.K, R = s.R, E = s.E, Nw = a.Nw;
  if (mode == kForward) {
    // rows in blocks of 8, a gated weight's gate and up blocks in turn
    const int64_t da[5] = {K, 8, s.gated ? 2 : 1, s.N / 8, E}, sa[4] = {K, s.N * K, 8 * K, Nw * K};
    const int ba[5] = {64, 8, s.gated ? 2 : 1, a.tile_m / 8, 1};
    const int64_t db[2] = {K, R}, sb[1] = {K};
    const int bb[2] = {64, a.tile_c / 2};
    ok = make_map(&maps[0], bf16, w, 5, da, sa, ba, true) && make_map(&maps[1], bf16, x, 2, db, sb, bb, true);
  } else if (mode == kInputGrad) {
    const int64_t da[3] = {K, Nw, E}, sa[2] = {K, Nw * K}, db[2] = {Nw, R}, sb[1] = {Nw};
    const int ba[3] = {64, depth, 1}, bb[2] = {64, a.tile_c / 2};
    ok = make_map(&maps[0], bf16, w, 3, da, sa, ba, true) && make_map(&maps[1], bf16, dz, 2, db, sb, bb, true);
  } else {
    const int64_t da[2] = {K, R}, sa[1] = {K}, db[2] = {Nw, R}, sb[1] = {Nw};
    const int box[2] = {64, depth};
    ok = make_map(&maps[0], bf16, x, 2, da, sa, box, true) && make_map(&maps[1], bf16, dz, 2, db, sb, box, true);
  }
  const int64_t width = a.width, planes = mode == kWeightGrad ? E : 1, lines = mode == kWeightGrad ? Nw : R;
  // the output: rows of `width` in planes; where the width is a multiple of 64, columns of 64 as
  // an extent of their own, so that one box takes both halves of a step
  const int rows = mode == kWeightGrad && a.split == 1 ? step_cols<kWeightGrad> : 32;
  a.one_store = width % 64 == 0;
  if (a.one_store) {
    const int64_t d[4] = {64, lines, width / 64, planes}, st4[3] = {width, 64, width * lines};
    const int box[4] = {64, rows, a.gated ? 1 : 2, 1};
    ok = ok && make_map(&maps[2], bf16, a.out, 4, d, st4, box, true);
  } else {
    const int64_t d[4] = {width, lines, 1, planes}, st4[3] = {width, width * lines, width * lines};
    const int box[4] = {64, rows, 1, 1};
    ok = ok && make_map(&maps[2], bf16, a.out, 4, d, st4, box, true);
  }
  if (a.preact) {
    const int64_t dzm[3] = {width, s.gated ? 2 : 1, R}, szm[2] = {width, Nw};
    const int bzm[3] = {64, 1, rows};
    ok = ok && make_map(&maps[3], bf16, a.preact, 3, dzm, szm, bzm, true);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int64_t most = mode == kWeightGrad ? E * a.tiles_m * a.tiles_c
                                           : int64_t(a.tiles_m) * ((R + a.tile_c - 1) / a.tile_c + (offsets ? E : 0));
  if (a.split > 1) {
    if (mode == kForward) return launch_tiles<kForward, 128, true>(a, maps, most, num_sms, st);
    if (mode == kInputGrad) return launch_tiles<kInputGrad, 128, true>(a, maps, most, num_sms, st);
    return launch_tiles<kWeightGrad, 128, true>(a, maps, most, num_sms, st);
  }
  if (mode == kForward) {
    if (cols == 32) return launch_tiles<kForward, 32>(a, maps, most, num_sms, st);
    if (cols == 128) return launch_tiles<kForward, 128>(a, maps, most, num_sms, st);
    return launch_tiles<kForward, 256>(a, maps, most, num_sms, st);
  }
  if (mode == kInputGrad) {
    if (cols == 32) return launch_tiles<kInputGrad, 32>(a, maps, most, num_sms, st);
    if (cols == 128) return launch_tiles<kInputGrad, 128>(a, maps, most, num_sms, st);
    return launch_tiles<kInputGrad, 256>(a, maps, most, num_sms, st);
  }
  if (cols == 128) return launch_tiles<kWeightGrad, 128>(a, maps, most, num_sms, st);
  return launch_tiles<kWeightGrad, 256>(a, maps, most, num_sms, st);
}

}  // namespace

cudaError_t init_linear_kernels() {
  cudaError_t err = init_tiles<kForward, 32>();
  if (err == cudaSuccess) err = init_tiles<kForward, 128>();
  if (err == cudaSuccess) err = init_tiles<kForward, 256>();
  if (err == cudaSuccess) err = init_tiles<kInputGrad, 32>();
  if (err == cudaSuccess) err = init_tiles<kInputGrad, 128>();
  if (err == cudaSuccess) err = init_tiles<kInputGrad, 256>();
  if (err == cudaSuccess) err = init_tiles<kWeightGrad, 128>();
  if (err == cudaSuccess) err = init_tiles<kWeightGrad, 256>();
  if (err == cudaSuccess) err = init_tiles<kForward, 128, true>();
  for (int n = 2; err == cudaSuccess && n <= kMaxSplit; ++n) {
    const Launch l(1, n, Config<kForward, 128, true>::smem, nullptr);
    int count = 0;
    err = cudaOccupancyMaxActiveClusters(&count, linear_kernel<kForward, 128, true>, &l.cfg);
    g_clusters[n] = count;
  }
  if (err == cudaSuccess) err = init_tiles<kInputGrad, 128, true>();
  if (err == cudaSuccess) err = init_tiles<kWeightGrad, 128, true>();
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
                                      void* dw, const float* partial, float* dbias, int32_t* err, int num_sms,
                                      cudaStream_t st) {
  Args a = {};
  a.partial = partial;
  a.dbias = dbias;
  a.block_rows = linear_block_rows(s.R);
  a.out = static_cast<uint16_t*>(dw);
  a.err = err;
  a.act = 3;
  return run_mode(s, kWeightGrad, offsets, x, nullptr, dz, a, num_sms, st);
}

}  // namespace moe
