// rows.cu -- token rows sorted by expert and back, with the router's weights, and
// the gradients of both (fp16, bf16 or fp32 rows).
//
//   dispatch           rows[pos[p]] = x[p / k] for every kept pair p, sorted by expert, p ascending
//   dispatch backward  dx[t] = sum_r drows[pos[t k + r]]
//   combine            out[t] = res[t] + sum_r w[t][r] rows[pos[t k + r]]
//   combine backward   drows[pos[p]] = w_p dout[t],  dw_p = <dout[t], rows[pos[p]]>,
//                      dlogits[t][e_r] += w_r (dw_r - sum_j w_j dw_j)  (softmax over the k selected)
//
// All four move each row once: they are bound by memory (dispatch (T + P) rows,
// combine backward (T + 2 P) rows; the arithmetic is one multiply-add per element).
// A token's pairs are handled together, so x and dout are read once, not k times,
// and the k rows of a token are summed in registers in rank order: no atomics, the
// same bits in every run.
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "row_vec.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;  // threads per CTA; at least one per expert (E <= 256)
static_assert(kMaxExperts <= kThreads, "one thread per expert");

// The expert of a pair, E for a dropped one (an id outside 0 .. E-1).
__device__ __forceinline__ int expert_of(int id, int E) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(E) ? id : E;
}

// ---------------------------------------------------------------- dispatch
//
// A stable counting sort.  The pairs are cut into chunks; a pair's row is
//   offset[e] + pairs of e in earlier chunks + earlier pairs of e in its chunk.
// Up to kOneChunkPairs pairs are one chunk and one launch: every CTA counts all ids
// itself (16 per thread at most, from L2), which costs less than a second launch.
// More pairs are counted per chunk first (count), the counts summed over chunks
// (prefix), and every CTA of the copy counts only the ids of its chunk before its
// own pairs.
constexpr int kOneChunkPairs = 4096;
constexpr int kChunkPairs = 512;  // pairs per chunk above that, about
constexpr int kCtaPairs = 64;     // pairs per CTA of the copy, at most: two warps place them
constexpr int kCopyLoads = 4;     // pieces a thread has in flight

// Tokens per CTA of the copy: about 64 KB of rows.  A CTA spends some microseconds on its
// pairs' places first, so many small ones hide each other's (16384 tokens top-8 of 4 KB rows:
// 108 us with 64 pairs per CTA, 98 us with 16), but below that the placing shows (1 KB rows:
// 33 us with 64 pairs, 40 us with 16).
inline int copy_tokens(const RowDims& s) {
  int pairs = 65536 / (s.nvec() * 16);
  pairs = pairs < 16 ? 16 : pairs > kCtaPairs ? kCtaPairs : pairs;
  return pairs / s.k;
}
inline int chunk_pairs(const RowDims& s) {  // whole CTAs of whole tokens
  const int cta = copy_tokens(s) * s.k;
  return kChunkPairs / cta * cta;
}

__global__ void __launch_bounds__(kThreads) dispatch_count_kernel(const int32_t* ids, int P, int E,
                                                                  int chunk, int32_t* hist) {
  __shared__ int cnt[kMaxExperts + 1];
  grid_dependents_launch();
  grid_dependency_wait();
  for (int e = threadIdx.x; e <= E; e += kThreads) cnt[e] = 0;
  __syncthreads();
  const int p0 = blockIdx.x * chunk, p1 = min(P, p0 + chunk);
  for (int p = p0 + threadIdx.x; p < p1; p += kThreads) atomicAdd(&cnt[expert_of(ids[p], E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) hist[static_cast<size_t>(blockIdx.x) * E + e] = cnt[e];
}

// hist[c][e] becomes the sum over chunks before c, tot[e] the sum over all.  Lane =
// expert; warp w takes a contiguous run of chunks.
__global__ void __launch_bounds__(1024) dispatch_prefix_kernel(int32_t* hist, int nchunks, int E,
                                                               int32_t* tot) {
  __shared__ int part[32][33];
  grid_dependents_launch();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  const int per = (nchunks + 31) / 32;
  const int c0 = min(nchunks, warp * per), c1 = min(nchunks, c0 + per);
  int s = 0;
  if (e < E) {
#pragma unroll 8
    for (int c = c0; c < c1; ++c) s += hist[static_cast<size_t>(c) * E + e];
  }
  part[warp][lane] = s;
  __syncthreads();
  int run = 0;
  for (int w = 0; w < warp; ++w) run += part[w][lane];
  if (e < E) {
    if (warp == 31) tot[e] = run + s;
    for (int c = c0; c < c1; ++c) {
      int32_t* h = hist + static_cast<size_t>(c) * E + e;
      const int v = *h;
      *h = run;
      run += v;
    }
  }
}

// One CTA places the pairs of `tpc` tokens (tpc * k <= kCtaPairs) and copies their rows: each
// 16-byte piece of a token is read once and written to the token's k rows.
// hist/tot are NULL when all pairs are one chunk.
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const int32_t* ids, int T, int k, int E,
                                                            int tpc, int chunk, const int32_t* hist,
                                                            const int32_t* tot,
                                                            const uint4* x, int nvec,
                                                            int32_t* offsets,
                                                            int32_t* pair_list,
                                                            int32_t* pair_pos, uint4* rows) {
  __shared__ int before[kMaxExperts + 1];  // pairs of an expert before the CTA's, then their first row
  __shared__ int total[kMaxExperts + 1];
  __shared__ int warp_tot[kThreads / 32];
  __shared__ int row_of[kCtaPairs];
  grid_dependents_launch();
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = T * k;
  const int t0 = blockIdx.x * tpc, nt = min(tpc, T - t0);
  const int p0 = t0 * k, np = nt * k;
  const int c = p0 / chunk, cp0 = c * chunk;  // a CTA's pairs lie in one chunk
  for (int e = tid; e <= E; e += kThreads) {
    before[e] = hist && e < E ? hist[static_cast<size_t>(c) * E + e] : 0;
    total[e] = tot && e < E ? tot[e] : 0;
  }
  __syncthreads();
  if (tot) {
    for (int p = cp0 + tid; p < p0; p += kThreads) atomicAdd(&before[expert_of(ids[p], E)], 1);
  } else {
    for (int p = tid; p < P; p += kThreads) {
      const int e = expert_of(ids[p], E);
      atomicAdd(&total[e], 1);
      if (p < p0) atomicAdd(&before[e], 1);
    }
  }
  __syncthreads();
  // exclusive scan of the totals: thread e holds expert e
  const int v = tid < E ? total[tid] : 0;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_tot[warp] = incl;
  __syncthreads();
  int base = incl - v, kept = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    base += w < warp ? warp_tot[w] : 0;
    kept += warp_tot[w];
  }
  if (tid < E) {
    before[tid] += base;
    if (blockIdx.x == 0) offsets[tid] = base;
  }
  if (blockIdx.x == 0 && tid == 0) offsets[E] = kept;
  __syncthreads();
  // the CTA's pairs in order, 32 per warp: the rank among the warp's earlier pairs of the
  // same expert; the second warp's pairs follow the first's
  int e = E, rank = 0, peers = 0;
  if (warp < 2) {
    e = tid < np ? expert_of(ids[p0 + tid], E) : E;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    rank = __popc(same & ((1u << lane) - 1u));
    peers = __popc(same);
  }
  for (int w = 0; w < 2; ++w) {
    if (warp == w && tid < np) {
      const int row = e < E ? before[e] + rank : -1;
      row_of[tid] = row;
      pair_pos[p0 + tid] = row;
      if (row >= 0) pair_list[row] = p0 + tid;
    }
    __syncwarp();
    if (warp == w && e < E && rank == 0) before[e] += peers;
    __syncthreads();
  }
  // pair_list behind the kept pairs
  for (int p = kept + blockIdx.x * kThreads + tid; p < P; p += gridDim.x * kThreads) pair_list[p] = -1;
  const uint4* src = x + static_cast<size_t>(t0) * nvec;
  const int total_pieces = nt * nvec;
  for (int j0 = tid; j0 < total_pieces; j0 += kThreads * kCopyLoads) {
    uint4 piece[kCopyLoads];
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u)
      if (j0 + u * kThreads < total_pieces) piece[u] = src[j0 + u * kThreads];
#pragma unroll
    for (int u = 0; u < kCopyLoads; ++u) {
      const int j = j0 + u * kThreads;
      if (j >= total_pieces) break;
      const int t = j / nvec, col = j - t * nvec;
#pragma unroll
      for (int r = 0; r < kMaxTopK; ++r)
        if (r < k) {
          const int row = row_of[t * k + r];
          if (row >= 0) rows[static_cast<size_t>(row) * nvec + col] = piece[u];
        }
    }
  }
}

// ----------------------------------------------------------------- combine
//
// One thread per 16-byte piece of a token's row; the pieces of the k rows are all
// requested before the first is used.  With topk_w NULL every weight is one (the
// gradient of dispatch).
// With few choices a thread takes several tokens' pieces at once, 8 / kChoices of them, so that
// eight loads are in flight whatever k is.
template <int kType, int kChoices>
__global__ void __launch_bounds__(kThreads) combine_rows_kernel(const int32_t* pair_pos, const float* topk_w,
                                                                const uint4* rows,
                                                                const uint4* residual,  // may equal out
                                                                uint4* out, int T, int k, int nvec, int tpc) {
  constexpr int kPieces = kMaxTopK / kChoices, N = Vec<kType>::n;
  grid_dependents_launch();
  grid_dependency_wait();
  const int P = T * k;
  const int t0 = blockIdx.x * tpc, n = min(tpc, T - t0) * nvec;
  for (int j0 = threadIdx.x; j0 < n; j0 += kThreads * kPieces) {
    int pos[kPieces][kChoices];
    float w[kPieces][kChoices];
    uint4 v[kPieces][kChoices], res[kPieces];
    size_t at[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int j = j0 + u * kThreads;
      const int tl = j / nvec, t = t0 + tl;
      at[u] = static_cast<size_t>(t0) * nvec + j;
#pragma unroll
      for (int r = 0; r < kChoices; ++r) {
        const bool on = j < n && r < k;
        pos[u][r] = on ? pair_pos[t * k + r] : -1;
        w[u][r] = on && topk_w ? topk_w[t * k + r] : 1.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int j = j0 + u * kThreads, col = j % nvec;
#pragma unroll
      for (int r = 0; r < kChoices; ++r)
        if (static_cast<unsigned>(pos[u][r]) < static_cast<unsigned>(P))
          v[u][r] = rows[static_cast<size_t>(pos[u][r]) * nvec + col];
      if (residual && j < n) res[u] = residual[at[u]];
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (j0 + u * kThreads >= n) break;
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
#pragma unroll
      for (int r = 0; r < kChoices; ++r)
        if (static_cast<unsigned>(pos[u][r]) < static_cast<unsigned>(P)) {
          float f[N];
          Vec<kType>::load(v[u][r], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = fmaf(w[u][r], f[i], acc[i]);
        }
      if (residual) {
        float f[N];
        Vec<kType>::load(res[u], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += f[i];
      }
      out[at[u]] = Vec<kType>::store(acc);
    }
  }
}

// -------------------------------------------------------- combine backward
//
// kGroup threads per token, 256 / kGroup tokens per CTA.  Each thread keeps the k
// partial products <dout, row_r> of its pieces, 8 / kChoices pieces at a time so that eight
// rows' loads are in flight whatever k is; they meet in a fixed tree (a butterfly that halves
// the values at each of its first three steps, then the warps of the group in order).
template <int kType, int kGroup, int kChoices>
__global__ void __launch_bounds__(kThreads) combine_rows_backward_kernel(
    const int32_t* topk_idx, const int32_t* pair_pos, const float* topk_w, const uint4* rows, const uint4* dout,
    uint4* drows, float* dtopk_w, float* dlogits, int T, int k, int E, int nvec) {
  constexpr int kTokens = kThreads / kGroup, kWarps = kGroup / 32, N = Vec<kType>::n;
  constexpr int kPieces = kMaxTopK / kChoices;
  __shared__ float part[kThreads / 32][kMaxTopK];
  grid_dependents_launch();
  grid_dependency_wait();
  const int P = T * k;
  const int tl = threadIdx.x / kGroup, g = threadIdx.x % kGroup, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kTokens + tl;
  const bool on = t < T;
  int pos[kMaxTopK];
  float w[kMaxTopK], dot[kMaxTopK];
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r) {
    pos[r] = on && r < kChoices && r < k ? pair_pos[t * k + r] : -1;
    w[r] = on && r < kChoices && r < k ? topk_w[t * k + r] : 0.f;
    dot[r] = 0.f;
  }
  if (on) {
    for (int col0 = g; col0 < nvec; col0 += kGroup * kPieces) {
      uint4 v[kPieces][kChoices], dv[kPieces];
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int col = col0 + u * kGroup;
        if (col < nvec) {
          dv[u] = dout[static_cast<size_t>(t) * nvec + col];
#pragma unroll
          for (int r = 0; r < kChoices; ++r)
            if (static_cast<unsigned>(pos[r]) < static_cast<unsigned>(P))
              v[u][r] = rows[static_cast<size_t>(pos[r]) * nvec + col];
        }
      }
#pragma unroll
      for (int u = 0; u < kPieces; ++u) {
        const int col = col0 + u * kGroup;
        if (col >= nvec) break;
        float d[N];
        Vec<kType>::load(dv[u], d);
#pragma unroll
        for (int r = 0; r < kChoices; ++r)
          if (static_cast<unsigned>(pos[r]) < static_cast<unsigned>(P)) {
            float f[N], o[N];
            Vec<kType>::load(v[u][r], f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dot[r] = fmaf(d[i], f[i], dot[r]);
              o[i] = w[r] * d[i];
            }
            if (drows) drows[static_cast<size_t>(pos[r]) * nvec + col] = Vec<kType>::store(o);
          }
      }
    }
  }
  // lane l ends with the warp's sum for r = l & 7: each step exchanges the half of the
  // values whose r differs from the lane's in one bit
  float h4[4], h2[2], h1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // r bit 2
    const bool up = lane & 4;
    const float keep = up ? dot[i + 4] : dot[i], give = up ? dot[i] : dot[i + 4];
    h4[i] = keep + __shfl_xor_sync(0xffffffffu, give, 4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {  // r bit 1
    const bool up = lane & 2;
    const float keep = up ? h4[i + 2] : h4[i], give = up ? h4[i] : h4[i + 2];
    h2[i] = keep + __shfl_xor_sync(0xffffffffu, give, 2);
  }
  {
    const bool up = lane & 1;  // r bit 0
    const float keep = up ? h2[1] : h2[0], give = up ? h2[0] : h2[1];
    h1 = keep + __shfl_xor_sync(0xffffffffu, give, 1);
  }
  h1 += __shfl_xor_sync(0xffffffffu, h1, 8);
  h1 += __shfl_xor_sync(0xffffffffu, h1, 16);
  if (kWarps > 1) {
    if (lane < kMaxTopK) part[threadIdx.x >> 5][lane] = h1;
    __syncthreads();
    h1 = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) h1 += part[tl * kWarps + i][lane & 7];
  }
  if (!on) return;
  float dw[kMaxTopK], mean = 0.f;
#pragma unroll
  for (int r = 0; r < kMaxTopK; ++r) {
    dw[r] = __shfl_sync(0xffffffffu, h1, r);
    // (a dropped pair has dw = 0, and its weight may be anything)
    if (static_cast<unsigned>(pos[r]) < static_cast<unsigned>(P)) mean = fmaf(w[r], dw[r], mean);
  }
  if (dtopk_w && g < k) dtopk_w[t * k + g] = h1;  // lane g of the group's first warp: r = g
  if (dlogits) {
    // a dropped choice too: its logit is in the softmax's sum, whatever became of its row
    int id[kMaxTopK];
#pragma unroll
    for (int r = 0; r < kMaxTopK; ++r) id[r] = r < k ? topk_idx[t * k + r] : -1;
    for (int e = g; e < E; e += kGroup) {
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < kMaxTopK; ++r)
        if (id[r] == e) s += w[r] * (dw[r] - mean);
      dlogits[static_cast<size_t>(t) * E + e] = s;
    }
  }
}

template <int kType>
cudaError_t launch_backward(const RowDims& s, const int32_t* topk_idx, const int32_t* pair_pos, const float* topk_w,
                            const uint4* rows, const uint4* dout, uint4* drows, float* dtopk_w, float* dlogits,
                            cudaStream_t st) {
  const int nvec = s.nvec();
  const auto go = [&](auto kernel, int group) {
    const int per = kThreads / group;
    return launch_pdl(kernel, dim3((s.T + per - 1) / per), dim3(kThreads), 0, st, topk_idx, pair_pos, topk_w, rows,
                      dout, drows, dtopk_w, dlogits, s.T, s.k, s.E, nvec);
  };
  // threads per token: one round of its pieces, at most
  if (s.k == 1) return go(combine_rows_backward_kernel<kType, 32, 1>, 32);
  if (s.k == 2) {
    if (nvec <= 128) return go(combine_rows_backward_kernel<kType, 32, 2>, 32);
    return go(combine_rows_backward_kernel<kType, 64, 2>, 64);
  }
  if (s.k <= 4) {
    if (nvec <= 64) return go(combine_rows_backward_kernel<kType, 32, 4>, 32);
    if (nvec <= 128) return go(combine_rows_backward_kernel<kType, 64, 4>, 64);
    return go(combine_rows_backward_kernel<kType, 128, 4>, 128);
  }
  if (nvec <= 32) return go(combine_rows_backward_kernel<kType, 32, 8>, 32);
  if (nvec <= 64) return go(combine_rows_backward_kernel<kType, 64, 8>, 64);
  if (nvec <= 128) return go(combine_rows_backward_kernel<kType, 128, 8>, 128);
  return go(combine_rows_backward_kernel<kType, 256, 8>, 256);
}

}  // namespace

size_t dispatch_ws_bytes(const RowDims& s) {
  const int64_t P = s.pairs();
  if (P <= kOneChunkPairs) return 16;
  const int chunk = chunk_pairs(s);
  return (size_t((P + chunk - 1) / chunk) + 1) * s.E * 4;
}

cudaError_t launch_dispatch(const RowDims& s, const int32_t* topk_idx, const void* x, int32_t* offsets,
                            int32_t* pair_list, int32_t* pair_pos, void* rows, void* workspace, cudaStream_t st) {
  const int P = static_cast<int>(s.pairs()), nvec = s.nvec();
  const auto* xv = static_cast<const uint4*>(x);
  auto* rv = static_cast<uint4*>(rows);
  if (P <= kOneChunkPairs) {
    // two CTAs per SM where the tokens suffice, whole tokens
    const int want = (s.T + 303) / 304, most = kCtaPairs / s.k, tpc = want < most ? want : most;
    return launch_pdl(dispatch_kernel, dim3((s.T + tpc - 1) / tpc), dim3(kThreads), 0, st, topk_idx, s.T, s.k, s.E,
                      tpc, P, static_cast<const int32_t*>(nullptr), static_cast<const int32_t*>(nullptr), xv, nvec,
                      offsets, pair_list, pair_pos, rv);
  }
  const int tpc = copy_tokens(s), chunk = chunk_pairs(s), nchunks = (P + chunk - 1) / chunk;
  auto* hist = static_cast<int32_t*>(workspace);
  int32_t* tot = hist + static_cast<size_t>(nchunks) * s.E;
  cudaError_t err =
      launch_pdl(dispatch_count_kernel, dim3(nchunks), dim3(kThreads), 0, st, topk_idx, P, s.E, chunk, hist);
  if (err != cudaSuccess) return err;
  err = launch_pdl(dispatch_prefix_kernel, dim3((s.E + 31) / 32), dim3(1024), 0, st, hist, nchunks, s.E, tot);
  if (err != cudaSuccess) return err;
  return launch_pdl(dispatch_kernel, dim3((s.T + tpc - 1) / tpc), dim3(kThreads), 0, st, topk_idx, s.T, s.k, s.E, tpc,
                    chunk, static_cast<const int32_t*>(hist), static_cast<const int32_t*>(tot), xv, nvec, offsets,
                    pair_list, pair_pos, rv);
}

cudaError_t launch_combine_rows(const RowDims& s, const int32_t* pair_pos, const float* topk_w, const void* rows,
                                const void* residual, void* out, cudaStream_t st) {
  const int nvec = s.nvec();
  const auto go = [&](auto kernel, int choices) {
    int tpc = kThreads * (kMaxTopK / choices) / nvec;  // one round of a CTA, whole tokens
    if (tpc < 1) tpc = 1;
    while (tpc > 1 && (s.T + tpc - 1) / tpc < 608) tpc = (tpc + 1) / 2;  // four CTAs per SM at least
    return launch_pdl(kernel, dim3((s.T + tpc - 1) / tpc), dim3(kThreads), 0, st, pair_pos, topk_w,
                      static_cast<const uint4*>(rows), static_cast<const uint4*>(residual), static_cast<uint4*>(out),
                      s.T, s.k, nvec, tpc);
  };
  const auto by_k = [&](auto type) {
    constexpr int t = decltype(type)::value;
    if (s.k == 1) return go(combine_rows_kernel<t, 1>, 1);
    if (s.k == 2) return go(combine_rows_kernel<t, 2>, 2);
    if (s.k <= 4) return go(combine_rows_kernel<t, 4>, 4);
    return go(combine_rows_kernel<t, 8>, 8);
  };
  if (s.type == 0) return by_k(std::integral_constant<int, 0>{});
  if (s.type == 1) return by_k(std::integral_constant<int, 1>{});
  return by_k(std::integral_constant<int, 2>{});
}

cudaError_t launch_combine_rows_backward(const RowDims& s, const int32_t* topk_idx, const int32_t* pair_pos,
                                         const float* topk_w, const void* rows, const void* dout, void* drows,
                                         float* dtopk_w, float* dlogits, cudaStream_t st) {
  const auto* rv = static_cast<const uint4*>(rows);
  const auto* dv = static_cast<const uint4*>(dout);
  auto* gv = static_cast<uint4*>(drows);
  if (s.type == 0) return launch_backward<0>(s, topk_idx, pair_pos, topk_w, rv, dv, gv, dtopk_w, dlogits, st);
  if (s.type == 1) return launch_backward<1>(s, topk_idx, pair_pos, topk_w, rv, dv, gv, dtopk_w, dlogits, st);
  return launch_backward<2>(s, topk_idx, pair_pos, topk_w, rv, dv, gv, dtopk_w, dlogits, st);
}

}  // namespace moe
