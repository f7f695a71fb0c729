// NoPE MLA of a step's new tokens over the paged latent cache: causal, with an
// optional sliding window beside which the first tokens stay visible.
//
// Module glm5next_dsa, "Traps carried from Slice 8" (NoPE: a score is the plain
// latent dot product) and Constants, MASKED_ATTN_MAX_KEYS (dense masked
// attention).  A token at position p sees the positions [0, s0) and [lo, p] with
// lo = max(0, p - window + 1) (0 without a window) and s0 = min(sinks, lo): two
// ranges, so no kernel ever holds a mask.
//
// This file: the dispatch, and the generic kernel for any geometry and type
// (fp32 activations, latent widths other than 512, fp32 pages).  One CTA of four
// warps = one token and four heads; a tile of visible rows is brought into shared
// memory as fp32 once, thread pairs (key, head) take the scores from it, threads
// (column, head) the output.  Running maximum, sum and outputs are fp32.  It is bound
// by the latency of a tile's row reads and barriers (the 200-token fp32 prompt: see
// the measurements); the tcgen05 kernels take the serving geometry.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "dsa_internal.cuh"

namespace dsa {
namespace {

constexpr int kChunkThreads = 128, kChunkHeads = 4, kChunkTile = 64;
constexpr int kChunkCols = 1024 / kChunkThreads;  // latent columns of a thread at most
constexpr int kChunkFloats = 16384;               // of a tile's rows
// keys of a tile: the rows (one float of padding each: columns of 32 rows in different
// banks) fit kChunkFloats
__host__ __device__ constexpr int chunk_tile(int L) {
  return kChunkFloats / (L + 1) < kChunkTile ? kChunkFloats / (L + 1) : kChunkTile;
}

__device__ __forceinline__ float page_value(const PagedKv& pk, long long row, int d, int L) {
  const long long o = row * L + d;
  if (pk.kv_dtype == DSA_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(pk.pages)[o]);
  if (pk.kv_dtype == DSA_F32) return static_cast<const float*>(pk.pages)[o];
  const __half_raw h =
      __nv_cvt_fp8_to_halfraw(static_cast<const __nv_fp8_storage_t*>(pk.pages)[o], __NV_E4M3);
  return __half2float(*reinterpret_cast<const __half*>(&h)) * pk.row_scale[row];
}

template <typename T>
__global__ void __launch_bounds__(kChunkThreads) mla_chunk_simt_kernel(ChunkArgs a) {
  extern __shared__ float rows[];  // [tile][L + 1], then the queries [kChunkHeads][L]
  __shared__ float sz[kChunkHeads][kChunkTile];
  __shared__ int srow[kChunkTile];
  __shared__ float s_m[kChunkHeads], s_l[kChunkHeads], s_alpha[kChunkHeads];
  const int L = a.L, Lp = a.L + 1, kt = chunk_tile(a.L);
  float* sq = rows + kt * Lp;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, h0 = blockIdx.y * kChunkHeads;
  const int nh = min(kChunkHeads, a.Hm - h0);
  const bool reports = blockIdx.y == 0;
  if (blockIdx.x == 0 && reports)
    for (int b = tid; b < a.B; b += kChunkThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b] > a.cu_new[b + 1] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  // the sequence that owns row t
  if (a.cu_new[0] > t) return;
  int b = 0;
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (a.cu_new[mid] <= t) b = mid; else hi = mid;
  }
  const int c0 = max(a.cu_new[b], 0), c1 = min(a.cu_new[b + 1], a.T);
  if (t < c0 || t >= c1) return;  // behind the last sequence: left as it was
  const int len = a.kv.seq_lens[b];
  const long long at = (long long)len - (c1 - c0) + (t - c0);
  if (at < 0 && reports && tid == 0) flag(a.status, DSA_DEV_BAD_LENGTH);
  const int pos = (int)max(at, -1ll);
  // (positions behind the table's width have no page)
  const long long width = (long long)a.kv.max_pages * a.kv.page_size;
  const int cap = (int)min(width, 0x7fffffffll);
  if (pos >= cap && reports && tid == 0) flag(a.status, DSA_DEV_BAD_PAGE);
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int s0 = min(min(a.sinks, lo), cap);
  const int nv = pos < 0 ? 0 : s0 + max(min(pos, cap - 1) - lo + 1, 0);  // visible positions

  const long long qh = (long long)t * a.Hm + h0;
  const T* q = static_cast<const T*>(a.q_lat) + qh * a.L;
  for (int i = tid; i < kChunkHeads * L; i += kChunkThreads)
    sq[i] = i < nh * L ? Act<T>::to_f(q[i]) : 0.f;
  if (tid < kChunkHeads) {
    s_m[tid] = -INFINITY;
    s_l[tid] = 0.f;
  }
  float acc[kChunkHeads][kChunkCols];
#pragma unroll
  for (int h = 0; h < kChunkHeads; ++h)
#pragma unroll
    for (int c = 0; c < kChunkCols; ++c) acc[h][c] = 0.f;

  for (int v0 = 0; v0 < nv; v0 += kt) {
    const int n = min(kt, nv - v0);
    __syncthreads();
    if (tid < n) {
      const int v = v0 + tid, p = v < s0 ? v : lo + (v - s0);
      const int blk = p / a.kv.page_size;
      const int page =
          blk < a.kv.max_pages ? a.kv.block_table[(long long)b * a.kv.max_pages + blk] : -1;
      const bool ok = page >= 0 && page < a.kv.n_pages;
      if (!ok && reports) flag(a.status, DSA_DEV_BAD_PAGE);
      srow[tid] = ok ? page * a.kv.page_size + p % a.kv.page_size : -1;
    }
    __syncthreads();
    for (int j = warp; j < n; j += kChunkThreads / 32) {  // (a position without a page: zeros)
      const int row = srow[j];
      for (int d = lane; d < L; d += 32)
        rows[j * Lp + d] = row >= 0 ? page_value(a.kv, row, d, L) : 0.f;
    }
    __syncthreads();
    for (int i = tid; i < n * kChunkHeads; i += kChunkThreads) {
      const int j = i % n, h = i / n;
      const float* x = rows + j * Lp;
      const float* y = sq + h * L;
      float d4[4] = {0.f, 0.f, 0.f, 0.f};
      for (int d = 0; d < L; d += 8) {  // L is a multiple of 8
#pragma unroll
        for (int u = 0; u < 8; ++u) d4[u & 3] = fmaf(x[d + u], y[d + u], d4[u & 3]);
      }
      sz[h][j] = srow[j] >= 0 ? ((d4[0] + d4[1]) + (d4[2] + d4[3])) * a.sm_scale : -INFINITY;
    }
    __syncthreads();
    if (warp < nh) {  // warp = head: two positions a lane
      const float za = lane < n ? sz[warp][lane] : -INFINITY;
      const float zb = lane + 32 < n ? sz[warp][lane + 32] : -INFINITY;
      const float m_old = s_m[warp], m = fmaxf(m_old, warp_max(fmaxf(za, zb)));
      const float ref = m == -INFINITY ? 0.f : m;
      const float ea = expf(za - ref), eb = expf(zb - ref);
      const float sum = warp_sum(ea + eb);
      __syncwarp();
      sz[warp][lane] = ea;
      sz[warp][lane + 32] = eb;
      if (lane == 0) {
        const float alpha = expf(m_old - ref);  // 0 before the first visible position
        s_m[warp] = m;
        s_l[warp] = s_l[warp] * alpha + sum;
        s_alpha[warp] = alpha;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kChunkHeads; ++h) {
      const float alpha = h < nh ? s_alpha[h] : 0.f;
#pragma unroll
      for (int c = 0; c < kChunkCols; ++c) acc[h][c] *= alpha;
    }
#pragma unroll
    for (int c = 0; c < kChunkCols; ++c) {
      const int d = c * kChunkThreads + tid;
      if (d >= L) break;
#pragma unroll 4
      for (int j = 0; j < n; ++j) {
        const float x = rows[j * Lp + d];
#pragma unroll
        for (int h = 0; h < kChunkHeads; ++h) acc[h][c] = fmaf(sz[h][j], x, acc[h][c]);
      }
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + qh * a.L;
#pragma unroll
  for (int h = 0; h < kChunkHeads; ++h) {
    if (h >= nh) break;
    const float l = s_l[h], inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
#pragma unroll
    for (int c = 0; c < kChunkCols; ++c) {
      const int d = c * kChunkThreads + tid;
      if (d < a.L) out[(long long)h * a.L + d] = Act<T>::from_f(acc[h][c] * inv);
    }
    if (a.lse && tid == 0) a.lse[qh + h] = l == 0.f ? -INFINITY : s_m[h] + logf(l);
  }
}

}  // namespace

size_t mla_chunk_workspace_size(int T, int Hm, int L, int dtype, int kv_dtype) {
  if (T < 1 || !mla_chunk_umma_ok(L, dtype, kv_dtype)) return 0;
  const size_t one = mla_chunk_umma_workspace_size(Hm);
  const size_t two = kv_dtype == DSA_FP8_E4M3 ? mla_chunk_f8_workspace_size(T, Hm)
                                              : (Hm > 32 ? mla_chunk_pair_workspace_size() : 0);
  return one > two ? one : two;
}

namespace {

// Whether pairs of CTAs are the faster kernel for bf16 pages: two row blocks of a step
// must share their keys (two new tokens of a sequence on average, or more than 64
// heads), and a row must see enough of them to pay for the exchange's start and end.
// The lengths live on the device: the window and the block table's width bound them.
// Measured on GB300, pair / single CTA in us (sequences x new tokens, 64 heads):
//   context  8,192, 32 x 4: 177 / 196, 16 x 16: 317 / 361, 4 x 256: 1,101 / 1,221
//   context  2,048, 32 x 4:  72 /  70, 16 x 16: 111 / 104, 4 x 256:   330 /   336
//   context    512, 32 x 4:  45 /  35, 16 x 16:  61 /  46, 4 x 256:   138 /   114
//   window   4,096 of 16,384, 4 x 256: 627 / 662; 2,048: 370 / 367; 512: 177 / 143
//   single tokens, context 8,192: 64 x 1: 165 / 111, 64 heads; 32 x 2: 106 / 109
bool pairs_pay(const ChunkArgs& a) {
  if (a.kv.kv_dtype != DSA_BF16 || (a.Hm <= 64 && a.T < 2ll * a.B)) return false;
  const long long table = (long long)a.kv.max_pages * a.kv.page_size;
  const long long seen = a.window > 0 ? (long long)a.window + a.sinks : table;
  return (seen < table ? seen : table) > 2048;
}

}  // namespace

int launch_mla_chunk(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  if (mla_chunk_umma_ok(a.L, a.dtype, a.kv.kv_dtype)) {
    if (a.kv.kv_dtype == DSA_FP8_E4M3 && a.kv.page_size % 8 == 0)
      return launch_mla_chunk_f8(a, workspace, stream);
    return pairs_pay(a) && mla_chunk_pair_ok(a.Hm, a.kv.page_size)
               ? launch_mla_chunk_pair(a, workspace, stream)
               : launch_mla_chunk_umma(a, workspace, stream);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.T, (a.Hm + kChunkHeads - 1) / kChunkHeads, 1);
  cfg.blockDim = dim3(kChunkThreads, 1, 1);
  cfg.dynamicSmemBytes =
      ((size_t)chunk_tile(a.L) * (a.L + 1) + (size_t)kChunkHeads * a.L) * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = a.dtype == DSA_BF16 ? mla_chunk_simt_kernel<__nv_bfloat16>
                                    : mla_chunk_simt_kernel<float>;
  if (cfg.dynamicSmemBytes > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)cfg.dynamicSmemBytes) != cudaSuccess)
    return DSA_ERR_CUDA;
  return launch_kernel(&cfg, kernel, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
