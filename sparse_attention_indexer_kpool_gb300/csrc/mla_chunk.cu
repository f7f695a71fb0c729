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
// warps = one token and four heads; a tile of up to 128 visible rows is brought into
// shared memory as fp32 once (16-byte pieces, four on their way a thread, the next
// tile's pages looked up meanwhile), a thread takes the score of a key and a head from
// it, and a thread's latent columns of four heads the output.  Running maximum, sum
// and outputs are fp32.  It is bound by the latency of a tile's loads and barriers: 200
// new fp32 tokens, 4 heads of latent 64, 11.7 us on GB300 (tiles of 64 rows copied
// element by element: 26.9 us).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "dsa_internal.cuh"

namespace dsa {
namespace {

constexpr int kChunkThreads = 128, kChunkHeads = 4, kChunkTile = 128;
constexpr int kChunkCols = 1024 / kChunkThreads;  // latent columns of a thread at most
constexpr int kChunkFloats = 16384;               // of a tile's rows
// A row in shared memory is L + 4 floats apart from the next (L is a multiple of 8: an
// odd number of 16-byte pieces), so that eight threads' pieces of eight rows lie in
// different banks, as those of one row do.
__host__ __device__ constexpr int chunk_pitch(int L) { return L + 4; }
__host__ __device__ constexpr int chunk_tile(int L) {
  return kChunkFloats / chunk_pitch(L) < kChunkTile ? kChunkFloats / chunk_pitch(L) : kChunkTile;
}

// Eight elements of a cache row.
template <int kKv> struct Piece;
template <> struct Piece<DSA_BF16> {
  uint4 v;
  __device__ __forceinline__ void load(const PagedKv& kv, long long row, int at, int L) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(kv.pages) +
                                             row * L + at));
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(u[i]);
      f[2 * i + 1] = bf16hi(u[i]);
    }
  }
};
template <> struct Piece<DSA_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const PagedKv& kv, long long row, int at, int L) {
    const float4* p =
        reinterpret_cast<const float4*>(static_cast<const float*>(kv.pages) + row * L + at);
    a = __ldg(p);
    b = __ldg(p + 1);
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
template <> struct Piece<DSA_FP8_E4M3> {
  uint2 v;
  float s;
  __device__ __forceinline__ void load(const PagedKv& kv, long long row, int at, int L) {
    v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(kv.pages) + row * L + at));
    s = __ldg(kv.row_scale + row);
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    const uint32_t u[4] = {v.x & 0xffffu, v.x >> 16, v.y & 0xffffu, v.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u[i], __NV_E4M3);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * i] = x.x * s;
      f[2 * i + 1] = x.y * s;
    }
  }
};

template <typename T, int kKv>
__global__ void __launch_bounds__(kChunkThreads) mla_chunk_simt_kernel(ChunkArgs a) {
  extern __shared__ __align__(16) float rows[];  // [tile][pitch], then queries [kChunkHeads][L]
  __shared__ __align__(16) float sz[kChunkTile][kChunkHeads];
  __shared__ int srow[2][kChunkTile];
  __shared__ float s_m[kChunkHeads], s_l[kChunkHeads];
  __shared__ __align__(16) float s_alpha[kChunkHeads];
  const int L = a.L, Lp = chunk_pitch(a.L), kt = chunk_tile(a.L);
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
  // thread j: the cache row of the tile's position j (-1: no page); v may pass an int in
  // the last tile
  auto find_row = [&](unsigned v, int* dst) {
    if (tid >= kt || v + tid >= (unsigned)nv) return;
    const int i = (int)(v + tid), p = i < s0 ? i : lo + (i - s0);
    const int page = a.kv.block_table[(long long)b * a.kv.max_pages + p / a.kv.page_size];
    const bool ok = page >= 0 && page < a.kv.n_pages;
    if (!ok && reports) flag(a.status, DSA_DEV_BAD_PAGE);
    dst[tid] = ok ? page * a.kv.page_size + p % a.kv.page_size : -1;
  };
  find_row(0, srow[0]);
  float acc[kChunkHeads][kChunkCols];
#pragma unroll
  for (int h = 0; h < kChunkHeads; ++h)
#pragma unroll
    for (int c = 0; c < kChunkCols; ++c) acc[h][c] = 0.f;

  const int pieces = L / 8;
  int par = 0;
  for (unsigned v0 = 0; v0 < (unsigned)nv; v0 += kt, par ^= 1) {
    const int n = min(kt, nv - (int)v0), total = n * pieces;
    __syncthreads();
    for (int i0 = tid; i0 < total; i0 += 4 * kChunkThreads) {
      Piece<kKv> x[4];  // four loads on their way at once
      int row[4], j[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kChunkThreads;
        j[u] = i / pieces;
        row[u] = i < total ? srow[par][j[u]] : -1;
        if (row[u] >= 0) x[u].load(a.kv, row[u], (i - j[u] * pieces) * 8, L);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u * kChunkThreads;
        if (i >= total) break;
        float f[8];
        x[u].values(f);
        float4* dst = reinterpret_cast<float4*>(rows + j[u] * Lp + (i - j[u] * pieces) * 8);
        const bool some = row[u] >= 0;  // (a position without a page: zeros)
        dst[0] = some ? make_float4(f[0], f[1], f[2], f[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        dst[1] = some ? make_float4(f[4], f[5], f[6], f[7]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    find_row(v0 + kt, srow[par ^ 1]);  // the next tile's, under this one's work
    __syncthreads();
    for (int i = tid; i < n * kChunkHeads; i += kChunkThreads) {
      const int h = i / n, j = i - h * n;
      const float4* x = reinterpret_cast<const float4*>(rows + j * Lp);
      const float4* y = reinterpret_cast<const float4*>(sq + h * L);
      float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < L / 4; ++k) {
        const float4 xv = x[k], yv = y[k];
        d.x = fmaf(xv.x, yv.x, d.x);
        d.y = fmaf(xv.y, yv.y, d.y);
        d.z = fmaf(xv.z, yv.z, d.z);
        d.w = fmaf(xv.w, yv.w, d.w);
      }
      sz[j][h] = srow[par][j] >= 0 ? ((d.x + d.y) + (d.z + d.w)) * a.sm_scale : -INFINITY;
    }
    __syncthreads();
    if (warp < nh) {  // warp = head: four positions a lane
      float z[kChunkTile / 32], top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int u = 0; u < kChunkTile / 32; ++u) {
        z[u] = lane + 32 * u < n ? sz[lane + 32 * u][warp] : -INFINITY;
        top = fmaxf(top, z[u]);
      }
      const float m_old = s_m[warp], m = fmaxf(m_old, warp_max(top));
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int u = 0; u < kChunkTile / 32; ++u) {
        z[u] = expf(z[u] - ref);
        sum += z[u];
        sz[lane + 32 * u][warp] = z[u];
      }
      sum = warp_sum(sum);
      if (lane == 0) {
        const float alpha = expf(m_old - ref);  // 0 before the first visible position
        s_m[warp] = m;
        s_l[warp] = s_l[warp] * alpha + sum;
        s_alpha[warp] = alpha;
      }
    } else {  // no such head
#pragma unroll
      for (int u = 0; u < kChunkTile / 32; ++u) sz[lane + 32 * u][warp] = 0.f;
      if (lane == 0) s_alpha[warp] = 0.f;
    }
    __syncthreads();
    const float4 alpha = *reinterpret_cast<const float4*>(s_alpha);
#pragma unroll
    for (int c = 0; c < kChunkCols; ++c) {
      const int d = c * kChunkThreads + tid;
      if (d >= L) break;
      acc[0][c] *= alpha.x;
      acc[1][c] *= alpha.y;
      acc[2][c] *= alpha.z;
      acc[3][c] *= alpha.w;
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float x = rows[j * Lp + d];
        const float4 w = *reinterpret_cast<const float4*>(sz[j]);
        acc[0][c] = fmaf(w.x, x, acc[0][c]);
        acc[1][c] = fmaf(w.y, x, acc[1][c]);
        acc[2][c] = fmaf(w.z, x, acc[2][c]);
        acc[3][c] = fmaf(w.w, x, acc[3][c]);
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

template <typename T>
auto simt_kernel(int kv_dtype) {
  return kv_dtype == DSA_BF16  ? mla_chunk_simt_kernel<T, DSA_BF16>
         : kv_dtype == DSA_F32 ? mla_chunk_simt_kernel<T, DSA_F32>
                               : mla_chunk_simt_kernel<T, DSA_FP8_E4M3>;
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
// heads), a row must see enough of them to pay for the exchange's start and end (2,048),
// and every pair must have enough tiles of 64 keys to hide it (64).  The lengths live on
// the device: T, the window and the block table's width stand for them, so a step
// whose table is wider than its contexts, or whose T is larger than its tokens, may take
// pairs where one CTA a row tile were faster, by what the short cases below say.
// Measured on GB300, pair / single CTA in us (sequences x new tokens, 64 heads; tiles a
// pair), table and T as large as the step:
//   context  8,192, 32 x 4: 182 / 197, 16 x 16: 321 / 362, 4 x 256: 1,109 / 1,245
//   context  4,096, 4 x 8 (13): 51 / 37, 8 x 8 (27): 70 / 59, 1 x 128 (54): 105 / 103,
//            32 x 4 (54): 113 / 123, 1 x 256 (108): 175 / 179
//   context  2,048, 16 x 16: 118 / 105, 4 x 256: 341 / 339
//   context    512, 16 x 16:  66 /  45, 4 x 256: 149 / 113
//   one sequence, 4 on 65,536 (27): 63 / 60, 8 on 131,072 (108): 159 / 169
//   window   4,096 of 16,384, 4 x 256: 638 / 673; 2,048: 382 / 371; 512: 192 / 142
//   context  8,192, 32 x 2: 110 / 111, single tokens 64 x 1: 171 / 111
//   128 heads, context 8,192, 4 x 4 (27): 65 / 55, 16 x 4 (108): 180 / 208
bool pairs_pay(const ChunkArgs& a) {
  if (a.kv.kv_dtype != DSA_BF16 || (a.Hm <= 64 && a.T < 2ll * a.B)) return false;
  const long long table = (long long)a.kv.max_pages * a.kv.page_size;
  const long long bound = a.window > 0 ? (long long)a.window + a.sinks : table;
  const long long seen = bound < table ? bound : table;
  const long long row_tiles = a.Hm <= 64 ? (a.T + 1ll) / 2 : a.T;
  return seen > 2048 && row_tiles * ((seen + 63) / 64) >= 64 * (num_sms() / 2);
}

}  // namespace

int launch_mla_chunk(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  if (mla_chunk_umma_ok(a.L, a.dtype, a.kv.kv_dtype)) {
    // E4M3 codes as they are need TMA's boxes of 8 rows; other page sizes are widened
    // (pages of 64, 16 heads, 64 single tokens on 8,192 keys: 65 us, widened 141; 64
    // heads, 4 x 128 tokens on 4,096 keys: 352 and 516)
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
      ((size_t)chunk_tile(a.L) * chunk_pitch(a.L) + (size_t)kChunkHeads * a.L) * sizeof(float);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  auto kernel = a.dtype == DSA_BF16 ? simt_kernel<__nv_bfloat16>(a.kv.kv_dtype)
                                    : simt_kernel<float>(a.kv.kv_dtype);
  // (the largest size once a kernel: another thread's call may come between)
  static std::atomic<unsigned long long> done[2][3];
  if (!allow_smem(kernel, (kChunkFloats + kChunkHeads * 1024) * sizeof(float),
                  done[a.dtype == DSA_BF16][a.kv.kv_dtype]))
    return DSA_ERR_CUDA;
  return launch_kernel(&cfg, kernel, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
