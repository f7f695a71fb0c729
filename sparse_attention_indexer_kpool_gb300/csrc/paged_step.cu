// The paged serving step around the attention: the step plan (block tables and
// slot maps from request lengths) and the append of new latent rows.
//
// ---- Step plan --------------------------------------------------------------
// For B requests with c_b cached and n_b new tokens (page size s):
//   cu_b   = min(sum_{a<b} n_a, T)                 (the token axis of the step)
//   have_b = ceil(c_b / s),  need_b = ceil((c_b + n_b) / s) - have_b
//   off_b  = sum_{a<b} need_a                      (of the free pages taken)
//   table[b, have_b + j] = free[begin + off_b + j]                j < need_b
//   token cu_b + i: position c_b + i, page table[b, position / s]
// Both sums are scans over B values.  Every CTA scans all B of them into its own
// shared memory (12 bytes a request) and then writes its share of the tokens, so
// one launch without any exchange between CTAs does the step; a token finds its
// request by a binary search over the shared sums, and its page from the free
// list itself, never from a table entry that another CTA is writing.
// What bounds it: the launch and two dependent round trips to memory (lengths,
// then free pages).  When seq_lens or free_end are written in place, the CTAs
// form one cluster (8 at most) and write only after a cluster barrier behind
// everyone's reads.  Measured on GB300: 64 decode requests 3.5 us, 512 requests with
// 64,536 new tokens in place 4.9 us.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>

#include "dsa_internal.cuh"

namespace dsa {
namespace {

constexpr int kClusterMax = 8;

// Exclusive scan of one value per thread (sums at most cap; saturating addition
// of non-negative values is associative); *total gets the whole sum.
__device__ __forceinline__ unsigned block_exclusive(unsigned v, unsigned cap, unsigned* warp_sums,
                                                    unsigned* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  unsigned inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc = min(inc + u, cap);
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    unsigned w = lane < nw ? warp_sums[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = min(w + u, cap);
    }
    warp_sums[lane] = w;  // 32 slots
  }
  __syncthreads();
  const unsigned before = warp ? warp_sums[warp - 1] : 0u;
  *total = warp_sums[nw - 1];
  unsigned ex = __shfl_up_sync(0xffffffffu, inc, 1);
  if (lane == 0) ex = 0u;
  __syncthreads();
  return min(before + ex, cap);
}

// Largest b in [0, n) with off[b] <= t (off[0] = 0 <= t).
__device__ __forceinline__ int find_segment(const int* off, int n, int t) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(int tokens, int page_size) {
  return tokens / page_size + (tokens % page_size != 0);
}

__global__ void __launch_bounds__(1024) paged_plan_kernel(PlanArgs a, int clustered) {
  extern __shared__ int32_t plan_sh[];
  int* cu = plan_sh;            // [B + 1]
  int* off = cu + a.B + 1;      // [B + 1] pages taken before request b
  int* ctx = off + a.B + 1;     // [B]
  __shared__ unsigned warp_sums[32];
  const int B = a.B, ps = a.page_size;
  const bool first = blockIdx.x == 0;
  pdl_wait();
  pdl_launch_dependents();
  const int per = (B + (int)blockDim.x - 1) / (int)blockDim.x;
  const int b0 = min(B, (int)threadIdx.x * per), b1 = min(B, b0 + per);
  const int begin = a.free_begin[0];

  // tokens: cu[b] holds the clean n_b until the scan has run
  unsigned mine = 0;
  const unsigned cap = (unsigned)a.T;
  for (int b = b0; b < b1; ++b) {
    int n = a.new_lens[b], c = a.ctx_lens[b];
    if (n < 0 || c < 0 || c > INT_MAX - n) {
      if (first) flag(a.status, DSA_DEV_BAD_LENGTH);
      n = 0;
      c = max(c, 0);
    }
    cu[b] = n;
    ctx[b] = c;
    mine = min(mine + min((unsigned)n, cap), cap);
  }
  unsigned total_tokens, total_pages;
  unsigned at = block_exclusive(mine, cap, warp_sums, &total_tokens);
  unsigned pages = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = cu[b];
    const unsigned next = min(at + min((unsigned)n, cap), cap);
    const int kept = (int)(next - at);
    if (kept < n && first) flag(a.status, DSA_DEV_TOKEN_CAP);
    cu[b] = (int)at;
    at = next;
    const int have = blocks_of(ctx[b], ps), after = blocks_of(ctx[b] + kept, ps);
    if (kept > 0 && after > a.max_pages && first) flag(a.status, DSA_DEV_NO_PAGE);
    off[b] = max(0, min(after, a.max_pages) - have);
    pages += (unsigned)off[b];
  }
  unsigned pat = block_exclusive(pages, 0x7fffffffu, warp_sums, &total_pages);
  for (int b = b0; b < b1; ++b) {
    const int need = off[b];
    off[b] = (int)pat;
    pat += (unsigned)need;
  }
  if (threadIdx.x == 0) {
    cu[B] = (int)total_tokens;
    off[B] = (int)total_pages;
  }
  __syncthreads();
  if (clustered) cooperative_groups::this_cluster().sync();  // every CTA has read its inputs

  const int avail = begin < 0 ? 0 : max(0, a.n_free - begin);
  if (first && threadIdx.x == 0) {
    if (begin < 0) flag(a.status, DSA_DEV_BAD_LENGTH);
    if ((int)total_pages > avail) flag(a.status, DSA_DEV_NO_PAGE);
    a.free_end[0] = begin + min((int)total_pages, avail);
  }
  auto free_page = [&](int k) {  // the k-th page that the step takes
    if (k >= avail) return -1;
    const int id = a.free_pages[begin + k];
    if (id >= 0 && id < a.n_pages) return id;
    flag(a.status, DSA_DEV_BAD_PAGE);
    return -1;
  };
  const int stride = gridDim.x * blockDim.x, tid0 = blockIdx.x * blockDim.x + threadIdx.x;
  for (int b = tid0; b <= B; b += stride) {
    a.cu_new[b] = cu[b];
    if (b < B) a.seq_lens[b] = ctx[b] + (cu[b + 1] - cu[b]);
  }
  for (int k = tid0; k < (int)total_pages; k += stride) {
    const int b = find_segment(off, B, k);
    const int blk = blocks_of(ctx[b], ps) + k - off[b];
    a.block_table[(long long)b * a.max_pages + blk] = free_page(k);
  }
  for (int t = tid0; t < a.T; t += stride) {
    if (t >= (int)total_tokens) {  // padding: sees nothing, is stored nowhere
      a.q_seq[t] = 0;
      a.q_pos[t] = -1;
      a.kv_rows[t] = -1;
      if (a.key_rows) a.key_rows[t] = -1;
      continue;
    }
    const int b = find_segment(cu, B, t);
    const int pos = ctx[b] + (t - cu[b]), blk = pos / ps, have = blocks_of(ctx[b], ps);
    int id = -1;
    if (blk < a.max_pages) {
      if (blk >= have) {
        id = free_page(off[b] + blk - have);
      } else {
        id = a.block_table[(long long)b * a.max_pages + blk];  // held before this step
        if (id < 0 || id >= a.n_pages) {
          flag(a.status, DSA_DEV_BAD_PAGE);
          id = -1;
        }
      }
    }
    a.q_seq[t] = b;
    a.q_pos[t] = pos;
    a.kv_rows[t] = id < 0 ? -1 : id * ps + (pos - blk * ps);
    if (a.key_rows) a.key_rows[t] = a.row_base[b] + pos;
  }
}

// ---- Append -----------------------------------------------------------------
// Row t of kv_new goes to cache row kv_rows[t].  E4M3 pages hold code = rn(x / s)
// with one fp32 scale per row, s = max|x| / 448 over the row's finite elements
// (1 where that is zero): the row's largest magnitude lands on the largest code,
// and both divisions are correctly rounded, so the stored row is a function of the
// row alone.  The elements' divisions share their divisor: q = x r with r = rn(1 / s),
// then q + (x - q s) r, the residual exact in an FMA (Markstein's correction, IBM J.
// Res. Dev. 34(1), 1990), which rounds x / s correctly where nothing underflows;
// rows with an extreme scale take the plain division.
// One warp per row, 8 elements (16 or 32 bytes) a lane and step; the row stays in
// registers between the maximum and the conversion, so it is read once.
// What bounds it: HBM bandwidth (a row is 2 L bytes in, L or 2 L out) and, for E4M3, the
// conversions.  Measured on GB300, L = 512: 65,536 bf16 rows to E4M3 18.4 us (101 MB: 5.5
// TB/s, 0.81 of the measured copy rate; two and four rows a warp were slower), 16,383 to
// bf16 4.7 us, 64 rows 1.1 us.
template <typename T> struct Load8;
template <> struct Load8<__nv_bfloat16> {
  static __device__ __forceinline__ void get(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = ld_stream_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf16lo(w[i]);
      x[2 * i + 1] = bf16hi(w[i]);
    }
  }
};
template <> struct Load8<float> {
  static __device__ __forceinline__ void get(const float* p, float (&x)[8]) {
    const uint4 u = ld_stream_v4(p), v = ld_stream_v4(p + 4);
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
};

constexpr int kAppendWarps = 8;

// kSteps: 8-element pieces per lane (L <= 256 kSteps)
template <typename T, int kKv, int kSteps>
__global__ void __launch_bounds__(kAppendWarps * 32)
    paged_append_kernel(const T* __restrict__ kv_new, const int32_t* __restrict__ kv_rows, int n_t,
                        int L, void* __restrict__ pages, float* __restrict__ row_scale,
                        int n_rows, int32_t* status) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= n_t) return;
  const int row = kv_rows[t];
  const T* src = kv_new + (long long)t * L;
  float x[kSteps][8];
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {  // (beside the row number, not behind it)
    const int d = (s * 32 + lane) * 8;
    if (d < L) {
      Load8<T>::get(src + d, x[s]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[s][i] = 0.f;
    }
  }
  if (row < 0) return;
  if (row >= n_rows) {
    if (lane == 0) flag(status, DSA_DEV_BAD_PAGE);
    return;
  }
  const long long dst = (long long)row * L;
  float scale = 1.f, r = 1.f;
  bool easy = true;
  if (kKv == DSA_FP8_E4M3) {
    float m = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[s][i]));  // (a NaN is passed over)
    m = warp_max(m);
    if (m == INFINITY) {  // an infinity does not set the scale either
      m = 0.f;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (fabsf(x[s][i]) < INFINITY) m = fmaxf(m, fabsf(x[s][i]));
      m = warp_max(m);
    }
    const float q = __fdiv_rn(m, 448.f);
    scale = q > 0.f ? q : 1.f;
    r = __frcp_rn(scale);
    easy = scale > 0x1p-80f && scale < 0x1p80f;
    if (lane == 0) row_scale[row] = scale;
  }
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int d = (s * 32 + lane) * 8;
    if (d >= L) continue;
    if (kKv == DSA_BF16) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pages) + dst + d) =
          make_uint4(pack_bf16(x[s][0], x[s][1]), pack_bf16(x[s][2], x[s][3]),
                     pack_bf16(x[s][4], x[s][5]), pack_bf16(x[s][6], x[s][7]));
    } else if (kKv == DSA_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(pages) + dst + d);
      o[0] = make_float4(x[s][0], x[s][1], x[s][2], x[s][3]);
      o[1] = make_float4(x[s][4], x[s][5], x[s][6], x[s][7]);
    } else {
      // a non-finite element stays visible as NaN (E4M3 has no infinity): the residual
      // of an infinity is one
      if (easy) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float q = x[s][i] * r;
          x[s][i] = fmaf(fmaf(-q, scale, x[s][i]), r, q);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          x[s][i] = fabsf(x[s][i]) < INFINITY ? __fdiv_rn(x[s][i], scale) : NAN;
      }
      uint32_t w[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[s][4 * h], x[s][4 * h + 1]),
                                                     __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(x[s][4 * h + 2], x[s][4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
        w[h] = lo | (hi << 16);
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + dst + d) = make_uint2(w[0], w[1]);
    }
  }
}

cudaLaunchConfig_t pdl_config(int grid, int block, size_t smem, cudaStream_t stream,
                              cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int kKv>
int append_steps(const void* kv_new, const int32_t* kv_rows, int n_t, int L, void* pages,
                 float* row_scale, int n_rows, int32_t* status, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = pdl_config((int)((n_t + kAppendWarps - 1ll) / kAppendWarps),
                                            kAppendWarps * 32, 0, stream, attr);
  auto kernel = L <= 256 ? paged_append_kernel<T, kKv, 1>
                         : (L <= 512 ? paged_append_kernel<T, kKv, 2>
                                     : paged_append_kernel<T, kKv, 4>);
  return launch_kernel(&cfg, kernel, static_cast<const T*>(kv_new), kv_rows, n_t, L, pages,
                       row_scale, n_rows, status) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <typename T>
int append_kv(const void* kv_new, const int32_t* kv_rows, int n_t, int L, int kv_dtype,
              void* pages, float* row_scale, int n_rows, int32_t* status, cudaStream_t stream) {
  if (kv_dtype == DSA_BF16)
    return append_steps<T, DSA_BF16>(kv_new, kv_rows, n_t, L, pages, row_scale, n_rows, status,
                                     stream);
  if (kv_dtype == DSA_F32)
    return append_steps<T, DSA_F32>(kv_new, kv_rows, n_t, L, pages, row_scale, n_rows, status,
                                    stream);
  return append_steps<T, DSA_FP8_E4M3>(kv_new, kv_rows, n_t, L, pages, row_scale, n_rows, status,
                                       stream);
}

}  // namespace

int launch_paged_plan(const PlanArgs& a, cudaStream_t stream) {
  const size_t smem = (size_t)(3 * a.B + 2) * 4;
  // (the largest size once: another thread's call may come between)
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(paged_plan_kernel, (3 * DSA_PLAN_MAX_B + 2) * 4, done)) return DSA_ERR_CUDA;
  // one thread a token up to the CTAs that the scans are repeated in
  const long long work = a.T > a.B ? a.T : a.B;
  const int block = work <= 256 ? 256 : 1024;
  const bool in_place = a.seq_lens == a.ctx_lens || a.free_end == a.free_begin;
  const long long want = (work + block - 1) / block;
  int grid = (int)(want < num_sms() ? want : num_sms());
  if (in_place && grid > kClusterMax) grid = kClusterMax;
  if (grid < 1) grid = 1;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = pdl_config(grid, block, smem, stream, attr);
  const int clustered = in_place && grid > 1;
  if (clustered) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = grid;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return launch_kernel(&cfg, paged_plan_kernel, a, clustered) == cudaSuccess ? DSA_OK
                                                                             : DSA_ERR_CUDA;
}

int launch_paged_append(const void* kv_new, const int32_t* kv_rows, int T, int L, int dtype,
                        int kv_dtype, void* pages, float* row_scale, int n_rows,
                        int32_t* status_dev, cudaStream_t stream) {
  return dtype == DSA_BF16
             ? append_kv<__nv_bfloat16>(kv_new, kv_rows, T, L, kv_dtype, pages, row_scale, n_rows,
                                        status_dev, stream)
             : append_kv<float>(kv_new, kv_rows, T, L, kv_dtype, pages, row_scale, n_rows,
                                status_dev, stream);
}

}  // namespace dsa
