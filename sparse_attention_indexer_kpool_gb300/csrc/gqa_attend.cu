// Attention of a step's new tokens over the paged 8-bit cache of a grouped-query layer:
// causal, with an optional sliding window and first tokens, or over listed blocks.
//
// This file: the dispatch, and the generic kernel for any geometry and type.  One CTA of
// four warps = one token, one KV head and up to four of its query heads; tiles of 32 visible
// rows are brought into shared memory as fp32, a warp takes a head's scores and softmax,
// a thread two output columns of every head.  Running maximum, sum and outputs are fp32.
// Bound by latency (a tile's loads, dot products and barriers in turn) and fp32 products: 117
// tokens of 8 KV heads of 80 on up to 160 keys 19 us, 22 tokens on lists of 85 blocks 21 us.
#include "gqa.cuh"

namespace dsa {
namespace {

using namespace gqa;

constexpr int kThreads = 128, kHeads = 4, kTile = 32;

template <typename T>
__global__ void __launch_bounds__(kThreads) gqa_attend_simt_kernel(GqaArgs a) {
  extern __shared__ __align__(16) float rows[];  // keys [kTile][D + 4], values, queries
  __shared__ float sz[kHeads][kTile], s_m[kHeads], s_l[kHeads], s_alpha[kHeads];
  __shared__ int srow[kTile], spage[kTile];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const GqaKv& kv = a.kv;
  const int D = kv.D, Dp = D + 4, ps = kv.page_size, G = a.Hq / kv.Hkv;
  const int hb = (G + kHeads - 1) / kHeads;
  const int t = blockIdx.x, h = blockIdx.y / hb, g0 = (blockIdx.y - h * hb) * kHeads;
  const int nh = min(kHeads, G - g0);
  const bool reports = blockIdx.y == 0;
  if (t == 0 && reports)
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  const int b = sequence_of(a.cu_new, a.B, t);
  const int c0 = max(a.cu_new[b], 0), c1 = min(a.cu_new[b + 1], a.T);
  if (t < c0 || t >= c1) return;  // behind the last sequence: left as it was
  const long long at = (long long)kv.seq_lens[b] - (c1 - c0) + (t - c0);
  if (at < 0 && reports && tid == 0) flag(a.status, DSA_DEV_BAD_LENGTH);
  const int pos = (int)max(at, -1ll), cap = table_cap(kv.max_pages, ps);
  if (!a.block_ids && pos >= cap && reports && tid == 0) flag(a.status, DSA_DEV_BAD_PAGE);
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int s0 = min(min(a.sinks, lo), cap);
  const int32_t* ids =
      a.block_ids ? a.block_ids + ((long long)t * kv.Hkv + h) * a.K : nullptr;
  // rows to look at: [0, s0) and [lo, pos], or the listed blocks' rows
  const int nv = pos < 0 ? 0 : (ids ? a.K * ps : s0 + max(min(pos, cap - 1) - lo + 1, 0));

  float* sk = rows;
  float* sv = rows + kTile * Dp;
  float* sq = sv + kTile * Dp;
  const long long head0 = (long long)t * a.Hq + (long long)h * G + g0;
  const T* q = static_cast<const T*>(a.q) + head0 * D;
  for (int i = tid; i < kHeads * D; i += kThreads)
    sq[i] = i < nh * D ? Act<T>::to_f(q[i]) : 0.f;
  if (tid < kHeads) {
    s_m[tid] = -INFINITY;
    s_l[tid] = 0.f;
  }
  float acc[kHeads][2];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) acc[i][0] = acc[i][1] = 0.f;
  const int per = D / 16;
  for (unsigned v0 = 0; v0 < (unsigned)nv; v0 += kTile) {
    __syncthreads();
    int page = -1;
    if (tid < kTile) {
      const unsigned v = v0 + tid;
      int p = 0;
      if (v < (unsigned)nv) {
        long long x;
        if (ids) {
          const int id = ids[v / ps];
          x = id < 0 ? -1 : (long long)id * ps + v % ps;
        } else {
          x = (int)v < s0 ? (int)v : lo + ((int)v - s0);
        }
        if (x >= 0 && x <= pos) {
          p = (int)x;
          page = p < cap ? kv.block_table[(long long)b * kv.max_pages + p / ps] : -1;
          if (page < 0 || page >= kv.n_pages) {
            flag(a.status, DSA_DEV_BAD_PAGE);
            page = -1;
          }
        }
      }
      spage[tid] = page;
      srow[tid] = p % ps;
    }
    if (!__syncthreads_or(page >= 0)) continue;  // (a list's -1 entries)
    for (int i = tid; i < kTile * per * 2; i += kThreads) {
      const bool key = i < kTile * per;
      const int j = key ? i : i - kTile * per, r = j / per, d = (j - r * per) * 16;
      const int page = spage[r];
      float* dst = (key ? sk : sv) + r * Dp + d;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      float s = 0.f;
      if (page >= 0) {
        const long long unit = (long long)page * kv.Hkv + h;
        x = __ldg(reinterpret_cast<const uint4*>((key ? kv.k_pages : kv.v_pages) +
                                                 (unit * ps + srow[r]) * D + d));
        s = __ldg((key ? kv.k_scale : kv.v_scale) + unit);
      }
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float2 m = codes2(w[u] & 0xffffu), n = codes2(w[u] >> 16);
        *reinterpret_cast<float4*>(dst + 4 * u) =
            make_float4(m.x * s, m.y * s, n.x * s, n.y * s);
      }
    }
    __syncthreads();
    {  // warp = head, lane = row
      float d = 0.f;
#pragma unroll 4
      for (int i = 0; i < D / 4; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(sk + lane * Dp + 4 * i);
        const float4 y = *reinterpret_cast<const float4*>(sq + warp * D + 4 * i);
        d = fmaf(x.x, y.x, d);
        d = fmaf(x.y, y.y, d);
        d = fmaf(x.z, y.z, d);
        d = fmaf(x.w, y.w, d);
      }
      const float z = spage[lane] >= 0 ? d * a.sm_scale : -INFINITY;
      const float m_old = s_m[warp], m = fmaxf(m_old, warp_max(z));
      const float ref = m == -INFINITY ? 0.f : m;
      const float w = expf(z - ref);
      sz[warp][lane] = w;
      const float sum = warp_sum(w);
      __syncwarp();
      if (lane == 0) {
        const float alpha = expf(m_old - ref);  // 0 before the first visible row
        s_m[warp] = m;
        s_l[warp] = s_l[warp] * alpha + sum;
        s_alpha[warp] = alpha;
      }
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = tid + c * kThreads;
      if (d >= D) break;
#pragma unroll
      for (int i = 0; i < kHeads; ++i) acc[i][c] *= s_alpha[i];
#pragma unroll 4
      for (int r = 0; r < kTile; ++r) {
        const float x = sv[r * Dp + d];
#pragma unroll
        for (int i = 0; i < kHeads; ++i) acc[i][c] = fmaf(sz[i][r], x, acc[i][c]);
      }
    }
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + head0 * D;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (i >= nh) break;
    const float l = s_l[i], inv = l == 0.f ? 0.f : 1.f / l;  // a NaN sum stays one
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int d = tid + c * kThreads;
      if (d < D) out[(long long)i * D + d] = Act<T>::from_f(acc[i][c] * inv);
    }
    if (a.lse && tid == 0) a.lse[head0 + i] = l == 0.f ? -INFINITY : s_m[i] + logf(l);
  }
}

}  // namespace

size_t gqa_attend_workspace_size(int, int Hq, int Hkv, int D, int dtype) {
  if (!gqa_split_ok(D, dtype)) return 0;
  const size_t one = gqa_split_workspace_size(Hq, Hkv, D), two = gqa_chunk_workspace_size(D);
  return one > two ? one : two;
}

int launch_gqa_attend(const GqaArgs& a, void* workspace, cudaStream_t stream) {
  if (gqa_split_ok(a.kv.D, a.dtype)) {
    // Rows of a sequence together (tcgen05, 128 a tile) or each token's by themselves, in us, by
    // new tokens of each sequence (8 KV heads of 8 query heads):
    //   4 sequences on 1,500 keys: 4 tokens 31.4 / 15.8, 8 tokens 32.4 / 35.0, 12 32.4 / 38.0
    //   16 on 8,000: 4 tokens 150 / 131, 8 153 / 235, 32 180 / 856
    //   16 on 64: 4 tokens 18.8 / 21.2, 8 18.9 / 24.9, 64 30.6 / 72.5
    //   16 on 8,000 with one query head a KV head, 2 of them: 4 tokens 53.5 / 39.8, 8 53.9 / 77
    // and a few short rows, however many a sequence has, by a cluster each (gqa_split.cu).  The
    // sequences of each of these have as many tokens as one another.  The host knows the average
    // alone: a prompt beside so many decode tokens that it is below eight goes the way of those,
    // and reads its keys anew for each token (16 x 32 tokens on 8,000: 856 us for 180).
    if (a.block_ids || a.T < 8ll * a.B) return launch_gqa_split(a, workspace, stream);
    const int rc = launch_gqa_split(a, workspace, stream, true);
    return rc == kElsewhere ? launch_gqa_chunk(a, workspace, stream) : rc;
  }
  const int G = a.Hq / a.kv.Hkv;
  auto kernel =
      a.dtype == DSA_BF16 ? gqa_attend_simt_kernel<__nv_bfloat16> : gqa_attend_simt_kernel<float>;
  static std::atomic<unsigned long long> done[2];
  constexpr size_t kMost = (size_t)(2 * kTile * (256 + 4) + kHeads * 256) * sizeof(float);
  if (!allow_smem(kernel, kMost, done[a.dtype == DSA_BF16])) return DSA_ERR_CUDA;
  Launch l(dim3(a.T, a.kv.Hkv * ((G + kHeads - 1) / kHeads), 1), kThreads,
           (size_t)(2 * kTile * (a.kv.D + 4) + kHeads * a.kv.D) * sizeof(float), stream);
  return launch_kernel(&l.cfg, kernel, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
