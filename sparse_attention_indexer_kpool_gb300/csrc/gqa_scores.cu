// Block scores of a grouped-query layer: how much each new token's heads look at each
// complete block, by the blocks' mean keys.
//   z[g, j] = sm_scale <q_g, k_mean_j>;  s[j] = sum_g exp(z[g, j] - m_g) / l_g
// with m_g, l_g the maximum and the sum of exp(z - m) over the candidates j < n: two passes
// over the means, the first for m and l, the second for the sum over the group's heads.
//
// Generic kernel (any geometry and type): a CTA a token and KV head, a warp a block.
#include "gqa.cuh"

namespace dsa {
namespace {

using namespace gqa;

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxG = 128;

struct Row {        // of a token and KV head
  int b, mine;      // sequence, own block (-1: no position)
  int n;            // candidates
  bool live;
};
__device__ __forceinline__ Row row_of(const GqaScoreArgs& a, int t, bool reports) {
  Row r{0, -1, 0, false};
  r.b = sequence_of(a.cu_new, a.B, t);
  const int c0 = max(a.cu_new[r.b], 0), c1 = min(a.cu_new[r.b + 1], a.T);
  if (t < c0 || t >= c1) return r;
  r.live = true;
  const long long pos = (long long)a.seq_lens[r.b] - (c1 - c0) + (t - c0);
  if (pos < 0) {
    if (reports) flag(a.status, DSA_DEV_BAD_LENGTH);
    return r;
  }
  r.mine = (int)(pos / a.page_size);
  const int whole = (int)((pos + 1) / a.page_size);
  r.n = min(min(whole, a.NB), a.max_pages);
  if (reports && r.mine >= a.NB) flag(a.status, DSA_DEV_POOL_RANGE);
  if (reports && r.mine >= a.max_pages) flag(a.status, DSA_DEV_BAD_PAGE);
  return r;
}
__device__ __forceinline__ int page_of(const GqaScoreArgs& a, int b, int j) {
  const int page = a.block_table[(long long)b * a.max_pages + j];
  return page >= 0 && page < a.n_pages ? page : -1;
}
__device__ __forceinline__ bool forced(const GqaScoreArgs& a, int mine, int j) {
  return j <= mine && (j < a.sink_blocks || (long long)j > (long long)mine - a.local_blocks);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) gqa_scores_kernel(GqaScoreArgs a) {
  extern __shared__ float sq[];  // [G][D], then the warps' maxima and sums [kWarps][G] each
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int t = blockIdx.x, h = blockIdx.y, G = a.Hq / a.Hkv, D = a.D;
  if (t == 0 && h == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  const Row r = row_of(a, t, h == 0 && tid == 0);
  if (!r.live) return;
  float* sm = sq + G * D;
  float* sl = sm + kWarps * G;
  const T* q = static_cast<const T*>(a.q) + ((long long)t * a.Hq + (long long)h * G) * D;
  const float unit = a.sm_scale * kLog2e;
  for (int i = tid; i < G * D; i += kThreads) sq[i] = Act<T>::to_f(q[i]) * unit;
  for (int i = tid; i < kWarps * G; i += kThreads) {
    sm[i] = -INFINITY;
    sl[i] = 0.f;
  }
  __syncthreads();
  // z of block j and the warp's head g (base 2), in every lane
  float k[8];
  auto load = [&](int j) -> bool {
    const int page = page_of(a, r.b, j);
    if (page < 0) return false;
    const __nv_bfloat16* p = a.k_mean + ((long long)page * a.Hkv + h) * D;
#pragma unroll
    for (int i = 0; i < 8; ++i) k[i] = lane + 32 * i < D ? __bfloat162float(p[lane + 32 * i]) : 0.f;
    return true;
  };
  auto dot = [&](int g) -> float {
    float d = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < D) d = fmaf(k[i], sq[g * D + lane + 32 * i], d);
    return warp_sum(d);
  };
  bool missing = false;
  for (int j = warp; j < r.n; j += kWarps) {
    if (!load(j)) {
      missing = true;
      continue;
    }
    for (int g = 0; g < G; ++g) {
      const float z = dot(g);
      if (lane == 0) {
        float& m = sm[warp * G + g];
        float& l = sl[warp * G + g];
        const float top = fmaxf(m, z), ref = top == -INFINITY ? 0.f : top;
        l = l * exp2f(m - ref) + exp2f(z - ref);
        m = top;
      }
      __syncwarp();
    }
  }
  if (missing && lane == 0) flag(a.status, DSA_DEV_BAD_PAGE);
  __syncthreads();
  for (int g = tid; g < G; g += kThreads) {
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w * G + g]);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) sum += sl[w * G + g] * exp2f(sm[w * G + g] - ref);
    sm[g] = ref;
    sl[g] = 1.f / sum;
  }
  __syncthreads();
  float* out = a.scores + ((long long)t * a.Hkv + h) * a.NB;
  for (int j = warp; j < a.NB; j += kWarps) {
    float s = -INFINITY;
    if (forced(a, r.mine, j)) {
      s = INFINITY;
    } else if (j < r.n && load(j)) {
      s = 0.f;
      for (int g = 0; g < G; ++g) s = fmaf(exp2f(dot(g) - sm[g]), sl[g], s);
    }
    if (lane == 0) out[j] = s;
  }
}

}  // namespace

int launch_gqa_scores(const GqaScoreArgs& a, int dtype, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  auto kernel = dtype == DSA_BF16 ? gqa_scores_kernel<__nv_bfloat16> : gqa_scores_kernel<float>;
  static std::atomic<unsigned long long> done[2];
  constexpr size_t kMost = (size_t)(kMaxG * 256 + 2 * kWarps * kMaxG) * sizeof(float);
  if (!allow_smem(kernel, kMost, done[dtype == DSA_BF16])) return DSA_ERR_CUDA;
  Launch l(dim3(a.T, a.Hkv, 1), kThreads, (size_t)(G * a.D + 2 * kWarps * G) * sizeof(float),
           stream);
  return launch_kernel(&l.cfg, kernel, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
