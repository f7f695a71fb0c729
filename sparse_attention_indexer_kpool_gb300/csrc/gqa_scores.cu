// Block scores of a grouped-query layer: how much each new token's heads look at each
// complete block, by the blocks' mean keys.
//   z[g, j] = sm_scale <q_g, k_mean_j>;  s[j] = sum_g exp(z[g, j] - m_g) / l_g
// with m_g, l_g the maximum and the sum of exp(z - m) over the candidates j < n: two passes
// over the means, the first for m and l, the second for the sum over the group's heads.
//
// Here: a kernel on the tensor cores for few tokens (bf16 queries, head dim 64 or 128, groups of
// up to 32 heads), and a generic one (any geometry and type), a CTA a token and KV head, a warp a
// block (21 tokens on up to 230 keys, fp32, 9.7 us: latency).  That for chunks is
// gqa_scores_chunk.cu.
#include <cooperative_groups.h>

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

// ---- generic ---------------------------------------------------------------------
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
    sl[g] = sum == 0.f ? 0.f : 1.f / sum;  // (logits of minus infinity alone weigh nothing)
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

// ---- tensor cores ------------------------------------------------------------------
// The means of 16 blocks are the rows of a product, up to 8 kN query heads of a token and KV
// head its columns: z^T = K_mean Q^T, bf16 in, fp32 out.  Lane (g, t) of a warp
// loads 16-byte pieces t, t + 4, .. of the rows g and g + 8 straight from memory and uses
// them as they come; the queries' pieces, kept in registers, follow the same order.  A lane
// then has two columns' z of its rows: it keeps their maximum and sum alone, and only at
// the end of the first pass do lanes (and warps, and CTAs) exchange them.
// The warps of a cluster's CTAs share the blocks of one token, so that many SMs
// read one long context's means.  Bound by round trips to the table and the means: four tokens on
// 262,144 keys (8 KV heads of 8 query heads of 128) 9.5 us, 13.8 with cold caches, where the
// means' 34 MB take 5; with 16 query heads a KV head 10.7.
constexpr int kPadG = 32;            // heads of a group, at most
struct GroupArgs {
  GqaScoreArgs a;
  int pad;                           // G up to a power of two
};

// Sums over the token's `pad` columns, left in the first: a lane's two, its neighbours', n tiles.
template <int kN>
__device__ __forceinline__ void sum_heads(float (&z)[kN][4], int pad) {
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    if (pad >= 2) {
      z[n][0] += z[n][1];
      z[n][2] += z[n][3];
    }
    if (pad >= 4) {
      z[n][0] += __shfl_xor_sync(0xffffffffu, z[n][0], 1);
      z[n][2] += __shfl_xor_sync(0xffffffffu, z[n][2], 1);
    }
    if (pad >= 8) {
      z[n][0] += __shfl_xor_sync(0xffffffffu, z[n][0], 2);
      z[n][2] += __shfl_xor_sync(0xffffffffu, z[n][2], 2);
    }
  }
  if constexpr (kN >= 2)
    if (pad >= 16) {
#pragma unroll
      for (int n = 0; n < kN; n += 2) {
        z[n][0] += z[n + 1][0];
        z[n][2] += z[n + 1][2];
      }
    }
  if constexpr (kN >= 4)
    if (pad >= 32) {
      z[0][0] += z[2][0];
      z[0][2] += z[2][2];
    }
}

template <int kD, int kN>
__global__ void __launch_bounds__(kThreads)
    gqa_scores_mma_kernel(const GroupArgs ga) {
  constexpr int kSteps = kD / 16, kCols = 8 * kN;
  __shared__ float2 s_part[kWarps][kCols];
  __shared__ float2 s_cta[kCols];
  pdl_wait();
  pdl_launch_dependents();
  const GqaScoreArgs& a = ga.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, G = a.Hq / a.Hkv;
  namespace cg = cooperative_groups;
  const int splits = (int)cg::this_cluster().num_blocks();
  const int rank = (int)cg::this_cluster().block_rank();
  if (blockIdx.x == 0 && h == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  const int row = (int)blockIdx.x / splits;  // the token's row of the step
  const int b = sequence_of(a.cu_new, a.B, row);
  const StepRows rows = rows_between(a.cu_new[b], a.cu_new[b + 1], a.T);
  const int c0 = rows.first, n_new = rows.n;
  const int i0 = row - c0;
  if (i0 < 0 || i0 >= n_new) return;  // (all of a cluster's CTAs alike)
  const long long pos = (long long)a.seq_lens[b] - n_new + i0;
  const int most =  // candidates
      pos < 0 ? 0 : (int)min((long long)min(a.NB, a.max_pages), (pos + 1) / a.page_size);
  const int mine = pos < 0 ? -1 : (int)(pos / a.page_size);
  if (h == 0 && rank == 0 && tid == 0) {
    if (pos < 0) flag(a.status, DSA_DEV_BAD_LENGTH);
    if (mine >= a.NB) flag(a.status, DSA_DEV_POOL_RANGE);
    if (mine >= a.max_pages) flag(a.status, DSA_DEV_BAD_PAGE);
  }

  // queries: lane (g, t) has column g of every n tile; candidates of columns 2 t, 2 t + 1
  uint32_t q[kN][kSteps][2];
  int cand[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int head = n * 8 + g;
    const bool real = head < G;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((long long)row * a.Hq + (long long)h * G + (real ? head : 0)) * kD);
#pragma unroll
    for (int k = 0; k < kD / 32; ++k) {
      const uint4 x = real ? __ldg(src + 4 * k + t) : make_uint4(0u, 0u, 0u, 0u);
      q[n][2 * k][0] = x.x;
      q[n][2 * k][1] = x.y;
      q[n][2 * k + 1][0] = x.z;
      q[n][2 * k + 1][1] = x.w;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) cand[n][j] = n * 8 + 2 * t + j < G ? most : 0;
  }
  const float unit = a.sm_scale * kLog2e;
  const int32_t* table = a.block_table + (long long)b * a.max_pages;
  const int step = kWarps * splits, first = warp * splits + rank;
  const int tiles = (most + 15) / 16;
  // z (base 2) of the tile's blocks j0 + g and j0 + g + 8; -inf where there is no candidate
  auto page_at = [&](int j) -> int {
    if (j >= most) return -1;
    const int page = __ldg(table + j);
    return page >= 0 && page < a.n_pages ? page : -2;
  };
  auto scores_of = [&](int j0, int p0, int p1, float (&z)[kN][4]) {
    uint4 x[kD / 32], y[kD / 32];
    const uint4* k0 = reinterpret_cast<const uint4*>(
        a.k_mean + ((long long)max(p0, 0) * a.Hkv + h) * kD);
    const uint4* k1 = reinterpret_cast<const uint4*>(
        a.k_mean + ((long long)max(p1, 0) * a.Hkv + h) * kD);
#pragma unroll
    for (int k = 0; k < kD / 32; ++k) {
      x[k] = p0 >= 0 ? __ldg(k0 + 4 * k + t) : make_uint4(0u, 0u, 0u, 0u);
      y[k] = p1 >= 0 ? __ldg(k1 + 4 * k + t) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) z[n][i] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kD / 32; ++k)
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        mma_bf16_16816(z[n], x[k].x, y[k].x, x[k].y, y[k].y, q[n][2 * k][0], q[n][2 * k][1]);
        mma_bf16_16816(z[n], x[k].z, y[k].z, x[k].w, y[k].w, q[n][2 * k + 1][0],
                       q[n][2 * k + 1][1]);
      }
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        z[n][i] = (i < 2 ? p0 : p1) >= 0 && j0 + g + (i < 2 ? 0 : 8) < cand[n][i & 1]
                      ? z[n][i] * unit
                      : -INFINITY;
  };

  // ---- first pass: maximum and sum of every column
  float m[kN][2], l[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  auto add = [&](const float (&z)[kN][4]) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float top = fmaxf(z[n][i], z[n][i + 2]);
        if (top > m[n][i] + 24.f) {  // (a sum of 2^24 times as much still fits)
          l[n][i] *= ex2_fast(m[n][i] - top);
          m[n][i] = top;
        }
        const float ref = m[n][i] == -INFINITY ? 0.f : m[n][i];
        l[n][i] += ex2_fast(z[n][i] - ref) + ex2_fast(z[n][i + 2] - ref);
      }
  };
  // A warp's first tiles: their pages are looked up at once, and their z stay in registers (262,144
  // tokens, 4 x 8 rows: 15.5 us with the second pass reading them again).
  constexpr int kHeld = 8 / kN;
  float held[kHeld][kN][4];
  int pages[kHeld][2];
  bool missing = false;
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int j = (first + k * step) * 16 + g;
    pages[k][0] = page_at(j);
    pages[k][1] = page_at(j + 8);
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    if (first + k * step >= tiles) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) held[k][n][i] = -INFINITY;
      continue;
    }
    missing |= pages[k][0] == -2 || pages[k][1] == -2;
    scores_of((first + k * step) * 16, pages[k][0], pages[k][1], held[k]);
  }
#pragma unroll
  for (int k = 0; k < kHeld; ++k) add(held[k]);
  const int next = first + kHeld * step;
  int p0 = page_at(next * 16 + g), p1 = page_at(next * 16 + g + 8);
#pragma unroll 1
  for (int v = next; v < tiles; v += step) {
    const int n0 = page_at((v + step) * 16 + g), n1 = page_at((v + step) * 16 + g + 8);
    missing |= p0 == -2 || p1 == -2;
    float z[kN][4];
    scores_of(v * 16, p0, p1, z);
    add(z);
    p0 = n0;
    p1 = n1;
  }
  if (missing) flag(a.status, DSA_DEV_BAD_PAGE);
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = m[n][i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float ref = top == -INFINITY ? 0.f : top;
      float sum = l[n][i] * (m[n][i] == -INFINITY ? 1.f : ex2_fast(m[n][i] - ref));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      m[n][i] = ref;
      l[n][i] = sum;
      if (g == 0) s_part[warp][n * 8 + 2 * t + i] = make_float2(top, sum);
    }
  __syncthreads();
  if (tid < kCols) {
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_part[w][tid].x);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = s_part[w][tid];
      sum += x.y * (x.x == -INFINITY ? 1.f : ex2_fast(x.x - ref));
    }
    s_cta[tid] = make_float2(top, sum);
  }
  cg::this_cluster().sync();
  if (tid < kCols) {
    float top = -INFINITY, sum = 0.f;
    for (int r = 0; r < splits; ++r)
      top = fmaxf(top, cg::this_cluster().map_shared_rank(s_cta, r)[tid].x);
    const float ref = top == -INFINITY ? 0.f : top;
    for (int r = 0; r < splits; ++r) {
      const float2 x = cg::this_cluster().map_shared_rank(s_cta, r)[tid];
      sum += x.y * (x.x == -INFINITY ? 1.f : ex2_fast(x.x - ref));
    }
    s_part[0][tid] = make_float2(ref, sum);
  }
  cg::this_cluster().sync();  // (nobody leaves while its sums are read)
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 x = s_part[0][n * 8 + 2 * t + i];
      m[n][i] = x.x;
      l[n][i] = x.y;
    }
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (a column that is none adds nothing; without a candidate no weight is looked at)
      l[n][i] = n * 8 + 2 * t + i < G ? 1.f / l[n][i] : 0.f;
      if (l[n][i] == INFINITY) l[n][i] = 0.f;
    }

  // ---- second pass: weights, summed over the token's heads
  float* out = a.scores + ((long long)row * a.Hkv + h) * a.NB;
  auto write = [&](int v, int p0, int p1, float (&z)[kN][4]) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[n][i] = ex2_fast(z[n][i] - m[n][i & 1]) * l[n][i & 1];
    sum_heads<kN>(z, ga.pad);
    if (t != 0) return;  // the first column writes
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = v * 16 + g + 8 * r, page = r ? p1 : p0;
      if (j >= a.NB) continue;
      out[j] = forced(a, mine, j) ? INFINITY : page >= 0 && j < most ? z[0][2 * r] : -INFINITY;
    }
  };
  const int all = (a.NB + 15) / 16;
#pragma unroll
  for (int k = 0; k < kHeld; ++k)
    if (first + k * step < all) write(first + k * step, pages[k][0], pages[k][1], held[k]);
  p0 = page_at(next * 16 + g);
  p1 = page_at(next * 16 + g + 8);
#pragma unroll 1
  for (int v = next; v < all; v += step) {
    const int n0 = page_at((v + step) * 16 + g), n1 = page_at((v + step) * 16 + g + 8);
    float z[kN][4];
    if (v < tiles) {
      scores_of(v * 16, p0, p1, z);
    } else {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[n][i] = -INFINITY;
    }
    write(v, p0, p1, z);
    p0 = n0;
    p1 = n1;
  }
}

template <int kD, int kN>
int launch_decode(const GroupArgs& ga, int splits, cudaStream_t stream) {
  Launch l(dim3((unsigned)(ga.a.T * splits), ga.a.Hkv, 1), kThreads, 0, stream);
  cudaLaunchAttribute attr[2];
  attr[0] = l.attr;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  l.cfg.attrs = attr;
  l.cfg.numAttrs = 2;
  return launch_kernel(&l.cfg, gqa_scores_mma_kernel<kD, kN>, ga) == cudaSuccess ? DSA_OK
                                                                                 : DSA_ERR_CUDA;
}

template <int kD>
int launch_groups(const GqaScoreArgs& a, cudaStream_t stream) {
  GroupArgs ga{a, 1};
  const int G = a.Hq / a.Hkv;
  while (ga.pad < G) ga.pad *= 2;
  const long long rows = (long long)a.T * a.Hkv;
  // Tokens together (128 columns a CTA) or a CTA (or several) for each, tables of 48 / 470 blocks,
  // in us, 8 query heads a KV head: 256 rows (tokens x KV heads) 7.6 / 17.3 and 5.9 / 9.0, 512
  // rows 7.4 / 17.1 and 10.5 / 16.7, 1,024 rows 7.5 / 17.4 and 19.4 / 31.6, 4,096 rows 9.5 / 21.9
  // and 66 / 108; 512 rows of sequences with one token each 16.3 / 38.5 and 11.7 / 17.8, with two
  // (1,024 rows) 16.6 / 39.5 and 21.7 / 33.9.  With 16 query heads a KV head 256 rows 7.1 / 16.1
  // and 6.4 / 10.2, 512 rows 7.1 / 16.3 and 11.1 / 18.7.  (Equal lengths throughout; T is what the
  // step has room for, and its sequences may differ: the host knows neither.)
  if (rows >= 3ll * num_sms() && a.T >= 2ll * a.B) return launch_gqa_scores_chunk(a, stream);
  // otherwise CTAs for a token until there is one an SM, each with 64 blocks at least
  int splits = 1;
  while (splits < 8 && rows * splits < num_sms() && a.NB >= 128 * splits) splits *= 2;
  if ((long long)a.T * splits > 0x7fffffffll) splits = 1;
  if (ga.pad <= 8) return launch_decode<kD, 1>(ga, splits, stream);
  if (ga.pad <= 16) return launch_decode<kD, 2>(ga, splits, stream);
  return launch_decode<kD, 4>(ga, splits, stream);
}

}  // namespace

int launch_gqa_scores(const GqaScoreArgs& a, int dtype, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  if (dtype == DSA_BF16 && G <= kPadG && a.D == 128) return launch_groups<128>(a, stream);
  if (dtype == DSA_BF16 && G <= kPadG && a.D == 64) return launch_groups<64>(a, stream);
  auto kernel = dtype == DSA_BF16 ? gqa_scores_kernel<__nv_bfloat16> : gqa_scores_kernel<float>;
  static std::atomic<unsigned long long> done[2];
  constexpr size_t kMost = (size_t)(kMaxG * 256 + 2 * kWarps * kMaxG) * sizeof(float);
  if (!allow_smem(kernel, kMost, done[dtype == DSA_BF16])) return DSA_ERR_CUDA;
  Launch l(dim3(a.T, a.Hkv, 1), kThreads, (size_t)(G * a.D + 2 * kWarps * G) * sizeof(float),
           stream);
  return launch_kernel(&l.cfg, kernel, a) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
