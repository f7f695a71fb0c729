// Block scores of a grouped-query layer: how much each new token's heads look at each
// complete block, by the blocks' mean keys.
//   z[g, j] = sm_scale <q_g, k_mean_j>;  s[j] = sum_g exp(z[g, j] - m_g) / l_g
// with m_g, l_g the maximum and the sum of exp(z - m) over the candidates j < n: two passes
// over the means, the first for m and l, the second for the sum over the group's heads.
//
// Two kernels: one on the tensor cores (bf16 queries, head dim 64 or 128, groups of up to 32
// heads), and a generic one (any geometry and type), a CTA a token and KV head, a warp a block.
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
__device__ __forceinline__ bool forced(const GqaScoreArgs& a, int mine, int j) {
  return j <= mine && (j < a.sink_blocks || (long long)j > (long long)mine - a.local_blocks);
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

// ---- tensor cores ------------------------------------------------------------------
// The means of 16 blocks are the rows of a product, 8 kN (token, head) pairs of one
// sequence and KV head its columns: z^T = K_mean Q^T, bf16 in, fp32 out.  Lane (g, t) of a warp
// loads 16-byte pieces t, t + 4, .. of the rows g and g + 8 straight from memory and uses
// them as they come; the queries' pieces, kept in registers, follow the same order.  A lane
// then has two columns' z of its rows: it keeps their maximum and sum alone, and only at
// the end of the first pass do lanes (and warps, and CTAs) exchange them.
// Here (decode) the warps of a cluster's CTAs share the blocks of one token, so that many SMs
// read one long context's means.  Bound by round trips to the table and the means.
constexpr int kPadG = 32;            // heads of a group, at most
struct GroupArgs {
  GqaScoreArgs a;
  int pad;                           // G up to a power of two
  int tokens;                        // of a warp (chunks)
};

// Sums over a token's `pad` columns, left in its first: a lane's two, its neighbours', n tiles.
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
  const int c0 = min(max(a.cu_new[b], 0), a.T), n_new = min(a.cu_new[b + 1], a.T) - c0;
  const int i0 = row - c0;
  if (i0 < 0 || i0 >= n_new) return;  // (all of a cluster's CTAs alike)
  constexpr int live = 1;
  const long long base = (long long)a.seq_lens[b] - n_new + i0;  // the first token's position
  auto whole_at = [&](long long pos) {
    return pos < 0 ? 0 : (int)min((long long)min(a.NB, a.max_pages), (pos + 1) / a.page_size);
  };
  const int most = whole_at(base + live - 1);  // candidates of the last token
  if (h == 0 && rank == 0 && tid == 0) {
    if (base < 0) flag(a.status, DSA_DEV_BAD_LENGTH);
    const long long last = (base + live - 1) / a.page_size;
    if (base + live > 0 && last >= a.NB) flag(a.status, DSA_DEV_POOL_RANGE);
    if (base + live > 0 && last >= a.max_pages) flag(a.status, DSA_DEV_BAD_PAGE);
  }

  // queries: lane (g, t) has column g of every n tile; candidates of columns 2 t, 2 t + 1
  uint32_t q[kN][kSteps][2];
  int cand[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int col = n * 8 + g, i = col / ga.pad, head = col - i * ga.pad;
    const bool real = i < live && head < G;
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((long long)(c0 + i0 + (real ? i : 0)) * a.Hq + (long long)h * G + (real ? head : 0)) * kD);
#pragma unroll
    for (int k = 0; k < kD / 32; ++k) {
      const uint4 x = real ? __ldg(src + 4 * k + t) : make_uint4(0u, 0u, 0u, 0u);
      q[n][2 * k][0] = x.x;
      q[n][2 * k][1] = x.y;
      q[n][2 * k + 1][0] = x.z;
      q[n][2 * k + 1][1] = x.w;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = n * 8 + 2 * t + j, ic = c / ga.pad;
      cand[n][j] = ic < live && c - ic * ga.pad < G ? whole_at(base + ic) : 0;
    }
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
      const int c = n * 8 + 2 * t + i, ic = c / ga.pad;
      // (a column that is none adds nothing; without a candidate no weight is looked at)
      l[n][i] = ic < live && c - ic * ga.pad < G ? 1.f / l[n][i] : 0.f;
      if (l[n][i] == INFINITY) l[n][i] = 0.f;
    }

  // ---- second pass: weights, summed over a token's heads
  const long long pos = base;
  const int mine = pos < 0 ? -1 : (int)(pos / a.page_size);
  float* out = a.scores + ((long long)(c0 + i0) * a.Hkv + h) * a.NB;
  auto write = [&](int v, int p0, int p1, float (&z)[kN][4]) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) z[n][i] = ex2_fast(z[n][i] - m[n][i & 1]) * l[n][i & 1];
    sum_heads<kN>(z, ga.pad);
    if (t != 0) return;  // the token's first column writes
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

// Prompt chunks: a CTA takes neighbouring tokens of a sequence and one KV head, each warp 32
// columns of them (32 / G tokens, G up to a power of two), and runs through the means in
// tiles of 64 blocks that all its warps read from shared memory.  The products, and the two
// passes, are those above.  Three tiles are in the ring: one in use, two on their way, whose
// pages were looked up a tile earlier.  A row's 16-byte piece c lies at c ^ (row & 7), so that
// ldmatrix reads eight rows' pieces without a bank conflict, and hands them over in the order
// that a product takes them (pieces read by the lanes themselves cost two moves a product).
constexpr int kBlocks = 64, kRing = 3;

// kPad: G up to a power of two where that is known (0: any)
template <int kD, int kN, int kPad>
__global__ void __launch_bounds__(kThreads, 2) gqa_scores_chunk_kernel(const GroupArgs ga) {
  constexpr int kSteps = kD / 16, kPieces = kD / 8;  // 16-byte pieces of a row
  constexpr int kCopies = kBlocks * kPieces / kThreads;       // of a thread and tile
  extern __shared__ __align__(16) unsigned char ring[];       // [kRing][kBlocks][kD] bf16
  __shared__ uint32_t s_none[kRing][2];                       // blocks of a tile without a page
  pdl_wait();
  pdl_launch_dependents();
  const GqaScoreArgs& a = ga.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, G = a.Hq / a.Hkv, cta = ga.tokens * kWarps;  // tokens of a CTA
  if (blockIdx.x == 0 && h == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  // slots from floor(cu / cta) + b on are sequence b's
  auto first_slot = [&](int b) { return min(max(a.cu_new[b], 0), a.T) / cta + b; };
  int b = 0;
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (first_slot(mid) <= (int)blockIdx.x) b = mid; else hi = mid;
  }
  const int c0 = min(max(a.cu_new[b], 0), a.T), n_new = min(a.cu_new[b + 1], a.T) - c0;
  const int j0 = ((int)blockIdx.x - first_slot(b)) * cta;  // the CTA's first token
  if (j0 < 0 || j0 >= n_new) return;
  const int i0 = j0 + warp * ga.tokens, live = max(0, min(ga.tokens, n_new - i0));
  const long long base = (long long)a.seq_lens[b] - n_new + i0;  // the first token's position
  auto whole_at = [&](long long pos) {
    return pos < 0 ? 0 : (int)min((long long)min(a.NB, a.max_pages), (pos + 1) / a.page_size);
  };
  const long long end = (long long)a.seq_lens[b] - n_new + min(j0 + cta, n_new);
  const int most = whole_at(end - 1);  // candidates of the CTA's last token
  if (h == 0 && tid == 0) {
    if (base < 0) flag(a.status, DSA_DEV_BAD_LENGTH);
    if (end > 0 && (end - 1) / a.page_size >= a.NB) flag(a.status, DSA_DEV_POOL_RANGE);
    if (end > 0 && (end - 1) / a.page_size >= a.max_pages) flag(a.status, DSA_DEV_BAD_PAGE);
  }
  // queries: lane (g, t) has column g of every n tile; candidates of columns 2 t, 2 t + 1
  uint32_t q[kN][kSteps][2];
  int cand[kN][2], mine[kN][2];
  float* out[kN][2];
  int least = 0x7fffffff;  // candidates that every column has
  int near = 0x7fffffff;   // the first block that some column's token takes as a near one
  const int pad = kPad ? kPad : ga.pad, log = 31 - __clz(pad);
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int col = n * 8 + g, i = col >> log, head = col & (pad - 1);
    const bool real = i < live && head < G;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(
        static_cast<const __nv_bfloat16*>(a.q) +
        ((long long)(c0 + (real ? i0 + i : j0)) * a.Hq + (long long)h * G + (real ? head : 0)) *
            kD);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      q[n][k][0] = real ? __ldg(src + 8 * k + t) : 0u;
      q[n][k][1] = real ? __ldg(src + 8 * k + 4 + t) : 0u;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = n * 8 + 2 * t + j, ic = c >> log;
      const long long pos = base + ic;
      cand[n][j] = ic < live ? whole_at(pos) : 0;
      mine[n][j] = ic < live && pos >= 0 ? (int)(pos / a.page_size) : -1;
      if (ic < live) {
        least = min(least, cand[n][j]);
        near = min(near, (int)max((long long)mine[n][j] - a.local_blocks + 1, 0ll));
      }
      // a token's first column writes its row
      out[n][j] = ic < live && (c & (pad - 1)) == 0
                      ? a.scores + ((long long)(c0 + i0 + ic) * a.Hkv + h) * a.NB + g
                      : nullptr;
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  near = __reduce_min_sync(0xffffffffu, near);
  const float unit = a.sm_scale * kLog2e;
  const int32_t* table = a.block_table + (long long)b * a.max_pages;
  const int tiles = (most + kBlocks - 1) / kBlocks, all = (a.NB + kBlocks - 1) / kBlocks;

  // ---- the ring: tile v of both passes (2 tiles in all) in slot v % kRing
  int page[kCopies];  // of the next tile to copy: this thread's rows
  auto look_up = [&](int v) {
    const int w = v < tiles ? v : v - tiles;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int j = w * kBlocks + (tid + i * kThreads) / kPieces;
      page[i] = -1;
      if (v < 2 * tiles && j < most) {
        const int pg = __ldg(table + j);
        page[i] = pg >= 0 && pg < a.n_pages ? pg : -2;
      }
    }
  };
  auto copy = [&](int v) {  // (always a group of copies, if an empty one)
    if (v < 2 * tiles) {
      const int s = v % kRing;
      if (tid < 2) s_none[s][tid] = 0u;  // (nobody reads this slot's now)
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int p = tid + i * kThreads, r = p / kPieces, c = p - r * kPieces;
        const __nv_bfloat16* src =
            a.k_mean + ((long long)max(page[i], 0) * a.Hkv + h) * kD + c * 8;
        unsigned char* dst = ring + (((size_t)s * kBlocks + r) * kPieces + (c ^ (r & 7))) * 16;
        cp_async16(smem_u32(dst), src, page[i] >= 0);
        if (page[i] == -2) {
          if (c == 0) atomicOr(&s_none[s][r >> 5], 1u << (r & 31));
          flag(a.status, DSA_DEV_BAD_PAGE);
        }
      }
    }
    cp_async_commit();
  };
  float ref[kN][2], l[kN][2];  // references (-inf: none yet) and sums of the columns
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    ref[n][0] = ref[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }
  // products of the blocks 16 i + g, + 8 of the tile in slot s with the queries
  auto products = [&](int s, int i, float (&z)[kN][4]) {
    // (lane: row `lane & 15` of the 16, the first or the second piece of a step)
    const uint32_t at =
        smem_u32(ring + ((size_t)s * kBlocks + 16 * i + (lane & 15)) * kPieces * 16);
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) z[n][k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      uint32_t x[4];
      ldmatrix_x4(x[0], x[1], x[2], x[3], at + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
      for (int n = 0; n < kN; ++n)
        mma_bf16_16816(z[n], x[0], x[1], x[2], x[3], q[n][k][0], q[n][k][1]);
    }
  };
  // exponents z unit - ref of the blocks from block0 on; -inf where there is no candidate
  auto exponents = [&](const float (&z)[kN][4], int block0, uint32_t none, float (&e)[kN][4]) {
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) e[n][k] = fmaf(z[n][k], unit, -ref[n][k & 1]);
    if (block0 + 16 > least || none) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int r = g + (k < 2 ? 0 : 8);
          if (block0 + r >= cand[n][k & 1] || ((none >> r) & 1u)) e[n][k] = -INFINITY;
        }
    }
  };
  look_up(0);
  copy(0);
  look_up(1);
  copy(1);
  look_up(2);
  // ---- first pass: maximum and sum of every column
#pragma unroll 1
  for (int v = 0; v < tiles; ++v) {
    cp_async_wait<1>();
    __syncthreads();  // tile v is there; the slot of tile v + 2 is read
    copy(v + 2);
    look_up(v + 3);
    const int s = v % kRing, rows = min(kBlocks, most - v * kBlocks);
    const uint32_t none[2] = {s_none[s][0], s_none[s][1]};
#pragma unroll 1
    for (int i = 0; i * 16 < rows; ++i) {
      const int block0 = v * kBlocks + 16 * i;
      const uint32_t no = (i < 2 ? none[0] : none[1]) >> (16 * (i & 1)) & 0xffffu;
      float z[kN][4], e[kN][4], top = -INFINITY;
      products(s, i, z);
      exponents(z, block0, no, e);
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, e[n][k]);
      if (top > 24.f) {  // (a sum of 2^24 times as much still fits)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            // (without a reference: every candidate's exponent is +inf)
            const float z0 = e[n][k] == -INFINITY ? -INFINITY : z[n][k] * unit;
            const float z1 = e[n][k + 2] == -INFINITY ? -INFINITY : z[n][k + 2] * unit;
            const float to = fmaxf(z0, z1);
            if (to > ref[n][k] + 24.f) {
              l[n][k] *= ex2_fast(ref[n][k] - to);
              ref[n][k] = to;
            }
          }
        exponents(z, block0, no, e);
      }
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) l[n][k] += ex2_fast(e[n][k]) + ex2_fast(e[n][k + 2]);
    }
  }
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float top = ref[n][k];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float to = top == -INFINITY ? 0.f : top;
      float sum = l[n][k] * (ref[n][k] == -INFINITY ? 1.f : ex2_fast(ref[n][k] - to));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      ref[n][k] = to;
      // (a column that is none adds nothing; without a candidate no weight is looked at)
      const int c = n * 8 + 2 * t + k;
      l[n][k] = (c >> log) < live && (c & (pad - 1)) < G && sum != 0.f ? 1.f / sum : 0.f;
    }
  // ---- second pass: weights, summed over a token's heads
#pragma unroll 1
  for (int v = 0; v < all; ++v) {
    const int u = tiles + v, s = u % kRing;
    if (v < tiles) {
      cp_async_wait<1>();
      __syncthreads();
      copy(u + 2);
      look_up(u + 3);
    }
    uint32_t none[2] = {0u, 0u};
    if (v < tiles) {
      none[0] = s_none[s][0];
      none[1] = s_none[s][1];
    }
    const int rows = min(kBlocks, a.NB - v * kBlocks);
#pragma unroll 1
    for (int i = 0; i * 16 < rows; ++i) {
      const int block0 = v * kBlocks + 16 * i;
      const uint32_t no = (i < 2 ? none[0] : none[1]) >> (16 * (i & 1)) & 0xffffu;
      float z[kN][4];
      if (block0 < most) {
        products(s, i, z);
        // (columns without a candidate here come to weights that nobody looks at)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            z[n][k] = ex2_fast(fmaf(z[n][k], unit, -ref[n][k & 1])) * l[n][k & 1];
        sum_heads<kN>(z, pad);
      }
      // every one a candidate, none forced, none past the rows' end
      const bool plain = block0 >= a.sink_blocks && block0 + 16 <= min(min(least, near), a.NB) &&
                         no == 0u;
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (kPad >= 2 && (k == 1 || (n * 8) % kPad != 0)) continue;
          float* dst = out[n][k];
          if (dst == nullptr) continue;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = block0 + g + 8 * r;
            float x = z[n][2 * r + k];
            if (!plain) {
              if (j >= a.NB) continue;
              const bool some = j < cand[n][k] && !((no >> (g + 8 * r)) & 1u);
              x = forced(a, mine[n][k], j) ? INFINITY : some ? x : -INFINITY;
            }
            dst[block0 + 8 * r] = x;
          }
        }
    }
  }
  cp_async_wait<0>();
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

template <int kD, int kN, int kPad>
int launch_chunk(const GroupArgs& ga, cudaStream_t stream) {
  constexpr size_t kSmem = (size_t)kRing * kBlocks * kD * 2;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(gqa_scores_chunk_kernel<kD, kN, kPad>, kSmem, done)) return DSA_ERR_CUDA;
  Launch l(dim3((unsigned)(ga.a.T / (ga.tokens * kWarps) + ga.a.B), ga.a.Hkv, 1), kThreads, kSmem,
           stream);
  return launch_kernel(&l.cfg, gqa_scores_chunk_kernel<kD, kN, kPad>, ga) == cudaSuccess ? DSA_OK
                                                                                   : DSA_ERR_CUDA;
}

template <int kD>
int launch_groups(const GqaScoreArgs& a, cudaStream_t stream) {
  GroupArgs ga{a, 1, 1};
  const int G = a.Hq / a.Hkv;
  while (ga.pad < G) ga.pad *= 2;
  const long long rows = (long long)a.T * a.Hkv;
  const int n_tiles = ga.pad <= 16 ? 2 : 4, tokens = 8 * n_tiles / ga.pad;
  // Tokens together or a CTA (or several) for each, tables of 48 / 470 blocks, in us: 256 rows
  // (tokens x KV heads) 9.6 / 34.8 and 7.2 / 10.3, 512 rows 9.7 / 34.8 and 12.8 / 18.4, 1,024 rows
  // 9.8 / 34.8 and 22.7 / 34.5, 4,096 rows 11.9 / 45.7 and 76 / 116.
  if (rows >= 7ll * num_sms() || (rows >= 3ll * num_sms() && a.NB <= 128)) {
    ga.tokens = tokens;
    if (ga.pad == 8) return launch_chunk<kD, 2, 8>(ga, stream);
    if (ga.pad == 16) return launch_chunk<kD, 2, 16>(ga, stream);
    return n_tiles == 2 ? launch_chunk<kD, 2, 0>(ga, stream) : launch_chunk<kD, 4, 32>(ga, stream);
  }
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
