// Block scores of a grouped-query layer (gqa_scores.cu) for chunks of many new tokens (bf16
// queries, head dim 64 or 128, groups of up to 32 heads): tcgen05 products of 128 columns and
// 128 blocks.
//
// A column is a (token, head) pair: 128 / G neighbouring tokens of a sequence (G up to a power
// of two) with the query heads of one KV head, a CTA's.  The CTA runs through the tiles of 128
// blocks twice:
//   first   S = Q K_mean^T, a thread a column and half of the blocks: the column's reference and
//           sum stay in its registers
//   second  S^T = K_mean Q^T, the same operands the other way round, a thread a block and half
//           of the columns: exp(z - reference) / sum is summed over a token's heads in registers,
//           and a warp writes 32 neighbouring blocks' scores
// so that neither pass exchanges anything between threads.  The second pass takes the tiles from
// the last to the first: the last two are still in shared memory.
//
// The products of step u + 1 run while step u's numbers are taken, and step u + 2's means are on
// their way; two CTAs an SM.  2,048 tokens of 64 query heads on 16,384 keys (256 blocks): 45 us
// (mma.sync products of 16 x 8, which read each mean again for every 16 columns: 86 us).  The
// bytes of the scores and the queries take 6 us, the exponentials (two for each column and block,
// 36 a clock and SM) 6 us: what is left is the instructions around them, by 16 warps an SM, and
// the start of each CTA.  Without the numbers it is 33 us, without the exponentials alone 43.
// Not faster: CTAs that stay and take one group of tokens after the other (52 us), a warp for the
// products alone (52), 16 warps a CTA (70).
#include "gqa.cuh"
#include "mla_chunk.cuh"
#include "umma.cuh"

namespace dsa {
namespace {

using namespace gqa;
using chunk::add2;
using chunk::fma2;
using chunk::wait_on;

constexpr int kThreads = 256, kCols = 128, kBlocks = 128;
// A sum of 32 weights, relative to a column's reference, above which that is raised (2^104 such
// sums still fit)
constexpr float kHigh = 16777216.f;

struct Ctl {
  uint64_t s_full[2], drain;
  int page[4][kBlocks];        // of step u in u & 3; -1: no candidate, -2: a bad page
  uint32_t none[8][4];         // candidates without a page, of step u in u & 7
  float2 part[2][kCols];       // reference and sum of a column, by halves of the tiles
  alignas(16) float ref[kCols];  // negated
  alignas(16) float inv[kCols];  // 1 / sum (0: not a column)
  int cand[kCols], mine[kCols];  // of a token: candidates, own block
  uint32_t tmem;
  int dead;
};
template <int kD>
struct Smem {
  static constexpr int kAtom = 128 * 128, kTile = kD / 64 * kAtom;  // 128 rows, SW128
  static constexpr size_t kMeans = kTile, kCtl = 3 * (size_t)kTile;
  static constexpr size_t kBytes = 1024 + kCtl + sizeof(Ctl);
};
static_assert(2 * (Smem<128>::kBytes + 1024) <= 228 * 1024, "two CTAs an SM");

// a += b c, two at a time
__device__ __forceinline__ void fma2v(float& a0, float& a1, float b0, float b1, float c0,
                                      float c1) {
  unsigned long long a, b, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(b), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// kPad: G up to a power of two
template <int kD, int kPad>
__global__ void __launch_bounds__(kThreads, 2)
    gqa_scores_chunk_kernel(const GqaScoreArgs a, const int drill) {
  using S = Smem<kD>;
  constexpr int kPieces = kD / 8, kPer = kCols / kPad, kTmem = 256;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl& c = *reinterpret_cast<Ctl*>(sb + S::kCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, G = a.Hq / a.Hkv;
  pdl_wait();
  if (blockIdx.x == 0 && h == 0)
    for (int b = tid; b < a.B; b += kThreads)
      if (a.cu_new[b] < 0 || a.cu_new[b + 1] < a.cu_new[b] || a.cu_new[b + 1] > a.T)
        flag(a.status, DSA_DEV_BAD_LENGTH);
  // slots from floor(cu / kPer) + b on are sequence b's
  auto first_slot = [&](int b) { return min(max(a.cu_new[b], 0), a.T) / kPer + b; };
  int b = 0;
  for (int hi = a.B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (first_slot(mid) <= (int)blockIdx.x) b = mid; else hi = mid;
  }
  const StepRows rows = rows_between(a.cu_new[b], a.cu_new[b + 1], a.T);
  const int c0 = rows.first, n_new = rows.n;
  const int j0 = ((int)blockIdx.x - first_slot(b)) * kPer;  // the CTA's first token
  if (j0 < 0 || j0 >= n_new) return;
  const int live = min(kPer, n_new - j0);
  const long long base = (long long)a.seq_lens[b] - n_new + j0, end = base + live;
  const unsigned limit = min(a.NB, a.max_pages), ps = a.page_size;
  auto whole_at = [&](long long pos) {  // (positions are below 2^31)
    return pos < 0 ? 0 : (int)min(limit, ((unsigned)pos + 1u) / ps);
  };
  const int most = whole_at(end - 1);  // candidates of the last token; of the first:
  const int least = whole_at(base);
  const int n = (most + kBlocks - 1) / kBlocks, steps = 2 * n;
  auto tile_of = [&](int u) { return u < n ? u : steps - 1 - u; };
  for (int i = tid; i < kPer; i += kThreads) {
    const long long pos = base + i;
    c.cand[i] = i < live ? whole_at(pos) : 0;
    c.mine[i] = i < live && pos >= 0 ? (int)((unsigned)pos / ps) : -1;
  }
  if (h == 0 && tid == 0) {
    if (base < 0) flag(a.status, DSA_DEV_BAD_LENGTH);
    if (end > 0 && (end - 1) / a.page_size >= a.NB) flag(a.status, DSA_DEV_POOL_RANGE);
    if (end > 0 && (end - 1) / a.page_size >= a.max_pages) flag(a.status, DSA_DEV_BAD_PAGE);
  }
  if (tid == 0) {
    mbar_init(&c.s_full[0], 1);
    mbar_init(&c.s_full[1], 1);
    mbar_init(&c.drain, 1);
    fence_mbar_init();
    c.dead = 0;
  }
  __syncwarp();
  if (warp == 0 && n > 0) {
    tmem_alloc<kTmem>(&c.tmem);
    tc_fence_before();
  }
  float* out = a.scores + ((long long)(c0 + j0) * a.Hkv + h) * a.NB;  // of the first token
  const long long next = (long long)a.Hkv * a.NB;

  // ---- what a step needs
  const int32_t* table = a.block_table + (long long)b * a.max_pages;
  auto page_at = [&](int u) {  // of this thread's block of the step's tile
    if (u >= steps || tid >= kBlocks) return -1;
    const int j = tile_of(u) * kBlocks + tid;
    if (j >= most) return -1;
    const int page = __ldg(table + j);
    return page >= 0 && page < a.n_pages ? page : -2;
  };
  auto keep = [&](int u, int page) {
    if (u >= steps || tid >= kBlocks) return;
    c.page[u & 3][tid] = page;
    const uint32_t bad = __ballot_sync(0xffffffffu, page == -2);
    if (lane == 0) c.none[u & 7][warp] = bad;
    if (page == -2) flag(a.status, DSA_DEV_BAD_PAGE);
  };
  auto load = [&](int u) {  // the means of a step's tile, where they are not there already
    if (u >= steps || u == n || u == n + 1) return;
    unsigned char* to = sb + S::kMeans + (tile_of(u) & 1) * S::kTile;
#pragma unroll
    for (int i = 0; i < kBlocks * kPieces / kThreads; ++i) {
      const int p = tid + i * kThreads, r = p / kPieces, k = p - r * kPieces;
      const int page = c.page[u & 3][r];
      cp_async16(smem_u32(to + (k >> 3) * S::kAtom + r * 128 + (((k & 7) ^ (r & 7)) << 4)),
                 a.k_mean + ((long long)max(page, 0) * a.Hkv + h) * kD + k * 8, page >= 0);
    }
  };
  constexpr uint32_t idesc = umma_idesc_bf16(128, 128, false);
  const uint64_t d_q = sw128_desc(smem_u32(sb)), d_k = sw128_desc(smem_u32(sb + S::kMeans));
  auto products = [&](int u, uint32_t tmem) {  // by warp 0
    if (u >= steps || drill) return;  // (a failure drill multiplies nothing)
    const uint64_t dk = d_k + (uint32_t)((tile_of(u) & 1) * (S::kTile >> 4));
#pragma unroll
    for (int s = 0; s < kD / 16; ++s) {
      const uint32_t at = ((s >> 2) * S::kAtom + (s & 3) * 32) >> 4;
      umma_bf16_elect(tmem + (u & 1) * 128, (u < n ? d_q : dk) + at, (u < n ? dk : d_q) + at,
                      idesc, s ? 1u : 0u);
    }
    umma_commit_elect(&c.s_full[u & 1]);
  };

  if (n > 0) {
#pragma unroll
    for (int i = 0; i < kCols * kPieces / kThreads; ++i) {
      const int p = tid + i * kThreads, r = p / kPieces, k = p - r * kPieces;
      const int token = r / kPad, head = r - token * kPad;
      const bool real = token < live && head < G;
      cp_async16(smem_u32(sb + (k >> 3) * S::kAtom + r * 128 + (((k & 7) ^ (r & 7)) << 4)),
                 static_cast<const __nv_bfloat16*>(a.q) +
                     ((long long)(c0 + j0 + (real ? token : 0)) * a.Hq + (long long)h * G +
                      (real ? head : 0)) * kD + k * 8,
                 real);
    }
    for (int u = 0; u < 3; ++u) keep(u, page_at(u));
    __syncthreads();
    // behind the barrier that follows the allocation: a dependent kernel's CTA on this SM might
    // take the tensor memory that this CTA still waits for, and itself wait for this grid
    pdl_launch_dependents();
    load(0);
    cp_async_commit();
    load(1);
    cp_async_commit();
    cp_async_wait<1>();
    fence_proxy_async_smem();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    if (warp == 0) products(0, tmem);

    const float unit = a.sm_scale * kLog2e;
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;  // TMEM lane; columns of S, S^T
    const uint32_t ts = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 64;
    const int token = row / kPad, cand = c.cand[token];
    const int near = max(c.mine[0] - max(a.local_blocks, 0) + 1, 0);  // the first near block
    const unsigned long long wait_ns = drill ? kDrillWaitNs : kWaitNs;
    float ref = -INFINITY, sum = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int u = 0; u < steps; ++u) {
      const int page = page_at(u + 3);
      ok = wait_on(&c.s_full[u & 1], (u >> 1) & 1, &c.dead, wait_ns);
      load(u + 2);  // (its place was step u's)
      cp_async_commit();
      keep(u + 3, page);
      cp_async_wait<1>();
      fence_proxy_async_smem();
      tc_fence_before();
      ok = __syncthreads_and(ok);
      if (!ok) break;
      tc_fence_after();
      if (warp == 0) products(u + 1, tmem);
      __syncwarp();
      const int j0 = tile_of(u) * kBlocks;
      const uint32_t* none = c.none[u & 7];
      if (u < n) {
        // ---- a column's reference and sum
#pragma unroll 1
        for (int k0 = 0; k0 < 64; k0 += 32) {
          const int block0 = j0 + half * 64 + k0;
          if (block0 >= most) break;
          float z[32], e[32];
          tmem_ld32(ts + (u & 1) * 128 + k0, z);
          const int seen = min(max(cand - block0, 0), 32);
          const uint32_t see = (seen < 32 ? (1u << seen) - 1u : ~0u) & ~none[half * 2 + k0 / 32];
          const bool all = __all_sync(0xffffffffu, see == ~0u);
          float part;
          auto weigh = [&]() {
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              e[k] = z[k];
              e[k + 1] = z[k + 1];
              fma2(e[k], e[k + 1], unit, -ref, -ref);
            }
            if (!all)
#pragma unroll
              for (int k = 0; k < 32; ++k) e[k] = (see >> k) & 1u ? e[k] : -INFINITY;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              add2(s[0], s[1], ex2_fast(e[k]), ex2_fast(e[k + 1]));
              add2(s[2], s[3], ex2_fast(e[k + 2]), ex2_fast(e[k + 3]));
            }
            part = (s[0] + s[1]) + (s[2] + s[3]);
          };
          weigh();
          // Without a reference every candidate's weight is infinite, or NaN where its logit is
          // minus infinity: that sets no reference and weighs nothing.
          if (!(part <= kHigh)) {
            float top = ref, nan = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if ((see >> k) & 1u) {
                const float x = z[k] * unit;
                top = fmaxf(top, x);
                nan = x != x ? x : nan;
              }
            if (top == -INFINITY) {
              part = nan;
            } else {
              sum *= ex2_fast(ref - top);
              ref = top;
              weigh();
            }
          }
          __syncwarp();
          sum += part;
        }
        if (u < n - 1) continue;
        c.part[half][row] = make_float2(ref, sum);
        __syncthreads();
        if (tid < kCols) {
          const float2 x = c.part[0][tid], y = c.part[1][tid];
          const float top = fmaxf(x.x, y.x), to = top == -INFINITY ? 0.f : top;
          const float l = x.y * (x.x == -INFINITY ? 1.f : ex2_fast(x.x - to)) +
                          y.y * (y.x == -INFINITY ? 1.f : ex2_fast(y.x - to));
          c.ref[tid] = -to;
          // (a column that is none adds nothing; without a candidate no weight is looked at)
          c.inv[tid] = tid / kPad < live && tid % kPad < G && l != 0.f ? 1.f / l : 0.f;
        }
        __syncthreads();
        continue;
      }
      // ---- the scores of a block, for half of the tokens
      const int j = j0 + row, warp0 = j0 + (warp & 3) * 32;
      if (warp0 >= a.NB) continue;
      const bool gone = (none[warp & 3] >> lane) & 1u;
      const bool plain = warp0 >= a.sink_blocks &&
                         warp0 + 32 <= min(min(least, near), a.NB) && none[warp & 3] == 0u;
#pragma unroll 1
      for (int k0 = 0; k0 < 64; k0 += 32) {
        const int col = half * 64 + k0;
        if (col / kPad >= live) break;
        float z[32], s[32 / kPad];
        tmem_ld32(ts + (u & 1) * 128 + k0, z);
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 r = *reinterpret_cast<const float4*>(c.ref + col + k);
          fma2(z[k], z[k + 1], unit, r.x, r.y);
          fma2(z[k + 2], z[k + 3], unit, r.z, r.w);
        }
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 v = *reinterpret_cast<const float4*>(c.inv + col + k);
          const float e[4] = {ex2_fast(z[k]), ex2_fast(z[k + 1]), ex2_fast(z[k + 2]),
                              ex2_fast(z[k + 3])};
          if constexpr (kPad == 1) {
            s[k] = e[0] * v.x;
            s[k + 1] = e[1] * v.y;
            s[k + 2] = e[2] * v.z;
            s[k + 3] = e[3] * v.w;
          } else if constexpr (kPad == 2) {
            s[k / 2] = fmaf(e[0], v.x, e[1] * v.y);
            s[k / 2 + 1] = fmaf(e[2], v.z, e[3] * v.w);
          } else {
            fma2v(s0, s1, e[0], e[1], v.x, v.y);
            fma2v(s0, s1, e[2], e[3], v.z, v.w);
            if ((k + 4) % kPad == 0) {
              s[k / kPad] = s0 + s1;
              s0 = s1 = 0.f;
            }
          }
        }
        constexpr int kTok = 32 / kPad;
        float* to = out + (col / kPad) * next + j;
        if (plain && col / kPad + kTok <= live) {
#pragma unroll
          for (int i = 0; i < kTok; ++i) to[i * next] = s[i];
        } else if (j < a.NB) {
#pragma unroll 1
          for (int i = 0; i < kTok; ++i) {
            const int tok = col / kPad + i;
            if (tok >= live) break;
            float x = s[0];
#pragma unroll
            for (int k = 1; k < kTok; ++k) x = k == i ? s[k] : x;
            to[i * next] =
                forced(a, c.mine[tok], j) ? INFINITY : j < c.cand[tok] && !gone ? x : -INFINITY;
          }
        }
      }
    }
    cp_async_wait<0>();
    if (!ok && warp == 0) {  // what was issued, before the CTA's memory is given back
      umma_commit_elect(&c.drain);
      mbar_wait_bounded(&c.drain, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && c.dead) flag(a.status, DSA_DEV_TIMEOUT);  // outputs unspecified
    if (warp == 0) {
      tc_fence_after();
      tmem_dealloc<kTmem>(tmem);
    }
  } else {
    __syncthreads();
  }
  // blocks that no token has as a candidate
  for (int j = n * kBlocks + tid; j < a.NB; j += kThreads)
    for (int i = 0; i < live; ++i)
      out[i * next + j] = forced(a, c.mine[i], j) ? INFINITY : -INFINITY;
}

template <int kD, int kPad>
int launch(const GqaScoreArgs& a, cudaStream_t stream) {
  auto kernel = gqa_scores_chunk_kernel<kD, kPad>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(kernel, Smem<kD>::kBytes, done)) return DSA_ERR_CUDA;
  Launch l(dim3((unsigned)(a.T / (kCols / kPad) + a.B), a.Hkv, 1), kThreads, Smem<kD>::kBytes,
           stream);
  return launch_kernel(&l.cfg, kernel, a, failure_drill()) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
template <int kD>
int launch_pad(const GqaScoreArgs& a, cudaStream_t stream) {
  const int G = a.Hq / a.Hkv;
  if (G == 1) return launch<kD, 1>(a, stream);
  if (G == 2) return launch<kD, 2>(a, stream);
  if (G <= 4) return launch<kD, 4>(a, stream);
  if (G <= 8) return launch<kD, 8>(a, stream);
  if (G <= 16) return launch<kD, 16>(a, stream);
  return launch<kD, 32>(a, stream);
}

}  // namespace

int launch_gqa_scores_chunk(const GqaScoreArgs& a, cudaStream_t stream) {
  return a.D == 128 ? launch_pad<128>(a, stream) : launch_pad<64>(a, stream);
}

}  // namespace dsa
