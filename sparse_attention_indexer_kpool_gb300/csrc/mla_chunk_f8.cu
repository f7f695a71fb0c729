// The chunk attention over E4M3 pages on the 8-bit tensor-core products (bf16
// activations, latent 512, page size a multiple of 8): the codes go to the tensor
// cores as they are.
//
// Work, row tiles, key tiles, masks and the join are those of the bf16 kernel.  What
// differs is where the precision comes from: an E4M3 code keeps its value, and the
// other factor of each product is split into 8-bit parts whose sum it is.
//   S^T = C q_hi^T + 2^-4 C q_lo^T   E4M3 x E4M3.  A head's query row is scaled by a power
//     of two to a largest magnitude in [128, 256); hi is the nearest E4M3 value (off by
//     8 at most), lo that of 16 times the rest.  A bf16 value has 8 significant bits, an
//     E4M3 value 4, so the two are the value itself down to 2^-6 of the scaled row, and
//     off by at most 2^-14 below: 2^-21 of the row's largest element.  (Beside an element
//     2^12 times as large, a bf16 element's own rounding is as coarse.)
//   O^T += C^T (p_1 + p_2 + p_3)^T   E4M3 x E5M2.  A weight u = 2^(z - m) * row scale,
//     times 2^8, is cut to 3 significant bits twice and its rest rounded: off by at
//     most 2^-9 of itself (a bf16 weight: up to 2^-8), and, where a part falls below
//     E5M2's least normal value, by 2^-17 a part, 2^-23 of a weight at the reference in
//     all.  The sums keep the unrounded fp32 weights.
// The reference m of a head is kept for u rather than for the bare weight, so that u
// stays below 2^7 and its parts inside E5M2's range.  Row scales are taken relative to a power
// of two near those of the first key tile, the base, and count in the reference as at least
// 2^-80 of it, which bounds the bare weight as well.  A row whose codes are all zero adds to
// the sums alone: its scale, whatever it is, does not set the reference.
//
// Why.  Widening the codes to bf16 in shared memory took 1,960 cycles of conversions
// and 2,000 of shared-memory traffic a tile and kept one tile at a time in the 128 KB
// that its bf16 rows fill: 8,100 cycles a tile.  As codes a tile is 64 KB: two are in
// flight, the softmax of one under the products of the other.
//
// What bounds it.  64 heads: the products.  S^T is 16 MMAs of 128 x 128 x 32 (both query
// parts as N, 66 cycles each), O^T 48 of 128 x 64 x 32 (50 cycles, 6 KB of shared memory
// each), about 4,000 cycles a tile with the next tile's rows through the same port; 5,500
// by counters, row tiles' ends and raised references included: the rest is the hand-over
// between the two tiles in flight.  32 heads and fewer: S^T 16 of N = 64 and
// O^T 16 of N = 96 (the three weight parts beside one another), 1,700 cycles, so the
// chain load, S^T, softmax, O^T of a tile, two in flight: 4,000 cycles.  16 heads and fewer
// leave room for a third tile.
// Measured on GB300 in graphs of calls: 12 sequences of 1 to 300 new tokens on up to 5,000
// keys, 64 heads, 681 us (726 TFLOP/s counted once; of these, 15 us keep row scales of any size
// and zero rows right; one part of the queries after the other: 16 % more); 16 heads, 64
// single tokens on 4,096 to 16,000 keys in pages of 16, 77 us (334 MB: 4.3 TB/s, 0.64 of the
// measured copy rate; two tiles in flight: 10 % more, and 32 % with the parts one after the
// other).  A softmax thread has half of a tile's heads; a quarter each, on twice the warps,
// took 6 % longer on the former.
#include "mla_chunk.cuh"

namespace dsa {
namespace {

using namespace chunk;

constexpr int kKeys = 128;
constexpr int kBlock = kKeys * 128;       // 128 rows x 128 codes, 16 KB
constexpr int kStage = 4 * kBlock;        // a tile
constexpr int kTmaWarps = 2;
__host__ __device__ constexpr int cta_threads(int n) {
  return soft_threads(n) + 32 * (kTmaWarps + 1);
}
constexpr float kRaise8 = 7.f;            // base-2 growth of u that raises a reference
constexpr float kUp = 256.f;              // weights in E5M2 are scaled by 2^8
constexpr float kLeastLog = -80.f;
// The base lies 2^30 below the largest row scale of a segment's first key tile, so that up to
// 2^60 above that one and 2^110 below it weights and products stay in range; partials times
// 2^base do between these two.
constexpr int kBelow = 30, kBaseMin = -110, kBaseMax = 64;
constexpr float kLoUp = 16.f;             // of the queries' lo parts

template <int kStages>
struct Ctl {
  // per head; first: read as float4.  alpha: the square root of a rescale (of weights that may
  // lie above and below the reference by more than a float's range: taken twice)
  float m[64], nm[64], alpha[64], l[64], move[64];
  float sq[64];                           // the query rows' scales
  float red[4][64];
  uint64_t full[kStages][4], empty[kStages][4];  // by block of 128 codes
  uint64_t s_full[kStages], p_full, o_full, q_full, q_empty, drain;
  Start start;
  uint32_t tmem;
  unsigned groups[kStages];            // TMA boxes of the tile that hold rows
  int raise;
  int soft_dead[2];
  int dead;
};

template <int kN>
struct Smem {
  static constexpr int kStages = kN == 16 ? 3 : 2;      // tiles in flight: what fits
  static constexpr int kQBlock = kN * 128;              // kN heads x 128 codes
  // One MMA takes both parts of the queries as 2 kN rows, [block][part][head], and the
  // three parts of up to 32 heads' weights as 3 kN columns of P; each part has its own
  // columns of the result, which the softmax (and the end) adds.  (64 heads' outputs in
  // three parts do not fit TMEM: there the parts add up in the accumulator.)
  static constexpr int kOParts = kN == 64 ? 1 : 3, kON = kOParts * kN;
  static constexpr uint32_t kSCols = 2 * kN, kOCols = (kON + 31) / 32 * 32;  // stage, chunk
  // P: rows of a key's weights, 64 or 32 bytes each: a part of 64 or of 32 heads, or two
  // parts of 16 (the third has half a buffer)
  static constexpr int kPRow = kN == 64 ? 64 : 32, kPBufs = kN == 16 ? 2 : 3;
  static constexpr int kPPart = kKeys * kPRow;
  static constexpr size_t kKv = 0;
  static constexpr size_t kQ = (size_t)kStages * kStage;
  static constexpr size_t kP = kQ + 8 * (size_t)kQBlock;
  static constexpr size_t kCtl = kP + kPBufs * (size_t)kPPart;
  static constexpr size_t kBytes = 1024 + kCtl + sizeof(Ctl<kStages>);
};
static_assert(Smem<64>::kBytes <= 227 * 1024 && Smem<16>::kBytes <= 227 * 1024,
              "shared memory budget");

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, E4M3 A, E4M3 or E5M2 B.
constexpr uint32_t idesc_f8(int m, int n, bool a_mn, bool b_e5m2, bool b_mn) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void umma_f8_elect(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Shared-memory matrix descriptor, 32-byte swizzle: an atom is 8 rows of 32 bytes; the
// 16-byte chunk c of row r is stored at chunk position c ^ ((r >> 2) & 1).
__device__ __forceinline__ uint64_t umma_desc_sw32(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)((lbo >> 4) & 0x3FFF) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFF) << 32) | ((uint64_t)1 << 46) | ((uint64_t)6 << 61);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e5m2x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// 2^x of a whole number
__device__ __forceinline__ float pow2(int x) {
  return __uint_as_float((uint32_t)(127 + x) << 23);
}
// the leading 3 significant bits (of a NaN: one)
__device__ __forceinline__ float cut3(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffe00000u);
}

// The query rows in two E4M3 parts, for the kernel below: row r's 512 hi codes, then
// its 512 lo codes, and its scale.  A warp a row, 16 elements a lane.  Bound by its
// 1 KB in and 1 KB out a row; inside the attention the same work held every row
// tile's first product back (20,000 cycles of one warp's latency a tile).
__global__ void __launch_bounds__(256)
    mla_chunk_query_kernel(const __nv_bfloat16* __restrict__ q_lat, long long rows,
                           uint8_t* __restrict__ codes, float* __restrict__ scale) {
  pdl_wait();
  pdl_launch_dependents();
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  const __nv_bfloat16* src = q_lat + row * kL + lane * 16;
  const uint4 r0 = ld_stream_v4(src), r1 = ld_stream_v4(src + 8);
  const uint32_t u[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
  float x[16], top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = bf16lo(u[i]);
    x[2 * i + 1] = bf16hi(u[i]);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (fabsf(x[i]) < INFINITY) top = fmaxf(top, fabsf(x[i]));
  top = warp_max(top);
  // exponent of the largest magnitude: 2^ex <= top < 2^(ex + 1) (below the normal numbers:
  // theirs, at which the elements are still multiples of 1); 2^(7 - ex) in two factors
  const int ex = max((int)(__float_as_uint(top) >> 23) - 127, -126), half = (7 - ex) >> 1;
  const float up0 = pow2(half), up1 = pow2(7 - ex - half);
  const float down = pow2(-half) * pow2(half + ex - 7);  // 2^(ex - 7)
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    hi[j] = lo[j] = 0u;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      // a NaN or an infinity becomes the NaN code: its head's logits are NaN
      float a = x[4 * j + 2 * k] * up0 * up1, b = x[4 * j + 2 * k + 1] * up0 * up1;
      a = fabsf(a) < INFINITY ? a : NAN;
      b = fabsf(b) < INFINITY ? b : NAN;
      const uint32_t h2 = e4m3x2(a, b) & 0xffffu;
      const float2 f = from_e4m3x2(h2);
      hi[j] |= h2 << (16 * k);
      lo[j] |= (e4m3x2((a - f.x) * kLoUp, (b - f.y) * kLoUp) & 0xffffu) << (16 * k);
    }
  }
  uint8_t* dst = codes + row * (2 * kL) + lane * 16;
  *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(dst + kL) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  if (lane == 0) scale[row] = down;
}

template <int kN>
__global__ void __launch_bounds__(cta_threads(kN), 1)
    mla_chunk_f8_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap kv_map,
                        const __grid_constant__ CUtensorMap ahead_map,
                        const float* __restrict__ q_scale, const Params p) {
  using S = Smem<kN>;
  constexpr int kStages = S::kStages, kSoft = soft_threads(kN);
  auto stage_of = [](int tile) { return (int)((unsigned)tile % (unsigned)kStages); };
  auto phase_of = [](int tile) { return (unsigned)tile / (unsigned)kStages & 1u; };
  constexpr int kW = heads_of(kN), kGroups = kN / kW;  // heads of a softmax thread
  constexpr int kTma0 = kSoft / 32, kMmaWarp = kTma0 + kTmaWarps;
  constexpr uint32_t kOCol = kStages * S::kSCols;
  constexpr int kTmemCols = 512;
  static_assert(kOCol + 4 * S::kOCols <= kTmemCols, "TMEM columns");
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto& c = *reinterpret_cast<Ctl<S::kStages>*>(sb + S::kCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hb = (p.Hm + kN - 1) / kN;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      for (int blk = 0; blk < 4; ++blk) {
        mbar_init(&c.full[i][blk], 1);
        mbar_init(&c.empty[i][blk], 1);
      }
      mbar_init(&c.s_full[i], 1);
    }
    mbar_init(&c.p_full, kSoft / 32);
    mbar_init(&c.o_full, 1);
    mbar_init(&c.q_full, 1);
    mbar_init(&c.q_empty, 1);
    mbar_init(&c.drain, 1);
    fence_mbar_init();
    c.soft_dead[0] = c.soft_dead[1] = c.dead = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc<kTmemCols>(&c.tmem);
    tc_fence_before();
  }
  if (tid < 64) {
    c.m[tid] = -INFINITY;
    c.nm[tid] = 0.f;
  }
  pdl_wait();  // every input may come from the kernel just before
  pdl_launch_dependents();

  const unsigned long long units = find_share<kKeys, false, cta_threads(kN)>(
      p, hb, blockIdx.x, gridDim.x, &c.start, blockIdx.x == 0);
  const uint32_t tmem = c.tmem;
  Walk<kKeys, false> w(p, hb, c.start, units);
  // a failure drill loads nothing and issues no MMA: the first waits run out
  const bool issue = p.drill == 0;
  const unsigned long long wait_ns = p.drill ? kDrillWaitNs : kWaitNs;
  volatile int* dead = &c.dead;

  if (warp < kTma0) {
    // ================= softmax and epilogue =================
    const int qw = warp & 3;      // TMEM lanes 32 qw ..: this thread's key row r
    const int hq = warp >> 2;     // heads kW hq ..
    const int r = qw * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16);
    Header hd = {-1, -1, 0, 0};
    int tiles = 0, segs = 0;
    bool ok = true;
    // this thread's row scale in a tile (0: not seen or no page)
    auto scale_of = [&](const Keys<kKeys>& k, int b, int v) -> float {
      const int t = k.at(v, r);
      if (!k.sees(t)) return 0.f;
      const int blk = t / p.kv.page_size;
      if (blk >= p.kv.max_pages) return 0.f;
      const int page = __ldg(p.kv.block_table + (long long)b * p.kv.max_pages + blk);
      if (page < 0 || page >= p.kv.n_pages) return 0.f;
      return __ldg(p.kv.row_scale + (long long)page * p.kv.page_size + t % p.kv.page_size);
    };
    // Whether this thread's row has no code but zeros: looked for only where its scores
    // are (e: minus the references) zero or, by the queries, NaN.
    auto adds_nothing = [&](const float (&e)[kW], float sc, int st, int tile) -> bool {
      bool zero = fabsf(sc) < INFINITY;
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const float nm = c.nm[hq * kW + i];
        zero = zero && !(e[i] < nm || e[i] > nm);
      }
#pragma unroll 1
      for (int i = 0; zero && i < 32; ++i) {
        if ((i & 7) == 0 && !mbar_test(&c.full[st][i >> 3], phase_of(tile))) return false;
        const uint4 x = *reinterpret_cast<const uint4*>(
            sb + S::kKv + st * kStage + (i >> 3) * kBlock + r * 128 + (((i & 7) ^ (r & 7)) << 4));
        zero = ((x.x | x.y | x.z | x.w) & 0x7f7f7f7fu) == 0u;
      }
      return zero;
    };
    while (ok && w.next()) {
      float l[kW];                // this row's sums
      bool unset = true;          // some head here has no reference yet
#pragma unroll
      for (int i = 0; i < kW; ++i) l[i] = 0.f;
      float rs = w.ta < w.tb ? scale_of(w.k, w.b, w.ta) : 0.f;
      const float4* sq4 = reinterpret_cast<const float4*>(c.sq + hq * kW);
      const int heads = min(kN, p.Hm - w.h0 * kN);
      const long long row0 = (long long)w.token * p.Hm + w.h0 * kN;
      if (tid < kN) c.sq[tid] = tid < heads ? __ldg(q_scale + row0 + tid) : 0.f;
      {  // (c.red: the last segment's sums are read)
        const float lg = warp_max(fabsf(rs) < INFINITY ? log2f(fabsf(rs)) : -INFINITY);
        if (hq == 0 && lane == 0) c.red[0][qw] = lg;
      }
      sync_soft<kSoft>();
      // the segment's row scales are taken relative to 2^base (as floats: converted in every
      // tile they cost 15 us of the mixed step)
      const float top_lg =
          fmaxf(fmaxf(c.red[0][0], c.red[0][1]), fmaxf(c.red[0][2], c.red[0][3]));
      const int lowest = (top_lg > -INFINITY ? (int)floorf(top_lg) : 0) - kBelow;
      const int exponent = min(max(lowest, kBaseMin), kBaseMax);
      const float base = (float)exponent, unit = kUp * pow2(-exponent);
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        const int st = stage_of(tiles), dead_at = tiles & 1;
        const float rs_next = v + 1 < w.tb ? scale_of(w.k, w.b, v + 1) : 0.f;
        const int t = w.k.at(v, r);
        if (!wait_on(&c.s_full[st], phase_of(tiles), dead, wait_ns))
          c.soft_dead[dead_at] = 1;
        __syncwarp();
        tc_fence_after();
        const bool valid = w.k.sees(t) && ((c.groups[st] >> (r >> w.k.log)) & 1u);
        if (!valid) {  // the part of this row that this thread clears
#pragma unroll 1
          for (int blk = 4 / kGroups * hq; blk < 4 / kGroups * (hq + 1); ++blk)
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)  // (neighbouring rows in different banks)
              *reinterpret_cast<uint4*>(sb + S::kKv + st * kStage + blk * kBlock + r * 128 +
                                        ((ch ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        // (a hidden key's scale may be anything)
        const float sc = valid ? rs : 0.f, zs = p.zscale * sc;
        float lg = fmaxf(log2f(fabsf(sc)) - base, kLeastLog);  // in u's reference
        float up = sc * unit;
        const float high_at = kRaise8 - lg;
        float e[kW];
        // z = S * query scale * row scale * softmax scale, S of both parts
        {
          const uint32_t ts = tl + st * S::kSCols + (uint32_t)(hq * kW);
          tmem_ldw<kW>(ts, e);
#pragma unroll
          for (int g = 0; g < kW; g += 16) {
            float lo[16];
            tmem_ld16(ts + kN + g, lo);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              fma2(lo[i], lo[i + 1], 1.f / kLoUp, e[g + i], e[g + i + 1]);
              e[g + i] = lo[i];
              e[g + i + 1] = lo[i + 1];
            }
          }
#pragma unroll
          for (int q = 0; q < kW / 4; ++q) {
            const float4 s4 = sq4[q];
            e[4 * q] *= s4.x;
            e[4 * q + 1] *= s4.y;
            e[4 * q + 2] *= s4.z;
            e[4 * q + 3] *= s4.w;
          }
        }
        bool high = unset;
#pragma unroll
        for (int q = 0; q < kW / 4; ++q) {  // minus the references (0: none yet)
          const float4 nm = reinterpret_cast<const float4*>(c.nm + hq * kW)[q];
          fma2(e[4 * q], e[4 * q + 1], zs, nm.x, nm.y);
          fma2(e[4 * q + 2], e[4 * q + 3], zs, nm.z, nm.w);
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) {
          e[i] = valid ? e[i] : -INFINITY;
          high |= e[i] > high_at;
        }
        // every thread takes the same branch; the flag of a failed wait was
        // written before this barrier
        const bool full = vote_soft<kSoft>(high);
        if (c.soft_dead[dead_at]) {
          ok = false;
          break;
        }
        if (full) {
          const bool nothing = high && adds_nothing(e, sc, st, tiles);
          __syncwarp();
          if (nothing) {
            lg = kLeastLog;
            up = 0.f;
          }
          float top[kW];  // of u, relative to the references so far
#pragma unroll
          for (int i = 0; i < kW; ++i) top[i] = e[i] + lg;
          const float m = across_rows<kW, true>(top, lane);
          if (lane < kW) c.red[qw][hq * kW + lane] = m;
          if (tid == 0) c.raise = 0;
          sync_soft<kSoft>();
          if (tid < kN) {
            const float rel = fmaxf(fmaxf(c.red[0][tid], c.red[1][tid]),
                                    fmaxf(c.red[2][tid], c.red[3][tid]));
            const float m_old = c.m[tid];
            float a = 1.f, move = 0.f;
            if (m_old == -INFINITY) {  // nothing accumulated for this head yet
              c.m[tid] = rel;
              if (rel != -INFINITY) move = -rel;
            } else if (rel > kRaise8) {
              c.m[tid] = m_old + rel;
              a = ex2_fast(-0.5f * rel);
              move = -rel;
              c.raise = 1;
            }
            c.alpha[tid] = a;
            c.move[tid] = move;
            c.nm[tid] = c.m[tid] == -INFINITY ? 0.f : -c.m[tid];
          }
          sync_soft<kSoft>();
          unset = false;
#pragma unroll
          for (int i = 0; i < kW; ++i) unset |= c.m[hq * kW + i] == -INFINITY;
          // (an infinite maximum: its key's weight is NaN, as in the formula)
#pragma unroll
          for (int i = 0; i < kW; ++i) e[i] += c.move[hq * kW + i];
        }
        if (full && c.raise) {
#pragma unroll
          for (int i = 0; i < kW; ++i) l[i] = l[i] * c.alpha[hq * kW + i] * c.alpha[hq * kW + i];
        }
        // the weights and their parts (in registers: the last tile's may still be read)
        uint32_t part[3][kW / 4];
#pragma unroll
        for (int j = 0; j < kW / 4; ++j) {
          float a[4], x[3][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float& ei = e[4 * j + i];
            ei = ex2_fast(ei);
            a[i] = ei * up;
            x[0][i] = cut3(a[i]);
            a[i] -= x[0][i];
            x[1][i] = cut3(a[i]);
            x[2][i] = a[i] - x[1][i];
          }
#pragma unroll
          for (int k = 0; k < 3; ++k)
            part[k][j] = e5m2x2(x[k][0], x[k][1]) | (e5m2x2(x[k][2], x[k][3]) << 16);
          add2(l[4 * j], l[4 * j + 1], e[4 * j], e[4 * j + 1]);
          add2(l[4 * j + 2], l[4 * j + 3], e[4 * j + 2], e[4 * j + 3]);
        }
        // P's place and O^T: the last tile's product is done with both
        if (tiles > 0 && !wait_on(&c.empty[stage_of(tiles - 1)][3],
                                  phase_of(tiles - 1), dead, wait_ns))
          c.soft_dead[dead_at ^ 1] = 1;
        __syncwarp();
        if (full && c.raise && v > w.ta) {
          tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < 4 * S::kOParts; ++i) {
            float o[kW];
            const uint32_t ta = tl + kOCol + (i / S::kOParts) * S::kOCols +
                                (uint32_t)(i % S::kOParts * kN + hq * kW);
            tmem_ldw<kW>(ta, o);
#pragma unroll
            for (int j = 0; j < kW; ++j) o[j] = o[j] * c.alpha[hq * kW + j] * c.alpha[hq * kW + j];
            tmem_stw<kW>(ta, o);
          }
        }
#pragma unroll
        for (int q = 0; q < kW / 16; ++q) {  // 16 heads: 16 bytes of each part
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            const int buf = kN == 16 ? k >> 1 : k;
            const int ch = kN == 16 ? k & 1 : hq * (kW / 16) + q;
            const int at = kN == 64 ? r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)
                                    : r * 32 + ((ch ^ ((r >> 2) & 1)) << 4);
            *reinterpret_cast<uint4*>(sb + S::kP + buf * S::kPPart + at) = make_uint4(
                part[k][4 * q], part[k][4 * q + 1], part[k][4 * q + 2], part[k][4 * q + 3]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&c.p_full);
        rs = rs_next;
      }
      if (!ok) break;
      const bool some = w.tb > w.ta, whole = w.ta == 0 && w.tb == w.k.n;
      const bool begins = some && w.ta == 0 && !whole;
      if (begins) hd.start_tile = w.tile_id;
      if (!whole && !begins && hd.cont_tile < 0) {
        hd.cont_tile = w.tile_id;
        hd.cont_some = some;
        hd.cont_ends = w.tb == w.k.n;
      }
      if (!some && !whole) continue;
      if (!some) {
        store_nothing<kSoft>(p, row0, heads, tid);
        continue;
      }
      {
        const float sum = across_rows<kW, false>(l, lane);
        if (lane < kW) c.red[qw][hq * kW + lane] = sum;
      }
      if (!wait_on(&c.o_full, segs & 1, dead, wait_ns)) c.soft_dead[tiles & 1] = 1;
      ++segs;
      __syncwarp();
      tc_fence_after();
      sync_soft<kSoft>();
      if (c.soft_dead[tiles & 1]) {
        ok = false;
        break;
      }
      if (tid < kN) {
        const float sum = (c.red[0][tid] + c.red[1][tid]) + (c.red[2][tid] + c.red[3][tid]);
        const float m = c.m[tid];
        c.m[tid] = -INFINITY;
        c.nm[tid] = 0.f;
        if (whole) {
          // a NaN sum stays one
          c.l[tid] = sum == 0.f ? 0.f : 1.f / (sum * kUp) * pow2(exponent);
          if (p.lse && tid < heads) p.lse[row0 + tid] = lse_of(m, sum);
        } else {
          // relative to its own sum: beside a part of other row scales the references alone
          // may lie too far apart
          int ex = 0;
          const float f = fabsf(sum) < INFINITY ? frexpf(sum, &ex) : sum;
          c.l[tid] = ldexpf(1.f, exponent - ex);
          const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
          p.part_ml[slot * kN + tid] = make_float2(m + (float)ex, f);
        }
      }
      sync_soft<kSoft>();
      if (whole)
        store_rows<kN, S::kOParts, S::kOCols>(p, c.l, tl + kOCol, row0, heads, qw, hq, lane);
      else
        store_part<kN, S::kOParts, S::kOCols>(p, 2 * blockIdx.x + (begins ? 1 : 0), tl + kOCol,
                                              heads, qw, hq, lane, c.l);
      tc_fence_before();  // O^T is read: the next segment's P releases it
    }
    if (!ok) hd = Header{-1, -1, 0, 0};
    if (tid == 0 && p.head) p.head[blockIdx.x] = hd;
  } else if (warp < kMmaWarp) {
    // ================= TMA: two warps, two blocks of 128 codes each =================
    const int team = warp - kTma0;
    const int R = 1 << p.box_log, ng = kKeys >> p.box_log;
    int tiles = 0, segs = 0;
    bool ok = issue;
    int issued = 0;  // blocks of tile `tiles` under way, up to this one
    // the cache row of this lane's box of a tile (-1: nothing seen, -2: no page)
    auto box_row = [&](const Keys<kKeys>& k, int b, int v) -> int {
      if (lane >= ng) return -1;
      const int t0 = k.at(v, lane * R);
      if (t0 > k.pos) return -1;
      const int blk = t0 / p.kv.page_size;
      if (blk >= p.kv.max_pages) return -2;
      const int page = __ldg(p.kv.block_table + (long long)b * p.kv.max_pages + blk);
      if (page < 0 || page >= p.kv.n_pages) return -2;
      return page * p.kv.page_size + t0 % p.kv.page_size;
    };
    while (ok && w.next()) {
      if (w.ta == w.tb) continue;
      int row = box_row(w.k, w.b, w.ta);
      if (team == 0) {
        // the queries' parts, once the last segment's products with them are done
        const bool free_q = segs == 0 || wait_on(&c.q_empty, (segs - 1) & 1, dead, wait_ns);
        ok = __all_sync(0xffffffffu, free_q);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&c.q_full, 8 * S::kQBlock);
          for (int i = 0; i < 8; ++i)
            tma_load_2d(sb + S::kQ + (2 * (i & 3) + (i >> 2)) * S::kQBlock, &q_map, i * 64,
                        w.token * p.Hm + w.h0 * kN, &c.q_full);
        }
        ++segs;
      }
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        const int row_next = v + 1 < w.tb ? box_row(w.k, w.b, v + 1) : -1;
        if (row == -2) {
          flag(p.status, DSA_DEV_BAD_PAGE);
          row = -1;
        }
        const unsigned boxes = __ballot_sync(0xffffffffu, row >= 0);
        const int st = stage_of(tiles);
#pragma unroll 1
        for (int blk = team; blk < 4; blk += 2) {
          const bool room = tiles < kStages ||
                            wait_on(&c.empty[st][blk], phase_of(tiles) ^ 1u, dead, wait_ns);
          ok = __all_sync(0xffffffffu, room);
          if (!ok) break;
          if (lane == 0) {
            if (blk == 0) c.groups[st] = boxes;
            mbar_arrive_expect_tx(&c.full[st][blk], __popc(boxes) * R * 128);
          }
          issued = blk + 1;
          __syncwarp();
          if (row >= 0)
            tma_load_2d(sb + S::kKv + st * kStage + blk * kBlock + lane * R * 128, &kv_map,
                        blk * 64, row, &c.full[st][blk]);
        }
        if (!ok) break;
        issued = 0;
        // the next tile's rows to L2 (32 heads' columns, 64 single tokens on 8,192 keys: 70.6
        // us, without 73.4; no difference where tokens share the rows)
        if (team == 0 && row_next >= 0) tma_prefetch_2d(&ahead_map, 0, row_next);
        row = row_next;
      }
    }
    // after a give-up: no copy into this CTA's memory may be in flight at its end
    if (*dead && lane == 0) {
      if (segs > 0) mbar_wait_bounded(&c.q_full, (segs - 1) & 1);
      for (int blk = team; blk < 4; blk += 2)
        for (int i = blk < issued ? 0 : 1; i <= kStages; ++i)
          if (tiles - i >= 0)
            mbar_wait_bounded(&c.full[stage_of(tiles - i)][blk], phase_of(tiles - i));
    }
  } else if (warp == kMmaWarp && issue) {
    // ================= MMA =================
    constexpr uint32_t id_s = idesc_f8(kKeys, 2 * kN, false, false, false);
    constexpr uint32_t id_o = idesc_f8(128, S::kON, true, true, true);
    const uint32_t kvb = smem_u32(sb + S::kKv), qb = smem_u32(sb + S::kQ);
    const uint32_t pb = smem_u32(sb + S::kP);
    // (a descriptor's low bits are the address in 16-byte units: steps add constants)
    const uint64_t d_k0 = sw128_desc(kvb), d_q = sw128_desc(qb);
    const uint64_t d_v0 = umma_desc_sw128(kvb, kBlock, 1024);
    const uint64_t d_p = kN == 64 ? umma_desc_sw64(pb, S::kPPart, 512)
                                  : umma_desc_sw32(pb, S::kPPart, 256);
    // Two streams over the same tiles: scores block by block as a stage's keys arrive,
    // outputs as soon as a tile's weights are there; outputs first (they free the
    // stage), also between the blocks of a tile whose keys are still under way.
    Walk<kKeys, false> wo(p, hb, c.start, units);
    auto segment = [](Walk<kKeys, false>& x) {
      while (x.next())
        if (x.tb > x.ta) return true;
      return false;
    };
    auto ready = [](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0;
    };
    bool ok = true, left_s = segment(w), left_o = segment(wo), have_q = false;
    int ns = 0, blk = 0, no = 0, vs = w.ta, vo = wo.ta, seg = 0;
    unsigned long long since = 0;  // time of the first idle look
    while (left_o) {
      if (no < ns && ready(&c.p_full, no & 1)) {
        const int st = stage_of(no);
        const uint64_t d_v = d_v0 + (uint32_t)(st * (kStage >> 4));
        const uint32_t more = vo > wo.ta ? 1u : 0u;
        tc_fence_after();
#pragma unroll
        for (int mc = 0; mc < 4; ++mc) {
#pragma unroll
          for (int kr = 0; kr < 4; ++kr)
#pragma unroll
            for (int k = 0; k < 3 / S::kOParts; ++k)
              umma_f8_elect(tmem + kOCol + mc * S::kOCols, d_v + ((mc * kBlock + kr * 4096) >> 4),
                            d_p + ((k * S::kPPart + kr * 32 * S::kPRow) >> 4), id_o,
                            (kr | k) ? 1u : more);
          umma_commit_elect(&c.empty[st][mc]);
        }
        ++no;
        if (++vo == wo.tb) {
          umma_commit_elect(&c.o_full);
          left_o = segment(wo);
          vo = wo.ta;
        }
        since = 0;
        continue;
      }
      if (left_s && ns - no < kStages) {
        have_q = have_q || ready(&c.q_full, seg & 1);
        // (the stage's keys imply that its last outputs are done: its scores are free)
        const int st = stage_of(ns);
        if (have_q && ready(&c.full[st][blk], phase_of(ns))) {
          const uint64_t d_k = d_k0 + (uint32_t)(st * (kStage >> 4) + blk * (kBlock >> 4));
          const uint64_t d_qb = d_q + (uint32_t)(blk * (2 * S::kQBlock >> 4));
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            umma_f8_elect(tmem + st * S::kSCols, d_k + (j * 32 >> 4), d_qb + (j * 32 >> 4),
                          id_s, (blk | j) ? 1u : 0u);
          if (++blk == 4) {
            blk = 0;
            umma_commit_elect(&c.s_full[st]);
            ++ns;
            if (++vs == w.tb) {
              umma_commit_elect(&c.q_empty);
              ++seg;
              left_s = segment(w);
              vs = w.ta;
              have_q = false;
            }
          }
          since = 0;
          continue;
        }
      }
      const unsigned long long now = global_ns();
      if (since == 0) since = now;
      const bool late = now - since > wait_ns;
      if (late) *dead = 1;
      if (__any_sync(0xffffffffu, late || *dead)) {
        ok = false;
        break;
      }
    }
    if (!ok) {  // drain what was issued before the CTA's memory is given back
      umma_commit_elect(&c.drain);
      mbar_wait_bounded(&c.drain, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && c.dead) flag(p.status, DSA_DEV_TIMEOUT);  // outputs unspecified
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kTmemCols>(tmem);
  }
}

// the partials' place at the workspace's front
template <int kN>
size_t part_bytes(int n_cta) {
  const size_t n = (size_t)n_cta * 2 * kN * (kL * 4 + 8) + (size_t)n_cta * sizeof(Header);
  return (n + 127) / 128 * 128;
}

template <int kN>
int launch(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  const int n_cta = num_sms();
  Params p = {};
  p.kv = a.kv;
  p.cu_new = a.cu_new;
  p.T = a.T;
  p.B = a.B;
  p.Hm = a.Hm;
  p.window = a.window;
  p.sinks = a.sinks;
  p.zscale = a.sm_scale * kLog2e;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.status = a.status;
  p.drill = failure_drill();
  p.cap = table_cap(a.kv);
  p.box_log = box_log_of(a.kv.page_size);
  p.o_scale = 1.f / kUp;
  p.extra = 1;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)n_cta * 2 * kN * kL);
  p.head = reinterpret_cast<Header*>(p.part_ml + (size_t)n_cta * 2 * kN);
  const long long q_rows = (long long)a.T * a.Hm;
  uint8_t* q_codes = static_cast<uint8_t*>(workspace) + part_bytes<kN>(n_cta);
  float* q_scale = reinterpret_cast<float*>(q_codes + (size_t)q_rows * 2 * kL);
  CUtensorMap q_map, kv_map, ahead_map;
  const uint64_t rows = (uint64_t)a.kv.n_pages * a.kv.page_size;
  if (!byte_map(&q_map, q_codes, (uint64_t)q_rows, 2 * kL, 64, kN, true) ||
      !row_map(&kv_map, a.kv.pages, rows, 1u << p.box_log, true) ||
      !prefetch_map(&ahead_map, a.kv.pages, rows, 1u << p.box_log, true))
    return DSA_ERR_CUDA;
  auto kernel = mla_chunk_f8_kernel<kN>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(kernel, Smem<kN>::kBytes, done)) return DSA_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((q_rows + 7) / 8), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  if (launch_kernel(&cfg, mla_chunk_query_kernel, static_cast<const __nv_bfloat16*>(a.q_lat),
                    q_rows, q_codes, q_scale) != cudaSuccess)
    return DSA_ERR_CUDA;
  cfg.gridDim = dim3(n_cta, 1, 1);
  cfg.blockDim = dim3(cta_threads(kN), 1, 1);
  cfg.dynamicSmemBytes = Smem<kN>::kBytes;
  if (launch_kernel(&cfg, kernel, q_map, kv_map, ahead_map, (const float*)q_scale, p) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  cfg.gridDim = dim3(2 * num_sms(), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return launch_kernel(&cfg, mla_chunk_join_kernel<kN, false>, p, n_cta) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace

size_t mla_chunk_f8_workspace_size(int T, int Hm) {
  const size_t parts = Hm <= 16   ? part_bytes<16>(num_sms())
                       : Hm <= 32 ? part_bytes<32>(num_sms())
                                  : part_bytes<64>(num_sms());
  return parts + (size_t)T * Hm * (2 * kL + 4);
}

int launch_mla_chunk_f8(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  // (16 heads, 64 single tokens on 8,192 keys: 65 us, as 32 heads 72, as 64 103; 4 x 128
  // tokens on 4,096 keys: 199, 226 and 330)
  return a.Hm <= 16   ? launch<16>(a, workspace, stream)
         : a.Hm <= 32 ? launch<32>(a, workspace, stream)
                      : launch<64>(a, workspace, stream);
}

}  // namespace dsa
