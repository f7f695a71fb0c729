// NoPE MLA of a step's new tokens over the paged latent cache on the tcgen05
// tensor cores, a CTA at a time (bf16 activations, latent 512, bf16 pages of any size;
// E4M3 pages whose size is no multiple of 8).
//
// Module glm5next_dsa, "Traps carried from Slice 8" (NoPE: a score is the plain
// latent dot product) and Constants, MASKED_ATTN_MAX_KEYS (dense masked
// attention).  In absorbed MLA the value of a latent row is the row itself, so
// one tile of rows feeds both products.
//
// Work.  A row tile is one token and up to kN of its heads; its keys are what it sees in
// aligned boxes of positions (the sinks' boxes, then those from the window's first
// position, 0 without one, to the token's own), 128 positions to a key tile.  A tile's
// rows share one mask, by position alone: what a token does not see is zeroed in
// shared memory before the second product reads it, so nothing there (NaN, infinity)
// reaches the output.  One persistent CTA per SM takes an equal, contiguous share of
// the (row tile, key tile) units of the whole batch, found from the lengths by a scan
// in every CTA; a row tile whose units fall to several CTAs leaves partials (O
// unnormalised, maximum, sum) that a second kernel joins in CTA order.  Units
// are counted with the longest token's tiles for every token of a sequence and
// scaled to the token's own; tokens are taken from both ends of the chunk in
// turn, so that a share of long and short ones evens out.
//
// Per key tile, S^T = C q^T (M = 128 rows, N = kN heads, K = 512) goes to TMEM; a
// thread holds one row's scores of kN / 2 heads, P = 2^(z - m) goes to shared
// memory row by row, and O^T += C^T P^T (M = 128 latent columns, four chunks)
// reads the same tile MN-major.  The reference m of a head is its maximum when
// it was last raised; it is raised, and O^T and the sums rescaled, only when a
// score passes it by more than kRaiseAt (base 2): bf16 and fp32 keep the same
// relative precision at any scale, so a stale reference costs nothing, and no
// tile but such a one needs a maximum across rows.
//
// What bounds it.  Single tokens: HBM, and a tile's latency.  Otherwise the tile itself:
// one 128 x 64 x 16 MMA reads 6 KB of shared memory at 128 bytes a cycle (measured 51
// cycles; the tensor cores alone would take 32), the next tile's rows are written
// through the same port (1,024 cycles), and the softmax of a tile stands between its two
// products: rows 128 KB, queries 64 KB and P 16 KB leave no room for a second tile, so
// the tile is handed on in four column chunks, each refilled as soon as its part of
// O^T is done.  About 5,500 cycles a tile, of which 4,300 are shared-memory traffic, in long
// row tiles; a row tile's queries, first rows, first references and end come to 12,500
// more (five key tiles a row tile: 8,000 cycles each in all, by counters).
// Measured on GB300 in graphs of calls, 64 heads: 64 single tokens on 4,096 to 16,000 keys
// 131 us (667 MB: 5.1 TB/s, 0.75 of the measured copy rate); chunks of 1 to 128 tokens of 16
// sequences under a window of 512 and 4 sinks 94 us (434 TFLOP/s); one token on 256 keys
// 14.5 us.
#include "mla_chunk.cuh"

namespace dsa {
namespace {

using namespace chunk;

constexpr int kKeys = 128;
constexpr int kKvBlock = kKeys * 128;  // 128 rows x 64 latent columns, 16 KB
constexpr int kSoftThreads = 256;      // warps 0..7

// Row sources: TMA boxes of bf16 rows (page size a multiple of 8); or, for any page
// size, four warps that copy bf16 rows or widen E4M3 rows from global memory.
constexpr int kSrcTma = 0, kSrcCopy = 1, kSrcCopy8 = 2;
// warps 8..: two TMA warps or four row warps, then the MMA warp
__host__ __device__ constexpr int load_warps(int src) { return src == kSrcTma ? 2 : 4; }
__host__ __device__ constexpr int cta_threads(int src) {
  return kSoftThreads + 32 * (load_warps(src) + 1);
}

struct Ctl {
  float m[64], nm[64], alpha[64], l[64], move[64];  // per head; first: read as float4
  float red[4][64];
  float rs[kKeys];
  int valid[kKeys];               // copied rows: the position is seen and has a page
  int prow[2][kKeys];
  uint64_t full[4], empty[4], s_full, p_full, o_full, q_full, q_empty, drain;
  Start start;
  uint32_t tmem;
  unsigned groups;                // TMA boxes of the tile that hold rows
  int raise;
  int soft_dead[2];
  int dead;
};

template <int kN>
struct Smem {
  static constexpr int kQBlock = kN * 128;
  static constexpr int kPRow = kN * 2;              // bytes of one key's probabilities
  static constexpr size_t kKv = 0;
  static constexpr size_t kQ = 8 * (size_t)kKvBlock;
  static constexpr size_t kP = kQ + 8 * (size_t)kQBlock;
  static constexpr size_t kCtl = kP + (size_t)kKeys * kPRow;
  static constexpr size_t kBytes = 1024 + kCtl + sizeof(Ctl);
};
static_assert(Smem<64>::kBytes <= 227 * 1024, "shared memory budget");

// ---- small pieces ------------------------------------------------------------
// whether any thread of the four row warps says so
__device__ __forceinline__ bool vote_rows(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void sync_load() {
  asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
}

// ---- the kernel --------------------------------------------------------------
template <int kN, int kSrc>
__global__ void __launch_bounds__(cta_threads(kSrc), 1)
    mla_chunk_kernel(const __grid_constant__ CUtensorMap q_map,
                     const __grid_constant__ CUtensorMap kv_map,
                     const __grid_constant__ CUtensorMap ahead_map, const Params p) {
  using S = Smem<kN>;
  constexpr int kW = kN / 2;  // heads per softmax thread
  constexpr int kLoad0 = kSoftThreads / 32, kMmaWarp = kLoad0 + load_warps(kSrc);
  constexpr int kTmemCols = kN == 64 ? 512 : 256;  // S^T (kN), O^T (4 kN)
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl& c = *reinterpret_cast<Ctl*>(sb + S::kCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hb = (p.Hm + kN - 1) / kN;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&c.full[i], kSrc == kSrcTma ? 1 : 4);
      mbar_init(&c.empty[i], 1);
    }
    mbar_init(&c.s_full, 1);
    mbar_init(&c.p_full, kSoftThreads / 32);
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

  const unsigned long long units = find_share<kKeys, false, cta_threads(kSrc)>(
      p, hb, blockIdx.x, gridDim.x, &c.start, blockIdx.x == 0);
  const uint32_t tmem = c.tmem;
  Walk<kKeys, false> w(p, hb, c.start, units);
  // a failure drill loads nothing and issues no MMA: the first waits run out
  const bool issue = p.drill == 0;
  const unsigned long long wait_ns = p.drill ? kDrillWaitNs : kWaitNs;
  const uint32_t kvb = smem_u32(sb + S::kKv), qb = smem_u32(sb + S::kQ);
  const uint32_t pb = smem_u32(sb + S::kP);
  volatile int* dead = &c.dead;

  if (warp < kLoad0) {
    // ================= softmax and epilogue =================
    const int qw = warp & 3;      // TMEM lanes 32 qw ..: this thread's key row r
    const int hq = warp >> 2;     // heads kW hq ..
    const int r = qw * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16);
    Header hd = {-1, -1, 0, 0};
    int tiles = 0, segs = 0;      // waits so far
    bool ok = true;
    while (ok && w.next()) {
      float l[kW];                // this row's sums
      bool unset = true;          // some head here has no reference yet
#pragma unroll
      for (int i = 0; i < kW; ++i) l[i] = 0.f;
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        const int t = w.k.at(v, r);
        if (!wait_on(&c.s_full, tiles & 1, dead, wait_ns)) c.soft_dead[tiles & 1] = 1;
        __syncwarp();  // (tcgen05.ld takes a converged warp)
        tc_fence_after();
        float e[kW];
        tmem_ldw<kW>(tl + hq * kW, e);
        bool valid;
        float rs = 1.f;
        if constexpr (kSrc == kSrcTma) {
          valid = w.k.sees(t) && ((c.groups >> (r >> w.k.log)) & 1u);
          if (!valid) {  // the half of this row that this thread clears
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
            for (int blk = 4 * hq; blk < 4 * hq + 4; ++blk)
#pragma unroll
              for (int ch = 0; ch < 8; ++ch)  // (neighbouring rows in different banks)
                *reinterpret_cast<uint4*>(sb + S::kKv + blk * kKvBlock + r * 128 +
                                          ((ch ^ (r & 7)) << 4)) = zero;
          }
        } else {
          valid = c.valid[r] != 0;
        }
        if constexpr (kSrc == kSrcCopy8) rs = valid ? c.rs[r] : 0.f;
        const float zs = (kSrc == kSrcCopy8) ? p.zscale * rs : p.zscale;
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
          high |= e[i] > kRaiseAt;
        }
        // every thread takes the same branch; the flag of a failed wait was
        // written before this barrier
        const bool full = vote_soft<kSoftThreads>(high);
        if (c.soft_dead[tiles & 1]) {
          ok = false;
          break;
        }
        if (full) {
          float top[kW];  // relative to the references so far
#pragma unroll
          for (int i = 0; i < kW; ++i) top[i] = e[i];
          const float m = across_rows<kW, true>(top, lane);
          if (lane < kW) c.red[qw][hq * kW + lane] = m;
          if (tid == 0) c.raise = 0;
          sync_soft<kSoftThreads>();
          if (tid < kN) {
            const float rel = fmaxf(fmaxf(c.red[0][tid], c.red[1][tid]),
                                    fmaxf(c.red[2][tid], c.red[3][tid]));
            const float m_old = c.m[tid];
            float a = 1.f, move = 0.f;
            if (m_old == -INFINITY) {  // nothing accumulated for this head yet
              c.m[tid] = rel;
              if (rel != -INFINITY) move = -rel;
            } else if (rel > kRaiseAt) {
              c.m[tid] = m_old + rel;
              a = ex2_fast(-rel);
              move = -rel;
              c.raise = 1;
            }
            c.alpha[tid] = a;
            c.move[tid] = move;
            c.nm[tid] = c.m[tid] == -INFINITY ? 0.f : -c.m[tid];
          }
          sync_soft<kSoftThreads>();
          unset = false;
#pragma unroll
          for (int i = 0; i < kW; ++i) unset |= c.m[hq * kW + i] == -INFINITY;
          if (c.raise) {  // O^T of the tiles so far is complete: S^T came after it
#pragma unroll
            for (int i = 0; i < kW; ++i) l[i] *= c.alpha[hq * kW + i];
            if (v > w.ta) {
#pragma unroll 1
              for (int mc = 0; mc < 4; ++mc) {
                float o[kW];
                const uint32_t ta = tl + (uint32_t)(kN + mc * kN + hq * kW);
                tmem_ldw<kW>(ta, o);
#pragma unroll
                for (int i = 0; i < kW; ++i) o[i] *= c.alpha[hq * kW + i];
                tmem_stw<kW>(ta, o);
              }
            }
          }
          // (an infinite maximum: its key's weight is NaN, as in the formula)
#pragma unroll
          for (int i = 0; i < kW; ++i) e[i] += c.move[hq * kW + i];
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) e[i] = ex2_fast(e[i]);
        // P is rounded to bf16 for the tensor cores; the sums keep the unrounded
        // weights.  An E4M3 row's scale goes to its weights, so the tile holds codes.
#pragma unroll
        for (int q = 0; q < kW / 8; ++q) {
          const float sc = (kSrc == kSrcCopy8) ? rs : 1.f;
          const uint4 pk4 = make_uint4(pack_bf16(e[8 * q] * sc, e[8 * q + 1] * sc),
                                 pack_bf16(e[8 * q + 2] * sc, e[8 * q + 3] * sc),
                                 pack_bf16(e[8 * q + 4] * sc, e[8 * q + 5] * sc),
                                 pack_bf16(e[8 * q + 6] * sc, e[8 * q + 7] * sc));
          const int ch = hq * (kW / 8) + q;
          const int at = kN == 64 ? r * 128 + ((ch ^ (r & 7)) << 4)
                                  : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
          *reinterpret_cast<uint4*>(sb + S::kP + at) = pk4;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&c.p_full);
#pragma unroll
        for (int i = 0; i < kW; i += 2) add2(l[i], l[i + 1], e[i], e[i + 1]);
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
      const int heads = min(kN, p.Hm - w.h0 * kN);
      const long long row0 = (long long)w.token * p.Hm + w.h0 * kN;
      if (!some) {  // a token that sees nothing
        store_nothing<kSoftThreads>(p, row0, heads, tid);
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
      sync_soft<kSoftThreads>();
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
          c.l[tid] = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays one
          if (p.lse && tid < heads)
            p.lse[row0 + tid] = sum == 0.f ? -INFINITY : (m + log2f(sum)) / kLog2e;
        } else {
          const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
          p.part_ml[slot * kN + tid] = make_float2(m, sum);
        }
      }
      sync_soft<kSoftThreads>();
      if (whole)
        store_rows<kN>(p, c.l, tl + kN, row0, heads, qw, hq, lane);
      else
        store_part<kN>(p, 2 * blockIdx.x + (begins ? 1 : 0), tl + kN, heads, qw, hq, lane);
      tc_fence_before();  // O^T is read: the next segment's P releases it
    }
    if (!ok) hd = Header{-1, -1, 0, 0};
    if (tid == 0 && p.head) p.head[blockIdx.x] = hd;
  } else if (kSrc == kSrcTma && warp < kMmaWarp) {
    // ================= TMA =================
    // Two warps take the chunks in turn: a copy costs the issuing warp 100 cycles and
    // more (16-row boxes: 1,340 a chunk, four times what its part of O^T takes).
    const int team = warp - kLoad0;
    const int R = 1 << p.box_log, ng = kKeys >> p.box_log;
    int tiles = 0, segs = 0;
    bool ok = issue;
    int issued = 0;  // chunks of tile `tiles` under way, up to this one
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
        // the queries, once the previous segment's last product with them is done
        const bool free_q = segs == 0 || wait_on(&c.q_empty, (segs - 1) & 1, dead, wait_ns);
        if (!__all_sync(0xffffffffu, free_q)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&c.q_full, 8 * S::kQBlock);
          for (int blk = 0; blk < 8; ++blk)
            tma_load_2d(sb + S::kQ + blk * S::kQBlock, &q_map, blk * 64,
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
        const uint32_t bytes = __popc(boxes) * R * 256;
#pragma unroll 1
        for (int mc = team; mc < 4; mc += 2) {
          const bool room = tiles == 0 || wait_on(&c.empty[mc], (tiles - 1) & 1, dead, wait_ns);
          ok = __all_sync(0xffffffffu, room);
          if (!ok) break;
          if (lane == 0) {
            if (mc == 0) c.groups = boxes;  // the last tile's softmax has read its own
            mbar_arrive_expect_tx(&c.full[mc], bytes);
          }
          issued = mc + 1;
          __syncwarp();
          if (row >= 0) {
            unsigned char* dst = sb + S::kKv + 2 * mc * kKvBlock + lane * R * 128;
            tma_load_2d(dst, &kv_map, mc * 128, row, &c.full[mc]);
            tma_load_2d(dst + kKvBlock, &kv_map, mc * 128 + 64, row, &c.full[mc]);
          }
        }
        if (!ok) break;
        issued = 0;
        // the next tile's rows to L2, half of a row each (64 single tokens on 8,192
        // keys: 111 us, without 122; no difference where tokens share the rows)
        if (row_next >= 0) tma_prefetch_2d(&ahead_map, team * 256, row_next);
        row = row_next;
      }
    }
    // after a give-up: no copy into this CTA's memory may be in flight at its end
    if (*dead && lane == 0) {
      for (int mc = team; mc < 4; mc += 2)
        if (mc < issued || tiles > 0)
          mbar_wait_bounded(&c.full[mc], (mc < issued ? tiles : tiles - 1) & 1);
      if (segs > 0) mbar_wait_bounded(&c.q_full, (segs - 1) & 1);
    }
  } else if (warp < kMmaWarp) {
    // ================= rows =================
    int tiles = 0, segs = 0;
    bool ok = issue;
    const int lt = tid - kSoftThreads;  // 0..127: its row of every tile
    {
      // the cache row of position t (-1: not seen or no page)
      auto row_of = [&](const Keys<kKeys>& k, int b, int t) -> int {
        if (t > k.pos) return -1;  // (single positions: none but visible ones)
        const int blk = t / p.kv.page_size;
        int page = -1;
        if (blk < p.kv.max_pages)
          page = __ldg(p.kv.block_table + (long long)b * p.kv.max_pages + blk);
        if (page < 0 || page >= p.kv.n_pages) {
          flag(p.status, DSA_DEV_BAD_PAGE);
          return -1;
        }
        return page * p.kv.page_size + t % p.kv.page_size;
      };
      constexpr int kPer = kSrc == kSrcCopy8 ? 8 : 16;  // 16-byte pieces a thread and chunk
      constexpr int kPieces = kSrc == kSrcCopy8 ? 8 : 16;  // of a row's chunk
      constexpr int kRowBytes = kSrc == kSrcCopy8 ? kL : 2 * kL;
      const unsigned char* pages = static_cast<const unsigned char*>(p.kv.pages);
      while (ok && w.next()) {
        if (w.ta == w.tb) continue;
        if (segs > 0 && !wait_on(&c.q_empty, (segs - 1) & 1, dead, wait_ns)) {
          ok = false;
        } else if (lt == 0) {
          mbar_arrive_expect_tx(&c.q_full, 8 * S::kQBlock);
          for (int blk = 0; blk < 8; ++blk)
            tma_load_2d(sb + S::kQ + blk * S::kQBlock, &q_map, blk * 64,
                        w.token * p.Hm + w.h0 * kN, &c.q_full);
        }
        ++segs;
        int row = row_of(w.k, w.b, w.k.at(w.ta, lt));
        for (int v = w.ta; v < w.tb; ++v, ++tiles) {
          // this tile's rows (in its slot since the tile before, but for the first)
          // and the next one's
          if (v == w.ta) c.prow[tiles & 1][lt] = row;
          float rs = 0.f;
          if (kSrc == kSrcCopy8 && row >= 0) rs = __ldg(p.kv.row_scale + row);
          const bool seen = row >= 0;
          row = v + 1 < w.tb ? row_of(w.k, w.b, w.k.at(v + 1, lt)) : -1;
          if (row >= 0) {
            const unsigned char* nx = pages + (long long)row * kRowBytes;
#pragma unroll
            for (int o = 0; o < kRowBytes; o += 128)
              asm volatile("prefetch.global.L2 [%0];" ::"l"(nx + o));
          }
          c.prow[(tiles + 1) & 1][lt] = row;
          sync_load();
          uint4 raw[kPer];
          auto fetch = [&](int mc) {
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
              const int i = u * 128 + lt, rr = i / kPieces, pc = i % kPieces;
              const int prow = c.prow[tiles & 1][rr];
              raw[u] = prow >= 0 ? __ldg(reinterpret_cast<const uint4*>(
                                     pages + (long long)prow * kRowBytes +
                                     (mc * kPieces + pc) * 16))
                               : make_uint4(0u, 0u, 0u, 0u);
            }
          };
          fetch(0);
#pragma unroll 1
          for (int mc = 0; mc < 4; ++mc) {
            if (mc > 0) fetch(mc);
            if (ok && tiles > 0 && !wait_on(&c.empty[mc], (tiles - 1) & 1, dead, wait_ns))
              ok = false;
            if (mc == 0) {  // the last tile's softmax has read its own
              c.valid[lt] = seen;
              c.rs[lt] = rs;
            }
            unsigned char* dst = sb + S::kKv + 2 * mc * kKvBlock;
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
              const int i = u * 128 + lt, rr = i / kPieces, pc = i % kPieces;
              if (kSrc == kSrcCopy8) {
                const uint32_t x[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                  const int ch = 2 * pc + hf;
                  *reinterpret_cast<uint4*>(dst + (ch >> 3) * kKvBlock + rr * 128 +
                                            (((ch & 7) ^ (rr & 7)) << 4)) =
                      make_uint4(e4m3x2_to_bf16x2(x[2 * hf] & 0xffffu),
                                 e4m3x2_to_bf16x2(x[2 * hf] >> 16),
                                 e4m3x2_to_bf16x2(x[2 * hf + 1] & 0xffffu),
                                 e4m3x2_to_bf16x2(x[2 * hf + 1] >> 16));
                }
              } else {
                *reinterpret_cast<uint4*>(dst + (pc >> 3) * kKvBlock + rr * 128 +
                                          (((pc & 7) ^ (rr & 7)) << 4)) = raw[u];
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive1(&c.full[mc]);
          }
          // after a give-up every thread leaves at the same tile (nobody waits for
          // the others in sync_load)
          if (vote_rows(!ok)) {
            ok = false;
            break;
          }
        }
        ok = !vote_rows(!ok);
      }
      if (*dead && lt == 0 && segs > 0) mbar_wait_bounded(&c.q_full, (segs - 1) & 1);
    }
  } else if (issue) {
    // ================= MMA =================
    // The whole warp runs the loop and one elected lane issues: the descriptors
    // stay in uniform registers (one lane alone: 73 instead of 51 cycles a step).
    constexpr uint32_t id_s = umma_idesc_bf16(kKeys, kN, false);
    constexpr uint32_t id_o = umma_idesc_bf16(128, kN, true, true);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_on(bar, parity, dead, wait_ns)) != 0;
    };
    // A descriptor's low bits are the address in 16-byte units (below 2^14): a step adds
    // a constant to a base.  (Built anew for each step they cost 70 cycles a step.)
    const uint64_t d_k = sw128_desc(kvb), d_q = sw128_desc(qb);
    const uint64_t d_v = umma_desc_sw128(kvb, kKvBlock, 1024);
    const uint64_t d_p = kN == 64 ? umma_desc_sw128(pb, kKeys * 128, 1024)
                                  : umma_desc_sw64(pb, kKeys * 64, 512);
    int tiles = 0, segs = 0;
    bool ok = true;
    while (ok && w.next()) {
      if (w.ta == w.tb) continue;
      ok = wait_all(&c.q_full, segs & 1);
      for (int v = w.ta; ok && v < w.tb; ++v, ++tiles) {
#pragma unroll
        for (int mc = 0; mc < 4; ++mc) {
          ok = ok && wait_all(&c.full[mc], tiles & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint32_t blk = 2 * mc + (j >> 2), off = (j & 3) * 32;
            umma_bf16_elect(tmem, d_k + ((blk * kKvBlock + off) >> 4),
                            d_q + ((blk * S::kQBlock + off) >> 4), id_s, (mc | j) ? 1u : 0u);
          }
        }
        if (!ok) break;
        umma_commit_elect(&c.s_full);
        if (v + 1 == w.tb) umma_commit_elect(&c.q_empty);
        ok = wait_all(&c.p_full, tiles & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int mc = 0; mc < 4; ++mc) {
#pragma unroll
          for (int kr = 0; kr < 8; ++kr) {
            umma_bf16_elect(tmem + kN + mc * kN, d_v + ((2 * mc * kKvBlock + kr * 2048) >> 4),
                            d_p + ((kr * (kN == 64 ? 2048 : 1024)) >> 4), id_o,
                            (v > w.ta || kr > 0) ? 1u : 0u);
          }
          umma_commit_elect(&c.empty[mc]);
        }
      }
      if (!ok) break;
      umma_commit_elect(&c.o_full);
      ++segs;
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

template <int kN>
size_t workspace_bytes(int n_cta) {
  return (size_t)n_cta * 2 * kN * (kL * 4 + 8) + (size_t)n_cta * sizeof(Header);
}

template <int kN, int kSrc>
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
  p.o_scale = 1.f;
  p.extra = 2;
  p.box_log = kSrc == kSrcTma ? box_log_of(a.kv.page_size) : 0;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)n_cta * 2 * kN * kL);
  p.head = reinterpret_cast<Header*>(p.part_ml + (size_t)n_cta * 2 * kN);
  CUtensorMap q_map, kv_map, ahead_map;
  if (!row_map(&q_map, a.q_lat, (uint64_t)a.T * a.Hm, kN)) return DSA_ERR_CUDA;
  kv_map = ahead_map = q_map;
  const uint64_t rows = (uint64_t)a.kv.n_pages * a.kv.page_size;
  if (kSrc == kSrcTma &&
      (!row_map(&kv_map, a.kv.pages, rows, 1u << p.box_log) ||
       !prefetch_map(&ahead_map, a.kv.pages, rows, 1u << p.box_log, false)))
    return DSA_ERR_CUDA;
  auto kernel = mla_chunk_kernel<kN, kSrc>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(kernel, Smem<kN>::kBytes, done)) return DSA_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(n_cta, 1, 1);
  cfg.blockDim = dim3(cta_threads(kSrc), 1, 1);
  cfg.dynamicSmemBytes = Smem<kN>::kBytes;
  if (launch_kernel(&cfg, kernel, q_map, kv_map, ahead_map, p) != cudaSuccess) return DSA_ERR_CUDA;
  cfg.gridDim = dim3(2 * num_sms(), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return launch_kernel(&cfg, mla_chunk_join_kernel<kN, false>, p, n_cta) == cudaSuccess ? DSA_OK
                                                                                 : DSA_ERR_CUDA;
}

// TMA takes boxes of 8 rows and more, so pages of a multiple of 8; any other page size is
// copied row by row (64 single tokens on 8,192 keys in pages of 64: 111 us by TMA, 190
// copied).
template <int kN>
int launch_src(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  if (a.kv.kv_dtype == DSA_FP8_E4M3) return launch<kN, kSrcCopy8>(a, workspace, stream);
  return a.kv.page_size % 8 == 0 ? launch<kN, kSrcTma>(a, workspace, stream)
                                 : launch<kN, kSrcCopy>(a, workspace, stream);
}

}  // namespace

bool mla_chunk_umma_ok(int L, int dtype, int kv_dtype) {
  return L == kL && dtype == DSA_BF16 && (kv_dtype == DSA_BF16 || kv_dtype == DSA_FP8_E4M3);
}

size_t mla_chunk_umma_workspace_size(int Hm) {
  return Hm <= 32 ? workspace_bytes<32>(num_sms()) : workspace_bytes<64>(num_sms());
}

// Up to 32 heads take half the columns (16 heads, 16 sequences x 32 tokens on 1,024 keys:
// 86 us, in 64 columns 103; 4 tokens on 4,096: 49 and 57).
int launch_mla_chunk_umma(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  return a.Hm <= 32 ? launch_src<32>(a, workspace, stream)
                    : launch_src<64>(a, workspace, stream);
}

}  // namespace dsa
