// The chunk attention on pairs of CTAs (bf16 activations, latent 512, more than 32
// heads, bf16 pages of a multiple of 8 rows): two row blocks of 64 (two tokens, or one
// token's two blocks of heads) share every key row.
//
// Why pairs.  One CTA cannot hold more than 64 rows: the fp32 output of a row takes
// 512 TMEM columns over 128 lanes, and every key row is fetched for one token.  A
// cluster of two CTAs splits the latent axis instead: CTA c holds latent columns
// 256 c .. of the queries (64 KB), of the keys (32 KB for a tile of 64, four stages), and
// of the output (256 TMEM columns for all 128 rows).
//   S_c = Q_c K_c^T      M = 128 rows, N = 64 keys, K = 256: a partial sum
//   S   = S_0 + S_1      each CTA sends the partials of the other one's 64 rows
//                        through distributed shared memory and adds its own
//   P                    softmax weights of its 64 rows, written to its own TMEM and
//                        sent (bf16) to the other's
//   O_c += P V_c         A = P from TMEM, V_c = K_c read MN-major, N = 256, K = 64
// An MMA then reads 6 KB of shared memory for 32 cycles' work (QK) or 8 KB for 128 (PV):
// 20 MMAs, about 1,350 cycles a tile of 128 x 64; the single-CTA kernel takes 6,200
// for the same scores.  A key row is fetched once for two tokens, and no product is
// done twice.  What bounds it is the exchange: scores, send, sum, weights, send and PV are
// a chain of about 9,500 cycles a tile, of which four tiles are on their way at once (what
// shared memory holds).  Measured on GB300, 64 heads, 2,048 tokens behind 14,336:
// 4.00 ms, 1,031 TFLOP/s (0.55 of the measured bf16 rate; the single-CTA kernel: 4.62 ms).
//
// The two tokens of a pair see the same keys but for the last one and the first of a
// window.  A key that neither sees is zeroed in shared memory before PV, and so is one that
// only one of them sees if it holds a NaN or an infinity: nothing masked reaches a row.
// The seeing token's logit is then NaN or infinite, too, and its sums NaN, unless the
// logit is minus infinity: a weight of 0 times the infinity is NaN in that latent column
// alone, so these columns are noted and stored as NaN.
//
// Every wait is bounded; both CTAs meet at a cluster barrier before either ends.
#include "mla_chunk.cuh"

namespace dsa {
namespace {

using namespace chunk;

constexpr int kKT = 64;                      // keys of a tile
constexpr int kBoxLog = 3;                   // a TMA box: 8 rows of this CTA's 256 latent
constexpr int kBoxes = kKT >> kBoxLog;       // columns, [64-column block][row][128 B]
constexpr int kBoxBytes = 4096;
constexpr unsigned kAllBoxes = (1u << kBoxes) - 1;
constexpr int kStageBytes = kBoxes * kBoxBytes;
constexpr int kStages = 4;
constexpr int kQBlock = 128 * 128;           // 128 rows x 64 latent columns
// Warps 0..15 by TMEM lane quarter (warp mod 4).  The quarters of this CTA's row block
// have two teams of softmax warps that take the tiles in turn (a tile's weights take
// longer than its products; only raising a reference has an order); the other block's
// have warps that send its partial scores and warps that receive its weights.  Two
// warps share a quarter's keys: 32 a thread.
constexpr int kRowWarps = 16;
constexpr int kTeamWarps = 4;
constexpr int kW = kKT / 2;
constexpr int kThreads = 32 * (kRowWarps + 4);
constexpr size_t kOffQ = 0;
constexpr size_t kOffK = 4 * (size_t)kQBlock;
constexpr size_t kOffS = kOffK + (size_t)kStages * kStageBytes;   // [16][64 rows] x 16 B
constexpr size_t kOffP = kOffS + (size_t)(kKT / 4) * 64 * 16;     // [16][64 rows] x 8 B
constexpr uint32_t kSBytes = kKT * 64 * 4, kPBytes = kKT * 64 * 2 + 64 * 4;

struct Ctl {
  float alpha[64];                 // from the other CTA: its rows' rescale of this tile
  float inv[128];                  // 1 / sum of every row (the other CTA's rows: sent)
  float m[64];                     // own rows: the reference (base 2)
  float mx[2][2][64];              // [team][half of the keys]: a tile's row maxima
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages];
  uint64_t s_full[kStages], p_full[kStages], o_full, drain;
  // [2]: by the tile's team, so that each waiter sees every phase of its barrier
  uint64_t in_s[2], in_p, in_l;    // data from the other CTA
  uint64_t free_s, free_p[2];      // the other CTA has read what was sent
  uint64_t turn[2];                // the references of this tile stand
  uint64_t sums, epi;              // the sums of a segment's rows
  uint64_t o_free;                 // a segment's outputs are read
  Start start;
  uint32_t tmem;
  unsigned groups[kStages];        // boxes of the tile that have a page
  // by segment (its parity) and row block: latent columns in which a zeroed key that only
  // this block sees is not finite
  uint32_t odd[2][2][8];
  int team_dead[2][2];
  int dead;
};
constexpr size_t kOffCtl = kOffP + (size_t)(kKT / 4) * 64 * 8;
constexpr size_t kSmem = 1024 + kOffCtl + sizeof(Ctl);
static_assert(kSmem <= 227 * 1024, "shared memory budget");
static_assert(256 + kStages * kKT <= 512, "TMEM columns");

// ---- cluster pieces ------------------------------------------------------------
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// the address of this CTA's shared-memory location in CTA `rank`
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// 16 / 8 / 4 bytes to the other CTA; counted on its barrier
__device__ __forceinline__ void send16(uint32_t addr, uint4 v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1,%2,%3,%4},"
      " [%5];" ::"r"(addr),
      "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void send8(uint32_t addr, uint32_t x, uint32_t y, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1,%2}, [%3];" ::"r"(
          addr),
      "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void send4(uint32_t addr, float v, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
      "r"(__float_as_uint(v)), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
// a barrier of a team's warps: whether any of their threads says so
__device__ __forceinline__ bool vote_team(int team, bool v) {
  uint32_t r;
  if (team == 0)
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, 2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
  return r != 0;
}

// 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_st16(uint32_t ta, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(ta),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// O += P V with P (the A operand) in TMEM; one elected lane of a converged warp.
__device__ __forceinline__ void umma_tmem_a_elect(uint32_t d, uint32_t a, uint64_t b,
                                                  uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// What one row block (token) of the tile sees.
struct Sight {
  int pos, lo, sinks;
  __device__ __forceinline__ bool operator()(int t) const {
    return t <= pos && (t >= lo || t < sinks);
  }
};
__device__ __forceinline__ Sight sight_of(int pos, const Params& p) {
  return Sight{pos, p.window > 0 ? max(0, pos - p.window + 1) : 0, p.sinks};
}

using PairWalk = Walk<kKT, true>;
using PairKeys = Keys<kKT>;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mla_chunk_pair_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap kv_map, const Params p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl& c = *reinterpret_cast<Ctl*>(sb + kOffCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cta_rank(), other = rank ^ 1u;
  // the softmax warps sit on two of the SM's four schedulers (their lane quarters):
  // the TMA and the MMA warp go to the other two
  const int kTmaWarp = kRowWarps + (rank == 0 ? 2 : 0), kMmaWarp = kTmaWarp + 1;
  const int hb = (p.Hm + 63) / 64;
  const unsigned me = blockIdx.x >> 1, workers = gridDim.x >> 1;

  if (tid == 0) {
    mbar_init(&c.q_full, 1);
    mbar_init(&c.q_empty, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&c.k_full[i], 1);
      mbar_init(&c.k_empty[i], 1);
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_full[i], 2 * kTeamWarps);
    }
    mbar_init(&c.o_full, 1);
    mbar_init(&c.drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.in_s[i], 1);
      mbar_init(&c.free_p[i], kTeamWarps);
      mbar_init(&c.turn[i], kTeamWarps);
    }
    mbar_init(&c.in_p, 1);
    mbar_init(&c.in_l, 1);
    mbar_init(&c.free_s, kTeamWarps);
    mbar_init(&c.sums, 2 * kTeamWarps);
    mbar_init(&c.epi, 3 * kTeamWarps);
    mbar_init(&c.o_free, 3 * kTeamWarps);
    fence_mbar_init();
    c.team_dead[0][0] = c.team_dead[0][1] = c.team_dead[1][0] = c.team_dead[1][1] = c.dead = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc<512>(&c.tmem);
    tc_fence_before();
  }
  if (tid < 64) c.m[tid] = -INFINITY;
  if (tid < 32) c.odd[tid >> 4][(tid >> 3) & 1][tid & 7] = 0u;
  pdl_wait();  // every input may come from the kernel just before
  pdl_launch_dependents();
  const unsigned long long units = find_share<kKT, true, kThreads>(
      p, hb, me, workers, &c.start, blockIdx.x == 0);
  cluster_sync();  // the other CTA's barriers exist
  const uint32_t tmem = c.tmem;
  const bool any = c.start.b < p.B;
  PairWalk w(p, hb, c.start, units);
  // a failure drill loads nothing and issues no MMA: the first waits run out
  const bool issue = p.drill == 0;
  const unsigned long long wait_ns = p.drill ? kDrillWaitNs : kWaitNs;
  volatile int* dead = &c.dead;

  if (warp < kRowWarps) {
    const int qw = warp & 3, part = warp >> 2;  // TMEM lanes 32 qw ..
    const int g = qw >> 1;                      // row block of these lanes
    const bool own = g == (int)rank;
    const int r = (qw & 1) * 32 + lane;         // row of the block
    const uint32_t tl = tmem + ((uint32_t)(qw * 32) << 16);
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(0xffffffffu, wait_on(bar, parity, dead, wait_ns)) != 0;
    };
    if (!own && part < 2) {
      // ================= send the other block's partial scores =================
      const int h = part;  // keys 32 h ..
      const uint32_t to_s = map_to(smem_u32(sb + kOffS) + (h * (kW / 4) * 64 + r) * 16, other);
      const uint32_t bar_s[2] = {map_to(smem_u32(&c.in_s[0]), other),
                                 map_to(smem_u32(&c.in_s[1]), other)};
      int tiles = 0;
      bool ok = true;
      while (ok && w.next()) {
        for (int v = w.ta; v < w.tb; ++v, ++tiles) {
          const int st = tiles % kStages;
          ok = wait_all(&c.s_full[st], (tiles / kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          float e[kW];
          tmem_ld32(tl + 256 + (uint32_t)(st * kKT + h * kW), e);
          tc_fence_before();
          // the other CTA has read the last tile's
          ok = tiles == 0 || wait_all(&c.free_s, (tiles - 1) & 1);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < kW / 4; ++j)
            send16(to_s + j * 64 * 16,
                   make_uint4(__float_as_uint(e[4 * j]), __float_as_uint(e[4 * j + 1]),
                              __float_as_uint(e[4 * j + 2]), __float_as_uint(e[4 * j + 3])),
                   bar_s[tiles & 1]);
        }
      }
    } else {
      // ================= softmax of the own block; weights of the other =================
      const int team = part >> 1, h = part & 1;  // keys 32 h ..
      // O columns, in blocks of 32: of a segment's end, and of a rescale
      const int o0 = own ? part * 64 : h * 128, o_n = own ? 2 : 4;
      const bool first = own ? (warp & 3) == 2 * (int)rank && h == 0
                             : (warp & 3) == 2 * (int)other && h == 0;
      const uint32_t to_p = map_to(smem_u32(sb + kOffP) + (h * (kW / 4) * 64 + r) * 8, other);
      const uint32_t bar_p = map_to(smem_u32(&c.in_p), other),
                     bar_l = map_to(smem_u32(&c.in_l), other),
                     bar_free_s = map_to(smem_u32(&c.free_s), other),
                     bar_free_p[2] = {map_to(smem_u32(&c.free_p[0]), other),
                                      map_to(smem_u32(&c.free_p[1]), other)};
      const uint4* in_s = reinterpret_cast<const uint4*>(sb + kOffS) + h * (kW / 4) * 64 + r;
      const uint2* in_p = reinterpret_cast<const uint2*>(sb + kOffP) + h * (kW / 4) * 64 + r;
      const int ttid = ((warp & 1) + 2 * h) * 32 + lane;  // thread of the team
      Header hd = {-1, -1, 0, 0};
      int tiles = 0, segs = 0, sums = 0;
      bool ok = true;
      // The phases of the data from the other CTA are armed one ahead.  (Nothing of
      // the next phase is sent before every reader of this one has said so.)
      if (any && first && lane == 0) {
        if (own) {
          mbar_arrive_expect_tx(&c.in_s[team], kSBytes);
          if (team == 0) mbar_arrive_expect_tx(&c.in_l, 64 * 4);
        } else {
          mbar_arrive_expect_tx(&c.in_p, kPBytes);
        }
      }
      // O of the tiles so far, once the last of them is in it
      auto rescale = [&](int tiles, float alpha) {
        wait_on(&c.k_empty[(tiles - 1) % kStages], ((tiles - 1) / kStages) & 1, dead, wait_ns);
        __syncwarp();
        tc_fence_after();
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          float o[32];
          tmem_ld32(tl + h * 128 + cc * 32, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(tl + h * 128 + cc * 32, o);
        }
      };
      while (ok && w.next()) {
        // this thread's row block: its token, its heads, what it sees
        const bool there = p.Hm > 64 || g == 0 || w.two;
        const int token = p.Hm > 64 ? w.token : w.token + (there ? g : 0);
        const int head = p.Hm > 64 ? g * 64 + r : r;
        const bool live = there && head < p.Hm;
        const int pos_a = w.pos0 < 0 ? -1 : w.pos0;
        // (a missing second token sees what the first one does, for nobody)
        const int pos_b = w.two ? (w.pos0 + 1 < 0 ? -1 : w.pos0 + 1) : pos_a;
        const Sight sa = sight_of(pos_a, p), sbt = sight_of(pos_b, p);
        const Sight mine = g == 0 ? sa : sbt;
        float m = -INFINITY, l = 0.f;  // l: this thread's sum, relative to m
        for (int v = w.ta; v < w.tb; ++v, ++tiles) {
          if (own && (tiles & 1) != team) continue;
          const int st = tiles % kStages, ph = (tiles / kStages) & 1;
          const uint32_t tS = tl + 256 + (uint32_t)(st * kKT);
          if (own) {
            const int turn = (tiles >> 1) & 1;
            // is every key of the tile seen by both blocks (once it has its pages)?
            const int t0 = w.k.at(v, 0), t1 = w.k.at(v, kKT - 1);
            const bool span = t1 - t0 == kKT - 1 && t0 >= max(sa.lo, sbt.lo) &&
                              t1 <= min(sa.pos, sbt.pos);
            bool fine = wait_on(&c.s_full[st], ph, dead, wait_ns);
            __syncwarp();
            tc_fence_after();
            float e[kW];
            tmem_ld32(tS + h * kW, e);
            const bool plain = span && c.groups[st] == kAllBoxes;
            if (!plain && ttid < kKT) {
              // clear what neither sees, and what one does not see if it is not finite
              const int key = ttid;
              const int t = w.k.at(v, key);
              const bool paged = (c.groups[st] >> (key >> kBoxLog)) & 1u;
              const bool ina = paged && sa(t), inb = paged && sbt(t);
              if (!(ina && inb)) {
                unsigned char* kr = sb + kOffK + st * kStageBytes + (key >> 3) * kBoxBytes +
                                    (key & 7) * 128;
                bool odd = !(ina || inb);
                if (!odd) {
                  uint32_t* cols = c.odd[segs & 1][inb ? 1 : 0];  // (one such key a block)
                  for (int i = 0; i < 32; ++i) {
                    const uint4 x = *reinterpret_cast<const uint4*>(
                        kr + (i >> 3) * 1024 + (((i & 7) ^ (key & 7)) << 4));
                    const uint32_t wd[4] = {x.x, x.y, x.z, x.w};
                    uint32_t bits = 0u;
                    for (int j = 0; j < 4; ++j) {
                      if ((wd[j] & 0x7f80u) == 0x7f80u) bits |= 1u << (2 * j);
                      if ((wd[j] & 0x7f800000u) == 0x7f800000u) bits |= 2u << (2 * j);
                    }
                    if (bits) {
                      cols[i >> 2] |= bits << ((i & 3) * 8);
                      odd = true;
                    }
                  }
                }
                if (odd)
                  for (int i = 0; i < 32; ++i)
                    *reinterpret_cast<uint4*>(kr + (i >> 3) * 1024 +
                                              (((i & 7) ^ (key & 7)) << 4)) =
                        make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async_smem();
            }
            uint32_t see = 0xffffffffu;  // the keys of this warp that the own block sees
            if (!plain) {
              const int key = h * kW + lane;
              see = __ballot_sync(0xffffffffu, mine(w.k.at(v, key)) &&
                                                   ((c.groups[st] >> (key >> kBoxLog)) & 1u));
            }
            fine = fine && wait_on(&c.in_s[team], turn, dead, wait_ns);
            __syncwarp();
            // the next one (never while this one is still open)
            if (fine && first && lane == 0) mbar_arrive_expect_tx(&c.in_s[team], kSBytes);
#pragma unroll
            for (int j = 0; j < kW / 4; ++j) {
              const uint4 x = in_s[j * 64];
              add2(e[4 * j], e[4 * j + 1], __uint_as_float(x.x), __uint_as_float(x.y));
              add2(e[4 * j + 2], e[4 * j + 3], __uint_as_float(x.z), __uint_as_float(x.w));
            }
            __syncwarp();
            if (fine && lane == 0) arrive_remote(bar_free_s);
            // the references, once the last tile's team has settled them
            if (tiles > 0 && fine)
              fine = wait_on(&c.turn[team ^ 1], ((tiles - 1) >> 1) & 1, dead, wait_ns);
            __syncwarp();
            const float m_now = c.m[r];
            if (m_now != m) {
              l *= ex2_fast(m - m_now);  // (0 before the first key: m = -inf)
              m = m_now;
            }
            const float nm = m == -INFINITY ? 0.f : -m;
#pragma unroll
            for (int i = 0; i < kW; i += 2) fma2(e[i], e[i + 1], p.zscale, nm, nm);
            if (!plain) {
#pragma unroll
              for (int i = 0; i < kW; ++i)
                if (!((see >> i) & 1u)) e[i] = -INFINITY;
            }
            float t4[4] = {e[0], e[1], e[2], e[3]};
#pragma unroll
            for (int i = 4; i < kW; ++i) t4[i & 3] = fmaxf(t4[i & 3], e[i]);
            const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
            if (!fine) c.team_dead[team][turn] = 1;
            c.mx[team][h][r] = top;  // relative to the reference
            // (also: both threads of a row have read its scores, which P overlays)
            const bool full = vote_team(team, live && (m == -INFINITY || top > kRaiseAt));
            if (c.team_dead[team][turn]) {
              ok = false;
              break;
            }
            float alpha = 1.f;
            if (full) {
              const float both = fmaxf(c.mx[team][0][r], c.mx[team][1][r]);  // relative
              float step = 0.f;
              if (m == -INFINITY) {
                if (both > -INFINITY) {  // the first key that this row sees
                  m = both;              // (nothing accumulated: no rescale)
                  step = -both;
                }
              } else if (both > kRaiseAt) {
                m += both;
                step = -both;
                alpha = ex2_fast(-both);
                l *= alpha;
              }
              if (h == 0) c.m[r] = m;
              __syncwarp();
              // (an infinite maximum: its key's weight is NaN, as in the formula)
#pragma unroll
              for (int i = 0; i < kW; ++i) e[i] += step;
            }
            if (lane == 0) mbar_arrive1(&c.turn[team]);
#pragma unroll
            for (int i = 0; i < kW; ++i) e[i] = ex2_fast(e[i]);
            float s4[4] = {e[0], e[1], e[2], e[3]};
#pragma unroll
            for (int i = 4; i < kW; i += 4) {
              add2(s4[0], s4[1], e[i], e[i + 1]);
              add2(s4[2], s4[3], e[i + 2], e[i + 3]);
            }
            l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
            // P is rounded to bf16 for the tensor cores; the sums keep the unrounded
            // weights.
            uint32_t pk[kW / 2];
#pragma unroll
            for (int i = 0; i < kW / 2; ++i) pk[i] = pack_bf16(e[2 * i], e[2 * i + 1]);
            // the other CTA has taken the last tile's weights
            if (tiles > 0 &&
                !wait_on(&c.free_p[team ^ 1], ((tiles - 1) >> 1) & 1, dead, wait_ns)) {
              c.team_dead[team][turn ^ 1] = 1;
            } else {
#pragma unroll
              for (int j = 0; j < kW / 4; ++j)
                send8(to_p + j * 64 * 8, pk[2 * j], pk[2 * j + 1], bar_p);
              if (h == 0) send4(map_to(smem_u32(&c.alpha[r]), other), alpha, bar_p);
            }
            __syncwarp();
            if (v > w.ta && __any_sync(0xffffffffu, alpha != 1.f)) rescale(tiles, alpha);
            tmem_st16(tS + h * (kW / 2), pk);
          } else {
            // ---- the other block's weights (its scores here were read before the
            // other CTA could make them)
            ok = wait_all(&c.in_p, tiles & 1);
            if (!ok) break;
            if (first && lane == 0) mbar_arrive_expect_tx(&c.in_p, kPBytes);  // the next tile's
            uint32_t pk[kW / 2];
#pragma unroll
            for (int j = 0; j < kW / 4; ++j) {
              const uint2 x = in_p[j * 64];
              pk[2 * j] = x.x;
              pk[2 * j + 1] = x.y;
            }
            const float alpha = c.alpha[r];
            const bool raised = __any_sync(0xffffffffu, alpha != 1.f);
            if (lane == 0) arrive_remote(bar_free_p[tiles & 1]);
            if (v > w.ta && raised) rescale(tiles, alpha);
            tmem_st16(tS + h * (kW / 2), pk);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive1(&c.p_full[st]);
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
        const long long row = (long long)token * p.Hm + head;
        if (!some) {  // tokens that see nothing
          if (own && live) {
            __nv_bfloat16* dst = p.out + row * kL + part * 128;
            for (int i = 0; i < 16; ++i)
              *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse && part == 0) p.lse[row] = -INFINITY;
          }
          continue;
        }
        bool fine = wait_on(&c.o_full, segs & 1, dead, wait_ns);
        __syncwarp();
        tc_fence_after();
        const int slot = 2 * (int)me + (begins ? 1 : 0);
        if (own) {
          // the four threads of a row: relative to the last reference
          const float m_end = c.m[r];
          c.mx[team][h][r] = m == -INFINITY ? l : l * ex2_fast(m - m_end);  // (no key: 0 or NaN)
          __syncwarp();
          if (lane == 0) mbar_arrive1(&c.sums);
          fine = fine && wait_on(&c.sums, segs & 1, dead, wait_ns);
          __syncwarp();
          if (part == 0) {
            const float sum = (c.mx[0][0][r] + c.mx[0][1][r]) + (c.mx[1][0][r] + c.mx[1][1][r]);
            c.m[r] = -INFINITY;  // (every thread of the row has read it)
            // the next segment's columns (every warp has stored the one before's)
            if (r < 16) c.odd[(segs & 1) ^ 1][(r >> 3) & 1][r & 7] = 0u;
            if (whole) {
              const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a NaN sum stays one
              c.inv[64 * rank + r] = inv;
              send4(map_to(smem_u32(&c.inv[64 * rank + r]), other), inv, bar_l);
              if (p.lse && live)
                p.lse[row] = sum == 0.f ? -INFINITY : (m_end + log2f(sum)) / kLog2e;
            } else {
              p.part_ml[slot * 128 + 64 * rank + r] = make_float2(m_end, sum);
            }
          }
        }
        float inv = 0.f;
        if (whole) {
          fine = fine && wait_on(&c.in_l, sums & 1, dead, wait_ns);
          ++sums;
          // read before `epi`: the other CTA's next sums may follow one tile of the next
          // segment, whose weights come from warps that have passed it
          if (!own) inv = c.inv[64 * g + r];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive1(&c.epi);
        fine = wait_on(&c.epi, segs & 1, dead, wait_ns) && fine;
        ++segs;
        // a team's warps leave together
        if (own ? vote_team(team, !fine) : !__all_sync(0xffffffffu, fine)) {
          ok = false;
          break;
        }
        if (whole && own && first && team == 0 && lane == 0)
          mbar_arrive_expect_tx(&c.in_l, 64 * 4);
        // a thread holds latent columns 256 rank + o0 .. of its row
        const uint32_t* cols = c.odd[(segs - 1) & 1][g] + (o0 >> 5);
        auto load_o32 = [&](int cc, float (&o)[32]) {
          tmem_ld32(tl + o0 + cc * 32, o);
          const uint32_t bits = cols[cc];
          if (bits) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if ((bits >> i) & 1u) o[i] = NAN;
          }
        };
        if (whole) {
          if (own) inv = c.inv[64 * g + r];  // (part 0's, before `epi`)
          __nv_bfloat16* dst = p.out + row * kL + 256 * rank + o0;
#pragma unroll 1
          for (int cc = 0; cc < o_n; ++cc) {
            float o[32];
            load_o32(cc, o);
            if (live) {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<uint4*>(dst + cc * 32 + q * 8) = make_uint4(
                    pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv),
                    pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                    pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                    pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
            }
          }
        } else {
          float* dst = p.part_o + ((long long)slot * 128 + 64 * g + r) * kL + 256 * rank + o0;
#pragma unroll 1
          for (int cc = 0; cc < o_n; ++cc) {
            float o[32];
            load_o32(cc, o);
            if (live) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                *reinterpret_cast<float4*>(dst + cc * 32 + q * 4) =
                    make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          }
        }
        // O is read.  (This warp's next P does not say so in time: the next segment's
        // first tile is one team's, and the other team may still be reading.)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&c.o_free);
      }
      if (!ok) hd = Header{-1, -1, 0, 0};
      if (own && first && team == 0 && lane == 0 && rank == 0) p.head[me] = hd;
    }
  } else if (warp == kTmaWarp) {
    // ================= TMA =================
    int tiles = 0, segs = 0;
    bool ok = issue, armed = false;
    // the cache row of this lane's box of a tile (-1: nothing seen, -2: no page)
    auto group_row = [&](const PairKeys& k, int b, int v) -> int {
      if (lane >= kBoxes) return -1;
      const int t0 = k.at(v, lane << kBoxLog);
      if (t0 > k.pos) return -1;
      const int blk = t0 / p.kv.page_size;
      if (blk >= p.kv.max_pages) return -2;
      const int page = __ldg(p.kv.block_table + (long long)b * p.kv.max_pages + blk);
      if (page < 0 || page >= p.kv.n_pages) return -2;
      return page * p.kv.page_size + t0 % p.kv.page_size;
    };
    while (ok && w.next()) {
      if (w.ta == w.tb) continue;
      int row = group_row(w.k, w.b, w.ta);
      const bool free_q = segs == 0 || wait_on(&c.q_empty, (segs - 1) & 1, dead, wait_ns);
      if (!__all_sync(0xffffffffu, free_q)) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&c.q_full, 4 * kQBlock);
        for (int g = 0; g < 2; ++g) {
          // (a missing second token: the first one's rows again, never used)
          const int y = p.Hm > 64 ? w.token * p.Hm + g * 64 : (w.token + (w.two ? g : 0)) * p.Hm;
          for (int blk = 0; blk < 4; ++blk)
            tma_load_2d(sb + kOffQ + blk * kQBlock + g * 8192, &q_map, 256 * rank + blk * 64, y,
                        &c.q_full);
        }
      }
      ++segs;
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        const int row_next = v + 1 < w.tb ? group_row(w.k, w.b, v + 1) : -1;
        if (row == -2) {
          flag(p.status, DSA_DEV_BAD_PAGE);
          row = -1;
        }
        const int st = tiles % kStages;
        const unsigned groups = __ballot_sync(0xffffffffu, row >= 0);
        const bool room = tiles < kStages ||
                          wait_on(&c.k_empty[st], (tiles / kStages - 1) & 1, dead, wait_ns);
        ok = __all_sync(0xffffffffu, room);
        if (!ok) break;
        if (lane == 0) {
          c.groups[st] = groups;
          mbar_arrive_expect_tx(&c.k_full[st], __popc(groups) * kBoxBytes);
        }
        armed = true;
        __syncwarp();
        if (row >= 0)
          tma_load_3d(sb + kOffK + st * kStageBytes + lane * kBoxBytes, &kv_map, 0, row,
                      4 * (int)rank, &c.k_full[st]);
        row = row_next;
      }
    }
    // after a give-up: no copy into this CTA's memory may be in flight at its end
    if (*dead && lane == 0) {
      for (int i = 1; i <= kStages; ++i)
        if (armed && tiles - i >= 0)
          mbar_wait_bounded(&c.k_full[(tiles - i) % kStages], ((tiles - i) / kStages) & 1);
      if (segs > 0) mbar_wait_bounded(&c.q_full, (segs - 1) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ================= MMA =================
    if (issue) {
      constexpr uint32_t id_s = umma_idesc_bf16(128, kKT, false);
      constexpr uint32_t id_o = umma_idesc_bf16(128, 256, false, true);
      const uint32_t qb = smem_u32(sb + kOffQ), kb = smem_u32(sb + kOffK);
      // (a descriptor's low bits are the address in 16-byte units: steps add constants)
      const uint64_t d_q = sw128_desc(qb), d_k0 = umma_desc_sw128(kb, 16, kBoxBytes),
                     d_v0 = umma_desc_sw128(kb, 1024, kBoxBytes);
      // Two streams over the same tiles: scores as soon as a stage holds keys, outputs
      // as soon as a tile's weights are there; whichever is ready goes next (outputs
      // first: they free the stage).
      PairWalk wo(p, hb, c.start, units);
      auto segment = [](PairWalk& x) {
        while (x.next())
          if (x.tb > x.ta) return true;
        return false;
      };
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_on(bar, parity, dead, wait_ns)) != 0;
      };
      auto ready = [](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test(bar, parity)) != 0;
      };
      bool ok = true, left_s = segment(w), left_o = segment(wo), have_q = false;
      int ns = 0, no = 0, vs = w.ta, vo = wo.ta, seg = 0, ends = 0;
      unsigned long long since = 0;  // time of the first idle look
      while (left_o) {
        if (no < ns && ready(&c.p_full[no % kStages], (no / kStages) & 1)) {
          const int st = no % kStages;
          const uint64_t d_v = d_v0 + (uint32_t)(st * (kStageBytes >> 4));
          const uint32_t a0 = tmem + 256 + st * kKT;
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < kKT / 16; ++s)
            umma_tmem_a_elect(tmem, a0 + s * 8, d_v + s * (2 * kBoxBytes >> 4), id_o,
                              (vo > wo.ta || s > 0) ? 1u : 0u);
          umma_commit_elect(&c.k_empty[st]);
          ++no;
          if (++vo == wo.tb) {
            umma_commit_elect(&c.o_full);
            left_o = segment(wo);
            vo = wo.ta;
            // (every warp reads the segment's outputs before the next one's first product)
            if (left_o && !wait_all(&c.o_free, ends & 1)) {
              ok = false;
              break;
            }
            ++ends;
          }
          since = 0;
          continue;
        }
        if (left_s && ns - no < kStages) {
          have_q = have_q || ready(&c.q_full, seg & 1);
          // (the stage's keys imply that its last PV is done: its scores are free)
          if (have_q && ready(&c.k_full[ns % kStages], (ns / kStages) & 1)) {
            const int st = ns % kStages;
            const uint64_t d_k = d_k0 + (uint32_t)(st * (kStageBytes >> 4));
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const uint32_t blk = j >> 2, off = (j & 3) * 32;
              umma_bf16_elect(tmem + 256 + st * kKT, d_q + ((blk * kQBlock + off) >> 4),
                              d_k + ((blk * 1024 + off) >> 4), id_s, j ? 1u : 0u);
            }
            umma_commit_elect(&c.s_full[st]);
            ++ns;
            if (++vs == w.tb) {
              umma_commit_elect(&c.q_empty);
              ++seg;
              left_s = segment(w);
              vs = w.ta;
              have_q = false;
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
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && c.dead) flag(p.status, DSA_DEV_TIMEOUT);  // outputs unspecified
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<512>(tmem);
  }
  __syncwarp();
  cluster_sync();  // neither CTA's memory goes while the other may write to it
}

// [rows, 512] as blocks of 64 columns: boxes of 8 rows of a CTA's half of the latent
// columns, 128-byte swizzle.
bool half_map(CUtensorMap* m, const void* base, uint64_t rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {64, (cuuint64_t)rows, 8};
  const cuuint64_t strides[2] = {(cuuint64_t)kL * 2, 128};
  const cuuint32_t box[3] = {64, 1u << kBoxLog, 4};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// CTA pairs that the current device holds at once (0: none; asked once per device).
int max_pairs() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];  // pairs + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return 0;
  }
  int n = known[dev].load(std::memory_order_relaxed);
  if (n > 0) return n - 1;
  n = 0;
  if (cudaFuncSetAttribute(mla_chunk_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kSmem) == cudaSuccess) {
    cudaLaunchAttribute a;
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = 2;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms() / 2 * 2, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = kSmem;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, mla_chunk_pair_kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();  // a refused query leaves no error behind
  if (n > num_sms() / 2) n = num_sms() / 2;
  known[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

bool mla_chunk_pair_ok(int Hm, int page_size) {
  return Hm > 32 && page_size % 8 == 0 && max_pairs() > 0;
}

size_t mla_chunk_pair_workspace_size() {
  const size_t pairs = num_sms() / 2;
  return pairs * 2 * 128 * (kL * 4 + 8) + pairs * sizeof(Header);
}

int launch_mla_chunk_pair(const ChunkArgs& a, void* workspace, cudaStream_t stream) {
  const int pairs = max_pairs();
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
  p.extra = 4;
  p.box_log = kBoxLog;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)pairs * 2 * 128 * kL);
  p.head = reinterpret_cast<Header*>(p.part_ml + (size_t)pairs * 2 * 128);
  CUtensorMap q_map, kv_map;
  if (!row_map(&q_map, a.q_lat, (uint64_t)a.T * a.Hm, 64) ||
      !half_map(&kv_map, a.kv.pages, (uint64_t)a.kv.n_pages * a.kv.page_size))
    return DSA_ERR_CUDA;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(mla_chunk_pair_kernel, kSmem, done)) return DSA_ERR_CUDA;
  // Not launched beside the end of the kernel before it: pairs that are placed while other
  // blocks still hold SMs run slower to their end (2,048 tokens behind 14,336: 3 % beside a
  // kernel of 304 blocks, 5 % beside one of 1,216).
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  if (launch_kernel(&cfg, mla_chunk_pair_kernel, q_map, kv_map, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2 * num_sms(), 1, 1);
  cfg.blockDim = dim3(kJoinThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  return launch_kernel(&cfg, mla_chunk_join_kernel<128, true>, p, pairs) == cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

}  // namespace dsa
