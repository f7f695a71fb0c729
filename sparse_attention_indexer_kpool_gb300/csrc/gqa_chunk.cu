// Attention of a grouped-query layer over the paged 8-bit cache, for chunks of many new
// tokens (bf16 activations, head dim 64 or 128): tcgen05 products of 128 query rows and 128
// keys.
//
// A row tile is 128 / G tokens of a sequence with the G query heads of one KV head: up to 128
// rows.  An item is two of them, A and B, one behind the other; a CTA runs through its equal
// share of the batch's (item, tile of 128 keys) units.  Per tile, for A and B in turn:
//   S = Q C_k^T                   fp16 in, fp32 out in tensor memory
//   e = S * (query scale * (key scale * softmax scale)) + lv - m,  w = 2^e
//   O += W C_v                    W as the first factor in tensor memory, where S was
// with the codes C widened to fp16 (exact), the query rows scaled by a power of two, lv the
// exponent of the values' scale and m a row's reference, all as in the kernel for decode
// tokens (weights times 2^2; the sums, of 2^(z - m + B), in fp32).
//
// Roles (a thread of the softmax has a whole row, so that no reduction crosses threads):
//   warps 0 - 3, 4 - 7   softmax of A, of B: S from tensor memory, W back to it
//   warps 8 - 11         widen the codes into the 128-byte swizzled fp16 tiles
//   warp 12              TMA of the codes (16 KB of keys, 16 KB of values a tile)
//   warp 13              the products: O of the last tile, then S of this one, A before B,
//                        so that the tensor cores have B's while A's softmax runs
// A row's reference stays until a sum of 16 of its weights passes 2^15 (half of fp16's
// largest): only then, and at a row's first tile, is a maximum looked for.  It is raised by whole
// numbers, so that the tile's weights that are written already follow exactly.
//
// What no row may see is masked, and its values are zeros in the tile.  Keys that some rows of an
// item see and others do not (the diagonal, a window's edge) may hold NaN codes in their
// values: those are zeros in the tile too, and the rows that see them remember which columns
// they make NaN.
//
// Measured (head dim 128, join included): 2,048 tokens behind 14,336 keys, 4 KV heads of 16 query
// heads, 973 us, 1.06 PFLOP/s.  A tile of A and B took 3,950 clocks in a trace of a form that
// needed 996 us: the products 2,064, a softmax 1,900 (a row's 128 exponentials, its thread's
// alone) and handing S and W over, of which the two row tiles cover one another's half.  16
// sequences of 1 to 250 tokens, window 1,024, 8 KV heads of 4, 85 us: ten tiles an item do not hide
// its start and end (rows in, first reference, rows out: 14,000 clocks), and an item of up to 32
// tokens has no B to run under.
#include "gqa.cuh"
#include "gqa_join.cuh"
#include "mla_chunk.cuh"
#include "umma.cuh"

namespace dsa {
namespace {

using namespace gqa;
using chunk::add2;
using chunk::fma2;
using chunk::wait_on;

constexpr int kRows = 128, kKeys = 128, kGroups = kKeys / 16;
constexpr int kSoft = 256, kWiden = 128;
constexpr int kWidenWarp = kSoft / 32, kTmaWarp = kWidenWarp + kWiden / 32,
              kMmaWarp = kTmaWarp + 1;
constexpr int kThreads = 512, kWarps = kThreads / 32;  // (the last two warps idle)
// Registers: the launch's 128 a thread, moved from the eight other warps to the softmax.
constexpr int kSoftRegs = 152, kOtherRegs = 104;
static_assert(kSoftRegs + kOtherRegs == 2 * 128, "what the launch has");
constexpr int kMetas = 4;
constexpr float kFull = 32768.f;       // a sum of 16 weights above which a reference is raised
// and from which on it is where another row of the warp has to be: the long chunk below 969 us, 974
// with 1,024, 994 where each row waits for its own (931 if none were raised)
constexpr float kHigh = 128.f;
// What an item costs, in units: a tile of it, one without rows of B, and an item beside its tiles.
constexpr int kPairCost = 4, kSingleCost = 3, kExtra = 12;

struct Params {
  GqaArgs a;
  int G, per;          // query heads of a KV head; tokens of a row tile
  float zscale;        // softmax scale in base 2
  int cap;             // positions that the block table has room for
  int box_log;         // keys of a TMA box
  float* part_o;       // [2 CTAs][2 kRows][D]
  float4* part_ml;     // [2 CTAs][2 kRows]: reference; the sum f 2^z as z and f
  Header* head;
  int drill;
};

// ---- the batch as units ---------------------------------------------------------
struct Seq {
  int c0, n, base;     // rows c0 .. c0 + n - 1 of the step; position of the first
  unsigned count;      // items of a KV head
  unsigned u, tail;    // units of an item, of the last of a head
  __device__ __forceinline__ unsigned long long units() const {  // of a head
    return count ? (unsigned long long)(count - 1) * u + tail : 0;
  }
};
__device__ __forceinline__ Seq seq_of(int cu0, int cu1, int len, const Params& p) {
  Seq s;
  const StepRows rows = rows_between(cu0, cu1, p.a.T);
  s.c0 = rows.first;
  s.n = max(rows.n, 0);
  s.base = len < 0 ? -s.n : len - s.n;  // negative: rows before position 0
  const unsigned all = (unsigned)min(max(len, 0), p.cap);
  unsigned n = (all + kKeys - 1) / kKeys;  // key tiles of an item, at most
  if (p.a.window > 0) {
    const long long R = 1 << p.box_log;
    const long long span = (long long)p.a.window + 2 * p.per - 1;
    const long long keys = ((p.a.sinks + R - 1) / R + (R - 2 + span) / R + 1) * R;
    n = (unsigned)min((long long)n, (keys + kKeys - 1) / kKeys);
  }
  n = max(n, 1u);
  const unsigned pair = 2 * p.per;
  s.count = ((unsigned)s.n + pair - 1) / pair;
  s.u = n * kPairCost + kExtra;
  s.tail = s.count * pair - (unsigned)s.n >= (unsigned)p.per ? n * kSingleCost + kExtra : s.u;
  return s;
}

struct Start {
  unsigned long long n;
  int b;
  unsigned item, unit;
};
struct Walk {
  const Params& p;
  unsigned long long left;
  int b;
  unsigned item, unit;
  Seq s;
  int token, tokens, h, id, ta, tb, n;        // the segment: tiles [ta, tb) of n
  int pos0, pos1;                             // positions of its first and last token
  int lo, s0, first, sink_boxes, boxes;       // the keys that any of them sees

  __device__ __forceinline__ Walk(const Params& pp, const Start& st)
      : p(pp), left(st.b < pp.a.B ? st.n : 0), b(st.b), item(st.item), unit(st.unit) {
    if (left > 0) load();
  }
  __device__ __forceinline__ void load() {
    s = seq_of(__ldg(p.a.cu_new + b), __ldg(p.a.cu_new + b + 1), __ldg(p.a.kv.seq_lens + b), p);
  }
  __device__ __forceinline__ bool next() {
    if (left == 0) return false;
    const int Hkv = p.a.kv.Hkv, pair = 2 * p.per;
    while (item >= s.count * Hkv) {
      if (++b >= p.a.B) return false;  // (lengths that changed under the call)
      load();
      item = 0;
    }
    h = (int)(item / s.count);
    const unsigned k = item - (unsigned)h * s.count;
    // groups are taken from both ends in turn: a share of a long prompt's units is then its
    // share of the work
    const unsigned at = (k & 1) ? s.count - 1 - (k >> 1) : k >> 1;
    const unsigned u = at == s.count - 1 ? s.tail : s.u;
    const unsigned e = left < u - unit ? unit + (unsigned)left : u;
    const int i = (int)at * pair;
    token = s.c0 + i;
    tokens = min(pair, s.n - i);
    id = token * Hkv + h;
    pos0 = s.base + i;
    pos1 = pos0 + tokens - 1;
    const int end = min(pos1, p.cap - 1);
    lo = p.a.window > 0 ? max(0, max(pos0, -1) - p.a.window + 1) : 0;
    s0 = min(min(p.a.sinks, lo), p.cap);
    first = lo >> p.box_log;
    sink_boxes = min((s0 + (1 << p.box_log) - 1) >> p.box_log, first);
    boxes = end < 0 ? 0 : sink_boxes + max((end >> p.box_log) - first + 1, 0);
    const unsigned per_tile = kKeys >> p.box_log;
    n = (int)(((unsigned)boxes + per_tile - 1) / per_tile);
    ta = share_of(unit, n, u);
    tb = share_of(e, n, u);
    left -= e - unit;
    unit = e;
    if (e == u) {
      unit = 0;
      ++item;
    }
    return true;
  }
  static __device__ __forceinline__ int share_of(unsigned a, int n, unsigned u) {
    if (a == 0) return 0;
    if (a == u) return n;
    return (int)((unsigned long long)a * (unsigned)n / u);
  }
};

struct Meta {          // of a key tile, by 16 keys
  alignas(16) int pos[kGroups];  // first position (0x7fffffff: none)
  // keys' scale times 2^-14 times the softmax scale's size: what is left to a row is the power of
  // two of its largest element, always a normal number
  alignas(16) float ks[kGroups];
  alignas(16) int ev[kGroups];    // exponent of the values' scale
  int row[kGroups];    // first cache row
  uint32_t nan[4];     // keys whose NaN values were taken out of the tile
  int least;           // least exponent of the values' scales
  int partial;         // not every row of the item sees every key
};
struct Ctl {
  uint64_t raw_full[2], raw_empty[2];      // codes of keys, of values
  uint64_t wide_full[2][2], wide_empty[2][2];  // [stage][keys, values]
  uint64_t s_full[2], p_full[2], o_full[2], q_full[2], drain;
  Meta meta[kMetas];
  Start start;
  unsigned long long scan[kWarps];
  uint32_t tmem;
  int dead;
};

template <int kD>
struct Smem {
  static constexpr int kAtoms = kD / 64, kAtom = 128 * 128;  // 128 rows of 64 fp16
  static constexpr int kTile = kAtoms * kAtom, kRaw = kKeys * kD;
  static constexpr size_t kQ = 0, kWide = 2 * (size_t)kTile;         // [stage][keys, values]
  static constexpr size_t kCodes = kWide + 4 * (size_t)kTile;
  static constexpr size_t kCtl = kCodes + 2 * (size_t)kRaw;
  static constexpr size_t kBytes = 1024 + kCtl + sizeof(Ctl);
};
static_assert(Smem<128>::kBytes <= 227 * 1024, "shared memory of a CTA");

// The share of this CTA.  Ends with a barrier.
__device__ __forceinline__ void find_share(const Params& p, Ctl& c) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.a.B;
  const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  if (tid == 0) c.start.b = B;
  unsigned long long mine = 0;
  bool odd = false, past = false, falls = false;
  for (int b = b0; b < b1; ++b) {
    const int cu0 = p.a.cu_new[b], cu1 = p.a.cu_new[b + 1], len = p.a.kv.seq_lens[b];
    const Seq s = seq_of(cu0, cu1, len, p);
    odd |= cu0 < 0 || cu1 < cu0 || cu1 > p.a.T || (s.n > 0 && s.base < 0);
    past |= s.n > 0 && len > p.cap;
    falls |= cu1 < cu0;
    mine += s.units() * p.a.kv.Hkv;
  }
  if (blockIdx.x == 0) {
    if (odd) flag(p.a.status, DSA_DEV_BAD_LENGTH);
    if (past) flag(p.a.status, DSA_DEV_BAD_PAGE);
  }
  unsigned long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) c.scan[warp] = inc;
  // rows of several sequences at once (the work would have no bound): nothing is done
  falls = __syncthreads_or(falls);
  unsigned long long before = inc - mine, total = 0, v0, v1;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += c.scan[w];
    total += c.scan[w];
  }
  if (falls) total = 0;
  const unsigned me = blockIdx.x, workers = gridDim.x;
  if (total < workers) {
    v0 = me < total ? me : total;
    v1 = me < total ? me + 1 : total;
  } else {
    v0 = total * me / workers;
    v1 = total * (me + 1) / workers;
  }
  if (v0 < v1 && v0 >= before && v0 < before + mine) {
    unsigned long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = seq_of(p.a.cu_new[b], p.a.cu_new[b + 1], p.a.kv.seq_lens[b], p);
      const unsigned long long all = s.units() * p.a.kv.Hkv;
      if (v0 < at + all) {
        unsigned long long off = v0 - at;
        c.start.b = b;
        const unsigned h = (unsigned)(off / s.units());
        off -= h * s.units();
        // a head's items: its last group is the second (the first where there is one only)
        const unsigned last = s.count > 1;
        unsigned k = 0;
        if (off >= (unsigned long long)last * s.u) {
          off -= last * s.u;
          k = last;
          if (off >= s.tail) {
            off -= s.tail;
            k = last + 1 + (unsigned)(off / s.u);
            off %= s.u;
          }
        }
        c.start.item = h * s.count + k;
        c.start.unit = (unsigned)off;
        c.start.n = v1 - v0;
        break;
      }
      at += all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// ---- small pieces -----------------------------------------------------------------
// Instruction descriptor, kind::f16: fp32 accumulator, fp16 A and B.
constexpr uint32_t idesc_f16(int m, int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(m >> 4) << 24);
}
// A from tensor memory; run by a converged warp, one elected lane issues
__device__ __forceinline__ void umma_tmem_a_elect(uint32_t d, uint32_t a, uint64_t b,
                                                  uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b32 r;\n elect.sync r|e, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 16 consecutive columns of the warp's 32 TMEM lanes: the load, and the wait behind which its
// values may be used.
__device__ __forceinline__ void tmem_ld16_start(uint32_t ta, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(ta));
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
// The same with 32 columns.
__device__ __forceinline__ void tmem_ld32_start(uint32_t ta, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta));
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}
// Store 16 consecutive columns (done behind tmem_st_wait).
__device__ __forceinline__ void tmem_st16_start(uint32_t ta, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(ta),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32_start(uint32_t ta, const uint32_t (&v)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = v[i];
    b[i] = v[16 + i];
  }
  tmem_st16_start(ta, a);
  tmem_st16_start(ta + 16, b);
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <int kD>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_chunk_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const Params p) {
  using S = Smem<kD>;
  constexpr int kTmem = 512, kOCol = 256;   // S of A at 0, of B at 128; O of A at 256, B at 384
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Ctl& c = *reinterpret_cast<Ctl*>(sb + S::kCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const GqaKv& kv = p.a.kv;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.raw_full[i], 1);
      mbar_init(&c.raw_empty[i], kWiden / 32);
      for (int j = 0; j < 2; ++j) {
        mbar_init(&c.wide_full[i][j], kWiden / 32);
        mbar_init(&c.wide_empty[i][j], 1);
      }
      mbar_init(&c.s_full[i], 1);
      mbar_init(&c.p_full[i], 4);
      mbar_init(&c.o_full[i], 1);
      mbar_init(&c.q_full[i], 4);
    }
    mbar_init(&c.drain, 1);
    fence_mbar_init();
    c.dead = 0;
  }
  if (warp == kMmaWarp) {
    tmem_alloc<kTmem>(&c.tmem);
    tc_fence_before();
  }
  pdl_wait();
  find_share(p, c);
  // behind the barrier that follows the allocation: a dependent kernel's CTA on this SM might
  // take the tensor memory that this CTA still waits for, and itself wait for this grid
  pdl_launch_dependents();
  const uint32_t tmem = c.tmem;
  Walk w(p, c.start);
  const bool issue = p.drill == 0;  // a failure drill loads and multiplies nothing
  const unsigned long long wait_ns = p.drill ? kDrillWaitNs : kWaitNs;
  volatile int* dead = &c.dead;

  // (by whole warpgroups)
  if (warp < kWidenWarp)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (warp < kWidenWarp) {
    // ================= softmax: a thread a row of A or B =================
    const int ab = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + ab * 128, to = tmem + lanes + kOCol + ab * 128;
    const int my = r / p.G, g = r - my * p.G;
    // The warp's 32 rows of Q, in pieces of 16 bytes.  Rows come in and go out through it, so that
    // neighbouring lanes have neighbouring pieces of memory.  (With cold caches an item's take
    // 4,000 to 8,000 clocks to read and 6,000 to 10,000 to write; a row to a lane 12,000 and
    // 16,000.)
    constexpr int kChunks = kD / 8, kAtOnce = 32 / kChunks, kLoads = 32 / kAtOnce;
    auto piece = [&](int row, int k) {
      return reinterpret_cast<uint4*>(sb + S::kQ + ab * S::kTile + (k >> 3) * S::kAtom +
                                      ((r & ~31) + row) * 128 + (((k & 7) ^ (row & 7)) << 4));
    };
    Header hd = {-1, -1, 0, 0};
    int tiles = 0;                // key tiles so far
    int mine = 0, outs = 0;       // those of this row tile, its segments
    bool ok = true;
    while (ok && w.next()) {
      const bool some = w.tb > w.ta, whole = w.ta == 0 && w.tb == w.n;
      const bool begins = some && w.ta == 0 && !whole;
      if (begins) {
        hd.start_item = w.id;
        hd.tokens = w.tokens;
      }
      if (!whole && !begins && hd.cont_item < 0) {
        hd.cont_item = w.id;
        hd.cont = (some ? 1 : 0) | (w.tb == w.n ? 2 : 0);
      }
      if (!some && !whole) continue;
      const int i = ab * p.per + my;              // this row's token of the item
      const bool real = my < p.per && i < w.tokens;
      const bool used = ab == 0 || w.tokens > p.per;
      // the warp's rows are rel rows behind the item's first
      const long long first_row = (long long)w.token * p.a.Hq + w.h * p.G;
      const int rel = real ? i * p.a.Hq + g : 0;
      const long long row = first_row + rel;
      if (!some) {  // nothing seen
        if (real) {
          uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + row * kD);
          for (int k = 0; k < kD / 8; ++k) out[k] = make_uint4(0u, 0u, 0u, 0u);
          if (p.a.lse) p.a.lse[row] = -INFINITY;
        }
        continue;
      }
      if (!used) {
        tiles += w.tb - w.ta;
        continue;
      }
      float qs;
      const unsigned reals = __ballot_sync(0xffffffffu, real);
      {
        // (this place's last products are done: the outputs of the last segment are out)
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.q) + first_row * kD;
        uint4 x[kLoads];
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int in_row = k * kAtOnce + lane / kChunks;
          const int at = __shfl_sync(0xffffffffu, rel, in_row);
          x[k] = make_uint4(0u, 0u, 0u, 0u);
          if ((reals >> in_row) & 1u)
            x[k] = __ldg(reinterpret_cast<const uint4*>(src + (long long)at * kD) +
                         lane % kChunks);
        }
#pragma unroll
        for (int k = 0; k < kLoads; ++k)
          *piece(k * kAtOnce + lane / kChunks, lane % kChunks) = x[k];
        __syncwarp();
        // the largest element (of bits whose order is the values')
        uint32_t top = 0u;
#pragma unroll 8
        for (int k = 0; k < kChunks; ++k) {
          const uint4 y = *piece(lane, k);
          const uint32_t u[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            top = max(max(top, u[j] & 0x7fff0000u), (u[j] & 0x7fffu) << 16);
        }
        const bool odd = top >= 0x7f800000u;  // infinities or NaN: the largest of the others
        if (odd) {
          top = 0u;
#pragma unroll 1
          for (int k = 0; k < kD; ++k) {
            const unsigned char* at = reinterpret_cast<const unsigned char*>(piece(lane, k / 8));
            const uint32_t u = (reinterpret_cast<const uint16_t*>(at)[k % 8] & 0x7fffu) << 16;
            if (u < 0x7f800000u) top = max(top, u);
          }
        }
        const int ex = max((int)(top >> 23) - 127, -126), half = (14 - ex) >> 1;
        // (a negative scale's sign goes with the query: what scores are multiplied with is
        // positive, and what is masked may be -infinity before it)
        const float up0 = copysignf(pow2(half), p.zscale), up1 = pow2(14 - ex - half);
        qs = pow2(ex);
#pragma unroll 4
        for (int k = 0; k < kChunks; ++k) {
          const uint4 y = *piece(lane, k);
          const uint32_t u[4] = {y.x, y.y, y.z, y.w};
          uint32_t z[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            z[j] = pack_f16(bf16lo(u[j]) * up0 * up1, bf16hi(u[j]) * up0 * up1);
          *piece(lane, k) = make_uint4(z[0], z[1], z[2], z[3]);
        }
        if (odd) {  // an infinity becomes NaN too: its row's logits are NaN
#pragma unroll 1
          for (int k = 0; k < kD; ++k) {
            uint16_t* at = reinterpret_cast<uint16_t*>(piece(lane, k / 8)) + k % 8;
            if ((*at & 0x7fffu) == 0x7c00u) *at = 0x7fffu;
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive1(&c.q_full[ab]);

      const int pos = real ? min(w.pos0 + i, p.cap - 1) : -1;
      const int lo = p.a.window > 0 ? max(0, max(w.pos0 + i, -1) - p.a.window + 1) : 0;
      const int s0 = min(p.a.sinks, lo);
      float m = -INFINITY, l = 0.f;
      int base = 0;
      uint32_t bad[kD / 32] = {};  // columns that a NaN value reached by the long way
#pragma unroll 1
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        ok = wait_on(&c.s_full[ab], mine++ & 1, dead, wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        Meta& mt = c.meta[tiles % kMetas];
        const bool partial = mt.partial != 0;
        // What is masked becomes -infinity, a row's first reference the largest exponent of the
        // tile.
        const bool begin = __any_sync(0xffffffffu, real && m == -INFINITY);
        if (partial || begin) {
          float top = -INFINITY;
          int at = 0;
#pragma unroll 1
          for (int j = 0; j < kGroups / 2; ++j) {
            uint32_t s[32];
            tmem_ld32_start(ts + j * 32, s);
            tmem_ld32_wait(s);
            if (partial) {
              uint32_t see = 0;
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // positions t0 .. t0 + 15: [lo, pos] and [0, s0)
                const int t0 = mt.pos[2 * j + h];
                // bits of the positions before t (0 .. 2^31 - 1, as t0 is)
                auto below = [&](int t) { return (1u << min(max(t - t0, 0), 16)) - 1u; };
                see |= (below(max(pos + 1, 0)) & (~below(lo) | below(s0)) & 0xffffu) << (16 * h);
              }
#pragma unroll
              for (int k = 0; k < 32; ++k) s[k] = (see >> k) & 1u ? s[k] : 0xff800000u;
              tmem_st32_start(ts + j * 32, s);
            }
            if (begin) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float t = __uint_as_float(s[16 * h]);
#pragma unroll
                for (int k = 1; k < 16; ++k) t = fmaxf(t, __uint_as_float(s[16 * h + k]));
                const int lv = mt.ev[2 * j + h];
                t = fmaf(t, fmaxf(qs * mt.ks[2 * j + h], 0x1p-126f), (float)lv);
                if (t > top) {
                  top = t;
                  at = lv + kUp;
                }
              }
            }
          }
          if (m == -INFINITY && top != -INFINITY) {
            m = top;
            base = at;
          }
          tmem_st_wait();
        }
        // A larger reference, by a whole number: what is there already follows exactly.
        auto raise = [&](float by, int next, int cols) {
          m += by;
          if ((float)(next - base) - by > 60.f) next = (int)floorf((float)base + by + 60.f);
          if (by == 0.f) next = base;
          // (square roots, taken twice: weights may lie further apart than a float reaches)
          const float f = ex2_fast(0.5f * ((float)(next - base) - by)), a = ex2_fast(-0.5f * by);
          base = next;
          l = l * f * f;
          __syncwarp();
          if (v > w.ta) {
#pragma unroll 1
            for (int k = 0; k < kD / 16; ++k) {
              float o[16];
              tmem_ld16(to + k * 16, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = o[j] * a * a;
              chunk::tmem_st16(to + k * 16, o);
            }
          }
          tmem_st_wait();  // (the weights before these, read back)
          // (in two steps: 2^15 to 2^-24 is more than fp16 has below 1)
          const int half = (int)by >> 1, rest = (int)by - half;
          const __half2 down0 = __float2half2_rn(by < 40.f ? pow2(-half) : 0.f);
          const __half2 down1 = __float2half2_rn(by < 40.f ? pow2(-rest) : 0.f);
#pragma unroll 1
          for (int k = 0; k < cols; ++k) {
            uint32_t y[16];
            tmem_ld16_start(ts + k * 16, y);
            tmem_ld_wait(y);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const __half2 z = __hmul2(__hmul2(*reinterpret_cast<__half2*>(&y[j]), down0), down1);
              y[j] = *reinterpret_cast<const uint32_t*>(&z);
            }
            tmem_st16_start(ts + k * 16, y);
            tmem_st_wait();
          }
        };
        // The tile in two code paths: a short one for what most tiles are (scales not far apart,
        // weights that a float holds), and one for everything, from where that one leaves off.
        // (The code has to stay small: with the rare cases in the common loop, 1.25 ms; with that
        // loop unrolled over the tile, 1.5.)
        int i = 0;
        bool far = __any_sync(0xffffffffu, base - (mt.least + kUp) > 64);
        if (!far) {
          uint32_t raw[2][32];
          tmem_ld32_start(ts, raw[0]);
#pragma unroll 1
          for (; i < kGroups / 2; i += 2) {
            uint32_t wt[2][16];
            float part[4];
            const float4 ks = *reinterpret_cast<const float4*>(mt.ks + 2 * i);
            const int4 lv = *reinterpret_cast<const int4*>(mt.ev + 2 * i);
            const float zs[4] = {fmaxf(qs * ks.x, 0x1p-126f), fmaxf(qs * ks.y, 0x1p-126f),
                                 fmaxf(qs * ks.z, 0x1p-126f), fmaxf(qs * ks.w, 0x1p-126f)};
            const float ref = m == -INFINITY ? -INFINITY : (float)kUp - m;
            const int ev[4] = {lv.x, lv.y, lv.z, lv.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              tmem_ld32_wait(raw[j]);
              if (j == 0) tmem_ld32_start(ts + (i + 1) * 32, raw[1]);
              else if (i == 0) tmem_ld32_start(ts + 64, raw[0]);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float z = zs[2 * j + h], off = (float)ev[2 * j + h] + ref;
                float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
                for (int k = 16 * h; k < 16 * h + 16; k += 4) {
                  float e[4];
#pragma unroll
                  for (int u = 0; u < 4; ++u) e[u] = __uint_as_float(raw[j][k + u]);
                  fma2(e[0], e[1], z, off, off);
                  fma2(e[2], e[3], z, off, off);
#pragma unroll
                  for (int u = 0; u < 4; ++u) e[u] = ex2_fast(e[u]);
                  add2(a0, a1, e[0], e[1]);
                  add2(b0, b1, e[2], e[3]);
                  wt[j][k / 2] = pack_f16(e[0], e[1]);
                  wt[j][k / 2 + 1] = pack_f16(e[2], e[3]);
                }
                part[2 * j + h] = (a0 + b0) + (a1 + b1);
              }
            }
            const float high = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
            if (__any_sync(0xffffffffu, high > kFull)) {
              if (i == 0) tmem_ld32_wait(raw[0]);  // (a load that nobody waited for)
              far = __any_sync(0xffffffffu, high == INFINITY);
              if (far) break;
              // These columns again.  Rows with a sum that is high at all go along with those that
              // have to: to the sum's exponent less 4, so that the largest of its 16 weights is
              // not below the reference.
              const bool up = high >= kHigh;
              int next = ev[0];
#pragma unroll
              for (int h = 1; h < 4; ++h)
                if (part[h] == high) next = ev[h];
              raise(up ? (float)((int)(__float_as_uint(high) >> 23) - 127 - kUp - 4) : 0.f,
                    next + kUp, i);
              far = __any_sync(0xffffffffu, base - (mt.least + kUp) > 64);
              if (far) break;
              tmem_ld32_start(ts + i * 32, raw[0]);
              i -= 2;
              continue;
            }
#pragma unroll
            for (int h = 0; h < 4; ++h)
              l = fmaf(part[h], pow2(max(base - kUp - ev[h], -126)), l);
            // (where scores lay that are read)
            tmem_st16_start(ts + i * 16, wt[0]);
            tmem_st16_start(ts + i * 16 + 16, wt[1]);
          }
          tmem_st_wait();
        }
        // exponents of the weights of groups 2 i and 2 i + 1
        auto exponents = [&](int i, const uint32_t (&s)[32], float (&e)[32]) {
          const float2 ks = *reinterpret_cast<const float2*>(mt.ks + 2 * i);
          const int2 lv = *reinterpret_cast<const int2*>(mt.ev + 2 * i);
          const float ref = m == -INFINITY ? -INFINITY : (float)kUp - m;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float zs = fmaxf(qs * (h ? ks.y : ks.x), 0x1p-126f);
            const float off = (float)(h ? lv.y : lv.x) + ref;
#pragma unroll
            for (int k = 16 * h; k < 16 * h + 16; k += 2) {
              e[k] = __uint_as_float(s[k]);
              e[k + 1] = __uint_as_float(s[k + 1]);
              fma2(e[k], e[k + 1], zs, off, off);
            }
          }
        };
#pragma unroll 1
        for (; i < kGroups / 2; ++i) {
          uint32_t s[32];
          float e[32], part[2];
          tmem_ld32_start(ts + i * 32, s);
          tmem_ld32_wait(s);
          exponents(i, s, e);
          uint32_t wt[16];
#pragma unroll 1
          for (bool again = false;; again = true) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float a0 = 0.f, a1 = 0.f, b0 = 0.f, b1 = 0.f;
#pragma unroll
              for (int k = 16 * h; k < 16 * h + 16; k += 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) e[k + j] = ex2_fast(e[k + j]);
                add2(a0, a1, e[k], e[k + 1]);
                add2(b0, b1, e[k + 2], e[k + 3]);
                wt[k / 2] = pack_f16(e[k], e[k + 1]);
                wt[k / 2 + 1] = pack_f16(e[k + 2], e[k + 3]);
              }
              part[h] = (a0 + b0) + (a1 + b1);
            }
            const bool high = fmaxf(part[0], part[1]) > kFull;
            if (again || !__any_sync(0xffffffffu, high)) break;
            // (an infinite weight stays one)
            uint32_t x[32];
            tmem_ld32_start(ts + i * 32, x);
            tmem_ld32_wait(x);
            exponents(i, x, e);
            float top = e[0];
#pragma unroll
            for (int k = 1; k < 32; ++k) top = fmaxf(top, e[k]);
            raise(high ? fminf(fmaxf(ceilf(top) - (float)kUp, 0.f), 4096.f) : 0.f,
                  max(mt.ev[2 * i], mt.ev[2 * i + 1]) + kUp, i);
            exponents(i, x, e);
          }
          const int2 lv = *reinterpret_cast<const int2*>(mt.ev + 2 * i);
          far = far || __any_sync(0xffffffffu, base - (mt.least + kUp) > 64);
          if (far) {  // scales far below the reference's: their weights' sum by itself
            uint32_t x[32];
            tmem_ld32_start(ts + i * 32, x);
            tmem_ld32_wait(x);
            exponents(i, x, e);
            float top0 = e[0], top1 = e[16];
#pragma unroll
            for (int k = 1; k < 16; ++k) {
              top0 = fmaxf(top0, e[k]);
              top1 = fmaxf(top1, e[16 + k]);
            }
            if (fmaxf(top0 - (float)lv.x, top1 - (float)lv.y) + (float)(base - kUp) > 100.f) {
              base -= 100;
              l *= 0x1p-100f;
            }
            const float by0 = (float)(base - kUp - lv.x), by1 = (float)(base - kUp - lv.y);
#pragma unroll
            for (int k = 0; k < 16; ++k) l += ex2_fast(e[k] + by0) + ex2_fast(e[16 + k] + by1);
            __syncwarp();
          } else {
            l = fmaf(part[0], pow2(max(base - kUp - lv.x, -126)), l);
            l = fmaf(part[1], pow2(max(base - kUp - lv.y, -126)), l);
          }
          // (where scores lay that are read)
          tmem_st16_start(ts + i * 16, wt);
        }
        tmem_st_wait();
        if (partial) {
          // (before the weights are handed on: the tile's values stay where they are till then)
          ok = wait_on(&c.wide_full[tiles & 1][1], (tiles >> 1) & 1, dead, wait_ns);
          if (ok) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q)
#pragma unroll 1
              for (uint32_t left = mt.nan[q]; left; left &= left - 1) {
                const int k = q * 32 + __ffs(left) - 1;
                const long long t = (long long)mt.pos[k >> 4] + (k & 15);
                if (!(t <= pos && (t >= lo || t < s0))) continue;
                const uint8_t* codes = kv.v_pages + ((long long)mt.row[k >> 4] + (k & 15)) * kD;
#pragma unroll 1
                for (int d = 0; d < kD; ++d)
                  if ((codes[d] & 0x7f) == 0x7f) {
#pragma unroll
                    for (int j = 0; j < kD / 32; ++j)
                      if (j == (d >> 5)) bad[j] |= 1u << (d & 31);
                  }
              }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive1(&c.p_full[ab]);
      }
      if (!ok) break;

      // the segment's end
      ok = wait_on(&c.o_full[ab], outs & 1, dead, wait_ns);
      ++outs;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      int ex = 0;
      const float f = fabsf(l) < INFINITY ? frexpf(l, &ex) : l;
      const float z = m + (float)(ex - base);  // the sum is f 2^z
      const Factor by(f, base - ex);
      const int slot = (2 * blockIdx.x + (begins ? 1 : 0)) * (2 * kRows) + ab * kRows + r;
      auto outputs = [&](int k, float (&o)[16]) {
        __syncwarp();
        tmem_ld16(to + k * 16, o);
        uint32_t nans = 0u;
#pragma unroll
        for (int j = 0; j < kD / 32; ++j)
          if (j == (k >> 1)) nans = bad[j];
        nans = nans >> ((k & 1) * 16) & 0xffffu;
        if (nans)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if ((nans >> j) & 1u) o[j] = NAN;
      };
      if (whole) {
#pragma unroll 1
        for (int k = 0; k < kD / 16; ++k) {
          float o[16];
          outputs(k, o);
          uint32_t y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = pack_bf16(by(o[2 * j]), by(o[2 * j + 1]));
          *piece(lane, 2 * k) = make_uint4(y[0], y[1], y[2], y[3]);
          *piece(lane, 2 * k + 1) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        __syncwarp();
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + first_row * kD;
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int to_row = k * kAtOnce + lane / kChunks;
          const long long at = (long long)__shfl_sync(0xffffffffu, rel, to_row) * kD;
          if ((reals >> to_row) & 1u)
            reinterpret_cast<uint4*>(out + at)[lane % kChunks] = *piece(to_row, lane % kChunks);
        }
      } else {
        float* part = p.part_o + (long long)(slot - lane) * kD;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll 1
          for (int k = 0; k < kD / 32; ++k) {
            float o[16];
            outputs(half * (kD / 32) + k, o);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *piece(lane, 4 * k + j) =
                  make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                             __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3]));
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < kLoads; ++k) {
            const int to_row = k * kAtOnce + lane / kChunks;
            if ((reals >> to_row) & 1u)
              reinterpret_cast<uint4*>(part + to_row * kD + half * (kD / 2))[lane % kChunks] =
                  *piece(to_row, lane % kChunks);
          }
          __syncwarp();
        }
      }
      if (real) {
        if (!whole)
          p.part_ml[slot] = make_float4(m, z, f, 0.f);
        else if (p.a.lse)
          p.a.lse[row] = l == 0.f ? -INFINITY : (z + log2f(f)) / kLog2e;
      }
      __syncwarp();
      tc_fence_before();  // O is read: the next segment's first weights release it
    }
    if (!ok) hd = Header{-1, -1, 0, 0};
    if (tid == 0) p.head[blockIdx.x] = hd;
  } else if (warp < kTmaWarp) {
    // ================= widen the codes =================
    const int ww = warp - kWidenWarp, z = lane >> 3, cc = lane & 3;
    int tiles = 0;
    bool ok = issue;
    while (ok && w.next()) {
      const int end = min(w.pos1, p.cap - 1);
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        const int st = tiles & 1;
        Meta& mt = c.meta[tiles % kMetas];
#pragma unroll 1
        for (int kind = 0; kind < 2; ++kind) {
          ok = wait_on(&c.raw_full[kind], tiles & 1, dead, wait_ns) &&
               (tiles < 2 ||
                wait_on(&c.wide_empty[st][kind], ((tiles >> 1) & 1) ^ 1, dead, wait_ns));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const bool partial = kind == 1 && mt.partial != 0;
          const unsigned char* raw = sb + S::kCodes + kind * S::kRaw;
          unsigned char* wide = sb + S::kWide + (2 * st + kind) * S::kTile;
#pragma unroll 4
          for (int i = ww; i < 16 * S::kAtoms; i += kWiden / 32) {
            // eight lanes: four 16-byte pieces of the rows r and r ^ 5, whose places in both
            // tiles share no bank
            const int half = i % S::kAtoms;
            const int r = i / S::kAtoms * 8 + ((lane & 4) ? z ^ 5 : z), ch = half * 4 + cc;
            uint4 x = *reinterpret_cast<const uint4*>(
                raw + (kD == 128 ? r * 128 + ((ch ^ (r & 7)) << 4)
                                 : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4)));
            if (partial) {
              const long long t = (long long)mt.pos[r >> 4] + (r & 15);
              if (!(t <= end && (t >= w.lo || t < w.s0))) x = make_uint4(0u, 0u, 0u, 0u);
              uint32_t any = 0;
              auto clean = [&](uint32_t u) -> uint32_t {  // without NaN codes
                const uint32_t n = ((u & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                any |= n;
                return u & ~((n >> 7) * 0xffu);
              };
              x = make_uint4(clean(x.x), clean(x.y), clean(x.z), clean(x.w));
              if (any) atomicOr(&mt.nan[r >> 5], 1u << (r & 31));
            }
            unsigned char* dst = wide + half * S::kAtom + r * 128;
            *reinterpret_cast<uint4*>(dst + (((2 * cc) ^ (r & 7)) << 4)) =
                make_uint4(codes2_f16(x.x & 0xffffu), codes2_f16(x.x >> 16),
                           codes2_f16(x.y & 0xffffu), codes2_f16(x.y >> 16));
            *reinterpret_cast<uint4*>(dst + (((2 * cc + 1) ^ (r & 7)) << 4)) =
                make_uint4(codes2_f16(x.z & 0xffffu), codes2_f16(x.z >> 16),
                           codes2_f16(x.w & 0xffffu), codes2_f16(x.w >> 16));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive1(&c.wide_full[st][kind]);
            mbar_arrive1(&c.raw_empty[kind]);
          }
        }
        if (!ok) break;
      }
    }
  } else if (warp == kTmaWarp) {
    // ================= TMA =================
    const int R = 1 << p.box_log;
    int tiles = 0, sent = 0;  // sent: copies of tile `tiles` under way (1: keys)
    bool ok = issue;
    // group `lane` of tile v: position (0x7fffffff: none) and cache row
    auto look_up = [&](int v, int& pos, int& row) {
      pos = 0x7fffffff;
      row = -1;
      if (lane >= kGroups || v >= w.tb) return;
      const unsigned box = (unsigned)v * (unsigned)(kKeys >> p.box_log) +
                           ((unsigned)(lane * 16) >> p.box_log);
      if (box >= (unsigned)w.boxes) return;
      const long long b = (int)box < w.sink_boxes ? (int)box : w.first + ((int)box - w.sink_boxes);
      const long long at = (b << p.box_log) + ((lane * 16) & (R - 1));
      if (at > min(w.pos1, p.cap - 1)) return;
      const int blk = (int)at / kv.page_size;
      const int page = __ldg(kv.block_table + (long long)w.b * kv.max_pages + blk);
      if (page < 0 || page >= kv.n_pages) {
        flag(p.a.status, DSA_DEV_BAD_PAGE);
        return;
      }
      pos = (int)at;
      row = (page * kv.Hkv + w.h) * kv.page_size + ((int)at - blk * kv.page_size);
    };
    while (ok && w.next()) {
      if (w.ta == w.tb) continue;
      const int lo1 = p.a.window > 0 ? max(0, max(w.pos1, -1) - p.a.window + 1) : 0;
      int pos, row;
      look_up(w.ta, pos, row);
      for (int v = w.ta; v < w.tb; ++v, ++tiles) {
        float ks = 0.f;
        int ev = 0;
        if (row >= 0) {
          const int unit = row / kv.page_size;
          ks = __ldg(kv.k_scale + unit) * 0x1p-14f * fabsf(p.zscale);
          ev = exponent_of(__ldg(kv.v_scale + unit));
        }
        int next_pos, next_row;
        look_up(v + 1, next_pos, next_row);
        // every row sees every one of the 16 keys
        const long long last = (long long)pos + 15;
        const bool full = last <= w.pos0 && (pos >= lo1 || last < p.a.sinks);
        const bool partial = __any_sync(0xffffffffu, lane < kGroups && !full);
        const int least = __reduce_min_sync(0xffffffffu, row >= 0 ? ev : kExpMax);
        const bool box = row >= 0 && ((lane * 16) & (R - 1)) == 0;
        const unsigned boxes = __ballot_sync(0xffffffffu, box);
        Meta& mt = c.meta[tiles % kMetas];
#pragma unroll
        for (int kind = 0; kind < 2; ++kind) {
          ok = tiles == 0 || wait_on(&c.raw_empty[kind], (tiles - 1) & 1, dead, wait_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (kind == 0) {
            // (the tile four before this one is done with: its values' place was asked for again
            // before the last tile's keys were widened)
            if (lane < kGroups) {
              mt.pos[lane] = pos;
              mt.ks[lane] = ks;
              mt.ev[lane] = ev;
              mt.row[lane] = row;
            }
            if (lane < 4) mt.nan[lane] = 0u;
            if (lane == 0) {
              mt.least = least;
              mt.partial = partial;
            }
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(&c.raw_full[kind], __popc(boxes) * R * kD);
          sent = kind + 1;
          __syncwarp();
          if (box)
            tma_load_2d(sb + S::kCodes + kind * S::kRaw + lane * 16 * kD, kind ? &v_map : &k_map, 0,
                        row, &c.raw_full[kind]);
        }
        if (!ok) break;
        sent = 0;
        pos = next_pos;
        row = next_row;
      }
    }
    // after a give-up: no copy into this CTA's memory may be in flight at its end
    if (*dead && lane == 0)
      for (int kind = 0; kind < 2; ++kind) {
        const int n = tiles + (sent > kind ? 1 : 0);  // copies of this kind so far
        if (n > 0) mbar_wait_bounded(&c.raw_full[kind], (n - 1) & 1);
      }
  } else if (warp == kMmaWarp && issue) {
    // ================= the products =================
    constexpr uint32_t id_s = idesc_f16(kRows, kKeys, false), id_o = idesc_f16(kRows, kD, true);
    const uint64_t d_q = sw128_desc(smem_u32(sb + S::kQ));
    const uint64_t d_k = sw128_desc(smem_u32(sb + S::kWide));
    const uint64_t d_v = umma_desc_sw128(smem_u32(sb + S::kWide) + S::kTile, S::kAtom, 1024);
    int tiles = 0;
    unsigned used_a = 0, used_b = 0, done_a = 0, done_b = 0;  // segments, tiles of A, of B
    bool ok = true;
    auto wait = [&](uint64_t* bar, unsigned parity) {
      const bool got = wait_on(bar, parity, dead, wait_ns);
      return __all_sync(0xffffffffu, got) != 0;
    };
    // O += W C_v of tile j for A or B (a segment's first: O = W C_v)
    auto outputs = [&](int ab, unsigned& done, int j, bool more) {
      if (!wait(&c.p_full[ab], done & 1) || !wait(&c.wide_full[j & 1][1], (j >> 1) & 1))
        return false;
      ++done;
      tc_fence_after();
      const uint64_t dv = d_v + (uint32_t)((j & 1) * (2 * S::kTile >> 4));
#pragma unroll
      for (int s = 0; s < kKeys / 16; ++s)
        umma_tmem_a_elect(tmem + kOCol + ab * 128, tmem + ab * 128 + s * 8, dv + (s * 2048 >> 4),
                          id_o, (s || more) ? 1u : 0u);
      return true;
    };
    auto scores = [&](int ab, int j) {
      const uint64_t dk = d_k + (uint32_t)((j & 1) * (2 * S::kTile >> 4));
      const uint64_t dq = d_q + (uint32_t)(ab * (S::kTile >> 4));
      tc_fence_after();
#pragma unroll
      for (int s = 0; s < kD / 16; ++s) {
        const uint32_t at = ((s >> 2) * S::kAtom + (s & 3) * 32) >> 4;
        // (the types stand in the descriptor)
        umma_bf16_elect(tmem + ab * 128, dq + at, dk + at, id_s, s ? 1u : 0u);
      }
      umma_commit_elect(&c.s_full[ab]);
    };
    while (ok && w.next()) {
      if (w.ta == w.tb) continue;
      const bool two = w.tokens > p.per;
      // at v: the outputs of tile v - 1 and the scores of tile v, A's and then B's
#pragma unroll 1
      for (int v = w.ta; v <= w.tb; ++v) {
        const bool first = v == w.ta, end = v == w.tb, more = v - 1 > w.ta;
        if (!end && !(ok = wait(&c.wide_full[tiles & 1][0], (tiles >> 1) & 1))) break;
        if (first ? !(ok = wait(&c.q_full[0], used_a++ & 1))
                  : !(ok = outputs(0, done_a, tiles - 1, more)))
          break;
        if (end)
          umma_commit_elect(&c.o_full[0]);
        else
          scores(0, tiles);
        if (two) {
          if (first ? !(ok = wait(&c.q_full[1], used_b++ & 1))
                    : !(ok = outputs(1, done_b, tiles - 1, more)))
            break;
          if (end)
            umma_commit_elect(&c.o_full[1]);
          else
            scores(1, tiles);
        }
        if (!first) umma_commit_elect(&c.wide_empty[(tiles - 1) & 1][1]);
        if (!end) umma_commit_elect(&c.wide_empty[tiles & 1][0]);
        tiles += !end;
      }
    }
    if (!ok) {  // drain what was issued before the CTA's memory is given back
      umma_commit_elect(&c.drain);
      mbar_wait_bounded(&c.drain, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && c.dead) flag(p.a.status, DSA_DEV_TIMEOUT);  // outputs unspecified
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<kTmem>(tmem);
  }
}

// The rows of an item (gqa_join.cuh).
struct Rows {
  static constexpr int kRows = 2 * dsa::kRows;
  int Hq, Hkv, G, per;
  __device__ __forceinline__ int used() const { return kRows; }
  __device__ __forceinline__ long long operator()(int item, int tokens, int r) const {
    const int token = item / Hkv, h = item - token * Hkv;
    const int ab = r / dsa::kRows, rr = r - ab * dsa::kRows, my = rr / G, i = ab * per + my;
    return my < per && i < tokens ? (long long)(token + i) * Hq + h * G + (rr - my * G) : -1;
  }
};

template <int kD>
int launch(const GqaArgs& a, void* workspace, cudaStream_t stream) {
  const int n_cta = num_sms();
  Params p = {};
  p.a = a;
  p.G = a.Hq / a.kv.Hkv;
  p.per = kRows / p.G;
  p.zscale = a.sm_scale * kLog2e;
  p.cap = table_cap(a.kv.max_pages, a.kv.page_size);
  p.box_log = chunk::box_log_of(a.kv.page_size);
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + (size_t)n_cta * 4 * kRows * kD);
  p.head = reinterpret_cast<Header*>(p.part_ml + (size_t)n_cta * 4 * kRows);
  p.drill = failure_drill();
  CUtensorMap k_map, v_map;
  const uint64_t rows = (uint64_t)a.kv.n_pages * a.kv.Hkv * a.kv.page_size;
  if (!code_map(&k_map, a.kv.k_pages, rows, kD, 1u << p.box_log) ||
      !code_map(&v_map, a.kv.v_pages, rows, kD, 1u << p.box_log))
    return DSA_ERR_CUDA;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(gqa_chunk_kernel<kD>, Smem<kD>::kBytes, done)) return DSA_ERR_CUDA;
  Launch l(dim3(n_cta, 1, 1), kThreads, Smem<kD>::kBytes, stream);
  if (launch_kernel(&l.cfg, gqa_chunk_kernel<kD>, k_map, v_map, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  const JoinArgs j{p.part_o, p.part_ml, p.head, n_cta, static_cast<__nv_bfloat16*>(a.out), a.lse};
  return launch_join<kD>(j, Rows{a.Hq, a.kv.Hkv, p.G, p.per}, (long long)a.T * a.kv.Hkv, stream);
}

}  // namespace

size_t gqa_chunk_workspace_size(int D) {
  return (size_t)num_sms() * (4 * kRows * (D * 4 + 16) + sizeof(Header));
}

int launch_gqa_chunk(const GqaArgs& a, void* workspace, cudaStream_t stream) {
  return a.kv.D == 128 ? launch<128>(a, workspace, stream) : launch<64>(a, workspace, stream);
}

}  // namespace dsa
