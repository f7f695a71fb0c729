// What the tensor-core kernels of the chunk attention share: the batch as units of
// work, a walk over a CTA's (or CTA pair's) share of them, the join of partials.
//
// Equal shares of the whole batch's units, whatever its lengths, keep every SM at work
// to the end; the price is that a share may begin and end inside a row tile, whose two
// or more partials (fp32, 128 KB for 64 heads) go through memory once.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "dsa_internal.cuh"
#include "umma.cuh"

#include <cudaTypedefs.h>

namespace dsa {
namespace chunk {

constexpr int kL = 512;
constexpr float kLog2e = 1.4426950408889634f;
// A head's reference is raised when a score passes it by more than this (base 2).
constexpr float kRaiseAt = 20.f;

struct Header {        // what a worker (CTA or CTA pair) left for the join
  int start_tile;      // row tile whose first units it holds but not its last (-1: none)
  int cont_tile;       // row tile that an earlier worker began (-1: none)
  int cont_some;       // it has a partial of that
  int cont_ends;       // and its last units
};

struct Params {
  PagedKv kv;
  const int32_t* cu_new;
  int T, B, Hm, window, sinks;
  float zscale;              // sm_scale in base 2
  __nv_bfloat16* out;
  float* lse;
  float* part_o;             // [2 workers][rows of a tile][kL]
  float2* part_ml;           // [2 workers][rows of a tile]
  Header* head;
  int32_t* status;
  int drill;
  int box_log;               // positions of a box, 2^box_log (copied rows: 1)
  float o_scale;             // of the partials' output against their sums
  int extra;                 // what a row tile costs beside its key tiles, in units
  int cap;                   // positions that the block table has room for
};

// Positions behind the table's width have no page: nothing is walked there, so that a
// wrong length costs no more than the table's own.
inline int table_cap(const PagedKv& kv) {
  const long long n = (long long)kv.max_pages * kv.page_size;
  return n < 0x7fffffffll ? (int)n : 0x7fffffff;
}

// ---- the batch as units ------------------------------------------------------
// A unit is one key tile of kT positions for one row tile; its queries, its first
// tile's wait and its end count as Params::extra more.  kPair: a row tile is two
// tokens and a block of 64 heads, or one token and two such blocks (Hm > 64);
// otherwise one token and a block of heads.
struct Seq {
  int c0, n, base;             // rows c0 .. c0 + n - 1 of the step; position of the first
  unsigned u;                  // units per row tile
};
template <int kT, bool kPair>
__device__ __forceinline__ Seq seq_of(int cu0, int cu1, int len, const Params& p) {
  Seq s;
  s.c0 = min(max(cu0, 0), p.T);
  s.n = max(min(cu1, p.T) - s.c0, 0);
  s.base = len < 0 ? -s.n : len - s.n;   // negative: rows before position 0
  const unsigned all = (unsigned)min(max(len, 0), p.cap);
  s.u = (all + kT - 1) / kT;
  if (p.window > 0) {
    const long long R = 1 << p.box_log;
    const long long keys =
        ((p.sinks + R - 1) / R + (R - 2 + (kPair ? 1 : 0) + p.window) / R + 1) * R;
    if ((keys + kT - 1) / kT < (long long)s.u) s.u = (unsigned)((keys + kT - 1) / kT);
  }
  s.u = max(s.u, 1u) + (unsigned)p.extra;
  return s;
}

// Visible positions [0, s0) and [lo, pos] as boxes of R = 2^log positions (aligned;
// the window's first and last may reach past it), kT / R to a key tile.  A row tile of
// two tokens holds the union of theirs.
template <int kT>
struct Keys {
  int pos, lo, s0, log, sink_boxes, first, boxes, n;
  // position of row r of key tile v (past the last box: past pos); boxes of one position
  // may number 2^31 - 1, so that the last tile's count passes an int
  __device__ __forceinline__ int at(int v, int r) const {
    const unsigned g = (unsigned)v * (unsigned)(kT >> log) + (unsigned)(r >> log);
    if (g >= (unsigned)boxes) return 0x7fffffff;
    const int box = (int)g < sink_boxes ? (int)g : first + ((int)g - sink_boxes);
    return (box << log) + (r & ((1 << log) - 1));
  }
  __device__ __forceinline__ bool sees(int t) const { return t <= pos && (t >= lo || t < s0); }
};
// pos0: the first token's position (the window begins there), pos: the last one's
template <int kT>
__device__ __forceinline__ Keys<kT> keys_of(int pos0, int pos, const Params& p) {
  Keys<kT> k;
  k.pos = min(pos, p.cap - 1);
  k.log = p.box_log;
  k.lo = p.window > 0 ? max(0, max(pos0, -1) - p.window + 1) : 0;
  k.s0 = min(min(p.sinks, k.lo), p.cap);
  k.first = k.lo >> k.log;
  k.sink_boxes = min((k.s0 >> k.log) + ((k.s0 & ((1 << k.log) - 1)) != 0), k.first);
  k.boxes = pos < 0 ? 0 : k.sink_boxes + max((k.pos >> k.log) - k.first + 1, 0);
  const unsigned per = kT >> k.log;
  k.n = (int)(((unsigned)k.boxes + per - 1) / per);
  return k;
}

// a n / u, rounded down
__device__ __forceinline__ int share_of(unsigned a, unsigned n, unsigned u) {
  if (a == 0) return 0;
  if (a == u) return (int)n;
  if ((a | n) < 65536u) return (int)(a * n / u);
  return (int)((unsigned long long)a * n / u);
}

// Where a worker's share begins (in shared memory).
struct Start {
  unsigned long long scan[32];
  int b;                       // sequence (B: no share)
  unsigned row, unit;          // row tile of it, unit of that
};

template <int kT, bool kPair>
__device__ __forceinline__ unsigned row_tiles(const Seq& s, int hb) {
  return kPair ? (hb == 2 ? (unsigned)s.n : ((unsigned)s.n + 1) / 2) : (unsigned)s.n * hb;
}

// The share of worker `me` of `workers`: returns its number of units, and fills
// *st.  With fewer units than workers the first ones take one each, so that the
// workers of a row tile are always neighbours.  Run by all kThreads threads of a CTA;
// ends with a barrier.
template <int kT, bool kPair, int kThreads>
__device__ __forceinline__ unsigned long long find_share(const Params& p, int hb, unsigned me,
                                                         unsigned workers, Start* st,
                                                         bool reports) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per),
            b1 = min(p.B, b0 + per);
  if (tid == 0) st->b = p.B;
  unsigned long long mine = 0;
  bool odd = false, past = false, falls = false;
  for (int b = b0; b < b1; ++b) {
    const int cu0 = p.cu_new[b], cu1 = p.cu_new[b + 1], len = p.kv.seq_lens[b];
    const Seq s = seq_of<kT, kPair>(cu0, cu1, len, p);
    odd |= cu0 < 0 || cu1 < cu0 || cu1 > p.T || (s.n > 0 && s.base < 0);
    past |= s.n > 0 && len > p.cap;
    falls |= cu1 < cu0;
    mine += (unsigned long long)row_tiles<kT, kPair>(s, hb) * s.u;
  }
  if (odd && reports) flag(p.status, DSA_DEV_BAD_LENGTH);
  if (past && reports) flag(p.status, DSA_DEV_BAD_PAGE);
  unsigned long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) st->scan[warp] = inc;
  // rows of several sequences at once (the work would have no bound): nothing is done
  falls = __syncthreads_or(falls);
  unsigned long long before = inc - mine, total = 0, v0, v1;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += st->scan[w];
    total += st->scan[w];
  }
  if (falls) total = 0;
  if (total < workers) {
    v0 = me < total ? me : total;
    v1 = me < total ? me + 1 : total;
  } else if (total < (1ull << 32) / 256) {  // (fewer than 256 workers: a product of 32 bits)
    v0 = (unsigned)total * me / workers;
    v1 = (unsigned)total * (me + 1) / workers;
  } else {
    v0 = total * me / workers;
    v1 = total * (me + 1) / workers;
  }
  if (v0 < v1 && v0 >= before && v0 < before + mine) {
    unsigned long long at = before;
    for (int b = b0; b < b1; ++b) {
      const Seq s = seq_of<kT, kPair>(p.cu_new[b], p.cu_new[b + 1], p.kv.seq_lens[b], p);
      const unsigned long long all = (unsigned long long)row_tiles<kT, kPair>(s, hb) * s.u;
      if (v0 < at + all) {
        const unsigned long long off = v0 - at;
        st->b = b;
        st->row = (unsigned)(off >> 32 ? off / s.u : (unsigned)off / s.u);
        st->unit = (unsigned)(off - (unsigned long long)st->row * s.u);
        break;
      }
      at += all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return v1 - v0;
}

// A walk over a worker's units, row tile by row tile.  Every role walks alone; the
// next sequence's lengths are read one sequence ahead.
template <int kT, bool kPair>
struct Walk {
  const Params& p;
  int hb;                       // head blocks per token: 1 or 2
  unsigned long long left;      // units still to do
  int b;
  unsigned row, unit;           // of sequence b: row tile, unit of it
  Seq s;
  int cu_next, len_next;        // of sequence b + 1 (its end, its length)
  // the current segment: a row tile and its key tiles [ta, tb) (none: ta == tb)
  int token, h0, tile_id, ta, tb;
  int pos0;                     // the (first) token's position; -1 and below: sees nothing
  bool two;                     // kPair: a second token follows the first
  Keys<kT> k;

  __device__ __forceinline__ Walk(const Params& pp, int hb_, const Start& st,
                                  unsigned long long n)
      : p(pp), hb(hb_), left(st.b < pp.B ? n : 0), b(st.b), row(st.row), unit(st.unit) {
    if (left == 0) return;
    s = seq_of<kT, kPair>(__ldg(p.cu_new + b), __ldg(p.cu_new + b + 1),
                          __ldg(p.kv.seq_lens + b), p);
    ahead();
  }
  __device__ __forceinline__ void ahead() {
    if (b + 1 < p.B) {
      cu_next = __ldg(p.cu_new + b + 2);
      len_next = __ldg(p.kv.seq_lens + b + 1);
    }
  }
  __device__ __forceinline__ bool next() {
    if (left == 0) return false;
    while (row >= row_tiles<kT, kPair>(s, hb)) {  // units remain: a sequence with some follows
      if (++b >= p.B) return false;               // (lengths that changed under the call)
      const int cu0 = __ldg(p.cu_new + b);
      s = seq_of<kT, kPair>(cu0, cu_next, len_next, p);
      ahead();
      row = 0;
    }
    const unsigned e = left < s.u - unit ? unit + (unsigned)left : s.u;
    const int kk = (int)(!kPair && hb == 2 ? row >> 1 : row);
    h0 = !kPair && hb == 2 ? (int)(row & 1u) : 0;
    // row tiles are taken from both ends in turn
    const int n = kPair && hb == 1 ? (s.n + 1) / 2 : s.n;
    int i = (kk & 1) ? n - 1 - (kk >> 1) : kk >> 1;
    two = false;
    if (kPair && hb == 1) {
      i *= 2;
      two = i + 1 < s.n;
    }
    token = s.c0 + i;
    tile_id = kPair ? 2 * token + (two ? 1 : 0) : token * hb + h0;
    pos0 = s.base + i;
    const int last = pos0 + (two ? 1 : 0);
    k = keys_of<kT>(pos0, last < 0 ? -1 : last, p);
    ta = share_of(unit, k.n, s.u);
    tb = share_of(e, k.n, s.u);
    left -= e - unit;
    unit = e;
    if (e == s.u) {
      unit = 0;
      ++row;
    }
    return true;
  }
};

// ---- small pieces ------------------------------------------------------------
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void fma2(float& a0, float& a1, float b, float c0, float c1) {
  unsigned long long a, bb, c;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(bb) : "f"(b));
  asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(c0), "f"(c1));
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(a) : "l"(bb), "l"(c));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  unsigned long long a, b;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(b0), "f"(b1));
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// kW values per lane (one row, kW heads) reduced over the warp's 32 rows by
// halving exchanges; lane l ends with head l mod kW.
template <int kW, bool kMax>
__device__ __forceinline__ float across_rows(float (&v)[kW], int lane) {
  if (kW == 16) {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const float o = __shfl_xor_sync(0xffffffffu, v[i], 16);
      v[i] = kMax ? fmaxf(v[i], o) : v[i] + o;
    }
  }
#pragma unroll
  for (int s = kW / 2; s >= 1; s >>= 1) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = upper ? v[i] : v[i + s];
      const float keep = upper ? v[i + s] : v[i];
      const float recv = __shfl_xor_sync(0xffffffffu, send, s);
      v[i] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  return v[0];
}

template <int kW>
__device__ __forceinline__ void tmem_ldw(uint32_t ta, float (&v)[kW]) {
  if constexpr (kW == 32) tmem_ld32(ta, v); else tmem_ld16(ta, v);
}
// Store 16 consecutive fp32 columns of the warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
template <int kW>
__device__ __forceinline__ void tmem_stw(uint32_t ta, const float (&v)[kW]) {
  if constexpr (kW == 32) tmem_st32(ta, v); else tmem_st16(ta, v);
}

// Heads of a softmax thread, of kN a row tile: half of them, but 16 at least; four warps (a
// TMEM lane quarter each) for every such group.
__host__ __device__ constexpr int heads_of(int n) { return n == 64 ? 32 : 16; }
__host__ __device__ constexpr int soft_threads(int n) { return 128 * (n / heads_of(n)); }
// Barriers of the softmax threads (barrier 0 is the CTA's).
template <int kThreads>
__device__ __forceinline__ void sync_soft() {
  asm volatile("barrier.cta.sync 1, %0;" ::"n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ bool vote_soft(bool v) {  // whether any of them says so
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, 1, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(kThreads)
      : "memory");
  return r != 0;
}

// A chunk's output columns of a thread's heads: the sum of kParts accumulators side by
// side (kN columns each; the next chunk's begin kCols on).
template <int kN, int kParts, int kCols>
__device__ __forceinline__ void load_o(uint32_t to, int mc, int hq, float (&o)[heads_of(kN)]) {
  constexpr int kW = heads_of(kN);
  const uint32_t ta = to + (uint32_t)(mc * kCols + hq * kW);
  tmem_ldw<kW>(ta, o);
#pragma unroll
  for (int k = 1; k < kParts; ++k) {
    float x[kW];
    tmem_ldw<kW>(ta + k * kN, x);
#pragma unroll
    for (int i = 0; i < kW; ++i) o[i] += x[i];
  }
}

// A segment's end, by the softmax warps (lane quarter qw, heads heads_of(kN) hq ..):
// a row tile's rows, normalised by inv[head]; O^T (kN columns a chunk of 128 latent
// columns) from TMEM at `to`.  A lane pair holds two latent columns of every head:
// each lane of the pair stores both columns of one of two heads.
template <int kN, int kParts = 1, int kCols = kN>
__device__ __forceinline__ void store_rows(const Params& p, const float* inv, uint32_t to,
                                           long long row0, int heads, int qw, int hq, int lane) {
  constexpr int kW = heads_of(kN);
  const bool upper = lane & 1;
  float iv[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) iv[i] = inv[hq * kW + i];
#pragma unroll 1
  for (int mc = 0; mc < 4; ++mc) {
    float o[kW];
    load_o<kN, kParts, kCols>(to, mc, hq, o);
    __nv_bfloat16* dst =
        p.out + (row0 + hq * kW + (upper ? 1 : 0)) * kL + mc * 128 + qw * 32 + (lane & ~1);
#pragma unroll
    for (int i = 0; i < kW; i += 2) {
      const float a = o[i] * iv[i], b = o[i + 1] * iv[i + 1];
      const float got = __shfl_xor_sync(0xffffffffu, upper ? a : b, 1);
      if (hq * kW + i + (upper ? 1 : 0) < heads)
        *reinterpret_cast<uint32_t*>(dst + (long long)i * kL) =
            upper ? pack_bf16(got, b) : pack_bf16(a, got);
    }
  }
}
// an unnormalised part of a row tile for the join (times unit[head], if given)
template <int kN, int kParts = 1, int kCols = kN>
__device__ __forceinline__ void store_part(const Params& p, int slot, uint32_t to, int heads,
                                           int qw, int hq, int lane,
                                           const float* unit = nullptr) {
  constexpr int kW = heads_of(kN);
  float* dst = p.part_o + ((long long)slot * kN + hq * kW) * kL + qw * 32 + lane;
  float iv[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) iv[i] = unit ? unit[hq * kW + i] : 1.f;
#pragma unroll 1
  for (int mc = 0; mc < 4; ++mc) {
    float o[kW];
    load_o<kN, kParts, kCols>(to, mc, hq, o);
#pragma unroll
    for (int i = 0; i < kW; ++i)
      if (hq * kW + i < heads) dst[(long long)i * kL + mc * 128] = o[i] * iv[i];
  }
}
// a token that sees nothing
template <int kThreads>
__device__ __forceinline__ void store_nothing(const Params& p, long long row0, int heads,
                                              int tid) {
  for (int i = tid; i < heads * (kL / 8); i += kThreads)
    *reinterpret_cast<uint4*>(p.out + row0 * kL + (long long)i * 8) = make_uint4(0u, 0u, 0u, 0u);
  if (p.lse && tid < heads) p.lse[row0 + tid] = -INFINITY;
}
// whether the phase has completed, without waiting
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
// A bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* dead,
                                        unsigned long long limit_ns) {
  unsigned long long t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*dead) return false;
    if (t0 == 0) t0 = global_ns();
    if (global_ns() - t0 > limit_ns) {
      *dead = 1;
      return false;
    }
  }
}

// log of the sum of 2^z, from its reference and the sum relative to it: the sum's exponent is
// added to the reference first, so that a large one against a low reference costs no digits.
__device__ __forceinline__ float lse_of(float m, float sum) {
  if (sum == 0.f) return -INFINITY;
  int ex;
  const float f = frexpf(sum, &ex);
  return (m + (float)ex + log2f(f)) / kLog2e;
}

// Join the partials of the row tiles that were split over workers, in their order.  A
// tile's workers are neighbours: every block reads all headers and lists the workers that
// began a tile.  A piece of the work is half of a row (two 16-byte pieces a lane); the
// pieces of all tiles are dealt out to the warps of two blocks an SM, so that one wave of
// blocks does it.  Where few tiles leave many partials (16,384 keys of one token: 128 of
// 128 KB) a block takes a piece and each of its warps a sixteenth of its partials.
// Bound by round trips to memory (headers, maxima and sums, partial rows) and, where
// every worker left partials, by their 128 KB a part.
constexpr int kMaxWorkers = 256;
constexpr int kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
struct Joined {
  float mx, den;
  float4 acc[2];
};
// The parts s0 .. s1 - 1 of row h, latent columns col .. and col + 128 ..: 32 workers' maxima
// and sums at once, a lane each, then four partial rows on their way at once.
template <int kRows>
__device__ __forceinline__ Joined join_parts(const Params& p, const Header* heads, int g0, int s0,
                                             int s1, int h, int col, int lane) {
  Joined j;
  j.mx = -INFINITY;
  j.den = 0.f;
  j.acc[0] = j.acc[1] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (; s0 < s1; s0 += 32) {
    const int s = s0 + lane;
    const bool part = s < s1 && (s == g0 || heads[s].cont_some);
    const int slot = s == g0 ? 2 * s + 1 : 2 * s;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (part) ml = p.part_ml[(long long)slot * kRows + h];
    const bool some = part && ml.y != 0.f;  // (a part that saw no page adds nothing)
    const float top = fmaxf(j.mx, warp_max(some ? ml.x : -INFINITY));
    const float ref = top == -INFINITY ? 0.f : top;
    const float old = ex2_fast(j.mx - ref);   // 0 before the first part
    const float wgt = some ? ex2_fast(ml.x == -INFINITY ? 0.f : ml.x - ref) : 0.f;
    j.den = j.den * old + warp_sum(some ? ml.y * wgt : 0.f);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      j.acc[q].x *= old; j.acc[q].y *= old; j.acc[q].z *= old; j.acc[q].w *= old;
    }
    j.mx = top;
    unsigned todo = __ballot_sync(0xffffffffu, some);
    while (todo) {
      float4 v[4][2];
      float wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = todo ? __ffs(todo) - 1 : -1;
        const int sl = __shfl_sync(0xffffffffu, slot, i & 31);
        wv[u] = __shfl_sync(0xffffffffu, wgt, i & 31);
        if (i < 0) wv[u] = 0.f;
        const float4* src =
            reinterpret_cast<const float4*>(p.part_o + ((long long)sl * kRows + h) * kL + col);
#pragma unroll
        for (int q = 0; q < 2; ++q)
          v[u][q] = i < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcs(src + q * 32);
        todo &= todo - 1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          j.acc[q].x = fmaf(v[u][q].x, wv[u], j.acc[q].x);
          j.acc[q].y = fmaf(v[u][q].y, wv[u], j.acc[q].y);
          j.acc[q].z = fmaf(v[u][q].z, wv[u], j.acc[q].z);
          j.acc[q].w = fmaf(v[u][q].w, wv[u], j.acc[q].w);
        }
      }
    }
  }
  return j;
}

template <int kRows, bool kPair>
__global__ void __launch_bounds__(kJoinThreads, 2)
    mla_chunk_join_kernel(const Params p, int workers) {
  __shared__ __align__(16) Header heads[kMaxWorkers];
  __shared__ int begun[kMaxWorkers], n_begun;  // workers that began a tile
  __shared__ float s_mx[kJoinWarps], s_den[kJoinWarps];
  __shared__ __align__(16) float s_acc[kJoinWarps][256];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < workers; i += kJoinThreads)
    *reinterpret_cast<int4*>(heads + i) = *reinterpret_cast<const int4*>(p.head + i);
  __syncthreads();
  if (warp == 0) {
    int n = 0;
    for (int s = 0; s < workers; s += 32) {
      const bool hit = s + lane < workers && heads[s + lane].start_tile >= 0;
      const unsigned all = __ballot_sync(0xffffffffu, hit);
      if (hit) begun[n + __popc(all & ((1u << lane) - 1))] = s + lane;
      n += __popc(all);
    }
    if (lane == 0) n_begun = n;
  }
  __syncthreads();
  const int pieces = n_begun * 2 * kRows;
  const bool wide = pieces <= 2 * (int)gridDim.x;  // a block per piece
  const int step = wide ? gridDim.x : gridDim.x * kJoinWarps;
#pragma unroll 1
  for (int i = wide ? blockIdx.x : warp * gridDim.x + blockIdx.x; i < pieces; i += step) {
    const int g0 = begun[i / (2 * kRows)], h = (i >> 1) & (kRows - 1), c0 = (i & 1) * 256;
    const int tile = heads[g0].start_tile;
    int token, head;
    if (kPair) {
      token = tile >> 1;
      head = h;
      if (p.Hm <= 64 && h >= 64) {  // the second token's rows
        if (!(tile & 1)) continue;
        ++token;
        head = h - 64;
      }
    } else {
      const int hb = (p.Hm + kRows - 1) / kRows;
      token = tile / hb;
      head = (tile - token * hb) * kRows + h;
    }
    if (head >= p.Hm) continue;
    const long long row = (long long)token * p.Hm + head;
    int n = 1;  // its workers: g0 .. g0 + n - 1
    for (unsigned stop = 0; !stop;) {
      const int s = g0 + n + lane;
      const Header hd = heads[min(s, workers - 1)];
      const bool mine = s < workers && hd.cont_tile == tile;
      stop = __ballot_sync(0xffffffffu, !mine || hd.cont_ends);
      const int k = stop ? __ffs(stop) - 1 : 32;  // before the stopping one
      n += k + (stop ? __shfl_sync(0xffffffffu, (int)mine, k & 31) : 0);
    }
    const int per = wide ? (n + kJoinWarps - 1) / kJoinWarps : n;
    const int s0 = g0 + (wide ? min(n, warp * per) : 0);
    const Joined j = join_parts<kRows>(p, heads, g0, s0, min(s0 + per, g0 + n), h,
                                       c0 + lane * 4, lane);
    if (!wide) {
      const float inv = j.den == 0.f ? 0.f : p.o_scale / j.den;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        *reinterpret_cast<uint2*>(p.out + row * kL + c0 + q * 128 + lane * 4) =
            make_uint2(pack_bf16(j.acc[q].x * inv, j.acc[q].y * inv),
                       pack_bf16(j.acc[q].z * inv, j.acc[q].w * inv));
      if (p.lse && lane == 0 && c0 == 0)
        p.lse[row] = lse_of(j.mx, j.den);
      continue;
    }
    if (lane == 0) {
      s_mx[warp] = j.mx;
      s_den[warp] = j.den;
    }
    *reinterpret_cast<float4*>(&s_acc[warp][lane * 4]) = j.acc[0];
    *reinterpret_cast<float4*>(&s_acc[warp][128 + lane * 4]) = j.acc[1];
    __syncthreads();
    if (tid < 128) {
      float mx = -INFINITY, den = 0.f, a = 0.f, b = 0.f;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) mx = fmaxf(mx, s_mx[w]);
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        // (no maximum: no part, or a NaN sum, which stays one)
        const float e = s_mx[w] == -INFINITY ? 1.f : ex2_fast(s_mx[w] - ref);
        const float2 x = *reinterpret_cast<const float2*>(&s_acc[w][tid * 2]);
        den = fmaf(s_den[w], e, den);
        a = fmaf(x.x, e, a);
        b = fmaf(x.y, e, b);
      }
      const float inv = den == 0.f ? 0.f : p.o_scale / den;
      *reinterpret_cast<uint32_t*>(p.out + row * kL + c0 + tid * 2) = pack_bf16(a * inv, b * inv);
      if (p.lse && tid == 0 && c0 == 0)
        p.lse[row] = lse_of(mx, den);
    }
    __syncthreads();
  }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// Rows of `row_bytes` bytes as 2-byte elements (an E4M3 row is 256 of them: with
// 1-byte elements the same boxes landed at a third of the rate), boxes of box_cols x
// box_rows; rows at or beyond `rows` read as zeros.
inline bool byte_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t row_bytes,
                     uint32_t box_cols, uint32_t box_rows, bool swizzle) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {row_bytes / 2, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// blocks of 128 bytes x box_rows rows, 128-byte swizzle
inline bool row_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows,
                    bool codes = false) {
  return byte_map(m, base, rows, codes ? kL : 2 * kL, 64, box_rows, true);
}
// blocks of 512 bytes x box_rows rows, to bring rows into L2
inline bool prefetch_map(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows,
                         bool codes) {
  return byte_map(m, base, rows, codes ? kL : 2 * kL, 256, box_rows, false);
}

inline int box_log_of(int page_size) {  // largest power of two that divides it, 128 at most
  int log = 0;
  while (log < 7 && page_size % (2 << log) == 0) ++log;
  return log;
}

}  // namespace chunk
}  // namespace dsa
