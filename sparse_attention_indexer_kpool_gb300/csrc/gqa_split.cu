// Attention of a grouped-query layer over the paged 8-bit cache, for decode tokens and for
// tokens on selected blocks (bf16 activations, head dim 64 or 128): every warp on its own
// share of the keys.
//
// A row tile is one token, one KV head and up to 8 kN of its query heads.  Per tile of 32
// keys, with the keys as the rows of the products (16 x 8 x 16, fp16 in, fp32 out):
//   S^T = C_k Q^T                 the codes of the keys, widened to fp16 (exact)
//   e = S * (query scale * (key scale * softmax scale)) + lv - m,  w = 2^e
//   O^T += C_v^T W^T              the codes of the values, widened likewise
// Query rows are scaled by a power of two to a largest magnitude in [2^14, 2^15): a bf16
// element keeps its 8 bits in fp16 down to 2^-28 of the row's largest.  lv is the exponent of the
// values' scale (a power of two), which so multiplies the weight.  The reference m of a head
// is that of z + lv, raised when a weight passes it by 2^13; weights are held times 2^2, so
// that fp16 keeps 11 bits of them down to 2^-16 of the reference and none is off by more than
// 2^-27 of it.  The sum of a head takes lv off again: it is that of 2^(z - m + B) in fp32, B
// the lv of the key that set the reference, so that scales as far apart as their exponents
// go neither overflow it nor lose a weight to it.
//
// Why like this.  A decode step reads every key and value once and computes 2 G products for
// each byte: it is bound by memory, and what counts is bytes on their way and no pause in
// them.  So no warp waits for another: each has a ring of two 8 KB tiles (32 keys and
// their values) that TMA fills in the 128-byte swizzle, runs through its share of the
// batch's tiles, and keeps scores, weights and outputs in registers: an S^T accumulator
// holds a key's row in four lanes, movmatrix turns it into the second factor of O^T, and
// a value's 16 bytes are widened in the lane that needs them.  The keys of a tile are taken in
// an order that keeps both kinds of rows free of bank conflicts.
// Shares are equal in tiles whatever the lengths; a row tile that two or more warps share
// leaves partials (fp32) that the join kernel adds in their order.
// Where a step has few row tiles of few keys, a cluster of CTAs takes each (kCluster): its warps
// share the tiles evenly, and the partials meet in (distributed) shared memory, so that no
// second kernel follows.
// Measured (head dim 128, join included): 64 tokens on 4,096 to 16,000 keys, 8 KV heads of 8 query
// heads, 212 us: 6.2 TB/s, memory-bound (the join is 8 of them).  1,024 tokens on 32 blocks of
// 64 each, 4 KV heads of 16 query heads, 318 us: 2.1 GB of codes out of L2 at 6.7 TB/s, two warps
// a scheduler, so that an instruction's latency shows.  One token on 256 keys, 8 x 8 heads, 10.4
// us: start, lengths, table, scales, one or two tiles, the cluster's exchange (under a table of 17
// blocks; under one of 4,096, whose width the host takes for the keys, shares and a join: 15).
#include <cooperative_groups.h>

#include "gqa.cuh"
#include "gqa_join.cuh"
#include "mla_chunk.cuh"
#include "umma.cuh"

namespace dsa {
namespace {

using namespace gqa;

constexpr int kW = 8, kThreads = 32 * kW;
constexpr int kKeys = 32;                      // of a tile
constexpr float kRaise = 15.f;                 // e above which a reference is raised
constexpr int kExtra = 1;                      // what a row tile costs beside its tiles, in tiles
constexpr int kLeast = 2;                      // tiles of a share, at least
// Tiles of a warp, at most, where a cluster takes a row tile; and where these are three quarters
// of the SMs.  Measured, cluster / shares in us (sequences x KV heads, 8 query heads each):
//   1 x 8 on 2,048 keys 11.1 / 14.0, 16,384 (8 tiles) 18.6 / 22.7, 32,768 (16) 26.1 / 25.4
//   2 x 2 on 2,048 11.1 / 13.1, 16,384 (8) 18.3 / 21.0, 32,768 (16) 26.7 / 24.9
//   4 x 8 on 8,192 (8) 17.6 / 24.5, 32,768 (32) 49.0 / 57.3, 65,536 (64) 87.7 / 94.3
//   16 x 8 on 2,048 (8) 16.8 / 27.5, 8,192 (32) 48.2 / 59.9
// (lengths that differ leave a cluster waiting for its longest: so no more than that)
constexpr int kMost = 12, kMostFull = 32;
// and where there are tokens enough for the chunk kernel (8 KV heads of 8 query heads, 16 tokens
// of one sequence, cluster / chunk: on 64 keys 9.4 / 17.5, on 1,500 16.1 / 24.9, on 8,000 (32)
// 40.6 / 33.5)
constexpr int kMostTogether = 16;
constexpr int kRingBytes = 2 * 2 * kKeys * 128;  // of a warp

struct Params {
  GqaArgs a;
  int G, hb;                 // query heads of a KV head, row tiles of those
  float zscale;              // softmax scale in base 2
  int cap;                   // positions that the block table has room for
  int per_block;             // boxes of a block
  float* part_o;             // [2 workers][8 kN][D]
  float4* part_ml;           // [2 workers][8 kN]: reference; the sum f 2^z as z and f
  Header* head;              // [workers]
  int workers;               // warps that take a share, at most gridDim.x * kW
  int drill;                 // a failure drill loads nothing: the first waits run out
};

// ---- the batch as tiles --------------------------------------------------------
struct Seq {
  int c0, n, base;           // rows c0 .. c0 + n - 1 of the step; position of the first
  unsigned u;                // tiles of a row tile, at most, and kExtra
};
template <int kR>
__device__ __forceinline__ Seq seq_of(int cu0, int cu1, int len, const Params& p) {
  Seq s;
  const StepRows rows = rows_between(cu0, cu1, p.a.T);
  s.c0 = rows.first;
  s.n = max(rows.n, 0);
  s.base = len < 0 ? -s.n : len - s.n;  // negative: rows before position 0
  if (p.a.block_ids) {
    s.u = (unsigned)(((long long)p.a.K * p.per_block * kR + kKeys - 1) / kKeys);
  } else {
    const unsigned all = (unsigned)min(max(len, 0), p.cap);
    s.u = (all + kKeys - 1) / kKeys;
    if (p.a.window > 0) {
      const long long boxes = (p.a.sinks + kR - 1ll) / kR + (kR - 2ll + p.a.window) / kR + 1;
      const long long most = (boxes * kR + kKeys - 1) / kKeys;
      if (most < (long long)s.u) s.u = (unsigned)most;
    }
  }
  s.u = max(s.u, 1u) + kExtra;
  return s;
}

struct Start {
  unsigned long long n;      // tiles of the share
  int b;                     // its first sequence (B: no share)
  unsigned row, unit;        // row tile of it, tile of that
};

// A row tile's part of a share.
template <int kR>
struct Walk {
  const Params& p;
  unsigned long long left;
  int b;
  unsigned row, unit;
  Seq s;
  int part, parts;                          // kCluster: this warp's part of every row tile
  int token, h, cb, tile_id, ta, tb, n;     // the segment: tiles [ta, tb) of n
  int pos, lo, s0, sink_boxes, first, boxes;  // what its token sees

  __device__ __forceinline__ Walk(const Params& pp, const Start& st, int part_, int parts_)
      : p(pp), left(st.b < pp.a.B ? st.n : 0), b(st.b), row(st.row), unit(st.unit), part(part_),
        parts(parts_) {
    if (left > 0) load();
  }
  __device__ __forceinline__ void load() {
    s = seq_of<kR>(__ldg(p.a.cu_new + b), __ldg(p.a.cu_new + b + 1), __ldg(p.a.kv.seq_lens + b),
                   p);
  }
  __device__ __forceinline__ bool next() {
    if (left == 0) return false;
    const unsigned per = (unsigned)(p.a.kv.Hkv * p.hb);
    while (row >= (unsigned)s.n * per) {
      if (++b >= p.a.B) return false;  // (lengths that changed under the call)
      load();
      row = 0;
    }
    const unsigned e = left < s.u - unit ? unit + (unsigned)left : s.u;
    const int i = (int)(row / per), rest = (int)(row - (unsigned)i * per);
    h = rest / p.hb;
    cb = rest - h * p.hb;
    token = s.c0 + i;
    tile_id = token * (int)per + rest;
    const int at = s.base + i;
    if (p.a.block_ids) {
      pos = at;
      lo = s0 = 0;
      sink_boxes = first = 0;
      boxes = at < 0 ? 0 : p.a.K * p.per_block;
    } else {
      pos = min(at, p.cap - 1);
      lo = p.a.window > 0 ? max(0, max(at, -1) - p.a.window + 1) : 0;
      s0 = min(min(p.a.sinks, lo), p.cap);
      first = lo / kR;
      sink_boxes = min((s0 + kR - 1) / kR, first);
      boxes = at < 0 ? 0 : sink_boxes + max(pos / kR - first + 1, 0);
    }
    n = (boxes * kR + kKeys - 1) / kKeys;
    if (parts > 1) {
      ta = share_of(part, n, parts);
      tb = share_of(part + 1, n, parts);
    } else {
      ta = share_of(unit, n, s.u);
      tb = share_of(e, n, s.u);
    }
    left -= e - unit;
    unit = e;
    if (e == s.u) {
      unit = 0;
      ++row;
    }
    return true;
  }
  static __device__ __forceinline__ int share_of(unsigned a, int n, unsigned u) {
    if (a == 0) return 0;
    if (a == u) return n;
    return (int)((unsigned long long)a * (unsigned)n / u);
  }
};

// The share of worker `me` for each warp of this CTA.  Ends with a barrier.
template <int kR>
__device__ __forceinline__ void find_shares(const Params& p, Start* st,
                                            unsigned long long* scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, B = p.a.B;
  const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
  const unsigned tiles = (unsigned)(p.a.kv.Hkv * p.hb);
  if (tid < kW) st[tid].b = B;
  unsigned long long mine = 0;
  bool odd = false, past = false, falls = false;
  for (int b = b0; b < b1; ++b) {
    const int cu0 = p.a.cu_new[b], cu1 = p.a.cu_new[b + 1], len = p.a.kv.seq_lens[b];
    const Seq s = seq_of<kR>(cu0, cu1, len, p);
    odd |= cu0 < 0 || cu1 < cu0 || cu1 > p.a.T || (s.n > 0 && s.base < 0);
    past |= s.n > 0 && len > p.cap;
    falls |= cu1 < cu0;
    mine += (unsigned long long)((unsigned)s.n * tiles) * s.u;
  }
  if (blockIdx.x == 0) {
    if (odd) flag(p.a.status, DSA_DEV_BAD_LENGTH);
    if (past && !p.a.block_ids) flag(p.a.status, DSA_DEV_BAD_PAGE);
  }
  unsigned long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) scan[warp] = inc;
  // rows of several sequences at once (the work would have no bound): nothing is done
  falls = __syncthreads_or(falls);
  unsigned long long before = inc - mine, total = 0;
  for (int w = 0; w < kW; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  if (falls) total = 0;
  // the shares' ends, by a thread for each warp
  if (tid < kW) {
    // neighbours in the keys are neighbours in their numbers, and few shares lie on many SMs
    const unsigned me = (unsigned)tid * gridDim.x + blockIdx.x, workers = (unsigned)p.workers;
    unsigned long long v0 = 0, v1 = 0;
    if (me < workers) {
      if (total < workers) {
        v0 = me < total ? me : total;
        v1 = me < total ? me + 1 : total;
      } else if (total < (1u << 21)) {  // (2,048 workers at most: a product of 32 bits)
        v0 = (unsigned)total * me / workers;
        v1 = (unsigned)total * (me + 1) / workers;
      } else {
        v0 = total * me / workers;
        v1 = total * (me + 1) / workers;
      }
    }
    st[tid].n = v1 - v0;
    scan[kW + tid] = v0;
  }
  __syncthreads();
  for (int w = 0; w < kW; ++w) {
    const unsigned long long v0 = scan[kW + w], v1 = v0 + st[w].n;
    if (v0 < v1 && v0 >= before && v0 < before + mine) {
      unsigned long long at = before;
      for (int b = b0; b < b1; ++b) {
        const Seq s = seq_of<kR>(p.a.cu_new[b], p.a.cu_new[b + 1], p.a.kv.seq_lens[b], p);
        const unsigned long long all = (unsigned long long)((unsigned)s.n * tiles) * s.u;
        if (v0 < at + all) {
          const unsigned long long off = v0 - at;
          st[w].b = b;
          st[w].row = (unsigned)(off >> 32 ? off / s.u : (unsigned)off / s.u);
          st[w].unit = (unsigned)(off - (unsigned long long)st[w].row * s.u);
          break;
        }
        at += all;
      }
    }
  }
  __syncthreads();
}

// kCluster: the row tile of this cluster, for all its warps; false: there is none (no row of a
// sequence, or faulty lengths).  Ends with a barrier.
template <int kR>
__device__ __forceinline__ bool find_row(const Params& p, Start* st, unsigned tile) {
  const int tid = threadIdx.x, B = p.a.B, per = p.a.kv.Hkv * p.hb;
  const int token = (int)(tile / (unsigned)per), rest = (int)tile - token * per;
  bool odd = false, past = false, falls = false;
  int below = 0;  // sequences that begin at or before the token
  for (int b = tid; b < B; b += kThreads) {
    const int cu0 = p.a.cu_new[b], cu1 = p.a.cu_new[b + 1], len = p.a.kv.seq_lens[b];
    const Seq s = seq_of<kR>(cu0, cu1, len, p);
    odd |= cu0 < 0 || cu1 < cu0 || cu1 > p.a.T || (s.n > 0 && s.base < 0);
    past |= s.n > 0 && len > p.cap;
    falls |= cu1 < cu0;
    if (token >= s.c0 && token < s.c0 + s.n) {  // (its owner: one, where cu_new does not fall)
      st->b = b;
      st->row = (unsigned)((token - s.c0) * per + rest);
      st->unit = 0;
      st->n = s.u;
      below = 1;
    }
  }
  if (blockIdx.x == 0) {
    if (odd) flag(p.a.status, DSA_DEV_BAD_LENGTH);
    if (past && !p.a.block_ids) flag(p.a.status, DSA_DEV_BAD_PAGE);
  }
  falls = __syncthreads_or(falls);
  return __syncthreads_or(below) && !falls;
}

// ---- small pieces ----------------------------------------------------------------
// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 in, fp32 out
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// an 8 x 8 matrix of fp16, a row in four lanes, transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// row of a tile that row r of the products holds (r < 8; the other eight follow alike)
__device__ __forceinline__ int key_of(int r) { return (r & 1) ? r ^ 4 : r; }
// where the 16-byte chunk c of a row of kD bytes lies in the tile
template <int kD>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return kD == 128 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// the maximum over the keys of a product's column (lanes of the same t)
__device__ __forceinline__ float across_keys(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
struct Meta {          // of a tile in the ring, by box
  int pos[2];          // first position (0x7fffffff: no such box)
  float ks[2];         // keys' scale times 2^-14 times the softmax scale: what is left to a query
                       // row is the power of two of its largest element, always a normal number
  int ev[2];           // exponent of the values' scale
};
template <int kStages>
struct Ctl {
  uint64_t full[kW][kStages];
  Meta meta[kW][kStages];
  Start start[kW];
  unsigned long long scan[2 * kW];
};
// kCluster: a CTA's sums for the others
template <int kD, int kN>
struct Shared {
  float4 ml[kW][8 * kN], cta_ml[8 * kN];   // reference; the sum f 2^z as z and f
  float cta_x[8 * kN][kD];
};

template <int kD>
constexpr int stages() { return kRingBytes / (2 * kKeys * kD); }
template <int kD, int kN, bool kCluster>
constexpr size_t smem_bytes() {
  return 1024 + (size_t)kW * kRingBytes + sizeof(Ctl<stages<kD>()>) +
         (kCluster ? 16 + sizeof(Shared<kD, kN>) : 0);
}

// kD: head dim, kN: blocks of 8 query heads, kR: keys of a TMA box (a divisor of the page)
template <int kD, int kN, int kR, bool kCluster>
__global__ void __launch_bounds__(kThreads, 1)
    gqa_split_kernel(const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map, const Params p) {
  constexpr int kStages = stages<kD>(), kBoxes = kKeys / kR;
  constexpr int kSteps = kD / 16, kM = kD / 16;   // k steps of S^T, m tiles of O^T
  constexpr int kTile = kKeys * kD;               // bytes of a tile's keys (its values follow)
  extern __shared__ __align__(16) unsigned char smem_raw[];
  unsigned char* sb = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  auto& c = *reinterpret_cast<Ctl<kStages>*>(sb + (size_t)kW * kRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const GqaKv& kv = p.a.kv;
  if (tid < kW * kStages) {  // (each thread's fence covers its own)
    mbar_init(&c.full[tid / kStages][tid % kStages], 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  namespace cg = cooperative_groups;
  const int ctas = kCluster ? (int)cg::this_cluster().num_blocks() : 1;
  const int rank = kCluster ? (int)cg::this_cluster().block_rank() : 0;
  if constexpr (kCluster) {
    if (!find_row<kR>(p, c.start, blockIdx.x / ctas)) return;  // (all CTAs of the cluster alike)
  } else {
    find_shares<kR>(p, c.start, c.scan);
  }
  const int worker = kCluster ? rank * kW + warp : warp * gridDim.x + blockIdx.x;
  const int parts = kCluster ? ctas * kW : 1;
  const Start& st = c.start[kCluster ? 0 : warp];
  Shared<kD, kN>* sh = reinterpret_cast<Shared<kD, kN>*>(
      reinterpret_cast<unsigned char*>(&c) + (sizeof(c) + 15) / 16 * 16);
  unsigned char* ring = sb + (size_t)warp * kRingBytes;
  const uint32_t ring_at = smem_u32(ring);

  // ---- the loads, kStages tiles ahead
  Walk<kR> wl(p, st, worker, parts);
  bool more = false;
  int lv = 0, held = 0;                     // next tile; first tile that the lanes hold
  int row[kBoxes], bpos[kBoxes], bev[kBoxes];
  float bks[kBoxes];
  int issued = 0;
  auto look_up = [&]() {                    // the next 32 tiles, one a lane
    held = lv;
#pragma unroll
    for (int i = 0; i < kBoxes; ++i) {
      row[i] = -1;
      bpos[i] = 0x7fffffff;
      bks[i] = 0.f;
      bev[i] = 0;
      const int box = (lv + lane) * kBoxes + i;
      if (lv + lane >= wl.tb || box >= wl.boxes) continue;
      long long at;
      if (p.a.block_ids) {
        const int j = box / p.per_block;
        const int id =
            __ldg(p.a.block_ids + ((long long)wl.token * kv.Hkv + wl.h) * p.a.K + j);
        at = id < 0 ? -1 : (long long)id * kv.page_size + (box - j * p.per_block) * kR;
      } else {
        at = (long long)(box < wl.sink_boxes ? box : wl.first + (box - wl.sink_boxes)) * kR;
      }
      if (at < 0 || at > wl.pos) continue;
      const int blk = (int)at / kv.page_size;
      const int page =
          at < p.cap ? __ldg(kv.block_table + (long long)wl.b * kv.max_pages + blk) : -1;
      if (page < 0 || page >= kv.n_pages) {
        flag(p.a.status, DSA_DEV_BAD_PAGE);
        continue;
      }
      const int unit = page * kv.Hkv + wl.h;
      row[i] = unit * kv.page_size + ((int)at - blk * kv.page_size);
      bpos[i] = (int)at;
      bks[i] = __ldg(kv.k_scale + unit) * 0x1p-14f * p.zscale;
      bev[i] = exponent_of(__ldg(kv.v_scale + unit));
    }
  };
  auto advance = [&]() {                    // to the next segment with tiles
    while ((more = wl.next()) && wl.ta == wl.tb) {}
    if (more) {
      lv = wl.ta;
      look_up();
    }
  };
  auto issue = [&]() {
    if (!more) return;
    if (lv - held == 32) look_up();
    const int src = lv - held, s = issued % kStages;
    if (lane == src && p.drill == 0) {
      Meta& m = c.meta[warp][s];
#pragma unroll
      for (int i = 0; i < kBoxes; ++i) {
        m.pos[i] = bpos[i];
        m.ks[i] = bks[i];
        m.ev[i] = bev[i];
      }
      int boxes = 0;
#pragma unroll
      for (int i = 0; i < kBoxes; ++i) boxes += row[i] >= 0;
      mbar_arrive_expect_tx(&c.full[warp][s], boxes * 2 * kR * kD);
      unsigned char* dst = ring + s * 2 * kTile;
#pragma unroll
      for (int i = 0; i < kBoxes; ++i)
        if (row[i] >= 0) {
          tma_load_2d(dst + i * kR * kD, &k_map, 0, row[i], &c.full[warp][s]);
          tma_load_2d(dst + kTile + i * kR * kD, &v_map, 0, row[i], &c.full[warp][s]);
        }
    }
    __syncwarp();
    ++issued;
    if (++lv == wl.tb) advance();
  };
  advance();
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) issue();

  // ---- the work
  Walk<kR> w(p, st, worker, parts);
  Header hd = {-1, -1, 0, 0};
  int done = 0;
  bool ok = true;
  const unsigned long long wait_ns = p.drill ? kDrillWaitNs : kWaitNs;
  while (ok && w.next()) {
    const bool some = w.tb > w.ta, whole = !kCluster && w.ta == 0 && w.tb == w.n;
    const bool begins = some && w.ta == 0 && !whole;
    if (kCluster && !some) break;  // (no part of the row tile)
    if (begins) hd.start_item = w.tile_id;
    if (!whole && !begins && hd.cont_item < 0) {
      hd.cont_item = w.tile_id;
      hd.cont = (some ? 1 : 0) | (w.tb == w.n ? 2 : 0);
    }
    if (!some && !whole) continue;
    const int head0 = w.cb * 8 * kN, heads = min(8 * kN, p.G - head0);
    const long long row0 = (long long)w.token * p.a.Hq + w.h * p.G + head0;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + row0 * kD;
    if (!some) {  // nothing seen
      for (int i = lane; i < heads * (kD / 8); i += 32)
        reinterpret_cast<uint4*>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
      if (p.a.lse)
        for (int i = lane; i < heads; i += 32) p.a.lse[row0 + i] = -INFINITY;
      continue;
    }
    // the queries: lane (g, t) holds head g's elements 16 t .. and, of 128, 64 + 16 t ..
    uint32_t q[kN][kSteps][2];
    float qs[kN][2];
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      uint4 x[kD / 64][2];
      const bool real = n * 8 + g < heads;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.q) +
                                 (row0 + (real ? n * 8 + g : 0)) * kD + 16 * t;
#pragma unroll
      for (int i = 0; i < kD / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          x[i][j] = real ? __ldg(reinterpret_cast<const uint4*>(src + 64 * i) + j)
                         : make_uint4(0u, 0u, 0u, 0u);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < kD / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = fabsf(bf16lo(u[k])), b = fabsf(bf16hi(u[k]));
            if (a < INFINITY) top = fmaxf(top, a);
            if (b < INFINITY) top = fmaxf(top, b);
          }
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max((int)(__float_as_uint(top) >> 23) - 127, -126), half = (14 - ex) >> 1;
      const float up0 = pow2(half), up1 = pow2(14 - ex - half);
#pragma unroll
      for (int i = 0; i < kD / 64; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t u[4] = {x[i][j].x, x[i][j].y, x[i][j].z, x[i][j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // a NaN or an infinity becomes NaN: its head's logits are NaN
            float a = bf16lo(u[k]) * up0 * up1, b = bf16hi(u[k]) * up0 * up1;
            a = fabsf(a) < INFINITY ? a : NAN;
            b = fabsf(b) < INFINITY ? b : NAN;
            q[n][4 * i + 2 * j + (k >> 1)][k & 1] = pack_f16(a, b);
          }
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        qs[n][j] = __shfl_sync(0xffffffffu, pow2(ex), (2 * t + j) * 4);
    }
    float o[kM][kN][4], l[kN][2], m[kN][2];
    int base[kN][2];  // B
#pragma unroll
    for (int n = 0; n < kN; ++n) {
#pragma unroll
      for (int i = 0; i < kM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][n][j] = 0.f;
      l[n][0] = l[n][1] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      base[n][0] = base[n][1] = 0;
    }
    bool unset = true;  // some head here has no reference yet

#pragma unroll 1
    for (int v = w.ta; v < w.tb; ++v, ++done) {
      const int s = done % kStages;
      ok = mbar_wait_bounded(&c.full[warp][s], (unsigned)(done / kStages) & 1u, wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const Meta& mt = c.meta[warp][s];
      const uint32_t kb = ring_at + s * 2 * kTile, vb = kb + kTile;
      bool all = true;  // every key of the tile is seen
#pragma unroll
      for (int i = 0; i < kBoxes; ++i) {
        const long long p0 = mt.pos[i], p1 = p0 + kR - 1;
        all = all && p1 <= w.pos && (p0 >= w.lo || p1 < w.s0);
      }
      auto seen = [&](int r) -> bool {
        const int i = kBoxes == 1 ? 0 : r / kR;
        const long long at = (long long)mt.pos[i] + (kBoxes == 1 ? r : r % kR);
        return at <= w.pos && (at >= w.lo || at < w.s0);
      };
      // The tile, in two forms: a short one for what most are (kPlain: every key seen, every head
      // with a reference that holds, scales not far apart), which does nothing and says so where a
      // weight is too large, and one for everything.
      auto tile = [&](auto form) -> bool {
        constexpr bool kPlain = decltype(form)::value;
        // S^T: 16 keys at a time
        float e[2][kN][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) e[j][n][i] = 0.f;
          const int r0 = 16 * j + key_of(g);
#pragma unroll
          for (int i = 0; i < kD / 64; ++i) {
            const uint4 x = lds128(kb + chunk_at<kD>(r0, 4 * i + t));
            const uint4 y = lds128(kb + chunk_at<kD>(r0 + 8, 4 * i + t));
            const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a0 = codes2_f16(xa[k] & 0xffffu), a2 = codes2_f16(xa[k] >> 16);
              const uint32_t a1 = codes2_f16(ya[k] & 0xffffu), a3 = codes2_f16(ya[k] >> 16);
#pragma unroll
              for (int n = 0; n < kN; ++n)
                mma_f16(e[j][n], a0, a1, a2, a3, q[n][4 * i + k][0], q[n][4 * i + k][1]);
            }
          }
        }
        // exponents of the weights; columns 2 t and 2 t + 1
        bool raise = !kPlain && unset;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int box = kBoxes == 1 ? 0 : j;
          const float ks = mt.ks[box], lv8 = (float)(mt.ev[box] + kUp);
          const bool see0 = kPlain || all || seen(16 * j + key_of(g));
          const bool see1 = kPlain || all || seen(16 * j + key_of(g) + 8);
          float top = -INFINITY;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float mm = m[n][i & 1], ref = !kPlain && mm == -INFINITY ? 0.f : mm;
              const float x = fmaf(e[j][n][i], qs[n][i & 1] * ks, lv8 - ref);
              e[j][n][i] = (i < 2 ? see0 : see1) ? x : -INFINITY;
              top = fmaxf(top, e[j][n][i]);
            }
          raise |= top > kRaise;
        }
        raise = __any_sync(0xffffffffu, raise);
        if (kPlain && raise) return false;
        if (!kPlain && raise) {
          unset = false;
#pragma unroll
          for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float top0 = across_keys(fmaxf(e[0][n][i], e[0][n][i + 2]));
              const float top1 = across_keys(fmaxf(e[1][n][i], e[1][n][i + 2]));
              const int lv = mt.ev[kBoxes == 2 && top1 > top0 ? 1 : 0] + kUp;
              const float rel = fmaxf(top0, top1) - (float)kUp;
              float move = 0.f;
              if (m[n][i] == -INFINITY) {  // nothing accumulated for this head yet
                if (rel != -INFINITY) {
                  m[n][i] = rel;
                  move = -rel;
                  base[n][i] = lv;
                }
              } else if (rel > kRaise - (float)kUp) {
                m[n][i] += rel;
                move = -rel;
                // (square roots, taken twice: weights may lie further apart than a float reaches)
                const float a = ex2_fast(-0.5f * rel);
                int to = lv;
                if ((float)(lv - base[n][i]) - rel > 60.f)
                  to = (int)floorf((float)base[n][i] + rel + 60.f);
                const float f = ex2_fast(0.5f * ((float)(to - base[n][i]) - rel));
                base[n][i] = to;
                l[n][i] = l[n][i] * f * f;
#pragma unroll
                for (int k = 0; k < kM; ++k) {
                  o[k][n][i] = o[k][n][i] * a * a;
                  o[k][n][i + 2] = o[k][n][i + 2] * a * a;
                }
              }
              // (an infinite maximum: its key's weight is NaN, as in the formula)
              e[0][n][i] += move;
              e[0][n][i + 2] += move;
              e[1][n][i] += move;
              e[1][n][i + 2] += move;
              unset |= m[n][i] == -INFINITY;
            }
        }
        // weights; O^T
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int box = kBoxes == 1 ? 0 : j;
          const int lv = mt.ev[box] + kUp;
          uint32_t b[kN][2];
          bool far = false;  // this box's scale lies far below the reference's
          if (!kPlain) {
#pragma unroll
            for (int n = 0; n < kN; ++n) far |= max(base[n][0], base[n][1]) - lv > 64;
            far = __any_sync(0xffffffffu, far);
          }
          if (far) {
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float d = (float)(base[n][i] - lv);
                float x = e[j][n][i] + d, y = e[j][n][i + 2] + d;
                if (across_keys(fmaxf(x, y)) > 100.f) {
                  base[n][i] -= 100;
                  l[n][i] *= 0x1p-100f;
                  x -= 100.f;
                  y -= 100.f;
                }
                l[n][i] += ex2_fast(x) + ex2_fast(y);
              }
          }
#pragma unroll
          for (int n = 0; n < kN; ++n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[j][n][i] = ex2_fast(e[j][n][i]);
            if (!far) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                l[n][i] = fmaf(e[j][n][i] + e[j][n][i + 2], pow2(max(base[n][i] - lv, -126)),
                               l[n][i]);
            }
            b[n][0] = transpose8(pack_f16(e[j][n][0], e[j][n][1]));
            b[n][1] = transpose8(pack_f16(e[j][n][2], e[j][n][3]));
          }
          // the values of four keys: of the products' k = 2 t, 2 t + 1 and eight on
          const int r0 = 16 * j + key_of(2 * t), r1 = 16 * j + key_of(2 * t + 1);
          const int rs[4] = {r0, r1, r0 + 8, r1 + 8};
          if constexpr (kD == 128) {  // lane (g, t): columns 16 g ..
            uint32_t x[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 y = lds128(vb + chunk_at<kD>(rs[i], g));
              if (!kPlain && !all && !seen(rs[i])) y = make_uint4(0u, 0u, 0u, 0u);
              x[i][0] = y.x; x[i][1] = y.y; x[i][2] = y.z; x[i][3] = y.w;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint32_t sel = u ? 0x7362u : 0x5140u;
                const uint32_t a0 = __byte_perm(x[0][k], x[1][k], sel);
                const uint32_t a1 = __byte_perm(x[0][k + 2], x[1][k + 2], sel);
                const uint32_t a2 = __byte_perm(x[2][k], x[3][k], sel);
                const uint32_t a3 = __byte_perm(x[2][k + 2], x[3][k + 2], sel);
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t f0 = codes2_f16(z ? a0 >> 16 : a0 & 0xffffu);
                  const uint32_t f1 = codes2_f16(z ? a1 >> 16 : a1 & 0xffffu);
                  const uint32_t f2 = codes2_f16(z ? a2 >> 16 : a2 & 0xffffu);
                  const uint32_t f3 = codes2_f16(z ? a3 >> 16 : a3 & 0xffffu);
#pragma unroll
                  for (int n = 0; n < kN; ++n)
                    mma_f16(o[4 * k + 2 * u + z][n], f0, f1, f2, f3, b[n][0], b[n][1]);
                }
              }
          } else {  // columns 8 g ..
            uint32_t x[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint2 y = lds64(vb + chunk_at<kD>(rs[i], g >> 1) + 8 * (g & 1));
              if (!kPlain && !all && !seen(rs[i])) y = make_uint2(0u, 0u);
              x[i][0] = y.x; x[i][1] = y.y;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t sel = u ? 0x7362u : 0x5140u;
              const uint32_t a0 = __byte_perm(x[0][0], x[1][0], sel);
              const uint32_t a1 = __byte_perm(x[0][1], x[1][1], sel);
              const uint32_t a2 = __byte_perm(x[2][0], x[3][0], sel);
              const uint32_t a3 = __byte_perm(x[2][1], x[3][1], sel);
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint32_t f0 = codes2_f16(z ? a0 >> 16 : a0 & 0xffffu);
                const uint32_t f1 = codes2_f16(z ? a1 >> 16 : a1 & 0xffffu);
                const uint32_t f2 = codes2_f16(z ? a2 >> 16 : a2 & 0xffffu);
                const uint32_t f3 = codes2_f16(z ? a3 >> 16 : a3 & 0xffffu);
#pragma unroll
                for (int n = 0; n < kN; ++n)
                  mma_f16(o[2 * u + z][n], f0, f1, f2, f3, b[n][0], b[n][1]);
              }
            }
          }
        }
        return true;
      };
      int far = 0;
#pragma unroll
      for (int n = 0; n < kN; ++n) far = max(far, max(base[n][0], base[n][1]));
      far -= (kBoxes == 1 ? mt.ev[0] : min(mt.ev[0], mt.ev[1])) + kUp;
      // (nothing there: a list's -1 entries)
      const bool none = mt.pos[0] == 0x7fffffff && mt.pos[kBoxes - 1] == 0x7fffffff;
      if ((__any_sync(0xffffffffu, !all || unset || far > 64) || !tile(std::true_type{})) && !none)
        tile(std::false_type{});
      __syncwarp();  // the tile is read
      issue();
    }
    if (!ok) break;

    // the row tile's end: lane (g, t) holds columns kD / 8 * g .. of heads 2 t and 2 t + 1
    constexpr int kC = kD / 8;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[n][i];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int col = n * 8 + 2 * t + i;
        if (col >= heads) continue;
        float x[kC];
#pragma unroll
        for (int k = 0; k < kM; ++k) {
          x[k] = o[k][n][i];
          x[kC / 2 + k] = o[k][n][i + 2];
        }
        int ex = 0;
        const float f = fabsf(sum) < INFINITY ? frexpf(sum, &ex) : sum;
        const float z = m[n][i] + (float)(ex - base[n][i]);  // the sum is f 2^z
        if (whole) {
          const Factor by(f, base[n][i] - ex);
          uint32_t y[kC / 2];
#pragma unroll
          for (int k = 0; k < kC / 2; ++k) y[k] = pack_bf16(by(x[2 * k]), by(x[2 * k + 1]));
          uint4* dst = reinterpret_cast<uint4*>(out + (long long)col * kD + kC * g);
#pragma unroll
          for (int k = 0; k < kC / 8; ++k)
            dst[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          if (p.a.lse && g == 0)
            p.a.lse[row0 + col] = sum == 0.f ? -INFINITY : (z + log2f(f)) / kLog2e;
        } else if (kCluster) {  // to where the ring was: every tile is read
          float4* dst = reinterpret_cast<float4*>(ring) + (col * kD + kC * g) / 4;
#pragma unroll
          for (int k = 0; k < kC / 4; ++k)
            dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          if (g == 0) sh->ml[warp][col] = make_float4(m[n][i], z, f, 0.f);
        } else {
          const long long slot = (long long)(2 * worker + (begins ? 1 : 0)) * (8 * kN) + col;
          float4* dst = reinterpret_cast<float4*>(p.part_o + slot * kD + kC * g);
#pragma unroll
          for (int k = 0; k < kC / 4; ++k)
            dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          if (g == 0) p.part_ml[slot] = make_float4(m[n][i], z, f, 0.f);
        }
      }
  }
  if (!ok) {  // a wait ran out: no copy into this CTA's memory may be in flight at its end
    for (; done < issued; ++done)
      mbar_wait_bounded(&c.full[warp][done % kStages], (unsigned)(done / kStages) & 1u, wait_ns);
    if (lane == 0) flag(p.a.status, DSA_DEV_TIMEOUT);
    hd = Header{-1, -1, 0, 0};
  }
  if constexpr (!kCluster) {
    if (lane == 0 && worker < p.workers) p.head[worker] = hd;
  } else {
    // the CTA's warps' partials, a head a warp, then those of the cluster's CTAs
    const int per = kv.Hkv * p.hb, tile = (int)(blockIdx.x / ctas), token = tile / per;
    const int rest = tile - token * per, h = rest / p.hb, head0 = (rest - h * p.hb) * 8 * kN;
    const int heads = min(8 * kN, p.G - head0), mine = max(w.tb - w.ta, 0);
    static_assert(8 * kN * kD * 4 <= kRingBytes, "a warp's partial takes its ring's place");
    if (mine == 0 || !ok)  // (after a give-up: no sums of whoever had the memory before)
      for (int i = lane; i < 8 * kN; i += 32)
        sh->ml[warp][i] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
    __syncthreads();
    for (int col = warp; col < heads; col += kW) {
      Joined j = nothing();
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        const float4 ml = sh->ml[i][col];
        if (ml.z == 0.f) continue;  // (a warp without a tile, or that saw no page)
        Joined x{ml.x, ml.y, ml.z, {0.f, 0.f, 0.f, 0.f}};
        load_part<kD>(x, reinterpret_cast<const float*>(sb + (size_t)i * kRingBytes) + col * kD,
                      lane);
        merge(j, x);
      }
      if (lane == 0) sh->cta_ml[col] = make_float4(j.m, j.z, j.f, 0.f);
#pragma unroll
      for (int k = 0; k < kD / 32; ++k) sh->cta_x[col][lane * (kD / 32) + k] = j.x[k];
    }
    cg::this_cluster().sync();
    for (int i = warp; i * ctas + rank < heads; i += kW) {
      const int col = i * ctas + rank;
      Joined j = nothing();
#pragma unroll 4
      for (int r = 0; r < ctas; ++r) {
        const Shared<kD, kN>* other = cg::this_cluster().map_shared_rank(sh, r);
        const float4 ml = other->cta_ml[col];
        if (ml.z == 0.f) continue;
        Joined x{ml.x, ml.y, ml.z, {0.f, 0.f, 0.f, 0.f}};
        load_part<kD>(x, other->cta_x[col], lane);
        merge(j, x);
      }
      const JoinArgs out{nullptr, nullptr, nullptr, 0, static_cast<__nv_bfloat16*>(p.a.out),
                         p.a.lse};
      store_joined<kD>(out, (long long)token * p.a.Hq + h * p.G + head0 + col, j, lane);
    }
    cg::this_cluster().sync();  // (nobody leaves while its sums are read)
  }
}

// ---- launches ----------------------------------------------------------------------
int workers_of() { return num_sms() * kW < kMaxWorkers ? num_sms() * kW : kMaxWorkers / kW * kW; }

// The heads of a row tile (gqa_join.cuh).
template <int kN>
struct Rows {
  static constexpr int kRows = 8 * kN;
  int Hq, Hkv, G, hb;
  __device__ __forceinline__ int used() const { return min(kRows, G); }
  __device__ __forceinline__ long long operator()(int tile, int, int r) const {
    const int rows = Hkv * hb, token = tile / rows, rest = tile - token * rows;
    const int h = rest / hb, head = (rest - h * hb) * kRows + r;
    return head < G ? (long long)token * Hq + h * G + head : -1;
  }
};

// Clusters of `ctas` CTAs (one an SM) that the device holds at once; asked once for each kernel
// (all of them have one type), device and size.
template <auto kKernel>
int clusters_of(size_t bytes, int ctas) {
  static std::atomic<int> held[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  std::atomic<int>& h = held[dev][ctas == 8 ? 3 : ctas == 4 ? 2 : ctas - 1];
  int n = h.load(std::memory_order_relaxed);
  if (n) return n - 1;
  Launch l(dim3(ctas, 1, 1), kThreads, bytes, nullptr);
  l.attr.id = cudaLaunchAttributeClusterDimension;
  l.attr.val.clusterDim.x = ctas;
  l.attr.val.clusterDim.y = l.attr.val.clusterDim.z = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kKernel, &l.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  h.store(n + 1, std::memory_order_relaxed);
  return n;
}

// together: only where a cluster takes a row tile and does so in few rounds (kElsewhere if not)
template <int kD, int kN, int kR>
int launch(const GqaArgs& a, void* workspace, cudaStream_t stream, bool together) {
  Params p = {};
  p.a = a;
  p.G = a.Hq / a.kv.Hkv;
  p.hb = (p.G + 8 * kN - 1) / (8 * kN);
  p.zscale = a.sm_scale * kLog2e;
  p.cap = table_cap(a.kv.max_pages, a.kv.page_size);
  p.per_block = a.kv.page_size / kR;
  p.drill = failure_drill();
  const long long row_tiles = (long long)a.T * a.kv.Hkv * p.hb;
  const long long seen = a.block_ids ? (long long)a.K * a.kv.page_size
                         : a.window > 0 && (long long)a.window + a.sinks < p.cap
                             ? (long long)a.window + a.sinks : p.cap;
  // a cluster for a row tile where the device holds all of them at once (16 of 8 CTAs are more
  // than it does: 17.7 us instead of 9.6 for as many of 4)
  auto kernel = gqa_split_kernel<kD, kN, kR, true>;
  constexpr size_t kBytes = smem_bytes<kD, kN, true>();
  int ctas = 8;
  if (row_tiles <= num_sms()) {
    static std::atomic<unsigned long long> done{0};
    if (!allow_smem(kernel, kBytes, done)) return DSA_ERR_CUDA;
    while (ctas > 1 && (row_tiles * ctas > num_sms() ||
                        row_tiles > clusters_of<gqa_split_kernel<kD, kN, kR, true>>(kBytes, ctas)))
      ctas >>= 1;
  }
  const long long all = row_tiles * ctas;
  const int most = together ? kMostTogether : all * 4 >= 3ll * num_sms() ? kMostFull : kMost;
  const bool cluster =
      row_tiles <= num_sms() && (seen + kKeys - 1) / kKeys <= (long long)most * kW * ctas;
  if (together && !cluster) return kElsewhere;
  CUtensorMap k_map, v_map;
  const uint64_t rows = (uint64_t)a.kv.n_pages * a.kv.Hkv * a.kv.page_size;
  if (!code_map(&k_map, a.kv.k_pages, rows, kD, kR) ||
      !code_map(&v_map, a.kv.v_pages, rows, kD, kR))
    return DSA_ERR_CUDA;
  if (cluster) {
    Launch l(dim3((unsigned)all, 1, 1), kThreads, kBytes, stream);
    cudaLaunchAttribute attr[2];
    attr[0] = l.attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    l.cfg.attrs = attr;
    l.cfg.numAttrs = 2;
    return launch_kernel(&l.cfg, kernel, k_map, v_map, p) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  }
  // Workers: a warp for each kLeast tiles of what the step can hold, all of them at most.
  const long long bound = row_tiles * ((seen + kKeys - 1) / kKeys + kExtra);
  const long long want = (bound + kLeast - 1) / kLeast;
  const int limit = workers_of(), workers = want < limit ? (int)want : limit;
  const int grid = workers < num_sms() ? workers : num_sms();
  p.workers = workers;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + (size_t)workers * 2 * 8 * kN * kD);
  p.head = reinterpret_cast<Header*>(p.part_ml + (size_t)workers * 2 * 8 * kN);
  auto shares = gqa_split_kernel<kD, kN, kR, false>;
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem(shares, smem_bytes<kD, kN, false>(), done)) return DSA_ERR_CUDA;
  Launch l(dim3(grid, 1, 1), kThreads, smem_bytes<kD, kN, false>(), stream);
  if (launch_kernel(&l.cfg, shares, k_map, v_map, p) != cudaSuccess) return DSA_ERR_CUDA;
  const JoinArgs j{p.part_o, p.part_ml, p.head, workers, static_cast<__nv_bfloat16*>(a.out), a.lse};
  return launch_join<kD>(j, Rows<kN>{a.Hq, a.kv.Hkv, p.G, p.hb}, row_tiles, stream);
}

// Boxes of 32 keys, or of 16 where the page is no multiple of 32: 64 decode tokens on 4,096 to
// 16,000 keys 212.5 / 214.5 us, 1,024 tokens on 32 blocks 319 / 344.
template <int kD, int kN>
int launch_r(const GqaArgs& a, void* workspace, cudaStream_t stream, bool together) {
  return a.kv.page_size % 32 == 0 ? launch<kD, kN, 32>(a, workspace, stream, together)
                                  : launch<kD, kN, 16>(a, workspace, stream, together);
}

}  // namespace

bool gqa_split_ok(int D, int dtype) { return dtype == DSA_BF16 && (D == 64 || D == 128); }

size_t gqa_split_workspace_size(int Hq, int Hkv, int D) {
  const size_t cols = Hq / Hkv <= 8 ? 8 : 16;
  return (size_t)workers_of() * (2 * cols * (D * 4 + 16) + sizeof(Header));
}

int launch_gqa_split(const GqaArgs& a, void* workspace, cudaStream_t stream, bool together) {
  const bool one = a.Hq / a.kv.Hkv <= 8;
  if (a.kv.D == 128)
    return one ? launch_r<128, 1>(a, workspace, stream, together)
               : launch_r<128, 2>(a, workspace, stream, together);
  return one ? launch_r<64, 1>(a, workspace, stream, together)
             : launch_r<64, 2>(a, workspace, stream, together);
}

}  // namespace dsa
