// The paged cache of a grouped-query layer: keys and values as E4M3 codes with one
// power of two for each block of tokens (page) and KV head.
//
// ---- Append -----------------------------------------------------------------
// For a block, a KV head, and keys and values apart, over the block's new rows x and
// the codes c of the rows before them (scale 2^e0):
//   a = max finite |x|;  e = least exponent >= -64 with a <= 448 2^e, and e0 at least
//   c <- RN(c 2^(e0 - e));  code = RN(x 2^-e);  scale = 2^e
// and, for keys, the mean of a block that is complete:
//   k_mean = RN_bf16(2^e / page_size * sum of its codes)
// A CTA takes a block of a KV head, its keys with one half of its threads and its values with
// the other.  With head dims of 64 and 128 and up to 8,192 elements a block, a thread keeps
// its 64 elements (of 4 or 8 rows' pieces of 16) in registers between the maximum and the
// conversion, all its loads in flight at once, and adds the mean's columns from them; other
// blocks are read a second time, from L1 or L2.  The sum of a block's codes is exact in fp32 up
// to 64 rows (whole multiples of 2^-9 below 2^15): the order of the additions does not count.
// Which blocks a step touches is known on the GPU only.  A sequence with n new tokens
// touches at most floor(n / page_size) + 2, so with cu its place on the step's token axis
// the slots from floor(cu / page_size) + 2 b on are its own: a CTA finds its sequence among
// them with one or two rounds of loads by all its threads (a binary search's dependent loads
// were half of a decode step's 7.9 us).
// What bounds it: memory in a chunk (65,000 tokens of 8 heads of 128 in bf16 72 us, 5.5 TB/s),
// round trips to memory in a decode step: cu_new, the lengths, the table, then rows and scale
// (64 sequences with a token each 2.9 us, 3.2 with cold caches) and, where a block becomes
// complete, its keys for the mean (6.2 to 6.9, 7.1 to 8.5): among 64 tokens one mostly does.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gqa.cuh"

namespace dsa {
namespace {

using namespace gqa;

constexpr int kThreads = 128;  // of the append, for keys and for values

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p));
  const float4 v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}
__device__ __forceinline__ void unpack8(uint2 v, float (&x)[8]) {
  const float2 a = codes2(v.x & 0xffffu), b = codes2(v.x >> 16), c = codes2(v.y & 0xffffu),
               d = codes2(v.y >> 16);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  x[4] = c.x; x[5] = c.y; x[6] = d.x; x[7] = d.y;
}
// (a value above 448 would saturate; none is, but by a wrong scale)
__device__ __forceinline__ uint2 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The place of a slot's block in step and cache; the same for all threads (ends with a barrier).
struct Place {
  bool some;                 // (false: nothing to do)
  int page;                  // as the table has it; -1: past the table
  int lo, hi;                // new rows lo .. hi - 1 of the page
  long long t0;              // row lo on the step's token axis
};
struct Lens {                // of up to 2 kThreads - 1 sequences
  int cu[2 * kThreads], len[2 * kThreads];
};
// by_token: slots are the step's tokens, and the first of a block in it (the first new one of its
// sequence, or the block's first) stands for it: fewer slots where tokens are few.
// One CTA (`first`) reports faulty boundaries and lengths of all sequences: a faulty sequence need
// not have a slot of its own.
__device__ __forceinline__ Place find_place(const int32_t* __restrict__ cu_new, int n_t, int B,
                                            const GqaKv& kv, Lens& s, bool by_token,
                                            int32_t* status, bool first) {
  const int tid = threadIdx.x, ps = kv.page_size, slot = (int)blockIdx.x;
  Place p{false, -1, 0, 0, 0};
  auto check = [&](int cu0, int cu1, int len) {
    const int n = rows_between(cu0, cu1, n_t).n;
    if (cu0 < 0 || cu1 < cu0 || cu1 > n_t || (n > 0 && len < n)) flag(status, DSA_DEV_BAD_LENGTH);
  };
  auto first_slot = [&](int cu, int b) {
    const int c = min(max(cu, 0), n_t);
    return by_token ? c : c / ps + 2 * b;
  };
  int b = 0, cu0, cu1, len;
  if (B < 2 * kThreads) {  // everything in one round
    int cu = 0;
    if (tid <= B) {
      cu = cu_new[tid];
      s.cu[tid] = cu;
      if (tid < B) s.len[tid] = kv.seq_lens[tid];
    }
    b = max(__syncthreads_count(tid < B && first_slot(cu, tid) <= slot) - 1, 0);
    cu0 = s.cu[b];
    cu1 = s.cu[b + 1];
    len = s.len[b];
    if (first && tid < B) check(cu, s.cu[tid + 1], s.len[tid]);
  } else {  // first among every `step`th, then among those between (at most 8192 / 256)
    const int step = (B + 2 * kThreads - 1) / (2 * kThreads), i = tid * step;
    b = max(__syncthreads_count(i < B && first_slot(cu_new[i], i) <= slot) - 1, 0) * step;
    const bool in = tid < step && b + tid < B;
    b += max(__syncthreads_count(in && first_slot(cu_new[b + tid], b + tid) <= slot) - 1, 0);
    cu0 = cu_new[b];
    cu1 = cu_new[b + 1];
    len = kv.seq_lens[b];
    if (first)
      for (int k = tid; k < B; k += 2 * kThreads) check(cu_new[k], cu_new[k + 1], kv.seq_lens[k]);
  }
  const StepRows mine = rows_between(cu0, cu1, n_t);
  const int c0 = mine.first, n = mine.n;
  const int i = slot - first_slot(cu0, b);
  if (n <= 0 || i < 0 || len <= 0) return p;
  const long long ctx = (long long)len - n;
  // (rows before position 0 have no place)
  const int from = (int)max(ctx, 0ll);
  int blk = from / ps + i;
  if (by_token) {
    const long long pos = ctx + i;
    if (i >= n || pos < 0) return p;
    blk = (int)pos / ps;
    if (pos != from && (int)pos != blk * ps) return p;
  }
  if ((long long)blk * ps >= len) return p;
  p.some = true;
  if (blk < kv.max_pages) p.page = __ldg(kv.block_table + (long long)b * kv.max_pages + blk);
  p.lo = max(from - blk * ps, 0);
  p.hi = (int)min((long long)ps, len - (long long)blk * ps);
  p.t0 = c0 + (long long)blk * ps + p.lo - ctx;
  return p;
}
__device__ __forceinline__ bool page_ok(int page, const GqaKv& kv, int32_t* status, bool reports) {
  const bool ok = page >= 0 && page < kv.n_pages;
  if (!ok && reports) flag(status, DSA_DEV_BAD_PAGE);
  return ok;
}

// 32 bytes: at once where the tensor begins on a multiple of them (its rows are multiples).  Two
// accesses of 16, each with gaps between the lanes, took a read of 59,400 rows from 58 to 66 us.
__device__ __forceinline__ bool is_wide(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 31) == 0;
}
__device__ __forceinline__ void load32(uint4 (&v)[2], const void* p, bool wide) {
  if (wide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x),
                   "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                 : "l"(p));
  } else {
    v[0] = ld_stream_v4(p);
    v[1] = ld_stream_v4(static_cast<const uint4*>(p) + 1);
  }
}
__device__ __forceinline__ void store32(void* p, const uint4 (&v)[2], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0].x),
                 "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
                 "r"(v[1].w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = v[0];
    static_cast<uint4*>(p)[1] = v[1];
  }
}

// Sixteen elements as they lie in memory.
template <typename T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool wide) {
    load32(v, p, wide);
  }
  __device__ __forceinline__ void clear() { v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void half(int i, float (&x)[8]) const {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = bf16lo(w[k]);
      x[2 * k + 1] = bf16hi(w[k]);
    }
  }
  // the largest magnitude (a NaN is passed over)
  __device__ __forceinline__ float top() const {
    __nv_bfloat162 m = __habs2(pair(v[0].x));
    const uint32_t w[7] = {v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
    for (int k = 0; k < 7; ++k) m = __hmax2(m, __habs2(pair(w[k])));
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t u) {
    return *reinterpret_cast<const __nv_bfloat162*>(&u);
  }
};
template <> struct Raw16<float> {
  uint4 v[4];
  __device__ __forceinline__ void load(const float* p, bool wide) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint4 w[2];
      load32(w, p + 8 * i, wide);
      v[2 * i] = w[0];
      v[2 * i + 1] = w[1];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void half(int i, float (&x)[8]) const {
    const uint32_t w[8] = {v[2 * i].x, v[2 * i].y, v[2 * i].z, v[2 * i].w,
                           v[2 * i + 1].x, v[2 * i + 1].y, v[2 * i + 1].z, v[2 * i + 1].w};
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(w[k]);
  }
  __device__ __forceinline__ float top() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x[8];
      half(i, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
    }
    return m;
  }
};

// Blocks of up to 8,192 elements: a thread's stay in registers.
template <typename T, int kD>
__global__ void __launch_bounds__(2 * kThreads, sizeof(T) == 2 ? 4 : 2)
    gqa_append_block_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                            const int32_t* __restrict__ cu_new, int n_t, int B, GqaKv kv,
                            __nv_bfloat16* __restrict__ k_mean, int32_t* status) {
  constexpr int kRowPieces = kD / 16, kStep = kThreads / kRowPieces;  // rows between a thread's
  constexpr int kMine = 4;                                            // its pieces
  __shared__ Lens s_lens;
  __shared__ float s_top[2][kThreads / 32];
  __shared__ float s_sum[kThreads / 32][kD];
  pdl_wait();
  pdl_launch_dependents();
  const int all = threadIdx.x, tid = all & (kThreads - 1), kind = all / kThreads;
  const int lane = tid & 31, warp = tid >> 5, h = blockIdx.y, ps = kv.page_size;
  const Place p =
      find_place(cu_new, n_t, B, kv, s_lens, false, status, blockIdx.x == 0 && h == 0);
  if (!p.some) return;
  const long long pitch = (long long)kv.Hkv * kD;
  const T* src = (kind ? v_new : k_new) + (p.t0 * kv.Hkv + h) * kD;
  const int r0 = tid / kRowPieces, c = (tid & (kRowPieces - 1)) * 16;
  const bool mean = kind == 0 && k_mean != nullptr && p.hi == ps;

  const bool wide = is_wide(kind ? v_new : k_new);
  Raw16<T> x[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int r = r0 + i * kStep;
    if (r >= p.lo && r < p.hi)
      x[i].load(src + (r - p.lo) * pitch + c, wide);
    else
      x[i].clear();
  }
  // (the rows are on their way beside the table's entry)
  if (!page_ok(p.page, kv, status, all == 0 && h == 0)) return;
  const long long unit = (long long)p.page * kv.Hkv + h;
  uint8_t* codes = (kind ? kv.v_pages : kv.k_pages) + unit * ps * kD;
  float* scale = (kind ? kv.v_scale : kv.k_scale) + unit;
  const int e0 = p.lo > 0 ? exponent_of(*scale) : kExpMin;  // read by all before it is written
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kMine; ++i) top = fmaxf(top, x[i].top());
  const bool infinite = top == INFINITY;
  if (infinite) {  // an infinity does not set the scale
    top = 0.f;
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[8];
        x[i].half(j, f);
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (fabsf(f[u]) < INFINITY) top = fmaxf(top, fabsf(f[u]));
      }
  }
  top = warp_max(top);
  if (lane == 0) s_top[kind][warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_top[kind][w]);
  const int e = max(exponent_for(top), e0);
  if (tid == 0) *scale = pow2(e);
  const bool moves = e > e0 && p.lo > 0;
  const float up = pow2(-e), down = pow2(max(e0 - e, -126));  // (2^-126: all zero by then)
  uint2 first[kMine];  // codes of the pieces' first halves
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // half a piece at a time, written together
    float sum[8] = {};
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = r0 + i * kStep;
      uint2* dst = reinterpret_cast<uint2*>(codes + (long long)r * kD + c);
      float f[8];
      uint2 y;
      if (r >= p.hi) continue;
      if (r >= p.lo) {
        x[i].half(j, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] *= up;
        if (infinite) {  // (a NaN stays one anyway)
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] = fabsf(f[u]) < INFINITY ? f[u] : NAN;
        }
        y = pack8(f);
      } else {  // a row before the new ones
        if (!moves && !mean) continue;
        y = dst[j];
        if (moves) {
          unpack8(y, f);
#pragma unroll
          for (int u = 0; u < 8; ++u) f[u] *= down;
          y = pack8(f);
        }
      }
      if (j == 0)
        first[i] = y;
      else if (r >= p.lo || moves)
        *reinterpret_cast<uint4*>(dst) = make_uint4(first[i].x, first[i].y, y.x, y.y);
      if (mean) {
        unpack8(y, f);
#pragma unroll
        for (int u = 0; u < 8; ++u) sum[u] += f[u];
      }
    }
    if (mean) {  // over the warp's rows
#pragma unroll
      for (int u = 0; u < 8; ++u) {
#pragma unroll
        for (int o = kRowPieces; o < 32; o <<= 1)
          sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
        if (lane < kRowPieces) s_sum[warp][c + 8 * j + u] = sum[u];
      }
    }
  }
  if (k_mean == nullptr || p.hi < ps) return;
  __syncthreads();
  if (mean && tid < kD / 2) {  // and over the warps
    const float share = pow2(e) / (float)ps;
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      a += s_sum[w][2 * tid];
      b += s_sum[w][2 * tid + 1];
    }
    *reinterpret_cast<uint32_t*>(k_mean + unit * kD + 2 * tid) = pack_bf16(a * share, b * share);
  }
}

// Blocks of any size and head dim: kLanes threads take a block's keys or values, its new rows read
// for the maximum and again for the codes.  kLanes = 32 is for steps of few tokens (decode): a
// CTA takes one token's block for several heads, a warp each, so that little of an SM is
// taken and the next kernel can be there already.
template <typename T, int kLanes>
__global__ void __launch_bounds__(2 * kThreads)
    gqa_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                      const int32_t* __restrict__ cu_new, int n_t, int B, GqaKv kv,
                      __nv_bfloat16* __restrict__ k_mean, int32_t* status) {
  constexpr int kTeams = 2 * kThreads / kLanes;
  __shared__ Lens s_lens;
  __shared__ float s_top[kTeams][kLanes / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x & (kLanes - 1), team = threadIdx.x / kLanes;
  const int which = blockIdx.y * kTeams + team, h = which >> 1, kind = which & 1;
  const int ps = kv.page_size, D = kv.D;
  const bool reports = threadIdx.x == 0 && blockIdx.y == 0;
  const Place p = find_place(cu_new, n_t, B, kv, s_lens, kLanes == 32, status,
                             blockIdx.x == 0 && blockIdx.y == 0);
  if (!p.some || !page_ok(p.page, kv, status, reports)) return;
  if (kLanes == 32 && h >= kv.Hkv) return;  // (no barrier follows for single warps)
  const int lo = p.lo, hi = p.hi;
  const long long unit = (long long)p.page * kv.Hkv + h;
  uint8_t* codes = (kind ? kv.v_pages : kv.k_pages) + unit * ps * D;
  float* scale = (kind ? kv.v_scale : kv.k_scale) + unit;
  const T* src = (kind ? v_new : k_new) + (p.t0 * kv.Hkv + h) * D;
  const int per = D / 8, pieces = (hi - lo) * per;
  const long long pitch = (long long)kv.Hkv * D;

  const int e0 = lo > 0 ? exponent_of(*scale) : kExpMin;  // read by all before it is written
  float top = 0.f;
  for (int j = tid; j < pieces; j += kLanes) {
    const int r = j / per;
    float x[8];
    load8<T>(src + r * pitch + (j - r * per) * 8, x);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (fabsf(x[u]) < INFINITY) top = fmaxf(top, fabsf(x[u]));
  }
  top = warp_max(top);
  if (kLanes > 32) {
    if ((tid & 31) == 0) s_top[team][tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kLanes / 32; ++w) top = fmaxf(top, s_top[team][w]);
  }
  const int e = max(exponent_for(top), e0);
  __syncwarp();
  if (tid == 0) *scale = pow2(e);
  if (e > e0 && lo > 0) {
    const float down = pow2(max(e0 - e, -126));  // (2^-126: all zero by then)
    for (int j = tid; j < lo * per; j += kLanes) {
      uint2* q = reinterpret_cast<uint2*>(codes) + j;
      float x[8];
      unpack8(*q, x);
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] *= down;
      *q = pack8(x);
    }
  }
  const float up = pow2(-e);
  for (int j = tid; j < pieces; j += kLanes) {
    const int r = j / per, c = (j - r * per) * 8;
    float x[8];
    load8<T>(src + r * pitch + c, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = fabsf(x[u]) < INFINITY ? x[u] * up : NAN;
    *reinterpret_cast<uint2*>(codes + (long long)(lo + r) * D + c) = pack8(x);
  }
  if (k_mean == nullptr || hi < ps) return;
  // the block's codes are written
  if (kLanes > 32) __syncthreads(); else __syncwarp();
  if (kind) return;
  // a warp's lanes: 16 columns c of every `step`th row, eight rows on their way at once
  const float share = pow2(e) / (float)ps;
  const int cols = D / 16, step = 32 / cols, lane = tid & 31;
  if (tid >= 32) return;
  const int c = lane % cols, r0 = lane / cols;
  float sum[16] = {};
#pragma unroll 8
  for (int r = r0; r < ps; r += step) {
    if (r0 >= step) break;  // (lanes behind the last whole row)
    const uint4 y = *reinterpret_cast<const uint4*>(codes + (long long)r * D + c * 16);
    float f[8];
    unpack8(make_uint2(y.x, y.y), f);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] += f[u];
    unpack8(make_uint2(y.z, y.w), f);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[8 + u] += f[u];
  }
  __syncwarp();
  for (int g = 1; g < step; ++g) {  // the rows' groups, in their order
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      const float other = __shfl_sync(0xffffffffu, sum[u], (g * cols + c) & 31);
      if (r0 == 0) sum[u] += other;
    }
  }
  if (r0 == 0) {
    uint32_t w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = pack_bf16(sum[2 * u] * share, sum[2 * u + 1] * share);
    uint4* dst = reinterpret_cast<uint4*>(k_mean + unit * D + c * 16);
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ---- Read-back ----------------------------------------------------------------
// value = code * scale.  A CTA takes 16 rows of the outputs, finds their sequences and
// pages once, and walks over their (KV head, 16 codes) pieces: 16 bytes in, 32 or 64 out a
// thread and step, two steps' loads at once.  59,400 rows of 8 heads of 128 in bf16: 57.7 us,
// 6.3 TB/s (one step at a time 65, with 16-byte stores 66; 32 and 64 rows 58 and 59.5); 1,001
// rows of 4 heads 3.4 us (with 64 rows a CTA 5.4).
constexpr int kReadRows = 16, kReadThreads = 256;

// wide: 32 bytes at once (p is a multiple of them)
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16], bool wide);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[16],
                                                       bool wide) {
  uint4 w[2];
  w[0] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
  w[1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]),
                    pack_bf16(x[14], x[15]));
  store32(p, w, wide);
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&x)[16], bool wide) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint4 w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = make_uint4(__float_as_uint(x[8 * i + 4 * k]), __float_as_uint(x[8 * i + 4 * k + 1]),
                        __float_as_uint(x[8 * i + 4 * k + 2]),
                        __float_as_uint(x[8 * i + 4 * k + 3]));
    store32(p + 8 * i, w, wide);
  }
}

template <typename T>
__global__ void __launch_bounds__(kReadThreads)
    gqa_read_kernel(GqaKv kv, const int32_t* __restrict__ cu_out,
                    const int32_t* __restrict__ begin, int n_t, int B, T* __restrict__ k_out,
                    T* __restrict__ v_out, int32_t* status) {
  __shared__ int s_page[kReadRows], s_off[kReadRows];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, t_first = blockIdx.x * kReadRows;
  if (tid < kReadRows) {
    const int t = t_first + tid;
    int page = -2, off = 0;  // -2: left as it was, -1: zeros
    if (t < n_t) {
      const int b = sequence_of(cu_out, B, t);
      const int c0 = max(cu_out[b], 0), c1 = min(cu_out[b + 1], n_t);
      if (t >= c0 && t < c1) {
        const long long pos = (long long)t - cu_out[b] + (begin ? begin[b] : 0);
        page = -1;
        if (pos < 0 || pos >= kv.seq_lens[b]) {
          flag(status, DSA_DEV_BAD_LENGTH);
        } else {
          const int blk = (int)pos / kv.page_size;
          off = (int)pos - blk * kv.page_size;
          if (blk < kv.max_pages) page = kv.block_table[(long long)b * kv.max_pages + blk];
          if (page < 0 || page >= kv.n_pages) {
            flag(status, DSA_DEV_BAD_PAGE);
            page = -1;
          }
        }
      }
    }
    s_page[tid] = page;
    s_off[tid] = off;
  }
  if (blockIdx.x == 0)
    for (int b = tid; b < B; b += kReadThreads)
      if (cu_out[b] < 0 || cu_out[b + 1] < cu_out[b] || cu_out[b + 1] > n_t)
        flag(status, DSA_DEV_BAD_LENGTH);
  __syncthreads();
  const int per = kv.D / 16, row = kv.Hkv * per, rows = min(kReadRows, n_t - t_first);
  const uint8_t* pages = blockIdx.y == 0 ? kv.k_pages : kv.v_pages;
  const float* scales = blockIdx.y == 0 ? kv.k_scale : kv.v_scale;
  T* out = blockIdx.y == 0 ? k_out : v_out;
  const bool wide = is_wide(out);
  // piece `rest` of row r, and how far the thread's next one is; its head by a product (exact:
  // rest < 2^11, per <= 2^4)
  const unsigned inv = 65536u / per + 1;
  const int more_r = kReadThreads / row, more = kReadThreads - more_r * row;
  int r = tid / row, rest = tid - r * row;
  auto ahead = [&](int& r, int& rest) {
    r += more_r;
    rest += more;
    if (rest >= row) {
      rest -= row;
      ++r;
    }
  };
  constexpr int kAhead = 2;  // pieces on their way
#pragma unroll 1
  while (r < rows) {
    uint4 v[kAhead];
    float s[kAhead];
    int r1 = r, rest1 = rest;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      v[i] = make_uint4(0u, 0u, 0u, 0u);  // (no page: zeros)
      s[i] = 0.f;
      const int page = r1 < rows ? s_page[r1] : -2;
      if (page >= 0) {
        const int h = (int)((unsigned)rest1 * inv >> 16);
        const long long unit = (long long)page * kv.Hkv + h;
        v[i] = ld_stream_v4(pages + (unit * kv.page_size + s_off[r1]) * kv.D +
                            (rest1 - h * per) * 16);
        s[i] = __ldg(scales + unit);
      }
      ahead(r1, rest1);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (r < rows && s_page[r] != -2) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float x[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 a = codes2(w[k] & 0xffffu), c = codes2(w[k] >> 16);
          x[4 * k] = a.x * s[i];
          x[4 * k + 1] = a.y * s[i];
          x[4 * k + 2] = c.x * s[i];
          x[4 * k + 3] = c.y * s[i];
        }
        store16<T>(out + ((long long)(t_first + r) * row + rest) * 16, x, wide);
      }
      ahead(r, rest);
    }
  }
}

}  // namespace

namespace {

template <typename T>
int append(const void* k_new, const void* v_new, const int32_t* cu_new, int n_t, int B,
           const GqaKv& kv, void* k_mean, int32_t* status, cudaStream_t stream) {
  // A warp a token's block where that is no more of them than of blocks, in us, of 64 sequences
  // with 1 / 2 / 3 / 8 tokens each (8 heads of 128, pages of 64, no block becomes complete): 2.9 /
  // 3.2 / 5.0 / 6.2, a CTA a block 5.5 / 5.6 / 5.7 / 5.8.  Elements kept in registers where they
  // fit, of 64 sequences with 8 / 128 / 512 tokens: 5.8 / 13.4 / 41, read twice 5.3 / 23.8 / 74.
  const int slots = n_t / kv.page_size + 2 * B;
  const bool few = n_t <= slots, block = kv.page_size * kv.D <= 64 * kThreads;
  const dim3 grid = few ? dim3((unsigned)n_t, (unsigned)(2 * kv.Hkv + 7) / 8, 1)
                        : dim3((unsigned)slots, (unsigned)kv.Hkv, 1);
  static_assert(2 * kThreads / 32 == 8, "warps of a CTA");
  Launch l(grid, 2 * kThreads, 0, stream);
  auto kernel = few                    ? gqa_append_kernel<T, 32>
                : block && kv.D == 128 ? gqa_append_block_kernel<T, 128>
                : block && kv.D == 64  ? gqa_append_block_kernel<T, 64>
                                       : gqa_append_kernel<T, kThreads>;
  return launch_kernel(&l.cfg, kernel, static_cast<const T*>(k_new), static_cast<const T*>(v_new),
                       cu_new, n_t, B, kv, static_cast<__nv_bfloat16*>(k_mean),
                       status) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

int launch_gqa_append(const void* k_new, const void* v_new, const int32_t* cu_new, int T, int B,
                      int dtype, const GqaKv& kv, void* k_mean, int32_t* status,
                      cudaStream_t stream) {
  return dtype == DSA_BF16
             ? append<__nv_bfloat16>(k_new, v_new, cu_new, T, B, kv, k_mean, status, stream)
             : append<float>(k_new, v_new, cu_new, T, B, kv, k_mean, status, stream);
}

int launch_gqa_read(const GqaKv& kv, const int32_t* cu_out, const int32_t* begin, int T, int B,
                    int dtype, void* k_out, void* v_out, int32_t* status, cudaStream_t stream) {
  Launch l(dim3((unsigned)((T + kReadRows - 1ll) / kReadRows), 2, 1), kReadThreads, 0, stream);
  const cudaError_t e =
      dtype == DSA_BF16
          ? launch_kernel(&l.cfg, gqa_read_kernel<__nv_bfloat16>, kv, cu_out, begin, T, B,
                          static_cast<__nv_bfloat16*>(k_out), static_cast<__nv_bfloat16*>(v_out),
                          status)
          : launch_kernel(&l.cfg, gqa_read_kernel<float>, kv, cu_out, begin, T, B,
                          static_cast<float*>(k_out), static_cast<float*>(v_out), status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
