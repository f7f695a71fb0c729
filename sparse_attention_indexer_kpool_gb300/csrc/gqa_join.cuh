// What the attention kernels of the grouped-query layer share: the tensor maps of the codes, and
// the join of the partials of items (row tiles) whose tiles were shared out over several
// workers (warps or CTAs).
#pragma once

#include <type_traits>

#include "gqa.cuh"
#include "mla_chunk.cuh"

namespace dsa {
namespace gqa {

// Weights are held times 2^2, and so are the outputs: 2^13 above a head's first reference before it
// has to be raised (held times 2^8, with 2^7 above, a chunk of 2,048 tokens behind 14,336 keys took
// 8 % longer), and 2^-27 of it below.
constexpr int kUp = 2;

struct Header {        // what a worker left
  int start_item;      // item whose first tiles it holds but not its last (-1: none)
  int cont_item;       // item that an earlier worker began (-1: none)
  int cont;            // 1: it has a partial of that, 2: and its last tiles
  int tokens;          // of start_item, where items differ in them
};

// x 2^(e - kUp) / f, in steps that stay in range where the result does (0 for f = 0: no sum)
struct Factor {
  float inv, a, b;
  __device__ __forceinline__ Factor(float f, int e) {
    inv = f == 0.f ? 0.f : 1.f / (f * (float)(1 << kUp));
    const int third = max(min(e / 3, 126), -126);
    a = pow2(third);
    b = pow2(max(min(e - 2 * third, 126), -126));
  }
  __device__ __forceinline__ float operator()(float x) const { return x * inv * a * a * b; }
};

struct JoinArgs {
  const float* part_o;    // [2 workers][kRows][D], outputs relative to 2^reference
  const float4* part_ml;  // [2 workers][kRows]: reference; the sum f 2^z as z and f
  const Header* head;     // [workers]
  int workers;
  __nv_bfloat16* out;
  float* lse;
};

// Partials are joined in the workers' order.  An item's workers are neighbours in their numbers:
// every block reads all headers and lists the ones that began an item.  A piece is one row
// of such an item: a warp's where there are many, a block's, each warp a part of the
// partials, where there are few.
constexpr int kMaxWorkers = 1280, kJoinThreads = 512, kJoinWarps = kJoinThreads / 32;
struct Joined {
  float m, z, f, x[4];  // outputs relative to 2^m; the sum f 2^z
};
__device__ __forceinline__ Joined nothing() {
  return Joined{-INFINITY, -INFINITY, 0.f, {0.f, 0.f, 0.f, 0.f}};
}
__device__ __forceinline__ float finite_or_0(float x) { return x == -INFINITY ? 0.f : x; }

// a <- a and b together, in this order (nothing: f and x are 0)
__device__ __forceinline__ void merge(Joined& a, const Joined& b) {
  const float m = fmaxf(a.m, b.m), z = fmaxf(a.z, b.z);
  const float ref = finite_or_0(m), zref = finite_or_0(z);
  // square roots, taken twice (no reference: nothing, or a NaN sum, which stays one)
  const float wa = a.m == -INFINITY ? 1.f : ex2_fast(0.5f * (a.m - ref));
  const float wb = b.m == -INFINITY ? 1.f : ex2_fast(0.5f * (b.m - ref));
  const float za = a.z == -INFINITY ? 1.f : ex2_fast(0.5f * (a.z - zref));
  const float zb = b.z == -INFINITY ? 1.f : ex2_fast(0.5f * (b.z - zref));
  a.m = m;
  a.z = z;
  a.f = a.f * za * za + b.f * zb * zb;
#pragma unroll
  for (int k = 0; k < 4; ++k) a.x[k] = a.x[k] * wa * wa + b.x[k] * wb * wb;
}
// a lane's columns of a row
template <int kD>
__device__ __forceinline__ void load_part(Joined& j, const float* row, int lane) {
  if constexpr (kD == 128) {
    const float4 x = reinterpret_cast<const float4*>(row)[lane];
    j.x[0] = x.x; j.x[1] = x.y; j.x[2] = x.z; j.x[3] = x.w;
  } else {
    const float2 x = reinterpret_cast<const float2*>(row)[lane];
    j.x[0] = x.x; j.x[1] = x.y;
  }
}

template <int kD, int kRows>
__device__ __forceinline__ Joined join_parts(const JoinArgs& p, const Header* heads, int g0,
                                             int s0, int s1, int r, int lane) {
  Joined j = nothing();
#pragma unroll 1
  for (; s0 < s1; s0 += 32) {
    const int s = s0 + lane;
    const bool part = s < s1 && (s == g0 || (heads[s].cont & 1));
    const int slot = (s == g0 ? 2 * s + 1 : 2 * s) * kRows + r;
    float4 ml = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
    if (part) ml = p.part_ml[slot];
    const bool some = part && ml.z != 0.f;  // (a part that saw no page adds nothing)
    const float m = fmaxf(j.m, warp_max(some ? ml.x : -INFINITY));
    const float z = fmaxf(j.z, warp_max(some ? ml.y : -INFINITY));
    const float ref = finite_or_0(m), zref = finite_or_0(z);
    // square roots, taken twice; 0 before the first part
    const float old = ex2_fast(0.5f * (j.m - ref)), zold = ex2_fast(0.5f * (j.z - zref));
    // (no reference: a NaN sum, which stays one)
    const float wgt = some ? ex2_fast(ml.x == -INFINITY ? 0.f : 0.5f * (ml.x - ref)) : 0.f;
    const float zw = some ? ex2_fast(ml.y == -INFINITY ? 0.f : 0.5f * (ml.y - zref)) : 0.f;
    j.f = j.f * zold * zold + warp_sum(some ? ml.z * zw * zw : 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) j.x[k] = j.x[k] * old * old;
    j.m = m;
    j.z = z;
    unsigned todo = __ballot_sync(0xffffffffu, some);
    while (todo) {
      float v[4][4], wv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // four partial rows on their way at once
        const int i = todo ? __ffs(todo) - 1 : -1;
        const int sl = __shfl_sync(0xffffffffu, slot, i & 31);
        wv[u] = __shfl_sync(0xffffffffu, wgt, i & 31);
        if (i < 0) wv[u] = 0.f;
        const float* src = p.part_o + (long long)sl * kD + lane * (kD / 32);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][k] = 0.f;
        if (i >= 0) {
          if constexpr (kD == 128) {
            const float4 f = __ldcs(reinterpret_cast<const float4*>(src));
            v[u][0] = f.x; v[u][1] = f.y; v[u][2] = f.z; v[u][3] = f.w;
          } else {
            const float2 f = __ldcs(reinterpret_cast<const float2*>(src));
            v[u][0] = f.x; v[u][1] = f.y;
          }
        }
        todo &= todo - 1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) j.x[k] = fmaf(v[u][k] * wv[u], wv[u], j.x[k]);
    }
  }
  return j;
}
template <int kD>
__device__ __forceinline__ void store_row(const JoinArgs& p, long long row, const float (&x)[4],
                                          int lane) {
  __nv_bfloat16* out = p.out + row * kD + lane * (kD / 32);
  if constexpr (kD == 128)
    *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  else
    *reinterpret_cast<uint32_t*>(out) = pack_bf16(x[0], x[1]);
}
template <int kD>
__device__ __forceinline__ void store_joined(const JoinArgs& p, long long row, const Joined& j,
                                             int lane) {
  // (m - z: a whole part and a rest below 1)
  const float d = j.f == 0.f || j.m == -INFINITY ? 0.f : j.m - j.z;
  const float whole = fabsf(d) < 1000.f ? floorf(d) : 0.f;
  const Factor by(j.f * ex2_fast(whole - d), (int)whole);
  float x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) x[k] = by(j.x[k]);
  store_row<kD>(p, row, x, lane);
  if (p.lse && lane == 0)
    p.lse[row] = j.f == 0.f ? -INFINITY : (j.z + log2f(j.f)) / kLog2e;
}

// Rows: kRows rows of an item, `used` of them in any; the output row of one (-1: none)
template <int kD, typename Rows>
__global__ void __launch_bounds__(kJoinThreads, 2)
    gqa_join_kernel(const JoinArgs p, const Rows rows) {
  constexpr int kRows = Rows::kRows;
  const int workers = p.workers;
  __shared__ __align__(16) Header heads[kMaxWorkers];
  __shared__ unsigned short begun[kMaxWorkers];
  __shared__ int counts[kMaxWorkers / 32];
  __shared__ Joined parts[kJoinWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < workers; i += kJoinThreads)
    *reinterpret_cast<int4*>(heads + i) = *reinterpret_cast<const int4*>(p.head + i);
  __syncthreads();
  // (32 of them a warp and step, behind those of the steps before)
  const int steps = (workers + 31) / 32;
  auto began = [&](int s) {
    return __ballot_sync(0xffffffffu, s + lane < workers && heads[s + lane].start_item >= 0);
  };
  for (int i = warp; i < steps; i += kJoinWarps) {
    const unsigned all = began(32 * i);
    if (lane == 0) counts[i] = __popc(all);
  }
  __syncthreads();
  int n_begun = 0;
  for (int i = 0; i < steps; ++i) n_begun += counts[i];
  for (int i = warp; i < steps; i += kJoinWarps) {
    const unsigned all = began(32 * i);
    int n = __popc(all & ((1u << lane) - 1));
    for (int k = 0; k < i; ++k) n += counts[k];
    if ((all >> lane) & 1u) begun[n] = (unsigned short)(32 * i + lane);
  }
  __syncthreads();
  const int used = rows.used(), pieces = n_begun * used;
  // workers of the item that g0 began: g0 .. g0 + n - 1
  auto workers_of = [&](int g0, int item) {
    int n = 1;
    for (unsigned stop = 0; !stop;) {
      const int s = g0 + n + lane;
      const Header hd = heads[min(s, workers - 1)];
      const bool mine = s < workers && hd.cont_item == item;
      stop = __ballot_sync(0xffffffffu, !mine || (hd.cont & 2));
      const int k = stop ? __ffs(stop) - 1 : 32;  // before the stopping one
      n += k + (stop ? __shfl_sync(0xffffffffu, (int)mine, k & 31) : 0);
    }
    return n;
  };
  if (pieces > 2 * (int)gridDim.x) {
    // A warp takes kRowsOnce rows of an item at a time.  Of up to eight partials lane 8 p + r takes
    // the numbers of partials p and p + 4 of row r, so that each is worked out once; the outputs
    // are then sums of products with two factors each (2^64 apart and more, in steps that stay in
    // range).  A chunk's 39,000 rows: 13 us, and 19 with each lane working out all numbers.  Eight
    // rows where half of the warps have as many, else two.
    auto join_rows = [&](auto rows_at_once) {
      constexpr int kRowsOnce = decltype(rows_at_once)::value, kU = kRowsOnce < 4 ? kRowsOnce : 4;
      const int groups = (used + kRowsOnce - 1) / kRowsOnce, r = lane & 7;
#pragma unroll 1
      for (int i = warp * gridDim.x + blockIdx.x; i < n_begun * groups;
           i += gridDim.x * kJoinWarps) {
        const int g0 = begun[i / groups], r0 = i % groups * kRowsOnce, item = heads[g0].start_item;
        const int n = workers_of(g0, item);
        const int row = r < kRowsOnce && r0 + r < used ? (int)rows(item, heads[g0].tokens, r0 + r)
                                                       : -1;
        if (n > 8) {
#pragma unroll 1
          for (int u = 0; u < kRowsOnce; ++u) {
            const int to = __shfl_sync(0xffffffffu, row, u);
            if (to >= 0)
              store_joined<kD>(p, to,
                               join_parts<kD, kRows>(p, heads, g0, g0, g0 + n, r0 + u, lane), lane);
          }
          continue;
        }
        auto slot_of = [&](int part) { return (2 * (g0 + part) + (part == 0)) * kRows + r0; };
        auto there = [&](int part) {
          return part < n && (part == 0 || (heads[g0 + part].cont & 1));
        };
        float m[2], z[2], f[2], top = -INFINITY;
        bool some[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int part = (lane >> 3) + 4 * v;
          float4 ml = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
          if (there(part) && row >= 0) ml = __ldcs(p.part_ml + slot_of(part) + r);
          m[v] = ml.x;
          z[v] = ml.y;
          f[v] = ml.z;
          some[v] = ml.z != 0.f;  // (a part that saw no page adds nothing)
          if (some[v]) top = fmaxf(top, z[v]);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const float ref = finite_or_0(top);
        float sum = 0.f, c1[2], c2[2];
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          // square roots, taken twice (no reference: a NaN sum, which stays one)
          const float a = z[v] == -INFINITY ? 1.f : ex2_fast(0.5f * (z[v] - ref));
          sum += some[v] ? f[v] * a * a : 0.f;
          c1[v] = !some[v] ? 0.f : m[v] == -INFINITY ? 1.f : ex2_fast(0.5f * (m[v] - ref));
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const float inv = sum == 0.f ? 0.f : 1.f / (sum * (float)(1 << kUp));
        c2[0] = c1[0] * inv;
        c2[1] = c1[1] * inv;
        if (p.lse && lane < 8 && row >= 0)
          p.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) / kLog2e;
#pragma unroll
        for (int u0 = 0; u0 < kRowsOnce; u0 += kU) {
          int to[kU];
          float x[kU][4];
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            to[u] = __shfl_sync(0xffffffffu, row, u0 + u);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[u][k] = 0.f;
          }
#pragma unroll 2
          for (int part = 0; part < n; ++part) {
            if (!there(part)) continue;
            const float* src = p.part_o + (long long)(slot_of(part) + u0) * kD;
            const float s1 = part < 4 ? c1[0] : c1[1], s2 = part < 4 ? c2[0] : c2[1];
            const int from = (part & 3) * 8 + u0;
            Joined j[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              j[u] = nothing();
              if (to[u] >= 0) load_part<kD>(j[u], src + u * kD, lane);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
              const float a = __shfl_sync(0xffffffffu, s1, from + u);
              const float b = __shfl_sync(0xffffffffu, s2, from + u);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[u][k] = fmaf(j[u].x[k] * a, b, x[u][k]);
            }
          }
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (to[u] >= 0) store_row<kD>(p, to[u], x[u], lane);
        }
      }
    };
    if (pieces >= 4 * (int)gridDim.x * kJoinWarps)
      join_rows(std::integral_constant<int, 8>{});
    else
      join_rows(std::integral_constant<int, 2>{});
    return;
  }
  // a block a row, each warp a part of the partials
#pragma unroll 1
  for (int i = blockIdx.x; i < pieces; i += gridDim.x) {
    const int g0 = begun[i / used], r = i % used, item = heads[g0].start_item;
    const long long row = rows(item, heads[g0].tokens, r);
    if (row < 0) continue;
    const int n = workers_of(g0, item), per = (n + kJoinWarps - 1) / kJoinWarps;
    const int s0 = g0 + min(n, warp * per);
    const Joined j =
        join_parts<kD, kRows>(p, heads, g0, s0, min(s0 + per, g0 + n), r, lane);
    parts[warp][lane] = j;
    __syncthreads();
    if (warp == 0) {
      Joined all = nothing();
#pragma unroll
      for (int u = 0; u < kJoinWarps; ++u) {
        all.m = fmaxf(all.m, parts[u][lane].m);
        all.z = fmaxf(all.z, parts[u][lane].z);
      }
      const float ref = finite_or_0(all.m), zref = finite_or_0(all.z);
#pragma unroll
      for (int u = 0; u < kJoinWarps; ++u) {
        const Joined& x = parts[u][lane];
        // (no reference: no part, or a NaN sum, which stays one)
        const float e = x.m == -INFINITY ? 1.f : ex2_fast(0.5f * (x.m - ref));
        const float ze = x.z == -INFINITY ? 1.f : ex2_fast(0.5f * (x.z - zref));
        all.f = fmaf(x.f * ze, ze, all.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) all.x[k] = fmaf(x.x[k] * e, e, all.x[k]);
      }
      store_joined<kD>(p, row, all, lane);
    }
    __syncthreads();
  }
}

// Rows of D codes (as 2-byte elements), boxes of box_rows of them.
inline bool code_map(CUtensorMap* m, const void* base, uint64_t rows, int D, uint32_t box_rows) {
  auto fn = chunk::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D / 2, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)D / 2, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// items: of the step, at most
template <int kD, typename Rows>
int launch_join(const JoinArgs& p, const Rows& rows, long long items, cudaStream_t stream) {
  const long long pieces = (items < p.workers ? items : p.workers) * Rows::kRows;
  const int grid = pieces < 2 * num_sms() ? (int)pieces : 2 * num_sms();
  Launch l(dim3(grid, 1, 1), kJoinThreads, 0, stream);
  return launch_kernel(&l.cfg, gqa_join_kernel<kD, Rows>, p, rows) == cudaSuccess ? DSA_OK
                                                                                  : DSA_ERR_CUDA;
}

}  // namespace gqa
}  // namespace dsa
