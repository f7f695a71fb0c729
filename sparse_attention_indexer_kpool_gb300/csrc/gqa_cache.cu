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
// A CTA takes one such block: its rows are read for the maximum and again (from L1) for
// the codes, so that memory sees them once.  The sum of a block's codes is exact in fp32
// up to 64 rows (whole multiples of 2^-9 below 2^15): the order of the additions does
// not count.
// Which blocks a step touches is known on the GPU only.  A sequence with n new tokens
// touches at most floor(n / page_size) + 2, so with cu its place on the step's token axis
// the slots from floor(cu / page_size) + 2 b on are its own: a CTA finds its sequence by
// a binary search in cu_new, and no pass over the lengths comes first.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "gqa.cuh"

namespace dsa {
namespace {

using namespace gqa;

constexpr int kThreads = 128;

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

template <typename T>
__global__ void __launch_bounds__(kThreads)
    gqa_append_kernel(const T* __restrict__ k_new, const T* __restrict__ v_new,
                      const int32_t* __restrict__ cu_new, int n_t, int B, GqaKv kv,
                      __nv_bfloat16* __restrict__ k_mean, int32_t* status) {
  __shared__ float s_top[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, h = blockIdx.y, ps = kv.page_size, D = kv.D;
  const bool keys = blockIdx.z == 0, reports = tid == 0 && h == 0 && keys;
  // the sequence of this slot
  auto first_slot = [&](int b) { return min(max(cu_new[b], 0), n_t) / ps + 2 * b; };
  int b = 0;
  for (int hi = B; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (first_slot(mid) <= (int)blockIdx.x) b = mid; else hi = mid;
  }
  const int cu0 = cu_new[b], cu1 = cu_new[b + 1];
  const int c0 = min(max(cu0, 0), n_t), n = min(cu1, n_t) - c0;
  const int i = (int)blockIdx.x - (c0 / ps + 2 * b);
  if (reports && i == 0 && (cu0 < 0 || cu1 < cu0 || cu1 > n_t)) flag(status, DSA_DEV_BAD_LENGTH);
  if (n <= 0 || i < 0) return;
  const int len = kv.seq_lens[b];
  const long long ctx = (long long)len - n;
  if (ctx < 0 && reports && i == 0) flag(status, DSA_DEV_BAD_LENGTH);
  // (rows before position 0 have no place)
  const long long blk = max(ctx, 0ll) / ps + i;
  if (blk * ps >= len) return;
  const int page =
      blk < kv.max_pages ? kv.block_table[(long long)b * kv.max_pages + blk] : -1;
  if (page < 0 || page >= kv.n_pages) {
    if (reports) flag(status, DSA_DEV_BAD_PAGE);
    return;
  }
  const int lo = (int)max(ctx - blk * ps, 0ll);             // new rows lo .. hi - 1 of the page
  const int hi = (int)min((long long)ps, len - blk * ps);
  const long long t0 = c0 + blk * ps + lo - ctx;            // row lo on the step's token axis
  const long long unit = (long long)page * kv.Hkv + h;
  uint8_t* codes = (keys ? kv.k_pages : kv.v_pages) + unit * ps * D;
  float* scale = (keys ? kv.k_scale : kv.v_scale) + unit;
  const T* src = (keys ? k_new : v_new) + (t0 * kv.Hkv + h) * D;
  const int per = D / 8, pieces = (hi - lo) * per;
  const long long pitch = (long long)kv.Hkv * D;

  float top = 0.f;
  for (int j = tid; j < pieces; j += kThreads) {
    const int r = j / per;
    float x[8];
    load8<T>(src + r * pitch + (j - r * per) * 8, x);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (fabsf(x[u]) < INFINITY) top = fmaxf(top, fabsf(x[u]));
  }
  top = warp_max(top);
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  const int e0 = lo > 0 ? exponent_of(*scale) : kExpMin;    // read by all before it is written
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  const int e = max(exponent_for(top), e0);
  if (tid == 0) *scale = pow2(e);
  if (e > e0 && lo > 0) {
    const float down = pow2(max(e0 - e, -126));  // (E4M3 values below 2^126: all zero by then)
    for (int j = tid; j < lo * per; j += kThreads) {
      uint2* p = reinterpret_cast<uint2*>(codes) + j;
      float x[8];
      unpack8(*p, x);
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] *= down;
      *p = pack8(x);
    }
  }
  const float up = pow2(-e);
  for (int j = tid; j < pieces; j += kThreads) {
    const int r = j / per, c = (j - r * per) * 8;
    float x[8];
    load8<T>(src + r * pitch + c, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = fabsf(x[u]) < INFINITY ? x[u] * up : NAN;
    *reinterpret_cast<uint2*>(codes + (long long)(lo + r) * D + c) = pack8(x);
  }
  if (!keys || k_mean == nullptr || hi < ps) return;
  __syncthreads();  // the block's codes are written
  const float share = pow2(e) / (float)ps;
  for (int d = tid * 2; d < D; d += kThreads * 2) {
    float a = 0.f, c = 0.f;
#pragma unroll 8
    for (int r = 0; r < ps; ++r) {
      const float2 x = codes2(*reinterpret_cast<const uint16_t*>(codes + (long long)r * D + d));
      a += x.x;
      c += x.y;
    }
    *reinterpret_cast<uint32_t*>(k_mean + unit * D + d) = pack_bf16(a * share, c * share);
  }
}

// ---- Read-back ----------------------------------------------------------------
// value = code * scale.  A CTA takes 32 rows of the outputs, finds their sequences and
// pages once, and walks over their (KV head, 16 codes) pieces: 16 bytes in, 32 or 64 out a
// thread and step.
constexpr int kReadRows = 32, kReadThreads = 256;

template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&x)[16]);
template <>
__device__ __forceinline__ void store16<__nv_bfloat16>(__nv_bfloat16* p, const float (&x)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  uint4* o = reinterpret_cast<uint4*>(p);
  o[0] = make_uint4(w[0], w[1], w[2], w[3]);
  o[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
template <>
__device__ __forceinline__ void store16<float>(float* p, const float (&x)[16]) {
  float4* o = reinterpret_cast<float4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
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
        const long long pos = (long long)(t - cu_out[b]) + (begin ? begin[b] : 0);
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
  for (int j = tid; j < rows * row; j += kReadThreads) {
    const int r = j / row, rest = j - r * row, h = rest / per, d = (rest - h * per) * 16;
    const int page = s_page[r];
    if (page == -2) continue;
    float x[16];
    if (page < 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    } else {
      const long long unit = (long long)page * kv.Hkv + h;
      const uint4 v = ld_stream_v4(pages + (unit * kv.page_size + s_off[r]) * kv.D + d);
      const float s = __ldg(scales + unit);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = codes2(w[i] & 0xffffu), c = codes2(w[i] >> 16);
        x[4 * i] = a.x * s;
        x[4 * i + 1] = a.y * s;
        x[4 * i + 2] = c.x * s;
        x[4 * i + 3] = c.y * s;
      }
    }
    store16<T>(out + ((long long)(t_first + r) * kv.Hkv + h) * kv.D + d, x);
  }
}

}  // namespace

int launch_gqa_append(const void* k_new, const void* v_new, const int32_t* cu_new, int T, int B,
                      int dtype, const GqaKv& kv, void* k_mean, int32_t* status,
                      cudaStream_t stream) {
  Launch l(dim3((unsigned)(T / kv.page_size + 2 * B), kv.Hkv, 2), kThreads, 0, stream);
  __nv_bfloat16* mean = static_cast<__nv_bfloat16*>(k_mean);
  const cudaError_t e =
      dtype == DSA_BF16
          ? launch_kernel(&l.cfg, gqa_append_kernel<__nv_bfloat16>,
                          static_cast<const __nv_bfloat16*>(k_new),
                          static_cast<const __nv_bfloat16*>(v_new), cu_new, T, B, kv, mean, status)
          : launch_kernel(&l.cfg, gqa_append_kernel<float>, static_cast<const float*>(k_new),
                          static_cast<const float*>(v_new), cu_new, T, B, kv, mean, status);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
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
