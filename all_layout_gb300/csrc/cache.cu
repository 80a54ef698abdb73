// The quantised key/value cache: rows of keys and values into pages in e4m3 with a scale
// each (xs_cache_write), and back (xs_cache_read).
//
// Row x of d values (one token, one k/v head): with a = max |x|
//     e = the least integer with a <= 448 * 2^e   (in [-120, 119]; 0 for a row of zeros),
//     code = e4m3(x * 2^-e), to nearest even,   scale byte = e + 127,
// and what a code stands for is code * 2^e. A power of two costs no precision beside a
// scale of full width (the codes are floating-point numbers themselves; only what lies 2^15
// below the row's maximum loses bits to the range), and makes both x * 2^-e and code * 2^e
// exact, so that a code is the only rounding between a key and what attention sees of it:
// e4m3 has 4 significant bits, bf16 8. A row that holds a NaN or an infinity gets the scale
// byte 255 and reads as NaN.
//
// Bound: HBM, every value read once and written once (3 bytes a value from or to bf16). A lane
// has eight columns of a row, a row the power of two of lanes at or above d / 8, its maximum
// comes by shuffles; kRows rows a thread are loaded before the first is used.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>

#include "../../include/xs.h"
#include "cache.h"
#include "internal.h"

namespace xs {
namespace {

constexpr int kCacheThreads = 256, kRows = 4;

struct CacheParams {
  PageLists lists;
  uint8_t *codes[2], *scales[2];        // of k and v
  const void *x[2];                     // rows outside the cache: read by a write, written by a read
  long long x_b[2], x_h[2], x_n[2];     // strides in elements: batch, head, token
  const int *start, *lens;              // [B] or null
  int B, Hk, N, d;
  int lanes;                            // lanes of a row
};

// Eight values to and from fp32.
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
  const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half *p, float (&f)[8]) {
  const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h;
    memcpy(&h, &u[i], 4);
    const float2 t = __half22float2(h);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  __stcs(reinterpret_cast<float4 *>(p), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ uint32_t pair_of(__nv_bfloat16, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t pair_of(__half, float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
template <class T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(pair_of(T(), f[0], f[1]), pair_of(T(), f[2], f[3]),
                                                  pair_of(T(), f[4], f[5]), pair_of(T(), f[6], f[7])));
}

// Four values to e4m3, to nearest even, the largest finite code beyond it.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// What two codes stand for without the scale (exact in fp16).
__device__ __forceinline__ float2 values2(uint32_t codes) {
  uint32_t r;
  asm("{.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;}" : "=r"(r) : "r"(codes));
  __half2 h;
  memcpy(&h, &r, 4);
  return __half22float2(h);
}

// The scale byte of a row from the bits of its largest magnitude.
__device__ __forceinline__ int scale_byte(uint32_t big) {
  if (big == 0) return 127;
  if (big >= 0x7f800000u) return kNanScale;
  // big = 2^(E - 127) (1 + f): 448 * 2^e = 1.75 * 2^(8 + e) holds it for e = E - 135, or one more
  // where 1 + f > 1.75.
  const int e = static_cast<int>(big >> 23) - 135 + ((big & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -120), 119) + 127;
}

// Place of row (b, h, n) in the cache, in rows; -1 where there is none.
__device__ __forceinline__ long long row_at(const CacheParams &p, int b, int h, int n, long long first) {
  const long long pos = first + n;
  const int page = page_of(p.lists, b, pos);
  if (page < 0) return -1;
  return (static_cast<long long>(page) * p.Hk + h) * p.lists.page + (pos & (p.lists.page - 1));
}

template <class T, bool WRITE>
__global__ void __launch_bounds__(kCacheThreads) cache_kernel(const __grid_constant__ CacheParams p) {
  const int kv = blockIdx.y & 1;
  const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, groups = kCacheThreads / p.lanes;
  const long long base = static_cast<long long>(blockIdx.x) * groups * kRows + group;
  const bool in_row = lane * 8 < p.d;
  const long long rows = static_cast<long long>(p.Hk) * p.N;
  for (int b = blockIdx.y >> 1; b < p.B; b += gridDim.y >> 1) {
    const int live = p.lens ? min(max(__ldg(p.lens + b), 0), p.N) : p.N;
    const long long first = p.start ? __ldg(p.start + b) : 0;
    long long at[kRows];
    T *x[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const long long r = base + static_cast<long long>(u) * groups;
      const int h = static_cast<int>(static_cast<unsigned>(min(r, rows - 1)) / static_cast<unsigned>(p.N));
      const int n = static_cast<int>(r - static_cast<long long>(h) * p.N);
      at[u] = r < rows && n < live ? row_at(p, b, h, n, first) : -2;
      x[u] = const_cast<T *>(static_cast<const T *>(p.x[kv])) + b * p.x_b[kv] + h * p.x_h[kv] + n * p.x_n[kv] + lane * 8;
    }
    if constexpr (WRITE) {
      float f[kRows][8];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (at[u] >= 0 && in_row) {
          load8(x[u], f[u]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[u][i] = 0.f;
        }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        uint32_t big = 0;   // magnitudes order as their bits do, infinities and NaN above all
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(f[u][i]) & 0x7fffffffu);
        for (int o = 1; o < p.lanes; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        if (at[u] < 0) continue;
        const int byte = scale_byte(big);
        uint2 code = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
        if (byte != kNanScale) {
          const float s = __int_as_float((254 - byte) << 23);   // 2^-e
          code.x = codes4(f[u][0] * s, f[u][1] * s, f[u][2] * s, f[u][3] * s);
          code.y = codes4(f[u][4] * s, f[u][5] * s, f[u][6] * s, f[u][7] * s);
        }
        if (in_row) *reinterpret_cast<uint2 *>(p.codes[kv] + at[u] * p.d + lane * 8) = code;
        if (lane == 0) p.scales[kv][at[u]] = static_cast<uint8_t>(byte);
      }
    } else {
      uint2 code[kRows];
      int byte[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        code[u] = make_uint2(0, 0);
        byte[u] = kNanScale;   // a place that no page holds
        if (at[u] >= 0 && in_row) {
          code[u] = __ldcs(reinterpret_cast<const uint2 *>(p.codes[kv] + at[u] * p.d + lane * 8));
          byte[u] = __ldg(p.scales[kv] + at[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (at[u] == -2 || !in_row) continue;
        const float s = power_of(byte[u]);
        float f[8];
        const uint32_t w[4] = {code[u].x, code[u].x >> 16, code[u].y, code[u].y >> 16};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 t = values2(w[i]);
          f[2 * i] = t.x * s;
          f[2 * i + 1] = t.y * s;
        }
        store8(x[u], f);
      }
    }
  }
}

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

xs_status cache_call(bool write, const xs_cache *c, const void *k, const void *v, const long long *k_stride,
                     const long long *v_stride, const xs_pages *pages, const int *start, const int *lens, int B,
                     int N, int type, void *stream) {
  if (B < 0 || N < 0 || (type != XS_BF16 && type != XS_FP16 && type != XS_FP32)) return XS_ERR_INVALID;
  xs_status st = check_cache(c);
  if (st != XS_OK) return st;
  if (!k || !v || !k_stride || !v_stride) return XS_ERR_INVALID;
  const long long extent[3] = {B, c->H_kv, N};
  const void *x[2] = {k, v};
  const long long *strides[2] = {k_stride, v_stride};
  const bool empty = B == 0 || N == 0 || c->H_kv == 0;
  for (int t = 0; t < 2 && !empty; ++t)
    for (int i = 0; i < 3; ++i)
      if (extent[i] > 1 && (strides[t][i] < 0 || (!write && strides[t][i] < c->d))) return XS_ERR_INVALID;
  st = check_pages(pages, B);
  if (st != XS_OK) return st;
  if (c->d % 16 != 0 || c->d < 16 || c->d > 256) return XS_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->H_kv) * N > 0x7fffffffLL) return XS_ERR_UNSUPPORTED;
  const int vec = type == XS_FP32 ? 4 : 8;
  for (int t = 0; t < 2; ++t) {
    if (!aligned(x[t], 16)) return XS_ERR_ALIGN;
    for (int i = 0; i < 3 && !empty; ++i)
      if (extent[i] > 1 && strides[t][i] % vec != 0) return XS_ERR_ALIGN;
  }
  if (!aligned(start, 4) || !aligned(lens, 4)) return XS_ERR_ALIGN;
  if (empty) return XS_OK;
  CacheParams p;
  std::memset(&p, 0, sizeof(p));
  p.lists = lists_of(*c, pages);
  p.codes[0] = static_cast<uint8_t *>(c->k);
  p.codes[1] = static_cast<uint8_t *>(c->v);
  p.scales[0] = c->k_scale;
  p.scales[1] = c->v_scale;
  for (int t = 0; t < 2; ++t) {
    p.x[t] = x[t];
    p.x_b[t] = strides[t][0];
    p.x_h[t] = strides[t][1];
    p.x_n[t] = strides[t][2];
  }
  p.start = start;
  p.lens = lens;
  p.B = B;
  p.Hk = c->H_kv;
  p.N = N;
  p.d = c->d;
  p.lanes = 2;
  while (p.lanes * 8 < c->d) p.lanes *= 2;
  const long long rows = static_cast<long long>(c->H_kv) * N, each = kCacheThreads / p.lanes * kRows;
  const dim3 grid(static_cast<unsigned>((rows + each - 1) / each), 2u * static_cast<unsigned>(B < 32767 ? B : 32767));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto one) {
    using T = decltype(one);
    if (write)
      cache_kernel<T, true><<<grid, kCacheThreads, 0, s>>>(p);
    else
      cache_kernel<T, false><<<grid, kCacheThreads, 0, s>>>(p);
  };
  if (type == XS_BF16)
    launch(__nv_bfloat16());
  else if (type == XS_FP16)
    launch(__half());
  else
    launch(0.f);
  return cudaGetLastError() == cudaSuccess ? XS_OK : XS_ERR_CUDA;
}

}  // namespace

xs_status check_cache(const xs_cache *c) {
  if (!c || c->n_pages < 0 || c->H_kv < 0 || c->page_size < 1 || c->d < 0) return XS_ERR_INVALID;
  if (c->n_pages > 0 && c->H_kv > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return XS_ERR_INVALID;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0) return XS_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16)) return XS_ERR_ALIGN;
  return XS_OK;
}

xs_status check_pages(const xs_pages *l, int B) {
  if (!l || l->count < 0 || (l->count > 0 && B > 0 && !l->pages)) return XS_ERR_INVALID;
  if (B > 1 && l->stride < 0) return XS_ERR_INVALID;
  if (!aligned(l->pages, 4)) return XS_ERR_ALIGN;
  return XS_OK;
}

PageLists lists_of(const xs_cache &c, const xs_pages *l) {
  PageLists r{l->pages, l->stride, l->count, c.n_pages, c.page_size, 0};
  while ((1 << r.shift) < c.page_size) ++r.shift;
  return r;
}

}  // namespace xs

extern "C" __attribute__((visibility("default"))) xs_status xs_cache_write(
    const xs_cache *cache, const void *k, const void *v, const long long *k_stride, const long long *v_stride,
    const xs_pages *pages, const int *start, const int *lens, int B, int N, int in_type, void *stream) {
  return xs::cache_call(true, cache, k, v, k_stride, v_stride, pages, start, lens, B, N, in_type, stream);
}

extern "C" __attribute__((visibility("default"))) xs_status xs_cache_read(
    const xs_cache *cache, void *k, void *v, const long long *k_stride, const long long *v_stride,
    const xs_pages *pages, const int *start, const int *lens, int B, int N, int out_type, void *stream) {
  return xs::cache_call(false, cache, k, v, k_stride, v_stride, pages, start, lens, B, N, out_type, stream);
}
