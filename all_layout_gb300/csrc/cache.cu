// The quantised key/value cache: rows of keys and values into pages in e4m3 with a scale
// each (xs_cache_write), and back (xs_cache_read).
//
// Row x of d values (one token, one k/v head): with a = max |x|
//     e = the least integer with a <= 448 * 2^e   (in [-120, 119]; 0 for a row of zeros),
//     code = e4m3(x * 2^-e), to nearest even,   scale byte = e + 127,
// and what a code stands for is code * 2^e. A power of two costs no precision beside a
// scale of full width (the codes are floating-point numbers themselves: values down to 2^-13 of
// the row's maximum keep all 4 bits, and smaller ones are off by at most 2^-10 * 2^e), and makes both x * 2^-e and code * 2^e
// exact, so that a code is the only rounding between a key and what attention sees of it:
// e4m3 has 4 significant bits, bf16 8. A row that holds a NaN or an infinity gets the scale
// byte 255 and reads as NaN.
//
// Bound: HBM, every value read once and written once (3 bytes a value from or to bf16), once the
// instructions are few enough. So a lane has 16 columns of a row (one vector of codes, two or four
// of values), a row the power of two of lanes at or above d / 16; 16-bit magnitudes are compared in
// pairs, the maximum of a row comes by shuffles; and a thread's two rows are loaded before the first
// is used. Measured at 65536 rows of 24 heads of 128 (1.21 GB): read 178 us = 6.8 TB/s, write 202 us
// = 6.0 TB/s; with 8 columns a lane and four rows 246 and 382 us, with 16 and one row 211 and 243,
// with four rows 194 and 194 but the small calls up to 1.6 times as long. To and from fp32 (2.02 GB): read 384 us = 5.3 TB/s,
// write 315 us = 6.4 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/xs.h"
#include "cache.h"
#include "internal.h"

namespace xs {
namespace {

constexpr int kCacheThreads = 256, kRows = 2, kColumns = 16;
// CTAs that an SM holds: what bounds the registers, without spills.
template <class T, bool WRITE>
constexpr int kBlocks = !WRITE ? 8 : sizeof(T) == 4 ? 4 : 5;

struct CacheParams {
  PageLists lists;
  uint8_t *codes[2], *scales[2];        // of k and v
  const void *x[2];                     // rows outside the cache: read by a write, written by a read
  long long x_b[2], x_h[2], x_n[2];     // strides in elements: batch, head, token
  const int *start, *lens;              // [B] or null
  int B, Hk, N, d;
  int lanes;                            // lanes of a row
};

// A lane's columns of a row as they lie in memory, and the pairs of values that they are.
template <class T>
struct Columns {
  static constexpr int kVecs = kColumns * static_cast<int>(sizeof(T)) / 16;
  uint4 w[kVecs];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint32_t word(int i) const {
    const uint4 &v = w[i >> 2];
    return (i & 3) == 0 ? v.x : (i & 3) == 1 ? v.y : (i & 3) == 2 ? v.z : v.w;
  }
};
__device__ __forceinline__ float2 pair_at(const Columns<float> &c, int i) {
  return make_float2(__uint_as_float(c.word(2 * i)), __uint_as_float(c.word(2 * i + 1)));
}
__device__ __forceinline__ float2 pair_at(const Columns<__nv_bfloat16> &c, int i) {
  const uint32_t u = c.word(i);
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_at(const Columns<__half> &c, int i) {
  const uint32_t u = c.word(i);
  __half2 h;
  memcpy(&h, &u, 4);
  return __half22float2(h);
}

// The bits of the largest magnitude of a row, as fp32, over its lanes. Magnitudes order as their
// bits do, infinities and NaN above all; 16-bit ones are compared in pairs.
__device__ __forceinline__ uint32_t biggest(const Columns<float> &c, int lanes) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < kColumns; ++i) big = max(big, c.word(i) & 0x7fffffffu);
  for (int o = 1; o < lanes; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
  return big;
}
template <class T>
__device__ __forceinline__ uint32_t biggest(const Columns<T> &c, int lanes) {
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < kColumns / 2; ++i) big = __vmaxu2(big, c.word(i) & 0x7fff7fffu);
  for (int o = 1; o < lanes; o <<= 1) big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, o));
  big = max(big >> 16, big & 0xffffu);
  if constexpr (std::is_same<T, __half>::value) {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(big))));
  } else {
    return big << 16;
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

// Place of a row of request b in the cache, in rows; -1 where there is none.
__device__ __forceinline__ long long row_at(const CacheParams &p, int b, const TokenAt &t, long long first) {
  const long long pos = first + t.n;
  const int page = page_of(p.lists, b, pos);
  if (page < 0) return -1;
  return (static_cast<long long>(page) * p.Hk + t.h) * p.lists.page + (pos & (p.lists.page - 1));
}

template <class T, bool WRITE>
__global__ void __launch_bounds__(kCacheThreads, kBlocks<T, WRITE>) cache_kernel(const __grid_constant__ CacheParams p) {
  const int kv = blockIdx.y & 1;
  const int lane = threadIdx.x & (p.lanes - 1), group = threadIdx.x / p.lanes, groups = kCacheThreads / p.lanes;
  const int c0 = lane * kColumns;
  const bool in_row = c0 < p.d;
  // Rows base, base + groups, ... of the Hk * N; the division is done for the first of them.
  const long long base = static_cast<long long>(blockIdx.x) * groups * kRows + group, rows = static_cast<long long>(p.Hk) * p.N;
  for (int b = blockIdx.y >> 1; b < p.B; b += gridDim.y >> 1) {
    const unsigned N = p.N, live = p.lens ? min(max(__ldg(p.lens + b), 0), p.N) : p.N;
    const long long first = p.start ? __ldg(p.start + b) : 0;
    T *const xb = const_cast<T *>(static_cast<const T *>(p.x[kv])) + b * p.x_b[kv] + c0;
    TokenAt t = token_at(static_cast<unsigned>(min(base, rows)), N);
    long long at[kRows];
    T *x[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      at[u] = t.h < p.Hk && t.n < live ? row_at(p, b, t, first) : -2;
      x[u] = xb + t.h * p.x_h[kv] + t.n * p.x_n[kv];
      step_token(t, groups, N, p.Hk);
    }
    if constexpr (WRITE) {
      Columns<T> c[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (at[u] >= 0 && in_row)
          c[u].load(x[u]);
        else
          c[u].clear();
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int byte = scale_byte(biggest(c[u], p.lanes));
        if (at[u] < 0) continue;
        const float s = __int_as_float((254 - byte) << 23);   // 2^-e
        uint32_t code[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 l = pair_at(c[u], 2 * j), r = pair_at(c[u], 2 * j + 1);
          code[j] = byte == kNanScale ? 0x7f7f7f7fu : codes4(l.x * s, l.y * s, r.x * s, r.y * s);
        }
        if (in_row) *reinterpret_cast<uint4 *>(p.codes[kv] + at[u] * p.d + c0) = make_uint4(code[0], code[1], code[2], code[3]);
        if (lane == 0) p.scales[kv][at[u]] = static_cast<uint8_t>(byte);
      }
    } else {
      uint4 code[kRows];
      int byte[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        code[u] = make_uint4(0, 0, 0, 0);
        byte[u] = kNanScale;   // a place that no page holds
        if (at[u] >= 0 && in_row) {
          code[u] = __ldcs(reinterpret_cast<const uint4 *>(p.codes[kv] + at[u] * p.d + c0));
          byte[u] = __ldg(p.scales[kv] + at[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (at[u] == -2 || !in_row) continue;
        const float s = power_of(byte[u]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[8];
          const uint32_t a = j ? code[u].z : code[u].x, b = j ? code[u].w : code[u].y;
          const uint32_t w[4] = {a, a >> 16, b, b >> 16};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 t = values2(w[i]);
            f[2 * i] = t.x * s;
            f[2 * i + 1] = t.y * s;
          }
          store8(x[u] + 8 * j, f);
        }
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
  p.lanes = 1;
  while (p.lanes * kColumns < c->d) p.lanes *= 2;
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
