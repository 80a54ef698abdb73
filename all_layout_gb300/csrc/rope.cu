// Rotary positions with several axes, with the per-head RMS norm of q and k, from
// the token-major output of the QKV projection [B][N][heads][d] to the head-major
// tensors [B][heads][N][d] that attention reads (any strides on both sides; in
// place when a tensor's two sides are the same).
//
// Per row x (one token, one head) of a tensor with a weight w:
//     x <- x / sqrt(mean(x^2) + eps) * w,
// and of a rotated tensor, for every pair (a, b) of its first `rot` columns, with
// the pair's axis and frequency f: angle = pos[axis] * f,
//     (a, b) <- (a cos - b sin, b cos + a sin).
//
// Angles. A frequency is held as a 64-bit fixed-point fraction of a turn (turns.h: off by
// 2^-65 of one at most), so pos * f modulo one turn is one wrapping integer product: off by
// 2^-34 of a turn at most for every 32-bit position, negative ones included, with no range
// reduction. Its top 32 bits, as a signed fraction of a half turn, go to sincospif in fp32
// (in all below 2^-25 of a turn, plus sincospif's own error).
//
// Bound: HBM. Every value is read once and written once. A thread keeps one token
// and eight columns and walks the heads, so the sines and cosines of its four pairs
// are computed once and stay in registers for all heads of q and k; the norm's sum
// runs over the lanes of the row by shuffles. Half pairs: a thread takes four columns
// and their four partners (two 8-byte accesses), which needs no exchange between
// lanes. There is no shared memory and no barrier; UNROLL rows are loaded before the
// first is used, and blocks of 128 threads at no more than 64 registers keep 32 warps
// on an SM. Measured (GB300, device time): 65536 tokens x 72 heads x 128 with the norm
// 377 us = 6.41 TB/s, 95% of the copy rate; 4096 tokens of the same 31.6 us (71%: one
// wave, whose start and end show); 16384 tokens x 36 x 256 fp16 half pairs 105.7 us
// (84%); 65536 x 25 x 80 fp32 to bf16 149 us (78%: a row takes the power of two of lanes
// at or above d / 8, of whose 16 ten work). Tried at the first three sizes, then 378, 30.9
// and 105.9 us: blocks of 256 threads 381, 34.1 and 107.3; the weight and the rotation as
// two factors per column (fewer operations, 72-90 registers) 402, 36 and 174; the partner
// columns by shuffle 384, 32.6 and 119.7.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/xs.h"
#include "internal.h"
#include "turns.h"

namespace xs {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxPairs = 128;

struct RopeTensor {
  const void *x;
  void *y;
  const float *w;                 // [d] or null
  long long x_b, x_n, x_h;        // strides in elements: batch, token, head
  long long y_b, y_n, y_h;
  int heads, rotate;
};

struct RopeParams {
  RopeTensor t[3];
  int n_tensors, items;           // items: heads of all tensors
  const int *pos;                 // [B or 1][N][n_axes]
  long long pos_b;                // elements between batch entries (0: shared)
  int n_axes, adjacent;
  int B, N, d, rot;
  int lanes;                      // lanes per row, the power of two >= d / 8
  int items_per_block;            // of the heads of all tensors, per blockIdx.y
  float eps, inv_d;
  unsigned long long freq[kRopeMaxPairs];   // turns per position step, 64-bit fraction
  unsigned char axis[kRopeMaxPairs];
};

// Four values of a type: 8 bytes (bf16, fp16) or 16 (fp32), to and from fp32.
template <class T>
struct Quad {
  uint32_t u[sizeof(T)];
};
__device__ __forceinline__ void ld(Quad<float> &q, const float *p) {
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.u[0]), "=r"(q.u[1]), "=r"(q.u[2]), "=r"(q.u[3])
               : "l"(p)
               : "memory");
}
template <class T>
__device__ __forceinline__ void ld(Quad<T> &q, const T *p) {
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(q.u[0]), "=r"(q.u[1])
               : "l"(p)
               : "memory");
}
// A thread's eight columns: two quads, next to each other (PAIRED: one 16-byte access for
// 2-byte types) or half a rotation apart.
template <bool PAIRED, class T>
__device__ __forceinline__ void ld_row(Quad<T> (&q)[2], const T *a, const T *b) {
  if constexpr (PAIRED && sizeof(T) == 2) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(q[0].u[0]), "=r"(q[0].u[1]), "=r"(q[1].u[0]), "=r"(q[1].u[1])
                 : "l"(a)
                 : "memory");
  } else {
    ld(q[0], a);
    ld(q[1], b);
  }
}
__device__ __forceinline__ void widen(const Quad<float> &q, float *f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(q.u[i]);
}
__device__ __forceinline__ void widen(const Quad<__nv_bfloat16> &q, float *f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[2 * i] = __uint_as_float(q.u[i] << 16);
    f[2 * i + 1] = __uint_as_float(q.u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen(const Quad<__half> &q, float *f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    __half2 h;
    memcpy(&h, &q.u[i], 4);
    const float2 g = __half22float2(h);
    f[2 * i] = g.x;
    f[2 * i + 1] = g.y;
  }
}
// The one rounding of an output value, to nearest even.
__device__ __forceinline__ uint2 narrow(const float *f, __nv_bfloat16) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  uint2 u;
  memcpy(&u.x, &a, 4);
  memcpy(&u.y, &b, 4);
  return u;
}
__device__ __forceinline__ uint2 narrow(const float *f, __half) {
  const __half2 a = __floats2half2_rn(f[0], f[1]), b = __floats2half2_rn(f[2], f[3]);
  uint2 u;
  memcpy(&u.x, &a, 4);
  memcpy(&u.y, &b, 4);
  return u;
}
template <bool PAIRED, class T>
__device__ __forceinline__ void st_row(T *a, T *b, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4 *>(a) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4 *>(b) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    const uint2 lo = narrow(f, T()), hi = narrow(f + 4, T());
    if constexpr (PAIRED) {
      *reinterpret_cast<uint4 *>(a) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      *reinterpret_cast<uint2 *>(a) = lo;
      *reinterpret_cast<uint2 *>(b) = hi;
    }
  }
}

// cos and sin of a pair at position `pos`.
__device__ __forceinline__ void pair_angle(const RopeParams &p, const int *pos, int pair, float &c,
                                           float &s) {
  const long long at = pos[p.axis[pair]];
  const unsigned long long turn = static_cast<unsigned long long>(at) * p.freq[pair];
  const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;
  sincospif(half_turns, &s, &c);
}

// The rotation of a thread's four pairs; the columns past the rotated part stay, infinities among them.
template <bool ADJ>
__device__ __forceinline__ void turn_pairs(float (&f)[8], const float (&cs)[4], const float (&sn)[4], int c,
                                           int half) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = ADJ ? 2 * i : i, ib = ADJ ? 2 * i + 1 : i + 4;
    const float a = f[ia], e = f[ib];
    if (4 * c + i < half) {
      f[ia] = a * cs[i] - e * sn[i];
      f[ib] = e * cs[i] + a * sn[i];
    }
  }
}
// Sum over a row's lanes.
__device__ __forceinline__ float row_sum(float x, int lanes) {
  for (int m = lanes / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}
// Whether t = mean(x^2) + eps is as good as its formula: no square that counts has left fp32's range. (None of
// an fp16 does: 2^-48 to 2^32.)
__device__ __forceinline__ bool norm_fits(float t) { return t >= 0x1p-80f && t <= 0x1p120f; }

// The rows of heads h, h + 1, ... that do not fit, by the bits of `left`: their values become x * s, with s the
// power of two that brings the largest near 1 (exact), and their factor 1 / sqrt(mean((x s)^2) + eps s^2).
// Rows with an infinity or NaN keep s = 1; a row of zeros with eps = 0 stays zeros. The kernel stores the
// other rows and leaves these as they were read, in place too. (Once for 32 heads, behind the kernel's loop
// over them: 16384 tokens x 72 heads x 128, half pairs, 107.1 us, without any of this 106.8. In the loop 109.6;
// called from it 121.7.)
template <class TI, class TO, bool ADJ>
__device__ __forceinline__ void rope_scaled(const RopeParams &p, int ti, int b, int n, bool live, int h, unsigned left) {
  const RopeTensor &t = p.t[ti];
  const int c = threadIdx.x & (p.lanes - 1), half = p.rot / 2;
  const bool turned = c * 8 < p.rot;
  const int col_a = ADJ || !turned ? 8 * c : 4 * c;
  const int col_b = ADJ || !turned ? 8 * c + 4 : half + 4 * c;
  const int *pos = p.pos + b * p.pos_b + static_cast<long long>(n) * p.n_axes;
#pragma unroll 1
  for (; __any_sync(0xffffffffu, left != 0); ++h, left >>= 1) {
    const bool mine = left & 1;
    Quad<TI> raw[2];
    memset(&raw, 0, sizeof(raw));
    const TI *x = static_cast<const TI *>(t.x) + b * t.x_b + n * t.x_n + h * t.x_h;
    if (live && mine) ld_row<ADJ>(raw, x + col_a, x + col_b);
    float f[8], ss = 0.f, big = 0.f;
    widen(raw[0], f);
    widen(raw[1], f + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fmaf(f[i], f[i], ss);
      big = fmaxf(big, fabsf(f[i]));   // (passes a NaN over: ss tells)
    }
    ss = row_sum(ss, p.lanes);
    for (int m = p.lanes / 2; m > 0; m >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, m));
    float s = 1.f;
    if (ss == ss && big < INFINITY) {
      const int e = __float_as_int(fmaxf(big, sqrtf(p.eps))) >> 23;
      s = __int_as_float((254 - min(max(e, 1), 253)) << 23);
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] *= s;
      ss = fmaf(f[i], f[i], ss);
    }
    const float mean = fmaf(row_sum(ss, p.lanes), p.inv_d, p.eps * s * s);
    const float r = mean == 0.f ? 0.f : rsqrtf(mean);
    if (!live || !mine) continue;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= r * __ldg(t.w + (i < 4 ? col_a + i : col_b + i - 4));
    if (t.rotate) {
      float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * c + i < half) pair_angle(p, pos, 4 * c + i, cs[i], sn[i]);
      turn_pairs<ADJ>(f, cs, sn, c, half);
    }
    TO *y = static_cast<TO *>(t.y) + b * t.y_b + n * t.y_n + h * t.y_h;
    st_row<ADJ>(y + col_a, y + col_b, f);
  }
}

template <class TI, class TO, bool ADJ>
__global__ void __launch_bounds__(kRopeThreads, 1024 / kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int UNROLL = sizeof(TI) == 2 ? 4 : 2;
  constexpr bool SCALED = !std::is_same_v<TI, __half>;   // rows may be left to rope_scaled
  const int lanes = p.lanes;
  const int c = threadIdx.x & (lanes - 1);
  const long long token = static_cast<long long>(blockIdx.x) * (kRopeThreads / lanes) +
                          threadIdx.x / lanes;
  const long long tokens = static_cast<long long>(p.B) * p.N;
  // Idle lanes (past the row, past the last token) load nothing and store nothing but take part
  // in the shuffles.
  const bool live = token < tokens && c * 8 < p.d;
  const int b = live ? static_cast<int>(token / p.N) : 0;
  const int n = live ? static_cast<int>(token - static_cast<long long>(b) * p.N) : 0;

  // The thread's columns: eight in a row, or (half pairs, rotated part) four and their partners.
  const int half = p.rot / 2;
  const bool turned = c * 8 < p.rot;
  const int col_a = ADJ || !turned ? 8 * c : 4 * c;
  const int col_b = ADJ || !turned ? 8 * c + 4 : half + 4 * c;
  float cs[4], sn[4];
  {
    const int *pos = p.pos + b * p.pos_b + static_cast<long long>(n) * p.n_axes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = 4 * c + i;
      cs[i] = 1.f;
      sn[i] = 0.f;
      if (live && pair < half) pair_angle(p, pos, pair, cs[i], sn[i]);
    }
  }

  const int item0 = blockIdx.y * p.items_per_block;
  const int item1 = min(item0 + p.items_per_block, p.items);
  int first = 0;   // item of the tensor's head 0
#pragma unroll 1
  for (int ti = 0; ti < p.n_tensors; ++ti) {
    const RopeTensor &t = p.t[ti];
    const int h0 = max(item0 - first, 0), h1 = min(item1 - first, t.heads);
    first += t.heads;
    if (h0 >= h1) continue;
    const TI *x = static_cast<const TI *>(t.x) + b * t.x_b + n * t.x_n + col_a;
    TO *y = static_cast<TO *>(t.y) + b * t.y_b + n * t.y_n + col_a;
    const int step = col_b - col_a;
    const bool norm = t.w != nullptr, rotate = t.rotate != 0;
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (norm && live) {
      const float4 wa = __ldg(reinterpret_cast<const float4 *>(t.w + col_a));
      const float4 wb = __ldg(reinterpret_cast<const float4 *>(t.w + col_b));
      w[0] = wa.x, w[1] = wa.y, w[2] = wa.z, w[3] = wa.w;
      w[4] = wb.x, w[5] = wb.y, w[6] = wb.z, w[7] = wb.w;
    }
#pragma unroll 1
    for (int hc = h0; SCALED ? hc < h1 : hc == h0; hc += 32) {   // 32 heads at a time, or all
      const int h2 = SCALED ? min(hc + 32, h1) : h1;
      unsigned left = 0;   // a bit for each head whose row is left to rope_scaled
#pragma unroll 1
      for (int h = hc; h < h2; h += UNROLL) {
        Quad<TI> raw[UNROLL][2];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          memset(&raw[k], 0, sizeof(raw[k]));
          const TI *row = x + (h + k) * t.x_h;
          if (live && h + k < h2) ld_row<ADJ>(raw[k], row, row + step);
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
          if (h + k >= h2) break;
          float f[8];
          widen(raw[k][0], f);
          widen(raw[k][1], f + 4);
          bool fits = true;
          if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
            const float mean = fmaf(row_sum(ss, lanes), p.inv_d, p.eps);
            float r = rsqrtf(mean);
            if constexpr (!SCALED) {
              if (mean == 0.f) r = 0.f;
            } else {
              fits = !live || norm_fits(mean);
              if (!fits) left |= 1u << (h + k - hc);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= r * w[i];
          }
          if (rotate) turn_pairs<ADJ>(f, cs, sn, c, half);
          TO *row = y + (h + k) * t.y_h;
          if (live && fits) st_row<ADJ>(row, row + step, f);
        }
      }
      if constexpr (SCALED)
        if (__any_sync(0xffffffffu, left != 0)) rope_scaled<TI, TO, ADJ>(p, ti, b, n, live, hc, left);
    }
  }
}

template <class TI, class TO>
cudaError_t launch_typed(const RopeParams &p, dim3 grid, cudaStream_t s) {
  if (p.adjacent)
    rope_kernel<TI, TO, true><<<grid, kRopeThreads, 0, s>>>(p);
  else
    rope_kernel<TI, TO, false><<<grid, kRopeThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_rope(const RopeParams &p, int in, int out, dim3 grid, cudaStream_t s) {
  if (in == XS_BF16 && out == XS_BF16) return launch_typed<__nv_bfloat16, __nv_bfloat16>(p, grid, s);
  if (in == XS_FP16 && out == XS_FP16) return launch_typed<__half, __half>(p, grid, s);
  if (in == XS_FP16) return launch_typed<__half, __nv_bfloat16>(p, grid, s);
  if (out == XS_FP32) return launch_typed<float, float>(p, grid, s);
  return launch_typed<float, __nv_bfloat16>(p, grid, s);
}

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace
}  // namespace xs

extern "C" __attribute__((visibility("default"))) xs_status xs_rope(
    const xs_rope_tensor *tensors, int n_tensors, const int *pos, long long pos_batch_stride,
    const int *axis_dims, int n_axes, const double *freqs, int B, int N, int d, float eps,
    int flags, int in_type, int out_type, void *stream) {
  using namespace xs;
  if (!tensors || !pos || !axis_dims || !freqs || n_tensors < 1 || n_tensors > 3 || B < 0 ||
      N < 0 || d < 0 || n_axes < 1 || n_axes > 4 || (flags & ~XS_ROPE_ADJACENT) != 0 ||
      !(eps >= 0.f) || std::isinf(eps) || pos_batch_stride < 0)
    return XS_ERR_INVALID;
  for (int t : {in_type, out_type})
    if (t != XS_BF16 && t != XS_FP16 && t != XS_FP32) return XS_ERR_INVALID;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  for (int a = 0; a < n_axes; ++a) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 != 0 || axis_dims[a] > d - p.rot) return XS_ERR_INVALID;
    p.rot += axis_dims[a];
  }
  const bool adjacent = (flags & XS_ROPE_ADJACENT) != 0;
  long long items = 0;
  // The strides of a tensor without rows say nothing.
  auto has_rows = [&](const xs_rope_tensor &t) { return B > 0 && N > 0 && t.heads > 0; };
  for (int i = 0; i < n_tensors; ++i) {
    const xs_rope_tensor &t = tensors[i];
    if (t.heads < 0 || (t.heads > 0 && (!t.x || !t.y))) return XS_ERR_INVALID;
    if (!has_rows(t)) {
      items += t.heads;
      continue;
    }
    const long long extent[3] = {B, N, t.heads};
    bool same = true;
    for (int k = 0; k < 3; ++k) {
      if (t.x_stride[k] < 0 || t.y_stride[k] < 0) return XS_ERR_INVALID;
      if (extent[k] > 1 && t.y_stride[k] < d) return XS_ERR_INVALID;   // rows of y would overlap
      if (extent[k] > 1 && t.x_stride[k] != t.y_stride[k]) same = false;
    }
    // In place only where every row is written to where it was read.
    if (t.x == t.y && (!same || in_type != out_type)) return XS_ERR_INVALID;
    items += t.heads;
  }
  if (d < 8 || d > 256 || d % 8 != 0 || (!adjacent && p.rot % 8 != 0)) return XS_ERR_UNSUPPORTED;
  if (!(in_type == out_type || (in_type != XS_BF16 && out_type == XS_BF16))) return XS_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > 0x7fffffffLL || items > 65535) return XS_ERR_UNSUPPORTED;
  const int in_vec = in_type == XS_FP32 ? 4 : 8, out_vec = out_type == XS_FP32 ? 4 : 8;
  for (int i = 0; i < n_tensors; ++i) {
    const xs_rope_tensor &t = tensors[i];
    if (!aligned(t.x, 16) || !aligned(t.y, 16) || !aligned(t.weight, 16)) return XS_ERR_ALIGN;
    if (!has_rows(t)) continue;
    const long long extent[3] = {B, N, t.heads};
    for (int k = 0; k < 3; ++k)
      if (extent[k] > 1 && (t.x_stride[k] % in_vec != 0 || t.y_stride[k] % out_vec != 0))
        return XS_ERR_ALIGN;
  }
  if (!aligned(pos, 4)) return XS_ERR_ALIGN;
  for (int a = 0, pair = 0; a < n_axes; ++a)
    for (int i = 0; i < axis_dims[a] / 2; ++i, ++pair) {
      if (!std::isfinite(freqs[pair])) return XS_ERR_INVALID;
      if (!turns_fit(freqs[pair])) return XS_ERR_UNSUPPORTED;
      p.freq[pair] = turns_per_step(freqs[pair]);
      p.axis[pair] = static_cast<unsigned char>(a);
    }
  if (B == 0 || N == 0 || items == 0) return XS_OK;
  for (int i = 0; i < n_tensors; ++i) {
    const xs_rope_tensor &t = tensors[i];
    p.t[i] = RopeTensor{t.x, t.y, t.weight, t.x_stride[0], t.x_stride[1], t.x_stride[2],
                        t.y_stride[0], t.y_stride[1], t.y_stride[2], t.heads, t.rotate};
  }
  p.n_tensors = n_tensors;
  p.items = static_cast<int>(items);
  p.pos = pos;
  p.pos_b = pos_batch_stride;
  p.n_axes = n_axes;
  p.adjacent = adjacent;
  p.B = B;
  p.N = N;
  p.d = d;
  p.eps = eps;
  p.inv_d = 1.f / static_cast<float>(d);
  p.lanes = 1;
  while (p.lanes * 8 < d) p.lanes *= 2;
  const int sms = sm_count();
  if (sms <= 0) return XS_ERR_CUDA;
  const long long rows = kRopeThreads / p.lanes;   // tokens of a block
  const long long gx = (static_cast<long long>(B) * N + rows - 1) / rows;
  // Few tokens: the heads are spread over blocks too, down to four per block, until there are
  // four blocks for every SM; each repeats its tokens' sines and cosines. (Measured at 4096
  // tokens x 72 heads: 4 blocks 30.9 us, 8 32.9, 16 34.0.)
  long long gy = (4LL * sms + gx - 1) / gx;
  if (gy > (items + 3) / 4) gy = (items + 3) / 4;
  p.items_per_block = static_cast<int>((items + gy - 1) / gy);
  gy = (items + p.items_per_block - 1) / p.items_per_block;
  return launch_rope(p, in_type, out_type, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)),
                     static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? XS_OK
             : XS_ERR_CUDA;
}
