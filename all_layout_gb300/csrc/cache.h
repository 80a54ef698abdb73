// What the calls that use the quantised key/value cache share (cache.cu, prefix_api.cu).
#pragma once
#include <cstdint>

#include "../../include/xs.h"

namespace xs {

constexpr int kNanScale = 255;   // scale byte of a row that is not a number

// Lists of pages as a kernel sees them.
struct PageLists {
  const int *pages;      // list of request b at pages + b * stride
  long long stride;
  int count, n_pages;    // entries of a list; pages of the cache
  int page, shift;       // rows of a page, a power of two
};

#ifdef __CUDACC__
#define XS_HOST_DEVICE __host__ __device__
#else
#define XS_HOST_DEVICE
#endif
// Head and token of row h * N + n among H * N < 2^31; h = H: past the last one. The token is unsigned, as N and
// a step together may pass 2^31.
struct TokenAt {
  int h;
  unsigned n;
};
XS_HOST_DEVICE inline TokenAt token_at(unsigned row, unsigned N) {
  const unsigned h = row / N;
  return TokenAt{static_cast<int>(h), row - h * N};
}
// `by` rows on.
XS_HOST_DEVICE inline void step_token(TokenAt &t, unsigned by, unsigned N, int H) {
  t.n += by;
  while (t.n >= N && t.h < H) t.n -= N, ++t.h;
}

xs_status check_cache(const xs_cache *c);
xs_status check_pages(const xs_pages *l, int B);
PageLists lists_of(const xs_cache &c, const xs_pages *l);

#ifdef __CUDACC__
// The page that holds place `pos` of request b; -1 where the list ends before it or names none.
__device__ __forceinline__ int page_of(const PageLists &l, int b, long long pos) {
  if (pos < 0 || (pos >> l.shift) >= l.count) return -1;
  const int page = __ldg(l.pages + b * l.stride + (pos >> l.shift));
  return page >= 0 && page < l.n_pages ? page : -1;
}
// 2^(byte - 127), or NaN for kNanScale.
__device__ __forceinline__ float power_of(int byte) {
  return __int_as_float(byte == kNanScale ? 0x7fffffff : byte == 0 ? 0x00400000 : byte << 23);
}
#endif

}  // namespace xs
