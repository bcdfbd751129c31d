// pages.cuh -- copies of cache pages: forking a sequence, copying on write, compaction.
//
// A page holds rows of every layer's codes and scales (and a sequence's slot its sink, window and tensor
// scale), so one page is `outer` pieces of `item` bytes in each of several arrays.  One launch moves all
// pieces of all arrays for a list of (source, destination) pages given by the caller on the host: the list
// travels in the kernel's parameters, so it needs no device buffer and no copy of its own.  Bytes are read
// once and written once, which bounds it: a CTA moves up to 16 KB of one piece with 32-byte accesses (16, 4 or 1
// where the piece's size or address asks for it).  Measured: 128 pages of 64 tokens in 16 layers, K and V, 8 heads of 128
// channels (302 MB moved) 47.2 us, 6.4 TB/s, 0.98 of the copy rate; 8 pages in 8 layers (9.4 MB) 2.7 us, most of it the
// launch.
#pragma once

#include <type_traits>

#include "device.cuh"

namespace nvfp4 {

constexpr int kPagesMaxArrays = 16, kPagesPairs = 1024, kPagesThreads = 256;
constexpr int64_t kPagesPiece = 16384;     // bytes per CTA

struct PagesArray {
  char* base;
  int64_t stride, item;                    // bytes between outer pieces; bytes of a page within one
  int outer, width;                        // width: bytes per access (32, 16, 4, 1)
  int64_t parts;                           // CTAs per piece: ceil(item / kPagesPiece)
};
struct PagesParams {
  PagesArray a[kPagesMaxArrays];
  int64_t start[kPagesMaxArrays + 1];      // CTAs of the arrays before
  int count, n;
  int src[kPagesPairs], dst[kPagesPairs];
};
static_assert(sizeof(PagesParams) <= 32764, "kernel parameters are limited to 32764 bytes");

template <int N>
__device__ __forceinline__ void pages_move(const char* s, char* d, int64_t bytes) {
  constexpr int U = 2;                       // loads in flight per thread
  const int64_t n = bytes / N;
  for (int64_t i = threadIdx.x; i < n; i += U * kPagesThreads) {
    if constexpr (N == 32) {
      uint32_t v[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kPagesThreads < n) ld_v8(s + (i + u * kPagesThreads) * 32, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kPagesThreads < n) st_v8(d + (i + u * kPagesThreads) * 32, v[u]);
    } else {
      using T = typename std::conditional<N == 16, uint4, typename std::conditional<N == 4, uint32_t, uint8_t>::type>::type;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i + u * kPagesThreads < n)
          reinterpret_cast<T*>(d)[i + u * kPagesThreads] = reinterpret_cast<const T*>(s)[i + u * kPagesThreads];
    }
  }
}

__global__ void __launch_bounds__(kPagesThreads) copy_pages_kernel(const __grid_constant__ PagesParams p) {
  int64_t x = blockIdx.x;
  int k = 0;
  while (x >= p.start[k + 1]) ++k;
  x -= p.start[k];
  const PagesArray& a = p.a[k];
  const int64_t part = x % a.parts;
  x /= a.parts;
  const int pair = (int)(x % p.n);
  const int64_t outer = x / p.n;
  char* base = a.base + outer * a.stride + part * kPagesPiece;
  const char* s = base + (int64_t)p.src[pair] * a.item;
  char* d = base + (int64_t)p.dst[pair] * a.item;
  const int64_t bytes = min(kPagesPiece, a.item - part * kPagesPiece);
  if (a.width == 32) pages_move<32>(s, d, bytes);
  else if (a.width == 16) pages_move<16>(s, d, bytes);
  else if (a.width == 4) pages_move<4>(s, d, bytes);
  else pages_move<1>(s, d, bytes);
}

}  // namespace nvfp4
