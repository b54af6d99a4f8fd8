// What the kernels that write pages share: an append's runs of pages, the rule of
// the page exponent, the upkeep of a page's other rows, and the host's side of an
// append.
#pragma once

#include "iq_paged.cuh"

namespace iq {
namespace paged {

// One contiguous run of pages of one entry: `rows` rows of the call, from row
// `row0`, go to positions pos .. pos + rows - 1 of the slot, which lie in pages
// page, page + 1, ...; the rows that the first page already holds come from
// page `from` (another one when the page was shared and is being copied).
struct Segment {
  int entry, slot, row0, rows, pos, page, from;
};
constexpr int kSegments = 256;  // per launch, by value

struct AppendParams {
  const uint16_t* keys;
  const uint16_t* values;
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  int* table;
  unsigned* status;
  int heads, n, max_pages;
  Segment seg[kSegments];
};

// The checks of an append, without a change, and the checked append: `launch` is
// given the runs of pages (segs of them, the widest of so many pages) and enqueues
// the kernel that fills them.
using AppendLaunch = cudaError_t (*)(const AppendParams& p, int widest, int segs, cudaStream_t stream, const void* more);
int check_append(iq_paged* c, const void* keys, const void* values, int n, const int32_t* slots, const int32_t* counts,
                 int n_slots);
int do_append(iq_paged* c, const void* keys, const void* values, int n, const int32_t* slots, const int32_t* counts,
              int n_slots, iq_stream_t stream, AppendLaunch launch, const void* more);

// NaN: 0; infinity: the largest value of its sign.
__device__ __forceinline__ uint32_t drop_non_finite(uint32_t w) {
#pragma unroll
  for (int s = 0; s < 32; s += 16) {
    const uint32_t h = (w >> s) & 0x7FFFu;
    if (h >= 0x7F80u) w = (w & ~(0x7FFFu << s)) | ((h == 0x7F80u ? 0x7F7Fu : 0u) << s);
  }
  return w;
}
// The larger magnitude of both halves of eight bf16 values (they order as integers).
__device__ __forceinline__ uint32_t magnitude(const uint4& x) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(t & 0xFFFFu, t >> 16);
}
// The least e >= kEMin with |x| <= 448 * 2^e, of the bits of a finite |x|:
// x = 1.m * 2^k, and 448 * 2^e = 1.75 * 2^(8+e) is reached from e = k - 8 on, or
// k - 7 where 1.m is above 1.75.
__device__ __forceinline__ int least_exponent(uint32_t bits) {
  if (bits < 0x00800000u) return kEMin;
  return max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0), kEMin);
}
// The other rows of a page into which rows [begin, end) go (256 threads): those
// before come from `src` (moved: another page), rescaled where the exponent grew
// from `old` to `e`; where the page is new to its slot, those behind are zero, so
// that whole pages can enter matrix products before they are full.
__device__ __forceinline__ void upkeep(const uint8_t* src, uint8_t* dst, int begin, int end, bool moved, int old, int e) {
  const int warp = threadIdx.x >> 5, at = (threadIdx.x & 31) * 8;
  if (begin > 0 && (moved || e > old)) {
    const float f = power2(max(old - e, -126));
    for (int r = warp; r < begin; r += 8) {
      uint2 c = *reinterpret_cast<const uint2*>(src + r * kHeadDim + at);
      if (e > old) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 lo = f16x2_to_f32(e4m3x2_to_f16x2(w[j] & 0xFFFFu)), hi = f16x2_to_f32(e4m3x2_to_f16x2(w[j] >> 16));
          w[j] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
        }
      }
      *reinterpret_cast<uint2*>(dst + r * kHeadDim + at) = c;
    }
  }
  if (begin == 0 || moved)
    for (int r = warp; r < kPage; r += 8)
      if (r >= end) *reinterpret_cast<uint2*>(dst + r * kHeadDim + at) = make_uint2(0, 0);
}

}  // namespace paged
}  // namespace iq
