// libiqkv: rotary positions of queries and keys, each head's vector normed in the
// same pass, and the paged cache's append that takes a projection's rows as they are.
//
// Mathematics.  y = x * (mean(x^2) + eps)^-1/2 * weight (where a weight is given), then
// the pairs (a, b) of the leading rotary dims become (a c - b s, a s + b c) * amplitude
// with c, s the cosine and sine of position * frequency.  fp32 throughout, rounded once.
//
// Angles.  A far position times a frequency has a fraction of a turn that fp32 cannot
// tell (at 2^20, 2^-4 of a radian is lost), so a frequency is held as its turns per
// position modulo 1 in 64 bits of fixed point: the product with a position, modulo
// 2^64, is the angle modulo a turn, off by at most position * 2^-64 and what the
// frequency itself was off.  One integer product; no table in memory, no fp64.  The
// eighth of a turn around the nearest quarter goes to sincospif, the quarter swaps
// and negates.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "iq_pages.cuh"

namespace iq {
namespace paged {
namespace {

// Where the pairs of a lane's dims are.  Lane l of a row's warp holds dims 4l .. 4l+3
// and 128 + 4l .. 128 + 4l+3: then halves that are 128 apart meet in one lane, and a
// row's cosines are read from shared memory without conflicts.
enum Layout {
  kNone,    // nothing turns
  kPairs,   // dims 2i and 2i + 1
  kNear,    // dims i and i + pairs, pairs <= 64: all among the first 128 dims
  kAcross,  // pairs == 128
  kFar      // between
};

struct Turn {
  const unsigned long long* turns;
  const float* q_weight;
  const float* k_weight;
  float amplitude, eps;
  int pairs;
};
struct Rows {
  const uint8_t* at;
  long long entry, head, row;  // strides in bytes
};

template <bool F32>
struct Raw;
template <>
struct Raw<false> {
  static constexpr int kBytes = 2;
  uint2 x[2];
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    x[0] = __ldcs(reinterpret_cast<const uint2*>(row + lane * 8));
    x[1] = __ldcs(reinterpret_cast<const uint2*>(row + 256 + lane * 8));
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      y[4 * g] = __uint_as_float(x[g].x << 16);
      y[4 * g + 1] = __uint_as_float(x[g].x & 0xFFFF0000u);
      y[4 * g + 2] = __uint_as_float(x[g].y << 16);
      y[4 * g + 3] = __uint_as_float(x[g].y & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(uint8_t* row, int lane, const float (&y)[8]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint2 o;
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.x) : "f"(y[4 * g + 1]), "f"(y[4 * g]));
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o.y) : "f"(y[4 * g + 3]), "f"(y[4 * g + 2]));
      *reinterpret_cast<uint2*>(row + 256 * g + lane * 8) = o;
    }
  }
};
template <>
struct Raw<true> {
  static constexpr int kBytes = 4;
  float4 x[2];
  __device__ __forceinline__ void load(const uint8_t* row, int lane) {
    x[0] = __ldcs(reinterpret_cast<const float4*>(row + lane * 16));
    x[1] = __ldcs(reinterpret_cast<const float4*>(row + 512 + lane * 16));
  }
  __device__ __forceinline__ void get(float (&y)[8]) const {
#pragma unroll
    for (int g = 0; g < 2; ++g) y[4 * g] = x[g].x, y[4 * g + 1] = x[g].y, y[4 * g + 2] = x[g].z, y[4 * g + 3] = x[g].w;
  }
  static __device__ __forceinline__ void store(uint8_t* row, int lane, const float (&y)[8]) {
#pragma unroll
    for (int g = 0; g < 2; ++g) *reinterpret_cast<float4*>(row + 512 * g + lane * 16) = make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]);
  }
};

// Cosine and sine of an angle of `a` / 2^32 turns.
__device__ __forceinline__ float2 unit_at(unsigned a, float amplitude) {
  const unsigned quarter = (a + 0x20000000u) >> 30;
  const int rest = static_cast<int>(a - (quarter << 30));  // an eighth of a turn at most
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c * amplitude, s * amplitude);
}
// Row r of the table: the cosines of its pairs, then their sines.
template <typename Position>
__device__ __forceinline__ void fill_table(const Turn& t, float* table, int rows, Position position) {
  int r = threadIdx.x / t.pairs, j = threadIdx.x - r * t.pairs;
  const int down = blockDim.x / t.pairs, across = blockDim.x - down * t.pairs;
  while (r < rows) {
    const long long p = position(r);
    const float2 u = unit_at(static_cast<unsigned>((static_cast<unsigned long long>(p) * __ldg(t.turns + j)) >> 32), t.amplitude);
    table[(2 * r) * t.pairs + j] = u.x;
    table[(2 * r + 1) * t.pairs + j] = u.y;
    r += down;
    j += across;
    if (j >= t.pairs) {
      j -= t.pairs;
      ++r;
    }
  }
}

// (a c - b s, a s + b c)
__device__ __forceinline__ void spin(float& a, float& b, float c, float s) {
  const float x = fmaf(a, c, -(b * s));
  b = fmaf(a, s, b * c);
  a = x;
}
// a c + b s, with the sine's sign given by the half that `a` is in
__device__ __forceinline__ float spun(float a, float b, float c, float s, bool upper) { return fmaf(a, c, upper ? b * s : -(b * s)); }

// A row's vector, turned.  row: its cosines, then its sines.
template <int LAYOUT>
__device__ __forceinline__ void turn_row(float (&x)[8], const float* row, int pairs, int lane) {
  if constexpr (LAYOUT == kPairs) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int j = 64 * g + 2 * lane;
      if (j >= pairs) continue;
      const float2 c = *reinterpret_cast<const float2*>(row + j), s = *reinterpret_cast<const float2*>(row + pairs + j);
      spin(x[4 * g], x[4 * g + 1], c.x, s.x);
      spin(x[4 * g + 2], x[4 * g + 3], c.y, s.y);
    }
  } else if constexpr (LAYOUT == kAcross) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * lane), s = *reinterpret_cast<const float4*>(row + 128 + 4 * lane);
    spin(x[0], x[4], c.x, s.x);
    spin(x[1], x[5], c.y, s.y);
    spin(x[2], x[6], c.z, s.z);
    spin(x[3], x[7], c.w, s.w);
  } else if constexpr (LAYOUT == kNear || LAYOUT == kFar) {
    constexpr int kParts = LAYOUT == kNear ? 1 : 2;  // of 128 dims
    float y[8];
#pragma unroll
    for (int g = 0; g < kParts; ++g) {
      const int d = 128 * g + 4 * lane;
      const bool upper = d >= pairs;
      const int other = upper ? d - pairs : d + pairs;  // (beyond 2 pairs: unused)
      float b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        b[i] = __shfl_sync(0xFFFFFFFFu, x[i], other >> 2);
        if constexpr (LAYOUT == kFar) {
          const float far = __shfl_sync(0xFFFFFFFFu, x[4 + i], other >> 2);
          if (other >= 128) b[i] = far;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) y[4 * g + i] = x[4 * g + i];
      if (d < 2 * pairs) {
        const float* at = row + (upper ? d - pairs : d);
        const float4 c = *reinterpret_cast<const float4*>(at), s = *reinterpret_cast<const float4*>(at + pairs);
        y[4 * g] = spun(x[4 * g], b[0], c.x, s.x, upper);
        y[4 * g + 1] = spun(x[4 * g + 1], b[1], c.y, s.y, upper);
        y[4 * g + 2] = spun(x[4 * g + 2], b[2], c.z, s.z, upper);
        y[4 * g + 3] = spun(x[4 * g + 3], b[3], c.w, s.w, upper);
      }
    }
#pragma unroll
    for (int i = 0; i < 4 * kParts; ++i) x[i] = y[i];
  }
}

__device__ __forceinline__ float square_sum(const float (&x)[8]) {
  float a = x[0] * x[0], b = x[4] * x[4];
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    a = fmaf(x[i], x[i], a);
    b = fmaf(x[4 + i], x[4 + i], b);
  }
  a += b;
#pragma unroll
  for (int d = 16; d; d >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, d);
  return a;
}
// 1 / sqrt(mean of squares + eps) of a warp's row
__device__ __forceinline__ float inverse_norm(const float (&x)[8], float eps) {
  float sum = square_sum(x);
  float unit = 1.0f;
  if (sum == __int_as_float(0x7F800000)) {  // above 2^63 or so the squares pass fp32's range, not their root
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * 0x1p-80f;
    sum = square_sum(y);
    unit = 0x1p-80f;
    eps = 0.0f;
  }
  return __frsqrt_rn(fmaf(sum, 1.0f / kHeadDim, eps)) * unit;
}

// A lane's weights of the norm.
struct Weights {
  float w[8];
  __device__ __forceinline__ void load(const float* at, int lane) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(at) + lane), b = __ldg(reinterpret_cast<const float4*>(at) + 32 + lane);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
  __device__ __forceinline__ void apply(float (&x)[8], float inv) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
  }
};

// ------------------------------------------------------------------ rows to rows

struct RotateParams {
  Turn turn;
  Rows q, k;
  uint8_t* q_out;
  uint8_t* k_out;
  const int* positions;
  int n, rows, q_heads, k_heads, group, q_groups, block_shift;
  unsigned n_mul, n_shift;  // division by n of row numbers, see Quotient
  int start[IQ_MAX_BATCH];
};
// floor(r / n) for r < 2^31: with s = floor(log2 n) and mul = ceil(2^(32+s) / n) < 2^32,
// umulhi(r, mul) >> s (its error is below r / 2^(32+s) < 1 / n); a shift for powers of two.
struct Quotient {
  unsigned mul = 0, shift = 0;
  explicit Quotient(int n) {
    while ((2LL << shift) <= n) ++shift;
    if (n & (n - 1)) mul = static_cast<unsigned>(((1ull << (32 + shift)) + n - 1) / n);
  }
};
__device__ __forceinline__ int divided(unsigned r, unsigned mul, unsigned shift) {
  return static_cast<int>((mul ? __umulhi(r, mul) : r) >> shift);
}

// A CTA takes a block of 2^block_shift token rows of (entries x rows) and a group of
// heads; a warp takes one row of one head at a time, eight (fp32: four) in flight.
template <int LAYOUT, bool F32>
__global__ void __launch_bounds__(256) rotate_kernel(const __grid_constant__ RotateParams p) {
  extern __shared__ __align__(16) float table[];
  constexpr int kInFlight = F32 ? 4 : 8;
  wait_for_last_kernel();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = blockIdx.x << p.block_shift, rows = min(1 << p.block_shift, p.rows - r0), mask = (1 << p.block_shift) - 1;
  const bool is_k = static_cast<int>(blockIdx.y) >= p.q_groups;
  const int head0 = (static_cast<int>(blockIdx.y) - (is_k ? p.q_groups : 0)) * p.group, all = is_k ? p.k_heads : p.q_heads;
  const int items = min(p.group, all - head0) << p.block_shift;
  const Rows in = is_k ? p.k : p.q;
  uint8_t* out = is_k ? p.k_out : p.q_out;
  const float* weight = is_k ? p.turn.k_weight : p.turn.q_weight;

  Raw<F32> raw[kInFlight];
  auto load = [&](int item0) {
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int item = item0 + 8 * i, r = item & mask, e = divided(r0 + r, p.n_mul, p.n_shift);
      if (item >= items || r >= rows) continue;
      raw[i].load(in.at + e * in.entry + (head0 + (item >> p.block_shift)) * in.head + (r0 + r - e * p.n) * in.row, lane);
    }
  };
  load(warp);
  Weights w;
  if (weight) w.load(weight, lane);
  if constexpr (LAYOUT != kNone) {
    fill_table(p.turn, table, rows, [&](int r) {
      const int e = divided(r0 + r, p.n_mul, p.n_shift);
      return static_cast<long long>(p.positions ? __ldg(p.positions + r0 + r) : p.start[e]) + (p.positions ? 0 : r0 + r - e * p.n);
    });
    __syncthreads();
  }
  for (int item0 = warp;; ) {
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int item = item0 + 8 * i, r = item & mask;
      if (item >= items || r >= rows) continue;
      float x[8];
      raw[i].get(x);
      if (weight) w.apply(x, inverse_norm(x, p.turn.eps));
      turn_row<LAYOUT>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, lane);
      const int e = divided(r0 + r, p.n_mul, p.n_shift);
      const long long to = (static_cast<long long>(e) * all + head0 + (item >> p.block_shift)) * p.n + (r0 + r - e * p.n);
      Raw<F32>::store(out + to * kHeadDim * Raw<F32>::kBytes, lane, x);
    }
    item0 += 8 * kInFlight;
    if (item0 >= items) break;
    load(item0);
  }
}

// ------------------------------------------------------------------ rows into pages

struct RotaryAppendParams {
  AppendParams a;  // (keys and values: unused)
  Turn turn;
  Rows q, k, v;
  uint8_t* q_out;
  const int* positions;
  int q_heads, group;
};

// CTA (page of a segment, y, segment): the keys of kv head y, the values of kv head y -
// heads, or the queries of a group of heads at the page's new rows.  A page's rows
// stay in registers as they came, eight to a warp; keys are turned twice, for the page's
// largest element and for the codes, which takes fewer registers than keeping them in
// fp32.  Codes are rounded from fp32, once.
template <int LAYOUT>
__global__ void __launch_bounds__(256, 3) paged_append_rotary_kernel(const __grid_constant__ RotaryAppendParams p) {
  extern __shared__ __align__(16) float table[];  // of the page's new rows
  __shared__ uint32_t tops[8];
  wait_for_last_kernel();
  const Segment sg = p.a.seg[blockIdx.z];
  const int k = blockIdx.x, heads = p.a.heads, y = blockIdx.y;
  const int off = sg.pos % kPage;                 // rows of the segment's first page before it
  const int begin = k == 0 ? off : 0;             // this page's new rows: [begin, end)
  const int end = min(kPage, off + sg.rows - k * kPage);
  if (end <= begin) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = sg.row0 + k * kPage - off;     // the call's row of this page's row 0
  const bool is_v = y >= heads && y < 2 * heads;
  Raw<false> raw[8];
  auto fill = [&]() {
    if constexpr (LAYOUT != kNone) {
      fill_table(p.turn, table, end - begin, [&](int r) {
        return static_cast<long long>(p.positions ? __ldg(p.positions + static_cast<long long>(sg.entry) * p.a.n + row0 + begin + r)
                                                  : sg.pos - off + k * kPage + begin + r);
      });
      __syncthreads();
    }
  };
  auto turned = [&](const Raw<false>& from, int r, const float* weight, const Weights& w, float inv, float (&x)[8]) {  // r: of the new rows
    from.get(x);
    if (weight) w.apply(x, inv);
    turn_row<LAYOUT>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, lane);
  };

  if (y >= 2 * heads) {
    // ---------------------------------------------------------------- queries
    const int head0 = (y - 2 * heads) * p.group, rows = end - begin, items = min(p.group, p.q_heads - head0) * rows;
    const unsigned mul = 0xFFFFFFFFu / rows + 1;  // item / rows = umulhi(item, mul): item < 2^16, rows <= 64 (rows 1: mul 0)
    auto head_of = [&](int item) { return rows == 1 ? item : static_cast<int>(__umulhi(item, mul)); };
    auto load = [&](int item0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int item = item0 + 8 * i, h = head_of(item), r = item - h * rows;
        if (item < items) raw[i].load(p.q.at + sg.entry * p.q.entry + (head0 + h) * p.q.head + (row0 + begin + r) * p.q.row, lane);
      }
    };
    load(warp);
    Weights w;
    if (p.turn.q_weight) w.load(p.turn.q_weight, lane);
    fill();
    for (int item0 = warp;;) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int item = item0 + 8 * i, h = head_of(item), r = item - h * rows;
        if (item >= items) break;
        float x[8];
        raw[i].get(x);
        if (p.turn.q_weight) w.apply(x, inverse_norm(x, p.turn.eps));
        turn_row<LAYOUT>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, lane);
        const long long to = (static_cast<long long>(sg.entry) * p.q_heads + head0 + h) * p.a.n + row0 + begin + r;
        Raw<false>::store(p.q_out + to * kHeadDim * 2, lane, x);
      }
      item0 += 64;
      if (item0 >= items) break;
      load(item0);
    }
    return;
  }
  // ---------------------------------------------------------------- keys, values
  const int h = is_v ? y - heads : y;
  const int page = sg.page + k, from = k == 0 ? sg.from : page;
  const long long at = static_cast<long long>(page) * heads + h, at_from = static_cast<long long>(from) * heads + h;
  uint8_t* codes = (is_v ? p.a.v_codes : p.a.k_codes) + at * kPageBytes;
  float* scales = is_v ? p.a.v_scales : p.a.k_scales;
  {
    const Rows& in = is_v ? p.v : p.k;
    const uint8_t* rows = in.at + sg.entry * in.entry + h * in.head;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = warp + 8 * i;
      raw[i].x[0] = raw[i].x[1] = make_uint2(0, 0);
      if (r >= begin && r < end) raw[i].load(rows + (row0 + r) * in.row, lane);
    }
  }
  Weights w;
  float inv[8] = {};
  uint32_t top = 0;
  bool odd;  // not a number, held as 0, or infinite, held as the largest value
  if (is_v) {
    auto largest = [&]() {
      top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(make_uint4(raw[i].x[0].x, raw[i].x[0].y, raw[i].x[1].x, raw[i].x[1].y)));
    };
    largest();
    odd = top >= 0x7F80u;
    if (odd) {  // rare
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int g = 0; g < 2; ++g) raw[i].x[g] = make_uint2(drop_non_finite(raw[i].x[g].x), drop_non_finite(raw[i].x[g].y));
      largest();
    }
    top <<= 16;
  } else {
    if (p.turn.k_weight) w.load(p.turn.k_weight, lane);
    fill();
    uint32_t bits = 0;
    float most = 0.0f;  // (a maximum leaves out what is not a number)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = warp + 8 * i;
      if (r < begin || r >= end) continue;
      float x[8];
      if (p.turn.k_weight) {
        raw[i].get(x);
        inv[i] = inverse_norm(x, p.turn.eps);
      }
      turned(raw[i], r - begin, p.turn.k_weight, w, inv[i], x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        most = fmaxf(most, fabsf(x[j]));
        bits = max(bits, __float_as_uint(x[j]) & 0x7FFFFFFFu);
      }
    }
    odd = bits >= 0x7F800000u;
    top = min(__float_as_uint(most), 0x7F7FFFFFu);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, tops[i]);
  int e = least_exponent(top);
  const bool beyond = e > kEMax;
  e = min(e, kEMax);
  const int old = begin > 0 ? exponent_of(scales[at_from]) : e;
  e = max(e, old);
  const float unit = power2(-e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = warp + 8 * i;
    if (r < begin || r >= end) continue;
    float x[8];
    if (is_v) raw[i].get(x);
    else turned(raw[i], r - begin, p.turn.k_weight, w, inv[i], x);
    if (odd)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] != x[j] ? 0.0f : x[j];
#pragma unroll
    for (int g = 0; g < 2; ++g)
      *reinterpret_cast<uint32_t*>(codes + r * kHeadDim + 128 * g + 4 * lane) =
          e4m3x2(x[4 * g] * unit, x[4 * g + 1] * unit) | e4m3x2(x[4 * g + 2] * unit, x[4 * g + 3] * unit) << 16;
  }
  upkeep((is_v ? p.a.v_codes : p.a.k_codes) + at_from * kPageBytes, codes, begin, end, from != page, old, e);
  if (odd || beyond) atomicOr(p.a.status, IQ_STATUS_RANGE);
  __syncthreads();  // the old scale has been read by every thread
  if (threadIdx.x == 0) {
    scales[at] = power2(e);
    if (y == 0) p.a.table[static_cast<long long>(sg.slot) * p.a.max_pages + sg.pos / kPage + k] = page;
  }
}


// The turns per position of a frequency, modulo 1, times 2^64.
struct TurnsParams {
  int n;
  unsigned long long turns[kHeadDim / 2];
};
__global__ void turns_kernel(const __grid_constant__ TurnsParams p, unsigned long long* out) {
  wait_for_last_kernel();
  if (threadIdx.x < p.n) out[threadIdx.x] = p.turns[threadIdx.x];
}

// ------------------------------------------------------------------ host

Layout layout_of(const iq_rotary* r) {
  const int pairs = r->rotary_dim / 2;
  return pairs == 0 ? kNone : r->interleaved ? kPairs : pairs == 128 ? kAcross : pairs <= 64 ? kNear : kFar;
}
Turn turn_of(const iq_rotary* r) {
  return {reinterpret_cast<const unsigned long long*>(r->turns), r->q_weight, r->k_weight, r->amplitude, r->eps, r->rotary_dim / 2};
}

int check_rotary(const iq_rotary* r) {
  clear_error();
  if (!r) return fail(IQ_ERR_INVALID_ARG, "null rotary plan");
  if (r->rotary_dim < 0 || r->rotary_dim > kHeadDim || r->rotary_dim % 16)
    return fail(IQ_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 in [0, 256]");
  if (r->interleaved != 0 && r->interleaved != 1) return fail(IQ_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (r->rotary_dim > 0) {
    if (!r->turns) return fail(IQ_ERR_INVALID_ARG, "null turns");
    if (misaligned(r->turns, 8)) return fail(IQ_ERR_INVALID_ARG, "turns not 8-byte aligned");
    if (!(r->amplitude - r->amplitude == 0.0f)) return fail(IQ_ERR_INVALID_ARG, "amplitude is not finite");
  }
  if (r->q_weight || r->k_weight) {
    if (misaligned(r->q_weight) || misaligned(r->k_weight)) return fail(IQ_ERR_INVALID_ARG, "weights not 16-byte aligned");
    if (!(r->eps >= 1e-30f && r->eps < __builtin_huge_valf())) return fail(IQ_ERR_INVALID_ARG, "eps must be 1e-30 or more, and finite");
  }
  return IQ_OK;
}

// Rows [entries][heads][n] of `size`-byte elements: aligned, and where in memory they are.
int check_rows(const iq_rows* r, int entries, int heads, int n, int size, const char* name, Rows* rows, Range* range) {
  *range = {nullptr, 0};
  if (!r || !r->at) return fail(IQ_ERR_INVALID_ARG, std::string("null ") + name);
  const int64_t strides[3] = {r->entry, r->head, r->row};
  const int counts[3] = {entries, heads, n};
  int64_t in_bytes[3], last = kHeadDim * size;
  bool bad = misaligned(r->at);
  for (int i = 0; i < 3; ++i) {
    if (counts[i] <= 1) {  // never stepped by
      in_bytes[i] = 0;
      continue;
    }
    if (strides[i] < 0 || strides[i] > (1LL << 40)) return fail(IQ_ERR_INVALID_ARG, std::string(name) + ": stride outside [0, 2^40]");
    in_bytes[i] = strides[i] * size;
    bad |= in_bytes[i] % 16 != 0;
    last += in_bytes[i] * (counts[i] - 1);
  }
  if (bad) return fail(IQ_ERR_INVALID_ARG, std::string(name) + ": rows not 16-byte aligned");
  *rows = {static_cast<const uint8_t*>(r->at), in_bytes[0], in_bytes[1], in_bytes[2]};
  *range = {r->at, static_cast<size_t>(last)};
  return IQ_OK;
}
bool overlap(Range a, Range b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return x < y + b.bytes && y < x + a.bytes;
}

template <bool F32>
const void* rotate_kernel_of(Layout l) {
  switch (l) {
    case kPairs: return reinterpret_cast<const void*>(&rotate_kernel<kPairs, F32>);
    case kNear: return reinterpret_cast<const void*>(&rotate_kernel<kNear, F32>);
    case kAcross: return reinterpret_cast<const void*>(&rotate_kernel<kAcross, F32>);
    case kFar: return reinterpret_cast<const void*>(&rotate_kernel<kFar, F32>);
    default: return reinterpret_cast<const void*>(&rotate_kernel<kNone, F32>);
  }
}
const void* append_kernel_of(Layout l) {
  switch (l) {
    case kPairs: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kPairs>);
    case kNear: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kNear>);
    case kAcross: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kAcross>);
    case kFar: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kFar>);
    default: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kNone>);
  }
}

struct RotaryAppend {
  Turn turn;
  Layout layout;
  Rows q, k, v;
  uint8_t* q_out;
  const int* positions;
  int q_heads;
};
cudaError_t launch_append_rotary(const AppendParams& a, int widest, int segs, cudaStream_t stream, const void* more) {
  const RotaryAppend& m = *static_cast<const RotaryAppend*>(more);
  RotaryAppendParams p;
  p.a = a;
  p.turn = m.turn;
  p.q = m.q;
  p.k = m.k;
  p.v = m.v;
  p.q_out = m.q_out;
  p.positions = m.positions;
  p.q_heads = m.q_heads;
  p.group = 8;
  int rows = 0;  // the most new rows of a page
  for (int i = 0; i < segs; ++i) rows = std::max(rows, std::min(kPage, a.seg[i].rows));
  const int smem = rows * 2 * m.turn.pairs * static_cast<int>(sizeof(float));
  const void* kernel = append_kernel_of(m.layout);
  static std::atomic<uint64_t> seen[kFar + 1] = {};
  const cudaError_t e = smem > 48 * 1024 ? allow_smem(kernel, 64 * 1024, seen[m.layout]) : cudaSuccess;
  void* args[] = {&p};
  return e == cudaSuccess ? launch_after(kernel, dim3(widest, 2 * a.heads + (m.q_heads + p.group - 1) / p.group, segs), 256, smem, stream, args) : e;
}

}  // namespace
}  // namespace paged
}  // namespace iq

using namespace iq;
using namespace iq::paged;

extern "C" {

int iq_rotary_frequencies(int rotary_dim, double base, int scaling, double factor, double original, double low, double high,
                          double* frequencies, double* amplitude) {
  clear_error();
  if (!frequencies || !amplitude) return fail(IQ_ERR_INVALID_ARG, "null frequencies/amplitude");
  if (rotary_dim <= 0 || rotary_dim > kHeadDim || rotary_dim % 16)
    return fail(IQ_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 in [16, 256]");
  if (scaling < IQ_SCALING_NONE || scaling > IQ_SCALING_BANDED) return fail(IQ_ERR_INVALID_ARG, "unknown scaling");
  if (!(base > 1.0 && std::isfinite(base))) return fail(IQ_ERR_INVALID_ARG, "base must be finite and above 1");
  const bool by_length = scaling == IQ_SCALING_YARN || scaling == IQ_SCALING_BANDED;
  if (scaling != IQ_SCALING_NONE && !(factor >= 1.0 && std::isfinite(factor))) return fail(IQ_ERR_INVALID_ARG, "factor must be 1 or more");
  if (by_length && !(original >= 1.0 && std::isfinite(original))) return fail(IQ_ERR_INVALID_ARG, "original must be 1 or more");
  if (by_length && !(low > 0.0 && high > low && std::isfinite(high))) return fail(IQ_ERR_INVALID_ARG, "0 < low < high is needed");
  const double pi2 = 6.283185307179586476925;
  const int n = rotary_dim / 2;
  if (scaling == IQ_SCALING_NTK) base *= std::pow(factor, static_cast<double>(rotary_dim) / (rotary_dim - 2));
  // YaRN's ramp runs between the pairs that turn `high` and `low` times within the original length
  auto pair_of = [&](double turns) { return n * std::log(original / (turns * pi2)) / std::log(base); };
  double first = 0.0, last = 0.0;
  if (scaling == IQ_SCALING_YARN) {
    first = std::max(std::floor(pair_of(high)), 0.0);
    last = std::min(std::ceil(pair_of(low)), static_cast<double>(rotary_dim - 1));
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -static_cast<double>(i) / n);
    double keep = 1.0;  // the share of f; the rest is stretched
    if (scaling == IQ_SCALING_LINEAR) keep = 0.0;
    if (scaling == IQ_SCALING_YARN) keep = 1.0 - std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
    if (scaling == IQ_SCALING_BANDED) keep = std::min(std::max((original * f / pi2 - low) / (high - low), 0.0), 1.0);
    frequencies[i] = keep == 1.0 ? f : f * keep + f / factor * (1.0 - keep);
  }
  *amplitude = scaling == IQ_SCALING_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return IQ_OK;
}

int iq_rotary_turns(const double* frequencies, int pairs, uint64_t* turns, iq_stream_t stream) {
  clear_error();
  if (!frequencies || !turns) return fail(IQ_ERR_INVALID_ARG, "null frequencies/turns");
  if (pairs <= 0 || pairs > kHeadDim / 2) return fail(IQ_ERR_INVALID_ARG, "pairs outside [1, 128]");
  if (misaligned(turns, 8)) return fail(IQ_ERR_INVALID_ARG, "turns not 8-byte aligned");
  TurnsParams p;
  p.n = pairs;
  for (int i = 0; i < pairs; ++i) {
    if (!std::isfinite(frequencies[i])) return fail(IQ_ERR_INVALID_ARG, "a frequency is not finite");
    const double t = frequencies[i] / 6.283185307179586476925, part = t - std::floor(t);  // in [0, 1]
    p.turns[i] = part < 1.0 ? static_cast<unsigned long long>(std::ldexp(part, 64)) : 0;
  }
  unsigned long long* out = reinterpret_cast<unsigned long long*>(turns);
  void* args[] = {&p, &out};
  IQ_CUDA(launch_after(reinterpret_cast<const void*>(&turns_kernel), dim3(1), kHeadDim / 2, 0, static_cast<cudaStream_t>(stream), args));
  return IQ_OK;
}

int iq_rotary_apply(const iq_rotary* rotary, int dtype, const iq_rows* q, int q_heads, const iq_rows* k, int k_heads, int entries,
                    int n, const int32_t* start, const int32_t* positions, void* q_out, void* k_out, iq_stream_t stream) {
  int st = check_rotary(rotary);
  if (st != IQ_OK) return st;
  if (dtype != IQ_DTYPE_BF16 && dtype != IQ_DTYPE_F32) return fail(IQ_ERR_INVALID_ARG, "unknown dtype");
  if (q_heads < 0 || k_heads < 0 || entries < 0 || n < 0) return fail(IQ_ERR_INVALID_ARG, "negative size");
  if (entries > IQ_MAX_BATCH) return fail(IQ_ERR_INVALID_ARG, "entries above IQ_MAX_BATCH");
  if (start && positions) return fail(IQ_ERR_INVALID_ARG, "give either start or positions");
  if (misaligned(positions, 4)) return fail(IQ_ERR_INVALID_ARG, "positions not 4-byte aligned");
  if (static_cast<long long>(entries) * n >= (1LL << 30)) return fail(IQ_ERR_UNSUPPORTED, "entries * n exceeds 2^30");
  if (q_heads > (1 << 16) || k_heads > (1 << 16)) return fail(IQ_ERR_UNSUPPORTED, "too many heads");
  if (entries == 0 || n == 0 || q_heads + k_heads == 0) return IQ_OK;
  RotateParams p;
  const int size = dtype == IQ_DTYPE_F32 ? 4 : 2;
  Range in[2] = {}, out[2] = {};
  p.q = p.k = {nullptr, 0, 0, 0};
  if (q_heads > 0 && (st = check_rows(q, entries, q_heads, n, size, "q", &p.q, &in[0])) != IQ_OK) return st;
  if (k_heads > 0 && (st = check_rows(k, entries, k_heads, n, size, "k", &p.k, &in[1])) != IQ_OK) return st;
  const size_t head = static_cast<size_t>(entries) * n * kHeadDim * size;
  if (q_heads > 0) out[0] = {q_out, head * q_heads};
  if (k_heads > 0) out[1] = {k_out, head * k_heads};
  for (const Range& o : out) {
    if (o.bytes && !o.at) return fail(IQ_ERR_INVALID_ARG, "null output");
    if (misaligned(o.at)) return fail(IQ_ERR_INVALID_ARG, "output not 16-byte aligned");
    for (const Range& i : in)
      if (o.bytes && i.bytes && overlap(o, i)) return fail(IQ_ERR_INVALID_ARG, "an output overlaps an input");
  }
  if (out[0].bytes && out[1].bytes && overlap(out[0], out[1])) return fail(IQ_ERR_INVALID_ARG, "the outputs overlap");
  p.turn = turn_of(rotary);
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.positions = positions;
  p.n = n;
  p.rows = entries * n;
  p.q_heads = q_heads;
  p.k_heads = k_heads;
  const Quotient by_n(n);
  p.n_mul = by_n.mul;
  p.n_shift = by_n.shift;
  for (int i = 0; i < entries; ++i) p.start[i] = start ? start[i] : 0;
  p.group = 16;
  p.block_shift = 5;
  auto groups = [&](int heads) { return (heads + p.group - 1) / p.group; };
  auto blocks = [&]() { return (p.rows + (1 << p.block_shift) - 1) >> p.block_shift; };
  while (p.block_shift > 0 && static_cast<long long>(blocks()) * (groups(q_heads) + groups(k_heads)) < 4ll * num_sms()) --p.block_shift;
  if (p.block_shift == 0) p.group = 8;
  p.q_groups = groups(q_heads);
  const Layout layout = layout_of(rotary);
  void* args[] = {&p};
  IQ_CUDA(launch_after(dtype == IQ_DTYPE_F32 ? rotate_kernel_of<true>(layout) : rotate_kernel_of<false>(layout),
                       dim3(blocks(), p.q_groups + groups(k_heads)), 256, static_cast<int>(sizeof(float)) * (2 * p.turn.pairs << p.block_shift),
                       static_cast<cudaStream_t>(stream), args));
  launched_outputs(stream, out[0], out[1]);
  return IQ_OK;
}

int iq_paged_append_rotary(iq_paged* c, const iq_rotary* rotary, const iq_rows* q, int q_heads, const iq_rows* k, const iq_rows* v, int n,
                           const int32_t* slots, const int32_t* counts, int n_slots, const int32_t* positions, void* q_out,
                           iq_stream_t stream) {
  int st = check_rotary(rotary);
  if (st != IQ_OK) return st;
  st = check_append(c, k ? k->at : nullptr, v ? v->at : nullptr, n, slots, counts, n_slots);
  if (st != IQ_OK) return st;
  if (q_heads < 0 || q_heads > (1 << 16)) return fail(IQ_ERR_INVALID_ARG, "bad q_heads");
  if (misaligned(positions, 4)) return fail(IQ_ERR_INVALID_ARG, "positions not 4-byte aligned");
  if (n_slots == 0 || n == 0) return IQ_OK;
  RotaryAppend m;
  m.turn = turn_of(rotary);
  m.layout = layout_of(rotary);
  Range in[3] = {};
  m.q = {nullptr, 0, 0, 0};
  if (q_heads > 0 && (st = check_rows(q, n_slots, q_heads, n, 2, "q", &m.q, &in[0])) != IQ_OK) return st;
  if ((st = check_rows(k, n_slots, c->kv_heads, n, 2, "k", &m.k, &in[1])) != IQ_OK) return st;
  if ((st = check_rows(v, n_slots, c->kv_heads, n, 2, "v", &m.v, &in[2])) != IQ_OK) return st;
  const Range out{q_out, q_heads > 0 ? static_cast<size_t>(n_slots) * q_heads * n * kHeadDim * 2 : 0};
  if (out.bytes) {
    if (!q_out) return fail(IQ_ERR_INVALID_ARG, "null q_out");
    if (misaligned(q_out)) return fail(IQ_ERR_INVALID_ARG, "q_out not 16-byte aligned");
    for (const Range& i : in)
      if (i.bytes && overlap(out, i)) return fail(IQ_ERR_INVALID_ARG, "q_out overlaps an input");
  }
  m.q_out = static_cast<uint8_t*>(q_out);
  m.positions = positions;
  m.q_heads = q_heads;
  st = do_append(c, nullptr, nullptr, n, slots, counts, n_slots, stream, launch_append_rotary, &m);
  if (st == IQ_OK) launched_outputs(stream, out);
  return st;
}

}  // extern "C"
