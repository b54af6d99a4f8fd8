// libiqkv: rotary positions of queries and keys, each head's vector normed in the
// same pass, and the paged cache's append that takes a projection's rows as they are.
//
// Mathematics.  y = x * (mean(x^2) + eps)^-1/2 * weight (where a weight is given), then
// the pairs (a, b) of the leading rotary dims become (a c - b s, a s + b c) * amplitude
// with c, s the cosine and sine of position * frequency.  fp32 throughout, rounded once;
// the codes and page exponents that this leaves open come from fp64 (see Bound, exact_codes).
//
// Angles.  A far position times a frequency has a fraction of a turn that fp32 cannot
// tell (at 2^20, 2^-4 of a radian is lost), so a frequency is held as its turns per
// position modulo 1 in 64 bits of fixed point: the product with a position, modulo
// 2^64, is the angle modulo a turn, off by at most position * 2^-64 and what the
// frequency itself was off.  One integer product; no table in memory.
//
// Rows.  Eight lanes hold a row, 32 elements each in pieces of 16 bytes, 128 bytes apart:
// what a row costs besides its elements (its address, the norm's sum over lanes and root)
// a warp then does for four rows at once.  With a row per warp that was most of 210
// instructions a row, and 16 x 2048 rows of 18 heads took 202 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "iq_pages.cuh"

namespace iq {
namespace paged {
namespace {

struct Turn {
  const unsigned long long* turns;
  const float* q_weight;
  const float* k_weight;
  double amplitude, eps;
  float unit_off;  // what cosines and sines may be off by, in 2^-24 of the amplitude
  int pairs;
};
struct Rows {
  const uint8_t* at;
  long long entry, head, row;  // strides in bytes
};

// Lane l of eight holds V elements of each of C pieces: c * 8V + V * l + i.
template <bool F32>
struct Raw {
  static constexpr int V = F32 ? 4 : 8, C = 32 / V, kRowBytes = kHeadDim * (F32 ? 4 : 2);
  uint4 x[C];
  __device__ __forceinline__ void load(const uint8_t* row, int l) {
#pragma unroll
    for (int c = 0; c < C; ++c) x[c] = __ldcs(reinterpret_cast<const uint4*>(row + c * 128 + l * 16));
  }
  __device__ __forceinline__ void get(float (&y)[32]) const {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
          y[4 * c + i] = __uint_as_float(w[i]);
        } else {
          y[8 * c + 2 * i] = __uint_as_float(w[i] << 16);
          y[8 * c + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(uint8_t* row, int l, const float (&y)[32]) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (F32) w[i] = __float_as_uint(y[4 * c + i]);
        else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(y[8 * c + 2 * i + 1]), "f"(y[8 * c + 2 * i]));
      }
      *reinterpret_cast<uint4*>(row + c * 128 + l * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

// Where the pairs of a lane's elements are.  With pairs = 8V * K + V * shift:
enum Layout {
  kNone,   // nothing turns
  kPairs,  // elements 2i and 2i + 1
  kHere,   // halves, shift 0: K pieces on, in the same lane
  kSwap,   // halves, K = 0, shift 4: the same piece of the lane four on
  kShift   // halves, any other: K pieces on, or one more, of the lane `shift` on
};

// Cosine and sine, times the amplitude, of an angle of a / 2^64 turns.  The nearest
// quarter is taken off, and of what is left, t = h + l with |t| <= pi / 4 and l of half a step
// of h or 2^-32 of a turn, Taylor's series: what follows their first terms is below 2^-3 of
// them, so the results are a half and some hundredths of a step off at most (codes are rounded
// from what they turn: the nearer, the fewer land on the wrong side of a border).  Of the
// angle's lower half 23 bits count, so that it is held to 2^-55 of a turn (without them the sine of
// 10^-4 radians was off by 10^-5 of it).
__device__ __forceinline__ float2 unit_at(unsigned long long angle, float amplitude) {
  const unsigned a = static_cast<unsigned>(angle >> 32), quarter = (a + 0x20000000u) >> 30;
  const int rest = static_cast<int>(a - (quarter << 30));
  constexpr float kHi = 0x1.921fb6p-30f, kLo = -0x1.777a5cp-55f;  // 2 pi / 2^32
  const float lower = __uint_as_float(0x3F800000u | static_cast<unsigned>(angle) >> 9) - 1.0f;
  const float u = static_cast<float>(rest), v = static_cast<float>(rest - static_cast<int>(u)) + lower;
  const float h = u * kHi, l = fmaf(u, kHi, -h) + fmaf(u, kLo, v * kHi);
  const float h2 = h * h, rounded = fmaf(h, h, -h2);  // h^2 = h2 + rounded
  float p = fmaf(h2, 1.0f / 362880, -1.0f / 5040);
  p = fmaf(h2, p, 1.0f / 120);
  p = fmaf(h2, p, -1.0f / 6);
  const float s1 = fmaf(h * h2, p, l * fmaf(h2, -0.5f, 1.0f));  // sin t - h
  float q = fmaf(h2, -1.0f / 3628800, 1.0f / 40320);
  q = fmaf(h2, q, -1.0f / 720);
  q = fmaf(h2, q, 1.0f / 24);
  const float c0 = fmaf(h2, -0.5f, 1.0f), c1 = fmaf(h2, -0.5f, 1.0f - c0);  // 1 - h2 / 2 = c0 + c1
  const float c2 = c1 + fmaf(h2 * h2, q, -fmaf(0.5f, rounded, l * h));      // cos t - c0
  float s = fmaf(amplitude, h, amplitude * s1), c = fmaf(amplitude, c0, amplitude * c2);
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) {
    c = -c;
    s = -s;
  }
  return make_float2(c, s);
}
// Row r of the table: the cosines of its pairs, then their sines.  In halves' layouts a
// lane reads V of them, four at a time: the first fours of all lanes stand side by side,
// then the second fours, so that eight lanes read 128 bytes in a row.
template <int V>
__device__ __forceinline__ int table_place(int j, int pairs) {
  return V == 8 ? (j & 4) * (pairs / 8) + (j >> 3) * 4 + (j & 3) : j;
}
template <int V, typename Position>
__device__ __forceinline__ void fill_table(const Turn& t, float* table, int rows, Position position) {
  const float amplitude = static_cast<float>(t.amplitude);
  int r = threadIdx.x / t.pairs, j = threadIdx.x - r * t.pairs;
  const int down = blockDim.x / t.pairs, across = blockDim.x - down * t.pairs;
  while (r < rows) {
    const long long p = position(r);
    const float2 u = unit_at(static_cast<unsigned long long>(p) * __ldg(t.turns + j), amplitude);
    const int to = 2 * r * t.pairs + table_place<V>(j, t.pairs);
    table[to] = u.x;
    table[to + t.pairs] = u.y;
    r += down;
    j += across;
    if (j >= t.pairs) {
      j -= t.pairs;
      ++r;
    }
  }
}
template <int LAYOUT, bool F32>
constexpr int kTableOrder = LAYOUT == kPairs ? 1 : Raw<F32>::V;

// a c - b s, or a c + b s.  EXACT: off by the roundings of its sum and of what makes the
// first product's good (for float32 results and codes, see unit_at).
template <bool EXACT>
__device__ __forceinline__ float less(float a, float c, float b, float s) {
  const float t = b * s, x = fmaf(a, c, -t);
  if constexpr (EXACT) return x - fmaf(b, s, -t);
  return x;
}

// What looks at the results of turn_row: y0 and y1 of elements e and e + 1, which were turned from
// elements whose magnitudes' sums are m0 and m1, or do not turn.
struct NoLook {
  __device__ __forceinline__ void turned(int, float, float, float, float) {}
  __device__ __forceinline__ void rest(int, float, float) {}
};

// A row's vector, turned (a whole warp, four rows).  row: its cosines, then its sines.
template <int LAYOUT, int K, bool F32, bool EXACT, class Look>
__device__ __forceinline__ void turn_row(float (&x)[32], const float* row, int pairs, int l, Look& look) {
  constexpr int V = Raw<F32>::V, C = Raw<F32>::C;
  auto rest = [&](int c) {  // a piece that does not turn
#pragma unroll
    for (int i = 0; i < V; i += 2) look.rest(V * c + i, x[V * c + i], x[V * c + i + 1]);
  };
  if constexpr (LAYOUT == kNone) {
#pragma unroll
    for (int c = 0; c < C; ++c) rest(c);
  } else if constexpr (LAYOUT == kPairs) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int j = (c * 8 * V + V * l) / 2;
      if (j >= pairs) {
        rest(c);
        continue;
      }
      float co[4], si[4];
      if constexpr (F32) {
        const float2 a = *reinterpret_cast<const float2*>(row + j), b = *reinterpret_cast<const float2*>(row + pairs + j);
        co[0] = a.x, co[1] = a.y, si[0] = b.x, si[1] = b.y;
      } else {
        const float4 a = *reinterpret_cast<const float4*>(row + j), b = *reinterpret_cast<const float4*>(row + pairs + j);
        co[0] = a.x, co[1] = a.y, co[2] = a.z, co[3] = a.w, si[0] = b.x, si[1] = b.y, si[2] = b.z, si[3] = b.w;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float a = x[V * c + 2 * i], b = x[V * c + 2 * i + 1];
        x[V * c + 2 * i] = less<EXACT>(a, co[i], b, si[i]);
        x[V * c + 2 * i + 1] = less<EXACT>(a, si[i], -b, co[i]);
        const float m = fabsf(a) + fabsf(b);
        look.turned(V * c + 2 * i, x[V * c + 2 * i], m, x[V * c + 2 * i + 1], m);
      }
    }
  } else if constexpr (LAYOUT == kHere) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float* at = row + i * (pairs / V) + (c * 8 + l) * 4;
        const float4 co = *reinterpret_cast<const float4*>(at), si = *reinterpret_cast<const float4*>(at + pairs);
        const float cs[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
        float m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = x[V * c + i + k], b = x[V * (c + K) + i + k];
          x[V * c + i + k] = less<EXACT>(a, cs[k], b, ss[k]);
          x[V * (c + K) + i + k] = less<EXACT>(a, ss[k], -b, cs[k]);
          m[k] = fabsf(a) + fabsf(b);
        }
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const int e = V * c + i + k, f = e + V * K;
          look.turned(e, x[e], m[k], x[e + 1], m[k + 1]);
          look.turned(f, x[f], m[k], x[f + 1], m[k + 1]);
        }
      }
    }
#pragma unroll
    for (int c = 2 * K; c < C; ++c) rest(c);
  } else if constexpr (LAYOUT == kSwap || LAYOUT == kShift) {
    const int shift = pairs / V - 8 * K, lane = threadIdx.x & 31;
    const int up = (lane & 24) + ((l + shift) & 7), down = (lane & 24) + ((l - shift) & 7);
    const int carry = l + shift >= 8, borrow = l < shift;
    constexpr int kPieces = LAYOUT == kSwap ? 1 : 2 * K + 2 < C ? 2 * K + 2 : C;  // that turn
    float from_up[kPieces * V], from_down[kPieces * V];
#pragma unroll
    for (int i = 0; i < kPieces * V; ++i) {
      from_up[i] = __shfl_sync(0xFFFFFFFFu, x[i], up);
      if constexpr (LAYOUT == kShift) from_down[i] = __shfl_sync(0xFFFFFFFFu, x[i], down);
    }
#pragma unroll
    for (int c = 0; c < kPieces; ++c) {
      const int unit = c * 8 + l, half = pairs / V;
      if (unit >= 2 * half) {
        rest(c);
        continue;
      }
      const bool upper = unit >= half;
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float* at = row + i * half + (upper ? unit - half : unit) * 4;
        const float4 co = *reinterpret_cast<const float4*>(at), si = *reinterpret_cast<const float4*>(at + pairs);
        const float cs[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
        float m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float b;
          if constexpr (LAYOUT == kSwap) {
            b = from_up[i + k];
          } else {
            // (pieces that are not there belong to units beyond the pairs)
            constexpr int kLast = kPieces - 1;
            const int e = i + k;
            const float on = carry ? from_up[V * (c + K + 1 < kLast ? c + K + 1 : kLast) + e] : from_up[V * (c + K < kLast ? c + K : kLast) + e];
            const float back = borrow ? from_down[V * (c - K - 1 > 0 ? c - K - 1 : 0) + e] : from_down[V * (c - K > 0 ? c - K : 0) + e];
            b = upper ? back : on;
          }
          m[k] = fabsf(x[V * c + i + k]) + fabsf(b);
          x[V * c + i + k] = less<EXACT>(x[V * c + i + k], cs[k], upper ? -b : b, ss[k]);
        }
        const int e = V * c + i;
        look.turned(e, x[e], m[0], x[e + 1], m[1]);
        look.turned(e + 2, x[e + 2], m[2], x[e + 3], m[3]);
      }
    }
#pragma unroll
    for (int c = kPieces; c < C; ++c) rest(c);
  }
}

__device__ __forceinline__ float square_sum(const float (&x)[32], float unit) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (x[i] * unit) * (x[i] * unit);
#pragma unroll
  for (int i = 8; i < 32; ++i) a[i & 7] = fmaf(x[i] * unit, x[i] * unit, a[i & 7]);
  float sum = ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
#pragma unroll
  for (int d = 4; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  return sum;
}
// 1 / sqrt(mean of squares + eps) of each of a warp's four rows
__device__ __forceinline__ float inverse_norm(const float (&x)[32], float eps) {
  const float sum = square_sum(x, 1.0f);
  float inv = __frsqrt_rn(fmaf(sum, 1.0f / kHeadDim, eps));
  if (__any_sync(0xFFFFFFFFu, sum == __int_as_float(0x7F800000))) {  // above 2^63 or so the squares pass fp32's range, not their root
    const float small = square_sum(x, 0x1p-80f);
    if (sum == __int_as_float(0x7F800000)) inv = __frsqrt_rn(fmaf(small, 1.0f / kHeadDim, eps * 0x1p-80f * 0x1p-80f)) * 0x1p-80f;
  }
  return inv;
}

// A row times the norm's weights, which are in shared memory (in registers they would
// leave room for two CTAs instead of three), in an order like the table's.
template <bool F32>
__device__ __forceinline__ void put_weight(float* weights, const float* from) {
  const int d = threadIdx.x;
  weights[F32 ? d : (d & ~63) + (d & 4) * 8 + ((d & 63) >> 3) * 4 + (d & 3)] = __ldg(from + d);
}
template <bool F32>
__device__ __forceinline__ void weigh(float (&x)[32], float inv, const float* weights, int l) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>(weights + 8 * i + 4 * l);
    x[i] = x[i] * inv * w.x;
    x[i + 1] = x[i + 1] * inv * w.y;
    x[i + 2] = x[i + 2] * inv * w.z;
    x[i + 3] = x[i + 3] * inv * w.w;
  }
}

// ------------------------------------------------------------------ rows to rows

struct RotateParams {
  Turn turn;
  Rows q, k;
  uint8_t* q_out;
  uint8_t* k_out;
  const int* positions;
  int n, rows, q_heads, k_heads, block, group;  // rows of a CTA, heads of a CTA (queries', then keys')
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

// item / n = umulhi(item, mul) for item < 2^16, n <= 64; 0 stands for n == 1.
struct Split {
  unsigned mul;
  int n;
  __device__ __forceinline__ explicit Split(int n) : mul(0xFFFFFFFFu / n + 1), n(n) {}
  __device__ __forceinline__ int operator()(int item) const { return n == 1 ? item : static_cast<int>(__umulhi(item, mul)); }
};

// A CTA takes a block of token rows of (entries x rows) and a group of heads: their
// items, 32 at a time, the next ones' loads in front of these ones' arithmetic.
// Bound by HBM.  16 x 2048 rows of 16 / 2 heads, norms, 64 dims turning: 98 us, 604 MB at 6.2
// TB/s (91% of a measured copy), DRAM traffic that of the rows, 106 instructions of a warp per
// row, half of the issue slots.  2047 rows of 12 / 4 heads in float32, all dims, 10.6 us; a
// single token of 32 entries 2.3 us, a launch's latency.  Halves of dims that are no
// multiple of 128 nor 64 (kShift: pairs in other lanes, two CTAs to an SM instead of three), the first's
// sizes: 109 us at 16 or 32 dims, 112 at 96, 129 at 192, 142 at 240; in float32, where a lane's
// pieces are 4 elements, 182 at 16 or 32, 186 at 96 and 196 at 192 (64: 189; the rows take 178).
template <int LAYOUT, int K, bool F32>
__global__ void __launch_bounds__(256, LAYOUT == kShift ? 2 : 3) rotate_kernel(const __grid_constant__ RotateParams p) {
  extern __shared__ __align__(16) float table[];
  __shared__ __align__(16) float weights[2][kHeadDim];
  wait_for_last_kernel();
  const int octet = threadIdx.x >> 3, l = threadIdx.x & 7;
  const int r0 = blockIdx.x * p.block, rows = min(p.block, p.rows - r0);
  const int head0 = blockIdx.y * p.group, items = min(p.group, p.q_heads + p.k_heads - head0) * rows;
  const Split by_rows(rows);

  Raw<F32> raw;
  auto load = [&](int item) {
    const int h = by_rows(item), head = head0 + h, row = r0 + item - h * rows, e = divided(row, p.n_mul, p.n_shift);
    const bool is_k = head >= p.q_heads;
    const Rows& in = is_k ? p.k : p.q;
    if (item < items) raw.load(in.at + e * in.entry + (is_k ? head - p.q_heads : head) * in.head + (row - e * p.n) * in.row, l);
  };
#pragma unroll
  for (int c = 0; c < Raw<F32>::C; ++c) raw.x[c] = make_uint4(0, 0, 0, 0);
  load(octet);
  if (p.turn.q_weight) put_weight<F32>(weights[0], p.turn.q_weight);
  if (p.turn.k_weight) put_weight<F32>(weights[1], p.turn.k_weight);
  if constexpr (LAYOUT != kNone)
    fill_table<kTableOrder<LAYOUT, F32>>(p.turn, table, rows, [&](int r) {
      const int e = divided(r0 + r, p.n_mul, p.n_shift);
      return static_cast<long long>(p.positions ? __ldg(p.positions + r0 + r) : p.start[e]) + (p.positions ? 0 : r0 + r - e * p.n);
    });
  __syncthreads();
  for (int item0 = 0; item0 < items; item0 += 32) {  // the same turns for every lane: rows are exchanged among them
    const int item = item0 + octet, h = by_rows(item), head = head0 + h, r = item - h * rows;
    const bool is_k = head >= p.q_heads;
    float x[32];
    raw.get(x);
    load(item + 32);
    if (p.turn.q_weight || p.turn.k_weight) {
      const float inv = inverse_norm(x, static_cast<float>(p.turn.eps));
      if (is_k ? p.turn.k_weight : p.turn.q_weight) weigh<F32>(x, inv, weights[is_k], l);
    }
    NoLook look;
    turn_row<LAYOUT, K, F32, F32>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, l, look);
    if (item >= items) continue;
    const int e = divided(r0 + r, p.n_mul, p.n_shift), all = is_k ? p.k_heads : p.q_heads;
    const long long to = (static_cast<long long>(e) * all + (is_k ? head - p.q_heads : head)) * p.n + (r0 + r - e * p.n);
    Raw<F32>::store((is_k ? p.k_out : p.q_out) + to * Raw<F32>::kRowBytes, l, x);
  }
}

// ------------------------------------------------------------------ rows into pages

// A lane's codes, and the pairs of elements (bit e: e and e + 1) whose codes fp32 leaves open:
// the ends of what it may be off by have other codes, their signs apart (of zeros).  With u = 2^-24, y the result and m the sum of the
// magnitudes that it is turned from: the norm's sum 9 u at most (chains of 4, 6 levels of a tree), its
// factor then 6, of y; the product's rounding and its correction's 2, of y; the weight's products 2 and
// the cosines' 1.7, of m, or 2.7 where the amplitude is rounded to fp32 too.  Elements that do not
// turn: 8 u, or nothing without a norm.
// About one element in 60,000.  32 x 4096 rows of 16 / 2 heads and their read-back take 488 us, 481 where
// each such code is left to fp32; 16 x 2048 rows of 8 / 8 heads 171 and 158.  At worst, 32 x 4096 rows of two
// heads without queries (149 us): 1.5 ms where every key is one number on a border, 3 ms with a NaN in
// every row.
struct Bound {
  float of_y, of_m, of_rest;  // of elements times unit
  __device__ __forceinline__ Bound(float unit, const Turn& t)
      : of_y((t.k_weight ? 8.1f : 2.1f) * 0x1p-24f * unit),
        of_m((t.k_weight ? 2.0f + t.unit_off : t.unit_off) * 0x1p-24f * unit * fabsf(static_cast<float>(t.amplitude))),
        of_rest(t.k_weight ? of_y : 0.0f) {}
};
struct NearBorder : Bound {
  float unit;
  uint32_t elements = 0, words[8];
  __device__ __forceinline__ NearBorder(float unit, const Turn& t) : Bound(unit, t), unit(unit) {}
  __device__ __forceinline__ void ends(int e, float y0, float off0, float y1, float off1) {
    const uint32_t code = e4m3x2(fmaf(y0, unit, off0), fmaf(y1, unit, off1)), other = e4m3x2(fmaf(y0, unit, -off0), fmaf(y1, unit, -off1));
    if ((code ^ other) & 0x7F7Fu) elements |= 1u << e;
    words[e / 4] = e % 4 ? words[e / 4] | code << 16 : code;
  }
  __device__ __forceinline__ void turned(int e, float y0, float m0, float y1, float m1) {
    ends(e, y0, fmaf(fabsf(y0), of_y, m0 * of_m), y1, fmaf(fabsf(y1), of_y, m1 * of_m));
  }
  __device__ __forceinline__ void rest(int e, float y0, float y1) { ends(e, y0, fabsf(y0) * of_rest, y1, fabsf(y1) * of_rest); }
};
// Whether a lane's elements are above a limit, and those (bit e: e and e + 1) that fp32 leaves open.
struct AboveLimit : Bound {
  float limit;
  uint32_t elements = 0;
  bool above = false;
  __device__ __forceinline__ AboveLimit(float limit, const Turn& t) : Bound(1.0f, t), limit(limit) {}
  __device__ __forceinline__ void look(int e, float y, float off) {
    const float d = fabsf(y) - limit;  // (exact where it is small)
    if (d > off) above = true;
    else if (d > -off) elements |= 1u << e;
  }
  __device__ __forceinline__ void turned(int e, float y0, float m0, float y1, float m1) {
    look(e, y0, fmaf(fabsf(y0), of_y, m0 * of_m));
    look(e, y1, fmaf(fabsf(y1), of_y, m1 * of_m));
  }
  __device__ __forceinline__ void rest(int e, float y0, float y1) {
    look(e, y0, fabsf(y0) * of_rest);
    look(e, y1, fabsf(y1) * of_rest);
  }
};
// Cosine and sine of a / 2^64 turns in fp64: the nearest quarter taken off, Taylor's series.
__device__ __forceinline__ double2 exact_unit_at(unsigned long long a) {
  const unsigned quarter = static_cast<unsigned>((a + (1ull << 61)) >> 62);
  const double t = static_cast<double>(static_cast<long long>(a - (static_cast<unsigned long long>(quarter) << 62))) * (6.283185307179586476925 * 0x1p-64);
  const double t2 = t * t;
  const double t4 = t2 * t2, t8 = t4 * t4;  // (in a tree: a step takes 60 cycles)
  double s = fma(fma(t2, -1.0 / 1307674368000, 1.0 / 6227020800), t8,
                 fma(fma(t2, -1.0 / 39916800, 1.0 / 362880), t4, fma(t2, -1.0 / 5040, 1.0 / 120)));
  s = fma(fma(s, t2, -1.0 / 6) * t2, t, t);
  double c = fma(fma(t4, 1.0 / 20922789888000, fma(t2, -1.0 / 87178291200, 1.0 / 479001600)), t8,
                 fma(fma(t2, -1.0 / 3628800, 1.0 / 40320), t4, fma(t2, -1.0 / 720, 1.0 / 24)));
  c = fma(c, t4, fma(t2, -0.5, 1.0));
  if (quarter & 1) {
    const double x = c;
    c = -s;
    s = x;
  }
  return quarter & 2 ? make_double2(-c, -s) : make_double2(c, s);
}
__device__ __forceinline__ float bf16_at(const uint8_t* row, int d) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(row) + d)) << 16);
}
// Such elements again, in fp64, and those of lanes that hold what is not finite (NaN: 0), a warp's rows
// octet and octet + 32 of a page (`first`, `second`: the lane's pairs of each; rows: where the
// page's row 0 would be).  fp64 runs at a sixtieth of fp32's rate, so squares, which fp32 holds,
// are summed there with what is rounded off, a row by the whole warp; where they leave its range, in
// fp64.  Loops are not unrolled: what a warp waits for here is mostly instructions.
// Without codes to store: whether some element of the lane's is above 448 / unit.
template <bool PAIRS>
__device__ __noinline__ bool exact_codes(const Turn& t, const uint8_t* rows, long long stride, const int* positions, int position, float unit,
                                         uint32_t first, uint32_t second, uint8_t* codes) {
  const int lane = threadIdx.x & 31, l = lane & 7;
  bool above = false;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    uint32_t elements = i ? second : first, wanted = __ballot_sync(0xFFFFFFFFu, elements != 0);
    const bool here = (wanted >> (lane & 24) & 0xFF) != 0;  // some lane of the row's eight
    const int r = (threadIdx.x >> 3) + 32 * i;
    const uint8_t* row = rows + r * stride;
    double norm = 1.0;
    if (t.k_weight)
#pragma unroll 1
      while (wanted) {
        const int of = (__ffs(wanted) - 1) & 24;
        wanted &= ~(0xFFu << of);
        const uint4 raw = __ldg(reinterpret_cast<const uint4*>(rows + ((threadIdx.x >> 5) * 4 + of / 8 + 32 * i) * stride) + lane);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float s = 0.0f, off = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16), q = x * x, sum = s + q, back = sum - s;
          off += (s - (sum - back)) + (q - back);
          s = sum;
        }
        double sum = static_cast<double>(s) + off;
        if (__any_sync(0xFFFFFFFFu, !(s < 1e30f && (s > 1e-20f || s == 0.0f)))) {
          sum = 0.0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const double x = __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
            sum = fma(x, x, sum);
          }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        sum = fma(sum, 1.0 / kHeadDim, t.eps);
        double inv = __frsqrt_rn(static_cast<float>(sum));  // off by 2^-23, and after a step of Newton's 2^-45
        inv = sum < 1e30 && sum > 1e-30 ? inv * fma(-0.5 * sum * inv, inv, 1.5) : 1.0 / sqrt(sum);
        if ((lane & 24) == of) norm = inv;
      }
    const int at = !positions ? position + r : here ? __ldg(positions + r) : 0;
    auto element = [&](int d) {
      const double x = bf16_at(row, d);
      return t.k_weight ? x * norm * static_cast<double>(__ldg(t.k_weight + d)) : x;
    };
    __syncwarp();  // the codes of other lanes' elements are stored
#pragma unroll 1
    for (int half = 0; __any_sync(0xFFFFFFFFu, elements != 0); half ^= 1) {
      // the first pairs of the even lanes, of the odd ones: an element by either of two lanes
      const uint32_t pairs = __shfl_sync(0xFFFFFFFFu, elements, (lane & ~1) | half);
      if (pairs) {
        const int e = __ffs(pairs) - 1, d = (e >> 3) * 64 + ((l & ~1) | half) * 8 + (e & 7) + (lane & 1);
        double y = element(d);
        if (d < 2 * t.pairs) {
          const bool upper = PAIRS ? lane & 1 : d >= t.pairs;
          const int j = PAIRS ? d >> 1 : upper ? d - t.pairs : d;
          const double other = element(PAIRS ? d ^ 1 : upper ? d - t.pairs : d + t.pairs);
          const double2 u = exact_unit_at(__ldg(t.turns + j) * static_cast<unsigned long long>(static_cast<long long>(at)));
          y = t.amplitude * fma(y, u.x, upper ? other * u.y : -other * u.y);
        }
        y = y == y ? y * unit : 0.0;
        above |= fabs(y) > 448.0;
        float z = __double2float_rz(y);  // to odd, so that the code's rounding is the only one
        if (static_cast<double>(z) != y) z = __uint_as_float(__float_as_uint(z) | 1u);
        if (codes) codes[r * kHeadDim + d] = static_cast<uint8_t>(e4m3x2(z, 0.0f));
      }
      if ((lane & 1) == half) elements &= elements - 1;
    }
  }
  return above;
}

struct RotaryAppendParams {
  AppendParams a;  // (keys and values: unused)
  Turn turn;
  Rows q, k, v;
  uint8_t* q_out;
  const int* positions;
  int keys_first;  // in the order of CTAs: those of all segments' keys before others
  int q_heads, group, groups, part_rows;  // queries: of `groups` groups of heads, so many rows of a page
};

// Whether one of the lane's new elements of a page's rows [begin, end) is above 448 * 2^e.  The page's
// exponent hangs on it where the largest element, in fp32, is as near to that as it may be off
// (four pages in a million; where elements that are exact are the largest, one in 200, which need no fp64).
template <int LAYOUT, int K>
__device__ __noinline__ bool key_above(const Turn& t, const uint8_t* rows, long long stride, const int* positions, int position, int begin,
                                       int end, const float* weights, const float* table, int e) {
  const int octet = threadIdx.x >> 3, l = threadIdx.x & 7, octet0 = octet & ~3;
  uint32_t open[2] = {};
  bool above = false;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    if (octet0 + 32 * i + 4 <= begin || octet0 + 32 * i >= end) continue;  // no new row in this warp
    const int r = octet + 32 * i;
    const bool is_new = r >= begin && r < end;
    Raw<false> raw;
#pragma unroll
    for (int c = 0; c < 4; ++c) raw.x[c] = make_uint4(0, 0, 0, 0);
    if (is_new) raw.load(rows + r * stride, l);
    float x[32];
    raw.get(x);
    if (t.k_weight) weigh<false>(x, inverse_norm(x, static_cast<float>(t.eps)), weights, l);
    AboveLimit look(448.0f * power2(e), t);
    turn_row<LAYOUT, K, false, true>(x, table + 2 * (min(max(r, begin), end - 1) - begin) * t.pairs, t.pairs, l, look);
    if (!is_new) continue;
    (i ? open[1] : open[0]) = look.elements;
    above |= look.above;
  }
  if (__any_sync(0xFFFFFFFFu, (open[0] | open[1]) != 0))
    above |= exact_codes<LAYOUT == kPairs>(t, rows, stride, positions, position, power2(-e), open[0], open[1], nullptr);
  return above;
}

// CTA (page of a segment, y, segment; y last where keys come first): the keys of kv head y, the values of
// kv head y - heads, or the queries of a group of heads at the page's new rows.  A page's rows
// stay in registers as they came, two to eight lanes; keys are turned twice, for the
// page's largest element and for the codes, which takes fewer registers than keeping
// them in fp32.  Codes are those nearest to the exact keys (see NearBorder).
// Bound by HBM: 32 x 4096 rows of 16 / 2 heads, 64 dims turning, take 421 us, 2.52 GB at 6.0 TB/s
// (88% of a measured copy).  With all dims turning and few rows by a
// page's 8192 cosines in front of its keys: 7 x 513 rows of 8 / 4 heads 29 us, read back with them.
// Three CTAs to an SM leave 80 registers, of which two rows as they came take 32: instances that
// turn keep 40 to 140 bytes in local memory (none at kNone; the 128 of kShift<1> 52).  kShift: the large append
// and its read-back take 536 us at 32 dims, 584 at 96, 736 at 192 (64: 488).
template <int LAYOUT, int K>
__global__ void __launch_bounds__(256, LAYOUT == kShift ? 2 : 3) paged_append_rotary_kernel(const __grid_constant__ RotaryAppendParams p) {
  extern __shared__ __align__(16) float table[];  // of the page's new rows
  __shared__ __align__(16) float weights[kHeadDim];
  __shared__ uint32_t tops[8];
  wait_for_last_kernel();
  const Segment sg = p.a.seg[p.keys_first ? blockIdx.y : blockIdx.z];
  const int k = blockIdx.x, heads = p.a.heads, y = p.keys_first ? blockIdx.z : blockIdx.y;
  const int off = sg.pos % kPage;                 // rows of the segment's first page before it
  const int begin = k == 0 ? off : 0;             // this page's new rows: [begin, end)
  const int end = min(kPage, off + sg.rows - k * kPage);
  if (end <= begin) return;
  const int octet = threadIdx.x >> 3, l = threadIdx.x & 7;
  const int row0 = sg.row0 + k * kPage - off;     // the call's row of this page's row 0
  // the weights, and the table of rows [first, last) of the page
  auto fill = [&](const float* weight, int first, int last) {
    if (weight) put_weight<false>(weights, weight);
    if constexpr (LAYOUT != kNone)
      fill_table<kTableOrder<LAYOUT, false>>(p.turn, table, last - first, [&](int r) {
        return static_cast<long long>(p.positions ? __ldg(p.positions + static_cast<long long>(sg.entry) * p.a.n + row0 + first + r)
                                                  : sg.pos - off + k * kPage + first + r);
      });
    __syncthreads();
  };
  Raw<false> raw[2];
  auto clear = [&]() {
#pragma unroll
    for (int c = 0; c < 4; ++c) raw[0].x[c] = raw[1].x[c] = make_uint4(0, 0, 0, 0);
  };
  clear();

  if (y >= 2 * heads) {
    // ---------------------------------------------------------------- queries
    const int part = (y - 2 * heads) / p.groups, head0 = (y - 2 * heads - part * p.groups) * p.group;
    const int first = max(begin, part * p.part_rows), rows = min(end, (part + 1) * p.part_rows) - first;
    if (rows <= 0) return;
    const int items = min(p.group, p.q_heads - head0) * rows;
    const Split head_of(rows);
    auto load = [&](int item) {
      const int h = head_of(item), r = item - h * rows;
      if (item < items) raw[0].load(p.q.at + sg.entry * p.q.entry + (head0 + h) * p.q.head + (row0 + first + r) * p.q.row, l);
    };
    load(octet);
    fill(p.turn.q_weight, first, first + rows);
    for (int item0 = 0; item0 < items; item0 += 32) {  // the same turns for every lane: rows are exchanged among them
      const int item = item0 + octet, h = head_of(item), r = item - h * rows;
      float x[32];
      raw[0].get(x);
      load(item + 32);
      if (p.turn.q_weight) weigh<false>(x, inverse_norm(x, static_cast<float>(p.turn.eps)), weights, l);
      NoLook look;
      turn_row<LAYOUT, K, false, false>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, l, look);
      if (item >= items) continue;
      const long long to = (static_cast<long long>(sg.entry) * p.q_heads + head0 + h) * p.a.n + row0 + first + r;
      Raw<false>::store(p.q_out + to * Raw<false>::kRowBytes, l, x);
    }
    return;
  }
  // ---------------------------------------------------------------- keys, values
  const bool is_v = y >= heads;
  const int h = is_v ? y - heads : y;
  const int page = sg.page + k, from = k == 0 ? sg.from : page;
  const long long at = static_cast<long long>(page) * heads + h, at_from = static_cast<long long>(from) * heads + h;
  uint8_t* codes = (is_v ? p.a.v_codes : p.a.k_codes) + at * kPageBytes;
  float* scales = is_v ? p.a.v_scales : p.a.k_scales;
  const float* weight = p.turn.k_weight;
  auto load_rows = [&]() {
    const Rows& in = is_v ? p.v : p.k;
    const uint8_t* rows = in.at + sg.entry * in.entry + h * in.head;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = octet + 32 * i;
      if (r >= begin && r < end) raw[i].load(rows + (row0 + r) * in.row, l);
    }
  };
  load_rows();
  const int octet0 = octet & ~3;
  auto idle = [&](int i) { return octet0 + 32 * i + 4 <= begin || octet0 + 32 * i >= end; };  // no new row in this warp
  float inv[2] = {};
  auto turned = [&](int i, float (&x)[32], auto& look) {  // (rows that are not new are all zeros)
    raw[i].get(x);
    if (weight) weigh<false>(x, inv[i], weights, l);
    const int r = min(max(octet + 32 * i, begin), end - 1) - begin;
    turn_row<LAYOUT, K, false, true>(x, table + 2 * r * p.turn.pairs, p.turn.pairs, l, look);
  };
  uint32_t top = 0;
  bool odd;  // not a number, held as 0, or infinite, held as the largest value
  if (is_v) {
    auto largest = [&]() {
      top = 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) top = max(top, magnitude(raw[c >> 2].x[c & 3]));
    };
    largest();
    odd = top >= 0x7F80u;
    if (odd) {  // rare
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint4& x = raw[c >> 2].x[c & 3];
        x = make_uint4(drop_non_finite(x.x), drop_non_finite(x.y), drop_non_finite(x.z), drop_non_finite(x.w));
      }
      largest();
    }
    top <<= 16;
  } else {
    fill(weight, begin, end);
    uint32_t bits = 0;
    float most = 0.0f;  // (a maximum leaves out what is not a number)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (idle(i)) continue;
      float x[32];
      if (weight) {
        raw[i].get(x);
        inv[i] = inverse_norm(x, static_cast<float>(p.turn.eps));
      }
      NoLook look;
      turned(i, x, look);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        most = fmaxf(most, fabsf(x[j]));
        bits = max(bits, __float_as_uint(x[j]) & 0x7FFFFFFFu);
      }
    }
    odd = bits >= 0x7F800000u;
    top = min(__float_as_uint(most), 0x7F7FFFFFu);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, tops[i]);
  const uint8_t* key_rows = p.k.at + sg.entry * p.k.entry + h * p.k.head + row0 * p.k.row;
  const int* key_positions = p.positions ? p.positions + static_cast<long long>(sg.entry) * p.a.n + row0 : nullptr;
  const int key_position = sg.pos - off + k * kPage;
  int e = least_exponent(top);
  if (!is_v) {
    // The largest key is off by 2^-24 * (8.1 + 2 * 4.7) of it at most: of the pair that it is turned from, the magnitudes' sum
    // times the amplitude is at most twice the larger of the pair's results.
    const float most = __uint_as_float(top);
    const int least = least_exponent(__float_as_uint(most * (1.0f - 0x1.4p-20f)));
    if (least != least_exponent(__float_as_uint(most * (1.0f + 0x1.4p-20f)))) {
      e = least + __syncthreads_or(key_above<LAYOUT, K>(p.turn, key_rows, p.k.row, key_positions, key_position, begin, end, weights, table, least));
      clear();  // (the rows again, rather than in registers over the call)
      load_rows();
    }
  }
  const bool beyond = e > kEMax;
  e = min(e, kEMax);
  const int old = begin > 0 ? exponent_of(scales[at_from]) : e;
  e = max(e, old);
  const float unit = power2(-e);
  uint32_t again[2] = {};  // elements whose codes fp32 leaves open
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (idle(i)) continue;
    const int r = octet + 32 * i;
    float x[32];
    uint32_t words[8];
    if (is_v) {
      raw[i].get(x);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* z = x + 4 * j;
        words[j] = e4m3x2(z[0] * unit, z[1] * unit) | e4m3x2(z[2] * unit, z[3] * unit) << 16;
      }
    } else {
      NearBorder near(unit, p.turn);
      turned(i, x, near);
      again[i] = r < begin || r >= end ? 0 : odd ? 0x55555555u : near.elements;
#pragma unroll
      for (int j = 0; j < 8; ++j) words[j] = near.words[j];
    }
    if (r < begin || r >= end) continue;
#pragma unroll
    for (int c = 0; c < 4; ++c) *reinterpret_cast<uint2*>(codes + r * kHeadDim + 64 * c + 8 * l) = make_uint2(words[2 * c], words[2 * c + 1]);
  }
  if (__any_sync(0xFFFFFFFFu, (again[0] | again[1]) != 0))
    exact_codes<LAYOUT == kPairs>(p.turn, key_rows, p.k.row, key_positions, key_position, unit, again[0], again[1], codes);
  upkeep((is_v ? p.a.v_codes : p.a.k_codes) + at_from * kPageBytes, codes, begin, end, from != page, old, e);
  if (odd || beyond) atomicOr(p.a.status, IQ_STATUS_RANGE);
  __syncthreads();  // the old scale has been read by every thread
  if (threadIdx.x == 0) {
    scales[at] = power2(e);
    if (y == 0) p.a.table[static_cast<long long>(sg.slot) * p.a.max_pages + sg.pos / kPage + k] = page;
  }
}

// The queries of rows behind an entry's count: zeros, a warp to four rows.  (Filling all of
// the output before the append wrote 15 MB for 7 x 8 x 513 rows, and cost the host 15 us.)
struct PaddingParams {
  uint8_t* out;
  int n, heads, count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) padding_kernel(const __grid_constant__ PaddingParams p) {
  wait_for_last_kernel();
  const int e = blockIdx.z, lane = threadIdx.x & 31, r0 = p.count[e] + (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
  uint8_t* at = p.out + (static_cast<long long>(e) * p.heads + blockIdx.y) * p.n * (kHeadDim * 2) + lane * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (r0 + i < p.n) *reinterpret_cast<uint4*>(at + static_cast<long long>(r0 + i) * (kHeadDim * 2)) = make_uint4(0, 0, 0, 0);
}
int zero_padding(uint8_t* out, int entries, int heads, int n, const int32_t* counts, cudaStream_t stream) {
  PaddingParams p;
  p.out = out;
  p.n = n;
  p.heads = heads;
  int most = 0;  // rows behind a count
  for (int i = 0; i < entries; ++i) {
    p.count[i] = counts[i];
    most = std::max(most, n - counts[i]);
  }
  if (most == 0) return IQ_OK;
  void* args[] = {&p};
  IQ_CUDA(launch_after(reinterpret_cast<const void*>(&padding_kernel), dim3((most + 31) / 32, heads, entries), 256, 0, stream, args));
  return IQ_OK;
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

struct Kind {
  Layout layout;
  int k;
};
Kind kind_of(const iq_rotary* r, bool f32) {
  const int pairs = r->rotary_dim / 2, piece = f32 ? 32 : 64;  // 8V elements
  if (pairs == 0) return {kNone, 0};
  if (r->interleaved) return {kPairs, 0};
  if (pairs % piece == 0) return {kHere, pairs / piece};
  return {!f32 && pairs == 32 ? kSwap : kShift, pairs / piece};
}
Turn turn_of(const iq_rotary* r) {
  const bool rounded = static_cast<double>(static_cast<float>(r->amplitude)) != r->amplitude;
  return {reinterpret_cast<const unsigned long long*>(r->turns), r->q_weight, r->k_weight, r->amplitude, r->eps, rounded ? 2.7f : 1.7f, r->rotary_dim / 2};
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
    if (!std::isfinite(static_cast<float>(r->amplitude))) return fail(IQ_ERR_INVALID_ARG, "amplitude is not finite");
  }
  if (r->q_weight || r->k_weight) {
    if (misaligned(r->q_weight) || misaligned(r->k_weight)) return fail(IQ_ERR_INVALID_ARG, "weights not 16-byte aligned");
    if (!(r->eps >= 1e-30 && std::isfinite(static_cast<float>(r->eps)))) return fail(IQ_ERR_INVALID_ARG, "eps must be 1e-30 or more, and finite");
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
    if (in_bytes[i] > (1LL << 56) / (counts[i] - 1)) return fail(IQ_ERR_INVALID_ARG, std::string(name) + ": rows past any address");
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

template <int LAYOUT, int K = 0>
const void* rotate_of(bool f32) {
  return f32 ? reinterpret_cast<const void*>(&rotate_kernel<LAYOUT, K, true>) : reinterpret_cast<const void*>(&rotate_kernel<LAYOUT, K, false>);
}
const void* rotate_kernel_of(Kind kind, bool f32) {
  switch (kind.layout) {
    case kPairs: return rotate_of<kPairs>(f32);
    case kSwap: return reinterpret_cast<const void*>(&rotate_kernel<kSwap, 0, false>);
    case kHere:
      if (kind.k == 3) return reinterpret_cast<const void*>(&rotate_kernel<kHere, 3, true>);
      if (kind.k == 4) return reinterpret_cast<const void*>(&rotate_kernel<kHere, 4, true>);
      return kind.k == 1 ? rotate_of<kHere, 1>(f32) : rotate_of<kHere, 2>(f32);
    case kShift:
      if (kind.k == 2) return reinterpret_cast<const void*>(&rotate_kernel<kShift, 2, true>);
      if (kind.k == 3) return reinterpret_cast<const void*>(&rotate_kernel<kShift, 3, true>);
      return kind.k == 0 ? rotate_of<kShift, 0>(f32) : rotate_of<kShift, 1>(f32);
    default: return rotate_of<kNone>(f32);
  }
}
const void* append_kernel_of(Kind kind) {
  switch (kind.layout) {
    case kPairs: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kPairs, 0>);
    case kSwap: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kSwap, 0>);
    case kHere: return kind.k == 1 ? reinterpret_cast<const void*>(&paged_append_rotary_kernel<kHere, 1>) : reinterpret_cast<const void*>(&paged_append_rotary_kernel<kHere, 2>);
    case kShift: return kind.k == 0 ? reinterpret_cast<const void*>(&paged_append_rotary_kernel<kShift, 0>) : reinterpret_cast<const void*>(&paged_append_rotary_kernel<kShift, 1>);
    default: return reinterpret_cast<const void*>(&paged_append_rotary_kernel<kNone, 0>);
  }
}

struct RotaryAppend {
  Turn turn;
  Kind kind;
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
  int rows = 0;  // the most new rows of a page
  for (int i = 0; i < segs; ++i) rows = std::max(rows, std::min(kPage, a.seg[i].rows));
  p.group = rows == 1 ? 8 : 16;
  p.groups = (m.q_heads + p.group - 1) / p.group;
  p.part_rows = kPage;
  while (p.part_rows > 8 && static_cast<long long>(widest) * segs * p.groups * (kPage / p.part_rows) < 4ll * num_sms()) p.part_rows /= 2;
  if (rows == 1) p.part_rows = kPage;
  const int smem = rows * 2 * m.turn.pairs * static_cast<int>(sizeof(float));
  const void* kernel = append_kernel_of(m.kind);
  static std::atomic<uint64_t> seen[kShift + 1][3] = {};  // (48 KB need no leave, the kernel's own shared memory included)
  const cudaError_t e = smem > 32 * 1024 ? allow_smem(kernel, 64 * 1024, seen[m.kind.layout][m.kind.k]) : cudaSuccess;
  const int parts = 2 * a.heads + p.groups * (kPage / p.part_rows);
  // Keys' CTAs take longest.  In a few waves of CTAs they come first, so that none of them is the
  // last (8 x 512 rows of 8 / 4 heads: 27 us, by segments 33); in more, CTAs that follow one another
  // read the same segment's rows, which lie side by side (16 x 2048: 101 us, keys first 109).
  p.keys_first = static_cast<long long>(widest) * segs * parts <= 4 * 3ll * num_sms();
  const dim3 grid = p.keys_first ? dim3(widest, segs, parts) : dim3(widest, parts, segs);
  void* args[] = {&p};
  return e == cudaSuccess ? launch_after(kernel, grid, 256, smem, stream, args) : e;
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
                    int n, const int32_t* start, int n_start, const int32_t* positions, void* q_out, void* k_out, iq_stream_t stream) {
  int st = check_rotary(rotary);
  if (st != IQ_OK) return st;
  if (dtype != IQ_DTYPE_BF16 && dtype != IQ_DTYPE_F32) return fail(IQ_ERR_INVALID_ARG, "unknown dtype");
  if (q_heads < 0 || k_heads < 0 || entries < 0 || n < 0) return fail(IQ_ERR_INVALID_ARG, "negative size");
  if (entries > IQ_MAX_BATCH) return fail(IQ_ERR_INVALID_ARG, "entries above IQ_MAX_BATCH");
  if (n_start != 0 && n_start != 1 && n_start != entries) return fail(IQ_ERR_INVALID_ARG, "n_start must be 0, 1 or entries");
  if (n_start > 0 && !start) return fail(IQ_ERR_INVALID_ARG, "null start");
  if (n_start > 0 && positions) return fail(IQ_ERR_INVALID_ARG, "give either start or positions");
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
  for (int i = 0; i < entries; ++i) p.start[i] = n_start > 0 ? start[n_start == 1 ? 0 : i] : 0;
  // A CTA holds all heads of its rows (24 at most), so that angles are worked out once, and as many rows as make
  // whole waves of CTAs, three to an SM; where there are fewer rows than that, fewer heads, down to 8.
  const int heads = q_heads + k_heads, room = 3 * num_sms();
  int groups = (heads + 23) / 24;
  while (static_cast<long long>(p.rows) * groups * 2 <= room && (heads + 2 * groups - 1) / (2 * groups) >= 8) groups *= 2;
  p.group = (heads + groups - 1) / groups;
  groups = (heads + p.group - 1) / p.group;
  const long long abreast = std::max(room / groups, 1);
  const long long waves = (p.rows + 32 * abreast - 1) / (32 * abreast);
  p.block = static_cast<int>((p.rows + waves * abreast - 1) / (waves * abreast));
  void* args[] = {&p};
  IQ_CUDA(launch_after(rotate_kernel_of(kind_of(rotary, size == 4), size == 4),
                       dim3((p.rows + p.block - 1) / p.block, groups), 256, static_cast<int>(sizeof(float)) * 2 * p.turn.pairs * p.block,
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
  if (q_heads < 0) return fail(IQ_ERR_INVALID_ARG, "bad q_heads");
  if (q_heads > (1 << 14)) return fail(IQ_ERR_UNSUPPORTED, "q_heads above 2^14");
  if (misaligned(positions, 4)) return fail(IQ_ERR_INVALID_ARG, "positions not 4-byte aligned");
  if (n_slots == 0 || n == 0) return IQ_OK;
  RotaryAppend m;
  m.turn = turn_of(rotary);
  m.kind = kind_of(rotary, false);
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
  if (counts && out.bytes && (st = zero_padding(m.q_out, n_slots, q_heads, n, counts, static_cast<cudaStream_t>(stream))) != IQ_OK) return st;
  st = do_append(c, nullptr, nullptr, n, slots, counts, n_slots, stream, launch_append_rotary, &m);
  if (st == IQ_OK) launched_outputs(stream, out);
  return st;
}

}  // extern "C"
