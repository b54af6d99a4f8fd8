// libiqkv: attention over the paged 8-bit cache.
//
// Two kernels.  Calls with at most 32 query rows per kv head (decode, verify)
// run paged_split_kernel, below: the keys are the matrix products' M dimension,
// the codes go from HBM through shared memory into tcgen05.mma untouched, and
// the keys of all (slot, kv head) pairs are split evenly over the GPU.  More
// rows run paged_prefill_kernel (iq_paged_prefill.cu).
//
// Mathematics of the split kernel.  With a query as two e4m3 parts, x = 2^eq
// (hi + lo / 16), and key codes K of a page under 2^ek, the scores in log2 units
// are  s = (K.hi + K.lo / 16) * 2^ek * (2^eq * scale * log2 e): exact products,
// summed in fp32 by the tensor cores, hi and lo as columns of their own.  With
// value codes V of a page under 2^ev, a key weighs 2^(s + ev - ref) = p * 2^ev up
// to a common factor, so o = sum p 2^ev V / sum p : the value scales ride in the
// exponents.  The second product is block-scaled: with e the exponent s + ev - ref
// of the largest weight of a row's 32 keys (a warp's), rounded up, they are held as
// w = 2^(s + ev - ref - e + 6) under the scale 2^(e - 6).  w has two e4m3 parts, hi +
// lo / 128, in columns of their own again: off by at most 2^-8 of it, at random, and
// below e4m3's range by half a step of the least codes, 2^-22 of the largest weight
// among its 32 keys.  (One reference for the whole row left 2^-17 of the row's
// largest: next to one key with half of it, 131072 others were off by 8% in norm.)
// The sum of p, in fp32, takes w as the parts hold it: where one key dominates, its
// rounding then cancels (0.00035 off in norm for 32 x 32768 tokens, 0.0006 with w
// itself; no slower).  ref only keeps the sums in fp32's range: it moves, to the row's
// maximum, when the weights pass it by 2^kAhead, so steady-state tiles need no
// exchange between warps but a vote.
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "iq_paged_mma.cuh"

namespace iq {
namespace paged {

// ------------------------------------------------------------------ decode and verify

constexpr float kPlace = 6.0f;  // the place of a block's largest weight
constexpr float kPLo = 128.0f;  // the low parts' scale: half a step at 2^6 is 2, times 128 below 448

template <int NR>
struct SplitShape {
  static constexpr int kGroups = NR >= 32 ? 2 : 1;    // warpgroups on the softmax, NR / kGroups rows each
  static constexpr int kRows = NR / kGroups;
  static constexpr int kCols = 2 * NR;                // high and low parts
  static constexpr int kSlots = 6;                    // tiles of keys or values in flight
  static constexpr int kQ = kSlots * kSlotBytes;      // [2 halves of the dims][kCols rows][128 bytes]
  static constexpr int kP = kQ + 2 * kCols * 128;     // [2][kCols rows][128 keys]
  static constexpr int kScales = kP + 2 * kCols * 128;  // [2] the weights'
  static constexpr int kMisc = kScales + 2 * kScaleBytes;
  static constexpr int kRing = Loader<kSlots, false>::kRing;
  static constexpr int kFloats = 2 * NR + 4 * NR;     // factors, references; reductions
  static constexpr int kBars = 2 * kSlots + kRing + 10;
  static constexpr int kSmem = kMisc + kFloats * 4 + kRing * 16 + kBars * 8 + 8;
  static constexpr int kThreads = kGroups * 128 + 64;
  static constexpr int kTmem = 4 * kCols;             // S twice, O of both halves of the dims
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

// One persistent CTA per SM: warps 0 .. 4 kGroups - 1 hold a key per thread
// (warp w reaches tensor-memory lanes 32 (w % 4) ..), then one warp streams the
// pages and one issues the matrix products.
// Why keys as M: M is 128 whatever it holds, so 8 query rows as M would leave 15
// of 16 lanes idle; as N they fill 16 columns (two parts each), a product takes
// its least time (65 cycles) and a tile's 16 products a third of the time that
// its 64 KB take from HBM.  Six tiles of keys or values in flight (192 KB per SM)
// cover HBM's latency.  Up to 32 rows, where the row work is still shorter than the
// stream (see kMaxSplitRows).
// Bound by HBM.  32 slots x 32768 tokens, 16 / 2 heads, one query: 170 us, 1.07 GB
// at 6.3 TB/s (93% of a measured copy), DRAM traffic within 0.1% of the keys and
// values.  8 x 131072 tokens, four queries: 175 us.  One slot of 4096 tokens: 10.9
// us with the join, a launch's and a pipeline's latency.  The weights' block scales
// cost 1 us of the first.  A thread's own loads of
// its page's scale, one tile ahead, cost 5%: under a full HBM they take longer
// than a tile; the loading warp hands them over instead.
template <int NR>
__global__ void __launch_bounds__(SplitShape<NR>::kThreads, 1) paged_split_kernel(const __grid_constant__ AttendParams p) {
  using C = SplitShape<NR>;
  constexpr int RT = C::kRows;
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled operands need it; no room to align by hand
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // (the kernel has no other shared memory in front)
    wait_for_last_kernel();
    if (threadIdx.x == 0) atomicOr(p.status, kLostMma);
    return;
  }
  float* factor = reinterpret_cast<float*>(smem + C::kMisc);  // [NR] 2^eq * scale * log2 e
  float* ref = factor + NR;                                   // [NR]
  float* red = ref + NR;                                      // [4 warps][NR]
  float4* scales = reinterpret_cast<float4*>(red + 4 * NR);   // [kRing] of a tile's two pages: keys', values'
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + C::kRing);  // [kSlots]
  uint64_t* empty = full + C::kSlots;                         // [kSlots]
  uint64_t* scales_in = empty + C::kSlots;                    // [kRing]
  uint64_t* s_full = scales_in + C::kRing;                    // [2] scores of a tile in tensor memory
  uint64_t* s_free = s_full + 2;                              // [2] and read
  uint64_t* p_ready = s_free + 2;                             // [2] weights of a tile in shared memory
  uint64_t* o_done = p_ready + 2;                             // [2] and multiplied with its values
  uint64_t* q_ready = o_done + 2;
  uint64_t* drained = q_ready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert(NR % 8 == 0 && C::kMisc % 16 == 0, "scales and barriers are aligned");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kLoader = 4 * C::kGroups, kIssuer = kLoader + 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kRing; ++s) mbar_init(&scales_in[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], 4 * C::kGroups);
      mbar_init(&p_ready[s], 4 * C::kGroups);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(q_ready, 4 * C::kGroups);
    mbar_init(drained, 1);
    *abort = 0;
    mbar_fence_init();
  }
  wait_only();
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(C::kTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  release_dependents();
  const uint32_t tmem = *tslot;
  const uint32_t t_o = tmem + 2 * C::kCols;  // O: [half of the dims][kCols]
  const Waits wait{abort, p.status};

  const int first = range_begin(blockIdx.x, gridDim.x, p.total), last = range_begin(blockIdx.x + 1, gridDim.x, p.total);
  const Place start = place_of(p, first);  // every role walks the same segments from here

  if (warp == kLoader) {
    Loader<C::kSlots, false>{p, smem, full, empty, scales, scales_in, wait}.run(start, first, last, policy_evict_first());
  } else if (warp == kIssuer) {
    // ---------------------------------------------------------------- products
    {
      constexpr uint32_t kS = shape(128, C::kCols, false, false);
      // descriptors count in 16 bytes: those of other pieces are sums
      const uint64_t queries = operand(sbase + C::kQ), weights = operand(sbase + C::kP), at_slot = operand(sbase);
      int it = 0, used = 0, segment = 0;
      bool ok = true;
      Place w = start;
      for (int at = first; at < last && ok; ++segment, next_unit(p, w)) {
        const int tiles = tiles_at(p, w).n, n = part_of(p, w, tiles, last - at).n;
        at += tiles + p.cost - w.j;
        if (n == 0) break;
        ok = wait.together(q_ready, segment, kLostMma);
        for (int j = 0; j <= n && ok; ++j) {
          if (j < n) {
            const int b = (it + j) & 1, s = used % C::kSlots;
            if (it + j >= 2) ok = wait.together(&s_free[b], (it + j) / 2 - 1, kLostMma);
            ok = ok && wait.together(&full[s], used / C::kSlots, kLostMma);
            if (!ok) break;
            tc_after();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_e4m3(tmem + b * C::kCols, at_slot + ((s * kSlotBytes + (k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                       queries + (((k >> 2) * C::kCols * 128 + (k & 3) * 32) >> 4), kS, k > 0);
            mma_commit(&s_full[b]);
            mma_commit(&empty[s]);
            ++used;
          }
          if (j > 0) {
            const int b = (it + j - 1) & 1, s = used % C::kSlots;
            ok = wait.together(&p_ready[b], (it + j - 1) / 2, kLostMma) && wait.together(&full[s], used / C::kSlots, kLostMma);
            if (!ok) break;
            tc_after();
            const uint32_t place = tmem + b * C::kCols;  // of the scales, where the scores were; the values' behind them
            copy_scales(place, sbase + C::kScales + b * kScaleBytes);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_scaled(t_o + half * C::kCols, at_slot + ((s * kSlotBytes + half * kHalfBytes + k * 32 * 128) >> 4),
                           weights + ((b * C::kCols * 128 + k * 32) >> 4), shape_scaled(128, C::kCols, true, false, 0, k), place + 4, place,
                           j > 1 || k > 0);
            mma_commit(&o_done[b]);
            mma_commit(&empty[s]);
            ++used;
          }
        }
        it += n;
      }
      if (!ok) {  // given up: what is in flight ends before the tensor memory goes
        mma_commit(drained);
        wait.drain(drained, 0);
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax: a key per thread
    const int group = warp >> 2, key = threadIdx.x & 127, r0 = group * RT;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if (threadIdx.x == 0) p.cuts[blockIdx.x].last = -1;
    float l[RT];
    int it = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t phase) {  // a lost wait changes no path: every barrier below is still reached
      if (ok) ok = wait(bar, phase, kLostRows);
      __syncwarp();
    };
    Place at_unit = start;
    for (int at = first; at < last; next_unit(p, at_unit)) {
      const int e = at_unit.e;
      const Tiles tiles = tiles_at(p, at_unit);
      const Part part = part_of(p, at_unit, tiles.n, last - at);
      const int k0 = part.begin, n = part.n, len = p.len[e], count = p.count[e], rows = count * p.rep;
      const bool whole = n == tiles.n;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (at == first ? 0 : 1);
      if (n > 0 && n < tiles.n && k0 == 0 && threadIdx.x == 0) tell_cut(p, at_unit, at, tiles.n, slot);
      at += tiles.n + p.cost - at_unit.j;
      if (n == 0) break;
      // the query rows, a warp each
      constexpr int kEach = NR / (4 * C::kGroups);
      uint4 raw[kEach];
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = warp + i * 4 * C::kGroups;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (r < rows) raw[i] = __ldcg(reinterpret_cast<const uint4*>(p.q + row_index(p, at_unit, r) * kHeadDim) + lane);
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = warp + i * 4 * C::kGroups;
        uint2 hi, lo;
        const float f = clamp_finite(split_query<16>(raw[i], hi, lo) * (p.scale * kLog2e));
        uint8_t* to = smem + C::kQ + (lane >> 4) * C::kCols * 128;
        *reinterpret_cast<uint2*>(to + swizzled(r, (lane & 15) * 8)) = hi;
        *reinterpret_cast<uint2*>(to + swizzled(NR + r, (lane & 15) * 8)) = lo;
        if (lane == 0) {
          factor[r] = f;
          ref[r] = r < rows ? kUnset : kDead;
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      named_bar(3, 128 * C::kGroups);
#pragma unroll
      for (int r = 0; r < RT; ++r) l[r] = 0.0f;

      for (int j = 0; j < n; ++j, ++it) {
        const int b = it & 1;
        await(&scales_in[it % C::kRing], it / C::kRing);
        const float* sc = reinterpret_cast<const float*>(&scales[it % C::kRing]) + (key >> 6);  // this key's page
        const float ks = sc[0];
        const float ev = static_cast<float>(exponent_of(sc[2]));
        const int t0 = tiles.tile(k0 + j) * kTile;
        await(&s_full[b], it / 2);
        tc_after();
        float s[RT], w[RT];
        tmem_ld<RT>(tmem + lanes + b * C::kCols + r0, s);
        tmem_ld<RT>(tmem + lanes + b * C::kCols + NR + r0, w);
        ld_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[b]);
#pragma unroll
        for (int r = 0; r < RT; ++r) s[r] = fmaf(w[r], 1.0f / 16, s[r]) * clamp_finite(factor[r0 + r] * ks);
        // masks, in tiles that some row does not see whole
        const bool low_ok = p.window == 0 || t0 > tiles.p_hi - p.window || t0 + kTile <= p.sinks;
        if (!(t0 + kTile <= (p.causal ? tiles.p_lo + 1 : len) && low_ok)) {
          const int t = t0 + key;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int x = r0 + r < rows ? tiles.p_lo + query_of(p, r0 + r) : -1;
            const bool see = t < len && (!p.causal || (t <= x && (p.window == 0 || x < p.window || t > x - p.window || t < p.sinks)));
            if (!see) s[r] = kNothing;
          }
        }
        // lane r: the largest score of row r among the warp's keys
        float top = kNothing;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          const float m = warp_max(s[r]);
          if (lane == r) top = m;
        }
        const int own = r0 + lane % RT;
        int far = lane < RT && top + ev - ref[own] > kAhead;
        asm volatile("{\n.reg .pred a, b;\nsetp.ne.s32 a, %0, 0;\nbarrier.cta.red.or.pred b, %1, 128, a;\nselp.s32 %0, 1, 0, b;\n}"
                     : "+r"(far)
                     : "r"(1 + group)
                     : "memory");
        if (far) {
          // some row's scores passed its reference by 2^kAhead, or are its first: move
          // the references of such rows to their maxima, and what was summed with them
          if (lane < RT) red[(warp & 3) * NR + own] = top + ev;
          named_bar(1 + group, 128);
          if (j > 0) await(&o_done[b ^ 1], (it - 1) / 2);
          tc_after();
#pragma unroll
          for (int r = 0; r < RT; r += 8) {
            float change[8];
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              const int x = r0 + r + y;
              const float m = fmaxf(fmaxf(red[x], red[NR + x]), fmaxf(red[2 * NR + x], red[3 * NR + x])), old = ref[x];
              change[y] = m - old > kAhead ? ex2_approx(old - m) : 1.0f;
              l[r + y] *= change[y];
            }
            if (j > 0) {
#pragma unroll
              for (int part = 0; part < 4; ++part) {  // both halves of the dims, high and low parts
                const uint32_t c = t_o + lanes + (part >> 1) * C::kCols + (part & 1) * NR + r0 + r;
                float o[8];
                tmem_ld<8>(c, o);
                ld_wait();
#pragma unroll
                for (int y = 0; y < 8; ++y) o[y] *= change[y];
                tmem_st<8>(c, o);
              }
            }
          }
          if (j > 0) st_wait();
          named_bar(1 + group, 128);
          if (key < RT) {
            const int x = r0 + key;
            const float m = fmaxf(fmaxf(red[x], red[NR + x]), fmaxf(red[2 * NR + x], red[3 * NR + x]));
            if (m - ref[x] > kAhead) ref[x] = m;
          }
          named_bar(1 + group, 128);
        }
        // weights, their sums, their two parts (the buffer is free once tile it - 2 is multiplied)
        if (it >= 2) await(&o_done[b], it / 2 - 1);
        uint8_t* pb = smem + C::kP + b * C::kCols * 128;
        const float real = top + ev - ref[own], above = fmaxf(ceilf(real), kUnset), back = ex2_approx(above - ev - kPlace);
        const float below = real - above + kPlace;  // the exponent of the row's largest weight here
        top = fmaxf(top, kUnset);                   // (kUnset: no key is seen)
#pragma unroll
        for (int r = 0; r < RT; r += 2) {
          // (the difference first: it is exact near the maximum however large the scores are)
          const float a = ex2_approx(s[r] - __shfl_sync(0xFFFFFFFFu, top, r) + __shfl_sync(0xFFFFFFFFu, below, r));
          const float c = ex2_approx(s[r + 1] - __shfl_sync(0xFFFFFFFFu, top, r + 1) + __shfl_sync(0xFFFFFFFFu, below, r + 1));
          const uint32_t hi = e4m3x2(a, c);
          const float2 f = f16x2_to_f32(e4m3x2_to_f16x2(hi));
          const uint32_t lo = e4m3x2((a - f.x) * kPLo, (c - f.y) * kPLo);
          const float2 g = f16x2_to_f32(e4m3x2_to_f16x2(lo));
          l[r] = fmaf(fmaf(g.x, 1.0f / kPLo, f.x), __shfl_sync(0xFFFFFFFFu, back, r), l[r]);
          l[r + 1] = fmaf(fmaf(g.y, 1.0f / kPLo, f.y), __shfl_sync(0xFFFFFFFFu, back, r + 1), l[r + 1]);
          pb[swizzled(r0 + r, key)] = static_cast<uint8_t>(hi);
          pb[swizzled(r0 + r + 1, key)] = static_cast<uint8_t>(hi >> 8);
          pb[swizzled(NR + r0 + r, key)] = static_cast<uint8_t>(lo);
          pb[swizzled(NR + r0 + r + 1, key)] = static_cast<uint8_t>(lo >> 8);
        }
        if (lane < RT) {  // down to the least that a byte holds
          constexpr float kLeast = 127.0f - kPlace;
          const uint8_t x = static_cast<uint8_t>(static_cast<int>(fminf(fmaxf(above, -kLeast), kAhead) + kLeast));
          uint8_t* to = smem + C::kScales + b * kScaleBytes;
          to[scale_at(r0 + lane, warp & 3)] = x;
          to[scale_at(NR + r0 + lane, warp & 3)] = x;
        }
        if (group == 0) {  // the values' scales, 1; the scores' place is free until this tile is multiplied
          const float one = __uint_as_float(0x7F7F7F7Fu), ones[4] = {one, one, one, one};
          tmem_st<4>(tmem + lanes + b * C::kCols + 4, ones);
          st_wait();
        }
        proxy_fence();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[b]);
      }
      // ---- the segment's end: sums over the keys, then the results
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float x = l[r];
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        if (lane == 0) red[(warp & 3) * NR + r0 + r] = x;
      }
      await(&o_done[(it - 1) & 1], (it - 1) / 2);
      tc_after();
      named_bar(3, 128 * C::kGroups);
#pragma unroll 1
      for (int x = 0; x < rows; x += 8) {
        float o[2][16];  // both halves of the dims, or this group's: high parts, low parts
#pragma unroll
        for (int i = 0; i < 2 / C::kGroups; ++i) {
          const uint32_t c = t_o + lanes + (C::kGroups == 2 ? group : i) * C::kCols + x;
          tmem_ld<8>(c, o[i]);
          tmem_ld<8>(c + NR, o[i] + 8);
        }
        ld_wait();
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int r = x + y;
          if (r >= rows) break;
          const float sum = red[r] + red[NR + r] + red[2 * NR + r] + red[3 * NR + r];
          const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
          const long long to = whole ? row_index(p, at_unit, r) * kHeadDim : (static_cast<long long>(slot) * NR + r) * kHeadDim;
#pragma unroll
          for (int i = 0; i < 2 / C::kGroups; ++i) {
            const int d = (C::kGroups == 2 ? group : i) * 128 + key;
            const float v = fmaf(o[i][8 + y], 1.0f / kPLo, o[i][y]);
            if (whole) store_out(p.out, p.out_f32, to + d, v * inv);
            else p.part_o[to + d] = v;
          }
          if (!whole && threadIdx.x == 0) p.part_ml[slot * NR + r] = make_float2(ref[r], sum);
        }
      }
      tc_before();
      named_bar(3, 128 * C::kGroups);  // red, ref and the query buffer are free again
    }
  }
  __syncthreads();
  if (warp == kIssuer) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem));
  }
}

// Joins the partial results of the units that ranges cut, in the order of the
// ranges.  CTA (g, y) takes `rows` rows of the unit that range g's end cuts, 8 /
// rows warps each, a lane per 8 dims: one row where the partials are many
// (eight warps share them, then add up through shared memory), eight where the
// rows are.  Latency: 5 us for 32 partials of 16 rows, 11 us for 150 cut units of
// 128 rows (39 MB, L2).
struct JoinParams {
  const float* part_o;
  const float2* part_ml;
  const Cut* cuts;
  void* out;
  int out_f32, heads, rep, nq, unit_rows, rows;
  short entry[IQ_MAX_BATCH];
  int count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ JoinParams p) {
  wait_for_last_kernel();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.last < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = 8 / p.rows;
  const int x = blockIdx.y * p.rows + warp / share, r = cut.z * p.unit_rows + x, j = r / p.rep;
  const bool live = x < p.unit_rows && r < p.count[cut.e] * p.rep;
  auto row = [&](int g) { return static_cast<long long>(g == static_cast<int>(blockIdx.x) ? cut.slot : 2 * g) * p.unit_rows + x; };
  __shared__ float part[8][kHeadDim + 2];
  float m = kUnset, sum = 0.0f, o[8] = {};
  if (live) {
    for (int g = blockIdx.x + lane; g <= cut.last; g += 32) m = fmaxf(m, __ldcg(&p.part_ml[row(g)]).x);  // every lane a partial
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll 4
    for (int g = blockIdx.x + warp % share; g <= cut.last; g += share) {
      const long long i = row(g);
      const float2 ml = __ldcg(&p.part_ml[i]);
      const float4* v = reinterpret_cast<const float4*>(p.part_o + i * kHeadDim + lane * 8);
      const float4 v0 = __ldcg(v), v1 = __ldcg(v + 1);
      const float f = ex2_approx(ml.x - m);
      sum = fmaf(f, ml.y, sum);
      o[0] = fmaf(f, v0.x, o[0]), o[1] = fmaf(f, v0.y, o[1]), o[2] = fmaf(f, v0.z, o[2]), o[3] = fmaf(f, v0.w, o[3]);
      o[4] = fmaf(f, v1.x, o[4]), o[5] = fmaf(f, v1.y, o[5]), o[6] = fmaf(f, v1.z, o[6]), o[7] = fmaf(f, v1.w, o[7]);
    }
  }
  if (share > 1) {
#pragma unroll
    for (int d = 0; d < 8; ++d) part[warp][d * 32 + lane] = o[d];
    if (lane == 0) part[warp][kHeadDim] = sum;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < 8; ++w) {
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] += part[w][d * 32 + lane];
      sum += part[w][kHeadDim];
    }
  }
  if (!live) return;
  const long long to = static_cast<long long>((p.entry[cut.e] * p.heads + cut.h) * p.rep + r - j * p.rep) * p.nq + j;
  store_out8(p.out, p.out_f32, to * kHeadDim + lane * 8, o, sum == 0.0f ? 0.0f : 1.0f / sum);
}

// Rows of entries without a key: zeros.
struct ZeroParams {
  void* out;
  int q_heads, nq, out_bytes;
  short entry[IQ_MAX_BATCH];
  int count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) paged_zero_kernel(const __grid_constant__ ZeroParams p) {
  wait_for_last_kernel();
  const int pieces = kHeadDim * p.out_bytes / 16;
  const long long n = static_cast<long long>(p.count[blockIdx.y]) * pieces;
  for (int h = 0; h < p.q_heads; ++h) {
    uint4* out = static_cast<uint4*>(p.out) + (static_cast<long long>(p.entry[blockIdx.y]) * p.q_heads + h) * p.nq * pieces;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) out[i] = make_uint4(0, 0, 0, 0);
  }
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Up to 32 query rows per kv head the split kernel, beyond the prefill kernel.
// Measured over 8 x 131072 tokens (and 4 x 16384, 1 x 4096 with 8 kv heads): 32 rows
// 173.5 us split (28.3, 20.3); 33 rows 194.6 prefill (29.4, 21.0); a split kernel of
// 64 rows, which spills and stores its weights byte by byte, took 255.5 us at 33
// rows (37.7, 24.7) and 265.6 at 64 (45.9, 33.0), the prefill kernel 197.0 (31.2, 22.7).
constexpr int kMaxSplitRows = 32;
int unit_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kMaxSplitRows ? 32 : 128; }

// The tiles of one head of an entry whose units hold `each` rows, and how many units those are.
long long tiles_of_entry(int len, int count, int rep, int each, int causal, int window, int sinks, int* units) {
  long long n = 0;
  const int all = count * rep;
  *units = 0;
  for (long long r = 0; r < all; r += each, ++*units)
    n += tiles_of(len, len - count + static_cast<int>(r) / rep, len - count + (static_cast<int>(std::min<long long>(r + each, all)) - 1) / rep,
                  causal, window, sinks).n;
  return n;
}
// What a unit's beginning and end take, in tiles, where a range has 8 tiles or
// more (shorter ones are left at a tile's grain).  Measured, 0 / 1 / 2 / 4 / 6:
// 4 x 1531 prompts - / 137 / 131 / 138 / 145 us; batched decode under a window
// of 4096 - / 34.5 / 33.9 / 32.9 / - us.
constexpr int unit_cost(int each) { return each == 128 ? 2 : 4; }

template <int NR>
cudaError_t launch_split(const AttendParams& p, int grid, cudaStream_t stream) {
  using C = SplitShape<NR>;
  static std::atomic<uint64_t> seen{0};
  const void* kernel = reinterpret_cast<const void*>(&paged_split_kernel<NR>);
  const cudaError_t e = allow_smem(kernel, C::kSmem, seen);
  void* args[] = {const_cast<AttendParams*>(&p)};
  return e == cudaSuccess ? launch_after(kernel, dim3(grid), C::kThreads, C::kSmem, stream, args) : e;
}

}  // namespace

thread_local int launch_to_fail = -1;
thread_local bool stall_next = false;

cudaError_t launch_after(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t stream, void** args) {
  if (launch_to_fail >= 0 && launch_to_fail-- == 0) return cudaErrorLaunchFailure;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && seen.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) seen.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

bool code_map(CUtensorMap* map, const uint8_t* codes, long long rows, int box_rows) {
  const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(rows)}, strides[1] = {kHeadDim};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, unit[2] = {1, 1};
  auto fn = encode_fn();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int store_zeros(const iq_paged* c, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, void* out,
                int out_f32, iq_stream_t stream) {
  ZeroParams z;
  z.out = out;
  z.q_heads = q_heads;
  z.nq = n_queries;
  z.out_bytes = out_f32 ? 4 : 2;
  int n = 0, most = 0;
  for (int i = 0; i < n_slots; ++i) {
    const int count = counts ? counts[i] : n_queries;
    if (count == 0 || c->lens[slot_of(slots, i)] > 0) continue;
    z.entry[n] = static_cast<short>(i);
    z.count[n++] = count;
    most = std::max(most, count);
  }
  if (n == 0) return IQ_OK;
  void* args[] = {&z};
  IQ_CUDA(launch_after(reinterpret_cast<const void*>(&paged_zero_kernel), dim3(std::min(64, (most + 7) / 8), n), 256, 0,
                       static_cast<cudaStream_t>(stream), args));
  launched_outputs(stream, {out, static_cast<size_t>(n_slots) * q_heads * n_queries * kHeadDim * (out_f32 ? 4 : 2)});
  return IQ_OK;
}

int check_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                 const int32_t* counts, int n_slots, int added, float scale, int causal, int window, int sinks,
                 const void* out, int out_f32, const void* workspace, size_t workspace_bytes) {
  size_t need = 0;
  int st = iq_paged_attend_workspace(c, q_heads, n_queries, n_slots, &need);
  if (st != IQ_OK) return st;
  st = check_slots(c, slots, n_slots, false);
  if (st != IQ_OK) return st;
  if (causal != 0 && causal != 1) return fail(IQ_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (window < 0 || sinks < 0) return fail(IQ_ERR_INVALID_ARG, "negative window or sinks");
  if (window > 0 && !causal) return fail(IQ_ERR_INVALID_ARG, "a window needs causal attention");
  if (sinks > 0 && window == 0) return fail(IQ_ERR_INVALID_ARG, "sinks need a window");
  if (out_f32 != 0 && out_f32 != 1) return fail(IQ_ERR_INVALID_ARG, "out_f32 must be 0 or 1");
  if (!(scale - scale == 0.0f)) return fail(IQ_ERR_INVALID_ARG, "scale is not finite");
  if (counts)
    for (int i = 0; i < n_slots; ++i)
      if (counts[i] < 0 || counts[i] > n_queries) return fail(IQ_ERR_INVALID_ARG, "counts[i] outside [0, n_queries]");
  if (n_slots == 0 || n_queries == 0) return IQ_OK;
  if (!q || !out) return fail(IQ_ERR_INVALID_ARG, "null q/out");
  if (misaligned(q) || misaligned(out)) return fail(IQ_ERR_INVALID_ARG, "q/out not 16-byte aligned");
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return fail(IQ_ERR_WORKSPACE, "workspace missing or too small");
    if (misaligned(workspace, 256)) return fail(IQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  }
  // the slots of all units stay below 2^31: told by a bound, counted where that passes it
  const int rep = q_heads / c->kv_heads, each = unit_rows(n_queries * rep);
  for (int exact = 0; exact < 2; ++exact) {
    long long total = 0;
    for (int i = 0; i < n_slots; ++i) {
      const int count = counts ? counts[i] : n_queries, len = c->lens[slot_of(slots, i)] + (counts && added ? counts[i] : added);
      if (len <= 0 || count <= 0) continue;
      int units = (count * rep + each - 1) / each;
      const long long tiles = exact ? tiles_of_entry(len, count, rep, each, causal, window, sinks, &units)
                                    : static_cast<long long>(units) * (len / kTile + 1);
      total += (tiles + static_cast<long long>(units) * unit_cost(each)) * c->kv_heads;
    }
    if (total < (1LL << 31)) return IQ_OK;
  }
  return fail(IQ_ERR_UNSUPPORTED, "too many queries and keys for one call");
}

}  // namespace paged
}  // namespace iq

using namespace iq;
using namespace iq::paged;

extern "C" {

int iq_paged_attend_workspace(const iq_paged* c, int q_heads, int n_queries, int n_slots, size_t* bytes) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  if (!bytes) return fail(IQ_ERR_INVALID_ARG, "null bytes");
  if (q_heads <= 0 || n_queries < 0 || n_slots < 0) return fail(IQ_ERR_INVALID_ARG, "bad q_heads, n_queries or n_slots");
  if (n_slots > IQ_MAX_BATCH) return fail(IQ_ERR_INVALID_ARG, "bad number of slots");
  if (q_heads % c->kv_heads) return fail(IQ_ERR_UNSUPPORTED, "q_heads must be a multiple of kv_heads");
  if (q_heads / c->kv_heads > kMaxRep) return fail(IQ_ERR_UNSUPPORTED, "at most 64 query heads per kv head");
  if (static_cast<long long>(n_queries) * (q_heads / c->kv_heads) >= (1LL << 30)) return fail(IQ_ERR_UNSUPPORTED, "too many query rows");
  const int rows = n_queries * (q_heads / c->kv_heads);
  const size_t parts = rows > 0 && n_slots > 0 ? 2 * static_cast<size_t>(num_sms()) * unit_rows(rows) : 0;
  *bytes = parts ? parts * (kHeadDim * sizeof(float) + sizeof(float2)) + num_sms() * sizeof(Cut) : 0;
  if (rows > kMaxSplitRows) {  // the queries' two parts and factors
    const size_t all = static_cast<size_t>(n_slots) * q_heads * n_queries;
    if (all >= (1u << 30)) return fail(IQ_ERR_UNSUPPORTED, "too many query rows");
    *bytes += all * (2 * kHeadDim + sizeof(float));
  }
  return IQ_OK;
}

int iq_paged_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                    const int32_t* counts, int n_slots, float scale, int causal, int window, int sinks, void* out,
                    int out_f32, void* workspace, size_t workspace_bytes, iq_stream_t stream) {
  const int st = check_attend(c, q, q_heads, n_queries, slots, counts, n_slots, 0, scale, causal, window, sinks, out, out_f32,
                              workspace, workspace_bytes);
  if (st != IQ_OK || n_slots == 0 || n_queries == 0) return st;
  const int rep = q_heads / c->kv_heads, rows = rep * n_queries;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const Range written{out, static_cast<size_t>(n_slots) * q_heads * n_queries * kHeadDim * (out_f32 ? 4 : 2)};
  int longest = 0;
  for (int i = 0; i < n_slots; ++i) longest = std::max(longest, c->lens[slot_of(slots, i)]);
  if (window >= longest) window = sinks = 0;  // nothing is out of it, and positions less a window stay in 32 bits
  const int zeroed = store_zeros(c, q_heads, n_queries, slots, counts, n_slots, out, out_f32, stream);
  if (zeroed != IQ_OK) return zeroed;
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.unit_rows = unit_rows(rows);
  long long tiles = 0, per[IQ_MAX_BATCH];
  int units[IQ_MAX_BATCH];
  for (int i = 0; i < n_slots; ++i) {
    const int len = c->lens[slot_of(slots, i)], count = counts ? counts[i] : n_queries;
    per[i] = units[i] = 0;
    if (len > 0 && count > 0) tiles += (per[i] = tiles_of_entry(len, count, rep, p.unit_rows, causal, window, sinks, &units[i])) * c->kv_heads;
  }
  const int grid = static_cast<int>(std::min<long long>(num_sms(), tiles));
  if (grid == 0) return IQ_OK;
  p.cost = tiles >= 8ll * grid ? unit_cost(p.unit_rows) : 0;
  long long total = 0;
  for (int i = 0; i < n_slots; ++i) {
    const int s = slot_of(slots, i), len = c->lens[s], count = counts ? counts[i] : n_queries;
    if (count == 0 || len == 0) continue;
    const int e = p.entries++;
    p.entry[e] = static_cast<short>(i);
    p.slot[e] = static_cast<short>(s);
    p.len[e] = len;
    p.count[e] = count;
    p.cum[e] = static_cast<int>(total);
    per[i] += static_cast<long long>(units[i]) * p.cost;
    total += per[i] * c->kv_heads;
    p.per[e] = static_cast<int>(per[i]);
  }
  p.cum[p.entries] = p.total = static_cast<int>(total);
  const long long pool_rows = static_cast<long long>(c->pages) * c->kv_heads * kPage;
  if (!code_map(&p.k_map, c->k_codes, pool_rows) || !code_map(&p.v_map, c->v_codes, pool_rows))
    return fail(IQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.q = static_cast<const uint16_t*>(q);
  p.out = out;
  p.out_f32 = out_f32;
  p.heads = c->kv_heads;
  p.rep = rep;
  while ((2 << p.rep_shift) <= rep) ++p.rep_shift;
  if (rep & (rep - 1)) p.rep_mul = static_cast<unsigned>(((1ull << (32 + p.rep_shift)) + rep - 1) / rep);
  p.nq = n_queries;
  p.pages = c->pages;
  p.max_pages = c->max_pages;
  p.causal = causal;
  p.window = window;
  p.sinks = sinks;
  p.scale = scale;
  p.stall = stall_next ? 1 : 0;
  stall_next = false;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2ll * num_sms() * p.unit_rows * kHeadDim);
  p.cuts = reinterpret_cast<Cut*>(p.part_ml + 2ll * num_sms() * p.unit_rows);
  int all_counts[IQ_MAX_BATCH];
  if (p.unit_rows == 128) {
    const long long all = static_cast<long long>(n_slots) * q_heads * n_queries;
    p.cut = reinterpret_cast<uint8_t*>(p.cuts + num_sms());  // 16-byte aligned
    p.factors = reinterpret_cast<float*>(p.cut + all * 2 * kHeadDim);
    p.slots_n = n_slots;
    for (int i = 0; i < n_slots; ++i) all_counts[i] = counts ? counts[i] : n_queries;
    if (!code_map(&p.q_map, p.cut, 2 * all, 128)) return fail(IQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  }
  cudaError_t err = p.unit_rows == 8    ? launch_split<8>(p, grid, cs)
                    : p.unit_rows == 16 ? launch_split<16>(p, grid, cs)
                    : p.unit_rows == 32 ? launch_split<32>(p, grid, cs)
                                        : launch_prefill(p, all_counts, grid, cs);
  if (err == cudaSuccess && grid > 1) {
    const int each = p.unit_rows == 128 ? 8 : 1, most = std::min(p.unit_rows, rows);
    JoinParams j;
    j.part_o = p.part_o;
    j.part_ml = p.part_ml;
    j.cuts = p.cuts;
    j.out = p.out;
    j.out_f32 = p.out_f32;
    j.heads = p.heads;
    j.rep = p.rep;
    j.nq = p.nq;
    j.unit_rows = p.unit_rows;
    j.rows = each;
    std::memcpy(j.entry, p.entry, sizeof(j.entry));
    std::memcpy(j.count, p.count, sizeof(j.count));
    void* args[] = {&j};
    err = launch_after(reinterpret_cast<const void*>(&paged_join_kernel), dim3(grid - 1, (most + each - 1) / each), 256, 0, cs, args);
  }
  if (err != cudaSuccess) return cuda_fail(err, "paged attention");
  launched_outputs(stream, written);
  return IQ_OK;
}

}  // extern "C"
