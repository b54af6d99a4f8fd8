// Attention of few query rows per kv head over the paged 8-bit cache: what a CTA does.
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
#pragma once

#include <type_traits>

#include "iq_paged_mma.cuh"

namespace iq {
namespace paged {
namespace split {

constexpr int kMu = 4, kHu = 1;  // products unrolled in a tree
constexpr float kPlace = 6.0f;  // the place of a block's largest weight
constexpr float kPLo = 128.0f;  // the low parts' scale: half a step at 2^6 is 2, times 128 below 448

template <int NR, int TURNS = 1>
struct Shape {
  static constexpr int kTurns = TURNS;                // tiles of the sequence on the softmax at once
  static constexpr int kGroups = NR >= 32 ? 2 : 1;    // warpgroups on a tile, NR / kGroups rows each
  static constexpr int kRows = NR / kGroups;
  static constexpr int kWarps = 4 * kGroups * TURNS;  // on the softmax
  static constexpr int kCols = 2 * NR;                // high and low parts
  static constexpr int kSlots = 6;                    // tiles of keys or values in flight
  static constexpr int kQ = kSlots * kSlotBytes;      // [2 halves of the dims][kCols rows][128 bytes]
  static constexpr int kP = kQ + 2 * kCols * 128;     // [2][kCols rows][128 keys]
  static constexpr int kScales = kP + 2 * kCols * 128;  // [2] the weights'
  static constexpr int kMisc = kScales + 2 * kScaleBytes;
  static constexpr int kRing = Loader<kSlots, false>::kRing;
  static constexpr int kFloats = NR + TURNS * (NR + 4 * NR);  // factors; references, reductions
  static constexpr int kBars = 2 * kSlots + kRing + 10;
  static constexpr int kSmem = kMisc + kFloats * 4 + kRing * 16 + kBars * 8 + 8;
  static constexpr int kThreads = kWarps * 32 + 64;
  static constexpr int kTmem = (TURNS == 2 ? 8 : 4) * kCols;  // S twice, O of both halves of the dims (of every turn)
  static_assert(TURNS == 1 || kGroups == 1, "eight warps at most");
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};
// In a tree only some of the SMs stream leaves, each at more than its share of HBM, so the
// row threads' chain (1.1 us a tile) would set the pace: up to 16 rows, two warpgroups take the
// tiles in turn, each with references, sums and results of its own.  Mean of 14 trees of 32 to
// 250 paths with leaves of 500 to 2048 tokens: 48.9 us with one warpgroup, 48.2 with two at
// 8 rows, 74.3 and 70.8 at 16.  (32 rows take two warpgroups for a tile as it is.)
template <int NR>
using TreeShape = Shape<NR, NR <= 16 ? 2 : 1>;

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
// P: AttendParams, or TreeParams: leaves of slots that share pages, all of whose results
// are partial.  smem: the whole of the CTA's, 1024-byte aligned; warps behind Shape's wait
// for the others.
template <int NR, class P>
__device__ __forceinline__ void run(const P& p, const Work& work, uint8_t* smem) {
  using C = std::conditional_t<P::kTree, TreeShape<NR>, Shape<NR>>;
  constexpr int kTurns = C::kTurns;
  constexpr int RT = C::kRows;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // (the kernel has no other shared memory in front)
    wait_for_last_kernel();
    if (threadIdx.x == 0) atomicOr(p.status, kLostMma);
    return;
  }
  float* factor = reinterpret_cast<float*>(smem + C::kMisc);  // [NR] 2^eq * scale * log2 e
  float* ref0 = factor + NR;                                  // [kTurns][NR]
  float* red0 = ref0 + kTurns * NR;                           // [kTurns][4 warps][NR]
  float4* scales = reinterpret_cast<float4*>(red0 + kTurns * 4 * NR);  // [kRing] of a tile's two pages: keys', values'
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
  constexpr int kLoader = C::kWarps, kIssuer = kLoader + 1;
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
    mbar_init(q_ready, C::kWarps);
    mbar_init(drained, 1);
    *abort = 0;
    mbar_fence_init();
  }
  // In a tree what the kernel in front writes is not read here, and that one began when
  // all before it was done (see the rows' kernel); it is waited for before the first results.
  if constexpr (!P::kTree) wait_only();
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(C::kTmem));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  release_dependents();
  const uint32_t tmem = *tslot;
  const uint32_t t_o = tmem + 2 * C::kCols;  // O: [turn][half of the dims][kCols]
  const Waits wait{abort, p.status};

  const int first = range_begin(work.block, work.grid, work.total), last = range_begin(work.block + 1, work.grid, work.total);
  const Place start = place_of(p, work, first);  // every role walks the same segments from here

  if (warp == kLoader) {
    Loader<C::kSlots, false, P>{p, work, smem, full, empty, scales, scales_in, wait}.run(start, first, last, policy_evict_first());
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
        const int tiles = tiles_at(p, w).n, n = part_of(work, w, tiles, last - at).n;
        at += tiles + work.cost - w.j;
        if (n == 0) break;
        ok = wait.together(q_ready, segment, kLostMma);
        for (int j = 0; j <= n && ok; ++j) {
          if (j < n) {
            const int b = (it + j) & 1, s = used % C::kSlots;
            if (it + j >= 2) ok = wait.together(&s_free[b], (it + j) / 2 - 1, kLostMma);
            ok = ok && wait.together(&full[s], used / C::kSlots, kLostMma);
            if (!ok) break;
            tc_after();
#pragma unroll P::kTree ? kMu : 8
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
#pragma unroll P::kTree ? kHu : 2
            for (int half = 0; half < 2; ++half)
#pragma unroll P::kTree ? kMu : 4
              for (int k = 0; k < 4; ++k)
                mma_scaled(t_o + ((kTurns == 2 ? 2 * b : 0) + half) * C::kCols, at_slot + ((s * kSlotBytes + half * kHalfBytes + k * 32 * 128) >> 4),
                           weights + ((b * C::kCols * 128 + k * 32) >> 4), shape_scaled(128, C::kCols, true, false, 0, k), place + 4, place,
                           j > kTurns || k > 0);
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
  } else if (warp < kLoader) {
    // ---------------------------------------------------------------- softmax: a key per thread
    // tiles of both parities, or this warpgroup's; all rows, or its half; its barrier
    const int turn = kTurns == 2 ? warp >> 2 : 0, group = kTurns == 2 ? 0 : warp >> 2, own_bar = 1 + (warp >> 2);
    const int key = threadIdx.x & 127, r0 = group * RT;
    float *ref = ref0 + turn * NR, *red = red0 + turn * 4 * NR;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    if constexpr (!P::kTree) {
      if (threadIdx.x == 0) p.cuts[work.block].last = -1;
    }
    float l[RT];
    int it0 = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t phase) {  // a lost wait changes no path: every barrier below is still reached
      if (ok) ok = wait(bar, phase, kLostRows);
      __syncwarp();
    };
    bool at_first = true;
    Place at_unit = start;
    // the query rows, a warp each; with turns, which leave the registers, those of the next unit
    // are fetched before this one's tiles
    constexpr int kEach = NR / C::kWarps;
    uint4 raw[kEach];
    auto fetch = [&](const Place& unit) {
      const int rows = rows_at(p, unit);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = warp + i * C::kWarps;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (r < rows) raw[i] = __ldcg(reinterpret_cast<const uint4*>(p.q + row_index(p, unit, r) * kHeadDim) + lane);
      }
    };
    if (kTurns == 2 && first < last) fetch(start);
    for (int at = first; at < last; next_unit(p, at_unit)) {
      const Tiles tiles = tiles_at(p, at_unit);
      const Part part = part_of(work, at_unit, tiles.n, last - at);
      const int k0 = part.begin, n = part.n, rows = rows_at(p, at_unit);
      const bool whole = !P::kTree && n == tiles.n;
      int row0, len;  // the partial results' first row; keys that there are
      if constexpr (P::kTree) {
        row0 = k0 == 0 ? p.part0[at_unit.e] + at_unit.h * rows : p.narrow_cont + work.block * NR;
        len = tiles.p_hi + 1;
      } else {
        const int slot = 2 * work.block + (at == first ? 0 : 1);
        if (n > 0 && n < tiles.n && k0 == 0 && threadIdx.x == 0) tell_cut(p, work, at_unit, at, tiles.n, slot);
        row0 = slot * NR;
        len = p.len[at_unit.e];
      }
      at += tiles.n + work.cost - at_unit.j;
      if (n == 0) break;
      if (kTurns == 1) fetch(at_unit);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int r = warp + i * C::kWarps;
        uint2 hi, lo;
        const float f = clamp_finite(split_query<16>(raw[i], hi, lo) * (p.scale * kLog2e));
        uint8_t* to = smem + C::kQ + (lane >> 4) * C::kCols * 128;
        *reinterpret_cast<uint2*>(to + swizzled(r, (lane & 15) * 8)) = hi;
        *reinterpret_cast<uint2*>(to + swizzled(NR + r, (lane & 15) * 8)) = lo;
        if (lane == 0) {
          factor[r] = f;
#pragma unroll
          for (int x = 0; x < kTurns; ++x) ref0[x * NR + r] = r < rows ? kUnset : kDead;
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      if (kTurns == 2 && at < last) {
        Place next = at_unit;
        next_unit(p, next);
        fetch(next);
      }
      named_bar(3, C::kWarps * 32);
#pragma unroll
      for (int r = 0; r < RT; ++r) l[r] = 0.0f;

      // (a tree's first turn is a rehearsal: it fetches the instructions, see the rows' kernel)
      const int j0 = kTurns == 2 ? (turn - it0) & 1 : 0;  // the first tile of this turn
      for (int j = P::kTree && at_first ? j0 - kTurns : j0; j < n; j += kTurns) {
        const int it = it0 + j, b = it & 1;
        const bool rehearsal = P::kTree && j < 0;
        if (!rehearsal) await(&scales_in[it % C::kRing], it / C::kRing);
        static_assert((C::kRing & (C::kRing - 1)) == 0, "tile -1 has a place");
        const float* sc = reinterpret_cast<const float*>(&scales[it & (C::kRing - 1)]) + (key >> 6);  // this key's page
        const float ks = sc[0];
        const float ev = static_cast<float>(exponent_of(sc[2]));
        const int t0 = tiles.tile(k0 + j) * kTile;
        if (!rehearsal) await(&s_full[b], it / 2);
        tc_after();
        float s[RT], w[RT];
        tmem_ld<RT>(tmem + lanes + b * C::kCols + r0, s);
        tmem_ld<RT>(tmem + lanes + b * C::kCols + NR + r0, w);
        ld_wait();
        tc_before();
        __syncwarp();
        if (lane == 0 && !rehearsal) mbar_arrive(&s_free[b]);
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
        int far = (lane < RT && top + ev - ref[own] > kAhead) || rehearsal;
        asm volatile("{\n.reg .pred a, b;\nsetp.ne.s32 a, %0, 0;\nbarrier.cta.red.or.pred b, %1, 128, a;\nselp.s32 %0, 1, 0, b;\n}"
                     : "+r"(far)
                     : "r"(own_bar)
                     : "memory");
        if (far) {
          // some row's scores passed its reference by 2^kAhead, or are its first: move
          // the references of such rows to their maxima, and what was summed with them
          if (lane < RT) red[(warp & 3) * NR + own] = top + ev;
          named_bar(own_bar, 128);
          const bool had = j >= kTurns;  // a tile before this one, in the same sums
          if (had) await(&o_done[(it - kTurns) & 1], (it - kTurns) / 2);
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
            if (had) {
#pragma unroll
              for (int part = 0; part < 4; ++part) {  // both halves of the dims, high and low parts
                const uint32_t c = t_o + lanes + (2 * turn + (part >> 1)) * C::kCols + (part & 1) * NR + r0 + r;
                float o[8];
                tmem_ld<8>(c, o);
                ld_wait();
#pragma unroll
                for (int y = 0; y < 8; ++y) o[y] *= change[y];
                tmem_st<8>(c, o);
              }
            }
          }
          if (had) st_wait();
          named_bar(own_bar, 128);
          if (key < RT) {
            const int x = r0 + key;
            const float m = fmaxf(fmaxf(red[x], red[NR + x]), fmaxf(red[2 * NR + x], red[3 * NR + x]));
            if (m - ref[x] > kAhead) ref[x] = m;
          }
          named_bar(own_bar, 128);
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
        if (P::kTree && rehearsal) {
          named_bar(own_bar, 128);
          if (key < RT) ref[r0 + key] = r0 + key < rows ? kUnset : kDead;
#pragma unroll
          for (int r = 0; r < RT; ++r) l[r] = 0.0f;
          named_bar(own_bar, 128);
          continue;
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
      if (P::kTree && at_first) wait_only();
      at_first = false;
      it0 += n;
      // ---- the segment's end: sums over the keys, then the results
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float x = l[r];
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        if (lane == 0) red[(warp & 3) * NR + r0 + r] = x;
      }
      // The last tile's product (products end in order).  With turns the other warps' barrier comes first: a
      // warp that had no part in that tile cannot tell the end of its phase from that of the one
      // before, two tiles earlier, which the warps that had waited for.
      if constexpr (kTurns == 2) named_bar(3, C::kWarps * 32);
      await(&o_done[(it0 - 1) & 1], (it0 - 1) / 2);
      tc_after();
      if constexpr (kTurns == 1) named_bar(3, C::kWarps * 32);
      if constexpr (kTurns == 2) {
        // half of the dims each: both turns' results, under the larger of their references
        const bool had0 = n > 1 || (it0 & 1), had1 = n > 1 || !(it0 & 1);
#pragma unroll 1
        for (int x = 0; x < rows; x += 8) {
          float o[2][16];  // of each turn: high parts, low parts
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t c = t_o + lanes + (2 * i + turn) * C::kCols + x;
            tmem_ld<8>(c, o[i]);
            tmem_ld<8>(c + NR, o[i] + 8);
          }
          ld_wait();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int r = x + y;
            if (r >= rows) break;
            float sums[2], f[2];
            const float top = fmaxf(ref0[r], ref0[NR + r]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float* of = red0 + i * 4 * NR + r;
              sums[i] = of[0] + of[NR] + of[2 * NR] + of[3 * NR];
              f[i] = ex2_approx(ref0[i * NR + r] - top);
            }
            // (a turn that had no tile: its sums are 0, its results another unit's)
            const float v0 = had0 ? fmaf(o[0][8 + y], 1.0f / kPLo, o[0][y]) : 0.0f;
            const float v1 = had1 ? fmaf(o[1][8 + y], 1.0f / kPLo, o[1][y]) : 0.0f;
            p.part_o[static_cast<long long>(row0 + r) * kHeadDim + turn * 128 + key] = fmaf(f[0], v0, f[1] * v1);
            if (threadIdx.x == 0)
              p.part_ml[row0 + r] = make_float2(top, fmaf(f[0], sums[0], f[1] * sums[1]));
          }
        }
      } else {
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
            const long long to = (whole ? row_index(p, at_unit, r) : row0 + r) * kHeadDim;
#pragma unroll
            for (int i = 0; i < 2 / C::kGroups; ++i) {
              const int d = (C::kGroups == 2 ? group : i) * 128 + key;
              const float v = fmaf(o[i][8 + y], 1.0f / kPLo, o[i][y]);
              if (whole) store_out(p.out, p.out_f32, to + d, v * inv);
              else p.part_o[to + d] = v;
            }
            if (!whole && threadIdx.x == 0) p.part_ml[row0 + r] = make_float2(ref[r], sum);
          }
        }
      }
      tc_before();
      named_bar(3, C::kWarps * 32);  // red, ref and the query buffer are free again
    }
  }
  __syncthreads();
  if (warp == kIssuer) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmem));
  }
}

}  // namespace split
}  // namespace paged
}  // namespace iq
