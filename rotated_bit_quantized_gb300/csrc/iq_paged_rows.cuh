// Attention of many query rows per kv head over the paged 8-bit cache: what a CTA does.
//
// The same mathematics as the split kernel (iq_paged_split.cuh) with the query
// rows as the products' M dimension: S = Q.K^T with Q as two e4m3 parts summed
// into one accumulator, S (128 rows x 128 keys) twice in tensor memory, and
// O += W.V with the weights W as two e4m3 parts that the row threads write over
// the scores they came from.  Keys and values are the pages' codes as they lie
// in HBM.  Each product runs twice (high and low part) at e4m3's rate, twice
// bf16's, so the bound is bf16's rate; no code is ever converted.
//
// Rounding.  The second product is block-scaled: with e the exponent s + ev - ref of
// the largest weight of a row's 32 keys, rounded up, they are held as 2^(s + ev - ref
// - e + 8) under the scale 2^(e - 8).  A weight, as fp16 at first (2^-11 of it), leaves
// at most 2^-8 of it behind its two parts, and half a step of the least codes, 2^-10,
// where it lies below their range: 2^-17 of the largest weight among its 32 keys,
// whatever the row's other keys weigh.  (One reference for a row's whole tile, its running
// maximum at 2^5, left a floor of 2^-15 of the row's largest weight: next to one
// key with half of it, 32768 others were off by 12% in norm, 131072 by 32%.)
// The scales also carry what a row's reference does not: that one only keeps the
// sums in fp32's range, and moves when the weights pass it by 2^kAhead.  It is the
// row's maximum as it was then, not rounded, so that this key's weight is exact.
// In norm, on random rows with outliers, the weights leave 0.0006 to 0.0007 of the
// result (bfloat16 weights 0.0016); with references that move at 2^6, so that the
// heaviest key is exact more often, 0.0005, but 5 to 8% slower where units are
// short; with sums of the weights as they are held, 0.0004, but 4% slower.  In a tree
// the sums are those: its rows would run in the split kernel, whose sums are, if their pages
// were not shared.  32 paths of 32768 common tokens: 0.00037 off in norm, apart 0.00037, for
// 2% of the time (5% where the held weights were converted before they were added).  A
// query's second part has the first one's scale here and 16 times it there: elements 2^10
// (there 2^14) below the row's largest are held to 2^-17 of that one (2^-21), half a step of
// the least code, far below the weights' own roundings.
#pragma once

#include "iq_paged_mma.cuh"

namespace iq {
namespace paged {
namespace rows {

constexpr int kMu = 4;  // products unrolled in a tree (fully: 9 KB more to fetch; rolled: 2.2 us a tile instead of 1.45 then)
constexpr int kRows = 128;
constexpr int kSlots = 4;                         // tiles of keys or values in flight, from L2 mostly (3: no slower, 5: 1.5% slower)
constexpr int kQ = kSlots * kSlotBytes;           // [high, low][2 halves of the dims][128 rows][128 bytes]
constexpr int kScales = kQ + 4 * kHalfBytes;      // of the weights of a tile, twice; ones, the values'
constexpr int kMisc = kScales + 3 * kScaleBytes;
constexpr int kRing = Loader<kSlots, true>::kRing;
constexpr int kSmem = kMisc + 2 * kRows * 4 + kRing * 16 + 32 * 8;
constexpr int kStage = (kSmem + 127) / 128 * 128;  // trees: partial results on their way out, 4 KB per warp
constexpr int kTreeSmem = kStage + 8 * 4096;
constexpr int kThreads = 384;
constexpr int kLoader = 8, kIssuer = 9, kAsker = 10;
constexpr int kRowRegs = 208, kRestRegs = 88;     // 2 * 208 + 88 = 3 * 168, what the CTA is launched with
constexpr float kPlace = 8.0f;                    // the place of a block's largest weight (2^8.8 = 448 is the largest code)
constexpr float kFar = 16384.0f;                  // scores from here on take differences first
constexpr int kWeightScales = 32, kOnes = 96;     // their columns among a tile's 128, where its scores were
static_assert(kTreeSmem <= 232448, "shared memory of one CTA");

// One persistent CTA per SM, three warpgroups.  Warps 0-7: two threads per query
// row (warp w reaches tensor-memory lanes 32 (w % 4) ..), each with the 64 keys
// of one page of a tile; warps w and w + 4 hold the same rows and settle the
// rows' references between themselves.  Then one warp streams the pages, one
// issues the products, S of the next tile but one behind O of this tile, and one
// fetches a unit's queries once the last unit's scores are done.  A unit's
// results are stored after the next unit's first weights are written, so the
// products wait for the stores alone.
// Bound by the row threads' chain (scores out of tensor memory, maximum, vote,
// exponentials, two parts, back), 2.6 K cycles a tile, next to the products' 2.1 K
// (measured alone, of 2.05 K at the nominal rate).  2048 queries of 16 / 2 heads
// over 32768 keys: 736 us, 1450 TFLOP/s, 76% of a measured bf16 matrix product
// (710 with weights that are not block-scaled, whose second product reads no
// scales); a unit's beginning and end cost 4 to 5 tiles' time, which shows where
// units are short: 4 x 1531 tokens 116 us, 8191 under a window of 1023 171 us.  What counted
// on the way: the queries cut beforehand (260 to 214 us on the last), products
// issued by a whole warp (745 to 673 us on the first), the references' rescaling
// behind the weights, scores issued over a unit's end.
// P: AttendParams, or TreeParams: units of slots that share pages, all of whose results
// are partial.  smem: the whole of the CTA's, 1024-byte aligned.
// In a tree a CTA has ten tiles or so, and its beginning counts: 32 paths of 32768 common
// tokens, 16 / 2 heads, take 6 us until the first scores (instructions are fetched by all
// CTAs at once, 0.14 us a kilobyte), 1.5 us a tile and 3 us for the results.
template <class P>
__device__ __forceinline__ void run(const P& p, const Work& work, uint8_t* smem) {
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // (the kernel has no other shared memory in front)
    wait_for_last_kernel();
    if (threadIdx.x == 0) atomicOr(p.status, kLostMma);
    return;
  }
  float* xch = reinterpret_cast<float*>(smem + kMisc);          // [2][128] what the two threads of a row exchange
  float4* scales = reinterpret_cast<float4*>(xch + 2 * kRows);  // [kRing] of a tile's two pages: keys', values'
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + kRing);
  uint64_t* empty = full + kSlots;
  uint64_t* scales_in = empty + kSlots;
  uint64_t* s_full = scales_in + kRing;  // [2] scores of a tile in tensor memory
  uint64_t* p_ready = s_full + 2;      // [2] weights of a tile in their place
  uint64_t* o_done = p_ready + 2;      // [2] and multiplied with its values
  uint64_t* q_ready = o_done + 2;      // a segment's queries in shared memory
  uint64_t* q_free = q_ready + 1;      // a segment's last scores done
  uint64_t* drained = q_free + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert(2 * kSlots + kRing + 10 < 31, "the barriers and the two words behind them fit");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kRing; ++s) mbar_init(&scales_in[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_ready[s], 8);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(q_ready, 1);
    mbar_init(q_free, 1);
    mbar_init(drained, 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (threadIdx.x < kScaleBytes / 4) reinterpret_cast<uint32_t*>(smem + kScales + 2 * kScaleBytes)[threadIdx.x] = 0x7F7F7F7Fu;
  proxy_fence();
  // In a tree the kernel in front is the one that cuts the queries, which takes no tensor
  // memory and lets this one begin when all before it is done: only what it writes is waited for,
  // by the threads that read it, and by every CTA before it stores a result.  Pages, scales and the table
  // are read in front of that wait.  This rests on the cutting kernel: each of its threads has waited for
  // the kernels that wrote them, whose writes are then in L2, before it lets this kernel begin, and
  // all of these reads go to L2 (bulk copies, ld.cg), none to what an L1 may have kept.
  if constexpr (!P::kTree) wait_only();
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_before();
  __syncthreads();
  tc_after();
  release_dependents();
  const uint32_t tmem = *tslot, t_o = tmem + 256;  // S or W: 0..127, 128..255; O: 256..511
  const Waits wait{abort, p.status};

  const int first = range_begin(work.block, work.grid, work.total), last = range_begin(work.block + 1, work.grid, work.total);
  const Place start = place_of(p, work, first);
  int q_rows;  // high parts, then as many rows of low parts
  if constexpr (P::kTree) q_rows = p.heads * p.rows;
  else q_rows = p.slots_n * p.heads * p.rep * p.nq;

  if (warp < kLoader) {
    // ---------------------------------------------------------------- softmax: half a row per thread
    setmaxnreg_inc<kRowRegs>();
    const int group = warp >> 2, quad = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int it = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t phase) {  // a lost wait changes no path: every barrier below is still reached
      if (ok) ok = wait(bar, phase, kLostRows);
      __syncwarp();
    };
    if constexpr (!P::kTree) {
      if (threadIdx.x == 0) p.cuts[work.block].last = -1;
    }
    // the unit whose results are still in tensor memory
    Place done{};
    bool pending = false, done_whole = false;
    int done_row = 0;  // of partial results: its first row's place
    float done_l = 0.0f, done_ref = 0.0f;
    auto store_results = [&](int last_tile) {  // the sums of a row's two halves, half of its dims per thread
      xch[group * kRows + r] = done_l;
      named_bar(1 + quad, 64);
      const float sum = done_l + xch[(group ^ 1) * kRows + r];
      named_bar(1 + quad, 64);
      const int rows = min(kRows, rows_at(p, done));
      const float inv = !done_whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      const bool wide = !done_whole || p.out_f32;
      long long to = done_row + r;
      if constexpr (!P::kTree) {
        if (done_whole) to = row_index(p, done, done.z * kRows + min(r, rows - 1));
      }
      uint8_t* out = static_cast<uint8_t*>(done_whole ? p.out : p.part_o) + (to * kHeadDim + group * 128) * (wide ? 4 : 2);
      await(&o_done[last_tile & 1], last_tile / 2);
      tc_after();
      if constexpr (P::kTree) {
        // Short units: through 4 KB of shared memory per warp, so that a store covers four
        // rows' 128 bytes instead of 16 bytes of 32 rows (4 us less at a unit's end).
        uint8_t* stage = smem + kStage + warp * 4096;
        if (quad * 32 < rows) {
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float o[32];
            tmem_ld<32>(t_o + lanes + group * 128 + c, o);
            ld_wait();
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int x = 4 * i + (lane >> 3), piece = lane & 7, at = quad * 32 + x;
              const float4 v = *reinterpret_cast<const float4*>(stage + x * 128 + ((piece ^ (x & 7)) << 4));
              if (at < rows) *reinterpret_cast<float4*>(p.part_o + static_cast<long long>(done_row + at) * kHeadDim + group * 128 + c + piece * 4) = v;
            }
            __syncwarp();
          }
        }
      } else {
        // A thread stores its row in 32-byte pieces.  Slower, for 8191 queries under
        // a window of 1023 in 190 us: four lanes' pieces side by side through shuffles
        // (201), through shared memory and a warp that stores whole rows (213), kept as
        // bf16 and stored an eighth per tile (224, spills).
#pragma unroll 1
        for (int c = 0; c < 128; c += 32) {
          float o[32];
          tmem_ld<32>(t_o + lanes + group * 128 + c, o);
          ld_wait();
          if (r >= rows) continue;
          if (wide) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(out + (c + i) * 4) = make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x[k]) : "f"(o[i + 2 * k + 1] * inv), "f"(o[i + 2 * k] * inv));
              *reinterpret_cast<uint4*>(out + (c + i) * 2) = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        }
      }
      if (!done_whole && r < rows && group == 0) p.part_ml[done_row + r] = make_float2(done_ref, sum);
    };
    // the factor of this thread's row, and in a tree its position, fetched a unit ahead
    int next_pos = 0;
    auto factor_of = [&](const Place& u) {
      if (r >= rows_at(p, u)) return 0.0f;
      if constexpr (P::kTree) next_pos = __ldcg(&p.place[p.row0[u.e] + u.z * kRows + r].x);
      return __ldcg(p.factors + cut_row(p, u) + r);
    };
    bool at_first = true;
    Place w = start;
    float next_factor = !P::kTree && first < last ? factor_of(w) : 0.0f;
    for (int at = first;; next_unit(p, w)) {
      Tiles tiles{};
      Part part{0, 0};
      if (at < last) {
        tiles = tiles_at(p, w);
        part = part_of(work, w, tiles.n, last - at);
      }
      const int n = part.n;
      if (n == 0 && !pending) break;
      if (n == 0) w = start;  // no unit follows: one turn more, for the last one's results alone
      const int k0 = part.begin;
      const bool whole = !P::kTree && n == tiles.n, exists = r < rows_at(p, w);
      int row, pos = 0, len = 0;
      if constexpr (P::kTree) {
        row = k0 == 0 ? p.part0[w.e] + w.h * p.n[w.e] + w.z * kRows : p.wide_cont + work.block * kRows;
      } else {
        const int slot = 2 * work.block + (at == first ? 0 : 1);
        if (n > 0 && n < tiles.n && k0 == 0 && threadIdx.x == 0) tell_cut(p, work, w, at, tiles.n, slot);
        row = slot * kRows;
        len = p.len[w.e];
        pos = len - p.count[w.e] + query_of(p, w.z * kRows + r);
      }
      at += tiles.n + work.cost - w.j;
      const bool causal = P::kTree || p.causal;  // (in a tree a query that sees all has the last position)
      // a row that has seen no key yet has no reference (its weights are all 0)
      bool unset = exists;
      float ref = exists ? 0.0f : 0.5f * kFar, l = 0.0f;  // (rows that do not exist weigh next to nothing)

      int stop = 0, low = 0;  // this row's keys
      float fq = 0.0f;
      auto begin_unit = [&]() {
        if constexpr (P::kTree) pos = next_pos;
        stop = !exists ? 0 : causal ? pos + 1 : len;
        low = p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
        fq = next_factor;
        if (n > 0 && at < last) {
          Place after = w;
          next_unit(p, after);
          next_factor = factor_of(after);
        }
      };
      // A tree's units are short, and all SMs fetch the instructions of their first tile, some
      // 40 KB, at once: several microseconds, which one turn without effect spends while the
      // queries are being cut and the first pages come.
      bool rehearsal = P::kTree && at_first;
      if (!rehearsal) begin_unit();
      int j = 0;
      do {
        const int b = it & 1;
        if (n > 0) {
          if (!rehearsal) await(&scales_in[it % kRing], it / kRing);
          const float* sc = reinterpret_cast<const float*>(&scales[it % kRing]) + group;  // this thread's page
          float f = fminf(fmaxf(fq * sc[0], 2e-38f), 3e38f);  // (above 0: a hidden key's score stays below all)
          const float ev = static_cast<float>(exponent_of(sc[2]));
          const int t0 = tiles.tile(k0 + j) * kTile;
          // whether some row of the unit does not see the whole tile
          const bool masked = t0 + kTile > (causal ? tiles.p_lo + 1 : len) ||
                              (p.window > 0 && t0 <= tiles.p_hi - p.window && t0 + kTile > p.sinks);
          const uint32_t t_s = tmem + lanes + b * 128 + group * 64;
          if (!rehearsal) await(&s_full[b], it / 2);
          tc_after();
          // keys that this thread's row sees, of its 64
          unsigned long long see = ~0ull;
          if (masked) {
            const int tb = t0 + group * 64;
            auto below = [&](int x) { return x <= tb ? 0ull : x - tb >= 64 ? ~0ull : (1ull << (x - tb)) - 1; };  // keys before x
            see = below(stop) & (~below(low) | below(p.sinks));
          }
          float s[64], m0, m1;
          tmem_ld<32>(t_s, s);
          tmem_ld<32>(t_s + 32, s + 32);
          ld_wait();
          if (masked) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (!(static_cast<uint32_t>(see >> (i & 32)) & 1u << (i & 31))) s[i] = kNothing;
          }
          m0 = s[0], m1 = s[32];
#pragma unroll
          for (int i = 1; i < 31; i += 2) {
            m0 = fmaxf(fmaxf(m0, s[i]), s[i + 1]);
            m1 = fmaxf(fmaxf(m1, s[32 + i]), s[33 + i]);
          }
          m0 = __fmul_rn(fmaxf(m0, s[31]), f);
          m1 = __fmul_rn(fmaxf(m1, s[63]), f);
          float top = fmaxf(m0, m1) + ev;
          int far = top - ref > kAhead || (unset && top > kUnset) || rehearsal;
          asm volatile("{\n.reg .pred a, b;\nsetp.ne.s32 a, %0, 0;\nbarrier.cta.red.or.pred b, %1, 64, a;\nselp.s32 %0, 1, 0, b;\n}"
                       : "+r"(far)
                       : "r"(1 + quad)
                       : "memory");
          float change = 1.0f;
          if (far) {
            // some row of the quad passed its reference: move such rows' references
            // to their maxima
            xch[group * kRows + r] = top;
            named_bar(1 + quad, 64);
            top = fmaxf(top, xch[(group ^ 1) * kRows + r]);
            named_bar(1 + quad, 64);
            if (top - ref > kAhead || (unset && top > kUnset)) {
              if (!unset) change = ex2_approx(ref - top);  // (else there is nothing yet)
              ref = top;
              unset = false;
            }
            l *= change;
          }
          // the blocks' scales, 2^(above - kPlace), down to the least that a byte holds
          const float real0 = m0 + ev - ref, real1 = m1 + ev - ref;
          const float above0 = fmaxf(ceilf(real0), kUnset), above1 = fmaxf(ceilf(real1), kUnset);  // (kUnset: no key is seen)
          float shift0 = kPlace - above0 + (ev - ref), shift1 = kPlace - above1 + (ev - ref);
          if (fmaxf(fmaxf(m0 > kNothing ? fabsf(m0) : 0.0f, m1 > kNothing ? fabsf(m1) : 0.0f), fabsf(ref)) >= kFar) {
            // sums with scores this large are off by 2^-9 and more: differences from
            // the block's maximum first, which are exact near it
            m0 = fmaxf(m0, kUnset);
            m1 = fmaxf(m1, kUnset);
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = __fsub_rn(__fmul_rn(s[i], f), i < 32 ? m0 : m1);
            f = 1.0f;
            shift0 = kPlace + (real0 - above0);
            shift1 = kPlace + (real1 - above1);
          }
          __syncwarp();
          const int least = 127 - static_cast<int>(kPlace);
          const int scale0 = static_cast<int>(fminf(fmaxf(above0, static_cast<float>(-least)), kAhead)) + least;
          const int scale1 = static_cast<int>(fminf(fmaxf(above1, static_cast<float>(-least)), kAhead)) + least;
          if (!rehearsal) *reinterpret_cast<uint16_t*>(smem + kScales + b * kScaleBytes + scale_at(r, 2 * group)) = static_cast<uint16_t>(scale0 | scale1 << 8);
          // the weights; as fp16 pairs (11 bits), cut into two parts of 4 bits, over
          // the scores that this thread has read
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float shift = x ? shift1 : shift0;
            float s0 = 0.0f, s1 = 0.0f;
            uint32_t hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t ha, hb;
              {
                const int c = 32 * x + 4 * i;
                const float w0 = ex2_approx(fmaf(s[c], f, shift)), w1 = ex2_approx(fmaf(s[c + 1], f, shift));
                const float w2 = ex2_approx(fmaf(s[c + 2], f, shift)), w3 = ex2_approx(fmaf(s[c + 3], f, shift));
                if constexpr (!P::kTree) {
                  s0 += w0;
                  s1 += w1;
                  s0 += w2;
                  s1 += w3;
                }
                ha = f16x2(w0, w1);
                hb = f16x2(w2, w3);
              }
              const uint32_t a = e4m3x2_of_f16x2(ha), d = e4m3x2_of_f16x2(hb);
              hi[i] = a | d << 16;
              if constexpr (P::kTree) {
                const uint32_t a16 = e4m3x2_to_f16x2(a), d16 = e4m3x2_to_f16x2(d);
                const uint32_t a_lo = e4m3x2_of_f16x2(sub_f16x2(ha, a16)), d_lo = e4m3x2_of_f16x2(sub_f16x2(hb, d16));
                lo[i] = a_lo | d_lo << 16;
                // summed as they are held: multiples of the last place of their fp16 form, so exact there
                add_to(s0, s1, add_f16x2(a16, e4m3x2_to_f16x2(a_lo)));
                add_to(s0, s1, add_f16x2(d16, e4m3x2_to_f16x2(d_lo)));
              } else {
                lo[i] = e4m3x2_of_f16x2(sub_f16x2(ha, e4m3x2_to_f16x2(a))) | e4m3x2_of_f16x2(sub_f16x2(hb, e4m3x2_to_f16x2(d))) << 16;
              }
            }
            if (!rehearsal) {
              tmem_st<8>(t_s + 8 * x, reinterpret_cast<const float*>(hi));
              tmem_st<8>(t_s + 16 + 8 * x, reinterpret_cast<const float*>(lo));
            }
            l = fmaf(s0 + s1, ex2_approx((x ? above1 : above0) - ev - kPlace), l);
          }
          if (P::kTree && rehearsal) {
            rehearsal = at_first = false;
            wait_only();  // for the cut queries' factors and positions
            next_factor = factor_of(w);
            begin_unit();
            unset = exists;
            ref = exists ? 0.0f : 0.5f * kFar;
            l = 0.0f;
            j = -1;
            continue;
          }
          if (far && j > 0) {
            // what was summed with the old references, this thread's half of the
            // row; last, so that the product with the tile before, which has to end
            // first, ran under the work on the weights
            await(&o_done[b ^ 1], (it - 1) / 2);
            tc_after();
            constexpr int kStep = P::kTree ? 16 : 64;
#pragma unroll 1
            for (int c = 0; c < 128; c += kStep) {
              float o[kStep];
#pragma unroll
              for (int i = 0; i < kStep; i += 16) tmem_ld<16>(t_o + lanes + group * 128 + c + i, o + i);
              ld_wait();
#pragma unroll
              for (int i = 0; i < kStep; ++i) o[i] *= change;
#pragma unroll
              for (int i = 0; i < kStep; i += 16) tmem_st<16>(t_o + lanes + group * 128 + c + i, o + i);
            }
          }
          st_wait();
          proxy_fence();
        }
        if (j == 0 && pending) store_results(it - 1);
        if (n > 0) {
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_ready[b]);
          ++it;
        }
      } while (++j < n);
      if (n == 0) break;
      pending = true;
      done = w;
      done_whole = whole;
      done_row = row;
      done_l = l;
      done_ref = unset ? kUnset : ref;
    }
  } else {
    setmaxnreg_dec<kRestRegs>();
    if (warp == kLoader) {
      uint64_t policy;  // other row tiles read the same pages
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      Loader<kSlots, true, P>{p, work, smem, full, empty, scales, scales_in, wait}.run(start, first, last, policy);
    } else if (warp == kIssuer) {
      // ---------------------------------------------------------------- products
      constexpr uint32_t kS = shape(128, kTile, false, false);
      int used = 0;
      bool ok = true;
      // descriptors count in 16 bytes: those of other pieces are sums
      const uint64_t queries = operand(sbase + kQ), at_slot = operand(sbase), at_values = operand(sbase, kHalfBytes);
      // the scores run two tiles ahead, over the segments' ends
      Place ws = start;
      int at_s = first, left = 0, tile = 0, segment = 0;
      auto scores = [&]() {  // S of the next tile, if there is one
        if (left == 0) {
          if (at_s >= last) return;
          const int tiles = tiles_at(p, ws).n;
          left = part_of(work, ws, tiles, last - at_s).n;
          at_s += tiles + work.cost - ws.j;
          next_unit(p, ws);
          if (left == 0) return;
          ok = wait.together(q_ready, segment++, kLostMma);
        }
        const int b = tile++ & 1, s = used % kSlots;
        ok = ok && wait.together(&full[s], used / kSlots, kLostMma);
        if (!ok) return;
        tc_after();
        const uint64_t keys = at_slot + s * (kSlotBytes >> 4);
#pragma unroll P::kTree ? kMu : 16
        for (int k = 0; k < 16; ++k)  // high parts, low parts; halves of the dims; 32 dims at a time
          mma_e4m3(tmem + b * 128, queries + (((k >> 2) * kHalfBytes + (k & 3) * 32) >> 4),
                   keys + ((((k >> 2) & 1) * kHalfBytes + (k & 3) * 32) >> 4), kS, k > 0);
        mma_commit(&s_full[b]);
        mma_commit(&empty[s]);
        if (--left == 0) mma_commit(q_free);
        ++used;
      };
      Place w = start;
      int at = first, n = 0, j = 0;
      for (int it = -2; ok; ++it) {
        if (it >= 0) {
          if (j == n) {  // the next segment
            if (at >= last) break;
            const int tiles = tiles_at(p, w).n;
            n = part_of(work, w, tiles, last - at).n;
            at += tiles + work.cost - w.j;
            next_unit(p, w);
            if (n == 0) break;
            j = 0;
          }
          const int b = it & 1, s = used % kSlots;
          ok = wait.together(&p_ready[b], it / 2, kLostMma) && wait.together(&full[s], used / kSlots, kLostMma);
          if (!ok) break;
          tc_after();
          // The weights' scales (a copy of 75 cycles, which the products wait for) and
          // the values'.  Told to this warp by a barrier of their own and copied before
          // the weights are there: 756 against 741 us for the chunk below, as the row
          // threads then stop once more; before the scores ahead: 790.
          const uint32_t weights = tmem + b * 128;
          copy_scales(weights + kWeightScales, sbase + kScales + b * kScaleBytes);
          copy_scales(weights + kOnes, sbase + kScales + 2 * kScaleBytes);
          copy_scales(weights + kOnes + 4, sbase + kScales + 2 * kScaleBytes);
#pragma unroll P::kTree ? kMu : 8
          for (int k = 0; k < 8; ++k)  // 32 keys at a time, their high and low parts in turn
            mma_scaled_tmem(t_o, weights + (k >> 2) * 64 + ((k >> 1) & 1) * 8 + (k & 1) * 16,
                            at_values + ((s * kSlotBytes + (k >> 1) * 32 * 128) >> 4),
                            shape_scaled(128, kHeadDim, false, true, k >> 1, 0), weights + kWeightScales, weights + kOnes, j > 0 || k > 0);
          mma_commit(&o_done[b]);
          mma_commit(&empty[s]);
          ++used;
          ++j;
        }
        scores();  // runs behind O of this tile, whose weights it overwrites
      }
      if (!ok) {  // given up: what is in flight ends before the tensor memory goes
        mma_commit(drained);
        wait.drain(drained, 0);
      }
    } else if (warp == kAsker && lane == 0) {
      // ---------------------------------------------------------------- queries to shared memory
      if constexpr (P::kTree) wait_only();
      int segment = 0;
      Place w = start;
      for (int at = first; at < last; ++segment, next_unit(p, w)) {
        const int tiles = tiles_at(p, w).n, n = part_of(work, w, tiles, last - at).n;
        at += tiles + work.cost - w.j;
        if (n == 0 || (segment > 0 && !wait(q_free, segment - 1, kLostLoad))) break;
        mbar_arrive_expect_tx(q_ready, 4 * kHalfBytes);
        const int y = cut_row(p, w);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // high parts, low parts; halves of the dims (rows behind the unit's are others', or zeros)
          tensor2d_g2s(smem + kQ + k * kHalfBytes, &p.q_map, 128 * (k & 1), y + (k >> 1) * q_rows, q_ready, policy_evict_first());
      }
      if (segment > 0) wait.drain(q_ready, segment - 1);  // no copy left in flight
    }
  }
  __syncthreads();
  if (warp == kIssuer) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace rows
}  // namespace paged
}  // namespace iq
