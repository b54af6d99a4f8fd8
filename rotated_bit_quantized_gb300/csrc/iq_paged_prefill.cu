// libiqkv: attention of many query rows per kv head (prompts and their chunks)
// over the paged 8-bit cache.
//
// The same mathematics as the split kernel (iq_paged_attend.cu) with the query
// rows as the products' M dimension: S = Q.K^T with Q as two e4m3 parts summed
// into one accumulator, S (128 rows x 128 keys) twice in tensor memory, and
// O += W.V with the weights W = 2^(s + ev - ref) as two e4m3 parts that the
// row threads write over the scores they came from.  Keys and values are the
// pages' codes as they lie in HBM.  Each product runs twice (high and low
// part) at e4m3's rate, twice bf16's, so the bound is bf16's rate; no code is
// ever converted.
//
// Rounding.  A weight's two parts leave at most 2^-8 of it, and 2^-10 below
// e4m3's range: a row's reference puts its running maximum at 2^5 and moves
// when a weight would pass 2^8.75 (448 is the largest code), so that floor is
// 2^-15 of the largest weight or less.
#include <cuda_runtime.h>

#include "iq_paged_mma.cuh"

namespace iq {
namespace paged {
namespace {

constexpr int kRows = 128;
constexpr int kSlots = 5;                         // tiles of keys or values in flight
constexpr int kQ = kSlots * kSlotBytes;           // [high, low][2 halves of the dims][128 rows][128 bytes]
constexpr int kMisc = kQ + 4 * kHalfBytes;
constexpr int kSmem = 1024 + kMisc + 3 * kRows * 4 + 32 * 8;
constexpr int kThreads = 320;
constexpr int kLoader = 8, kIssuer = 9;
constexpr float kPlace = 5.0f, kTop = 8.75f;      // the running maximum's place, and how far a weight may grow
constexpr float kUnset = -1e30f, kDead = 1e30f;
static_assert(kSmem <= 232448, "shared memory of one CTA");

__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_of_f16x2(uint32_t h2) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(h2));
  return d;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One persistent CTA per SM.  Warps 0-7: two threads per query row (warp w
// reaches tensor-memory lanes 32 (w % 4) ..), each with the 64 keys of one
// page of a tile; warps w and w + 4 hold the same rows and settle the rows'
// references between themselves.  Then one warp streams the pages and one
// issues the products, S of the next tile but one behind O of this tile.
__global__ void __launch_bounds__(kThreads, 1) paged_prefill_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  float* factor = reinterpret_cast<float*>(smem + kMisc);  // [128] 2^eq * scale * log2 e
  float* xch = factor + kRows;                             // [2][128] what the two threads of a row exchange
  uint64_t* full = reinterpret_cast<uint64_t*>(xch + 2 * kRows);
  uint64_t* empty = full + kSlots;
  uint64_t* s_full = empty + kSlots;   // [2] scores of a tile in tensor memory
  uint64_t* p_ready = s_full + 2;      // [2] weights of a tile in their place
  uint64_t* o_done = p_ready + 2;      // [2] and multiplied with its values
  uint64_t* q_ready = o_done + 2;
  uint64_t* drained = q_ready + 1;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tslot + 1);
  static_assert(2 * kSlots + 8 < 31, "the barriers and the two words behind them fit");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_ready[s], 8);
      mbar_init(&o_done[s], 1);
    }
    mbar_init(q_ready, 8);
    mbar_init(drained, 1);
    *abort = 0;
    mbar_fence_init();
  }
  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tslot, t_o = tmem + 256;  // S or W: 0..127, 128..255; O: 256..511
  const Waits wait{abort, p.status};

  const int first = range_begin(blockIdx.x, gridDim.x, p.total), last = range_begin(blockIdx.x + 1, gridDim.x, p.total);
  const Place start = place_of(p, first);

  if (warp == kLoader) {
    // ---------------------------------------------------------------- pages to shared memory
    uint64_t pol;  // other row tiles read the same pages
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    int issued = 0;
    bool ok = true;
    Place w = start;
    for (int at = first; at < last && ok; next_unit(p, w)) {
      const int e = w.e, h = w.h, k0 = w.j;
      const Tiles tiles = tiles_at(p, w);
      const int n = min(tiles.n - k0, last - at);
      const int* row = p.table + static_cast<long long>(p.slot[e]) * p.max_pages;
      const int end_page = (p.len[e] + kPage - 1) / kPage - 1;
      // lanes fetch the ids of 16 tiles' pages at a time, one such piece ahead
      auto fetch = [&](int j) { return __ldcg(row + min(2 * tiles.tile(k0 + min(j + (lane >> 1), n - 1)) + (lane & 1), end_page)); };
      auto load = [&](const CUtensorMap* map, int id0, int id1) {
        const int s = issued % kSlots;
        if (issued >= kSlots) ok = __all_sync(0xFFFFFFFFu, wait(&empty[s], issued / kSlots - 1, kLostLoad));
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&full[s], kSlotBytes);
          uint8_t* to = smem + s * kSlotBytes;
          const int y0 = (id0 * p.heads + h) * kPage, y1 = (id1 * p.heads + h) * kPage;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tensor2d_g2s(to + half * kHalfBytes, map, 128 * half, y0, &full[s], pol);
            tensor2d_g2s(to + half * kHalfBytes + kHalfBytes / 2, map, 128 * half, y1, &full[s], pol);
          }
        }
        if (ok) ++issued;
        __syncwarp();
      };
      int ids = fetch(0), next = fetch(16), v0 = 0, v1 = 0;
      for (int j = 0; j <= n && ok; ++j) {  // in the order of the products: K0, K1, V0, K2, V1, ...
        int k0id = 0, k1id = 0;
        if (j < n) {
          if (j % 16 == 0) {
            if (j) {
              ids = next;
              next = fetch(j + 16);
            }
            ids = page_in_pool(ids, p.pages, p.status);
          }
          k0id = __shfl_sync(0xFFFFFFFFu, ids, 2 * (j % 16));
          k1id = __shfl_sync(0xFFFFFFFFu, ids, 2 * (j % 16) + 1);
          load(&p.k_map, k0id, k1id);
        }
        if (j > 0 && ok) load(&p.v_map, v0, v1);
        v0 = k0id;
        v1 = k1id;
      }
      at += n;
    }
    if (lane == 0)  // no copy left in flight
      for (int s = 0; s < kSlots && s < issued; ++s) wait.drain(&full[s], (issued - 1 - s) / kSlots);
  } else if (warp == kIssuer) {
    // ---------------------------------------------------------------- products
    if (lane == 0) {
      constexpr uint32_t kS = shape(128, kTile, false, false), kO = shape(128, kHeadDim, false, true);
      int it = 0, used = 0, segment = 0;
      bool ok = true;
      auto scores = [&](int j) {  // S of the segment's tile j
        const int b = (it + j) & 1, s = used % kSlots;
        ok = wait(&full[s], used / kSlots, kLostMma);
        if (!ok) return;
        tc_after();
#pragma unroll
        for (int k = 0; k < 16; ++k)  // high parts, low parts; halves of the dims; 32 dims at a time
          mma_e4m3(tmem + b * 128, operand(sbase + kQ + (k >> 2) * kHalfBytes + (k & 3) * 32),
                   operand(sbase + s * kSlotBytes + ((k >> 2) & 1) * kHalfBytes + (k & 3) * 32), kS, k > 0);
        mma_commit(&s_full[b]);
        mma_commit(&empty[s]);
        ++used;
      };
      Place w = start;
      for (int at = first; at < last && ok; ++segment, next_unit(p, w)) {
        const int n = min(tiles_at(p, w).n - w.j, last - at);
        ok = wait(q_ready, segment, kLostMma);
        if (ok) scores(0);
        if (ok && n > 1) scores(1);
        for (int j = 0; j < n && ok; ++j) {
          const int b = (it + j) & 1, s = used % kSlots;
          ok = wait(&p_ready[b], (it + j) / 2, kLostMma) && wait(&full[s], used / kSlots, kLostMma);
          if (!ok) break;
          tc_after();
#pragma unroll
          for (int k = 0; k < 8; ++k)  // high and low parts in turn, 32 keys at a time (so that one read of V may serve both)
            mma_tmem_a(t_o, tmem + b * 128 + (k >> 2) * 64 + ((k >> 1) & 1) * 8 + (k & 1) * 16,
                       operand(sbase + s * kSlotBytes + (k >> 1) * 32 * 128, kHalfBytes), kO, j > 0 || k > 0);
          mma_commit(&o_done[b]);
          mma_commit(&empty[s]);
          ++used;
          if (j + 2 < n) scores(j + 2);  // runs behind O of this tile, whose weights it overwrites
        }
        it += n;
        at += n;
      }
      if (!ok) {  // given up: what is in flight ends before the tensor memory goes
        mma_commit(drained);
        wait.drain(drained, 0);
      }
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax: half a row per thread
    const int group = warp >> 2, quad = warp & 3, r = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    int it = 0;
    bool ok = true;
    auto await = [&](uint64_t* bar, uint32_t phase) {  // a lost wait changes no path: every barrier below is still reached
      if (ok) ok = wait(bar, phase, kLostRows);
      __syncwarp();
    };
    // a unit's queries into the operand buffer, 16 of the quad's 32 rows per warp
    auto put_queries = [&](const Place& w) {
      const int rows = min(kRows, p.count[w.e] * p.rep - w.z * kRows);
#pragma unroll 1
      for (int i = 0; i < 16; i += 8) {
        uint4 raw[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int x = quad * 32 + group * 16 + i + k;
          raw[k] = make_uint4(0, 0, 0, 0);
          if (x < rows) raw[k] = __ldcg(reinterpret_cast<const uint4*>(p.q + row_index(p, w, w.z * kRows + x) * kHeadDim) + lane);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int x = quad * 32 + group * 16 + i + k;
          uint2 hi, lo;
          const float f = split_query<1>(raw[k], hi, lo);
          uint8_t* to = smem + kQ + (lane >> 4) * kHalfBytes + swizzled(x, (lane & 15) * 8);
          *reinterpret_cast<uint2*>(to) = hi;
          *reinterpret_cast<uint2*>(to + 2 * kHalfBytes) = lo;
          if (lane == 0) factor[x] = clamp_finite(f * (p.scale * kLog2e));
        }
      }
      proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
      named_bar(1 + quad, 64);  // the quad's factors
    };
    Place w = start;
    put_queries(w);
    for (int at = first; at < last;) {
      const Tiles tiles = tiles_at(p, w);
      const int e = w.e, k0 = w.j, n = min(tiles.n - k0, last - at), len = p.len[e];
      const bool whole = n == tiles.n, exists = w.z * kRows + r < p.count[e] * p.rep;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (at == first ? 0 : 1);
      const float fq = factor[r];
      const int x = len - p.count[e] + (w.z * kRows + r) / p.rep;  // the row's position
      const int stop = !exists ? 0 : p.causal ? x + 1 : len;
      const int low = p.window > 0 && x >= p.window ? x - p.window + 1 : 0;
      float ref = exists ? kUnset : kDead, l = 0.0f;

      const int* row = p.table + static_cast<long long>(p.slot[e]) * p.max_pages;
      const int end_page = (len + kPage - 1) / kPage - 1;
      // this thread's page of tile j: ids two tiles ahead, scales one
      auto id_of = [&](int j) { return __ldcg(row + min(2 * tiles.tile(k0 + min(j, n - 1)) + group, end_page)); };
      auto scales_of = [&](int id) {
        const long long i = static_cast<long long>(page_in_pool(id, p.pages, p.status)) * p.heads + w.h;
        return make_float2(__ldcg(p.k_scales + i), __ldcg(p.v_scales + i));
      };
      int id = id_of(1);
      float2 sc = scales_of(id_of(0));
      for (int j = 0; j < n; ++j, ++it) {
        const int b = it & 1;
        const float f = clamp_finite(fq * sc.x);
        const int ev = exponent_of(sc.y);
        sc = scales_of(id);
        id = id_of(j + 2);
        const int t0 = tiles.tile(k0 + j) * kTile, tb = t0 + group * 64;  // the tile's, this thread's first key
        // whether some row of the unit does not see the whole tile
        const bool masked = t0 + kTile > (p.causal ? tiles.p_lo + 1 : len) ||
                            (p.window > 0 && t0 <= tiles.p_hi - p.window && t0 + kTile > p.sinks);
        const uint32_t t_s = tmem + lanes + b * 128 + group * 64;
        await(&s_full[b], it / 2);
        tc_after();
        uint32_t h[32];  // the weights as fp16 pairs: 11 bits, to be cut into two parts of 4
        float sum;
        auto weights = [&]() {  // returns the largest exponent, for the references, only where asked: see below
          const float shift = static_cast<float>(ev) - ref;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float s[32];
            tmem_ld<32>(t_s + c, s);
            ld_wait();
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int t = tb + c + i;
                if (!(t < stop && (t >= low || t < p.sinks))) s[i] = -__builtin_huge_valf();
                else s[i] = fmaf(s[i], f, shift);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) s[i] = fmaf(s[i], f, shift);
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float a = ex2_approx(s[i]), d = ex2_approx(s[i + 1]);
              s0 += a;
              s1 += d;
              h[(c + i) / 2] = f16x2(a, d);
            }
          }
          sum = s0 + s1;
          uint32_t m = h[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) m = max_f16x2(m, h[i]);
          const float2 mm = f16x2_to_f32(m);
          return fmaxf(mm.x, mm.y);
        };
        int far = weights() > 430.0f;  // 2^8.75: e4m3 ends at 448
        asm volatile("{\n.reg .pred a, b;\nsetp.ne.s32 a, %0, 0;\nbarrier.cta.red.or.pred b, %1, 64, a;\nselp.s32 %0, 1, 0, b;\n}"
                     : "+r"(far)
                     : "r"(1 + quad)
                     : "memory");
        if (far) {
          // some row of the quad passed its reference: the rows' maxima in log2
          // units, the references moved so that they land at 2^kPlace, and what
          // was summed with the old ones
          float m = -__builtin_huge_valf();
#pragma unroll
          for (int c = 0; c < 64; c += 32) {
            float s[32];
            tmem_ld<32>(t_s + c, s);
            ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int t = tb + c + i;
              if (t < stop && (t >= low || t < p.sinks)) m = fmaxf(m, fmaf(s[i], f, static_cast<float>(ev)));
            }
          }
          xch[group * kRows + r] = m;
          named_bar(1 + quad, 64);
          m = fmaxf(m, xch[(group ^ 1) * kRows + r]);
          named_bar(1 + quad, 64);
          float change = 1.0f;
          if (m - ref > kTop - 0.01f) {
            change = ex2_approx(ref - (m - kPlace));
            ref = m - kPlace;
            l *= change;
          }
          if (j > 0) {  // this thread's half of the row's results
            await(&o_done[b ^ 1], (it - 1) / 2);
            tc_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              float o[16];
              tmem_ld<16>(t_o + lanes + group * 128 + c, o);
              ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= change;
              tmem_st<16>(t_o + lanes + group * 128 + c, o);
            }
            st_wait();
          }
          weights();
        }
        l = fmaf(sum, power2(-ev), l);
        // the two parts, over the scores that this thread has read
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t a = e4m3x2_of_f16x2(h[2 * i]), d = e4m3x2_of_f16x2(h[2 * i + 1]);
          hi[i] = a | d << 16;
          lo[i] = e4m3x2_of_f16x2(sub_f16x2(h[2 * i], e4m3x2_to_f16x2(a))) |
                  e4m3x2_of_f16x2(sub_f16x2(h[2 * i + 1], e4m3x2_to_f16x2(d))) << 16;
        }
        tmem_st<16>(t_s, reinterpret_cast<const float*>(hi));
        tmem_st<16>(t_s + 16, reinterpret_cast<const float*>(lo));
        st_wait();
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[b]);
      }
      at += n;
      // the next unit's queries, while the last product runs (its scores are done with these)
      Place next = w;
      next_unit(p, next);
      if (at < last) put_queries(next);
      // ---- the results: the sums of a row's two halves, half of its dims per thread
      xch[group * kRows + r] = l;
      named_bar(1 + quad, 64);
      const float total = l + xch[(group ^ 1) * kRows + r];
      named_bar(1 + quad, 64);
      await(&o_done[(it - 1) & 1], (it - 1) / 2);
      tc_after();
      const float inv = total == 0.0f ? 0.0f : 1.0f / total;
      const long long to = whole ? row_index(p, w, w.z * kRows + r) * kHeadDim + group * 128
                                 : (static_cast<long long>(slot) * kRows + r) * kHeadDim + group * 128;
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        float o[16];
        tmem_ld<16>(t_o + lanes + group * 128 + c, o);
        ld_wait();
        if (exists) {
          const float(&o0)[8] = *reinterpret_cast<const float(*)[8]>(o);
          const float(&o1)[8] = *reinterpret_cast<const float(*)[8]>(o + 8);
          if (whole) {
            store_out8(p.out, p.out_f32, to + c, o0, inv);
            store_out8(p.out, p.out_f32, to + c + 8, o1, inv);
          } else {
            store_out8(p.part_o, 1, to + c, o0, 1.0f);
            store_out8(p.part_o, 1, to + c + 8, o1, 1.0f);
          }
        }
      }
      if (!whole && exists && group == 0) p.part_ml[slot * kRows + r] = make_float2(ref, total);
      tc_before();
      w = next;
    }
  }
  __syncthreads();
  if (warp == kIssuer) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace

cudaError_t launch_prefill(const AttendParams& p, int grid, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(paged_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  return e == cudaSuccess ? launch_after<AttendParams>(paged_prefill_kernel, dim3(grid), kThreads, kSmem, stream, p) : e;
}

}  // namespace paged
}  // namespace iq
