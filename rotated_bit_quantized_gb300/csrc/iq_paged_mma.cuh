// tcgen05 pieces shared by the paged cache's attention kernels: e4m3 operands
// in 128-byte-swizzled shared memory, fp32 accumulators in tensor memory, and
// waits that end.
#pragma once

#include <cuda.h>

#include "iq_paged.cuh"

namespace iq {
namespace paged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNothing = -__builtin_huge_valf();      // the score of a key that a row does not see
constexpr float kAhead = 40.0f;  // how far, in binades, a row's weights may pass its reference before that moves
constexpr float kUnset = -3e38f, kDead = 3e38f;         // a row's reference before its first key, and of rows that do not exist
constexpr int kTile = 128;                    // keys per tile: two pages
constexpr int kHalfBytes = kTile * 128;       // 128 rows of half a head's dims
constexpr int kSlotBytes = 2 * kHalfBytes;    // a tile of keys or of values in shared memory

// The tensor map of a code pool: rows of 256 bytes, boxes of one page of one
// kv head by half of the dims (64 x 128 bytes, 128-byte swizzle).
bool code_map(CUtensorMap* map, const uint8_t* codes, long long rows, int box_rows = kPage);

// ------------------------------------------------------------------ work

// The arguments of an attention launch.  A unit is (entry, kv head, tile of
// unit_rows query rows); row r of an entry and kv head is query r / rep of head
// r % rep.  The key tiles of all units, laid end to end, are cut into gridDim
// ranges of equal length, one for each CTA; a unit that lies in one range is
// stored at once, the others leave a partial result per range.
// A unit that lies in several ranges, told by the range that holds its first
// tile: the slots of the partial results are `slot` and, for the ranges behind,
// 2 g.  last < 0: the range's end cuts no unit that begins in it.
struct Cut {
  int last, slot, e, h, z, pad[3];
};
struct AttendBase {
  CUtensorMap k_map, v_map, q_map;  // (q_map: the prefill kernel's queries, cut beforehand)
  const float* k_scales;
  const float* v_scales;
  const int* table;
  unsigned* status;
  const uint16_t* q;
  void* out;
  float* part_o;    // rows of 256 unnormalised partial results
  float2* part_ml;  // their references and sums
  uint8_t* cut;     // prefill: [high, low parts][entry][kv head][row][256] e4m3
  float* factors;   // prefill: [entry][kv head][row] 2^e * scale * log2 e
  int out_f32, heads, rep, nq, pages, max_pages, causal, window, sinks;
  int stall;                    // test hook (iq_paged_debug_stall): no page is loaded, so the waits for them run out
  float scale;
};
struct AttendParams : AttendBase {
  static constexpr bool kTree = false;
  // part_o, part_ml: [2 * grid][unit_rows], a range's first segment, its last
  Cut* cuts;        // [grid] the unit that a range's end cuts
  int unit_rows, entries, cost, total, slots_n;
  unsigned rep_mul, rep_shift;  // division by rep, see query_of
  // per entry that has queries and keys: its place in the call, its slot, what the slot holds,
  // its queries; cum: slots before it (all heads), per: slots of one of its heads
  short entry[IQ_MAX_BATCH], slot[IQ_MAX_BATCH];
  int len[IQ_MAX_BATCH], count[IQ_MAX_BATCH], cum[IQ_MAX_BATCH + 1], per[IQ_MAX_BATCH];
};

// The key tiles of a unit: those of the sinks, then those of the window up to
// its last row's position.  A unit that sees no key keeps one tile, all masked.
struct Tiles {
  int sinks, skip, n;  // tiles of the sinks; tiles between them and the window; all
  int p_lo, p_hi;      // the least and the largest position of a row
  int base;            // the tile before which nothing is of the unit's
  __host__ __device__ int tile(int j) const { return base + (j < sinks ? j : j + skip); }
};
__host__ __device__ inline Tiles tiles_of(int len, int first_pos, int last_pos, int causal, int window, int sinks) {
  Tiles t;
  t.p_lo = first_pos;
  t.p_hi = last_pos;
  const int stop = !causal ? len : t.p_hi < 0 ? 1 : t.p_hi + 1;
  const int low = window > 0 && t.p_lo >= window ? t.p_lo - window + 1 : 0;  // where the first row's window begins
  const int begin = low / kTile, reach = sinks < low ? sinks : low, n = (reach + kTile - 1) / kTile;
  t.sinks = n < begin ? n : begin;
  t.skip = n < begin ? begin - n : 0;
  t.n = (stop + kTile - 1) / kTile - t.skip;
  t.base = 0;
  return t;
}

// The first slot of a range, and the range of a slot.
__host__ __device__ inline int range_begin(int g, int grid, int total) {
  return static_cast<int>(static_cast<long long>(g) * total / grid);
}
__host__ __device__ inline int range_of(int tile, int grid, int total) {
  return static_cast<int>((static_cast<long long>(tile + 1) * grid - 1) / total);
}

// What the CTAs of a launch, or some of them, share: `count` entries from `first` on,
// whose slots are cut into `grid` ranges; this CTA's is number `block`.
struct Work {
  int first, count, cost, total, block, grid;
};

// A place in the slots of all units: entry, head, row tile, slot j of the unit.
struct Place {
  int e, h, z, j;
};
// The attention of slots that share pages.  The pages that a group of slots has in
// common, and others have not, are a node of a tree; its leaves are what a slot holds
// alone.  A node's rows are those of all its slots, which lie side by side in the cut
// queries, and its units are (node, kv head, 128 of these rows).  Every unit leaves
// partial results, at its rows' place, and in ranges behind its first in these ranges';
// those of the nodes that a slot is under are joined.
// Leaves of few rows are units of the split kernel's shape: one launch holds CTAs of
// both kinds, `wide` ranges of the nodes before `leaves`, and `narrow` of those from there on.
constexpr int kInner = 64, kNodes = IQ_MAX_BATCH + kInner, kDepth = 4;  // inner nodes of a call, all; nodes above one another
constexpr int kUnitRows = 128;
struct TreeParams : AttendBase {
  static constexpr bool kTree = true;
  int rows;                       // of one kv head
  int nodes, leaves, wide, narrow, wide_cost, narrow_cost, wide_total, narrow_total;
  int wide_cont, narrow_cont, narrow_rows;  // where the ranges' partial results begin; rows of a narrow range's
  unsigned rep_mul, rep_shift;    // division by rep, see query_of
  const int2* place;              // [rows] a row's position, its place in q and out for kv head 0
  short slot[kNodes];             // that holds the node's pages
  short parent[kNodes];           // < 0: none
  short entry[kNodes];            // of a leaf: its place in the call
  int end_page[kNodes];           // the slot's last page
  int row0[kNodes], n[kNodes], part0[kNodes];  // its first row, how many, their place in the partial results
  int cum[kNodes];                // slots before it, of its kind
  int tiles[kNodes], base[kNodes], sink_tiles[kNodes], skip[kNodes], p_lo[kNodes], p_hi[kNodes];  // of its units, see Tiles
};

// The tiles of a unit that a range takes from slot w.j on, `left` slots of the
// range being left: [begin, begin + n), none where it ends in the unit's empty slots.
struct Part {
  int begin, n;
};
__device__ __forceinline__ Part part_of(const Work& work, const Place& w, int tiles, int left) {
  const int begin = max(w.j - work.cost, 0), end = min(max(w.j + left - work.cost, 0), tiles);
  return {begin, end - begin};
}
// floor(r / rep) for r < 2^31: a shift where rep is a power of two; else, with s =
// floor(log2 rep) and mul = ceil(2^(32+s) / rep) < 2^32, umulhi(r, mul) >> s (its
// error is below r / 2^(32+s) < 1 / rep).
template <class P>
__device__ __forceinline__ int query_of(const P& p, int r) {
  return static_cast<int>((p.rep_mul ? __umulhi(static_cast<unsigned>(r), p.rep_mul) : static_cast<unsigned>(r)) >> p.rep_shift);
}
__device__ __forceinline__ Tiles tiles_at(const AttendParams& p, const Place& w) {
  const int rows = p.count[w.e] * p.rep, r0 = w.z * p.unit_rows, before = p.len[w.e] - p.count[w.e];
  return tiles_of(p.len[w.e], before + query_of(p, r0), before + query_of(p, min(r0 + p.unit_rows, rows) - 1), p.causal, p.window,
                  p.sinks);
}
__device__ __forceinline__ Tiles tiles_at(const TreeParams& p, const Place& w) {
  return {p.sink_tiles[w.e], p.skip[w.e], p.tiles[w.e], p.p_lo[w.e], p.p_hi[w.e], p.base[w.e]};
}
__device__ __forceinline__ int rows_at(const AttendParams& p, const Place& w) { return p.count[w.e] * p.rep - w.z * p.unit_rows; }
__device__ __forceinline__ int rows_at(const TreeParams& p, const Place& w) { return p.n[w.e] - w.z * kUnitRows; }
__device__ __forceinline__ int last_page(const AttendParams& p, int e) { return (p.len[e] + kPage - 1) / kPage - 1; }
__device__ __forceinline__ int last_page(const TreeParams& p, int e) { return p.end_page[e]; }
// the cut queries' row of a unit's first
__device__ __forceinline__ int cut_row(const AttendParams& p, const Place& w) {
  return (p.entry[w.e] * p.heads + w.h) * p.nq * p.rep + w.z * p.unit_rows;
}
__device__ __forceinline__ int cut_row(const TreeParams& p, const Place& w) { return w.h * p.rows + p.row0[w.e] + w.z * kUnitRows; }
// For the joining kernel: the unit at w, whose first slot in the range is `at`,
// of which the range takes all tiles from the first on, but not all.
__device__ __forceinline__ void tell_cut(const AttendParams& p, const Work& work, const Place& w, int at, int tiles, int slot) {
  const int end = at - w.j + work.cost + tiles - 1;  // the unit's last slot
  p.cuts[work.block] = {range_of(end, work.grid, work.total), slot, w.e, w.h, w.z, {0, 0, 0}};
}
// Of slot t (a whole warp calls it together).
__device__ inline Place place_of(const AttendParams& p, const Work& work, int t) {
  Place w;
  int hi = work.count - 1;
  w.e = 0;
  while (w.e < hi) {
    const int mid = (w.e + hi + 1) / 2;
    if (p.cum[mid] <= t) w.e = mid;
    else hi = mid - 1;
  }
  t -= p.cum[w.e];
  w.h = t / p.per[w.e];
  w.z = 0;
  w.j = t % p.per[w.e];
  const int units = (p.count[w.e] * p.rep + p.unit_rows - 1) / p.unit_rows;
  if (units == 1) return w;
  const int lane = threadIdx.x & 31;
  for (int z0 = 0;; z0 += 32) {  // 32 row tiles at a time, their slots summed up
    const int z = z0 + lane;
    int sum = 0;
    if (z < units) sum = tiles_at(p, {w.e, w.h, z, 0}).n + work.cost;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += x;
    }
    const unsigned beyond = __ballot_sync(0xFFFFFFFFu, sum > w.j);
    if (beyond) {
      const int i = __ffs(beyond) - 1;
      const int before = __shfl_sync(0xFFFFFFFFu, sum, i ? i - 1 : 0);
      w.z = z0 + i;
      w.j -= i ? before : 0;
      return w;
    }
    w.j -= __shfl_sync(0xFFFFFFFFu, sum, 31);
    if (z0 + 32 >= units) return w;  // not reached: t is a slot of this head
  }
}
__device__ inline Place place_of(const TreeParams& p, const Work& work, int t) {
  Place w;
  int hi = work.first + work.count - 1;
  w.e = work.first;
  while (w.e < hi) {
    const int mid = (w.e + hi + 1) / 2;
    if (p.cum[mid] <= t) w.e = mid;
    else hi = mid - 1;
  }
  t -= p.cum[w.e];
  const int per = p.tiles[w.e] + work.cost, units = (p.n[w.e] + kUnitRows - 1) / kUnitRows, u = t / per;
  w.j = t - u * per;
  w.h = u / units;
  w.z = u - w.h * units;
  return w;
}
// The unit after w's.
__device__ __forceinline__ void next_unit(const AttendParams& p, Place& w) {
  w.j = 0;
  if (++w.z * p.unit_rows < p.count[w.e] * p.rep) return;
  w.z = 0;
  if (++w.h < p.heads) return;
  w.h = 0;
  ++w.e;
}
__device__ __forceinline__ void next_unit(const TreeParams& p, Place& w) {
  w.j = 0;
  if (++w.z * kUnitRows < p.n[w.e]) return;
  w.z = 0;
  if (++w.h < p.heads) return;
  w.h = 0;
  ++w.e;
}
// The index of row r of an entry (a leaf) and kv head among the rows [entry][query head][query] of q and out.
template <class P>
__device__ __forceinline__ long long row_index(const P& p, const Place& w, int r) {
  const int j = query_of(p, r);
  return static_cast<long long>((p.entry[w.e] * p.heads + w.h) * p.rep + r - j * p.rep) * p.nq + j;
}

// counts: of every entry of the call, also those without keys
cudaError_t launch_prefill(const AttendParams& p, const int* counts, int grid, cudaStream_t stream);
// zeros for the queries of empty slots
int store_zeros(const iq_paged* c, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, void* out,
                int out_f32, iq_stream_t stream);

// Waits end: after a second (no stage takes a thousandth of it) the CTA's
// abort flag is raised, every later wait of the CTA returns at once, and the
// kernel runs out with a status bit set.
__device__ __forceinline__ unsigned long long now_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
struct Waits {
  volatile int* abort;  // shared memory
  unsigned* status;
  __device__ __forceinline__ bool slow(uint64_t* bar, uint32_t parity, unsigned bit) const {
    const unsigned long long t0 = now_ns();
    for (;;) {
      if (mbar_try_wait(bar, parity, 20000u)) return true;
      if (*abort) return false;
      if (now_ns() - t0 > 1000000000ull) {
        *abort = 1;
        atomicOr(status, bit);
        return false;
      }
    }
  }
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, unsigned bit) const {
    return mbar_try_wait(bar, parity & 1, 20000u) || slow(bar, parity & 1, bit);
  }
  // for a warp that runs as one: the same answer to every lane
  __device__ __forceinline__ bool together(uint64_t* bar, uint32_t parity, unsigned bit) const {
    return __all_sync(0xFFFFFFFFu, (*this)(bar, parity, bit));
  }
  // the same whether or not the CTA has given up: for what is in flight at the end
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    const unsigned long long t0 = now_ns();
    while (!mbar_try_wait(bar, parity & 1, 20000u))
      if (now_ns() - t0 > 1000000000ull) return;
  }
};
// status bits of the waits that ran out
constexpr unsigned kLostLoad = 0x1, kLostMma = 0x2, kLostRows = 0x8;

// Shared-memory operand descriptors, 128-byte swizzle.  K-major: rows of 128
// bytes, groups of 8 rows 1024 bytes apart.  MN-major: the 128 contiguous
// bytes run along M or N, `wide` bytes to the next 128 of them, and groups of
// 8 rows of K lie 1024 bytes apart.
__device__ __forceinline__ uint64_t operand(uint32_t saddr, uint32_t wide = 16) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(wide >> 4) << 16 |
         static_cast<uint64_t>(1024 >> 4) << 32 | static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(2) << 61;
}
// kind::f8f6f4, e4m3 x e4m3 -> fp32; which operands are MN-major
__host__ __device__ constexpr uint32_t shape(int m, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
// The products are issued by a whole warp that runs as one, an elected lane (always
// the same) executing them: their operands then live in uniform registers.  From
// a lane that runs alone each operand is moved there first, and next to the row
// threads' work the issue, not the tensor cores, sets the pace.
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(add ? 1u : 0u)
      : "memory");
}
// kind::mxf8f6f4: the same product with a power-of-two scale (an exponent + 127 in a
// byte) for every row of A or B and 32 elements of K.  A scale is byte `id` of the
// 32-bit word in lane r % 32, column r / 32 of its operand's place in tensor memory,
// the same in all four groups of 32 lanes.
constexpr int kScaleBytes = 512;  // of 128 rows and four ids in shared memory: [r % 32][r / 32][id]
__device__ __forceinline__ int scale_at(int r, int id) { return (r & 31) * 16 + (r >> 5) * 4 + id; }
__host__ __device__ constexpr uint32_t shape_scaled(int m, int n, bool a_mn, bool b_mn, int a_id, int b_id) {
  return (static_cast<uint32_t>(b_id) << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) |
         (static_cast<uint32_t>(a_id) << 29);
}
// the scales of 128 rows from shared memory to four columns; runs in order with the products behind it
__device__ __forceinline__ void copy_scales(uint32_t to, uint32_t saddr) {
  const uint64_t from = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | static_cast<uint64_t>(1) << 16 |
                        static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;  // rows of 16 bytes, not swizzled
  asm volatile(
      "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n}\n" ::"r"(to),
      "l"(from)
      : "memory");
}
__device__ __forceinline__ void mma_scaled_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t a_scales, uint32_t b_scales,
                                                bool add) {  // A in tensor memory
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], [%1], %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(a_scales), "r"(b_scales), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t a_scales, uint32_t b_scales, bool add) {
  asm volatile(
      "{\n.reg .pred p, q;\nsetp.ne.b32 p, %6, 0;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(a_scales), "r"(b_scales), "r"(add ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "{\n.reg .pred q;\nelect.sync _|q, 0xFFFFFFFF;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The loading warp of an attention kernel (a whole warp): streams the key and
// value tiles of a range's segments through a ring of SLOTS shared-memory slots,
// in the order of the products, K0, K1, V0, K2, V1, ... (each segment to its
// end, or ACROSS segments as one stream), and hands
// the tiles' page scales to the row threads through a ring of their own, so
// that those touch no global memory between a segment's begin and its end (a
// load under a saturated HBM takes a tile's time and more).  A lane holds the
// id and the scales of one page of 16 tiles.  Ids are fetched 16 tiles or two
// segments ahead, scales half of that.
template <int SLOTS, bool ACROSS, class P = AttendParams>
struct Loader {
  // a tile's scales live until its weights are written: K(j + 4) takes, of 4 slots, that of K(j + 2), free
  // once its scores are done, which the prefill kernel issues behind tile j's last product; K(j + 8) takes,
  // of 6 slots, that of K(j + 5), whose scores wait for the weights of tile j + 3
  static constexpr int kRing = SLOTS == 4 ? 4 : 8;
  static_assert(SLOTS == 4 || SLOTS == 6, "the ring's length is reasoned above");

  // up to 16 tiles of a segment, a lane's page of them and its scales
  struct Block {
    int n, h, id;
    bool last;  // of its segment
    float2 scales;
  };
  const P& p;
  const Work& work;
  uint8_t* smem;
  uint64_t *full, *empty;
  float4* scales;      // [kRing] keys' scales of the tile's two pages, values'
  uint64_t* scales_in; // [kRing]
  const Waits& wait;

  // One place in the code for every kind of step: the first pass through it is fetched while
  // all of the GPU fetches its own (see the rows' kernel).
  __device__ __forceinline__ void run(Place w, int first, int last, uint64_t policy) const {
    if (p.stall) return;
    const int lane = threadIdx.x & 31;
    // the segment whose blocks are being taken
    Tiles tiles{};
    const int* row = nullptr;
    int at = first, begin = 0, left = 0, end_page = 0, h = 0;
    // the block being loaded, the next (its ids are there), the one behind it (asked for)
    Block a{}, b{}, c{};
    int ahead = 0, j = 0, issued = 0, it = 0;
    int v0 = 0, v1 = 0, v_head = -1;  // the tile whose values come next
    for (bool ok = true; ok;) {
      while (j == a.n && ahead < 4) {
        if (left == 0 && at < last) {
          tiles = tiles_at(p, w);
          const Part part = part_of(work, w, tiles.n, last - at);
          begin = part.begin;
          left = part.n;
          row = p.table + static_cast<long long>(p.slot[w.e]) * p.max_pages;
          end_page = last_page(p, w.e);
          h = w.h;
          at += tiles.n + work.cost - w.j;
          next_unit(p, w);
        }
        a = b;
        b = c;
        c.n = min(left, 16);
        c.h = h;
        if (c.n > 0) c.id = __ldcg(row + min(2 * tiles.tile(begin + min(lane >> 1, c.n - 1)) + (lane & 1), end_page));
        begin += c.n;
        left -= c.n;
        c.last = left == 0;
        if (b.n > 0) {
          b.id = page_in_pool(b.id, p.pages, p.status);
          const long long x = static_cast<long long>(b.id) * p.heads + b.h;
          b.scales = make_float2(__ldcg(p.k_scales + x), __ldcg(p.v_scales + x));
        }
        j = 0;
        ahead = ahead < 2 ? ahead + 1 : a.n == 0 ? 4 : 3;
        if (ahead == 4) break;
        if (ahead == 3 && a.n > 0) break;
      }
      const bool more = j < a.n;
      if (!more && v_head < 0) break;
      const int id0 = __shfl_sync(0xFFFFFFFFu, a.id, 2 * j & 31), id1 = __shfl_sync(0xFFFFFFFFu, a.id, (2 * j + 1) & 31);
      const bool closes = !ACROSS && more && a.last && j == a.n - 1;  // its own values too
#pragma unroll 1
      for (int kind = 0; kind < 3 && ok; ++kind) {  // the tile's keys, the values of the one before, its own
        if (kind == 0 ? !more : kind == 1 ? v_head < 0 : !closes) continue;
        const int s = issued % SLOTS;
        if (issued >= SLOTS) ok = __all_sync(0xFFFFFFFFu, wait(&empty[s], issued / SLOTS - 1, kLostLoad));
        if (!ok) break;
        if (lane == 0) {
          const CUtensorMap* map = kind == 0 ? &p.k_map : &p.v_map;
          const int y0 = ((kind == 1 ? v0 : id0) * p.heads + (kind == 1 ? v_head : a.h)) * kPage;
          const int y1 = ((kind == 1 ? v1 : id1) * p.heads + (kind == 1 ? v_head : a.h)) * kPage;
          mbar_arrive_expect_tx(&full[s], kSlotBytes);
          uint8_t* to = smem + s * kSlotBytes;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            tensor2d_g2s(to + half * kHalfBytes, map, 128 * half, y0, &full[s], policy);
            tensor2d_g2s(to + half * kHalfBytes + kHalfBytes / 2, map, 128 * half, y1, &full[s], policy);
          }
        }
        ++issued;
        __syncwarp();
        if (kind > 0) continue;
        const int x = lane - 2 * j;
        if (x == 0 || x == 1) {
          float* to = reinterpret_cast<float*>(&scales[it % kRing]);
          to[x] = a.scales.x;
          to[2 + x] = a.scales.y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&scales_in[it % kRing]);
        ++it;
      }
      v0 = id0;
      v1 = id1;
      v_head = more && !closes ? a.h : -1;
      j += more;
    }
    if (lane == 0)  // no copy left in flight
      for (int s = 0; s < SLOTS && s < issued; ++s) wait.drain(&full[s], (issued - 1 - s) / SLOTS);
  }
};

// n consecutive columns of this thread's lane (volatile, and read only after ld_wait)
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* v);
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const float* v);

template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t addr, float* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t addr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
        "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]),
        "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_st<4>(uint32_t addr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<8>(uint32_t addr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t addr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}

template <>
__device__ __forceinline__ void tmem_st<32>(uint32_t addr, const float* v) {
  tmem_st<16>(addr, v);
  tmem_st<16>(addr + 16, v + 16);
}

// Byte offset of byte `c` of row `r` in a 128-byte-swizzled block of 128-byte rows.
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return static_cast<uint32_t>(r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 15));
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
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// both halves added to fp32 sums
__device__ __forceinline__ void add_to(float& lo, float& hi, uint32_t h2) {
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\nadd.rn.f32.f16 %0, l, %0;\nadd.rn.f32.f16 %1, h, %1;\n}" : "+f"(lo), "+f"(hi) : "r"(h2));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One query row (a warp; lane l holds dims 8l .. 8l+7 as bf16) as two e4m3
// parts: x * 2^-e = hi + lo / QLO, with the row's largest element in (224,
// 448].  A bf16 has 8 significant bits and an e4m3 code 4, so the two parts
// hold it exactly but for elements 2^14 (QLO 16) or 2^10 (QLO 1) below the row's
// largest.  Returns 2^e; a row with a NaN or an infinity becomes all NaN.
template <int QLO>  // 1 or 16
__device__ __forceinline__ float split_query(uint4 raw, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));  // bf16 magnitudes order as integers
  const uint32_t bad = top >= 0x7F80u ? 0x7F7F7F7Fu : 0u;  // no branch, so that several rows interleave
  int e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  e = min(max(e, -100), 120);
  const float inv = power2(-e);
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // as fp16, exact (8 significant bits, at most 448) but for elements 2^23 below the row's largest
    const uint32_t x = f16x2(bf16_to_f32(w[j] & 0xFFFFu) * inv, __uint_as_float(w[j] & 0xFFFF0000u) * inv);
    h[j] = e4m3x2_of_f16x2(x);
    uint32_t rest = sub_f16x2(x, e4m3x2_to_f16x2(h[j]));
    if constexpr (QLO > 1) rest = mul_f16x2(rest, 0x4C004C00u);  // 16
    l[j] = e4m3x2_of_f16x2(rest);
  }
  hi = make_uint2(h[0] | h[1] << 16 | bad, h[2] | h[3] << 16 | bad);
  lo = make_uint2(l[0] | l[1] << 16 | bad, l[2] | l[3] << 16 | bad);
  return power2(e);
}
// the largest of a whole warp's values (of those that are numbers)
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(m) : "f"(x));
  return m;
}
__device__ __forceinline__ float clamp_finite(float x) { return fminf(fmaxf(x, -3e38f), 3e38f); }

__device__ __forceinline__ void store_out(void* out, int out_f32, long long at, float x) {
  if (out_f32) static_cast<float*>(out)[at] = x;
  else static_cast<uint16_t*>(out)[at] = static_cast<uint16_t>(f32_to_bf16_bits(x));
}

__device__ __forceinline__ void store_out8(void* out, int out_f32, long long at, const float (&x)[8], float f) {
  if (out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
    o[0] = make_float4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
    o[1] = make_float4(x[4] * f, x[5] * f, x[6] * f, x[7] * f);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f32_to_bf16_bits(x[2 * j] * f) | f32_to_bf16_bits(x[2 * j + 1] * f) << 16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace paged
}  // namespace iq
