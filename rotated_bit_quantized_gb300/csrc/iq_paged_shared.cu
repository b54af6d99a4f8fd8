// libiqkv: attention of slots that share pages of the paged 8-bit cache.
//
// softmax(s) . v over a union of key sets is the weighted mean of the sets' own
// results, weights 2^(their maximum) * their sum; so the pages that several slots
// hold are multiplied once, with the rows of all of them side by side, and each slot's
// own pages apart, and the partial results are joined.  What is shared is found on the
// host, from the page ids of the table: a tree whose nodes are runs of pages that a
// group of slots holds and others do not.  One launch has CTAs of two kinds: nodes of many
// rows as in the prefill kernel (iq_paged_rows.cuh), whose M dimension the rows of many
// slots fill; what a slot holds alone as in the split kernel (iq_paged_split.cuh).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "iq_paged_rows.cuh"
#include "iq_paged_split.cuh"
#include "iq_pages.cuh"

namespace iq {
namespace paged {
namespace {

// ------------------------------------------------------------------ queries

struct TreeCutParams {
  const uint16_t* q;
  uint8_t* cut;
  float* factors;
  int2* place;
  int4* results;
  int rows, entries, causal;
  float scale;
  short entry[IQ_MAX_BATCH], lowest[IQ_MAX_BATCH];  // place in the call, lowest node
  int row0[IQ_MAX_BATCH + 1], pos0[IQ_MAX_BATCH];   // first row, first query's position
};

// The range that holds slot t of `total` in `grid`: the last g with g * total / grid <= t,
// that is, g * total < (t + 1) * grid.
__device__ __forceinline__ int range_with(int t, int grid, int total) {
  const unsigned long long x = static_cast<unsigned long long>(t + 1u) * grid;
  int g = static_cast<int>(__fdividef(static_cast<float>(x), static_cast<float>(total)));  // off by one at most
  if (static_cast<unsigned long long>(g) * total >= x) --g;
  else if (static_cast<unsigned long long>(g + 1) * total < x) ++g;
  return g;
}

// Where the partial results of a row at a node are: `first`, and from `behind` on those of the
// ranges behind, `step` rows apart; `count` in all.
struct Results {
  int first, behind, step, count;
};
__device__ inline Results results_of(const TreeParams& p, int e, int h, int row) {
  const bool narrow = e >= p.leaves;
  const int cost = narrow ? p.narrow_cost : p.wide_cost, grid = narrow ? p.narrow : p.wide, total = narrow ? p.narrow_total : p.wide_total;
  const int step = narrow ? p.narrow_rows : kUnitRows, per = p.tiles[e] + cost;
  const int x = row - p.row0[e], z = x / kUnitRows, units = (p.n[e] + kUnitRows - 1) / kUnitRows;  // (a leaf's: one)
  const int begin = p.cum[e] + (h * units + z) * per;
  const int g0 = range_with(begin + cost, grid, total), g1 = range_with(begin + per - 1, grid, total);
  return {p.part0[e] + h * p.n[e] + x, (narrow ? p.narrow_cont : p.wide_cont) + (g0 + 1) * step + x - z * kUnitRows, step, 1 + g1 - g0};
}

// 3 us for 256 rows of 2 heads, latency that the next kernel's start hides (it fetches its first
// pages meanwhile).
// Every row of (entry, kv head): two e4m3 parts, the factor of its scores, where it
// stands, and where its partial results will be (a lane for each node that it is under: the
// joining kernel, of eight warps to a row, spent most of its time on that); a warp takes
// four rows.
__global__ void __launch_bounds__(256) paged_tree_cut_kernel(const __grid_constant__ TreeCutParams c, const __grid_constant__ TreeParams p) {
  wait_for_last_kernel();
  const int lane = threadIdx.x & 31, w0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4, h = blockIdx.y;
  uint4 raw[4];
  int entry[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = min(w0 + k, c.rows - 1);
    int s = 0, hi = c.entries - 1;  // the last entry that begins at or before the row
    while (s < hi) {
      const int mid = (s + hi + 1) / 2;
      if (c.row0[mid] <= row) s = mid;
      else hi = mid - 1;
    }
    const int x = row - c.row0[s], j = query_of(p, x);
    const int at = (c.entry[s] * p.heads * p.rep + x - j * p.rep) * p.nq + j;
    raw[k] = __ldcs(reinterpret_cast<const uint4*>(c.q + (static_cast<long long>(h) * p.rep * p.nq + at) * kHeadDim) + lane);
    entry[k] = s;
    if (h == 0 && lane == 0 && w0 + k < c.rows) c.place[row] = make_int2(c.pos0[s] + (c.causal ? j : 0), at);
  }
  // lane (k, level): row k's results at its node of that level, the lowest first (while the
  // queries are on their way)
  if (const int k = lane / kDepth, level = lane % kDepth, row = w0 + k; k < 4 && row < c.rows) {
    int e = c.lowest[k == 0 ? entry[0] : k == 1 ? entry[1] : k == 2 ? entry[2] : entry[3]];
    for (int i = 0; i < level && e >= 0; ++i) e = p.parent[e];
    const Results r = e >= 0 ? results_of(p, e, h, row) : Results{0, 0, 0, 0};
    c.results[(static_cast<long long>(h) * c.rows + row) * kDepth + level] = make_int4(r.first, r.behind, r.step, r.count);
  }
  if (c.scale < 0.0f) {  // the factors are positive, so that the largest product is the largest score
#pragma unroll
    for (int k = 0; k < 4; ++k)
      raw[k] = make_uint4(raw[k].x ^ 0x80008000u, raw[k].y ^ 0x80008000u, raw[k].z ^ 0x80008000u, raw[k].w ^ 0x80008000u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint2 hi, lo;
    const float f = split_query<1>(raw[k], hi, lo);
    if (w0 + k >= c.rows) break;
    const long long w = static_cast<long long>(h) * c.rows + w0 + k;
    reinterpret_cast<uint2*>(c.cut + w * kHeadDim)[lane] = hi;
    reinterpret_cast<uint2*>(c.cut + (static_cast<long long>(p.heads) * c.rows + w) * kHeadDim)[lane] = lo;
    if (lane == 0) c.factors[w] = fminf(f * (fabsf(c.scale) * kLog2e), 3e38f);
  }
}

// ------------------------------------------------------------------ products

// CTAs of both kinds, so that neither waits for the other's end.  16 / 2 heads, with the other two
// launches: 32 paths of 32768 common tokens 31 us (540 TFLOP/s; every path's pages apart 132),
// bound by a tile's row threads next to its products and by a launch of short CTAs, tensor
// pipe 35%; 128 paths of 8192 common tokens and 16 tiles each of their own 66 us (apart
// 167), 284 MB from HBM at 4.6 TB/s under a profiler, bound by its beginning, HBM and the
// tiles of many rows, which take a quarter longer beside it.
template <int NR>
__global__ void __launch_bounds__(rows::kThreads, 1) paged_tree_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled operands need it; no room to align by hand
  const int block = static_cast<int>(blockIdx.x);
  if (block < p.wide) rows::run(p, {0, p.leaves, p.wide_cost, p.wide_total, block, p.wide}, smem);
  else split::run<NR>(p, {p.leaves, p.nodes - p.leaves, p.narrow_cost, p.narrow_total, block - p.wide, p.narrow}, smem);
}
template <int NR>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  using Few = split::TreeShape<NR>;
  constexpr int kSmem = rows::kTreeSmem > Few::kSmem ? rows::kTreeSmem : Few::kSmem;
  static_assert(Few::kThreads <= rows::kThreads, "threads of one CTA");
  static std::atomic<uint64_t> seen{0};
  const void* kernel = reinterpret_cast<const void*>(&paged_tree_kernel<NR>);
  const cudaError_t e = allow_smem(kernel, kSmem, seen);
  void* args[] = {const_cast<TreeParams*>(&p)};
  return e == cudaSuccess ? launch_after(kernel, dim3(p.wide + p.narrow), rows::kThreads, kSmem, stream, args) : e;
}

// ------------------------------------------------------------------ join

// CTA (x, h) joins rows of kv head h, 2^shift warps a row, a lane per 8 dims, in the
// order of nodes and ranges.  A warp asks for four partial results at a time, references
// and sums with them, so that it takes a trip to memory or two.  Bound by these, and by
// L2, which the results of all CTAs pass at once (17 MB for 32 paths of 32768 common
// tokens: 5 us).
struct TreeJoinParams {
  const float* part_o;
  const float2* part_ml;
  const int2* place;
  const int4* results;
  void* out;
  int out_f32, rows, stride, shift;  // stride: from a kv head's rows to the next one's in out
};
__global__ void __launch_bounds__(256, 4) paged_tree_join_kernel(const __grid_constant__ TreeJoinParams p) {
  wait_for_last_kernel();
  constexpr int kAtOnce = 4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, shift = p.shift, share = 1 << shift, h = blockIdx.y;
  const int wanted = static_cast<int>(blockIdx.x) * (8 >> shift) + (warp >> shift), row = min(wanted, p.rows - 1);
  const int4* results = p.results + (static_cast<long long>(h) * p.rows + row) * kDepth;
  __shared__ float part[8][kHeadDim + 2];
  float m = kUnset, sum = 0.0f, o[8] = {};
  int4 next = __ldcg(results);
  const int at = __ldcg(&p.place[row].y);
  int before = 0;  // partial results of the nodes before
#pragma unroll 1
  for (int level = 1; next.w > 0; ++level) {
    const int4 r = next;
    next = level < kDepth ? __ldcg(results + level) : make_int4(0, 0, 0, 0);
#pragma unroll 1
    for (int turn = (warp - before) & (share - 1); turn < r.w; turn += kAtOnce * share) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce][2];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int k = turn + i * share;
        ml[i] = make_float2(-__builtin_huge_valf(), 0.0f);
        v[i][0] = v[i][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (k >= r.w) continue;
        const long long x = k == 0 ? r.x : r.y + (k - 1) * r.z;
        const float4* from = reinterpret_cast<const float4*>(p.part_o + x * kHeadDim + lane * 8);
        ml[i] = __ldcg(&p.part_ml[x]);
        v[i][0] = __ldcg(from);
        v[i][1] = __ldcg(from + 1);
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
      const float old = ex2_approx(m - top);
      m = top;
      sum *= old;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] *= old;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float f = ex2_approx(ml[i].x - m);
        sum = fmaf(f, ml[i].y, sum);
        o[0] = fmaf(f, v[i][0].x, o[0]), o[1] = fmaf(f, v[i][0].y, o[1]), o[2] = fmaf(f, v[i][0].z, o[2]), o[3] = fmaf(f, v[i][0].w, o[3]);
        o[4] = fmaf(f, v[i][1].x, o[4]), o[5] = fmaf(f, v[i][1].y, o[5]), o[6] = fmaf(f, v[i][1].z, o[6]), o[7] = fmaf(f, v[i][1].w, o[7]);
      }
    }
    before += r.w;
  }
  if (share > 1) {
#pragma unroll
    for (int d = 0; d < 8; ++d) part[warp][d * 32 + lane] = o[d];
    if (lane < 2) part[warp][kHeadDim + lane] = lane ? m : sum;
    __syncthreads();
    if (warp & (share - 1)) return;
#pragma unroll 1
    for (int w = warp + 1; w < warp + share; ++w) {
      const float other = part[w][kHeadDim + 1], top = fmaxf(m, other), f = ex2_approx(other - top), old = ex2_approx(m - top);
      m = top;
      sum = fmaf(f, part[w][kHeadDim], sum * old);
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] = fmaf(f, part[w][d * 32 + lane], o[d] * old);
    }
  }
  if (wanted < p.rows)
    store_out8(p.out, p.out_f32, (static_cast<long long>(h) * p.stride + at) * kHeadDim + lane * 8, o, sum == 0.0f ? 0.0f : 1.0f / sum);
}

// ------------------------------------------------------------------ what is shared

// Microseconds, fitted to calls of 2 to 32 paths of 256 to 32768 common tokens, 2 and 8 kv
// heads, 1 to 8 queries.  kFetch: all CTAs of a launch fetch the same code at once, some 50 KB,
// which the GPU hands out at a rate, so each more delays them all.  kTile: a tile of 128
// rows; kFewTile: one of at most 8, 16, 32, beside which the first take a quarter longer (so
// these are below what a tile of few rows takes; fitted to the best split of the SMs on 14 trees
// of 32 to 250 paths, 500 to 2048 tokens each of their own: a third more or less of them costs 3 to
// 8%); a unit's beginning and end take as long as kUnitCost tiles.  kLaunches: the three launches without these.  kOrdinary, kOrdinaryTile: the
// launches of the attention of every slot apart, its tile of at most 8, 16, 32 and of
// more rows.  Shared and apart, 2 kv heads: 2 paths of 2048 tokens 13 and 10.5 us,
// 8 of 4096 14 and 17, 32 of 8192 22 and 43.
constexpr double kFetch = 0.05, kTile = 1.45, kFewTile[4] = {0.8, 1.0, 1.5, 0.0}, kLaunches = 9.25;
constexpr double kOrdinary = 8.5, kOrdinaryTile[4] = {1.2, 1.8, 3.2, 2.2};
constexpr int kUnitCost = 3;
constexpr int narrow_kind(int rows) { return rows <= 8 ? 0 : rows <= 16 ? 1 : rows <= 32 ? 2 : 3; }

struct Planner {
  int rep, window, sinks, inner = 0;
  bool forced;  // test hook (iq_paged_debug_share): shared wherever pages are
  // per entry, in the tree's order once it is built
  int n = 0;
  struct Entry {
    const int32_t* row;  // its page ids
    int pages, len, count, p_lo, p_hi, place, slot, lowest;
  } e[IQ_MAX_BATCH];
  // a node before the order of the entries, and with it of the rows, is known
  struct Node {
    int first, last, parent;  // entries [first, last)
    bool leaf;
    Tiles tiles;
  } node[kNodes];
  int nodes = 0;

  // The tiles of [start, stop) that some row of entries [a, b) sees.
  Tiles seen(int a, int b, int start, int stop) const {
    int lo = e[a].p_lo, hi = e[a].p_hi, len = e[a].len;
    for (int i = a + 1; i < b; ++i) {
      lo = std::min(lo, e[i].p_lo);
      hi = std::max(hi, e[i].p_hi);
      len = std::max(len, e[i].len);
    }
    Tiles t = tiles_of(len, lo, hi, 1, window, sinks);
    const int end = std::min(t.n + t.skip, stop);
    const int a1 = std::min(t.sinks, stop), b0 = std::max(t.sinks + t.skip, start);  // sinks' tiles [start, a1), others [b0, end)
    const int near = std::max(a1 - start, 0), far = std::max(end - b0, 0);
    t.sinks = near;
    t.n = near + far;
    t.base = near ? start : b0;
    t.skip = near ? b0 - a1 : 0;
    return t;
  }
  int row_units(int a, int b) const {
    int rows = 0;
    for (int i = a; i < b; ++i) rows += e[i].count * rep;
    return (rows + kUnitRows - 1) / kUnitRows;
  }
  int add(int a, int b, int parent, bool leaf, const Tiles& t) {
    node[nodes] = {a, b, parent, leaf, t};
    return nodes++;
  }
  // Where [from, to) of two rows begins to differ, 64 ids at a time as long as it does not (one
  // at a time, 32 paths of 512 pages took the host 6 us).
  static int alike(const int32_t* u, const int32_t* v, int from, int to) {
    constexpr int kAtOnce = 64;
    while (from + kAtOnce <= to && std::memcmp(u + from, v + from, kAtOnce * sizeof(int32_t)) == 0) from += kAtOnce;
    while (from < to && u[from] == v[from]) ++from;
    return from;
  }
  // Entries [a, b) hold the same first `page` pages; tiles before `start` are those of `parent` and above.
  void split(int a, int b, int page, int start, int parent, int depth) {
    const auto before = [&](const Entry& x, const Entry& y) {
      const int i = x.pages > page ? x.row[page] : -1, j = y.pages > page ? y.row[page] : -1;
      return i != j ? i < j : x.place < y.place;
    };
    if (!std::is_sorted(e + a, e + b, before)) std::sort(e + a, e + b, before);  // (mostly they are)
    for (int x = a, y; x < b; x = y) {
      y = x + 1;
      if (e[x].pages > page)
        while (y < b && e[y].pages > page && e[y].row[page] == e[x].row[page]) ++y;
      if (y - x == 1) {  // a leaf
        const Tiles t = seen(x, y, start, (e[x].pages + 1) / 2);
        e[x].lowest = t.n > 0 ? add(x, y, parent, true, t) : parent;
        continue;
      }
      int common = e[x].pages, most = e[x].pages;
      for (int i = x + 1; i < y; ++i) {
        common = alike(e[x].row, e[i].row, page, std::min(common, e[i].pages));
        most = std::max(most, e[i].pages);
      }
      const int stop = common == most ? (common + 1) / 2 : common / 2;
      const Tiles t = seen(x, y, start, stop);
      const bool once = depth < kDepth - 1 && inner < kInner &&
                        (forced ? t.n > 0 : static_cast<long long>(row_units(x, y)) * (t.n + kUnitCost) < static_cast<long long>(y - x) * t.n);
      int under = parent;
      if (once) {
        ++inner;
        under = add(x, y, parent, false, t);
      }
      split(x, y, common, once ? stop : start, under, depth + (once ? 1 : 0));
    }
  }

  // How the nodes' units are shared out among the SMs; false: every slot's pages apart are faster.
  // (tiles, units: of nodes of many rows, and of leaves of few, where these are apart)
  long long tiles[2] = {}, units[2] = {};
  int wide = 0, narrow = 0;
  bool share_out(int heads, int leaf_rows, int sms) {
    const int kind = narrow_kind(leaf_rows);
    bool alike = true;  // all units of many rows have one length
    int length = -1;
    for (int k = 0; k < nodes; ++k) {
      const Node& a = node[k];
      const int few = a.leaf && kind < 3;
      const long long u = static_cast<long long>(heads) * row_units(a.first, a.last);
      units[few] += u;
      tiles[few] += u * a.tiles.n;
      if (few) continue;
      alike &= length < 0 || length == a.tiles.n;
      length = a.tiles.n;
    }
    // the SMs go to the two kinds by what each has to do
    const double many = kTile * (tiles[0] + units[0] * kUnitCost), few = kFewTile[kind] * (tiles[1] + units[1] * kUnitCost);
    narrow = tiles[1] == 0 ? 0 : std::min(std::max(static_cast<int>(sms * few / (many + few) + 0.5), 1), sms - 1);
    const int room = sms - narrow;
    narrow = static_cast<int>(std::min<long long>(narrow, tiles[1]));
    // Units of one length are cut into as many ranges each, so that none is of two units.
    alike &= units[0] <= room && static_cast<int>(room % units[0]) * 16 <= room;
    const long long sets = alike ? units[0] : 1, whole = alike ? length : tiles[0], most = room / sets;
    // tiles of a range: so many that one CTA less saves no more than a tile costs
    long long each = (whole + most - 1) / most;
    auto ranges = [&](long long x) { return (whole + x - 1) / x; };
    while (each < whole && kFetch * sets * (ranges(each) - ranges(each + 1)) > kTile) ++each;
    wide = static_cast<int>(sets * ranges(each));
    if (forced) return true;
    long long apart = 0;
    for (int i = 0; i < n; ++i) apart += static_cast<long long>(seen(i, i + 1, 0, (e[i].pages + 1) / 2).n) * heads;
    // (kLaunches has a unit's beginning and end for every CTA; many short units have more)
    const double longest = std::max({kTile * each, many / wide - kTile * kUnitCost, narrow ? few / narrow : 0.0});
    const double shared = kLaunches + kFetch * (wide + narrow) + longest;
    return shared < kOrdinary + kFetch / 2 * std::min<long long>(apart, sms) + kOrdinaryTile[kind] * apart / sms;
  }
};

// The rows of all nodes of one kv head are at most kDepth times the call's.
size_t tree_bytes(size_t rows, size_t heads) {
  const size_t parts = kDepth * heads * rows + static_cast<size_t>(num_sms()) * kUnitRows;
  return parts * (kHeadDim * sizeof(float) + sizeof(float2)) + rows * sizeof(int2) +
         heads * rows * (2 * kHeadDim + sizeof(float) + kDepth * sizeof(int4));
}
// Where pages are shared among slots of more rows, their own products fill the tensor cores already.
bool tree_rows(const iq_paged* c, int q_heads, int n_queries, int n_slots) {
  const long long rows = static_cast<long long>(q_heads / c->kv_heads) * n_queries;
  return rows > 0 && rows <= kUnitRows && n_slots > 1 && kDepth * rows * n_slots * c->kv_heads < (1LL << 30);
}

thread_local bool share_next = false;

int check_shared(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots,
                 int added, float scale, int causal, int window, int sinks, const void* out, int out_f32, const void* workspace,
                 size_t workspace_bytes) {
  const int st = check_attend(c, q, q_heads, n_queries, slots, counts, n_slots, added, scale, causal, window, sinks, out, out_f32, workspace,
                              workspace_bytes);
  if (st != IQ_OK || !tree_rows(c, q_heads, n_queries, n_slots)) return st;
  if (workspace_bytes < tree_bytes(static_cast<size_t>(q_heads / c->kv_heads) * n_queries * n_slots, c->kv_heads))
    return fail(IQ_ERR_WORKSPACE, "workspace missing or too small");
  return IQ_OK;
}

// The tree of shared pages of a call, where there is one and it is the faster way (or `forced`): everything of
// the launches' parameters but addresses, and how many rows of partial results there are.
bool plan_tree(const iq_paged* c, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, int causal, int window,
               int sinks, bool forced, TreeParams* tree, TreeCutParams* cutting, long long* results) {
  const int heads = c->kv_heads;
  Planner t;
  t.rep = q_heads / heads;
  t.forced = forced;
  int longest = 0;
  for (int i = 0; i < n_slots; ++i) longest = std::max(longest, c->lens[slot_of(slots, i)]);
  if (window >= longest) window = sinks = 0;  // nothing is out of it, and positions less a window stay in 32 bits
  t.window = window;
  t.sinks = sinks;
  for (int i = 0; i < n_slots; ++i) {
    const int s = slot_of(slots, i), len = c->lens[s], count = counts ? counts[i] : n_queries;
    if (len == 0 || count == 0) continue;
    const int first = causal ? len - count : len - 1;
    t.e[t.n++] = {c->table_host + static_cast<long long>(s) * c->max_pages, pages_for(len), len, count, first, len - 1, i, s, -1};
  }
  if (t.n < 2) return false;
  t.split(0, t.n, 0, 0, -1, 0);
  const int leaf_rows = t.rep * n_queries, sms = num_sms();
  if (t.inner == 0 || !t.share_out(heads, leaf_rows, sms)) return false;

  TreeParams& p = *tree;
  std::memset(&p, 0, sizeof(p));
  TreeCutParams& cut = *cutting;
  std::memset(&cut, 0, sizeof(cut));
  // leaves of at most 32 rows, as the split kernel's calls, behind the other nodes
  short number[kNodes];
  for (int few = 0; few < 2; ++few)
    for (int k = 0; k < t.nodes; ++k) {
      if ((t.node[k].leaf && leaf_rows <= 32) != (few == 1)) continue;
      number[k] = static_cast<short>(p.nodes++);
      p.leaves += few == 0;
    }
  for (int i = 0; i < t.n; ++i) {
    cut.entry[i] = static_cast<short>(t.e[i].place);
    cut.lowest[i] = static_cast<short>(t.e[i].lowest < 0 ? -1 : number[t.e[i].lowest]);
    cut.pos0[i] = t.e[i].p_lo;
    cut.row0[i + 1] = cut.row0[i] + t.e[i].count * t.rep;
  }
  p.rows = cut.row0[t.n];
  long long parts = 0;
  for (int i = 0; i < t.nodes; ++i) {
    const Planner::Node& a = t.node[i];
    const Planner::Entry& holder = t.e[a.first];
    const int k = number[i];
    p.slot[k] = static_cast<short>(holder.slot);
    p.entry[k] = static_cast<short>(holder.place);
    p.parent[k] = static_cast<short>(a.parent < 0 ? -1 : number[a.parent]);
    p.end_page[k] = holder.pages - 1;
    p.row0[k] = cut.row0[a.first];
    p.n[k] = cut.row0[a.last] - p.row0[k];
    p.part0[k] = static_cast<int>(parts);
    p.tiles[k] = a.tiles.n;
    p.base[k] = a.tiles.base;
    p.sink_tiles[k] = a.tiles.sinks;
    p.skip[k] = a.tiles.skip;
    p.p_lo[k] = a.tiles.p_lo;
    p.p_hi[k] = a.tiles.p_hi;
    parts += static_cast<long long>(heads) * p.n[k];
  }
  p.wide = t.wide;
  p.narrow = t.narrow;
  p.narrow_rows = leaf_rows <= 8 ? 8 : leaf_rows <= 16 ? 16 : 32;
  // where ranges are shorter than units, these are cut at a tile's grain
  p.wide_cost = t.tiles[0] >= 8ll * p.wide || t.units[0] >= p.wide ? kUnitCost : 0;
  p.narrow_cost = t.tiles[1] >= 8ll * p.narrow || t.units[1] >= p.narrow ? kUnitCost : 0;
  long long total[2] = {};
  for (int k = 0; k < p.nodes; ++k) {
    const int kind = k >= p.leaves;
    p.cum[k] = static_cast<int>(total[kind]);
    total[kind] += static_cast<long long>(heads) * ((p.n[k] + kUnitRows - 1) / kUnitRows) * (p.tiles[k] + (kind ? p.narrow_cost : p.wide_cost));
    if (total[kind] >= (1LL << 31)) return false;
  }
  p.wide_total = static_cast<int>(total[0]);
  p.narrow_total = static_cast<int>(total[1]);
  p.wide_cont = static_cast<int>(parts);
  parts += static_cast<long long>(p.wide) * kUnitRows;
  p.narrow_cont = static_cast<int>(parts);
  parts += static_cast<long long>(p.narrow) * p.narrow_rows;
  p.heads = heads;
  p.rep = t.rep;
  p.nq = n_queries;
  while ((2 << p.rep_shift) <= t.rep) ++p.rep_shift;
  if (t.rep & (t.rep - 1)) p.rep_mul = static_cast<unsigned>(((1ull << (32 + p.rep_shift)) + t.rep - 1) / t.rep);
  p.causal = causal;
  p.window = window;
  p.sinks = sinks;
  cut.rows = p.rows;
  cut.entries = t.n;
  cut.causal = causal;
  *results = parts;
  return true;
}

// The attention by the tree of shared pages, where there is one; *done says whether.
int attend_tree(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots,
                float scale, int causal, int window, int sinks, void* out, int out_f32, void* workspace, iq_stream_t stream, bool forced,
                bool* done) {
  *done = false;
  TreeParams p;
  TreeCutParams cut;
  long long parts = 0;
  if (!plan_tree(c, q_heads, n_queries, slots, counts, n_slots, causal, window, sinks, forced, &p, &cut, &parts)) return IQ_OK;
  const int heads = c->kv_heads;
  const long long pool_rows = static_cast<long long>(c->pages) * heads * kPage, cut_rows = static_cast<long long>(heads) * p.rows;
  p.part_o = static_cast<float*>(workspace);
  p.cut = reinterpret_cast<uint8_t*>(p.part_o + parts * kHeadDim);
  cut.results = reinterpret_cast<int4*>(p.cut + cut_rows * 2 * kHeadDim);
  p.part_ml = reinterpret_cast<float2*>(cut.results + cut_rows * kDepth);
  cut.place = reinterpret_cast<int2*>(p.part_ml + parts);
  p.factors = reinterpret_cast<float*>(cut.place + p.rows);
  p.place = cut.place;
  if (!code_map(&p.k_map, c->k_codes, pool_rows) || !code_map(&p.v_map, c->v_codes, pool_rows) ||
      !code_map(&p.q_map, p.cut, 2 * cut_rows, kUnitRows))
    return fail(IQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.q = static_cast<const uint16_t*>(q);
  p.out = out;
  p.out_f32 = out_f32;
  p.scale = scale;
  p.pages = c->pages;
  p.max_pages = c->max_pages;
  p.stall = stall_next ? 1 : 0;
  stall_next = false;
  cut.q = static_cast<const uint16_t*>(q);
  cut.cut = p.cut;
  cut.factors = p.factors;
  cut.scale = scale;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int st = store_zeros(c, q_heads, n_queries, slots, counts, n_slots, out, out_f32, stream);
  if (st != IQ_OK) return st;
  void* cut_args[] = {&cut, &p};
  cudaError_t err = launch_after(reinterpret_cast<const void*>(&paged_tree_cut_kernel), dim3((p.rows + 31) / 32, heads), 256, 0, cs, cut_args);
  if (err == cudaSuccess) err = p.narrow_rows == 8 ? launch_tree<8>(p, cs) : p.narrow_rows == 16 ? launch_tree<16>(p, cs) : launch_tree<32>(p, cs);
  if (err == cudaSuccess) {
    TreeJoinParams j;
    j.part_o = p.part_o;
    j.part_ml = p.part_ml;
    j.place = p.place;
    j.results = cut.results;
    j.out = out;
    j.out_f32 = out_f32;
    j.rows = p.rows;
    j.stride = p.rep * n_queries;
    // warps to a row, so that each has some six partial results, but all CTAs at once
    const long long of_row = parts / cut_rows;
    j.shift = of_row <= 6 ? 0 : of_row <= 12 ? 1 : of_row <= 24 ? 2 : 3;
    while (j.shift > 0 && (cut_rows << j.shift) / 8 > 4ll * num_sms()) --j.shift;
    const int each = 8 >> j.shift;
    void* args[] = {&j};
    err = launch_after(reinterpret_cast<const void*>(&paged_tree_join_kernel), dim3((p.rows + each - 1) / each, heads), 256, 0, cs, args);
  }
  if (err != cudaSuccess) return cuda_fail(err, "paged attention of shared pages");
  launched_outputs(stream, {out, static_cast<size_t>(n_slots) * q_heads * n_queries * kHeadDim * (out_f32 ? 4 : 2)});
  *done = true;
  return IQ_OK;
}

}  // namespace
}  // namespace paged
}  // namespace iq

using namespace iq;
using namespace iq::paged;

extern "C" {

int iq_paged_debug_share(void) {
  clear_error();
  share_next = true;
  return IQ_OK;
}

int iq_paged_debug_plan(const iq_paged* c, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, int causal,
                        int window, int sinks, int forced, int32_t* plan) {
  size_t need = 0;
  int st = iq_paged_attend_shared_workspace(c, q_heads, n_queries, n_slots, &need);
  if (st != IQ_OK) return st;
  if (!plan) return fail(IQ_ERR_INVALID_ARG, "null plan");
  const void* any = reinterpret_cast<const void*>(uintptr_t{256});  // (never followed)
  st = check_attend(c, any, q_heads, n_queries, slots, counts, n_slots, 0, 1.0f, causal, window, sinks, any, 0, any, SIZE_MAX);
  if (st != IQ_OK) return st;
  std::fill(plan, plan + IQ_PLAN_WORDS, 0);
  TreeParams p;
  TreeCutParams cut;
  long long parts = 0;
  if (!tree_rows(c, q_heads, n_queries, n_slots) ||
      !plan_tree(c, q_heads, n_queries, slots, counts, n_slots, causal, window, sinks, forced != 0, &p, &cut, &parts))
    return IQ_OK;
  static_assert(IQ_PLAN_WORDS == 12 + 13 * kNodes + 4 * IQ_MAX_BATCH, "the largest plan fits");
  int32_t* to = plan;
  for (int x : {p.nodes, p.leaves, cut.entries, p.rows, p.wide, p.narrow, p.wide_cost, p.narrow_cost, p.wide_total, p.narrow_total,
                p.narrow_rows, static_cast<int>(parts)})
    *to++ = x;
  for (int k = 0; k < p.nodes; ++k)
    for (int x : {static_cast<int>(p.slot[k]), static_cast<int>(p.parent[k]), p.end_page[k], p.row0[k], p.n[k], p.part0[k], p.cum[k], p.tiles[k],
                  p.base[k], p.sink_tiles[k], p.skip[k], p.p_lo[k], p.p_hi[k]})
      *to++ = x;
  for (int i = 0; i < cut.entries; ++i)
    for (int x : {static_cast<int>(cut.entry[i]), static_cast<int>(cut.lowest[i]), cut.row0[i], cut.pos0[i]}) *to++ = x;
  return IQ_OK;
}

int iq_paged_attend_shared_workspace(const iq_paged* c, int q_heads, int n_queries, int n_slots, size_t* bytes) {
  const int st = iq_paged_attend_workspace(c, q_heads, n_queries, n_slots, bytes);
  if (st == IQ_OK && tree_rows(c, q_heads, n_queries, n_slots))
    *bytes = std::max(*bytes, tree_bytes(static_cast<size_t>(q_heads / c->kv_heads) * n_queries * n_slots, c->kv_heads));
  return st;
}

int iq_paged_attend_shared(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts,
                           int n_slots, float scale, int causal, int window, int sinks, void* out, int out_f32, void* workspace,
                           size_t workspace_bytes, iq_stream_t stream) {
  const int st = check_shared(c, q, q_heads, n_queries, slots, counts, n_slots, 0, scale, causal, window, sinks, out, out_f32, workspace,
                              workspace_bytes);
  const bool forced = share_next;
  share_next = false;
  if (st != IQ_OK || n_slots == 0 || n_queries == 0) return st;
  if (tree_rows(c, q_heads, n_queries, n_slots)) {
    bool done = false;
    const int tree = attend_tree(c, q, q_heads, n_queries, slots, counts, n_slots, scale, causal, window, sinks, out, out_f32, workspace,
                                 stream, forced, &done);
    if (tree != IQ_OK || done) return tree;
  }
  return iq_paged_attend(c, q, q_heads, n_queries, slots, counts, n_slots, scale, causal, window, sinks, out, out_f32, workspace,
                         workspace_bytes, stream);
}

int iq_paged_append_attend_shared(iq_paged* c, const void* keys, const void* values, int n, const void* q, int q_heads, int n_queries,
                                  const int32_t* slots, const int32_t* counts, int n_slots, float scale, int causal, int window, int sinks,
                                  void* out, int out_f32, void* workspace, size_t workspace_bytes, iq_stream_t stream) {
  int st = check_append(c, keys, values, n, slots, counts, n_slots);
  if (st != IQ_OK) return st;
  if (counts && n != n_queries) return fail(IQ_ERR_INVALID_ARG, "counts need as many rows as queries");
  st = check_shared(c, q, q_heads, n_queries, slots, counts, n_slots, n, scale, causal, window, sinks, out, out_f32, workspace,
                    workspace_bytes);
  if (st != IQ_OK) return st;
  st = iq_paged_append(c, keys, values, n, slots, counts, n_slots, stream);
  if (st != IQ_OK) return st;
  return iq_paged_attend_shared(c, q, q_heads, n_queries, slots, counts, n_slots, scale, causal, window, sinks, out, out_f32, workspace,
                                workspace_bytes, stream);
}

}  // extern "C"
