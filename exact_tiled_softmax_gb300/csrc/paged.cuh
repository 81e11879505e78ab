// Attention over a paged key/value cache: the problem, the way its work is
// shared out over the workers of one launch, and the two ways a row leaves it.
//
// Sequence b owns the packed tokens s0 .. s0 + nq - 1 and len cached keys, of
// which its tokens are the last nq; token i sits at position len - nq + i.  The
// group = heads / kv_heads query heads of one key head read the same keys, so
// the rows of (b, key head h) are the nq * group pairs (i, g), row = i * group + g.
//
// Work.  A row tile is kRT consecutive rows of one (b, h); its keys, from the
// first that any of its rows allows to the last, are cut at multiples of
// kUnitKeys into units.  All units of the launch stand in one line, ordered by
// (b, h, row tile, key), each row tile's rounded up to a multiple of `least`, and worker r
// (a warp or a CTA, as the kernel has it) takes run r of W consecutive ones, W = total /
// workers, in a small launch rounded up to such a multiple too: every worker reads the same
// number of keys, however unequal the lengths are and without the host knowing them (they are
// read on the device, so a captured launch follows them), and in a launch with few units none
// has two tiles to end.  (A tail of short runs, taken from a counter by the workers that are done
// first, changed nothing: 332 us for 2.1 GB either way, although the first worker is done
// at 271 us; the memory is what is shared.)
// A run is a list of segments, one for each row tile that it touches.  A segment that
// holds all of its row tile's units writes Y and L; any other writes its summary
// (m, l, z) of "Exact tiled softmax attention with block-recomputed vector-Jacobian
// products", Forward procedure, to a slot of the workspace: slot 2 r + 1 when it starts
// the row tile, slot 2 r when it continues one (run r has at most one of each), and a
// merge kernel joins the slots with the star rule.
//
// A shared prefix is one more sequence of the line: all T tokens over the prefix's keys,
// without a mask.  Its rows and the sequences' own are two sets of results of the same
// [T][heads], of which `info` says where each stands; paged_join_kernel joins them.
#pragma once

#include <math.h>

#include <atomic>

#include "common.cuh"

namespace exattn {

constexpr int kPagedMaxBatch = 1024;  // prefix sums of the units stay in shared memory
constexpr int kPagedSums = kPagedMaxBatch + 2;

// Division by a number that is fixed for a launch (n < 2^31): a high product, an
// addition and a shift (Granlund and Montgomery, "Division by invariant integers
// using multiplication", PLDI 1994, figure 4.1).
struct FastDiv {
  unsigned mul, shift;
  int d;
};
inline FastDiv fast_div(int d) {
  FastDiv f{0, 0, d};
  while ((1ll << f.shift) < d) ++f.shift;
  f.mul = static_cast<unsigned>(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ int div_by(int n, const FastDiv& f) {
  return static_cast<int>((__umulhi(static_cast<unsigned>(n), f.mul) + static_cast<unsigned>(n)) >> f.shift);
}

struct PagedArgs {
  const void* Q;
  const void* Kp;
  const void* Vp;
  const int* table;   // [B][max_pages]
  const int* prefix_table;
  int prefix_at, prefix_len;  // sequence of the line that is the prefix (-1: none), its keys
  const int* lens;    // [B]
  const int* starts;  // [B + 1], or null: T / B tokens for every sequence
  int B, T, Hk, G, d, v, dtype;  // B: sequences of the line, the prefix among them
  FastDiv by_group, by_heads;  // G, Hk
  int each;                       // tokens of a sequence without starts
  int lps;  // log2(page_size)
  int num_pages, max_pages;
  int mask_kind, window;
  float sl2;  // scale * log2(e)
  long long q_stride;  // elements between tokens of Q
  void* Y;             // [T][Hk * G][v] of dtype
  float* L;            // [T][Hk * G], natural log
  // With a shared prefix, instead of both: [2][T][Hk * G][v] and [2][T][Hk * G] in fp32, the
  // sequences' own rows and the prefix's, and of each (first run, runs that hold a piece),
  // the latter 0 where the row is finished.
  float* Yf;
  int2* info;
  float* Lout;  // the call's L
  int* sane;  // whether q_starts ascends and the lengths fit, for the join
  // Workspace.
  unsigned* status;  // written by the merge kernel; null: left for a later launch
  unsigned* flags;   // [n_flags] status bits, one word for each CTA of each launch
  int n_flags;       // words that the merge kernel joins (from flags0)
  const unsigned* flags0;
  // [runs] Of run r: the row tile that it starts and others end, as (first row of the
  // tile among (b, h)'s, rows of (b, h), s0, h << 16 | runs that hold a piece); the last
  // is 0 where there is none.
  int4* desc;
  float* pm;  // [2 runs][RT] exp2 domain
  float* pl;  // [2 runs][RT]
  float* pz;  // [2 runs][RT][v]
  FastDiv by_runs;
  int runs;   // and workers
  int least;  // units that a row tile's (and a short run's) are a multiple of (a power of 2)
  bool second;  // launched early behind another attention launch, independent of it
};

struct PagedSeq {
  int s0, nq, len;
  bool prefix;  // all tokens over the shared prefix
  bool bad;     // the caller's numbers do not fit (they are clamped)
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  PagedSeq s;
  s.bad = false;
  s.prefix = b == a.prefix_at;
  if (s.prefix) {
    s.s0 = 0;
    s.nq = a.T;
    s.len = a.prefix_len;
    return s;
  }
  if (a.starts) {
    const int x = __ldg(a.starts + b), y = __ldg(a.starts + b + 1);
    s.s0 = min(max(x, 0), a.T);
    const int s1 = min(max(y, s.s0), a.T);
    s.nq = s1 - s.s0;
    s.bad = x != s.s0 || y != s1;
  } else {
    s.nq = a.each;
    s.s0 = b * s.nq;
  }
  const int n = __ldg(a.lens + b);
  s.len = min(max(n, 0), a.max_pages << a.lps);
  s.bad |= s.len != n;
  return s;
}

// Keys [lo, hi) that row token i allows (an empty range is lo >= hi).  A: PagedArgs,
// or what of them a row tile's keys depend on (for functions that are called).
struct PagedRule {
  FastDiv by_group;
  int G, mask_kind, window, least;
};
__device__ __forceinline__ PagedRule paged_rule(const PagedArgs& a) {
  return {a.by_group, a.G, a.mask_kind, a.window, a.least};
}
template <typename A>
__device__ __forceinline__ void paged_row_span(const A& a, const PagedSeq& s, int i, int& lo,
                                               int& hi) {
  lo = 0;
  hi = s.len;
  if (s.prefix) return;
  const int pos = s.len - s.nq + i;
  if (a.mask_kind != kMaskNone) hi = min(hi, pos + 1);
  if (a.mask_kind == kMaskWindow) lo = max(0, pos + 1 - a.window);
}

// A row tile's rows and keys: units [kt0, kt0 + cnt), keys [lo, hi).
struct PagedTile {
  int rows, i0, i1;  // rows in the tile, first and last token
  int lo, hi, kt0, cnt;
};

template <int RT, int UK, typename A>
__device__ __forceinline__ PagedTile paged_tile(const A& a, const PagedSeq& s, int rt) {
  PagedTile t;
  const int r0 = rt * RT, all = s.nq * a.G;
  t.rows = min(RT, all - r0);
  t.i0 = div_by(r0, a.by_group);
  t.i1 = div_by(r0 + t.rows - 1, a.by_group);
  int x;
  paged_row_span(a, s, t.i0, t.lo, x);
  paged_row_span(a, s, t.i1, x, t.hi);
  if (t.hi <= t.lo) t.hi = t.lo = 0;
  t.kt0 = static_cast<unsigned>(t.lo) / UK;
  t.cnt = max(1, static_cast<int>((static_cast<unsigned>(t.hi) + UK - 1) / UK) - t.kt0);  // a tile without keys still writes its rows
  return t;
}

// n / d for n >= 0: a fixed divisor's fast form wherever n fits 31 bits.
__device__ __forceinline__ long long paged_div(long long n, const FastDiv& d) {
  return (n >> 31) == 0 ? div_by(static_cast<int>(n), d) : static_cast<long long>(static_cast<unsigned long long>(n) / d.d);
}
// n / d for n >= 0, d > 0: in 32 bits wherever they fit.
__device__ __forceinline__ long long paged_div(long long n, long long d) {
  if (((n | d) >> 32) == 0) return static_cast<unsigned>(n) / static_cast<unsigned>(d);
  return static_cast<long long>(static_cast<unsigned long long>(n) / static_cast<unsigned long long>(d));
}

__device__ __forceinline__ long long round_up(long long x, int to) { return (x + to - 1) & -static_cast<long long>(to); }
// Units of a run, W.  A long run may begin inside a tile's rounded end; rounding it up too left
// workers without any (24 rows over 3200 keys, 4 x 16 heads of 112 fp32 columns, 21 units a run:
// 113 us, 102 without).
constexpr int kRunLong = 2;
__device__ __forceinline__ long long run_units(const PagedArgs& a, long long total) {
  const long long n = max(1ll, paged_div(total + a.runs - 1, a.by_runs));
  return n > kRunLong * a.least ? n : round_up(n, a.least);
}

// A place in the line of units.
struct PagedWalk {
  long long u, end;   // next unit, the run's end
  int b, h, rt, rem;  // of unit u: sequence, key head, row tile, unit in the tile
  PagedSeq s;
  PagedTile t;
  int tiles;  // row tiles of (b, h)
};

// Units of row tile rt, and of the tiles [first, end) of one (b, h).
template <int RT, int UK, typename A>
__device__ __forceinline__ int paged_tile_units(const A& a, const PagedSeq& s, int rt) {
  return static_cast<int>(round_up(paged_tile<RT, UK>(a, s, rt).cnt, a.least));
}
template <int RT, int UK, typename A>
__device__ __forceinline__ long long paged_tiles_units(const A& a, const PagedSeq& s, int first, int end) {
  long long u = 0;
#pragma unroll 1
  for (int rt = first; rt < end; ++rt) u += paged_tile_units<RT, UK>(a, s, rt);
  return u;
}
// Whether all row tiles have the same keys.
template <typename A>
__device__ __forceinline__ bool paged_flat(const A& a, const PagedSeq& s) {
  return s.prefix || a.mask_kind == kMaskNone;
}
__device__ __forceinline__ long long sum_over_lanes_upto(long long x) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Every worker finds the start of its run in the line by itself, before its first copy.  A
// sequence may have as many row tiles as tokens and more: above kFewTiles a warp's lanes share
// them out, and where all tiles have the same keys one is enough.  (One lane over all tiles: 65536
// fp32 tokens of 4 heads over 64 keys each 2.4 ms, now 0.15; 65536 of 8 heads over a window of 128
// 5.2 ms, now 0.70.)  That part is two functions, out of the way of other launches: inlined, they
// cost the tall tiles behind a prefix 1.5 of 29 us in instruction fetches.
constexpr int kFewTiles = 32;

// Units of each lane's sequence of `tiles` row tiles where these are many, by a whole warp.
template <int RT, int UK>
__device__ __noinline__ long long paged_many_units(const PagedRule a, int nq, int len, bool prefix, int tiles) {
  const int lane = threadIdx.x & 31;
  const PagedSeq s{0, nq, len, prefix, false};
  const bool flat = paged_flat(a, s);
  long long u = flat ? static_cast<long long>(tiles) * paged_tile_units<RT, UK>(a, s, 0) : 0;
#pragma unroll 1
  for (unsigned todo = __ballot_sync(0xFFFFFFFFu, !flat && tiles > kFewTiles); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1;
    PagedSeq of{0, 0, 0, false, false};
    of.nq = __shfl_sync(0xFFFFFFFFu, nq, who);
    of.len = __shfl_sync(0xFFFFFFFFu, len, who);
    const int n = __shfl_sync(0xFFFFFFFFu, tiles, who), per = (n + 31) / 32;
    long long sum = paged_tiles_units<RT, UK>(a, of, min(lane * per, n), min(lane * per + per, n));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    if (lane == who) u = sum;
  }
  return u;
}
// Units of each lane's sequence (nq = 0: none), by a whole warp.
template <int RT, int UK>
__device__ __forceinline__ long long paged_units(const PagedArgs& a, const PagedSeq& s) {
  const int tiles = (s.nq * a.G + RT - 1) / RT;
  const bool many = tiles > kFewTiles;
  long long u = paged_tiles_units<RT, UK>(a, s, 0, many ? 0 : tiles);
  if (__any_sync(0xFFFFFFFFu, many)) {
    const long long x = paged_many_units<RT, UK>(paged_rule(a), s.nq, s.len, s.prefix, tiles);
    if (many) u = x;
  }
  return u * a.Hk;
}

// All threads of a CTA: `pre` (shared, kPagedSums words) receives the number
// of units before each sequence.  Status bits that the caller's numbers raise go to
// `bits` (of CTA 0).
template <int RT, int UK, int NT>
__device__ __forceinline__ void paged_scan(const PagedArgs& a, long long* pre, long long* scan,
                                           unsigned& bits) {
  const int tid = threadIdx.x;
  const int per = (a.B + NT - 1) / NT;
  long long mine = 0;
  bool bad = false;
#pragma unroll 1
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    PagedSeq s{0, 0, 0, false, false};
    if (b < a.B) s = paged_seq(a, b);
    bad |= s.bad;
    mine += paged_units<RT, UK>(a, s);  // by the whole warp
    if (b < a.B) pre[b + 1] = mine;
  }
  // Exclusive sum of `mine` over the threads.
  const int lane = tid & 31, warp = tid >> 5;
  const long long inc = sum_over_lanes_upto(mine);
  if (lane == 31) scan[warp] = inc;
  const int any_bad = __syncthreads_or(bad);
  if (blockIdx.x == 0) {
    if (any_bad) bits |= kStatusBadPage;
    if (a.info && tid == 0 && a.prefix_at != 0) *a.sane = !any_bad;
  }
  long long before = inc - mine;
#pragma unroll 1
  for (int k = 0; k < warp; ++k) before += scan[k];
#pragma unroll 1
  for (int k = 0; k < per; ++k) {
    const int b = tid * per + k;
    if (b >= a.B) break;
    pre[b + 1] += before;
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
}

// The row tile that holds unit `rem` of the `left` tiles of one (b, h), and the unit in it, by a
// whole warp whose lanes agree on them.
struct PagedTileUnit {
  int rt;
  long long rem;
};
template <int RT, int UK>
__device__ __noinline__ PagedTileUnit paged_find(const PagedRule a, int nq, int len, bool prefix, int left,
                                                 long long rem) {
  const int lane = threadIdx.x & 31;
  const PagedSeq s{0, nq, len, prefix, false};
  const int same = paged_flat(a, s) ? paged_tile_units<RT, UK>(a, s, 0) : 0;
  int rt = 0;
#pragma unroll 1
  while (left > 1) {  // it is in [rt, rt + left): each lane sums a share of them
    const int per = (left + 31) / 32;
    const int first = min(lane * per, left), end = min(lane * per + per, left);
    const long long mine = same ? static_cast<long long>(end - first) * same
                                : paged_tiles_units<RT, UK>(a, s, rt + first, rt + end);
    const long long upto = sum_over_lanes_upto(mine);
    const unsigned behind = __ballot_sync(0xFFFFFFFFu, rem < upto);
    const int who = min(behind ? __ffs(behind) - 1 : 31, (left - 1) / per);
    rem -= __shfl_sync(0xFFFFFFFFu, upto - mine, who);
    rt += who * per;
    left = min(per, left - who * per);
  }
  return {rt, rem};
}
// w at unit `local` of the `units` of its sequence, by a whole warp whose lanes agree on them.
template <int RT, int UK>
__device__ __forceinline__ void paged_enter(const PagedArgs& a, PagedWalk& w, long long units, long long local) {
  w.tiles = (w.s.nq * a.G + RT - 1) / RT;
  const long long per_head = paged_div(units, a.by_heads);
  w.h = static_cast<int>(paged_div(local, per_head));
  long long rem = local - w.h * per_head;
  w.rt = 0;
  if (w.tiles > kFewTiles) {
    const PagedTileUnit at = paged_find<RT, UK>(paged_rule(a), w.s.nq, w.s.len, w.s.prefix, w.tiles, rem);
    w.rt = at.rt;
    rem = at.rem;
  }
  w.t = paged_tile<RT, UK>(a, w.s, w.rt);
  for (long long n; rem >= (n = round_up(w.t.cnt, a.least)) && w.rt + 1 < w.tiles;) {
    rem -= n;
    w.t = paged_tile<RT, UK>(a, w.s, ++w.rt);
  }
  w.rem = static_cast<int>(rem);
}

// Run r's first unit; false when it has none.
template <int RT, int UK>
__device__ __forceinline__ bool paged_begin(const PagedArgs& a, const long long* pre, int r, PagedWalk& w) {
  const long long total = pre[a.B];
  const long long n = run_units(a, total);
  w.u = n * r;
  w.end = min(total, w.u + n);
  if (w.u >= w.end) return false;
  int b0 = 0, b1 = a.B;  // pre[b0] <= u < pre[b1]
#pragma unroll 1
  while (b1 - b0 > 1) {
    const int mid = (b0 + b1) >> 1;
    if (pre[mid] <= w.u) b0 = mid;
    else b1 = mid;
  }
  w.b = b0;
  w.s = paged_seq(a, w.b);
  paged_enter<RT, UK>(a, w, pre[b0 + 1] - pre[b0], w.u - pre[b0]);
  return true;
}

// The same for a batch of at most 32 sequences, by one warp without the CTA's sums: lane b
// looks at sequence b.  `total` receives the units of the line.
template <int RT, int UK>
__device__ __forceinline__ bool paged_begin_warp(const PagedArgs& a, int r, PagedWalk& w, long long& total,
                                                 unsigned& bits) {
  const int lane = threadIdx.x & 31;
  PagedSeq s{0, 0, 0, false, false};
  if (lane < a.B) s = paged_seq(a, lane);
  long long units = paged_units<RT, UK>(a, s);
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    const bool any_bad = __any_sync(0xFFFFFFFFu, s.bad);
    if (any_bad) bits |= kStatusBadPage;
    if (a.info && lane == 0 && a.prefix_at != 0) *a.sane = !any_bad;
  }
  const long long upto = sum_over_lanes_upto(units);
  total = __shfl_sync(0xFFFFFFFFu, upto, 31);
  const long long n = run_units(a, total);
  w.u = n * r;
  w.end = min(total, w.u + n);
  if (w.u >= w.end) return false;
  w.b = __ffs(__ballot_sync(0xFFFFFFFFu, upto - units <= w.u && w.u < upto)) - 1;
  w.s.s0 = __shfl_sync(0xFFFFFFFFu, s.s0, w.b);
  w.s.nq = __shfl_sync(0xFFFFFFFFu, s.nq, w.b);
  w.s.len = __shfl_sync(0xFFFFFFFFu, s.len, w.b);
  w.s.prefix = w.b == a.prefix_at;
  w.s.bad = false;
  units = __shfl_sync(0xFFFFFFFFu, units, w.b);
  paged_enter<RT, UK>(a, w, units, w.u - __shfl_sync(0xFFFFFFFFu, upto, w.b) + units);
  return true;
}

// Past the segment that starts at w.u; false at the run's end.
template <int RT, int UK>
__device__ __forceinline__ bool paged_next(const PagedArgs& a, PagedWalk& w) {
  w.u += round_up(w.t.cnt, a.least) - w.rem;
  if (w.u >= w.end) return false;
  w.rem = 0;
  if (++w.rt == w.tiles) {
    w.rt = 0;
    if (++w.h == a.Hk) {
      w.h = 0;
#pragma unroll 1
      do {  // a sequence without tokens has no units
        ++w.b;
        w.s = paged_seq(a, w.b);
      } while (w.s.nq == 0);
      w.tiles = (w.s.nq * a.G + RT - 1) / RT;
    }
  }
  w.t = paged_tile<RT, UK>(a, w.s, w.rt);
  return true;
}

// Units of the segment that starts at w.u (0: only what the tile was rounded up by), and
// the keys they stand for.
template <int UK>
__device__ __forceinline__ int paged_segment(const PagedWalk& w, int& j0, int& j1) {
  const int n = max(0, static_cast<int>(min(static_cast<long long>(w.t.cnt - w.rem), w.end - w.u)));
  const int kt = w.t.kt0 + w.rem;
  j0 = max(w.t.lo, kt * UK);
  j1 = min(w.t.hi, (kt + n) * UK);
  return n;
}

// Where run r's present segment of n units goes: its slot, or -1 when the segment holds
// the whole row tile; where the tile starts here, the runs that hold a piece of it (0: all
// of it).  The thread `one` describes such a tile to the merge.
struct PagedPlace {
  int slot, parts;
};
template <int RT>
__device__ __forceinline__ PagedPlace paged_place(const PagedArgs& a, long long total, const PagedWalk& w, int n,
                                                  int r, bool one) {
  if (w.rem > 0) return {2 * r, -1};
  if (n == w.t.cnt) return {-1, 0};
  const int last = static_cast<int>(paged_div(w.u + w.t.cnt - 1, run_units(a, total)));
  if (one)
    a.desc[r] = make_int4(w.rt * RT, w.s.nq * a.G, w.s.s0,
                          static_cast<int>((static_cast<unsigned>(w.h) << 16) |
                                           static_cast<unsigned>(last - r + 1)));
  return {2 * r + 1, last - r + 1};
}

__device__ __forceinline__ const int* paged_table(const PagedArgs& a, int b) {
  return b == a.prefix_at ? a.prefix_table : a.table + static_cast<size_t>(b) * a.max_pages;
}

// Programmatic dependent launch.  Every kernel here is launched early: its CTAs may start
// while its predecessor in the stream runs, and wait, before they touch global memory,
// until that is complete; only then do they let their own successor start, so that a
// kernel that has not waited itself (a.second) still finds all that came before the launch
// in front of it.  Between calls this hides the launches, not the work.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Row r of key head h as an index into [T][heads], the prefix's behind the sequences'.
__device__ __forceinline__ size_t paged_out_row(const PagedArgs& a, int s0, int h, int r, bool prefix) {
  const int i = div_by(r, a.by_group);
  return static_cast<size_t>(s0 + i + (prefix ? a.T : 0)) * (a.Hk * a.G) + h * a.G + (r - i * a.G);
}

// A finished row (m in the exp2 domain, l): Y = z / l, and L.  Empty rows: 0 and -inf.
struct PagedScale {
  float fz, L;
};
__device__ __forceinline__ PagedScale paged_finish(float m, float l) {
  if (!(l > 0.f) && l == l) return {0.f, -INFINITY};  // a NaN score stays one
  return {1.f / l, (m + log2f(l)) * kLn2};
}

__device__ __forceinline__ void paged_store(const PagedArgs& a, size_t row, int col, float y) {
  const size_t at = row * a.v + col;
  if (a.Yf) a.Yf[at] = y;
  else if (a.dtype == kF32) static_cast<float*>(a.Y)[at] = y;
  else static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(y);
}
// Four columns into Y.
__device__ __forceinline__ void paged_store4(const PagedArgs& a, size_t row, int col, const float4& y) {
  const size_t at = row * a.v + col;
  if (a.dtype == kF32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + at) = y;
  } else {
    const __nv_bfloat162 p = __floats2bfloat162_rn(y.x, y.y), q = __floats2bfloat162_rn(y.z, y.w);
    uint2 raw;
    raw.x = *reinterpret_cast<const uint32_t*>(&p);
    raw.y = *reinterpret_cast<const uint32_t*>(&q);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.Y) + at) = raw;
  }
}

// The CTA's status bits, at its end (`joined`: a word in shared memory, zero since an
// earlier barrier).
__device__ __forceinline__ void paged_end(const PagedArgs& a, unsigned bits, unsigned* joined) {
  if (bits) atomicOr(joined, bits);
  __syncthreads();
  if (threadIdx.x == 0) a.flags[blockIdx.x] = *joined;
}

// The row of page table entries of sequence b, and the row of a key in the
// pool (pages [num_pages][Hk][page_size][width]); -1 for a page outside it.
__device__ __forceinline__ long long paged_key_row(const PagedArgs& a, const int* trow, int h, int key) {
  const int page = __ldg(trow + (key >> a.lps));
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) return -1;
  return ((static_cast<long long>(page) * a.Hk + h) << a.lps) + (key & ((1 << a.lps) - 1));
}

// Allows a kernel its dynamic shared memory, once for each device.
template <auto kernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};  // a bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}

// A launch that may start before its predecessor in the stream is complete.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         Args... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Host side: rows of a tile, CTAs and workers of the launch, the least multiple of units.
struct PagedKernel {
  int rt, ctas, workers, least;
};
PagedKernel paged_simt_kernel(bool one_row);
cudaError_t launch_paged_simt(const PagedArgs& a, bool one_row, cudaStream_t s);
bool paged_mma_shape(int d, int v);
PagedKernel paged_mma_kernel_of(int dtype, int d, int v, int rows);  // rows: 8 or 16
cudaError_t launch_paged_mma(const PagedArgs& a, int rows, cudaStream_t s);
bool paged_tc_supported(const PagedArgs& a);
PagedKernel paged_tc_kernel_of();
cudaError_t launch_paged_tc(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedArgs& a, int rt, cudaStream_t s);
// own, prefix: the launches that hold the two sets (the same one, or two), with their tiles' rows.
cudaError_t launch_paged_join(const PagedArgs& own, int own_rt, const PagedArgs& prefix, int prefix_rt,
                              cudaStream_t s);

struct AppendArgs {
  const void* q;  // may be null
  const void* k;
  const void* v;
  const int* starts;
  const int* table;
  const int* lens;
  const float* inv_freq;
  int pairs, interleaved, pos_offset;
  int B, T, H, Hk, d, vw, dtype, lps, num_pages, max_pages;
  long long qs, ks, vs;
  void* q_out;
  void* kp;
  void* vp;
  unsigned* status;
  // Set by the launcher: units of a row of q or k, accesses of a row of v, warps that
  // share a token; T / B.
  FastDiv by_units, by_vch, by_shares;
  int each;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);

}  // namespace exattn
