// Paged attention without tensor cores, for every width and type the library
// takes, and the merge of the row tiles that several CTAs share.
//
// paged_simt_kernel: kW warps share a segment's keys.  A group of G lanes
// covers one key row in 16-byte pieces (CPL a lane), so a warp-wide load reads
// 32 / G rows; scores are partial dot products summed inside the group, and
// each group keeps the running maximum, sum and output of NQ rows in registers
// (the running-max recurrence of "txf-modern-flash-attention", Hints, in the
// exp2 domain).  Groups, then warps, are joined with the star rule.  Keys and
// values are read straight into registers, so nothing outside a segment's keys
// is ever read or multiplied: what stale rows of a page hold does not matter.  Scores are
// products of exact bf16 or fp32 values summed in fp32.  A CTA is a worker; up to four rows
// share each read.  Bound by issue: every key costs 2 (d + v) multiply-adds a row and the
// shuffles of a group.  Heads of 256 columns, 537 MB of keys and values: one row 97 us in bf16
// (5.5 TB/s), 84 in fp32 (6.4), four rows 246 in bf16.  One row of 128 columns: 333 us for 2.1
// GB against the tensor cores' 325, which take eight rows in that time.
#include "paged.cuh"

namespace exattn {
namespace {

constexpr int kW = 4;
constexpr int kUnit = 64;  // keys of a unit of work
// CTAs of an SM, all at once.  With registers as the compiler likes (2 or 3 CTAs of 4) 151 us for
// one row of 256 bf16 columns, 272 for four; with three 111 and 246, with four 97 and 252.
template <int NQ>
constexpr int kCtas = NQ == 1 ? 4 : 3;

__device__ __forceinline__ float pexp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T> struct Row16;
template <> struct Row16<float> {
  static constexpr int E = 4;
  __device__ static void unpack(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
};
template <> struct Row16<__nv_bfloat16> {
  static constexpr int E = 8;
  __device__ static void unpack(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};

__device__ __forceinline__ uint4 ldg_once16(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

template <typename T, int G, int CPL, int NQ>
__global__ void __launch_bounds__(32 * kW, kCtas<NQ>) paged_simt_kernel(const PagedArgs a) {
  constexpr int E = Row16<T>::E;
  constexpr int KPW = 32 / G;
  constexpr int U = (NQ == 1 ? 8 : 4) / CPL;  // key steps in flight
  constexpr int STEP = KPW * U;
  constexpr int W = CPL * E;
  __shared__ long long pre[kPagedSums], scan[kW];
  __shared__ float red_m[kW][NQ], red_l[kW][NQ];
  __shared__ __align__(16) float red_z[kW][NQ][256];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane / G, gl = lane % G;
  const int d = a.d, v = a.v;
  const int kch = d / E, vch = v / E;
  const T* Q = static_cast<const T*>(a.Q);
  const T* Kp = static_cast<const T*>(a.Kp);
  const T* Vp = static_cast<const T*>(a.Vp);
  unsigned bits = 0;
  __shared__ unsigned joined;
  if (!a.second) wait_for_previous();
  let_next_start();
  if (threadIdx.x == 0) {
    a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    joined = 0;
  }
  PagedWalk w;
  paged_scan<NQ, kUnit, 32 * kW>(a, pre, scan, bits);
  bool more = paged_begin<NQ, kUnit>(a, pre, blockIdx.x, w);
  while (more) {
    int j0, j1;
    const int n = paged_segment<kUnit>(w, j0, j1);
    const int r0 = w.rt * NQ, rows = w.t.rows;
    const int* trow = paged_table(a, w.b);

    // Rows of Q with scale * log2(e) folded in, and the keys that each allows.
    float qf[NQ][W];
    int lo[NQ], hi[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = r0 + (q < rows ? q : 0), i = div_by(r, a.by_group);
      paged_row_span(a, w.s, i, lo[q], hi[q]);
      if (q < rows && lo[q] >= hi[q] && w.rem == 0 && !a.info) bits |= kStatusEmptyRow;
      const T* qr = Q + (w.s.s0 + i) * a.q_stride + (w.h * a.G + r - i * a.G) * d;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int pc = gl + c * G;
        float f[E];
        if (pc < kch) {
          Row16<T>::unpack(*reinterpret_cast<const uint4*>(qr + pc * E), f);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) qf[q][c * E + e] = f[e] * a.sl2;
      }
    }
    float m[NQ], l[NQ], z[NQ][W];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
#pragma unroll
      for (int e = 0; e < W; ++e) z[q][e] = 0.f;
    }

    for (int jb = j0 + warp * STEP; jb < j1; jb += kW * STEP) {
      uint4 kr[U][CPL], vr[U][CPL];
      bool have[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int key = jb + u * KPW + g;
        long long row = -1;
        if (key < j1) {
          row = paged_key_row(a, trow, w.h, key);
          if (row < 0) bits |= kStatusBadPage;
        }
        have[u] = row >= 0;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int pc = gl + c * G;
          kr[u][c] = have[u] && pc < kch ? ldg_once16(Kp + row * d + pc * E) : make_uint4(0u, 0u, 0u, 0u);
          vr[u][c] = have[u] && pc < vch ? ldg_once16(Vp + row * v + pc * E) : make_uint4(0u, 0u, 0u, 0u);
        }
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q >= rows) break;
        float s[U];
        bool ok[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            float f[E];
            Row16<T>::unpack(kr[u][c], f);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              acc0 = fmaf(qf[q][c * E + e], f[e], acc0);
              acc1 = fmaf(qf[q][c * E + e + 1], f[e + 1], acc1);
            }
          }
          float part = acc0 + acc1;
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, o);
          const int key = jb + u * KPW + g;
          ok[u] = have[u] && key >= lo[q] && key < hi[q];
          s[u] = ok[u] ? part : -INFINITY;
        }
        float mx = m[q];
#pragma unroll
        for (int u = 0; u < U; ++u) mx = fmaxf(mx, s[u]);
        const float ref = mx == -INFINITY ? 0.f : mx;
        const float alpha = pexp2(m[q] - ref);
        float psum = 0.f;
#pragma unroll
        for (int e = 0; e < W; ++e) z[q][e] *= alpha;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float p = pexp2(s[u] - ref);
          psum += p;
          if (ok[u]) {  // a key that this row does not allow leaves no trace, whatever its value
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
              float f[E];
              Row16<T>::unpack(vr[u][c], f);
#pragma unroll
              for (int e = 0; e < E; ++e) z[q][c * E + e] = fmaf(p, f[e], z[q][c * E + e]);
            }
          }
        }
        l[q] = l[q] * alpha + psum;
        m[q] = mx;
      }
    }

    // Groups of the warp, then warps.
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      float M = m[q];
#pragma unroll
      for (int o = G; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
      const float f = M == -INFINITY ? 0.f : pexp2(m[q] - M);
      float lq = l[q] * f;
#pragma unroll
      for (int o = G; o < 32; o <<= 1) lq += __shfl_xor_sync(0xFFFFFFFFu, lq, o);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        float ze = z[q][e] * f;
#pragma unroll
        for (int o = G; o < 32; o <<= 1) ze += __shfl_xor_sync(0xFFFFFFFFu, ze, o);
        z[q][e] = ze;
      }
      if (q < rows && lane < G) {
        if (lane == 0) {
          red_m[warp][q] = M;
          red_l[warp][q] = lq;
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int pc = gl + c * G;
          if (pc < vch)
#pragma unroll
            for (int e = 0; e < E; ++e) red_z[warp][q][pc * E + e] = z[q][c * E + e];
        }
      }
    }
    const PagedPlace place = paged_place<NQ>(a, pre[a.B], w, n, blockIdx.x, threadIdx.x == 0);
    const int slot = place.slot;
    __syncthreads();
    for (int idx = threadIdx.x; idx < rows * v; idx += 32 * kW) {
      const int q = idx / v, col = idx - q * v;
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kW; ++k) M = fmaxf(M, red_m[k][q]);
      // Also where no maximum was found: sums of NaN scores alone are NaN and stay it.
      const float ref = M == -INFINITY ? 0.f : M;
      float zc = 0.f, lq = 0.f;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const float f = pexp2(red_m[k][q] - ref);
        zc = fmaf(f, red_z[k][q][col], zc);
        lq = fmaf(f, red_l[k][q], lq);
      }
      const size_t out = paged_out_row(a, w.s.s0, w.h, r0 + q, w.s.prefix);
      if (a.info && col == 0 && place.parts >= 0) a.info[out] = make_int2(blockIdx.x, place.parts);
      if (slot < 0) {
        const PagedScale f = paged_finish(M, lq);
        paged_store(a, out, col, zc * f.fz);
        if (col == 0) a.L[out] = f.L;
      } else {
        const size_t row = static_cast<size_t>(slot) * NQ + q;
        a.pz[row * v + col] = zc;
        if (col == 0) {
          a.pm[row] = M;
          a.pl[row] = lq;
        }
      }
    }
    more = paged_next<NQ, kUnit>(a, w);
    __syncthreads();  // the joined rows are read before the next segment's
  }
  if (a.second) wait_for_previous();
  paged_end(a, bits, &joined);
}

// The star merge of the row tiles that one run starts and others end.  Piece 0 of run
// c's tile is in slot 2c + 1, piece k > 0 in slot 2 (c + k).  Each kernel is
// launched early and waits for the attention kernel at its start; CTA (0, 0) also joins
// the status bits of every CTA of the attention launches.  Bound by latency where few tiles
// are shared (the launch and three dependent loads, 2 to 3 us behind the attention kernel), by
// the summaries' traffic in the L2 cache where most are: 14 us for the 40 MB that 152 runs of
// 256-row tiles leave, 8 for 8 tiles of 152 runs each.
//
// A row's state while its pieces come in, four at a time so that their loads overlap.
template <int N>
struct Gather {
  float m = -INFINITY, l = 0.f;
  float4 z[N];
  __device__ __forceinline__ Gather() {
#pragma unroll
    for (int x = 0; x < N; ++x) z[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // Pieces first, first + step, ... below `parts`; row(k): piece k's index into pm and pl,
  // at(k, x): its x-th four columns, or null.
  template <typename A, typename R, typename F>
  __device__ __forceinline__ void take(const A& a, int first, int step, int parts, R row, F at) {
#pragma unroll 1
    for (int k0 = first; k0 < parts; k0 += 4 * step) {
      float pm[4], pl[4];
      float4 p[4][N];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + j * step;
        const bool on = k < parts;
        pm[j] = on ? a.pm[row(k)] : -INFINITY;
        pl[j] = on ? a.pl[row(k)] : 0.f;
#pragma unroll
        for (int x = 0; x < N; ++x) {
          const float4* from = on ? at(k, x) : nullptr;
          p[j][x] = from ? *from : make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      const float top = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])), m);
      const float ref = top == -INFINITY ? 0.f : top;
      const float f0 = pexp2(m - ref);
      m = top;
      l *= f0;
#pragma unroll
      for (int x = 0; x < N; ++x) z[x] = make_float4(z[x].x * f0, z[x].y * f0, z[x].z * f0, z[x].w * f0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = pexp2(pm[j] - ref);
        l = fmaf(f, pl[j], l);
#pragma unroll
        for (int x = 0; x < N; ++x)
          z[x] = make_float4(fmaf(f, p[j][x].x, z[x].x), fmaf(f, p[j][x].y, z[x].y), fmaf(f, p[j][x].z, z[x].z),
                             fmaf(f, p[j][x].w, z[x].w));
      }
    }
  }
};

__device__ __forceinline__ float4 scaled(const float4& z, float f) {
  return make_float4(z.x * f, z.y * f, z.z * f, z.w * f);
}

__device__ __forceinline__ void join_status(const PagedArgs& a) {
  if (!a.status || blockIdx.x != 0 || blockIdx.y != 0) return;
  __shared__ unsigned joined;
  if (threadIdx.x == 0) joined = 0;
  __syncthreads();
  unsigned bits = 0;
  for (int k = threadIdx.x; k < a.n_flags; k += blockDim.x) bits |= a.flags0[k];
  if (bits) atomicOr(&joined, bits);
  __syncthreads();
  if (threadIdx.x == 0) *a.status = joined;
}

// Tiles of up to 16 rows, summaries row by row ([rows][v]).  kSpread: CTA (x, y) takes
// row y of the tiles of every gridDim.x-th run from x on (at most 32), its warps sharing a row's
// pieces; else a warp takes a row of each.  (A CTA for every run and row cost 2 us a
// thousand CTAs, most of them without a tile.)
constexpr int kMergeW = 16;

// N: times 128 columns.
template <bool kSpread, int N>
__global__ void __launch_bounds__(32 * kMergeW) paged_merge_kernel(const PagedArgs a, int rt) {
  __shared__ float red_m[kMergeW], red_l[kMergeW];
  __shared__ __align__(16) float red_z[kSpread ? kMergeW : 1][128 * N];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, v = a.v;
  wait_for_previous();
  let_next_start();
  // Runs far apart: in a small launch only the first ones have tiles.
  const int cl = blockIdx.x + lane * gridDim.x;
  int4 mine = make_int4(0, 0, 0, 0);
  if (cl < a.runs) mine = a.desc[cl];
  for (unsigned todo = __ballot_sync(0xFFFFFFFFu, mine.w != 0); todo; todo &= todo - 1) {
    const int who = __ffs(todo) - 1, c = blockIdx.x + who * gridDim.x;
    const int q = kSpread ? blockIdx.y : warp;
    const int r = __shfl_sync(0xFFFFFFFFu, mine.x, who) + q, all = __shfl_sync(0xFFFFFFFFu, mine.y, who),
              s0 = __shfl_sync(0xFFFFFFFFu, mine.z, who), hp = __shfl_sync(0xFFFFFFFFu, mine.w, who);
    const int parts = hp & 0xFFFF;
    if (q >= rt || r >= all) continue;  // kSpread: all warps alike
    const size_t row = paged_out_row(a, s0, static_cast<unsigned>(hp) >> 16, r, false);
    Gather<N> x;
    auto at = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)) * rt + q; };
    x.take(a, kSpread ? warp : 0, kSpread ? kMergeW : 1, parts, at, [&](int k, int y) -> const float4* {
      const int col = 4 * lane + 128 * y;
      return col < v ? reinterpret_cast<const float4*>(a.pz + at(k) * v + col) : nullptr;
    });
    if constexpr (kSpread) {
      if (lane == 0) {
        red_m[warp] = x.m;
        red_l[warp] = x.l;
      }
#pragma unroll
      for (int y = 0; y < N; ++y) *reinterpret_cast<float4*>(&red_z[warp][4 * lane + 128 * y]) = x.z[y];
      __syncthreads();
      const int col = threadIdx.x;
      if (col < v) {
        float M = -INFINITY, l = 0.f, z = 0.f;
#pragma unroll
        for (int k = 0; k < kMergeW; ++k) M = fmaxf(M, red_m[k]);
        const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int k = 0; k < kMergeW; ++k) {
          const float f = pexp2(red_m[k] - ref);
          l = fmaf(f, red_l[k], l);
          z = fmaf(f, red_z[k][col], z);
        }
        const PagedScale f = paged_finish(M, l);
        paged_store(a, row, col, z * f.fz);
        if (col == 0) a.L[row] = f.L;
      }
      __syncthreads();
    } else {
      const PagedScale f = paged_finish(x.m, x.l);
#pragma unroll
      for (int y = 0; y < N; ++y) {
        const int col = 4 * lane + 128 * y;
        if (col < v) paged_store4(a, row, col, scaled(x.z[y], f.fz));
      }
      if (lane == 0) a.L[row] = f.L;
    }
  }
  join_status(a);
}

// Tiles of 256 rows, summaries column by column ([v / 8][256] pieces of eight): a thread a
// row, so that loads are whole lines.  CTA (x, y) takes four columns N y .. (in fours) of
// the tiles of runs kPer x ..: N = 4, kPer = 1 where most runs start a tile that others end,
// else N = 2 and kPer = 8.
constexpr int kTall = 256;
// Four columns, number c, of row q of slot s.
__device__ __forceinline__ size_t tall_at(size_t s, int v, int c, int q) {
  return ((s * (v / 8) + c / 2) * kTall + q) * 2 + (c & 1);
}

template <int N, int kPer>
__global__ void __launch_bounds__(kTall) paged_merge_tall_kernel(const PagedArgs a) {
  const int q = threadIdx.x, n4 = a.v / 4, first = N * blockIdx.y;
  const float4* z = reinterpret_cast<const float4*>(a.pz);
  wait_for_previous();
  let_next_start();
#pragma unroll 1
  for (int c = blockIdx.x * kPer; c < min(a.runs, (static_cast<int>(blockIdx.x) + 1) * kPer); ++c) {
    const int4 t = a.desc[c];
    const int r = t.x + q;
    if (t.w == 0 || r >= t.y) continue;
    const size_t row = paged_out_row(a, t.z, static_cast<unsigned>(t.w) >> 16, r, false);
    Gather<N> x;
    auto slot = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)); };
    x.take(a, 0, 1, t.w & 0xFFFF, [&](int k) { return slot(k) * kTall + q; },
           [&](int k, int y) -> const float4* {
             return first + y < n4 ? z + tall_at(slot(k), a.v, first + y, q) : nullptr;
           });
    const PagedScale f = paged_finish(x.m, x.l);
#pragma unroll
    for (int y = 0; y < N; ++y)
      if (first + y < n4)
        paged_store4(a, row, 4 * (first + y), scaled(x.z[y], f.fz));
    if (first == 0) a.L[row] = f.L;
  }
  join_status(a);
}

// A token's row over the shared prefix and over its own keys, joined: a finished row is
// one piece (m = L log2(e), l = 1), an unfinished one as many as runs hold some of it.
// kWarps warps share a row's pieces: four where the prefix's tiles may each be spread over
// more than 16 runs (a CTA a row), else one (a CTA eight rows).  One warp's loads are four
// pieces at a time: with 4 warps in place of 1, 28 to 64 runs a tile took 33.5 us in place of
// 38.4 and 16.2 of 20.8 (whole calls, about 16,000 and 50,000 prefix keys); below 16 runs a
// tile, 59.2 us with one and 60.9 with four (64 sequences behind 16384 keys).
constexpr int kJoinRows = 8;
constexpr int kJoinSpread = 16;

struct JoinSide {
  const float* pm;
  const float* pl;
  const float* pz;
  int rt;
};

template <int N, int kWarps>
__global__ void __launch_bounds__(kWarps > 1 ? 32 * kWarps : 32 * kJoinRows)
    paged_join_kernel(const PagedArgs a, const JoinSide own, const JoinSide prefix) {
  __shared__ float red_m[kWarps], red_l[kWarps];
  __shared__ __align__(16) float red_z[kWarps][128 * N];
  const int lane = threadIdx.x & 31, v = a.v, n4 = v / 4;
  const int warp = kWarps > 1 ? threadIdx.x >> 5 : 0;
  const int heads = a.Hk * a.G;
  const int index = kWarps > 1 ? blockIdx.x : blockIdx.x * kJoinRows + (threadIdx.x >> 5);
  const size_t row = index, behind = static_cast<size_t>(a.T) * heads;
  const int tok = index / heads, head = index - tok * heads;
  wait_for_previous();
  let_next_start();
  join_status(a);
  if (tok >= a.T) return;
  // Rows of tokens that no sequence owns stay as they are.
  int s0 = 0;
  if (a.starts) {
    const int end = min(max(__ldg(a.starts + a.prefix_at), 0), a.T);
    // The owner, for the row's place in its tile (and, where q_starts is not sane, at all).
    int b = 0, b1 = a.prefix_at;
    if (*a.sane) {
      if (tok < __ldg(a.starts) || tok >= end) return;
#pragma unroll 1
      while (b1 - b > 1) {
        const int mid = (b + b1) >> 1;
        if (__ldg(a.starts + mid) <= tok) b = mid;
        else b1 = mid;
      }
      s0 = __ldg(a.starts + b);
    } else {
#pragma unroll 1
      for (; b < b1; ++b) {
        const PagedSeq s = paged_seq(a, b);
        s0 = s.s0;
        if (tok >= s0 && tok < s0 + s.nq) break;
      }
      if (b == b1) return;
    }
  } else {
    s0 = tok / a.each * a.each;
  }
  const int g = head - div_by(head, a.by_group) * a.G;
  float m = -INFINITY, l = 0.f;
  float4 z[N];
#pragma unroll
  for (int y = 0; y < N; ++y) z[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const JoinSide& of = side ? prefix : own;
    const size_t from = row + (side ? behind : 0);
    const int2 at = a.info[from];
    Gather<N> x;
    if (at.y == 0) {
      if (warp != 0) continue;
      const float4* p = reinterpret_cast<const float4*>(a.Yf + from * v);
      x.m = a.L[from] * kLog2e;
      x.l = x.m == -INFINITY ? 0.f : 1.f;
#pragma unroll
      for (int y = 0; y < N; ++y)
        if (lane + 32 * y < n4) x.z[y] = p[lane + 32 * y];
    } else {
      const int c = at.x, q = ((side ? tok : tok - s0) * a.G + g) % of.rt;
      auto slot = [&](int k) { return static_cast<size_t>(k == 0 ? 2 * c + 1 : 2 * (c + k)); };
      const float4* pz = reinterpret_cast<const float4*>(of.pz);
      x.take(of, warp, kWarps, at.y, [&](int k) { return slot(k) * of.rt + q; },
             [&](int k, int y) -> const float4* {
               const int col = lane + 32 * y;
               if (col >= n4) return nullptr;
               return of.rt == kTall ? pz + tall_at(slot(k), v, col, q) : pz + (slot(k) * of.rt + q) * n4 + col;
             });
    }
    const float top = fmaxf(m, x.m), ref = top == -INFINITY ? 0.f : top;
    const float f0 = pexp2(m - ref), f1 = pexp2(x.m - ref);
    m = top;
    l = l * f0 + x.l * f1;
#pragma unroll
    for (int y = 0; y < N; ++y)
      z[y] = make_float4(fmaf(x.z[y].x, f1, z[y].x * f0), fmaf(x.z[y].y, f1, z[y].y * f0),
                         fmaf(x.z[y].z, f1, z[y].z * f0), fmaf(x.z[y].w, f1, z[y].w * f0));
  }
  if constexpr (kWarps == 1) {
    const PagedScale f = paged_finish(m, l);
#pragma unroll
    for (int y = 0; y < N; ++y)
      if (lane + 32 * y < n4) paged_store4(a, row, 4 * (lane + 32 * y), scaled(z[y], f.fz));
    if (lane == 0) a.Lout[row] = f.L;
  } else {
    if (lane == 0) {
      red_m[warp] = m;
      red_l[warp] = l;
    }
#pragma unroll
    for (int y = 0; y < N; ++y) *reinterpret_cast<float4*>(&red_z[warp][4 * lane + 128 * y]) = z[y];
    __syncthreads();
    float M = -INFINITY, sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, red_m[k]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) sum = fmaf(pexp2(red_m[k] - ref), red_l[k], sum);
    const PagedScale f = paged_finish(M, sum);
#pragma unroll 1
    for (int col = threadIdx.x; col < v; col += 32 * kWarps) {
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) y = fmaf(pexp2(red_m[k] - ref), red_z[k][col], y);
      y *= f.fz;
      if (a.dtype == kF32) static_cast<float*>(a.Y)[row * v + col] = y;
      else static_cast<__nv_bfloat16*>(a.Y)[row * v + col] = __float2bfloat16_rn(y);
    }
    if (threadIdx.x == 0) a.Lout[row] = f.L;
  }
}

template <typename T, int G, int CPL>
cudaError_t simt_launch(const PagedArgs& a, bool one_row, cudaStream_t s) {
  auto kern = one_row ? paged_simt_kernel<T, G, CPL, 1> : paged_simt_kernel<T, G, CPL, 4>;
  before_launch(kKernPaged, s);
  const cudaError_t e = launch_early(kern, dim3(a.runs), 32 * kW, 0, s, a);
  after_launch(kKernPaged, s);
  return e;
}

}  // namespace

PagedKernel paged_simt_kernel(bool one_row) {
  const int ctas = 152 * (one_row ? kCtas<1> : kCtas<4>);
  return {one_row ? 1 : 4, ctas, ctas, 1};
}

cudaError_t launch_paged_simt(const PagedArgs& a, bool one_row, cudaStream_t s) {
  const int bytes = (a.d > a.v ? a.d : a.v) * (a.dtype == kF32 ? 4 : 2);
  if (a.dtype == kF32) {
    if (bytes <= 128) return simt_launch<float, 8, 1>(a, one_row, s);
    if (bytes <= 256) return simt_launch<float, 16, 1>(a, one_row, s);
    if (bytes <= 512) return simt_launch<float, 32, 1>(a, one_row, s);
    return simt_launch<float, 32, 2>(a, one_row, s);
  }
  if (bytes <= 128) return simt_launch<__nv_bfloat16, 8, 1>(a, one_row, s);
  if (bytes <= 256) return simt_launch<__nv_bfloat16, 16, 1>(a, one_row, s);
  return simt_launch<__nv_bfloat16, 32, 1>(a, one_row, s);
}

// Rows that a tile can have (q_starts hides how many tokens a sequence has).  Tiles that
// may be spread over more than 16 runs give a row to all of a CTA's warps: a warp alone
// takes four pieces of 512 bytes after four.
cudaError_t launch_paged_merge(const PagedArgs& a, int rt, cudaStream_t s) {
  const long long all = static_cast<long long>(a.starts ? a.T : a.each) * a.G;
  const unsigned rows = static_cast<unsigned>(all < rt ? all : rt);
  const unsigned n4 = a.v / 4, runs = a.runs;
  const long long usual = (static_cast<long long>(a.T + a.B - 1) / a.B * a.G + rt - 1) / rt;
  const long long tiles = usual * a.B * a.Hk;
  const bool spread = runs > (rt == kTall ? 8 : 16) * tiles;
  cudaError_t e;
  before_launch(kKernPagedMerge, s);
  if (rt == kTall)
    e = spread ? launch_early(paged_merge_tall_kernel<2, 8>, dim3((runs + 7) / 8, (n4 + 1) / 2), kTall, 0, s, a)
               : launch_early(paged_merge_tall_kernel<4, 1>, dim3(runs, (n4 + 3) / 4), kTall, 0, s, a);
  else  // 61: a prime number, so that tiles that start at every so manyth run do not meet in one CTA
    e = spread ? launch_early(a.v <= 128 ? paged_merge_kernel<true, 1> : paged_merge_kernel<true, 2>, dim3(61, rows),
                              32 * kMergeW, 0, s, a, rt)
               : launch_early(a.v <= 128 ? paged_merge_kernel<false, 1> : paged_merge_kernel<false, 2>,
                              dim3((runs + 1) / 2), 32 * kMergeW, 0, s, a, rt);
  after_launch(kKernPagedMerge, s);
  return e;
}

cudaError_t launch_paged_join(const PagedArgs& own, int own_rt, const PagedArgs& prefix, int prefix_rt,
                              cudaStream_t s) {
  const JoinSide o{own.pm, own.pl, own.pz, own_rt}, p{prefix.pm, prefix.pl, prefix.pz, prefix_rt};
  before_launch(kKernPagedMerge, s);
  const int rows = own.T * own.Hk * own.G;
  const long long tiles = (static_cast<long long>(own.T) * own.G + prefix_rt - 1) / prefix_rt * own.Hk;
  const bool spread = prefix.runs > kJoinSpread * tiles;
  const dim3 grid(spread ? rows : (rows + kJoinRows - 1) / kJoinRows);
  const int threads = 32 * (spread ? 4 : kJoinRows);
  const cudaError_t e =
      own.v <= 128 ? launch_early(spread ? paged_join_kernel<1, 4> : paged_join_kernel<1, 1>, grid, threads, 0, s, own, o, p)
                   : launch_early(spread ? paged_join_kernel<2, 4> : paged_join_kernel<2, 1>, grid, threads, 0, s, own, o, p);
  after_launch(kKernPagedMerge, s);
  return e;
}

}  // namespace exattn
