// Paged attention for few rows to a key head (a decode step, a few guessed
// tokens), widths up to 128: bound by reading K and V once.
//
// A row tile is 16 rows, the rows of one tensor-core tile: the rows of a key head's
// whole group share each key that is read.  A worker is a warp.  It streams the key
// tiles of its units (16 keys in bf16, 8 in fp32: 8 KB of K and V at width 128)
// through a ring of kStages tiles of its own in shared memory (asynchronous 16-byte
// copies, row by row through the page table), and holds maximum, sum and output of
// its rows in registers.  No barrier and no other warp is involved between a
// segment's first copy and its last store.  The copies run ahead of the products by
// kStages - 1 tiles, over the ends of segments too, so that short sequences stream as
// long ones do; 8 warps to an SM keep 128 KB in flight.
//
// bf16: m16n8k16.  p enters P.V as the sum of two bf16 values, its rounding and what
// the rounding left out (2^-17 of p remains): the products are free beside the
// loads, and Y is then rounded once, on its way out.
// fp32: m16n8k8 on tf32 parts, x = hi + lo, three products for one (lo lo, 2^-22 of
// the product, is left out; lo is cut to tf32, 2^-21 of x).
// The reference point of the exponentials moves only when a row's maximum passes
// it by more than 2^8, so p <= 2^8.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

using tc::ex2;
using tc::ld_shared_v4;
using tc::pack_bf16x2;
using tc::smem_u32;
using tc::tf32_hi;

constexpr int kW = 4;
constexpr int kRows = 16;
constexpr int kCtas = 2 * 152;
constexpr float kRescale = 8.f;

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma8(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The tf32 parts of x, as operands.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  const float h = tf32_hi(x);
  hi = __float_as_uint(h);
  lo = __float_as_uint(x - h);
}

// A worker's rows over a segment: maximum (the reference point), sum over the
// thread's keys, output.  Thread (g, t) = (lane / 4, lane % 4) holds rows g and g + 8.
template <int D>
struct RowState {
  float m[2], l[2], o[D / 8][4];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;
  }
  // The reference point of rows whose tile maximum is top[].
  __device__ __forceinline__ void refer(const float (&top)[2]) {
    const bool move = top[0] > m[0] + kRescale || top[1] > m[1] + kRescale;
    if (!__any_sync(0xFFFFFFFFu, move)) return;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float to = fmaxf(m[x], top[x]);
      const float f = m[x] == -INFINITY ? 0.f : ex2(m[x] - to);
      m[x] = to;
      l[x] *= f;
#pragma unroll
      for (int y = 0; y < D / 8; ++y) {
        o[y][2 * x] *= f;
        o[y][2 * x + 1] *= f;
      }
    }
  }
};

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
}

// The keys that a thread's two rows allow, and those that every row of the tile does.
struct Spans {
  int lo[2], hi[2], all_lo, all_hi;
};

// What the two types differ in: the tile, its place in shared memory, Q's
// fragments, and one tile's products.
template <typename T, int D> struct Step;

template <int D>
struct Step<__nv_bfloat16, D> {
  static constexpr int kTile = 16, kCh = D / 8, kStages = D == 128 ? 3 : 6;
  uint32_t qa[D / 16][4];
  static __device__ __forceinline__ int kpiece(int r, int c) { return c ^ (r & 7); }
  static __device__ __forceinline__ int vpiece(int r, int c) { return c ^ (r & 7); }
  __device__ __forceinline__ void load_q(const __nv_bfloat16* (&row)[2], const bool (&on)[2], int t, int d) {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int c = ks * 16 + y * 8 + 2 * t;
          qa[ks][x + 2 * y] = on[x] && c < d ? *reinterpret_cast<const uint32_t*>(row[x] + c) : 0u;
        }
  }
  __device__ __forceinline__ void tile(RowState<D>& st, uint32_t kt, uint32_t vt, unsigned have, int key0,
                                       const Spans& sp, float sl2) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const int r = ((lane >> 4) << 3) + (lane & 7), c = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t b[4];
        ldm4(b, kt + r * (D * 2) + (kpiece(r, 2 * ks + c) << 4));
        mma16(sc[0], qa[ks], b[0], b[1]);
        mma16(sc[1], qa[ks], b[2], b[3]);
      }
    }
    const bool whole = have == 0xFFFFu && key0 >= sp.all_lo && key0 + kTile <= sp.all_hi;
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[y][e] *= sl2;
        if (!whole) {
          const int k = y * 8 + 2 * t + (e & 1), x = e >> 1;
          if (!((have >> k) & 1u) || key0 + k < sp.lo[x] || key0 + k >= sp.hi[x]) sc[y][e] = -INFINITY;
        }
      }
    float top[2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
      top[x] = quad_max(fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1])));
    st.refer(top);
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float ref = st.m[x] == -INFINITY ? 0.f : st.m[x];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float p0 = ex2(sc[y][2 * x] - ref), p1 = ex2(sc[y][2 * x + 1] - ref);
        st.l[x] += p0 + p1;
        const uint32_t h = pack_bf16x2(p0, p1);
        ph[x + 2 * y] = h;
        pl[x + 2 * y] = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xFFFF0000u));
      }
    }
    const int r = (((lane >> 3) & 1) << 3) + (lane & 7), c = lane >> 4;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
      uint32_t b[4];
      ldm4t(b, vt + r * (D * 2) + (vpiece(r, 2 * y + c) << 4));
      mma16(st.o[2 * y], ph, b[0], b[1]);
      mma16(st.o[2 * y + 1], ph, b[2], b[3]);
      mma16(st.o[2 * y], pl, b[0], b[1]);
      mma16(st.o[2 * y + 1], pl, b[2], b[3]);
    }
  }
  // put(x, column, values): the thread's columns of its row x, two at a time.
  template <typename F>
  static __device__ __forceinline__ void out(const RowState<D>& st, int t, F put) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int y = 0; y < D / 8; ++y) put(x, y * 8 + 2 * t, make_float2(st.o[y][2 * x], st.o[y][2 * x + 1]));
  }
};

// fp32.  The products' inner index is permuted so that a thread's operands are
// 16-byte pieces: of K, piece 4 s + t of key g gives steps 2 s and 2 s + 1 (columns
// 16 s + 4 t + {0, 1} and {2, 3}); of V, piece 8 q + g of keys 2 t and 2 t + 1 gives
// output tiles 4 q + {0..3}, whose column n stands for 32 q + 4 n + {0..3}.
template <int D>
struct Step<float, D> {
  static constexpr int kTile = 8, kCh = D / 4, kStages = D == 128 ? 3 : 6;
  float qa[D / 16][2][4];
  static __device__ __forceinline__ int kpiece(int r, int c) { return c ^ ((r & 1) << 2); }
  static __device__ __forceinline__ int vpiece(int r, int c) { return c ^ (r & 6); }
  __device__ __forceinline__ void load_q(const float* (&row)[2], const bool (&on)[2], int t, int d) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int c = 16 * s + 4 * t;
        const float4 q = on[x] && c < d ? *reinterpret_cast<const float4*>(row[x] + c)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
        qa[s][x][0] = q.x;
        qa[s][x][1] = q.y;
        qa[s][x][2] = q.z;
        qa[s][x][3] = q.w;
      }
  }
  __device__ __forceinline__ void tile(RowState<D>& st, uint32_t kt, uint32_t vt, unsigned have, int key0,
                                       const Spans& sp, float sl2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float hh[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}}, hl[4] = {0.f, 0.f, 0.f, 0.f},
          lh[4] = {0.f, 0.f, 0.f, 0.f};  // four chains
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint4 raw = ld_shared_v4(kt + g * (D * 4) + (kpiece(g, 4 * s + t) << 4));
      const float kf[4] = {__uint_as_float(raw.x), __uint_as_float(raw.y), __uint_as_float(raw.z),
                           __uint_as_float(raw.w)};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t ah[4], al[4], bh[2], bl[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          split(kf[2 * y + z], bh[z], bl[z]);
#pragma unroll
          for (int x = 0; x < 2; ++x) split(qa[s][x][2 * y + z], ah[x + 2 * z], al[x + 2 * z]);
        }
        mma8(hh[y], ah, bh[0], bh[1]);
        mma8(hl, ah, bl[0], bl[1]);
        mma8(lh, al, bh[0], bh[1]);
      }
    }
    const bool whole = have == 0xFFu && key0 >= sp.all_lo && key0 + kTile <= sp.all_hi;
    float sc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sc[e] = ((hl[e] + lh[e]) + (hh[0][e] + hh[1][e])) * sl2;
      if (!whole) {
        const int k = 2 * t + (e & 1), x = e >> 1;
        if (!((have >> k) & 1u) || key0 + k < sp.lo[x] || key0 + k >= sp.hi[x]) sc[e] = -INFINITY;
      }
    }
    const float top[2] = {quad_max(fmaxf(sc[0], sc[1])), quad_max(fmaxf(sc[2], sc[3]))};
    st.refer(top);
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const float ref = st.m[x] == -INFINITY ? 0.f : st.m[x];
      const float p0 = ex2(sc[2 * x] - ref), p1 = ex2(sc[2 * x + 1] - ref);
      st.l[x] += p0 + p1;
      split(p0, ph[x], pl[x]);
      split(p1, ph[x + 2], pl[x + 2]);
    }
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      const uint4 r0 = ld_shared_v4(vt + (2 * t) * (D * 4) + (vpiece(2 * t, 8 * q + g) << 4));
      const uint4 r1 = ld_shared_v4(vt + (2 * t + 1) * (D * 4) + (vpiece(2 * t + 1, 8 * q + g) << 4));
      const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        uint32_t bh[2], bl[2];
        split(__uint_as_float(w0[y]), bh[0], bl[0]);
        split(__uint_as_float(w1[y]), bh[1], bl[1]);
        mma8(st.o[4 * q + y], ph, bh[0], bh[1]);
        mma8(st.o[4 * q + y], ph, bl[0], bl[1]);
        mma8(st.o[4 * q + y], pl, bh[0], bh[1]);
      }
    }
  }
  template <typename F>
  static __device__ __forceinline__ void out(const RowState<D>& st, int t, F put) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int q = 0; q < D / 32; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            put(x, 32 * q + 8 * t + 4 * z + 2 * y,
                make_float2(st.o[4 * q + 2 * y][2 * x + z], st.o[4 * q + 2 * y + 1][2 * x + z]));
  }
};

template <typename T, int D>
struct MmaLayout {
  using St = Step<T, D>;
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(T));
  static constexpr int kTileBytes = St::kTile * kRowBytes;  // of K or V
  static constexpr int kWarpBytes = 2 * St::kStages * kTileBytes;
  static constexpr int kBytes = kW * kWarpBytes;
};

template <typename T, int D>
__global__ void __launch_bounds__(32 * kW, 2) paged_mma_kernel(const PagedArgs a) {
  using St = Step<T, D>;
  using Lay = MmaLayout<T, D>;
  constexpr int S = St::kStages, KT = St::kTile, CH = St::kCh, E = 16 / sizeof(T);
  constexpr unsigned kAll = (1u << KT) - 1u;
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ long long pre[kPagedMaxBatch + 1], scan[kW];
  __shared__ PagedWalk walks[kW][2];     // the present segment of the copies, of the products
  __shared__ unsigned tile_keys[kW][S];  // bit r: key r of the staged tile exists
  __shared__ unsigned joined;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // Neighbouring workers on different SMs: a small launch spreads out.
  const int c = warp * gridDim.x + blockIdx.x;
  const int d = a.d, v = a.v, kch = d / E, vch = v / E;
  const T* Kp = static_cast<const T*>(a.Kp);
  const T* Vp = static_cast<const T*>(a.Vp);
  uint8_t* own = sm + warp * Lay::kWarpBytes;
  const uint32_t kbase = smem_u32(own), vbase = kbase + S * Lay::kTileBytes;
  unsigned bits = 0;
  let_next_start();
  if (lane == 0) a.desc[c] = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) joined = 0;
  // Columns of K that the rows do not have stay zero: no copy writes them.
  if (kch < CH)
    for (int x = lane; x < S * Lay::kTileBytes / 16; x += 32)
      *reinterpret_cast<uint4*>(own + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
  paged_scan<kRows, KT, 32 * kW>(a, pre, scan, bits);
  int todo = 0;  // tiles of the worker
  {
    PagedWalk w;
    if (paged_begin<kRows, KT>(a, pre, c, w)) {
      todo = static_cast<int>(w.end - w.u);
      if (lane < 2) walks[warp][lane] = w;
    }
  }
  __syncwarp();

  // The copies' segment: tiles left, the next tile's first key, the keys that count.
  // Lane l holds the table entries of the keys from p_base + (l << lpk) on, and of as
  // many again behind those: one load for 512 keys, long before they are needed.
  int p_left = 0, p_key = 0, p_base = 0, p_j0 = 0, p_j1 = 0, p_h = 0;
  int pages = -1, pages_next = -1;
  const int* p_row = nullptr;
  constexpr int kLogTile = KT == 16 ? 4 : 3;
  const int lpk = min(a.lps, kLogTile), span = 32 << lpk;
  auto entries = [&](int base) {
    const int key = base + (lane << lpk);
    int page = -1;
    if (key < p_j1 && key + (1 << lpk) > p_j0) {
      page = __ldg(p_row + (key >> a.lps));
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(a.num_pages)) {
        page = -1;
        bits |= kStatusBadPage;
      }
    }
    return page;
  };
  // The products' segment.
  int left = 0, key0 = 0;
  Spans sp;
  St step;
  RowState<D> st;

  // One loop: step `it` copies tile it in and multiplies tile i = it - (S - 1).  Every
  // part of the code stands in one place, also while the ring fills: code that runs
  // once costs its instruction fetches.
#pragma unroll 1
  for (int it = 0, i = 1 - S; i < todo; ++it, ++i) {
    // Segments that start here: who = 0 the copies', 1 the products'.
#pragma unroll 1
    for (int who = 0; who < 2; ++who) {
      const bool starts = who == 0 ? p_left == 0 && it < todo : left == 0 && i >= 0;
      if (!starts) continue;
      PagedWalk w = walks[warp][who];
      if (who == 0 ? it > 0 : i > 0) {
        int x, y;
        paged_next<kRows, KT>(a, w, paged_segment<KT>(w, x, y));
        __syncwarp();
        if (lane == 0) walks[warp][who] = w;
        __syncwarp();
      }
      int j0, j1;
      const int n = paged_segment<KT>(w, j0, j1);
      const int key = (w.t.kt0 + w.rem) * KT;
      if (who == 0) {
        p_left = n;
        p_base = p_key = key;
        p_j0 = j0;
        p_j1 = j1;
        p_h = w.h;
        p_row = a.table + static_cast<size_t>(w.b) * a.max_pages;
        pages = entries(p_base);
        pages_next = entries(p_base + span);
      } else {
        left = n;
        key0 = key;
        const int r0 = w.rt * kRows;
        const T* qr[2];
        bool on[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int q = g + 8 * x, r = r0 + (q < w.t.rows ? q : 0), tok = div_by(r, a.by_group);
          on[x] = q < w.t.rows;
          paged_row_span(a, w.s, tok, sp.lo[x], sp.hi[x]);
          if (on[x] && sp.lo[x] >= sp.hi[x] && w.rem == 0 && !a.initL) bits |= kStatusEmptyRow;
          qr[x] = static_cast<const T*>(a.Q) + (w.s.s0 + tok) * a.q_stride + (w.h * a.G + r - tok * a.G) * d;
        }
        step.load_q(qr, on, t, d);
        int unused;
        paged_row_span(a, w.s, w.t.i1, sp.all_lo, unused);
        paged_row_span(a, w.s, w.t.i0, unused, sp.all_hi);
        st.clear();
      }
    }
    __syncwarp();  // every lane is done with tile i - 1
    if (it < todo) {
      if (p_key - p_base >= span) {
        p_base += span;
        pages = pages_next;
        pages_next = entries(p_base + span);
      }
      // Lane r: key r of the tile as a row of the pool, -1 for none.
      const int key = p_key + lane % KT;
      const int page = __shfl_sync(0xFFFFFFFFu, pages, (key - p_base) >> lpk);
      const long long row = page < 0 || key < p_j0 || key >= p_j1
                                ? -1
                                : ((static_cast<long long>(page) * a.Hk + p_h) << a.lps) +
                                      (key & ((1 << a.lps) - 1));
      const int s = it % S;
      const unsigned have = __ballot_sync(0xFFFFFFFFu, row >= 0) & kAll;
      if (lane == 0) tile_keys[warp][s] = have;
      const uint32_t kd = kbase + s * Lay::kTileBytes, vd = vbase + s * Lay::kTileBytes;
#pragma unroll
      for (int x = 0; x < KT * CH / 32; ++x) {
        const int idx = x * 32 + lane, r = idx / CH, pc = idx % CH;
        const long long at = __shfl_sync(0xFFFFFFFFu, row, r);
        const long long from = at < 0 ? 0 : at;
        const uint32_t off = r * Lay::kRowBytes;
        if (pc < kch) cp16(kd + off + (St::kpiece(r, pc) << 4), Kp + from * d + pc * E, at < 0 ? 0 : 16);
        if (pc < vch) cp16(vd + off + (St::vpiece(r, pc) << 4), Vp + from * v + pc * E, at < 0 ? 0 : 16);
      }
      p_key += KT;
      --p_left;
    }
    cp_commit();
    if (i < 0) continue;
    cp_wait<S - 1>();
    __syncwarp();  // tile i is in
    const int s = i % S;
    step.tile(st, kbase + s * Lay::kTileBytes, vbase + s * Lay::kTileBytes, tile_keys[warp][s], key0, sp, a.sl2);
    key0 += KT;
    if (--left > 0) continue;

    // The segment's rows.
    if (a.second) wait_for_previous();
    const PagedWalk w = walks[warp][1];
    int j0, j1;
    const int n = paged_segment<KT>(w, j0, j1);
    const int slot = paged_slot<kRows>(a, w, n, c, lane == 0);
    size_t to[2];
    bool on[2];
    PagedScale f[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int q = g + 8 * x;
      on[x] = q < w.t.rows;
      float l = st.l[x];
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (slot < 0) {
        to[x] = paged_out_row(a, w.s.s0, w.h, w.rt * kRows + (on[x] ? q : 0));
        f[x] = paged_finish(a, to[x], st.m[x], l);
        if (on[x] && t == 0) a.L[to[x]] = f[x].L;
      } else {
        to[x] = static_cast<size_t>(slot) * kRows + q;
        if (on[x] && t == 0) {
          a.pm[to[x]] = st.m[x];
          a.pl[to[x]] = l;
        }
      }
    }
    if (slot >= 0) {
      St::out(st, t, [&](int x, int col, const float2& z) {
        if (on[x] && col < v) *reinterpret_cast<float2*>(a.pz + to[x] * v + col) = z;
      });
    } else {
      St::out(st, t, [&](int x, int col, const float2& z) {
        if (!on[x] || col >= v) return;
        const size_t at = to[x] * v + col;
        float2 y = make_float2(z.x * f[x].fz, z.y * f[x].fz);
        if (a.initY) {
          const float2 p = *reinterpret_cast<const float2*>(a.initY + at);
          y = make_float2(fmaf(p.x, f[x].fi, y.x), fmaf(p.y, f[x].fi, y.y));
        }
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float2*>((a.Yf ? a.Yf : static_cast<float*>(a.Y)) + at) = y;
        } else {
          if (a.Yf) *reinterpret_cast<float2*>(a.Yf + at) = y;
          else *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.Y) + at) = pack_bf16x2(y.x, y.y);
        }
      });
    }
  }
  cp_wait<0>();
  if (a.second) wait_for_previous();  // warps without units too: the next launch counts on it
  paged_end(a, bits, &joined);
}

template <typename T, int D>
cudaError_t mma_launch(const PagedArgs& a, cudaStream_t s) {
  auto kern = paged_mma_kernel<T, D>;
  constexpr int bytes = MmaLayout<T, D>::kBytes;
  const cudaError_t e = allow_smem<paged_mma_kernel<T, D>>(bytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  cudaError_t le = cudaSuccess;
  if (a.second) le = launch_early(kern, dim3(kCtas), 32 * kW, bytes, s, a);
  else kern<<<kCtas, 32 * kW, bytes, s>>>(a);
  after_launch(kKernPaged, s);
  return le != cudaSuccess ? le : cudaGetLastError();
}

}  // namespace

bool paged_mma_shape(int d, int v) { return d <= 128 && v <= 128; }
PagedKernel paged_mma_kernel() { return {kRows, kCtas, kCtas * kW, 4}; }

cudaError_t launch_paged_mma(const PagedArgs& a, cudaStream_t s) {
  const bool narrow = a.d <= 64 && a.v <= 64;
  if (a.dtype == kF32) return narrow ? mma_launch<float, 64>(a, s) : mma_launch<float, 128>(a, s);
  return narrow ? mma_launch<__nv_bfloat16, 64>(a, s) : mma_launch<__nv_bfloat16, 128>(a, s);
}

}  // namespace exattn
