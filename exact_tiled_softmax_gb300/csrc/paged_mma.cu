// Paged attention for few rows to a key head (a decode step, a few guessed
// tokens), widths up to 128: bound by reading K and V once.
//
// A row tile is 8 or 16 rows, one or two tensor-core tiles in their N dimension: the
// products are transposed, S^T = K Q^T and O^T = V^T P^T, so that keys and columns fill
// the 16 of M whatever few rows there are, and a key head's whole group shares each key
// that is read.  A worker is a warp.  It streams the 16-key tiles of its units through a
// ring of kStages tiles of its own in shared memory (asynchronous 16-byte copies through
// the page table), and holds maximum, sum and output of its rows in registers.  No
// barrier and no other warp is involved between a segment's first copy and its last
// store.  The copies run ahead of the products by kStages - 1 tiles, over the ends of
// segments too, so that short sequences stream as long ones do; an SM keeps 96 to 144 KB in
// flight.  (As a CTA's worker, with tiles of 64 keys and barriers, 8 sequences of 16384 keys
// and 32 heads of 128 columns took 341 us.)
//
// Measured in bf16: those 2.1 GB 320 to 334 us, 6.4 to 6.7 TB/s or 95 to 98% of the measured
// copy; 64 sequences of 2048 to 32768 keys, 64 query heads over 8 key heads 674 to 707 us, 96 to
// 100%; 16 rows over 262147 keys 174 to 180 us, 88 to 91%, of which 8 are the merge.  fp32 is bound by its
// products: 12 sequences of 6000 keys of 16 heads of 80 and 96 columns 133 us, 6.1 TB/s for 4
// rows, 5.1 for 16.
//
// bf16: m16n8k16.  p enters P.V as the sum of two bf16 values, its rounding and what
// the rounding left out (2^-17 of p remains): the products are free beside the
// loads, and Y is then rounded once, on its way out.
// fp32: m16n8k8 on tf32 parts, x = hi + lo, three products for one (lo lo, 2^-22 of
// the product, is left out; lo is cut to tf32, 2^-21 of x).
// A part may be zero or of the other sign, so an infinite V, or fp32 K or Q, that a row allows may
// give NaN (stated in the header).
// The reference point of the exponentials moves only when a row's maximum passes
// it by more than 2^8, so p <= 2^8.
#include <type_traits>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

using tc::ex2;
using tc::ld_shared_v4;
using tc::pack_bf16x2;
using tc::smem_u32;
using tc::tf32_hi;

constexpr int kTile = 16;  // keys of a tile, a unit of work
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

// The 8x8 matrix of 16-bit values whose rows the warp's lanes hold in fours, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float max_over_keys(float x) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}

// A worker's rows over a segment.  Thread (g, t) = (lane / 4, lane % 4) holds, of rows
// 8 n + 2 t + x, the reference point m, the sum over its own keys l, and of the output
// the columns of o[n] (see Step).
template <int D, int NT>
struct RowState {
  float m[NT][2], l[NT][2], o[NT][D / 16][4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int y = 0; y < D / 16; ++y) o[n][y][0] = o[n][y][1] = o[n][y][2] = o[n][y][3] = 0.f;
    }
  }
  // sc[n][2 k + x]: row x's score of the thread's key k = 0, 1, masked.  Moves the
  // reference points and leaves p in sc.
  __device__ __forceinline__ void softmax(float (&sc)[NT][4]) {
    float top[NT][2];
    bool move = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[n][x] = max_over_keys(fmaxf(sc[n][x], sc[n][2 + x]));
        move |= top[n][x] > m[n][x] + kRescale;
      }
    if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float to = fmaxf(m[n][x], top[n][x]);
          const float f = m[n][x] == -INFINITY ? 0.f : ex2(m[n][x] - to);
          m[n][x] = to;
          l[n][x] *= f;
#pragma unroll
          for (int y = 0; y < D / 16; ++y) {
            o[n][y][x] *= f;
            o[n][y][2 + x] *= f;
          }
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ref = m[n][x] == -INFINITY ? 0.f : m[n][x];
        sc[n][x] = ex2(sc[n][x] - ref);
        sc[n][2 + x] = ex2(sc[n][2 + x] - ref);
        l[n][x] += sc[n][x] + sc[n][2 + x];
      }
  }
};

// The keys that a thread's rows allow, and those that every row of the tile does.
template <int NT>
struct Spans {
  int lo[NT][2], hi[NT][2], all_lo, all_hi;
};

// Scores into the exp2 domain, those that do not count to -inf.
template <int NT>
__device__ __forceinline__ void mask_scores(float (&sc)[NT][4], const Spans<NT>& sp, unsigned have, int key0,
                                            float sl2) {
  const int g = (threadIdx.x & 31) >> 2;
  const bool whole = have == 0xFFFFu && key0 >= sp.all_lo && key0 + kTile <= sp.all_hi;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sc[n][e] *= sl2;
      if (!whole) {
        const int k = g + 8 * (e >> 1), x = e & 1;
        if (!((have >> k) & 1u) || key0 + k < sp.lo[n][x] || key0 + k >= sp.hi[n][x]) sc[n][e] = -INFINITY;
      }
    }
}

// What the two types differ in: a tile's place in shared memory, Q's fragments, one
// tile's products, and the columns that a thread's outputs stand for.
template <typename T, int D, int NT> struct Step;

// bf16.  o[n][y]: columns 16 y + g (rows x = 0, 1) and 16 y + g + 8.
template <int D, int NT>
struct Step<__nv_bfloat16, D, NT> {
  // 64 columns: six warps with four stages 26.2 us, four with six 29.5 (12 sequences of 2000
  // keys, 16 key heads); 96: four with four 86.6, five with three 93.9 (6000 keys, 16 rows; 94.3 on
  // the kernel of 128).
  static constexpr int kW = D == 64 ? 6 : 4, kStages = D == 128 ? 3 : 4;
  static constexpr bool kSplit = false;  // see fp32
  uint32_t qb[NT][D / 16][2];
  // Eight rows' pieces in eight banks' groups (192-byte rows: every second begins there already).
  static __device__ __forceinline__ int kpiece(int r, int c) { return D == 96 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); }
  static __device__ __forceinline__ int vpiece(int r, int c) { return kpiece(r, c); }
  // Row n of the tile's row 8 n + g.
  __device__ __forceinline__ void load_q(int n, const __nv_bfloat16* row, bool on, int t, int d) {
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int c = ks * 16 + y * 8 + 2 * t;
        qb[n][ks][y] = on && c < d ? *reinterpret_cast<const uint32_t*>(row + c) : 0u;
      }
  }
  template <typename F>
  __device__ __forceinline__ void tile(RowState<D, NT>& st, uint32_t kt, uint32_t vt, unsigned have, int key0,
                                       const Spans<NT>& sp, float sl2, F after_scores) {
    const int lane = threadIdx.x & 31, i = lane >> 3;
    float sc[NT][4], sb[NT][4];  // two chains each
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] = sb[n][e] = 0.f;
    {
      const int r = ((i & 1) << 3) + (lane & 7), c = i >> 1;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        uint32_t k[4];
        ldm4(k, kt + r * (D * 2) + (kpiece(r, 2 * ks + c) << 4));
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16(ks & 1 ? sb[n] : sc[n], k, qb[n][ks][0], qb[n][ks][1]);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[n][e] += sb[n][e];
    mask_scores<NT>(sc, sp, have, key0, sl2);
    st.softmax(sc);
    after_scores();
    uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float p0 = sc[n][2 * k], p1 = sc[n][2 * k + 1];
        const uint32_t h = pack_bf16x2(p0, p1);
        ph[n][k] = transpose8(h);
        pl[n][k] = transpose8(pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xFFFF0000u)));
      }
    const int r = ((i >> 1) << 3) + (lane & 7), c = i & 1;
#pragma unroll
    for (int y = 0; y < D / 16; ++y) {
      uint32_t v[4];
      ldm4t(v, vt + r * (D * 2) + (vpiece(r, 2 * y + c) << 4));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16(st.o[n][y], v, ph[n][0], ph[n][1]);
        mma16(st.o[n][y], v, pl[n][0], pl[n][1]);
      }
    }
  }
  // Row pair n of the summary to z0, z1 (null: no such row).
  static __device__ __forceinline__ void put_summary(const RowState<D, NT>& st, int n, float* z0, float* z1, int v) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int y = 0; y < D / 16; ++y)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int col = 16 * y + 8 * h + g;
        if (col >= v) continue;
        if (z0) z0[col] = st.o[n][y][2 * h];
        if (z1) z1[col] = st.o[n][y][2 * h + 1];
      }
  }
  // Row pair n finished: rows to[0], to[1] of [T][heads], where on[].
  static __device__ __forceinline__ void put_rows(const PagedArgs& a, const RowState<D, NT>& st, int n,
                                                  const size_t (&to)[2], const bool (&on)[2],
                                                  const PagedScale (&f)[2]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (a.Yf) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < D / 8; ++y)
          if (on[x] && 8 * y + g < a.v)
            a.Yf[to[x] * a.v + 8 * y + g] = st.o[n][y / 2][2 * (y & 1) + x] * f[x].fz;
      return;
    }
    // Lane (g, t) stores row g of the tile, two columns at a time, after a transposition.
    const size_t r0 = __shfl_sync(0xFFFFFFFFu, to[0], g >> 1), r1 = __shfl_sync(0xFFFFFFFFu, to[1], g >> 1);
    const int o0 = __shfl_sync(0xFFFFFFFFu, static_cast<int>(on[0]), g >> 1),
              o1 = __shfl_sync(0xFFFFFFFFu, static_cast<int>(on[1]), g >> 1);
    __nv_bfloat16* mine = static_cast<__nv_bfloat16*>(a.Y) + (g & 1 ? r1 : r0) * a.v;
    const bool mine_on = g & 1 ? o1 : o0;
#pragma unroll
    for (int y = 0; y < D / 8; ++y) {
      const float *o = &st.o[n][y / 2][2 * (y & 1)];
      const uint32_t pair = transpose8(pack_bf16x2(o[0] * f[0].fz, o[1] * f[1].fz));  // row g, columns 2 t and 2 t + 1 of eight
      if (mine_on && 8 * y < a.v) *reinterpret_cast<uint32_t*>(mine + 8 * y + 2 * t) = pair;
    }
  }
};

// fp32.  The products' inner index is permuted so that a thread's operands are 16-byte
// pieces: of K, piece 4 s + t of keys g and g + 8 gives steps 2 s and 2 s + 1 (columns
// 16 s + 4 t + {0, 1} and {2, 3}); of V, piece 8 q + g of keys t and t + 4 (then t + 8 and
// t + 12) gives output tiles 2 q and 2 q + 1, so that o[n][2 q] and o[n][2 q + 1] are
// columns 32 q + 4 g + {0, 1} and {2, 3}.
template <int D, int NT>
struct Step<float, D, NT> {
  // Warps before stages: the products, 1000 to 2000 cycles a tile, are a warp's latency, and
  // four of a CTA load the SM's quarters evenly.  96 columns: four warps with two stages 133 us, two
  // with four 158 (12 sequences of 6000 keys, 16 key heads of 80 and 96 columns; 178 on a kernel of
  // 128).  128 columns: two whole stages fit three warps only; kSplit, keys and values of the
  // tiles one after another in a ring of three halves, fits four: 19 sequences of 1600 keys, 16
  // heads of 112 columns 89 -> 80 us, 34 x 8 rows over 12672 common keys 122 -> 106.
  static constexpr int kW = 4, kStages = D == 64 ? 3 : 2;
  static constexpr bool kSplit = D == 128;
  float qb[NT][D / 16][4];
  static __device__ __forceinline__ int kpiece(int r, int c) { return c ^ ((r & 1) << 2); }
  static __device__ __forceinline__ int vpiece(int r, int c) { return c ^ ((r & 3) << 1); }
  __device__ __forceinline__ void load_q(int n, const float* row, bool on, int t, int d) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const int c = 16 * s + 4 * t;
      const float4 q = on && c < d ? *reinterpret_cast<const float4*>(row + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      qb[n][s][0] = q.x;
      qb[n][s][1] = q.y;
      qb[n][s][2] = q.z;
      qb[n][s][3] = q.w;
    }
  }
  template <typename F>
  __device__ __forceinline__ void tile(RowState<D, NT>& st, uint32_t kt, uint32_t vt, unsigned have, int key0,
                                       const Spans<NT>& sp, float sl2, F after_scores) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float hh[2][NT][4], hl[NT][4], lh[NT][4];  // four chains
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) hh[0][n][e] = hh[1][n][e] = hl[n][e] = lh[n][e] = 0.f;
    // Pieces are read a step ahead of their products (128 columns, 24 rows over 3200 keys, 4 x 16
    // heads: 102 -> 94 us; nothing at 96 and 64, and a register there is spilt).
    constexpr bool kAhead = D == 128;
    auto k_piece = [&](int s, int z) {
      const int r = g + 8 * z;
      return ld_shared_v4(kt + r * (D * 4) + (kpiece(r, 4 * s + t) << 4));
    };
    auto v_piece = [&](int step, int z) {  // step 2 q + half
      const int r = 8 * (step & 1) + 4 * z + t;
      return ld_shared_v4(vt + r * (D * 4) + (vpiece(r, 8 * (step >> 1) + g) << 4));
    };
    uint4 ahead[2];
#pragma unroll
    for (int z = 0; z < 2; ++z) ahead[z] = k_piece(0, z);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      uint32_t kh[4][2], kl[4][2];  // [column of the piece][key g, g + 8]
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint4 raw = kAhead || s == 0 ? ahead[z] : k_piece(s, z);
        if (kAhead && s + 1 < D / 16) ahead[z] = k_piece(s + 1, z);
        split(__uint_as_float(raw.x), kh[0][z], kl[0][z]);
        split(__uint_as_float(raw.y), kh[1][z], kl[1][z]);
        split(__uint_as_float(raw.z), kh[2][z], kl[2][z]);
        split(__uint_as_float(raw.w), kh[3][z], kl[3][z]);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const uint32_t ah[4] = {kh[2 * y][0], kh[2 * y][1], kh[2 * y + 1][0], kh[2 * y + 1][1]};
        const uint32_t al[4] = {kl[2 * y][0], kl[2 * y][1], kl[2 * y + 1][0], kl[2 * y + 1][1]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t bh[2], bl[2];
          split(qb[n][s][2 * y], bh[0], bl[0]);
          split(qb[n][s][2 * y + 1], bh[1], bl[1]);
          mma8(hh[y][n], ah, bh[0], bh[1]);
          mma8(hl[n], ah, bl[0], bl[1]);
          mma8(lh[n], al, bh[0], bh[1]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) hh[0][n][e] = (hh[0][n][e] + hh[1][n][e]) + (hl[n][e] + lh[n][e]);
    float(&sc)[NT][4] = hh[0];
    mask_scores<NT>(sc, sp, have, key0, sl2);
    st.softmax(sc);
    after_scores();
    // p as B operands: row g, keys t and t + 4 of each half of the tile.
    uint32_t ph[NT][4], pl[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int from = ((k & 1) * 4 + t) * 4 + (g >> 1);  // the thread of key t + 4 (k & 1), rows g, g ^ 1
        const float a0 = __shfl_sync(0xFFFFFFFFu, sc[n][2 * (k >> 1)], from),
                    a1 = __shfl_sync(0xFFFFFFFFu, sc[n][2 * (k >> 1) + 1], from);
        split(g & 1 ? a1 : a0, ph[n][k], pl[n][k]);
      }
    // A tile's products are summed by the tensor cores, which cut their sums instead of
    // rounding them, and added to the output in rounded fp32.
#pragma unroll
    for (int z = 0; z < 2; ++z) ahead[z] = v_piece(0, z);
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      float sum[2][NT][4];
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int n = 0; n < NT; ++n) sum[y][n][0] = sum[y][n][1] = sum[y][n][2] = sum[y][n][3] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t vh[4][2], vl[4][2];  // [column of the piece][key t, t + 4]
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int step = 2 * q + half;
          const uint4 raw = kAhead || step == 0 ? ahead[z] : v_piece(step, z);
          if (kAhead && step + 1 < D / 16) ahead[z] = v_piece(step + 1, z);
          split(__uint_as_float(raw.x), vh[0][z], vl[0][z]);
          split(__uint_as_float(raw.y), vh[1][z], vl[1][z]);
          split(__uint_as_float(raw.z), vh[2][z], vl[2][z]);
          split(__uint_as_float(raw.w), vh[3][z], vl[3][z]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t ah[4] = {vh[2 * y][0], vh[2 * y + 1][0], vh[2 * y][1], vh[2 * y + 1][1]};
          const uint32_t al[4] = {vl[2 * y][0], vl[2 * y + 1][0], vl[2 * y][1], vl[2 * y + 1][1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma8(sum[y][n], ah, ph[n][2 * half], ph[n][2 * half + 1]);
            mma8(sum[y][n], al, ph[n][2 * half], ph[n][2 * half + 1]);
            mma8(sum[y][n], ah, pl[n][2 * half], pl[n][2 * half + 1]);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) st.o[n][2 * q + y][e] += sum[y][n][e];
    }
  }
  static __device__ __forceinline__ float4 columns(const RowState<D, NT>& st, int n, int q, int x) {
    return make_float4(st.o[n][2 * q][x], st.o[n][2 * q][2 + x], st.o[n][2 * q + 1][x], st.o[n][2 * q + 1][2 + x]);
  }
  static __device__ __forceinline__ void put_summary(const RowState<D, NT>& st, int n, float* z0, float* z1, int v) {
    const int g = (threadIdx.x & 31) >> 2;
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {
      const int col = 32 * q + 4 * g;
      if (col >= v) continue;
      if (z0) *reinterpret_cast<float4*>(z0 + col) = columns(st, n, q, 0);
      if (z1) *reinterpret_cast<float4*>(z1 + col) = columns(st, n, q, 1);
    }
  }
  static __device__ __forceinline__ void put_rows(const PagedArgs& a, const RowState<D, NT>& st, int n,
                                                  const size_t (&to)[2], const bool (&on)[2],
                                                  const PagedScale (&f)[2]) {
    const int g = (threadIdx.x & 31) >> 2;
    float* Y = a.Yf ? a.Yf : static_cast<float*>(a.Y);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int q = 0; q < D / 32; ++q)
        if (on[x] && 32 * q + 4 * g < a.v) {
          const float4 z = columns(st, n, q, x);
          *reinterpret_cast<float4*>(Y + to[x] * a.v + 32 * q + 4 * g) =
              make_float4(z.x * f[x].fz, z.y * f[x].fz, z.z * f[x].fz, z.w * f[x].fz);
        }
  }
};

template <typename T, int D, int NT>
struct MmaLayout {
  using St = Step<T, D, NT>;
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(T));
  static constexpr int kTileBytes = kTile * kRowBytes;  // of K or V
  static constexpr int kWarpBytes = (St::kSplit ? 3 : 2 * St::kStages) * kTileBytes;
  static constexpr int kBytes = St::kW * kWarpBytes;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * Step<T, D, NT>::kW, 2) paged_mma_kernel(const PagedArgs a) {
  using St = Step<T, D, NT>;
  using Lay = MmaLayout<T, D, NT>;
  constexpr int S = St::kStages, kW = St::kW, kRows = 8 * NT, E = 16 / sizeof(T);
  constexpr int CH = D / E;                 // pieces of a row
  constexpr int kCopies = kTile * CH / 32;  // pieces of K or V that a lane copies of a tile
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ long long pre[kPagedSums], scan[kW];
  __shared__ PagedWalk walks[kW][2];     // the present segment of the copies, of the products
  __shared__ unsigned tile_keys[kW][S];  // bit r: key r of the staged tile exists
  __shared__ unsigned joined;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // Neighbouring workers on different SMs: a small launch spreads out.
  const int worker = warp * gridDim.x + blockIdx.x;
  const int d = a.d, v = a.v, kch = d / E, vch = v / E;
  const T* Kp = static_cast<const T*>(a.Kp);
  const T* Vp = static_cast<const T*>(a.Vp);
  uint8_t* own = sm + warp * Lay::kWarpBytes;
  const uint32_t kbase = smem_u32(own), vbase = kbase + (St::kSplit ? 0 : S * Lay::kTileBytes);
  // Where tile i's keys and values are, from kbase and vbase on.  Split: K and V of the tiles
  // follow one another in a ring of three.
  auto k_slot = [&](int i) { return static_cast<uint32_t>(St::kSplit ? 2 * i % 3 : i % S) * Lay::kTileBytes; };
  auto v_slot = [&](int i) { return static_cast<uint32_t>(St::kSplit ? (2 * i + 1) % 3 : i % S) * Lay::kTileBytes; };
  unsigned bits = 0;
  if (threadIdx.x == 0) joined = 0;
  // Columns of K that the rows do not have stay zero: no copy writes them (split: each does).
  if (!St::kSplit && kch < CH)
    for (int x = lane; x < S * Lay::kTileBytes / 16; x += 32)
      *reinterpret_cast<uint4*>(own + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();  // `joined` is zero
  if (!a.second) wait_for_previous();
  let_next_start();
  if (lane == 0) a.desc[worker] = make_int4(0, 0, 0, 0);
  // The run's start, for both walks.
  long long total;
  bool more;  // more tiles to copy
  {
    PagedWalk w;
    if (a.B <= 32) {
      more = paged_begin_warp<kRows, kTile>(a, worker, w, total, bits);
    } else {
      paged_scan<kRows, kTile, 32 * kW>(a, pre, scan, bits);
      total = pre[a.B];
      more = paged_begin<kRows, kTile>(a, pre, worker, w);
    }
    if (more && lane < 2) walks[warp][lane] = w;
    __syncwarp();
  }
  // The copies' segment: tiles left, the next tile's first key, the keys that count.
  // Lane l holds the table entries of the keys from p_base + (l << lpk) on, and of as
  // many again behind those: one load for 512 keys, long before they are needed.
  int p_left = 0, p_key = 0, p_base = 0, p_j0 = 0, p_j1 = 0, p_h = 0;
  int pages = -1, pages_next = -1;
  const int* p_row = nullptr;
  const int lpk = min(a.lps, 4), span = 32 << lpk;
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
  // A lane's pieces: numbers lane + 32 x of the tile's kTile * CH.  Every kCols-th is in the
  // same column, kColRows rows on; every kAts-th also in the same place of a swizzle, which
  // repeats every kSwizzle rows.
  constexpr int kSwizzle = sizeof(T) == 4 ? 4 : 8;
  constexpr int kCols = 32 % CH == 0 ? 1 : 3, kColRows = kCols * 32 / CH;
  constexpr int kAts = kCols == 1 && kColRows < kSwizzle ? kSwizzle / kColRows : kCols, kAtRows = kAts * 32 / CH;
  static_assert(kCols * 32 % CH == 0 && kCopies % kAts == 0 && kAtRows % kSwizzle == 0 && 8 % kColRows == 0 &&
                    kCopies % (2 * kCols) == 0,
                "pieces of a lane");
  int rows_at[kCols], pc[kCols];
#pragma unroll
  for (int z = 0; z < kCols; ++z) {
    rows_at[z] = (lane + 32 * z) / CH;
    pc[z] = (lane + 32 * z) % CH;
  }
  uint32_t k_at[kAts], v_at[kAts];
#pragma unroll
  for (int x = 0; x < kAts; ++x) {
    const int r = (lane + 32 * x) / CH, c = pc[x % kCols];
    k_at[x] = kbase + r * Lay::kRowBytes + (St::kpiece(r, c) << 4);
    v_at[x] = vbase + r * Lay::kRowBytes + (St::vpiece(r, c) << 4);
  }
  int issued = 0;  // tiles copied so far
  // The products' segment.
  int left = 0, key0 = 0;
  Spans<NT> sp;
  St step;
  RowState<D, NT> st;

  // One loop: step `it` copies tile it in and multiplies tile i = it - (S - 1).  Every
  // part of the code stands in one place, also while the ring fills: code that runs
  // once costs its instruction fetches.
#pragma unroll 1
  for (int it = 0, i = 1 - S; more || p_left > 0 || i < issued; ++it, ++i) {
    // Segments that start here: who = 0 the copies', 1 the products'.
#pragma unroll 1
    for (int who = 0; who < 2; ++who) {
      const bool starts = who == 0 ? p_left == 0 && more : left == 0 && i >= 0 && i < issued;
      if (!starts) continue;
      PagedWalk w = walks[warp][who];
      int n = 0, j0 = 0, j1 = 0;
      bool on = (who == 0 ? it == 0 : i == 0) || paged_next<kRows, kTile>(a, w);
      // A segment may hold only what its tile was rounded up by.
#pragma unroll 1
      while (on && (n = paged_segment<kTile>(w, j0, j1)) == 0) on = paged_next<kRows, kTile>(a, w);
      if (!on) {  // the copies' end
        more = false;
        continue;
      }
      __syncwarp();
      if (lane == 0) walks[warp][who] = w;
      __syncwarp();
      const int key = (w.t.kt0 + w.rem) * kTile;
      if (who == 0) {
        p_left = n;
        p_base = p_key = key;
        p_j0 = j0;
        p_j1 = j1;
        p_h = w.h;
        p_row = paged_table(a, w.b);
        pages = entries(p_base);
        pages_next = entries(p_base + span);
      } else {
        left = n;
        key0 = key;
        const int r0 = w.rt * kRows;
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          // Row g of the tile for the operand, rows 2 t and 2 t + 1 for the statistics.
          const int q = 8 * y + g, r = r0 + (q < w.t.rows ? q : 0), tok = div_by(r, a.by_group);
          step.load_q(y,
                      static_cast<const T*>(a.Q) + (w.s.s0 + tok) * a.q_stride + (w.h * a.G + r - tok * a.G) * d,
                      q < w.t.rows, t, d);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = 8 * y + 2 * t + x;
            const bool on = row < w.t.rows;
            paged_row_span(a, w.s, div_by(r0 + (on ? row : 0), a.by_group), sp.lo[y][x], sp.hi[y][x]);
            if (on && sp.lo[y][x] >= sp.hi[y][x] && w.rem == 0 && !a.info) bits |= kStatusEmptyRow;
          }
        }
        int unused;
        paged_row_span(a, w.s, w.t.i1, sp.all_lo, unused);
        paged_row_span(a, w.s, w.t.i0, unused, sp.all_hi);
        st.clear();
      }
    }
    __syncwarp();  // every lane is done with tile i - 1
    // Copies of tile it, keys, values or both.  All sixteen keys, in pages of eight or more: rows
    // behind one another, the first eight from `row` of the pool on, the others from `row8` (pages
    // of eight row by row: 482 us in place of 326, 42 sequences of 3000 keys, 16 heads of 128 fp32
    // columns).
    auto copy_whole = [&](long long row, long long row8, auto with_k, auto with_v) {
      const uint32_t ks = k_slot(it), vs = v_slot(it);
      const T *kf[kCols], *vf[kCols];
#pragma unroll
      for (int z = 0; z < kCols; ++z) {
        kf[z] = Kp + (row + rows_at[z]) * d + pc[z] * E;
        vf[z] = Vp + (row + rows_at[z]) * v + pc[z] * E;
      }
#pragma unroll
      for (int x = 0; x < kCopies; ++x) {
        const uint32_t up = (x / kAts) * kAtRows * Lay::kRowBytes;
        const int z = x % kCols, on = x % (kCopies / 2) / kCols * kColRows;
        if (x == kCopies / 2) {
#pragma unroll
          for (int y = 0; y < kCols; ++y) {
            kf[y] += (row8 - row) * d;
            vf[y] += (row8 - row) * v;
          }
        }
        if constexpr (with_k) {
          if (St::kSplit) cp16(k_at[x % kAts] + ks + up, pc[z] < kch ? kf[z] + on * d : Kp, pc[z] < kch ? 16 : 0);
          else if (pc[z] < kch) cp16(k_at[x % kAts] + ks + up, kf[z] + on * d, 16);
        }
        if constexpr (with_v)
          if (pc[z] < vch) cp16(v_at[x % kAts] + vs + up, vf[z] + on * v, 16);
      }
    };
    // Else lane r's `row`: key r of the tile as a row of the pool, -1 for none.
    auto copy_rows = [&](long long row, auto with_k, auto with_v) {
      const uint32_t ks = k_slot(it), vs = v_slot(it);
#pragma unroll 1
      for (int x = 0; x < kCopies; ++x) {
        const int r = (lane + 32 * x) / CH, c = (lane + 32 * x) % CH;
        const long long at = __shfl_sync(0xFFFFFFFFu, row, r);
        const long long from = at < 0 ? 0 : at;
        const uint32_t off = r * Lay::kRowBytes;
        if constexpr (with_k) {
          const bool in = c < kch;
          if (St::kSplit || in)
            cp16(kbase + ks + off + (St::kpiece(r, c) << 4), in ? Kp + from * d + c * E : Kp, in && at >= 0 ? 16 : 0);
        }
        if constexpr (with_v)
          if (c < vch) cp16(vbase + vs + off + (St::vpiece(r, c) << 4), Vp + from * v + c * E, at < 0 ? 0 : 16);
      }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    constexpr std::bool_constant<!St::kSplit> at_once{};
    [[maybe_unused]] int left_over = 0;  // split: V of this tile is to be copied, 1 whole, 2 row by row
    [[maybe_unused]] long long v_row = -1, v_row8 = -1;
    if (p_left > 0) {
      if (p_key - p_base >= span) {
        p_base += span;
        pages = pages_next;
        pages_next = entries(p_base + span);
      }
      const int s = issued++ % S;
      const int first = __shfl_sync(0xFFFFFFFFu, pages, (p_key - p_base) >> lpk);
      unsigned have = 0xFFFFu;
      const int second = lpk == 3 ? __shfl_sync(0xFFFFFFFFu, pages, (p_key + 8 - p_base) >> 3) : first;
      if (lpk >= 3 && first >= 0 && second >= 0 && p_key >= p_j0 && p_key + kTile <= p_j1) {
        const long long row = ((static_cast<long long>(first) * a.Hk + p_h) << a.lps) + (p_key & ((1 << a.lps) - 1));
        const long long row8 = lpk == 3 ? (static_cast<long long>(second) * a.Hk + p_h) << 3 : row + 8;
        copy_whole(row, row8, yes, at_once);
        left_over = 1;
        v_row = row;
        v_row8 = row8;
      } else {
        const int key = p_key + (lane & 15);
        const int page = __shfl_sync(0xFFFFFFFFu, pages, (key - p_base) >> lpk);
        const long long row = page < 0 || key < p_j0 || key >= p_j1
                                  ? -1
                                  : ((static_cast<long long>(page) * a.Hk + p_h) << a.lps) +
                                        (key & ((1 << a.lps) - 1));
        have = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFFFu;
        copy_rows(row, yes, at_once);
        left_over = 2;
        v_row = row;
      }
      if (lane == 0) tile_keys[warp][s] = have;
      p_key += kTile;
      --p_left;
    }
    cp_commit();
    // Split: V(it), into the slot of K(i), which every lane is done with.
    [[maybe_unused]] auto rest = [&]() {
      if (left_over == 1) copy_whole(v_row, v_row8, no, yes);
      else if (left_over == 2) copy_rows(v_row, no, yes);
      cp_commit();
    };
    if (i < 0 || i >= issued) {
      if constexpr (St::kSplit) rest();
      continue;
    }
    cp_wait<St::kSplit ? 2 : S - 1>();
    __syncwarp();  // tile i is in (split: its keys)
    step.tile(st, kbase + k_slot(i), vbase + v_slot(i), tile_keys[warp][i % S], key0, sp, a.sl2, [&]() {
      if constexpr (St::kSplit) {
        __syncwarp();
        rest();
        cp_wait<2>();
        __syncwarp();  // V(i) is in
      }
    });
    key0 += kTile;
    if (--left > 0) continue;

    // The segment's rows.
    const PagedWalk w = walks[warp][1];
    int j0, j1;
    const int n = paged_segment<kTile>(w, j0, j1);
    const PagedPlace place = paged_place<kRows>(a, total, w, n, worker, lane == 0);
    const int slot = place.slot;
#pragma unroll
    for (int y = 0; y < NT; ++y) {
      size_t to[2];
      bool on[2];
      PagedScale f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int q = 8 * y + 2 * t + x;
        on[x] = q < w.t.rows;
        float l = st.l[y][x];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        to[x] = paged_out_row(a, w.s.s0, w.h, w.rt * kRows + (on[x] ? q : 0), w.s.prefix);
        if (a.info && place.parts >= 0 && on[x] && g == 0) a.info[to[x]] = make_int2(worker, place.parts);
        if (slot < 0) {
          f[x] = paged_finish(st.m[y][x], l);
          if (on[x] && g == 0) a.L[to[x]] = f[x].L;
        } else {
          to[x] = static_cast<size_t>(slot) * kRows + q;
          if (on[x] && g == 0) {
            a.pm[to[x]] = st.m[y][x];
            a.pl[to[x]] = l;
          }
        }
      }
      if (slot >= 0)
        St::put_summary(st, y, on[0] ? a.pz + to[0] * v : nullptr, on[1] ? a.pz + to[1] * v : nullptr, v);
      else
        St::put_rows(a, st, y, to, on, f);
    }
  }
  cp_wait<0>();
  if (a.second) wait_for_previous();  // the next launch waits for this one alone
  paged_end(a, bits, &joined);
}

template <typename T, int D, int NT>
cudaError_t mma_launch(const PagedArgs& a, cudaStream_t s) {
  auto kern = paged_mma_kernel<T, D, NT>;
  constexpr int bytes = MmaLayout<T, D, NT>::kBytes, threads = 32 * Step<T, D, NT>::kW;
  const cudaError_t e = allow_smem<paged_mma_kernel<T, D, NT>>(bytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  const cudaError_t le = launch_early(kern, dim3(kCtas), threads, bytes, s, a);
  after_launch(kKernPaged, s);
  return le;
}

template <typename T, int D>
cudaError_t mma_rows(const PagedArgs& a, int rows, cudaStream_t s) {
  return rows == 8 ? mma_launch<T, D, 1>(a, s) : mma_launch<T, D, 2>(a, s);
}

// The columns that a kernel is made for.
int columns_of(int d, int v) {
  const int most = d > v ? d : v;
  return most <= 64 ? 64 : most <= 96 ? 96 : 128;
}
template <typename T>
cudaError_t mma_columns(const PagedArgs& a, int columns, int rows, cudaStream_t s) {
  return columns == 64   ? mma_rows<T, 64>(a, rows, s)
         : columns == 96 ? mma_rows<T, 96>(a, rows, s)
                         : mma_rows<T, 128>(a, rows, s);
}
template <typename T>
int warps_of(int columns) {
  return columns == 64 ? Step<T, 64, 1>::kW : columns == 96 ? Step<T, 96, 1>::kW : Step<T, 128, 1>::kW;
}

}  // namespace

bool paged_mma_shape(int d, int v) { return d <= 128 && v <= 128; }
PagedKernel paged_mma_kernel_of(int dtype, int d, int v, int rows) {
  const int columns = columns_of(d, v), warps = dtype == kF32 ? warps_of<float>(columns) : warps_of<__nv_bfloat16>(columns);
  // Least units: what a worker streams before it ends a tile, against the workers that join it.
  // One sequence of 1000 keys, 8 key heads of 128 bf16 columns: 12.3 us with 2, 14.3 with 4, 16.4
  // with 8; 16 key heads of 64 columns and 2000 common keys: 13.1, 12.6, 13.1; fp32, 2 key heads of
  // 112 columns, 25 sequences of 600 keys behind 804: 30.3, 25.9, 37.9.
  const int least = dtype == kBF16 && columns > 64 ? 2 : 4;
  return {rows, kCtas, kCtas * warps, least};
}

cudaError_t launch_paged_mma(const PagedArgs& a, int rows, cudaStream_t s) {
  const int columns = columns_of(a.d, a.v);
  return a.dtype == kF32 ? mma_columns<float>(a, columns, rows, s) : mma_columns<__nv_bfloat16>(a, columns, rows, s);
}

}  // namespace exattn
