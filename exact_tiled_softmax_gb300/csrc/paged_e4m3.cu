// Paged attention over pages in 8 bits for few rows to a key head: bound by reading K and V once.
//
// The shape of the kernel for 16-bit pages: a row tile is 8 or 16 rows in the N of the products
// S^T = K Q^T and O^T = V^T P^T, a worker is a warp that streams the 32-key tiles of its units
// through a ring of its own (16-byte asynchronous copies through the page table, running ahead over
// the ends of segments) and holds maximum, sum and output of its rows in registers.  An 8-bit tile
// of 32 keys is the bytes of a 16-bit one of 16.
//
// Operands are fp16 (m16n8k16): an e4m3 number is one exactly, and two come out of each conversion.
// (mma.sync of e4m3 operands is two of fp16 here, with its conversions once more for each.)  No row's
// power of two enters them.
// A key's comes out of its score.  A value's goes into its
// weight: with s in the exp2 domain and e the exponent of V's row, w = s + e, and the operand is
// 2^(w - M + 7) with M a reference point of its own (the sum l keeps s's), so that unequal rows of V
// lose nothing; 2^7 puts the largest weight in the middle of fp16's range above its subnormals, and a
// weight is held to 2^-11 of itself or 2^-32 of the row's largest.  A row of Q is scaled by an even power of
// two that brings its largest entry to [2^13, 2^15).  fp32 queries and their weights are two fp16 parts,
// 2^-22 of themselves.
// The reference points move only when a row's maximum passes them by more than 2^8, which a vote
// tells without the maximum.
//
// Measured: one token of 8 sequences over 16384 keys, 32 key heads of 128 columns, 1.08 GB: 168 us, 6.4 TB/s or
// 95% of the measured copy (16-bit pages: 333); of 96 columns 143 us (5.6 TB/s), 80 136, 64 98; fp32 queries 174.
// 64 ragged sequences, 8 rows to a key head: 351 us, 98%.  16 rows, 262147 keys of 8 heads: 90 us, 6.0 TB/s, and 9
// of merge: registers for two row tiles leave two warps to a scheduler.  256 columns, 537 MB: 104 us for one row,
// 103 for four.  Pages of 8 or 16 keys 184 us in place of 168.
//
// The products' inner index is permuted freely, as long as both operands agree: a lane of a quad has four
// columns of 16 of a key or a query, which is what a 16-bit matrix load gives it of the bytes.  V comes
// transposed byte by byte (four keys of one column), and two conversions make two pairs of keys of
// it; the rows of the scores follow: row g of the half z of sixteen keys is key 4 (g / 2) + g % 2 + 2 z.
#include <cuda_fp16.h>

#include <type_traits>
#include <utility>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

using tc::ex2;
using tc::fadd2;
using tc::ld_shared_v4;
using tc::pack_bf16x2;
using tc::smem_u32;

constexpr int kTile = 32;  // keys of a tile, a unit of work
constexpr float kRescale = 8.f;
constexpr float kLift = 7.f;  // weights are held times 2^7
constexpr float kNoKey = -3.402823466e38f;  // a reference point below every score

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int kTo, int kFrom>
__device__ __forceinline__ void cp16_at(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kTo), "n"(kFrom) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t x;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return x;
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Two 16 x 16 matrices of bytes, transposed: lane (g, t) has row t .. t + 3 of columns g and g + 8 of each.
__device__ __forceinline__ void ldm2t8(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
// What the rounding of pack_f16x2 left out, packed.
__device__ __forceinline__ uint32_t rest_f16x2(float lo, float hi, uint32_t packed) {
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_f16x2(lo - x.x, hi - x.y);
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
__device__ __forceinline__ float max4(const float (&x)[2][4], int at) {
  return fmaxf(fmaxf(x[0][at], x[0][2 + at]), fmaxf(x[1][at], x[1][2 + at]));
}

// A tile in shared memory: rows of D bytes in lines of 128, their 16-byte pieces swizzled so that
// the eight rows of a matrix load meet eight banks' groups: keys 4 i + {0, 1} or {2, 3} for K, eight in a row for V.
template <int D>
struct Place {
  static constexpr int CH = D / 16;        // pieces of a row
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kRows = 32 / CH;    // rows that a warp copies at once, 512 bytes
  static constexpr __host__ __device__ int k_swizzle(int r) { return D >= 128 ? ((r >> 1) & 6) | (r & 1) : (r >> 2) & 3; }
  static constexpr __host__ __device__ int v_swizzle(int r) { return D >= 128 ? r & 7 : (r >> 1) & 3; }
  static __device__ __forceinline__ uint32_t at(int r, int c, int swizzle) {
    return D >= 128 ? r * D + ((c ^ swizzle) << 4) : (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ swizzle) << 4);
  }
  static __device__ __forceinline__ uint32_t k_at(int r, int c) { return at(r, c, k_swizzle(r)); }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) { return at(r, c, v_swizzle(r)); }
  // What kRows x rows further on the swizzle of a piece's address turns over (a lane's first row is below kRows,
  // a power of two).
  static constexpr uint32_t k_turn(int x) { return k_swizzle(kRows * x) << 4; }
  static constexpr uint32_t v_turn(int x) { return v_swizzle(kRows * x) << 4; }
};

// C columns (64, 96, 128 or 256) in rows of D bytes.  Up to 128: 12 warps of an SM with two stages (8 sequences of
// 16384 keys, 32 heads of 128: 169 us; 8 warps with three 177) where 168 registers are enough, else 8 with three.
template <typename T, int C, int NT>
struct Config {
  static constexpr int D = C <= 64 ? 64 : C <= 128 ? 128 : 256;
  static constexpr bool kMany = std::is_same<T, __nv_bfloat16>::value && NT == 1 && D <= 128;
  // Two row tiles of fp32 queries, whose parts are 64 registers: they stay in shared memory, in place of a stage
  // (32 sequences of 8192 keys, 8 key heads of 128 columns, 16 rows: 124 us in place of 148, 96 and 64 columns the
  // same; the 32 registers of bf16 ones: 147 in place of 109).
  static constexpr bool kQueries = std::is_same<T, float>::value && NT == 2;
  static constexpr int kW = D == 256 ? 6 : 4, kStages = kMany || D == 256 || kQueries ? 2 : 3,
                       kCtas = (D == 256 ? 1 : kMany ? 3 : 2) * 152;
  static constexpr int kQueryBytes = kQueries ? 32 * 16 * NT * (C / 16) : 0;  // of a warp
};

template <typename T> struct Parts;  // N: of a query's entry and of a weight
template <> struct Parts<__nv_bfloat16> {
  static constexpr int N = 1;
  using Raw = uint2;  // four columns
  static __device__ __forceinline__ void to(const Raw& raw, float (&x)[4]) {
    x[0] = __uint_as_float(raw.x << 16), x[1] = __uint_as_float(raw.x & 0xFFFF0000u);
    x[2] = __uint_as_float(raw.y << 16), x[3] = __uint_as_float(raw.y & 0xFFFF0000u);
  }
};
template <> struct Parts<float> {
  static constexpr int N = 2;
  using Raw = float4;
  static __device__ __forceinline__ void to(const Raw& q, float (&x)[4]) {
    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
  }
};

// The keys that a thread's rows allow, and those that every row of the tile does.
template <int NT>
struct Spans {
  int lo[NT][2], hi[NT][2], all_lo, all_hi;
};

// A worker's rows over a segment.  Thread (g, t) = (lane / 4, lane % 4) holds the operands of rows
// 8 n + g, and of rows 8 n + 2 t + x the root f of their power of two, the reference points m and M, the sum
// over its own keys l, and of the output o[n][y] columns 16 y + g (x = 0, 1) and 16 y + g + 8.
template <typename T, int C, int NT>
struct Rows {
  static constexpr int D = Config<T, C, NT>::D, P = Parts<T>::N, K = C / 16;
  static constexpr bool kQueries = Config<T, C, NT>::kQueries;
  uint32_t qb[kQueries ? 1 : NT][P][K][2];  // kQueries: of the row tile that is loaded
  float f[NT][2], m[NT][2], M[NT][2], l[NT][2], o[NT][K][4];

  using Raw = typename Parts<T>::Raw;
  // The tile's row 8 n + g.
  static __device__ __forceinline__ void load_q(Raw (&raw)[K], const T* row, bool on, int d) {
#pragma unroll
    for (int c = 0; c < K; ++c) {
      raw[c] = Raw{};
      if (on && 16 * c < d) raw[c] = *reinterpret_cast<const Raw*>(row + 16 * c + 4 * (threadIdx.x & 3));
    }
  }
  // Its operands.  qs: the warp's place for them in shared memory.
  __device__ __forceinline__ void take_q(int n, const Raw (&raw)[K], uint32_t qs) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float x[K][4];
    unsigned top = 0u;
#pragma unroll
    for (int c = 0; c < K; ++c) {
      Parts<T>::to(raw[c], x[c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[c][e]) & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    // The largest is below 2^(e - 126), and brought to [2^13, 2^15) by an even power of two, whose root is normal.
    const unsigned e = max((top >> 23) | 1u, 15u);
    const float up = __uint_as_float((268u - e) << 23), root = __uint_as_float((e + 113u) >> 1 << 23);
#pragma unroll
    for (int c = 0; c < K; ++c) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float p = x[c][2 * y] * up, q = x[c][2 * y + 1] * up;
        const uint32_t hi = pack_f16x2(p, q);
        qb[kQueries ? 0 : n][0][c][y] = hi;
        if (P == 2) qb[kQueries ? 0 : n][P - 1][c][y] = rest_f16x2(p, q, hi);
      }
    }
    if constexpr (kQueries) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int s = 0; s < C / 32; ++s)  // four registers of a lane at once, read by the same
          tc::st_shared_v4(qs + ((n * P + p) * (C / 32) + s) * 512 + 16 * lane, qb[0][p][2 * s][0], qb[0][p][2 * s][1],
                           qb[0][p][2 * s + 1][0], qb[0][p][2 * s + 1][1]);
    }
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) f[n][x2] = __shfl_sync(0xFFFFFFFFu, root, 4 * (2 * t + x2));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = M[n][0] = M[n][1] = kNoKey;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int y = 0; y < K; ++y) o[n][y][0] = o[n][y][1] = o[n][y][2] = o[n][y][3] = 0.f;
    }
  }

  // The tile at kt, vt, its exponents at et (32 of keys, 32 of values).
  __device__ __forceinline__ void tile(uint32_t kt, uint32_t vt, uint32_t et, unsigned have, int key0,
                                       const Spans<NT>& sp, int v, float sl2, uint32_t qs) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    // Of the sixteen keys q, half z (key `first` + 16 q + 2 z): bytes 2 z of the words.
    const int first = 4 * (g >> 1) + (g & 1);
    uint32_t ke[2], ve[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ke[q] = lds32(et + 16 * q + 4 * (g >> 1)) >> 8 * (g & 1);
      ve[q] = lds32(et + 32 + 16 * q + 4 * (g >> 1)) >> 8 * (g & 1);
    }
    float sc[NT][2][4];  // [row tile][sixteen keys][2 z + row]
    {
      const int i = lane & 7, b = lane >> 3;  // matrices: half b % 2, piece b / 2 of two
      const uint32_t at = kt + Place<D>::k_at(4 * (i >> 1) + (i & 1) + 2 * (b & 1), b >> 1);
#pragma unroll
      for (int s = 0; s < C / 32; ++s) {
        uint32_t qk[NT][P][4];
        if constexpr (kQueries) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const uint4 x = ld_shared_v4(qs + ((n * P + p) * (C / 32) + s) * 512 + 16 * lane);
              qk[n][p][0] = x.x, qk[n][p][1] = x.y, qk[n][p][2] = x.z, qk[n][p][3] = x.w;
            }
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
              for (int e = 0; e < 4; ++e) qk[n][p][e] = qb[n][p][2 * s + e / 2][e % 2];
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t k[4];
          ldm4(k, (at ^ (s << 5)) + q * (16 * D));
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t a[4] = {e4m3_pair(k[2 * c]), e4m3_pair(k[2 * c + 1]), e4m3_pair_high(k[2 * c]),
                                   e4m3_pair_high(k[2 * c + 1])};
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int p = 0; p < P; ++p) {
                const uint32_t b0 = qk[n][p][2 * c], b1 = qk[n][p][2 * c + 1];
                if (s == 0 && c == 0 && p == 0) mma16_first(sc[n][q], a, b0, b1);
                else mma16(sc[n][q], a, b0, b1);
              }
          }
        }
      }
    }
    // Scores into the exp2 domain but for f, those that do not count to -inf; w beside them.  The power of two of a row
    // of Q comes as its root f, before and after the key's: their product may leave fp32 where the score does not.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float f0 = f[n][0] * sl2, f1 = f[n][1] * sl2;
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const float kf = e4m3_scale((ke[q] >> (16 * z)) & 255u);
          float &s0 = sc[n][q][2 * z], &s1 = sc[n][q][2 * z + 1];
          s0 *= f0 * kf;
          s1 *= f1 * kf;
        }
    }
    if (have != 0xFFFFFFFFu || key0 < sp.all_lo || key0 + kTile > sp.all_hi) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = first + 16 * q + 2 * (e >> 1), x = e & 1;
            if (!((have >> key) & 1u) || key0 + key < sp.lo[n][x] || key0 + key >= sp.hi[n][x]) sc[n][q][e] = -INFINITY;
          }
    }
    float wt[NT][2][4], over = kNoKey;
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const float vx = __uint_as_float(0x4B000000u | ((ve[q] >> (16 * z)) & 255u)) - 8388735.f;  // byte - 127
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float s = sc[n][q][2 * z + x], w = wt[n][q][2 * z + x] = fmaf(s, f[n][x], vx);
            over = tc::fmax3(over, fmaf(s, f[n][x], -m[n][x]), w - M[n][x]);
          }
      }
    if (__any_sync(0xFFFFFFFFu, over > kRescale)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // Each row by itself: what the others hold does not change its bits.
          const float to = max_over_keys(max4(sc[n], x)) * f[n][x], To = max_over_keys(max4(wt[n], x));
          if (to > m[n][x] + kRescale) {
            l[n][x] *= ex2(m[n][x] - to);
            m[n][x] = to;
          }
          if (!(To > M[n][x] + kRescale)) continue;
          const float F = ex2(M[n][x] - To);
          M[n][x] = To;
#pragma unroll
          for (int y = 0; y < K; ++y) {
            o[n][y][x] *= F;
            o[n][y][2 + x] *= F;
          }
        }
    }
    uint32_t pb[NT][P][2][2];  // [pair of quarters][quarter]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float R0 = kLift - M[n][0], R1 = kLift - M[n][1];
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float s0, s1, w0, w1;
          tc::ffma2(s0, s1, sc[n][q][2 * z], sc[n][q][2 * z + 1], f[n][0], f[n][1], -m[n][0], -m[n][1]);
          fadd2(w0, w1, wt[n][q][2 * z], wt[n][q][2 * z + 1], R0, R1);
          fadd2(l[n][0], l[n][1], l[n][0], l[n][1], ex2(s0), ex2(s1));
          const float p0 = ex2(w0), p1 = ex2(w1);
          const uint32_t hi = pack_f16x2(p0, p1);
          pb[n][0][q][z] = transpose8(hi);
          if (P == 2) pb[n][P - 1][q][z] = transpose8(rest_f16x2(p0, p1, hi));
        }
    }
    {
      const uint32_t at = vt + Place<D>::v_at(lane, 0);
#pragma unroll
      for (int y = 0; y < K; ++y) {
        // (A branch for every y keeps the steps apart: 16 rows over 262147 keys 103 us in place of 100, 24 over 32 x 8192
        // 187 of 179, 16 of fp32 131 of 121.)
        if (y == K / 2 && 16 * y >= v) break;
        uint32_t r[4];  // of sixteen keys q: keys 4 t to 4 t + 3 of columns 16 y + g and 16 y + g + 8
        ldm2t8(r, at ^ (y << 4));
        uint32_t a[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            a[q][h] = e4m3_pair(r[2 * q + h]);
            a[q][2 + h] = e4m3_pair_high(r[2 * q + h]);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (P == 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q) mma16(o[n][y], a[q], pb[n][0][q][0], pb[n][0][q][1]);
          } else {
            // A tile's products are summed by the tensor cores, which cut their sums instead of
            // rounding them, and added to the output in rounded fp32.
            float sum[4];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int p = P - 1; p >= 0; --p) {
                if (q == 0 && p == P - 1) mma16_first(sum, a[q], pb[n][p][q][0], pb[n][p][q][1]);
                else mma16(sum, a[q], pb[n][p][q][0], pb[n][p][q][1]);
              }
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][y][e] += sum[e];
          }
        }
      }
    }
  }
};

// A whole tile of rows of D bytes behind one another; x: see the general copy.
template <int CH, int... X>
__device__ __forceinline__ void copy_dense(uint32_t k, uint32_t v, uint32_t up, const uint8_t* kf, const uint8_t* vf,
                                           std::integer_sequence<int, X...>) {
  (cp16_at<512 * X, 512 * X>((k ^ Place<16 * CH>::k_turn(X)) + up, kf), ...);
  (cp16_at<512 * X, 512 * X>((v ^ Place<16 * CH>::v_turn(X)) + up, vf), ...);
}

template <typename T, int C, int NT>
constexpr int smem_bytes() {
  return Config<T, C, NT>::kW * Config<T, C, NT>::kStages * (2 * Place<Config<T, C, NT>::D>::kTileBytes + 64) +
         Config<T, C, NT>::kW * Config<T, C, NT>::kQueryBytes + 256;
}

template <typename T, int C, int NT>
__global__ void __launch_bounds__(32 * Config<T, C, NT>::kW, Config<T, C, NT>::kCtas / 152)
    paged_e4m3_kernel(const PagedArgs a) {
  constexpr int D = Config<T, C, NT>::D;
  using At = Place<D>;
  constexpr int S = Config<T, C, NT>::kStages, kW = Config<T, C, NT>::kW, kRows = 8 * NT, CH = At::CH;
  constexpr int kStage = 2 * At::kTileBytes;
  extern __shared__ __align__(128) uint8_t sm_raw[];
  uint8_t* sm = sm_raw + (0u - smem_u32(sm_raw) & 255u);  // pieces are found by turning bits of an address over
  __shared__ long long pre[kPagedSums], scan[kW];
  __shared__ PagedWalk walks[kW][2];     // the present segment of the copies, of the products
  __shared__ unsigned tile_keys[kW][S];  // bit r: key r of the staged tile exists
  __shared__ unsigned joined;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // Neighbouring workers on different SMs: a small launch spreads out.
  const int worker = warp * gridDim.x + blockIdx.x;
  const int d = a.d, v = a.v;
  uint8_t* own = sm + warp * (S * kStage);
  const uint32_t base = smem_u32(own), scales = smem_u32(sm) + kW * S * kStage + warp * (S * 64);
  const uint32_t qs = smem_u32(sm) + kW * S * (kStage + 64) + warp * Config<T, C, NT>::kQueryBytes;
  unsigned bits = 0;
  if (threadIdx.x == 0) joined = 0;
  // Columns of K that the rows do not have stay zero: no copy writes them.
  if (d < D)
    for (int x = lane; x < S * kStage / 16; x += 32) *reinterpret_cast<uint4*>(own + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
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
  // many again behind those.
  int p_left = 0, p_key = 0, p_base = 0, p_j0 = 0, p_j1 = 0, p_h = 0;
  int pages = -1, pages_next = -1;
  const int* p_row = nullptr;
  const int lpk = min(a.lps, 5), span = 32 << lpk;
  const bool small = a.lps < 3;  // pages of fewer keys than the copies count in
  auto entries = [&](int first) {
    const int key = first + (lane << lpk);
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
  // The lane's pieces of a tile: column piece pc of rows pr + kRows x.
  const int pr = lane / CH, pc = lane % CH;
  const uint32_t k_to = base + At::k_at(pr, pc), v_to = base + At::kTileBytes + At::v_at(pr, pc);
  const bool k_on = 16 * pc < d, v_on = 16 * pc < v;
  const uint8_t* Kp = static_cast<const uint8_t*>(a.Kp) + static_cast<size_t>(pr) * d + 16 * pc;
  const uint8_t* Vp = static_cast<const uint8_t*>(a.Vp) + static_cast<size_t>(pr) * v + 16 * pc;
  const uint8_t* Ep = lane < 8 ? a.Ks : a.Vs;  // lanes 0 to 7 copy keys' exponents, 8 to 15 values'
  // Tiles that are copied as one stretch: rows of D bytes, or of any width where the kernel's columns are fewer.
  // (Both in one kernel cost the first: 8 sequences of 16384 keys 177 us in place of 169.)
  const bool stretch = lpk == 5 && (C != D || (d == D && v == D));
  int issued = 0;  // tiles copied so far
  // Row q of a segment's row tile (of the first, where the tile has no such).
  auto query = [&](const PagedWalk& w, int q) {
    const int r = w.rt * kRows + (q < w.t.rows ? q : 0), tok = div_by(r, a.by_group);
    return static_cast<const T*>(a.Q) + (w.s.s0 + tok) * a.q_stride + (w.h * a.G + r - tok * a.G) * d;
  };
  const int lines = (d * static_cast<int>(sizeof(T)) + 127) / 128;  // of 128 bytes, of a row
  // The products' segment.
  int left = 0, key0 = 0;
  Spans<NT> sp;
  Rows<T, C, NT> st;

  // One loop: step `it` copies tile it in and multiplies tile i = it - (S - 1).  Every
  // part of the code stands in one place, also while the ring fills: code that runs
  // once costs its instruction fetches.
#pragma unroll 1
  for (int it = 0, i = 1 - S; more || p_left > 0 || i < issued; ++it, ++i) {
    // Segments that start here: who = 0 the copies', 1 the products'.
#pragma unroll 1
    for (int who = (p_left == 0 && more) || (left == 0 && i >= 0 && i < issued) ? 0 : 2; who < 2; ++who) {
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
        // The segment's rows of Q, on their way before its first product: a miss waits some 4 us behind the streams
        // (16 fp32 rows over 262147 keys 119 us in place of 121, one bf16 row of 8 x 16384 keys 168.9 of 169.4).
#pragma unroll 1
        for (int x = lane; x < w.t.rows * lines; x += 32) {
          const T* at = query(w, x / lines) + x % lines * (128 / sizeof(T));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
        pages = entries(p_base);
        pages_next = entries(p_base + span);
      } else {
        left = n;
        key0 = key;
        const int r0 = w.rt * kRows;
        // Row g of the tile for the operand, rows 2 t and 2 t + 1 for the statistics.  All loads first, for the same
        // reason: one row tile after the other 16 rows over 262147 keys take 105 us in place of 99, 4 x 4000 keys 26.7
        // of 23.2.
        typename Parts<T>::Raw raw[NT][C / 16];
#pragma unroll
        for (int y = 0; y < NT; ++y) st.load_q(raw[y], query(w, 8 * y + g), 8 * y + g < w.t.rows, d);
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          st.take_q(y, raw[y], qs);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int row = 8 * y + 2 * t + x;
            const bool has = row < w.t.rows;
            paged_row_span(a, w.s, div_by(r0 + (has ? row : 0), a.by_group), sp.lo[y][x], sp.hi[y][x]);
            if (has && sp.lo[y][x] >= sp.hi[y][x] && w.rem == 0 && !a.info) bits |= kStatusEmptyRow;
          }
        }
        int unused;
        paged_row_span(a, w.s, w.t.i1, sp.all_lo, unused);
        paged_row_span(a, w.s, w.t.i0, unused, sp.all_hi);
        st.clear();
      }
    }
    __syncwarp();  // every lane is done with tile i - 1
    if (p_left > 0) {
      if (p_key - p_base >= span) {
        p_base += span;
        pages = pages_next;
        pages_next = entries(p_base + span);
      }
      const int s = issued++ % S;
      const uint32_t up = s * kStage;
      unsigned have = 0u;
      const int page0 = __shfl_sync(0xFFFFFFFFu, pages, (p_key - p_base) >> lpk);
      if (stretch && page0 >= 0 && p_key >= p_j0 && p_key + kTile <= p_j1) {
        // All keys, of one page: one stretch of memory.
        const long long row = ((static_cast<long long>(page0) * a.Hk + p_h) << a.lps) + (p_key & ((1 << a.lps) - 1));
        if constexpr (C == D) {
          copy_dense<CH>(k_to, v_to, up, Kp + row * D, Vp + row * D, std::make_integer_sequence<int, CH>{});
        } else {
          const uint8_t *kf = Kp + row * d, *vf = Vp + row * v;
#pragma unroll
          for (int x = 0; x < CH; ++x, kf += At::kRows * d, vf += At::kRows * v) {
            if (k_on) cp16((k_to ^ At::k_turn(x)) + up + 512 * x, kf, 16);
            if (v_on) cp16((v_to ^ At::v_turn(x)) + up + 512 * x, vf, 16);
          }
        }
        if (lane < 16) cp4(scales + s * 64 + 4 * lane, Ep + row + 4 * (lane & 7), 4);
        have = 0xFFFFFFFFu;
      } else if (!small) {
        // Eight keys at a time are one page's rows behind one another; pool rows of the four eights.
        long long row[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int key = p_key + 8 * z, page = __shfl_sync(0xFFFFFFFFu, pages, (key - p_base) >> lpk);
          if (page >= 0) have |= 0xFFu << 8 * z;
          row[z] = page < 0 ? 0 : ((static_cast<long long>(page) * a.Hk + p_h) << a.lps) + (key & ((1 << a.lps) - 1));
        }
        if (p_j0 > p_key) have &= 0xFFFFFFFFu << min(31, p_j0 - p_key);  // below 32: the segment has keys here
        if (p_j1 < p_key + kTile) have &= 0xFFFFFFFFu >> min(31, p_key + kTile - p_j1);
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          const int z = At::kRows * x / 8, on = At::kRows * x % 8;
          const int bytes = ((have >> (pr + At::kRows * x)) & 1u) << 4;
          if (k_on) cp16((k_to ^ At::k_turn(x)) + up + 512 * x, Kp + (row[z] + on) * d, bytes);
          if (v_on) cp16((v_to ^ At::v_turn(x)) + up + 512 * x, Vp + (row[z] + on) * v, bytes);
        }
        if (lane < 16) {
          const int z = (lane >> 1) & 3;
          const long long from = z == 0 ? row[0] : z == 1 ? row[1] : z == 2 ? row[2] : row[3];
          cp4(scales + s * 64 + 4 * lane, Ep + from + 4 * (lane & 1), (have >> 8 * z) & 0xFFu ? 4 : 0);
        }
      } else {
        // Key by key: lane l finds key l.
        const int key = p_key + lane, page = __shfl_sync(0xFFFFFFFFu, pages, (key - p_base) >> lpk);
        const bool on = page >= 0 && key >= p_j0 && key < p_j1;
        const long long mine = on ? ((static_cast<long long>(page) * a.Hk + p_h) << a.lps) + (key & ((1 << a.lps) - 1)) : 0;
        have = __ballot_sync(0xFFFFFFFFu, on);
#pragma unroll 1
        for (int x = 0; x < CH; ++x) {
          const int r = pr + At::kRows * x, bytes = ((have >> r) & 1u) << 4;
          const long long row = __shfl_sync(0xFFFFFFFFu, mine, r) - pr;  // Kp and Vp are at row pr
          const uint8_t* none = static_cast<const uint8_t*>(a.Kp);
          if (k_on) cp16(base + up + At::k_at(r, pc), bytes ? Kp + row * d : none, bytes);
          if (v_on) cp16(base + up + At::kTileBytes + At::v_at(r, pc), bytes ? Vp + row * v : none, bytes);
        }
        // Exponents byte by byte; the products' loads come after the next barriers of the warp.
        const unsigned ke = on ? __ldg(a.Ks + mine) : 0u, ve = on ? __ldg(a.Vs + mine) : 0u;
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + s * 64 + lane), "r"(ke) : "memory");
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(scales + s * 64 + 32 + lane), "r"(ve) : "memory");
      }
      if (lane == 0) tile_keys[warp][s] = have;
      p_key += kTile;
      --p_left;
    }
    cp_commit();
    if (i < 0 || i >= issued) continue;
    cp_wait<S - 1>();
    __syncwarp();  // tile i is in
    const uint32_t at = base + (i % S) * kStage;
    st.tile(at, at + At::kTileBytes, scales + (i % S) * 64, tile_keys[warp][i % S], key0, sp, v, a.sl2, qs);
    key0 += kTile;
    if (--left > 0) continue;

    // The segment's rows.
    const PagedWalk w = walks[warp][1];
    int j0, j1;
    const int n = paged_segment<kTile>(w, j0, j1);
    const PagedPlace place = paged_place<kRows>(a, total, w, n, worker, lane == 0);
#pragma unroll
    for (int y = 0; y < NT; ++y) {
      size_t to[2];
      bool on[2];
      float f0[2], f1[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int q = 8 * y + 2 * t + x;
        on[x] = q < w.t.rows;
        float l = st.l[y][x];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        const size_t out = paged_out_row(a, w.s.s0, w.h, w.rt * kRows + (on[x] ? q : 0), w.s.prefix);
        const bool none = l == 0.f;  // no key
        const float m = none ? -INFINITY : st.m[y][x];
        PagedScale f{1.f, 0.f};
        if (place.slot < 0) f = paged_finish(m, l);
        to[x] = place.slot < 0 ? out : static_cast<size_t>(place.slot) * kRows + q;
        if (on[x] && g == 0) {
          if (a.info && place.parts >= 0) a.info[out] = make_int2(worker, place.parts);
          if (place.slot < 0) {
            a.L[out] = f.L;
          } else {
            a.pm[to[x]] = m;
            a.pl[to[x]] = l;
          }
        }
        // From the weights' reference point to the scores', in two factors: 2^(M - m) may be
        // subnormal where what it multiplies is not.
        f0[x] = none ? 0.f : ex2(0.5f * (st.M[y][x] - kLift - st.m[y][x]));
        f1[x] = f0[x] * f.fz;
      }
      float* z = place.slot < 0 ? a.Yf : a.pz;
      if (sizeof(T) == 4 && !z) z = static_cast<float*>(a.Y);
      if (z) {
#pragma unroll
        for (int c = 0; c < C / 8; ++c)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (on[x] && 8 * c < v) z[to[x] * v + 8 * c + g] = st.o[y][c >> 1][2 * (c & 1) + x] * f0[x] * f1[x];
        continue;
      }
      // Lane (g, t) stores row g of the tile, two columns at a time, after a transposition.
      const size_t r0 = __shfl_sync(0xFFFFFFFFu, to[0], g >> 1), r1 = __shfl_sync(0xFFFFFFFFu, to[1], g >> 1);
      __nv_bfloat16* mine = static_cast<__nv_bfloat16*>(a.Y) + (g & 1 ? r1 : r0) * v + 2 * t;
      const bool mine_on = 8 * y + g < w.t.rows;
#pragma unroll
      for (int c = 0; c < C / 8; ++c) {
        const float* o = &st.o[y][c >> 1][2 * (c & 1)];
        const uint32_t pair = transpose8(pack_bf16x2(o[0] * f0[0] * f1[0], o[1] * f0[1] * f1[1]));
        if (mine_on && 8 * c < v) *reinterpret_cast<uint32_t*>(mine + 8 * c) = pair;
      }
    }
  }
  cp_wait<0>();
  if (a.second) wait_for_previous();  // the next launch waits for this one alone
  paged_end(a, bits, &joined);
}

template <typename T, int C, int NT>
cudaError_t e4m3_launch(const PagedArgs& a, cudaStream_t s) {
  constexpr int bytes = smem_bytes<T, C, NT>();
  const cudaError_t e = allow_smem<paged_e4m3_kernel<T, C, NT>>(bytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  const cudaError_t le = launch_early(paged_e4m3_kernel<T, C, NT>, dim3(Config<T, C, NT>::kCtas), 32 * Config<T, C, NT>::kW, bytes, s, a);
  after_launch(kKernPaged, s);
  return le;
}

// The columns that a kernel is made for; of 256 with 8-row tiles alone, whose registers suffice.
int columns_of(int d, int v) {
  const int most = d > v ? d : v;
  return most <= 64 ? 64 : most <= 96 ? 96 : most <= 128 ? 128 : 256;
}
template <typename T>
cudaError_t e4m3_columns(const PagedArgs& a, int columns, int rows, cudaStream_t s) {
  switch (columns) {
    case 64: return rows == 8 ? e4m3_launch<T, 64, 1>(a, s) : e4m3_launch<T, 64, 2>(a, s);
    case 96: return rows == 8 ? e4m3_launch<T, 96, 1>(a, s) : e4m3_launch<T, 96, 2>(a, s);
    case 128: return rows == 8 ? e4m3_launch<T, 128, 1>(a, s) : e4m3_launch<T, 128, 2>(a, s);
    default: return e4m3_launch<T, 256, 1>(a, s);
  }
}
// Least units: see launch_paged_mma's; two, and one where the tables hold no more (place_pass).
template <typename T, int C, int NT>
constexpr PagedKernel e4m3_kernel() {
  return {8 * NT, Config<T, C, NT>::kCtas, Config<T, C, NT>::kCtas * Config<T, C, NT>::kW, 2};
}
template <typename T>
PagedKernel e4m3_kernel(int columns, int rows) {
  switch (columns) {
    case 64: return rows == 8 ? e4m3_kernel<T, 64, 1>() : e4m3_kernel<T, 64, 2>();
    case 96: return rows == 8 ? e4m3_kernel<T, 96, 1>() : e4m3_kernel<T, 96, 2>();
    case 128: return rows == 8 ? e4m3_kernel<T, 128, 1>() : e4m3_kernel<T, 128, 2>();
    default: return e4m3_kernel<T, 256, 1>();
  }
}

}  // namespace

PagedKernel paged_e4m3_kernel_of(int dtype, int d, int v, int rows) {
  const int columns = columns_of(d, v);
  return dtype == kF32 ? e4m3_kernel<float>(columns, rows) : e4m3_kernel<__nv_bfloat16>(columns, rows);
}
cudaError_t launch_paged_e4m3(const PagedArgs& a, int rows, cudaStream_t s) {
  const int columns = columns_of(a.d, a.v);
  return a.dtype == kF32 ? e4m3_columns<float>(a, columns, rows, s) : e4m3_columns<__nv_bfloat16>(a, columns, rows, s);
}

}  // namespace exattn
