// Paged attention over pages in 8 bits for few rows to a key head, widths up to 128: bound by
// reading K and V once.
//
// The shape of the kernel for 16-bit pages: a row tile is 8 or 16 rows in the N of the products
// S^T = K Q^T and O^T = V^T P^T, a worker is a warp that streams the 32-key tiles of its units
// through a ring of its own (16-byte asynchronous copies through the page table, running ahead over
// the ends of segments) and holds maximum, sum and output of its rows in registers.  An 8-bit tile
// of 32 keys is the bytes of a 16-bit one of 16.
//
// K meets Q as it is (m16n8k32 of e4m3, whose products are summed in fp32 as fp16's are, to 2^-24 of
// their magnitudes): a row of Q, scaled by the power of two that brings its largest entry to [128, 256),
// is the sum of two e4m3 parts, the second times 2^-4.  A part leaves 2^-5 of what it is given, so that
// two hold a bf16 entry exactly, down to a floor of 2^-21 of the row's largest.  (K as fp16, two
// conversions and a shift for four numbers: 8 sequences of 16384 keys 215 us in place of 185.)  fp32
// queries would be five parts; they are two fp16 parts, 2^-22 of themselves, their row's largest in
// [2^14, 2^15), and K is fp16 for them (18 us in place of 28, 12 x 2 rows of 80 columns over 3001 keys).
// V is fp16 (m16n8k16): an e4m3 number is one exactly.  No row's power of two enters an operand.
// A key's comes out of its score.  A value's goes into its
// weight: with s in the exp2 domain and e the exponent of V's row, w = s + e, and the operand is
// 2^(w - M + 7) with M a reference point of its own (the sum l keeps s's), so that unequal rows of V
// lose nothing; 2^7 puts the largest weight in the middle of fp16's range above its subnormals, and a
// weight is held to 2^-11 of itself or 2^-32 of the row's largest; for fp32 queries two parts, 2^-22.
// The reference points move only when a row's maximum passes them by more than 2^8, which a vote
// tells without the maximum.
//
// A lane reads 16 columns of a key at once: the products' inner index is permuted so that lane t of
// a quad has columns 16 t .. 16 t + 15 (and those 64 on), eight a step, of the queries
// too.  Key 4 g + j of the tile is row g of the quarter j, so that a lane's four keys' exponents are one
// word and its masks one nibble.  V comes transposed in 16-bit units (ldmatrix): two columns of
// one key, which two byte permutations and two conversions turn into two keys of one column.
#include <cuda_fp16.h>

#include <type_traits>
#include <utility>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

using tc::ex2;
using tc::fadd2;
using tc::ffma2;
using tc::fmul2;
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
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
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
__device__ __forceinline__ void mma32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two numbers as e4m3, a in the low byte; x becomes what the rounding left out, times 16.
__device__ __forceinline__ uint32_t take_e4m3(float& a, float& b) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b), "f"(a));
  const uint32_t h = e4m3_pair(y);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
  a = (a - x.x) * 16.f;
  b = (b - x.y) * 16.f;
  return y;
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
// the eight lanes of a phase meet eight banks' groups: keys 4 g + j of neighbouring g for K (bit 2 of
// the row), of eight g for V.
template <int D>
struct Place {
  static constexpr int CH = D / 16;        // pieces of a row
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kRows = 32 / CH;    // rows that a warp copies at once, 512 bytes
  static __device__ __forceinline__ uint32_t at(int r, int c, int swizzle) {
    return D == 128 ? r * 128 + ((c ^ swizzle) << 4) : (r >> 1) * 128 + (((((r & 1) << 2) | c) ^ swizzle) << 4);
  }
  static __device__ __forceinline__ uint32_t k_at(int r, int c) { return at(r, c, r & 4); }
  static __device__ __forceinline__ uint32_t v_at(int r, int c) { return at(r, c, (r >> 2) & 7); }
};

template <typename T, int D, int NT>
struct Config {
  static constexpr bool kMany = std::is_same<T, __nv_bfloat16>::value && NT == 1;
  static constexpr int kW = 4, kStages = kMany ? 2 : 3, kCtas = (kMany ? 3 : 2) * 152;
};

template <typename T> struct Parts;  // of a query's entry and of a weight
template <> struct Parts<__nv_bfloat16> {
  static constexpr int N = 1;
  static constexpr bool kE4m3 = true;  // the query's, two; else N fp16 parts
  // Sixteen columns.
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* x) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint4 raw = *reinterpret_cast<const uint4*>(p + 8 * y);
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[8 * y + 2 * i] = __uint_as_float(w[i] << 16);
        x[8 * y + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};
template <> struct Parts<float> {
  static constexpr int N = 2;
  static constexpr bool kE4m3 = false;
  static __device__ __forceinline__ void load(const float* p, float* x) {
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const float4 q = *reinterpret_cast<const float4*>(p + 4 * y);
      x[4 * y] = q.x, x[4 * y + 1] = q.y, x[4 * y + 2] = q.z, x[4 * y + 3] = q.w;
    }
  }
};

// The keys that a thread's rows allow, and those that every row of the tile does.
template <int NT>
struct Spans {
  int lo[NT][2], hi[NT][2], all_lo, all_hi;
};

// A worker's rows over a segment.  Thread (g, t) = (lane / 4, lane % 4) holds the operands of rows
// 8 n + g, and of rows 8 n + 2 t + x the factor of their scores, the reference points m and M, the sum
// over its own keys l, and of the output o[n][y] columns 16 y + 2 g (x = 0, 1) and 16 y + 2 g + 1.
template <typename T, int D, int NT>
struct Rows {
  static constexpr int P = Parts<T>::N, K = D / 16;
  static constexpr bool kE4m3 = Parts<T>::kE4m3;
  static constexpr int kSteps = kE4m3 ? D / 32 : K;
  uint32_t qb[NT][2][kSteps][2];
  float f[NT][2], m[NT][2], M[NT][2], l[NT][2], o[NT][K][4];

  // Row n of the tile's row 8 n + g.
  __device__ __forceinline__ void load_q(int n, const T* row, bool on, int d, float sl2) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float x[D / 64][16];
    unsigned top = 0u;
#pragma unroll
    for (int h = 0; h < D / 64; ++h) {
      const int c = 64 * h + 16 * t;
      if (on && c < d) {
        Parts<T>::load(row + c, x[h]);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[h][e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[h][e]) & 0x7FFFFFFFu);
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const unsigned e = max(top >> 23, 15u);  // the largest is below 2^(e - 126)
    constexpr unsigned kUp = kE4m3 ? 261u : 268u;  // 254 and 8 bits, or 15
    const float up = __uint_as_float((kUp - e) << 23), down = __uint_as_float((e - (kUp - 254u)) << 23) * sl2;
#pragma unroll
    for (int h = 0; h < D / 64; ++h)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float(&z)[16] = x[h];
#pragma unroll
        for (int c = 4 * w; c < 4 * w + 4; ++c) z[c] = fmaf(z[c], up, z[c] * 0.f);  // an infinity: NaN
        if constexpr (kE4m3) {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t lo = take_e4m3(z[4 * w], z[4 * w + 1]), hi = take_e4m3(z[4 * w + 2], z[4 * w + 3]);
            qb[n][p][2 * h + (w >> 1)][w & 1] = lo | hi << 16;
          }
        } else {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float a = z[4 * w + 2 * y], b = z[4 * w + 2 * y + 1];
            const uint32_t hi = pack_f16x2(a, b);
            qb[n][0][4 * h + w][y] = hi;
            qb[n][1][4 * h + w][y] = rest_f16x2(a, b, hi);
          }
        }
      }
#pragma unroll
    for (int x2 = 0; x2 < 2; ++x2) f[n][x2] = __shfl_sync(0xFFFFFFFFu, down, 4 * (2 * t + x2));
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
                                       const Spans<NT>& sp, int v) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const uint32_t ke = lds32(et + 4 * g), ve = lds32(et + 32 + 4 * g);
    // [row tile][pair of quarters j = 2 q, 2 q + 1][2 (j & 1) + row]; the second e4m3 part's.
    float sc[NT][2][4], low[NT][2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[n][q][e] = low[n][q][e] = 0.f;
    {
      const uint32_t at = kt + Place<D>::k_at(4 * g, lane & 3);
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        uint4 k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          k[j] = ld_shared_v4(D == 128 ? (at ^ (h << 6)) + j * 128 : (at ^ ((j & 1) << 6)) + (j >> 1) * 128);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            auto word = [&](const uint4& x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; };
            if constexpr (kE4m3) {
              if (w & 1) continue;  // two words a step
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                  mma32(p ? low[n][q] : sc[n][q], word(k[2 * q], w), word(k[2 * q + 1], w), word(k[2 * q], w + 1),
                        word(k[2 * q + 1], w + 1), qb[n][p][2 * h + (w >> 1)][0], qb[n][p][2 * h + (w >> 1)][1]);
            } else {
              const uint32_t x0 = word(k[2 * q], w), x1 = word(k[2 * q + 1], w);
              const uint32_t a[4] = {e4m3_pair(x0), e4m3_pair(x1), e4m3_pair_high(x0), e4m3_pair_high(x1)};
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < 2; ++p)
                  mma16(sc[n][q], a, qb[n][p][4 * h + w][0], qb[n][p][4 * h + w][1]);
            }
          }
      }
    }
    // Scores into the exp2 domain, those that do not count to -inf; w beside them.
    const bool whole = have == 0xFFFFFFFFu && key0 >= sp.all_lo && key0 + kTile <= sp.all_hi;
    float wt[NT][2][4], over = kNoKey;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int j = 2 * q + z;
          const float kf = e4m3_scale((ke >> (8 * j)) & 255u);
          const float vx = __uint_as_float(0x4B000000u | ((ve >> (8 * j)) & 255u)) - 8388735.f;  // byte - 127
          float &s0 = sc[n][q][2 * z], &s1 = sc[n][q][2 * z + 1], f0, f1;
          if (kE4m3) ffma2(s0, s1, low[n][q][2 * z], low[n][q][2 * z + 1], 0x1p-4f, 0x1p-4f, s0, s1);
          fmul2(f0, f1, f[n][0], f[n][1], kf, kf);
          fmul2(s0, s1, s0, s1, f0, f1);
          if (!whole) {
            const int key = 4 * g + j;
#pragma unroll
            for (int x = 0; x < 2; ++x)
              if (!((have >> key) & 1u) || key0 + key < sp.lo[n][x] || key0 + key >= sp.hi[n][x])
                sc[n][q][2 * z + x] = -INFINITY;
          }
          float &w0 = wt[n][q][2 * z], &w1 = wt[n][q][2 * z + 1];
          fadd2(w0, w1, s0, s1, vx, vx);
          over = fmaxf(over, fmaxf(fmaxf(s0 - m[n][0], s1 - m[n][1]), fmaxf(w0 - M[n][0], w1 - M[n][1])));
        }
    if (__any_sync(0xFFFFFFFFu, over > kRescale)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // Each row by itself: what the others hold does not change its bits.
          const float to = max_over_keys(max4(sc[n], x)), To = max_over_keys(max4(wt[n], x));
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
          fadd2(s0, s1, sc[n][q][2 * z], sc[n][q][2 * z + 1], -m[n][0], -m[n][1]);
          fadd2(w0, w1, wt[n][q][2 * z], wt[n][q][2 * z + 1], R0, R1);
          fadd2(l[n][0], l[n][1], l[n][0], l[n][1], ex2(s0), ex2(s1));
          const float p0 = ex2(w0), p1 = ex2(w1);
          const uint32_t hi = pack_f16x2(p0, p1);
          pb[n][0][q][z] = transpose8(hi);
          if (P == 2) pb[n][P - 1][q][z] = transpose8(rest_f16x2(p0, p1, hi));
        }
    }
    {
      const uint32_t at = vt + Place<D>::v_at(4 * (lane & 7) + (lane >> 3), 0);
#pragma unroll
      for (int y = 0; y < K; ++y) {
        // (A branch for every y keeps the steps apart: 16 rows over 262147 keys 141 us in place of 129.)
        if (y == 4 && v <= 64) break;
        uint32_t r[4];  // quarter j: columns 2 g and 2 g + 1 of keys 2 t and 2 t + 1 of it
        ldm4t(r, at ^ (y << 4));
        uint32_t a[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[j >> 1][2 * (j & 1)] = e4m3_pair(__byte_perm(r[j], 0u, 0x4420));
          a[j >> 1][2 * (j & 1) + 1] = e4m3_pair(__byte_perm(r[j], 0u, 0x4431));
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (P == 1) {
#pragma unroll
            for (int q = 0; q < 2; ++q) mma16(o[n][y], a[q], pb[n][0][q][0], pb[n][0][q][1]);
          } else {
            // A tile's products are summed by the tensor cores, which cut their sums instead of
            // rounding them, and added to the output in rounded fp32.
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int p = P - 1; p >= 0; --p) mma16(sum, a[q], pb[n][p][q][0], pb[n][p][q][1]);
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
  (cp16_at<512 * X, 512 * X>((k ^ (CH == 8 ? (X & 1) << 6 : 0)) + up, kf), ...);
  (cp16_at<512 * X, 512 * X>((v ^ (CH == 8 ? X << 4 : X << 5)) + up, vf), ...);
}

template <typename T, int D, int NT>
constexpr int smem_bytes() {
  return Config<T, D, NT>::kW * Config<T, D, NT>::kStages * (2 * Place<D>::kTileBytes + 64);
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * Config<T, D, NT>::kW, Config<T, D, NT>::kCtas / 152)
    paged_e4m3_kernel(const PagedArgs a) {
  using At = Place<D>;
  constexpr int S = Config<T, D, NT>::kStages, kW = Config<T, D, NT>::kW, kRows = 8 * NT, CH = At::CH;
  constexpr int kStage = 2 * At::kTileBytes;
  extern __shared__ __align__(128) uint8_t sm[];
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
  const bool dense = d == D && v == D && lpk == 5;
  int issued = 0;  // tiles copied so far
  // The products' segment.
  int left = 0, key0 = 0;
  Spans<NT> sp;
  Rows<T, D, NT> st;

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
          st.load_q(y, static_cast<const T*>(a.Q) + (w.s.s0 + tok) * a.q_stride + (w.h * a.G + r - tok * a.G) * d,
                    q < w.t.rows, d, a.sl2);
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
      if (dense && page0 >= 0 && p_key >= p_j0 && p_key + kTile <= p_j1) {
        // All keys, of one page, in rows of D bytes: one stretch of memory.
        const long long row = ((static_cast<long long>(page0) * a.Hk + p_h) << a.lps) + (p_key & ((1 << a.lps) - 1));
        copy_dense<CH>(k_to, v_to, up, Kp + row * D, Vp + row * D, std::make_integer_sequence<int, CH>{});
        if (lane < 16) cp4(scales + s * 64 + 4 * lane, Ep + row + 4 * (lane & 7), 4);
        have = 0xFFFFFFFFu;
      } else {
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
      auto copy = [&](auto whole) {
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          const int z = CH == 8 ? x >> 1 : x, on = CH == 8 ? 4 * (x & 1) : 0;
          const int bytes = whole ? 16 : ((have >> (pr + At::kRows * x)) & 1u) << 4;
          // Rows kRows x further: 512 bytes, and the swizzle's bits of x.
          const uint32_t k_x = CH == 8 ? (x & 1) << 6 : 0, v_x = CH == 8 ? x << 4 : x << 5;
          if (k_on) cp16((k_to ^ k_x) + up + 512 * x, Kp + (row[z] + on) * d, bytes);
          if (v_on) cp16((v_to ^ v_x) + up + 512 * x, Vp + (row[z] + on) * v, bytes);
        }
      };
      if (have == 0xFFFFFFFFu) copy(std::true_type{});
      else copy(std::false_type{});
      if (lane < 16) {
        const int z = (lane >> 1) & 3;
        const long long from = z == 0 ? row[0] : z == 1 ? row[1] : z == 2 ? row[2] : row[3];
        cp4(scales + s * 64 + 4 * lane, Ep + from + 4 * (lane & 1), (have >> 8 * z) & 0xFFu ? 4 : 0);
      }
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
    st.tile(at, at + At::kTileBytes, scales + (i % S) * 64, tile_keys[warp][i % S], key0, sp, v);
    key0 += kTile;
    if (--left > 0) continue;

    // The segment's rows.
    const PagedWalk w = walks[warp][1];
    int j0, j1;
    const int n = paged_segment<kTile>(w, j0, j1);
    const PagedPlace place = paged_place<kRows>(a, total, w, n, worker, lane == 0);
#pragma unroll
    for (int y = 0; y < NT; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int q = 8 * y + 2 * t + x;
        const bool on = q < w.t.rows;
        float l = st.l[y][x];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (!on) continue;
        const size_t out = paged_out_row(a, w.s.s0, w.h, w.rt * kRows + q, w.s.prefix);
        if (a.info && place.parts >= 0 && g == 0) a.info[out] = make_int2(worker, place.parts);
        // From the weights' reference point to the scores', in two factors: 2^(M - m) may be
        // subnormal where what it multiplies is not.
        const bool none = l == 0.f;  // no key
        const float half = none ? 0.f : ex2(0.5f * (st.M[y][x] - kLift - st.m[y][x])), m = none ? -INFINITY : st.m[y][x];
        PagedScale f{1.f, 0.f};
        if (place.slot < 0) {
          f = paged_finish(m, l);
          if (g == 0) a.L[out] = f.L;
        } else if (g == 0) {
          a.pm[static_cast<size_t>(place.slot) * kRows + q] = m;
          a.pl[static_cast<size_t>(place.slot) * kRows + q] = l;
        }
        const float rest = half * f.fz;
        float* z = place.slot < 0 ? a.Yf : a.pz;
        const size_t to = (place.slot < 0 ? out : static_cast<size_t>(place.slot) * kRows + q) * v;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const int col = 16 * c + 2 * g;
          if (16 * c >= v) break;
          const float z0 = st.o[y][c][x] * half * rest, z1 = st.o[y][c][2 + x] * half * rest;
          if (z) *reinterpret_cast<float2*>(z + to + col) = make_float2(z0, z1);
          else if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(static_cast<float*>(a.Y) + to + col) = make_float2(z0, z1);
          else *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.Y) + to + col) = pack_bf16x2(z0, z1);
        }
      }
  }
  cp_wait<0>();
  if (a.second) wait_for_previous();  // the next launch waits for this one alone
  paged_end(a, bits, &joined);
}

template <typename T, int D, int NT>
cudaError_t e4m3_launch(const PagedArgs& a, cudaStream_t s) {
  constexpr int bytes = smem_bytes<T, D, NT>();
  const cudaError_t e = allow_smem<paged_e4m3_kernel<T, D, NT>>(bytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  const cudaError_t le = launch_early(paged_e4m3_kernel<T, D, NT>, dim3(Config<T, D, NT>::kCtas), 32 * Config<T, D, NT>::kW, bytes, s, a);
  after_launch(kKernPaged, s);
  return le;
}

template <typename T>
cudaError_t e4m3_columns(const PagedArgs& a, int rows, cudaStream_t s) {
  if (a.d <= 64 && a.v <= 64) return rows == 8 ? e4m3_launch<T, 64, 1>(a, s) : e4m3_launch<T, 64, 2>(a, s);
  return rows == 8 ? e4m3_launch<T, 128, 1>(a, s) : e4m3_launch<T, 128, 2>(a, s);
}
template <typename T, int D, int NT>
constexpr PagedKernel e4m3_kernel() {
  return {8 * NT, Config<T, D, NT>::kCtas, Config<T, D, NT>::kCtas * Config<T, D, NT>::kW, 2};
}
template <typename T>
PagedKernel e4m3_kernel(bool narrow, int rows) {
  if (narrow) return rows == 8 ? e4m3_kernel<T, 64, 1>() : e4m3_kernel<T, 64, 2>();
  return rows == 8 ? e4m3_kernel<T, 128, 1>() : e4m3_kernel<T, 128, 2>();
}

}  // namespace

// Eight rows of a page behind one another are what the copies count in.
bool paged_e4m3_shape(int d, int v, int lps) { return d <= 128 && v <= 128 && lps >= 3; }
PagedKernel paged_e4m3_kernel_of(int dtype, int d, int v, int rows) {
  const bool narrow = d <= 64 && v <= 64;
  return dtype == kF32 ? e4m3_kernel<float>(narrow, rows) : e4m3_kernel<__nv_bfloat16>(narrow, rows);
}
cudaError_t launch_paged_e4m3(const PagedArgs& a, int rows, cudaStream_t s) {
  return a.dtype == kF32 ? e4m3_columns<float>(a, rows, s) : e4m3_columns<__nv_bfloat16>(a, rows, s);
}

}  // namespace exattn
