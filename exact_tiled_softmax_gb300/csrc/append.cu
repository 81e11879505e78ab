// New keys and values into a paged cache, with the rotary position embedding
// applied to keys (and to the queries beside them) on the way.
//
// Token t of sequence b is at position pos = len - nq + i.  Pair f of a
// rotated row turns by (pos + pos_offset) * inv_freq[f]:
//   x' = x cos - y sin,  y' = y cos + x sin,
// pairs (f, f + pairs) or, interleaved, (2f, 2f + 1); other columns pass.
// Bound by memory: every element is read once and written once, in 16-byte accesses
// where the rotated halves allow them.  A warp takes a token (or a share of its rows):
// it finds the token's place and angles once for all heads.  What hides the latency is
// warps, not loads of a lane: six CTAs to an SM with 32 bytes in flight a lane move 36
// thousand tokens of 48 rows of 128 bf16 columns at 6.20 TB/s (91% of the measured copy);
// before the angles left double precision it was 5.94, and then two rows at four CTAs 5.41,
// four rows at two CTAs 4.05, and in fp32 six CTAs 5.74, five 5.01.  One CTA more checks
// that every token has a place and writes the status word.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kMaxPairs = 128;
// Pages in 8 bits.  CTAs of an SM: seven of four warps 144 us for 37 thousand tokens of 32 + 8 + 8 rows of 128
// bf16 columns (5.7 TB/s, 84% of the measured copy), six 148, five 154; three of eight 151, four, which
// spill, 161.  A second pass's loads ahead: no difference.
constexpr int kThreads8 = 128, kWarps8 = kThreads8 / 32, kAppendCtas8 = 7;
constexpr int kMaxPasses = 1 << 17;  // more than a token's rows

// The sequence that owns token t, or -1.
__device__ __forceinline__ int owner(const AppendArgs& a, int t) {
  if (!a.starts) return t / a.each;
  if (t >= __ldg(a.starts + a.B) || t < __ldg(a.starts)) return -1;
  int b0 = 0, b1 = a.B;  // starts[b0] <= t < starts[b1]
  while (b1 - b0 > 1) {
    const int mid = (b0 + b1) >> 1;
    if (__ldg(a.starts + mid) <= t) b0 = mid;
    else b1 = mid;
  }
  return b0;
}

// W consecutive elements in one access, and as fp32.
template <typename T, int W>
struct alignas(W * sizeof(T)) Piece {
  T x[W];
};
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float& x, float f) { x = f; }
__device__ __forceinline__ void from_float(__nv_bfloat16& x, float f) { x = __float2bfloat16_rn(f); }

// Whole turns that an angle of `freq` radians makes are dropped in fixed point: the turns of
// one position, freq / (2 pi) modulo 1 in units of 2^-64.  freq is M 2^E, M below 2^24, and
// 2^64 / (2 pi) an integer to 2^-65, so the result is off by 2^-64 (1 + |freq| / 2) at most,
// and by p times that after p positions.  (Double precision, 2 operations a clock and SM,
// took 1 us of a decode step's 4.7 and 6% of a long prompt's time.)
__device__ __forceinline__ unsigned long long turns_of(float freq) {
  constexpr unsigned long long kInv2Pi = 0x28be60db9391054aull;  // 2^64 / (2 pi)
  const unsigned x = __float_as_uint(freq), e = (x >> 23) & 255u;
  const unsigned long long m = (x & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int down = 150 - static_cast<int>(e ? e : 1u);  // -E
  unsigned long long f;
  if (down <= 0) f = down > -64 ? lo << -down : 0ull;
  else if (down < 64) f = (lo >> down) | (hi << (64 - down));
  else f = down < 128 ? hi >> (down - 64) : 0ull;
  return x >> 31 ? 0ull - f : f;
}

// cos and sin of pos * freq.  Quarter turns are taken out in fixed point too: what is left is
// rounded to fp32 at an eighth of a turn at most, off by 2^-28 turns, four times less than whole
// angles.
__device__ __forceinline__ void angle(long long pos, float freq, float& sn, float& cs) {
  const unsigned long long t = static_cast<unsigned long long>(pos) * turns_of(freq);
  const unsigned long long quarter = (t + (1ull << 61)) >> 62;
  const int rest = static_cast<int>((t - (quarter << 62)) >> 32);  // 2^-32 turns are cut off
  float s, c;
  sincospif(isfinite(freq) ? static_cast<float>(rest) * 0x1p-31f : NAN, &s, &c);
  sn = quarter & 1 ? c : s;
  cs = quarter & 1 ? -s : c;
  if (quarter & 2) {
    sn = -sn;
    cs = -cs;
  }
}

// Status: whether every new token has a place.  A thread takes a sequence at a time, a
// warp the pages of a long one.
__device__ void append_check(const AppendArgs& a) {
  bool bad = false;
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int b0 = (threadIdx.x & ~31); b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + lane;
    int first = 0, last = -1;  // pages of the new tokens
    if (b < a.B) {
      int nq = a.T / a.B;
      if (a.starts) {
        const int x = __ldg(a.starts + b), y = __ldg(a.starts + b + 1);
        bad |= x < 0 || y < x || y > a.T;
        nq = min(max(y, 0), a.T) - min(max(x, 0), a.T);
      }
      const int n = __ldg(a.lens + b);
      const int cap = a.max_pages << a.lps;
      bad |= n < 0 || n > cap;
      if (nq > 0) {
        bad |= n < nq;
        first = max(0, min(n, cap) - nq) >> a.lps;
        last = n > 0 ? (min(n, cap) - 1) >> a.lps : -1;
      }
    }
    auto outside = [&](int of, int p) {
      return static_cast<unsigned>(__ldg(a.table + static_cast<size_t>(of) * a.max_pages + p)) >=
             static_cast<unsigned>(a.num_pages);
    };
    const bool many = last - first >= 4;
#pragma unroll 1
    for (int p = first; !many && p <= last; ++p) bad |= outside(b, p);
#pragma unroll 1
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, many); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      const int f = __shfl_sync(0xFFFFFFFFu, first, who), e = __shfl_sync(0xFFFFFFFFu, last, who);
      for (int p = f + lane; p <= e; p += 32) bad |= outside(b0 + who, p);
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = any ? kStatusBadPage : 0u;
}

// The pairs (2f, 2f + 1) of a 16-byte piece, which starts at column `col`, turned.
template <typename T, int W>
__device__ __forceinline__ void turn_inside(Piece<T, W>& x, const float* cs, const float* sn, int col, int pairs) {
  const Piece<float, W / 2> c = *reinterpret_cast<const Piece<float, W / 2>*>(cs + col / 2),
                            s = *reinterpret_cast<const Piece<float, W / 2>*>(sn + col / 2);
#pragma unroll
  for (int e = 0; e < W; e += 2) {
    if ((col + e) >> 1 >= pairs) continue;
    const float x0 = as_float(x.x[e]), x1 = as_float(x.x[e + 1]);
    from_float(x.x[e], x0 * c.x[e / 2] - x1 * s.x[e / 2]);
    from_float(x.x[e + 1], x1 * c.x[e / 2] + x0 * s.x[e / 2]);
  }
}

// W: elements of an access.  A row of q or k is cut into units: interleaved, unit u is
// access u; else units below pairs / W are the accesses u W and pairs + u W of the two
// halves, those above two neighbouring accesses of the columns that pass.
template <typename T, int W, bool kInterleaved>
__global__ void __launch_bounds__(kAppendThreads, 6) append_kernel(const __grid_constant__ AppendArgs a) {
  wait_for_previous();
  let_next_start();
  if (blockIdx.x == gridDim.x - 1) {
    append_check(a);
    return;
  }
  __shared__ __align__(32) float cs[kAppendWarps][kMaxPairs];
  __shared__ __align__(32) float sn[kAppendWarps][kMaxPairs];
  using P = Piece<T, W>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int job = blockIdx.x * kAppendWarps + warp;  // share `job % shares` of token job / shares
  const int t = div_by(job, a.by_shares), share = job - t * a.by_shares.d;
  if (t >= a.T) return;
  const int b = owner(a, t);
  if (b < 0) return;  // behind the last sequence
  int s0 = b * a.each, nq = a.each;
  if (a.starts) {  // clamped, as the attention does
    s0 = max(__ldg(a.starts + b), 0);
    nq = min(__ldg(a.starts + b + 1), a.T) - s0;
  }
  const int pos = max(__ldg(a.lens + b), 0) - nq + (t - s0);
  long long slot = -1;  // the token's row of the pool (of key head 0); -1: nowhere
  if (pos >= 0 && pos < a.max_pages << a.lps) {
    const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (pos >> a.lps));
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
      slot = (static_cast<long long>(page) * a.Hk << a.lps) + (pos & ((1 << a.lps) - 1));
  }
  const long long at = static_cast<long long>(pos) + a.pos_offset;
  for (int f = lane; f < a.pairs; f += 32) angle(at, __ldg(a.inv_freq + f), sn[warp][f], cs[warp][f]);
  __syncwarp();

  const int units = a.by_units.d, half = a.pairs / W;
  const int rows = (a.q ? a.H : 0) + a.Hk, q_rows = rows - a.Hk;
  const T* qsrc = static_cast<const T*>(a.q) + t * a.qs;
  const T* ksrc = static_cast<const T*>(a.k) + t * a.ks;
  T* qdst = static_cast<T*>(a.q_out) + static_cast<size_t>(t) * a.H * a.d;
  T* kdst = static_cast<T*>(a.kp) + slot * a.d;
  if constexpr (kInterleaved) {
    // Every lane a piece, whatever the row's width, and two pieces in flight.
    const int all = (slot < 0 ? q_rows : rows) * units;
#pragma unroll 1
    for (int i0 = share * 64 + lane; i0 < all; i0 += 64 * a.by_shares.d) {
      P x[2];
      T* dst[2];
      int col[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int i = min(i0 + 32 * z, all - 1), r = div_by(i, a.by_units);
        col[z] = (i - r * units) * W;
        x[z] = *reinterpret_cast<const P*>((r < q_rows ? qsrc + r * a.d : ksrc + (r - q_rows) * a.d) + col[z]);
        dst[z] = (r < q_rows ? qdst + r * a.d : kdst + (static_cast<long long>(r - q_rows) << a.lps) * a.d) + col[z];
      }
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        turn_inside<T, W>(x[z], cs[warp], sn[warp], col[z], a.pairs);
        if (z == 0 || i0 + 32 < all) *reinterpret_cast<P*>(dst[z]) = x[z];
      }
    }
  } else {
    const int across = units < 32 ? units : 32, rpp = units < 32 ? div_by(32, a.by_units) : 1;  // rows of a pass
    const int sub = units < 32 ? div_by(lane, a.by_units) : 0;
    const int step = rpp * a.by_shares.d;
#pragma unroll 1
    for (int u0 = 0; u0 < units; u0 += 32) {
      const int u = u0 + lane - sub * across;
      const bool two = u < half;
      const int col = (two ? u : 2 * u) * W, to_second = two ? a.pairs : W;
      const bool second = col + to_second < a.d;
      if (sub >= rpp || u >= units) continue;
#pragma unroll 1
      for (int r = share * rpp + sub; r < rows; r += step) {
        const bool is_q = r < q_rows;
        const T* src = (is_q ? qsrc + r * a.d : ksrc + (r - q_rows) * a.d) + col;
        P x = *reinterpret_cast<const P*>(src), y;
        if (second) y = *reinterpret_cast<const P*>(src + to_second);
        if (!is_q && slot < 0) continue;
        if (two) {
          const Piece<float, W> c = *reinterpret_cast<const Piece<float, W>*>(&cs[warp][u * W]),
                                s = *reinterpret_cast<const Piece<float, W>*>(&sn[warp][u * W]);
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float x0 = as_float(x.x[e]), x1 = as_float(y.x[e]);
            from_float(x.x[e], x0 * c.x[e] - x1 * s.x[e]);
            from_float(y.x[e], x1 * c.x[e] + x0 * s.x[e]);
          }
        }
        T* dst = (is_q ? qdst + r * a.d : kdst + (static_cast<long long>(r - q_rows) << a.lps) * a.d) + col;
        *reinterpret_cast<P*>(dst) = x;
        if (second) *reinterpret_cast<P*>(dst + to_second) = y;
      }
    }
  }
  if (slot < 0) return;
  const int vch = a.by_vch.d;
  const uint4* vsrc = reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + t * a.vs);
  uint4* vdst = reinterpret_cast<uint4*>(static_cast<T*>(a.vp) + slot * a.vw);
#pragma unroll 2
  for (int i = share * 32 + lane; i < a.Hk * vch; i += 32 * a.by_shares.d) {
    const int h = div_by(i, a.by_vch);
    vdst[(static_cast<long long>(h) << a.lps) * vch + (i - h * vch)] = vsrc[i];
  }
}

template <typename T, int W, bool kInterleaved>
cudaError_t append_launch(AppendArgs a, cudaStream_t s) {
  a.each = a.T / a.B;
  a.by_units = fast_div(kInterleaved ? a.d / W : (a.d / W + 1) / 2);
  a.by_vch = fast_div(a.vw * static_cast<int>(sizeof(T)) / 16);
  // A token's rows are shared out while that leaves warps without work: a decode step's
  // few tokens are a matter of latency.
  int shares = 1;
  while (shares < kAppendWarps && (long long)a.T * shares * 2 <= 152 * 16 && shares < a.Hk) shares *= 2;
  a.by_shares = fast_div(shares);
  const unsigned ctas = (static_cast<unsigned>(a.T) * shares + kAppendWarps - 1) / kAppendWarps;
  before_launch(kKernAppend, s);
  const cudaError_t e = launch_early(append_kernel<T, W, kInterleaved>, dim3(ctas + 1), kAppendThreads, 0, s, a);
  after_launch(kKernAppend, s);
  return e;
}

template <typename T>
cudaError_t append_dispatch(const AppendArgs& a, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  // The widest access that neither half of the rotated columns breaks up.
  if (a.interleaved) return append_launch<T, E, true>(a, s);
  if (a.pairs % E == 0) return append_launch<T, E, false>(a, s);
  if (a.pairs % (E / 2) == 0) return append_launch<T, E / 2, false>(a, s);
  return append_launch<T, 1, false>(a, s);
}

// ------------------------------------------------------------------ pages in 8 bits
//
// A row y of w columns (rotated or not) becomes an exponent byte b, the smallest from 1 on with
// max |y| <= 448 * 2^(b - 127), and RN_e4m3(y * 2^(127 - b)): the scaling is exact.  kLanes lanes
// hold a row, 16 columns each, so that its maximum is three or four shuffles away and nothing is
// read twice.
//
// A rotated entry's fp32 value is off by some 2^-22 of the pair's length (sine and cosine by 2^-23.5,
// products and sum by 2^-24 each), so its rounding to 4 bits is settled unless a border lies that
// near: once in 2^16 entries.  Such entries are computed again in 64 bits (FP64 does two operations
// a clock and SM: a pair costs a warp half a microsecond), and so are the largest of a row whose
// maximum lies that near to 448 times a power of two.  The codes are those of 64-bit arithmetic.
// Behind the first position the bound does not know of pairs that their rotation leaves as they are (frequencies of zero):
// of their bf16 entries one in 16 lies on a border, and 37 thousand tokens with half of 64 such take 612 us in place of
// 144.  Nor does it know of columns behind the last pair in a lane that has pairs, in halves of a number of pairs that is
// no multiple of 8.
constexpr float kTurnError = 4e-7f;  // > 2^-22 sqrt(2), of the sum of the pair's magnitudes, before or after

// Where the pairs of a row are: halves that 8-column accesses reach, neighbours, or anywhere.
enum PairForm { kHalves, kInside, kAnywhere };

// Entry c of a row, rotated in 64 bits by the exact angle.
template <typename T>
__device__ __noinline__ double turned64(const T* row, int c, int pairs, bool inside, long long pos,
                                        const float* inv_freq) {
  if (c >= 2 * pairs) return as_float(row[c]);
  const int f = inside ? c >> 1 : c < pairs ? c : c - pairs;
  const bool first = inside ? !(c & 1) : c < pairs;
  const int other = inside ? c ^ 1 : first ? c + pairs : f;
  // Behind position 2^29 the angle may not fit 53 bits: what its rounding left out, at most 2^-16 radians, is
  // turned by afterwards (1 - rest^2 / 2 and rest are its cosine and sine to 2^-50).
  const double at = static_cast<double>(pos), freq = static_cast<double>(__ldg(inv_freq + f));
  const double angle = at * freq, rest = fma(at, freq, -angle);
  double s0, k0;
  sincos(angle, &s0, &k0);
  const double less = 0.5 * rest * rest, s = fma(k0, rest, fma(-s0, less, s0)), k = fma(-s0, rest, fma(-k0, less, k0));
  const double x = as_float(row[c]), y = as_float(row[other]);
  return first ? x * k - y * s : x * k + y * s;
}

// (a, b) rounded to e4m3, a in the low byte; magnitudes up to 448, NaN stays.
__device__ __forceinline__ uint32_t e4m3_of(float a, float b) {
  uint16_t y;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(b), "f"(a));
  return y;
}
__device__ __forceinline__ uint32_t e4m3_of(double z) {
  float f = __double2float_rz(z);  // to odd, so that the second rounding is the only one
  if (static_cast<double>(f) != z) f = __uint_as_float(__float_as_uint(f) | 1u);
  return e4m3_of(f, 0.f) & 0xFFu;
}

// The exponent byte of a row whose largest magnitude has these fp32 bits.  448 is 1.75 * 2^8.
__device__ __forceinline__ int exponent_of(unsigned top) {
  return top == 0u ? 0 : max(1, static_cast<int>((top + 0x1FFFFFu) >> 23) - 8);
}
__device__ __forceinline__ int exponent_of(unsigned long long top) {
  return top == 0ull ? 0 : max(1, static_cast<int>((top + 0x3FFFFFFFFFFFFull) >> 52) - 1023 + 127 - 8);
}

// Eight columns from each of two places of a row, as they are loaded.
template <typename T> struct Raw16;
template <> struct Raw16<__nv_bfloat16> {
  uint4 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
    a = *reinterpret_cast<const uint4*>(p);
    b = *reinterpret_cast<const uint4*>(q);
  }
  __device__ __forceinline__ void to(float (&x)[16]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <> struct Raw16<float> {
  float4 v[4];
  __device__ __forceinline__ void load(const float* p, const float* q) {
    v[0] = *reinterpret_cast<const float4*>(p);
    v[1] = *reinterpret_cast<const float4*>(p + 4);
    v[2] = *reinterpret_cast<const float4*>(q);
    v[3] = *reinterpret_cast<const float4*>(q + 4);
  }
  __device__ __forceinline__ void to(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * i] = v[i].x, x[4 * i + 1] = v[i].y, x[4 * i + 2] = v[i].z, x[4 * i + 3] = v[i].w;
  }
};
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  Piece<__nv_bfloat16, 8> y;
#pragma unroll
  for (int e = 0; e < 8; ++e) from_float(y.x[e], x[e]);
  *reinterpret_cast<Piece<__nv_bfloat16, 8>*>(p) = y;
}
// Where pair f's cosine stands: the fours of a lane's eight apart, so that lanes read next to one another.
__device__ __forceinline__ int pair_at(int f) { return ((f & 4) << 4) + ((f >> 3) << 2) + (f & 3); }
__device__ __forceinline__ void load_pairs(const float* c, int u, float (&x)[8]) {
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const float4 v = *reinterpret_cast<const float4*>(c + 64 * y + 4 * u);
    x[4 * y] = v.x, x[4 * y + 1] = v.y, x[4 * y + 2] = v.z, x[4 * y + 3] = v.w;
  }
}

enum RowKind { kQuery, kKey, kValue };
// What the rows of a token share.
struct TokenRows {
  long long slot, at;  // row of the pool of key head 0, position with its offset
  const float* cs;
  const float* sn;
};
// A lane's columns of a row: eight from c0 on, eight from c1 on.
struct Columns {
  int c0, c1, w;
  bool has;
};
template <PairForm kForm, RowKind kKind>
__device__ __forceinline__ Columns columns_of(const AppendArgs& a, int u) {
  Columns c;
  c.w = kKind == kValue ? a.vw : a.d;
  c.c0 = 16 * u;
  c.c1 = c.c0 + 8;
  c.has = 16 * u < c.w;
  if (kKind != kValue && kForm == kHalves && a.pairs > 0) {
    const int half = a.pairs >> 3;
    c.c0 = u < half ? 8 * u : 2 * a.pairs + 16 * (u - half);
    c.c1 = u < half ? a.pairs + 8 * u : c.c0 + 8;
  }
  return c;
}

// One pass over rows of one kind: a row for each kLanes lanes (where it has one: `on`), the lane's columns `raw`;
// rotated, and into q_row or quantised into the page's row and its exponent byte.
template <typename T, int kLanes, PairForm kForm, RowKind kKind>
__device__ __forceinline__ void append_pass(const AppendArgs& a, const TokenRows& t, const Columns& col, bool on, const T* row,
                                            T* q_row, uint8_t* page_row, uint8_t* exponent, const Raw16<T>& raw) {
  constexpr bool kTurns = kKind != kValue;
  const int u = threadIdx.x % kLanes, pairs = a.pairs, c0 = col.c0, c1 = col.c1;
  const bool turned = kTurns && col.has && (kForm == kAnywhere ? c0 < 2 * pairs : 8 * u < pairs);
  {
    float y[16];
    if (on) {
      raw.to(y);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = 0.f;
    }
    [[maybe_unused]] float x0[16], x1[16];  // the pairs, where a lane does not have both of each
    if (turned && on) {
      if constexpr (kForm == kAnywhere) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int c = c0 + e;
          x0[e] = x1[e] = 0.f;
          if (c >= 2 * pairs) continue;
          const bool first = c < pairs;
          const int f = first ? c : c - pairs;
          const float other = as_float(row[first ? c + pairs : f]), k = t.cs[pair_at(f)], s = t.sn[pair_at(f)];
          x0[e] = y[e];
          x1[e] = other;
          y[e] = first ? y[e] * k - other * s : y[e] * k + other * s;
        }
      } else {
        float k[8], s[8];
        load_pairs(t.cs, u, k);
        load_pairs(t.sn, u, s);
        if constexpr (kForm == kHalves) {  // two pairs at once
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float p0, p1, q0, q1;
            tc::fmul2(p0, p1, y[8 + e], y[9 + e], -s[e], -s[e + 1]);
            tc::fmul2(q0, q1, y[e], y[e + 1], s[e], s[e + 1]);
            tc::ffma2(p0, p1, y[e], y[e + 1], k[e], k[e + 1], p0, p1);
            tc::ffma2(y[8 + e], y[9 + e], y[8 + e], y[9 + e], k[e], k[e + 1], q0, q1);
            y[e] = p0;
            y[e + 1] = p1;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (8 * u + e >= pairs) continue;
            float &p = y[2 * e], &q = y[2 * e + 1];
            const float u0 = p, u1 = q;
            p = u0 * k[e] - u1 * s[e];
            q = u1 * k[e] + u0 * s[e];
          }
        }
      }
    }
    if constexpr (kKind == kQuery) {
      if (kForm == kAnywhere) __syncwarp();  // q_out may be q: every lane has read the pairs' others
      if (on) {
        store8(q_row + c0, y);
        store8(q_row + c1, y + 8);
      }
      return;
    }
    // Every lane of a row's, also those without columns.  An infinity is found by the maximum.
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) most = tc::fmax3(most, fabsf(y[e]), fabsf(y[e + 1]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
    unsigned top = __float_as_uint(most);
    if (__any_sync(0xFFFFFFFFu, top == 0x7F800000u)) {  // the largest finite one
      // The other entry of a pair with an infinity is NaN too.  (Where one is NaN the other is not finite: both come
      // of the same two entries, and finite ones give infinities at most.)
      [[maybe_unused]] bool other[16];
      if constexpr (kTurns) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if constexpr (kForm == kAnywhere) {
            const int c = c0 + e;
            other[e] = false;
            if (!turned || !on || c >= 2 * pairs) continue;
            const bool first = c < pairs;
            const int f = first ? c : c - pairs;
            const float k = t.cs[pair_at(f)], s = t.sn[pair_at(f)];
            other[e] = !isfinite(first ? x1[e] * k + x0[e] * s : x1[e] * k - x0[e] * s);
          } else {
            const int o = kForm == kInside ? e ^ 1 : e ^ 8, pair = 8 * u + (kForm == kInside ? e >> 1 : e & 7);
            other[e] = turned && pair < pairs && !isfinite(y[o]);
          }
        }
      }
      top = 0u;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        if constexpr (kTurns)
          if (other[e]) y[e] = NAN;
        const unsigned m = __float_as_uint(y[e]) & 0x7FFFFFFFu;
        top = max(top, m < 0x7F800000u ? m : 0u);
        if (m == 0x7F800000u) y[e] = NAN;
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    int ex = exponent_of(top);
    uint32_t again = 0u;  // entries to be computed again
    // No turn, no error: one bf16 value in 16 is on a border itself.  (Prompts from their first token on: 3 thousand
    // tokens 20 us in place of 70.)
    [[maybe_unused]] const bool exact = t.at == 0;
    if constexpr (kTurns) {
      // (8 units of the last place are more than the error of a pair that is no longer than twice its row's largest.)
      const bool near = pairs > 0 && top > 8u && exponent_of(top - 8u) != exponent_of(top + 8u);
      if (__any_sync(0xFFFFFFFFu, near)) {
        // Of the entries that may be the largest.  Columns that pass are often on the border itself (one bf16 value in
        // 128): 3 thousand tokens of 16 key heads, half of 128 columns rotated, 21 us in place of 145.
        uint32_t may = 0u;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const unsigned m = __float_as_uint(y[e]) & 0x7FFFFFFFu;
          may |= m + 16u >= top && m < 0x7F800000u ? 1u << e : 0u;
        }
        unsigned long long largest = 0ull;
#pragma unroll 1
        for (uint32_t left = near && on ? may : 0u; left; left &= left - 1) {
          const int e = __ffs(left) - 1;
          const double z = turned64(row, (e < 8 ? c0 : c1 - 8) + e, pairs, kForm == kInside, t.at, a.inv_freq);
          const unsigned long long m = static_cast<unsigned long long>(__double_as_longlong(fabs(z)));
          if (m < 0x7FF0000000000000ull) largest = max(largest, m);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) largest = max(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, o));
        if (near) ex = exponent_of(largest);
      }
    }
    if (!on) return;
    const float inv = __uint_as_float(static_cast<unsigned>(254 - max(ex, 1)) << 23);
    uint32_t code[4];
    if (turned) {
      // Rounded from either end of what an entry may be.  Zeros of either sign are the same.
      const float err = exact ? 0.f : inv * kTurnError, least = exact ? 0.f : 0x1p-22f;
      float d[kForm == kAnywhere ? 16 : 8];  // of an entry or a pair; 2^-22: of subnormal numbers' own spacing
#pragma unroll
      for (int e = 0; e < (kForm == kAnywhere ? 16 : 8); ++e) {
        const float u0 = kForm == kAnywhere ? x0[e] : kForm == kInside ? y[2 * e] : y[e];
        const float u1 = kForm == kAnywhere ? x1[e] : kForm == kInside ? y[2 * e + 1] : y[8 + e];
        d[e] = fmaf(fabsf(u0), err, fmaf(fabsf(u1), err, least));
        // Columns that pass, of the lane that has the last pairs: no error, whatever stands beside them.
        if (kForm == kInside && 8 * u + e >= pairs) d[e] = 0.f;
      }
      uint32_t down[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e0 = kForm == kAnywhere ? 2 * i : kForm == kInside ? i : 2 * i & 7;
        const int e1 = kForm == kAnywhere ? 2 * i + 1 : kForm == kInside ? i : (2 * i + 1) & 7;
        float z0, z1, h0, h1, l0, l1;
        tc::fmul2(z0, z1, y[2 * i], y[2 * i + 1], inv, inv);
        tc::fadd2(h0, h1, z0, z1, d[e0], d[e1]);
        tc::fadd2(l0, l1, z0, z1, -d[e0], -d[e1]);
        const uint32_t p = e4m3_of(h0, h1), q = e4m3_of(l0, l1);
        code[i >> 1] = i & 1 ? code[i >> 1] | p << 16 : p;
        down[i >> 1] = i & 1 ? down[i >> 1] | q << 16 : q;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t diff = (code[i] ^ down[i]) & 0x7F7F7F7Fu;
        if (diff)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if ((diff >> 8 * k) & 0xFFu) again |= 1u << (4 * i + k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        code[i] = e4m3_of(y[4 * i] * inv, y[4 * i + 1] * inv) | e4m3_of(y[4 * i + 2] * inv, y[4 * i + 3] * inv) << 16;
    }
#pragma unroll 1
    for (; again; again &= again - 1) {
      const int e = __ffs(again) - 1;
      const double z = turned64(row, (e < 8 ? c0 : c1 - 8) + e, pairs, kForm == kInside, t.at, a.inv_freq);
      const uint32_t x = e4m3_of(z * static_cast<double>(inv)) << 8 * (e & 3), keep = ~(0xFFu << 8 * (e & 3));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e >> 2 == i) code[i] = (code[i] & keep) | x;
    }
    if (c1 == c0 + 8) {
      *reinterpret_cast<uint4*>(page_row + c0) = make_uint4(code[0], code[1], code[2], code[3]);
    } else {
      *reinterpret_cast<uint2*>(page_row + c0) = make_uint2(code[0], code[1]);
      *reinterpret_cast<uint2*>(page_row + c1) = make_uint2(code[2], code[3]);
    }
    if (u == 0) *exponent = static_cast<uint8_t>(ex);
  }
}

// All passes of a warp over the n rows of one kind, from row r (of the lane) on in steps of `step`.  `next` holds
// the first one's columns; a pass's loads are in flight during the one before.
template <typename T, int kLanes, PairForm kForm, RowKind kKind>
__device__ __forceinline__ void append_rows(const AppendArgs& a, const TokenRows& t, const Columns& col, const T* rows, T* q_out,
                                            uint8_t* pages, uint8_t* exponents, int n, int r, int step, Raw16<T>& next) {
  const int sub = (threadIdx.x & 31) / kLanes;
  const T* row = rows + r * col.w;
#pragma unroll 1
  for (int left = n - r; left + sub > 0; left -= step) {
    const Raw16<T> raw = next;
    const T* at = row;
    row += step * col.w;
    if (col.has && left > step) next.load(row + col.c0, row + col.c1);
    const long long h = n - left;  // the lane's row
    append_pass<T, kLanes, kForm, kKind>(
        a, t, col, col.has && left > 0, at, kKind == kQuery ? q_out + h * col.w : nullptr,
        kKind == kQuery ? nullptr : pages + (t.slot + (h << a.lps)) * col.w,
        kKind == kQuery ? nullptr : exponents + t.slot + (h << a.lps), raw);
  }
}

template <typename T, int kLanes, PairForm kForm>
__global__ void __launch_bounds__(kThreads8, kAppendCtas8) append_e4m3_kernel(const __grid_constant__ AppendArgs a) {
  wait_for_previous();
  let_next_start();
  if (blockIdx.x == gridDim.x - 1) {
    append_check(a);
    return;
  }
  __shared__ __align__(16) float cs[kWarps8][kMaxPairs];
  __shared__ __align__(16) float sn[kWarps8][kMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int job = blockIdx.x * kWarps8 + warp;
  const int t = div_by(job, a.by_shares), share = job - t * a.by_shares.d;
  if (t >= a.T) return;
  // Passes over the token's rows, kPass of one kind each, dealt out to the warps that share it; the first ones'
  // loads stand before the look-up of the token's place.
  constexpr int kPass = 32 / kLanes;
  const int sub = lane / kLanes, shares = a.by_shares.d, step = kPass * shares;
  const T* q = static_cast<const T*>(a.q) + t * a.qs;
  const T* k = static_cast<const T*>(a.k) + t * a.ks;
  const T* v = static_cast<const T*>(a.v) + t * a.vs;
  const int H = a.q ? a.H : 0, q_passes = (H + kPass - 1) / kPass, k_passes = (a.Hk + kPass - 1) / kPass;
  auto first = [&](int base) { return (share + shares * kMaxPasses - base) % shares * kPass + sub; };  // row, of the kind behind `base` passes
  const int rq = first(0), rk = first(q_passes), rv = first(q_passes + k_passes);
  const Columns key = columns_of<kForm, kKey>(a, lane % kLanes), val = columns_of<kForm, kValue>(a, lane % kLanes);
  Raw16<T> next, next_k;
  if (key.has && rq < H) next.load(q + rq * key.w + key.c0, q + rq * key.w + key.c1);
  if (key.has && rk < a.Hk) next_k.load(k + rk * key.w + key.c0, k + rk * key.w + key.c1);
  const int b = owner(a, t);
  if (b < 0) return;  // behind the last sequence
  int s0 = b * a.each, nq = a.each;
  if (a.starts) {  // clamped, as the attention does
    s0 = max(__ldg(a.starts + b), 0);
    nq = min(__ldg(a.starts + b + 1), a.T) - s0;
  }
  const int pos = max(__ldg(a.lens + b), 0) - nq + (t - s0);
  long long slot = -1;  // the token's row of the pool (of key head 0); -1: nowhere
  if (pos >= 0 && pos < a.max_pages << a.lps) {
    const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (pos >> a.lps));
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
      slot = (static_cast<long long>(page) * a.Hk << a.lps) + (pos & ((1 << a.lps) - 1));
  }
  const long long at = static_cast<long long>(pos) + a.pos_offset;
  for (int f = lane; f < a.pairs; f += 32) angle(at, __ldg(a.inv_freq + f), sn[warp][pair_at(f)], cs[warp][pair_at(f)]);
  __syncwarp();
  const TokenRows x{slot, at, cs[warp], sn[warp]};
  append_rows<T, kLanes, kForm, kQuery>(a, x, key, q, static_cast<T*>(a.q_out) + static_cast<size_t>(t) * a.H * a.d, nullptr,
                                        nullptr, H, rq, step, next);
  if (slot < 0) return;
  if (val.has && rv < a.Hk) next.load(v + rv * val.w + val.c0, v + rv * val.w + val.c1);
  append_rows<T, kLanes, kForm, kKey>(a, x, key, k, nullptr, static_cast<uint8_t*>(a.kp), a.k_scales, a.Hk, rk, step, next_k);
  append_rows<T, kLanes, kForm, kValue>(a, x, val, v, nullptr, static_cast<uint8_t*>(a.vp), a.v_scales, a.Hk, rv, step, next);
}

template <typename T, int kLanes, PairForm kForm>
cudaError_t append_e4m3_launch(AppendArgs a, cudaStream_t s) {
  a.each = a.T / a.B;
  int shares = 1;
  while (shares < 8 && (long long)a.T * shares * 2 <= 152 * 16 && shares < 2 * a.Hk) shares *= 2;
  a.by_shares = fast_div(shares);
  const unsigned ctas = (static_cast<unsigned>(a.T) * shares + kWarps8 - 1) / kWarps8;
  before_launch(kKernAppend, s);
  const cudaError_t e = launch_early(append_e4m3_kernel<T, kLanes, kForm>, dim3(ctas + 1), kThreads8, 0, s, a);
  after_launch(kKernAppend, s);
  return e;
}

template <typename T, int kLanes>
cudaError_t append_e4m3_form(const AppendArgs& a, cudaStream_t s) {
  if (a.interleaved) return append_e4m3_launch<T, kLanes, kInside>(a, s);
  if (a.pairs % 8 == 0) return append_e4m3_launch<T, kLanes, kHalves>(a, s);
  return append_e4m3_launch<T, kLanes, kAnywhere>(a, s);
}

template <typename T>
cudaError_t append_e4m3_dispatch(const AppendArgs& a, cudaStream_t s) {
  return a.d <= 128 && a.vw <= 128 ? append_e4m3_form<T, 8>(a, s) : append_e4m3_form<T, 16>(a, s);
}

}  // namespace

cudaError_t launch_append_e4m3(const AppendArgs& a, cudaStream_t s) {
  return a.dtype == kF32 ? append_e4m3_dispatch<float>(a, s) : append_e4m3_dispatch<__nv_bfloat16>(a, s);
}

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  return a.dtype == kF32 ? append_dispatch<float>(a, s) : append_dispatch<__nv_bfloat16>(a, s);
}

}  // namespace exattn
