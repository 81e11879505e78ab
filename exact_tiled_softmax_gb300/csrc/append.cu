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

namespace exattn {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kMaxPairs = 128;

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
  for (int b0 = (threadIdx.x & ~31); b0 < a.B; b0 += kAppendThreads) {
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

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  return a.dtype == kF32 ? append_dispatch<float>(a, s) : append_dispatch<__nv_bfloat16>(a, s);
}

}  // namespace exattn
