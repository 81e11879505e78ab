// New keys and values into a paged cache, with the rotary position embedding
// applied to keys (and to the queries beside them) on the way.
//
// Token t of sequence b is at position pos = len - nq + i.  Pair f of a
// rotated row turns by (pos + pos_offset) * inv_freq[f]:
//   x' = x cos - y sin,  y' = y cos + x sin,
// pairs (f, f + pairs) or, interleaved, (2f, 2f + 1); other columns pass.
// Bound by memory: every element is read once and written once.
#include "paged.cuh"

namespace exattn {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kMaxPairs = 128;

// The sequence that owns token t, or -1.
__device__ __forceinline__ int owner(const AppendArgs& a, int t) {
  if (!a.starts) return t / (a.T / a.B);
  if (t >= __ldg(a.starts + a.B) || t < __ldg(a.starts)) return -1;
  int b0 = 0, b1 = a.B;  // starts[b0] <= t < starts[b1]
  while (b1 - b0 > 1) {
    const int mid = (b0 + b1) >> 1;
    if (__ldg(a.starts + mid) <= t) b0 = mid;
    else b1 = mid;
  }
  return b0;
}

// N consecutive elements as fp32, in accesses of N * sizeof(T) bytes.
template <typename T, int N> struct Vec;
template <int N> struct Vec<float, N> {
  struct alignas(4 * N) Raw { float x[N]; };
  __device__ static void load(const float* p, float (&f)[N]) {
    const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = r.x[i];
  }
  __device__ static void store(float* p, const float (&f)[N]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.x[i] = f[i];
    *reinterpret_cast<Raw*>(p) = r;
  }
};
template <int N> struct Vec<__nv_bfloat16, N> {
  struct alignas(2 * N) Raw { __nv_bfloat16 x[N]; };
  __device__ static void load(const __nv_bfloat16* p, float (&f)[N]) {
    const Raw r = *reinterpret_cast<const Raw*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __bfloat162float(r.x[i]);
  }
  __device__ static void store(__nv_bfloat16* p, const float (&f)[N]) {
    Raw r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.x[i] = __float2bfloat16_rn(f[i]);
    *reinterpret_cast<Raw*>(p) = r;
  }
};

// W: elements of an access.  Interleaved pairs stay inside an access; the two
// halves of the other form are W apart in units when W divides `pairs`.
template <typename T, int W>
__device__ __forceinline__ void rotate_row(const AppendArgs& a, const T* src, T* dst, int unit,
                                           const float* cs, const float* sn) {
  if (a.interleaved) {
    float x[W];
    Vec<T, W>::load(src + unit * W, x);
    if constexpr (W > 1) {
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const int f = (unit * W + e) >> 1;
        if (f < a.pairs) {
          const float c = cs[f], s = sn[f], x0 = x[e], x1 = x[e + 1];
          x[e] = x0 * c - x1 * s;
          x[e + 1] = x1 * c + x0 * s;
        }
      }
    }
    Vec<T, W>::store(dst + unit * W, x);
    return;
  }
  const int half = a.pairs / W;
  if (unit < half) {
    float x[W], y[W], p[W], q[W];
    Vec<T, W>::load(src + unit * W, x);
    Vec<T, W>::load(src + a.pairs + unit * W, y);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const float c = cs[unit * W + e], s = sn[unit * W + e];
      p[e] = x[e] * c - y[e] * s;
      q[e] = y[e] * c + x[e] * s;
    }
    Vec<T, W>::store(dst + unit * W, p);
    Vec<T, W>::store(dst + a.pairs + unit * W, q);
  } else {
    float x[W];
    const int col = (unit + half) * W;
    Vec<T, W>::load(src + col, x);
    Vec<T, W>::store(dst + col, x);
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a) {
  __shared__ float cs[kMaxPairs], sn[kMaxPairs];
  const int t = blockIdx.x;
  const int b = owner(a, t);
  if (b < 0) return;  // behind the last sequence
  int s0, nq;
  if (a.starts) {
    s0 = __ldg(a.starts + b);
    nq = __ldg(a.starts + b + 1) - s0;
  } else {
    nq = a.T / a.B;
    s0 = b * nq;
  }
  const int pos = __ldg(a.lens + b) - nq + (t - s0);
  for (int f = threadIdx.x; f < a.pairs; f += kAppendThreads) {
    // Whole turns are dropped in 64 bits: far positions keep their angle.
    constexpr double kInv2Pi = 0.15915494309189533577;
    const double turns = (static_cast<double>(pos) + a.pos_offset) *
                         (static_cast<double>(a.inv_freq[f]) * kInv2Pi);
    sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn[f], &cs[f]);
  }
  // Where the token's key and value go; -1: nowhere.
  long long slot = -1;
  if (pos >= 0 && pos < a.max_pages << a.lps) {
    const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (pos >> a.lps));
    if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
      slot = (static_cast<long long>(page) * a.Hk << a.lps) + (pos & ((1 << a.lps) - 1));
  }
  __syncthreads();
  const int units = (a.interleaved ? a.d : a.d - a.pairs) / W;  // of a row of q or k
  if (a.q) {
    const T* src = static_cast<const T*>(a.q) + t * a.qs;
    T* dst = static_cast<T*>(a.q_out) + static_cast<size_t>(t) * a.H * a.d;
    for (int x = threadIdx.x; x < a.H * units; x += kAppendThreads) {
      const int h = x / units, u = x - h * units;
      rotate_row<T, W>(a, src + h * a.d, dst + h * a.d, u, cs, sn);
    }
  }
  if (slot < 0) return;
  const T* ks = static_cast<const T*>(a.k) + t * a.ks;
  T* kd = static_cast<T*>(a.kp) + slot * a.d;
  for (int x = threadIdx.x; x < a.Hk * units; x += kAppendThreads) {
    const int h = x / units, u = x - h * units;
    rotate_row<T, W>(a, ks + h * a.d, kd + (static_cast<size_t>(h) << a.lps) * a.d, u, cs, sn);
  }
  constexpr int E = 16 / sizeof(T);
  const int vch = a.vw / E;
  const T* vs = static_cast<const T*>(a.v) + t * a.vs;
  T* vd = static_cast<T*>(a.vp) + slot * a.vw;
  for (int x = threadIdx.x; x < a.Hk * vch; x += kAppendThreads) {
    const int h = x / vch, u = x - h * vch;
    *reinterpret_cast<uint4*>(vd + (static_cast<size_t>(h) << a.lps) * a.vw + u * E) =
        *reinterpret_cast<const uint4*>(vs + h * a.vw + u * E);
  }
}

// Status: whether every new token has a place.  One CTA; a thread takes a
// sequence at a time, a warp the pages of a long one.
__global__ void __launch_bounds__(kAppendThreads) append_check_kernel(const AppendArgs a) {
  bool bad = false;
  const int lane = threadIdx.x & 31;
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
        last = (min(n, cap) - 1) >> a.lps;  // below `first` when n <= 0
        if (n <= 0) last = -1;
      }
    }
    const bool many = last - first >= 4;
    for (int p = first; !many && p <= last; ++p)
      bad |= static_cast<unsigned>(__ldg(a.table + static_cast<size_t>(b) * a.max_pages + p)) >=
             static_cast<unsigned>(a.num_pages);
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, many); todo; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      const int f = __shfl_sync(0xFFFFFFFFu, first, who), e = __shfl_sync(0xFFFFFFFFu, last, who);
      for (int p = f + lane; p <= e; p += 32)
        bad |= static_cast<unsigned>(__ldg(a.table + static_cast<size_t>(b0 + who) * a.max_pages + p)) >=
               static_cast<unsigned>(a.num_pages);
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) *a.status = any ? kStatusBadPage : 0u;
}

template <typename T, int W>
cudaError_t append_launch(const AppendArgs& a, cudaStream_t s) {
  before_launch(kKernAppend, s);
  append_check_kernel<<<1, kAppendThreads, 0, s>>>(a);
  append_kernel<T, W><<<a.T, kAppendThreads, 0, s>>>(a);
  after_launch(kKernAppend, s);
  return cudaGetLastError();
}

template <typename T>
cudaError_t append_dispatch(const AppendArgs& a, cudaStream_t s) {
  constexpr int E = 16 / sizeof(T);
  // The widest access that neither half of the rotated columns breaks up.
  if (a.interleaved || a.pairs % E == 0) return append_launch<T, E>(a, s);
  if (a.pairs % (E / 2) == 0) return append_launch<T, E / 2>(a, s);
  return append_launch<T, 1>(a, s);
}

}  // namespace

int append_max_pairs() { return kMaxPairs; }

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  return a.dtype == kF32 ? append_dispatch<float>(a, s) : append_dispatch<__nv_bfloat16>(a, s);
}

}  // namespace exattn
