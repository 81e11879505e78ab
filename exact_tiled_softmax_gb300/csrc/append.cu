// New keys and values into a paged cache, with the rotary position embedding
// applied to keys (and to the queries beside them) on the way.
//
// Token t of sequence b is at position pos = len - nq + i.  Pair f of a
// rotated row turns by (pos + pos_offset) * inv_freq[f]:
//   x' = x cos - y sin,  y' = y cos + x sin,
// pairs (f, f + pairs) or, interleaved, (2f, 2f + 1); other columns pass.
// Bound by memory: every element is read once and written once, in 16-byte accesses
// where the rotated halves allow them.  A CTA takes the accesses of a few tokens as one
// list.  A thread's source addresses need no table, so it loads first and works out
// angles and places while the loads are under way.  One CTA more checks that every
// token has a place and writes the status word.
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

constexpr int kMaxPer = 8;    // tokens of a CTA
constexpr int kPerThread = 2;  // accesses of a thread whose loads overlap

// W: elements of an access.  A rotated row is cut into units: interleaved, unit u is
// access u; else units below pairs / W are the accesses u W and pairs + u W of the two
// halves, those above one access of the columns that pass.
template <typename T, int W>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  if (blockIdx.x == gridDim.x - 1) {
    append_check(a);
    return;
  }
  __shared__ float cs[kMaxPer][kMaxPairs], sn[kMaxPer][kMaxPairs];
  __shared__ long long slots[kMaxPer];  // the token's row of the pool (key head 0); -1: nowhere
  __shared__ bool owned[kMaxPer];
  constexpr int E = 16 / sizeof(T);
  const int t0 = blockIdx.x * a.per, tokens = min(a.per, a.T - t0);
  const int total = tokens * a.by_items.d, half = a.pairs / W;
  bool placed = false;
#pragma unroll 1
  for (int base = 0; base < total; base += kPerThread * kAppendThreads) {
    float x[kPerThread][W], y[kPerThread][W];
    uint4 raw[kPerThread];
    int tok[kPerThread], head[kPerThread], unit[kPerThread], kind[kPerThread];  // kind: 0 q, 1 k, 2 v, 3 none
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const int idx = base + j * kAppendThreads + threadIdx.x;
      kind[j] = 3;
      if (idx >= total) continue;
      tok[j] = div_by(idx, a.by_items);
      int i = idx - tok[j] * a.by_items.d;
      const int t = t0 + tok[j];
      if (i < a.qk_items) {
        kind[j] = i < a.q_items ? 0 : 1;
        if (kind[j] == 1) i -= a.q_items;
        head[j] = div_by(i, a.by_units);
        unit[j] = i - head[j] * a.by_units.d;
        const T* src = (kind[j] == 0 ? static_cast<const T*>(a.q) + t * a.qs : static_cast<const T*>(a.k) + t * a.ks) +
                       head[j] * a.d;
        if (a.interleaved) {
          Vec<T, W>::load(src + unit[j] * W, x[j]);
        } else if (unit[j] < half) {
          Vec<T, W>::load(src + unit[j] * W, x[j]);
          Vec<T, W>::load(src + a.pairs + unit[j] * W, y[j]);
        } else {
          Vec<T, W>::load(src + (unit[j] + half) * W, x[j]);
        }
      } else {
        i -= a.qk_items;
        kind[j] = 2;
        head[j] = div_by(i, a.by_vch);
        unit[j] = i - head[j] * a.by_vch.d;
        raw[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + t * a.vs + head[j] * a.vw + unit[j] * E);
      }
    }
    if (!placed) {
      placed = true;
#pragma unroll 1
      for (int i = threadIdx.x; i < tokens * max(a.pairs, 1); i += kAppendThreads) {
        const int k = i / max(a.pairs, 1), f = i - k * max(a.pairs, 1), t = t0 + k;
        const int b = owner(a, t);
        if (f == 0) owned[k] = b >= 0;
        if (b < 0) continue;
        int s0, nq;
        if (a.starts) {
          s0 = __ldg(a.starts + b);
          nq = __ldg(a.starts + b + 1) - s0;
        } else {
          nq = a.T / a.B;
          s0 = b * nq;
        }
        const int pos = __ldg(a.lens + b) - nq + (t - s0);
        if (f == 0) {
          long long slot = -1;
          if (pos >= 0 && pos < a.max_pages << a.lps) {
            const int page = __ldg(a.table + static_cast<size_t>(b) * a.max_pages + (pos >> a.lps));
            if (static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages))
              slot = (static_cast<long long>(page) * a.Hk << a.lps) + (pos & ((1 << a.lps) - 1));
          }
          slots[k] = slot;
        }
        if (f < a.pairs) {
          // Whole turns are dropped in 64 bits: far positions keep their angle.
          constexpr double kInv2Pi = 0.15915494309189533577;
          const double turns = (static_cast<double>(pos) + a.pos_offset) *
                               (static_cast<double>(a.inv_freq[f]) * kInv2Pi);
          sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn[k][f], &cs[k][f]);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (kind[j] == 3 || !owned[tok[j]]) continue;
      const long long slot = slots[tok[j]];
      if (kind[j] == 2) {
        if (slot >= 0)
          *reinterpret_cast<uint4*>(static_cast<T*>(a.vp) +
                                    (slot + (static_cast<long long>(head[j]) << a.lps)) * a.vw + unit[j] * E) = raw[j];
        continue;
      }
      if (kind[j] == 1 && slot < 0) continue;
      T* dst = kind[j] == 0 ? static_cast<T*>(a.q_out) + (static_cast<size_t>(t0 + tok[j]) * a.H + head[j]) * a.d
                            : static_cast<T*>(a.kp) + (slot + (static_cast<long long>(head[j]) << a.lps)) * a.d;
      const float *c = cs[tok[j]], *s = sn[tok[j]];
      if (a.interleaved) {
        if constexpr (W > 1) {
#pragma unroll
          for (int e = 0; e < W; e += 2) {
            const int f = (unit[j] * W + e) >> 1;
            if (f < a.pairs) {
              const float x0 = x[j][e], x1 = x[j][e + 1];
              x[j][e] = x0 * c[f] - x1 * s[f];
              x[j][e + 1] = x1 * c[f] + x0 * s[f];
            }
          }
        }
        Vec<T, W>::store(dst + unit[j] * W, x[j]);
      } else if (unit[j] < half) {
        float p[W], q[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const int f = unit[j] * W + e;
          p[e] = x[j][e] * c[f] - y[j][e] * s[f];
          q[e] = y[j][e] * c[f] + x[j][e] * s[f];
        }
        Vec<T, W>::store(dst + unit[j] * W, p);
        Vec<T, W>::store(dst + a.pairs + unit[j] * W, q);
      } else {
        Vec<T, W>::store(dst + (unit[j] + half) * W, x[j]);
      }
    }
  }
}

template <typename T, int W>
cudaError_t append_launch(AppendArgs a, cudaStream_t s) {
  const int units = (a.interleaved ? a.d : a.d - a.pairs) / W, vch = a.vw * static_cast<int>(sizeof(T)) / 16;
  a.by_units = fast_div(units);
  a.by_vch = fast_div(vch);
  a.q_items = a.q ? a.H * units : 0;
  a.qk_items = a.q_items + a.Hk * units;
  a.by_items = fast_div(a.qk_items + a.Hk * vch);
  // Tokens of a CTA: enough for two accesses a thread, unless that leaves SMs idle.
  a.per = 1;
  while (a.per < kMaxPer && a.per * a.by_items.d < kPerThread * kAppendThreads && a.T / (2 * a.per) >= 4 * 152)
    a.per *= 2;
  before_launch(kKernAppend, s);
  append_kernel<T, W><<<(a.T + a.per - 1) / a.per + 1, kAppendThreads, 0, s>>>(a);
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
