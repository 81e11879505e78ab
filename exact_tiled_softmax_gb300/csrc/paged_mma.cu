// Paged attention for few rows to a key head (a decode step, a few guessed
// tokens) in bf16, widths up to 128: bound by reading K and V once.
//
// A row tile is 16 rows, one m16n8k16 tensor-core tile: the rows of a key head's
// whole group share each key that is read.  kW warps take the 16-key tiles of a
// unit in turn, each with a ring of kStages tiles of its own in shared memory
// (asynchronous 16-byte copies, row by row through the page table), its own
// running maximum, sum and output in registers, and no barrier until the
// segment's end, where the warps are joined with the star rule.  Two CTAs to an
// SM hold 2 x 4 x (kStages - 1) x 8 KB in flight, and one streams while the other
// starts or ends a segment.
//
// The reference point of the exponentials moves only when a row's maximum passes
// it by more than 2^8, so p <= 2^8.  p enters P.V as the sum of two bf16 values,
// its rounding and what the rounding left out (2^-17 of p remains): the products
// are free beside the loads, and Y is then rounded once, on its way out.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {
namespace {

using tc::ex2;
using tc::ld_shared_v4;
using tc::pack_bf16x2;
using tc::smem_u32;

constexpr int kW = 4;
constexpr int kRows = 16;
constexpr int kTile = 16;          // keys of a warp's tile
constexpr int kUnit = kW * kTile;  // keys of a unit of work
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

template <int D>
struct MmaLayout {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTileBytes = kTile * D * 2;  // of K or V
  static constexpr int kWarpBytes = 2 * kStages * kTileBytes;
  static constexpr int kBytes = kW * kWarpBytes;
  static_assert(kStages * kTileBytes >= kRows * D * 4, "a warp's output fits its V ring");
};

template <int D>
__global__ void __launch_bounds__(32 * kW, 2) paged_mma_kernel(const PagedArgs a) {
  using Lay = MmaLayout<D>;
  constexpr int S = Lay::kStages;
  constexpr int CH = D / 8;   // 16-byte pieces of a row
  constexpr int NT = D / 8;   // output columns in tiles of 8
  constexpr int KS = D / 16;  // steps of the score product
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ long long pre[kPagedMaxBatch + 1], scan[kW];
  __shared__ float red_m[kW][kRows], red_l[kW][kRows];
  __shared__ unsigned tile_keys[kW][S];  // bit r: key r of the staged tile exists

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int d = a.d, v = a.v, kch = d / 8, vch = v / 8;
  const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
  const __nv_bfloat16* Kp = static_cast<const __nv_bfloat16*>(a.Kp);
  const __nv_bfloat16* Vp = static_cast<const __nv_bfloat16*>(a.Vp);
  uint8_t* own = sm + warp * Lay::kWarpBytes;
  const uint32_t kbase = smem_u32(own), vbase = kbase + S * Lay::kTileBytes;
  unsigned bits = 0;
  if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  // Columns of K that the rows do not have stay zero: no copy writes them.
  if (kch < CH)
    for (int x = lane; x < S * Lay::kTileBytes / 16; x += 32)
      *reinterpret_cast<uint4*>(own + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
  PagedWalk w;
  bool more = paged_begin<kRows, kUnit, 32 * kW>(a, pre, scan, w, bits);
  while (more) {
    int j0, j1;
    const int n = paged_segment<kUnit>(w, j0, j1);
    const int r0 = w.rt * kRows, rows = w.t.rows;
    const int* trow = a.table + static_cast<size_t>(w.b) * a.max_pages;
    const int first = (w.t.kt0 + w.rem) * kUnit + warp * kTile;  // the warp's tile of unit 0
    const int i0 = first + kTile > j0 ? 0 : 1;
    const int i1 = j1 <= j0 ? i0 : first + (n - 1) * kUnit < j1 ? n : n - 1;

    // Lane r < 16: key r of tile i as a row of the pool, -1 outside [j0, j1) or the pool.
    auto find = [&](int i) {
      long long row = -1;
      const int key = first + i * kUnit + (lane & 15);
      if (i < i1 && key >= j0 && key < j1) {
        row = paged_key_row(a, trow, w.h, key);
        if (row < 0) bits |= kStatusBadPage;
      }
      return row;
    };
    auto issue = [&](int i, long long row) {
      if (i < i1) {
        const int s = i % S;
        const unsigned have = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFFFu;
        if (lane == 0) tile_keys[warp][s] = have;
        const uint32_t kd = kbase + s * Lay::kTileBytes, vd = vbase + s * Lay::kTileBytes;
#pragma unroll
        for (int x = 0; x < kTile * CH / 32; ++x) {
          const int idx = x * 32 + lane, r = idx / CH, c = idx % CH;
          const long long at = __shfl_sync(0xFFFFFFFFu, row, r);
          const uint32_t off = r * (D * 2) + ((c ^ (r & 7)) << 4);
          const long long from = at < 0 ? 0 : at;
          if (c < kch) cp16(kd + off, Kp + from * d + c * 8, at < 0 ? 0 : 16);
          if (c < vch) cp16(vd + off, Vp + from * v + c * 8, at < 0 ? 0 : 16);
        }
      }
      cp_commit();
    };
    long long row = find(i0);
#pragma unroll
    for (int k = 0; k < S - 1; ++k) {
      const long long next = find(i0 + k + 1);
      issue(i0 + k, row);
      row = next;
    }

    // The rows of Q as A operands: thread (g, t) holds rows g and g + 8.
    int lo[2], hi[2];
    uint32_t qa[KS][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int q = g + 8 * x, r = r0 + (q < rows ? q : 0), i = r / a.G;
      paged_row_span(a, w.s, i, lo[x], hi[x]);
      if (q < rows && lo[x] >= hi[x] && w.rem == 0 && !a.initL) bits |= kStatusEmptyRow;
      const __nv_bfloat16* qr = Q + (w.s.s0 + i) * a.q_stride + (w.h * a.G + r - i * a.G) * d;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int c = ks * 16 + y * 8 + 2 * t;
          qa[ks][x + 2 * y] = q < rows && c < d ? *reinterpret_cast<const uint32_t*>(qr + c) : 0u;
        }
    }
    // Keys that every row of the tile allows need no row mask.
    int all_lo, all_hi, unused;
    paged_row_span(a, w.s, w.t.i1, all_lo, unused);
    paged_row_span(a, w.s, w.t.i0, unused, all_hi);

    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.f;

    for (int i = i0; i < i1; ++i) {
      cp_wait<S - 2>();
      __syncwarp();  // tile i is in, and every lane is done with tile i - 1
      {
        const long long next = find(i + S);
        issue(i + S - 1, row);
        row = next;
      }
      const int s = i % S;
      const uint32_t kt = kbase + s * Lay::kTileBytes, vt = vbase + s * Lay::kTileBytes;
      const unsigned have = tile_keys[warp][s];
      float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      {
        const int r = ((lane >> 4) << 3) + (lane & 7), c = (lane >> 3) & 1;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if (ks * 16 >= d) break;
          uint32_t b[4];
          ldm4(b, kt + r * (D * 2) + (((2 * ks + c) ^ (r & 7)) << 4));
          mma16(sc[0], qa[ks], b[0], b[1]);
          mma16(sc[1], qa[ks], b[2], b[3]);
        }
      }
      const int key0 = first + i * kUnit;
      const bool whole = have == 0xFFFFu && key0 >= all_lo && key0 + kTile <= all_hi;
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[y][e] *= a.sl2;
          if (!whole) {
            const int k = y * 8 + 2 * t + (e & 1), x = e >> 1;
            if (!((have >> k) & 1u) || key0 + k < lo[x] || key0 + k >= hi[x]) sc[y][e] = -INFINITY;
          }
        }
      bool move = false;
      float top[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float mx = fmaxf(fmaxf(sc[0][2 * x], sc[0][2 * x + 1]), fmaxf(sc[1][2 * x], sc[1][2 * x + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
        top[x] = mx;
        move |= mx > m[x] + kRescale;
      }
      if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float to = fmaxf(m[x], top[x]);
          const float f = m[x] == -INFINITY ? 0.f : ex2(m[x] - to);
          m[x] = to;
          l[x] *= f;
#pragma unroll
          for (int y = 0; y < NT; ++y) {
            o[y][2 * x] *= f;
            o[y][2 * x + 1] *= f;
          }
        }
      }
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float ref = m[x] == -INFINITY ? 0.f : m[x];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float p0 = ex2(sc[y][2 * x] - ref), p1 = ex2(sc[y][2 * x + 1] - ref);
          l[x] += p0 + p1;
          const uint32_t h = pack_bf16x2(p0, p1);
          ph[x + 2 * y] = h;
          pl[x + 2 * y] = pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xFFFF0000u));
        }
      }
      {
        const int r = (((lane >> 3) & 1) << 3) + (lane & 7), c = lane >> 4;
#pragma unroll
        for (int y = 0; y < NT / 2; ++y) {
          if (y * 16 >= v) break;
          uint32_t b[4];
          ldm4t(b, vt + r * (D * 2) + (((2 * y + c) ^ (r & 7)) << 4));
          mma16(o[2 * y], ph, b[0], b[1]);
          mma16(o[2 * y + 1], ph, b[2], b[3]);
          mma16(o[2 * y], pl, b[0], b[1]);
          mma16(o[2 * y + 1], pl, b[2], b[3]);
        }
      }
    }
    cp_wait<0>();
    __syncwarp();

    // The warp's rows into its V ring, then all warps' together.
    float* z = reinterpret_cast<float*>(own + S * Lay::kTileBytes);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 1);
      l[x] += __shfl_xor_sync(0xFFFFFFFFu, l[x], 2);
      if (t == 0) {
        red_m[warp][g + 8 * x] = m[x];
        red_l[warp][g + 8 * x] = l[x];
      }
#pragma unroll
      for (int y = 0; y < NT; ++y)
        *reinterpret_cast<float2*>(z + (g + 8 * x) * D + y * 8 + 2 * t) =
            make_float2(o[y][2 * x], o[y][2 * x + 1]);
    }
    const int slot = paged_slot(a, w, n);
    __syncthreads();
    for (int idx = threadIdx.x; idx < rows * (v / 4); idx += 32 * kW) {
      const int q = idx / (v / 4), col = 4 * (idx - q * (v / 4));
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < kW; ++k) M = fmaxf(M, red_m[k][q]);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 zc = make_float4(0.f, 0.f, 0.f, 0.f);
      float lq = 0.f;
#pragma unroll
      for (int k = 0; k < kW; ++k) {
        const float f = ex2(red_m[k][q] - ref);
        const float4 x = *reinterpret_cast<const float4*>(sm + k * Lay::kWarpBytes + S * Lay::kTileBytes +
                                                          (q * D + col) * 4);
        zc.x = fmaf(f, x.x, zc.x);
        zc.y = fmaf(f, x.y, zc.y);
        zc.z = fmaf(f, x.z, zc.z);
        zc.w = fmaf(f, x.w, zc.w);
        lq = fmaf(f, red_l[k][q], lq);
      }
      if (slot < 0) {
        const size_t row_out = paged_out_row(a, w.s, w.h, r0 + q);
        const PagedScale f = paged_finish(a, row_out, M, lq);
        paged_store4(a, row_out, col, paged_join4(a, f, row_out, col, zc));
        if (col == 0) a.L[row_out] = f.L;
      } else {
        const size_t at = static_cast<size_t>(slot) * kRows + q;
        *reinterpret_cast<float4*>(a.pz + at * v + col) = zc;
        if (col == 0) {
          a.pm[at] = M;
          a.pl[at] = lq;
        }
      }
    }
    more = paged_next<kRows, kUnit>(a, w, n);
    __syncthreads();  // the joined rows are read before the next segment's copies land there
  }
  paged_end(a, bits);
}

template <int D>
cudaError_t mma_launch(const PagedArgs& a, cudaStream_t s) {
  auto kern = paged_mma_kernel<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MmaLayout<D>::kBytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  kern<<<a.ctas, 32 * kW, MmaLayout<D>::kBytes, s>>>(a);
  after_launch(kKernPaged, s);
  return cudaGetLastError();
}

}  // namespace

bool paged_mma_shape(int dtype, int d, int v) { return dtype == kBF16 && d <= 128 && v <= 128; }
PagedKernel paged_mma_kernel() { return {kRows, 2 * 152}; }

cudaError_t launch_paged_mma(const PagedArgs& a, cudaStream_t s) {
  return a.d <= 64 && a.v <= 64 ? mma_launch<64>(a, s) : mma_launch<128>(a, s);
}

}  // namespace exattn
