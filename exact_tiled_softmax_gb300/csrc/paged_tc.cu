// Paged attention for many rows to a key head (a chunk of a prompt, a batch over
// its shared prefix) in bf16, widths up to 128, on tcgen05, TMA and TMEM: bound by
// the tensor cores and the exponentials.
//
// A row tile is 256 rows, two 128-row halves A and B that share every key block
// of 128.  Roles (12 warps; for 8-bit pages four more): warps 0-3 and 4-7 the softmax of A and B, one thread a
// row; warp 8 the loads, warp 9 the products, warps 10-11 the rows of Q.  Warp 11
// also walks the CTA's segments and hands each to the others through a ring of two.  Per
// key block t the MMA warp issues S_A(t), PV_B(t-1), S_B(t), PV_A(t), so each half's softmax
// overlaps two products of the other.  TMEM: S_A [0,128), S_B [128,256), O_A, O_B behind; P
// (bf16) overwrites half of S and is the TMEM operand of P.V.  The reference point of the exponentials moves only when a
// row's maximum passes it by 2^8.  p is rounded to bf16 for P.V, as the dense
// forward does: the second product that would carry its remainder costs a third of
// the tensor time that bounds this kernel.
//
// Measured: chunks of 512 tokens of 4 sequences, 32 query heads over 8 key heads of 128
// columns, 8192 keys, causal: 197 to 200 us, 1.36 PFLOP/s or 73% of the measured peak, as the dense
// forward; the merge of the tiles that two CTAs share adds 14, launch and start 1 to 3.  (215 us
// a call at 2070 MHz; in a loop of seconds the power limit leaves 1807 MHz, and a call takes 226.)
// Pages of 8 keys, a box each: 347 us a call.  A short share costs its start
// and end: 6.7 key blocks a CTA (64 sequences' tokens over 16384 common keys) 28 us, 13 of
// them in the blocks.  Without the ring of segments, rows of Q read lane by lane, 281 us in
// place of 223 for the chunks and their merge.
//
// Pages.  A key block is loaded as boxes of min(page_size, 128) rows, one TMA load
// per box and 64 columns; lanes of the load warp look the pages up and issue their
// own box.  Rows that no key owns (behind the last key, before a window, on a page
// outside the pool) are not part of any row's mask (`keep`, four words a block,
// written beside the block's V), and the MMA warp zeroes them in V before P.V, so
// that what they hold, NaN included, meets no product that counts.
//
// Pages in 8 bits.  Their tiles are loaded as they are, and warps 12-15 turn them into the bf16 tiles of the
// products, a row's power of two folded in: an e4m3 number times it is a bf16 value, subnormal ones among them (under
// bytes 3 to 246; see bytes_to_bf16).  Tensor memory, full of
// S and O, has no room for the scales of a block-scaled product.  Measured: the chunks above 241 us a launch (258 a
// call, 1.03 PFLOP/s): converting shares the schedulers and shared memory with the softmax.  Without the
// conversion's work a call takes 221 us, without the softmax's 241, without both 172.  Pages of 8 keys: 353 us.
//
// Every wait is bounded; on a timeout the CTA records EXATTN_TIMEOUT, drains its
// own copies and products, frees TMEM and returns.
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace exattn {

PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder();

namespace {

using namespace tc;

constexpr int kHalf = 128;
constexpr int kRows = 2 * kHalf;
constexpr int kUnit = 128;
constexpr int kCtas = 152;
constexpr int kWarpTMA = 8, kWarpMMA = 9, kWarpQ = 10, kWarpConvert = 12;
// kBytes: pages in 8 bits, with four warps more, which convert them.  (Eight leave the softmax too few
// registers: 268 us in place of 257 for the chunks below.)
constexpr int kConverters = 4;
template <bool kBytes>
struct Warps {
  static constexpr int kSoftmaxRegs = kBytes ? 160 : 208;
  static constexpr int kProducerRegs = kBytes ? 96 : 88;
  static constexpr int kThreads = 384 + (kBytes ? 32 * kConverters : 0);
  static constexpr int kTakers = 11 + (kBytes ? kConverters : 0);  // warps that read a segment from the ring
};
constexpr int kQThreads = 64;
constexpr float kRescale = 8.f;
constexpr uint32_t kTmemCols = 512;

struct TcParams {
  CUtensorMap tk, tv;  // the pools as [num_pages * Hk * page_size][width], boxes 64 (bytes: D) x box_rows
  PagedArgs a;
  int box_rows;
};

// A segment, as warp 11 hands it out; n == 0: no more.
struct TcSegment {
  int n, kb0, j0, j1, rows, r0, h, b, slot, parts, s0, nq, len;  // parts: see PagedPlace
};

template <int D, bool kBytes>
struct TcLayout {
  static constexpr int CHUNKS = D / 64;
  static constexpr int QTILE = kHalf * D * 2;
  static constexpr int SLOT = kUnit * D * 2;
  // K and V of a block take one each.  Pages in 8 bits: and one each of the tiles as they are loaded.
  static constexpr int NSLOT = kBytes ? (D == 128 ? 3 : 6) : D == 128 ? 4 : 8;
  static constexpr int NRAW = kBytes ? (D == 128 ? 3 : 6) : 0;
  static constexpr int RAW = kUnit * D;
  // Blocks whose masks are kept: K of block t + 4 is converted when K of t + 1 (NSLOT 6) or V of t + 2 (3) is
  // done with, and the softmax with block t before that.
  static constexpr int kKeepBlocks = 4;
  static constexpr int Q_OFF = 0;
  static constexpr int SLOT_OFF = 2 * QTILE;
  static constexpr int RAW_OFF = SLOT_OFF + NSLOT * SLOT;
  static constexpr int BAR_OFF = RAW_OFF + NRAW * RAW;
  static constexpr int B_Q = 0, B_QFREE = 1, B_KVF = 2, B_KVE = B_KVF + NSLOT, B_S = B_KVE + NSLOT,
                       B_P = B_S + 2, B_O = B_P + 2, B_OREAD = B_O + 2, B_SEGF = B_OREAD + 2, B_SEGE = B_SEGF + 2, B_DRAIN = B_SEGE + 2,
                       B_RF = B_DRAIN + 1, B_RE = B_RF + NRAW, NBAR = B_RE + NRAW;
  static constexpr int KEEP_OFF = BAR_OFF + (NBAR * 8 + 15) / 16 * 16;  // 4 words a slot (bytes: a block)
  static constexpr int RKEEP_OFF = KEEP_OFF + (kBytes ? kKeepBlocks : NSLOT) * 16;  // the same of the raw tiles
  static constexpr int EXP_OFF = RKEEP_OFF + NRAW * 16;                 // and their keys' exponent bytes
  static constexpr int MISC_OFF = EXP_OFF + NRAW * kUnit;               // TMEM base, abort flag, status bits
  static constexpr int SEG_OFF = MISC_OFF + 16;
  static constexpr int TOTAL = SEG_OFF + 2 * 64;
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(ALLOC + kPagedSums * 8 + 256 <= 232448, "shared memory");
};

__device__ __forceinline__ uint32_t range_bits(int a, int b) {  // bits [a, b] of a word
  a = max(a, 0);
  b = min(b, 31);
  if (a > b) return 0u;
  const uint32_t width = static_cast<uint32_t>(b - a + 1);
  return (width == 32 ? 0xFFFFFFFFu : ((1u << width) - 1u)) << a;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                            int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// mbar_wait of a whole warp: all lanes go on, or none does.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, abort));
}

// Sixteen e4m3 numbers of a row with factor f, as bf16: exact from f = 2^-124 to 2^119.  Above, numbers may be 2^128 and
// infinite, below they may end under bf16's last place, 2^-133.
__device__ __forceinline__ void bytes_to_bf16(const uint4& raw, float f, uint32_t (&y)[8]) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = i & 1 ? e4m3_pair_high(w[i >> 1]) : e4m3_pair(w[i >> 1]);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    float x0, x1;
    fmul2(x0, x1, x.x, x.y, f, f);
    y[i] = pack_bf16x2(x0, x1);
  }
}

// A block's softmax for sixteen warps, which leave these 160 registers: the row's scores are read
// twice, 64 at a time, once for the maximum.  Keys lo to hi of the block where `mw` has them.
template <int D>
__device__ __forceinline__ void softmax_by_halves(uint32_t t_s, uint32_t t_o, bool whole, const uint32_t (&mw)[4],
                                                  int lo, int hi, float sl2, float& m_ref, float& l) {
  auto load = [&](int half, uint32_t (&s)[64]) {
    tmem_ld32(t_s + 64 * half, *reinterpret_cast<uint32_t(*)[32]>(s));
    tmem_ld32(t_s + 64 * half + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
    tmem_ld_wait();
    reg_fence(s);
    if (!whole) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t w = mw[2 * half + q] & range_bits(lo - 32 * (2 * half + q), hi - 32 * (2 * half + q));
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (!((w >> c) & 1u)) s[32 * q + c] = __float_as_uint(-INFINITY);
      }
    }
  };
  float mx = -INFINITY;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t s[64];
    load(half, s);
    float mx4[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) mx4[k] = __uint_as_float(s[k]);
#pragma unroll
    for (int c = 4; c + 8 <= 64; c += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) mx4[k] = fmax3(mx4[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + 4 + k]));
#pragma unroll
    for (int k = 0; k < 4; ++k) mx = fmax3(mx, mx4[k], __uint_as_float(s[60 + k]));
  }
  const float m_new = fmaxf(m_ref, mx * sl2);  // sl2 > 0
  const bool need = m_ref != -INFINITY && m_new > m_ref + kRescale;
  if (m_ref == -INFINITY) m_ref = m_new;
  if (__any_sync(0xFFFFFFFFu, need)) {
    const float alpha = need ? ex2(m_ref - m_new) : 1.f;
    if (need) m_ref = m_new;
    l *= alpha;
#pragma unroll
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t o[32];
      tmem_ld32(t_o + ch * 32, o);
      tmem_ld_wait();
      reg_fence(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
      tmem_st32(t_o + ch * 32, o);
    }
  }
  const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
  float sum2[4][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t s[64], pk[32];
    load(half, s);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float x0, x1;
      ffma2(x0, x1, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), sl2, sl2, neg, neg);
      const float p0 = ex2(x0), p1 = ex2(x1);
      fadd2(sum2[e & 3][0], sum2[e & 3][1], sum2[e & 3][0], sum2[e & 3][1], p0, p1);
      pk[e] = pack_bf16x2(p0, p1);
    }
    tmem_st32(t_s + 32 * half, pk);
  }
  l += ((sum2[0][0] + sum2[0][1]) + (sum2[1][0] + sum2[1][1])) + ((sum2[2][0] + sum2[2][1]) + (sum2[3][0] + sum2[3][1]));
  tmem_st_wait();
}

template <int D, bool kBytes>
__global__ void __launch_bounds__(Warps<kBytes>::kThreads, 1)
    paged_tc_kernel(const __grid_constant__ TcParams p) {
  using Lay = TcLayout<D, kBytes>;
  constexpr int NS = Lay::NSLOT, NR = kBytes ? Lay::NRAW : 1;
  constexpr int kThreads = Warps<kBytes>::kThreads;
  extern __shared__ uint8_t smem_raw[];
  __shared__ long long pre[kPagedSums], scan[kThreads / 32];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Lay::BAR_OFF;
  auto bar = [&](int k) { return bar0 + 8u * k; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + Lay::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile uint32_t* keep = reinterpret_cast<volatile uint32_t*>(smem + Lay::KEEP_OFF);
  const PagedArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(bar(Lay::B_Q), kQThreads);
    mbar_init(bar(Lay::B_QFREE), 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(bar(Lay::B_KVF + s), kBytes ? 32 * kConverters : 1);
      mbar_init(bar(Lay::B_KVE + s), 1);
    }
    for (int s = 0; s < Lay::NRAW; ++s) {
      mbar_init(bar(Lay::B_RF + s), 1);
      mbar_init(bar(Lay::B_RE + s), kConverters);
    }
    for (int X = 0; X < 2; ++X) {
      mbar_init(bar(Lay::B_S + X), 1);
      mbar_init(bar(Lay::B_P + X), kHalf);
      mbar_init(bar(Lay::B_O + X), 1);
      mbar_init(bar(Lay::B_OREAD + X), kHalf);
      mbar_init(bar(Lay::B_SEGF + X), 1);
      mbar_init(bar(Lay::B_SEGE + X), Warps<kBytes>::kTakers);
    }
    mbar_init(bar(Lay::B_DRAIN), 1);
    misc[1] = misc[2] = 0;
    fence_mbar_init();
  }
  if (warp == kWarpMMA) {
    tmem_alloc(sbase + Lay::MISC_OFF, kTmemCols);
    tmem_relinquish();
    tc_fence_before();
  }
  unsigned bits = 0;
  if (!a.second) wait_for_previous();
  let_next_start();
  if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  paged_scan<kRows, kUnit, kThreads>(a, pre, scan, bits);  // two barriers of the CTA
  tc_fence_after();
  const uint32_t tmem = misc[0];
  // Segment `seg` from the ring; false when there is none (or a wait gave up: ok).
  volatile int* ring = reinterpret_cast<volatile int*>(smem + Lay::SEG_OFF);
  auto take = [&](int seg, TcSegment& t, bool& ok) {
    const int e = seg & 1;
    if (!(ok = wait_all(bar(Lay::B_SEGF + e), (seg >> 1) & 1, abort_flag))) return false;
    volatile int* r = ring + 16 * e;
    t.n = r[0];
    t.kb0 = r[1];
    t.j0 = r[2];
    t.j1 = r[3];
    t.rows = r[4];
    t.r0 = r[5];
    t.h = r[6];
    t.b = r[7];
    t.slot = r[8];
    t.parts = r[9];
    t.s0 = r[10];
    t.nq = r[11];
    t.len = r[12];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(Lay::B_SEGE + e));
    return t.n > 0;
  };
  // Roles count segments (`seg`) and key blocks; K of block blk is fill 2 blk of the
  // ring of tiles, V fill 2 blk + 1.

  if (warp >= 8) {
    regs_dec<Warps<kBytes>::kProducerRegs>();
    const bool leader = elect_one();
    if constexpr (kBytes) {
      if (warp >= kWarpConvert) {
        // A raw tile to bf16 in the products' 128-byte swizzled layout, its rows' powers of two in: warp
        // by warp.  A lane takes 16 columns: quads have four pieces of a row, and neighbouring rows
        // the two halves of one, so that neither the loads nor the stores of eight lanes meet in a bank.
        constexpr int kRowsOf = kUnit / kConverters;
        static_assert(kRowsOf == 32, "a word of the mask each");
        const int wr = (warp - kWarpConvert) * kRowsOf, q = lane & 3, odd = (lane >> 2) & 1;
        volatile uint32_t* rkeep = reinterpret_cast<volatile uint32_t*>(smem + Lay::RKEEP_OFF);
        bool ok = true;
        int fill = 0;
        TcSegment t;
        for (int seg = 0; take(seg, t, ok); ++seg) {
          for (int u = 0; u < 2 * t.n && ok; ++u, ++fill) {
            const int rs = fill % NR, ks = fill % NS;
            if (!(ok = wait_all(bar(Lay::B_RF + rs), (fill / NR) & 1, abort_flag))) break;
            if (!(ok = wait_all(bar(Lay::B_KVE + ks), ((fill / NS) & 1) ^ 1, abort_flag))) break;
            // V: rows without a key are zero, whatever their page holds (K's scores do not count).
            uint32_t mine = rkeep[rs * 4 + (wr >> 5)];
            if (!(u & 1)) {
              if (lane == 0) keep[(fill / 2 % Lay::kKeepBlocks) * 4 + (wr >> 5)] = mine;
              mine = 0xFFFFFFFFu;
            }
            const uint8_t* ex = smem + Lay::EXP_OFF + rs * kUnit + wr;
            const uint32_t raw = sbase + Lay::RAW_OFF + rs * Lay::RAW + wr * D;
            const uint32_t to = sbase + Lay::SLOT_OFF + ks * Lay::SLOT + wr * 128;
            // All loads before the first use: beside the products' own reads a shared load takes long.
            constexpr int kPieces = D / 16 * kRowsOf / 32;
            uint4 x[kPieces];
            float f[kPieces];
            auto row_of = [&](int y) { return (D == 128 ? y >> 1 : y) * 8 + 2 * (lane >> 3) + odd; };  // of the warp's
            auto piece_of = [&](int y) { return q + (D == 128 ? 4 * (odd ^ (y & 1)) : 0); };
#pragma unroll
            for (int y = 0; y < kPieces; ++y) x[y] = ld_shared_v4(raw + row_of(y) * D + piece_of(y) * 16);
#pragma unroll
            for (int y = 0; y < kPieces; ++y) f[y] = e4m3_scale(ex[row_of(y)]);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(Lay::B_RE + rs));
            if (mine != 0xFFFFFFFFu) {  // the same for the whole warp
#pragma unroll
              for (int y = 0; y < kPieces; ++y)
                if (!((mine >> row_of(y)) & 1u)) {
                  x[y] = make_uint4(0u, 0u, 0u, 0u);
                  f[y] = 0.f;
                }
            }
#pragma unroll
            for (int y = 0; y < kPieces; ++y) {
              const int r = row_of(y);
              uint32_t z[8];
              bytes_to_bf16(x[y], f[y], z);
              const uint32_t row = to + (piece_of(y) >> 2) * (kUnit * 128) + r * 128;
              st_shared_v4(row + (((2 * q) ^ (r & 7)) << 4), z[0], z[1], z[2], z[3]);
              st_shared_v4(row + (((2 * q + 1) ^ (r & 7)) << 4), z[4], z[5], z[6], z[7]);
            }
            fence_proxy_async_smem();
            mbar_arrive(bar(Lay::B_KVF + ks));
          }
          if (!ok) break;  // not on to the next segment, whose wait may succeed
        }
        if (!ok) {
          bits |= kStatusTimeout;
          *abort_flag = 1;
        }
      }
    }
    if (warp == kWarpTMA) {
      if (leader) {
        prefetch_tmap(&p.tk);
        prefetch_tmap(&p.tv);
      }
      const int br = p.box_rows, nb = kUnit / br;
      bool ok = true;
      int fill = 0;
      TcSegment t;
      for (int seg = 0; take(seg, t, ok); ++seg) {
        const int* trow = paged_table(a, t.b);
        // Lane l: the pool row of box l of block u, or -1.
        auto find = [&](int u) {
          int row = -1;
          const int key = t.kb0 + u * kUnit + lane * br;
          if (u < t.n && lane < nb && key < t.j1 && key + br > t.j0) {
            const long long at = paged_key_row(a, trow, t.h, key);
            if (at < 0) bits |= kStatusBadPage;
            row = static_cast<int>(at);
          }
          return row;
        };
        // Bytes: the exponents of keys 4 lane to 4 lane + 3 of the block whose boxes are at `rows`.
        auto exponents = [&](int rows) {
          uint2 e = make_uint2(0u, 0u);
          if constexpr (kBytes) {
            const int at = __shfl_sync(0xFFFFFFFFu, rows, 4 * lane / br);
            if (at >= 0) {
              const size_t from = static_cast<size_t>(at) + 4 * lane % br;
              e.x = __ldg(reinterpret_cast<const unsigned*>(a.Ks + from));
              e.y = __ldg(reinterpret_cast<const unsigned*>(a.Vs + from));
            }
          }
          return e;
        };
        int row = find(0);
        uint2 ex = exponents(row);
        for (int u = 0; u < t.n && ok; ++u) {
          const int next = find(u + 1);
          const uint2 ex_next = exponents(next);
          const int kb = t.kb0 + u * kUnit;
          const unsigned boxes = __ballot_sync(0xFFFFFFFFu, row >= 0);
          const uint32_t bytes = __popc(boxes) * br * (kBytes ? D : 128 * Lay::CHUNKS);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            // The ring that is loaded into.
            constexpr int N = kBytes ? NR : NS, kFull = kBytes ? Lay::B_RF : Lay::B_KVF,
                          kEmpty = kBytes ? Lay::B_RE : Lay::B_KVE, kKeep = kBytes ? Lay::RKEEP_OFF : Lay::KEEP_OFF;
            const int slot = fill % N, phase = (fill / N) & 1;
            if (!(ok = wait_all(bar(kEmpty + slot), phase ^ 1, abort_flag))) break;
            ++fill;
            if constexpr (kBytes)
              reinterpret_cast<volatile uint32_t*>(smem + Lay::EXP_OFF)[slot * (kUnit / 4) + lane] = kv ? ex.y : ex.x;
            if ((kBytes || kv == 1) && lane < 4) {
              uint32_t word = range_bits(t.j0 - kb - 32 * lane, t.j1 - 1 - kb - 32 * lane);
              for (int b = 0; b < nb; ++b)
                if (!((boxes >> b) & 1u)) word &= ~range_bits(b * br - 32 * lane, b * br + br - 1 - 32 * lane);
              reinterpret_cast<volatile uint32_t*>(smem + kKeep)[slot * 4 + lane] = word;
            }
            __syncwarp();
            if (leader) mbar_arrive_expect_tx(bar(kFull + slot), bytes);
            __syncwarp();
            if constexpr (kBytes) {
              if (row >= 0)
                tma_load_2d(sbase + Lay::RAW_OFF + slot * Lay::RAW + lane * br * D, kv ? &p.tv : &p.tk,
                            bar(kFull + slot), 0, row);
            } else {
              const uint32_t dst = sbase + Lay::SLOT_OFF + slot * Lay::SLOT + lane * br * 128;
              if (row >= 0)
#pragma unroll
                for (int c = 0; c < Lay::CHUNKS; ++c)
                  tma_load_2d(dst + c * (kUnit * 128), kv ? &p.tv : &p.tk, bar(kFull + slot), 64 * c, row);
            }
            __syncwarp();
          }
          row = next;
          ex = ex_next;
        }
        if (!ok) break;
      }
      if (!ok) {
        bits |= kStatusTimeout;
        if (leader) *abort_flag = 1;
      }
      // Never leave with copies in flight: the last fill of every slot has landed.
      constexpr int N = kBytes ? NR : NS, kFull = kBytes ? Lay::B_RF : Lay::B_KVF;
      for (int u = 0; u < N && u < fill; ++u) {
        const int i = fill - 1 - u;
        mbar_wait_inflight(bar(kFull + i % N), (i / N) & 1);
      }
    } else if (warp == kWarpMMA) {
      constexpr uint32_t kIdescS = idesc_bf16(kHalf, kUnit, false, false);
      constexpr uint32_t kIdescPV = idesc_bf16(kHalf, D, false, true);
      const uint64_t dq0 = sdesc_sw128(sbase + Lay::Q_OFF, 16, 1024);
      const uint64_t dk0 = sdesc_sw128(sbase + Lay::SLOT_OFF, 16, 1024);
      const uint64_t dv0 = sdesc_sw128(sbase + Lay::SLOT_OFF, kUnit * 128, 1024);
      bool ok = true;
      int fill = 0, p_phase[2] = {0, 0};
      auto commit = [&](int b) {
        if (leader) tc_commit(bar(b));
      };
      auto issue_s = [&](int X, int slot) {
        const uint64_t qd = dq0 + static_cast<uint64_t>(X * (Lay::QTILE >> 4));
        const uint64_t kd = dk0 + static_cast<uint64_t>(slot * (Lay::SLOT >> 4));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * (kHalf * 128) + (kk & 3) * 32) >> 4;
            mma_ss(tmem + X * kUnit, qd + off, kd + off, kIdescS, kk > 0 ? 1u : 0u);
          }
        }
        commit(Lay::B_S + X);
      };
      auto issue_pv = [&](int X, int slot, bool first) {
        const uint64_t vd = dv0 + static_cast<uint64_t>(slot * (Lay::SLOT >> 4));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kUnit / 16; ++kk)
            mma_ts(tmem + 2 * kUnit + X * D, tmem + X * kUnit + kk * 8, vd + kk * 128, kIdescPV,
                   kk > 0 || !first ? 1u : 0u);
        }
      };
      TcSegment t;
      for (int seg = 0; take(seg, t, ok); ++seg) {
        const int n = t.n;
        const bool two = t.rows > kHalf;
        if (!(ok = wait_all(bar(Lay::B_Q), seg & 1, abort_flag))) break;
        tc_fence_after();
        int v_prev = -1;  // V slot whose P.V of half B is still to come
        for (int u = 0; u < n && ok; ++u) {
          const int ks = fill % NS, kphase = (fill / NS) & 1;
          const int vs = (fill + 1) % NS, vphase = ((fill + 1) / NS) & 1;
          fill += 2;
          if (!(ok = wait_all(bar(Lay::B_KVF + ks), kphase, abort_flag))) break;
          tc_fence_after();
          issue_s(0, ks);
          if (u > 0) {
            if (two) {
              if (!(ok = wait_all(bar(Lay::B_P + 1), p_phase[1] & 1, abort_flag))) break;
              tc_fence_after();
              ++p_phase[1];
              issue_pv(1, v_prev, u == 1);
            }
            commit(Lay::B_KVE + v_prev);
          }
          if (two) issue_s(1, ks);
          if (u == n - 1) commit(Lay::B_QFREE);
          commit(Lay::B_KVE + ks);
          if (!(ok = wait_all(bar(Lay::B_KVF + vs), vphase, abort_flag))) break;
          // Rows without a key are zeroed in V (bytes: they are already).
          uint32_t kw[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) kw[q] = kBytes ? 0xFFFFFFFFu : keep[vs * 4 + q];
          if ((kw[0] & kw[1] & kw[2] & kw[3]) != 0xFFFFFFFFu) {
            const uint32_t vt = sbase + Lay::SLOT_OFF + vs * Lay::SLOT;
#pragma unroll 1
            for (int r = lane >> 3; r < kUnit; r += 4) {
              const uint32_t word = r < 64 ? (r < 32 ? kw[0] : kw[1]) : (r < 96 ? kw[2] : kw[3]);
              if (!((word >> (r & 31)) & 1u))
#pragma unroll
                for (int c = 0; c < Lay::CHUNKS; ++c)
                  st_shared_v4(vt + c * (kUnit * 128) + r * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          tc_fence_after();
          if (!(ok = wait_all(bar(Lay::B_P + 0), p_phase[0] & 1, abort_flag))) break;
          tc_fence_after();
          ++p_phase[0];
          issue_pv(0, vs, u == 0);
          v_prev = vs;
        }
        if (ok && two) {
          if ((ok = wait_all(bar(Lay::B_P + 1), p_phase[1] & 1, abort_flag))) {
            tc_fence_after();
            ++p_phase[1];
            issue_pv(1, v_prev, n == 1);
          }
        }
        if (ok) commit(Lay::B_KVE + v_prev);
        for (int X = 0; X < 2 && ok; ++X) {
          if (seg > 0 && !(ok = wait_all(bar(Lay::B_OREAD + X), (seg - 1) & 1, abort_flag))) break;
          commit(Lay::B_O + X);
        }
        __syncwarp();
        if (!ok) break;
      }
      if (!ok) {
        bits |= kStatusTimeout;
        if (leader) *abort_flag = 1;
      }
      __syncwarp();
      commit(Lay::B_DRAIN);
      mbar_wait_inflight(bar(Lay::B_DRAIN), 0);
    } else if (warp < kWarpConvert) {
      // The rows of Q, in the 128-byte swizzled layout of the products' operand: warp
      // 10 the even groups of 32 rows, warp 11 the odd ones.  A lane finds one row, the
      // warp copies them together.
      const __nv_bfloat16* Q = static_cast<const __nv_bfloat16*>(a.Q);
      constexpr int CH = D / 8, kPass = 32 / CH;  // rows that a warp copies at once
      const int kch = a.d / 8;
      bool ok = true;
      auto copy_q = [&](const TcSegment& t) {
        const int groups = t.rows > kHalf ? kRows / 32 : kHalf / 32;
#pragma unroll 1
        for (int x = warp - kWarpQ; x < groups; x += 2) {
          const int mine = x * 32 + lane, r = t.r0 + (mine < t.rows ? mine : 0);
          const int i = div_by(r, a.by_group);
          const long long src = reinterpret_cast<long long>(Q + (t.s0 + i) * a.q_stride +
                                                            (t.h * a.G + r - i * a.G) * a.d);
          const uint32_t half = sbase + Lay::Q_OFF + (x / (kHalf / 32)) * Lay::QTILE;
          const int c = lane % CH;
          const uint32_t piece = half + (c >> 3) * (kHalf * 128);
#pragma unroll 4
          for (int y = 0; y < 32; y += kPass) {
            const int rr = y + lane / CH, row = x * 32 + rr;  // of the tile
            const char* from = reinterpret_cast<const char*>(__shfl_sync(0xFFFFFFFFu, src, rr));
            const bool has = row < t.rows && c < kch;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             piece + (row % kHalf) * 128 + (((c & 7) ^ (row & 7)) << 4)),
                         "l"(from + (c < kch ? c * 16 : 0)), "r"(has ? 16 : 0)
                         : "memory");
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(bar(Lay::B_Q));
      };
      TcSegment t;
      if (warp == kWarpQ) {
        for (int seg = 0; take(seg, t, ok); ++seg) {
          if (seg > 0 && !(ok = wait_all(bar(Lay::B_QFREE), (seg - 1) & 1, abort_flag))) break;
          copy_q(t);
        }
      } else {
        PagedWalk w;
        bool more = paged_begin<kRows, kUnit>(a, pre, blockIdx.x, w);
        for (int seg = 0; ok; ++seg) {
          const int e = seg & 1;
          t.n = 0;
          if (more) {
            t.n = paged_segment<kUnit>(w, t.j0, t.j1);
            t.kb0 = (w.t.kt0 + w.rem) * kUnit;
            t.rows = w.t.rows;
            t.r0 = w.rt * kRows;
            t.h = w.h;
            t.b = w.b;
            const PagedPlace place = paged_place<kRows>(a, pre[a.B], w, t.n, blockIdx.x, lane == 0);
            t.slot = place.slot;
            t.parts = place.parts;
            t.s0 = w.s.s0;
            t.nq = w.s.nq;
            t.len = w.s.len;
          }
          if (seg >= 2 && !(ok = wait_all(bar(Lay::B_SEGE + e), ((seg >> 1) - 1) & 1, abort_flag))) break;
          if (lane == 0) {
            volatile int* r = ring + 16 * e;
            r[0] = t.n;
            r[1] = t.kb0;
            r[2] = t.j0;
            r[3] = t.j1;
            r[4] = t.rows;
            r[5] = t.r0;
            r[6] = t.h;
            r[7] = t.b;
            r[8] = t.slot;
            r[9] = t.parts;
            r[10] = t.s0;
            r[11] = t.nq;
            r[12] = t.len;
            mbar_arrive(bar(Lay::B_SEGF + e));
          }
          __syncwarp();
          if (!more) break;
          if (seg > 0 && !(ok = wait_all(bar(Lay::B_QFREE), (seg - 1) & 1, abort_flag))) break;
          copy_q(t);
          more = paged_next<kRows, kUnit>(a, w);
        }
      }
      if (!ok) {
        bits |= kStatusTimeout;
        *abort_flag = 1;
      }
    }
  } else {
    regs_inc<Warps<kBytes>::kSoftmaxRegs>();
    const int X = warp >> 2;
    const int wl = warp & 3;
    const int rl = X * kHalf + wl * 32 + lane;  // row of the tile
    const uint32_t lane_off = static_cast<uint32_t>(wl * 32) << 16;
    const uint32_t t_s = tmem + lane_off + X * kUnit;
    const uint32_t t_o = tmem + lane_off + 2 * kUnit + X * D;
    const float sl2 = a.sl2;
    bool ok = true;
    int blk = 0, cnt = 0;
    TcSegment t;
    for (int seg = 0; take(seg, t, ok); ++seg) {
      const int n = t.n, r0 = t.r0, rows = t.rows, kb0 = t.kb0;
      const PagedSeq sq{t.s0, t.nq, t.len, t.b == a.prefix_at, false};
      const bool on = X * kHalf < rows;  // this half has rows
      const bool valid = rl < rows;
      int lo, hi, all_lo = 0, all_hi = 0;
      paged_row_span(a, sq, div_by(r0 + (valid ? rl : 0), a.by_group), lo, hi);
      if (valid && lo >= hi && t.parts >= 0 && !a.info) bits |= kStatusEmptyRow;
      if (on) {
        int unused;
        paged_row_span(a, sq, div_by(r0 + min(rows, X * kHalf + kHalf) - 1, a.by_group), all_lo, unused);
        paged_row_span(a, sq, div_by(r0 + X * kHalf, a.by_group), unused, all_hi);
      }
      float m_ref = -INFINITY, l = 0.f;
      for (int u = 0; u < n && on; ++u) {
        const int vf = 2 * (blk + u) + 1, vs = vf % NS;
        uint32_t mw[4];
        if constexpr (!kBytes) {
          if (!(ok = wait_all(bar(Lay::B_KVF + vs), (vf / NS) & 1, abort_flag))) break;
#pragma unroll
          for (int q = 0; q < 4; ++q) mw[q] = keep[vs * 4 + q];
        }
        const int kb = kb0 + u * kUnit;
        if (!(ok = wait_all(bar(Lay::B_S + X), cnt & 1, abort_flag))) break;
        if constexpr (kBytes) {  // written before K was there for the product
#pragma unroll
          for (int q = 0; q < 4; ++q) mw[q] = keep[((blk + u) % Lay::kKeepBlocks) * 4 + q];
        }
        const bool whole = (mw[0] & mw[1] & mw[2] & mw[3]) == 0xFFFFFFFFu && kb >= all_lo && kb + kUnit <= all_hi;
        tc_fence_after();
        ++cnt;
        if constexpr (kBytes) {
          softmax_by_halves<D>(t_s, t_o, whole, mw, lo - kb, hi - 1 - kb, sl2, m_ref, l);
          tc_fence_before();
          mbar_arrive(bar(Lay::B_P + X));
          continue;
        }
        uint32_t s[128];
        tmem_ld32(t_s + 0, *reinterpret_cast<uint32_t(*)[32]>(s + 0));
        tmem_ld32(t_s + 32, *reinterpret_cast<uint32_t(*)[32]>(s + 32));
        tmem_ld32(t_s + 64, *reinterpret_cast<uint32_t(*)[32]>(s + 64));
        tmem_ld32(t_s + 96, *reinterpret_cast<uint32_t(*)[32]>(s + 96));
        tmem_ld_wait();
        reg_fence(s);
        if (!whole) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mw[q] &= range_bits(lo - kb - 32 * q, hi - 1 - kb - 32 * q);
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!((mw[c >> 5] >> (c & 31)) & 1u)) s[c] = __float_as_uint(-INFINITY);
        }
        float mx8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = __uint_as_float(s[k]);
#pragma unroll
        for (int c = 8; c + 16 <= 128; c += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx8[k] = fmax3(mx8[k], __uint_as_float(s[c + k]), __uint_as_float(s[c + 8 + k]));
#pragma unroll
        for (int k = 0; k < 8; ++k) mx8[k] = fmaxf(mx8[k], __uint_as_float(s[120 + k]));
        const float mx =
            fmaxf(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float m_new = fmaxf(m_ref, mx * sl2);  // sl2 > 0
        const bool need = m_ref != -INFINITY && m_new > m_ref + kRescale;
        if (m_ref == -INFINITY) m_ref = m_new;
        if (__any_sync(0xFFFFFFFFu, need)) {
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;
          if (need) m_ref = m_new;
          l *= alpha;
#pragma unroll
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t o[32];
            tmem_ld32(t_o + ch * 32, o);
            tmem_ld_wait();
            reg_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(t_o + ch * 32, o);
          }
        }
        const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
        float sum2[4][2] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(s[64 * half + 2 * e]), __uint_as_float(s[64 * half + 2 * e + 1]), sl2,
                  sl2, neg, neg);
            const float p0 = ex2(x0), p1 = ex2(x1);
            fadd2(sum2[e & 3][0], sum2[e & 3][1], sum2[e & 3][0], sum2[e & 3][1], p0, p1);
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st32(t_s + 32 * half, pk);
        }
        l += ((sum2[0][0] + sum2[0][1]) + (sum2[1][0] + sum2[1][1])) +
             ((sum2[2][0] + sum2[2][1]) + (sum2[3][0] + sum2[3][1]));
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(Lay::B_P + X));
      }
      if (!ok) break;
      blk += n;
      if (!(ok = wait_all(bar(Lay::B_O + X), seg & 1, abort_flag))) break;
      tc_fence_after();
      const float m = l > 0.f || l != l ? m_ref : -INFINITY;
      const size_t row = paged_out_row(a, sq.s0, t.h, r0 + (valid ? rl : 0), sq.prefix);
      if (a.info && t.parts >= 0 && valid) a.info[row] = make_int2(blockIdx.x, t.parts);
      if (t.slot >= 0) {
        // The summary, [v / 8][256] pieces of eight columns: a warp's stores are whole lines.
        float* z = a.pz + (static_cast<size_t>(t.slot) * (a.v / 8) * kRows + rl) * 8;
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          if (!on || ch * 32 >= a.v) break;
          uint32_t o[32];
          tmem_ld32(t_o + ch * 32, o);
          tmem_ld_wait();
          reg_fence(o);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (valid && ch * 32 + 8 * e < a.v)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                               z + static_cast<size_t>(ch * 4 + e) * kRows * 8),
                           "r"(o[8 * e]), "r"(o[8 * e + 1]), "r"(o[8 * e + 2]), "r"(o[8 * e + 3]), "r"(o[8 * e + 4]),
                           "r"(o[8 * e + 5]), "r"(o[8 * e + 6]), "r"(o[8 * e + 7])
                           : "memory");
        }
        tc_fence_before();
        mbar_arrive(bar(Lay::B_OREAD + X));
        if (valid) {
          a.pm[static_cast<size_t>(t.slot) * kRows + rl] = m;
          a.pl[static_cast<size_t>(t.slot) * kRows + rl] = l;
        }
      } else {
        PagedScale f{0.f, 0.f};
        if (valid) {
          f = paged_finish(m, l);
          a.L[row] = f.L;
        }
#pragma unroll
        for (int ch = 0; ch < D / 32; ++ch) {
          if (!on || ch * 32 >= a.v) break;
          uint32_t o[32];
          tmem_ld32(t_o + ch * 32, o);
          tmem_ld_wait();
          reg_fence(o);
          if (!valid) continue;
          if (!a.Yf) {
            uint4* y = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.Y) + row * a.v + ch * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // eight columns a store (v is a multiple of 8)
              if (ch * 32 + 8 * e >= a.v) break;
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                h[k] = pack_bf16x2(__uint_as_float(o[8 * e + 2 * k]) * f.fz,
                                   __uint_as_float(o[8 * e + 2 * k + 1]) * f.fz);
              y[e] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else {
            float4* y = reinterpret_cast<float4*>(a.Yf + row * a.v + ch * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (ch * 32 + 4 * e < a.v)
                y[e] = make_float4(__uint_as_float(o[4 * e]) * f.fz, __uint_as_float(o[4 * e + 1]) * f.fz,
                                   __uint_as_float(o[4 * e + 2]) * f.fz, __uint_as_float(o[4 * e + 3]) * f.fz);
          }
        }
        tc_fence_before();
        mbar_arrive(bar(Lay::B_OREAD + X));
      }
    }
    if (!ok) {
      bits |= kStatusTimeout;
      *abort_flag = 1;
    }
  }

  tc_fence_before();
  if (a.second) wait_for_previous();
  paged_end(a, bits, reinterpret_cast<unsigned*>(misc + 2));
  if (warp == kWarpMMA) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// width: of the pool's rows; box: of a box, in elements.
bool pool_map(CUtensorMap* m, const void* base, const PagedArgs& a, int width, int box, int box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return false;
  const bool bytes = a.Ks != nullptr;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(width),
                        (static_cast<cuuint64_t>(a.num_pages) * a.Hk) << a.lps};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(width) * (bytes ? 1 : 2)};
  cuuint32_t boxes[2] = {static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                         const_cast<void*>(base), dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) record_error("cuTensorMapEncodeTiled", static_cast<int>(r), "");
  return r == CUDA_SUCCESS;
}

template <int D, bool kBytes>
cudaError_t tc_launch(const PagedArgs& a, cudaStream_t s) {
  TcParams p;
  p.a = a;
  p.box_rows = min(1 << a.lps, kUnit);
  const int box = kBytes ? D : 64;
  if (!pool_map(&p.tk, a.Kp, a, a.d, box, p.box_rows) || !pool_map(&p.tv, a.Vp, a, a.v, box, p.box_rows))
    return cudaErrorInvalidValue;
  constexpr int bytes = TcLayout<D, kBytes>::ALLOC;
  const cudaError_t e = allow_smem<paged_tc_kernel<D, kBytes>>(bytes);
  if (e != cudaSuccess) return e;
  before_launch(kKernPaged, s);
  const cudaError_t le =
      launch_early(paged_tc_kernel<D, kBytes>, dim3(kCtas), Warps<kBytes>::kThreads, bytes, s, p);
  after_launch(kKernPaged, s);
  return le;
}
template <int D>
cudaError_t tc_pages(const PagedArgs& a, cudaStream_t s) {
  return a.Ks ? tc_launch<D, true>(a, s) : tc_launch<D, false>(a, s);
}

}  // namespace

// Pages of at least 8 rows (a swizzle atom), pool rows within TMA's 32-bit
// coordinates, a scale whose sign keeps the maximum a maximum.
bool paged_tc_supported(const PagedArgs& a) {
  return a.dtype == kBF16 && paged_mma_shape(a.d, a.v) && a.lps >= 3 && a.sl2 > 0.f &&
         ((static_cast<long long>(a.num_pages) * a.Hk) << a.lps) < (1ll << 31) && tmap_encoder() != nullptr;
}
PagedKernel paged_tc_kernel_of() { return {kRows, kCtas, kCtas, 1}; }

cudaError_t launch_paged_tc(const PagedArgs& a, cudaStream_t s) {
  return a.d <= 64 && a.v <= 64 ? tc_pages<64>(a, s) : tc_pages<128>(a, s);
}

}  // namespace exattn
