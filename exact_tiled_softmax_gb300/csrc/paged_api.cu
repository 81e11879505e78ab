// The C ABI of the paged-cache operators (include/exattn.h): argument checks,
// workspace layout and kernel dispatch.  No memory is allocated here.
#include <stdint.h>

#include <algorithm>

#include "../../include/exattn.h"
#include "paged.cuh"

namespace exattn {
extern thread_local char g_last_error[256];
int current_path();
}  // namespace exattn

namespace {

using namespace exattn;

constexpr int kMaxWidth = 256;
constexpr int kMaxTokens = 1 << 20;
constexpr int kMaxKeys = 1 << 30;
constexpr int kMaxPageSize = 1024;
constexpr long long kMaxRows = (1ll << 31) - 1024;  // a row and a tile more still count in an int

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int log2_of(int x) {
  int k = 0;
  while ((1 << k) < x) ++k;
  return k;
}

int check_paged(const exattn_paged_shape* s) {
  if (!s) return EXATTN_INVALID_ARG;
  if (s->batch < 1 || s->tokens < 1 || s->heads < 1 || s->kv_heads < 1 || s->d < 1 || s->v < 1 ||
      s->page_size < 1 || s->num_pages < 1 || s->max_pages < 1)
    return EXATTN_INVALID_ARG;
  if (s->dtype != EXATTN_F32 && s->dtype != EXATTN_BF16) return EXATTN_INVALID_ARG;
  if (s->heads % s->kv_heads != 0) return EXATTN_INVALID_ARG;
  const int per16 = s->dtype == EXATTN_BF16 ? 8 : 4;
  const long long qw = (long long)s->heads * s->d, kw = (long long)s->kv_heads * s->d,
                  vw = (long long)s->kv_heads * s->v;
  if ((s->q_stride != 0 && s->q_stride < qw) || (s->k_stride != 0 && s->k_stride < kw) ||
      (s->v_stride != 0 && s->v_stride < vw))
    return EXATTN_INVALID_ARG;
  if (s->d > kMaxWidth || s->v > kMaxWidth || s->d % per16 != 0 || s->v % per16 != 0)
    return EXATTN_UNSUPPORTED;
  if (s->q_stride % per16 != 0 || s->k_stride % per16 != 0 || s->v_stride % per16 != 0)
    return EXATTN_MISALIGNED;
  if (s->page_size > kMaxPageSize || (s->page_size & (s->page_size - 1)) != 0) return EXATTN_UNSUPPORTED;
  if (s->batch > kPagedMaxBatch || s->tokens > kMaxTokens || s->heads > 65535 ||
      (long long)s->tokens * s->heads > kMaxRows ||
      (long long)s->max_pages * s->page_size > kMaxKeys)
    return EXATTN_UNSUPPORTED;
  return EXATTN_OK;
}

// The kernel of a call.
enum Kind { kSimtOne, kSimt, kMma8, kMma16, kTc };

PagedKernel kernel_of(Kind k, int dtype, int d, int v) {
  switch (k) {
    case kTc: return paged_tc_kernel_of();
    case kMma8: return paged_mma_kernel_of(dtype, d, v, 8);
    case kMma16: return paged_mma_kernel_of(dtype, d, v, 16);
    default: return paged_simt_kernel(k == kSimtOne);
  }
}

struct Choice {
  Kind kind;
  PagedKernel k;
};

// Rows of a key head on average: all that the host knows of them.
long long rows_of(const PagedArgs& a) { return (long long)(a.T + a.B - 1) / a.B * a.G; }
// From 17 rows on a second 16-row tile would read K and V again; the 256-row tiles read them
// once.  32 sequences of 8192 keys, 8 key heads of 128 columns: 16 rows 183 us (186 on the
// tall tiles), 24 rows 331 (190), 64 rows 644 (194); 4 of 4000: 16 rows 31 (31), 32 rows 42 (27).
constexpr int kTcRows = 16;

Choice choose(const PagedArgs& a) {
  Choice c;
  if (current_path() != EXATTN_PATH_SIMT && paged_mma_shape(a.d, a.v))
    c.kind = rows_of(a) > kTcRows && paged_tc_supported(a) ? kTc : rows_of(a) > 8 ? kMma16 : kMma8;
  else c.kind = !a.starts && a.T == a.B && a.G == 1 ? kSimtOne : kSimt;
  c.k = kernel_of(c.kind, a.dtype, a.d, a.v);
  return c;
}

// Workspace of one attention launch and its merge: tile descriptions | m | l | z of the
// runs' slots.
size_t pass_bytes(const PagedKernel& k, int v) {
  const size_t rows = 2 * (size_t)k.workers * k.rt;
  return align256(sizeof(int4) * (size_t)k.workers) + 2 * align256(sizeof(float) * rows) +
         align256(sizeof(float) * rows * v);
}
constexpr size_t kFlagBytes = 8192;  // status bits of the CTAs of two passes (at most 2048)

// The most that any kernel of this shape needs (the path may change between the query and
// the call, and q_starts is not part of the shape).
size_t most_bytes(const exattn_paged_shape* s) {
  size_t most = 0;
  for (const Kind k : {kSimtOne, kSimt, kMma8, kMma16, kTc}) {
    if (k >= kMma8 && !paged_mma_shape(s->d, s->v)) continue;
    // A prefix's pass takes all tokens as one sequence's.
    if (k == kTc && (s->dtype != EXATTN_BF16 || (long long)s->tokens * (s->heads / s->kv_heads) <= kTcRows)) continue;
    const size_t x = pass_bytes(kernel_of(k, s->dtype, s->d, s->v), s->v);
    most = x > most ? x : most;
  }
  return most;
}

// With a shared prefix: both sets' rows and statistics, where each stands, a word.
size_t join_bytes(size_t rows, int v) {
  return align256(sizeof(float) * 2 * rows * v) + align256(sizeof(float) * 2 * rows) +
         align256(sizeof(int2) * 2 * rows) + 256;
}

// The most units that the tables can hold (paged_mma_kernel's, of 16 keys).
long long most_units(const PagedArgs& a, int rt) {
  const long long rows = (long long)a.T * a.G, own = a.prefix_at < 0 ? a.B : a.B - 1;
  long long keys = ((long long)a.max_pages << a.lps) + 16;
  if (a.mask_kind == EXATTN_MASK_WINDOW) keys = std::min(keys, (long long)a.window + rt + 32);
  const long long tiles = a.starts ? rows / rt + own : own * (((long long)a.each * a.G + rt - 1) / rt);
  long long units = own > 0 ? tiles * (keys / 16) : 0;
  if (a.prefix_at >= 0) units += (rows + rt - 1) / rt * ((a.prefix_len + 15ll) / 16);
  return units * a.Hk;
}

void place_pass(PagedArgs& a, const PagedKernel& k, char* at) {
  a.runs = k.workers;
  a.by_runs = fast_div(k.workers);
  // Where two units a worker are all there can be, tiles are rounded up to no more: 2 sequences of
  // 600 keys behind 162, 8 key heads of 80 and 96 fp32 columns 14.4 us in place of 18.2, 5 tokens over
  // 7382 keys of one head of 112 columns 17.0 of 20.9.  (2 for 3 to 5 units a worker: 30.3 in
  // place of 25.9, 17.6 of 15.9.)
  a.least = k.least > 2 && most_units(a, k.rt) <= 2ll * k.workers ? 2 : k.least;
  const size_t rows = 2 * (size_t)a.runs * k.rt;
  a.desc = reinterpret_cast<int4*>(at);
  at += align256(sizeof(int4) * (size_t)a.runs);
  a.pm = reinterpret_cast<float*>(at);
  at += align256(sizeof(float) * rows);
  a.pl = reinterpret_cast<float*>(at);
  at += align256(sizeof(float) * rows);
  a.pz = reinterpret_cast<float*>(at);
}

PagedArgs make_args(const exattn_paged_shape* s, const void* Q, const void* Kp, const void* Vp,
                    const int* table, const int* lens, const int* starts, float scale, int mask_kind,
                    int window, void* Y, float* L) {
  PagedArgs a{};
  a.Q = Q;
  a.Kp = Kp;
  a.Vp = Vp;
  a.table = table;
  a.lens = lens;
  a.starts = starts;
  a.B = s->batch;
  a.T = s->tokens;
  a.Hk = s->kv_heads;
  a.G = s->heads / s->kv_heads;
  a.by_group = fast_div(a.G);
  a.by_heads = fast_div(a.Hk);
  a.each = a.T / a.B;
  a.prefix_at = -1;
  a.d = s->d;
  a.v = s->v;
  a.dtype = s->dtype;
  a.lps = log2_of(s->page_size);
  a.num_pages = s->num_pages;
  a.max_pages = s->max_pages;
  a.mask_kind = mask_kind;
  a.window = mask_kind == EXATTN_MASK_WINDOW ? (window < kMaxKeys ? window : kMaxKeys) : 0;
  a.sl2 = scale * kLog2e;
  a.q_stride = s->q_stride ? s->q_stride : (long long)s->heads * s->d;
  a.Y = Y;
  a.L = L;
  return a;
}

int cuda_result(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return EXATTN_OK;
  record_error(where, static_cast<int>(e), cudaGetErrorString(e));
  return EXATTN_CUDA_ERROR;
}

cudaError_t run_kernel(const PagedArgs& a, const Choice& c, cudaStream_t s) {
  return c.kind == kTc     ? launch_paged_tc(a, s)
         : c.kind >= kMma8 ? launch_paged_mma(a, c.k.rt, s)
                           : launch_paged_simt(a, c.kind == kSimtOne, s);
}

int check_call(const exattn_paged_shape* shape, const void* Q, const void* Kp, const void* Vp,
               const int* table, const int* lens, const int* starts, int mask_kind, int window,
               const void* Y, const void* L, const void* workspace) {
  if (mask_kind < EXATTN_MASK_NONE || mask_kind > EXATTN_MASK_BITMASK) return EXATTN_INVALID_ARG;
  if (mask_kind == EXATTN_MASK_BITMASK) return EXATTN_UNSUPPORTED;
  if (mask_kind == EXATTN_MASK_WINDOW && window < 1) return EXATTN_INVALID_ARG;
  if (!Q || !Kp || !Vp || !table || !lens || !Y || !L || !workspace) return EXATTN_INVALID_ARG;
  if (!starts && shape->tokens % shape->batch != 0) return EXATTN_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(Kp, 16) || !aligned(Vp, 16) || !aligned(Y, 16) || !aligned(L, 16) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(starts, 4) || !aligned(workspace, 256))
    return EXATTN_MISALIGNED;
  return EXATTN_OK;
}

}  // namespace

extern "C" {

size_t exattn_paged_workspace_size(const exattn_paged_shape* shape) {
  if (check_paged(shape) != EXATTN_OK) return 0;
  return kStatusBytes + kFlagBytes + most_bytes(shape);
}

size_t exattn_prefix_workspace_size(const exattn_paged_shape* shape) {
  if (check_paged(shape) != EXATTN_OK) return 0;
  const size_t rows = (size_t)shape->tokens * shape->heads;
  return kStatusBytes + kFlagBytes + 2 * most_bytes(shape) + join_bytes(rows, shape->v);
}

int attn_append_paged(const exattn_paged_shape* shape, const void* q, const void* k, const void* v,
                      const int* page_table, const int* seq_lens, const int* q_starts,
                      const float* inv_freq, int rot_pairs, int interleaved, int pos_offset,
                      void* q_out, void* k_pages, void* v_pages, void* workspace,
                      size_t workspace_bytes, void* cuda_stream) {
  const int st = check_paged(shape);
  if (st != EXATTN_OK) return st;
  if (!k || !v || !page_table || !seq_lens || !k_pages || !v_pages || !workspace || (q && !q_out) ||
      (rot_pairs > 0 && !inv_freq) || rot_pairs < 0 || 2 * (long long)rot_pairs > shape->d ||
      pos_offset < 0)
    return EXATTN_INVALID_ARG;
  if (!q_starts && shape->tokens % shape->batch != 0) return EXATTN_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(page_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(q_starts, 4) || !aligned(inv_freq, 4) || !aligned(workspace, 256))
    return EXATTN_MISALIGNED;
  if (workspace_bytes < kStatusBytes) return EXATTN_WORKSPACE_TOO_SMALL;
  g_last_error[0] = 0;
  AppendArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.starts = q_starts;
  a.table = page_table;
  a.lens = seq_lens;
  a.inv_freq = inv_freq;
  a.pairs = rot_pairs;
  a.interleaved = interleaved != 0;
  a.pos_offset = pos_offset;
  a.B = shape->batch;
  a.T = shape->tokens;
  a.H = shape->heads;
  a.Hk = shape->kv_heads;
  a.d = shape->d;
  a.vw = shape->v;
  a.dtype = shape->dtype;
  a.lps = log2_of(shape->page_size);
  a.num_pages = shape->num_pages;
  a.max_pages = shape->max_pages;
  a.qs = shape->q_stride ? shape->q_stride : (long long)shape->heads * shape->d;
  a.ks = shape->k_stride ? shape->k_stride : (long long)shape->kv_heads * shape->d;
  a.vs = shape->v_stride ? shape->v_stride : (long long)shape->kv_heads * shape->v;
  a.q_out = q_out;
  a.kp = k_pages;
  a.vp = v_pages;
  a.status = static_cast<unsigned*>(workspace);
  return cuda_result(launch_append(a, static_cast<cudaStream_t>(cuda_stream)),
                     "attn_append_paged: launch");
}

int attn_fwd_paged(const exattn_paged_shape* shape, const void* Q, const void* k_pages,
                   const void* v_pages, const int* page_table, const int* seq_lens,
                   const int* q_starts, float scale, int mask_kind, int window, void* Y, float* L,
                   void* workspace, size_t workspace_bytes, void* cuda_stream) {
  int st = check_paged(shape);
  if (st != EXATTN_OK) return st;
  st = check_call(shape, Q, k_pages, v_pages, page_table, seq_lens, q_starts, mask_kind, window, Y, L,
                  workspace);
  if (st != EXATTN_OK) return st;
  if (workspace_bytes < exattn_paged_workspace_size(shape)) return EXATTN_WORKSPACE_TOO_SMALL;
  g_last_error[0] = 0;
  char* ws = static_cast<char*>(workspace);
  PagedArgs a = make_args(shape, Q, k_pages, v_pages, page_table, seq_lens, q_starts, scale, mask_kind,
                          window, Y, L);
  const Choice c = choose(a);
  a.status = static_cast<unsigned*>(workspace);
  a.flags = reinterpret_cast<unsigned*>(ws + kStatusBytes);
  a.flags0 = a.flags;
  a.n_flags = c.k.ctas;
  place_pass(a, c.k, ws + kStatusBytes + kFlagBytes);
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = run_kernel(a, c, s);
  if (e == cudaSuccess) e = launch_paged_merge(a, c.k.rt, s);
  return cuda_result(e, "attn_fwd_paged: launch");
}

int attn_fwd_prefix(const exattn_paged_shape* shape, const void* Q, const void* k_pages,
                    const void* v_pages, const int* prefix_table, int prefix_len,
                    const int* page_table, const int* seq_lens, const int* q_starts, float scale,
                    int mask_kind, void* Y, float* L, void* workspace, size_t workspace_bytes,
                    void* cuda_stream) {
  int st = check_paged(shape);
  if (st != EXATTN_OK) return st;
  if (mask_kind == EXATTN_MASK_WINDOW) return EXATTN_UNSUPPORTED;
  st = check_call(shape, Q, k_pages, v_pages, page_table, seq_lens, q_starts, mask_kind, 0, Y, L,
                  workspace);
  if (st != EXATTN_OK) return st;
  if (prefix_len < 0 || (prefix_len > 0 && !prefix_table)) return EXATTN_INVALID_ARG;
  if (prefix_len > kMaxKeys - kMaxPageSize) return EXATTN_UNSUPPORTED;
  if (!aligned(prefix_table, 4)) return EXATTN_MISALIGNED;
  if (workspace_bytes < exattn_prefix_workspace_size(shape)) return EXATTN_WORKSPACE_TOO_SMALL;
  if (prefix_len == 0)
    return attn_fwd_paged(shape, Q, k_pages, v_pages, page_table, seq_lens, q_starts, scale, mask_kind,
                          0, Y, L, workspace, workspace_bytes, cuda_stream);
  g_last_error[0] = 0;
  cudaStream_t s = static_cast<cudaStream_t>(cuda_stream);
  char* ws = static_cast<char*>(workspace);
  const size_t rows = (size_t)shape->tokens * shape->heads;
  char* area = ws + kStatusBytes + kFlagBytes;
  char* sets = area + 2 * most_bytes(shape);
  PagedArgs a = make_args(shape, Q, k_pages, v_pages, page_table, seq_lens, q_starts, scale, mask_kind, 0, Y, L);
  a.Yf = reinterpret_cast<float*>(sets);
  a.L = reinterpret_cast<float*>(sets + align256(sizeof(float) * 2 * rows * a.v));
  a.info = reinterpret_cast<int2*>(reinterpret_cast<char*>(a.L) + align256(sizeof(float) * 2 * rows));
  a.sane = reinterpret_cast<int*>(reinterpret_cast<char*>(a.info) + align256(sizeof(int2) * 2 * rows));
  a.Lout = L;
  a.prefix_table = prefix_table;
  a.prefix_len = prefix_len;
  a.flags = reinterpret_cast<unsigned*>(ws + kStatusBytes);
  a.flags0 = a.flags;
  // All tokens over the prefix are one sequence: of as many rows to a key head as the batch
  // has, which may ask for another kernel than the sequences' own.
  PagedArgs p = a;
  p.B = 1;
  p.each = p.T;
  p.starts = nullptr;
  p.prefix_at = 0;
  Choice own = choose(a), of = choose(p);
  if (own.kind != of.kind && of.kind == kTc && own.kind >= kMma8) {
    // Tall tiles for the prefix alone mean a launch of their own, 6 us; 16-row tiles read the
    // prefix again for each, at some 6.5 TB/s (of the L2 cache).
    const double bytes = (double)prefix_len * a.Hk * (a.d + a.v) * 2, again = (double)((rows_of(p) + 15) / 16 - 1);
    if (again * bytes < 40e6) {
      of.kind = kMma16;
      of.k = kernel_of(of.kind, a.dtype, a.d, a.v);
    }
  }
  const bool together = own.kind == of.kind || own.kind <= kSimt || (own.kind == kMma8 && of.kind == kMma16);
  int launches_ctas = 0;
  cudaError_t e;
  if (together) {
    // One launch over B + 1 sequences, with the larger tiles.
    own = of;
    ++a.B;
    a.prefix_at = a.B - 1;
    place_pass(a, own.k, area);
    launches_ctas = own.k.ctas;
    e = run_kernel(a, own, s);
    p = a;
  } else {
    place_pass(p, of.k, area);
    place_pass(a, own.k, area + most_bytes(shape));
    a.flags = p.flags + of.k.ctas;
    a.second = true;
    launches_ctas = of.k.ctas + own.k.ctas;
    e = run_kernel(p, of, s);
    if (e == cudaSuccess) e = run_kernel(a, own, s);
  }
  if (e != cudaSuccess) return cuda_result(e, "attn_fwd_prefix: launch");
  a.prefix_at = shape->batch;  // for the join: q_starts' last entry
  a.Y = Y;
  a.status = static_cast<unsigned*>(workspace);
  a.n_flags = launches_ctas;
  return cuda_result(launch_paged_join(a, own.k.rt, p, of.k.rt, s), "attn_fwd_prefix: join launch");
}

int exattn_paged_run(int op, const exattn_paged_call* c) {
  if (!c) return EXATTN_INVALID_ARG;
  switch (op) {
    case EXATTN_PAGED_APPEND:
      return attn_append_paged(&c->shape, c->q, c->k, c->v, c->page_table, c->seq_lens, c->q_starts,
                               c->inv_freq, c->rot_pairs, c->interleaved, c->prefix_len, c->y, c->k_pages,
                               c->v_pages, c->workspace, c->workspace_bytes, c->cuda_stream);
    case EXATTN_PAGED_FWD:
      return attn_fwd_paged(&c->shape, c->q, c->k_pages, c->v_pages, c->page_table, c->seq_lens, c->q_starts,
                            c->scale, c->mask_kind, c->window, c->y, c->L, c->workspace, c->workspace_bytes,
                            c->cuda_stream);
    case EXATTN_PAGED_PREFIX:
      return attn_fwd_prefix(&c->shape, c->q, c->k_pages, c->v_pages, c->prefix_table, c->prefix_len,
                             c->page_table, c->seq_lens, c->q_starts, c->scale, c->mask_kind, c->y, c->L,
                             c->workspace, c->workspace_bytes, c->cuda_stream);
    default: return EXATTN_INVALID_ARG;
  }
}

}  // extern "C"
