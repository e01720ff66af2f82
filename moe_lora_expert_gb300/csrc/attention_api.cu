// C ABI of the attention half: argument checks of moe_rope, moe_kv_append and
// moe_paged_attention, and the choice of the width of their accesses.
#include <cstddef>

#include "attention.cuh"

namespace {

using moe::AttentionForms;
using moe::AttentionParams;
using moe::KvAppendParams;
using moe::RopeAxes;
using moe::RopeParams;
using moe::RopeTensor;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int done(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }
inline int element_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

// Which attention kernel: rows a key head has (new tokens x query heads of its
// group) and how many (sequence, key head) pairs there are.  The kernel for
// few rows reads the cache once for every 16 rows; the other one does 256 rows
// at the price of 128 and needs some pairs to fill its CTAs.  Both measured on
// 4 key heads (4 or 8 query heads each: the same times), few / many in us:
//   heads of 128: 16 sequences of 2048 keys: 16 rows 26 / 37, 32 rows 33 / 37, 48 rows 41 / 37;
//     8 of 16384: 16 rows 52 / 78, 32 rows 79 / 78;  1 of 32768: 64 rows 49 / 53, 96 rows 64 / 53;
//     1 of 2048: 96 rows 23 / 30, 192 rows 23 / 33;
//   heads of 64: 16 of 2048: 32 rows 29 / 30, 48 rows 36 / 30;  8 of 16384: 16 rows 43 / 64, 32 rows 67 / 64;
//     1 of 32768: 32 rows 31 / 38, 64 rows 43 / 38, 96 rows 56 / 38;  1 of 2048: 96 rows 20 / 24.
// So 32 rows are where the sides cross for many pairs.  For few pairs it is
// between 32 and over 192, later the shorter the contexts, whose lengths the
// host does not have: 96 saves 15 to 25% on a short one and costs up to 46% on
// one long context (on 8 key heads 77%: 109 / 62).
bool few_rows(int64_t rows, int64_t pairs) { return rows <= 32 || (rows <= 96 && pairs <= 16); }

// Whether prefixes are read once for their groups, by what the host has: the
// sequences, the groups, a bound on the tokens of the largest, and a bound on the
// lengths.  The call has three kernels then.  Outside a graph it takes the host 26
// to 30 us, so it pays only where the plain call takes the GPU longer: where the
// plain call's passes over the cache are 80 MB, which is 12 us of it.  And a unit
// (256 rows of a group and key head) takes a key tile 2 us of an SM, however few
// its rows are, which the plain call's reading for them has to outweigh.
// Shared / plain, us a call outside graphs (query heads of 128, 8 to a key head; in
// graphs plain calls take 0.8 less, shared ones 1 to 12):
//   4 key heads, one group, of 4 sequences: 8192 shared tokens 26.3 / 23.2, 16384 25.6 / 28.4, 65536 45.5 / 57.2;
//     of 8: 4096 26.1 / 21.4, 8192 26.5 / 26.0, 16384 27.6 / 34.9;  of 16: 4096 26.9 / 25.3, 8192 27.4 / 34.8, 65536 52 / 165;
//   1 key head, 8 sequences: 16384 28.2 / 23.6, 65536 29.8 / 37.0;  8 key heads: 4096 29.1 / 25.9, 8192 29.0 / 34.5;
//   4 key heads, groups of 2 (16 rows): 4 of 16384 38.9 / 37.9, 65536 107 / 85;  16 of 4096 61.9 / 33.2, 65536 545 / 254;
//   groups of 4 (32 rows): 4 of 4096 27.0 / 24.3, 8192 31.0 / 31.2, 16384 41.8 / 46.9;  8 of 8192 48.5 / 47.7, 65536 223 / 257;
//     16 of 16384 166 / 138, 65536 548 / 487;
//   groups of 8 (64 rows): 8 of 1024 29.7 / 25.8, 4096 40.0 / 48.1;  16 of 2048 55 / 53, 4096 82 / 83, 8192 134 / 142;
//     40 of 4096 161 / 178;  groups of 16: 16 of 2048 92 / 86, 4096 92 / 146;
//   heads of 64: 8 sequences 8192 29.7 / 23.3, 16384 29.5 / 31.3;  4 groups of 4: 8192 29.6 / 27.6, 16384 36.9 / 39.6;
//   16 sequences of 4 new tokens: 1024 30.3 / 25.8, 4096 29.7 / 41.4;  of 8: 1024 36 / 32, 4096 38 / 53;  of 16: 4096 66 / 53, 16384 109 / 125.
// Sequences of many rows fill the products' tiles by themselves, and their own
// keys are then in the kernel that is made for few.  A list of groups may be
// uneven, so with few units the bound on the largest counts and not the mean (4
// groups of 2 or 3 sequences, 5 query heads on each of 2 key heads, and no bound: 65536 63 / 54).
bool pays(const AttentionParams& p, int groups, int max_tokens) {
  const int64_t heads = p.Hq / p.cache.kv_heads, rows = p.max_q_len * heads, longest = p.max_seq_len;
  const int64_t mean_rows = (p.N + groups - 1ll) / groups * heads, units = groups * ((mean_rows + 255) / 256) * p.cache.kv_heads;
  if (max_tokens * heads < 32 || (mean_rows < 32 && units > 8) || (mean_rows < 64 && units > 32)) return false;
  if (rows > 128 || (rows > 32 && rows * rows > longest) || longest < 4096) return false;
  const double plain_bytes = 2.0 * p.cache.head_dim * static_cast<double>(longest) * static_cast<double>((rows + 15) / 16 * p.B * p.cache.kv_heads);
  return plain_bytes >= 80e6 && plain_bytes >= 8.4e6 * static_cast<double>(units);
}
// How many pieces the prefix pass may leave for a row: with one group whose
// rows fill 256-row units, twice as many as give each SM one of them, and no more
// than give each SM one of a unit that every key head has.  8 sequences with 8
// query heads a key head, 32 pieces and so many, in us: 1 key head, 65536 shared
// tokens 40.9 / 28.6, 131072 68.8 / 38.8; 2 key heads 42.6 / 34.7, 73.5 / 47.2.
// What a caller allocates who names no key heads holds 32.
constexpr int kPieces = 32;
int most_pieces(int N, int Hq, int kv_heads) {
  const int64_t rows = static_cast<int64_t>(N) * Hq, n = 2ll * 160 * 256 / rows;
  const int most = kv_heads > 0 && kv_heads < 5 ? 160 / kv_heads : kPieces;
  return n < 2 ? 2 : n > most ? most : static_cast<int>(n);
}

size_t partial_bytes(int pieces, int64_t rows, int head_dim, int groups) {
  return (pieces + 1) * static_cast<size_t>(rows) * (static_cast<size_t>(head_dim) * 4 + 8) + static_cast<size_t>(groups) * 4;
}

// Elements a thread may move at once, of 8, 4 and 1: V elements of a type
// with e bytes need addresses and strides in multiples of V * e bytes (16 at
// most), and the rotated part and the rest whole stretches.
int widest(int V, int e, int D, int R, const RopeTensor& x, int V_so_far) {
  if (x.heads == 0) return V_so_far;
  for (; V > 1; V /= 2) {
    const int bytes = V * e < 16 ? V * e : 16, n = bytes / e;
    if (D % (2 * V) == 0 && (R / 2) % V == 0 && R % (2 * V) == 0 && aligned(x.in, bytes) && aligned(x.out, bytes) &&
        x.in_token % n == 0 && x.in_head % n == 0 && x.out_token % n == 0 && x.out_head % n == 0)
      break;
  }
  if (V == 2) V = 1;
  return V < V_so_far ? V : V_so_far;
}

int check_cache(const moe_kv_cache_t& c) {
  if (c.num_pages < 0 || c.kv_heads <= 0 || c.page_size <= 0 || c.head_dim <= 0) return MOE_ERR_SHAPE;
  if (c.head_dim % 16 != 0 || c.head_dim > 128 || c.page_size % 8 != 0 || c.page_size > 256 || c.kv_heads > 1024)
    return MOE_ERR_UNSUPPORTED;
  if (c.k == nullptr || c.v == nullptr || c.k_scale == nullptr || c.v_scale == nullptr) return MOE_ERR_NULL;
  const int64_t strides[6] = {c.k_stride_page, c.k_stride_head, c.k_stride_token,
                              c.v_stride_page, c.v_stride_head, c.v_stride_token};
  for (int64_t s : strides) {
    if (s < 0) return MOE_ERR_SHAPE;
    if (s % 16 != 0) return MOE_ERR_ALIGN;
  }
  if (!aligned(c.k, 16) || !aligned(c.v, 16) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)) return MOE_ERR_ALIGN;
  return MOE_OK;
}

// The part of the arguments that says which tokens belong to which sequence.
int check_batch(int N, int B, int table_width, int max_q_len, const int32_t* table, const int32_t* lens,
                const int32_t* cu_q) {
  if (N < 0 || B < 0 || table_width < 0 || max_q_len < 0) return MOE_ERR_SHAPE;
  if (cu_q == nullptr && N != B) return MOE_ERR_SHAPE;
  if (N > 0 && B > 0 && (lens == nullptr || (table == nullptr && table_width > 0))) return MOE_ERR_NULL;
  return MOE_OK;
}

// The axes of a rotation's pairs, two bits each.
int pack_axes(const moe_rope_axes_t* x, int rotary_dim, RopeAxes* to) {
  if (x == nullptr) return MOE_ERR_NULL;
  if (x->struct_size != sizeof(*x)) return MOE_ERR_UNSUPPORTED;
  if (x->num_axes < 1 || x->positions_stride < 0 || rotary_dim < 2) return MOE_ERR_SHAPE;
  if (x->num_axes > moe::kMaxAxes || rotary_dim > 2 * moe::kMaxPairs) return MOE_ERR_UNSUPPORTED;
  *to = RopeAxes{};
  to->stride = x->positions_stride;
  to->count = x->num_axes;
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (x->axis_of_pair[i] >= x->num_axes) return MOE_ERR_SHAPE;
    to->of_pair[i / 16] |= static_cast<uint32_t>(x->axis_of_pair[i]) << (2 * (i % 16));
  }
  return MOE_OK;
}

int rope(const moe_rope_args_t* a, bool with_axes, const moe_rope_axes_t* x, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_NULL;
  if (a->struct_size != sizeof(*a)) return MOE_ERR_UNSUPPORTED;
  if (a->dtype < MOE_DTYPE_BF16 || a->dtype > MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (a->N < 0 || a->Hq < 0 || a->Hk < 0 || a->D <= 0 || a->rotary_dim < 2 || a->rotary_dim > a->D ||
      a->rotary_dim % 2 != 0 || a->D % 2 != 0 || a->num_positions < 0)
    return MOE_ERR_SHAPE;
  RopeAxes axes;
  if (with_axes) {
    const int st = pack_axes(x, a->rotary_dim, &axes);
    if (st != MOE_OK) return st;
  }
  if (a->D > 1024 || a->Hq + static_cast<int64_t>(a->Hk) > 65536 ||
      a->N * (a->Hq + static_cast<int64_t>(a->Hk)) * (a->D / 2) > (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  if (a->N == 0 || a->Hq + a->Hk == 0) return MOE_OK;
  if ((a->Hq > 0 && (a->q == nullptr || a->q_out == nullptr)) || (a->Hk > 0 && (a->k == nullptr || a->k_out == nullptr)) ||
      a->positions == nullptr || (a->cos_sin == nullptr && a->num_positions > 0))
    return MOE_ERR_NULL;
  if (!aligned(a->cos_sin, 16)) return MOE_ERR_ALIGN;
  RopeParams p = {};
  p.q = {a->q, a->q_out, a->q_stride_token, a->q_stride_head, a->q_out_stride_token, a->q_out_stride_head, a->Hq};
  p.k = {a->k, a->k_out, a->k_stride_token, a->k_stride_head, a->k_out_stride_token, a->k_out_stride_head, a->Hk};
  p.positions = a->positions;
  p.cos_sin = a->cos_sin;
  p.status = a->status;
  p.N = a->N, p.D = a->D, p.R = a->rotary_dim, p.num_positions = a->num_positions;
  p.interleaved = a->interleaved != 0, p.inverse = a->inverse != 0;
  const int e = element_bytes(a->dtype), most = e == 4 ? 4 : 8;
  int V = widest(most, e, p.D, p.R, p.q, most);
  V = widest(most, e, p.D, p.R, p.k, V);
  (void)cudaGetLastError();
  return done(moe::launch_rope(p, with_axes ? &axes : nullptr, a->dtype, V, reinterpret_cast<cudaStream_t>(stream)));
}

int kv_append(const moe_kv_append_args_t* a, bool with_axes, const moe_rope_axes_t* x, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_NULL;
  if (a->struct_size != sizeof(*a)) return MOE_ERR_UNSUPPORTED;
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
  int st = check_cache(a->cache);
  if (st != MOE_OK) return st;
  st = check_batch(a->N, a->B, a->table_width, a->max_q_len, a->block_table, a->seq_lens, a->cu_q);
  if (st != MOE_OK) return st;
  const moe_kv_cache_t& c = a->cache;
  if (a->Hq < 0 || a->rotary_dim < 0 || a->rotary_dim > c.head_dim || a->rotary_dim % 2 != 0 || a->num_positions < 0)
    return MOE_ERR_SHAPE;
  if ((a->cos_sin == nullptr) != (a->rotary_dim == 0)) return MOE_ERR_NULL;
  RopeAxes axes;
  if (with_axes) {
    st = pack_axes(x, a->rotary_dim, &axes);
    if (st != MOE_OK) return st;
  }
  if (!aligned(a->cos_sin, 16)) return MOE_ERR_ALIGN;
  if (a->Hq > 65536) return MOE_ERR_UNSUPPORTED;
  if (a->N == 0 || a->B == 0 || a->max_q_len == 0) return MOE_OK;
  if (with_axes && a->positions == nullptr) return MOE_ERR_NULL;
  if (a->k == nullptr || a->v == nullptr || (a->Hq > 0 && (a->q == nullptr || a->q_out == nullptr))) return MOE_ERR_NULL;
  KvAppendParams p = {};
  p.cache = c;
  p.k = a->k, p.v = a->v;
  p.k_token = a->k_stride_token, p.k_head = a->k_stride_head, p.v_token = a->v_stride_token, p.v_head = a->v_stride_head;
  p.q = {a->q, a->q_out, a->q_stride_token, a->q_stride_head, a->q_out_stride_token, a->q_out_stride_head, a->Hq};
  p.block_table = a->block_table, p.seq_lens = a->seq_lens, p.cu_q = a->cu_q, p.positions = a->positions;
  p.cos_sin = a->cos_sin;
  p.status = a->status;
  p.N = a->N, p.B = a->B, p.table_width = a->table_width, p.R = a->rotary_dim, p.num_positions = a->num_positions;
  p.interleaved = a->interleaved != 0;
  const int longest = a->cu_q == nullptr ? 1 : a->max_q_len < a->N ? a->max_q_len : a->N;
  p.max_q_len = longest;
  p.slots = (longest + c.page_size - 2) / c.page_size + 1;
  if (2ll * p.B * p.slots * c.kv_heads > (1ll << 30) || static_cast<int64_t>(a->N) * a->Hq * (c.head_dim / 2) > (1ll << 31))
    return MOE_ERR_UNSUPPORTED;
  const RopeTensor k = {a->k, nullptr, a->k_stride_token, a->k_stride_head, 0, 0, c.kv_heads};
  const RopeTensor v = {a->v, nullptr, a->v_stride_token, a->v_stride_head, 0, 0, c.kv_heads};
  int V = widest(8, 2, c.head_dim, p.R, k, 8);
  V = widest(8, 2, c.head_dim, 0, v, V);
  V = widest(8, 2, c.head_dim, p.R, p.q, V);
  (void)cudaGetLastError();
  return done(moe::launch_kv_append(p, with_axes ? &axes : nullptr, a->dtype, V, reinterpret_cast<cudaStream_t>(stream)));
}

// The arguments of a call, checked; MOE_OK with p.N = 0 where there is nothing to do.
int check_attention(const moe_paged_attention_args_t* a, AttentionParams& p) {
  if (a == nullptr) return MOE_ERR_NULL;
  if (a->struct_size != sizeof(*a)) return MOE_ERR_UNSUPPORTED;
  if (a->dtype != MOE_DTYPE_BF16 && a->dtype != MOE_DTYPE_F16) return MOE_ERR_UNSUPPORTED;
  int st = check_cache(a->cache);
  if (st != MOE_OK) return st;
  st = check_batch(a->N, a->B, a->table_width, a->max_q_len, a->block_table, a->seq_lens, a->cu_q);
  if (st != MOE_OK) return st;
  const moe_kv_cache_t& c = a->cache;
  if (a->Hq <= 0 || a->Hq % c.kv_heads != 0 || a->max_seq_len < 0 || a->window < 0 || a->wait_timeout_ms < 0)
    return MOE_ERR_SHAPE;
  if (a->Hq / c.kv_heads > 256 || (a->debug_flags & ~MOE_DEBUG_STALL_ATTENTION) != 0) return MOE_ERR_UNSUPPORTED;
  p.N = 0;
  if (a->N == 0 || a->B == 0 || a->max_q_len == 0) return MOE_OK;
  if (a->q == nullptr || a->out == nullptr) return MOE_ERR_NULL;
  const int64_t strides[4] = {a->q_stride_token, a->q_stride_head, a->out_stride_token, a->out_stride_head};
  for (int64_t s : strides)
    if (s % 8 != 0) return MOE_ERR_ALIGN;
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return MOE_ERR_ALIGN;
  if (a->workspace == nullptr || !aligned(a->workspace, 256) || a->workspace_bytes < moe_paged_attention_workspace_size())
    return MOE_ERR_WORKSPACE;
  p = AttentionParams{};
  p.cache = c;
  p.q = a->q, p.out = a->out, p.lse = a->lse;
  p.q_token = a->q_stride_token, p.q_head = a->q_stride_head;
  p.out_token = a->out_stride_token, p.out_head = a->out_stride_head;
  p.block_table = a->block_table, p.seq_lens = a->seq_lens, p.cu_q = a->cu_q;
  p.status = a->status;
  p.N = a->N, p.B = a->B, p.Hq = a->Hq, p.table_width = a->table_width;
  p.max_q_len = a->cu_q == nullptr ? 1 : a->max_q_len < a->N ? a->max_q_len : a->N;
  // A window past any position is cut so that a row before the first key may take it from its position.
  const int most_window = 0x7fffffff - (a->N < 1 << 30 ? a->N : 1 << 30);
  p.window = a->window < most_window ? a->window : most_window;
  p.max_seq_len = a->max_seq_len;
  p.scale = a->scale;
  p.workspace = a->workspace;
  p.wait_limit_ns = 1000000ull * static_cast<uint64_t>(a->wait_timeout_ms > 0 ? a->wait_timeout_ms : 2000);
  p.debug_flags = a->debug_flags;
  return MOE_OK;
}

int64_t rows_of(const AttentionParams& p) { return static_cast<int64_t>(p.max_q_len) * (p.Hq / p.cache.kv_heads); }
int attend(const AttentionParams& p, const AttentionForms* forms, int dtype, cudaStream_t on) {
  if (few_rows(rows_of(p), static_cast<int64_t>(p.B) * p.cache.kv_heads)) return moe::launch_decode_attention(p, forms, dtype, on);
  return moe::launch_prefill_attention(p, forms, dtype, on);
}

int check_shared(const moe_paged_attention_args_t* a, const moe_shared_prefix_t* x) {
  if (x == nullptr) return MOE_ERR_NULL;
  if (x->struct_size != sizeof(*x)) return MOE_ERR_UNSUPPORTED;
  if (x->groups < 0 || x->max_tokens < 0) return MOE_ERR_SHAPE;
  return a->window != 0 ? MOE_ERR_UNSUPPORTED : MOE_OK;   // with a window its rows would see different parts of a prefix
}

// Whether a call's prefixes are read for their groups, and then what the prefix
// pass is given; else the call is the plain one.  All three kernels have to take
// it, which is known before the first is launched.
bool shares(const AttentionParams& p, const moe_shared_prefix_t* x, AttentionParams& prefix) {
  if (p.N == 0 || x->groups == 0 || x->max_tokens == 0) return false;
  prefix = p;
  prefix.B = x->groups;
  prefix.max_q_len = x->max_tokens < p.N ? x->max_tokens : p.N;
  return pays(p, x->groups, prefix.max_q_len) && moe::prefill_attention_fits(prefix) && moe::decode_attention_fits(p) &&
         moe::shared_join_fits(p);
}

}  // namespace

extern "C" {

int moe_rope(const moe_rope_args_t* a, moe_stream_t stream) { return rope(a, false, nullptr, stream); }
int moe_rope_axes(const moe_rope_args_t* a, const moe_rope_axes_t* axes, moe_stream_t stream) { return rope(a, true, axes, stream); }
int moe_kv_append(const moe_kv_append_args_t* a, moe_stream_t stream) { return kv_append(a, false, nullptr, stream); }
int moe_kv_append_axes(const moe_kv_append_args_t* a, const moe_rope_axes_t* axes, moe_stream_t stream) { return kv_append(a, true, axes, stream); }

size_t moe_paged_attention_workspace_size(void) { return moe::decode_attention_workspace_bytes() + moe::prefill_attention_workspace_bytes(); }

int moe_paged_attention_workspace_init(void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < moe_paged_attention_workspace_size())
    return MOE_ERR_WORKSPACE;
  (void)cudaGetLastError();
  const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = moe::clear_decode_counters(workspace, on);
  return done(e != cudaSuccess ? e : moe::clear_prefill_counters(workspace, on));
}

int moe_stream_capture_id(moe_stream_t stream, uint64_t* id) {
  if (id == nullptr) return MOE_ERR_NULL;
  *id = 0;
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  unsigned long long capture = 0;
  if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(stream), &status, &capture) != cudaSuccess) return MOE_ERR_CUDA;
  if (status == cudaStreamCaptureStatusActive) *id = capture;
  return MOE_OK;
}

int moe_paged_attention(const moe_paged_attention_args_t* a, moe_stream_t stream) {
  AttentionParams p;
  const int st = check_attention(a, p);
  if (st != MOE_OK || p.N == 0) return st;
  (void)cudaGetLastError();
  return attend(p, nullptr, a->dtype, reinterpret_cast<cudaStream_t>(stream));
}

int moe_paged_attention_sinks(const moe_paged_attention_args_t* a, int sinks, moe_stream_t stream) {
  AttentionParams p;
  const int st = check_attention(a, p);
  if (st != MOE_OK) return st;
  if (sinks < 0) return MOE_ERR_SHAPE;
  if (p.N == 0) return MOE_OK;
  (void)cudaGetLastError();
  AttentionForms f = {};
  f.sinks = sinks < (1 << 30) ? sinks : 1 << 30;
  return attend(p, sinks == 0 || p.window == 0 ? nullptr : &f, a->dtype, reinterpret_cast<cudaStream_t>(stream));
}

size_t moe_shared_prefix_partial_size(int N, int Hq, int head_dim, int groups) {
  if (N <= 0 || Hq <= 0 || head_dim <= 0 || groups <= 0) return 0;
  return partial_bytes(most_pieces(N, Hq, 0), static_cast<int64_t>(N) * Hq, head_dim, groups);
}

size_t moe_paged_attention_shared_partial_size(const moe_paged_attention_args_t* a, const moe_shared_prefix_t* x) {
  AttentionParams p, prefix;
  if (x == nullptr || check_attention(a, p) != MOE_OK || check_shared(a, x) != MOE_OK || !shares(p, x, prefix)) return 0;
  return partial_bytes(most_pieces(p.N, p.Hq, p.cache.kv_heads), static_cast<int64_t>(p.N) * p.Hq, p.cache.head_dim, x->groups);
}

int moe_paged_attention_shared(const moe_paged_attention_args_t* a, const moe_shared_prefix_t* x, moe_stream_t stream) {
  AttentionParams p, prefix;
  int st = check_attention(a, p);
  if (st == MOE_OK) st = check_shared(a, x);
  if (st != MOE_OK || p.N == 0) return st;
  (void)cudaGetLastError();
  const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  if (x->groups == 0 || x->max_tokens == 0) return attend(p, nullptr, a->dtype, on);
  if (x->lens == nullptr || (x->seqs == nullptr && x->groups != 1)) return MOE_ERR_NULL;
  const bool some = x->partial != nullptr || x->partial_bytes != 0, whole = shares(p, x, prefix);
  if (some ? x->partial == nullptr || !aligned(x->partial, 32) || x->partial_bytes < moe_shared_prefix_partial_size(p.N, p.Hq, p.cache.head_dim, x->groups)
           : whole)
    return MOE_ERR_WORKSPACE;
  if (!whole) return attend(p, nullptr, a->dtype, on);
  AttentionForms f = {};
  f.groups = x->groups, f.sequences = p.B;
  f.max_tokens = prefix.max_q_len;
  f.seqs = x->seqs, f.lens = x->lens;
  f.rows = static_cast<int64_t>(p.N) * p.Hq;
  f.most_pieces = most_pieces(p.N, p.Hq, p.cache.kv_heads);
  while (partial_bytes(f.most_pieces, f.rows, p.cache.head_dim, x->groups) > x->partial_bytes) --f.most_pieces;   // 2 fit
  f.sums = static_cast<float*>(x->partial);
  f.refs = reinterpret_cast<float2*>(f.sums + (f.most_pieces + 1) * f.rows * p.cache.head_dim);
  f.pieces = reinterpret_cast<int32_t*>(f.refs + (f.most_pieces + 1) * f.rows);
  f.pass = moe::kPrefixPass;
  moe::decode_attention_shape(p, f.own_row_tiles, f.own_per_sm);
  const int sms = moe::sm_count();
  f.sms = sms < 255 ? sms : 255;
  int error = moe::launch_prefill_attention(prefix, &f, a->dtype, on);
  if (error != MOE_OK) return error;
  f.pass = moe::kOwnPass;
  error = moe::launch_decode_attention(p, &f, a->dtype, on);
  return error != MOE_OK ? error : moe::launch_shared_join(p, f, a->dtype, on);
}

}  // extern "C"
