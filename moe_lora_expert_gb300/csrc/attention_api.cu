// C ABI of the attention half: argument checks of moe_rope, moe_kv_append and
// moe_paged_attention, and the choice of the width of their accesses.
#include <cstddef>

#include "attention.cuh"

namespace {

using moe::AttentionParams;
using moe::KvAppendParams;
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

}  // namespace

extern "C" {

int moe_rope(const moe_rope_args_t* a, moe_stream_t stream) {
  if (a == nullptr) return MOE_ERR_NULL;
  if (a->struct_size != sizeof(*a)) return MOE_ERR_UNSUPPORTED;
  if (a->dtype < MOE_DTYPE_BF16 || a->dtype > MOE_DTYPE_F32) return MOE_ERR_UNSUPPORTED;
  if (a->N < 0 || a->Hq < 0 || a->Hk < 0 || a->D <= 0 || a->rotary_dim < 2 || a->rotary_dim > a->D ||
      a->rotary_dim % 2 != 0 || a->D % 2 != 0 || a->num_positions < 0)
    return MOE_ERR_SHAPE;
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
  return done(moe::launch_rope(p, a->dtype, V, reinterpret_cast<cudaStream_t>(stream)));
}

int moe_kv_append(const moe_kv_append_args_t* a, moe_stream_t stream) {
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
  if (!aligned(a->cos_sin, 16)) return MOE_ERR_ALIGN;
  if (a->Hq > 65536) return MOE_ERR_UNSUPPORTED;
  if (a->N == 0 || a->B == 0 || a->max_q_len == 0) return MOE_OK;
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
  return done(moe::launch_kv_append(p, a->dtype, V, reinterpret_cast<cudaStream_t>(stream)));
}

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
  if (a->N == 0 || a->B == 0 || a->max_q_len == 0) return MOE_OK;
  if (a->q == nullptr || a->out == nullptr) return MOE_ERR_NULL;
  const int64_t strides[4] = {a->q_stride_token, a->q_stride_head, a->out_stride_token, a->out_stride_head};
  for (int64_t s : strides)
    if (s % 8 != 0) return MOE_ERR_ALIGN;
  if (!aligned(a->q, 16) || !aligned(a->out, 16)) return MOE_ERR_ALIGN;
  if (a->workspace == nullptr || !aligned(a->workspace, 256) || a->workspace_bytes < moe_paged_attention_workspace_size())
    return MOE_ERR_WORKSPACE;
  AttentionParams p = {};
  p.cache = c;
  p.q = a->q, p.out = a->out, p.lse = a->lse;
  p.q_token = a->q_stride_token, p.q_head = a->q_stride_head;
  p.out_token = a->out_stride_token, p.out_head = a->out_stride_head;
  p.block_table = a->block_table, p.seq_lens = a->seq_lens, p.cu_q = a->cu_q;
  p.status = a->status;
  p.N = a->N, p.B = a->B, p.Hq = a->Hq, p.table_width = a->table_width;
  p.max_q_len = a->cu_q == nullptr ? 1 : a->max_q_len < a->N ? a->max_q_len : a->N;
  p.window = a->window;
  p.max_seq_len = a->max_seq_len;
  p.scale = a->scale;
  p.workspace = a->workspace;
  p.wait_limit_ns = 1000000ull * static_cast<uint64_t>(a->wait_timeout_ms > 0 ? a->wait_timeout_ms : 2000);
  p.debug_flags = a->debug_flags;
  (void)cudaGetLastError();
  const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = static_cast<int64_t>(p.max_q_len) * (a->Hq / c.kv_heads);
  if (few_rows(rows, static_cast<int64_t>(a->B) * c.kv_heads)) return moe::launch_decode_attention(p, a->dtype, on);
  return moe::launch_prefill_attention(p, a->dtype, on);
}

}  // extern "C"
