// What the kernels of the attention half share: element types, the rotation of
// one stretch of a head, float8 e4m3 conversions, and the launch interfaces of
// rope.cu, kv_append.cu, decode_attention.cu and prefill_attention.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe_lora.h"

namespace moe {

// ---------------------------------------------------------------- elements
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// N elements (N * sizeof(T) bytes, aligned to min(16, that)) to and from float32.
template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Pack {
  T v[N];
};
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&x)[N]) {
  const Pack<T, N> r = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f32(r.v[i]);
}
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&x)[N]) {
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = r;
}

// -------------------------------------------------------------------- e4m3
// Two e4m3 codes (low byte first) to two float16 values, exact; NaN codes give NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}
// The four codes of a word: the lower two to ``lo``, the upper two to ``hi``.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t word, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(word));
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint16_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// 2^x, to 2 units in the last place; 2^-infinity is 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A bf16 row becomes float16 by taking a power of two out of it: its exponent,
// given that of the row's largest magnitude (-127 to 127; 128: not finite).
// The largest then lies in [2^14, 2^15), so that all values down to 2^-31 of
// it stay exact; 112 and -126 hold the ends of bf16's range.
__device__ __forceinline__ int query_exponent(int largest) {
  return largest > 127 ? 0 : max(-126, min(112, largest - 14));
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Two float32 values to float16, first in the low half.
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float first, float second) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(second), "f"(first));
  return r;
}
// Two float32 values to e4m3 codes (first in the low byte): nearest, ties to
// even, magnitudes past 448 give 448, NaN stays NaN.
__device__ __forceinline__ uint16_t f32x2_to_e4m3x2(float first, float second) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(second), "f"(first));
  return r;
}

// ---------------------------------------------------------------- rotation
// A head is cut into D / 2V stretches of 2V elements that one thread handles.
// Stretch c of the rotated part holds the pairs of frequencies [Vc, Vc + V):
// two runs of V elements R/2 apart (half layout) or one run of 2V elements
// (interleaved).  Past the rotated part a stretch is one run of 2V elements.
// V divides R/2, and 2V divides D.
template <int V>
struct Stretch {
  int a, b;       // first elements of the two runs
  bool turned;    // in the rotated part
  __device__ __forceinline__ Stretch(int c, int R, bool interleaved) {
    turned = 2 * V * c < R;
    const bool split = turned && !interleaved;
    a = split ? V * c : 2 * V * c;
    b = split ? R / 2 + V * c : a + V;
  }
};

// cos and sin of frequencies [Vc, Vc + V) from a table row (R/2 cosines, then R/2 sines).
template <int V>
__device__ __forceinline__ void load_cos_sin(const float* row, int c, int R, float (&cs)[V], float (&sn)[V]) {
  load_f32<float, V>(row + V * c, cs);
  load_f32<float, V>(row + R / 2 + V * c, sn);
}

// Positions of several axes (time, height, width): each pair has an axis, two
// bits each in of_pair, and a token a position on each axis, [count][N] with
// ``stride`` between axes.  By value with a launch, so that a captured call
// keeps it.
constexpr int kMaxAxes = 4, kMaxPairs = 512;
struct RopeAxes {
  int64_t stride;
  int count;
  uint32_t of_pair[kMaxPairs / 16];
};
struct OneAxis {};
// The axis of pair i.
__device__ __forceinline__ uint32_t axis_of(const RopeAxes& axes, int i) { return axes.of_pair[i / 16] >> (2 * (i % 16)) & 3; }
// Whether token t's positions on all axes are in the table.
__device__ __forceinline__ bool in_table(const RopeAxes& axes, const int32_t* positions, int64_t t, int num_positions) {
  bool good = true;
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) {
    if (a >= axes.count) break;
    good &= static_cast<uint32_t>(positions[a * axes.stride + t]) < static_cast<uint32_t>(num_positions);
  }
  return good;
}
// The most tokens that ``threads`` consecutive items lie in.
__host__ __device__ __forceinline__ uint32_t axes_tokens(uint32_t threads, uint32_t per_token) { return (threads - 2) / per_token + 2; }
// The angles of tokens [t0, t0 + tokens) as rows of cosines and sines, each
// pair's from its own axis's row of the table, by all threads of a CTA; good[j]
// (if asked for): whether token t0 + j has all its positions in the table.  Each
// angle is looked up once and not by every head, a thread's all of one column
// and so of one axis; a row then serves as one of the table does.
__device__ __forceinline__ void gather_angles(float* rows, int* good, const RopeAxes& axes, const int32_t* positions, const float* cos_sin,
                                              int64_t t0, int tokens, int R, int num_positions) {
  const int threads = blockDim.x * blockDim.y * blockDim.z, tid = threadIdx.x + blockDim.x * (threadIdx.y + blockDim.y * threadIdx.z);
  const int at_once = threads / R;                      // tokens; 0: a thread has several columns
  const int first = at_once > 0 ? tid / R : 0, step = at_once > 0 ? at_once : 1;
  for (int col = tid - first * R; col < R && first < step; col += threads) {
    const int32_t* pos = positions + axis_of(axes, col < R / 2 ? col : col - R / 2) * axes.stride + t0;
    const float* column = cos_sin + col;
#pragma unroll 4
    for (int j = first; j < tokens; j += step) {
      const int p = pos[j];
      rows[j * R + col] = static_cast<uint32_t>(p) < static_cast<uint32_t>(num_positions) ? column[static_cast<int64_t>(p) * R] : 0.f;
    }
  }
  if (good != nullptr)
    for (int j = tid; j < tokens; j += threads) good[j] = in_table(axes, positions, t0 + j, num_positions);
}

// (u, w) -> (u cos - w sin, w cos + u sin), in float32.  ROUNDED: each product
// is rounded, for keys that become codes.  Next to the table's rounding that
// changes little, but a key close to the middle of two codes then gets the
// code that a program gets which does not fuse them; fused, a few of 2 million
// did not.  (4096 tokens 18.7 us, fused 18.2.  The products as packed pairs
// take the same time; with packed sums too the assembler fused them after all.)
template <bool ROUNDED>
__device__ __forceinline__ void turn_pair(float& u, float& w, float cs, float sn) {
  const float x = u;
  if constexpr (ROUNDED) {
    u = __fsub_rn(__fmul_rn(x, cs), __fmul_rn(w, sn));
    w = __fadd_rn(__fmul_rn(w, cs), __fmul_rn(x, sn));
  } else {
    u = x * cs - w * sn;
    w = w * cs + x * sn;
  }
}
// Each pair of a stretch.  In the interleaved layout the 2V elements (a, b)
// hold the pairs side by side.
template <int V, bool ROUNDED>
__device__ __forceinline__ void rotate(float (&a)[V], float (&b)[V], const float (&cs)[V], const float (&sn)[V],
                                       bool interleaved) {
  if (!interleaved || V == 1) {
#pragma unroll
    for (int i = 0; i < V; ++i) turn_pair<ROUNDED>(a[i], b[i], cs[i], sn[i]);
  } else if constexpr (V > 1) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      turn_pair<ROUNDED>(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
      turn_pair<ROUNDED>(b[2 * i], b[2 * i + 1], cs[V / 2 + i], sn[V / 2 + i]);
    }
  }
}

// ------------------------------------------------------------------ launch
// One operand of a rotation: [N, H, D] with strides in elements.
struct RopeTensor {
  const void* in;
  void* out;
  int64_t in_token, in_head, out_token, out_head;
  int heads;
};
// Raw stretches, moved as they are so that several can be on their way.
template <typename T, int V>
__device__ __forceinline__ void to_f32s(const Pack<T, V>& r, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = to_f32(r.v[i]);
}

// Work item ``item`` of a rotation: one stretch of HEADS consecutive heads of
// one token (of x's heads, then y's, which may be none).  The constructor puts
// the loads on their way; finish() takes the token's position, which may be
// looked up meanwhile, or kUnturned for none, or kSkipped to leave it out.
constexpr int kUnturned = -1, kSkipped = -2;
template <int V>
__host__ __device__ __forceinline__ uint32_t rotation_items(int heads, int per_thread, int D) {
  return static_cast<uint32_t>((heads + per_thread - 1) / per_thread * (D / (2 * V)));
}
template <typename T, int V, int HEADS>
struct RotationItem {
  Pack<T, V> ra[HEADS], rb[HEADS];
  uint32_t t;
  int h0, c;
  bool live;
  __device__ __forceinline__ RotationItem(const RopeTensor& x, const RopeTensor& y, uint32_t item, uint32_t per_token, int N, int D,
                                          int R, bool interleaved) {
    const uint32_t per_head = static_cast<uint32_t>(D / (2 * V));
    t = item / per_token;
    const uint32_t j = item - t * per_token;
    h0 = static_cast<int>(j / per_head) * HEADS;
    c = static_cast<int>(j - j / per_head * per_head);
    live = t < static_cast<uint32_t>(N);
    const Stretch<V> s(c, R, interleaved);
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      const int h = h0 + u;
      if (!live || h >= x.heads + y.heads) break;
      const T* in = h < x.heads ? static_cast<const T*>(x.in) + t * x.in_token + h * x.in_head
                                : static_cast<const T*>(y.in) + t * y.in_token + (h - x.heads) * y.in_head;
      ra[u] = *reinterpret_cast<const Pack<T, V>*>(in + s.a);
      rb[u] = *reinterpret_cast<const Pack<T, V>*>(in + s.b);
    }
  }
  __device__ __forceinline__ void finish(const RopeTensor& x, const RopeTensor& y, int pos, int R, bool interleaved, bool inverse,
                                         const float* cos_sin) const {
    if (!live || pos == kSkipped) return;
    turn_by(x, y, pos >= 0 ? cos_sin + static_cast<int64_t>(pos) * R : nullptr, R, interleaved, inverse);
  }
  // ``row``: the token's cosines and sines, or nullptr for none.
  __device__ __forceinline__ void turn_by(const RopeTensor& x, const RopeTensor& y, const float* row, int R, bool interleaved, bool inverse) const {
    const Stretch<V> s(c, R, interleaved);
    const bool turn = s.turned && row != nullptr;
    float cs[V], sn[V];
    if (turn) {
      load_cos_sin<V>(row, c, R, cs, sn);
      if (inverse) {
#pragma unroll
        for (int i = 0; i < V; ++i) sn[i] = -sn[i];
      }
    }
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
      const int h = h0 + u;
      if (h >= x.heads + y.heads) break;
      float a[V], b[V];
      to_f32s<T, V>(ra[u], a);
      to_f32s<T, V>(rb[u], b);
      if (turn) rotate<V, false>(a, b, cs, sn, interleaved);
      T* out = h < x.heads ? static_cast<T*>(x.out) + t * x.out_token + h * x.out_head
                           : static_cast<T*>(y.out) + t * y.out_token + (h - x.heads) * y.out_head;
      store_f32<T, V>(out + s.a, a);
      store_f32<T, V>(out + s.b, b);
    }
  }
};

struct RopeParams {
  RopeTensor q, k;
  const int32_t* positions;
  const float* cos_sin;
  int32_t* status;
  int N, D, R, num_positions, interleaved, inverse;
};
cudaError_t launch_rope(const RopeParams& p, const RopeAxes* axes, int dtype, int V, cudaStream_t s);   // axes: NULL = one

struct KvAppendParams {
  moe_kv_cache_t cache;
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;
  RopeTensor q;                 // heads 0: none
  const int32_t *block_table, *seq_lens, *cu_q, *positions;
  const float* cos_sin;
  int32_t* status;
  int N, B, table_width, max_q_len, R, num_positions, interleaved;
  int slots;                    // pages that one sequence's new tokens can touch
  uint32_t q_items;             // work items of a token's q
};
cudaError_t launch_kv_append(const KvAppendParams& p, const RopeAxes* axes, int dtype, int V, cudaStream_t s);

// Attention.  A "row" is one (new token, query head) of a key head's group:
// row r of sequence b and key head h is token r / group, query head h * group
// + r % group.
struct AttentionParams {
  moe_kv_cache_t cache;
  const void* q;
  void* out;
  float* lse;
  int64_t q_token, q_head, out_token, out_head;
  const int32_t *block_table, *seq_lens, *cu_q;
  int32_t* status;
  int N, B, Hq, table_width, max_q_len, max_seq_len;
  int window;                   // keys a row sees, itself included; 0 = all before it
  float scale;
  void* workspace;
  uint64_t wait_limit_ns;
  uint32_t debug_flags;
};
// What an attention call may ask for besides, in kernels of their own.
//
// Sinks: the first ``sinks`` keys stay visible to every row of a window.
//
// Shared prefixes: sequences [seqs[g], seqs[g + 1]) of a group (seqs NULL: all)
// begin with the same lens[g] tokens.  The prefix pass (the kernel for many
// rows) takes a group as one sequence whose rows are all of its new tokens' and
// all see the prefix's keys, through the block table's row of the group's first
// sequence.  It cuts the keys in pieces and leaves each piece's unnormalised
// sums with their references.  The own pass (the kernel for few rows) takes
// each sequence's other keys, beside it on the SMs that it leaves free, and
// leaves the same as one more piece; a third kernel joins them.  A sequence
// that begins inside the prefix, or whose tokens are not all among the group's
// first max_tokens, takes no part: the own pass reads all of its keys.
constexpr int kOwnUnit = 14;
enum AttentionPass { kWholePass, kPrefixPass, kOwnPass };
struct AttentionForms {
  int sinks;
  int pass;                     // AttentionPass
  int groups, sequences, max_tokens;
  const int32_t *seqs, *lens;
  int most_pieces;
  int own_row_tiles, own_per_sm; // of the own pass: row tiles of a sequence, CTAs an SM
  int sms;
  int64_t rows;                 // N * Hq
  float* sums;                  // [most_pieces + 1][rows][head_dim], the last of the own pass
  float2* refs;                 // [most_pieces + 1][rows]: reference and denominator
  int32_t* pieces;              // [groups]

  // What both passes take, in us (as measured: a CTA's time before and after its
  // tiles, and a tile's with the other pass beside it), if the prefix pass, with
  // ``tiles`` key tiles of its units in pieces of ``least`` or more, has n SMs,
  // and the own pass, with ``own`` key tiles of its row tiles, the others
  // meanwhile (or all of them after it).  Both passes look for the same best n:
  // they have times of their own before and after their tiles, so a CTA should
  // do all it can in one go.  A row tile takes the own pass kOwnUnit tiles' time
  // besides its own, counted in ``own``.  The times are those of heads of 128 in
  // row tiles of 8.  Against the best of n = 16, 24, ... the plan's n was 0 to 3%
  // slower on 64 to 256 sequences with heads of 64 and 128 and 1 to 8 key heads, 5
  // to 8% with row tiles of 16, and 20% (93 / 77 us) and 23% (134 / 109 us) where
  // units come out in uneven pieces: 8 units of 235 tiles on 88 SMs, 64 units of 64 on 152.
  __device__ __forceinline__ float time(int n, int tiles, int least, int own) const {
    const int left = sms - n, ctas = own_per_sm * (left > 0 ? left : sms);
    const float first = 15.f + 2.6f * static_cast<float>(max(least, (tiles + n - 1) / n)), second = 12.f + 0.85f * static_cast<float>((own + ctas - 1) / ctas);
    return left > 0 ? fmaxf(first, second) : first + second;
  }
  // The key tiles that a piece has at least, where the longest unit has ``longest``.
  __device__ __forceinline__ int least_piece(int longest) const { return (longest + most_pieces - 1) / most_pieces; }
  // The time and n as one number that orders by time.
  __device__ __forceinline__ int choice(int n, int tiles, int least, int own) const {
    return static_cast<int>(fminf(8.f * time(n, tiles, least, own), 8.0e6f)) << 8 | n;
  }
  // Group g's sequences and their tokens; nothing, where the list is out of order.
  __device__ __forceinline__ void group(const int32_t* cu_q, int g, int& s0, int& s1, int& q0, int& q1) const {
    s0 = seqs == nullptr ? 0 : max(0, min(sequences, seqs[g]));
    s1 = seqs == nullptr ? sequences : max(s0, min(sequences, seqs[g + 1]));
    q0 = cu_q == nullptr ? s0 : cu_q[s0];
    q1 = cu_q == nullptr ? s1 : cu_q[s1];
  }
  // Whether a sequence whose rows are tokens [q_first, q_first + q_len) and begin
  // at position ``start`` takes part in a prefix of n tokens of the group with
  // tokens [q0, q1).
  __device__ __forceinline__ bool takes_part(int n, int q0, int q1, int q_first, int q_len, int start) const {
    return n > 0 && start >= n && q_first >= q0 && q_first + q_len <= min(q1, q0 + max_tokens);
  }
  // Whether some row of a group's sequences [s0, s1) does.  Where none does,
  // nobody has to have the prefix's pages yet.
  __device__ __forceinline__ bool some_take_part(const int32_t* cu_q, const int32_t* seq_lens, int n, int s0, int s1, int q0, int q1) const {
    bool some = false;
#pragma unroll 1
    for (int s = s0; s < s1 && !some; s += 4) {          // nearly always the first one does
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = min(s + i, s1 - 1), q_first = cu_q == nullptr ? b : cu_q[b], q_len = cu_q == nullptr ? 1 : cu_q[b + 1] - q_first;
        some |= q_len > 0 && takes_part(n, q0, q1, q_first, q_len, seq_lens[b] - q_len);
      }
    }
    return some;
  }
  // How many keys of sequence b, whose rows are tokens [q_first, q_first +
  // q_len) and begin at position ``start``, the prefix pass has taken, and in
  // which group.
  __device__ __forceinline__ int taken(const int32_t* cu_q, int b, int q_first, int q_len, int start, int& g) const {
    g = 0;
    if (seqs != nullptr) {
      int hi = groups;                                   // the last group that begins at b or before
      while (hi - g > 1) {
        const int mid = (g + hi) / 2;
        if (seqs[mid] <= b) g = mid; else hi = mid;
      }
      if (b < seqs[g] || b >= seqs[g + 1]) return 0;
    }
    const int n = lens[g];
    int s0, s1, q0, q1;
    group(cu_q, g, s0, s1, q0, q1);
    return takes_part(n, q0, q1, q_first, q_len, start) ? n : 0;
  }
};
bool encode_cache_map(CUtensorMap* map, const moe_kv_cache_t& c, bool values, int rows);
bool encode_query_map(CUtensorMap* map, const AttentionParams& a, bool f16, int group, int tokens);
int sm_count();
size_t prefill_attention_workspace_bytes();
cudaError_t clear_prefill_counters(void* workspace, cudaStream_t s);
bool prefill_attention_fits(const AttentionParams& p);  // else the launch is MOE_ERR_UNSUPPORTED
int launch_prefill_attention(const AttentionParams& p, const AttentionForms* forms, int dtype, cudaStream_t s);  // a moe_status_t; forms NULL: none
bool shared_join_fits(const AttentionParams& p);     // whether its grid can be launched
int launch_shared_join(const AttentionParams& p, const AttentionForms& forms, int dtype, cudaStream_t s);   // a moe_status_t
size_t decode_attention_workspace_bytes();
cudaError_t clear_decode_counters(void* workspace, cudaStream_t s);
void decode_attention_shape(const AttentionParams& p, int& row_tiles, int& per_sm);   // row tiles of a sequence, CTAs an SM
bool decode_attention_fits(const AttentionParams& p);   // likewise
int launch_decode_attention(const AttentionParams& p, const AttentionForms* forms, int dtype, cudaStream_t s);   // a moe_status_t

}  // namespace moe
