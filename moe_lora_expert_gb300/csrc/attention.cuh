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
    const Stretch<V> s(c, R, interleaved);
    const bool turn = s.turned && pos >= 0;
    float cs[V], sn[V];
    if (turn) {
      load_cos_sin<V>(cos_sin + static_cast<int64_t>(pos) * R, c, R, cs, sn);
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
cudaError_t launch_rope(const RopeParams& p, int dtype, int V, cudaStream_t s);

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
cudaError_t launch_kv_append(const KvAppendParams& p, int dtype, int V, cudaStream_t s);

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
bool encode_cache_map(CUtensorMap* map, const moe_kv_cache_t& c, bool values, int rows);
bool encode_query_map(CUtensorMap* map, const AttentionParams& a, bool f16, int group, int tokens);
int sm_count();
size_t prefill_attention_workspace_bytes();
cudaError_t clear_prefill_counters(void* workspace, cudaStream_t s);
int launch_prefill_attention(const AttentionParams& p, int dtype, cudaStream_t s);  // a moe_status_t
size_t decode_attention_workspace_bytes();
cudaError_t clear_decode_counters(void* workspace, cudaStream_t s);
int launch_decode_attention(const AttentionParams& p, int dtype, cudaStream_t s);   // a moe_status_t

}  // namespace moe
