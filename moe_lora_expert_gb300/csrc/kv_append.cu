// New keys (rotated) and values into a paged cache of e4m3 codes with one
// scale for each (page, head), and the queries' rotation in the same launch.
//
// The scale of a page and head is the power of two 2^k with the smallest k
// for which its largest magnitude is at most 448 * 2^k (448 = 1.75 * 2^8 is
// the largest code).  A floating-point code keeps its relative precision
// under any scale, so the power of two costs nothing there, and it makes the
// step that a cache filled token by token needs exact: when new tokens raise
// the scale of a page that holds others, their codes are multiplied by
// s_old / s_new, which moves their exponents and rounds only what becomes
// subnormal.  With an arbitrary scale every raise would round every code again.
#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kHeld = 4;  // stretches a thread keeps in registers between the maximum and the codes

// Smallest 2^k (k >= -42) with amax <= 448 * 2^k; amax >= 0, not NaN.
__device__ __forceinline__ float page_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int k = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  k = k < -42 ? -42 : k > 120 ? 120 : k;   // infinity: 2^120, where code 448 reads as infinity again
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// The sequence that token t belongs to: the largest b with cu_q[b] <= t.
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu_q[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[V], float inv) {
  if constexpr (V == 1) {
    *p = static_cast<uint8_t>(f32x2_to_e4m3x2(x[0] * inv, 0.f));
  } else {
    Pack<uint16_t, V / 2> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = f32x2_to_e4m3x2(x[2 * i] * inv, x[2 * i + 1] * inv);
    *reinterpret_cast<Pack<uint16_t, V / 2>*>(p) = r;
  }
}

// CTAs [0, 2 * B * slots * Hkv): one (sequence, page of it, head, K or V) each.
// The rest rotate q.
template <typename T, int V>
__global__ void kv_append_kernel(KvAppendParams p) {
  __shared__ float s_max[32];
  pdl_wait();
  const moe_kv_cache_t& ca = p.cache;
  const int per_head = ca.head_dim / (2 * V);
  const int units = 2 * p.B * p.slots * ca.kv_heads;
  const int tid = threadIdx.x;

  if (blockIdx.x >= static_cast<unsigned>(units)) {  // q
    const int64_t total = static_cast<int64_t>(p.N) * p.q.heads * per_head;
    const int64_t stride = static_cast<int64_t>(gridDim.x - units) * blockDim.x;
    for (int64_t j = static_cast<int64_t>(blockIdx.x - units) * blockDim.x + tid; j < total; j += stride) {
      const int64_t th = j / per_head;
      const int c = static_cast<int>(j - th * per_head);
      const int t = static_cast<int>(th / p.q.heads), h = static_cast<int>(th - static_cast<int64_t>(t) * p.q.heads);
      if (p.cu_q != nullptr && t >= p.cu_q[p.B]) continue;  // a row of no sequence
      int pos;
      if (p.positions != nullptr) {
        pos = p.positions[t];
      } else {
        const int b = p.cu_q == nullptr ? t : sequence_of(p.cu_q, p.B, t);
        pos = p.cu_q == nullptr ? p.seq_lens[b] - 1 : p.seq_lens[b] - p.cu_q[b + 1] + t;
      }
      const bool known = pos >= 0 && pos < p.num_positions;
      const T* in = static_cast<const T*>(p.q.in) + t * p.q.in_token + h * p.q.in_head;
      T* out = static_cast<T*>(p.q.out) + t * p.q.out_token + h * p.q.out_head;
      const Stretch<V> s(c, p.R, p.interleaved);
      float a[V], b[V];
      load_f32<T, V>(in + s.a, a);
      load_f32<T, V>(in + s.b, b);
      if (s.turned && known) {
        float cs[V], sn[V];
        load_cos_sin<V>(p.cos_sin + static_cast<int64_t>(pos) * p.R, c, p.R, cs, sn);
        rotate<V>(a, b, cs, sn, p.interleaved);
      } else if (s.turned) {
        set_status(p.status, MOE_ERR_BAD_POSITION);
      }
      store_f32<T, V>(out + s.a, a);
      store_f32<T, V>(out + s.b, b);
    }
    return;
  }

  int u = blockIdx.x;
  const bool is_k = (u & 1) == 0;
  u >>= 1;
  const int head = u % ca.kv_heads;
  u /= ca.kv_heads;
  const int slot = u % p.slots, b = u / p.slots;
  const int t_first = p.cu_q == nullptr ? b : p.cu_q[b];
  int t_end = p.cu_q == nullptr ? b + 1 : p.cu_q[b + 1];
  if (t_end > p.N) t_end = p.N;
  const int len = p.seq_lens[b];
  const int start = len - (t_end - t_first);          // position of the first new token
  const int P = ca.page_size;
  if (start < 0 && tid == 0) set_status(p.status, MOE_ERR_BAD_POSITION);
  const int page_at = (start < 0 ? 0 : start) / P + slot;
  const int p0 = max(start < 0 ? 0 : start, page_at * P), p1 = min(len, (page_at + 1) * P);
  if (p0 >= p1) return;
  const int page = page_at < p.table_width ? p.block_table[static_cast<int64_t>(b) * p.table_width + page_at] : -1;
  if (page < 0 || page >= ca.num_pages) {
    if (tid == 0) set_status(p.status, MOE_ERR_BAD_PAGE);
    return;
  }
  const int rows = p1 - p0, off = p0 - page_at * P, items = rows * per_head;
  const T* x = is_k ? static_cast<const T*>(p.k) + head * p.k_head : static_cast<const T*>(p.v) + head * p.v_head;
  const int64_t x_token = is_k ? p.k_token : p.v_token;
  uint8_t* codes = is_k ? ca.k + page * ca.k_stride_page + head * ca.k_stride_head
                        : ca.v + page * ca.v_stride_page + head * ca.v_stride_head;
  const int64_t row_bytes = is_k ? ca.k_stride_token : ca.v_stride_token;
  float* scale = (is_k ? ca.k_scale : ca.v_scale) + static_cast<int64_t>(page) * ca.kv_heads + head;
  const float s_old = off > 0 ? *scale : 0.f;         // a page with no earlier token keeps nothing of its last use
  const bool turn = is_k && p.cos_sin != nullptr;

  auto fetch = [&](int j, float (&a)[V], float (&bb)[V]) {
    const int r = j / per_head, c = j - r * per_head;
    const int t = t_first + (p0 - start) + r;
    const T* row = x + t * x_token;
    const Stretch<V> s(c, turn ? p.R : 0, p.interleaved);
    load_f32<T, V>(row + s.a, a);
    load_f32<T, V>(row + s.b, bb);
    if (s.turned) {
      const int pos = p.positions != nullptr ? p.positions[t] : p0 + r;
      if (pos >= 0 && pos < p.num_positions) {
        float cs[V], sn[V];
        load_cos_sin<V>(p.cos_sin + static_cast<int64_t>(pos) * p.R, c, p.R, cs, sn);
        rotate<V>(a, bb, cs, sn, p.interleaved);
      } else {
        set_status(p.status, MOE_ERR_BAD_POSITION);
      }
    }
  };

  float held_a[kHeld][V], held_b[kHeld][V];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = tid + i * blockDim.x;
    if (j < items) {
      fetch(j, held_a[i], held_b[i]);
#pragma unroll
      for (int e = 0; e < V; ++e) amax = fmaxf(amax, fmaxf(fabsf(held_a[i][e]), fabsf(held_b[i][e])));
    }
  }
  for (int j = tid + kHeld * blockDim.x; j < items; j += blockDim.x) {
    float a[V], bb[V];
    fetch(j, a, bb);
#pragma unroll
    for (int e = 0; e < V; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[e]), fabsf(bb[e])));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) amax = fmaxf(amax, s_max[w]);
  const float s_new = fmaxf(s_old, page_scale(amax));
  const float inv = 1.f / s_new;

  auto put = [&](int j, const float (&a)[V], const float (&bb)[V]) {
    const int r = j / per_head, c = j - r * per_head;
    const Stretch<V> s(c, turn ? p.R : 0, p.interleaved);
    uint8_t* row = codes + (off + r) * row_bytes;
    store_codes<V>(row + s.a, a, inv);
    store_codes<V>(row + s.b, bb, inv);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int j = tid + i * blockDim.x;
    if (j < items) put(j, held_a[i], held_b[i]);
  }
  for (int j = tid + kHeld * blockDim.x; j < items; j += blockDim.x) {
    float a[V], bb[V];
    fetch(j, a, bb);
    put(j, a, bb);
  }
  if (off > 0 && s_new != s_old) {                     // the codes that the page held before
    const float ratio = s_old * inv;
    const int chunks = ca.head_dim / 16;
    for (int j = tid; j < off * chunks; j += blockDim.x) {
      const int r = j / chunks, c = j - r * chunks;
      Pack<uint16_t, 8>* at = reinterpret_cast<Pack<uint16_t, 8>*>(codes + r * row_bytes + 16 * c);
      Pack<uint16_t, 8> w = *at;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = e4m3x2_to_f32x2(w.v[e]);
        w.v[e] = f32x2_to_e4m3x2(f.x * ratio, f.y * ratio);
      }
      *at = w;
    }
  }
  if (tid == 0 && s_new != *scale) *scale = s_new;     // every thread has its s_old since the barrier
}

template <typename T, int V>
cudaError_t launch(const KvAppendParams& p, cudaStream_t s) {
  const int per_head = p.cache.head_dim / (2 * V);
  const int rows = p.slots > 1 ? p.cache.page_size : 1;
  int threads = 64;
  while (threads < 512 && threads * kHeld < rows * per_head) threads *= 2;
  const int64_t units = 2ll * p.B * p.slots * p.cache.kv_heads;
  const int64_t q_items = static_cast<int64_t>(p.N) * p.q.heads * per_head;
  const int64_t q_ctas = (q_items + threads - 1) / threads;
  return launch_pdl(kv_append_kernel<T, V>, dim3(static_cast<unsigned>(units + (q_ctas < 65536 ? q_ctas : 65536))),
                    dim3(threads), 0, s, p);
}

template <typename T>
cudaError_t launch_v(const KvAppendParams& p, int V, cudaStream_t s) {
  if (V >= 8) return launch<T, 8>(p, s);
  if (V == 4) return launch<T, 4>(p, s);
  return launch<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendParams& p, int dtype, int V, cudaStream_t s) {
  return dtype == MOE_DTYPE_F16 ? launch_v<__half>(p, V, s) : launch_v<__nv_bfloat16>(p, V, s);
}

}  // namespace moe
