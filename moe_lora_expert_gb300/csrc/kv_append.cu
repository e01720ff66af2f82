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
//
// A CTA takes the new tokens of one (sequence, page of it, head, K or V), so
// that a maximum is one CTA's and nothing depends on the order of atomics; the
// CTAs after those rotate q.  What bounds it: bytes (read k, v and q once,
// write codes and q) once there are enough; 4096 tokens of 32 and 4 heads of
// 128 take 18.7 us, 82 MB at 4.4 TB/s, 65% of the copy rate (64 registers a
// thread: with 126, which held the rotated stretches, 20.5 us; 4 stretches held
// instead of 2 the same there, 11.3 instead of 10.3 us on ragged chunks).  64
// single tokens take 5.8 us: the chain from lengths to table to scale.
#include <type_traits>

#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kMaxThreads = 512;
constexpr int kMinCtas = 2;           // of kMaxThreads an SM: 64 registers a thread
constexpr int kManyItems = 1 << 17;   // stretches of q from which on a thread takes two heads (4096 tokens: one 21.2, two 18.0 us)
constexpr int kHeld = 2;  // stretches a thread keeps in registers between the maximum and the codes

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

// Codes of x / by, or of x * by.
template <bool DIVIDE, int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&x)[V], float by) {
  auto scaled = [&](int i) { return DIVIDE ? x[i] / by : x[i] * by; };
  if constexpr (V == 1) {
    *p = static_cast<uint8_t>(f32x2_to_e4m3x2(scaled(0), 0.f));
  } else {
    Pack<uint16_t, V / 2> r;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.v[i] = f32x2_to_e4m3x2(scaled(2 * i), scaled(2 * i + 1));
    *reinterpret_cast<Pack<uint16_t, V / 2>*>(p) = r;
  }
}

// CTAs [0, 2 * B * slots * Hkv): one (sequence, page of it, head, K or V) each.
// The rest rotate q.
template <typename T, int V, int HEADS>
__global__ void __launch_bounds__(kMaxThreads, kMinCtas) kv_append_kernel(KvAppendParams p) {
  __shared__ float s_max[32];
  __shared__ int s_pos[kMaxThreads];
  pdl_launch_dependents();
  pdl_wait();
  const moe_kv_cache_t& ca = p.cache;
  const int per_head = ca.head_dim / (2 * V);
  const int units = 2 * p.B * p.slots * ca.kv_heads;
  const int tid = threadIdx.x;

  if (blockIdx.x >= static_cast<unsigned>(units)) {  // q
    const uint32_t item0 = (blockIdx.x - units) * blockDim.x, token0 = item0 / p.q_items;
    const RotationItem<T, V, HEADS> x(p.q, RopeTensor{}, item0 + tid, p.q_items, p.N, ca.head_dim, p.R, p.interleaved);
    // the positions of the CTA's tokens, a thread each
    const uint32_t t = token0 + tid;
    if (t <= (item0 + blockDim.x - 1) / p.q_items && t < static_cast<uint32_t>(p.N)) {
      int pos = kSkipped;
      if (p.cu_q == nullptr || static_cast<int>(t) < p.cu_q[p.B]) {          // else a row of no sequence
        if (p.positions != nullptr) {
          pos = p.positions[t];
        } else {
          const int b = p.cu_q == nullptr ? t : sequence_of(p.cu_q, p.B, t);
          pos = p.cu_q == nullptr ? p.seq_lens[b] - 1 : p.seq_lens[b] - p.cu_q[b + 1] + static_cast<int>(t);
        }
        if (pos < 0 || pos >= p.num_positions) {
          const bool padding = p.cu_q == nullptr && p.seq_lens[t] == 0;       // a slot without a sequence
          if (p.R > 0 && !padding) set_status(p.status, MOE_ERR_BAD_POSITION);
          pos = kUnturned;
        }
      }
      s_pos[tid] = pos;
    }
    __syncthreads();
    if (x.live) x.finish(p.q, RopeTensor{}, s_pos[x.t - token0], p.R, p.interleaved, false, p.cos_sin);
    return;
  }

  int u = blockIdx.x;
  const bool is_k = (u & 1) == 0;
  u >>= 1;
  const int head = u % ca.kv_heads;
  u /= ca.kv_heads;
  const int slot = u % p.slots, b = u / p.slots;
  const int t_first = p.cu_q == nullptr ? b : p.cu_q[b];
  const int t_end = p.cu_q == nullptr ? b + 1 : p.cu_q[b + 1];
  const int len = p.seq_lens[b];
  if (p.cu_q == nullptr && len == 0) return;          // a slot without a sequence
  const int start = len - (t_end - t_first);          // position of the first new token
  const int P = ca.page_size;
  if (start < 0 && tid == 0) set_status(p.status, MOE_ERR_BAD_POSITION);
  const int page_at = (start < 0 ? 0 : start) / P + slot;
  const int end = min(len, start + min(p.max_q_len, p.N - t_first));          // after the last token that is appended
  const int p0 = max(start < 0 ? 0 : start, page_at * P), p1 = min(end, (page_at + 1) * P);
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

  auto load = [&](int j, Pack<T, V>& ra, Pack<T, V>& rb) {
    const int r = j / per_head, c = j - r * per_head;
    const T* row = x + (t_first + (p0 - start) + r) * x_token;
    const Stretch<V> s(c, turn ? p.R : 0, p.interleaved);
    ra = *reinterpret_cast<const Pack<T, V>*>(row + s.a);
    rb = *reinterpret_cast<const Pack<T, V>*>(row + s.b);
  };
  auto rotated = [&](int j, const Pack<T, V>& ra, const Pack<T, V>& rb, float (&a)[V], float (&bb)[V]) {
    const int r = j / per_head, c = j - r * per_head;
    to_f32s<T, V>(ra, a);
    to_f32s<T, V>(rb, bb);
    if (turn && 2 * V * c < p.R) {
      const int pos = p.positions != nullptr ? p.positions[t_first + (p0 - start) + r] : p0 + r;
      if (pos >= 0 && pos < p.num_positions) {
        float cs[V], sn[V];
        load_cos_sin<V>(p.cos_sin + static_cast<int64_t>(pos) * p.R, c, p.R, cs, sn);
        rotate<V, true>(a, bb, cs, sn, p.interleaved);
      } else {
        set_status(p.status, MOE_ERR_BAD_POSITION);
      }
    }
  };

  // The maximum first, then the codes.  The stretches stay in registers as
  // they came and are rotated twice: rotated ones would take twice the
  // registers, and with them half of the threads that keep loads on their way.
  Pack<T, V> ra[kHeld], rb[kHeld];
  float amax = 0.f;
  auto reduce = [&](int j, const Pack<T, V>& pa, const Pack<T, V>& pb) {
    float a[V], bb[V];
    rotated(j, pa, pb, a, bb);
#pragma unroll
    for (int e = 0; e < V; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[e]), fabsf(bb[e])));
  };
  const int step = static_cast<int>(blockDim.x);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < items) load(tid + i * step, ra[i], rb[i]);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * step < items) reduce(tid + i * step, ra[i], rb[i]);
  for (int j = tid + kHeld * step; j < items; j += step) {
    Pack<T, V> pa, pb;
    load(j, pa, pb);
    reduce(j, pa, pb);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((tid & 31) == 0) s_max[tid >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (step >> 5); ++w) amax = fmaxf(amax, s_max[w]);
  const float s_new = fmaxf(s_old, page_scale(amax));
  const float inv = 1.f / s_new;

  auto put = [&](int j, const Pack<T, V>& pa, const Pack<T, V>& pb, auto divide) {
    const int r = j / per_head, c = j - r * per_head;
    float a[V], bb[V];
    rotated(j, pa, pb, a, bb);
    const Stretch<V> s(c, turn ? p.R : 0, p.interleaved);
    uint8_t* row = codes + (off + r) * row_bytes;
    constexpr bool kDivide = decltype(divide)::value;
    store_codes<kDivide, V>(row + s.a, a, kDivide ? s_new : inv);
    store_codes<kDivide, V>(row + s.b, bb, kDivide ? s_new : inv);
  };
  if ((__float_as_uint(s_new) & 0x7FFFFFu) == 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (tid + i * step < items) put(tid + i * step, ra[i], rb[i], std::false_type());
    for (int j = tid + kHeld * step; j < items; j += step) {
      Pack<T, V> pa, pb;
      load(j, pa, pb);
      put(j, pa, pb, std::false_type());
    }
  } else {   // a scale of the caller's own, which the page has kept: dividing is not multiplying by its inverse
#pragma unroll 1
    for (int j = tid; j < items; j += step) {
      Pack<T, V> pa, pb;
      load(j, pa, pb);
      put(j, pa, pb, std::true_type());
    }
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

template <typename T, int V, int HEADS>
cudaError_t launch_heads(KvAppendParams p, cudaStream_t s) {
  const int per_head = p.cache.head_dim / (2 * V);
  const int rows = p.slots > 1 ? p.cache.page_size : 1;
  int threads = 64;
  while (threads < kMaxThreads && threads * kHeld < rows * per_head) threads *= 2;
  const int64_t units = 2ll * p.B * p.slots * p.cache.kv_heads;
  p.q_items = p.q.heads > 0 ? rotation_items<V>(p.q.heads, HEADS, p.cache.head_dim) : 1;
  const int64_t q_ctas = p.q.heads > 0 ? (static_cast<int64_t>(p.N) * p.q_items + threads - 1) / threads : 0;
  return launch_pdl(kv_append_kernel<T, V, HEADS>, dim3(static_cast<unsigned>(units + q_ctas)), dim3(threads), 0, s, p);
}

template <typename T, int V>
cudaError_t launch(const KvAppendParams& p, cudaStream_t s) {
  return static_cast<int64_t>(p.N) * rotation_items<V>(p.q.heads, 1, p.cache.head_dim) >= kManyItems ? launch_heads<T, V, 2>(p, s)
                                                                                                     : launch_heads<T, V, 1>(p, s);
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
