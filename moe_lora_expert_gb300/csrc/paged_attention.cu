// Attention over the paged cache, one warp for each (token, query head): the
// definition written down, for every size and mask.  A lane holds four
// columns of the head; a running maximum and sum make one pass over the keys.
#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

template <typename T>
__global__ void attention_rows_kernel(AttentionParams p) {
  pdl_wait();
  const moe_kv_cache_t& ca = p.cache;
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / p.Hq), h = static_cast<int>(w - static_cast<int64_t>(t) * p.Hq);
  if (t >= p.N) return;
  int b = t, t0 = t, t1 = t + 1;
  if (p.cu_q != nullptr) {
    if (t >= p.cu_q[p.B]) return;
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    b = lo;
    t0 = p.cu_q[b];
    t1 = p.cu_q[b + 1];
  }
  const int at = p.seq_lens[b] - (t1 - t0) + (t - t0);      // position of this row
  const int first = p.window > 0 && at + 1 > p.window ? at + 1 - p.window : 0;
  const int head = h / (p.Hq / ca.kv_heads), d = 4 * lane;
  const bool mine = d < ca.head_dim;
  float q[4] = {}, o[4] = {};
  if (mine) load_f32<T, 4>(static_cast<const T*>(p.q) + t * p.q_token + h * p.q_head + d, q);
  float top = -INFINITY, sum = 0.f;
  for (int j = first; j <= at; ++j) {
    const int page_at = j / ca.page_size, off = j - page_at * ca.page_size;
    const int page = page_at < p.table_width ? p.block_table[static_cast<int64_t>(b) * p.table_width + page_at] : -1;
    if (page < 0 || page >= ca.num_pages) {
      set_status(p.status, MOE_ERR_BAD_PAGE);
      continue;
    }
    float k[4] = {}, v[4] = {};
    if (mine) {
      const uint2 kv = make_uint2(
          *reinterpret_cast<const uint32_t*>(ca.k + page * ca.k_stride_page + head * ca.k_stride_head + off * ca.k_stride_token + d),
          *reinterpret_cast<const uint32_t*>(ca.v + page * ca.v_stride_page + head * ca.v_stride_head + off * ca.v_stride_token + d));
      const float2 k0 = e4m3x2_to_f32x2(kv.x & 0xFFFF), k1 = e4m3x2_to_f32x2(kv.x >> 16);
      const float2 v0 = e4m3x2_to_f32x2(kv.y & 0xFFFF), v1 = e4m3x2_to_f32x2(kv.y >> 16);
      k[0] = k0.x; k[1] = k0.y; k[2] = k1.x; k[3] = k1.y;
      v[0] = v0.x; v[1] = v0.y; v[2] = v1.x; v[3] = v1.y;
    }
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    const int64_t sc = static_cast<int64_t>(page) * ca.kv_heads + head;
    s *= p.scale * ca.k_scale[sc];
    const float now = fmaxf(top, s);
    const float keep = top == -INFINITY ? 0.f : expf(top - now), e = s == -INFINITY ? 0.f : expf(s - now);  // NaN stays
    const float ev = e * ca.v_scale[sc];
    sum = sum * keep + e;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + ev * v[i];
    top = now;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] *= inv;
  if (mine) store_f32<T, 4>(static_cast<T*>(p.out) + t * p.out_token + h * p.out_head + d, o);
  if (lane == 0 && p.lse != nullptr) p.lse[static_cast<int64_t>(t) * p.Hq + h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_paged_attention(const AttentionParams& p, int dtype, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(p.N) * p.Hq;
  const dim3 grid(static_cast<unsigned>((warps + 3) / 4));
  if (dtype == MOE_DTYPE_F16) return launch_pdl(attention_rows_kernel<__half>, grid, dim3(128), 0, s, p);
  return launch_pdl(attention_rows_kernel<__nv_bfloat16>, grid, dim3(128), 0, s, p);
}

}  // namespace moe
