// Rotary positions: q and k rotated in one launch.
//
// For each pair (u, w) of a head and its frequency i at position p:
//   u' = u cos(p f_i) - w sin(p f_i),  w' = w cos(p f_i) + u sin(p f_i),
// cos and sin from a float32 table that was made in float64 (an angle p f_i
// in float32 is off by p f_i 2^-24, a tenth of a radian at a million).  The
// gradient is the transposed rotation: the same with -sin.
#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

// One CTA a token; a thread takes one stretch of one head at a time.
template <typename T, int V>
__global__ void rope_kernel(RopeParams p) {
  pdl_wait();
  const int per_head = p.D / (2 * V);
  const int items = (p.q.heads + p.k.heads) * per_head;
  for (int64_t t = blockIdx.x; t < p.N; t += gridDim.x) {
    const int pos = p.positions[t];
    const bool known = pos >= 0 && pos < p.num_positions;
    if (!known && threadIdx.x == 0) set_status(p.status, MOE_ERR_BAD_POSITION);
    const float* row = p.cos_sin + static_cast<int64_t>(known ? pos : 0) * p.R;
    for (int j = threadIdx.x; j < items; j += blockDim.x) {
      const int h = j / per_head, c = j - h * per_head;
      const bool is_q = h < p.q.heads;
      const RopeTensor& x = is_q ? p.q : p.k;
      const int hh = is_q ? h : h - p.q.heads;
      const T* in = static_cast<const T*>(x.in) + t * x.in_token + hh * x.in_head;
      T* out = static_cast<T*>(x.out) + t * x.out_token + hh * x.out_head;
      const Stretch<V> s(c, p.R, p.interleaved);
      float a[V], b[V];
      load_f32<T, V>(in + s.a, a);
      load_f32<T, V>(in + s.b, b);
      if (s.turned && known) {
        float cs[V], sn[V];
        load_cos_sin<V>(row, c, p.R, cs, sn);
        if (p.inverse) {
#pragma unroll
          for (int i = 0; i < V; ++i) sn[i] = -sn[i];
        }
        rotate<V>(a, b, cs, sn, p.interleaved);
      }
      store_f32<T, V>(out + s.a, a);
      store_f32<T, V>(out + s.b, b);
    }
  }
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  const int items = (p.q.heads + p.k.heads) * (p.D / (2 * V));
  const int threads = items >= 1024 ? 1024 : (items + 31) / 32 * 32;
  return launch_pdl(rope_kernel<T, V>, dim3(static_cast<unsigned>(p.N)), dim3(threads), 0, s, p);
}

template <typename T>
cudaError_t launch_v(const RopeParams& p, int V, cudaStream_t s) {
  if (V >= 8) return launch<T, 8>(p, s);
  if (V == 4) return launch<T, 4>(p, s);
  return launch<T, 1>(p, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, int V, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F32) return V >= 4 ? launch<float, 4>(p, s) : launch<float, 1>(p, s);
  if (dtype == MOE_DTYPE_F16) return launch_v<__half>(p, V, s);
  return launch_v<__nv_bfloat16>(p, V, s);
}

}  // namespace moe
