// Rotary positions: q and k rotated in one launch.
//
// For each pair (u, w) of a head and its frequency i at position p:
//   u' = u cos(p f_i) - w sin(p f_i),  w' = w cos(p f_i) + u sin(p f_i),
// cos and sin from a float32 table that was made in float64 (an angle p f_i
// in float32 is off by p f_i 2^-24, a tenth of a radian at a million).  The
// gradient is the transposed rotation: the same with -sin.
//
// What bounds it: bytes, each read and written once.  A thread takes one
// stretch of one head (two 16-byte loads): 4096 tokens of 36 heads of 128 take
// 14.6 us cold, 78 MB at 5.3 TB/s, 78% of the copy rate.  Two, four heads a
// thread to share its angles 15.1, 20.8 us: they come from the first-level
// cache anyway, and fewer threads keep fewer loads on their way.
#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;

// A thread a stretch of a head.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) rope_kernel(RopeParams p, uint32_t per_token) {
  pdl_launch_dependents();
  pdl_wait();
  const RotationItem<T, V, 1> x(p.q, p.k, blockIdx.x * kThreads + threadIdx.x, per_token, p.N, p.D, p.R, p.interleaved);
  if (!x.live) return;
  int pos = p.positions[x.t];
  if (pos < 0 || pos >= p.num_positions) {
    set_status(p.status, MOE_ERR_BAD_POSITION);
    pos = kUnturned;
  }
  x.finish(p.q, p.k, pos, p.R, p.interleaved, p.inverse, p.cos_sin);
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, cudaStream_t s) {
  const uint32_t per_token = rotation_items<V>(p.q.heads + p.k.heads, 1, p.D);
  const int64_t ctas = (static_cast<int64_t>(p.N) * per_token + kThreads - 1) / kThreads;
  return launch_pdl(rope_kernel<T, V>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, p, per_token);
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
