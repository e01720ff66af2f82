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

// The same with an axis for each pair: a token has a position on each axis.
// Finding the angles takes more then, and the CTA gathers those of its tokens:
// 4096 tokens of 36 heads of 128 take 19.9 us, whatever the axes' order (by each
// thread for itself 24 with a run of pairs for each axis, 33 with axes in turns;
// by each warp for its own tokens 21.9 and 23.2).  Bytes would take 11.5; half
// of the warp slots are empty for want of registers (63 a thread, 40 in the
// kernel above), and a warp waits for positions, angles and the others.  128
// threads: 256 20.2, 512 21.1 us; one head a thread 25.3, four 26.7.
constexpr int kAxesThreads = 128;
constexpr int kAxesHeads = 2;              // of a thread
constexpr int kAxesCtas = 8;
template <typename T, int V>
__global__ void __launch_bounds__(kAxesThreads, kAxesCtas) rope_axes_kernel(RopeParams p, const __grid_constant__ RopeAxes axes, uint32_t per_token) {
  extern __shared__ __align__(16) float angles[];      // [tokens][R], then whether each token has any
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t item0 = blockIdx.x * kAxesThreads, t0 = item0 / per_token;
  const RotationItem<T, V, kAxesHeads> x(p.q, p.k, item0 + threadIdx.x, per_token, p.N, p.D, p.R, p.interleaved);
  const int tokens = static_cast<int>(min((item0 + kAxesThreads - 1) / per_token + 1, static_cast<uint32_t>(p.N)) - t0);
  int* good = reinterpret_cast<int*>(angles + axes_tokens(kAxesThreads, per_token) * p.R);
  gather_angles(angles, good, axes, p.positions, p.cos_sin, t0, tokens, p.R, p.num_positions);
  __syncthreads();
  if (!x.live) return;
  const int j = static_cast<int>(x.t - t0);
  if (!good[j]) set_status(p.status, MOE_ERR_BAD_POSITION);
  x.turn_by(p.q, p.k, good[j] ? angles + j * p.R : nullptr, p.R, p.interleaved, p.inverse);
}

template <typename T, int V>
cudaError_t launch_axes(const RopeParams& p, const RopeAxes& axes, cudaStream_t s) {
  const uint32_t per_token = rotation_items<V>(p.q.heads + p.k.heads, kAxesHeads, p.D);
  const int64_t ctas = (static_cast<int64_t>(p.N) * per_token + kAxesThreads - 1) / kAxesThreads;
  // at most 17 KB: a token has R / 2V stretches at least, or one
  const size_t bytes = static_cast<size_t>(axes_tokens(kAxesThreads, per_token)) * (p.R + 1) * 4;
  return launch_pdl(rope_axes_kernel<T, V>, dim3(static_cast<unsigned>(ctas)), dim3(kAxesThreads), bytes, s, p, axes, per_token);
}

template <typename T, int V>
cudaError_t launch(const RopeParams& p, const RopeAxes* axes, cudaStream_t s) {
  const uint32_t per_token = rotation_items<V>(p.q.heads + p.k.heads, 1, p.D);
  if (axes != nullptr) return launch_axes<T, V>(p, *axes, s);
  const int64_t ctas = (static_cast<int64_t>(p.N) * per_token + kThreads - 1) / kThreads;
  return launch_pdl(rope_kernel<T, V>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, s, p, per_token);
}

template <typename T>
cudaError_t launch_v(const RopeParams& p, const RopeAxes* axes, int V, cudaStream_t s) {
  if (V >= 8) return launch<T, 8>(p, axes, s);
  if (V == 4) return launch<T, 4>(p, axes, s);
  return launch<T, 1>(p, axes, s);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, const RopeAxes* axes, int dtype, int V, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F32) return V >= 4 ? launch<float, 4>(p, axes, s) : launch<float, 1>(p, axes, s);
  if (dtype == MOE_DTYPE_F16) return launch_v<__half>(p, axes, V, s);
  return launch_v<__nv_bfloat16>(p, axes, V, s);
}

}  // namespace moe
