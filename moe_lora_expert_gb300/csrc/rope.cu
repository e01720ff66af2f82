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
// Finding the angles takes more then: a CTA has whole tokens, gathers their
// angles together, and nothing is divided: threadIdx is (stretch, head, token).
constexpr int kAxesThreads = 256;          // of a CTA, about
constexpr int kAxesHeads = 1;              // of a thread
constexpr int kAxesMost = 512, kAxesCtas = 3;
template <typename T, int V>
__global__ void __launch_bounds__(kAxesMost, kAxesCtas) rope_axes_kernel(RopeParams p, const __grid_constant__ RopeAxes axes) {
  extern __shared__ __align__(16) float angles[];      // [tokens][R], then whether each token has any
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * blockDim.z, tokens = min(static_cast<int>(blockDim.z), p.N - t0), z = threadIdx.z;
  const int c = threadIdx.x, heads = z < tokens ? p.q.heads + p.k.heads : 0, step = gridDim.y * blockDim.y;
  const int h0 = blockIdx.y * blockDim.y + threadIdx.y;
  const int64_t t = t0 + z;
  int* good = reinterpret_cast<int*>(angles + blockDim.z * p.R);
  Pack<T, V> ra[kAxesHeads], rb[kAxesHeads];
  const Stretch<V> s(c, p.R, p.interleaved);
#pragma unroll
  for (int u = 0; u < kAxesHeads; ++u) {
    const int h = h0 + u * step;
    if (h >= heads) break;
    const T* in = h < p.q.heads ? static_cast<const T*>(p.q.in) + t * p.q.in_token + h * p.q.in_head
                                : static_cast<const T*>(p.k.in) + t * p.k.in_token + (h - p.q.heads) * p.k.in_head;
    ra[u] = *reinterpret_cast<const Pack<T, V>*>(in + s.a);
    rb[u] = *reinterpret_cast<const Pack<T, V>*>(in + s.b);
  }
  gather_angles(angles, good, axes, p.positions, p.cos_sin, t0, tokens, p.R, p.num_positions);
  __syncthreads();
  if (h0 >= heads) return;
  const bool turn = s.turned && good[z];
  if (!good[z]) set_status(p.status, MOE_ERR_BAD_POSITION);
  float cs[V], sn[V];
  if (turn) {
    load_cos_sin<V>(angles + z * p.R, c, p.R, cs, sn);
    if (p.inverse) {
#pragma unroll
      for (int i = 0; i < V; ++i) sn[i] = -sn[i];
    }
  }
#pragma unroll
  for (int u = 0; u < kAxesHeads; ++u) {
    const int h = h0 + u * step;
    if (h >= heads) break;
    float a[V], b[V];
    to_f32s<T, V>(ra[u], a);
    to_f32s<T, V>(rb[u], b);
    if (turn) rotate<V, false>(a, b, cs, sn, p.interleaved);
    T* out = h < p.q.heads ? static_cast<T*>(p.q.out) + t * p.q.out_token + h * p.q.out_head
                           : static_cast<T*>(p.k.out) + t * p.k.out_token + (h - p.q.heads) * p.k.out_head;
    store_f32<T, V>(out + s.a, a);
    store_f32<T, V>(out + s.b, b);
  }
}

template <typename T, int V>
cudaError_t launch_axes(const RopeParams& p, const RopeAxes& axes, cudaStream_t s) {
  const uint32_t across = p.D / (2 * V);                                       // 512 at most
  const uint32_t heads = (p.q.heads + p.k.heads + kAxesHeads - 1) / kAxesHeads;
  const uint32_t most = kAxesMost / across, ctas = (heads + most - 1) / most, rows = (heads + ctas - 1) / ctas;
  uint32_t tokens = kAxesThreads / (across * rows);
  tokens = tokens < 1 ? 1 : tokens > 64 ? 64 : tokens;
  const dim3 grid((static_cast<uint32_t>(p.N) + tokens - 1) / tokens, ctas);
  return launch_pdl(rope_axes_kernel<T, V>, grid, dim3(across, rows, tokens), static_cast<size_t>(tokens) * (p.R + 1) * 4, s, p, axes);
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
