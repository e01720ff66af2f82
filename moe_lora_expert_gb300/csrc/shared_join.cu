// The last step of attention over shared prefixes: for each row that takes
// part, the prefix pass's pieces and the own pass's sums become its output.
//
// With piece i's reference m_i, denominator l_i and sums O_i (relative to 2^m_i),
//   out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,  m = max_i m_i.
// A warp a row, a lane four columns; 16 pieces' loads are on their way together.
// What bounds it: the pieces' bytes, from the second-level cache.  2048 rows of
// 8 pieces take 3 us of a call, 8 by themselves from cold caches.
#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kAtOnce = 16;
constexpr float kLn2 = 0.6931471805599453f;

template <typename T>
__global__ void __launch_bounds__(32 * kWarps) shared_join_kernel(const __grid_constant__ AttentionParams a, const __grid_constant__ AttentionForms f,
                                                                  uint32_t rows_each) {
  pdl_launch_dependents();
  // what the caller has given is there since the prefix pass has begun
  const int lane = threadIdx.x & 31, col = 4 * lane, D = a.cache.head_dim;
  const uint32_t r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int b = static_cast<int>(r / rows_each), in = static_cast<int>(r - b * rows_each), t = in / a.Hq, h = in - t * a.Hq;
  int tok = 0, g = 0, count = 0;
  if (b < a.B) {
    const int q_first = a.cu_q == nullptr ? b : a.cu_q[b], q_len = a.cu_q == nullptr ? 1 : a.cu_q[b + 1] - q_first;
    tok = q_first + t;
    if (t < min(min(q_len, a.max_q_len), a.N - q_first)) count = f.taken(a.cu_q, b, q_first, q_len, a.seq_lens[b] - q_len, g) > 0;
  }
  pdl_wait();
  if (count == 0) return;
  count = min(__ldcg(f.pieces + g), f.most_pieces);
  const int64_t row = static_cast<int64_t>(tok) * a.Hq + h;
  const float2* refs = f.refs + row;
  const float* sums = f.sums + row * D + col;
  const int64_t step = f.rows * D;
  const bool live = col < D;

  // the own pass's first
  const float2 own = __ldcg(refs + f.most_pieces * f.rows);
  float4 acc = live ? __ldcg(reinterpret_cast<const float4*>(sums + f.most_pieces * step)) : make_float4(0, 0, 0, 0);
  float m = own.x, l = own.y;
#pragma unroll 1
  for (int i = 0; i < count; i += kAtOnce) {
    float4 v[kAtOnce];
    float2 z = make_float2(-INFINITY, 0.f);                // lane k's is piece i + k's
    if (lane < kAtOnce && i + lane < count) z = __ldcg(refs + (i + lane) * f.rows);
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      v[k] = live && i + k < count ? __ldcg(reinterpret_cast<const float4*>(sums + (i + k) * step)) : make_float4(0, 0, 0, 0);
    float top = z.x;
#pragma unroll
    for (int x = 1; x < kAtOnce; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    top = fmaxf(m, __shfl_sync(0xffffffffu, top, 0));
    const float base = top == -INFINITY ? 0.f : top, keep = fast_exp2(m - base), e = fast_exp2(z.x - base);
    float part = z.y * e;
#pragma unroll
    for (int x = 1; x < kAtOnce; x *= 2) part += __shfl_xor_sync(0xffffffffu, part, x);
    l = fmaf(l, keep, __shfl_sync(0xffffffffu, part, 0));
    acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const float w = __shfl_sync(0xffffffffu, e, k);
      acc.x = fmaf(v[k].x, w, acc.x);
      acc.y = fmaf(v[k].y, w, acc.y);
      acc.z = fmaf(v[k].z, w, acc.z);
      acc.w = fmaf(v[k].w, w, acc.w);
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const float y[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  if (live) store_f32<T, 4>(static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head + col, y);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

namespace {
int64_t rows_each_of(const AttentionParams& p) { return static_cast<int64_t>(p.max_q_len) * p.Hq; }
int64_t ctas_of(const AttentionParams& p) { return (rows_each_of(p) * p.B + kWarps - 1) / kWarps; }
}  // namespace

bool shared_join_fits(const AttentionParams& p) { return ctas_of(p) <= 0x7fffffff / kWarps; }

int launch_shared_join(const AttentionParams& p, const AttentionForms& forms, int dtype, cudaStream_t s) {
  if (!shared_join_fits(p)) return MOE_ERR_UNSUPPORTED;
  const int64_t rows_each = rows_each_of(p), ctas = ctas_of(p);
  const dim3 grid(static_cast<unsigned>(ctas)), block(32 * kWarps);
  const cudaError_t e = dtype == MOE_DTYPE_F16
                            ? launch_pdl(shared_join_kernel<__half>, grid, block, 0, s, p, forms, static_cast<uint32_t>(rows_each))
                            : launch_pdl(shared_join_kernel<__nv_bfloat16>, grid, block, 0, s, p, forms, static_cast<uint32_t>(rows_each));
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
