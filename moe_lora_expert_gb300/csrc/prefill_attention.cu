// Attention of many new tokens over the paged cache, on tcgen05.
//
// A CTA takes 256 rows (new tokens x query heads of one key head's group) as
// two tiles of 128 and walks the keys they see in tiles of 128:
//   S = Q K^T (TMEM), P = 2^(S k_scale' + log2 v_scale - m) (float16, back into
//   S's columns), O += P V (TMEM), with the running maximum m of a softmax.
// The weights carry the pages' value scales, as in decode_attention.cu, so K
// and V enter the tensor cores as the codes themselves.  A code is exact in
// float16; four warps convert each tile once for both row tiles, from where
// the TMA put its bytes to the layout that tcgen05.mma reads.  (Feeding e4m3
// directly would need q and P as sums of three e4m3 parts each to keep their
// precision: 1.5 times the float16 work and the splitting of every weight.)
//
// Warps: 0-3 and 4-7 the softmax of a row tile each, a thread a row; 8-11
// convert; 12 issues the products; 13 looks up pages and issues the copies.
// While one row tile is in its softmax the tensor cores work for the other.
#include <cuda.h>

#include <type_traits>

#include "attention.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kKeys = 128;
constexpr int kTileRows = 128;
constexpr int kCtaRows = 256;
constexpr int kThreads = 512;
constexpr int kSlots = 4;                  // converted tiles: K0, V0, K1, V1, ...
constexpr int kStages = 2;                 // tiles of codes, in the same order
constexpr int kInfo = 8;                   // key tiles whose scales are held
constexpr int kConvertWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;

struct alignas(16) Group {                 // 8 keys, which lie in one page
  float k, lv, inv_v;
  int valid;
};

struct Control {
  Group group[kInfo][kKeys / 8];
  uint64_t code_full[kStages], code_empty[kStages], full[kSlots], empty[kSlots];
  uint64_t info_full[kInfo], q_full, s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int abort_flag, nan_seen;
};

template <int DP>
struct Layout {
  static constexpr int kHalves = DP / 64;
  static constexpr int kHalfBytes = kKeys * 128;                  // 128 keys (or rows) x 64 float16
  static constexpr int kSlotBytes = kHalves * kHalfBytes;
  static constexpr int kQBytes = 2 * kHalves * kHalfBytes;
  static constexpr int kCodeBytes = kKeys * 128;
  static constexpr int kQ = 0, kRing = kQBytes, kCode = kRing + kSlots * kSlotBytes,
                       kControl = kCode + kStages * kCodeBytes, kBytes = kControl + static_cast<int>(sizeof(Control));
};
static_assert(Layout<128>::kBytes <= 232448, "shared memory of a CTA");

struct Launch {
  AttentionParams a;
  int row_tiles;                           // of 256, of the longest sequence
  int box;                                 // keys of one TMA box: gcd(page_size, 128)
};

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// V as the B operand with its columns contiguous: 64-column halves kHalfBytes
// apart (leading offset), groups of 8 keys 1024 bytes apart (stride offset).
__device__ __forceinline__ uint64_t mn_major_sdesc(uint32_t saddr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(half_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
__device__ __forceinline__ void mma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 lanes x 32 columns; the registers are valid after tmem_wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ kernel
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
prefill_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const Launch p) {
  using L = Layout<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& s = *reinterpret_cast<Control*>(smem + L::kControl);
  const AttentionParams& a = p.a;
  const moe_kv_cache_t& ca = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / ca.kv_heads;
  pdl_wait();

  // Row tiles from a sequence's end first: they see the most keys.
  int u = blockIdx.x;
  const int head = u % ca.kv_heads;
  u /= ca.kv_heads;
  const int b = u % a.B, row0 = (p.row_tiles - 1 - u / a.B) * kCtaRows;
  const int q_first = a.cu_q == nullptr ? b : a.cu_q[b];
  const int q_len = a.cu_q == nullptr ? 1 : a.cu_q[b + 1] - q_first;
  const int n_rows = min(min(q_len, a.max_q_len), a.N - q_first) * group - row0;
  if (n_rows <= 0) return;
  const int rows = min(n_rows, kCtaRows), tiles = rows > kTileRows ? 2 : 1;
  const int start = a.seq_lens[b] - q_len;
  auto position = [&](int row) { return start + (row0 + row) / group; };
  const int lo = a.window > 0 ? max(0, position(0) + 1 - a.window) : 0;
  const int64_t most = static_cast<int64_t>(a.table_width) * ca.page_size;
  int end = max(0, position(rows - 1) + 1);
  if (end > most) {
    if (tid == 0) set_status(a.status, MOE_ERR_BAD_PAGE);
    end = static_cast<int>(most);
  }
  const int tile0 = lo / kKeys, n = end > lo ? (end + kKeys - 1) / kKeys - tile0 : 0;
  // Whether every row in [r0, r1] sees every key of the tile (if its pages are there).
  auto whole = [&](int tile, int r0, int r1) {
    const int key0 = tile * kKeys;
    return key0 + kKeys - 1 <= position(r0) && (a.window == 0 || key0 > position(r1) - a.window);
  };

  if (tid == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.code_full[i], 1);
      mbar_init(&s.code_empty[i], 4);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s.full[i], 4);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(&s.info_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], kTileRows);
      mbar_init(&s.o_full[i], 1);
    }
    mbar_init(&s.q_full, 2 * kTileRows);
    mbar_init(&s.drained, 1);
    s.abort_flag = 0;
    s.nan_seen = 0;
    fence_mbarrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s.tmem;
  auto s_cols = [&](int i) { return tmem + 128 * i; };
  auto o_cols = [&](int i) { return tmem + 256 + 128 * i; };

  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(smem_u32(bar), parity) || *static_cast<volatile int*>(&s.abort_flag)) return;
    if (!mbar_wait(bar, parity, a.wait_limit_ns)) {
      set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
      *static_cast<volatile int*>(&s.abort_flag) = 1;
    }
  };

  if (warp == kLoadWarp) {
    // ------------------------------------------------ pages, scales, copies
    struct Ahead {
      int page, off;
      Group g;
    };
    auto find = [&](int j) {
      Ahead f = {-1, 0, {0.f, 0.f, 0.f, 0}};
      const int key = (tile0 + j) * kKeys + 8 * (lane & 15);
      if (j < n && key < end && (key & ~(p.box - 1)) + p.box > lo) {
        const int page_at = key / ca.page_size;
        f.off = key - page_at * ca.page_size;
        f.page = a.block_table[static_cast<int64_t>(b) * a.table_width + page_at];
        if (f.page < 0 || f.page >= ca.num_pages) {
          f.page = -1;
          set_status(a.status, MOE_ERR_BAD_PAGE);
        } else {
          const int64_t i = static_cast<int64_t>(f.page) * ca.kv_heads + head;
          const float vs = fmaxf(ca.v_scale[i], 5.421010862427522e-20f);   // 2^-64: a zero scale gives zero values
          f.g = {ca.k_scale[i] * fabsf(a.scale) * kLog2e, log2f(vs), 1.f / vs, 1};
        }
      }
      return f;
    };
    const bool stalled = (a.debug_flags & MOE_DEBUG_STALL_ATTENTION) != 0;   // a failure for the tests: no tile arrives
    auto aborted = [&] { return *static_cast<volatile int*>(&s.abort_flag) != 0; };
    int issued = 0;
    Ahead now = find(0);
    for (int j = 0; j < n && !stalled && !aborted(); ++j) {
      const Ahead next = find(j + 1);
      if (lane < 16) s.group[j % kInfo][lane] = now.g;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.info_full[j % kInfo]);
      const bool issues = lane < 16 && now.page >= 0 && (8 * lane) % p.box == 0;
      const unsigned boxes = __ballot_sync(0xffffffffu, issues);
      for (int v = 0; v < 2; ++v) {
        const int k = 2 * j + v, st = k % kStages;
        if (k >= kStages) wait(&s.code_empty[st], (k / kStages - 1) & 1);
        if (__any_sync(0xffffffffu, aborted())) break;               // a stage that was not freed is not filled again
        issued = k + 1;
        if (lane == 0) mbar_arrive_expect_tx(&s.code_full[st], __popc(boxes) * p.box * 128);
        __syncwarp();
        if (issues)
          tma_load_4d(smem_u32(smem + L::kCode + st * L::kCodeBytes) + 8 * lane * 128, v == 0 ? &k_map : &v_map, &s.code_full[st],
                      now.off, head, now.page);
      }
      now = next;
    }
    if (aborted())                                                   // nothing of this CTA stays in flight
      for (int k = max(0, issued - kStages); k < issued; ++k) mbar_wait(&s.code_full[k % kStages], (k / kStages) & 1, a.wait_limit_ns);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0 && n > 0) {
      constexpr uint32_t kScores = idesc_f16(kTileRows, kKeys, false), kValues = idesc_f16(kTileRows, DP, true);
      const uint32_t q_base = smem_u32(smem + L::kQ), ring = smem_u32(smem + L::kRing);
      auto scores = [&](int i, int slot) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t at = (k / 4) * L::kHalfBytes + (k % 4) * 32;
          tc_mma_bf16(s_cols(i), make_sdesc_sw128(q_base + i * L::kHalves * L::kHalfBytes + at),
                      make_sdesc_sw128(ring + slot * L::kSlotBytes + at), kScores, k > 0);
        }
      };
      auto values = [&](int i, int slot, bool more) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts_f16(o_cols(i), s_cols(i) + 8 * k, mn_major_sdesc(ring + slot * L::kSlotBytes + 2048 * k, L::kHalfBytes), kValues,
                     more || k > 0);
      };
      wait(&s.q_full, 0);
      wait(&s.full[0], 0);
      tc_fence_after_sync();
      for (int i = 0; i < tiles; ++i) {
        scores(i, 0);
        tc_commit(&s.s_full[i]);
      }
      tc_commit(&s.empty[0]);
      for (int j = 0; j < n; ++j) {
        const int v = 2 * j + 1, k = 2 * j + 2;
        wait(&s.full[v % kSlots], (v / kSlots) & 1);
        for (int i = 0; i < tiles; ++i) {
          wait(&s.p_full[i], j & 1);
          tc_fence_after_sync();
          values(i, v % kSlots, j > 0);
          if (i == tiles - 1) tc_commit(&s.empty[v % kSlots]);
          if (j + 1 < n) {
            if (i == 0) {
              wait(&s.full[k % kSlots], (k / kSlots) & 1);
              tc_fence_after_sync();
            }
            scores(i, k % kSlots);
            tc_commit(&s.s_full[i]);
            if (i == tiles - 1) tc_commit(&s.empty[k % kSlots]);
          } else {
            tc_commit(&s.o_full[i]);
          }
        }
      }
      tc_commit(&s.drained);
      mbar_wait(&s.drained, 0, a.wait_limit_ns);
    }
    __syncwarp();
  } else if (warp >= kConvertWarp && warp < kConvertWarp + 4) {
    // --------------------------------------------------------- conversion
    // A lane converts 16 codes to two 16-byte chunks.  Eight lanes at a time
    // take four chunks of keys k and k ^ 5, which fall on distinct banks for
    // both the load and the stores.
    const int w = warp - kConvertWarp, sub = lane & 3, key8 = (lane >> 3) ^ (5 * ((lane >> 2) & 1));
    for (int k = 0; k < 2 * n; ++k) {
      const int st = k % kStages, slot = k % kSlots;
      wait(&s.code_full[st], (k / kStages) & 1);
      if (k >= kSlots) wait(&s.empty[slot], (k / kSlots - 1) & 1);
      const uint8_t* src = smem + L::kCode + st * L::kCodeBytes;
      uint8_t* dst = smem + L::kRing + slot * L::kSlotBytes;
      // a weight of zero times a NaN code would be NaN: where some row does
      // not see some key, NaN values are left out here and added at the end
      bool drop = false;
      if ((k & 1) != 0) {
        drop = !whole(tile0 + k / 2, 0, rows - 1);
        const int ok = lane < 16 ? s.group[(k / 2) % kInfo][lane].valid : 1;
        drop = !__all_sync(0xffffffffu, ok) || drop;
      }
      uint32_t nan = 0;
      auto counts = [&](int key) {         // some row sees it
        const int at = (tile0 + k / 2) * kKeys + key;
        return at >= lo && at < end && s.group[(k / 2) % kInfo][key >> 3].valid;
      };
#pragma unroll 4
      for (int it = w; it < 16 * L::kHalves; it += 4) {
        const int key = 8 * (it / L::kHalves) + key8, half = it % L::kHalves, x = key & 7;
        uint4 c = *reinterpret_cast<const uint4*>(src + key * 128 + (((4 * half + sub) ^ x) * 16));
        if (drop) {
          uint32_t* cw = &c.x;
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const uint32_t bad = __vcmpeq4(cw[z] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
            nan |= bad != 0 && counts(key) ? 1 : 0;
            cw[z] &= ~bad;
          }
        }
        uint4 f0, f1;
        e4m3x4_to_f16x4(c.x, f0.x, f0.y);
        e4m3x4_to_f16x4(c.y, f0.z, f0.w);
        e4m3x4_to_f16x4(c.z, f1.x, f1.y);
        e4m3x4_to_f16x4(c.w, f1.z, f1.w);
        uint8_t* to = dst + half * L::kHalfBytes + key * 128;
        *reinterpret_cast<uint4*>(to + (((2 * sub) ^ x) * 16)) = f0;
        *reinterpret_cast<uint4*>(to + (((2 * sub + 1) ^ x) * 16)) = f1;
      }
      if (nan != 0) *static_cast<volatile int*>(&s.nan_seen) = 1;
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s.code_empty[st]);
        mbar_arrive(&s.full[slot]);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2, row = kTileRows * i + 32 * (warp & 3) + lane;
    const bool live = row < rows;
    const int pos = live ? position(row) : -1;
    const int gr = row0 + row, tok = q_first + gr / group, h = head * group + gr % group;

    // Q in float16, a power of two taken out of bf16 rows, in the layout of
    // the A operand.
    float row_scale = 1.f;
    {
      const T* src = static_cast<const T*>(a.q) + tok * a.q_token + h * a.q_head;
      float inv = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
        float amax = 0.f;
#pragma unroll 4
        for (int d = 0; d < ca.head_dim; d += 8) {
          float v[8] = {};
          if (live) load_f32<T, 8>(src + d, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(v[e]));
        }
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        if (ex > -120 && ex < 120) {
          row_scale *= __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
          inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        }
      }
      if (a.scale < 0.f) inv = -inv;       // the sign goes into q, so that a larger score is a larger weight
      const int r = row & 127, x = r & 7;
      uint8_t* dst = smem + L::kQ + i * L::kHalves * L::kHalfBytes + r * 128;
#pragma unroll 4
      for (int d = 0; d < DP; d += 8) {
        float v[8] = {};
        if (live && d < ca.head_dim) load_f32<T, 8>(src + d, v);
        uint4 f;
        f.x = f32x2_to_f16x2(v[0] * inv, v[1] * inv);
        f.y = f32x2_to_f16x2(v[2] * inv, v[3] * inv);
        f.z = f32x2_to_f16x2(v[4] * inv, v[5] * inv);
        f.w = f32x2_to_f16x2(v[6] * inv, v[7] * inv);
        *reinterpret_cast<uint4*>(dst + (d / 64) * L::kHalfBytes + ((((d / 8) & 7) ^ x) * 16)) = f;
      }
      fence_proxy_async_shared();
      mbar_arrive(&s.q_full);
    }

    float m = -INFINITY, base = 0.f, l = 0.f;    // base: m, or 0 while there is none
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t sc = s_cols(i) + lanes, oc = o_cols(i) + lanes;
    if (i < tiles) {
      const int r0 = kTileRows * i, r1 = min(rows, r0 + kTileRows) - 1;
      for (int j = 0; j < n; ++j) {
        const int key0 = (tile0 + j) * kKeys;
        const Group* info = s.group[j % kInfo];
        wait(&s.info_full[j % kInfo], (j / kInfo) & 1);
        const bool all = __all_sync(0xffffffffu, lane < 16 ? info[lane].valid : 1) && whole(tile0 + j, r0, r1);
        wait(&s.s_full[i], j & 1);
        tc_fence_after_sync();

        auto seen = [&](int key, int valid) { return valid && key <= pos && (a.window == 0 || key > pos - a.window); };
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(sc + 32 * c, r);
          tmem_wait(r);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const Group gi = info[4 * c + g];
            float t = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x = __uint_as_float(r[8 * g + e]);
              t = all || seen(key0 + 32 * c + 8 * g + e, gi.valid) ? fmaxf(t, x) : t;
            }
            top = fmaxf(top, t == -INFINITY ? t : fmaf(t, gi.k * row_scale, gi.lv));
          }
        }
        if (__any_sync(0xffffffffu, top > m + kSlack)) {
          const float now = fmaxf(m, top);
          const float keep = m == -INFINITY ? 0.f : fast_exp2(m - now);
          m = now;
          base = now == -INFINITY ? 0.f : now;
          l *= keep;
          if (j > 0) {       // O holds the products up to tile j - 1: they came before these scores
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {
              uint32_t r[32];
              tmem_ld32(oc + 32 * c, r);
              tmem_wait(r);
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * keep);
              tmem_st32(oc + 32 * c, r);
            }
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32], w[16];
          tmem_ld32(sc + 32 * c, r);
          tmem_wait(r);
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const Group gi = info[4 * c + g];
            const float kk = gi.k * row_scale, off = gi.lv - base;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              float y0 = fmaf(__uint_as_float(r[8 * g + e]), kk, off), y1 = fmaf(__uint_as_float(r[8 * g + e + 1]), kk, off);
              if (!all) {
                const int key = key0 + 32 * c + 8 * g + e;
                if (!seen(key, gi.valid)) y0 = -INFINITY;
                if (!seen(key + 1, gi.valid)) y1 = -INFINITY;
              }
              y0 = fast_exp2(y0);
              y1 = fast_exp2(y1);
              sum += y0 + y1;
              w[4 * g + e / 2] = f32x2_to_f16x2(y0, y1);
            }
            l = fmaf(sum, gi.inv_v, l);
          }
          tmem_st16(sc + 16 * c, w);       // 32 weights over the first of the 32 scores' columns, all read by now
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&s.p_full[i]);
      }
    }

    // ------------------------------------------------------------ output
    if (n > 0 && i < tiles) {
      wait(&s.o_full[i], 0);
      tc_fence_after_sync();
    }
    // NaN values of partly hidden tiles, for the rows that see them
    uint32_t nan[4] = {};
    if (live && *static_cast<volatile int*>(&s.nan_seen) != 0) {
      for (int j = 0; j < n; ++j) {
        if (whole(tile0 + j, 0, rows - 1)) continue;
        for (int key = max((tile0 + j) * kKeys, a.window > 0 ? pos - a.window + 1 : 0); key <= min(pos, (tile0 + j) * kKeys + kKeys - 1); ++key) {
          if (key >= end || key < 0) continue;
          const int page_at = key / ca.page_size, page = a.block_table[static_cast<int64_t>(b) * a.table_width + page_at];
          if (page < 0 || page >= ca.num_pages) continue;
          const uint8_t* codes = ca.v + page * ca.v_stride_page + head * ca.v_stride_head + (key - page_at * ca.page_size) * ca.v_stride_token;
          for (int d = 0; d < ca.head_dim; ++d)
            if ((codes[d] & 0x7F) == 0x7F) nan[d >> 5] |= 1u << (d & 31);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    T* dst = static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head;
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
      uint32_t r[32] = {};
      if (n > 0 && i < tiles) {
        tmem_ld32(oc + 32 * c, r);
        tmem_wait(r);
      }
      if (live) {
#pragma unroll
        for (int d = 0; d < 32; d += 8) {
          if (32 * c + d >= ca.head_dim) continue;
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = n > 0 ? __uint_as_float(r[d + e]) * inv : 0.f;
            if ((nan[c] >> (d + e)) & 1) v[e] = __uint_as_float(0x7FC00000u);
          }
          store_f32<T, 8>(dst + 32 * c + d, v);
        }
      }
    }
    if (live && a.lse != nullptr) a.lse[static_cast<int64_t>(tok) * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    tc_fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DP>
int launch(const AttentionParams& a, cudaStream_t stream) {
  CUtensorMap k_map, v_map;
  Launch p = {};
  p.a = a;
  p.box = 8;
  while (p.box < kKeys && a.cache.page_size % (2 * p.box) == 0) p.box *= 2;
  if (!encode_cache_map(&k_map, a.cache, false, p.box) || !encode_cache_map(&v_map, a.cache, true, p.box)) return MOE_ERR_CUDA;
  auto kernel = prefill_attention_kernel<T, DP>;
  constexpr int bytes = Layout<DP>::kBytes;
  if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes) != cudaSuccess) return MOE_ERR_CUDA;
  const int64_t rows = static_cast<int64_t>(a.max_q_len) * (a.Hq / a.cache.kv_heads);
  p.row_tiles = static_cast<int>((rows + kCtaRows - 1) / kCtaRows);
  const int64_t grid = static_cast<int64_t>(p.row_tiles) * a.B * a.cache.kv_heads;
  if (grid > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, stream, k_map, v_map, p) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

int launch_prefill_attention(const AttentionParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F16) return p.cache.head_dim <= 64 ? launch<__half, 64>(p, s) : launch<__half, 128>(p, s);
  return p.cache.head_dim <= 64 ? launch<__nv_bfloat16, 64>(p, s) : launch<__nv_bfloat16, 128>(p, s);
}

}  // namespace moe
