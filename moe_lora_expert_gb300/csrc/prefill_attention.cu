// Attention of many new tokens over the paged cache, on tcgen05.
//
// A unit is up to 256 rows (new tokens x query heads of one key head's group)
// as two tiles of 128; a CTA walks the keys they see in tiles of 128:
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
// While one row tile is in its softmax the tensor cores work for the other,
// and while a unit ends the next one's keys are on their way.
//
// All units' key tiles form one line that the CTAs cut into equal stretches,
// so ragged batches and long contexts fill the GPU alike.  A unit whose tiles
// lie in several stretches is joined by the CTA that finishes it last.
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
constexpr int kThreads = 448;
constexpr int kSlots = 4;                  // converted tiles: K0, V0, K1, V1, ...
constexpr int kStages = 2;                 // tiles of codes, in the same order
constexpr int kInfo = 4;                   // key tiles whose scales are held (see the copies)
constexpr int kMinTiles = 4;               // a CTA takes at least this many key tiles
constexpr int kMaxCtas = 160;
constexpr int kJoin = 8;                   // pieces that are joined at a time
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
  uint64_t info_full[kInfo], q_raw, q_full, q_empty, s_full[2], p_full[2], o_full[2], drained;
  int8_t q_exponent[kCtaRows];             // of the power of two taken out of each row
  int sums[kThreads / 32];
  uint32_t tmem;
  int abort_flag, nan_seen, first_entry, first_prefix, last[2];
};

// Partial sums of a row tile [slot][row tile][column / 4][row] of four columns
// each, (m, l) [slot][row tile][row], counters [2][slot][row tile].
constexpr int kParts = 2 * kMaxCtas;
constexpr size_t kPartialBytes = static_cast<size_t>(kParts) * kCtaRows * 128 * 4;
constexpr size_t kMlBytes = static_cast<size_t>(kParts) * kCtaRows * 8;
constexpr size_t kCounterBytes = static_cast<size_t>(kParts) * 2 * 2 * 4;

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
  int unit_rows;                           // whole tokens' rows, at most 256
  int row_tiles;                           // units of the longest sequence
  uint8_t* workspace;
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

// -------------------------------------------------------- pairs of float32
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------- units
// The rows of one (sequence, row tile) and the keys they see.
struct Entry {
  int b, q_first, row0, rows, start, lo, end, tile0, count;
  __device__ __forceinline__ void load(const Launch& p, int e, int group) {
    const AttentionParams& a = p.a;
    b = e / p.row_tiles;
    row0 = (e - b * p.row_tiles) * p.unit_rows;
    q_first = a.cu_q == nullptr ? b : a.cu_q[b];
    const int q_len = a.cu_q == nullptr ? 1 : a.cu_q[b + 1] - q_first;
    start = a.seq_lens[b] - q_len;
    rows = max(0, min(p.unit_rows, min(min(q_len, a.max_q_len), a.N - q_first) * group - row0));
    lo = end = tile0 = count = 0;
    if (rows > 0) {
      lo = a.window > 0 ? max(0, position(0, group) + 1 - a.window) : 0;
      const int64_t most = static_cast<int64_t>(a.table_width) * a.cache.page_size;
      end = static_cast<int>(min(static_cast<int64_t>(max(0, position(rows - 1, group) + 1)), most));
      tile0 = lo / kKeys;
      count = max(1, (end + kKeys - 1) / kKeys - tile0);      // one at least, so that someone writes the rows
    }
  }
  __device__ __forceinline__ int position(int row, int group) const { return start + (row0 + row) / group; }
  // Whether rows r0 to r1 all see every key of a tile (if its pages are there).
  __device__ __forceinline__ bool whole(int tile, int r0, int r1, int group, int window) const {
    const int key0 = tile * kKeys;
    return key0 + kKeys - 1 <= position(r0, group) && (window == 0 || key0 > position(r1, group) - window);
  }
};

// A CTA's stretch of the line, unit by unit; every warp walks it by itself.
struct Walk {
  Entry en;
  int e, head, tile, x, x1, n;             // this piece: tiles [tile, tile + n) of the unit
  __device__ __forceinline__ bool next(const Launch& p, int group, bool first, int first_entry, int first_prefix) {
    const int heads = p.a.cache.kv_heads;
    if (first) {
      e = first_entry;
      en.load(p, e, group);
      const int in = x - first_prefix * heads;
      head = in / en.count;
      tile = in - head * en.count;
    } else {
      x += n;
      tile = 0;
      if (++head == heads) head = -1;
    }
    if (x >= x1) return false;
    if (head < 0) {
      head = 0;
      do en.load(p, ++e, group);
      while (en.count == 0);
    }
    n = min(en.count - tile, x1 - x);
    return true;
  }
};

// ------------------------------------------------------------------ kernel
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
prefill_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const Launch p) {
  using L = Layout<DP>;
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& s = *reinterpret_cast<Control*>(smem + L::kControl);
  const AttentionParams& a = p.a;
  const moe_kv_cache_t& ca = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / ca.kv_heads;

  if (tid == 0) {
    tma_prefetch_map(&q_map);
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
    mbar_init(&s.q_raw, 1);
    mbar_init(&s.q_full, 4);
    mbar_init(&s.q_empty, 1 + 2 * kTileRows);    // the last scores, and every row's thread has its exponent
    mbar_init(&s.drained, 1);
    s.abort_flag = 0;
    s.nan_seen = 0;
    fence_mbarrier_init();
  }
  pdl_wait();

  // The line's length, and where this CTA's stretch of it begins.
  const int entries = a.B * p.row_tiles, per = (entries + kThreads - 1) / kThreads;
  const int from = min(tid * per, entries), to = min(from + per, entries);
  int mine = 0;
  for (int e = from; e < to; ++e) {
    Entry en;
    en.load(p, e, group);
    mine += en.count;
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s.sums[warp] = incl;
  __syncthreads();
  int all_tiles = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) incl += s.sums[w];
    all_tiles += s.sums[w];
  }
  const int total = all_tiles * ca.kv_heads;
  const int ctas = min(static_cast<int>(gridDim.x), max(1, total / kMinTiles));
  if (total == 0 || static_cast<int>(blockIdx.x) >= ctas) return;
  auto begin_of = [&](int cta) { return static_cast<int>(static_cast<int64_t>(total) * cta / ctas); };
  Walk walk;
  walk.x = begin_of(blockIdx.x);
  walk.x1 = begin_of(blockIdx.x + 1);
  if (walk.x < incl * ca.kv_heads && walk.x >= (incl - mine) * ca.kv_heads) {
    int before = incl - mine;
    for (int e = from; e < to; ++e) {
      Entry en;
      en.load(p, e, group);
      if (walk.x < (before + en.count) * ca.kv_heads) {
        s.first_entry = e;
        s.first_prefix = before;
        break;
      }
      before += en.count;
    }
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

  // A wait that runs out, here or in another role, ends the CTA's work: no
  // role then issues a copy or a product or touches TMEM any more.
  auto aborted = [&] { return *static_cast<volatile int*>(&s.abort_flag) != 0; };
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {      // by one thread
    if (!mbar_try_wait(smem_u32(bar), parity) && (aborted() || !mbar_wait(bar, parity, a.wait_limit_ns))) {
      set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
      *static_cast<volatile int*>(&s.abort_flag) = 1;
      return false;
    }
    return true;
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {          // by a warp, which leaves it together
    const bool ok = wait_one(bar, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  auto next = [&](bool first) { return walk.next(p, group, first, s.first_entry, s.first_prefix); };
  const Entry& en = walk.en;

  if (warp == kLoadWarp) {
    // ------------------------------------------------ pages, scales, copies
    // Scales are held for kInfo tiles: when tile t's are written the codes of
    // K(t - 1) have been converted, so S(t - 3) is done, which was issued
    // after both softmaxes had delivered P(t - 4), their last use of t - 4's.
    struct Ahead {
      int page, off;
      Group g;
    };
    auto find = [&](int j) {
      Ahead f = {-1, 0, {0.f, 0.f, 0.f, 0}};
      const int key = (en.tile0 + walk.tile + j) * kKeys + 8 * (lane & 15);
      if (j < walk.n && key < en.end && (key & ~(p.box - 1)) + p.box > en.lo) {
        const int page_at = key / ca.page_size;
        f.off = key - page_at * ca.page_size;
        f.page = a.block_table[static_cast<int64_t>(en.b) * a.table_width + page_at];
        if (f.page < 0 || f.page >= ca.num_pages) {
          f.page = -1;
          set_status(a.status, MOE_ERR_BAD_PAGE);
        } else {
          const int64_t i = static_cast<int64_t>(f.page) * ca.kv_heads + walk.head;
          const float vs = fmaxf(ca.v_scale[i], 5.421010862427522e-20f);   // 2^-64: a zero scale gives zero values
          f.g = {ca.k_scale[i] * fabsf(a.scale) * kLog2e, log2f(vs), 1.f / vs, 1};
        }
      }
      return f;
    };
    int issued = 0, units = 0;
    bool stop = false;
    for (bool more = next(true); more && !stop; more = next(false)) {
      if (en.position(en.rows - 1, group) >= static_cast<int64_t>(a.table_width) * ca.page_size) set_status(a.status, MOE_ERR_BAD_PAGE);
      Ahead now = find(0);
      for (int j = 0; j < walk.n && !stop; ++j) {
        const Ahead later = find(j + 1);
        const int t = issued / 2;
        const bool issues = lane < 16 && now.page >= 0 && (8 * lane) % p.box == 0;
        const unsigned boxes = __ballot_sync(0xffffffffu, issues);
        for (int v = 0; v < 2; ++v) {
          const int st = issued % kStages;
          if (issued >= kStages && !wait(&s.code_empty[st], (issued / kStages - 1) & 1)) {
            stop = true;                                             // a stage that was not freed is not filled again
            break;
          }
          if (v == 0 && lane < 16) s.group[t % kInfo][lane] = now.g;
          __syncwarp();
          if (lane == 0) {
            if (v == 0) mbar_arrive(&s.info_full[t % kInfo]);
            mbar_arrive_expect_tx(&s.code_full[st], __popc(boxes) * p.box * 128);
          }
          __syncwarp();
          if (issues)
            tma_load_4d(smem_u32(smem + L::kCode + st * L::kCodeBytes) + 8 * lane * 128, v == 0 ? &k_map : &v_map,
                        &s.code_full[st], now.off, walk.head, now.page);
          ++issued;
          if (j == 0 && v == 0) {                                    // the unit's queries, after its first keys
            if (units > 0 && !wait(&s.q_empty, (units - 1) & 1)) {
              stop = true;
              break;
            }
            if (lane == 0) {
              mbar_arrive_expect_tx(&s.q_raw, L::kHalves * p.unit_rows * 128);
              for (int h = 0; h < L::kHalves; ++h)
                tma_load_3d(smem_u32(smem + L::kQ + 2 * h * L::kHalfBytes), &q_map, &s.q_raw, 64 * h, walk.head * group,
                            en.q_first + en.row0 / group);
            }
            ++units;
          }
        }
        now = later;
      }
    }
    if (stop) {                                          // nothing of this CTA stays in flight
      for (int k = max(0, issued - kStages); k < issued; ++k) mbar_wait(&s.code_full[k % kStages], (k / kStages) & 1, a.wait_limit_ns);
      if (units > 0) mbar_wait(&s.q_raw, (units - 1) & 1, a.wait_limit_ns);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t kScores = idesc_f16(kTileRows, kKeys, false), kValues = idesc_f16(kTileRows, DP, true);
      const uint32_t q_base = smem_u32(smem + L::kQ), ring = smem_u32(smem + L::kRing);
      auto scores = [&](int i, int slot) {
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          const uint32_t at = (k % 4) * 32;
          tc_mma_bf16(s_cols(i), make_sdesc_sw128(q_base + (2 * (k / 4) + i) * L::kHalfBytes + at),
                      make_sdesc_sw128(ring + slot * L::kSlotBytes + (k / 4) * L::kHalfBytes + at), kScores, k > 0);
        }
        tc_commit(&s.s_full[i]);
      };
      auto values = [&](int i, int slot, bool more) {
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          mma_ts_f16(o_cols(i), s_cols(i) + 8 * k, mn_major_sdesc(ring + slot * L::kSlotBytes + 2048 * k, L::kHalfBytes), kValues,
                     more || k > 0);
      };
      int t = 0, p_count[2] = {0, 0}, units = 0;
      bool ok = true, issued = false;
      for (bool more = next(true); more && ok; more = next(false)) {
        const int tiles = en.rows > kTileRows ? 2 : 1;
        int k = 2 * t;
        ok = wait_one(&s.q_full, units & 1) && wait_one(&s.full[k % kSlots], (k / kSlots) & 1);
        if (!ok) break;
        tc_fence_after_sync();
        issued = true;
        for (int i = 0; i < tiles; ++i) scores(i, k % kSlots);
        tc_commit(&s.empty[k % kSlots]);
        if (walk.n == 1) tc_commit(&s.q_empty);
        for (int j = 0; j < walk.n && ok; ++j, ++t) {
          const int v = 2 * t + 1;
          k = 2 * t + 2;
          ok = wait_one(&s.full[v % kSlots], (v / kSlots) & 1);
          for (int i = 0; i < tiles && ok; ++i) {
            ok = wait_one(&s.p_full[i], p_count[i]++ & 1);
            if (!ok) break;
            tc_fence_after_sync();
            values(i, v % kSlots, j > 0);
            if (i == tiles - 1) tc_commit(&s.empty[v % kSlots]);
            if (j + 1 < walk.n) {
              if (i == 0) {
                ok = wait_one(&s.full[k % kSlots], (k / kSlots) & 1);
                if (!ok) break;
                tc_fence_after_sync();
              }
              scores(i, k % kSlots);
              if (i == tiles - 1) {
                tc_commit(&s.empty[k % kSlots]);
                if (j + 2 == walk.n) tc_commit(&s.q_empty);
              }
            } else {
              tc_commit(&s.o_full[i]);
            }
          }
        }
        ++units;
      }
      if (issued) {
        tc_commit(&s.drained);
        mbar_wait(&s.drained, 0, a.wait_limit_ns);
      }
    }
    __syncwarp();
  } else if (warp >= kConvertWarp && warp < kMmaWarp) {
    // --------------------------------------------------------- conversion
    // A lane converts 16 codes to two 16-byte chunks.  Eight lanes at a time
    // take four chunks of keys k and k ^ 5, which fall on distinct banks for
    // both the load and the stores.
    const int w = warp - kConvertWarp, sub = lane & 3, key8 = (lane >> 3) ^ (5 * ((lane >> 2) & 1));
    int k = 0, units = 0;
    bool good = true;
    for (bool more = next(true); more && good; more = next(false), ++units) {
      for (int j = 0; j < 2 * walk.n; ++j, ++k) {
        const int st = k % kStages, slot = k % kSlots;
        const Group* info = s.group[(k / 2) % kInfo];
        good = wait(&s.code_full[st], (k / kStages) & 1) && (k < kSlots || wait(&s.empty[slot], (k / kSlots - 1) & 1));
        if (!good) break;
        const uint8_t* src = smem + L::kCode + st * L::kCodeBytes;
        uint8_t* dst = smem + L::kRing + slot * L::kSlotBytes;
        // a weight of zero times a NaN code would be NaN: where some row does
        // not see some key, NaN values are left out here and added at the end
        const int tile = en.tile0 + walk.tile + j / 2;
        bool drop = false;
        if ((j & 1) != 0) {
          const int ok = lane < 16 ? info[lane].valid : 1;
          drop = !__all_sync(0xffffffffu, ok) || !en.whole(tile, 0, en.rows - 1, group, a.window);
        }
        bool nan = false;
#pragma unroll 4
        for (int it = w; it < 16 * L::kHalves; it += 4) {
          const int key = 8 * (it / L::kHalves) + key8, half = it % L::kHalves, x = key & 7;
          uint4 c = *reinterpret_cast<const uint4*>(src + key * 128 + (((4 * half + sub) ^ x) * 16));
          if (drop) {
            uint32_t seen = 0;
            auto clean = [&](uint32_t& word) {
              const uint32_t bad = __vcmpeq4(word & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              seen |= bad;
              word &= ~bad;
            };
            clean(c.x), clean(c.y), clean(c.z), clean(c.w);
            const int at = tile * kKeys + key;
            nan |= seen != 0 && at >= en.lo && at < en.end && info[key >> 3].valid;      // some row sees it
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
        if (nan) *static_cast<volatile int*>(&s.nan_seen) = 1;
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&s.code_empty[st]);
          mbar_arrive(&s.full[slot]);
        }
        if (j == 0) {
          // The queries, which the TMA has put where the A operand goes: bf16
          // rows become float16 in place, a power of two taken out of each.
          good = wait(&s.q_raw, units & 1);
          if (!good) break;
          if constexpr (kBf16) {
#pragma unroll 1
            for (int row = 32 * w + lane; row < kCtaRows; row += 128) {
              uint8_t* at = smem + L::kQ + row * 128;      // half h of row r: (2 h + r / 128) * 128 rows + r % 128
              auto chunk = [&](int c) { return reinterpret_cast<uint4*>(at + 2 * (c / 8) * L::kHalfBytes + (((c & 7) ^ (row & 7)) * 16)); };
              uint32_t amax = 0;                           // of the magnitudes' bits, which order as they do
#pragma unroll 4
              for (int c = 0; c < DP / 8; ++c) {
                const uint4 u = *chunk(c);
                amax = __vmaxu2(amax, __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu)));
              }
              int ex = static_cast<int>(max(amax & 0xFFFF, amax >> 16) >> 7) - 127;
              if (ex <= -120 || ex >= 120) ex = 0;         // zero, or not finite: nothing to gain
              s.q_exponent[row] = static_cast<int8_t>(ex);
              float inv = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
              if (a.scale < 0.f) inv = -inv;               // the sign goes into q, so that a larger score is a larger weight
#pragma unroll 4
              for (int c = 0; c < DP / 8; ++c) {
                uint4 u = *chunk(c);
                auto turn = [&](uint32_t v) {
                  return f32x2_to_f16x2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
                };
                u = make_uint4(turn(u.x), turn(u.y), turn(u.z), turn(u.w));
                *chunk(c) = u;
              }
            }
            fence_proxy_async_shared();
            __syncwarp();
          } else if (a.scale < 0.f) {
            for (int c = 32 * w + lane; c < L::kQBytes / 16; c += 128) {
              uint4* at = reinterpret_cast<uint4*>(smem + L::kQ) + c;
              const uint4 u = *at;
              *at = make_uint4(u.x ^ 0x80008000u, u.y ^ 0x80008000u, u.z ^ 0x80008000u, u.w ^ 0x80008000u);
            }
            fence_proxy_async_shared();
            __syncwarp();
          }
          if (lane == 0) mbar_arrive(&s.q_full);
        }
      }
    }
  } else if (warp < kConvertWarp) {
    // ------------------------------------------------------------- softmax
    const int i = warp >> 2, row = kTileRows * i + 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t sc = s_cols(i) + lanes, oc = o_cols(i) + lanes;
    int t = 0, s_count = 0, o_count = 0, units = 0;
    bool good = true;
    for (bool more = next(true); more; more = next(false), ++units) {
      // after a timeout a unit's rows are left as they are, but its part in the
      // join is still played, so that the counters end at zero
      good = good && wait(&s.q_full, units & 1);
      const float row_scale = kBf16 ? __uint_as_float(static_cast<uint32_t>(127 + s.q_exponent[row]) << 23) : 1.f;
      // Only now may the next unit's queries come: a unit of one tile has its
      // last scores before its rows' threads have begun it, and two of them
      // would carry q_full past the phase that they wait for.
      mbar_arrive(&s.q_empty);
      if (kTileRows * i >= en.rows) {
        t += walk.n;
        continue;
      }
      const bool live = row < en.rows;
      const int pos = live ? en.position(row, group) : -1;
      const int r0 = kTileRows * i, r1 = min(en.rows, r0 + kTileRows) - 1;
      // weights are relative to 2^base; a row's limit is how far above it a
      // weight may be before the sums are rescaled
      float base = 0.f, limit = -INFINITY, l = 0.f;

      for (int j = 0; j < walk.n && good; ++j, ++t) {
        const int tile = en.tile0 + walk.tile + j, key0 = tile * kKeys;
        const Group* info = s.group[t % kInfo];
        good = wait(&s.info_full[t % kInfo], (t / kInfo) & 1) && wait(&s.s_full[i], s_count++ & 1);
        if (!good) break;
        const bool all = __all_sync(0xffffffffu, lane < 16 ? info[lane].valid : 1) && en.whole(tile, r0, r1, group, a.window);
        tc_fence_after_sync();

        // which of 32 keys from key0 + 32 c on this row sees, a bit each
        const int low = a.window > 0 ? pos - a.window + 1 - key0 : 0;
        auto seen = [&](int c) {
          const int first = low - 32 * c, last = pos - key0 - 32 * c;    // [first, last]
          uint32_t mask = last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u;
          mask &= first <= 0 ? 0xffffffffu : first > 31 ? 0u : ~((1u << first) - 1u);
#pragma unroll
          for (int g = 0; g < 4; ++g)
            if (!info[4 * c + g].valid) mask &= ~(0xFFu << (8 * g));
          return mask;
        };
        // 32 scores to weights, in the columns of the first 16: what was
        // there has been read
        auto weigh = [&](int c, uint32_t (&r)[32]) {
          float4 gi[4];
          float top = -INFINITY;
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            gi[g] = *reinterpret_cast<const float4*>(&info[4 * c + g]);
            const uint64_t kk = f32x2(gi[g].x * row_scale, gi[g].x * row_scale), off = f32x2(gi[g].y - base, gi[g].y - base);
#pragma unroll
            for (int e = 8 * g; e < 8 * g + 8; e += 2) {
              float y0, y1;
              unpack(fma2(f32x2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), kk, off), y0, y1);
              r[e] = __float_as_uint(y0);
              r[e + 1] = __float_as_uint(y1);
            }
          }
          if (!all) {
            const uint32_t mask = seen(c);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = (mask >> e) & 1 ? r[e] : 0xFF800000u;
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2) top = max3(top, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
          if (__any_sync(0xffffffffu, top > limit)) {
            // a new maximum: what this unit has summed so far, and this
            // tile's earlier weights, become relative to it
            const float rise = limit == -INFINITY ? (top == -INFINITY ? 0.f : top) : fmaxf(top, 0.f);
            const float keep = limit == -INFINITY ? 0.f : fast_exp2(-rise);
            base += rise;
            if (top > -INFINITY) limit = kSlack;
            l *= keep;
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) - rise);
            if (j > 0) {       // O holds the products up to the tile before: they came before these scores
#pragma unroll 1
              for (int d = 0; d < DP / 32; ++d) {
                uint32_t o[32];
                tmem_ld32(oc + 32 * d, o);
                tmem_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st32(oc + 32 * d, o);
              }
            }
#pragma unroll 1
            for (int d = 0; d < c; ++d) {
              float o[16];
              tmem_ld16(sc + 16 * d, o);
              uint32_t wd[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t bits = __float_as_uint(o[e]);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&bits));
                wd[e] = f32x2_to_f16x2(f.x * keep, f.y * keep);
              }
              tmem_st16(sc + 16 * d, wd);
            }
          }
          uint32_t wd[16];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            uint64_t sum = 0;
#pragma unroll
            for (int e = 8 * g; e < 8 * g + 8; e += 2) {
              const float y0 = fast_exp2(__uint_as_float(r[e])), y1 = fast_exp2(__uint_as_float(r[e + 1]));
              sum = e == 8 * g ? f32x2(y0, y1) : add2(sum, f32x2(y0, y1));
              wd[e / 2] = f32x2_to_f16x2(y0, y1);
            }
            float s0, s1;
            unpack(sum, s0, s1);
            l = fmaf(s0 + s1, gi[g].z, l);
          }
          tmem_st16(sc + 16 * c, wd);
        };
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(sc + 32 * c, r);
          tmem_wait(r);
          weigh(c, r);
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(&s.p_full[i]);
      }

      // ---------------------------------------------------------- output
      good = good && wait(&s.o_full[i], o_count++ & 1);
      tc_fence_after_sync();
      // NaN values of partly hidden tiles, for the rows that see them
      uint32_t nan[4] = {};
      if (live && good && *static_cast<volatile int*>(&s.nan_seen) != 0) {
        for (int tile = en.tile0 + walk.tile; tile < en.tile0 + walk.tile + walk.n; ++tile) {
          const int k0 = max(tile * kKeys, a.window > 0 ? pos - a.window + 1 : 0), k1 = min(min(pos, en.end - 1), tile * kKeys + kKeys - 1);
          for (int key = k0; key <= k1; ++key) {
            const int page_at = key / ca.page_size, page = a.block_table[static_cast<int64_t>(en.b) * a.table_width + page_at];
            if (page < 0 || page >= ca.num_pages) continue;
            const uint8_t* codes = ca.v + page * ca.v_stride_page + walk.head * ca.v_stride_head + (key - page_at * ca.page_size) * ca.v_stride_token;
            for (int d = 0; d < ca.head_dim; ++d)
              if ((codes[d] & 0x7F) == 0x7F) nan[d >> 5] |= 1u << (d & 31);
          }
        }
      }
      const float m = limit == -INFINITY ? -INFINITY : base;
      const int gr = en.row0 + row, tok = en.q_first + gr / group, h = walk.head * group + gr % group;
      T* dst = static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head;
      auto put = [&](int d, const float (&v)[32], float inv) {        // columns [d, d + 32)
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (d + e >= ca.head_dim) continue;
          float y[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) y[z] = v[e + z] * inv;
          store_f32<T, 8>(dst + d + e, y);
        }
      };
      auto put_lse = [&](float mm, float ll) {
        if (a.lse != nullptr) a.lse[static_cast<int64_t>(tok) * a.Hq + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      };
      auto summed = [&](int d, float (&v)[32]) {                       // O's columns [d, d + 32)
        uint32_t r[32] = {};
        if (good) {
          tmem_ld32(oc + d, r);
          tmem_wait(r);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = (nan[d / 32] >> e) & 1 ? __uint_as_float(0x7FC00000u) : __uint_as_float(r[e]);
      };
      if (walk.n == en.count) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int d = 0; d < DP; d += 32) {
          float v[32];
          summed(d, v);
          if (live) put(d, v, inv);
        }
        if (live) put_lse(m, l);
        tc_fence_before_sync();
        continue;
      }

      // A part of the unit: pieces of it are in CTAs [cta0, cta1], joined
      // eight at a time by whoever finishes last among them, then those
      // results likewise.
      float4* parts = reinterpret_cast<float4*>(p.workspace);
      float2* ml = reinterpret_cast<float2*>(p.workspace + kPartialBytes);
      int* counters = reinterpret_cast<int*>(p.workspace + kPartialBytes + kMlBytes);
      const int u0 = walk.x - walk.tile, u1 = u0 + en.count;
      auto cta_of = [&](int y) {                                       // the CTA that holds tile y of the line
        int cta = static_cast<int>(static_cast<int64_t>(y) * ctas / total);
        while (cta + 1 < ctas && begin_of(cta + 1) <= y) ++cta;
        while (begin_of(cta) > y) --cta;
        return cta;
      };
      const int cta0 = cta_of(u0), pieces = cta_of(u1 - 1) - cta0 + 1, mine_at = static_cast<int>(blockIdx.x) - cta0;
      // two slots a CTA: for the unit that began before its stretch, and for one that began in it
      auto slot_of = [&](int piece) { return (2 * (cta0 + piece) + (piece == 0 ? 1 : 0)) * 2 + i; };
      const int r = row & 127;
      auto part = [&](int slot, int d) { return parts + (static_cast<size_t>(slot) * 32 + d / 4) * kTileRows + r; };
#pragma unroll
      for (int d = 0; d < DP; d += 32) {
        float v[32];
        summed(d, v);
#pragma unroll
        for (int e = 0; e < 32; e += 4) __stcg(part(slot_of(mine_at), d + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
      }
      __stcg(ml + static_cast<size_t>(slot_of(mine_at)) * kTileRows + r, make_float2(m, l));
      tc_fence_before_sync();
      int step = 1, lead = mine_at / kJoin * kJoin, count = min(kJoin, pieces - lead);
      for (int level = 0;; ++level) {
        __threadfence();
        named_barrier_sync(1 + i, kTileRows);
        if ((tid & 127) == 0) {
          int* counter = counters + level * 2 * kParts + slot_of(lead);
          const bool last = atomicAdd(counter, 1) == count - 1;
          if (last) *counter = 0;                                      // ready for the next call
          s.last[i] = last;
        }
        named_barrier_sync(1 + i, kTileRows);
        const bool last = s.last[i] != 0;
        named_barrier_sync(1 + i, kTileRows);
        if (!last) break;
        __threadfence();
        const bool finish = count == pieces || level == 1;
        auto ml_of = [&](int q) { return __ldcg(ml + static_cast<size_t>(slot_of(lead + q * step)) * kTileRows + r); };
        float mx = -INFINITY, lx = 0.f;
        for (int q = 0; q < count; ++q) mx = fmaxf(mx, ml_of(q).x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        for (int q = 0; q < count; ++q) {
          const float2 z = ml_of(q);
          lx = fmaf(z.y, fast_exp2(z.x - ref), lx);
        }
        const float inv = lx == 0.f ? 0.f : 1.f / lx;
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
          float v[32] = {};
          for (int q = 0; q < count; ++q) {
            const float f = fast_exp2(ml_of(q).x - ref);
            const int slot = slot_of(lead + q * step);
            float4 y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = __ldcg(part(slot, d + 4 * e));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              v[4 * e] = fmaf(y[e].x, f, v[4 * e]);
              v[4 * e + 1] = fmaf(y[e].y, f, v[4 * e + 1]);
              v[4 * e + 2] = fmaf(y[e].z, f, v[4 * e + 2]);
              v[4 * e + 3] = fmaf(y[e].w, f, v[4 * e + 3]);
            }
          }
          if (finish) {
            if (live) put(d, v, inv);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4) __stcg(part(slot_of(lead), d + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
          }
        }
        if (finish) {
          if (live) put_lse(mx, lx);
          break;
        }
        __stcg(ml + static_cast<size_t>(slot_of(lead)) * kTileRows + r, make_float2(mx, lx));
        step = kJoin;
        lead = 0;
        count = (pieces + kJoin - 1) / kJoin;
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <typename T, int DP>
int launch(const AttentionParams& a, cudaStream_t stream) {
  CUtensorMap q_map, k_map, v_map;
  Launch p = {};
  p.a = a;
  p.workspace = static_cast<uint8_t*>(a.workspace) + decode_attention_workspace_bytes();
  p.box = 8;
  while (p.box < kKeys && a.cache.page_size % (2 * p.box) == 0) p.box *= 2;
  const int group = a.Hq / a.cache.kv_heads;
  p.unit_rows = kCtaRows / group * group;
  if (!encode_cache_map(&k_map, a.cache, false, p.box) || !encode_cache_map(&v_map, a.cache, true, p.box) ||
      !encode_query_map(&q_map, a, std::is_same<T, __half>::value, group, kCtaRows / group))
    return MOE_ERR_CUDA;
  auto kernel = prefill_attention_kernel<T, DP>;
  constexpr int bytes = Layout<DP>::kBytes;
  if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes) != cudaSuccess) return MOE_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int64_t row_tiles = (static_cast<int64_t>(a.max_q_len) * group + p.unit_rows - 1) / p.unit_rows;
  const int64_t line = row_tiles * a.B * ((static_cast<int64_t>(a.table_width) * a.cache.page_size) / kKeys + 1) * a.cache.kv_heads;
  if (line > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  p.row_tiles = static_cast<int>(row_tiles);
  int64_t grid = sms < kMaxCtas ? sms : kMaxCtas;
  const int64_t units = row_tiles * a.B * a.cache.kv_heads * ((a.max_seq_len + kKeys - 1) / kKeys + 1);
  if (grid > units) grid = units;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, stream, q_map, k_map, v_map, p) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

size_t prefill_attention_workspace_bytes() { return kPartialBytes + kMlBytes + kCounterBytes; }

int launch_prefill_attention(const AttentionParams& p, int dtype, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F16) return p.cache.head_dim <= 64 ? launch<__half, 64>(p, s) : launch<__half, 128>(p, s);
  return p.cache.head_dim <= 64 ? launch<__nv_bfloat16, 64>(p, s) : launch<__nv_bfloat16, 128>(p, s);
}

}  // namespace moe
