// Attention of many new tokens over the paged cache, on tcgen05.
//
// A unit is up to 256 rows (new tokens x query heads of one key head's group)
// as two tiles of 128; a CTA walks the keys they see in tiles of 128:
//   S = Q K^T (TMEM), P = 2^(S k_scale' + log2 v_scale - m) (float16, back into
//   S's columns), O += P V (TMEM), with a reference m that follows the keys.
// The weights carry the pages' value scales, and m keeps the largest of every
// 64 keys where float16 has all its bits, both as in decode_attention.cu; so K
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
// lie in several stretches is joined by the CTA that finishes it last.  A cut
// costs a CTA that writes its part or joins it about four key tiles' time, so
// where whole units can be dealt out nearly as evenly they are.
//
// What bounds it.  2 x 2048 tokens of 32 heads of 128 on 4 key heads take 90.6
// us, 759 TFLOP/s of what the causal mask leaves, 40% of the measured bf16
// rate (37 us).  The products of a pair of row tiles and a key tile take 2.05
// thousand cycles, 2.8 with the gaps between groups of them; a softmax takes
// about 3 (each row tile's four warps share their schedulers with the other's
// and the converter's: 0.6 thousand instructions a warp, waits on TMEM and
// on each other), and a row tile's products and softmax follow one another.
// For heads of 64 the softmax is the same for half the products: 116 us for
// ragged chunks on up to 8191 keys, 25%.  Scores of 64 keys in two buffers a
// row tile took the wait out but cost more than it (an M = 128, N = 64
// product takes the time of N = 128): 148 against 130 us then.  A reference
// that falls as well costs nothing on scores of standard deviation 1 and 3
// (91 and 99 us), 1% on 6 and 2% on 12 there; 1, 1, 5 and 12% on chunks of 1000
// with heads of 64.
#include <cuda.h>

#include <type_traits>

#include "attention.cuh"
#include "attention_line.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kKeys = 128;
constexpr int kHalf = 64;                  // keys whose weights are handed over at a time
constexpr int kTileRows = 128;
constexpr int kCtaRows = 256;
constexpr int kThreads = 448;
constexpr int kSlots = 4;                  // converted tiles: K0, V0, K1, V1, ...
constexpr int kStages = 2;                 // tiles of codes, in the same order
constexpr int kInfo = 4;                   // key tiles whose scales are held (see the copies)
constexpr int kUnitCost = 2;               // key tiles' worth of time that a unit takes besides its tiles; 2 x 2048 tokens, cut from the line: 1 122, 2 103, 3 103, 4 105 us
constexpr int kMinTiles = 4;               // least length of a CTA's stretch (a join costs about as much as four tiles)
constexpr int kMaxCtas = 160;
constexpr int kMaxUnits = 16;              // whole units a CTA may be given (see the kernel)
constexpr int kJoinCost = 8;               // key tiles' worth of time that cutting the line may cost a CTA: part of a unit written, another joined
constexpr int kJoin = 8;                   // pieces that are joined at a time
constexpr int kNanTiles = 8;               // tiles with NaN that a warp notes for a unit; hidden in part are 6 at most where all pages are there
constexpr int kConvertWarp = 8, kMmaWarp = 12, kLoadWarp = 13;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMost = 15.9f, kNew = 7.f; // as in decode_attention.cu: a weight past 2^15.9 makes the reference rise, so that it becomes 2^7;
constexpr float kLow = -8.f, kBack = -5.f; // all of 64 keys' under 2^-8 make it fall, so that the largest becomes 2^-5,
constexpr float kRoom = 24.f;              // by 2^24 at most below its highest,
constexpr int kLook = 4;                   // looked for at every fourth tile
constexpr int kOColumns = 256;             // TMEM: two row tiles' scores, then their sums, 128 columns each

struct alignas(16) Group {                 // 8 keys, which lie in one page
  float k, lv, inv_v;
  int valid;
};

// Partial sums of a row tile [slot][row tile][column / 4][row] of four columns
// each, (m, l) [slot][row tile][row], counters [level][slot][row tile].
constexpr int kParts = 2 * kMaxCtas;
constexpr size_t kPartialBytes = static_cast<size_t>(kParts) * kCtaRows * 128 * 4;
constexpr size_t kMlBytes = static_cast<size_t>(kParts) * kCtaRows * 8;
constexpr size_t kCounterBytes = static_cast<size_t>(kParts) * 2 * 3 * 4;   // three levels of eight: up to 512 pieces

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
// A shared-memory descriptor's low word: the address, and for V (as the B
// operand with its columns contiguous) the distance of its 64-column halves.
// The high word is the same for both: groups of 8 rows 1024 bytes apart,
// 128-byte swizzle.  The one thread that issues the products adds constants
// to low words instead of building descriptors.
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t leading) { return (saddr >> 4) | (leading >> 4) << 16; }
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
// True in one lane of a converged warp.  The compiler knows that of this
// instruction but not of a comparison of lane numbers: behind that, each
// product is issued in a loop over the lanes that might be there (123 instead
// of 103 us on 2 x 2048 tokens).
__device__ __forceinline__ bool elect_one() {
  uint32_t elected;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected));
  return elected != 0;
}
__device__ __forceinline__ void mma_ss_f16(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "n"(kDescHigh), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "n"(kDescHigh), "r"(idesc), "r"(accumulate)
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
// On the line a unit is kUnitCost places and then a place a key tile.  Where
// ``whole`` is given the CTA has those units instead, x to x1.
struct Walk {
  Entry en;
  int e, head, tile, x, x1, n, u0, span;   // this piece: tiles [tile, tile + n) of the unit that begins at u0
  __device__ __forceinline__ bool next(const Launch& p, int group, const int* whole, bool first, int first_entry, int first_prefix) {
    const int heads = p.a.cache.kv_heads;
    if (whole != nullptr) {
      if (x == x1) return false;
      const int unit = whole[x++];
      e = unit / heads;
      head = unit - e * heads;
      en.load(p, e, group);
      tile = 0;
      n = en.count;
      return true;
    }
    int v = 0;
    if (first) {
      e = first_entry;
      en.load(p, e, group);
      const int in = x - first_prefix * heads;
      head = in / (en.count + kUnitCost);
      v = in - head * (en.count + kUnitCost);
      span = 0;
    } else {
      ++head;
    }
    while (true) {
      x += span;
      if (x >= x1) return false;
      if (head == heads) {
        head = 0;
        do en.load(p, ++e, group);
        while (en.count == 0);
      }
      u0 = x - v;
      span = min(en.count + kUnitCost - v, x1 - x);
      tile = max(0, v - kUnitCost);
      n = max(0, v + span - kUnitCost) - tile;
      if (n > 0) return true;
      v = 0;
      ++head;
    }
  }
};

// The kernel's roles share one instruction cache: what is called once a unit,
// or to wait, is not inlined into each of them.
// A walk lies in memory that ``lanes`` share, who all call this: the barriers
// keep each from writing the next piece while another still reads this one or
// has yet to take the same step (the loops that come here end in code which a
// warp's lanes may leave one by one).
__device__ __noinline__ bool walk_next(Walk* at, const Launch& p, int group, const int* whole, int first_entry, int first_prefix, uint32_t lanes) {
  __syncwarp(lanes);
  Walk w = *at;
  const bool more = w.next(p, group, whole, first_entry >= 0, first_entry, first_prefix);
  __syncwarp(lanes);
  *at = w;
  __syncwarp(lanes);
  return more;
}
// Which columns of keys k0 to k1 (of one tile) of sequence b hold NaN values.
__device__ __noinline__ uint4 nan_columns(const AttentionParams& a, int b, int head, int k0, int k1) {
  const moe_kv_cache_t& ca = a.cache;
  uint32_t nan[4] = {};
#pragma unroll 1
  for (int key = k0; key <= k1; ++key) {
    const int page_at = key / ca.page_size, page = a.block_table[static_cast<int64_t>(b) * a.table_width + page_at];
    if (page < 0 || page >= ca.num_pages) continue;
    const uint8_t* codes = ca.v + page * ca.v_stride_page + head * ca.v_stride_head + (key - page_at * ca.page_size) * ca.v_stride_token;
    uint4 c[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) c[d] = 16 * d < ca.head_dim ? *reinterpret_cast<const uint4*>(codes + 16 * d) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      // a bit for each of a word's four codes
      auto bits = [](uint32_t w) { return ((__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & 0x08040201u) * 0x01010101u) >> 24; };
      nan[d / 2] |= (bits(c[d].x) | bits(c[d].y) << 4 | bits(c[d].z) << 8 | bits(c[d].w) << 12) << (16 * (d & 1));
    }
  }
  return make_uint4(nan[0], nan[1], nan[2], nan[3]);
}
// ----------------------------------------------------------- shared memory
struct Control {
  Group group[kInfo][kKeys / 8];
  uint64_t code_full[kStages], code_empty[kStages], full[kSlots], empty[kSlots];
  uint64_t info_full[kInfo], q_raw, q_full, q_empty, s_full[2], p_full[2][2], first_done[2], o_full[2], drained;
  int8_t q_exponent[kCtaRows];             // of the power of two taken out of each row
  int sums[kThreads / 32];
  int units[kMaxUnits];                    // this CTA's, if it has whole ones
  Walk walk[kThreads / 32];                // each warp's own, here and not in its registers
  // Of a unit and the next: the key tiles, hidden from some rows, in which a
  // converting warp has met and left out NaN values that some row sees.
  int nan_count[2][4], nan_tiles[2][4][kNanTiles];
  uint32_t tmem;
  int abort_flag, first_entry, first_prefix, given, last[2], issued, issued_units;
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

// The queries of a unit by plain loads, to where and how the TMA would put
// them (f16 rows with the sign of the scale): rows first, first + 128, ...
template <typename T, int DP>
__device__ __noinline__ void load_queries(const AttentionParams& a, const Entry& en, int head, int group, uint8_t* to, int first) {
#pragma unroll 1
  for (int row = first; row < kCtaRows; row += kTileRows) {
    const int gr = en.row0 + row;
    const T* src = static_cast<const T*>(a.q) + (en.q_first + gr / group) * a.q_token + (head * group + gr % group) * a.q_head;
#pragma unroll 4
    for (int c = 0; c < DP / 8; ++c) {
      uint4 u = row < en.rows && 8 * c < a.cache.head_dim ? *reinterpret_cast<const uint4*>(src + 8 * c) : make_uint4(0, 0, 0, 0);
      if (std::is_same<T, __half>::value && a.scale < 0.f) u = make_uint4(u.x ^ 0x80008000u, u.y ^ 0x80008000u, u.z ^ 0x80008000u, u.w ^ 0x80008000u);
      *reinterpret_cast<uint4*>(to + row * 128 + 2 * (c / 8) * Layout<DP>::kHalfBytes + (((c & 7) ^ (row & 7)) * 16)) = u;
    }
  }
}

// ------------------------------------------------------------------ kernel
// MAPPED: queries come by TMA.  A tensor map holds no strides of zero or below;
// with those they come by plain loads, in a kernel of its own, as the other one
// has no instructions to spare (117.5 instead of 116.5 us on ragged chunks).
template <typename T, int DP, bool MAPPED>
__global__ void __launch_bounds__(kThreads, 1)
prefill_attention_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const __grid_constant__ Launch p) {
  using L = Layout<DP>;
  constexpr bool kBf16 = !std::is_same<T, __half>::value;
  extern __shared__ __align__(1024) uint8_t smem[];
  Control& s = *reinterpret_cast<Control*>(smem + L::kControl);
  const AttentionParams& a = p.a;
  const moe_kv_cache_t& ca = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / ca.kv_heads;

  if (tid == 0) {
    if (MAPPED) tma_prefetch_map(&q_map);
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.code_full[i], 1);
      mbar_init(&s.code_empty[i], 4);
    }
#pragma unroll 1
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s.full[i], 4);
      mbar_init(&s.empty[i], 1);
    }
#pragma unroll 1
    for (int i = 0; i < kInfo; ++i) mbar_init(&s.info_full[i], 1);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
#pragma unroll 1
      for (int h = 0; h < 2; ++h) mbar_init(&s.p_full[i][h], kTileRows / 32);
      mbar_init(&s.first_done[i], 1);
      mbar_init(&s.o_full[i], 1);
    }
    mbar_init(&s.q_raw, 1);
    mbar_init(&s.q_full, 4);
    mbar_init(&s.q_empty, 1 + 2 * kTileRows / 32);   // the last scores, and every row's thread has its exponent
    mbar_init(&s.drained, 1);
    s.abort_flag = 0;
    fence_mbarrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // The line's length, and where this CTA's stretch of it begins.
  const int entries = a.B * p.row_tiles, per = (entries + kThreads - 1) / kThreads;
  const int from = min(tid * per, entries), to = min(from + per, entries);
  int mine = 0;
#pragma unroll 1
  for (int e = from; e < to; ++e) {
    Entry en;
    en.load(p, e, group);
    if (en.count > 0) mine += en.count + kUnitCost;
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
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) incl += s.sums[w];
    all_tiles += s.sums[w];
  }
  const int total = all_tiles * ca.kv_heads;
  const int ctas = min(static_cast<int>(gridDim.x), max(1, total / kMinTiles));
  if (total == 0) return;

  // Whole units, longest first and to the CTAs forwards and backwards in turn,
  // need no joins.  They are taken where the CTA with the most to do then has
  // no more than a stretch of the line and its joins.  Every CTA finds the
  // same: each thread places one entry and adds up one CTA's share.
  // 512 units of 2 x 2048 tokens: 92 us, cut from the line 104; 220 units of
  // four ragged chunks: 149 and 120.
  bool whole = false;
  if (per == 1) {
    int* costs = reinterpret_cast<int*>(smem + L::kRing);    // not in use yet
    int* sorted = costs + kThreads;
    costs[tid] = mine;
    const int units = __syncthreads_count(mine > 0) * ca.kv_heads, across = gridDim.x;
    if (units <= kMaxUnits * across) {
      int place = 0;
#pragma unroll 1
      for (int e = 0; e < entries; e += 4) {
        const int4 c = *reinterpret_cast<const int4*>(costs + e);
        place += (c.x > mine || (c.x == mine && e < tid)) + (c.y > mine || (c.y == mine && e + 1 < tid)) +
                 (c.z > mine || (c.z == mine && e + 2 < tid)) + (c.w > mine || (c.w == mine && e + 3 < tid));
      }
      if (mine > 0) sorted[place] = tid;
      __syncthreads();
      int share = 0, given = 0;
      if (tid < across) {
#pragma unroll 1
        for (int i = 0; i * across < units; ++i) {
          const int at = i * across + (i % 2 == 0 ? tid : across - 1 - tid);
          if (at >= units) break;
          const int e = sorted[at / ca.kv_heads];
          share += costs[e];
          if (tid == static_cast<int>(blockIdx.x)) {
            s.units[i] = e * ca.kv_heads + at % ca.kv_heads;
            given = i + 1;
          }
        }
      }
      const int most = __reduce_max_sync(0xffffffffu, share);
      if (lane == 0) s.sums[warp] = most;
      if (tid == static_cast<int>(blockIdx.x)) s.given = given;
      __syncthreads();
      int longest = 0;
#pragma unroll 1
      for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, s.sums[w]);
      whole = longest <= (total + ctas - 1) / ctas + kJoinCost;
    }
  }
  if (whole ? s.given == 0 : static_cast<int>(blockIdx.x) >= ctas) return;
  const int x0 = stretch_begin(total, ctas, blockIdx.x);
  if (!whole && x0 < incl * ca.kv_heads && x0 >= (incl - mine) * ca.kv_heads) {
    int before = incl - mine;
#pragma unroll 1
    for (int e = from; e < to; ++e) {
      Entry en;
      en.load(p, e, group);
      const int places = en.count > 0 ? en.count + kUnitCost : 0;
      if (x0 < (before + places) * ca.kv_heads) {
        s.first_entry = e;
        s.first_prefix = before;
        break;
      }
      before += places;
    }
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_alloc(&s.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = s.tmem;
  auto s_cols = [&](int i) { return tmem + 128 * i; };
  auto o_cols = [&](int i) { return tmem + kOColumns + 128 * i; };

  // A wait that runs out, here or in another role, ends the CTA's work: no
  // role then issues a copy or a product or touches TMEM any more.
  auto aborted = [&] { return *static_cast<volatile int*>(&s.abort_flag) != 0; };
  auto wait_one = [&](uint64_t* bar, uint32_t parity) {      // by one thread
    return mbar_try_wait(smem_u32(bar), parity) || wait_long(bar, parity, a.wait_limit_ns, a.status, &s.abort_flag);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) {          // by a warp, which leaves it together
    const bool ok = wait_one(bar, parity);
    return __all_sync(0xffffffffu, ok) != 0;
  };
  Walk& walk = s.walk[warp];
  const Entry& en = walk.en;
  // who walks: a whole warp with the same values, or the one lane that issues the products
  const uint32_t walkers = warp == kMmaWarp ? 1u << lane : 0xffffffffu;
  auto next = [&](bool first) {
    if (first) {
      walk.x = whole ? 0 : x0;
      walk.x1 = whole ? s.given : stretch_begin(total, ctas, blockIdx.x + 1);
    }
    return walk_next(&walk, p, group, whole ? s.units : nullptr, first ? s.first_entry : -1, s.first_prefix, walkers);
  };

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
    bool stop = (a.debug_flags & MOE_DEBUG_STALL_ATTENTION) != 0;      // a failure for the tests: no tile arrives
#pragma unroll 1
    for (bool more = next(true); more && !stop; more = next(false)) {
      if (en.position(en.rows - 1, group) >= static_cast<int64_t>(a.table_width) * ca.page_size) set_status(a.status, MOE_ERR_BAD_PAGE);
      Ahead now = find(0);
#pragma unroll 1
      for (int j = 0; j < walk.n && !stop; ++j) {
        const Ahead later = find(j + 1);
        const int t = issued / 2;
        const bool issues = lane < 16 && now.page >= 0 && (8 * lane) % p.box == 0;
        const unsigned boxes = __ballot_sync(0xffffffffu, issues);
#pragma unroll 1
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
            if (!MAPPED) {
              if (lane == 0) mbar_arrive(&s.q_raw);
            } else if (lane == 0) {
              mbar_arrive_expect_tx(&s.q_raw, L::kHalves * p.unit_rows * 128);
#pragma unroll 1
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
    if (lane == 0) {
      s.issued = issued;
      s.issued_units = units;
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (elect_one()) {
      constexpr uint32_t kScores = idesc_f16(kTileRows, kKeys, false), kValues = idesc_f16(kTileRows, DP, true);
      constexpr uint32_t kSlot = L::kSlotBytes >> 4;
      const uint32_t q_low = desc_low(smem_u32(smem + L::kQ), 16), k_low = desc_low(smem_u32(smem + L::kRing), 16),
                     v_low = desc_low(smem_u32(smem + L::kRing), L::kHalfBytes);
      auto scores = [&](int i, int slot) {
        const uint32_t q = q_low + i * (L::kHalfBytes >> 4), k = k_low + slot * kSlot;
#pragma unroll
        for (int x = 0; x < DP / 16; ++x)
          mma_ss_f16(s_cols(i), q + ((2 * (x / 4) * L::kHalfBytes + (x % 4) * 32) >> 4),
                     k + (((x / 4) * L::kHalfBytes + (x % 4) * 32) >> 4), kScores, x > 0);
        tc_commit(&s.s_full[i]);
      };
      // what the weights of half h of a tile's keys add to O
      auto values = [&](int i, int h, int slot, bool more) {
        const uint32_t v = v_low + slot * kSlot + h * (kHalf * 128 >> 4), w = s_cols(i) + kHalf * h;
#pragma unroll
        for (int x = 0; x < kHalf / 16; ++x) mma_ts_f16(o_cols(i), w + 8 * x, v + (2048 * x >> 4), kValues, more || x > 0);
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
            for (int h = 0; h < 2 && ok; ++h) {
              ok = wait_one(&s.p_full[i][h], p_count[i] & 1);
              if (!ok) break;
              tc_fence_after_sync();
              values(i, h, v % kSlots, j > 0 || h > 0);
              if (h == 0) tc_commit(&s.first_done[i]);
            }
            if (!ok) break;
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
          for (int i = 0; i < tiles; ++i) ++p_count[i];
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
#pragma unroll 1
    for (bool more = next(true); more && good; more = next(false), ++units) {
#pragma unroll 1
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
        // a warp keeps to one half of the columns and every second (fourth) group of 8 keys
        constexpr int kStep = 8 * (4 / L::kHalves);
        const int half = L::kHalves == 2 ? w & 1 : 0, key0 = 8 * (L::kHalves == 2 ? w >> 1 : w) + key8, x = key8;
        src += key0 * 128 + (((4 * half + sub) ^ x) * 16);
        uint8_t* d0 = dst + half * L::kHalfBytes + key0 * 128 + (((2 * sub) ^ x) * 16);
        uint8_t* d1 = dst + half * L::kHalfBytes + key0 * 128 + (((2 * sub + 1) ^ x) * 16);
        auto put = [&](int it, const uint4& c) {
          uint4 f0, f1;
          e4m3x4_to_f16x4(c.x, f0.x, f0.y);
          e4m3x4_to_f16x4(c.y, f0.z, f0.w);
          e4m3x4_to_f16x4(c.z, f1.x, f1.y);
          e4m3x4_to_f16x4(c.w, f1.z, f1.w);
          *reinterpret_cast<uint4*>(d0 + it * kStep * 128) = f0;
          *reinterpret_cast<uint4*>(d1 + it * kStep * 128) = f1;
        };
        if (!drop) {
#pragma unroll
          for (int it = 0; it < kKeys / kStep; ++it) put(it, *reinterpret_cast<const uint4*>(src + it * kStep * 128));
        } else {
#pragma unroll 1
          for (int it = 0; it < kKeys / kStep; ++it) {
            uint4 c = *reinterpret_cast<const uint4*>(src + it * kStep * 128);
            uint32_t seen = 0;
            auto clean = [&](uint32_t& word) {
              const uint32_t bad = __vcmpeq4(word & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              seen |= bad;
              word &= ~bad;
            };
            clean(c.x), clean(c.y), clean(c.z), clean(c.w);
            const int key = key0 + it * kStep, at = tile * kKeys + key;
            nan |= seen != 0 && at >= en.lo && at < en.end && info[key >> 3].valid;      // some row sees it
            put(it, c);
          }
        }
        if (drop && __any_sync(0xffffffffu, nan) && lane == 0) {
          const int n = s.nan_count[units & 1][w]++;
          if (n < kNanTiles) s.nan_tiles[units & 1][w][n] = tile;
        }
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
          // the rows have begun the unit before, so they are done with the one before that
          if (lane == 0) s.nan_count[units & 1][w] = 0;
          if constexpr (!MAPPED) {
            load_queries<T, DP>(a, en, walk.head, group, smem + L::kQ, 32 * w + lane);
            fence_proxy_async_shared();
            __syncwarp();
          }
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
              const int ex = query_exponent(static_cast<int>(max(amax & 0xFFFF, amax >> 16) >> 7) - 127);
              s.q_exponent[row] = static_cast<int8_t>(ex);
              float inv = power_of_two(-ex);
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
          } else if (MAPPED && a.scale < 0.f) {
#pragma unroll 1
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
    const uint32_t sc = s_cols(i) + lanes;
    int t = 0, s_count = 0, o_count = 0, units = 0;
    bool good = true;
#pragma unroll 1
    for (bool more = next(true); more; more = next(false), ++units) {
      // after a timeout a unit's rows are left as they are, but its part in the
      // join is still played, so that the counters end at zero
      good = good && wait(&s.q_full, units & 1);
      const float row_scale = kBf16 ? power_of_two(s.q_exponent[row]) : 1.f;
      // Only now may the next unit's queries come: a unit of one tile has its
      // last scores before its rows' warps have begun it, and two of them
      // would carry q_full past the phase that they wait for.
      // (After a timeout nothing arrives any more: a phase must not get more
      // arrivals than it lacks.)
      __syncwarp();
      if (good && lane == 0) mbar_arrive(&s.q_empty);
      if (kTileRows * i >= en.rows) {
        t += walk.n;
        continue;
      }
      // the CTAs that have parts of the unit, here and not where the result waits
      int cta0 = 0, pieces = 1;
      if (walk.n != en.count) {
        const int first_at = walk.u0 + kUnitCost;
        cta0 = stretch_of(total, ctas, first_at);
        pieces = stretch_of(total, ctas, first_at + en.count - 1) - cta0 + 1;
      }
      const int pos = row < en.rows ? en.position(row, group) : -1;
      // keys below pos_lo are seen by every row of the tile, as far as the window goes
      const int pos_lo = en.position(kTileRows * i, group);
      const int pos_hi = en.position(min(en.rows, kTileRows * (i + 1)) - 1, group) - a.window;
      // weights are relative to 2^base; a row's room is how far the base may
      // still fall, negative before the row's first key.  Rows past the unit's
      // have weights of zero, whatever their queries are.
      float base = row < en.rows ? 0.f : INFINITY, room = -1.f, l = 0.f;

#pragma unroll 1
      for (int j = 0; j < walk.n && good; ++j, ++t, ++s_count) {
        const int tile_key = (en.tile0 + walk.tile + j) * kKeys;
        good = wait(&s.info_full[t % kInfo], (t / kInfo) & 1) && wait(&s.s_full[i], s_count & 1);
        if (!good) break;
        tc_fence_after_sync();

        // 64 keys at a time: their scores to weights, which go over scores
        // that have been read, and on to the products
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const Group* info = s.group[t % kInfo] + 8 * h;
          const int key0 = tile_key + kHalf * h;
          const uint32_t sh = sc + kHalf * h;
          uint32_t ra[32], rb[32];
          tmem_ld32(sh, ra);
          tmem_ld32(sh + 32, rb);
          tmem_wait(ra);
          tmem_wait(rb);
          const bool all = __all_sync(0xffffffffu, info[lane & 7].valid) && key0 + kHalf - 1 <= pos_lo && (a.window == 0 || key0 > pos_hi);
          float top = -INFINITY;
          auto exponents = [&](uint32_t (&r)[32], int c) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float2 gi = *reinterpret_cast<const float2*>(&info[4 * c + g]);
              const float kk = gi.x * row_scale, off = gi.y - base;
#pragma unroll
              for (int e = 8 * g; e < 8 * g + 8; e += 2) {
                r[e] = __float_as_uint(fmaf(__uint_as_float(r[e]), kk, off));
                r[e + 1] = __float_as_uint(fmaf(__uint_as_float(r[e + 1]), kk, off));
              }
            }
            if (!all) {
              // which of the 32 keys this row sees, a bit each: [first, last]
              const int first = a.window > 0 ? pos - a.window + 1 - key0 - 32 * c : 0, last = pos - key0 - 32 * c;
              uint32_t mask = last < 0 ? 0u : last >= 31 ? 0xffffffffu : (2u << last) - 1u;
              mask &= first <= 0 ? 0xffffffffu : first > 31 ? 0u : ~((1u << first) - 1u);
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (!info[4 * c + g].valid) mask &= ~(0xFFu << (8 * g));
#pragma unroll
              for (int e = 0; e < 32; ++e) r[e] = (mask >> e) & 1 ? r[e] : 0xFF800000u;
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              auto x = [&](int e) { return __uint_as_float(r[8 * g + e]); };
              top = max3(top, max3(x(0), x(1), x(2)), max3(max3(x(3), x(4), x(5)), x(6), x(7)));
            }
          };
          exponents(ra, 0);
          exponents(rb, 1);
          const bool above = top > (room < 0.f ? -INFINITY : kMost), below = all && j % kLook == 0 && top < kLow && room > 0.f;
          if (__any_sync(0xffffffffu, above | below)) {
            // New references: what this unit has summed so far becomes relative
            // to them.  A row that would rise by less gets one too, since it
            // costs nothing more (without: 107 instead of 99 us on 2 x 2048
            // tokens with scores of standard deviation 3).
            const float rise = room < 0.f ? (top > -INFINITY ? top - kNew : 0.f) : top > kNew ? top - kNew : below ? fmaxf(top - kBack, -room) : 0.f;
            const float keep = room < 0.f ? 0.f : fast_exp2(-rise);
            base += rise;
            room = room >= 0.f ? fminf(room + rise, kRoom) : top > -INFINITY ? kRoom : room;
            l *= keep;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              ra[e] = __float_as_uint(__uint_as_float(ra[e]) - rise);
              rb[e] = __float_as_uint(__uint_as_float(rb[e]) - rise);
            }
            // O: the tiles before came before these scores, this tile's first half has its own word
            if (h > 0) {
              good = wait(&s.first_done[i], s_count & 1);
              if (!good) break;
              tc_fence_after_sync();
            }
            if (j > 0 || h > 0) {
#pragma unroll 1
              for (int d = 0; d < DP; d += 16) {
                float o[16];
                tmem_ld16(sc + kOColumns + d, o);
                uint32_t now[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) now[e] = __float_as_uint(o[e] * keep);
                tmem_st16(sc + kOColumns + d, now);
              }
            }
          }
          // The denominator grows by 64 keys at a time.  8 at a time, what
          // many small weights add to a large one was rounded the same way
          // each time (lse off by 1e-3 on 131072 keys).
          float part = 0.f;
          auto weights = [&](uint32_t (&r)[32], int c) {
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
              part = fmaf(s0 + s1, info[4 * c + g].inv_v, part);
            }
            tmem_st16(sh + 16 * c, wd);
          };
          weights(ra, 0);
          weights(rb, 1);
          l += part;
          tmem_wait_st();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.p_full[i][h]);
          __syncwarp();                    // the next scores, or sums, are read by the warp as one
        }
      }

      // ---------------------------------------------------------- output
      const bool live = row < en.rows;
      good = good && wait(&s.o_full[i], o_count++ & 1);
      tc_fence_after_sync();
      // NaN values that were left out of partly hidden tiles, for the rows that
      // see them: of the tiles that were noted, one after another, or of all
      // where a warp met more of them than it could note
      uint32_t nan[4] = {};
      bool any_nan = false;
      const int(&counts)[4] = s.nan_count[units & 1];
      if (good && (counts[0] | counts[1] | counts[2] | counts[3]) != 0) {
        const int first = en.tile0 + walk.tile, end = first + walk.n;
#pragma unroll 1
        for (int at = first; at < end; ++at) {
          int tile = end;
#pragma unroll 1
          for (int w = 0; w < 4; ++w) {
            if (counts[w] > kNanTiles) tile = at;
#pragma unroll 1
            for (int e = 0; e < min(counts[w], kNanTiles); ++e) {
              const int noted = s.nan_tiles[units & 1][w][e];
              if (noted >= at) tile = min(tile, noted);
            }
          }
          if (tile == end) break;
          at = tile;
          if (live) {
            const int k0 = max(tile * kKeys, a.window > 0 ? pos - a.window + 1 : 0), k1 = min(min(pos, en.end - 1), tile * kKeys + kKeys - 1);
            const uint4 bits = nan_columns(a, en.b, walk.head, k0, k1);
            nan[0] |= bits.x, nan[1] |= bits.y, nan[2] |= bits.z, nan[3] |= bits.w;
          }
        }
        any_nan = (nan[0] | nan[1] | nan[2] | nan[3]) != 0;
      }
      const float m = room < 0.f ? -INFINITY : base;
      const int gr = en.row0 + row, tok = en.q_first + gr / group, h = walk.head * group + gr % group;
      T* dst = static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head;
      const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // whole sectors at a time
      auto put = [&](int d, const float (&v)[32], float inv) {        // columns [d, d + 32)
#pragma unroll
        for (int e = 0; e < 32; e += 16) {
          if (d + e >= ca.head_dim) continue;
          Pack<T, 16> y;
#pragma unroll
          for (int z = 0; z < 16; ++z) y.v[z] = from_f32<T>(v[e + z] * inv);
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&y);
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + d + e), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                         "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          } else {
            *reinterpret_cast<uint4*>(dst + d + e) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + d + e + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      };
      auto put_lse = [&](float mm, float ll) {
        if (a.lse != nullptr) a.lse[static_cast<int64_t>(tok) * a.Hq + h] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
      };
      // O's columns [d, d + 32): read by the warp as one, which it need not be after rows of its own
      auto summed = [&](int d, float (&v)[32]) {
        uint32_t r[32] = {};
        __syncwarp();
        if (good) {
          tmem_ld32(sc + kOColumns + d, r);
          tmem_wait(r);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]);
        if (any_nan) {
          const uint32_t bits = nan[d / 32];
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if ((bits >> e) & 1) v[e] = __uint_as_float(0x7FC00000u);
        }
      };
      if (walk.n == en.count) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
          float v[32];
          summed(d, v);
          if (live) put(d, v, inv);
        }
        if (live) put_lse(m, l);
        tc_fence_before_sync();
        continue;
      }

      // A part of the unit: pieces of it are in consecutive CTAs.  Eight at a
      // time are joined by whoever finishes last among them, then those
      // results likewise.  Who finds all others done need not write its own.
      float4* parts = reinterpret_cast<float4*>(p.workspace);
      float2* ml = reinterpret_cast<float2*>(p.workspace + kPartialBytes);
      int* counters = reinterpret_cast<int*>(p.workspace + kPartialBytes + kMlBytes);
      const int mine_at = static_cast<int>(blockIdx.x) - cta0;
      // two slots a CTA: for the unit that began before its stretch, and for one that began in it
      auto slot_of = [&](int piece) { return (2 * (cta0 + piece) + (piece == 0 ? 1 : 0)) * 2 + i; };
      const int r = row & 127;
      auto part = [&](int slot, int d) { return parts + (static_cast<size_t>(slot) * 32 + d / 4) * kTileRows + r; };
      float m_own = m, l_own = l;
      int step = 1;
#pragma unroll 1
      for (int level = 0;; ++level) {
        const int lead = mine_at / (kJoin * step) * (kJoin * step), count = min(kJoin, (pieces - lead + step - 1) / step);
        const int own = (mine_at - lead) / step;                       // this result's place among them
        int* counter = counters + level * 2 * kParts + slot_of(lead);
        const bool kept = level == 0;                                  // O is still in TMEM
        if ((tid & 127) == 0) s.last[i] = kept && ld_acquire_gpu(counter) == count - 1;
        named_barrier_sync(1 + i, kTileRows);
        bool last = s.last[i] != 0;
        const bool unwritten = last;
        if (!unwritten) {
          if (kept) {
#pragma unroll 1
            for (int d = 0; d < DP; d += 32) {
              float v[32];
              summed(d, v);
#pragma unroll
              for (int e = 0; e < 32; e += 4) __stcg(part(slot_of(lead + own * step), d + e), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
            }
            __stcg(ml + static_cast<size_t>(slot_of(lead + own * step)) * kTileRows + r, make_float2(m_own, l_own));
          }
          __threadfence();
          named_barrier_sync(1 + i, kTileRows);
          if ((tid & 127) == 0) s.last[i] = atomicAdd(counter, 1) == count - 1;
          named_barrier_sync(1 + i, kTileRows);
          last = s.last[i] != 0;
        }
        named_barrier_sync(1 + i, kTileRows);
        if (!last) break;
        if ((tid & 127) == 0) *counter = 0;                            // ready for the next call
        __threadfence();
        const bool finish = lead == 0 && count * step >= pieces;
        auto ml_of = [&](int q) {
          return unwritten && q == own ? make_float2(m_own, l_own)
                                       : __ldcg(ml + static_cast<size_t>(slot_of(lead + q * step)) * kTileRows + r);
        };
        float2 parts_ml[kJoin];                                        // read together
#pragma unroll
        for (int q = 0; q < kJoin; ++q) parts_ml[q] = q < count ? ml_of(q) : make_float2(-INFINITY, 0.f);
        float mx = -INFINITY, lx = 0.f;
#pragma unroll
        for (int q = 0; q < kJoin; ++q) mx = fmaxf(mx, parts_ml[q].x);
        const float ref = mx == -INFINITY ? 0.f : mx;
        float factor[kJoin];
#pragma unroll
        for (int q = 0; q < kJoin; ++q) {
          factor[q] = fast_exp2(parts_ml[q].x - ref);
          lx = fmaf(parts_ml[q].y, factor[q], lx);
        }
        const float inv = lx == 0.f ? 0.f : 1.f / lx;
#pragma unroll 1
        for (int d = 0; d < DP; d += 32) {
          float v[32] = {};
#pragma unroll 1
          for (int q = 0; q < count; ++q) {
            const float f = factor[q];
            float y[32];
            if (unwritten && q == own) {
              summed(d, y);
            } else {
              const float4* from_part = part(slot_of(lead + q * step), d);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 w = __ldcg(from_part + e * kTileRows);
                y[4 * e] = w.x, y[4 * e + 1] = w.y, y[4 * e + 2] = w.z, y[4 * e + 3] = w.w;
              }
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = fmaf(y[e], f, v[e]);
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
        step *= kJoin;
      }
      tc_fence_before_sync();
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  // Nothing of this CTA is in flight when it ends: every copy has been waited
  // for, unless a wait ran out.
  if (warp == kLoadWarp && aborted()) {
#pragma unroll 1
    for (int k = max(0, s.issued - kStages); k < s.issued; ++k) mbar_wait(&s.code_full[k % kStages], (k / kStages) & 1, a.wait_limit_ns);
    if (s.issued_units > 0) mbar_wait(&s.q_raw, (s.issued_units - 1) & 1, a.wait_limit_ns);
  }
}

template <typename T, int DP, bool MAPPED>
int launch(const AttentionParams& a, cudaStream_t stream) {
  CUtensorMap q_map = {}, k_map, v_map;
  Launch p = {};
  p.a = a;
  p.workspace = static_cast<uint8_t*>(a.workspace) + decode_attention_workspace_bytes();
  p.box = 8;
  while (p.box < kKeys && a.cache.page_size % (2 * p.box) == 0) p.box *= 2;
  const int group = a.Hq / a.cache.kv_heads;
  p.unit_rows = kCtaRows / group * group;
  if (!encode_cache_map(&k_map, a.cache, false, p.box) || !encode_cache_map(&v_map, a.cache, true, p.box) ||
      (MAPPED && !encode_query_map(&q_map, a, std::is_same<T, __half>::value, group, kCtaRows / group)))
    return MOE_ERR_CUDA;
  auto kernel = prefill_attention_kernel<T, DP, MAPPED>;
  constexpr int bytes = Layout<DP>::kBytes;
  if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes) != cudaSuccess) return MOE_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int64_t row_tiles = (static_cast<int64_t>(a.max_q_len) * group + p.unit_rows - 1) / p.unit_rows;
  const int64_t line = row_tiles * a.B * ((static_cast<int64_t>(a.table_width) * a.cache.page_size) / kKeys + 1 + kUnitCost) * a.cache.kv_heads;
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
cudaError_t clear_prefill_counters(void* workspace, cudaStream_t s) {
  return cudaMemsetAsync(static_cast<uint8_t*>(workspace) + decode_attention_workspace_bytes() + kPartialBytes + kMlBytes, 0, kCounterBytes, s);
}

namespace {
template <typename T>
int launch_type(const AttentionParams& p, cudaStream_t s) {
  const bool mapped = p.q_token > 0 && p.q_head > 0;
  if (p.cache.head_dim <= 64) return mapped ? launch<T, 64, true>(p, s) : launch<T, 64, false>(p, s);
  return mapped ? launch<T, 128, true>(p, s) : launch<T, 128, false>(p, s);
}
}  // namespace

int launch_prefill_attention(const AttentionParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DTYPE_F16 ? launch_type<__half>(p, s) : launch_type<__nv_bfloat16>(p, s);
}

}  // namespace moe
