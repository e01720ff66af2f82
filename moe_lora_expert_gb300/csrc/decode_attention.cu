// Attention of a few new tokens over the paged cache: decode, and the few
// tokens a draft proposes.
//
// Each key head's rows (new tokens x query heads of its group) are cut into
// tiles of 8 or 16 and the keys into tiles of 64.  All (row tile, key tile)
// pairs of the call form one line, which the CTAs of the grid share in equal
// stretches whatever the sequences' lengths are; a row tile whose keys lie in
// several stretches is joined by the CTA that finishes it last.
//
// Mathematics.  With t_j = log2(e) scale k_scale (q . k_j) the weights are
//   w_j = 2^(t_j + log2(v_scale) - m),  m a reference that follows the keys,
//   out = sum_j w_j code_j / sum_j (w_j / v_scale),
// so w_j is what multiplies the codes, whatever the pages' scales are, and
// both sums stay in float32.  Codes enter the tensor cores as float16, which
// holds each exactly; so it does q, down to 2^-31 of a bf16 row's largest
// value (a power of two is taken out of the row), and the scores are products
// summed in float32.  The weights are rounded to float16: 2^-12 of each that
// is normal, an eighth of what a bf16 output is rounded by and as much as a
// float16 one is (whose error grows from 2.1e-4 to 2.9e-4 by it; two parts to
// each weight would take it out at twice the products).
// Float16 ends at 2^16 and has full precision down to 2^-14 (2^-25 is 0), so m
// puts the largest weight of each warp's 16 keys of a tile between 2^-8 and
// 2^15.9: it rises when one would pass that, and falls again when all are below.
// With m the running maximum alone, one key that takes nearly all of the mass
// (and whose values may be zero) took the weights of the thousands after it
// away from the output but not from its denominator.  m falls by 2^24 at most
// below where it stood highest, and the sums stay inside float32: what is then
// still lost is under 2^-56 of the largest weight for each key.
// A fall costs a pass over the sums, and where scores are far apart low tiles
// lie between others, so that m would have to rise again.  It therefore falls
// no further than it has to, at every eighth tile, and not for tiles at the
// end of what a row sees, which have few keys.  The tiles in between lose under
// 2^-32 of the weight that made m rise, for each key: 2^-23 of the values'
// range in all.  (64 sequences of 16384 keys with scores of standard deviation
// 1, 6 and 12: 176, 176 and 179 us, 175 each without the fall; falling in any
// tile under 2^0, to 2^8: 177, 204 and 206.)
//
// What bounds it: one pass over the cache's bytes.  64 sequences of up to
// 32768 keys (8 query heads of 128 on each of 4 key heads) take 214 us, 6.3
// TB/s, 92% of the copy rate; one token on 262140 keys 57 us (40 at the copy
// rate: the first tiles come after 8 us and the join takes 5).  At smaller
// sizes it is the chain of latencies from the lengths to the block table, the
// first tile, and the join: one token on 1022 keys 11 us.
//
// Why mma.sync.  The products of 8 rows are far below even its rate, and its
// fragments go from shared memory to registers: a warp reads each code once,
// converts it (two codes an instruction) and multiplies.  A tcgen05 tile is
// 128 keys high and its codes would have to be converted and written back to
// shared memory first, or q and the weights split into three e4m3 parts each.
// The keys are the rows of the products and the query rows their columns, so
// that 8 rows fill an m16n8k16 (as the rows of the products they fill half of
// one: 291 us instead of 217 on the 64 sequences, with twice the products,
// weights and sums a key).
#include <cuda.h>

#include <type_traits>

#include "attention.cuh"
#include "attention_line.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kKeys = 64;                 // keys of a tile
constexpr int kMaxRows = 16;              // most rows of a row tile: 8 NT
constexpr int kWarps = 4;                 // 16 keys of a tile each
constexpr int kThreads = 32 * kWarps;
constexpr int kRing = 3;                  // tiles in a warp's ring (2 and 4 are no faster)
constexpr int kBatch = 16;                // tiles whose pages are looked up at once
// 8 rows: 3 CTAs of 168 registers (2: 262 instead of 217 us on 64 sequences of up to 32768 keys); 16 rows: 2 of 250 (3 of 168 spill:
// 82 instead of 50 us on 8 sequences of 16384 keys).
constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }
constexpr int kMaxCtas = 640;
constexpr int kMaxEntries = 512;          // (sequence, row tile) pairs of one launch
constexpr int kMinTiles = 2;              // a CTA's stretch of the line is at least so long; one token on 1022 keys: 1 13.0, 2 11.3, 4 12.7 us
constexpr int kJoin = 16;                 // pieces that are joined at a time; 16 sequences of up to 4096 keys: 8 27.6, 16 24.5 us
constexpr int kPitch = 128;               // bytes of a key in shared memory
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kMost = 15.9f, kNew = 7.f;// a weight past 2^15.9 makes the reference rise, so that it becomes 2^7;
constexpr float kLow = -8.f, kBack = -5.f;// all of a tile's under 2^-8 make it fall, so that the largest becomes 2^-5,
constexpr float kRoom = 24.f;             // by 2^24 at most below its highest,
constexpr int kLook = 8;                  // looked for at every eighth tile
constexpr float kNone = -3.0e38f;         // the reference before any key: every weight is 0 next to it, and its sums are

struct alignas(16) Group {                // 8 keys of a tile, which lie in one page
  float k;                                // log2(e) * scale * k_scale
  float lv;                               // log2(v_scale)
  float inv_v;                            // 1 / v_scale
  int valid;
};

struct Shared {
  Group group[kWarps][2][2 * kBatch];     // of two batches of tiles
  uint64_t full[kWarps][kRing];
  int prefix[kMaxEntries + 1];            // key tiles before each entry
  int begin[kMaxEntries];                 // first key that some row of each entry sees
  int end[kMaxEntries];                   // end of the keys that some row of it sees
  float m[kWarps][kMaxRows], l[kWarps][kMaxRows];
  int total, abort_flag, last;
};
constexpr int kSlotBytes = 2 * 16 * kPitch;
constexpr int kScratch(int rows) { return 2 * rows * 128 * 4; }              // two warps' sums
constexpr int kSmem(int rows) { return kWarps * kRing * kSlotBytes + kScratch(rows) + static_cast<int>(sizeof(Shared)) + 1024; }

// Partial sums of a row tile: [slot][row][128] and (m, l) [slot][row][2];
// counters [2][slots].
constexpr int kSlots = 2 * kMaxCtas;
constexpr size_t kPartialBytes = static_cast<size_t>(kSlots) * kMaxRows * 128 * 4;
constexpr size_t kMlBytes = static_cast<size_t>(kSlots) * kMaxRows * 2 * 4;
constexpr size_t kCounterBytes = static_cast<size_t>(kSlots) * 2 * 4;

struct Launch {
  AttentionParams a;
  int b0, B, row_tiles, tile_rows;        // sequences [b0, b0 + B), row tiles of each and their rows
  int box;                                // keys of one TMA box: gcd(page_size, 16)
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8 x 8 block of 16-bit values, thread (g, c) with (row g, columns 2c and
// 2c + 1), to its transpose.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// The rows of entry e (a sequence and a row tile of it).
struct Entry {
  int b, q_first, q_len, len, row0, rows;
  __device__ __forceinline__ Entry(const Launch& p, int e, int group) {
    b = p.b0 + e / p.row_tiles;
    row0 = (e % p.row_tiles) * p.tile_rows;
    q_first = p.a.cu_q == nullptr ? b : p.a.cu_q[b];
    q_len = p.a.cu_q == nullptr ? 1 : p.a.cu_q[b + 1] - q_first;
    len = p.a.seq_lens[b];
    const int n = min(min(q_len, p.a.max_q_len), p.a.N - q_first);
    rows = max(0, min(p.tile_rows, n * group - row0));
  }
  __device__ __forceinline__ int position(int row, int group) const { return len - q_len + (row0 + row) / group; }
};

// Where tile x of the line lies.
struct Place {
  int e, head, tile, count;
  __device__ __forceinline__ Place(const Shared& s, int entries, int kv_heads, int x) {
    int lo = 0, hi = entries;              // the last entry with prefix * heads <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s.prefix[mid] * kv_heads <= x) lo = mid; else hi = mid;
    }
    e = lo;
    count = s.prefix[e + 1] - s.prefix[e];
    const int in = x - s.prefix[e] * kv_heads;
    head = in / count;
    tile = in - head * count;
  }
};

// Removes the NaN codes of a word and remembers that there were some.
__device__ __forceinline__ uint32_t drop_nan(uint32_t w, uint32_t& seen) {
  const uint32_t nan = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  seen |= nan;
  return w & ~nan;
}

template <typename T, int DP, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT))
decode_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, const __grid_constant__ Launch p) {
  extern __shared__ uint8_t raw[];
  uint8_t* const rings = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  float* const scratch = reinterpret_cast<float*>(rings + kWarps * kRing * kSlotBytes);
  Shared& s = *reinterpret_cast<Shared*>(reinterpret_cast<uint8_t*>(scratch) + kScratch(8 * NT));
  const AttentionParams& a = p.a;
  const moe_kv_cache_t& ca = a.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = a.Hq / ca.kv_heads, entries = p.B * p.row_tiles;
  constexpr int kWords = DP / 16;          // 4-code words of a key in one thread: K steps
  constexpr int kTiles = DP / 16;          // output tiles of 16 columns

  if (tid == 0) {
    tma_prefetch_map(&k_map);
    tma_prefetch_map(&v_map);
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w)
#pragma unroll 1
      for (int i = 0; i < kRing; ++i) mbar_init(&s.full[w][i], 1);
    s.abort_flag = 0;
    fence_mbarrier_init();
  }
  pdl_launch_dependents();
  pdl_wait();

  // The line: each entry's key tiles, one at least so that someone writes its rows.
  const int64_t most = static_cast<int64_t>(a.table_width) * ca.page_size;
#pragma unroll 1
  for (int e = tid; e < entries; e += kThreads) {
    const Entry en(p, e, group);
    int n = 0, lo = 0, hi = 0;
    if (en.rows > 0) {
      const int pos0 = en.position(0, group), pos1 = en.position(en.rows - 1, group);
      lo = a.window > 0 && pos0 >= a.window ? pos0 + 1 - a.window : 0;
      hi = max(0, pos1 + 1);
      if (hi > most) {
        hi = static_cast<int>(most);
        set_status(a.status, MOE_ERR_BAD_PAGE);
      }
      n = max(1, (hi + kKeys - 1) / kKeys - lo / kKeys);
    }
    s.prefix[e + 1] = n;
    s.begin[e] = lo;
    s.end[e] = hi;
  }
  __syncthreads();
  if (warp == 0) {
    const int per = (entries + 31) / 32, from = min(lane * per, entries), to = min(from + per, entries);
    int sum = 0;
#pragma unroll 1
    for (int e = from; e < to; ++e) sum += s.prefix[e + 1];
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
#pragma unroll 1
    for (int e = from; e < to; ++e) {
      run += s.prefix[e + 1];
      s.prefix[e + 1] = run;
    }
    if (lane == 0) s.prefix[0] = 0;
    if (lane == 31) s.total = incl * ca.kv_heads;
  }
  __syncthreads();
  const int total = s.total, ctas = min(static_cast<int>(gridDim.x), (total + kMinTiles - 1) / kMinTiles);
  const bool idle = static_cast<int>(blockIdx.x) >= ctas;
  const int x0 = idle ? 0 : stretch_begin(total, ctas, blockIdx.x), x1 = idle ? 0 : stretch_begin(total, ctas, blockIdx.x + 1);

  auto wait = [&](uint64_t* bar, uint32_t parity) {          // by a warp, which leaves it together
    if (!mbar_try_wait(smem_u32(bar), parity)) wait_long(bar, parity, a.wait_limit_ns, a.status, &s.abort_flag);
    __syncwarp();
  };

  // Each warp streams its own 16 keys of every tile through a ring of its own:
  // it issues the copies three tiles ahead, and no warp waits for another.
  // Two lanes stand for a tile, one for each group of 8 keys; the 32 lanes
  // look up the pages of 16 tiles at once, two batches ahead, and their scales
  // one batch ahead.
  struct Ahead {
    int page, off, head;
    float ks, vs;
  };
  const int steps = x1 - x0;
  auto find = [&](int batch) {
    Ahead f = {-1, 0, 0, 0.f, 0.f};
    const int k = batch * kBatch + (lane >> 1);
    if (k < steps) {
      const Place at(s, entries, ca.kv_heads, x0 + k);
      const int key = (s.begin[at.e] / kKeys + at.tile) * kKeys + 16 * warp + 8 * (lane & 1);
      // boxes that no row sees are not looked up: their pages may be gone
      if (key < s.end[at.e] && (key & ~(p.box - 1)) + p.box > s.begin[at.e]) {
        const int page_at = key / ca.page_size;
        f.off = key - page_at * ca.page_size;
        f.head = at.head;
        f.page = a.block_table[static_cast<int64_t>(p.b0 + at.e / p.row_tiles) * a.table_width + page_at];
        if (f.page < 0 || f.page >= ca.num_pages) {
          f.page = -1;
          set_status(a.status, MOE_ERR_BAD_PAGE);
        }
      }
    }
    return f;
  };
  auto fetch = [&](Ahead& f) {
    if (f.page >= 0) {
      const int64_t i = static_cast<int64_t>(f.page) * ca.kv_heads + f.head;
      f.ks = ca.k_scale[i];
      f.vs = ca.v_scale[i];
    }
  };
  // The scales of a batch, where its tiles' weights will look for them.
  auto put_scales = [&](int batch, const Ahead& f) {
    const float vs = fmaxf(f.vs, 5.421010862427522e-20f);              // 2^-64: a zero scale gives zero values
    s.group[warp][batch & 1][lane] = {f.ks * a.scale * kLog2e, log2f(vs), 1.f / vs, f.page >= 0};
  };
  Ahead now = find(0), next, later;
  int issued = 0;
  const bool stalled = (a.debug_flags & MOE_DEBUG_STALL_ATTENTION) != 0;   // a failure for the tests: no tile arrives
  auto issue = [&]() {
    if (issued >= steps || stalled) return;
    if (__any_sync(0xffffffffu, *static_cast<volatile int*>(&s.abort_flag))) return;   // a slot that was not filled is not filled again
    const int in = issued % kBatch, slot = issued % kRing;
    if (in == 0 && issued > 0) {
      // the batch before last has been weighed: kRing tiles at most are between its last and this one's first
      now = next;
      put_scales(issued / kBatch, now);
      next = later;
      fetch(next);
      later = find(issued / kBatch + 2);
    }
    const bool mine = (lane >> 1) == in, issues = mine && now.page >= 0 && (now.off & (p.box - 1)) == 0;
    const unsigned boxes = __ballot_sync(0xffffffffu, issues);
    if (lane == 0) mbar_arrive_expect_tx(&s.full[warp][slot], __popc(boxes) * p.box * kPitch * 2);
    __syncwarp();
    if (issues) {
      const uint32_t dst = smem_u32(rings + (warp * kRing + slot) * kSlotBytes) + 8 * (lane & 1) * kPitch;
      tma_load_4d(dst, &k_map, &s.full[warp][slot], now.off, now.head, now.page);
      tma_load_4d(dst + 16 * kPitch, &v_map, &s.full[warp][slot], now.off, now.head, now.page);
    }
    ++issued;
  };
#pragma unroll 1
  for (int i = 0; i < kRing; ++i) issue();
  fetch(now);
  if (steps > kBatch) {
    next = find(1);
    later = find(2);
  }
  put_scales(0, now);
  if (steps > kBatch) fetch(next);
  __syncwarp();

  {
    const int g = lane >> 2, c = lane & 3;
    int taken = 0;                         // tiles consumed so far
#pragma unroll 1
    for (int x = x0; x < x1;) {
      const Place at(s, entries, ca.kv_heads, x);
      const Entry en(p, at.e, group);
      const int n = min(at.count - at.tile, x1 - x);
      const int first_tile = s.begin[at.e] / kKeys + at.tile;
      const int pos_min = en.position(0, group), pos_max = en.position(en.rows - 1, group);
      const int end = s.end[at.e];

      // Q^T as the B operand: K step w, column pair (0, 1) in b0 and (2, 3) in
      // b1 are columns DP/4 * c + 4 w + (0..3), the order in which a thread
      // reads the codes of a key.
      uint32_t qf[NT][kWords][2];
      float row_scale[NT][2];
      int pos[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + g, row = en.row0 + r, tok = en.q_first + row / group, h = at.head * group + row % group;
        const T* src = static_cast<const T*>(a.q) + tok * a.q_token + h * a.q_head;
        float q[DP / 4], amax = 0.f, scale = 1.f;
#pragma unroll
        for (int d = 0; d < DP / 4; d += 8) {
          const int col = DP / 4 * c + d;
          float v[8] = {};
          if (r < en.rows && col < ca.head_dim) load_f32<T, 8>(src + col, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            q[d + j] = v[j];
            amax = fmaxf(amax, fabsf(v[j]));
          }
        }
        if constexpr (!std::is_same<T, __half>::value) {
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          const int ex = query_exponent(static_cast<int>(__float_as_uint(amax) >> 23) - 127);
          scale = power_of_two(ex);
          const float inv = power_of_two(-ex);
#pragma unroll
          for (int d = 0; d < DP / 4; ++d) q[d] *= inv;
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          qf[t][w][0] = f32x2_to_f16x2(q[4 * w], q[4 * w + 1]);
          qf[t][w][1] = f32x2_to_f16x2(q[4 * w + 2], q[4 * w + 3]);
        }
        // a thread's scores belong to rows 2 c and 2 c + 1
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          row_scale[t][z] = __shfl_sync(0xffffffffu, scale, 4 * (2 * c + z));
          const int rz = 8 * t + 2 * c + z;
          pos[t][z] = rz < en.rows ? en.position(rz, group) : -1;
        }
      }

      float o[NT][kTiles][4];
      float m[NT][2], least[NT][2], l[NT][2];   // least: what m may fall to
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int j = 0; j < kTiles; ++j) o[t][j][0] = o[t][j][1] = o[t][j][2] = o[t][j][3] = 0.f;
#pragma unroll
        for (int z = 0; z < 2; ++z) m[t][z] = least[t][z] = kNone, l[t][z] = 0.f;
      }

#pragma unroll 1
      for (int i = 0; i < n; ++i, ++taken) {
        const int slot = taken % kRing;
        wait(&s.full[warp][slot], (taken / kRing) & 1);
        const int key0 = (first_tile + i) * kKeys + 16 * warp;
        const uint8_t* kt = rings + (warp * kRing + slot) * kSlotBytes;
        const uint8_t* vt = kt + 16 * kPitch;
        const Group* groups = &s.group[warp][taken / kBatch & 1][2 * (taken % kBatch)];
        const Group g0 = groups[0], g1 = groups[1];
        const bool some = key0 < end && (a.window == 0 || key0 + 15 > pos_min - a.window) && (g0.valid || g1.valid);
        if (some) {
          // S^T = K Q^T for 16 keys: sc[t] = (key g, rows 2c and 2c + 1), (key g + 8, the same)
          float sc[NT][4] = {};
          uint4 kw[2][DP / 64];
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < DP / 64; ++u)
              kw[h][u] = *reinterpret_cast<const uint4*>(kt + (8 * h + g) * kPitch + (((DP / 64) * c + u) ^ g) * 16);
#pragma unroll
          for (int w = 0; w < kWords; ++w) {
            auto word = [&](const uint4& u) { return (w & 3) == 0 ? u.x : (w & 3) == 1 ? u.y : (w & 3) == 2 ? u.z : u.w; };
            uint32_t af[4];
            e4m3x4_to_f16x4(word(kw[0][w / 4]), af[0], af[2]);
            e4m3x4_to_f16x4(word(kw[1][w / 4]), af[1], af[3]);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(sc[t], af, qf[t][w][0], qf[t][w][1]);
          }
          // V while the scores are on their way: DP / 8 columns of four keys
          uint32_t vw[4][kTiles / 2];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const int key = 8 * (h >> 1) + 2 * c + (h & 1);
            if constexpr (DP == 128) {
              const uint4 u = *reinterpret_cast<const uint4*>(vt + key * kPitch + ((g ^ (key & 7)) * 16));
              vw[h][0] = u.x, vw[h][1] = u.y, vw[h][2] = u.z, vw[h][3] = u.w;
            } else {
              const uint2 u = *reinterpret_cast<const uint2*>(vt + key * kPitch + (((g >> 1) ^ (key & 7)) * 16) + 8 * (g & 1));
              vw[h][0] = u.x, vw[h][1] = u.y;
            }
          }
          // exponents of the weights, and whether some reference has to move
          const bool whole = key0 + 15 <= pos_min && (a.window == 0 || key0 > pos_max - a.window) && g0.valid && g1.valid;
          bool move = false;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const Group& gr = j < 2 ? g0 : g1;
              float y = fmaf(sc[t][j], gr.k * row_scale[t][j & 1], gr.lv);
              if (!whole) {
                const int key = key0 + (j < 2 ? 0 : 8) + g, ps = pos[t][j & 1];
                if (!gr.valid || key > ps || (a.window > 0 && key <= ps - a.window)) y = -INFINITY;
              }
              sc[t][j] = y;
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) move |= fmaxf(sc[t][z], sc[t][z + 2]) > m[t][z] + kMost;
          }
          const bool look = whole && i % kLook == 0;
          if (look) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int z = 0; z < 2; ++z) {  // a row's 16 keys are with the 8 lanes of the same c
                const unsigned up = __ballot_sync(0xffffffffu, !(fmaxf(sc[t][z], sc[t][z + 2]) < m[t][z] + kLow));
                move |= (up & 0x11111111u << c) == 0 && m[t][z] > least[t][z];
              }
          }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                float top = fmaxf(sc[t][z], sc[t][z + 2]);
#pragma unroll
                for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                float now = m[t][z];
                if (top > m[t][z] + kNew) now = top - kNew;
                if (look && top < m[t][z] + kLow && m[t][z] > least[t][z]) now = fmaxf(top - kBack, least[t][z]);
                const float keep = fast_exp2(m[t][z] - now);
                m[t][z] = now;
                least[t][z] = fmaxf(least[t][z], now - kRoom);
                l[t][z] *= keep;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                  o[t][j][z] *= keep;
                  o[t][j][2 + z] *= keep;
                }
              }
          }
          // P^T as the B operand: the weights' 8 x 8 blocks transposed
          uint32_t pf[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w0 = fast_exp2(sc[t][2 * h] - m[t][0]), w1 = fast_exp2(sc[t][2 * h + 1] - m[t][1]);
              const float inv_v = h == 0 ? g0.inv_v : g1.inv_v;
              l[t][0] = fmaf(w0, inv_v, l[t][0]);
              l[t][1] = fmaf(w1, inv_v, l[t][1]);
              pf[t][h] = transpose_8x8(f32x2_to_f16x2(w0, w1));
            }
          uint32_t nan = 0;
          if (!whole) {                    // a weight of zero times a NaN code would be NaN
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
              for (int w = 0; w < kTiles / 2; ++w) vw[h][w] = drop_nan(vw[h][w], nan);
          }
          // O^T += V^T P^T: columns 2 j and 2 j + 1 of the thread's are rows g and g + 8 of tile j
#pragma unroll
          for (int w = 0; w < kTiles / 2; ++w) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t sel = half == 0 ? 0x5140 : 0x7362;
              uint32_t af[4];
              e4m3x4_to_f16x4(__byte_perm(vw[0][w], vw[1][w], sel), af[0], af[1]);
              e4m3x4_to_f16x4(__byte_perm(vw[2][w], vw[3][w], sel), af[2], af[3]);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_f16(o[t][2 * w + half], af, pf[t][0], pf[t][1]);
            }
          }
          if (!whole && __any_sync(0xffffffffu, nan != 0)) {
            // NaN codes of a partly hidden tile reach the rows that see them
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
              const int key = key0 + k;
              const bool ok = (k < 8 ? g0 : g1).valid != 0;
#pragma unroll
              for (int j = 0; j < kTiles; ++j)
#pragma unroll
                for (int d = 0; d < 2; ++d) {
                  const int col = (DP / 8) * g + 2 * j + d;
                  const uint8_t code = vt[k * kPitch + (((col >> 4) ^ (k & 7)) * 16) + (col & 15)];
                  const bool bad = ok && (code & 0x7F) == 0x7F;
#pragma unroll
                  for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int z = 0; z < 2; ++z)
                      if (bad && key <= pos[t][z] && (a.window == 0 || key > pos[t][z] - a.window)) o[t][j][2 * d + z] = __uint_as_float(0x7FC00000u);
                }
            }
          }
        }
        __syncwarp();                      // every lane has read the slot
        issue();
      }

      // Join the four warps.
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
          for (int x = 4; x < 32; x *= 2) l[t][z] += __shfl_xor_sync(0xffffffffu, l[t][z], x);
          if (g == 0) {
            s.m[warp][8 * t + 2 * c + z] = m[t][z];
            s.l[warp][8 * t + 2 * c + z] = l[t][z];
          }
        }
      __syncthreads();
      float M[NT][2], Ls[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int r = 8 * t + 2 * c + z;
          M[t][z] = kNone;
          Ls[t][z] = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M[t][z] = fmaxf(M[t][z], s.m[w][r]);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) Ls[t][z] += s.l[w][r] * fast_exp2(s.m[w][r] - M[t][z]);
          const float keep = fast_exp2(m[t][z] - M[t][z]);
#pragma unroll
          for (int j = 0; j < kTiles; ++j) {
            o[t][j][z] *= keep;
            o[t][j][2 + z] *= keep;
          }
        }
      constexpr int kSums = NT * kTiles * 4;
      auto put = [&](float* to) {
#pragma unroll
        for (int x = 0; x < kSums; ++x) to[x * 32 + lane] = o[x / (4 * kTiles)][x / 4 % kTiles][x % 4];
      };
      auto add = [&](const float* from) {
#pragma unroll
        for (int x = 0; x < kSums; ++x) o[x / (4 * kTiles)][x / 4 % kTiles][x % 4] += from[x * 32 + lane];
      };
      if (warp >= 2) put(scratch + (warp - 2) * kSums * 32);
      __syncthreads();
      if (warp < 2) add(scratch + warp * kSums * 32);
      __syncthreads();
      if (warp == 1) put(scratch);
      __syncthreads();
      if (warp == 0) add(scratch);

      const bool begun_before = at.tile > 0, goes_on = at.tile + n < at.count;
      const bool split = begun_before || goes_on;
      float* parts = static_cast<float*>(a.workspace);
      float* ml = parts + kPartialBytes / 4;
      int* counters = reinterpret_cast<int*>(ml + kMlBytes / 4);

      // A thread of warp 0 holds, for rows 2 c and 2 c + 1, columns [DP/8 g, DP/8 g + DP/8).
      if (warp == 0) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int row = 8 * t + 2 * c + z;
            if (row >= en.rows) continue;
            if (!split) {
              const float inv = Ls[t][z] == 0.f ? 0.f : 1.f / Ls[t][z];
              const int gr = en.row0 + row, tok = en.q_first + gr / group, h = at.head * group + gr % group;
              T* dst = static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head;
#pragma unroll
              for (int j = 0; j < kTiles; j += 4) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  v[2 * k] = o[t][j + k][z] * inv;
                  v[2 * k + 1] = o[t][j + k][2 + z] * inv;
                }
                const int col = (DP / 8) * g + 2 * j;
                if (col < ca.head_dim) store_f32<T, 8>(dst + col, v);
              }
              if (g == 0 && a.lse != nullptr)
                a.lse[static_cast<int64_t>(tok) * a.Hq + h] = Ls[t][z] == 0.f ? -INFINITY : (M[t][z] + log2f(Ls[t][z])) * kLn2;
            } else {
              const int slot = 2 * blockIdx.x + (begun_before ? 0 : 1);
              float* dst = parts + (static_cast<size_t>(slot) * kMaxRows + row) * 128;
#pragma unroll
              for (int j = 0; j < kTiles; j += 2) {
                const float v[4] = {o[t][j][z], o[t][j][2 + z], o[t][j + 1][z], o[t][j + 1][2 + z]};
                store_f32<float, 4>(dst + (DP / 8) * g + 2 * j, v);
              }
              if (g == 0)
                *reinterpret_cast<float2*>(ml + (static_cast<size_t>(slot) * kMaxRows + row) * 2) = make_float2(M[t][z], Ls[t][z]);
            }
          }
      }

      if (split) {
        // Pieces of this row tile: CTAs [cta0, cta1], joined kJoin at a time
        // by whoever finishes last among them, then those results likewise.
        const int u0 = x - at.tile, u1 = u0 + at.count;      // its stretch of the line
        const int cta0 = stretch_of(total, ctas, u0), cta1 = stretch_of(total, ctas, u1 - 1), pieces = cta1 - cta0 + 1;
        auto slot_of = [&](int piece) { return 2 * (cta0 + piece) + (piece == 0 ? 1 : 0); };
        const int mine = static_cast<int>(blockIdx.x) - cta0;
        int step = 1, from = mine / kJoin * kJoin, count = min(kJoin, pieces - from);
#pragma unroll 1
        for (int level = 0;; ++level) {
          __threadfence();
          __syncthreads();
          if (tid == 0) {
            int* counter = counters + level * kSlots + slot_of(from);
            const bool last = atomicAdd(counter, 1) == count - 1;
            if (last) *counter = 0;                           // ready for the next call
            s.last = last;
          }
          __syncthreads();
          const bool last = s.last != 0;
          __syncthreads();
          if (!last) break;
          __threadfence();
          const bool finish = count == pieces || level == 1;
          // thread: 4 columns of rows tid / 32, + 4, ...
          const int col = 4 * lane;
#pragma unroll 1
          for (int row = warp; row < en.rows; row += kWarps) {
            float Mx = -INFINITY, Lx = 0.f, acc[4] = {};
#pragma unroll 1
            for (int i = 0; i < count; i += 8) {
              float4 v[8];
              float2 z[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (i + k >= count) {
                  z[k] = make_float2(-INFINITY, 0.f);
                  v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                  continue;
                }
                const size_t at_row = static_cast<size_t>(slot_of(from + (i + k) * step)) * kMaxRows + row;
                z[k] = __ldcg(reinterpret_cast<const float2*>(ml + at_row * 2));
                v[k] = col < DP ? __ldcg(reinterpret_cast<const float4*>(parts + at_row * 128 + col)) : make_float4(0, 0, 0, 0);
              }
              float now = Mx;
#pragma unroll
              for (int k = 0; k < 8; ++k) now = fmaxf(now, z[k].x);
              const float base = now == -INFINITY ? 0.f : now, keep = fast_exp2(Mx - base);
              Lx *= keep;
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[q] *= keep;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float e = fast_exp2(z[k].x - base);
                Lx = fmaf(z[k].y, e, Lx);
                acc[0] = fmaf(v[k].x, e, acc[0]);
                acc[1] = fmaf(v[k].y, e, acc[1]);
                acc[2] = fmaf(v[k].z, e, acc[2]);
                acc[3] = fmaf(v[k].w, e, acc[3]);
              }
              Mx = now;
            }
            if (finish) {
              const float inv = Lx == 0.f ? 0.f : 1.f / Lx;
              const int gr = en.row0 + row, tok = en.q_first + gr / group, h = at.head * group + gr % group;
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[q] *= inv;
              if (col < ca.head_dim) store_f32<T, 4>(static_cast<T*>(a.out) + tok * a.out_token + h * a.out_head + col, acc);
              if (lane == 0 && a.lse != nullptr)
                a.lse[static_cast<int64_t>(tok) * a.Hq + h] = Lx == 0.f ? -INFINITY : (Mx + log2f(Lx)) * kLn2;
            } else {
              const size_t at_row = static_cast<size_t>(slot_of(from)) * kMaxRows + row;
              __syncwarp();
              if (col < DP) store_f32<float, 4>(parts + at_row * 128 + col, acc);
              if (lane == 0) *reinterpret_cast<float2*>(ml + at_row * 2) = make_float2(Mx, Lx);
            }
          }
          if (finish) break;
          step = kJoin;
          from = 0;
          count = (pieces + kJoin - 1) / kJoin;
        }
      }
      x += n;
    }
  }

  // Nothing of this warp is in flight when it ends: it has waited for every
  // tile, unless a wait ran out.
  if (*static_cast<volatile int*>(&s.abort_flag)) {
#pragma unroll 1
    for (int k = max(0, issued - kRing); k < issued; ++k) mbar_wait(&s.full[warp][k % kRing], (k / kRing) & 1, a.wait_limit_ns);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

}  // namespace

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Keys or values of the cache as {head_dim, page_size, kv_heads, num_pages}
// bytes; a box is ``rows`` tokens of one page and head, 128 bytes each (zeros
// past head_dim), with the 128-byte swizzle.
bool encode_cache_map(CUtensorMap* map, const moe_kv_cache_t& c, bool values, int rows) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.num_pages > 0 ? c.num_pages : 1)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(values ? c.v_stride_token : c.k_stride_token),
                                 static_cast<cuuint64_t>(values ? c.v_stride_head : c.k_stride_head),
                                 static_cast<cuuint64_t>(values ? c.v_stride_page : c.k_stride_page)};
  const cuuint32_t box[4] = {128, static_cast<cuuint32_t>(rows), 1, 1}, step[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, values ? c.v : c.k, dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as {head_dim, Hq, N}; a box is 64 columns (zeros past head_dim) of
// the ``group`` heads of one key head and ``tokens`` tokens, rows in the order
// of the attention's rows, with the 128-byte swizzle.
bool encode_query_map(CUtensorMap* map, const AttentionParams& a, bool f16, int group, int tokens) {
  const EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.cache.head_dim), static_cast<cuuint64_t>(a.Hq), static_cast<cuuint64_t>(a.N)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.q_head) * 2, static_cast<cuuint64_t>(a.q_token) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tokens)}, step[3] = {1, 1, 1};
  return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(a.q), dims, strides,
            box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t decode_attention_workspace_bytes() { return kPartialBytes + kMlBytes + kCounterBytes; }
cudaError_t clear_decode_counters(void* workspace, cudaStream_t s) {
  return cudaMemsetAsync(static_cast<uint8_t*>(workspace) + kPartialBytes + kMlBytes, 0, kCounterBytes, s);
}

namespace {

template <typename T, int DP, int NT>
int launch(const AttentionParams& a, cudaStream_t stream) {
  CUtensorMap k_map, v_map;
  Launch p = {};
  p.a = a;
  p.box = gcd(a.cache.page_size, 16);
  if (!encode_cache_map(&k_map, a.cache, false, p.box) || !encode_cache_map(&v_map, a.cache, true, p.box)) return MOE_ERR_CUDA;
  auto kernel = decode_attention_kernel<T, DP, NT>;
  constexpr int bytes = kSmem(8 * NT);
  p.tile_rows = 8 * NT;
  if (ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes) != cudaSuccess) return MOE_ERR_CUDA;
  const int sms = sm_count();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int group = a.Hq / a.cache.kv_heads;
  const int64_t row_tiles = (static_cast<int64_t>(a.max_q_len) * group + 8 * NT - 1) / (8 * NT);
  const int64_t entries = row_tiles * a.B < kMaxEntries ? row_tiles * a.B : kMaxEntries;
  const int64_t line = (static_cast<int64_t>(a.table_width) * a.cache.page_size / kKeys + 1) * entries * a.cache.kv_heads;
  if (row_tiles > kMaxEntries || line > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  p.row_tiles = static_cast<int>(row_tiles);
  const int per_launch = kMaxEntries / p.row_tiles;
  const int64_t longest = a.max_seq_len > 0 ? a.max_seq_len : 1;
#pragma unroll 1
  for (p.b0 = 0; p.b0 < a.B; p.b0 += per_launch) {
    p.B = a.B - p.b0 < per_launch ? a.B - p.b0 : per_launch;
    // no more CTAs than key tiles there can be
    const int64_t tiles = (longest + kKeys - 1) / kKeys * p.B * p.row_tiles * a.cache.kv_heads;
    int64_t grid = static_cast<int64_t>(sms) * ctas_per_sm(NT);
    if (grid > kMaxCtas) grid = kMaxCtas;
    if (grid > tiles) grid = tiles;
    if (launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), bytes, stream, k_map, v_map, p) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

namespace {
template <typename T>
int launch_rows(const AttentionParams& p, cudaStream_t s) {
  const bool few = static_cast<int64_t>(p.max_q_len) * (p.Hq / p.cache.kv_heads) <= 8;
  if (p.cache.head_dim <= 64) return few ? launch<T, 64, 1>(p, s) : launch<T, 64, 2>(p, s);
  return few ? launch<T, 128, 1>(p, s) : launch<T, 128, 2>(p, s);
}
}  // namespace

int launch_decode_attention(const AttentionParams& p, int dtype, cudaStream_t s) {
  return dtype == MOE_DTYPE_F16 ? launch_rows<__half>(p, s) : launch_rows<__nv_bfloat16>(p, s);
}

}  // namespace moe
