// k_attend_one.cu -- attention of one query a sequence over a paged cache, up to
// 16 query heads for each key and value head.
//
// The work is the reading of the cache: 4 d flops for every 2 d bytes (BF16) and
// head of a group, far below what the tensor cores do in that time.  So:
//  * Every row of the cache is read once, for all heads of its group, by 16-byte
//    asynchronous copies into shared memory; a warp keeps STAGES - 1 tiles (one of 8 KB;
//    three, 13 KB, of 8-bit heads of 64) on their way while it works on one.  Copies of places that are not there
//    (behind the end, a page out of range) read nothing and leave zeros.
//  * A sequence and kv head's visible positions (the first ones and the window, one
//    behind the other) are cut into units of the warps' tiles.  The call's units form one
//    line, which is divided evenly over the CTAs, whatever the lengths are; a
//    CTA's part of a (sequence, head) is a segment.  Copies run on across the
//    segments' ends.
//  * Warps work alone, each on its own tiles with its own running maxima, sums and
//    outputs (heads x head_dim in registers), and meet at a segment's end.
//  * A segment that is not a whole (sequence, head) goes to scratch and is joined with the
//    others (attend_join.cuh).
//
// Products are m16n8k16, turned so that the positions are the 16 rows and the heads
// the 8 columns (one or two groups of them): S^T = K Q^T and O^T = V^T P^T.  The order of
// the products' inner indexes is free as long as both factors use the same, and so is
// that of O's rows: lanes take their fragments as whole 16-byte pieces of K's and V's
// rows, and the fragments of Q and the rows of O^T follow.  Over a BF16 cache P goes in
// as two positive BF16 pieces (16 bits of it), over an 8-bit one everything is FP16: E4M3 fits
// it, Q is taken with a power of two off each head's row, and P carries the value's
// scale, 2^(x + log2 scale - its own running maximum + 7): from 2^15 down to 2^-24, so that
// what is lost of a weight below the normals is at most 2^-32 of the largest.
//
// Bound by memory where the caches are long: 64 sequences of 8192 positions, 48 heads on 8
// of 128, in 162 us, 6.6 TB/s (0.97 of a copy; 200 with products whose rows are heads, 191
// with one CTA of eight warps an SM, 173 with cuts wherever an even division puts them).  8 bits, 16 heads a kv head: the conversions and
// products share the time with the copies, 37 sequences of up to 16001 positions on 4 kv heads
// in 67 us (4.8 TB/s); 12 heads a kv head over BF16, 64 of 8192, in 169 us.  Few positions: trips through memory one after another (lengths, pages,
// rows, parts), 3.7 us for one unit, 8 for 700 positions cut and joined.
#include <algorithm>

#include "attend_join.cuh"
#include "attention.cuh"
#include "device_common.cuh"

namespace mhc {
namespace {

constexpr int EXTRA = 1;   // places on the line that a (sequence, head) takes besides its units
// Places that a cut inside one costs: its parts' way through memory and a join, and with as
// many (sequence, head) pairs as CTAs the CTA's second beginning, too, which an uneven load
// is worth.  In us, 8 kv heads of 128, with 2 and with 5: 32 sequences of 300 positions 11.2 and
// 8.3, of 500 15.6 and 11.4; with few pairs, which only cuts spread, 8 of 1000 9.2 and (with 4) 10.7.
constexpr int COST = 2, COST_MANY = 5;
static_assert(COST > EXTRA, "a cut has a unit on either side");
constexpr float GROWTH = 8.f;   // log2 of what a weight may reach
constexpr float ROOM = 7.f;     // log2 of FP16's largest weight over 2^GROWTH (8-bit cache)
constexpr float LEAST = 1.17549435e-38f;   // of a weight's second piece, 2^-126: nothing beside the first one

template <int D, bool FP8>
struct One {
  // CTAs an SM and warps of one
  static constexpr int SM_CTAS = 2, WARPS = 8 / SM_CTAS, THREADS = WARPS * 32;
  static constexpr int ROW = FP8 ? D : 2 * D;             // bytes of a cache row
  static constexpr int CHUNKS = ROW / 16;
  static constexpr int KEYS = !FP8 && D == 128 ? 16 : 32; // of a warp's tile
  static constexpr int TILE = KEYS * ROW;                 // bytes, keys or values
  static constexpr int STAGE = 2 * TILE + (FP8 ? KEYS * 8 : 0);
  static constexpr int STAGES = STAGE > 5000 ? 2 : 4;
  static constexpr int UNIT = WARPS * KEYS;
  static constexpr int PASS = 8;                          // rows that the warps meet over at a time
  static constexpr int MEET_ROW = D;                      // floats
  static constexpr int RING = WARPS * STAGES * STAGE;
  static constexpr int LOOK = 2 * KEYS * 4;                 // bytes: a tile's page numbers and places
  static constexpr int SMEM = RING + WARPS * (PASS * MEET_ROW * 4 + 16 * 16 + STAGES * (LOOK + 4));
  static_assert(SM_CTAS * (SMEM + 1024 + 256) <= 228 * 1024, "an SM's shared memory");
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
// 16 or 4 bytes to shared memory; zeros where `there` is false (nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ float lds4(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
template <bool FP8>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (FP8)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A transposed 8 x 8 matrix of 16-bit values, a row's pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Two E4M3 values (the lower or upper half of w) as an FP16 pair.
__device__ __forceinline__ uint32_t f16_lower(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(w)));
  return r;
}
__device__ __forceinline__ uint32_t f16_upper(uint32_t w) { return f16_lower(w >> 16); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What one query of a sequence sees: positions [0, sinks) and [first, length), the
// latter from `start` = first rounded down to a block of 16 (which lies in one page), the
// former up to there; in blocks of 16, the sinks' before the others.
constexpr int BLOCK = 16;
struct Seen {
  int length, first, start, sinks, sink_blocks, blocks;
};
__device__ __forceinline__ Seen seen_by_last(const AttendParams &p, int length) {
  Seen v;
  v.length = length;
  v.first = p.window && length > p.window ? length - p.window : 0;
  v.start = v.first / BLOCK * BLOCK;
  v.sinks = min(p.sinks, v.first);
  v.sink_blocks = (min(v.sinks, v.start) + BLOCK - 1) / BLOCK;
  v.blocks = v.sink_blocks + (length - v.start + BLOCK - 1) / BLOCK;
  return v;
}
// First position of block i.
__device__ __forceinline__ int block_position(const Seen &v, int i) {
  return i < v.sink_blocks ? i * BLOCK : v.start + (i - v.sink_blocks) * BLOCK;
}

// A place on the line: unit `unit` of `units` of (sequence s, head h); the EXTRA places before
// a pair's first unit have none (-EXTRA .. -1).
struct Cursor {
  int s, h, unit, units;
  Seen seen;
};

template <int D, bool FP8>
__device__ __forceinline__ int units_of(const Seen &v) {
  constexpr int N = One<D, FP8>::UNIT / BLOCK;
  return (v.blocks + N - 1) / N;
}

// To the first unit of the next (sequence, head); there has to be one.
template <int D, bool FP8>
__device__ __forceinline__ void next_head(const AttendParams &p, Cursor &c) {
  c.unit = -EXTRA;
  if (++c.h < p.kv_heads) return;
  c.h = 0;
  bool bad = false;
  do {
    if (c.s + 1 >= p.sequences) break;   // only if lengths change under the call
    c.seen = seen_by_last(p, sequence_length(p, ++c.s, bad));
    c.units = units_of<D, FP8>(c.seen);
  } while (c.units == 0);
}

// Over the places without a unit.
__device__ __forceinline__ void skip_extra(Cursor &c, int &left) {
  const int n = min(left, max(-c.unit, 0));
  c.unit += n;
  left -= n;
}

// Four elements of a head's output from its sums.
template <bool FP8>
__device__ __forceinline__ void store_row4(const AttendParams &p, int s, int head, int col, int dim, float all, float n,
                                           float all_out, const float4 &o) {
  const float b = all == -INFINITY ? 0.f : all, bo = all_out == -INFINITY ? 0.f : all_out;
  const float f = n != 0.f ? (FP8 ? exp2_fast(bo - b) : UP) / n : 0.f;
  *reinterpret_cast<uint2 *>(p.output + s * p.output_stride + int64_t(head) * dim + col) =
      make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
  if (p.lse && col == 0) p.lse[int64_t(s) * p.heads + head] = n != 0.f ? (b + log2f(n)) * 0.69314718056f : -INFINITY;
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__((One<D, FP8>::THREADS), (One<D, FP8>::SM_CTAS)) k_attend_one(const AttendParams p) {
  using F = One<D, FP8>;
  constexpr int M_TILES = D / 16;      // of 16 elements of a row of output
  constexpr int WARPS = F::WARPS, THREADS = F::THREADS;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int warp_total[WARPS];
  __shared__ Cursor begin_shared;
  __shared__ int bounds_shared[2];
  __shared__ Join joins[2];   // of the part's first and last (sequence, head)
  __shared__ int join_count, join_flag;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t = lane % 4;
  const int group = p.heads / p.kv_heads;
  bool bad = false;
  if (tid == 0) join_count = 0;

  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's part of the line.  Code that runs once comes from far, line after
  // line (a call's first microseconds are that): it is kept short.
  const int chunk = (p.sequences + THREADS - 1) / THREADS;
  auto places_of = [&](int s, Cursor &c, bool &wrong) {
    c.s = s;
    c.seen = seen_by_last(p, sequence_length(p, s, wrong));
    c.units = units_of<D, FP8>(c.seen);
    return c.units ? EXTRA + c.units : 0;
  };
  int mine = 0;
  bool empty = false;
#pragma unroll 1
  for (int s = tid * chunk; s < min(p.sequences, (tid + 1) * chunk); ++s) {
    Cursor c;
    const int n = places_of(s, c, bad);
    empty |= n == 0;
    mine += n * p.kv_heads;
  }
  int upto = mine;   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) warp_total[warp] = upto;
  const bool any_empty = __syncthreads_or(empty);
  Line line;
  line.total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) upto += warp_total[w];
    line.total += warp_total[w];
  }
  // Two places a CTA at least with 32 units a pair, four with 64: a join of fewer parts
  // ends sooner (one kv head of 32768 positions 23.2 us with one, 19.3 with four; 8 of 2000 11.5 and
  // 9.7 with two; at 16 units one is as good as two).
  const int pairs = p.sequences * p.kv_heads;
  line.divide(min(int(gridDim.x), line.total >> (line.total / 64 >= pairs ? 2 : line.total / 32 >= pairs)));
  const int cost = 2 * pairs >= int(gridDim.x) ? COST_MANY : COST;
  const int cta = min(int(blockIdx.x), line.grid);
  // thread k finds where this CTA's part begins (0), where it ends (1): the owner of the
  // place tells it what lies before
  const int place0 = line.begin(cta), place1 = line.begin(min(cta + 1, line.grid));
  const int owner0 = __syncthreads_count(upto <= place0), owner1 = __syncthreads_count(upto <= place1);
  if (tid == owner0) bounds_shared[0] = upto - mine;
  if (tid == owner1) bounds_shared[1] = upto - mine;
  __syncthreads();
  if (tid < 2) {
    const int place = tid ? place1 : place0;
    if (place >= line.total) {
      bounds_shared[tid] = line.total;
    } else {
      int rest = place - bounds_shared[tid];
      bool seen_before = false;
      Cursor c;
      bounds_shared[tid] = line.total;
      // (it ends at the break, unless lengths change under the call)
#pragma unroll 1
      for (int s = (tid ? owner1 : owner0) * chunk; s < p.sequences; ++s) {
        const int n = places_of(s, c, seen_before);
        if (rest < n * p.kv_heads) {
          c.h = rest / n;
          rest -= c.h * n;
          const int at = line.cut(place, place - rest, n, cost);
          c.unit = at - (place - rest) - EXTRA;
          bounds_shared[tid] = at;
          break;
        }
        rest -= n * p.kv_heads;
      }
      if (tid == 0) begin_shared = c;
    }
  }
  __syncthreads();
  const int end = bounds_shared[1];

  const uint32_t ring_at = smem_u32(smem + warp * F::STAGES * F::STAGE);
  float *meet = reinterpret_cast<float *>(smem + F::RING);             // [WARPS][PASS][MEET_ROW]
  float4 *stats = reinterpret_cast<float4 *>(meet + WARPS * F::PASS * F::MEET_ROW);   // [WARPS][16]
  int *looks = reinterpret_cast<int *>(stats + WARPS * 16) + warp * F::STAGES * 2 * F::KEYS + lane % F::KEYS;
  uint32_t *masks = reinterpret_cast<uint32_t *>(stats + WARPS * 16) + WARPS * F::STAGES * 2 * F::KEYS + warp * F::STAGES;

  Cursor at = begin_shared, ahead;
  int left = end - bounds_shared[0], left_ahead;
  if (left > 0 && at.unit == at.units) next_head<D, FP8>(p, at);
  skip_extra(at, left);
  ahead = at;
  left_ahead = left;

  // ---- copies.  A tile is looked up STAGES tiles before its copies are issued: its
  // pages' numbers (lane 16 i has block i's) come by a copy as well, into `looks` with the
  // places in the page; -1 for positions that the query does not see.
  constexpr int TILE_BLOCKS = F::KEYS / BLOCK;
  auto look = [&](int stage) {
    int place = -1;
    if (left_ahead > 0) {
      const int block = ahead.unit * (F::UNIT / BLOCK) + warp * TILE_BLOCKS + lane / BLOCK;
      const int position = block_position(ahead.seen, block) + lane % BLOCK;
      if (lane < F::KEYS && block < ahead.seen.blocks && position < ahead.seen.length &&
          (position >= ahead.seen.first || position < ahead.seen.sinks)) {
        place = (ahead.h << p.page_shift) + (position & ((1 << p.page_shift) - 1));
        copy4(smem_u32(looks + stage * 2 * F::KEYS), p.page_table + ahead.s * p.table_stride + (position >> p.page_shift), true);
      }
      --left_ahead;
      if (++ahead.unit == ahead.units && left_ahead > 0) {
        next_head<D, FP8>(p, ahead);
        skip_extra(ahead, left_ahead);
      }
    }
    if (lane < F::KEYS) looks[(stage * 2 + 1) * F::KEYS] = place;
  };
  // A warp's instruction copies ROWS rows; this lane's are row lane / CHUNKS of them, its piece of
  // a row lane % CHUNKS.
  constexpr int ROWS = 32 / F::CHUNKS, COPIES = BLOCK / ROWS, SIZE = FP8 ? 1 : 2;
  const int my_row = lane / F::CHUNKS, my_piece = lane % F::CHUNKS;
  auto issue = [&](int stage) {
    const uint32_t to = ring_at + stage * F::STAGE + my_row * F::ROW;
    const int page = looks[stage * 2 * F::KEYS], place = lane < F::KEYS ? looks[(stage * 2 + 1) * F::KEYS] : -1;
    const bool is_page = page >= 0 && page < p.pages, there = place >= 0 && is_page;
    bad |= place >= 0 && !is_page;
    const uint32_t all = __ballot_sync(0xffffffffu, there);
    if (lane == 0) masks[stage] = all;
    if (all) {
#pragma unroll
      for (int j = 0; j < TILE_BLOCKS; ++j) {
        // from the page and place of the block's first position that the query sees
        const uint32_t seen = all >> (j * BLOCK) & 0xffffu;
        const int first = seen ? __ffs(seen) - 1 : 0;
        const int64_t block_page = seen ? __shfl_sync(0xffffffffu, page, j * BLOCK + first) : 0;
        const int block_place = (__shfl_sync(0xffffffffu, place, j * BLOCK + first) - first) * D + lane * (16 / SIZE);
        const unsigned char *k = static_cast<const unsigned char *>(p.keys.data) + (block_page * p.keys.page_stride + block_place) * SIZE;
        const unsigned char *v = static_cast<const unsigned char *>(p.values.data) + (block_page * p.values.page_stride + block_place) * SIZE;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int row = i * ROWS + my_row;   // of the block
          const bool ok = seen >> row & 1;
          const int ck = F::CHUNKS >= 8 ? my_piece ^ ((row & 1) << 2) : my_piece;
          const int cv = F::CHUNKS >= 8 ? my_piece ^ ((row >> 1 & 3) << 1) : my_piece ^ (row >> 1 & 3);
          copy16(to + (j * BLOCK + i * ROWS) * F::ROW + ck * 16, k + i * 512, ok);
          copy16(to + F::TILE + (j * BLOCK + i * ROWS) * F::ROW + cv * 16, v + i * 512, ok);
        }
      }
      if (FP8) {
        const int64_t from = there ? ((int64_t(page) * p.kv_heads) << p.page_shift) + place : 0;
        const uint32_t scales = ring_at + stage * F::STAGE + 2 * F::TILE + lane * 4;
        copy4(scales, p.keys.scales + from, there);
        copy4(scales + F::KEYS * 4, p.values.scales + from, there);
      }
    }
    look(stage);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < F::STAGES; ++i) look(i);
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
  for (int i = 0; i < F::STAGES; ++i) issue(i);

  // ---- sequences that see nothing
  if (any_empty) {
    for (int s = blockIdx.x; s < p.sequences; s += gridDim.x) {
      if (sequence_length(p, s, bad) > 0) continue;
      for (int i = tid; i < p.heads * D / 8; i += THREADS)
        st_vec(p.output + s * p.output_stride + i * 8, make_uint4(0, 0, 0, 0));
      for (int i = tid; p.lse && i < p.heads; i += THREADS) p.lse[int64_t(s) * p.heads + i] = -INFINITY;
    }
  }

  const JoinCounters counters = {p.counters, p.counter_ctas};
  int stage = 0;
  while (left > 0) {
    // ---- a segment: units at.unit .. of (at.s, at.h), as far as this CTA's part goes
    const int unit0 = at.unit, count = min(left, at.units - at.unit);
    const uint16_t *q = p.q + at.s * p.q_stride + int64_t(at.h) * group * D;
    uint32_t qb[NT][D / 16][2];          // of head 8 n + g
    float head_scale[NT][2];             // of heads 8 n + 2 t, + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = 8 * n + g;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if (!FP8) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint4 v = head < group ? ld_vec(q + head * D + (4 * i + t) * 8) : zero;
          qb[n][2 * i][0] = v.x;
          qb[n][2 * i][1] = v.y;
          qb[n][2 * i + 1][0] = v.z;
          qb[n][2 * i + 1][1] = v.w;
        }
        head_scale[n][0] = head_scale[n][1] = p.scale_log2;
      } else {
        float x[D / 64][2][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            unpack8(head < group ? ld_vec(q + head * D + (4 * i + t) * 16 + e * 8) : zero, x[i][e]);
#pragma unroll
            for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(x[i][e][k]) & 0x7fffffffu);
          }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the head's largest magnitude to [1, 2)
        const int e2 = min(max(int(top >> 23) - 127, -126), 126);
        const float down = __uint_as_float(uint32_t(127 - e2) << 23);
        const float up = p.scale_log2 * __uint_as_float(uint32_t(127 + e2) << 23);
#pragma unroll
        for (int e = 0; e < 2; ++e) head_scale[n][e] = __shfl_sync(0xffffffffu, up, (2 * t + e) * 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *y = x[i][k / 2] + k % 2 * 4;
            qb[n][4 * i + k][0] = pack_f16x2(y[0] * down, y[1] * down);
            qb[n][4 * i + k][1] = pack_f16x2(y[2] * down, y[3] * down);
          }
      }
    }
    float acc[NT][M_TILES][4];
    float top[NT][2], top_out[NT][2], sum[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < M_TILES; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[n][e] = top_out[n][e] = -INFINITY;
        sum[n][e] = 0.f;
      }
    }

    for (int u = 0; u < count; ++u) {
      asm volatile("cp.async.wait_group %0;" ::"n"(F::STAGES - 1) : "memory");
      __syncwarp();
      const uint32_t from = ring_at + stage * F::STAGE;
      const uint32_t there = masks[stage];
      if (there) {
        constexpr int BLOCKS = F::KEYS / 16;   // of 16 positions: rows g and g + 8 are this lane's
        // ---- x = scale (q k) log2(e)
        float x[NT][BLOCKS][4];
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
#pragma unroll
          for (int n = 0; n < NT; ++n) x[n][j][0] = x[n][j][1] = x[n][j][2] = x[n][j][3] = 0.f;
          const int row = j * 16 + g;
#pragma unroll
          for (int i = 0; i < F::CHUNKS / 4; ++i) {
            const int c = 4 * i + t, ck = F::CHUNKS >= 8 ? c ^ ((row & 1) << 2) : c;
            const uint4 v = lds16(from + row * F::ROW + ck * 16), w = lds16(from + (row + 8) * F::ROW + ck * 16);
            const uint32_t a[4] = {v.x, v.y, v.z, v.w}, b[4] = {w.x, w.y, w.z, w.w};
            if (FP8) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t ka[4] = {f16_lower(a[k]), f16_lower(b[k]), f16_upper(a[k]), f16_upper(b[k])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<FP8>(x[n][j], ka, qb[n][4 * i + k][0], qb[n][4 * i + k][1]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t ka[4] = {a[2 * k], b[2 * k], a[2 * k + 1], b[2 * k + 1]};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma<FP8>(x[n][j], ka, qb[n][2 * i + k][0], qb[n][2 * i + k][1]);
              }
            }
          }
        }
        float y[FP8 ? NT : 1][FP8 ? BLOCKS : 1][4];   // x + log2 of the value's scale
        float now[NT][2], now_out[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) now[n][0] = now[n][1] = now_out[n][0] = now_out[n][1] = -INFINITY;
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = j * 16 + 8 * r + g;
            const bool ok = there >> row & 1;
            float ks = 1.f, vs = 0.f;
            if (FP8) {
              ks = lds4(from + 2 * F::TILE + row * 4);
              vs = log2_fast(lds4(from + 2 * F::TILE + (F::KEYS + row) * 4));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float v = x[n][j][2 * r + e] * head_scale[n][e];
                if (FP8) v *= ks;
                x[n][j][2 * r + e] = ok ? v : -INFINITY;
                now[n][e] = fmaxf(now[n][e], x[n][j][2 * r + e]);
                if (FP8) {
                  y[n][j][2 * r + e] = ok ? v + vs : -INFINITY;
                  now_out[n][e] = fmaxf(now_out[n][e], y[n][j][2 * r + e]);
                }
              }
          }
        // ---- the running references of the weights: a head's maximum, over its eight lanes, when
        // some lane's has grown past the reference by more than GROWTH (weights are then at
        // most 2^GROWTH).  Most tiles need no exchange of lanes (exchanged for every one: 70 us for
        // the 66.6 of 37 sequences over an 8-bit cache, 9.9 for 9.3 of one over 700 positions).
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            grew |= now[n][e] > top[n][e] + GROWTH;
            if (FP8) grew |= now_out[n][e] > top_out[n][e] + GROWTH;
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int o = 4; o < 32; o *= 2) {
                now[n][e] = fmaxf(now[n][e], __shfl_xor_sync(0xffffffffu, now[n][e], o));
                if (FP8) now_out[n][e] = fmaxf(now_out[n][e], __shfl_xor_sync(0xffffffffu, now_out[n][e], o));
              }
              const float up = fmaxf(now[n][e], top[n][e]), up_out = FP8 ? fmaxf(now_out[n][e], top_out[n][e]) : up;
              const float f = up == -INFINITY ? 1.f : exp2_fast(top[n][e] - up);
              const float fo = FP8 ? up_out == -INFINITY ? 1.f : exp2_fast(top_out[n][e] - up_out) : f;
              sum[n][e] *= f;
              top[n][e] = up;
              if (FP8) top_out[n][e] = up_out;
#pragma unroll
              for (int i = 0; i < M_TILES; ++i) {
                acc[n][i][e] *= fo;
                acc[n][i][2 + e] *= fo;
              }
            }
        }
        float base[NT][2], base_out[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            base_out[n][e] = base[n][e] = top[n][e] == -INFINITY ? 0.f : top[n][e];
            if (FP8) base_out[n][e] = top_out[n][e] == -INFINITY ? 0.f : top_out[n][e] - ROOM;
          }
        // ---- weights and their sum, values times weights, 16 positions at a time
#pragma unroll
        for (int j = 0; j < BLOCKS; ++j) {
          uint32_t pa[NT][2], pb[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float w0 = exp2_fast(x[n][j][2 * r] - base[n][0]), w1 = exp2_fast(x[n][j][2 * r + 1] - base[n][1]);
              sum[n][0] += w0;
              sum[n][1] += w1;
              if (FP8) {
                pa[n][r] = transpose8(pack_f16x2(exp2_fast(y[n][j][2 * r] - base_out[n][0]), exp2_fast(y[n][j][2 * r + 1] - base_out[n][1])));
              } else {
                const float v0 = w0 * (1.f / UP), v1 = w1 * (1.f / UP);
                // the first piece cut off, not rounded: the second is what is left, never negative and
                // never zero, so that both times an infinity are the same infinity
                const uint32_t w = __byte_perm(__float_as_uint(v0), __float_as_uint(v1), 0x7632);
                pa[n][r] = transpose8(w);
                pb[n][r] = transpose8(pack_bf16x2(fmaxf(v0 - bf16_lo(w), LEAST), fmaxf(v1 - bf16_hi(w), LEAST)));
              }
            }
          const int row = j * 16 + 2 * t;   // this lane's positions: row, row + 1, row + 8, row + 9
          if (!FP8) {
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh) {
              uint32_t v[4][4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int rr = row + (i & 1) + (i >> 1) * 8;
                const uint4 w = lds16(from + F::TILE + rr * F::ROW + ((hh * 8 + g) ^ ((rr >> 1 & 3) << 1)) * 16);
                v[i][0] = w.x; v[i][1] = w.y; v[i][2] = w.z; v[i][3] = w.w;
              }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t va[4] = {__byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
                                        __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  mma<FP8>(acc[n][hh * 4 + w], va, pa[n][0], pa[n][1]);
                  mma<FP8>(acc[n][hh * 4 + w], va, pb[n][0], pb[n][1]);
                }
              }
            }
          } else {
            uint32_t v[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int rr = row + (i & 1) + (i >> 1) * 8;
              if (D == 128) {
                const uint4 w = lds16(from + F::TILE + rr * F::ROW + (g ^ ((rr >> 1 & 3) << 1)) * 16);
                v[i][0] = w.x; v[i][1] = w.y; v[i][D / 32 - 2] = w.z; v[i][D / 32 - 1] = w.w;
              } else {
                const uint2 w = lds8(from + F::TILE + rr * F::ROW + ((g >> 1) ^ (rr >> 1 & 3)) * 16 + (g & 1) * 8);
                v[i][0] = w.x; v[i][1] = w.y;
              }
            }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5140), a1 = __byte_perm(v[2][w], v[3][w], 0x5140);
              const uint32_t b0 = __byte_perm(v[0][w], v[1][w], 0x7362), b1 = __byte_perm(v[2][w], v[3][w], 0x7362);
              const uint32_t va[4] = {f16_lower(a0), f16_upper(a0), f16_lower(a1), f16_upper(a1)};
              const uint32_t vb[4] = {f16_lower(b0), f16_upper(b0), f16_lower(b1), f16_upper(b1)};
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma<FP8>(acc[n][2 * w], va, pa[n][0], pa[n][1]);
                mma<FP8>(acc[n][2 * w + 1], vb, pa[n][0], pa[n][1]);
              }
            }
          }
        }
      }
      __syncwarp();
      issue(stage);
      if (++stage == F::STAGES) stage = 0;
    }

    // ---- the warps meet: rows PASS at a time, weighted to the common maximum
    const bool whole = count == at.units;
    // CTAs that have units of this (sequence, head), and where their parts are
    const int unit_place = end - left - unit0;   // its first unit on the line
    int cta0 = 0, cta1 = 0;
    if (!whole) line.owners(unit_place - EXTRA, EXTRA + at.units, cost, cta0, cta1);
    auto part_of = [&](int c, bool begins) { return p.parts + int64_t(2 * c + begins) * part_floats(16, D); };
    float *const part = part_of(blockIdx.x, int(blockIdx.x) == cta0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o *= 2) sum[n][e] += __shfl_xor_sync(0xffffffffu, sum[n][e], o);
        if (g == 0) stats[warp * 16 + 8 * n + 2 * t + e] = make_float4(top[n][e], sum[n][e], FP8 ? top_out[n][e] - ROOM : top[n][e], 0.f);
      }
    for (int r0 = 0; r0 < group; r0 += F::PASS) {
      const int rows = min(F::PASS, group - r0);
      __syncthreads();   // stats are there; the buffer's last readers are done
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * n + 2 * t + e - r0;
          if (row < 0 || row >= rows) continue;
          // a lane's elements: whole pieces of PIECE, the rows of its tiles in pairs
          constexpr int PIECE = FP8 && D == 128 ? 16 : 8;
          float *m = meet + (warp * F::PASS + row) * F::MEET_ROW + g * PIECE;
#pragma unroll
          for (int i = 0; i < M_TILES; i += 2) {
            const int d = i * 2 / PIECE * 64 + i * 2 % PIECE;
            *reinterpret_cast<float4 *>(m + d) = make_float4(acc[n][i][e], acc[n][i][2 + e], acc[n][i + 1][e], acc[n][i + 1][2 + e]);
          }
        }
      __syncthreads();
      for (int item = tid; item < rows * (D / 4); item += THREADS) {
        const int row = r0 + item / (D / 4), col = item % (D / 4) * 4;
        float all = -INFINITY, all_out = -INFINITY, n = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          all = fmaxf(all, stats[w * 16 + row].x);
          all_out = fmaxf(all_out, stats[w * 16 + row].z);
        }
        const float b = all == -INFINITY ? 0.f : all, bo = all_out == -INFINITY ? 0.f : all_out;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 st = stats[w * 16 + row];
          const float4 v = *reinterpret_cast<const float4 *>(meet + (w * F::PASS + row - r0) * F::MEET_ROW + col);
          n += st.y * exp2_fast(st.x - b);
          const float f = exp2_fast(st.z - bo);
          o.x += v.x * f;
          o.y += v.y * f;
          o.z += v.z * f;
          o.w += v.w * f;
        }
        if (whole) {
          store_row4<FP8>(p, at.s, at.h * group + row, col, D, all, n, all_out, o);
        } else {
          *reinterpret_cast<float4 *>(part + (col / 4 * 16 + row) * 4) = o;
          if (col == 0) *reinterpret_cast<float4 *>(part + (D / 4 * 16 + row) * 4) = make_float4(all, n, all_out, 0.f);
        }
      }
    }
    if (!whole) {
      // who writes the last part of sixteen joins them, once there is no other work
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int join_group = (int(blockIdx.x) - cta0) / JOIN_WIDTH;
        unsigned int *counter = counters.of_group(cta0, join_group);
        if (atomicAdd(counter, 1u) == unsigned(join_group_size(cta0, cta1, join_group) - 1)) {
          *counter = 0;
          joins[join_count++] = {at.s, at.h, 0, cta0, cta1, join_group};
        }
      }
    }
    __syncthreads();   // stats may be written again
    left -= count;
    at.unit += count;
    if (at.unit == at.units && left > 0) {
      next_head<D, FP8>(p, at);
      skip_extra(at, left);
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");

#pragma unroll 1
  for (int k = 0; k < join_count; ++k) {
    const Join join = joins[k];
    join_parts<D>(smem, F::RING, tid, THREADS, [] { __syncthreads(); }, join, group, 16, counters,
                  [&](int c, bool begins) { return p.parts + int64_t(2 * c + begins) * part_floats(16, D); },
                  [&](int row, int col, float all, float n, float all_out, const float4 &o) {
                    store_row4<FP8>(p, join.s, join.h * group + row, col, D, all, n, all_out, o);
                  },
                  &join_flag);
  }
  if (bad) atomicOr(p.err, ATTN_ERR_INDEX);
}

template <int D, bool FP8, int NT>
cudaError_t launch(const AttendParams &p, int sms, cudaStream_t stream) {
  // what a sequence can see at most, in units
  int64_t most = int64_t(p.table_width) << p.page_shift;
  if (p.window) most = std::min(most, int64_t(p.window) + p.sinks + 2 * BLOCK);
  const int64_t places = (EXTRA + (most + One<D, FP8>::UNIT - 1) / One<D, FP8>::UNIT) * p.kv_heads * p.sequences;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(places, One<D, FP8>::SM_CTAS * sms)));
  cfg.blockDim = dim3(One<D, FP8>::THREADS);
  cfg.dynamicSmemBytes = One<D, FP8>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend_one<D, FP8, NT>, p);
}

template <int D, bool FP8>
cudaError_t launch_groups(const AttendParams &p, int sms, cudaStream_t stream) {
  return p.heads / p.kv_heads <= 8 ? launch<D, FP8, 1>(p, sms, stream) : launch<D, FP8, 2>(p, sms, stream);
}

template <int D, bool FP8>
cudaError_t allow() {
  cudaError_t e = cudaFuncSetAttribute(k_attend_one<D, FP8, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize, One<D, FP8>::SMEM);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_attend_one<D, FP8, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize, One<D, FP8>::SMEM);
  return e;
}

}  // namespace

cudaError_t attend_one_setup() {
  cudaError_t e = allow<128, false>();
  if (e == cudaSuccess) e = allow<128, true>();
  if (e == cudaSuccess) e = allow<64, false>();
  if (e == cudaSuccess) e = allow<64, true>();
  return e;
}

size_t attend_one_scratch(int sms) { return size_t(2) * 2 * sms * part_floats(16, 128) * sizeof(float); }

cudaError_t launch_attend_one(const AttendParams &p, int sms, cudaStream_t stream) {
  if (p.dim == 128) return p.fp8 ? launch_groups<128, true>(p, sms, stream) : launch_groups<128, false>(p, sms, stream);
  return p.fp8 ? launch_groups<64, true>(p, sms, stream) : launch_groups<64, false>(p, sms, stream);
}

}  // namespace mhc
