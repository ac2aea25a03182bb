// attend_join.cuh -- how a call's work is divided over the CTAs, and how rows that
// several of them have parts of are joined: what the two attend kernels share.
//
// The call's items (a sequence and kv head; with several queries a block of them, too) lie
// one behind the other on a line, each with `places` by its work, and the line is cut
// evenly.  A cut inside an item costs its parts' way through memory and a join, `cost`
// places: within that of an end of the item it is moved to the nearer end.
//
// Of an item that the CTAs cta0 .. cta1 have a part of, each writes it to scratch: its rows'
// sums of weighted values and, for each row, the maximum that its weights are relative to
// (log2), their sum, and the maximum of the weights that went into the output (another
// one over an 8-bit cache).  Parts are joined in their order, so that the bits do not
// depend on who comes when: sixteen at a time by the CTA that writes the last of them,
// and what comes out (in the place of the first of the sixteen) once more by the one that
// is last there.  A CTA joins when its other work is done: then its shared memory has
// room for all parts of many rows at once, and no work waits for the trips.
#pragma once

#include "attention.cuh"
#include "device_common.cuh"

namespace mhc {

constexpr int JOIN_WIDTH = 16;   // parts that are joined at a time

// Weights go into sums of a BF16 cache's values 2^DOWN smaller than they are: at most 2^8 for each
// of 2^30 positions, no sum of finite values leaves FP32's range, however near to its end they
// are.  At the other end, sums stop at 2^-149: a position's part at 2^-111 of the output.
constexpr float DOWN = 38.f, UP = 274877906944.f;
static_assert(UP == float(1ull << 38), "2^DOWN");

// A CTA's parts: two (of what began with an earlier CTA, of what begins with it), each
// [dim / 4][rows][4] floats and then [rows][4]: threads that have a row each write whole
// lines.
constexpr int part_floats(int rows, int dim) { return rows * (dim + 4); }

// `total` places over `grid` CTAs: `each`, and one more for the first `more`.
struct Line {
  int total, grid, each, more;
  __device__ __forceinline__ void divide(int ctas) {
    grid = max(1, min(ctas, total));
    each = total / grid;
    more = total - each * grid;
  }
  // Where CTA c's part would begin but for what a cut costs.
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
  // The last CTA that begins at `place` or before.
  __device__ __forceinline__ int cta(int place) const {
    const int bound = more * (each + 1);
    return place < bound ? place / (each + 1) : more + (place - bound) / each;
  }
  // The cut at `place`, which is in the item [first, first + places).
  static __device__ __forceinline__ int cut(int place, int first, int places, int cost) {
    const int at = place - first;
    if (at >= cost && at <= places - cost) return place;
    return 2 * at < places ? first : first + places;
  }
  // The CTAs that an item is cut over.
  __device__ __forceinline__ void owners(int first, int places, int cost, int &cta0, int &cta1) const {
    cta0 = cta(first + cost - 1);
    cta1 = cta(first + places - cost);
  }
};

// A group of parts that this CTA joins.
struct Join {
  int s, h, block, cta0, cta1, group;
};

__device__ __forceinline__ float join_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The counters of one set of parts: [3][ctas].
struct JoinCounters {
  unsigned int *at;
  int ctas;
  // Of the group that `cta` is in: the first group's at its first CTA, another's in an
  // array of its own (a CTA may be the first of one set of parts and inside one other).
  __device__ __forceinline__ unsigned int *of_group(int cta0, int group) const {
    return at + (group ? ctas : 0) + cta0 + group * JOIN_WIDTH;
  }
  __device__ __forceinline__ unsigned int *of_groups(int cta0) const { return at + 2 * ctas + cta0; }
};

__device__ __forceinline__ int join_group_size(int cta0, int cta1, int group) {
  return min(JOIN_WIDTH, cta1 + 1 - cta0 - group * JOIN_WIDTH);
}

__device__ __forceinline__ void join_copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// A join, by `threads` threads of the CTA that `sync` lets wait for one another.  part(cta,
// begins) is a part, final(row, column, maximum, sum, maximum of the output's weights, four
// elements) writes output.
template <int D, class Sync, class Part, class Final>
__device__ __forceinline__ void join_parts(unsigned char *smem, int room, int tid, int threads, const Sync &sync, const Join &join,
                                           int rows, int max_rows, const JoinCounters &counters, const Part &part,
                                           const Final &final, volatile int *flag) {
  const int groups = (join.cta1 - join.cta0) / JOIN_WIDTH + 1;
  const float4 *there = reinterpret_cast<const float4 *>(smem);
  const uint32_t to = uint32_t(__cvta_generic_to_shared(smem));
  int first = join.cta0 + join.group * JOIN_WIDTH, step = 1, count = join_group_size(join.cta0, join.cta1, join.group);
  bool last = groups == 1;
  __threadfence();
#pragma unroll 1
  for (;;) {
    // rows at a time; a part in shared memory is [dim / 4 + 1][n + 1][4], the last of the rows
    // of stats
    const int pass = max(1, min(rows, room / (count * (D + 4) * 4) - 1));
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += pass) {
      const int n = min(pass, rows - r0), size = (D / 4 + 1) * (n + 1);   // of 16 bytes
      sync();
      const int shift = 32 - __clz(n - 1);   // rows to a power of two
#pragma unroll 4
      for (int i = tid; i < count * (D / 4 + 1) << shift; i += threads) {
        const int q = (i >> shift) / (D / 4 + 1), col = (i >> shift) % (D / 4 + 1), row = i & ((1 << shift) - 1), c = first + q * step;
        if (row < n)
          join_copy16(to + (q * size + col * (n + 1) + row) * 16, part(c, c == join.cta0) + (col * max_rows + r0 + row) * 4);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      sync();
#pragma unroll 1
      for (int item = tid; item < n * (D / 4); item += threads) {
        const int row = item / (D / 4), col = item % (D / 4);
        const float4 *stats = there + D / 4 * (n + 1) + row, *values = there + col * (n + 1) + row;
        float all = -INFINITY, all_out = -INFINITY, sum = 0.f;
#pragma unroll 2
        for (int q = 0; q < count; ++q) {
          all = fmaxf(all, stats[q * size].x);
          all_out = fmaxf(all_out, stats[q * size].z);
        }
        const float b = all == -INFINITY ? 0.f : all, bo = all_out == -INFINITY ? 0.f : all_out;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int q = 0; q < count; ++q) {
          const float4 st = stats[q * size], v = values[q * size];
          sum += st.y * join_exp2(st.x - b);
          const float f = join_exp2(st.z - bo);
          o.x += v.x * f;
          o.y += v.y * f;
          o.z += v.z * f;
          o.w += v.w * f;
        }
        if (last) {
          final(r0 + row, col * 4, all, sum, all_out, o);
        } else {
          float *mine = part(first, first == join.cta0) + (r0 + row) * 4;
          *reinterpret_cast<float4 *>(mine + col * max_rows * 4) = o;
          if (col == 0) *reinterpret_cast<float4 *>(mine + D * max_rows) = make_float4(all, sum, all_out, 0.f);
        }
      }
    }
    if (last) return;
    __threadfence();
    sync();
    if (tid == 0) {
      unsigned int *counter = counters.of_groups(join.cta0);
      *flag = atomicAdd(counter, 1u) == unsigned(groups - 1);
      if (*flag) *counter = 0;
    }
    sync();
    if (!*flag) return;
    __threadfence();
    first = join.cta0;
    step = JOIN_WIDTH;
    count = groups;
    last = true;
  }
}

}  // namespace mhc
