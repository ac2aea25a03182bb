// k_moe.cu -- a whole mixture-of-experts layer for up to 32 tokens in one
// kernel:
//   route      logits = x router^T, scores, the top_k experts of each token
//   up         g = x gate^T, u = x up^T of every reached expert, h = silu(g) u
//   down       y = sum over a token's experts of weight * (h down^T)
//
// What bounds it is the read of the reached experts' weights, 3 I H values
// each.  So the weights are the row operand of the tensor cores (tiles of 128
// rows x 128 bytes, moved by TMA straight to where tcgen05.mma reads them) and
// the few tokens are the columns; nothing but the tokens' columns passes
// through registers.
//
// 8-bit weights against BF16 activations: the tensor core multiplies E4M3 by
// E4M3, so an activation row is scaled by a power of two and split into E4M3
// pieces, each holding four significant bits of what the ones before leave
// (16 times larger than it stands for): two pieces hold a BF16 value (8 bits)
// exactly down to 2^-13 of the row's largest and to 2^-22 of it below, three
// hold the FP32 activation h to 12 bits.  The pieces are neighbouring
// columns, and their products are added with factors 1, 1/16, 1/256.  The
// weight's block scale multiplies each block of 128's sum in FP32.  BF16
// weights take x as it is and h as two BF16 pieces (16 bits).
//
// One persistent CTA per SM, launched cooperatively (the CTAs wait for one
// another twice, after `route` and between `up` and `down`).  The k blocks
// of all tiles of a phase form one sequence that is cut into equal runs, one
// for each CTA, so the read is balanced whatever the number of reached
// experts.  A run's partial sums of a tile go to scratch; the last run to
// arrive at a tile adds them in the order of the runs, so the result does not
// depend on timing.  The producer of the weight tiles does not take part in the
// waits after `route`: it fills the stage ring with the first `down` tiles while
// the `up` sums are still being joined; and the warps that join the pieces are
// not those that take the sums out of the tensor memory, so neither does the
// ring wait for a join.
//
// Warps: 0 weight tiles, 1 MMA, 2 TMEM, 3 activation tiles, 4-7 sums, 8-11
// joins.
#include <algorithm>
#include <type_traits>

#include "sublayer.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int NT = 384, WARPS = NT / 32;
constexpr int SUM_WARP0 = 4, JOIN_WARP0 = 8;
constexpr int STAGES_MAX = 12;
constexpr int BUFS = 4, BUF_COLS = 128;
constexpr int A_BYTES = 128 * 128;
constexpr int SMEM_BYTES = 227 * 1024;
constexpr int EXPERTS = MOE_EXPERTS_MAX + MOE_SHARED_MAX;
constexpr int SLOTS = MOE_TOKENS_MAX * (MOE_TOPK_MAX + MOE_SHARED_MAX);
constexpr uint32_t POLL_LIMIT = 1u << 22;

__device__ int g_stall_copies;   // test hook: the producers issue no copies

struct Shared {
  uint64_t full[STAGES_MAX], empty[STAGES_MAX], acc_full[BUFS], acc_empty[BUFS], sum_full[2], sum_empty[2], drain;
  uint32_t tmem;
  int abort, last, active, issued_a, issued_b;
  float red[WARPS][8];
  uint32_t red_max[WARPS];
  float x_scale[MOE_TOKENS_MAX];
  uint32_t mask[EXPERTS];       // tokens of an expert, one bit each
  uint32_t act_mask[EXPERTS];   // the same of the reached experts, in order
  uint16_t act_expert[EXPERTS], act_base[EXPERTS], position[EXPERTS];
  float slot_weight[SLOTS];
  int16_t chosen[MOE_TOKENS_MAX][MOE_TOPK_MAX];
  float chosen_weight[MOE_TOKENS_MAX][MOE_TOPK_MAX];
};
constexpr int SMEM_TABLES = (int(sizeof(Shared)) + 1023) / 1024 * 1024;
constexpr int SMEM_SLACK = 1024;   // an MMA's columns are rounded up to 16: it may read 8 rows past the last stage

// ------------------------------------------------------------------ waits
__device__ __forceinline__ unsigned ld_acquire(const unsigned *p) {
  unsigned v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Until *p reaches `want`, another thread of the CTA gave up, or the limit.
__device__ __noinline__ bool poll(const unsigned *p, unsigned want, volatile int *abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < POLL_LIMIT; ++i) {
    if (ld_acquire(p) >= want) return true;
    if (*abort) return false;
    if (i > 256) __nanosleep(128);
  }
  *abort = 1;
  return false;
}
// Orders generic-proxy accesses to global memory and the TMA's.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// ------------------------------------------------------------- the sequence
// A phase's k blocks, cut into `runs` equal runs (run c: [total c / runs,
// total (c + 1) / runs)).
struct Sequence {
  int64_t total;
  int runs;
  __device__ int64_t begin(int c) const { return c >= runs ? total : total * c / runs; }
  // the run that holds unit u
  __device__ int run_of(int64_t u) const { return int(((u + 1) * runs - 1) / total); }
  // runs that share units [u, u + n)
  __device__ int pieces(int64_t u, int64_t n) const { return run_of(u + n - 1) - run_of(u) + 1; }
};

struct Shape {
  int up_tiles, up_k;       // up: tiles of 128 rows of an expert's gate (and of its up) and their k blocks
  int down_tiles, down_k;   // down: row blocks of the output, k blocks of an expert
};

template <bool FP8>
__device__ __forceinline__ Shape shape_of(const MoeParams &p) {
  constexpr int KB = FP8 ? 128 : 64;
  return {(p.intermediate + 127) / 128, (p.hidden + KB - 1) / KB, (p.hidden + 127) / 128,
          (p.intermediate + KB - 1) / KB};
}
// up: units (expert, tile, gate / up, k); runs of at least half a tile's k
// blocks, so that at most MOE_UP_FRAGMENTS share a tile
__device__ __forceinline__ Sequence up_sequence(const Shape &s, int active) {
  Sequence q;
  q.total = int64_t(active) * s.up_tiles * 2 * s.up_k;
  q.runs = int(min(int64_t(gridDim.x), max(int64_t(1), q.total / ((s.up_k + 1) / 2))));
  return q;
}
// down: units (row block, expert, k); at most MOE_DOWN_SPLIT runs a row block
__device__ __forceinline__ Sequence down_sequence(const Shape &s, int active) {
  Sequence q;
  q.total = int64_t(s.down_tiles) * active * s.down_k;
  q.runs = int(min(min(int64_t(gridDim.x), int64_t(s.down_tiles) * MOE_DOWN_SPLIT), q.total));
  return q;
}

// The position in a sequence: a tile's run of k blocks at a time, so that the
// loops over k blocks hold nothing but steps (a division for each block would
// take as long as the block's read).
struct UpCursor {     // (expert, gate / up tile, k)
  int a, r, kb;
  __device__ UpCursor(const Shape &s, int64_t u) {
    const int64_t tile = u / s.up_k;
    kb = int(u - tile * s.up_k);
    a = int(tile / (2 * s.up_tiles));
    r = int(tile - int64_t(a) * 2 * s.up_tiles);
  }
  // k blocks of this tile among the next `left` units
  __device__ int run(const Shape &s, int left) const { return min(s.up_k - kb, left); }
  __device__ void step(const Shape &s, int blocks) {
    kb += blocks;
    if (kb == s.up_k) {
      kb = 0;
      if (++r == 2 * s.up_tiles) {
        r = 0;
        ++a;
      }
    }
  }
};
struct DownCursor {   // (row block, expert, k)
  int rb, a, kb;
  __device__ DownCursor(const Shape &s, int active, int64_t u) {
    const int64_t tile = u / s.down_k;
    kb = int(u - tile * s.down_k);
    rb = int(tile / active);
    a = int(tile - int64_t(rb) * active);
  }
  __device__ int run(const Shape &s, int left) const { return min(s.down_k - kb, left); }
  __device__ void step(const Shape &s, int active, int blocks) {
    kb += blocks;
    if (kb == s.down_k) {
      kb = 0;
      if (++a == active) {
        a = 0;
        ++rb;
      }
    }
  }
};

// A place in a ring of barriers and the phase of its current round.  A
// producer waits for a slot's release with the other parity: that wait
// returns at once in the first round.
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ void next(int size) {
    if (++at == size) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// ----------------------------------------------------------------- pieces
// Power of two that brings a largest magnitude (bit pattern) to [128, 256);
// NaN where it is not finite, so that the row's outputs are.
__device__ __forceinline__ float piece_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
  const int e = max(int(amax_bits >> 23), 27);   // magnitudes under 2^-100 count as 2^-100
  return __uint_as_float(uint32_t(e - 7) << 23);
}
// 1 / piece_scale (exact; 0 for the NaN scale)
__device__ __forceinline__ float piece_inverse(float scale) {
  const uint32_t e = __float_as_uint(scale) >> 23;
  return e == 255u ? 0.f : __uint_as_float((254u - e) << 23);
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)b));
  float f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;\n\t}" : "=f"(f) : "r"(h));
  return f;
}

// ------------------------------------------------------------------ route
// Logits of all tokens for this CTA's experts: eight tokens at a time, the
// hidden size spread over all threads.
__device__ __forceinline__ void route_logits(const MoeParams &p, Shared &sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int frags = p.hidden / 8;
  for (int e = blockIdx.x; e < p.experts; e += gridDim.x)
    for (int t0 = 0; t0 < p.m; t0 += 8) {
      float acc[8] = {};
#pragma unroll 2
      for (int f = threadIdx.x; f < frags; f += NT) {
        float w[8];
        uint4 xv[8];
        const size_t at = size_t(e) * p.hidden + size_t(f) * 8;
#pragma unroll
        for (int t = 0; t < 8; ++t)
          xv[t] = t0 + t < p.m ? ld_ro(p.x + size_t(t0 + t) * p.hidden + size_t(f) * 8) : make_uint4(0, 0, 0, 0);
        if (p.router_f32) {
          const float *r = static_cast<const float *>(p.router) + at;
          const float4 a = __ldg(reinterpret_cast<const float4 *>(r)), b = __ldg(reinterpret_cast<const float4 *>(r) + 1);
          w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
          w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
        } else {
          unpack8(ld_ro(static_cast<const uint16_t *>(p.router) + at), w);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (t0 + t < p.m) {
            float x[8];
            unpack8(xv[t], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[t] = fmaf(x[k], w[k], acc[t]);
          }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t0 + t < p.m) acc[t] = warp_sum(acc[t]);
      __syncthreads();
      if (lane == 0)
#pragma unroll
        for (int t = 0; t < 8; ++t) sh.red[warp][t] = acc[t];
      __syncthreads();
      if (threadIdx.x < 8 && t0 + int(threadIdx.x) < p.m) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) s += sh.red[w][threadIdx.x];
        p.scratch.logits[size_t(t0 + threadIdx.x) * p.experts + e] = s;
      }
    }
}

// The E4M3 pieces of x: a row a CTA, from the last CTA down (the first ones
// have experts' logits to compute).
__device__ __forceinline__ void split_x(const MoeParams &p, Shared &sh) {
  constexpr int HELD = 4;   // fragments a thread keeps in registers between the two passes
  const int frags = p.hidden / 8;
  for (int t = int(gridDim.x) - 1 - int(blockIdx.x); t < p.m; t += gridDim.x) {
    const uint16_t *x = p.x + size_t(t) * p.hidden;
    uint32_t a = 0;
    auto peak = [&](const uint4 &v) {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) a = max(a, max((w[k] << 16) & 0x7fff0000u, w[k] & 0x7fff0000u));
    };
    uint4 held[HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k) {
      const int f = threadIdx.x + k * NT;
      held[k] = f < frags ? ld_ro(x + size_t(f) * 8) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < HELD; ++k) peak(held[k]);
    for (int f = threadIdx.x + HELD * NT; f < frags; f += NT) peak(ld_ro(x + size_t(f) * 8));
    a = __reduce_max_sync(0xffffffffu, a);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sh.red_max[threadIdx.x / 32] = a;
    __syncthreads();
    a = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) a = max(a, sh.red_max[k]);
    const float scale = piece_scale(a), inv = piece_inverse(scale);
    uint8_t *hi = p.scratch.x_pieces + size_t(2 * t) * p.hidden, *lo = hi + p.hidden;
    auto split = [&](const uint4 &x8, int f) {
      float v[8];
      unpack8(x8, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
      const uint2 h = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = (v[k] - from_e4m3((k < 4 ? h.x : h.y) >> (k % 4 * 8) & 0xffu)) * 16.f;
      *reinterpret_cast<uint2 *>(hi + size_t(f) * 8) = h;
      *reinterpret_cast<uint2 *>(lo + size_t(f) * 8) =
          make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (int(threadIdx.x) + k * NT < frags) split(held[k], threadIdx.x + k * NT);
    for (int f = threadIdx.x + HELD * NT; f < frags; f += NT) split(ld_ro(x + size_t(f) * 8), f);
    if (threadIdx.x == 0) p.scratch.x_scale[t] = scale;
  }
}

// Order-preserving unsigned key of a score; a NaN is below every number.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 0u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp chooses token t's experts from its logits: lane l holds experts
// l, l + 32, ... (PER of them).
template <int PER>
__device__ __noinline__ void choose(const MoeParams &p, Shared &sh, int t) {
  const int lane = threadIdx.x % 32;
  float score[PER];
  uint32_t key[PER];
  float peak = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    score[i] = e < p.experts ? __ldcg(p.scratch.logits + size_t(t) * p.experts + e) : -INFINITY;
    peak = fmaxf(peak, score[i]);
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      score[i] = i * 32 + lane < p.experts ? expf(score[i] - peak) : 0.f;
      sum += score[i];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] = score[i] / sum;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] = 1.f / (1.f + expf(-score[i]));
  }
  uint32_t taken = 0;   // bit i: expert i * 32 + lane is chosen or does not exist
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    if (e >= p.experts) taken |= 1u << i;
    key[i] = e < p.experts ? score_key(p.bias ? score[i] + __ldg(p.bias + e) : score[i]) : 0u;
  }
  float total = 0.f, mine = 0.f;
  int mine_e = 0;
  for (int k = 0; k < p.top_k; ++k) {
    uint32_t best = 0, at = 0xffffffffu;
    float value = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (!(taken >> i & 1u) && (at == 0xffffffffu || key[i] > best)) {
        best = key[i];
        at = uint32_t(i * 32 + lane);
        value = score[i];
      }
    // the largest key, then the lowest expert among the lanes that hold it
    const bool any = at != 0xffffffffu;
    const uint32_t top = __reduce_max_sync(0xffffffffu, any ? best : 0u);
    const uint32_t winner = __reduce_min_sync(0xffffffffu, any && best == top ? at : 0xffffffffu);
    const float w = __shfl_sync(0xffffffffu, value, int(winner % 32));
    if (at == winner) taken |= 1u << (winner / 32);
    total += w;
    if (lane == k) {
      mine = w;
      mine_e = int(winner);
    }
  }
  if (lane < p.top_k) {
    const float w = (p.renormalize ? mine / total : mine) * p.routed_scale;
    sh.chosen[t][lane] = int16_t(mine_e);
    sh.chosen_weight[t][lane] = w;
    atomicOr(&sh.mask[mine_e], 1u << t);
    if (blockIdx.x == 0) {
      if (p.idx) p.idx[t * p.top_k + lane] = mine_e;
      if (p.weights) p.weights[t * p.top_k + lane] = w;
    }
  }
}

// The reached experts in order, each one's tokens and first slot (a slot is a
// token of an expert), and the slots' weights.  Every CTA computes the same.
__device__ __forceinline__ void build_plan(const MoeParams &p, Shared &sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int every = p.experts + p.shared;
  const uint32_t all = p.m == 32 ? 0xffffffffu : (1u << p.m) - 1u;
  for (int e = threadIdx.x; e < every; e += NT) sh.mask[e] = e < p.experts ? 0u : all;
  __syncthreads();
  for (int t = warp; t < p.m; t += WARPS) {
    if (p.experts <= 64) choose<2>(p, sh, t);
    else if (p.experts <= 256) choose<8>(p, sh, t);
    else choose<MOE_EXPERTS_MAX / 32>(p, sh, t);
  }
  if (p.fp8 && threadIdx.x < p.m) sh.x_scale[threadIdx.x] = __ldcg(p.scratch.x_scale + threadIdx.x);
  __syncthreads();
  if (warp == 0) {
    int active = 0, slots = 0;
    for (int e0 = 0; e0 < every; e0 += 32) {
      const uint32_t mask = e0 + lane < every ? sh.mask[e0 + lane] : 0u;
      const uint32_t reached = __ballot_sync(0xffffffffu, mask != 0u);
      const int n = __popc(mask);
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (mask) {
        const int a = active + __popc(reached & ((1u << lane) - 1u));
        sh.act_mask[a] = mask;
        sh.act_expert[a] = uint16_t(e0 + lane);
        sh.act_base[a] = uint16_t(slots + upto - n);
        sh.position[e0 + lane] = uint16_t(a);
      }
      active += __popc(reached);
      slots += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) sh.active = active;
  }
  __syncthreads();
  // a token a lane, a route a warp
  for (int k = warp; lane < p.m && k < p.top_k + p.shared; k += WARPS) {
    const int a = sh.position[k < p.top_k ? sh.chosen[lane][k] : p.experts + k - p.top_k];
    const int slot = sh.act_base[a] + __popc(sh.act_mask[a] & ((1u << lane) - 1u));
    sh.slot_weight[slot] = k < p.top_k ? sh.chosen_weight[lane][k] : 1.f;
  }
  __syncthreads();
}

// -------------------------------------------------------------------- sums
// COLS columns of this thread's TMEM lane.
template <int COLS>
__device__ __forceinline__ void load_cols(uint32_t taddr, uint32_t (&d)[COLS]) {
  static_assert(COLS % 16 == 0, "16 columns a load");
#pragma unroll
  for (int c = 0; c < COLS; c += 16) tc::tmem_ld16_async(taddr + c, reinterpret_cast<uint32_t(&)[16]>(d[c]));
  tc::tmem_wait_ld();
  tc::tmem_hold(d);
}

__device__ __forceinline__ float value(uint32_t bits) { return __uint_as_float(bits); }

// Sums of the k blocks [kb0, kb1) of a tile for this thread's row and CT
// columns' tokens (P pieces each): block sums from the accumulator ring,
// their pieces added, times the weight's block scale
// and, where `act` is given, the activation's (`count` of them a block,
// `act_step` apart from block to block).  What lies beyond `count` is not
// used.
template <bool FP8, int P, int CT>
__device__ __forceinline__ void sum_blocks(Shared &sh, uint32_t lane_base, Ring &ring, int kb0, int kb1, const float *sw,
                                           int sw_count, const float *act, int act_step, int count,
                                           float (&acc)[CT]) {
  constexpr int COLS = (CT * P + 15) / 16 * 16;
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int t = 0; t < CT; ++t) acc[t] = 0.f;
  float held = 0.f;     // lane l: the weight scale of block (kb & ~31) + l
  // lane l: the activation scale of token l, one block ahead
  float next = FP8 && act && lane < count ? __ldcg(act + size_t(kb0) * act_step + lane) : 0.f;
  for (int kb = kb0; kb < kb1; ++kb) {
    float scale = 1.f;
    if (FP8) {
      if (kb == kb0 || kb % 32 == 0) {
        const int k = kb / 32 * 32 + lane;
        held = k < sw_count ? __ldg(sw + k) : 0.f;
      }
      scale = __shfl_sync(0xffffffffu, held, kb % 32);
      if (act) {
        scale *= next;
        if (kb + 1 < kb1 && lane < count) next = __ldcg(act + size_t(kb + 1) * act_step + lane);
      }
    }
    tc::wait_or_abort(&sh.acc_full[ring.at], ring.phase, &sh.abort);
    __syncwarp();
    tc::fence_after_sync();
    uint32_t d[COLS];
    load_cols(lane_base + uint32_t(ring.at * BUF_COLS), d);
    tc::fence_before_sync();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.acc_empty[ring.at]);
    ring.next(BUFS);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      if (FP8) {
        float v = value(d[P * t + P - 1]);
#pragma unroll
        for (int c = P - 2; c >= 0; --c) v = fmaf(v, 0.0625f, value(d[P * t + c]));
        acc[t] = fmaf(v, act ? __shfl_sync(0xffffffffu, scale, t) : scale, acc[t]);
      } else {
#pragma unroll
        for (int c = 0; c < P; ++c) acc[t] += value(d[P * t + c]);
      }
    }
  }
}

// Takes the sums of a tile's run for `count` tokens and gives token t's to
// emit(t, sum); the width of the work follows the count.
template <bool FP8, int P, class Emit>
__device__ __forceinline__ void sum_tile(Shared &sh, uint32_t lane_base, Ring &ring, int kb0, int kb1, const float *sw,
                                         int sw_count, const float *act, int act_step, int count, const Emit &emit) {
  auto with = [&](auto ct) {
    constexpr int CT = decltype(ct)::value;
    float acc[CT];
    sum_blocks<FP8, P, CT>(sh, lane_base, ring, kb0, kb1, sw, sw_count, act, act_step, count, acc);
#pragma unroll
    for (int t = 0; t < CT; ++t)
      if (t < count) emit(t, acc[t]);
  };
  if (count <= 5) with(std::integral_constant<int, 5>());
  else if (count <= 10) with(std::integral_constant<int, 10>());
  else with(std::integral_constant<int, MOE_TOKENS_MAX>());
}

// ------------------------------------------------------------------- joins
// h = silu(g) u of one token's 128 rows (four a lane) to its pieces for the
// down product.
template <bool FP8>
__device__ __forceinline__ void store_act(const MoeParams &p, int slot, int j, const float4 &g4, const float4 &u4) {
  const int lane = threadIdx.x % 32, row = j * 128 + lane * 4;
  const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
  const bool live = row < p.intermediate;   // four rows are in or out together
  float h[4];
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = live ? g[k] / (1.f + expf(-g[k])) * u[k] : 0.f;
    top = max(top, __float_as_uint(h[k]) & 0x7fffffffu);
  }
  if (FP8) {
    const float scale = piece_scale(__reduce_max_sync(0xffffffffu, top)), inv = piece_inverse(scale);
    if (lane == 0) p.scratch.act_scale[size_t(j) * p.slots + slot] = scale;
    uint8_t *dst = static_cast<uint8_t *>(p.scratch.act) + size_t(slot) * 3 * p.intermediate + row;
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] *= inv;
    if (live)
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const uint32_t b = e4m3x4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint32_t *>(dst + size_t(c) * p.intermediate) = b;
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = (h[k] - from_e4m3(b >> (8 * k) & 0xffu)) * 16.f;
      }
  } else if (live) {
    uint16_t *dst = static_cast<uint16_t *>(p.scratch.act) + size_t(slot) * 2 * p.intermediate + row;
    const uint2 hi = make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
    *reinterpret_cast<uint2 *>(dst) = hi;
    *reinterpret_cast<uint2 *>(dst + p.intermediate) =
        make_uint2(pack_bf16x2(h[0] - bf16_lo(hi.x), h[1] - bf16_hi(hi.x)),
                   pack_bf16x2(h[2] - bf16_lo(hi.y), h[3] - bf16_hi(hi.y)));
  }
}

__device__ __forceinline__ float4 add4(const float4 &a, const float4 &b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 ldcg4(const float *p) { return __ldcg(reinterpret_cast<const float4 *>(p)); }

// A finished tile of an expert from the runs' pieces in scratch, added in the
// order of the runs; a warp a token.
template <bool FP8>
__device__ __forceinline__ void finish_up(const MoeParams &p, int base, int count, int j, int up_tiles, int gate_pieces,
                                          int up_pieces) {
  const int warp = threadIdx.x / 32 - JOIN_WARP0, lane = threadIdx.x % 32;
  const size_t width = size_t(up_tiles) * 128, step = size_t(p.slots) * 2 * width;
#pragma unroll 2
  for (int t = warp; t < count; t += 4) {
    const float *src = p.scratch.up + size_t(base + t) * 2 * width + j * 128 + lane * 4;
    float4 g[MOE_UP_FRAGMENTS], u[MOE_UP_FRAGMENTS];
#pragma unroll
    for (int f = 0; f < MOE_UP_FRAGMENTS; ++f) {
      g[f] = f < gate_pieces ? ldcg4(src + f * step) : make_float4(0.f, 0.f, 0.f, 0.f);
      u[f] = f < up_pieces ? ldcg4(src + f * step + width) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int f = 1; f < MOE_UP_FRAGMENTS; ++f) {
      if (f < gate_pieces) g[0] = add4(g[0], g[f]);
      if (f < up_pieces) u[0] = add4(u[0], u[f]);
    }
    store_act<FP8>(p, base + t, j, g[0], u[0]);
  }
}

// ----------------------------------------------------------------- kernel
template <bool FP8>
__global__ void __launch_bounds__(NT, 1)
k_moe(const MoeParams p, const __grid_constant__ CUtensorMap tm_gate_up, const __grid_constant__ CUtensorMap tm_down,
      const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x_token,
      const __grid_constant__ CUtensorMap tm_act) {
  constexpr int KB = FP8 ? 128 : 64;                        // values of a 128-byte k block
  constexpr int XP = FP8 ? 2 : 1, HP = FP8 ? 3 : 2;         // pieces of x and of h
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  float *sums = reinterpret_cast<float *>(smem + SMEM_TABLES);   // two buffers [m][128] from the sums to the joins
  unsigned char *ring = smem + SMEM_TABLES + p.m * 1024;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &sh.abort;
  const int stage_bytes = A_BYTES + p.b_bytes;
  unsigned *routed = p.scratch.control, *ups_done = routed + 1, *exits = routed + 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      tc::mbar_init(&sh.full[i], 2);
      tc::mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      tc::mbar_init(&sh.acc_full[i], 1);
      tc::mbar_init(&sh.acc_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.sum_full[i], 4);
      tc::mbar_init(&sh.sum_empty[i], 4);
    }
    tc::mbar_init(&sh.drain, 1);
    tc::mbar_init_fence();
    sh.abort = 0;
    sh.issued_a = sh.issued_b = 0;
    tc::tma_prefetch_desc(&tm_gate_up);
    tc::tma_prefetch_desc(&tm_down);
    tc::tma_prefetch_desc(&tm_x);
    tc::tma_prefetch_desc(&tm_x_token);
    tc::tma_prefetch_desc(&tm_act);
  }
  if (warp == 2) tc::tmem_alloc(&sh.tmem, BUFS * BUF_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  // ---- route
  route_logits(p, sh);
  if (FP8) split_x(p, sh);
  fence_proxy_async_global();
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    atomicAdd(routed, 1u);
    poll(routed, gridDim.x, abort);
  }
  __syncthreads();
  const bool gave_up = *abort != 0;   // the same in all threads: no role has begun
  build_plan(p, sh);

  const Shape s = shape_of<FP8>(p);
  const int active = sh.active;
  const Sequence up = up_sequence(s, active), down = down_sequence(s, active);
  const int cta = blockIdx.x;
  const int64_t up0 = up.begin(cta), up1 = up.begin(cta + 1), down0 = down.begin(cta), down1 = down.begin(cta + 1);
  const int up_n = int(up1 - up0), down_n = int(down1 - down0);
  UpCursor uc(s, up0);
  DownCursor dc(s, active, down0);
  const unsigned up_total = unsigned(active) * unsigned(s.up_tiles);

  if (gave_up) {
    // the logits never came: no role begins
  } else if (warp == 0) {
    // ----------------------------------------------------- weight tiles
    Ring at;
    int issued = 0;
    bool ok = !g_stall_copies;
    const bool leader = tc::elect_one();
    auto load = [&](const CUtensorMap *map, int kb, int row, int blocks) {
      for (int k = 0; k < blocks; ++k) {
        ok = ok && tc::wait_or_abort(&sh.empty[at.at], at.phase ^ 1u, abort);
        if (!ok) return;
        if (leader) {
          tc::mbar_arrive_expect_tx(&sh.full[at.at], A_BYTES);
          tc::tma_load_2d(ring + size_t(at.at) * stage_bytes, map, (kb + k) * KB, row, &sh.full[at.at]);
        }
        __syncwarp();
        at.next(p.stages);
        ++issued;
      }
    };
    for (int n = 0, run; n < up_n && ok; n += run) {
      run = uc.run(s, up_n - n);
      load(&tm_gate_up, uc.kb, (sh.act_expert[uc.a] * 2 + (uc.r & 1)) * p.intermediate + (uc.r >> 1) * 128, run);
      uc.step(s, run);
    }
    for (int n = 0, run; n < down_n && ok; n += run) {
      run = dc.run(s, down_n - n);
      load(&tm_down, dc.kb, sh.act_expert[dc.a] * p.hidden + dc.rb * 128, run);
      dc.step(s, active, run);
    }
    if (lane == 0) sh.issued_a = issued;
  } else if (warp == 3) {
    // ------------------------------------------------- activation tiles
    Ring at;
    int issued = 0;
    bool ok = !g_stall_copies;
    // `copies` copies of a k block, one a lane, of `bytes` in all: this lane's
    // from row `row` to byte `place` of the stage
    auto load = [&](const CUtensorMap *map, int kb, int blocks, int copies, int bytes, int row, int place) {
      for (int k = 0; k < blocks; ++k) {
        ok = ok && tc::wait_or_abort(&sh.empty[at.at], at.phase ^ 1u, abort);
        if (!ok) return;
        if (lane == 0) tc::mbar_arrive_expect_tx(&sh.full[at.at], uint32_t(bytes));
        __syncwarp();
        if (lane < copies)
          tc::tma_load_2d(ring + size_t(at.at) * stage_bytes + A_BYTES + place, map, (kb + k) * KB, row,
                          &sh.full[at.at]);
        __syncwarp();
        at.next(p.stages);
        ++issued;
      }
    };
    fence_proxy_async_global();
    const int x_rows = (p.m * XP + 7) / 8 * 8;
    for (int n = 0, run; n < up_n && ok; n += run) {
      run = uc.run(s, up_n - n);
      const uint32_t mask = sh.act_mask[uc.a];
      const int count = __popc(mask);
      // all tokens in one copy; else the expert's tokens only, a copy each:
      // their rows' swizzle goes by their place in shared memory, as the
      // tensor core reads them
      if (count == p.m) load(&tm_x, uc.kb, run, 1, x_rows * 128, 0, 0);
      else load(&tm_x_token, uc.kb, run, count, count * XP * 128, __fns(mask, 0, lane + 1) * XP, lane * XP * 128);
      uc.step(s, run);
    }
    if (down_n > 0 && ok) {
      ok = poll(ups_done, up_total, abort);
      ok = __all_sync(0xffffffffu, ok);
      fence_proxy_async_global();
    }
    for (int n = 0, run; n < down_n && ok; n += run) {
      run = dc.run(s, down_n - n);
      const int boxes = (__popc(sh.act_mask[dc.a]) * HP + 7) / 8;
      load(&tm_act, dc.kb, run, boxes, boxes * 1024, sh.act_base[dc.a] * HP + lane * 8, lane * 1024);
      dc.step(s, active, run);
    }
    if (lane == 0) sh.issued_b = issued;
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA
    Ring at, acc;
    bool ok = true;
    const bool leader = tc::elect_one();
    const uint64_t a0 = tc::desc_sw128(ring), b0 = tc::desc_sw128(ring + A_BYTES);
    auto multiply = [&](int columns, int blocks) {
      const int cols = (columns + 15) / 16 * 16;
      const uint32_t idesc = FP8 ? tc::idesc_e4m3_f32(128, cols) : tc::idesc_bf16_f32(128, cols);
      for (int k = 0; k < blocks; ++k) {
        ok = ok && tc::wait_or_abort(&sh.full[at.at], at.phase, abort) &&
             tc::wait_or_abort(&sh.acc_empty[acc.at], acc.phase ^ 1u, abort);
        if (!ok) return;
        tc::fence_after_sync();
        const uint64_t step = uint64_t(at.at * (stage_bytes >> 4));
        const uint32_t d = tmem + uint32_t(acc.at * BUF_COLS);
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            if (FP8) tc::mma_e4m3(d, a0 + step + 2 * ks, b0 + step + 2 * ks, idesc, ks != 0);
            else tc::mma_bf16(d, a0 + step + 2 * ks, b0 + step + 2 * ks, idesc, ks != 0);
          }
          tc::mma_commit(&sh.empty[at.at]);
          tc::mma_commit(&sh.acc_full[acc.at]);
        }
        __syncwarp();
        at.next(p.stages);
        acc.next(BUFS);
      }
    };
    for (int n = 0, run; n < up_n && ok; n += run) {
      run = uc.run(s, up_n - n);
      multiply(__popc(sh.act_mask[uc.a]) * XP, run);
      uc.step(s, run);
    }
    for (int n = 0, run; n < down_n && ok; n += run) {
      run = dc.run(s, down_n - n);
      multiply(__popc(sh.act_mask[dc.a]) * HP, run);
      dc.step(s, active, run);
    }
    // no MMA is in flight when the tensor memory goes
    if (leader) tc::mma_commit(&sh.drain);
    __syncwarp();
    tc::mbar_wait_bounded(&sh.drain, 0u, tc::SUB_WAIT_LIMIT);
  } else if (warp >= SUM_WARP0 && warp < JOIN_WARP0) {
    // ------------------------------------------------------------- sums
    // After a wait gave up these warps and the joins go through the rest of
    // their loops on whatever is there (the waits return at once), so that they
    // meet at their barriers and every arrival is counted.
    const int i = threadIdx.x - SUM_WARP0 * 32;   // row of the tile
    const uint32_t lane_base = tmem + (uint32_t((warp % 4) * 32) << 16);
    Ring acc;
    int given = 0;
    auto take = [&]() {   // the next buffer, once the joins have emptied it
      if (given >= 2) tc::wait_or_abort(&sh.sum_empty[given % 2], uint32_t((given / 2 - 1) & 1), abort);
      __syncwarp();
      return sums + size_t(given % 2) * p.m * 128 + i;
    };
    auto give = [&]() {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.sum_full[given % 2]);
      ++given;
    };
    // ---- up
    for (int n = 0, run; n < up_n; n += run) {
      run = uc.run(s, up_n - n);
      const float *sw = p.gate_up_scales +
                        ((size_t(sh.act_expert[uc.a]) * 2 + (uc.r & 1)) * s.up_tiles + (uc.r >> 1)) * s.up_k;
      uint32_t rest = sh.act_mask[uc.a];
      float *dst = nullptr;
      sum_tile<FP8, XP>(sh, lane_base, acc, uc.kb, uc.kb + run, sw, s.up_k, nullptr, 0, __popc(rest),
                        [&](int t, float v) {
                          if (t == 0) dst = take();
                          if (FP8) {
                            v *= sh.x_scale[__ffs(rest) - 1];
                            rest &= rest - 1u;
                          }
                          dst[t * 128] = v;
                        });
      give();
      uc.step(s, run);
    }
    // ---- down
    if (down_n > 0) poll(ups_done, up_total, abort);
    __syncwarp();
    for (int n = 0; n < down_n;) {
      const int rb = dc.rb;
      float *y = take();
      for (int t = 0; t < p.m; ++t) y[t * 128] = 0.f;
      for (int run; n < down_n && dc.rb == rb; n += run) {
        run = dc.run(s, down_n - n);
        const int base = sh.act_base[dc.a];
        const float *sw = p.down_scales + (size_t(sh.act_expert[dc.a]) * s.down_tiles + rb) * s.down_k;
        uint32_t rest = sh.act_mask[dc.a];
        sum_tile<FP8, HP>(sh, lane_base, acc, dc.kb, dc.kb + run, sw, s.down_k, p.scratch.act_scale + base, p.slots,
                          __popc(rest), [&](int t, float v) {
                            float *at = y + (__ffs(rest) - 1) * 128;
                            rest &= rest - 1u;
                            *at = fmaf(v, sh.slot_weight[base + t], *at);
                          });
        dc.step(s, active, run);
      }
      give();
    }
  } else if (warp >= JOIN_WARP0) {
    // ------------------------------------------------------------ joins
    const int jw = warp - JOIN_WARP0;
    const size_t width = size_t(s.up_tiles) * 128;
    int taken = 0;
    auto wait_sum = [&](int k) {
      tc::wait_or_abort(&sh.sum_full[k % 2], uint32_t((k / 2) & 1), abort);
      __syncwarp();
      return sums + size_t(k % 2) * p.m * 128;
    };
    auto release = [&](int k) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.sum_empty[k % 2]);
    };
    // whether this run is the last of `want` to arrive at a counter, what all
    // have written then being visible; the whole warps' threads call it
    auto arrive = [&](unsigned *counter, unsigned want) {
      __threadfence();
      tc::named_barrier(1, 128);
      if (threadIdx.x == JOIN_WARP0 * 32) {
        const bool last = atomicAdd(counter, 1u) == want - 1;
        if (last) *counter = 0;
        sh.last = last;
      }
      tc::named_barrier(1, 128);
      const bool last = sh.last != 0;
      if (last) __threadfence();
      return last;
    };
    // ---- up
    for (int n = 0; n < up_n;) {
      const int a = uc.a, r = uc.r, j = r >> 1;
      const int base = sh.act_base[a], count = __popc(sh.act_mask[a]);
      bool done = true;
      if (!(r & 1) && uc.kb == 0 && n + 2 * s.up_k <= up_n) {
        // gate and up of the tile lie in this run: no scratch
        const float *g = wait_sum(taken), *u = wait_sum(taken + 1);
        for (int t = jw; t < count; t += 4)
          store_act<FP8>(p, base + t, j, reinterpret_cast<const float4 *>(g + t * 128)[lane],
                         reinterpret_cast<const float4 *>(u + t * 128)[lane]);
        release(taken);
        release(taken + 1);
        taken += 2;
        n += 2 * s.up_k;
        uc.r = r + 1;
        uc.step(s, s.up_k);
      } else {
        const int run = uc.run(s, up_n - n);
        const int64_t u0 = (int64_t(a) * s.up_tiles + j) * 2 * s.up_k;
        const int gate_pieces = up.pieces(u0, s.up_k), up_pieces = up.pieces(u0 + s.up_k, s.up_k);
        const int piece = cta - up.run_of(u0 + (r & 1) * s.up_k);
        float *dst = p.scratch.up + (size_t(piece) * p.slots + base) * 2 * width + (r & 1) * width + j * 128;
        const float *src = wait_sum(taken);
        for (int t = jw; t < count; t += 4)
          __stcg(reinterpret_cast<float4 *>(dst + size_t(t) * 2 * width) + lane,
                 reinterpret_cast<const float4 *>(src + t * 128)[lane]);
        release(taken++);
        done = arrive(p.scratch.up_counters + a * s.up_tiles + j, unsigned(gate_pieces + up_pieces));
        if (done) finish_up<FP8>(p, base, count, j, s.up_tiles, gate_pieces, up_pieces);
        n += run;
        uc.step(s, run);
      }
      if (done) {
        fence_proxy_async_global();
        __threadfence();
        tc::named_barrier(1, 128);
        if (threadIdx.x == JOIN_WARP0 * 32) atomicAdd(ups_done, 1u);
      }
    }
    // ---- down
    const int64_t rb_units = int64_t(active) * s.down_k;
    for (int64_t u = down0; u < down1;) {
      const int rb = dc.rb;
      const int64_t rb_u0 = rb * rb_units;
      const int pieces = down.pieces(rb_u0, rb_units);
      const float *src = wait_sum(taken);
      // an item: a token's four neighbouring rows
      const size_t step = size_t(s.down_tiles) * p.m * 128;
      float *part = p.scratch.down + size_t(rb) * p.m * 128;
      auto store_y = [&](int k, const float4 &y) {
        const int row = rb * 128 + k % 32 * 4;   // hidden is a multiple of 8: four rows are in or out together
        if (row < p.hidden) {
          uint16_t *out = p.output + size_t(k / 32) * p.hidden + row;
          const uint32_t lo = pack_bf16x2(y.x, y.y), hi = pack_bf16x2(y.z, y.w);
          if (p.vector_out) {
            *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
          } else {
            out[0] = uint16_t(lo);
            out[1] = uint16_t(lo >> 16);
            out[2] = uint16_t(hi);
            out[3] = uint16_t(hi >> 16);
          }
        }
      };
      const int items = p.m * 32, first = threadIdx.x - JOIN_WARP0 * 32;
      if (pieces == 1) {
        for (int k = first; k < items; k += 128) store_y(k, reinterpret_cast<const float4 *>(src)[k]);
        release(taken++);
      } else {
        float *dst = part + (cta - down.run_of(rb_u0)) * step;
        for (int k = first; k < items; k += 128)
          __stcg(reinterpret_cast<float4 *>(dst) + k, reinterpret_cast<const float4 *>(src)[k]);
        release(taken++);
        if (arrive(p.scratch.down_counters + rb, unsigned(pieces)))
#pragma unroll 2
          for (int k = first; k < items; k += 128) {
            float4 y[MOE_DOWN_FRAGMENTS];
#pragma unroll
            for (int f = 0; f < MOE_DOWN_FRAGMENTS; ++f)
              y[f] = f < pieces ? ldcg4(part + f * step + size_t(k) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int f = 1; f < MOE_DOWN_FRAGMENTS; ++f)
              if (f < pieces) y[0] = add4(y[0], y[f]);
            store_y(k, y[0]);
          }
      }
      u = min(down1, rb_u0 + rb_units);
      ++dc.rb;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 2) tc::tmem_dealloc(tmem, BUFS * BUF_COLS);
  if (threadIdx.x == 0) {
    if (*abort) {
      atomicOr(p.err, 2u);
      // copies in flight land before the CTA's shared memory goes: the stages
      // that only one of the two producers filled lack one arrival
      const int lo = min(sh.issued_a, sh.issued_b), hi = max(sh.issued_a, sh.issued_b);
      for (int n = lo; n < hi; ++n) tc::mbar_arrive(&sh.full[n % p.stages]);
      for (int n = max(0, hi - p.stages); n < hi; ++n)
        tc::mbar_wait_bounded(&sh.full[n % p.stages], uint32_t((n / p.stages) & 1), tc::SUB_WAIT_LIMIT);
    }
    // the last CTA to leave puts the grid's counters back
    if (atomicAdd(exits, 1u) == gridDim.x - 1) {
      *routed = 0;
      *ups_done = 0;
      *exits = 0;
    }
  }
}

template <bool FP8>
cudaError_t launch(const MoeParams &p, int sms, const CUtensorMap *maps, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_moe<FP8>, p, maps[0], maps[1], maps[2], maps[3], maps[4]);
}

}  // namespace

cudaError_t moe_stall_copies(int on) { return cudaMemcpyToSymbol(g_stall_copies, &on, sizeof on); }

cudaError_t moe_set_attributes() {
  cudaError_t e = cudaSuccess;
  for (const void *k : {(const void *)k_moe<false>, (const void *)k_moe<true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  return e;
}

cudaError_t launch_moe(const MoeParams &args, int sms, cudaStream_t stream) {
  MoeParams p = args;
  const bool fp8 = p.fp8 != 0;
  const int every = p.experts + p.shared, elem = fp8 ? 1 : 2, kb = fp8 ? 128 : 64;
  const int xp = fp8 ? 2 : 1, hp = fp8 ? 3 : 2;
  p.b_bytes = (p.m * std::max(xp, hp) + 7) / 8 * 1024;
  p.stages = std::min(STAGES_MAX, (SMEM_BYTES - SMEM_TABLES - SMEM_SLACK - p.m * 1024) / (A_BYTES + p.b_bytes));
  p.vector_out = reinterpret_cast<uintptr_t>(p.output) % 8 == 0;
  const CUtensorMapDataType type = fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t H = p.hidden, I = p.intermediate;
  const void *x = fp8 ? static_cast<const void *>(p.scratch.x_pieces) : p.x;
  CUtensorMap maps[5];
  if (!encode_rows_sw128(&maps[0], type, p.gate_up, uint64_t(every) * 2 * I, H, H * elem, kb, 128) ||
      !encode_rows_sw128(&maps[1], type, p.down, uint64_t(every) * H, I, I * elem, kb, 128) ||
      !encode_rows_sw128(&maps[2], type, x, uint64_t(p.m) * xp, H, H * elem, kb, (p.m * xp + 7) / 8 * 8) ||
      !encode_rows_sw128(&maps[3], type, x, uint64_t(p.m) * xp, H, H * elem, kb, xp) ||
      !encode_rows_sw128(&maps[4], type, p.scratch.act, uint64_t(p.slots) * hp, I, I * elem, kb, 8))
    return cudaErrorInvalidValue;
  return fp8 ? launch<true>(p, sms, maps, stream) : launch<false>(p, sms, maps, stream);
}

}  // namespace mhc
