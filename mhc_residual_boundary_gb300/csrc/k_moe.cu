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
// (16 times larger than it stands for).  Three pieces hold a BF16 value (8 bits)
// exactly down to 2^-17 of the row's largest (2^-10 where that is in [128, 256):
// the last piece's smallest step, 2^-9, stands for 2^-17, an ulp of 2^-10) and
// to half that step, 2^-25 of the largest, below; two would end at 2^-13 and
// 2^-21.  Three hold the FP32 activation h to 12 bits.  The pieces are neighbouring
// columns, and their products are added with factors 1, 1/16, 1/256.  The
// weight's block scale multiplies each block of 128's sum in FP32.  BF16
// weights take x as it is and h as two BF16 pieces (16 bits).
//
// One persistent CTA per SM, launched cooperatively (after `route` the CTAs wait
// for one another).  The work is one list of items, a tile's chunk of k blocks
// each: first all of `up`, then all of `down`, both expert by expert.  A CTA
// takes the next item when its producer comes to it, so CTAs with experts of
// many tokens, whose blocks take longer, take fewer.  An item waits only for
// items before it (a `down` item for its expert's `up` tiles, which were taken
// long before), so the memory is read without a break from the first item to
// the last.  An item's sums go to scratch, by the item's place, and are added in
// the order of the chunks by whoever finds a tile complete: the result does not
// depend on who took which item when.
//
// Measured (a call among others in a graph; H 5120, I 2048, 64 experts, the best 8
// and a shared one, 8-bit weights): one token 63 us, 4.5 TB/s of weights, of which
// some 9 us pass before the first item's weights are asked for (logits, a meeting
// of all CTAs, the choice, each of them first fetches of code and memory trips) and
// 7 us after the last are there; 32 tokens, which reach nearly every expert, 342
// us, 5.9 TB/s or 0.87 of a copy.  With BF16 weights 94 us and 596 us, 6.0 and 6.8
// TB/s.  Five tokens of a small BF16 layer (1024 x 512, 16 experts) take 24 us, a
// chain of such trips.
//
// Warps: 0 items and weight tiles, 1 MMA, 2 scales, 3 activation tiles, 4-7 sums
// (tensor memory to buffers), 8-11 joins (buffers to scratch, activations).
#include <algorithm>
#include <type_traits>

#include "sublayer.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int NT = 384, WARPS = NT / 32;
constexpr int SUM_WARP0 = 4, JOIN_WARP0 = 8;
constexpr int STAGES_MAX = 12;
constexpr int ITEMS = MOE_ITEMS;
constexpr int BUFS = 4, BUF_COLS = 128;
constexpr int A_BYTES = MOE_STAGE_A;
constexpr int SMEM_BYTES = MOE_SMEM;
constexpr int EXPERTS = MOE_EXPERTS_MAX + MOE_SHARED_MAX;
constexpr uint32_t POLL_LIMIT = 1u << 22;

__device__ int g_stall_copies;   // test hook: the producers issue no copies

struct Shared {
  uint64_t full[STAGES_MAX], empty[STAGES_MAX], acc_full[BUFS], acc_empty[BUFS], sum_full[4], sum_empty[2],
      item_full[ITEMS], item_empty[ITEMS], scale_full[ITEMS], drain;
  uint32_t tmem;
  int abort, active, issued_a, issued_b;
  int item[ITEMS];
  float red[WARPS][8];
  uint32_t red_max[WARPS];
  float x_scale[MOE_TOKENS_MAX];
  int warp_active[WARPS], warp_slots[WARPS];
  uint32_t mask[EXPERTS];       // tokens of an expert, one bit each; the shared experts come first
  uint32_t act_mask[EXPERTS];   // the same of the reached experts, in that order
  uint16_t act_expert[EXPERTS], act_base[EXPERTS], position[EXPERTS];
  int16_t route_expert[MOE_TOKENS_MAX][MOE_TOPK_MAX];               // a token's chosen experts
  int16_t route_slot[MOE_TOKENS_MAX][MOE_TOPK_MAX + MOE_SHARED_MAX];  // the slots of its chosen and shared experts
  float route_weight[MOE_TOKENS_MAX][MOE_TOPK_MAX];
};
constexpr int SMEM_TABLES = (int(sizeof(Shared)) + 1023) / 1024 * 1024;
constexpr int SMEM_SLACK = 1024;   // an MMA's columns are rounded up to 16: it may read 8 rows past the last stage
// The sums read a block's scales for 5, 10 or 32 tokens, however many it has (what
// is read for the others is not used): so many words lie after the last block's.
constexpr int SCALE_SLACK = MOE_TOKENS_MAX * 4;

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
// Until experts [ready, need) are complete: the whole warp looks at the next 32
// counters with one read (it takes microseconds while the memory is busy) and
// returns how many experts, in order, are.
__device__ __noinline__ int poll_experts(const unsigned *done, unsigned tiles, int ready, int need, int active,
                                         volatile int *abort) {
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (uint32_t i = 0; i < POLL_LIMIT; ++i) {
    const bool complete = ready + lane >= active || ld_acquire(done + ready + lane) >= tiles;
    const uint32_t missing = ~__ballot_sync(0xffffffffu, complete);
    ready += missing ? __ffs(missing) - 1 : 32;
    if (ready >= need || __any_sync(0xffffffffu, *abort != 0)) break;
    if (i > 256) __nanosleep(128);
  }
  if (ready < need) *abort = 1;
  return ready;
}
// Orders generic-proxy accesses to global memory and the TMA's.
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// ---------------------------------------------------------------- the items
struct Shape {
  int up_tiles, up_k;       // up: tiles of 128 rows of an expert's gate (and of its up) and their k blocks
  int down_tiles, down_k;   // down: row blocks of the output, k blocks of an expert
  int up_chunks, down_chunks;
  int up_items, items;      // of `up`, of both
};

template <bool FP8>
__device__ __forceinline__ Shape shape_of(const MoeParams &p, int active) {
  constexpr int KB = FP8 ? 128 : 64;
  Shape s;
  s.up_tiles = (p.intermediate + 127) / 128;
  s.up_k = (p.hidden + KB - 1) / KB;
  s.down_tiles = (p.hidden + 127) / 128;
  s.down_k = (p.intermediate + KB - 1) / KB;
  s.up_chunks = p.up_chunks;
  s.down_chunks = p.down_chunks;
  s.up_items = active * s.up_tiles * 2 * s.up_chunks;
  s.items = s.up_items + active * s.down_tiles * s.down_chunks;
  return s;
}

struct Item {
  bool down;
  int a;        // reached expert
  int tile;     // up: tile of the intermediate size; down: row block of the output
  int half;     // up: 0 gate, 1 up
  int chunk, kb0, blocks;
};
__device__ __forceinline__ Item item_at(const Shape &s, int i) {
  Item it;
  it.down = i >= s.up_items;
  if (!it.down) {
    int q = i / s.up_chunks;
    it.chunk = i - q * s.up_chunks;
    it.half = q & 1;
    q >>= 1;
    it.a = q / s.up_tiles;
    it.tile = q - it.a * s.up_tiles;
    it.kb0 = s.up_k * it.chunk / s.up_chunks;
    it.blocks = s.up_k * (it.chunk + 1) / s.up_chunks - it.kb0;
  } else {
    i -= s.up_items;
    const int q = i / s.down_chunks;
    it.chunk = i - q * s.down_chunks;
    it.half = 0;
    it.a = q / s.down_tiles;
    it.tile = q - it.a * s.down_tiles;
    it.kb0 = s.down_k * it.chunk / s.down_chunks;
    it.blocks = s.down_k * (it.chunk + 1) / s.down_chunks - it.kb0;
  }
  return it;
}

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
// An item is an expert and eight tokens; a CTA's warps take as many items at a
// time (1, 2, 3 or 6) as spread them over all CTAs.
__device__ __forceinline__ int router_groups(const MoeParams &p) {
  int groups = 1;
  while (groups < 6 && p.experts * ((p.m + 7) / 8) > groups * int(gridDim.x)) groups = groups == 3 ? 6 : groups + 1;
  return groups;
}
// Logits, the hidden size being spread over the warps of an item.
__device__ __forceinline__ void route_logits(const MoeParams &p, Shared &sh) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int frags = p.hidden / 8, items = p.experts * ((p.m + 7) / 8);
  const int groups = router_groups(p);
  const int warps = WARPS / groups, group = warp / warps;
  for (int i0 = blockIdx.x * groups; i0 < items; i0 += gridDim.x * groups) {
    const int item = i0 + group, e = item % p.experts, t0 = item / p.experts * 8;
    float acc[8] = {};
    if (item < items) {
#pragma unroll 2
      for (int f = threadIdx.x - group * warps * 32; f < frags; f += warps * 32) {
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
    }
    __syncthreads();
    if (lane == 0)
#pragma unroll
      for (int t = 0; t < 8; ++t) sh.red[warp][t] = acc[t];
    __syncthreads();
    if (warp == group * warps && lane < 8 && item < items && t0 + lane < p.m) {
      float s = 0.f;
      for (int w = 0; w < warps; ++w) s += sh.red[warp + w][lane];
      p.scratch.logits[size_t(t0 + lane) * p.experts + e] = s;
    }
  }
}

// Asks for the router's rows of this CTA's first items and for the bias: they
// come from memory while the CTA sets itself up.
__device__ __forceinline__ void request_router(const MoeParams &p) {
  const int groups = router_groups(p), lines = (p.hidden * (p.router_f32 ? 4 : 2) + 127) / 128;
  const size_t row = size_t(p.hidden) * (p.router_f32 ? 4 : 2);
  const int items = min(groups, p.experts * ((p.m + 7) / 8) - int(blockIdx.x) * groups);
  for (int l = threadIdx.x; l < items * lines; l += NT) {
    const int g = l / lines, e = (int(blockIdx.x) * groups + g) % p.experts;
    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(p.router) + size_t(e) * row +
                                                 min(size_t(l - g * lines) * 128, row - 1)));
  }
  if (p.bias)
    for (int e = threadIdx.x * 32; e < p.experts; e += NT * 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.bias + e));
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
    uint8_t *pieces = p.scratch.x_pieces + size_t(3 * t) * p.hidden;
    auto split = [&](const uint4 &x8, int f) {
      float v[8];
      unpack8(x8, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
#pragma unroll
      for (int c = 0; c < 3; ++c) {
        const uint2 b = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
        *reinterpret_cast<uint2 *>(pieces + size_t(c) * p.hidden + size_t(f) * 8) = b;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = (v[k] - from_e4m3((k < 4 ? b.x : b.y) >> (k % 4 * 8) & 0xffu)) * 16.f;
      }
    };
#pragma unroll
    for (int k = 0; k < HELD; ++k)
      if (int(threadIdx.x) + k * NT < frags) split(held[k], threadIdx.x + k * NT);
    for (int f = threadIdx.x + HELD * NT; f < frags; f += NT) split(ld_ro(x + size_t(f) * 8), f);
    if (threadIdx.x == 0) p.scratch.x_scale[t] = scale;
  }
}

// Order-preserving unsigned key of a score, never 0; a NaN is below every
// number.
__device__ __forceinline__ uint32_t score_key(float v) {
  const uint32_t b = __float_as_uint(v);
  if ((b & 0x7fffffffu) > 0x7f800000u) return 1u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp chooses token t's experts from its logits (in scratch, or in shared
// memory): lane l holds experts l, l + 32, ... (PER of them).
template <int PER>
__device__ __noinline__ void choose(const MoeParams &p, Shared &sh, int t, const float *logits) {
  const int lane = threadIdx.x % 32;
  float score[PER];
  uint32_t key[PER];
  float peak = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    score[i] = e < p.experts ? *static_cast<const volatile float *>(logits + e) : -INFINITY;
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
    const float inverse = 1.f / warp_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] *= inverse;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) score[i] = sigmoid(score[i]);
  }
  // key 0: the expert is chosen already, or does not exist
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < p.experts ? score_key(p.bias ? score[i] + __ldg(p.bias + e) : score[i]) : 0u;
  }
  float total = 0.f, mine = 0.f;
  int mine_e = 0;
#pragma unroll 1
  for (int k = 0; k < p.top_k; ++k) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    // the largest key, then the lowest expert that has it
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    uint32_t at = 0xffffffffu;
    float value = 0.f;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == top) {
        at = uint32_t(i * 32 + lane);
        value = score[i];
      }
    const uint32_t winner = __reduce_min_sync(0xffffffffu, at);
    const float w = __shfl_sync(0xffffffffu, value, int(winner % 32));
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (winner == uint32_t(i * 32 + lane)) key[i] = 0u;
    total += w;
    if (lane == k) {
      mine = w;
      mine_e = int(winner);
    }
  }
  if (lane < p.top_k) {
    const float w = (p.renormalize ? mine / total : mine) * p.routed_scale;
    sh.route_expert[t][lane] = int16_t(mine_e);
    sh.route_weight[t][lane] = w;
    atomicOr(&sh.mask[p.shared + mine_e], 1u << t);
    if (blockIdx.x == 0) {
      if (p.idx) p.idx[t * p.top_k + lane] = mine_e;
      if (p.weights) p.weights[t * p.top_k + lane] = w;
    }
  }
}

// The reached experts in order (the shared ones first), each one's tokens and
// first slot (a slot is a token of an expert), and the tokens' slots.  Every
// CTA computes the same.
template <class Begin>
__device__ __forceinline__ void build_plan(const MoeParams &p, Shared &sh, float *held, const Begin &begin) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int every = p.experts + p.shared;
  // the logits of all tokens into shared memory (256 floats a token), where
  // they fit
  const bool fit = p.experts <= 256;
  if (fit)
    for (int i = threadIdx.x; i < p.m * p.experts; i += NT) held[i] = __ldcg(p.scratch.logits + i);
  if (p.fp8 && threadIdx.x < p.m) sh.x_scale[threadIdx.x] = __ldcg(p.scratch.x_scale + threadIdx.x);
  __syncthreads();
  for (int t = warp; t < p.m; t += WARPS) {
    const float *logits = (fit ? held : p.scratch.logits) + size_t(t) * p.experts;
    if (p.experts <= 64) choose<2>(p, sh, t, logits);
    else if (p.experts <= 256) choose<8>(p, sh, t, logits);
    else choose<MOE_EXPERTS_MAX / 32>(p, sh, t, logits);
  }
  begin();
  __syncthreads();
  int active0 = 0, slots0 = 0;   // before this round of one expert a thread
  for (int e0 = 0; e0 < every; e0 += NT) {
    const int e = e0 + threadIdx.x;
    const uint32_t mask = e < every ? sh.mask[e] : 0u;
    const uint32_t reached = __ballot_sync(0xffffffffu, mask != 0u);
    const int n = __popc(mask);
    int upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) {
      sh.warp_active[warp] = __popc(reached);
      sh.warp_slots[warp] = upto;
    }
    __syncthreads();
    int a = active0 + __popc(reached & ((1u << lane) - 1u)), slot = slots0 + upto - n;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) {
        a += sh.warp_active[w];
        slot += sh.warp_slots[w];
      }
      active0 += sh.warp_active[w];
      slots0 += sh.warp_slots[w];
    }
    if (mask) {
      sh.act_mask[a] = mask;
      sh.act_expert[a] = uint16_t(e < p.shared ? p.experts + e : e - p.shared);
      sh.act_base[a] = uint16_t(slot);
      sh.position[e] = uint16_t(a);
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) sh.active = active0;
  // a token a lane, a route a warp
  for (int k = warp; lane < p.m && k < p.top_k + p.shared; k += WARPS) {
    const int a = sh.position[k < p.top_k ? p.shared + sh.route_expert[lane][k] : k - p.top_k];
    sh.route_slot[lane][k] = int16_t(sh.act_base[a] + __popc(sh.act_mask[a] & ((1u << lane) - 1u)));
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

// Sums of an item's k blocks for this thread's row and CT columns' tokens (P
// pieces each): block sums from the accumulator ring, their pieces added, times
// the block's scale (8-bit weights): `scales` of m floats a block, one a token.
// What lies beyond the expert's tokens is not used.
template <bool FP8, int P, int CT>
__device__ __forceinline__ void sum_blocks(Shared &sh, uint32_t lane_base, Ring &ring, int blocks, const float *scales,
                                           int m, float (&acc)[CT]) {
  constexpr int COLS = (CT * P + 15) / 16 * 16;
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int t = 0; t < CT; ++t) acc[t] = 0.f;
  for (int k = 0; k < blocks; ++k, scales += m) {
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
        acc[t] = fmaf(v, scales[t], acc[t]);
      } else {
#pragma unroll
        for (int c = 0; c < P; ++c) acc[t] += value(d[P * t + c]);
      }
    }
  }
}

// Takes the sums of an item for `count` tokens and gives token t's to
// emit(t, sum); the width of the work follows the count.
template <bool FP8, int P, class Emit>
__device__ __forceinline__ void sum_item(Shared &sh, uint32_t lane_base, Ring &ring, int blocks, const float *scales,
                                         int m, int count, const Emit &emit) {
  auto with = [&](auto ct) {
    constexpr int CT = decltype(ct)::value;
    float acc[CT];
    sum_blocks<FP8, P, CT>(sh, lane_base, ring, blocks, scales, m, acc);
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

// The sum of a row piece's chunks, `step` apart, in their order.
__device__ __forceinline__ float4 add_chunks(const float *src, size_t step, int chunks) {
  float4 v[MOE_CHUNKS];
#pragma unroll
  for (int c = 0; c < MOE_CHUNKS; ++c) v[c] = c < chunks ? ldcg4(src + c * step) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int c = 1; c < MOE_CHUNKS; ++c)
    if (c < chunks) v[0] = add4(v[0], v[c]);
  return v[0];
}

// A complete tile of an expert: its tokens' activations; one warp.
template <bool FP8>
__device__ __forceinline__ void finish_up(const MoeParams &p, const Shape &s, int base, int count, int j) {
  const int lane = threadIdx.x % 32;
  const size_t width = size_t(s.up_tiles) * 128, step = size_t(p.slots) * 2 * width;
#pragma unroll 2
  for (int t = 0; t < count; ++t) {
    const float *src = p.scratch.up + size_t(base + t) * 2 * width + j * 128 + lane * 4;
    const float4 g = add_chunks(src, step, s.up_chunks), u = add_chunks(src + width, step, s.up_chunks);
    store_act<FP8>(p, base + t, j, g, u);
  }
}

// ----------------------------------------------------------------- kernel
// ---------------------------------------------------------------- the output
// y[t] = the sum over t's routes of weight * (the pieces of the route's slot).
__device__ __forceinline__ float route_factor(const MoeParams &p, const Shared &sh, int t, int k) {
  return k < p.top_k ? sh.route_weight[t][k] : 1.f;
}
// Few tokens: eight columns a warp, the routes over four groups of its lanes,
// three routes' pieces asked for at a time.
__device__ __forceinline__ void combine_few(const MoeParams &p, const Shared &sh, const Shape &s, size_t width) {
  const int lane = threadIdx.x % 32, per_token = s.down_tiles * 16, routes = p.top_k + p.shared;
  for (int n = blockIdx.x + threadIdx.x / 32 * gridDim.x; n < p.m * per_token; n += gridDim.x * WARPS) {
    const int t = n / per_token, col = (n - t * per_token) * 8 + lane % 8;
    float y = 0.f;
    for (int k0 = lane / 8; k0 < routes; k0 += 12) {
      float v[3][MOE_CHUNKS];
#pragma unroll
      for (int j = 0; j < 3; ++j)
#pragma unroll
        for (int c = 0; c < MOE_CHUNKS; ++c)
          v[j][c] = k0 + 4 * j < routes && c < s.down_chunks
                        ? __ldcg(p.scratch.down + (size_t(c) * p.slots + sh.route_slot[t][k0 + 4 * j]) * width + col)
                        : 0.f;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
#pragma unroll
        for (int c = 1; c < MOE_CHUNKS; ++c) v[j][0] += v[j][c];
        if (k0 + 4 * j < routes) y = fmaf(route_factor(p, sh, t, k0 + 4 * j), v[j][0], y);
      }
    }
    y += __shfl_xor_sync(0xffffffffu, y, 8);
    y += __shfl_xor_sync(0xffffffffu, y, 16);
    if (lane < 8 && col < p.hidden) p.output[size_t(t) * p.hidden + col] = uint16_t(pack_bf16x2(y, 0.f));
  }
}
// Many: four columns a thread, nine pieces at a time.
__device__ __forceinline__ void combine_many(const MoeParams &p, const Shared &sh, const Shape &s, size_t width) {
  const int lane = threadIdx.x % 32, terms = (p.top_k + p.shared) * s.down_chunks;
  for (int n = blockIdx.x + threadIdx.x / 32 * gridDim.x; n < p.m * s.down_tiles; n += gridDim.x * WARPS) {
    const int t = n / s.down_tiles, col = (n - t * s.down_tiles) * 128 + lane * 4;
    float y[4] = {};
    int k = 0, c = 0;
    for (int j0 = 0; j0 < terms; j0 += 9) {
      float4 v[9];
      float w[9];
#pragma unroll
      for (int j = 0; j < 9; ++j) {
        v[j] = ldcg4(p.scratch.down + (size_t(c) * p.slots + sh.route_slot[t][k]) * width + col);
        w[j] = route_factor(p, sh, t, k);
        if (j0 + j + 1 < terms && ++c == s.down_chunks) {
          c = 0;
          ++k;
        }
      }
#pragma unroll
      for (int j = 0; j < 9; ++j)
        if (j0 + j < terms) {
          y[0] = fmaf(w[j], v[j].x, y[0]);
          y[1] = fmaf(w[j], v[j].y, y[1]);
          y[2] = fmaf(w[j], v[j].z, y[2]);
          y[3] = fmaf(w[j], v[j].w, y[3]);
        }
    }
    if (col < p.hidden)   // hidden is a multiple of 8: four columns are in or out together
#pragma unroll
      for (int i = 0; i < 4; ++i) p.output[size_t(t) * p.hidden + col + i] = uint16_t(pack_bf16x2(y[i], 0.f));
  }
}

template <bool FP8>
__global__ void __launch_bounds__(NT, 1)
k_moe(const MoeParams p, const __grid_constant__ CUtensorMap tm_gate_up, const __grid_constant__ CUtensorMap tm_down,
      const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_x_token,
      const __grid_constant__ CUtensorMap tm_act) {
  constexpr int KB = FP8 ? 128 : 64;                        // values of a 128-byte k block
  constexpr int XP = FP8 ? 3 : 1, HP = FP8 ? 3 : 2;         // pieces of x and of h
  extern __shared__ __align__(1024) unsigned char smem[];
  Shared &sh = *reinterpret_cast<Shared *>(smem);
  float *sums = reinterpret_cast<float *>(smem + SMEM_TABLES);   // two buffers [m][128] from the sums to the joins
  unsigned char *ring = smem + p.ring_at;
  // scales of the items in flight (8-bit weights)
  float *scales = reinterpret_cast<float *>(smem + p.scales_at);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &sh.abort;
  const int stage_bytes = A_BYTES + p.b_bytes;
  unsigned *routed = p.scratch.control, *tickets = routed + 1, *downs_done = routed + 2, *exits = routed + 3;

  request_router(p);
  // a barrier a lane: one after another they would take a microsecond
  if (warp == 0) {
    if (lane < p.stages) {
      tc::mbar_init(&sh.full[lane], 2);
      tc::mbar_init(&sh.empty[lane], 1);
    }
    if (lane < BUFS) {
      tc::mbar_init(&sh.acc_full[lane], 1);
      tc::mbar_init(&sh.acc_empty[lane], 4);
    }
    if (lane < 4) tc::mbar_init(&sh.sum_full[lane], 4);   // one a join warp
    if (lane < 2) tc::mbar_init(&sh.sum_empty[lane], 1);  // one a buffer
    if (lane < ITEMS) {
      tc::mbar_init(&sh.item_full[lane], 1);
      tc::mbar_init(&sh.item_empty[lane], 11);   // scale, activation, MMA, four sum and four join warps
      tc::mbar_init(&sh.scale_full[lane], 1);
    }
    if (lane == 0) {
      tc::mbar_init(&sh.drain, 1);
      sh.abort = 0;
      sh.issued_a = sh.issued_b = 0;
    }
    tc::mbar_init_fence();
  } else if (warp == 1 && lane < 5) {
    tc::tma_prefetch_desc(lane == 0 ? &tm_gate_up : lane == 1 ? &tm_down : lane == 2 ? &tm_x : lane == 3 ? &tm_x_token
                                                                                                       : &tm_act);
  }
  if (warp == 2) tc::tmem_alloc(&sh.tmem, BUFS * BUF_COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const bool stall = g_stall_copies != 0;

  for (int e = threadIdx.x; e < p.experts + p.shared; e += NT)
    sh.mask[e] = e < p.shared ? (p.m == 32 ? 0xffffffffu : (1u << p.m) - 1u) : 0u;

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
  // The first items are the shared experts': their weights are requested before
  // the list of the reached experts is made (not earlier: with the memory busy the
  // choice itself, its instructions included, takes three times as long).
  int ahead = 0;   // blocks of this CTA's first item that are already requested
  build_plan(p, sh, sums, [&]() {
    if (warp != 0 || gave_up || int(blockIdx.x) >= p.shared * ((p.intermediate + 127) / 128) * 2 * p.up_chunks) return;
    const Item it = item_at(shape_of<FP8>(p, p.shared), blockIdx.x);
    ahead = min(it.blocks, p.stages);
    if (!stall && tc::elect_one())
      for (int k = 0; k < ahead; ++k) {
        tc::mbar_arrive_expect_tx(&sh.full[k], A_BYTES);
        tc::tma_load_2d(ring + size_t(k) * stage_bytes, &tm_gate_up, (it.kb0 + k) * KB,
                        ((p.experts + it.a) * 2 + it.half) * p.intermediate + it.tile * 128, &sh.full[k]);
      }
    __syncwarp();
  });

  const int active = sh.active;
  const Shape s = shape_of<FP8>(p, active);
  const size_t up_width = size_t(s.up_tiles) * 128, down_width = size_t(s.down_tiles) * 128;

  // the next item of this CTA, -1 after the last (and once a wait gave up)
  Ring items;
  auto next_item = [&]() {
    const bool ok = tc::wait_or_abort(&sh.item_full[items.at], items.phase, abort);
    if (!__all_sync(0xffffffffu, ok)) return -1;
    const int item = sh.item[items.at];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&sh.item_empty[items.at]);
    items.next(ITEMS);
    return item;
  };

  if (gave_up) {
    // the logits never came: no role begins
  } else if (warp == 0) {
    // ------------------------------------------- items and weight tiles
    Ring at;
    // The first two items go by the CTA's place; a later one is asked for two
    // items ahead, as the answer takes longer than a small item's requests.
    int issued = stall ? 0 : ahead, item = blockIdx.x, next = item + int(gridDim.x);
    bool ok = true;
    const bool leader = tc::elect_one();
    while (true) {
      ok = ok && tc::wait_or_abort(&sh.item_empty[items.at], items.phase ^ 1u, abort);
      ok = __all_sync(0xffffffffu, ok);
      const bool live = ok && item < s.items;
      if (lane == 0) {
        sh.item[items.at] = live ? item : -1;
        if (ok) tc::mbar_arrive(&sh.item_full[items.at]);
      }
      if (!live) break;
      items.next(ITEMS);
      const Item it = item_at(s, item);
      int after = 0;
      if (lane == 0) after = int(atomicAdd(tickets, 1u) + 2 * gridDim.x);
      const int e = sh.act_expert[it.a];
      const int row = it.down ? e * p.hidden + it.tile * 128 : (e * 2 + it.half) * p.intermediate + it.tile * 128;
      const CUtensorMap *map = it.down ? &tm_down : &tm_gate_up;
      for (int k = 0; k < it.blocks && ok; ++k) {
        if (ahead > 0) {
          // already requested; no wait for the stage, which may have been
          // released by now
          --ahead;
        } else {
          ok = tc::wait_or_abort(&sh.empty[at.at], at.phase ^ 1u, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && leader && !stall) {
            tc::mbar_arrive_expect_tx(&sh.full[at.at], A_BYTES);
            tc::tma_load_2d(ring + size_t(at.at) * stage_bytes, map, (it.kb0 + k) * KB, row, &sh.full[at.at]);
            ++issued;
          }
          __syncwarp();
        }
        at.next(p.stages);
      }
      item = __shfl_sync(0xffffffffu, next, 0);
      next = after;
    }
    if (leader) sh.issued_a = issued;
  } else if (warp == 3) {
    // ------------------------------------------------- activation tiles
    Ring at;
    int issued = 0, ready = 0;
    bool ok = true;
    fence_proxy_async_global();
    const int x_rows = (p.m * XP + 7) / 8 * 8;
    while (ok) {
      const int item = next_item();
      if (item < 0) break;
      const Item it = item_at(s, item);
      const uint32_t mask = sh.act_mask[it.a];
      const int count = __popc(mask);
      // a block's copies, one a lane: all tokens in one; or the expert's tokens
      // only, a copy each (their rows' swizzle goes by their place in shared
      // memory, as the tensor core reads them); or the expert's activations
      const CUtensorMap *map;
      int copies, bytes, row, place;
      if (it.down) {
        if (ready <= it.a) {
          ready = poll_experts(p.scratch.up_done, unsigned(s.up_tiles), ready, it.a + 1, active, abort);
          ok = ready > it.a;
          __syncwarp();
          fence_proxy_async_global();
        }
        map = &tm_act;
        copies = (count * HP + 7) / 8;
        bytes = copies * 1024;
        row = sh.act_base[it.a] * HP + lane * 8;
        place = lane * 1024;
      } else if (count == p.m) {
        map = &tm_x;
        copies = 1;
        bytes = x_rows * 128;
        row = place = 0;
      } else {
        map = &tm_x_token;
        copies = count;
        bytes = count * XP * 128;
        row = lane < count ? int(__fns(mask, 0, lane + 1)) * XP : 0;
        place = lane * XP * 128;
      }
      for (int k = 0; k < it.blocks && ok; ++k) {
        ok = tc::wait_or_abort(&sh.empty[at.at], at.phase ^ 1u, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && !stall) {
          if (lane == 0) tc::mbar_arrive_expect_tx(&sh.full[at.at], uint32_t(bytes));
          __syncwarp();
          if (lane < copies)
            tc::tma_load_2d(ring + size_t(at.at) * stage_bytes + A_BYTES + place, map, (it.kb0 + k) * KB, row,
                            &sh.full[at.at]);
          ++issued;
        }
        __syncwarp();
        at.next(p.stages);
      }
    }
    if (lane == 0) sh.issued_b = issued;
  } else if (warp == 2) {
    // ----------------------------------------------------------- scales
    // Read here, some items ahead: a read takes longer than several blocks.
    int ready = 0;
    while (true) {
      const int slot = items.at, item = next_item();
      if (item < 0) break;
      if (!FP8) continue;
      const Item it = item_at(s, item);
      const int count = __popc(sh.act_mask[it.a]), e = sh.act_expert[it.a];
      const float *sw = it.down ? p.down_scales + (size_t(e) * s.down_tiles + it.tile) * s.down_k
                                : p.gate_up_scales + ((size_t(e) * 2 + it.half) * s.up_tiles + it.tile) * s.up_k;
      const float *act = p.scratch.act_scale + size_t(it.kb0) * p.slots + sh.act_base[it.a];
      if (it.down && ready <= it.a) {
        ready = poll_experts(p.scratch.up_done, unsigned(s.up_tiles), ready, it.a + 1, active, abort);
        __syncwarp();
      }
      float *dst = scales + size_t(slot) * p.scale_blocks * p.m;
      // blocks in lanes; all reads of a token are under way together
      if (lane < it.blocks) {
        const float w = __ldg(sw + it.kb0 + lane);
#pragma unroll 4
        for (int t = 0; t < count; ++t) dst[lane * p.m + t] = it.down ? w * __ldcg(act + size_t(lane) * p.slots + t) : w;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.scale_full[slot]);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA
    Ring at, acc;
    bool ok = true;
    const bool leader = tc::elect_one();
    const uint64_t a0 = tc::desc_sw128(ring), b0 = tc::desc_sw128(ring + A_BYTES);
    while (ok) {
      const int item = next_item();
      if (item < 0) break;
      const Item it = item_at(s, item);
      const int cols = (__popc(sh.act_mask[it.a]) * (it.down ? HP : XP) + 15) / 16 * 16;
      const uint32_t idesc = FP8 ? tc::idesc_e4m3_f32(128, cols) : tc::idesc_bf16_f32(128, cols);
      for (int k = 0; k < it.blocks && ok; ++k) {
        ok = tc::wait_or_abort(&sh.full[at.at], at.phase, abort) &&
             tc::wait_or_abort(&sh.acc_empty[acc.at], acc.phase ^ 1u, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
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
    }
    // no MMA is in flight when the tensor memory goes
    if (leader) tc::mma_commit(&sh.drain);
    __syncwarp();
    tc::mbar_wait_bounded(&sh.drain, 0u, tc::SUB_WAIT_LIMIT);
  } else if (warp >= SUM_WARP0 && warp < JOIN_WARP0) {
    // ------------------------------------------------------------- sums
    const int i = threadIdx.x - SUM_WARP0 * 32;   // row of the tile
    const uint32_t lane_base = tmem + (uint32_t((warp % 4) * 32) << 16);
    Ring acc, out, join;
    while (true) {
      const Ring from = items;
      // the item's slot is given back after its scales are read
      const bool ok = tc::wait_or_abort(&sh.item_full[from.at], from.phase, abort);
      if (!__all_sync(0xffffffffu, ok)) break;
      const int item = sh.item[from.at];
      if (item < 0) break;
      const Item it = item_at(s, item);
      uint32_t rest = sh.act_mask[it.a];
      const int count = __popc(rest);
      float *dst = sums + size_t(out.at) * p.m * 128 + i;
      const float *scale = scales + size_t(from.at) * p.scale_blocks * p.m;
      if (FP8) {
        tc::wait_or_abort(&sh.scale_full[from.at], from.phase, abort);
        __syncwarp();
      }
      // emit(t, sum): into the buffer, once the joins have emptied it
      auto emit = [&](int t, float v) {
        if (t == 0) {
          tc::wait_or_abort(&sh.sum_empty[out.at], out.phase ^ 1u, abort);
          __syncwarp();
        }
        if (FP8 && !it.down) {
          v *= sh.x_scale[__ffs(rest) - 1];
          rest &= rest - 1u;
        }
        dst[t * 128] = v;
      };
      if (it.down) sum_item<FP8, HP>(sh, lane_base, acc, it.blocks, scale, p.m, count, emit);
      else sum_item<FP8, XP>(sh, lane_base, acc, it.blocks, scale, p.m, count, emit);
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&sh.sum_full[join.at]);
        tc::mbar_arrive(&sh.item_empty[from.at]);
      }
      out.next(2);
      join.next(4);
      items.next(ITEMS);
    }
  } else if (warp >= JOIN_WARP0) {
    // ------------------------------------------------------------ joins
    // Each warp takes every fourth item: a join is a chain of accesses that
    // other SMs must see, each of them microseconds long while the memory is
    // busy, so four are under way at a time.
    const int jw = warp - JOIN_WARP0;
    for (int n = 0;; ++n) {
      const int item = next_item();
      if (item < 0) break;
      if (n % 4 != jw) continue;
      const Item it = item_at(s, item);
      const int base = sh.act_base[it.a], count = __popc(sh.act_mask[it.a]);
      tc::wait_or_abort(&sh.sum_full[jw], uint32_t(n / 4 & 1), abort);
      __syncwarp();
      const float *src = sums + size_t(n % 2) * p.m * 128;
      float *dst;
      size_t row;
      if (!it.down) {
        row = 2 * up_width;
        dst = p.scratch.up + (size_t(it.chunk) * p.slots + base) * row + it.half * up_width + it.tile * 128;
      } else {
        row = down_width;
        dst = p.scratch.down + (size_t(it.chunk) * p.slots + base) * row + it.tile * 128;
      }
#pragma unroll 4
      for (int t = 0; t < count; ++t)
        __stcg(reinterpret_cast<float4 *>(dst + size_t(t) * row) + lane,
               reinterpret_cast<const float4 *>(src + t * 128)[lane]);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.sum_empty[n % 2]);
      if (it.down) continue;
      // a tile of `up` is complete with its last chunk
      __threadfence();
      __syncwarp();
      unsigned there = 0, *counter = p.scratch.up_counters + it.a * s.up_tiles + it.tile;
      if (lane == 0) there = atomicAdd(counter, 1u) + 1;
      if (__shfl_sync(0xffffffffu, there, 0) == unsigned(2 * s.up_chunks)) {
        __threadfence();
        finish_up<FP8>(p, s, base, count, it.tile);
        fence_proxy_async_global();
        __threadfence();
        __syncwarp();
        if (lane == 0) {
          *counter = 0;
          atomicAdd(p.scratch.up_done + it.a, 1u);
        }
      }
    }
    __threadfence();
  }
  // ---- the output, once every CTA's sums are there
  __syncthreads();
  if (threadIdx.x == 0) {
    atomicAdd(downs_done, 1u);
    poll(downs_done, gridDim.x, abort);
  }
  __syncthreads();
  __threadfence();
  // few: while a pass of the wide form would leave most warps idle
  if (p.m * s.down_tiles * 4 <= int(gridDim.x) * WARPS) combine_few(p, sh, s, down_width);
  else combine_many(p, sh, s, down_width);
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
      *tickets = 0;
      *downs_done = 0;
      *exits = 0;
      for (int a = 0; a < sh.active; ++a) p.scratch.up_done[a] = 0;
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

void moe_form(MoeParams &p, int sms) {
  const bool fp8 = p.fp8 != 0;
  const int kb = fp8 ? 128 : 64, pieces = fp8 ? 3 : 2;   // of x or h, at most
  p.b_bytes = (p.m * pieces + 7) / 8 * 1024;
  // Chunks of a tile's k blocks: of about ten blocks (`up`) or six (`down`,
  // whose last items decide when the kernel ends), or fewer blocks where the
  // tiles of the experts that are reached at least do not give every CTA an
  // item.
  auto chunks = [&](int k, int blocks, int tiles) {
    const int by_size = (k + blocks - 1) / blocks, by_ctas = std::min(sms / tiles, k / 2);
    return std::max(1, std::min(MOE_CHUNKS, std::max(by_size, by_ctas)));
  };
  const int up_k = (p.hidden + kb - 1) / kb, down_k = (p.intermediate + kb - 1) / kb;
  const int least = p.top_k + p.shared;
  p.up_chunks = chunks(up_k, 10, least * qblocks(p.intermediate) * 2);
  p.down_chunks = chunks(down_k, 6, least * qblocks(p.hidden));
  p.scale_blocks = std::max((up_k + p.up_chunks - 1) / p.up_chunks, (down_k + p.down_chunks - 1) / p.down_chunks);
  const int scale_bytes = fp8 ? ITEMS * p.scale_blocks * p.m * 4 + SCALE_SLACK : 0;
  p.ring_at = SMEM_TABLES + p.m * 1024;
  p.stages = std::min(STAGES_MAX, (SMEM_BYTES - p.ring_at - SMEM_SLACK - scale_bytes) / (A_BYTES + p.b_bytes));
  p.scales_at = p.ring_at + p.stages * (A_BYTES + p.b_bytes) + SMEM_SLACK;
}

cudaError_t launch_moe(const MoeParams &args, int sms, cudaStream_t stream) {
  MoeParams p = args;
  moe_form(p, sms);
  const bool fp8 = p.fp8 != 0;
  const int every = p.experts + p.shared, elem = fp8 ? 1 : 2, kb = fp8 ? 128 : 64;
  const int xp = fp8 ? 3 : 1, hp = fp8 ? 3 : 2;
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
