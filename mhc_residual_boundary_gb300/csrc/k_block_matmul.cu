// k_block_matmul.cu -- product of 8-bit matrices with a scale for each block
// of 128:
//   out[m][n] = sum_kb sa[m][kb] sw[n/128][kb] * sum_{k in kb} a[m][k] w[n][k]
//
// The inner sums (128 E4M3 products) run on the tensor cores into tensor
// memory; the scaled outer sum runs in FP32 registers.  A row of `a` is a TMEM
// lane, so its scale is one register of one thread, and the columns of an
// epilogue warp lie in one block of `w`, so the outer sum is one packed FP32
// fused multiply-add for every two elements and block.
//
// Two kernels share this.  Few rows, where the read of `w` bounds the call: a
// tile of 128 rows x BN columns a cluster, its k blocks cut over the cluster's
// CTAs, whose sums meet through distributed shared memory (no scratch, and the
// order of addition is that of the ranks).  Many rows, where the tensor cores
// do: a pair of CTAs works on a tile of 256 x 256 with cta_group::2 MMAs, each
// CTA loading half of both operands, persistent over the tiles.
//
// Roles (12 warps): 0 operand copies, 1 MMA, 2-3 scales (read some blocks ahead
// into shared memory: a read takes longer than a block's products), 4-11
// epilogue, two warps for each TMEM sub-partition.  Operands arrive in a ring of
// stages of one k block (128 bytes a row, 128-byte swizzled); the accumulator
// is a ring of buffers, so the tensor cores work on one block while the
// epilogue warps add the one before.
#include <algorithm>

#include "sublayer.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int BM = 128;                  // rows of a CTA
constexpr int NT = 384;
constexpr int SCALE_WARP0 = 2, EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int STAGES_MAX = 12;
constexpr int CHUNK = 8, CHUNKS = 4;     // k blocks of a chunk of scales, chunks in flight
constexpr int SMEM_CTRL = 1024;
constexpr int SMEM_SCALES = CHUNKS * CHUNK * (BM + 2) * 4 + 1024;   // and the ring's alignment
constexpr int SMEM_BYTES = 227 * 1024;
constexpr int RING_BYTES = (SMEM_BYTES - SMEM_CTRL - SMEM_SCALES) / 1024 * 1024;

__device__ int g_stall_copies;   // test hook: the producer issues no copies

struct Control {
  uint64_t full[STAGES_MAX], empty[STAGES_MAX], peer_full[STAGES_MAX], acc_full[4], acc_empty[4];
  uint64_t scale_full[CHUNKS], scale_empty[CHUNKS], drain;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Control) <= SMEM_CTRL, "control block");

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// An arrival on another CTA's barrier.  What it tells of lies in tensor memory
// (read, ordered by the tcgen05 fences) or came by asynchronous copies (ordered
// by their own completion), not in memory that this thread wrote, so it has no
// release at cluster scope, nor its wait an acquire: each costs hundreds of
// clocks, several times a block (matmul of 4096 x 4096 x 6144: 242 us with
// them).
__device__ __forceinline__ void arrive_peer(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------- cta_group::2 instructions
__device__ __forceinline__ void tmem_alloc2(uint32_t *slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_addr(slot)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma2_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// One arrival on the barrier at this place in both CTAs of the pair.
__device__ __forceinline__ void mma2_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_addr(bar)),
      "h"((unsigned short)3)
      : "memory");
}

// A place in a ring of barriers and the phase of its current round; a producer
// waits for a slot's release with the other parity, which returns at once in
// the first round.
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

// Scales of the k blocks [kb0, kb1): [block][row] of this CTA's rows, and the
// weight's [block][2]; one of the two scale warps writes 64 rows.
struct Scales {
  float *a;   // [CHUNKS][CHUNK][rows]
  float *w;   // [CHUNKS][CHUNK][2]
  int rows;   // of the tile, at most BM
};

__device__ __forceinline__ void load_scales(const MatmulParams &p, Control &c, const Scales &sc, Ring &ring, int m0,
                                            int n_block, int kb0, int kb1, int warp, int lane) {
  volatile int *abort = &c.abort;
  for (int kb = kb0; kb < kb1; kb += CHUNK) {
    tc::wait_or_abort(&c.scale_empty[ring.at], ring.phase ^ 1u, abort);
    __syncwarp();
    float *a = sc.a + ring.at * CHUNK * sc.rows, *w = sc.w + ring.at * CHUNK * 2;
    float v[2][CHUNK];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = m0 + warp * 64 + h * 32 + lane;
      const float *src = p.scales + size_t(row < p.m ? row : 0) * p.scales_stride + kb;
#pragma unroll
      for (int k = 0; k < CHUNK; ++k) v[h][k] = row < p.m && kb + k < kb1 ? __ldg(src + k) : 0.f;
    }
    // lane 8 b + k: block n_block + b
    float sw = 0.f;
    if (warp == 0 && lane < 2 * CHUNK && kb + lane % CHUNK < kb1)
      sw = __ldg(p.weight_scales + size_t(min(n_block + lane / CHUNK, p.n_blocks - 1)) * p.k_blocks + kb + lane % CHUNK);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < CHUNK; ++k) {
        const int row = warp * 64 + h * 32 + lane;
        if (row < sc.rows) a[k * sc.rows + row] = v[h][k];
      }
    if (warp == 0 && lane < 2 * CHUNK) w[lane % CHUNK * 2 + lane / CHUNK] = sw;
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&c.scale_full[ring.at]);
    ring.next(CHUNKS);
  }
}

// Adds the scaled block sums of `blocks` k blocks to acc: NC columns of this
// thread's row, from TMEM columns `col` of each accumulator buffer of
// buf_cols; `released` tells the MMA warp that a buffer is read.
template <int NC, class Release>
__device__ __forceinline__ void add_blocks(Control &c, const Scales &sc, Ring &acc_ring, Ring &scale_ring, int bufs,
                                           int buf_cols, uint32_t taddr, int row, int w_block, int blocks, bool rows_live,
                                           int lane, const Release &release, uint64_t (&acc)[NC / 2]) {
  volatile int *abort = &c.abort;
  for (int k = 0; k < blocks; ++k) {
    const int in_chunk = k % CHUNK;
    if (in_chunk == 0) {
      tc::wait_or_abort_inline(&c.scale_full[scale_ring.at], scale_ring.phase, abort);
      __syncwarp();
    }
    const int at = scale_ring.at * CHUNK + in_chunk;
    const float scale = sc.a[at * sc.rows + row] * sc.w[at * 2 + w_block];
    if (in_chunk == CHUNK - 1 || k == blocks - 1) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.scale_empty[scale_ring.at]);
      scale_ring.next(CHUNKS);
    }
    tc::wait_or_abort_inline(&c.acc_full[acc_ring.at], acc_ring.phase, abort);
    __syncwarp();
    tc::fence_after_sync();
    if (rows_live) {
      const uint64_t s2 = tc::pair(scale, scale);
      const uint32_t src = taddr + uint32_t(acc_ring.at * buf_cols);
      constexpr int STEP = NC > 64 ? 32 : NC;   // what the registers beside acc hold
#pragma unroll
      for (int h = 0; h < NC; h += STEP) {
        uint32_t d[STEP / 32][32];
#pragma unroll
        for (int q = 0; q < STEP / 32; ++q) tc::tmem_ld32_async(src + uint32_t(h + q * 32), d[q]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < STEP / 32; ++q) tc::tmem_hold(d[q]);
        if (h + STEP == NC) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) release(acc_ring.at);
        }
#pragma unroll
        for (int q = 0; q < STEP / 32; ++q)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            tc::fma_pair(acc[h / 2 + q * 16 + i], d[q][2 * i], d[q][2 * i + 1], s2);
      }
    } else if (lane == 0) {
      release(acc_ring.at);
    }
    acc_ring.next(bufs);
  }
}

// Eight neighbouring columns of a row to the output.
__device__ __forceinline__ void store8(const MatmulParams &p, int row, int col, const float (&v)[8]) {
  const size_t at = size_t(row) * p.output_stride + col;
  const bool whole = p.vector_out && col + 8 <= p.n;
  if (p.output_f32) {
    float *out = static_cast<float *>(p.output) + at;
    if (whole) {
      reinterpret_cast<float4 *>(out)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4 *>(out)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < p.n) out[k] = v[k];
    }
  } else {
    uint16_t *out = static_cast<uint16_t *>(p.output) + at;
    const uint4 w = pack8(v);
    if (whole) {
      st_vec(out, w);
    } else {
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (col + k < p.n) out[k] = uint16_t(u[k / 2] >> (k % 2 * 16));
    }
  }
}

template <int NC>
__device__ __forceinline__ void store_row(const MatmulParams &p, int row, int col, const uint64_t (&acc)[NC / 2]) {
#pragma unroll
  for (int i = 0; i < NC / 2; i += 4) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = tc::pair_lo(acc[i + k]);
      v[2 * k + 1] = tc::pair_hi(acc[i + k]);
    }
    if (col + 2 * i < p.n) store8(p, row, col + 2 * i, v);
  }
}

__device__ __forceinline__ void init_control(Control &c, int stages, int bufs, uint32_t acc_empty_count) {
  for (int i = 0; i < stages; ++i) {
    tc::mbar_init(&c.full[i], 1);
    tc::mbar_init(&c.empty[i], 1);
    tc::mbar_init(&c.peer_full[i], 1);
  }
  for (int i = 0; i < bufs; ++i) {
    tc::mbar_init(&c.acc_full[i], 1);
    tc::mbar_init(&c.acc_empty[i], acc_empty_count);
  }
  for (int i = 0; i < CHUNKS; ++i) {
    tc::mbar_init(&c.scale_full[i], 2);
    tc::mbar_init(&c.scale_empty[i], EPI_WARPS);
  }
  tc::mbar_init(&c.drain, 1);
  tc::mbar_init_fence();
  c.abort = 0;
}

// ------------------------------------------------------------ split kernel
// Cluster `tile` of p.splits CTAs: BM rows by BN columns, CTA r the k blocks
// [k_blocks r / splits, k_blocks (r + 1) / splits).  The roles hand each other
// groups of G blocks, each block with an accumulator of its own: a wait between
// two roles takes some hundred clocks, as long as the few rows' work for a block
// (one row of 6144 x 5120, a wait for each block: 11.0 us).
template <int BN, int G>
__global__ void __launch_bounds__(NT, 1)
k_matmul_split(const MatmulParams p, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w) {
  constexpr int BUFS = 2;                // accumulators of two groups
  constexpr int NC = BN / 2;             // columns of an epilogue warp group
  static_assert(BUFS * G * BN == 512 && CHUNK % G == 0, "all of the tensor memory; a group lies in a chunk of scales");
  extern __shared__ __align__(1024) unsigned char smem[];
  Control &c = *reinterpret_cast<Control *>(smem);
  unsigned char *ring = smem + SMEM_CTRL;
  const Scales sc = {reinterpret_cast<float *>(ring + RING_BYTES),
                     reinterpret_cast<float *>(ring + RING_BYTES) + CHUNKS * CHUNK * BM, BM};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  const int a_bytes = p.a_rows * 128, block_bytes = a_bytes + BN * 128;

  if (threadIdx.x == 0) {
    init_control(c, p.stages, BUFS, EPI_WARPS);
    tc::tma_prefetch_desc(&tm_a);
    tc::tma_prefetch_desc(&tm_w);
  }
  if (warp == SCALE_WARP0) tc::tmem_alloc(&c.tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int rank = p.splits > 1 ? int(cluster_rank()) : 0, tile = int(blockIdx.x) / p.splits;
  const int m0 = tile % p.m_tiles * BM, n0 = tile / p.m_tiles * BN;
  const int kb0 = p.k_blocks * rank / p.splits, kb1 = p.k_blocks * (rank + 1) / p.splits;
  const int rows = min(BM, p.m - m0);    // of the tile

  // The copies and the MMAs are issued by one thread that runs their whole
  // loop: under a predicate carried from outside a loop an MMA takes some 25
  // clocks more to issue (its operands leave the uniform registers).
  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (tc::elect_one()) {
      Ring at;
      int issued = 0;
      if (!g_stall_copies)
        for (int kb = kb0; kb < kb1; kb += G) {
          if (!tc::wait_or_abort(&c.empty[at.at], at.phase ^ 1u, abort)) break;
          const int blocks = min(G, kb1 - kb);
          unsigned char *dst = ring + size_t(at.at) * G * block_bytes;
          tc::mbar_arrive_expect_tx(&c.full[at.at], uint32_t(blocks * block_bytes));
          for (int q = 0; q < blocks; ++q, dst += block_bytes) {
            tc::tma_load_2d(dst + a_bytes, &tm_w, (kb + q) * 128, n0, &c.full[at.at]);
            tc::tma_load_2d(dst, &tm_a, (kb + q) * 128, m0, &c.full[at.at]);
          }
          at.next(p.stages);
          ++issued;
        }
      // copies in flight land before the CTA's shared memory goes
      if (*abort)
        for (int i = max(0, issued - p.stages); i < issued; ++i)
          tc::mbar_wait_bounded(&c.full[i % p.stages], uint32_t((i / p.stages) & 1), tc::SUB_WAIT_LIMIT);
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    const uint32_t idesc = tc::idesc_e4m3_f32(BM, BN);
    const uint64_t a0 = tc::desc_sw128(ring), b0 = tc::desc_sw128(ring + a_bytes);
    if (tc::elect_one()) {
      Ring at, acc;
      bool full = false, released = false;   // the next group's barriers, tested beside this one's products
      for (int kb = kb0; kb < kb1; kb += G) {
        if (!tc::wait_or_abort(full, &c.full[at.at], at.phase, abort) ||
            !tc::wait_or_abort(released, &c.acc_empty[acc.at], acc.phase ^ 1u, abort))
          break;
        const Ring at0 = at, acc0 = acc;
        at.next(p.stages);
        acc.next(BUFS);
        full = tc::mbar_try_wait(&c.full[at.at], at.phase);
        released = tc::mbar_try_wait(&c.acc_empty[acc.at], acc.phase ^ 1u);
        tc::fence_after_sync();
        const int blocks = min(G, kb1 - kb);
        for (int q = 0; q < blocks; ++q) {
          const uint64_t step = uint64_t((at0.at * G + q) * (block_bytes >> 4));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_e4m3(tmem + uint32_t((acc0.at * G + q) * BN), a0 + step + 2 * ks, b0 + step + 2 * ks, idesc,
                         ks != 0);
        }
        tc::mma_commit(&c.empty[at0.at]);
        tc::mma_commit(&c.acc_full[acc0.at]);
      }
      // no MMA is in flight when the tensor memory goes
      tc::mma_commit(&c.drain);
      tc::mbar_wait_bounded(&c.drain, 0u, tc::SUB_WAIT_LIMIT);
    }
  } else if (warp < EPI_WARP0) {
    Ring scales;
    load_scales(p, c, sc, scales, m0, n0 / QBLOCK, kb0, kb1, warp - SCALE_WARP0, lane);
  } else {
    // ---------------------------------------------------------- epilogue
    // After a wait gave up these warps go through the rest of their loops on
    // whatever is there (the waits return at once).
    const int sub = warp % 4, group = (warp - EPI_WARP0) / 4, r = sub * 32 + lane;
    const int col = group * NC;
    const bool rows_live = sub * 32 < rows;
    const uint32_t lane_base = tmem + (uint32_t(sub * 32) << 16) + uint32_t(col);
    Ring buf, chunk;
    uint64_t acc[NC / 2];
#pragma unroll
    for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
    for (int k = 0; k < kb1 - kb0; k += G) {
      const int blocks = min(G, kb1 - kb0 - k);
      if (k % CHUNK == 0) {
        tc::wait_or_abort_inline(&c.scale_full[chunk.at], chunk.phase, abort);
        __syncwarp();
      }
      const int s0 = chunk.at * CHUNK + k % CHUNK;
      float scale[G];
#pragma unroll
      for (int q = 0; q < G; ++q) scale[q] = sc.a[(s0 + q) * BM + r] * sc.w[(s0 + q) * 2];
      if (k % CHUNK + G == CHUNK || k + G >= kb1 - kb0) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&c.scale_empty[chunk.at]);
        chunk.next(CHUNKS);
      }
      tc::wait_or_abort_inline(&c.acc_full[buf.at], buf.phase, abort);
      __syncwarp();
      tc::fence_after_sync();
      if (rows_live) {
#pragma unroll
        for (int q = 0; q < G; ++q)
          if (q < blocks) {
            uint32_t d[NC / 32][32];
#pragma unroll
            for (int h = 0; h < NC / 32; ++h)
              tc::tmem_ld32_async(lane_base + uint32_t((buf.at * G + q) * BN + h * 32), d[h]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < NC / 32; ++h) tc::tmem_hold(d[h]);
            const uint64_t s2 = tc::pair(scale[q], scale[q]);
#pragma unroll
            for (int h = 0; h < NC / 32; ++h)
#pragma unroll
              for (int i = 0; i < 16; ++i) tc::fma_pair(acc[h * 16 + i], d[h][2 * i], d[h][2 * i + 1], s2);
          }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.acc_empty[buf.at]);
      buf.next(BUFS);
    }
    if (p.splits == 1) {
      if (r < rows) store_row<NC>(p, m0 + r, n0 + col, acc);
    } else if (r < rows) {
      // every MMA has completed, so the stages are free: [column][row]
      float *part = reinterpret_cast<float *>(ring) + size_t(col) * p.a_rows + r;
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) {
        part[size_t(2 * i) * p.a_rows] = tc::pair_lo(acc[i]);
        part[size_t(2 * i + 1) * p.a_rows] = tc::pair_hi(acc[i]);
      }
    }
  }
  if (p.splits > 1) {
    __syncwarp();
    cluster_sync();
    // this CTA's share of the tile: items of a row's eight columns
    const int items = rows * (BN / 8);
    const int i1 = items * (rank + 1) / p.splits;
    for (int i = items * rank / p.splits + threadIdx.x; i < i1; i += NT) {
      const int cg = i / rows, row = i - cg * rows;
      const float *at = reinterpret_cast<const float *>(ring) + size_t(cg) * 8 * p.a_rows + row;
      float v[8] = {};
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s) {
        const uint32_t src = peer_addr(at, uint32_t(s));
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += ld_peer(src + uint32_t(k * p.a_rows * 4));
      }
      if (n0 + cg * 8 < p.n) store8(p, m0 + row, n0 + cg * 8, v);
    }
    cluster_sync();   // no CTA leaves while another reads its sums
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == SCALE_WARP0) tc::tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && c.abort) atomicOr(p.err, 2u);
}

// ------------------------------------------------------------- pair kernel
// CTA pair: tiles of 256 rows x 256 columns; CTA r has rows 128 r .. and loads
// rows 128 r .. of the tile's part of w.  The MMAs, issued by rank 0, read both
// CTAs' stages and write both tensor memories.  Rank 1 tells rank 0 when its
// part of a stage has arrived; a stage's or buffer's release reaches both.
constexpr int PAIR_N = 256;
constexpr int PAIR_STAGE = 2 * BM * 128;
constexpr int PAIR_STAGES = RING_BYTES / PAIR_STAGE;

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NT, 1)
k_matmul_pair(const MatmulParams p, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w) {
  constexpr int BUFS = 2;
  constexpr int NC = PAIR_N / 2;
  extern __shared__ __align__(1024) unsigned char smem[];
  Control &c = *reinterpret_cast<Control *>(smem);
  unsigned char *ring = smem + SMEM_CTRL;
  const Scales sc = {reinterpret_cast<float *>(ring + RING_BYTES),
                     reinterpret_cast<float *>(ring + RING_BYTES) + CHUNKS * CHUNK * BM, BM};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  const uint32_t rank = cluster_rank();

  if (threadIdx.x == 0) {
    init_control(c, PAIR_STAGES, BUFS, 2 * EPI_WARPS);
    tc::tma_prefetch_desc(&tm_a);
    tc::tma_prefetch_desc(&tm_w);
  }
  if (warp == SCALE_WARP0) tmem_alloc2(&c.tmem, BUFS * PAIR_N);
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  pdl_launch_dependents();
  const int tiles = p.m_tiles * p.n_tiles, pairs = int(gridDim.x) / 2, first = int(blockIdx.x) / 2;

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      // -------------------------------------------------------- producer
      if (tc::elect_one()) {
        Ring at;
        int issued = 0;
        bool ok = !g_stall_copies;
        for (int tile = first; tile < tiles && ok; tile += pairs) {
          const int m0 = tile % p.m_tiles * 256 + int(rank) * BM, n0 = tile / p.m_tiles * PAIR_N + int(rank) * BM;
          for (int kb = 0; kb < p.k_blocks; ++kb) {
            ok = tc::wait_or_abort(&c.empty[at.at], at.phase ^ 1u, abort);
            if (!ok) break;
            unsigned char *dst = ring + size_t(at.at) * PAIR_STAGE;
            tc::mbar_arrive_expect_tx(&c.full[at.at], PAIR_STAGE);
            tc::tma_load_2d(dst, &tm_a, kb * 128, m0, &c.full[at.at]);
            tc::tma_load_2d(dst + BM * 128, &tm_w, kb * 128, n0, &c.full[at.at]);
            at.next(PAIR_STAGES);
            ++issued;
          }
        }
        if (*abort)
          for (int i = max(0, issued - PAIR_STAGES); i < issued; ++i)
            tc::mbar_wait_bounded(&c.full[i % PAIR_STAGES], uint32_t((i / PAIR_STAGES) & 1), tc::SUB_WAIT_LIMIT);
      }
    } else if (warp == 1) {
      // ------------------------------------------- MMA issuer / its peer
      const uint32_t idesc = tc::idesc_e4m3_f32(256, PAIR_N);
      const uint64_t a0 = tc::desc_sw128(ring), b0 = tc::desc_sw128(ring + BM * 128);
      const int blocks = (tiles - first + pairs - 1) / pairs * p.k_blocks;
      if (tc::elect_one()) {
        Ring at, acc;
        if (rank == 0) {
          bool full = false, peer = false, released = false;   // the next block's, tested beside this one's products
          for (int n = 0; n < blocks; ++n) {
            if (!tc::wait_or_abort(full, &c.full[at.at], at.phase, abort) ||
                !tc::wait_or_abort(peer, &c.peer_full[at.at], at.phase, abort) ||
                !tc::wait_or_abort(released, &c.acc_empty[acc.at], acc.phase ^ 1u, abort))
              break;
            const Ring at0 = at, acc0 = acc;
            at.next(PAIR_STAGES);
            acc.next(BUFS);
            full = tc::mbar_test_wait(&c.full[at.at], at.phase);
            peer = tc::mbar_test_wait(&c.peer_full[at.at], at.phase);
            released = tc::mbar_test_wait(&c.acc_empty[acc.at], acc.phase ^ 1u);
            tc::fence_after_sync();
            const uint64_t step = uint64_t(at0.at * (PAIR_STAGE >> 4));
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma2_e4m3(tmem + uint32_t(acc0.at * PAIR_N), a0 + step + 2 * ks, b0 + step + 2 * ks, idesc, ks != 0);
            mma2_commit(&c.empty[at0.at]);
            mma2_commit(&c.acc_full[acc0.at]);
          }
          // no MMA is in flight when the tensor memory goes
          mma2_commit(&c.drain);
          tc::mbar_wait_bounded(&c.drain, 0u, tc::SUB_WAIT_LIMIT);
        } else {
          const uint32_t told = peer_addr(&c.peer_full[0], 0);
          for (int n = 0; n < blocks; ++n) {
            if (!tc::wait_or_abort(&c.full[at.at], at.phase, abort)) break;
            arrive_peer(told + uint32_t(at.at) * 8);
            at.next(PAIR_STAGES);
          }
        }
      }
    } else {
      Ring scales;
      for (int tile = first; tile < tiles; tile += pairs)
        load_scales(p, c, sc, scales, tile % p.m_tiles * 256 + int(rank) * BM, tile / p.m_tiles * 2, 0, p.k_blocks,
                    warp - SCALE_WARP0, lane);
    }
  } else {
    // ---------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int sub = warp % 4, group = (warp - EPI_WARP0) / 4, r = sub * 32 + lane;
    const int col = group * NC;
    const uint32_t release0 = peer_addr(&c.acc_empty[0], 0);
    Ring acc_ring, scale_ring;
    for (int tile = first; tile < tiles; tile += pairs) {
      const int m0 = tile % p.m_tiles * 256 + int(rank) * BM, n0 = tile / p.m_tiles * PAIR_N;
      uint64_t acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
      add_blocks<NC>(c, sc, acc_ring, scale_ring, BUFS, PAIR_N, tmem + (uint32_t(sub * 32) << 16) + uint32_t(col), r,
                     group, p.k_blocks, m0 + sub * 32 < p.m, lane,
                     [&](int b) { arrive_peer(release0 + uint32_t(b) * 8); }, acc);
      if (m0 + r < p.m) store_row<NC>(p, m0 + r, n0 + col, acc);
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  cluster_sync();   // neither CTA leaves while the other's MMAs or arrivals reach it
  tc::fence_after_sync();
  if (warp == SCALE_WARP0) tmem_dealloc2(tmem, BUFS * PAIR_N);
  if (threadIdx.x == 0 && c.abort) atomicOr(p.err, 2u);
}

template <class Kernel>
cudaError_t launch(Kernel k, const MatmulParams &p, const CUtensorMap &tm_a, const CUtensorMap &tm_w, int grid,
                   int cluster, int smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, k, p, tm_a, tm_w);
}

template <class Kernel>
cudaError_t active_clusters(Kernel k, int cluster, int *out) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(cluster));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(out, k, &cfg);
}

}  // namespace

cudaError_t matmul_stall_copies(int on) { return cudaMemcpyToSymbol(g_stall_copies, &on, sizeof on); }

cudaError_t matmul_setup(int sms, MatmulPlan *plan) {
  cudaError_t e = cudaSuccess;
  for (const void *k : {(const void *)k_matmul_split<64, 4>, (const void *)k_matmul_split<128, 2>, (const void *)k_matmul_pair})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  plan->clusters[1] = sms;
  for (int s = 2; s <= MATMUL_SPLITS_MAX && e == cudaSuccess; ++s)
    e = active_clusters(k_matmul_split<128, 2>, s, &plan->clusters[s]);
  if (e == cudaSuccess) e = active_clusters(k_matmul_pair, 2, &plan->pairs);
  if (e == cudaSuccess && plan->pairs < 1) e = cudaErrorNotSupported;
  return e;
}

cudaError_t launch_block_matmul(const MatmulParams &args, const MatmulPlan &plan, cudaStream_t stream) {
  MatmulParams p = args;
  p.k_blocks = qblocks(p.k);
  p.n_blocks = qblocks(p.n);
  p.m_tiles = (p.m + BM - 1) / BM;
  // The form that takes the fewest clocks: waves of clusters, a block's clocks
  // for each of a CTA's k blocks (measured: the tile's products, or the read
  // of its weights where all CTAs stream), and what a wave costs beside them
  // (start, pipeline fill, the meeting of the sums).
  const double PAIR_BLOCK = 560, PAIR_WAVE = 3000, WAVE = 2500, MEET = 1500;
  const int64_t pair_tiles = int64_t((p.m + 255) / 256) * ((p.n + PAIR_N - 1) / PAIR_N);
  double best = double((pair_tiles + plan.pairs - 1) / plan.pairs) * (p.k_blocks * PAIR_BLOCK + PAIR_WAVE);
  int bn = 0;
  p.splits = 1;
  for (int n : {128, 64})
    for (int s = 1; s <= std::min(MATMUL_SPLITS_MAX, p.k_blocks); ++s) {
      if (plan.clusters[s] < 1) continue;
      const int64_t tiles = int64_t(p.m_tiles) * ((p.n + n - 1) / n);
      const double block = n == 128 ? 700 : 400;
      const double clocks = double((tiles + plan.clusters[s] - 1) / plan.clusters[s]) *
                            (double((p.k_blocks + s - 1) / s) * block + WAVE + (s > 1 ? MEET : 0));
      if (clocks < best) {
        best = clocks;
        bn = n;
        p.splits = s;
      }
    }
  CUtensorMap tm_a, tm_w;
  if (bn == 0) {
    p.m_tiles = (p.m + 255) / 256;
    p.n_tiles = (p.n + PAIR_N - 1) / PAIR_N;
    if (!encode_rows_sw128(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.values, p.m, p.k, p.values_stride, 128, BM) ||
        !encode_rows_sw128(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weight, p.n, p.k, p.weight_stride, 128, BM))
      return cudaErrorInvalidValue;
    const int pairs = int(std::min<int64_t>(pair_tiles, plan.pairs));
    return launch(k_matmul_pair, p, tm_a, tm_w, 2 * pairs, 1, SMEM_BYTES, stream);   // the kernel's own cluster size
  }
  p.n_tiles = (p.n + bn - 1) / bn;
  p.a_rows = std::min(BM, (p.m + 7) / 8 * 8);
  // the tensor core reads 128 rows of `values` whatever their number: the last
  // block's may reach past its own end
  const int block_bytes = p.a_rows * 128 + bn * 128, group = 256 / bn;
  p.stages = std::min(STAGES_MAX, (RING_BYTES - std::max(0, BM * 128 - block_bytes)) / (group * block_bytes));
  if (!encode_rows_sw128(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.values, p.m, p.k, p.values_stride, 128, p.a_rows) ||
      !encode_rows_sw128(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weight, p.n, p.k, p.weight_stride, 128, bn))
    return cudaErrorInvalidValue;
  const int grid = p.m_tiles * p.n_tiles * p.splits;
  return bn == 128 ? launch(k_matmul_split<128, 2>, p, tm_a, tm_w, grid, p.splits, SMEM_BYTES, stream)
                   : launch(k_matmul_split<64, 4>, p, tm_a, tm_w, grid, p.splits, SMEM_BYTES, stream);
}

}  // namespace mhc
