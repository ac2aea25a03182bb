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
// A tile is 128 rows x BN columns.  With few tiles (the read of `w` bounds the
// call) a cluster works on a tile: its CTAs share out the k blocks and their sums
// meet through distributed shared memory, without scratch and in the order of the
// ranks.  With many, CTAs are persistent over the tiles, and what bounds the call
// is the outer sum's chain beside the products and the copies: a block's 128 x 128
// products take the tensor cores 256 clocks and its 32 KB of operands as much of
// shared memory's bandwidth as the products do; the epilogue's turn (a wait, four
// reads of 32 columns from tensor memory, their multiply-adds, the release) some
// 900 clocks for two blocks.
//
// Measured (a call among others in a graph): 4096 x 4096 x 6144 102 us, 2020
// TFLOP/s (without its stores 96 us, without its copies 92, without its additions
// 95); one row of 6144 x 5120 10.2 us, 3.1 TB/s of weights (6.1
// once they flow); 37 rows of 2120 x 5120 7.1 us.
//
// Roles: warp 0 operand copies, 1 MMA, 2-3 scales and tensor memory, 4-11
// epilogue, two warps for each TMEM sub-partition (with four of half the columns
// 4096 x 4096 x 6144 took 118 us against 114).  Operands arrive in a ring
// of stages (128 bytes a row, 128-byte swizzled); the accumulator is a ring of
// buffers, so the tensor cores work on one group of blocks while the epilogue
// warps add the one before.
#include <algorithm>

#include "sublayer.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int BM = 128;                  // rows of a CTA
constexpr int TMEM_WARP = 2, SCALE_WARP0 = 2, EPI_WARP0 = 4, EPI_WARPS = 8;
constexpr int NT = (EPI_WARP0 + EPI_WARPS) * 32;
constexpr int STAGES_MAX = 12;
constexpr int SMEM_CTRL = 1024;
constexpr int SMEM_BYTES = 227 * 1024;
constexpr int CHUNKS_MAX = 2;
constexpr int SMEM_SCALES = 33 * 1024;
constexpr int RING_BYTES = SMEM_BYTES - SMEM_CTRL - SMEM_SCALES;

__device__ int g_stall_copies;   // test hook: the producer issues no copies

struct Control {
  uint64_t full[STAGES_MAX], empty[STAGES_MAX], acc_full[4], acc_empty[4];
  uint64_t scale_full[CHUNKS_MAX], scale_empty[CHUNKS_MAX], drain;
  uint32_t tmem;
  int abort;
  int issued;   // stages that the producer asked for
};
static_assert(sizeof(Control) <= SMEM_CTRL, "control block");

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, uint64_t a, uint64_t b) {
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
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

// The scales of a CTA's rows come through shared memory, CHUNK blocks at a time,
// read by two warps of their own: a row's scales lie side by side in memory, so
// a lane reads a block and a warp a row at a time (a lane a row would touch 32
// lines with every read, and all of the SM's accesses would queue behind them:
// 4096 x 4096 x 6144 took 141 us), and a transposed store makes them one word a
// row.
constexpr int CHUNK = 32, CHUNKS = CHUNKS_MAX;   // k blocks of a chunk, chunks in flight
constexpr int SCALE_ROW = BM + 1;        // words from block to block: no bank conflicts
struct Scales {
  float *a;   // [CHUNKS][CHUNK][SCALE_ROW]
  float *w;   // [CHUNKS][CHUNK]: of the column block that the tile lies in
};
static_assert(CHUNKS * CHUNK * (SCALE_ROW + 1) * 4 <= SMEM_SCALES, "scales");

// One word to shared memory without passing through a register, and the
// barrier's arrival once all of this thread's are there.
__device__ __forceinline__ void copy_word(float *dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(tc::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(tc::smem_addr(bar)) : "memory");
}

// One of the two scale warps: rows 64 * half .. of the k blocks [kb0, kb1).  All
// of a chunk's words are under way at once.
__device__ __forceinline__ void load_scales(const MatmulParams &p, Control &c, const Scales &sc, Ring &ring, int m0,
                                            int n_block, int kb0, int kb1, int half, int lane) {
  const int rows = max(0, min(64, p.m - m0 - half * 64));
  for (int kb = kb0; kb < kb1; kb += CHUNK) {
    tc::wait_or_abort(&c.scale_empty[ring.at], ring.phase ^ 1u, &c.abort);
    __syncwarp();
    if (kb + lane < kb1) {
      float *a = sc.a + (ring.at * CHUNK + lane) * SCALE_ROW + half * 64;
      const float *src = p.scales + size_t(m0 + half * 64) * p.scales_stride + kb + lane;
      if (half == 1)   // up to 64 rows leave this warp without any
        copy_word(sc.w + ring.at * CHUNK + lane, p.weight_scales + size_t(n_block) * p.k_blocks + kb + lane);
#pragma unroll 8
      for (int r = 0; r < rows; ++r, src += p.scales_stride) copy_word(a + r, src);
    }
    copies_arrive(&c.scale_full[ring.at]);
    ring.next(CHUNKS);
  }
}

// An epilogue warp's way through the chunks: the scales of this thread's row
// and of the tile's column block, G blocks (G divides CHUNK) at a time.
struct ScaleReader {
  Ring ring;
  int k = 0;   // blocks taken of this chunk
  template <int G>
  __device__ __forceinline__ void take(Control &c, const Scales &sc, int row, bool last, int lane,
                                       float (&scale)[G]) {
    if (k == 0) {
      tc::wait_or_abort_inline(&c.scale_full[ring.at], ring.phase, &c.abort);
      __syncwarp();
    }
    const int at = ring.at * CHUNK + k;
#pragma unroll
    for (int q = 0; q < G; ++q) scale[q] = sc.a[(at + q) * SCALE_ROW + row] * sc.w[at + q];
    k += G;
    if (k == CHUNK || last) {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.scale_empty[ring.at]);
      ring.next(CHUNKS);
      k = 0;
    }
  }
};

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

// Sixteen bytes of a row to the output.
template <bool F32>
__device__ __forceinline__ void store_piece(const MatmulParams &p, int row, int col, const uint4 &v) {
  constexpr int W = F32 ? 4 : 8;
  if (row >= p.m) return;
  const size_t at = size_t(row) * p.output_stride + col;
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  if (col + W <= p.n) {
    st_vec(static_cast<char *>(p.output) + at * (F32 ? 4 : 2), v);
  } else if (F32) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (col + k < p.n) static_cast<uint32_t *>(p.output)[at + k] = u[k];
  } else {
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (col + k < p.n) static_cast<uint16_t *>(p.output)[at + k] = uint16_t(u[k / 2] >> (k % 2 * 16));
  }
}

// A warp's 32 rows, one a lane, to the output where it takes 16 bytes at a
// time.  Four lanes exchange their rows' pieces (two rounds of a transposition)
// so that they write 64 neighbouring bytes: a lane for itself would write half a
// sector of each of 32 lines (4096 x 4096 x 6144: 111 us, with four lanes' exchange
// 105, with eight lanes' 107).
template <int NC, bool F32>
__device__ __forceinline__ void store_rows(const MatmulParams &p, int row0, int col, int lane,
                                           const uint64_t (&acc)[NC / 2]) {
  constexpr int W = F32 ? 4 : 8;   // columns of a piece
#pragma unroll
  for (int g = 0; g < NC / (4 * W); ++g) {
    uint4 piece[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t *a = acc + (g * 4 + k) * W / 2;
      if (F32) {
        piece[k] = make_uint4(uint32_t(a[0]), uint32_t(a[0] >> 32), uint32_t(a[1]), uint32_t(a[1] >> 32));
      } else {
        const float v[8] = {tc::pair_lo(a[0]), tc::pair_hi(a[0]), tc::pair_lo(a[1]), tc::pair_hi(a[1]),
                            tc::pair_lo(a[2]), tc::pair_hi(a[2]), tc::pair_lo(a[3]), tc::pair_hi(a[3])};
        piece[k] = pack8(v);
      }
    }
#pragma unroll
    for (int bit = 1; bit <= 2; bit <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!(k & bit)) {
          const bool odd = lane & bit;
          uint4 &lo = piece[k], &hi = piece[k | bit];
          auto swap = [&](uint32_t &x, uint32_t &y) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? x : y, bit);
            if (odd) x = got;
            else y = got;
          };
          swap(lo.x, hi.x);
          swap(lo.y, hi.y);
          swap(lo.z, hi.z);
          swap(lo.w, hi.w);
        }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      store_piece<F32>(p, row0 + (lane & ~3) + k, col + (g * 4 + lane % 4) * W, piece[k]);
  }
}

__device__ __forceinline__ void init_control(Control &c, int stages, int bufs) {
  for (int i = 0; i < stages; ++i) {
    tc::mbar_init(&c.full[i], 1);
    tc::mbar_init(&c.empty[i], 1);
  }
  for (int i = 0; i < bufs; ++i) {
    tc::mbar_init(&c.acc_full[i], 1);
    tc::mbar_init(&c.acc_empty[i], EPI_WARPS);
  }
  for (int i = 0; i < CHUNKS; ++i) {
    tc::mbar_init(&c.scale_full[i], 64);   // both scale warps' threads
    tc::mbar_init(&c.scale_empty[i], EPI_WARPS);
  }
  tc::mbar_init(&c.drain, 1);
  tc::mbar_init_fence();
  c.abort = 0;
  c.issued = 0;
}

// Clusters of p.splits CTAs, tile after tile: CTA r of a cluster has the k blocks
// [k_blocks r / splits, k_blocks (r + 1) / splits).  A split tile is its cluster's
// only one.  The roles hand each other groups of G blocks, each block with an
// accumulator of its own: a wait between two roles takes some hundred clocks, as
// long as a block's work (one row of 6144 x 5120 in 64-column tiles: 13.9 us with
// a wait for each block, 11.0 us with one for four).
template <int BN, int G>
__global__ void __launch_bounds__(NT, 1)
k_block_matmul(const MatmulParams p, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w) {
  constexpr int BUFS = 2;                // accumulators of two groups
  constexpr int NC = BN / 2;             // columns of an epilogue warp
  static_assert(BUFS * G * BN == 512, "all of the tensor memory");
  extern __shared__ __align__(1024) unsigned char smem[];
  Control &c = *reinterpret_cast<Control *>(smem);
  unsigned char *ring = smem + SMEM_CTRL;
  float *scales_at = reinterpret_cast<float *>(ring + RING_BYTES);
  const Scales sc = {scales_at, scales_at + CHUNKS * CHUNK * SCALE_ROW};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  const int a_bytes = p.a_rows * 128, block_bytes = a_bytes + BN * 128;
  const int rank = p.splits > 1 ? int(cluster_rank()) : 0;
  const int kb0 = p.k_blocks * rank / p.splits, kb1 = p.k_blocks * (rank + 1) / p.splits;
  const int tiles = p.m_tiles * p.n_tiles, first = int(blockIdx.x) / p.splits, step = int(gridDim.x) / p.splits;

  // The sums of a split tile: groups of eight columns, each summed by one CTA of
  // the cluster, [group of this CTA][rank they come from][row][8].
  constexpr int GROUPS = BN / 8;
  float *parts = reinterpret_cast<float *>(ring + p.parts_at);
  auto first_group = [&](int r) { return (r * GROUPS + p.splits - 1) / p.splits; };
  // once every CTA of the cluster runs and, where the parts are in the stages,
  // has no copy or MMA of its own left
  auto meet = [&]() {
    __syncwarp();
    if (p.parts_at == 0) cluster_arrive();
    cluster_wait();
  };
  if (p.splits > 1 && p.parts_at != 0) cluster_arrive();

  // The weights of the first stages are on their way to L2 while the kernel
  // before this one ends (a prefetch is no read: what that kernel may still write
  // is written there too) and this one sets itself up: the first blocks take two
  // microseconds from memory.
  if (warp == 1) {
    tc::tma_prefetch_desc(&tm_w);
    for (int kb = kb0 + lane; kb < min(kb1, kb0 + p.stages * G); kb += 32)
      tc::tma_prefetch_2d(&tm_w, kb * 128, first / p.m_tiles * BN);
    tc::tma_prefetch_desc(&tm_a);
  }
  if (threadIdx.x == 0) init_control(c, p.stages, BUFS);
  if (warp == TMEM_WARP) tc::tmem_alloc(&c.tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  pdl_launch_dependents();

  // The copies and the MMAs are issued by one thread that runs their whole
  // loop: under a predicate carried from outside a loop an MMA takes some 25
  // clocks more to issue (its operands leave the uniform registers).
  if (warp == 0) {
    // ---------------------------------------------------------- producer
    if (tc::elect_one()) {
      Ring at;
      int issued = 0;
      bool ok = !g_stall_copies;
      for (int tile = first; tile < tiles && ok; tile += step) {
        const int m0 = tile % p.m_tiles * BM, n0 = tile / p.m_tiles * BN;
        for (int kb = kb0; kb < kb1; kb += G) {
          ok = tc::wait_or_abort(&c.empty[at.at], at.phase ^ 1u, abort);
          if (!ok) break;
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
      }
      c.issued = issued;
    }
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    const uint32_t idesc = tc::idesc_e4m3_f32(BM, BN);
    const uint64_t a0 = tc::desc_sw128(ring), b0 = tc::desc_sw128(ring + a_bytes);
    if (tc::elect_one()) {
      Ring at, acc;
      bool full = false, released = false;   // the next group's barriers, tested beside this one's products
      const int per_tile = (kb1 - kb0 + G - 1) / G;
      int left = first < tiles ? (tiles - first + step - 1) / step * per_tile : 0;
      for (int g = 0; left > 0; --left, g = g + 1 == per_tile ? 0 : g + 1) {
        if (!tc::wait_or_abort(full, &c.full[at.at], at.phase, abort) ||
            !tc::wait_or_abort(released, &c.acc_empty[acc.at], acc.phase ^ 1u, abort))
          break;
        const Ring at0 = at, acc0 = acc;
        at.next(p.stages);
        acc.next(BUFS);
        full = tc::mbar_test_wait(&c.full[at.at], at.phase);
        released = tc::mbar_test_wait(&c.acc_empty[acc.at], acc.phase ^ 1u);
        tc::fence_after_sync();
        const int blocks = min(G, kb1 - kb0 - g * G);
#pragma unroll
        for (int q = 0; q < G; ++q) {
          if (q >= blocks) break;
          const uint64_t place = uint64_t((at0.at * G + q) * (block_bytes >> 4));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_e4m3(tmem + uint32_t((acc0.at * G + q) * BN), a0 + place + 2 * ks, b0 + place + 2 * ks, idesc,
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
    for (int tile = first; tile < tiles; tile += step)
      load_scales(p, c, sc, scales, tile % p.m_tiles * BM, tile / p.m_tiles * BN / QBLOCK, kb0, kb1,
                  warp - SCALE_WARP0, lane);
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ---------------------------------------------------------- epilogue
    // After a wait gave up these warps go through the rest of their loops on
    // whatever is there (the waits return at once).
    const int sub = warp % 4, group = (warp - EPI_WARP0) / 4, r = sub * 32 + lane;
    const int col = group * NC;
    const uint32_t lane_base = tmem + (uint32_t(sub * 32) << 16) + uint32_t(col);
    Ring buf;
    ScaleReader scales;
    // The first pass has no blocks and no rows: it brings the instructions of the
    // output, which would come from memory one line after another, while the
    // first operands are on their way.
    bool first_pass = true;
    for (int tile = first; tile < tiles; tile += first_pass ? 0 : step, first_pass = false) {
      const int m0 = first_pass ? p.m_tiles * BM : tile % p.m_tiles * BM, n0 = tile / p.m_tiles * BN;
      const bool rows_live = m0 + sub * 32 < p.m, live = m0 + r < p.m;
      uint64_t acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
      for (int k = first_pass ? kb1 : 0; k < kb1 - kb0; k += G) {
        const int blocks = min(G, kb1 - kb0 - k);
        float scale[G];
        scales.take(c, sc, r, k + G >= kb1 - kb0, lane, scale);
        tc::wait_or_abort_inline(&c.acc_full[buf.at], buf.phase, abort);
        __syncwarp();
        tc::fence_after_sync();
        // Parts of 32 columns: the next one is read while this one is added, and
        // the buffer is given back before the last is added (4096 x 4096 x 6144:
        // 105 us with each block's reads before its additions, 102 us so).
        constexpr int H = NC / 32;
        const uint32_t from = lane_base + uint32_t(buf.at * G * BN);
        auto release = [&]() {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&c.acc_empty[buf.at]);
        };
        auto add = [&](int j, const uint32_t (&d)[32]) {
          const uint64_t s2 = tc::pair(scale[j / H], scale[j / H]);
#pragma unroll
          for (int i = 0; i < 16; ++i) tc::fma_pair(acc[j % H * 16 + i], d[2 * i], d[2 * i + 1], s2);
        };
        if (rows_live && blocks == G) {
          uint32_t d[2][32];
          tc::tmem_ld32_async(from, d[0]);
#pragma unroll
          for (int j = 0; j < G * H; ++j) {
            tc::tmem_wait_ld();
            tc::tmem_hold(d[j % 2]);
            if (j + 1 < G * H) tc::tmem_ld32_async(from + uint32_t((j + 1) / H * BN + (j + 1) % H * 32), d[(j + 1) % 2]);
            else release();
            add(j, d[j % 2]);
          }
        } else {
          if (rows_live)
#pragma unroll
            for (int j = 0; j < G * H; ++j)
              if (j / H < blocks) {
                uint32_t d[32];
                tc::tmem_ld32_async(from + uint32_t(j / H * BN + j % H * 32), d);
                tc::tmem_wait_ld();
                tc::tmem_hold(d);
                add(j, d);
              }
          release();
        }
        buf.next(BUFS);
      }
      if (p.splits == 1) {
        if (!p.vector_out) {
          if (live) store_row<NC>(p, m0 + r, n0 + col, acc);
        } else if (p.output_f32) {
          store_rows<NC, true>(p, m0 + sub * 32, n0 + col, lane, acc);
        } else {
          store_rows<NC, false>(p, m0 + sub * 32, n0 + col, lane, acc);
        }
      } else {
        if (!first_pass) meet();
        int owner = col / 8 * p.splits / GROUPS, place = col / 8 - first_group(owner);
#pragma unroll
        for (int g = 0; g < NC / 8; ++g, ++place) {
          const int to = (col / 8 + g) * p.splits / GROUPS;
          if (to != owner) place = 0;
          owner = to;
          const uint32_t at =
              peer_addr(parts + (size_t(place * p.splits + rank) * p.a_rows + r) * 8, uint32_t(owner));
          if (live) {
            st_peer(at, acc[g * 4], acc[g * 4 + 1]);
            st_peer(at + 16, acc[g * 4 + 2], acc[g * 4 + 3]);
          }
        }
      }
    }
  }
  if (p.splits > 1) {
    if (warp < EPI_WARP0) meet();
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // this CTA's share of the tile, in the order of the ranks
    const int m0 = first % p.m_tiles * BM, n0 = first / p.m_tiles * BN, rows = min(BM, p.m - m0);
    const int g0 = first_group(rank), items = (first_group(rank + 1) - g0) * rows;
    for (int i = threadIdx.x; i < items; i += NT) {
      const int g = i / rows, row = i - g * rows;
      const float4 *at = reinterpret_cast<const float4 *>(parts + (size_t(g * p.splits) * p.a_rows + row) * 8);
      float v[8] = {};
#pragma unroll 4
      for (int s = 0; s < p.splits; ++s, at += p.a_rows * 2) {
        const float4 a = at[0], b = at[1];
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
      }
      if (n0 + (g0 + g) * 8 < p.n) store8(p, m0 + row, n0 + (g0 + g) * 8, v);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == TMEM_WARP) tc::tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && c.abort) {
    atomicOr(p.err, 2u);
    // copies in flight land before the CTA's shared memory goes, whoever gave up
    // and whenever (the producer may have left by then)
    for (int i = max(0, c.issued - p.stages); i < c.issued; ++i)
      tc::mbar_wait_bounded(&c.full[i % p.stages], uint32_t((i / p.stages) & 1), tc::SUB_WAIT_LIMIT);
  }
}

template <class Kernel>
cudaError_t launch(Kernel k, const MatmulParams &p, const CUtensorMap &tm_a, const CUtensorMap &tm_w, int grid,
                   int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM_BYTES;
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
  for (const void *k : {(const void *)k_block_matmul<64, 4>, (const void *)k_block_matmul<128, 2>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  plan->clusters[1] = sms;
  for (int s = 2; s <= MATMUL_SPLITS_MAX && e == cudaSuccess; ++s)
    e = active_clusters(k_block_matmul<128, 2>, s, &plan->clusters[s]);
  return e;
}

cudaError_t launch_block_matmul(const MatmulParams &args, const MatmulPlan &plan, cudaStream_t stream) {
  MatmulParams p = args;
  p.k_blocks = qblocks(p.k);
  p.m_tiles = (p.m + BM - 1) / BM;
  // The form that takes the fewest clocks: rounds of clusters, a block's clocks
  // for each of a CTA's k blocks, and what a call and a split tile cost beside
  // them (start, pipeline fill, the meeting of the sums).
  const double START = 6000, MEET = 1500;
  double best = 1e30;
  int bn = 0;
  for (int n : {128, 64})
    for (int s = 1; s <= std::min(MATMUL_SPLITS_MAX, p.k_blocks); ++s) {
      const int64_t tiles = int64_t(p.m_tiles) * ((p.n + n - 1) / n);
      if (plan.clusters[s] < 1 || (s > 1 && tiles > plan.clusters[s])) continue;
      const double block = n == 128 ? 600 : 400;
      const double clocks = START + double((tiles + plan.clusters[s] - 1) / plan.clusters[s]) *
                                        double((p.k_blocks + s - 1) / s) * block + (s > 1 ? MEET : 0);
      if (clocks < best) {
        best = clocks;
        bn = n;
        p.splits = s;
      }
    }
  p.n_tiles = (p.n + bn - 1) / bn;
  p.a_rows = std::min(BM, (p.m + 7) / 8 * 8);
  // the tensor core reads 128 rows of `values` whatever their number: the last
  // block's may reach past its own end
  const int block_bytes = p.a_rows * 128 + bn * 128, group = 256 / bn;
  int ring = RING_BYTES - std::max(0, BM * 128 - block_bytes);
  // A split tile's sums have a place of their own where that takes little from
  // the stages: the CTAs then meet once, not twice (one row of 6144 x 5120: 10.8 us
  // with two meetings).
  const int parts = p.splits > 1 ? (bn / 8 + p.splits - 1) * p.a_rows * 32 : 0;
  p.parts_at = 0;
  if (parts > 0 && parts <= RING_BYTES / 6) {
    ring -= parts;
    p.parts_at = RING_BYTES - parts;
  }
  p.stages = std::min(STAGES_MAX, ring / (group * block_bytes));
  CUtensorMap tm_a, tm_w;
  if (!encode_rows_sw128(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.values, p.m, p.k, p.values_stride, 128, p.a_rows) ||
      !encode_rows_sw128(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weight, p.n, p.k, p.weight_stride, 128, bn))
    return cudaErrorInvalidValue;
  const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles;
  const int grid = int(std::min<int64_t>(tiles, plan.clusters[p.splits])) * p.splits;
  if (bn == 64) return launch(k_block_matmul<64, 4>, p, tm_a, tm_w, grid, p.splits, stream);
  return launch(k_block_matmul<128, 2>, p, tm_a, tm_w, grid, p.splits, stream);
}

}  // namespace mhc
