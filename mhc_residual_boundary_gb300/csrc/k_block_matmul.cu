// k_block_matmul.cu -- product of 8-bit matrices with a scale for each block
// of 128:
//   out[m][n] = sum_kb sa[m][kb] sw[n/128][kb] * sum_{k in kb} a[m][k] w[n][k]
//
// The inner sums (128 E4M3 products) run on the tensor cores into tensor
// memory; the scaled outer sum runs in FP32 registers.  A CTA's tile is 128
// rows of `a` (a TMEM lane each, so the row's scale is one register of one
// thread) by BN rows of `w`; an epilogue warp group owns 128 (BN = 256) or 64
// columns, so the weight's scale is one value for all of them, and the outer
// sum is one packed FP32 fused multiply-add for every two elements and block.
//
// Roles (12 warps): TMA producer, MMA issuer, TMEM owner, and eight epilogue
// warps (two per TMEM sub-partition).  Operands arrive in a ring of stages of
// one k block (128 bytes a row, 128-byte swizzled); the accumulator is a ring
// of 512 / BN buffers, so the tensor cores work on one block while the
// epilogue warps add the one before.
//
// Few tiles: each tile's k blocks are split over `splits` work items.  Every
// item then writes its FP32 sums to scratch, and the last of a tile's items
// to arrive adds them in split order, so the result does not depend on the
// order of arrival.
#include <algorithm>

#include "sublayer.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int BM = 128;
constexpr int NT = 384;
constexpr int EPI_WARP0 = 4, EPI_THREADS = 256;
constexpr int STAGES_MAX = 12;
constexpr int SMEM_CTRL = 1024;
constexpr int SMEM_BYTES = 227 * 1024;

__device__ int g_stall_copies;   // test hook: the producer issues no copies

struct Control {
  uint64_t full[STAGES_MAX], empty[STAGES_MAX], acc_full[4], acc_empty[4], drain;
  uint32_t tmem;
  int abort, last;
};
static_assert(sizeof(Control) <= SMEM_CTRL, "control block");

template <int BN>
__global__ void __launch_bounds__(NT, 1)
k_block_matmul(const MatmulParams p, const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_w) {
  constexpr int BUFS = 512 / BN;
  constexpr int NC = BN / 2;             // columns of an epilogue warp group
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = smem_raw;
  Control &c = *reinterpret_cast<Control *>(smem);
  unsigned char *ring = smem + SMEM_CTRL;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  const int a_bytes = p.a_rows * 128, stage_bytes = a_bytes + BN * 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      tc::mbar_init(&c.full[i], 1);
      tc::mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      tc::mbar_init(&c.acc_full[i], 1);
      tc::mbar_init(&c.acc_empty[i], EPI_THREADS / 32);
    }
    tc::mbar_init(&c.drain, 1);
    tc::mbar_init_fence();
    c.abort = 0;
    tc::tma_prefetch_desc(&tm_a);
    tc::tma_prefetch_desc(&tm_w);
  }
  if (warp == 2) tc::tmem_alloc(&c.tmem, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = c.tmem;
  pdl_wait();
  pdl_launch_dependents();

  const int items = p.m_tiles * p.n_tiles * p.splits;
  if (warp == 0) {
    // ---------------------------------------------------------- producer
    int n = 0;
    bool ok = !g_stall_copies;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const WorkItem w = work_item(p, item);
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n) {
        const int s = n % p.stages;
        if (n >= p.stages && !tc::wait_or_abort(&c.empty[s], uint32_t((n / p.stages - 1) & 1), abort)) {
          ok = false;
          break;
        }
        if (tc::elect_one()) {
          unsigned char *dst = ring + size_t(s) * stage_bytes;
          tc::mbar_arrive_expect_tx(&c.full[s], uint32_t(stage_bytes));
          tc::tma_load_2d(dst, &tm_a, kb * 128, w.m0, &c.full[s]);
          tc::tma_load_2d(dst + a_bytes, &tm_w, kb * 128, w.n_tile * BN, &c.full[s]);
        }
        __syncwarp();
      }
    }
    // copies in flight land before the CTA's shared memory goes
    if (*abort)
      for (int i = max(0, n - p.stages); i < n; ++i)
        tc::mbar_wait_bounded(&c.full[i % p.stages], uint32_t((i / p.stages) & 1), tc::SUB_WAIT_LIMIT);
  } else if (warp == 1) {
    // -------------------------------------------------------- MMA issuer
    const uint32_t idesc = tc::idesc_e4m3_f32(BM, BN);
    int n = 0;
    bool ok = true;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const WorkItem w = work_item(p, item);
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n) {
        const int s = n % p.stages, b = n % BUFS;
        ok = tc::wait_or_abort(&c.full[s], uint32_t((n / p.stages) & 1), abort) &&
             (n < BUFS || tc::wait_or_abort(&c.acc_empty[b], uint32_t((n / BUFS - 1) & 1), abort));
        if (!ok) break;
        tc::fence_after_sync();
        const unsigned char *src = ring + size_t(s) * stage_bytes;
        const uint64_t ad = tc::desc_sw128(src), bd = tc::desc_sw128(src + a_bytes);
        if (tc::elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc::mma_e4m3(tmem + uint32_t(b * BN), ad + 2 * ks, bd + 2 * ks, idesc, ks != 0);
          tc::mma_commit(&c.empty[s]);
          tc::mma_commit(&c.acc_full[b]);
        }
        __syncwarp();
      }
    }
    // no MMA is in flight when the tensor memory goes
    if (tc::elect_one()) tc::mma_commit(&c.drain);
    __syncwarp();
    tc::mbar_wait_bounded(&c.drain, 0u, tc::SUB_WAIT_LIMIT);
  } else if (warp >= EPI_WARP0) {
    // ---------------------------------------------------------- epilogue
    // After a wait gave up these warps go through the rest of their loops on
    // whatever is there (the waits return at once), so that they meet at their
    // barriers and every arrival is counted.
    const int sub = warp % 4, group = (warp - EPI_WARP0) / 4;
    const uint32_t lane_base = tmem + (uint32_t(sub * 32) << 16) + uint32_t(group * NC);
    const int epi_tid = threadIdx.x - EPI_WARP0 * 32;
    int n = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      const WorkItem w = work_item(p, item);
      const int row = w.m0 + sub * 32 + lane;
      const int n0 = w.n_tile * BN + group * NC;
      const bool rows_live = w.m0 + sub * 32 < p.m, live = row < p.m;
      const float *sa = p.scales + size_t(live ? row : 0) * p.scales_stride;
      const float *sw = p.weight_scales + size_t(min(n0 / QBLOCK, p.n_blocks - 1)) * p.k_blocks;
      uint64_t acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
      float a_next = __ldg(sa + w.kb0), w_next = __ldg(sw + w.kb0);
      for (int kb = w.kb0; kb < w.kb1; ++kb, ++n) {
        const int b = n % BUFS;
        const float scale = a_next * w_next;
        if (kb + 1 < w.kb1) {
          a_next = __ldg(sa + kb + 1);
          w_next = __ldg(sw + kb + 1);
        }
        tc::wait_or_abort(&c.acc_full[b], uint32_t((n / BUFS) & 1), abort);
        __syncwarp();
        tc::fence_after_sync();
        if (rows_live) {
          const uint64_t s2 = tc::pair(scale, scale);
#pragma unroll
          for (int h = 0; h < NC; h += 64) {
            uint32_t d0[32], d1[32];
            tc::tmem_ld32_async(lane_base + uint32_t(b * BN + h), d0);
            tc::tmem_ld32_async(lane_base + uint32_t(b * BN + h + 32), d1);
            tc::tmem_wait_ld();
            tc::tmem_hold(d0);
            tc::tmem_hold(d1);
            if (h + 64 == NC) {
              tc::fence_before_sync();
              __syncwarp();
              if (lane == 0) tc::mbar_arrive(&c.acc_empty[b]);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) tc::fma_pair(acc[h / 2 + i], d0[2 * i], d0[2 * i + 1], s2);
#pragma unroll
            for (int i = 0; i < 16; ++i) tc::fma_pair(acc[h / 2 + 16 + i], d1[2 * i], d1[2 * i + 1], s2);
          }
        } else if (lane == 0) {
          tc::mbar_arrive(&c.acc_empty[b]);
        }
      }
      bool finish = true;
      if (p.splits > 1) {
        // fragment [column][row], rows padded to a_rows: neighbouring lanes
        // write neighbouring words
        const int tile = w.tile;
        const size_t frag = size_t(BN) * p.a_rows;
        float *mine = p.scratch + (size_t(tile) * p.splits + w.split) * frag;
        const int r = sub * 32 + lane;
        if (live) {
#pragma unroll
          for (int i = 0; i < NC / 2; ++i) {
            __stcg(mine + size_t(group * NC + 2 * i) * p.a_rows + r, tc::pair_lo(acc[i]));
            __stcg(mine + size_t(group * NC + 2 * i + 1) * p.a_rows + r, tc::pair_hi(acc[i]));
          }
        }
        __threadfence();
        tc::named_barrier(1, EPI_THREADS);
        if (epi_tid == 0) c.last = atomicAdd(p.counters + tile, 1u) == unsigned(p.splits - 1);
        tc::named_barrier(1, EPI_THREADS);
        finish = c.last != 0;
        tc::named_barrier(1, EPI_THREADS);   // c.last may be written again
        if (finish) {
          __threadfence();
          if (epi_tid == 0) p.counters[tile] = 0;
          if (live) {
            const float *all = p.scratch + size_t(tile) * p.splits * frag + r;
#pragma unroll
            for (int i = 0; i < NC / 2; ++i) acc[i] = 0ull;
            for (int s = 0; s < p.splits; ++s) {
#pragma unroll
              for (int i = 0; i < NC / 2; ++i) {
                const float *src = all + s * frag + size_t(group * NC + 2 * i) * p.a_rows;
                acc[i] = tc::pair(tc::pair_lo(acc[i]) + __ldcg(src), tc::pair_hi(acc[i]) + __ldcg(src + p.a_rows));
              }
            }
          }
        }
      }
      if (finish && live) {
        const size_t at = size_t(row) * p.output_stride;
        if (p.output_f32) {
          float *out = reinterpret_cast<float *>(p.output) + at;
#pragma unroll
          for (int i = 0; i < NC / 2; i += 2) {
            const int col = n0 + 2 * i;
            const float v[4] = {tc::pair_lo(acc[i]), tc::pair_hi(acc[i]), tc::pair_lo(acc[i + 1]), tc::pair_hi(acc[i + 1])};
            if (p.vector_out && col + 4 <= p.n) {
              *reinterpret_cast<float4 *>(out + col) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (col + k < p.n) out[col + k] = v[k];
            }
          }
        } else {
          uint16_t *out = reinterpret_cast<uint16_t *>(p.output) + at;
#pragma unroll
          for (int i = 0; i < NC / 2; i += 4) {
            const int col = n0 + 2 * i;
            uint32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = pack_bf16x2(tc::pair_lo(acc[i + k]), tc::pair_hi(acc[i + k]));
            if (p.vector_out && col + 8 <= p.n) {
              st_vec(out + col, make_uint4(v[0], v[1], v[2], v[3]));
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (col + k < p.n) out[col + k] = uint16_t(v[k / 2] >> (k % 2 * 16));
            }
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 2) tc::tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && c.abort) atomicOr(p.err, 2u);
}

template <int BN>
cudaError_t launch(const MatmulParams &p, const CUtensorMap &tm_a, const CUtensorMap &tm_w, int grid,
                   cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_block_matmul<BN>, p, tm_a, tm_w);
}

}  // namespace

cudaError_t matmul_stall_copies(int on) { return cudaMemcpyToSymbol(g_stall_copies, &on, sizeof on); }

cudaError_t matmul_set_attributes() {
  cudaError_t e = cudaFuncSetAttribute(k_block_matmul<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(k_block_matmul<256>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  return e;
}

cudaError_t launch_block_matmul(const MatmulParams &args, int sms, cudaStream_t stream) {
  MatmulParams p = args;
  p.k_blocks = qblocks(p.k);
  p.n_blocks = qblocks(p.n);
  p.m_tiles = (p.m + BM - 1) / BM;
  const int64_t tiles128 = int64_t(p.m_tiles) * p.n_blocks, tiles256 = int64_t(p.m_tiles) * ((p.n + 255) / 256);
  const bool wide = tiles256 >= sms;
  const int bn = wide ? 256 : 128;
  p.n_tiles = (p.n + bn - 1) / bn;
  p.a_rows = std::min(BM, (p.m + 7) / 8 * 8);
  p.splits = 1;
  if (tiles128 < sms) {
    // as many items as SMs, of at least two k blocks, within the scratch
    p.splits = int(std::min<int64_t>({sms / tiles128, std::max(1, p.k_blocks / 2),
                                      int64_t(p.scratch_floats / (size_t(tiles128) * bn * p.a_rows))}));
    if (p.splits < 1 || tiles128 > p.counter_count) p.splits = 1;
  }
  p.stages = std::min(STAGES_MAX, (SMEM_BYTES - SMEM_CTRL) / (p.a_rows * 128 + bn * 128));
  CUtensorMap tm_a, tm_w;
  if (!encode_rows_sw128(&tm_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.values, p.m, p.k, p.values_stride, 128, p.a_rows) ||
      !encode_rows_sw128(&tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.weight, p.n, p.k, p.weight_stride, 128, bn))
    return cudaErrorInvalidValue;
  const int64_t items = int64_t(p.m_tiles) * p.n_tiles * p.splits;
  const int grid = int(std::min<int64_t>(items, sms));
  return wide ? launch<256>(p, tm_a, tm_w, grid, stream) : launch<128>(p, tm_a, tm_w, grid, stream);
}

}  // namespace mhc
