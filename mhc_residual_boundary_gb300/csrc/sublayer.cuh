// sublayer.cuh -- parameter blocks and launchers of the sublayer operators
// (internal to the library; the public surface is include/mhc_sublayer.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mhc {

constexpr int QBLOCK = 128;              // values that share a scale
constexpr float E4M3_MAX = 448.0f;
constexpr int SUB_MAX_HIDDEN = 16384;    // widest row of the norm's register tiling

constexpr int qblocks(int n) { return (n + QBLOCK - 1) / QBLOCK; }

struct NormParams {
  int m, h;
  const uint16_t *x, *residual, *weight;  // residual may be null
  int64_t x_stride, residual_stride;
  float eps;
  uint16_t *residual_out, *output;        // null: not written
  uint8_t *values;                        // null: not written
  float *scales;
};

struct QuantParams {
  int m, h;
  const uint16_t *x;                      // [m][h], or [m][2h] gate and up
  int64_t x_stride;
  uint16_t *output;                       // null: not written
  uint8_t *values;
  float *scales;
  uint32_t row_mul;                       // division of a block's number by the blocks of a row
  int row_shift;
};

struct MatmulParams {
  int m, n, k;
  const uint8_t *values, *weight;         // e4m3
  int64_t values_stride, weight_stride;
  const float *scales, *weight_scales;    // [m][k_blocks], [n / 128 rounded up][k_blocks]
  int64_t scales_stride;
  void *output;                           // bf16 or f32
  int64_t output_stride;
  int output_f32;
  int vector_out;                         // the output's rows start on 16-byte boundaries
  unsigned int *err;                      // bit 1: a bounded wait gave up
  // set by the launcher
  int k_blocks, m_tiles, n_tiles, splits, stages;
  int a_rows;                             // rows of a stage's `values` tile
  int parts_at;                           // offset of a split tile's sums; 0: where the stages are
};

constexpr int MATMUL_SPLITS_MAX = 8;
// What runs at once on this GPU.
struct MatmulPlan {
  int clusters[MATMUL_SPLITS_MAX + 1];    // clusters of that many CTAs
};

cudaError_t matmul_setup(int sms, MatmulPlan *plan);
cudaError_t matmul_stall_copies(int on);  // test hook, see include/mhc_boundary_test.h
cudaError_t launch_block_matmul(const MatmulParams &p, const MatmulPlan &plan, cudaStream_t stream);

// MoE layer of up to MOE_TOKENS_MAX tokens (k_moe.cu).
constexpr int MOE_TOKENS_MAX = 32;
constexpr int MOE_EXPERTS_MAX = 512;
constexpr int MOE_SHARED_MAX = 8;
constexpr int MOE_TOPK_MAX = 16;
// Chunks of k blocks that a tile's work is cut into, at most.
constexpr int MOE_CHUNKS = 4;

// Scratch of one MoE handle, by its capacity.
struct MoeScratch {
  unsigned int *control;      // MOE_CONTROL words: grid counters (all counters are zero between calls)
  unsigned int *up_counters;  // [reached experts][I / 128] chunks of a tile that are there
  unsigned int *up_done;      // [reached experts] complete tiles
  float *logits;              // [tokens][E]
  uint8_t *x_pieces;          // [3 tokens][H] e4m3 (8-bit weights)
  float *x_scale;             // [tokens]
  float *up;                  // [MOE_CHUNKS][slots][2][I rounded up to 128]
  void *act;                  // [slots * pieces][I]: e4m3 x 3 or bf16 x 2
  float *act_scale;           // [I / 128][slots] (8-bit weights)
  float *down;                // [MOE_CHUNKS][slots][H rounded up to 128]
};
constexpr int MOE_CONTROL = 4;

struct MoeParams {
  int m, hidden, intermediate, experts, shared, top_k;
  int fp8, sigmoid, renormalize, router_f32;
  float routed_scale;
  const uint16_t *x;
  const void *router;
  const float *bias;
  const void *gate_up, *down;
  const float *gate_up_scales, *down_scales;
  uint16_t *output;
  int32_t *idx;
  float *weights;
  int slots;                  // slots of the scratch tensors
  MoeScratch scratch;
  unsigned int *err;
  // set by the launcher: how the work is cut and where things lie in a CTA's
  // shared memory
  int stages, b_bytes;
  int up_chunks, down_chunks; // chunks of a tile's k blocks
  int scale_blocks;           // k blocks of an item at most
  int ring_at, scales_at;     // offsets of the stages and of the items' scales
};
constexpr int MOE_ITEMS = 4;  // items between their taking and the last warp that reads them
constexpr int MOE_SMEM = 227 * 1024;
constexpr int MOE_STAGE_A = 128 * 128;   // bytes of a stage's weight tile

// The launcher's fields of p, on a GPU of that many SMs.
void moe_form(MoeParams &p, int sms);
cudaError_t moe_set_attributes();
cudaError_t moe_stall_copies(int on);   // test hook
cudaError_t launch_moe(const MoeParams &p, int sms, cudaStream_t stream);

cudaError_t launch_add_rms_norm(const NormParams &p, cudaStream_t stream);
cudaError_t launch_quantize(const QuantParams &p, bool swiglu, int sms, cudaStream_t stream);

}  // namespace mhc
