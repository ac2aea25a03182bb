// sublayer_tc.cuh -- what the sublayer operators' tensor-core kernels share
// beyond tcgen05.cuh: 8-bit MMAs, wide TMEM reads, packed FP32 arithmetic,
// waits that end when another warp of the CTA gave up, and tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "device_common.cuh"
#include "tcgen05.cuh"

namespace mhc {
namespace tc {

// Polls before a wait gives up (about a second).
constexpr uint32_t SUB_WAIT_LIMIT = 1u << 22;

// Waits for the phase with the given parity, until another thread of the CTA
// set *abort or the limit is reached (then this thread sets it).
static __device__ __noinline__ bool wait_poll(uint64_t *bar, uint32_t parity, volatile int *abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < SUB_WAIT_LIMIT; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (i > 64) __nanosleep(64);
  }
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
  return mbar_try_wait(bar, parity) || wait_poll(bar, parity, abort);
}

// A wait in two parts: a test, whose answer arrives (some hundred clocks later)
// while the thread goes on, and the wait for it.  The test is test_wait: a
// try_wait may suspend the thread until the phase completes.
__device__ __forceinline__ bool mbar_test_wait(uint64_t *bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait_or_abort(bool tested, uint64_t *bar, uint32_t parity, volatile int *abort) {
  return tested || wait_poll(bar, parity, abort);
}
// The same without a call: for code that holds most registers.
__device__ __forceinline__ void wait_or_abort_inline(uint64_t *bar, uint32_t parity, volatile int *abort) {
#pragma unroll 1
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
    if (*abort) break;
    if (i > 64) __nanosleep(64);
    if (i > SUB_WAIT_LIMIT) *abort = 1;
  }
}

// Instruction descriptor of kind::f8f6f4: FP32 accumulator, E4M3 A and B,
// both K-major, M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int m, int n) {
  return (1u << 4) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// Descriptor of a K-major operand of 128-byte rows in the 128-byte swizzled
// layout (8-row groups 1024 bytes apart); a K step of 32 bytes adds 2.
__device__ __forceinline__ uint64_t desc_sw128(const void *p) {
  return smem_desc(smem_addr(p), 16, 1024) | (uint64_t(2) << 61);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 / 16 consecutive 32-bit columns of this thread's TMEM lane, without
// waiting (see tmem_ld4_async); r is valid after tmem_wait_ld + tmem_hold.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Keeps uses of loaded columns behind the wait before it.
template <int N>
__device__ __forceinline__ void tmem_hold(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// acc += d * s on a pair of FP32 values (two IEEE fused multiply-adds).
__device__ __forceinline__ void fma_pair(uint64_t &acc, uint32_t d0, uint32_t d1, uint64_t s) {
  const uint64_t d = uint64_t(d1) << 32 | d0;
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s));
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ float pair_lo(uint64_t v) { return __uint_as_float(uint32_t(v)); }
__device__ __forceinline__ float pair_hi(uint64_t v) { return __uint_as_float(uint32_t(v >> 32)); }

}  // namespace tc

// Tensor map of a row-major [rows][cols] matrix (row_bytes apart) for boxes
// of box_rows rows x 128 bytes in the 128-byte swizzled layout; what a box
// covers outside the matrix reads as zero.  False if the driver refuses it.
inline bool encode_rows_sw128(CUtensorMap *map, CUtensorMapDataType type, const void *base, uint64_t rows,
                              uint64_t cols, uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_cols, box_rows}, ones[2] = {1, 1};
  return fn(map, type, 2, const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace mhc
