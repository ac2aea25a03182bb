// k_rowquant.cu -- RMS norm with the residual's addition, and the 8-bit
// quantisers (plain and SwiGLU), rows in BF16, 8-bit outputs as E4M3 values
// with one FP32 scale for each 128 values of a row.
//
//   r = x + residual; y = r * rsqrt(mean(r^2) + eps) * w
//   scale = max(amax, 2^-100) / 448, value = x * (448 / amax), the quotients by
//   rounded reciprocals (e4m3_scale.h)
// The norm moves 2 + 2 bytes in and up to 2 + 2 + 1 out for each element,
// quantize 2 in and 1 out, swiglu 4 in and 1 out.  Every value crosses the memory
// once: the row stays in registers between its reduction and its output.
//
// Measured (a call among others in a graph): norm of 4096 x 6144 with all outputs
// 37.5 us, 6.05 TB/s, bound by memory; one row of 5120 2.6 us, a launch and two
// memory trips one after another (x and residual, then the weight); quantize 1999 x
// 5064 7.4 us, 4.2 TB/s; swiglu 4096 x 2048 9.9 us, 4.3 TB/s, of which some 2.5 us
// are launch and ramp and the rest the SiLU's instructions as much as the bytes.  A
// thread holds
// one or two 16-byte fragments (8 values each), so 16 or 8 neighbouring lanes
// hold a block of 128 and its largest magnitude takes four shuffles or three.
// Magnitudes are compared as the bit patterns of |x|: their order is that of the
// numbers, with infinity above them and NaN above that, so a non-finite value
// always reaches the block's scale.
#include <algorithm>

#include "device_common.cuh"
#include "e4m3_scale.h"
#include "sublayer.cuh"

namespace mhc {
namespace {

constexpr uint32_t AMAX_FLOOR_BITS = uint32_t(127 - 100) << 23;   // 2^-100

// Bit pattern of the largest |y| of this lane's block (N values in each of 128 /
// N lanes).
template <int N>
__device__ __forceinline__ uint32_t block_amax(const float (&y)[N]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max(a, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
  for (int o = QBLOCK / N / 2; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  return max(a, AMAX_FLOOR_BITS);
}

__device__ __forceinline__ float inverse_of(float amax) { return e4m3_inverse(amax, rcp_fast(e4m3_divisor(amax))); }

// Eight values to E4M3 at inv = 448 / amax.
__device__ __forceinline__ uint2 quant8(const float *y, float inv) {
  return make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                    e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

// 16 bytes, read once, of a row that this thread may write later (residual_out may
// be residual): not through the read-only path.
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// One row per threadIdx.y, VPT fragments a thread.
template <int VPT>
__global__ void __launch_bounds__(256) k_add_rms_norm(const NormParams p) {
  __shared__ float part[8];
  const int tx = threadIdx.x, T = blockDim.x;
  const int warps = T / 32, warp = threadIdx.y * warps + tx / 32;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live_row = row < p.m;
  const int frags = p.h / 8;
  pdl_wait();
  pdl_launch_dependents();
  const uint16_t *x = p.x + size_t(live_row ? row : 0) * p.x_stride;
  const uint16_t *res = p.residual ? p.residual + size_t(live_row ? row : 0) * p.residual_stride : nullptr;
  uint4 xv[VPT], rv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int f = i * T + tx;
    const bool live = live_row && f < frags;
    xv[i] = live ? ld_once(x + size_t(f) * 8) : make_uint4(0, 0, 0, 0);
    rv[i] = live && res ? ld_once(res + size_t(f) * 8) : make_uint4(0, 0, 0, 0);
  }
  float r[VPT][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float b[8];
    unpack8(xv[i], r[i]);
    unpack8(rv[i], b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (res) r[i][k] += b[k];
      ss = fmaf(r[i][k], r[i][k], ss);
    }
  }
  ss = warp_sum(ss);
  if (warps > 1) {
    if (tx % 32 == 0) part[warp] = ss;
    __syncthreads();
    const int lane = tx % 32;
    ss = warp_sum(lane < warps ? part[threadIdx.y * warps + lane] : 0.f);
  }
  const float rstd = __frsqrt_rn(__fdiv_rn(ss, float(p.h)) + p.eps);
  const size_t base = size_t(row) * p.h;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int f = i * T + tx;
    const bool live = live_row && f < frags;
    const size_t at = base + size_t(f) * 8;
    if (live && p.residual_out) st_vec(p.residual_out + at, pack8(r[i]));
    if (!p.output && !p.values) continue;
    float w[8];
    unpack8(live ? ld_ro(p.weight + size_t(f) * 8) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) r[i][k] = r[i][k] * rstd * w[k];
    if (live && p.output) st_vec(p.output + at, pack8(r[i]));
  }
  if (!p.values) return;
  // the fragments' chains (shuffles, quotients) run side by side
  float amax[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) amax[i] = __uint_as_float(block_amax(r[i]));
  float inv[VPT], scale[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    inv[i] = inverse_of(amax[i]);
    scale[i] = e4m3_scale(amax[i]);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int f = i * T + tx;
    if (!live_row || f >= frags) continue;
    *reinterpret_cast<uint2 *>(p.values + base + size_t(f) * 8) = quant8(r[i], inv[i]);
    if (f % (QBLOCK / 8) == 0) p.scales[size_t(row) * qblocks(p.h) + f / (QBLOCK / 8)] = scale[i];
  }
}

// 32 bytes, read once.
__device__ __forceinline__ void ld_stream32(const void *p, uint4 (&v)[2]) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                 "=r"(v[1].w)
               : "l"(p));
}

// A lane has FR fragments of a block, 16 / FR lanes a block, and takes U blocks
// a round, all of their reads under way together.  WIDE: rows are read 32 bytes
// at a time.  Index: 32 bits while the blocks can be counted in them, with the
// division by the blocks of a row as a product (a 64-bit division for each block
// costs more than its bytes).
template <bool SWIGLU, int FR, int U, bool WIDE, class Index>
__global__ void __launch_bounds__(256) k_quantize(const QuantParams p) {
  constexpr int L = 16 / FR, WARP_BLOCKS = 32 / L, CTA_BLOCKS = 8 * WARP_BLOCKS;
  const Index per_row = qblocks(p.h), blocks = Index(p.m) * per_row;
  pdl_wait();
  pdl_launch_dependents();
  // all of a warp takes the same number of rounds (the shuffles need all 32
  // lanes)
  const Index step = Index(gridDim.x) * CTA_BLOCKS;
  for (Index b0 = Index(blockIdx.x) * CTA_BLOCKS + threadIdx.x / 32 * WARP_BLOCKS; b0 < blocks; b0 += step * U) {
    uint4 g[U][FR], u[U][FR];
    Index row[U];
    int f[U], left[U];   // first fragment; this lane's fragments inside the row
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const Index b = b0 + i * step + threadIdx.x % 32 / L;
      row[i] = sizeof(Index) == 4 ? Index((__umulhi(uint32_t(b), p.row_mul) + uint32_t(b)) >> p.row_shift) : b / per_row;
      f[i] = int(b - row[i] * per_row) * 16 + threadIdx.x % L * FR;
      left[i] = b < blocks ? p.h / 8 - f[i] : 0;
      const uint16_t *x = p.x + int64_t(row[i]) * p.x_stride + f[i] * 8;
      if (WIDE) {
        g[i][0] = g[i][FR - 1] = u[i][0] = u[i][FR - 1] = make_uint4(0, 0, 0, 0);
        if (left[i] > 0) {
          ld_stream32(x, reinterpret_cast<uint4(&)[2]>(g[i]));
          if (SWIGLU) ld_stream32(x + p.h, reinterpret_cast<uint4(&)[2]>(u[i]));
        }
      } else {
#pragma unroll
        for (int e = 0; e < FR; ++e) {
          g[i][e] = left[i] > e ? ld_stream(x + e * 8) : make_uint4(0, 0, 0, 0);
          if (SWIGLU) u[i][e] = left[i] > e ? ld_stream(x + p.h + e * 8) : make_uint4(0, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float y[FR * 8];
      const int64_t at = int64_t(row[i]) * p.h + f[i] * 8;
#pragma unroll
      for (int e = 0; e < FR; ++e) {
        float v[8];
        unpack8(g[i][e], v);
        if (SWIGLU) {
          float up[8];
          unpack8(u[i][e], up);
          // 1 / (1 + exp(-v)) within an ulp, FP32 like all else here (swiglu 4096 x
          // 2048: 9.9 us, with a correctly rounded quotient 12.3)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[k] * rcp_approx(1.f + expf(-v[k])) * up[k];
        }
        if (p.output && left[i] > e) st_vec(p.output + at + e * 8, pack8(v));
#pragma unroll
        for (int k = 0; k < 8; ++k) y[e * 8 + k] = v[k];
      }
      const float amax = __uint_as_float(block_amax(y)), inv = inverse_of(amax);
      if (WIDE) {
        const uint2 a = quant8(y, inv), c = quant8(y + (FR - 1) * 8, inv);
        if (left[i] > 0) *reinterpret_cast<uint4 *>(p.values + at) = make_uint4(a.x, a.y, c.x, c.y);
      } else {
#pragma unroll
        for (int e = 0; e < FR; ++e)
          if (left[i] > e) *reinterpret_cast<uint2 *>(p.values + at + e * 8) = quant8(y + e * 8, inv);
      }
      if (left[i] > 0 && f[i] % 16 == 0) p.scales[int64_t(row[i]) * per_row + f[i] / 16] = e4m3_scale(amax);
    }
  }
}

template <class Kernel, class Params>
cudaError_t launch_pdl(Kernel k, dim3 grid, dim3 block, const Params &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace

cudaError_t launch_add_rms_norm(const NormParams &p, cudaStream_t stream) {
  const int frags = p.h / 8;
  const int vpt = frags <= 256 ? 1 : frags <= 512 ? 2 : frags <= 1024 ? 4 : 8;
  const int T = ((frags + vpt - 1) / vpt + 31) / 32 * 32;
  const int rows = std::max(1, 256 / T);
  const dim3 grid((p.m + rows - 1) / rows), block(T, rows);
  switch (vpt) {
    case 1: return launch_pdl(k_add_rms_norm<1>, grid, block, p, stream);
    case 2: return launch_pdl(k_add_rms_norm<2>, grid, block, p, stream);
    case 4: return launch_pdl(k_add_rms_norm<4>, grid, block, p, stream);
    default: return launch_pdl(k_add_rms_norm<8>, grid, block, p, stream);
  }
}

namespace {

template <bool SWIGLU>
cudaError_t launch_quantize_as(const QuantParams &args, int sms, cudaStream_t stream) {
  // n / d = (mulhi(n, mul) + n) >> shift with shift = ceil(log2 d), mul = floor(2^32 (2^shift - d) / d) + 1
  QuantParams p = args;
  const uint64_t d = uint64_t(qblocks(p.h));
  p.row_shift = 0;
  while ((uint64_t(1) << p.row_shift) < d) ++p.row_shift;
  p.row_mul = uint32_t((uint64_t(1) << 32) * ((uint64_t(1) << p.row_shift) - d) / d + 1);
  const int64_t blocks = int64_t(p.m) * qblocks(p.h);
  const dim3 block(256);
  auto ctas = [&](int per) { return dim3(unsigned((blocks + per - 1) / per)); };
  // Once every SM is full: two fragments a lane, which halves what a block costs
  // beside its values, and 64 bytes under way a lane (swiglu 4096 x 2048: one
  // fragment 11.5 us, two 9.8, four 11.8; quantize 1999 x 5064: 7.9, one pair of
  // fragments 7.5, two 7.35).  Rows that allow it are read 32 bytes at a time.  No
  // loop over a resident grid, whose reads and writes would not overlap (quantize
  // 1999 x 5064: 9.5 us against 8.4).
  if (blocks > (int64_t(1) << 30))
    return launch_pdl(k_quantize<SWIGLU, 1, 2, false, int64_t>, dim3(1 << 22), block, p, stream);
  if (blocks < int64_t(sms) * 128) return launch_pdl(k_quantize<SWIGLU, 1, 1, false, int>, ctas(16), block, p, stream);
  constexpr int U = SWIGLU ? 1 : 2;
  const bool wide = reinterpret_cast<uintptr_t>(p.x) % 32 == 0 && p.x_stride % 16 == 0 && p.h % 16 == 0 &&
                    reinterpret_cast<uintptr_t>(p.values) % 16 == 0;
  if (wide) return launch_pdl(k_quantize<SWIGLU, 2, U, true, int>, ctas(32 * U), block, p, stream);
  return launch_pdl(k_quantize<SWIGLU, 2, U, false, int>, ctas(32 * U), block, p, stream);
}

}  // namespace

cudaError_t launch_quantize(const QuantParams &p, bool swiglu, int sms, cudaStream_t stream) {
  return swiglu ? launch_quantize_as<true>(p, sms, stream) : launch_quantize_as<false>(p, sms, stream);
}

}  // namespace mhc
