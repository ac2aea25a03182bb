// k_append_kv.cu -- new tokens' queries and keys rotated by their positions, keys
// and values written to their slots of a paged cache (BF16, or E4M3 with one
// FP32 scale for each position and head).
//
//   pair i of a rotated head: (a, b) -> (a cos w - b sin w, b cos w + a sin w),
//   w = position * f(i)
// The angle in turns is position * (f(i) / 2 pi); only its part behind the point
// matters.  f(i) / 2 pi is held as a 64-bit binary fraction, so the product in 64
// bits, which drops the whole turns, is exact but for the fraction's own last bit
// times the position: 2^-33 turns at positions of 2^31.  Its upper 32 bits, signed,
// give the angle between -pi and pi.
//
// Bound by memory for many tokens: 8192 of 48 + 2 x 8 heads of 128 in BF16 read and write
// 268 MB in 42 us, 6.4 TB/s, over an 8-bit cache 252 MB in 42 us, 6.0 TB/s; by latency for few:
// one token takes 1.6 us.
#include "attention.cuh"
#include "device_common.cuh"
#include "e4m3_scale.h"

namespace mhc {
namespace {

constexpr int APPEND_THREADS = 256;   // at most

// 16 bytes of a row that this thread may write later (q_out may be q).
__device__ __forceinline__ uint4 ld_once(const void *p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 quant8(const float (&y)[8], float inv) {
  return make_uint2(e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                    e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
}

// TOKENS tokens a blockIdx.x; a thread takes 16 elements of one head of each: two 16-byte
// fragments that a rotation pairs.  All are asked for before anything is waited for.
template <int DIM, int TOKENS>
__global__ void __launch_bounds__(APPEND_THREADS, 4) k_append_kv(const AppendParams p) {
  constexpr int UNITS = DIM / 16;   // threads a head
  __shared__ float2 turns[TOKENS][DIM / 2];  // cos, sin; of pair i at (i % 8) UNITS + i / 8: without bank conflicts (with them 45 us for 42)
  __shared__ int32_t slots[TOKENS];
  const int first = blockIdx.x * TOKENS, count = min(TOKENS, p.tokens - first);
  const int item = blockIdx.y * blockDim.x + threadIdx.x;
  const int unit = item % UNITS, row = item / UNITS;
  const int heads = p.q ? p.heads : 0;
  const bool live = row < heads + 2 * p.kv_heads;
  const bool is_q = row < heads, is_v = row >= heads + p.kv_heads;
  const int head = is_q ? row : is_v ? row - heads - p.kv_heads : row - heads;
  // its fragments: those that a rotation pairs, else the next two
  const bool rotated = unit < p.rotary / 16;
  const int fa = rotated && !p.interleaved ? unit : 2 * unit, fb = rotated && !p.interleaved ? unit + p.rotary / 16 : fa + 1;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t x_stride = is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride;
  const uint16_t *x = (is_q ? p.q : is_v ? p.v : p.k) + first * x_stride + int64_t(head) * DIM;
  uint4 va[TOKENS], vb[TOKENS];
#pragma unroll
  for (int n = 0; n < TOKENS; ++n) {
    va[n] = vb[n] = make_uint4(0, 0, 0, 0);
    if (live && n < count) {
      va[n] = ld_once(x + n * x_stride + fa * 8);
      vb[n] = ld_once(x + n * x_stride + fb * 8);
    }
  }
  if (threadIdx.x < count) slots[threadIdx.x] = p.slots[first + threadIdx.x];
  // a warp's threads take the angles of one token
  const int angles = p.rotary / 2;
  for (int job = threadIdx.x / 32; job < (angles + 31) / 32 * TOKENS; job += blockDim.x / 32) {
    const int n = job % TOKENS, i = job / TOKENS * 32 + threadIdx.x % 32;
    if (i < angles && n < count) {
      const uint64_t w = uint64_t(int64_t(p.positions[first + n])) * p.turns[i];
      float s, c;
      sincospif(float(int32_t(w >> 32)) * 0x1p-31f, &s, &c);
      turns[n][i % 8 * UNITS + i / 8] = make_float2(c, s);
    }
  }
  __syncthreads();
  const int64_t rows = int64_t(p.pages) << p.page_shift;
  const CacheParams &cache = is_v ? p.values : p.keys;
#pragma unroll
  for (int n = 0; n < TOKENS; ++n) {
    if (n >= count) break;
    const float2 *turn = turns[n];
    const int token = first + n, slot = slots[n];
    float a[8], b[8];
    unpack8(va[n], a);
    unpack8(vb[n], b);
    if (rotated && !is_v) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 ta = turn[i / 2 * UNITS + unit], tb = turn[(4 + i / 2) * UNITS + unit];
          const float a0 = a[i], b0 = b[i];
          a[i] = a0 * ta.x - a[i + 1] * ta.y;
          a[i + 1] = a[i + 1] * ta.x + a0 * ta.y;
          b[i] = b0 * tb.x - b[i + 1] * tb.y;
          b[i + 1] = b[i + 1] * tb.x + b0 * tb.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 t = turn[i * UNITS + unit];
          const float a0 = a[i];
          a[i] = a0 * t.x - b[i] * t.y;
          b[i] = b[i] * t.x + a0 * t.y;
        }
      }
    }
    if (live && is_q) {
      uint16_t *y = p.q_out + token * p.q_out_stride + int64_t(head) * DIM;
      st_vec(y + fa * 8, pack8(a));
      st_vec(y + fb * 8, pack8(b));
    }
    const bool keep = live && !is_q && slot >= 0 && slot < rows;
    if ((slot < -1 || slot >= rows) && threadIdx.x == 0) atomicOr(p.err, ATTN_ERR_INDEX);
    const int page = slot >> p.page_shift;
    const int64_t in_page = (int64_t(head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
    const int64_t at = page * cache.page_stride + in_page * DIM;
    if (!p.fp8) {
      if (keep) {
        uint16_t *y = static_cast<uint16_t *>(cache.data) + at;
        st_vec(y + fa * 8, pack8(a));
        st_vec(y + fb * 8, pack8(b));
      }
      continue;
    }
    // magnitudes compare as bit patterns: a NaN reaches the scale
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = max(top, max(__float_as_uint(a[i]) & 0x7fffffffu, __float_as_uint(b[i]) & 0x7fffffffu));
#pragma unroll
    for (int o = UNITS / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float amax = __uint_as_float(max(top, uint32_t(127 - 100) << 23));
    const float inv = e4m3_inverse(amax, rcp_fast(e4m3_divisor(amax)));
    if (keep) {
      uint8_t *y = static_cast<uint8_t *>(cache.data) + at;
      *reinterpret_cast<uint2 *>(y + fa * 8) = quant8(a, inv);
      *reinterpret_cast<uint2 *>(y + fb * 8) = quant8(b, inv);
      if (unit == 0) cache.scales[((int64_t(page) * p.kv_heads) << p.page_shift) + in_page] = e4m3_scale(amax);
    }
  }
}

template <int TOKENS>
cudaError_t launch(const AppendParams &p, int splits, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.tokens + TOKENS - 1) / TOKENS, splits);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.dim == 128 ? cudaLaunchKernelEx(&cfg, k_append_kv<128, TOKENS>, p) : cudaLaunchKernelEx(&cfg, k_append_kv<64, TOKENS>, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, int sms, cudaStream_t stream) {
  const int items = ((p.q ? p.heads : 0) + 2 * p.kv_heads) * (p.dim / 16);
  const int splits = (items + APPEND_THREADS - 1) / APPEND_THREADS;
  const int threads = ((items + splits - 1) / splits + 31) / 32 * 32;   // no more than the heads have: with
  // 16 + 2 x 2 heads of 64, 8192 tokens took 15.7 us in CTAs of 256 threads and take 9.3
  // Tokens a CTA, by the 256 threads that there would be for each SM with one: more loads
  // under way and fewer CTAs, against too few CTAs.  With 48 + 2 x 8 heads of 128, in us:
  // 32 tokens 1.58, 1.73 and 2.41 with one, two and four, 608 tokens 4.2, 3.3 and 3.7,
  // 2432 tokens 17.9, 14.7 and 14.2, 8192 tokens 55, 44 and 42.
  const int64_t all = int64_t(p.tokens) * splits * threads / APPEND_THREADS / sms;
  return all < 3 ? launch<1>(p, splits, threads, stream) : all < 24 ? launch<2>(p, splits, threads, stream)
                                                                  : launch<4>(p, splits, threads, stream);
}

}  // namespace mhc
