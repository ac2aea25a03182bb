// k_attend.cu -- attention over a paged cache, one warp for each (query, head):
// the plain form that is right for every call.
#include "attention.cuh"
#include "device_common.cuh"

namespace mhc {
namespace {

template <int DIM, bool FP8>
__global__ void __launch_bounds__(128) k_attend(const AttendParams p) {
  constexpr int N = DIM / 32;   // elements a lane
  const int lane = threadIdx.x % 32;
  const int64_t item = int64_t(blockIdx.x) * 4 + threadIdx.x / 32;
  pdl_wait();
  pdl_launch_dependents();
  const int token = int(item / p.heads), head = int(item % p.heads), kv = head / (p.heads / p.kv_heads);
  bool bad = false;
  for (int64_t i = item; p.q_starts && i < p.sequences && lane == 0; i += int64_t(gridDim.x) * 4) {
    query_start(p, int(i) + 1, bad);
    if (bad || p.q_starts[i] < 0 || p.q_starts[i] > p.q_starts[i + 1]) atomicOr(p.err, ATTN_ERR_INDEX);
  }
  if (token >= p.tokens) return;
  int s = token, begin = token, end = token + 1;
  if (p.q_starts) {
    // the last sequence that starts at or before the token
    int lo = 0, hi = p.sequences;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (query_start(p, mid, bad) <= token) lo = mid;
      else hi = mid;
    }
    s = lo;
    begin = query_start(p, s, bad);
    end = query_start(p, s + 1, bad);
    if (token < begin || token >= end) return;
  }
  const int length = sequence_length(p, s, bad);
  const int at = length - (end - begin) + token - begin;
  const uint16_t *q = p.q + token * p.q_stride + int64_t(head) * DIM + lane * N;
  float x[N], acc[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = __uint_as_float(uint32_t(q[i]) << 16);
  float top = -INFINITY, sum = 0.f;
  const int first = p.window && at >= p.window ? at - p.window + 1 : 0, sinks = min(p.sinks, first);
  for (int i = 0; i < sinks + at + 1 - first; ++i) {
    const int j = i < sinks ? i : i - sinks + first;
    const int page = p.page_table[s * p.table_stride + (j >> p.page_shift)];
    if (page < 0 || page >= p.pages) {
      bad = true;
      continue;
    }
    const int64_t in_page = (int64_t(kv) << p.page_shift) + (j & ((1 << p.page_shift) - 1));
    const int64_t ks = page * p.keys.page_stride + in_page * DIM + lane * N;
    const int64_t vs = page * p.values.page_stride + in_page * DIM + lane * N;
    float k[N], v[N];
    if (FP8) {
      const int64_t scale = ((int64_t(page) * p.kv_heads) << p.page_shift) + in_page;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        uint32_t w;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(w) : "h"(uint16_t(static_cast<const uint8_t *>(p.keys.data)[ks + e] | static_cast<const uint8_t *>(p.values.data)[vs + e] << 8)));
        asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(k[e]), "=f"(v[e]) : "r"(w));
        k[e] *= p.keys.scales[scale];
        v[e] *= p.values.scales[scale];
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        k[e] = __uint_as_float(uint32_t(static_cast<const uint16_t *>(p.keys.data)[ks + e]) << 16);
        v[e] = __uint_as_float(uint32_t(static_cast<const uint16_t *>(p.values.data)[vs + e]) << 16);
      }
    }
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) d = fmaf(x[e], k[e], d);
    d = warp_sum(d) * p.scale_log2;
    const float now = fmaxf(top, d) == -INFINITY ? 0.f : isnan(d) ? d : fmaxf(top, d);
    const float keep = exp2f(top - now), w = exp2f(d - now);
    top = isnan(d) ? d : fmaxf(top, d);
    sum = sum * keep + w;
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = acc[e] * keep + w * v[e];
  }
  uint16_t *out = p.output + token * p.output_stride + int64_t(head) * DIM + lane * N;
#pragma unroll
  for (int e = 0; e < N; ++e) out[e] = uint16_t(pack_bf16x2(sum != 0.f ? acc[e] / sum : 0.f, 0.f));
  if (lane == 0 && p.lse) p.lse[int64_t(token) * p.heads + head] = sum != 0.f ? (top + log2f(sum)) * 0.69314718056f : -INFINITY;
  if (bad && lane == 0) atomicOr(p.err, ATTN_ERR_INDEX);
}

}  // namespace

cudaError_t launch_attend(const AttendParams &p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((int64_t(p.tokens) * p.heads + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.dim == 128)
    return p.fp8 ? cudaLaunchKernelEx(&cfg, k_attend<128, true>, p) : cudaLaunchKernelEx(&cfg, k_attend<128, false>, p);
  return p.fp8 ? cudaLaunchKernelEx(&cfg, k_attend<64, true>, p) : cudaLaunchKernelEx(&cfg, k_attend<64, false>, p);
}

}  // namespace mhc
