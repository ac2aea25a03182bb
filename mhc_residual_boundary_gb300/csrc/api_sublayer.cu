// api_sublayer.cu -- host implementation of include/mhc_sublayer.h: argument
// checks, the handle's scratch, and one kernel launch for each call.  All but
// moe's are programmatic dependent launches, so a call's setup overlaps the end
// of the kernel before it on the stream; moe's is a cooperative one (its CTAs
// wait for one another) and begins when that kernel is done.
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <new>
#include <string>
#include <type_traits>

#include "mhc_boundary_test.h"
#include "mhc_sublayer.h"
#include "sublayer.cuh"

using namespace mhc;

struct mhc_sublayer {
  mhc_sublayer_config_t cfg;
  int device = 0;
  int sm_count = 0;
  unsigned int *err = nullptr;       // device error word
  MatmulPlan matmul = {};
  // moe (num_experts > 0): its scratch, in one allocation
  MoeScratch moe = {};
  unsigned char *moe_base = nullptr;
  size_t moe_counter_bytes = 0;      // the counters are its first bytes
  int moe_slots = 0;
  std::string last_error;
};

namespace {

thread_local std::string g_sublayer_create_error;

struct DeviceGuard {
  int prev = -1;
  explicit DeviceGuard(int device) {
    if (cudaGetDevice(&prev) != cudaSuccess) prev = -1;
    if (prev != device) cudaSetDevice(device);
  }
  ~DeviceGuard() {
    int now = -1;
    if (prev >= 0 && cudaGetDevice(&now) == cudaSuccess && now != prev) cudaSetDevice(prev);
  }
};

mhc_status_t fail(std::string &slot, mhc_status_t status, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  slot = buf;
  return status;
}

// One tensor of a call: what is checked before any launch.
struct Tensor {
  const char *name;
  const void *p;
  size_t align;
  bool required;
};

template <size_t N>
mhc_status_t check_tensors(std::string &msg, const Tensor (&tensors)[N]) {
  for (const Tensor &t : tensors) {
    if (!t.p) {
      if (t.required) return fail(msg, MHC_ERR_INVALID_ARG, "%s is NULL", t.name);
    } else if (reinterpret_cast<uintptr_t>(t.p) % t.align) {
      return fail(msg, MHC_ERR_INVALID_ARG, "%s is not %zu-byte aligned", t.name, t.align);
    }
  }
  return MHC_OK;
}

mhc_status_t check_stride(std::string &msg, const char *name, int64_t stride, int64_t width, int64_t step) {
  if (stride < width || stride % step || stride > (int64_t(1) << 40))
    return fail(msg, MHC_ERR_INVALID_ARG, "%s = %lld: at least %lld and a multiple of %lld", name, (long long)stride,
                (long long)width, (long long)step);
  return MHC_OK;
}

// Whether a dense output of `bytes` bytes meets one of `m` rows of an input, `row`
// bytes each and `stride` bytes apart.
bool meets(const void *out, int64_t bytes, const void *in, int64_t row, int64_t stride, int64_t m) {
  const int64_t at = int64_t(reinterpret_cast<uintptr_t>(in) - reinterpret_cast<uintptr_t>(out));
  const int64_t first = at + row > 0 ? 0 : (-at - row) / stride + 1;   // the first row that ends after the output begins
  return first < m && at + first * stride < bytes;
}

mhc_status_t launched(mhc_sublayer_t *s, cudaError_t e, const char *what) {
  if (e == cudaSuccess) return MHC_OK;
  return fail(s->last_error, MHC_ERR_CUDA, "%s kernel: %s", what, cudaGetErrorString(e));
}

mhc_status_t quantize_call(mhc_sublayer_t *s, const mhc_sublayer_quantize_args_t *a, bool swiglu,
                           mhc_stream_t stream) {
  if (!s) return MHC_ERR_INVALID_ARG;
  std::string &msg = s->last_error;
  if (!a) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (a->m < 0) return fail(msg, MHC_ERR_INVALID_ARG, "m is negative");
  if (a->h < 8 || a->h % 8) return fail(msg, MHC_ERR_INVALID_ARG, "h must be a positive multiple of 8");
  if (a->h > (1 << 28)) return fail(msg, MHC_ERR_UNSUPPORTED, "h > 2^28");
  if (a->m == 0) return MHC_OK;
  if (a->output && !swiglu) return fail(msg, MHC_ERR_INVALID_ARG, "quantize has no BF16 output");
  const Tensor tensors[] = {{swiglu ? "gate_up" : "x", a->x, 16, true}, {"output", a->output, 16, false},
                            {"values", a->values, 16, true}, {"scales", a->scales, 4, true}};
  mhc_status_t st = check_tensors(msg, tensors);
  if (st == MHC_OK) st = check_stride(msg, "x_stride", a->x_stride, int64_t(a->h) * (swiglu ? 2 : 1), 8);
  if (st != MHC_OK) return st;
  DeviceGuard guard(s->device);
  QuantParams p = {};
  p.m = a->m;
  p.h = a->h;
  p.x = static_cast<const uint16_t *>(a->x);
  p.x_stride = a->x_stride;
  p.output = static_cast<uint16_t *>(a->output);
  p.values = a->values;
  p.scales = a->scales;
  return launched(s, launch_quantize(p, swiglu, s->sm_count, reinterpret_cast<cudaStream_t>(stream)),
                  swiglu ? "swiglu" : "quantize");
}

// Carves the MoE scratch out of s->moe_base (null: returns its size only).
size_t moe_layout(mhc_sublayer_t *s) {
  const mhc_sublayer_config_t &c = s->cfg;
  const bool fp8 = (c.flags & MHC_SUBLAYER_FP8) != 0;
  const size_t m = c.max_moe_tokens, slots = m * (c.top_k + c.shared_experts);
  const size_t reached = size_t(c.shared_experts) + (size_t(c.num_experts) < m * c.top_k ? size_t(c.num_experts) : m * c.top_k);
  const size_t ib = qblocks(c.intermediate), hb = qblocks(c.hidden);
  size_t off = 0;
  auto take = [&](auto *&p, size_t bytes) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(s->moe_base + off);
    off += (bytes + 255) / 256 * 256;
  };
  MoeScratch &q = s->moe;
  take(q.control, MOE_CONTROL * 4);
  take(q.up_counters, reached * ib * 4);
  take(q.up_done, reached * 4);
  s->moe_counter_bytes = off;
  take(q.logits, m * c.num_experts * 4);
  take(q.x_pieces, fp8 ? 3 * m * c.hidden : 0);
  take(q.x_scale, m * 4);
  take(q.up, MOE_CHUNKS * slots * 2 * ib * QBLOCK * 4);
  unsigned char *act;
  take(act, slots * (fp8 ? 3 : 4) * c.intermediate);
  q.act = act;
  take(q.act_scale, fp8 ? ib * slots * 4 : 0);
  take(q.down, MOE_CHUNKS * slots * hb * QBLOCK * 4);
  s->moe_slots = int(slots);
  return off;
}

void release(mhc_sublayer_t *s) {
  if (s->moe_base) cudaFree(s->moe_base);
  if (s->err) cudaFree(s->err);
}

}  // namespace

extern "C" {

mhc_status_t mhc_sublayer_create(const mhc_sublayer_config_t *config, int device, mhc_sublayer_t **out) {
  std::string &msg = g_sublayer_create_error;
  msg.clear();
  if (!config || !out) return fail(msg, MHC_ERR_INVALID_ARG, "config and out are required");
  const mhc_sublayer_config_t &c = *config;
  if (c.num_experts < 0) return fail(msg, MHC_ERR_INVALID_ARG, "num_experts is negative");
  if (c.flags & ~uint32_t(MHC_SUBLAYER_FP8 | MHC_SUBLAYER_RENORMALIZE | MHC_SUBLAYER_ROUTER_F32))
    return fail(msg, MHC_ERR_INVALID_ARG, "unknown flag bits 0x%x", c.flags);
  if (c.num_experts > 0) {
    const int unit = c.flags & MHC_SUBLAYER_FP8 ? 16 : 8;
    if (c.hidden < unit || c.hidden % unit || c.intermediate < unit || c.intermediate % unit)
      return fail(msg, MHC_ERR_INVALID_ARG, "hidden and intermediate must be positive multiples of %d", unit);
    if (c.hidden > SUB_MAX_HIDDEN || c.intermediate > SUB_MAX_HIDDEN)
      return fail(msg, MHC_ERR_UNSUPPORTED, "hidden or intermediate > %d", SUB_MAX_HIDDEN);
    if (c.num_experts > MOE_EXPERTS_MAX) return fail(msg, MHC_ERR_UNSUPPORTED, "num_experts > %d", MOE_EXPERTS_MAX);
    if (c.shared_experts < 0 || c.shared_experts > MOE_SHARED_MAX)
      return fail(msg, MHC_ERR_INVALID_ARG, "shared_experts must be in [0, %d]", MOE_SHARED_MAX);
    if (c.top_k < 1 || c.top_k > MOE_TOPK_MAX || c.top_k > c.num_experts)
      return fail(msg, MHC_ERR_INVALID_ARG, "top_k must be in [1, %d] and at most num_experts", MOE_TOPK_MAX);
    if (c.max_moe_tokens < 1 || c.max_moe_tokens > MOE_TOKENS_MAX)
      return fail(msg, MHC_ERR_INVALID_ARG, "max_moe_tokens must be in [1, %d]", MOE_TOKENS_MAX);
    if (c.score != MHC_SCORE_SOFTMAX && c.score != MHC_SCORE_SIGMOID)
      return fail(msg, MHC_ERR_INVALID_ARG, "unknown score %d", c.score);
  }
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || device < 0 || device >= count)
    return fail(msg, MHC_ERR_CUDA, "device %d is not available", device);
  DeviceGuard guard(device);
  mhc_sublayer_t *s = new (std::nothrow) mhc_sublayer();
  if (!s) return fail(msg, MHC_ERR_OOM, "host allocation failed");
  s->cfg = c;
  s->device = device;
  cudaError_t e = cudaDeviceGetAttribute(&s->sm_count, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = matmul_setup(s->sm_count, &s->matmul);
  if (e == cudaSuccess) e = cudaMalloc(&s->err, sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemset(s->err, 0, sizeof(unsigned int));
  if (e == cudaSuccess && c.num_experts > 0) {
    e = moe_set_attributes();
    if (e == cudaSuccess) e = cudaMalloc(&s->moe_base, moe_layout(s));
    if (e == cudaSuccess) {
      moe_layout(s);
      e = cudaMemset(s->moe_base, 0, s->moe_counter_bytes);
    }
  }
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const mhc_status_t st = e == cudaErrorMemoryAllocation ? MHC_ERR_OOM : MHC_ERR_CUDA;
    cudaGetLastError();
    release(s);
    delete s;
    return fail(msg, st, "create: %s", cudaGetErrorString(e));
  }
  *out = s;
  return MHC_OK;
}

mhc_status_t mhc_sublayer_add_rms_norm(mhc_sublayer_t *s, const mhc_sublayer_norm_args_t *a, mhc_stream_t stream) {
  if (!s) return MHC_ERR_INVALID_ARG;
  std::string &msg = s->last_error;
  if (!a) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (a->m < 0) return fail(msg, MHC_ERR_INVALID_ARG, "m is negative");
  if (a->h < 8 || a->h % 8) return fail(msg, MHC_ERR_INVALID_ARG, "h must be a positive multiple of 8");
  if (a->h > SUB_MAX_HIDDEN) return fail(msg, MHC_ERR_UNSUPPORTED, "h > %d", SUB_MAX_HIDDEN);
  if (a->m == 0) return MHC_OK;
  if (!a->residual_out && !a->output && !a->values) return fail(msg, MHC_ERR_INVALID_ARG, "no output is given");
  if (a->residual_out && !a->residual) return fail(msg, MHC_ERR_INVALID_ARG, "residual_out needs residual");
  if (!a->values != !a->scales) return fail(msg, MHC_ERR_INVALID_ARG, "values and scales go together");
  const Tensor tensors[] = {{"x", a->x, 16, true}, {"residual", a->residual, 16, false},
                            {"norm_weight", a->norm_weight, 16, true}, {"residual_out", a->residual_out, 16, false},
                            {"output", a->output, 16, false}, {"values", a->values, 16, false},
                            {"scales", a->scales, 4, false}};
  mhc_status_t st = check_tensors(msg, tensors);
  if (st == MHC_OK) st = check_stride(msg, "x_stride", a->x_stride, a->h, 8);
  if (st == MHC_OK && a->residual) st = check_stride(msg, "residual_stride", a->residual_stride, a->h, 8);
  if (st != MHC_OK) return st;
  // A row's block reads its inputs before it writes, and other rows not at all:
  // a BF16 output may take the place of a dense input, row for row, and meet an
  // input in no other way.
  const int64_t m = a->m, h = a->h;
  const struct { const char *name; const void *p; int64_t bytes; bool rows; } outs[] = {
      {"residual_out", a->residual_out, m * h * 2, true}, {"output", a->output, m * h * 2, true},
      {"values", a->values, m * h, false}, {"scales", a->scales, m * qblocks(a->h) * 4, false}};
  const struct { const char *name; const void *p; int64_t stride, m; } ins[] = {
      {"x", a->x, a->x_stride, m}, {"residual", a->residual, a->residual_stride, m}, {"norm_weight", a->norm_weight, h, 1}};
  for (const auto &o : outs)
    for (int i = 0; o.p && i < 3; ++i) {
      if (!ins[i].p || !meets(o.p, o.bytes, ins[i].p, h * 2, ins[i].stride * 2, ins[i].m)) continue;
      if (i < 2 && o.rows && o.p == ins[i].p && (m == 1 || ins[i].stride == h)) continue;
      return fail(msg, MHC_ERR_INVALID_ARG, "%s overlaps %s (only residual_out and output may be a dense x or residual)",
                  o.name, ins[i].name);
    }
  DeviceGuard guard(s->device);
  NormParams p = {};
  p.m = a->m;
  p.h = a->h;
  p.x = static_cast<const uint16_t *>(a->x);
  p.residual = static_cast<const uint16_t *>(a->residual);
  p.weight = static_cast<const uint16_t *>(a->norm_weight);
  p.x_stride = a->x_stride;
  p.residual_stride = a->residual_stride;
  p.eps = a->eps;
  p.residual_out = static_cast<uint16_t *>(a->residual_out);
  p.output = static_cast<uint16_t *>(a->output);
  p.values = a->values;
  p.scales = a->scales;
  return launched(s, launch_add_rms_norm(p, reinterpret_cast<cudaStream_t>(stream)), "norm");
}

mhc_status_t mhc_sublayer_quantize(mhc_sublayer_t *s, const mhc_sublayer_quantize_args_t *a, mhc_stream_t stream) {
  return quantize_call(s, a, false, stream);
}

mhc_status_t mhc_sublayer_swiglu(mhc_sublayer_t *s, const mhc_sublayer_quantize_args_t *a, mhc_stream_t stream) {
  return quantize_call(s, a, true, stream);
}

mhc_status_t mhc_sublayer_matmul(mhc_sublayer_t *s, const mhc_sublayer_matmul_args_t *a, mhc_stream_t stream) {
  if (!s) return MHC_ERR_INVALID_ARG;
  std::string &msg = s->last_error;
  if (!a) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (a->m < 0) return fail(msg, MHC_ERR_INVALID_ARG, "m is negative");
  if (a->n < 1) return fail(msg, MHC_ERR_INVALID_ARG, "n must be positive");
  if (a->k < 16 || a->k % 16) return fail(msg, MHC_ERR_INVALID_ARG, "k must be a positive multiple of 16");
  if (a->m > (1 << 24) || a->n > (1 << 24) || a->k > (1 << 24))
    return fail(msg, MHC_ERR_UNSUPPORTED, "m, n or k > 2^24");
  if (a->m == 0) return MHC_OK;
  if (int64_t((a->m + 127) / 128) * qblocks(a->n) > (1 << 30))
    return fail(msg, MHC_ERR_UNSUPPORTED, "more than 2^30 output tiles");
  const Tensor tensors[] = {{"values", a->values, 16, true}, {"scales", a->scales, 4, true},
                            {"weight", a->weight, 16, true}, {"weight_scales", a->weight_scales, 4, true},
                            {"output", a->output, size_t(a->output_f32 ? 4 : 2), true}};
  mhc_status_t st = check_tensors(msg, tensors);
  if (st == MHC_OK) st = check_stride(msg, "values_stride", a->values_stride, a->k, 16);
  if (st == MHC_OK) st = check_stride(msg, "weight_stride", a->weight_stride, a->k, 16);
  if (st == MHC_OK) st = check_stride(msg, "scales_stride", a->scales_stride, qblocks(a->k), 1);
  if (st == MHC_OK) st = check_stride(msg, "output_stride", a->output_stride, a->n, 1);
  if (st != MHC_OK) return st;
  DeviceGuard guard(s->device);
  MatmulParams p = {};
  p.m = a->m;
  p.n = a->n;
  p.k = a->k;
  p.values = a->values;
  p.values_stride = a->values_stride;
  p.scales = a->scales;
  p.scales_stride = a->scales_stride;
  p.weight = a->weight;
  p.weight_stride = a->weight_stride;
  p.weight_scales = a->weight_scales;
  p.output = a->output;
  p.output_stride = a->output_stride;
  p.output_f32 = a->output_f32 != 0;
  const int64_t row_step = a->output_f32 ? 4 : 8;
  p.vector_out = reinterpret_cast<uintptr_t>(a->output) % 16 == 0 && a->output_stride % row_step == 0;
  p.err = s->err;
  return launched(s, launch_block_matmul(p, s->matmul, reinterpret_cast<cudaStream_t>(stream)), "matmul");
}

mhc_status_t mhc_sublayer_moe(mhc_sublayer_t *s, const mhc_sublayer_moe_args_t *a, mhc_stream_t stream) {
  if (!s) return MHC_ERR_INVALID_ARG;
  std::string &msg = s->last_error;
  const mhc_sublayer_config_t &c = s->cfg;
  if (c.num_experts == 0) return fail(msg, MHC_ERR_UNSUPPORTED, "created without experts");
  if (!a) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (a->m < 1 || a->m > c.max_moe_tokens)
    return fail(msg, MHC_ERR_CAPACITY, "M=%d is outside [1, %d]", a->m, c.max_moe_tokens);
  const bool fp8 = (c.flags & MHC_SUBLAYER_FP8) != 0;
  if (!fp8 && (a->gate_up_scales || a->down_scales))
    return fail(msg, MHC_ERR_INVALID_ARG, "BF16 weights have no scales");
  const Tensor tensors[] = {{"x", a->x, 16, true}, {"router", a->router, 16, true}, {"bias", a->bias, 4, false},
                            {"gate_up", a->gate_up, 16, true}, {"gate_up_scales", a->gate_up_scales, 4, fp8},
                            {"down", a->down, 16, true}, {"down_scales", a->down_scales, 4, fp8},
                            {"output", a->output, 2, true}, {"idx", a->idx, 4, false},
                            {"weights", a->weights, 4, false}};
  const mhc_status_t st = check_tensors(msg, tensors);
  if (st != MHC_OK) return st;
  DeviceGuard guard(s->device);
  MoeParams p = {};
  p.m = a->m;
  p.hidden = c.hidden;
  p.intermediate = c.intermediate;
  p.experts = c.num_experts;
  p.shared = c.shared_experts;
  p.top_k = c.top_k;
  p.fp8 = fp8;
  p.sigmoid = c.score == MHC_SCORE_SIGMOID;
  p.renormalize = (c.flags & MHC_SUBLAYER_RENORMALIZE) != 0;
  p.router_f32 = (c.flags & MHC_SUBLAYER_ROUTER_F32) != 0;
  p.routed_scale = c.routed_scale;
  p.x = static_cast<const uint16_t *>(a->x);
  p.router = a->router;
  p.bias = a->bias;
  p.gate_up = a->gate_up;
  p.down = a->down;
  p.gate_up_scales = a->gate_up_scales;
  p.down_scales = a->down_scales;
  p.output = static_cast<uint16_t *>(a->output);
  p.idx = a->idx;
  p.weights = a->weights;
  p.slots = s->moe_slots;
  p.scratch = s->moe;
  p.err = s->err;
  return launched(s, launch_moe(p, s->sm_count, reinterpret_cast<cudaStream_t>(stream)), "moe");
}

mhc_status_t mhc_sublayer_check_errors(mhc_sublayer_t *s) {
  if (!s) return MHC_ERR_INVALID_ARG;
  DeviceGuard guard(s->device);
  unsigned int flag = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&flag, s->err, sizeof flag, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && flag) {
    // a call that gave up leaves its arrival counters half way
    e = cudaMemset(s->err, 0, sizeof flag);
    if (e == cudaSuccess && s->moe_base) e = cudaMemset(s->moe_base, 0, s->moe_counter_bytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return fail(s->last_error, MHC_ERR_CUDA, "check_errors: %s", cudaGetErrorString(e));
  if (flag & 2u)
    return fail(s->last_error, MHC_ERR_TIMEOUT,
                "a kernel gave up one of its bounded waits (copies or tensor-core work); its outputs are not valid");
  return MHC_OK;
}

mhc_status_t mhc_sublayer_destroy(mhc_sublayer_t *s) {
  if (!s) return MHC_OK;
  {
    DeviceGuard guard(s->device);
    release(s);
  }
  delete s;
  return MHC_OK;
}

const char *mhc_sublayer_last_error(const mhc_sublayer_t *s) {
  return s ? s->last_error.c_str() : g_sublayer_create_error.c_str();
}

}  // extern "C"

mhc_status_t mhc_test_stall_sublayer_copies(int32_t on) {
  cudaError_t e = matmul_stall_copies(on ? 1 : 0);
  if (e == cudaSuccess) e = moe_stall_copies(on ? 1 : 0);
  return e == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

mhc_status_t mhc_test_moe_form(const mhc_sublayer_config_t *config, int32_t m, int32_t sms, mhc_test_moe_form_t *out) {
  if (!config || !out || m < 1 || m > MOE_TOKENS_MAX || sms < 1 || config->hidden < 1 || config->intermediate < 1 ||
      config->top_k < 1 || config->shared_experts < 0)
    return MHC_ERR_INVALID_ARG;
  MoeParams p = {};
  p.m = m;
  p.hidden = config->hidden;
  p.intermediate = config->intermediate;
  p.top_k = config->top_k;
  p.shared = config->shared_experts;
  p.fp8 = (config->flags & MHC_SUBLAYER_FP8) != 0;
  moe_form(p, sms);
  *out = {MOE_SMEM, p.ring_at, p.stages, MOE_STAGE_A + p.b_bytes, MOE_STAGE_A, p.scales_at, MOE_ITEMS, p.scale_blocks};
  return MHC_OK;
}
