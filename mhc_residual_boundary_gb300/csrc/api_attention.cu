// api_attention.cu -- host implementation of include/mhc_attention.h: argument
// checks, the handle's scratch, and one kernel launch for each call, each a
// programmatic dependent one, so that a call's setup overlaps the end of the
// kernel before it on the stream.
#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <new>
#include <string>
#include <vector>

#include "attention.cuh"
#include "mhc_attention.h"
#include "mhc_boundary_test.h"

using namespace mhc;

struct mhc_attention {
  mhc_attention_config_t cfg;
  int device = 0;
  int sm_count = 0;
  int page_shift = 0;
  unsigned int *err = nullptr;       // device error word
  uint64_t *turns = nullptr;         // [rotary_dim / 2], see k_append_kv.cu
  unsigned int *counters = nullptr;  // attend's scratch, see AttendParams
  float *parts = nullptr;
  std::string last_error;
};

namespace {

thread_local std::string g_attention_create_error;

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

constexpr size_t MESSAGE = 512;   // bytes of one, at most
mhc_status_t fail(std::string &slot, mhc_status_t status, const char *fmt, ...) {
  char buf[MESSAGE];
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

struct Stride {
  const char *name;
  int64_t stride, width, step;
};

template <size_t N>
mhc_status_t check_strides(std::string &msg, const Stride (&strides)[N]) {
  for (const Stride &s : strides)
    if (s.stride < s.width || s.stride % s.step || s.stride > (int64_t(1) << 40))
      return fail(msg, MHC_ERR_INVALID_ARG, "%s = %lld: at least %lld and a multiple of %lld", s.name,
                  (long long)s.stride, (long long)s.width, (long long)s.step);
  return MHC_OK;
}

// What a tensor of `rows` rows reaches over, in bytes.
struct Range {
  const char *name;
  const void *p;
  int64_t rows, stride, width;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + (rows - 1) * stride + width; }
};

bool meet(const Range &a, const Range &b) { return a.p && b.p && a.begin() < b.end() && b.begin() < a.end(); }

mhc_status_t launched(mhc_attention_t *a, cudaError_t e, const char *what) {
  if (e == cudaSuccess) return MHC_OK;
  return fail(a->last_error, MHC_ERR_CUDA, "%s kernel: %s", what, cudaGetErrorString(e));
}

// The cache's part of a call.
mhc_status_t check_cache(mhc_attention_t *a, int pages, const void *k, int64_t k_stride, const void *v,
                         int64_t v_stride, const float *k_scales, const float *v_scales) {
  std::string &msg = a->last_error;
  const mhc_attention_config_t &c = a->cfg;
  const bool fp8 = (c.flags & MHC_ATTENTION_FP8) != 0;
  if (pages < 1) return fail(msg, MHC_ERR_INVALID_ARG, "pages must be positive");
  if (int64_t(pages) * c.page_size > INT32_MAX) return fail(msg, MHC_ERR_UNSUPPORTED, "more than 2^31 - 1 slots");
  if (!fp8 && (k_scales || v_scales)) return fail(msg, MHC_ERR_INVALID_ARG, "a BF16 cache has no scales");
  const Tensor tensors[] = {{"k_cache", k, 16, true}, {"v_cache", v, 16, true},
                            {"k_scales", k_scales, 16, fp8}, {"v_scales", v_scales, 16, fp8}};
  mhc_status_t st = check_tensors(msg, tensors);
  if (st != MHC_OK) return st;
  const int64_t page = int64_t(c.kv_heads) * c.page_size * c.head_dim;
  const Stride strides[] = {{"k_page_stride", k_stride, page, fp8 ? 16 : 8}, {"v_page_stride", v_stride, page, fp8 ? 16 : 8}};
  return check_strides(msg, strides);
}

// two CTAs an SM at most; two sets of counters (attend_many's tiles)
int counter_ctas(const mhc_attention_t *a) { return 2 * a->sm_count; }
size_t counter_bytes(const mhc_attention_t *a) { return size_t(2) * 3 * counter_ctas(a) * sizeof(unsigned int); }

// f / 2 pi behind the point, in 64 bits: within one of the last of them.  1 / 2 pi is the sum of
// two doubles, off by 2^-110, so a product with less than 2^40 is off by less than 2^-67 (with
// 1 / 2 pi in one double it is off by up to 2^-55 for f = 1 already, 2^-24 turns 2^31 positions on).
constexpr double MOST_FREQUENCY = 0x1p40;
uint64_t turns_of(double f) {
  constexpr double INVERSE = 0x1.45f306dc9c883p-3, REST = -0x1.6b01ec5417056p-57;
  const double t = f * INVERSE, rest = std::fma(f, REST, std::fma(f, INVERSE, -t));
  const double high = std::ldexp(t - std::trunc(t), 64), whole = std::floor(high);   // exact
  const double low = std::floor(high - whole + std::ldexp(rest, 64) + 0.5);
  return uint64_t(__int128(whole)) + uint64_t(int64_t(low));
}

void release(mhc_attention_t *a) {
  if (a->turns) cudaFree(a->turns);
  if (a->counters) cudaFree(a->counters);
  if (a->parts) cudaFree(a->parts);
  if (a->err) cudaFree(a->err);
}

}  // namespace

extern "C" {

mhc_status_t mhc_attention_create(const mhc_attention_config_t *config, int device, mhc_attention_t **out) try {
  std::string &msg = g_attention_create_error;
  msg.clear();
  if (!config || !out) return fail(msg, MHC_ERR_INVALID_ARG, "config and out are required");
  const mhc_attention_config_t &c = *config;
  if (c.flags & ~uint32_t(MHC_ATTENTION_FP8 | MHC_ATTENTION_INTERLEAVED))
    return fail(msg, MHC_ERR_INVALID_ARG, "unknown flag bits 0x%x", c.flags);
  if (c.kv_heads < 1 || c.heads < 1 || c.heads % c.kv_heads)
    return fail(msg, MHC_ERR_INVALID_ARG, "heads must be a positive multiple of kv_heads");
  if (c.kv_heads > 1024 || c.heads / c.kv_heads > 128)
    return fail(msg, MHC_ERR_UNSUPPORTED, "more than 1024 kv_heads or 128 heads for each of them");
  if (c.head_dim != 64 && c.head_dim != 128) return fail(msg, MHC_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
    return fail(msg, MHC_ERR_UNSUPPORTED, "page_size must be 16, 32, 64 or 128");
  if (c.rotary_dim < 0 || c.rotary_dim > c.head_dim || c.rotary_dim % 16)
    return fail(msg, MHC_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim]");
  std::vector<uint64_t> turns(c.rotary_dim / 2);
  if (!c.frequencies && c.rotary_dim && !(c.theta > 0 && std::isfinite(c.theta)))
    return fail(msg, MHC_ERR_INVALID_ARG, "theta must be positive and finite");
  for (int i = 0; i < c.rotary_dim / 2; ++i) {
    const double f = c.frequencies ? c.frequencies[i] : std::pow(c.theta, -2.0 * i / c.rotary_dim);
    if (!(std::fabs(f) < MOST_FREQUENCY))
      return fail(msg, MHC_ERR_INVALID_ARG, "frequency %d is not between -2^40 and 2^40", i);
    turns[i] = turns_of(f);
  }
  int count = 0;
  if (cudaGetDeviceCount(&count) != cudaSuccess || device < 0 || device >= count)
    return fail(msg, MHC_ERR_CUDA, "device %d is not available", device);
  DeviceGuard guard(device);
  std::string message;
  message.reserve(MESSAGE);
  mhc_attention_t *a = new (std::nothrow) mhc_attention();
  if (!a) return fail(msg, MHC_ERR_OOM, "host allocation failed");
  a->last_error.swap(message);   // room for what the calls say: nothing is thrown out of them
  a->cfg = c;
  a->cfg.frequencies = nullptr;
  a->device = device;
  while (1 << a->page_shift < c.page_size) ++a->page_shift;
  cudaError_t e = cudaDeviceGetAttribute(&a->sm_count, cudaDevAttrMultiProcessorCount, device);
  if (e == cudaSuccess) e = cudaMalloc(&a->err, sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemset(a->err, 0, sizeof(unsigned int));
  if (e == cudaSuccess && !turns.empty()) {
    e = cudaMalloc(&a->turns, turns.size() * sizeof(uint64_t));
    if (e == cudaSuccess) e = cudaMemcpy(a->turns, turns.data(), turns.size() * sizeof(uint64_t), cudaMemcpyHostToDevice);
  }
  if (e == cudaSuccess) e = attend_one_setup();
  if (e == cudaSuccess) e = attend_many_setup();
  if (e == cudaSuccess)
    e = cudaMalloc(&a->parts, std::max(attend_one_scratch(a->sm_count), attend_many_scratch(a->sm_count)));
  if (e == cudaSuccess) e = cudaMalloc(&a->counters, counter_bytes(a));
  if (e == cudaSuccess) e = cudaMemset(a->counters, 0, counter_bytes(a));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const mhc_status_t st = e == cudaErrorMemoryAllocation ? MHC_ERR_OOM : MHC_ERR_CUDA;
    cudaGetLastError();
    release(a);
    delete a;
    return fail(msg, st, "create: %s", cudaGetErrorString(e));
  }
  *out = a;
  return MHC_OK;
} catch (const std::bad_alloc &) {
  return MHC_ERR_OOM;
}

mhc_status_t mhc_attention_append(mhc_attention_t *a, const mhc_attention_append_args_t *g, mhc_stream_t stream) {
  if (!a) return MHC_ERR_INVALID_ARG;
  std::string &msg = a->last_error;
  const mhc_attention_config_t &c = a->cfg;
  if (!g) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (g->tokens < 0) return fail(msg, MHC_ERR_INVALID_ARG, "tokens is negative");
  if (g->tokens == 0) return MHC_OK;
  if (!g->q != !g->q_out) return fail(msg, MHC_ERR_INVALID_ARG, "q and q_out go together");
  mhc_status_t st = check_cache(a, g->pages, g->k_cache, g->k_page_stride, g->v_cache, g->v_page_stride, g->k_scales,
                                g->v_scales);
  if (st != MHC_OK) return st;
  const Tensor tensors[] = {{"q", g->q, 16, false}, {"k", g->k, 16, true}, {"v", g->v, 16, true},
                            {"positions", g->positions, 4, true}, {"slots", g->slots, 4, true},
                            {"q_out", g->q_out, 16, false}};
  st = check_tensors(msg, tensors);
  if (st != MHC_OK) return st;
  const int64_t q_row = int64_t(c.heads) * c.head_dim, kv_row = int64_t(c.kv_heads) * c.head_dim;
  const Stride strides[] = {{"k_stride", g->k_stride, kv_row, 8}, {"v_stride", g->v_stride, kv_row, 8},
                            {"q_stride", g->q ? g->q_stride : q_row, q_row, 8},
                            {"q_out_stride", g->q ? g->q_out_stride : q_row, q_row, 8}};
  st = check_strides(msg, strides);
  if (st != MHC_OK) return st;
  if (g->q && !(g->q_out == g->q && g->q_out_stride == g->q_stride)) {
    const Range out = {"q_out", g->q_out, g->tokens, g->q_out_stride * 2, q_row * 2};
    const Range ins[] = {{"q", g->q, g->tokens, g->q_stride * 2, q_row * 2},
                         {"k", g->k, g->tokens, g->k_stride * 2, kv_row * 2},
                         {"v", g->v, g->tokens, g->v_stride * 2, kv_row * 2}};
    for (const Range &in : ins)
      if (meet(out, in)) return fail(msg, MHC_ERR_INVALID_ARG, "q_out reaches over %s (it may be q itself)", in.name);
  }
  DeviceGuard guard(a->device);
  AppendParams p = {};
  p.tokens = g->tokens;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.dim = c.head_dim;
  p.page_shift = a->page_shift;
  p.pages = g->pages;
  p.rotary = c.rotary_dim;
  p.interleaved = (c.flags & MHC_ATTENTION_INTERLEAVED) != 0;
  p.fp8 = (c.flags & MHC_ATTENTION_FP8) != 0;
  p.turns = a->turns;
  p.q = static_cast<const uint16_t *>(g->q);
  p.k = static_cast<const uint16_t *>(g->k);
  p.v = static_cast<const uint16_t *>(g->v);
  p.q_stride = g->q_stride;
  p.k_stride = g->k_stride;
  p.v_stride = g->v_stride;
  p.q_out_stride = g->q_out_stride;
  p.positions = g->positions;
  p.slots = g->slots;
  p.q_out = static_cast<uint16_t *>(g->q_out);
  p.keys = {g->k_cache, g->k_page_stride, g->k_scales};
  p.values = {g->v_cache, g->v_page_stride, g->v_scales};
  p.err = a->err;
  return launched(a, launch_append(p, a->sm_count, reinterpret_cast<cudaStream_t>(stream)), "append");
}

mhc_status_t mhc_attention_attend(mhc_attention_t *a, const mhc_attention_attend_args_t *g, mhc_stream_t stream) {
  if (!a) return MHC_ERR_INVALID_ARG;
  std::string &msg = a->last_error;
  const mhc_attention_config_t &c = a->cfg;
  if (!g) return fail(msg, MHC_ERR_INVALID_ARG, "args is NULL");
  if (g->tokens < 0 || g->sequences < 0) return fail(msg, MHC_ERR_INVALID_ARG, "tokens or sequences is negative");
  if (!g->q_starts && g->tokens != g->sequences)
    return fail(msg, MHC_ERR_INVALID_ARG, "without q_starts every sequence has one token");
  if (g->window < 0 || g->sinks < 0) return fail(msg, MHC_ERR_INVALID_ARG, "window or sinks is negative");
  const float scale_log2 = g->scale * 1.44269504088896340736f;
  if (!(g->scale > 0) || !std::isfinite(scale_log2)) return fail(msg, MHC_ERR_INVALID_ARG, "scale must be positive and finite");
  if (g->tokens == 0 || g->sequences == 0) return MHC_OK;
  if (g->tokens > (1 << 24) || g->sequences > (1 << 20))
    return fail(msg, MHC_ERR_UNSUPPORTED, "more than 2^24 tokens or 2^20 sequences");
  if (g->table_width < 1) return fail(msg, MHC_ERR_INVALID_ARG, "table_width must be positive");
  if (int64_t(g->table_width) * c.page_size > (1 << 30))
    return fail(msg, MHC_ERR_UNSUPPORTED, "a row of the page table holds more than 2^30 positions");
  // places on the kernels' line (attend_join.cuh), of what the call may hold at most
  const bool one = !g->q_starts && c.heads / c.kv_heads <= ATTEND_ONE_GROUP;
  const int64_t positions = int64_t(g->table_width) * c.page_size;
  const int64_t items = one ? g->sequences : g->sequences + g->tokens / (2 * (128 / (c.heads / c.kv_heads)));
  if (items * c.kv_heads > INT32_MAX / (one ? 2 + positions / 64 : 6 + positions / 128))
    return fail(msg, MHC_ERR_UNSUPPORTED, "tokens, sequences, kv_heads and table_width are too large together");
  mhc_status_t st = check_cache(a, g->pages, g->k_cache, g->k_page_stride, g->v_cache, g->v_page_stride, g->k_scales,
                                g->v_scales);
  if (st != MHC_OK) return st;
  const Tensor tensors[] = {{"q", g->q, 16, true}, {"q_starts", g->q_starts, 4, false}, {"lengths", g->lengths, 4, true},
                            {"page_table", g->page_table, 4, true}, {"output", g->output, 16, true},
                            {"lse", g->lse, 4, false}};
  st = check_tensors(msg, tensors);
  if (st != MHC_OK) return st;
  const int64_t row = int64_t(c.heads) * c.head_dim;
  const Stride strides[] = {{"q_stride", g->q_stride, row, 8}, {"output_stride", g->output_stride, row, 8},
                            {"table_stride", g->table_stride, g->table_width, 1}};
  st = check_strides(msg, strides);
  if (st != MHC_OK) return st;
  const Range q = {"q", g->q, g->tokens, g->q_stride * 2, row * 2};
  const Range outs[] = {{"output", g->output, g->tokens, g->output_stride * 2, row * 2},
                        {"lse", g->lse, g->tokens, c.heads * 4, c.heads * 4}};
  for (const Range &o : outs)
    if (meet(o, q)) return fail(msg, MHC_ERR_INVALID_ARG, "%s reaches over q", o.name);
  if (meet(outs[0], outs[1])) return fail(msg, MHC_ERR_INVALID_ARG, "lse reaches over output");
  DeviceGuard guard(a->device);
  AttendParams p = {};
  p.tokens = g->tokens;
  p.sequences = g->sequences;
  p.heads = c.heads;
  p.kv_heads = c.kv_heads;
  p.dim = c.head_dim;
  p.page_shift = a->page_shift;
  p.pages = g->pages;
  p.table_width = g->table_width;
  p.fp8 = (c.flags & MHC_ATTENTION_FP8) != 0;
  p.q = static_cast<const uint16_t *>(g->q);
  p.q_stride = g->q_stride;
  p.output_stride = g->output_stride;
  p.table_stride = g->table_stride;
  p.q_starts = g->q_starts;
  p.lengths = g->lengths;
  p.page_table = g->page_table;
  p.keys = {const_cast<void *>(g->k_cache), g->k_page_stride, const_cast<float *>(g->k_scales)};
  p.values = {const_cast<void *>(g->v_cache), g->v_page_stride, const_cast<float *>(g->v_scales)};
  p.scale_log2 = scale_log2;
  // a window that no sequence fills is none: positions less a window stay in range
  p.window = g->window < positions ? g->window : 0;
  p.sinks = p.window ? int(std::min<int64_t>(g->sinks, positions)) : 0;
  p.output = static_cast<uint16_t *>(g->output);
  p.lse = g->lse;
  p.parts = a->parts;
  p.counters = a->counters;
  p.counter_ctas = counter_ctas(a);
  p.err = a->err;
  const cudaStream_t on = reinterpret_cast<cudaStream_t>(stream);
  return launched(a, one ? launch_attend_one(p, a->sm_count, on) : launch_attend_many(p, a->sm_count, on), "attend");
}

mhc_status_t mhc_attention_check_errors(mhc_attention_t *a) {
  if (!a) return MHC_ERR_INVALID_ARG;
  DeviceGuard guard(a->device);
  unsigned int flag = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&flag, a->err, sizeof flag, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && flag) {
    // a call that gave up leaves its counters half way
    e = cudaMemset(a->err, 0, sizeof flag);
    if (e == cudaSuccess) e = cudaMemset(a->counters, 0, counter_bytes(a));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
  }
  if (e != cudaSuccess) return fail(a->last_error, MHC_ERR_CUDA, "check_errors: %s", cudaGetErrorString(e));
  if (flag & ATTN_ERR_WAIT)
    return fail(a->last_error, MHC_ERR_TIMEOUT,
                "a kernel gave up one of its bounded waits (copies or tensor-core work); its outputs are not valid");
  if (flag & ATTN_ERR_INDEX)
    return fail(a->last_error, MHC_ERR_INVALID_ARG, "a page, slot, length or start was out of range; it was not followed");
  return MHC_OK;
}

mhc_status_t mhc_attention_destroy(mhc_attention_t *a) {
  if (!a) return MHC_OK;
  {
    DeviceGuard guard(a->device);
    release(a);
  }
  delete a;
  return MHC_OK;
}

const char *mhc_attention_last_error(const mhc_attention_t *a) {
  return a ? a->last_error.c_str() : g_attention_create_error.c_str();
}

}  // extern "C"

mhc_status_t mhc_test_stall_attention_copies(int32_t on) {
  return attend_stall_copies(on ? 1 : 0) == cudaSuccess ? MHC_OK : MHC_ERR_CUDA;
}

uint64_t mhc_test_attention_turns(double frequency) { return turns_of(frequency); }
