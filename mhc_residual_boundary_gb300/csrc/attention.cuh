// attention.cuh -- parameter blocks, launchers and shared device steps of the
// attention kernels (internal to the library; the public surface is
// include/mhc_attention.h).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace mhc {

// Bits of the handle's error word.
constexpr unsigned int ATTN_ERR_INDEX = 1;   // a page, slot, length or start was out of range
constexpr unsigned int ATTN_ERR_WAIT = 2;    // a bounded wait gave up

// One cache (keys or values): pages of [kv_heads][page_size][head_dim].
struct CacheParams {
  void *data;
  int64_t page_stride;       // elements
  float *scales;             // [pages][kv_heads][page_size], 8-bit only
};

struct AppendParams {
  int tokens, heads, kv_heads, dim, page_shift, pages;
  int rotary, interleaved, fp8;
  const uint64_t *turns;     // [rotary / 2] turns a position, 64 bits behind the point
  const uint16_t *q, *k, *v; // q may be null
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const int32_t *positions, *slots;
  uint16_t *q_out;
  CacheParams keys, values;
  unsigned int *err;
};

struct AttendParams {
  int tokens, sequences, heads, kv_heads, dim, page_shift, pages, table_width, fp8;
  const uint16_t *q;
  int64_t q_stride, output_stride, table_stride;
  const int32_t *q_starts;   // null: one query a sequence
  const int32_t *lengths, *page_table;
  CacheParams keys, values;
  float scale_log2;          // scale * log2(e)
  int window, sinks;
  uint16_t *output;
  float *lse;                // may be null
  // scratch of the handle: parts of rows that several CTAs work on, and counters of
  // the parts that are there (zero between calls), see attend_join.cuh
  float *parts;
  unsigned int *counters;
  int counter_ctas;          // CTAs that there are counters for
  unsigned int *err;
  // set by the launcher of attend_many
  int tile_queries;          // queries of a tile
  uint32_t all_pages;        // a bit for each page of a unit
  bool whole_sectors;        // rows of output begin at multiples of 32 bytes
};

cudaError_t launch_append(const AppendParams &p, int sms, cudaStream_t stream);

// One query a sequence, up to 16 heads for each kv head.
constexpr int ATTEND_ONE_GROUP = 16;
cudaError_t attend_one_setup();
size_t attend_one_scratch(int sms);   // bytes of parts
cudaError_t launch_attend_one(const AttendParams &p, int sms, cudaStream_t stream);

// Any number of queries a sequence.
cudaError_t attend_many_setup();
size_t attend_many_scratch(int sms);
cudaError_t attend_stall_copies(int on);   // test hook, see include/mhc_boundary_test.h
cudaError_t launch_attend_many(const AttendParams &p, int sms, cudaStream_t stream);

#ifdef __CUDACC__
// A sequence's positions in the cache, within what its row of the table holds.
__device__ __forceinline__ int sequence_length(const AttendParams &p, int s, bool &bad) {
  const int n = p.lengths[s];
  const int64_t most = int64_t(p.table_width) << p.page_shift;
  bad |= n < 0 || n > most;
  return n < 0 ? 0 : n > most ? int(most) : n;
}
// First query of sequence s (s = sequences: the end of the last one's).
__device__ __forceinline__ int query_start(const AttendParams &p, int s, bool &bad) {
  if (!p.q_starts) return s;
  const int n = p.q_starts[s];
  bad |= n < 0 || n > p.tokens;
  return n < 0 ? 0 : n > p.tokens ? p.tokens : n;
}
#endif

}  // namespace mhc
