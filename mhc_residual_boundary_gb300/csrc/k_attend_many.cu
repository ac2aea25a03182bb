// k_attend_many.cu -- attention of any number of queries a sequence over a paged
// cache, on the tensor cores: prompts, chunks of them, a few proposed tokens, and
// single tokens of more than 16 heads a kv head.
//
// A row of the products is a (query, head of the group): 128 / group queries make a
// tile of up to 128 rows, two tiles (A and B) an item of one sequence and kv head.
// Items read the same keys and values 128 positions at a time (a unit); what no row of
// an item sees is not read.  The call's units form one line, sequence after sequence,
// head after head, item after item, which is divided evenly over one CTA an SM: long
// prompts and few rows over a long cache use every SM alike.  An item that lies in
// several CTAs' parts goes to scratch and is joined (attend_join.cuh).
//
// A CTA's warps:
//  0-3, 4-7  softmax of tile A, of tile B: a thread has a row.  S = Q K^T comes from
//            tensor memory, P = exp(S - m) goes back over it in BF16; the output stays
//            in tensor memory for the whole item and is rescaled only when the running
//            maximum grows by more than 2^8 (the sum of P is held in FP32; see DOWN_BY).
//            At the item's end the thread writes its row.
//  8         copies: queries, keys and values by TMA, page by page
//  9         the products: O_A += P_A V(j), S_A(j + 1), O_B += P_B V(j), S_B(j + 1), so that
//            one tile's softmax runs beside the other's products
//  10, 11    values of units that are hidden from some rows: P is zero there, but zero
//            times an infinity is not.  Infinities and NaN in such units are set to zero
//            before the product, and the rows that do see them are told (poison).  Over
//            an 8-bit cache also values to BF16 (exactly), for the product with P.  Keys are
//            taken as they are, by queries in two 8-bit pieces, which the softmax warps
//            make of their rows.  The scales go to the columns of S and of P.
//
// Bound by the chain S, softmax, P of a tile: two tiles in turn keep the tensor cores at
// work for 2048 of about 3000 clocks a unit (head_dim 128), and an item's ends cost two more
// units' time.  48 heads on 8 of 128: a prompt of 4096 in 178 us (1160 TFLOP/s, 0.60 of a
// library product's rate), 1024 more queries over 16384 positions in 273 us (0.76).  What
// runs once an item, and what few units need, is kept short or apart: instructions that
// are not in the SM's caches cost more than those that are executed.  Few rows over a long
// cache: the same chain with one tile, 8 sequences of 4 queries over up to 32768 positions in
// 62 us, 4.8 TB/s, and 64 single tokens of 32 heads a kv head over up to 8192 in 97 us, 5.5 TB/s.
// Over an 8-bit cache the scales' loads and products come on top of the
// softmax: 3 x 1024 queries of 40 heads on 8 over up to 8000 positions in 306 us, 0.44.
#include <algorithm>
#include <type_traits>

#include "attend_join.cuh"
#include "attention.cuh"
#include "device_common.cuh"
#include "sublayer_tc.cuh"

namespace mhc {
namespace {

constexpr int KEYS = 128;            // positions of a unit
constexpr int ROWS = 128;            // rows of a tile
constexpr int INFOS = 8;             // units whose notes are kept, and segments: no more of them can be under way
constexpr int CUT = 5;               // places that a cut through all rows costs besides EXTRA + 1
constexpr float GROWTH = 8.f;        // log2 of what P may reach over the reference
constexpr int EXTRA = 2;             // places on the line that an item takes besides its units, for its beginning and end

constexpr int TMEM_WARP = 11;        // has the tensor memory: a warp whose threads stay together

__device__ int g_stall_copies;       // test hook: the copying warp issues no copies

template <int D, bool FP8>
struct Many {
  static constexpr int THREADS = 384;
  static constexpr int SLOT = KEYS * 2 * D;             // keys or values of a unit in BF16
  static constexpr int SLOTS = D == 128 ? (FP8 ? 2 : 5) : (FP8 ? 4 : 8);   // of both, 8-bit: of values
  static constexpr int RAW = FP8 ? KEYS * D : 0;        // the same as they are in an 8-bit cache
  static constexpr int RAWS = FP8 ? (D == 128 ? 2 : 4) : 0;    // values to be converted
  static constexpr int KSLOTS = FP8 ? (D == 128 ? 3 : 4) : 0;  // keys
  static constexpr int Q = ROWS * 2 * D;                // a tile's queries
  static constexpr int Q_AT = 0, SLOTS_AT = 2 * Q, RAW_AT = SLOTS_AT + SLOTS * SLOT;
  static constexpr int K_AT = RAW_AT + RAWS * RAW;
  static constexpr int SCALES_AT = K_AT + KSLOTS * RAW; // [INFOS][keys, values][KEYS]
  static constexpr int CONTROL_AT = SCALES_AT + (FP8 ? INFOS * 2 * KEYS * 4 : 0);
  // registers a thread: at the launch, then the softmax warps', the others'
  static constexpr int R_START = 168, R_SOFT = 208, R_REST = 88;
  static_assert(256 * R_SOFT + 128 * R_REST <= THREADS * R_START, "registers of a CTA");
};

// Notes of a unit, which the copying warp writes for the others.
enum : uint32_t {
  LAST = 16,             // of a segment
  STOP = 32              // no unit: the CTA's part is done
};
struct Info {
  uint32_t flags;        // bits X: tile X has rows that see some of it, 2 + X: all rows see all of it
  int key0, end;         // positions [key0, key0 + KEYS), those before `end` there
  uint32_t all_there;    // no page is missing
  uint32_t there[4];     // a bit for each position: its page is there
  uint32_t poison[4];    // positions whose values were set to zero in part
};
// Notes of a segment: units from .. to of an item's.
struct Segment {
  int s, h, token;       // sequence, kv head, first query's row
  int count[2], position;
  int from, to, units;
  int cta0, cta1;        // CTAs that the item lies in
};

// What one item is.  Tiles: X = 0 (A), 1 (B).
struct Item {
  int s, h, block;       // sequence, kv head, block of queries
  int queries, length, query0, blocks;   // the sequence's
  int count[2];          // queries of the tiles
  int position;          // of the first query (may be negative)
  int sink_end, sink_units, first, end, units;   // positions [0, sink_end) and [first, end), in units
  __device__ __forceinline__ int places() const;
  __device__ __forceinline__ int cost(int group) const;
};

// A wait for a phase also passes while the phase before the last one is open, so whoever waits at a
// barrier has to see each of its phases.  Over a BF16 cache keys and values share a ring of slots, but
// not who waits for them: `full` (keys) and `raw_full` (values) go with the units, not with the
// slots.  (By slots, five of them, the third unit's values followed the first one's keys: they counted
// as there when the first two units' values came before those keys.  The product took what was in
// the slot, and the next copy into it, with that one on its way, ended the launch: one of some
// 300000 calls over long caches.)
struct Control {
  uint64_t full[8], empty[8], raw_full[8], raw_empty[8];
  uint64_t info_full[INFOS], info_empty[INFOS], ready[INFOS];
  uint64_t k_full[4], k_empty[4], q_ready[2];   // 8-bit cache
  uint64_t q_full, q_empty, s_full[2], p_ready[2][2], o_full[2], drain;
  Info info[INFOS];
  Segment segment[INFOS];
  uint32_t tmem;
  int abort;
  int issued, k_issued, q_issued;  // copies into the ring (8-bit cache: of values), of keys, of queries
  uint32_t warp_total[16];
  int warp_good[16];
  Item begin;
  int begin_place, bounds[2];
  Join joins[4];         // of the first and last item of the part, either tile
  int join_count, join_flag;
};

static_assert(INFOS <= 8, "keys and values have a barrier for each unit under way");

template <int D, bool FP8>
constexpr int smem_bytes() { return Many<D, FP8>::CONTROL_AT + int(sizeof(Control)); }
static_assert(smem_bytes<128, false>() <= 227 * 1024 && smem_bytes<128, true>() <= 227 * 1024 &&
              smem_bytes<64, false>() <= 227 * 1024 && smem_bytes<64, true>() <= 227 * 1024, "a CTA's shared memory");

// ----------------------------------------------------------------- items
__device__ __forceinline__ void load_sequence(const AttendParams &p, Item &it, int s, bool &bad, bool &bad_start) {
  it.s = s;
  it.length = sequence_length(p, s, bad);
  it.query0 = query_start(p, s, bad_start);
  const int to = query_start(p, s + 1, bad_start);
  bad_start |= to < it.query0;
  it.queries = max(to - it.query0, 0);
  const int per = 2 * p.tile_queries;
  it.blocks = (it.queries + per - 1) / per;
}

__device__ __forceinline__ void load_block(const AttendParams &p, Item &it, int block) {
  const int per = p.tile_queries, i0 = block * 2 * per;
  it.block = block;
  it.count[0] = min(per, it.queries - i0);
  it.count[1] = max(0, min(per, it.queries - i0 - per));
  it.position = it.length - it.queries + i0;
  const int low = p.window && it.position >= p.window ? it.position - p.window + 1 : 0;
  it.first = low >> p.page_shift << p.page_shift;
  it.end = max(0, it.position + it.count[0] + it.count[1]);
  it.sink_end = min(min(p.sinks, low), it.first);
  it.sink_units = (it.sink_end + KEYS - 1) / KEYS;
  it.units = it.end > 0 ? it.sink_units + (it.end - it.first + KEYS - 1) / KEYS : 0;
}

// To the next item with units; false if there is none.
__device__ __forceinline__ bool next_item(const AttendParams &p, Item &it) {
  bool bad = false;
  int block = it.block + 1;
  for (;;) {
    for (; block < it.blocks; ++block) {
      load_block(p, it, block);
      if (it.units > 0) return true;
    }
    block = 0;
    // a sequence whose last block sees nothing has no units
    if (it.blocks > 0 && it.length > 0 && ++it.h < p.kv_heads) continue;
    it.h = 0;
    if (it.s + 1 >= p.sequences) return false;
    load_sequence(p, it, it.s + 1, bad, bad);
    if (it.length == 0) it.blocks = 0;
  }
}

__device__ __forceinline__ int Item::places() const { return units > 0 ? EXTRA + units : 0; }
// Places that a cut inside it costs: by its rows.
__device__ __forceinline__ int Item::cost(int group) const { return EXTRA + 1 + CUT * (count[0] + count[1]) * group / (2 * ROWS); }

struct Unit {
  int key0, end;         // positions [key0, key0 + KEYS), those before `end` there
  bool sink;
};
__device__ __forceinline__ Unit unit_of(const Item &it, int j) {
  Unit u;
  u.sink = j < it.sink_units;
  u.key0 = u.sink ? j * KEYS : it.first + (j - it.sink_units) * KEYS;
  u.end = u.sink ? it.sink_end : it.end;
  return u;
}
// Whether some row of tile X sees something of the unit.
__device__ __forceinline__ bool active(const AttendParams &p, const Item &it, const Unit &u, int X) {
  const int n = it.count[X], from = it.position + X * p.tile_queries, to = from + n - 1;
  return n > 0 && u.key0 <= to && (!p.window || u.key0 < p.sinks || u.key0 + KEYS > from - p.window + 1);
}
// Whether every row of tile X sees all of it.
__device__ __forceinline__ bool whole(const AttendParams &p, const Item &it, const Unit &u, int X) {
  const int from = it.position + X * p.tile_queries, to = from + it.count[X] - 1;
  return u.key0 + KEYS - 1 <= from && u.key0 + KEYS <= u.end &&
         (!p.window || u.key0 >= to - p.window + 1 || u.key0 + KEYS <= p.sinks);
}

struct Ring {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++at == uint32_t(n)) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// Goes through a part's segments: units from .. to of item `it`.  An item's places on
// the line are EXTRA without units, then its units.
struct Segments {
  Item it;
  int at;                // place in the item that the part begins (or goes on) at
  int from, to;
  int left, end;         // places of the part that are left, its end on the line
  __device__ __forceinline__ Segments(const AttendParams &p, const Control &c)
      : it(c.begin), at(c.begin_place), left(c.bounds[1] - c.bounds[0]), end(c.bounds[1]) {
    cut(p);
  }
  __device__ __forceinline__ void cut(const AttendParams &p) {
    while (left > 0) {
      from = max(at - EXTRA, 0);
      to = min(it.units, at - EXTRA + left);
      if (to > from) return;
      advance(p);
    }
  }
  __device__ __forceinline__ void advance(const AttendParams &p) {
    left -= min(left, EXTRA + it.units - at);
    at = 0;
    if (left > 0 && !next_item(p, it)) left = 0;
  }
  __device__ __forceinline__ void next(const AttendParams &p) {
    advance(p);
    cut(p);
  }
  // The item's first place on the line.
  __device__ __forceinline__ int first() const { return end - left - at; }
};

// -------------------------------------------------------------- tensor cores
// BF16 A in tensor memory (K-major), B in shared memory with its columns
// contiguous, FP32 accumulator.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t at, const uint32_t *r);
template <>
__device__ __forceinline__ void tmem_st<16>(uint32_t at, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_st<32>(uint32_t at, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// A warp's registers a thread, drawn on (or given back to) what the CTA started with.
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// (a, b) times a pair; x * f + g; acc + (a, b).
__device__ __forceinline__ void mul_pair(uint32_t &a, uint32_t &b, uint64_t f) {
  asm("{.reg .b64 t;\n\tmov.b64 t, {%0, %1};\n\tmul.rn.f32x2 t, t, %2;\n\tmov.b64 {%0, %1}, t;}" : "+r"(a), "+r"(b) : "l"(f));
}
__device__ __forceinline__ void fma_pair(float &y0, float &y1, uint32_t x0, uint32_t x1, uint64_t f, uint64_t g) {
  asm("{.reg .b64 t;\n\tmov.b64 t, {%2, %3};\n\tfma.rn.f32x2 t, t, %4, %5;\n\tmov.b64 {%0, %1}, t;}"
      : "=f"(y0), "=f"(y1)
      : "r"(x0), "r"(x1), "l"(f), "l"(g));
}
__device__ __forceinline__ void add_pair(uint64_t &acc, float a, float b) {
  asm("{.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tadd.rn.f32x2 %0, %0, t;}" : "+l"(acc) : "f"(a), "f"(b));
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Tensor memory: S (and P over its first half) of A and B, then the outputs.
constexpr uint32_t S_COL(int X) { return X * 128; }
constexpr uint32_t O_COL(int X) { return 256 + X * 128; }

// Instruction descriptors: S = Q K^T, both K-major; O = P V, V's columns contiguous.
constexpr uint32_t IDESC_S = tc::idesc_bf16_f32(ROWS, KEYS), IDESC_S8 = tc::idesc_e4m3_f32(ROWS, KEYS);
template <int D>
constexpr uint32_t idesc_o() { return tc::idesc_bf16_f32(ROWS, D) | 1u << 16; }

// ------------------------------------------------------------------ softmax
// Whether some row of a tile that sees some of a unit does not see all of it.
__device__ __forceinline__ bool hides(uint32_t flags) { return (flags & 3u & ~(flags >> 2)) != 0; }

// lowest n bits
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// The columns of the positions `which` of a unit whose values are not finite: bits of +infinity [0, D / 32) and -infinity [4, 4 + D / 32), NaN both.
template <int D, bool FP8>
__device__ __noinline__ void read_poison(const AttendParams &p, int s, int h, int key0, uint4 which,
                                         uint32_t *bits) {
  const uint32_t words[4] = {which.x, which.y, which.z, which.w};
  for (int w = 0; w < 4; ++w)
    for (uint32_t m = words[w]; m; m &= m - 1) {
      const int key = key0 + w * 32 + __ffs(m) - 1;
      const int page = p.page_table[s * p.table_stride + (key >> p.page_shift)];
      const int64_t at = page * p.values.page_stride +
                         ((int64_t(h) << p.page_shift) + (key & ((1 << p.page_shift) - 1))) * D;
      for (int d = 0; d < D; ++d) {
        const uint32_t v = FP8 ? static_cast<const uint8_t *>(p.values.data)[at + d] : static_cast<const uint16_t *>(p.values.data)[at + d];
        const bool nan = FP8 ? (v & 0x7fu) == 0x7fu : (v & 0x7fffu) > 0x7f80u;
        if (nan || (!FP8 && v == 0x7f80u)) bits[d / 32] |= 1u << d % 32;
        if (nan || (!FP8 && v == 0xff80u)) bits[4 + d / 32] |= 1u << d % 32;
      }
    }
}

// 32 columns of a row of output, 32 bytes at a time: whole sectors of memory, without an
// exchange between the lanes (that, for 64 neighbouring bytes of four lanes, took 214 us
// for the 200 of 4096 queries of 48 heads).  Rows that begin at an odd multiple of 16 bytes take halves.
__device__ __forceinline__ void store32(uint16_t *out, bool whole_sectors, const uint32_t (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 16) {
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = pack_bf16x2(__uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
    if (whole_sectors) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + i), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                   "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                   : "memory");
    } else {
      st_vec(out + i, make_uint4(r[0], r[1], r[2], r[3]));
      st_vec(out + i + 8, make_uint4(r[4], r[5], r[6], r[7]));
    }
  }
}

// A row of queries in two E4M3 pieces, for products with 8-bit keys: y = q 2^(7 - e) with
// the largest |y| in [128, 256) is the sum of y rounded to E4M3 and the rest, which has no
// more than E4M3's four bits either, down to 2^-2; below that the rest is rounded to a
// multiple of 2^-9.  In place: 64 elements of BF16 give their row of 128 bytes to 64 of the
// first piece and 64 of the second.  Returns 2^(e - 7).  A row that is not finite becomes NaN,
// in its pieces and not in the factor: places that it does not see stay hidden.
template <int D>
__device__ __forceinline__ float split_queries(unsigned char *tile, int row) {
  uint32_t top = 0;
#pragma unroll 4
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = *reinterpret_cast<const uint4 *>(tile + i / 8 * ROWS * 128 + row * 128 + i % 8 * 16);
    top = __vmaxu2(__vmaxu2(top, v.x & 0x7fff7fffu), __vmaxu2(__vmaxu2(v.y & 0x7fff7fffu, v.z & 0x7fff7fffu), v.w & 0x7fff7fffu));
  }
  const int e2 = int(max(top >> 16, top & 0xffffu) >> 7);
  const int e = max(e2 - 127, -110);
  const float up = __uint_as_float(uint32_t(127 + 7 - e) << 23);
#pragma unroll 1
  for (int h = 0; h < D / 64; ++h) {
    unsigned char *at = tile + h * ROWS * 128 + row * 128;
    uint32_t hi[16], lo[16];
    const uint32_t nan = e2 == 255 ? 0x7f7f7f7fu : 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = *reinterpret_cast<const uint4 *>(at + ((i ^ (row & 7)) * 16));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        float y[4] = {bf16_lo(w[k]) * up, bf16_hi(w[k]) * up, bf16_lo(w[k + 1]) * up, bf16_hi(w[k + 1]) * up};
        const uint32_t a = e4m3x4(y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          uint32_t f;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(uint16_t(a >> q * 8)));
          float b0, b1;
          asm("{.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;}" : "=f"(b0), "=f"(b1) : "r"(f));
          y[q] -= b0;
          y[q + 1] -= b1;
        }
        hi[i * 2 + k / 2] = a | nan;
        lo[i * 2 + k / 2] = e4m3x4(y[0], y[1], y[2], y[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<uint4 *>(at + ((i ^ (row & 7)) * 16)) = make_uint4(hi[4 * i], hi[4 * i + 1], hi[4 * i + 2], hi[4 * i + 3]);
      *reinterpret_cast<uint4 *>(at + (((4 + i) ^ (row & 7)) * 16)) = make_uint4(lo[4 * i], lo[4 * i + 1], lo[4 * i + 2], lo[4 * i + 3]);
    }
  }
  return __uint_as_float(uint32_t(127 + e - 7) << 23);
}

// How far the maximum of the products may grow; finite, so that minus infinity grows.
__device__ __forceinline__ float slack_of(float scale) { return fminf(GROWTH / scale, 3.4e38f); }

// Over an 8-bit cache P has the value's scale in it, and both ends matter: it stops at BF16's
// 2^-126, and 2^30 positions with values of 2^110 (2^20 with 2^120) have their sum.
template <bool FP8>
constexpr float DOWN_BY = FP8 ? 20.f : DOWN;
template <bool FP8>
constexpr float UP_BY = FP8 ? 1048576.f : UP;
// What is added to x * scale: the reference becomes 2^-DOWN_BY.  As it is rounded it is part of
// what lse is made of.
template <bool FP8>
__device__ __forceinline__ float exponent_base(float top, float scale) { return fmaf(-top, scale, -DOWN_BY<FP8>); }
template <bool FP8>
__device__ __forceinline__ float reference(float top, float scale) { return -(exponent_base<FP8>(top, scale) + DOWN_BY<FP8>); }

template <int D, bool FP8>
__device__ __forceinline__ void softmax_role(const AttendParams &p, unsigned char *smem, Control &c, uint32_t tmem, int X) {
  using F = Many<D, FP8>;
  const int tid = threadIdx.x % 128, warp = tid / 32, lane = tid % 32;
  volatile int *abort = &c.abort;
  const uint32_t lanes = uint32_t(warp * 32) << 16;
  const uint32_t s_at = tmem + S_COL(X) + lanes, o_at = tmem + O_COL(X) + lanes;
  const int group = p.heads / p.kv_heads, query = tid / group, head = tid % group;
  float scale = p.scale_log2, slack = slack_of(scale);   // (8-bit cache: of this row)
  const float *scales = reinterpret_cast<const float *>(smem + F::SCALES_AT);
  uint32_t s_phase = 0, o_phase = 0, q_phase = 0;
  Ring info;
  bool fresh = true;        // a segment's first unit
  uint32_t bits[8];
  bool poisoned = false, any = false;
  float top = -INFINITY, sum = 0.f;

  for (uint32_t segment = 0;;) {
    const Ring my_info = info;
    info.next(INFOS);
    tc::wait_or_abort_inline(&c.info_full[my_info.at], my_info.phase, abort);
    __syncwarp();
    const Info &u = c.info[my_info.at];
    const uint32_t flags = u.flags;
    if (__any_sync(0xffffffffu, *abort) || (flags & STOP)) break;
    const Segment &seg = c.segment[segment % INFOS];
    if (FP8 && fresh) {
      fresh = false;
      if (seg.count[X] > 0) {
        tc::wait_or_abort_inline(&c.q_full, q_phase, abort);
        __syncwarp();
        scale = p.scale_log2 * split_queries<D>(smem + F::Q_AT + X * F::Q, tid);
        // no scale is zero or infinite (minus infinity times zero is not a number)
        scale = fminf(fmaxf(scale, 1.2e-38f), 3.4e38f);
        slack = slack_of(scale);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&c.q_ready[X]);
      }
      q_phase ^= 1u;
    }
    if (flags >> X & 1) {
      tc::wait_or_abort_inline(&c.s_full[X], s_phase, abort);
      s_phase ^= 1u;
      __syncwarp();
      tc::fence_after_sync();
      const float *ks = scales + my_info.at * 2 * KEYS, *vs = ks + KEYS;
      const bool whole = flags >> (2 + X) & 1, masked = !whole || !u.all_there;
      // columns 32 k .. of the unit that this row sees
      const int position = seg.position + X * p.tile_queries + query;
      const int upto = min(position, u.end - 1) - u.key0 + 1;
      const int low = p.window ? position - p.window + 1 - u.key0 : 0, sinks = p.sinks - u.key0;
      auto seen = [&](int k) {
        return u.there[k] & low_bits(upto - 32 * k) & (~low_bits(low - 32 * k) | low_bits(sinks - 32 * k));
      };
      // the row of S, 64 columns on their way while the others are worked on
      uint32_t x[4][32];
      auto hide = [&](int k) {
        const uint32_t w = seen(k);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[k][i] = w >> i & 1 ? x[k][i] : 0xff800000u;   // minus infinity
      };
      // The whole work twice, for units that hide something from some row and for the others:
      // what most units need has to lie together, it is about what the SM's instruction
      // caches hold (with the tests in their places 4096 queries of 48 heads took 189 us for
      // 181 and 3 x 1024 of 40 heads over an 8-bit cache of 8000 positions 420 for 332).
      auto work = [&](auto some) {
      constexpr bool SOME = decltype(some)::value;
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      tc::tmem_ld32_async(s_at, x[0]);
      tc::tmem_ld32_async(s_at + 32, x[1]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t (&v)[32] = x[k];
        if (k % 2 == 0) {
          tc::tmem_wait_ld();
          tc::tmem_hold(x[k]);
          tc::tmem_hold(x[k + 1]);
          if (k == 0) {
            tc::tmem_ld32_async(s_at + 64, x[2]);
            tc::tmem_ld32_async(s_at + 96, x[3]);
          }
        }
        if (FP8) {   // the keys' scales
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(ks + k * 32 + i);
            mul_pair(v[i], v[i + 1], f.x);
            mul_pair(v[i + 2], v[i + 3], f.y);
          }
        }
        if (SOME) hide(k);
        // four chains
#pragma unroll
        for (int i = 0; i < 32; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            m[e] = max3(m[e], __uint_as_float(v[i + 2 * e]), __uint_as_float(v[i + 2 * e + 1]));
      }
      const float now = max3(m[0], m[1], fmaxf(m[2], m[3]));
      // the reference of the exponentials follows the maximum when it has grown far
      const bool grew = now > top + slack;
      const bool first = !any;
      any = true;
      if (__any_sync(0xffffffffu, grew)) {
        const float f = grew ? exp2_fast((top - now) * scale) : 1.f;
        if (grew) top = now;
        sum *= f;
        if (!first) {
          // the product before this one is complete: S of this unit was issued behind it
#pragma unroll 1
          for (int k = 0; k < D; k += 32) {
            uint32_t r[32];
            tc::tmem_ld32_async(o_at + k, r);
            tc::tmem_wait_ld();
            tc::tmem_hold(r);
#pragma unroll
            for (int i = 0; i < 32; i += 2) mul_pair(r[i], r[i + 1], tc::pair(f, f));
            tmem_st<32>(o_at + k, r);
          }
        }
      }
      const float base = top == -INFINITY ? 0.f : exponent_base<FP8>(top, scale);
      const uint64_t scale2 = tc::pair(scale, scale), base2 = tc::pair(base, base);
      uint64_t sums[2] = {0ull, 0ull};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t (&v)[32] = x[k];
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float w[4];
          fma_pair(w[0], w[1], v[2 * i], v[2 * i + 1], scale2, base2);
          fma_pair(w[2], w[3], v[2 * i + 2], v[2 * i + 3], scale2, base2);
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = exp2_fast(w[e]);
          add_pair(sums[0], w[0], w[1]);
          add_pair(sums[1], w[2], w[3]);
          if (FP8) {   // the values' scales
            const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(vs + k * 32 + 2 * i);
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(w[e]);
            mul_pair(u[0], u[1], f.x);
            mul_pair(u[2], u[3], f.y);
            // what is hidden has none
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = SOME && w[e] == 0.f ? 0.f : __uint_as_float(u[e]);
          }
          r[i] = pack_bf16x2(w[0], w[1]);
          r[i + 1] = pack_bf16x2(w[2], w[3]);
        }
        tmem_st<16>(s_at + k * 16, r);
        if (k % 2) {   // half of P is there: its product can begin
          tmem_wait_st();
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&c.p_ready[X][k / 2]);
          __syncwarp();
        }
      }
      sum += (tc::pair_lo(sums[0]) + tc::pair_hi(sums[0])) + (tc::pair_lo(sums[1]) + tc::pair_hi(sums[1]));
      };
      if (!masked) work(std::false_type{});
      else work(std::true_type{});
      if (hides(flags)) {
        // values that were set to zero; P is on its way, so the wait costs little
        tc::wait_or_abort_inline(&c.ready[my_info.at], my_info.phase, abort);
        const volatile uint32_t *q = u.poison;
        const uint4 poison = make_uint4(q[0], q[1], q[2], q[3]);
        if (poison.x | poison.y | poison.z | poison.w) {
          if (!poisoned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) bits[i] = 0;
            poisoned = true;
          }
          if (query < seg.count[X])
            read_poison<D, FP8>(p, seg.s, seg.h, u.key0,
                                make_uint4(poison.x & seen(0), poison.y & seen(1), poison.z & seen(2), poison.w & seen(3)), bits);
        }
        __syncwarp();
      }
    }
    // the notes (and, once its row is written, the segment's) may be written over
    auto release = [&] {
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&c.info_empty[my_info.at]);
    };
    if (!(flags & LAST)) {
      release();
      continue;
    }
    // ---- the segment's end
    ++segment;
    fresh = true;
    const bool had = any, live = query < seg.count[X];
    const float top_now = top, sum_now = sum;
    any = false;
    top = -INFINITY;
    sum = 0.f;
    if (seg.count[X] == 0) {
      release();
      continue;
    }
    if (had) {
      tc::wait_or_abort_inline(&c.o_full[X], o_phase, abort);
      o_phase ^= 1u;
      __syncwarp();
      tc::fence_after_sync();
    }
    const bool item_whole = seg.from == 0 && seg.to == seg.units;
    const int64_t token = seg.token + X * p.tile_queries + query;
    uint16_t *out = p.output + token * p.output_stride + (int64_t(seg.h) * group + head) * D;
    float *lse = p.lse ? p.lse + token * p.heads + seg.h * group + head : nullptr;
    const float inverse = sum_now != 0.f ? 1.f / sum_now : 0.f;
    const int cta0 = seg.cta0, cta1 = seg.cta1;
    float *const part = p.parts + int64_t((2 * blockIdx.x + (int(blockIdx.x) == cta0)) * 2 + X) * part_floats(ROWS, D);
    // Not unrolled, and what is rare is apart: code that runs once an item comes from far,
    // line after line.
    if (item_whole) {
      if (live && !had) {   // saw nothing
#pragma unroll 1
        for (int i = 0; i < D; i += 8) st_vec(out + i, make_uint4(0, 0, 0, 0));
      }
      const uint64_t inverse2 = tc::pair(inverse, inverse);
#pragma unroll (FP8 ? 1 : 2)
      for (int k = 0; had && k < D / 32; ++k) {
        uint32_t v[32];
        __syncwarp();
        tc::tmem_ld32_async(o_at + k * 32, v);
        tc::tmem_wait_ld();
        tc::tmem_hold(v);
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul_pair(v[i], v[i + 1], inverse2);
        if (live) store32(out + k * 32, p.whole_sectors, v);
      }
      if (poisoned && live) {
#pragma unroll 1
        for (int i = 0; i < D; ++i) {
          float x = bf16_lo(out[i]);
          if (bits[0 + i / 32] >> i % 32 & 1) x += INFINITY;
          if (bits[4 + i / 32] >> i % 32 & 1) x -= INFINITY;
          out[i] = uint16_t(pack_bf16x2(x, 0.f));
        }
      }
      if (live && lse) *lse = sum_now != 0.f ? (reference<FP8>(top_now, scale) + log2f(sum_now * UP_BY<FP8>)) * 0.69314718056f : -INFINITY;
      poisoned = false;
      tc::fence_before_sync();
      release();
      continue;
    }
#pragma unroll 1
    for (int k = 0; k < D / 32; ++k) {
      uint32_t v[32];
      __syncwarp();
      tc::tmem_ld32_async(o_at + k * 32, v);
      tc::tmem_wait_ld();
      tc::tmem_hold(v);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        if (live)
          *reinterpret_cast<uint4 *>(part + ((k * 32 + i) * ROWS / 4 + tid) * 4) =
              had ? make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_uint4(0, 0, 0, 0);   // (saw nothing)
    }
    if (poisoned && live) {
#pragma unroll 1
      for (int i = 0; i < D; ++i) {
        float &x = part[(i / 4 * ROWS + tid) * 4 + i % 4];
        if (bits[0 + i / 32] >> i % 32 & 1) x += INFINITY;
        if (bits[4 + i / 32] >> i % 32 & 1) x -= INFINITY;
      }
    }
    poisoned = false;
    tc::fence_before_sync();
    if (live) {
      const float m = top_now != -INFINITY ? reference<FP8>(top_now, scale) : -INFINITY;
      *reinterpret_cast<float4 *>(part + ROWS * D + tid * 4) = make_float4(m, sum_now, m, 0.f);
    }
    // who writes the last part of sixteen joins them, once there is no other work
    __threadfence();
    __syncwarp();
    if (lane == 0) {
      const int join_group = (int(blockIdx.x) - cta0) / JOIN_WIDTH;
      unsigned int *counter = JoinCounters{p.counters + 3 * p.counter_ctas * X, p.counter_ctas}.of_group(cta0, join_group);
      if (atomicAdd(counter, 1u) == unsigned(4 * join_group_size(cta0, cta1, join_group) - 1)) {
        *counter = 0;
        c.joins[atomicAdd(&c.join_count, 1)] = {int(seg.token) + X * p.tile_queries, seg.h, seg.count[X] << 1 | X, cta0, cta1, join_group};
      }
    }
    release();
  }
}

// ------------------------------------------------------------------- copies
template <int D, bool FP8>
__device__ __forceinline__ void load_role(const AttendParams &p, unsigned char *smem, Control &c, const Line &line,
                                          const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v) {
  using F = Many<D, FP8>;
  constexpr int COLS = FP8 ? D : 64, HALVES = FP8 ? 1 : D / 64;   // a box: page rows of COLS values
  const int lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  const int unit_pages = KEYS >> p.page_shift, box = COLS * (FP8 ? 1 : 2) << p.page_shift;
  constexpr int BYTES = FP8 ? F::RAW : F::SLOT;
  Ring ring, k_ring, info;
  uint32_t q_phase = 1;
  int issued = 0, k_issued = 0, q_issued = 0;
  bool ok = !*static_cast<volatile int *>(&g_stall_copies), bad = false;
  // a unit's page numbers, one a lane; -1: not there
  auto look = [&](const Item &it, int j) {
    const Unit u = unit_of(it, j);
    const int key = u.key0 + (lane << p.page_shift);
    if (lane >= unit_pages || key >= u.end) return -1;
    const int page = p.page_table[it.s * p.table_stride + (key >> p.page_shift)];
    const bool there = page >= 0 && page < p.pages;
    bad |= !there;
    return there ? page : -1;
  };
  uint32_t segment = 0;
  for (Segments seg(p, c); seg.left > 0 && ok; seg.next(p), ++segment) {
    const Item &it = seg.it;
    int page = look(it, seg.from);
    // the notes that come next, of a unit and so of a segment, are no longer read
    ok = tc::wait_or_abort(&c.q_empty, q_phase, abort) && tc::wait_or_abort(&c.info_empty[info.at], info.phase ^ 1u, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    q_phase ^= 1u;
    if (lane == 0) {
      Segment &n = c.segment[segment % INFOS];
      n.s = it.s;
      n.h = it.h;
      n.token = it.query0 + it.block * 2 * p.tile_queries;
      n.count[0] = it.count[0];
      n.count[1] = it.count[1];
      n.position = it.position;
      n.from = seg.from;
      n.to = seg.to;
      n.units = it.units;
      if (seg.from > 0 || seg.to < it.units)
        line.owners(seg.first(), it.places(), it.cost(p.heads / p.kv_heads), n.cta0, n.cta1);
    }
    if (lane == 0) {
      const int tiles = it.count[1] > 0 ? 2 : 1;
      const int group = p.heads / p.kv_heads;
      tc::mbar_arrive_expect_tx(&c.q_full, uint32_t(tiles * p.tile_queries * group * 2 * D));
      for (int X = 0; X < tiles; ++X)
        for (int k = 0; k < D / 64; ++k)
          tc::tma_load_3d(smem + F::Q_AT + X * F::Q + k * ROWS * 128, tm_q, k * 64, it.h * group,
                          it.query0 + (it.block * 2 + X) * p.tile_queries, &c.q_full);
    }
    ++q_issued;
    for (int j = seg.from; j < seg.to; ++j) {
      const int next_page = j + 1 < seg.to ? look(it, j + 1) : -1;
      const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
      // places behind the end count as there: rows do not see them
      const Unit u = unit_of(it, j);
      const uint32_t inside = __ballot_sync(0xffffffffu, lane < unit_pages && u.key0 + (lane << p.page_shift) < u.end);
      for (int kv = 0; kv < 2; ++kv) {
        const bool keys = FP8 && kv == 0;   // have a ring of their own
        Ring &at = keys ? k_ring : ring;
        uint64_t *full = FP8 ? (keys ? c.k_full : c.raw_full) + at.at : (kv ? c.raw_full : c.full) + info.at;
        uint64_t *empty = (FP8 ? keys ? c.k_empty : c.raw_empty : c.empty) + at.at;
        ok = tc::wait_or_abort(empty, at.phase ^ 1u, abort) &&
             (kv == 1 || tc::wait_or_abort(&c.info_empty[info.at], info.phase ^ 1u, abort));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (kv == 0) {
          const uint32_t all = there | ~inside;   // a bit for each page
          if (lane < 4) {
            const int at0 = 32 * lane >> p.page_shift, at1 = 32 * lane + 16 >> p.page_shift;
            c.info[info.at].there[lane] = (all >> at0 & 1 ? 0xffffu : 0u) | (all >> at1 & 1 ? 0xffff0000u : 0u);
          }
          __syncwarp();
          if (lane == 0) {
            Info &n = c.info[info.at];
            uint32_t flags = j + 1 == seg.to ? LAST : 0u;
            for (int X = 0; X < 2; ++X)
              flags |= (active(p, it, u, X) ? 1u : 0u) << X | (whole(p, it, u, X) ? 4u : 0u) << X;
            n.flags = flags;
            n.key0 = u.key0;
            n.end = u.end;
            n.all_there = (~all & p.all_pages) == 0;
            n.poison[0] = n.poison[1] = n.poison[2] = n.poison[3] = 0;
            if (FP8) tc::mbar_arrive_expect_tx(&c.info_full[info.at], uint32_t(__popc(there) * 8 << p.page_shift));
            else tc::mbar_arrive(&c.info_full[info.at]);
          }
          __syncwarp();
          if (FP8 && page >= 0) {
            const int64_t from = (int64_t(page) * p.kv_heads + it.h) << p.page_shift;
            float *to = reinterpret_cast<float *>(smem + F::SCALES_AT) + info.at * 2 * KEYS + (lane << p.page_shift);
            tc::bulk_load(to, p.keys.scales + from, 4u << p.page_shift, &c.info_full[info.at]);
            tc::bulk_load(to + KEYS, p.values.scales + from, 4u << p.page_shift, &c.info_full[info.at]);
          }
        }
        if (lane == 0) tc::mbar_arrive_expect_tx(full, uint32_t(BYTES));
        __syncwarp();
        if (lane < unit_pages) {
          unsigned char *to = smem + (FP8 ? keys ? F::K_AT : F::RAW_AT : F::SLOTS_AT) + at.at * BYTES + lane * box;
          for (int k = 0; k < HALVES; ++k)   // a page that is not there: zeros
            tc::tma_load_3d(to + k * KEYS * 128, kv ? tm_v : tm_k, k * 64, it.h << p.page_shift, page, full);
        }
        at.next(FP8 ? keys ? F::KSLOTS : F::RAWS : F::SLOTS);
        if (keys) ++k_issued;
        else ++issued;
      }
      if (!ok) break;
      info.next(INFOS);
      page = next_page;
    }
  }
  // the others end (after a wait that gave up they have seen that as well)
  if (lane == 0) {
    c.issued = issued;
    c.k_issued = k_issued;
    c.q_issued = q_issued;
    if (ok && tc::wait_or_abort(&c.info_empty[info.at], info.phase ^ 1u, abort)) {
      c.info[info.at].flags = STOP;
      tc::mbar_arrive(&c.info_full[info.at]);
    }
  }
  if (bad) atomicOr(p.err, ATTN_ERR_INDEX);
}

// ----------------------------------------------------------------- products
template <int D, bool FP8>
__device__ __forceinline__ void mma_role(unsigned char *smem, Control &c, uint32_t tmem) {
  using F = Many<D, FP8>;
  volatile int *abort = &c.abort;
  // keys: rows of 128 bytes, 64 of them 8-bit ones of 64 elements (in the 64-byte swizzled layout)
  const uint64_t q_desc = tc::desc_sw128(smem + F::Q_AT);
  const uint64_t k_desc = FP8 && D == 64 ? tc::smem_desc(tc::smem_addr(smem + F::K_AT), 16, 512) | uint64_t(4) << 61
                                         : tc::desc_sw128(smem + (FP8 ? F::K_AT : F::SLOTS_AT));
  // values: 64 columns of 8 positions are 1024 bytes, the next 8 positions behind them, the
  // next 64 columns KEYS * 128 bytes on
  const uint64_t v_desc = tc::smem_desc(tc::smem_addr(smem + F::SLOTS_AT), KEYS * 128, 1024) | uint64_t(2) << 61;
  Ring at, info, value, value_info;   // the next unit's keys; the unit before's values
  uint32_t q_phase = 0, p_phase[2] = {0, 0};
  bool ok = true, pending[2] = {false, false}, any[2] = {false, false};
  bool first = true, flush = false;           // a segment's first unit; the step behind its last one
  Ring k_at;
  uint32_t segment = 0, ready_phase[2] = {0, 0};
  while (ok) {
    uint32_t flags = 0;
    if (!flush) {
      ok = tc::wait_or_abort(&c.info_full[info.at], info.phase, abort);
      if (!ok) break;
      flags = c.info[info.at].flags;
      if (flags & STOP) break;
      if (first) {
        if (FP8) {
          const Segment &seg = c.segment[segment++ % INFOS];
          for (int X = 0; X < 2 && ok; ++X)
            if (seg.count[X] > 0) {
              ok = tc::wait_or_abort(&c.q_ready[X], ready_phase[X], abort);
              ready_phase[X] ^= 1u;
            }
        } else {
          ok = tc::wait_or_abort(&c.q_full, q_phase, abort);
          q_phase ^= 1u;
        }
      }
      ok = ok && (FP8 ? tc::wait_or_abort(&c.k_full[k_at.at], k_at.phase, abort) : tc::wait_or_abort(&c.full[info.at], info.phase, abort));
      if (!ok) break;
    }
    if (!first) {
      ok = FP8 ? tc::wait_or_abort(&c.full[value.at], value.phase, abort)
               : tc::wait_or_abort(&c.ready[value_info.at], value_info.phase, abort);
      if (!ok) break;
    }
#pragma unroll
    for (int X = 0; X < 2; ++X) {
      if (pending[X]) {
#pragma unroll
        for (int half = 0; half < 2 && ok; ++half) {
          ok = tc::wait_or_abort(&c.p_ready[X][half], p_phase[X], abort);
          if (!ok) break;
          tc::fence_after_sync();
#pragma unroll
          for (int k = half * 4; k < half * 4 + 4; ++k)
            mma_tmem(tmem + O_COL(X), tmem + S_COL(X) + k * 8, v_desc + value.at * (F::SLOT >> 4) + k * 128, idesc_o<D>(),
                     any[X] || k != 0);
        }
        if (!ok) break;
        p_phase[X] ^= 1u;
        any[X] = true;
        pending[X] = false;
      }
      if (X == 1 && !first) tc::mma_commit(&c.empty[value.at]);
      if (flush) {
        if (any[X]) tc::mma_commit(&c.o_full[X]);
        any[X] = false;
      } else if (flags >> X & 1) {
        tc::fence_after_sync();
        if (FP8) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {   // 32 elements: of 64, of a piece
            const int h = k / 4, piece = k / 2 % 2, half = k % 2;
            tc::mma_e4m3(tmem + S_COL(X), q_desc + X * (F::Q >> 4) + h * (ROWS * 128 >> 4) + piece * 4 + half * 2,
                         k_desc + k_at.at * (F::RAW >> 4) + h * 4 + half * 2, IDESC_S8, k != 0);
          }
        } else
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t step = k / 4 * (ROWS * 128 >> 4) + k % 4 * 2;
          tc::mma_bf16(tmem + S_COL(X), q_desc + X * (F::Q >> 4) + step, k_desc + at.at * (F::SLOT >> 4) + step, IDESC_S, k != 0);
        }
        tc::mma_commit(&c.s_full[X]);
        pending[X] = true;
      }
    }
    if (!ok) break;
    if (!flush) {
      tc::mma_commit(FP8 ? &c.k_empty[k_at.at] : &c.empty[at.at]);
      if (flags & LAST) tc::mma_commit(&c.q_empty);
      if (FP8) k_at.next(F::KSLOTS);
      else at.next(F::SLOTS);
      value = at;
      at.next(F::SLOTS);
      value_info = info;
      info.next(INFOS);
    }
    first = flush;
    flush = !flush && (flags & LAST);
  }
  // no product is in flight when the tensor memory goes
  tc::mma_commit(&c.drain);
  tc::mbar_wait_bounded(&c.drain, 0u, tc::SUB_WAIT_LIMIT);
}

// Whether a BF16 pair holds an infinity or a NaN (in bits 15 and 31).
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }

// Positions of the unit with values that are not finite: those values to zero, the
// positions to `poison`.
template <int D>
__device__ __forceinline__ void clean_values(unsigned char *slot, uint32_t *poison, int thread, int threads) {
#pragma unroll 1
  for (int i0 = thread; i0 < KEYS * (D / 8); i0 += 8 * threads) {
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = reinterpret_cast<const uint4 *>(slot)[i0 + i * threads];
      any |= not_finite2(v.x) | not_finite2(v.y) | not_finite2(v.z) | not_finite2(v.w);
    }
    if (any == 0) continue;
#pragma unroll 1
    for (int i = i0; i < i0 + 8 * threads; i += threads) {
      uint32_t *w = reinterpret_cast<uint32_t *>(slot) + i * 4;
      const int row = i / 8 % KEYS;
      for (int k = 0; k < 4; ++k) {
        const uint32_t bad = not_finite2(w[k]);
        if (bad & 0x8000u) w[k] &= 0xffff0000u;
        if (bad & 0x80000000u) w[k] &= 0x0000ffffu;
        if (bad) atomicOr(poison + row / 32, 1u << row % 32);
      }
    }
  }
}

// Values that some row of a tile does not see (BF16 cache).
template <int D>
__device__ __forceinline__ void clean_role(unsigned char *smem, Control &c) {
  using F = Many<D, false>;
  const int thread = threadIdx.x % 64, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  Ring slot, info;
  for (;;) {
    if (!__all_sync(0xffffffffu, tc::wait_or_abort(&c.info_full[info.at], info.phase, abort))) break;
    const uint32_t flags = c.info[info.at].flags;
    if (flags & STOP) break;
    slot.next(F::SLOTS);
    if (!__all_sync(0xffffffffu, tc::wait_or_abort(&c.raw_full[info.at], info.phase, abort))) break;
    if (hides(flags)) {
      clean_values<D>(smem + F::SLOTS_AT + slot.at * F::SLOT, c.info[info.at].poison, thread, 64);
      tc::fence_proxy_async_smem();
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&c.ready[info.at]);
    slot.next(F::SLOTS);
    info.next(INFOS);
  }
}

// 8-bit values to BF16, two rows a thread; NaN as clean_values.
template <int D>
__device__ __forceinline__ void convert_role(unsigned char *smem, Control &c) {
  using F = Many<D, true>;
  const int thread = threadIdx.x % 64, lane = threadIdx.x % 32;
  volatile int *abort = &c.abort;
  Ring raw, slot, info;
  for (bool ok = true; ok;) {
    if (!__all_sync(0xffffffffu, tc::wait_or_abort(&c.info_full[info.at], info.phase, abort))) break;
    const uint32_t flags = c.info[info.at].flags;
    if (flags & STOP) break;
    const bool hidden = hides(flags);
    ok = __all_sync(0xffffffffu, tc::wait_or_abort(&c.raw_full[raw.at], raw.phase, abort) &&
                                     tc::wait_or_abort(&c.empty[slot.at], slot.phase ^ 1u, abort));
    if (!ok) break;
#pragma unroll 1
    for (int row = thread; row < KEYS; row += 64) {
      const unsigned char *from = smem + F::RAW_AT + raw.at * F::RAW + row * D;
      unsigned char *to = smem + F::SLOTS_AT + slot.at * F::SLOT + row * 128;
      uint32_t bad = 0;
#pragma unroll 2
      for (int i = 0; i < D / 16; ++i) {
        const int chunk = D == 128 ? i ^ (row & 7) : i ^ (row >> 1 & 3);   // as the copies laid them
        const uint4 v = *reinterpret_cast<const uint4 *>(from + chunk * 16);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t h;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(w[k / 2] >> k % 2 * 16)));
          float a, b;
          asm("{.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(h));
          o[k] = pack_bf16x2(a, b);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) bad |= not_finite2(o[k]);
        unsigned char *half = to + i / 4 * KEYS * 128;
        const int c0 = i % 4 * 2;
        *reinterpret_cast<uint4 *>(half + ((c0 ^ (row & 7)) * 16)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4 *>(half + (((c0 + 1) ^ (row & 7)) * 16)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      if (hidden && bad) {   // (rare: apart, and not unrolled)
        atomicOr(c.info[info.at].poison + row / 32, 1u << row % 32);
#pragma unroll 1
        for (int i = 0; i < D / 2; ++i) {
          uint32_t *w = reinterpret_cast<uint32_t *>(to + i / 32 * KEYS * 128) + i % 32;
          const uint32_t b = not_finite2(*w);
          if (b & 0x8000u) *w &= 0xffff0000u;
          if (b & 0x80000000u) *w &= 0x0000ffffu;
        }
      }
    }
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tc::mbar_arrive(&c.full[slot.at]);
      tc::mbar_arrive(&c.ready[info.at]);
      tc::mbar_arrive(&c.raw_empty[raw.at]);
    }
    raw.next(F::RAWS);
    slot.next(F::SLOTS);
    info.next(INFOS);
  }
}

// ------------------------------------------------------------------- kernel
template <int D, bool FP8>
__global__ void __launch_bounds__((Many<D, FP8>::THREADS), 1)
k_attend_many(const AttendParams p, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v) {
  using F = Many<D, FP8>;
  extern __shared__ __align__(1024) unsigned char smem[];
  Control &c = *reinterpret_cast<Control *>(smem + F::CONTROL_AT);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  constexpr int T = F::THREADS;

  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&c.full[i], FP8 ? 2 : 1);
      tc::mbar_init(&c.empty[i], 1);
      tc::mbar_init(&c.raw_full[i], 1);
      tc::mbar_init(&c.raw_empty[i], 2);
    }
    for (int i = 0; i < INFOS; ++i) {
      tc::mbar_init(&c.info_full[i], 1);
      tc::mbar_init(&c.info_empty[i], 8);   // the softmax warps
      tc::mbar_init(&c.ready[i], 2);
    }
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&c.k_full[i], 1);
      tc::mbar_init(&c.k_empty[i], 1);
    }
    for (int X = 0; X < 2; ++X) tc::mbar_init(&c.q_ready[X], 4);
    tc::mbar_init(&c.q_full, 1);
    tc::mbar_init(&c.q_empty, 1);
    for (int X = 0; X < 2; ++X) {
      tc::mbar_init(&c.s_full[X], 1);
      tc::mbar_init(&c.p_ready[X][0], 4);
      tc::mbar_init(&c.p_ready[X][1], 4);
      tc::mbar_init(&c.o_full[X], 1);
    }
    tc::mbar_init(&c.drain, 1);
    tc::mbar_init_fence();
    c.abort = c.issued = c.k_issued = c.q_issued = c.join_count = 0;
  }
  if (warp == TMEM_WARP) tc::tmem_alloc(&c.tmem, 512);
  if (warp == 8 && lane == 0) {
    tc::tma_prefetch_desc(&tm_q);
    tc::tma_prefetch_desc(&tm_k);
    tc::tma_prefetch_desc(&tm_v);
  }
  pdl_wait();
  pdl_launch_dependents();

  // ---- this CTA's part of the line: a thread has `chunk` sequences; those of many
  // blocks are gone through by their warp
  const int chunk = (p.sequences + T - 1) / T;
  bool bad = false, hidden = false;
  int mine = 0, good = p.sequences;   // places, and the first sequence whose starts are no good
  for (int i = 0; i < chunk; ++i) {
    const int s = tid * chunk + i;
    Item it;
    it.blocks = it.queries = it.length = 0;
    bool bad_start = false;
    if (s < good) load_sequence(p, it, s, bad, bad_start);
    if (bad_start) {
      good = s;
      it.blocks = it.queries = 0;
    }
    bad |= bad_start;
    hidden |= it.queries > it.length;   // queries that see nothing
    int units = 0;
    const bool many = it.blocks > 4;
    for (int b = 0; b < it.blocks && !many; ++b) {
      load_block(p, it, b);
      units += it.places();
    }
    for (uint32_t m = __ballot_sync(0xffffffffu, many); m; m &= m - 1) {
      const int from = __ffs(m) - 1;
      Item other;
      other.queries = __shfl_sync(0xffffffffu, it.queries, from);
      other.length = __shfl_sync(0xffffffffu, it.length, from);
      const int blocks = __shfl_sync(0xffffffffu, it.blocks, from);
      int n = 0;
      for (int b = lane; b < blocks; b += 32) {
        load_block(p, other, b);
        n += other.places();
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (lane == from) units = n;
    }
    mine += units * p.kv_heads;
  }
  if (lane == 0) c.warp_good[warp] = p.sequences;
  __syncwarp();
  if (good < p.sequences) atomicMin(&c.warp_good[warp], good);
  // The sequences before the first whose starts are no good follow one another: they have no
  // more queries than the call, and so no more places than the host has allowed.  The others
  // have none; with them the sum may have wrapped, so it is taken again without.
  Line line;
  int upto, sequences;
  bool any_hidden;
  uint32_t tmem;
#pragma unroll 1
  for (bool again = false;; again = true) {
    uint32_t sum = uint32_t(mine), total = 0;   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) c.warp_total[warp] = sum;
    tc::fence_before_sync();
    any_hidden = __syncthreads_or(hidden);
    tc::fence_after_sync();
    tmem = c.tmem;
    sequences = p.sequences;
#pragma unroll 1
    for (int w = 0; w < T / 32; ++w) {
      if (w < warp) sum += c.warp_total[w];
      total += c.warp_total[w];
      sequences = min(sequences, c.warp_good[w]);
    }
    upto = int(sum);
    line.total = int(total);
    if (again || sequences == p.sequences) break;
    if (tid * chunk > sequences) mine = 0;
    __syncthreads();
  }
  line.divide(gridDim.x);
  const int cta = min(int(blockIdx.x), line.grid);
  // warp k finds where this CTA's part begins (0), where it ends (1): the owner of the
  // place tells it what lies before
  const int place0 = line.begin(cta), place1 = line.begin(min(cta + 1, line.grid));
  const int owner0 = __syncthreads_count(upto <= place0), owner1 = __syncthreads_count(upto <= place1);
  if (tid == owner0) c.bounds[0] = upto - mine;
  if (tid == owner1) c.bounds[1] = upto - mine;
  __syncthreads();
  const int place = warp ? place1 : place0;
  if (warp < 2 && place >= line.total) c.bounds[warp] = line.total;
  if (warp < 2 && place < line.total) {
    int rest = place - c.bounds[warp];
    __syncwarp();
    if (lane == 0) c.bounds[warp] = line.total;
    __syncwarp();
    bool seen_before = false;
    // (it ends at the break, unless lengths change under the call)
#pragma unroll 1
    for (int s = (warp ? owner1 : owner0) * chunk; s < p.sequences; ++s) {
      Item it;
      load_sequence(p, it, s, seen_before, seen_before);
      int n = 0;
#pragma unroll 1
      for (int b = lane; b < it.blocks; b += 32) {
        load_block(p, it, b);
        n += it.places();
      }
#pragma unroll
      for (int o = 16; o > 0; o /= 2) n += __shfl_xor_sync(0xffffffffu, n, o);
      if (rest >= n * p.kv_heads) {
        rest -= n * p.kv_heads;
        continue;
      }
      it.h = rest / n;
      rest -= it.h * n;
#pragma unroll 1
      for (int b0 = 0;; b0 += 32) {
        it.units = 0;
        if (b0 + lane < it.blocks) load_block(p, it, b0 + lane);
        const int here = it.places();
        int to = here;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, to, o);
          if (lane >= o) to += v;
        }
        const uint32_t behind = __ballot_sync(0xffffffffu, to > rest);
        if (behind) {
          if (lane == __ffs(behind) - 1) {
            const int first = place - (rest - (to - here));
            const int at = line.cut(place, first, here, it.cost(p.heads / p.kv_heads));
            c.bounds[warp] = at;
            if (warp == 0) {
              c.begin_place = at - first;
              c.begin = it;
            }
          }
          break;
        }
        rest -= __shfl_sync(0xffffffffu, to, 31);
      }
      break;
    }
  }
  __syncthreads();

  // ---- queries before their sequence's first position see nothing
  if (any_hidden) {
    for (int s = blockIdx.x; s < sequences; s += gridDim.x) {
      Item it;
      load_sequence(p, it, s, bad, bad);
      const int n = min(it.queries, it.queries - it.length);
      // (query, 16 bytes of its row), stepped: their product may be more than 2^31
      const int row = p.heads * D / 8;
#pragma unroll 1
      for (int i = tid / row, at = tid % row; i < n;) {
        st_vec(p.output + (it.query0 + i) * p.output_stride + at * 8, make_uint4(0, 0, 0, 0));
        i += T / row;
        at += T % row;
        if (at >= row) {
          at -= row;
          ++i;
        }
      }
      const int64_t first = int64_t(it.query0) * p.heads, count = int64_t(n) * p.heads;
#pragma unroll 1
      for (int64_t i = tid; p.lse && i < count; i += T) p.lse[first + i] = -INFINITY;
    }
  }
  if (bad) atomicOr(p.err, ATTN_ERR_INDEX);

  __syncwarp();   // setmaxnreg is for whole warps
  if (c.bounds[0] < c.bounds[1]) {
    if (warp < 8) {
      registers_up<F::R_SOFT>();
      softmax_role<D, FP8>(p, smem, c, tmem, warp / 4);
    } else {
      registers_down<F::R_REST>();
      if (warp == 8) {
        load_role<D, FP8>(p, smem, c, line, &tm_q, &tm_k, &tm_v);
      } else if (warp == 9) {
        if (tc::elect_one()) mma_role<D, FP8>(smem, c, tmem);
      } else if (FP8) {
        convert_role<D>(smem, c);
      } else {
        clean_role<D>(smem, c);
      }
    }
  }
  // The thread with the products comes apart from the rest of its warp, and __syncwarp() does not
  // bring them together for good (seen by their masks): from here on that warp meets no
  // instruction for whole warps.  The barrier counts threads, and the tensor memory is another
  // warp's.
  __syncwarp();
  tc::fence_before_sync();
  sync_threads_apart();
  tc::fence_after_sync();
  __syncwarp();
  if (warp == TMEM_WARP) tc::tmem_dealloc(c.tmem, 512);
  if (!c.abort && warp < 8) {   // those with the most registers
    const int group = p.heads / p.kv_heads;
#pragma unroll 1
    for (int k = 0; k < c.join_count; ++k) {
      const Join join = c.joins[k];   // s: its first query's row; block: queries and tile
      const int X = join.block & 1;
      join_parts<D>(smem, F::CONTROL_AT, tid, 256, [] { asm volatile("barrier.sync 1, 256;" ::: "memory"); }, join,
                    (join.block >> 1) * group, ROWS, JoinCounters{p.counters + 3 * p.counter_ctas * X, p.counter_ctas},
                    [&](int cta, bool begins) { return p.parts + int64_t((2 * cta + begins) * 2 + X) * part_floats(ROWS, D); },
                    [&](int row, int col, float all, float n, float, const float4 &o) {
                      const int64_t token = join.s + row / group;
                      const int head = join.h * group + row % group;
                      const float f = n != 0.f ? 1.f / n : 0.f;
                      *reinterpret_cast<uint2 *>(p.output + token * p.output_stride + int64_t(head) * D + col) =
                          make_uint2(pack_bf16x2(o.x * f, o.y * f), pack_bf16x2(o.z * f, o.w * f));
                      if (p.lse && col == 0) p.lse[token * p.heads + head] = n != 0.f ? ((all == -INFINITY ? 0.f : all) + log2f(n * UP_BY<FP8>)) * 0.69314718056f : -INFINITY;
                    },
                    &c.join_flag);
    }
  }
  if (tid == 0 && c.abort) {
    atomicOr(p.err, ATTN_ERR_WAIT);
    // copies in flight land before the CTA's shared memory goes
    if (FP8) {
      for (int i = max(0, c.issued - F::RAWS); i < c.issued; ++i)
        tc::mbar_wait_bounded(&c.raw_full[i % max(F::RAWS, 1)], uint32_t(i / max(F::RAWS, 1) & 1), tc::SUB_WAIT_LIMIT);
    } else {   // keys, values, keys, ...
      for (int i = max(0, c.issued - 2 * INFOS); i < c.issued; ++i)
        tc::mbar_wait_bounded(&(i % 2 ? c.raw_full : c.full)[i / 2 % INFOS], uint32_t(i / 2 / INFOS & 1), tc::SUB_WAIT_LIMIT);
    }
    if (FP8)
      for (int i = max(0, c.k_issued - F::KSLOTS); i < c.k_issued; ++i)
        tc::mbar_wait_bounded(&c.k_full[i % max(F::KSLOTS, 1)], uint32_t(i / max(F::KSLOTS, 1) & 1), tc::SUB_WAIT_LIMIT);
    if (c.q_issued > 0) tc::mbar_wait_bounded(&c.q_full, uint32_t(c.q_issued - 1 & 1), tc::SUB_WAIT_LIMIT);
    for (int i = max(0, c.k_issued - INFOS); FP8 && i < c.k_issued; ++i)
      tc::mbar_wait_bounded(&c.info_full[i % INFOS], uint32_t(i / INFOS & 1), tc::SUB_WAIT_LIMIT);
  }
}

// A tensor map of three dimensions (the innermost contiguous) for boxes of them.
bool encode_3d(CUtensorMap *map, CUtensorMapDataType type, const void *base, const uint64_t (&dims)[3],
               const uint64_t (&strides)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swizzle) {
  const auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t d[3] = {dims[0], dims[1], dims[2]}, s[2] = {strides[0], strides[1]};
  const cuuint32_t b[3] = {box[0], box[1], box[2]}, ones[3] = {1, 1, 1};
  return fn(map, type, 3, const_cast<void *>(base), d, s, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8>
cudaError_t launch(const AttendParams &args, int sms, cudaStream_t stream) {
  using F = Many<D, FP8>;
  AttendParams p = args;
  const int group = p.heads / p.kv_heads, page = 1 << p.page_shift;
  p.tile_queries = ROWS / group;
  p.whole_sectors = reinterpret_cast<uintptr_t>(p.output) % 32 == 0 && p.output_stride % 16 == 0;
  p.all_pages = uint32_t((uint64_t(1) << (KEYS >> p.page_shift)) - 1);
  const int size = FP8 ? 1 : 2;
  CUtensorMap tm_q, tm_k, tm_v;
  const auto type = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto swizzle = FP8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  auto cache = [&](CUtensorMap *map, const CacheParams &c) {
    return encode_3d(map, type, c.data, {uint64_t(D), uint64_t(p.kv_heads) * page, uint64_t(p.pages)},
                     {uint64_t(D) * size, uint64_t(c.page_stride) * size}, {FP8 ? uint32_t(D) : 64u, uint32_t(page), 1u}, swizzle);
  };
  if (!encode_3d(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.q, {uint64_t(D), uint64_t(p.heads), uint64_t(p.tokens)},
                 {uint64_t(D) * 2, uint64_t(p.q_stride) * 2}, {64u, uint32_t(group), uint32_t(p.tile_queries)},
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !cache(&tm_k, p.keys) || !cache(&tm_v, p.values))
    return cudaErrorInvalidValue;
  // no more CTAs than there can be units
  int64_t most = int64_t(p.table_width) << p.page_shift;
  if (p.window) most = std::min(most, int64_t(p.window) + p.sinks + 2 * p.tile_queries + 2 * KEYS);
  const int64_t blocks = std::min<int64_t>(p.tokens, p.tokens / (2 * p.tile_queries) + p.sequences);
  const int64_t units = (most + KEYS - 1) / KEYS * blocks * p.kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(std::min<int64_t>(units, sms)));
  cfg.blockDim = dim3(F::THREADS);
  cfg.dynamicSmemBytes = smem_bytes<D, FP8>();
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend_many<D, FP8>, p, tm_q, tm_k, tm_v);
}

template <int D, bool FP8>
cudaError_t allow() {
  using F = Many<D, FP8>;
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, k_attend_many<D, FP8>);
  if (e != cudaSuccess) return e;
  // the warps' shares are drawn on what the CTA starts with: never wait for more
  if (a.numRegs != F::R_START) return cudaErrorInvalidKernelImage;
  return cudaFuncSetAttribute(k_attend_many<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<D, FP8>());
}

}  // namespace

cudaError_t attend_many_setup() {
  cudaError_t e = allow<128, false>();
  if (e == cudaSuccess) e = allow<128, true>();
  if (e == cudaSuccess) e = allow<64, false>();
  if (e == cudaSuccess) e = allow<64, true>();
  return e;
}

cudaError_t attend_stall_copies(int on) { return cudaMemcpyToSymbol(g_stall_copies, &on, sizeof on); }

size_t attend_many_scratch(int sms) { return size_t(4) * sms * part_floats(ROWS, 128) * sizeof(float); }

cudaError_t launch_attend_many(const AttendParams &p, int sms, cudaStream_t stream) {
  if (p.dim == 128) return p.fp8 ? launch<128, true>(p, sms, stream) : launch<128, false>(p, sms, stream);
  return p.fp8 ? launch<64, true>(p, sms, stream) : launch<64, false>(p, sms, stream);
}

}  // namespace mhc
