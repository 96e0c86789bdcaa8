// fq_attention.cu -- attention of one new token per sequence over a paged FP8 key-value cache, the work
// split over the caches' length and joined.
//
// Mathematics. For a query head with codes q, key rows k_j and value rows v_j (codes), in base 2:
//   x_j = (q . k_j) * (q_scale * softmax_scale * log2 e * k_scale_j),  m = max x,  l = sum 2^(x_j - m),
//   out = (sum 2^(x_j - m) v_scale_j v_j) / l,  lse = (m + log2 l) * ln 2.
// One pass with running m and l. The value sum has a running reference of its own, M = max (x_j + log2
// v_scale_j) - 7, so its weights 2^(x_j + log2 v_scale_j - M) fit fp16 for the tensor cores whatever the scales of
// the rows are, and partial results (m, l, M, O) join exactly: out = O * 2^(M - m) / l. The 7 uses fp16's range to
// the end: the largest weight is 2^7 when M is set and may grow to 2^15 before M follows (below), and weights are
// rounded by 2^-11 of themselves, or 2^-32 of the largest. (fp16 because it halves the value product's operands and
// rounds 128 times finer than the 8-bit codes it multiplies; sums stay in fp32.)
//
// What bounds it: up to 16 query heads per key head, every key and value byte is read once and used Hq/Hk times, so HBM;
// above 16, each 16 of them are a work item that reads its key head's cache again, and the instructions do (64 sequences
// of up to 8192 tokens, 128 query heads of 128: 146 us on 4, 2 or 1 key heads alike). The products are
// legacy-shape warp matrix instructions on purpose: eight query heads of a key head fill the 8 columns of m16n8k16
// with tokens (scores) or output columns (values) on the 16 rows, and the codes become fp16, exactly, on their way
// into the fragments; tcgen05 would need the value tile transposed through shared memory and 128 rows to fill.
// (mma.sync takes e4m3 as well, but here that costs more than converting: the conversions of both operands at each
// use showed as 246 ALU instructions per step of 16 tokens at head size 256, 51 us against what it is now.)
//
// Layout. Units of 128 tokens (64 and 32 for the larger items) stream through a ring of stages: a producer warp
// brings one TMA box of the rows of a page at a time where the page is a multiple of 8 tokens and such boxes hold 1 KB
// (heads of up to 64: a multiple of 16 tokens), else two producer warps copy row by row with 16-byte cp.async. Both products contract over an index whose order is free as long as both
// operands agree: thread (g, c) = (lane / 4, lane % 4) reads pieces 2c and 2c + 1 of key rows g and g + 8 as the k
// indices of its A fragments (scores: tokens x heads), and piece g of value rows 2c, 2c + 1, 2c + 8, 2c + 9 as A
// fragments of the value product (columns x heads). Pieces are stored at (piece ^ row % 8), the 128-byte swizzle,
// which puts the eight lanes of every 16-byte access phase in different banks for both readings. The weights go from
// accumulators to B fragments by two movmatrix.
//
// The running maxima are only brought up to date when a score exceeds one by more than 2^8 (a vote; then three
// shuffles per head and the rescaling): weights of up to 2^8, and 2^15 for the values, lose nothing in fp32 and fp16.
//
// Split. The work is a list of units in the order sequence, head, tokens, and behind each head one place more, which
// stands for the time its end takes (the warps' results are joined and written: about as long as a unit, 1.2 us; a
// batch with many short sequences was held up by the CTAs that had them). The n CTAs take equal ranges of places. The
// lengths are on the device, so each CTA finds its range itself. A run of units of one head that is not the whole head
// goes to the workspace as a partial result, at most two per CTA (its first and its last), and a second kernel joins
// them in order: no atomics, and the same bits on every run.
#include <math_constants.h>

#include "fq_device.cuh"
#include "fq_serving.h"
#include "fq_sync.cuh"
#include "fq_tensormap.h"

namespace fq {
namespace {

constexpr int kWarps = 8;                     // consumer warps
constexpr int kConsumers = kWarps * 32;
constexpr int kProducers = 2;                 // producer warps
constexpr int kThreads = kConsumers + 32 * kProducers;
constexpr int kStep = 16;                     // tokens of one warp per unit
constexpr int kHeads = 8;                     // query heads of one warp

// A work item is one key head with kHeads * HG of its query heads. The consumer warps are slabs (16 tokens of
// a unit each) x HG groups of heads x CG groups of 128 output columns; the column groups of a slab and head
// group all take its score product, which is the smaller one, so that a thread never holds more than
// 32 output accumulators and two CTAs fit an SM at every head size.
template <int DP, int HG>
struct Item {
  static constexpr int CG = DP > 128 ? 2 : 1;
  static constexpr int kSlabs = kWarps / (HG * CG);
  static constexpr int kUnit = kStep * kSlabs;    // tokens per unit
  static constexpr int kRows = kHeads * HG;       // query heads
  // Ring depth: what two CTAs per SM leave room for beside the scales (heavy at head size 64) and the query fragments
  // of the largest items.
  static constexpr int kStages = (DP == 64 ? 80 : DP > 128 && HG == 2 ? 88 : 98) * 1024 / (2 * kUnit * DP);
};
constexpr float kSlack = 8.f;                // powers of two by which a score may exceed its running maximum
constexpr float kRoom = 7.f;                 // powers of two of the largest value weight when M is set; 2^(7 + 8) fits fp16
constexpr float kUnroom = 0.0078125f;        // 2^-kRoom
constexpr float kLowest = -3.402823466e38f;  // below every score: a maximum before the first token

// A unit's rows are stored as kA tiles of [rows][128 bytes], then kB of [rows][64], keys before values.
template <int DP>
struct Shape {
  static constexpr int kA = DP / 128;
  static constexpr int kB = (DP % 128) / 64;
};

// Where 16-byte piece `piece` of row `row` sits in a tile of 128-byte (64-byte) rows.
__device__ __forceinline__ int spot128(int row, int piece) { return row * 128 + ((piece ^ (row & 7)) << 4); }
__device__ __forceinline__ int spot64(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

constexpr int kJoinStride = 36;  // floats per joined row of 32: float4 stores without bank conflicts

template <int DP, int HG>
struct Shared {
  static constexpr int kStages = Item<DP, HG>::kStages;
  static constexpr int kUnit = Item<DP, HG>::kUnit;
  alignas(1024) unsigned char codes[kStages][2][kUnit * DP];  // K then V
  alignas(16) float scales[kStages][2][kUnit];  // K then V
  uint16_t live[kStages][Item<DP, HG>::kSlabs];  // bit t of a slab's word: its token t counts
  alignas(16) float join[kWarps][kHeads][kJoinStride];
  // Above head size 128 the query fragments are read from here at each use: in registers they spill.
  uint4 query[DP > 128 ? HG : 1][DP > 128 ? DP / 32 : 1][32];
  float stat[kWarps][kHeads][3];  // m, M, l
  alignas(8) uint64_t full[kStages];
  uint64_t empty[kStages];
  int64_t scan[kThreads / 32];
  int32_t start_b, start_item, start_tile;  // where this CTA's first unit is
  int32_t before_begin, before_end;         // units before its first place and before the next CTA's
};

// What a CTA that begins inside a head leaves for the join of that head: the CTAs that have its first and last part,
// and which partial result of the first one's it is. b < 0: this CTA begins with a head.
struct alignas(16) Meta {
  int32_t b, item, first, last, slot;
};

struct SplitArgs {
  PagedArgs p;
  int32_t G;       // query heads per key head
  int32_t chunks;  // work items per key head
  int32_t slots;   // 2 * the first kernel's grid
  uint32_t page_magic;  // t / page_size = (t * page_magic) >> page_magic_shift for t < 2^31
  int32_t page_magic_shift;
  unsigned int* status;
  int32_t dtype;
  int32_t box_shift;    // TMA feed: log2 of the rows per box, which divide a page and a unit
  int32_t bulk_scales;  // TMA feed: the scales of a box are contiguous and 16-byte aligned
  Meta* meta;      // [grid]
  float* stats;    // [slots][rows of an item][4]: m, M, l
  float* part;     // [slots][rows of an item][DP]
};

// TMA feed: maps of the keys' and values' 128-byte and 64-byte pieces of a row ({D, slot, head, page}).
struct Maps {
  CUtensorMap k128, v128, k64, v64;
};

__device__ __forceinline__ int32_t length_of(const PagedArgs& p, int32_t b) {
  return max(0, min(p.lens[b], p.max_len));
}

// The tokens of a sequence that take part, [0, sunk) and [start, len), and the tiles that hold them: the first `low`, then
// all behind a gap of `skip` whole ones. Without a window, all of them.
template <int DP, int HG, bool kWindow>
struct Span {
  static constexpr int kUnit = Item<DP, HG>::kUnit;
  int32_t start = 0, sunk = 0, low = 0, skip = 0, tiles;

  __device__ __forceinline__ Span(const PagedArgs& p, int32_t len) {
    tiles = (len + kUnit - 1) / kUnit;
    if constexpr (kWindow) {
      start = max(len - p.window, 0);
      sunk = min(p.sinks, start);
      low = (sunk + kUnit - 1) / kUnit;
      skip = max(start / kUnit - low, 0);
      tiles -= skip;
    }
  }
  // First token of the k-th tile.
  __device__ __forceinline__ int32_t base(int32_t k) const { return (kWindow && k >= low ? k + skip : k) * kUnit; }
  __device__ __forceinline__ bool sees(int32_t t) const { return !kWindow || t < sunk || t >= start; }
};

template <int DP, int HG, bool kWindow>
__device__ __forceinline__ int32_t tiles_of(const PagedArgs& p, int32_t len) {
  return Span<DP, HG, kWindow>(p, len).tiles;
}

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// With subnormal results and arguments, for V scales at the lower end of fp32.
__device__ __forceinline__ float ex2_all(float v) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float lg2_all(float v) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// What turns a sum of weighted values into the output, 2^(M - m) / l, as factors 2^(M + 7 - m) and 2^-7 / l: their product
// may leave fp32's normal range where the output does not.
struct Norm {
  float scale, inv;
  __device__ __forceinline__ float operator()(float v) const { return v * inv * scale; }
  __device__ __forceinline__ float2 operator()(float2 v) const { return mul2(mul2(v, splat2(inv)), splat2(scale)); }
};

__device__ __forceinline__ Norm norm_of(float top, float topo, float l) {
  return l == 0.f ? Norm{0.f, 0.f} : Norm{ex2_all(topo + kRoom - top), kUnroom / l};
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory, or zeros (and nothing read) where `live` is false; 4 bytes.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// e4m3 codes at the same byte of two words (tokens t, t+1) -> the fp16 pair of a B fragment; exact.
__device__ __forceinline__ void pair_f16(uint32_t t0, uint32_t t1, uint32_t (&r)[4]) {
  const uint32_t lo = __byte_perm(t0, t1, 0x5140), hi = __byte_perm(t0, t1, 0x7362);
  asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(r[0]), "=r"(r[1])
      : "r"(lo));
  asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(r[2]), "=r"(r[3])
      : "r"(hi));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int k) {
  return k == 0 ? v.x : (k == 1 ? v.y : (k == 2 ? v.z : v.w));
}

// Four codes of a word -> two fp16 pairs; exact.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 p, q;\n\tmov.b32 {p, q}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, p;\n\tcvt.rn.f16x2.e4m3x2 %1, q;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// An 8 x 8 matrix of 16-bit values, two of a row per thread, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// The largest v of the eight lanes with the same lane % 4.
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A place in the list of units: a work item of sequence b (key head item / chunks, and the item % chunks-th
// part of its query heads) with `left` tiles to go, `len` tokens in all.
template <int DP, int HG, bool kWindow>
struct Place {
  int32_t b, item, len, left;

  // To the next head; `left` is its number of tiles.
  __device__ __forceinline__ void next_head(const SplitArgs& a) {
    if (++item == a.p.Hk * a.chunks) {
      item = 0;
      len = 0;
      while (len == 0 && ++b < a.p.B) len = length_of(a.p, b);
    }
    left = tiles_of<DP, HG, kWindow>(a.p, len);
  }
};

// The places of `total` that each of n CTAs takes: the first `rest` take each + 1, the others `each`.
struct Share {
  int32_t each, rest;
  __device__ __forceinline__ Share(int32_t total, int32_t n) : each(total / n), rest(total - total / n * n) {}
  __device__ __forceinline__ int32_t begin(int32_t cta) const { return cta * each + min(cta, rest); }
  __device__ __forceinline__ int32_t owner(int32_t place) const {
    const int32_t wide = rest * (each + 1);
    return place < wide ? place / (each + 1) : rest + (place - wide) / each;
  }
};

// The block's inclusive sum of v over its threads.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scan, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = v;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  *total = all;
  return v + before;
}

// What a sequence adds to the list: its units in the high half, its places in the low half. Sums of a whole batch fit
// 31 bits each.
template <int DP, int HG, bool kWindow>
__device__ __forceinline__ int64_t extent_of(const SplitArgs& a, int32_t b) {
  const int32_t tiles = b < a.p.B ? tiles_of<DP, HG, kWindow>(a.p, length_of(a.p, b)) : 0, heads = a.p.Hk * a.chunks;
  return tiles == 0 ? 0 : (static_cast<int64_t>(tiles * heads) << 32) + (tiles + 1) * heads;
}

__device__ __forceinline__ int32_t units_in(int64_t extent) { return static_cast<int32_t>(extent >> 32); }
__device__ __forceinline__ int32_t places_in(int64_t extent) { return static_cast<int32_t>(extent & 0xffffffffll); }

// Sequences without tokens get zeros and -inf, spread over the CTAs; by `threads` threads of each.
__device__ __forceinline__ void write_empty(const PagedArgs& p, int threads) {
  for (int32_t b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (length_of(p, b) != 0) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + static_cast<int64_t>(b) * p.Hq * p.D);
    for (int32_t i = threadIdx.x; i < p.Hq * p.D / 8; i += threads) o[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr)
      for (int32_t h = threadIdx.x; h < p.Hq; h += threads) p.lse[static_cast<int64_t>(b) * p.Hq + h] = -CUDART_INF_F;
  }
}

// A producer warp, any page size and layout of scales: copies its share (tokens kTok * half ..) of the units
// from the one at `at` into the ring, 16 bytes a lane: lane (row, piece) copies the same piece of the key and of
// the value row.
template <int DP, int HG, bool kWindow>
__device__ __forceinline__ void produce_rows(const SplitArgs& a, Shared<DP, HG>& sm, Place<DP, HG, kWindow> at, int32_t units,
                                             int half) {
  using S = Shape<DP>;
  constexpr int kUnit = Item<DP, HG>::kUnit, kStages = Shared<DP, HG>::kStages;
  constexpr int kTok = kUnit / kProducers;         // tokens of a unit that this warp copies
  constexpr int kQ = (kTok + 31) / 32;             // words of 32 tokens, the last one may be half
  const PagedArgs& p = a.p;
  const CacheView& cache = p.cache;
  const int lane = threadIdx.x & 31;
  Span<DP, HG, kWindow> span(p, at.len);
  int32_t tok = span.base(span.tiles - at.left) + kTok * half + lane;  // this lane's tokens: tok + 32*q
  int64_t head_off = 0, head_soff = 0;
  const int32_t* table = nullptr;
  auto enter = [&]() {
    const int32_t head = at.item / a.chunks;
    head_off = head * cache.head_stride;
    head_soff = head * cache.s_head_stride;
    table = p.table + static_cast<int64_t>(at.b) * p.table_stride;
  };
  auto page_index = [&](int32_t t) {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(t)) * a.page_magic) >> a.page_magic_shift);
  };
  // The pages of the next unit's tokens, loaded one unit ahead of their use; -1 behind the end.
  int32_t page[kQ];
  auto look_up = [&]() {
#pragma unroll
    for (int q = 0; q < kQ; ++q)
      page[q] = tok + 32 * q < at.len && lane + 32 * q < kTok && span.sees(tok + 32 * q) ? table[page_index(tok + 32 * q)] : -1;
  };
  enter();
  look_up();
  int stage = 0;
  uint32_t phase = 1;  // the first round finds every stage empty
  for (int32_t u = 0; u < units; ++u) {
    // one verdict for the whole warp: the votes and shuffles below are collective
    if (u >= kStages && !__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &sm.empty[stage], phase))) {
      flag_failure(a.status);
      break;
    }
    int64_t row[kQ];
    uint32_t mask[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      const int32_t t = tok + 32 * q;
      const int32_t off = t - page_index(t) * cache.page_size;
      const bool live = static_cast<uint32_t>(page[q]) < static_cast<uint32_t>(cache.pages);
      mask[q] = __ballot_sync(0xffffffffu, live);
      row[q] = live ? page[q] * cache.page_stride + head_off + off * cache.token_stride : -1;
      if (live) {
        const int64_t srow = page[q] * cache.s_page_stride + head_soff + off * cache.s_token_stride;
        cp_async4(smem_addr(&sm.scales[stage][0][kTok * half + 32 * q + lane]), cache.k_scale + srow);
        cp_async4(smem_addr(&sm.scales[stage][1][kTok * half + 32 * q + lane]), cache.v_scale + srow);
      }
    }
    if (lane == 0)
#pragma unroll
      for (int w = 0; w < kTok / kStep; ++w)
        sm.live[stage][kTok / kStep * half + w] = static_cast<uint16_t>(mask[w >> 1] >> (16 * (w & 1)));
    const uint32_t kd = smem_addr(sm.codes[stage][0]), vd = smem_addr(sm.codes[stage][1]);
#pragma unroll
    for (int w = 0; w < kTok / kStep; ++w) {
      const uint32_t here = (mask[w >> 1] >> (16 * (w & 1))) & 0xffffu;
      if (here == 0u) continue;
      const int slab = kTok / kStep * half + w;
      if constexpr (S::kA > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (lane >> 3) + 4 * j, piece = lane & 7;
          const int64_t from = __shfl_sync(0xffffffffu, row[w >> 1], 16 * (w & 1) + r) + 16 * piece;
          const int d = 2048 * slab + spot128(r, piece);
#pragma unroll
          for (int i = 0; i < S::kA; ++i) {
            const bool ok = from >= 16 * piece && 128 * i + 16 * piece < p.D;
            cp_async16_or_zero(kd + 128 * kUnit * i + d, cache.k + (ok ? from + 128 * i : 0), ok);
            cp_async16_or_zero(vd + 128 * kUnit * i + d, cache.v + (ok ? from + 128 * i : 0), ok);
          }
        }
      }
      if constexpr (S::kB > 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = (lane >> 2) + 8 * j, piece = lane & 3;
          const int64_t from = __shfl_sync(0xffffffffu, row[w >> 1], 16 * (w & 1) + r) + 16 * piece;
          const int d = 128 * kUnit * S::kA + 1024 * slab + spot64(r, piece);
          const bool ok = from >= 16 * piece && 128 * S::kA + 16 * piece < p.D;
          cp_async16_or_zero(kd + d, cache.k + (ok ? from + 128 * S::kA : 0), ok);
          cp_async16_or_zero(vd + d, cache.v + (ok ? from + 128 * S::kA : 0), ok);
        }
      }
    }
    // Each lane arrives once its copies have landed, lane 0 once more for the masks.
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sm.full[stage])) : "memory");
    if (lane == 0) mbar_arrive(&sm.full[stage]);
    if (u + 1 < units) {
      if (--at.left == 0) {
        at.next_head(a);
        if constexpr (kWindow) span = Span<DP, HG, kWindow>(p, at.len);
        tok = kTok * half + lane;  // a first tile is never behind the gap, unless there is none before it
        if constexpr (kWindow) tok += span.base(0);
        enter();
      } else if constexpr (kWindow) {
        tok = span.base(span.tiles - at.left) + kTok * half + lane;
      } else {
        tok += kUnit;
      }
      look_up();
    }
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // nothing in flight when the warp ends
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z, int32_t w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// The feed of a CTA by TMA boxes, one warp's: lane k brings the k-th box of each unit,
// 2^box_shift tokens of one page. Rows of a box behind the sequence's end are loaded too (they are inside the cache)
// and masked by the consumers.
template <int DP, int HG, bool kWindow>
struct BoxFeed {
  using S = Shape<DP>;
  static constexpr int kUnit = Item<DP, HG>::kUnit;

  Place<DP, HG, kWindow> at;
  Span<DP, HG, kWindow> span;
  int32_t base, head;  // the next unit's first token, its key head
  const int32_t* table;
  // Entries `window`..`window + 63` of the sequence's table row, two per lane, loaded at least 16 entries before a
  // unit needs them (a unit spans at most 16 pages); loading each unit's entries as it came cost their latency per
  // unit. Entries behind the sequence's last page are -1.
  int32_t window, near, far, pages_here;

  __device__ __forceinline__ BoxFeed(const SplitArgs& a, const Place<DP, HG, kWindow>& first)
      : at(first), span(a.p, first.len), base(span.base(span.tiles - first.left)) {
    enter(a);
  }
  __device__ __forceinline__ int32_t index_of(const SplitArgs& a, int32_t t) const {
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(t)) * a.page_magic) >> a.page_magic_shift);
  }
  __device__ __forceinline__ int32_t entry(int32_t i) const { return i < pages_here ? table[i] : -1; }

  // At unit `at`, whose first token is `base`.
  __device__ __forceinline__ void enter(const SplitArgs& a) {
    const int lane = threadIdx.x & 31;
    head = at.item / a.chunks;
    table = a.p.table + static_cast<int64_t>(at.b) * a.p.table_stride;
    pages_here = index_of(a, at.len - 1) + 1;
    window = index_of(a, base);
    near = entry(window + lane);
    far = entry(window + 32 + lane);
  }

  // Starts the copies of the next unit into `stage` and moves on (`more`: another unit follows).
  __device__ __forceinline__ void issue(const SplitArgs& a, const Maps& maps, Shared<DP, HG>& sm, int stage, bool more) {
    const PagedArgs& p = a.p;
    const CacheView& cache = p.cache;
    const int lane = threadIdx.x & 31, rows = 1 << a.box_shift;
    if (index_of(a, base) >= window + 32) {
      window += 32;
      near = far;
      far = entry(window + 32 + lane);
    }
    // Page and slot of this lane's box.
    const int32_t first = base + (lane << a.box_shift), index = index_of(a, first), in = index - window;
    const int32_t slot = first - index * cache.page_size;
    const int32_t from_near = __shfl_sync(0xffffffffu, near, in & 31), from_far = __shfl_sync(0xffffffffu, far, in & 31);
    bool wanted = (lane << a.box_shift) < kUnit && first < at.len;
    if constexpr (kWindow) wanted = wanted && (first < span.sunk || first + rows > span.start);
    const int32_t page = wanted ? (in < 32 ? from_near : from_far) : -1;
    const bool live = static_cast<uint32_t>(page) < static_cast<uint32_t>(cache.pages);
    const uint32_t boxes = __ballot_sync(0xffffffffu, live);
    // Lane w makes the mask of slab w: the tokens whose box is live, up to the sequence's end.
    if (lane < Item<DP, HG>::kSlabs) {
      uint32_t mask = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)  // boxes are at least 8 rows
        if ((boxes >> ((kStep * lane + 8 * h) >> a.box_shift)) & 1u) mask |= 0xffu << (8 * h);
      const int32_t last = at.len - base - kStep * lane;
      if (last < kStep) mask &= last > 0 ? (1u << last) - 1u : 0u;
      if constexpr (kWindow) {  // tokens [sunk, start) are out
        const int32_t from = min(max(span.sunk - base - kStep * lane, 0), kStep), to = min(max(span.start - base - kStep * lane, 0), kStep);
        mask &= ~(((1u << to) - 1u) & ~((1u << from) - 1u));
      }
      sm.live[stage][lane] = static_cast<uint16_t>(mask);
    }
    uint64_t* bar = &sm.full[stage];
    if (a.bulk_scales == 0) {
#pragma unroll
      for (int q = 0; q < kUnit / 32; ++q) {
        const int from = (32 * q + lane) >> a.box_shift;  // the lane whose box holds this lane's token
        const int32_t pg = __shfl_sync(0xffffffffu, page, from), sl = __shfl_sync(0xffffffffu, slot, from);
        if ((boxes >> from) & 1u) {
          const int64_t srow = pg * cache.s_page_stride + head * cache.s_head_stride +
                               (sl + ((32 * q + lane) & (rows - 1))) * cache.s_token_stride;
          cp_async4(smem_addr(&sm.scales[stage][0][32 * q + lane]), cache.k_scale + srow);
          cp_async4(smem_addr(&sm.scales[stage][1][32 * q + lane]), cache.v_scale + srow);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
    }
    __syncwarp();  // the masks are written before lane 0 arrives
    if (lane == 0)
      mbar_arrive_expect_tx(bar, static_cast<uint32_t>(__popc(boxes)) * static_cast<uint32_t>(rows) *
                                     (2u * DP + (a.bulk_scales != 0 ? 8u : 0u)));
    __syncwarp();
    if (live) {
      const int row = lane << a.box_shift;
      const uint32_t kd = smem_addr(sm.codes[stage][0]), vd = smem_addr(sm.codes[stage][1]);
#pragma unroll
      for (int i = 0; i < S::kA; ++i) {
        tma_load_4d(kd + 128 * (kUnit * i + row), &maps.k128, 128 * i, slot, head, page, bar);
        tma_load_4d(vd + 128 * (kUnit * i + row), &maps.v128, 128 * i, slot, head, page, bar);
      }
      if constexpr (S::kB > 0) {
        tma_load_4d(kd + 128 * kUnit * S::kA + 64 * row, &maps.k64, 128 * S::kA, slot, head, page, bar);
        tma_load_4d(vd + 128 * kUnit * S::kA + 64 * row, &maps.v64, 128 * S::kA, slot, head, page, bar);
      }
      if (a.bulk_scales != 0) {
        const int64_t srow = page * cache.s_page_stride + head * cache.s_head_stride + slot;
        bulk_g2s(&sm.scales[stage][0][row], cache.k_scale + srow, 4u * rows, bar);
        bulk_g2s(&sm.scales[stage][1][row], cache.v_scale + srow, 4u * rows, bar);
      }
    }
    if (more) {
      if (--at.left == 0) {
        at.next_head(a);
        if constexpr (kWindow) span = Span<DP, HG, kWindow>(a.p, at.len);
        base = kWindow ? span.base(0) : 0;
        enter(a);
      } else {
        base += kUnit;
        if constexpr (kWindow) {
          if (span.tiles - at.left == span.low && span.skip > 0) {  // over the gap: other entries of the table
            base += span.skip * kUnit;
            enter(a);
          }
        }
      }
    }
  }
};

// The producer warp: `units` units from the one at `at` on.
template <int DP, int HG, bool kWindow>
__device__ __forceinline__ void produce_boxes(const SplitArgs& a, const Maps& maps, Shared<DP, HG>& sm,
                                              const Place<DP, HG, kWindow>& at, int32_t units) {
  constexpr int kStages = Shared<DP, HG>::kStages;
  BoxFeed<DP, HG, kWindow> feed(a, at);
  int stage = 0;
  uint32_t phase = 1;  // the first round finds every stage empty
  int32_t u = 0;
  for (; u < units; ++u) {
    if (u >= kStages && !__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &sm.empty[stage], phase))) break;
    feed.issue(a, maps, sm, stage, u + 1 < units);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (u < units) {
    flag_failure(a.status);
    // Let the copies already issued land before this CTA's shared memory goes away.
    for (int32_t j = max(0, u - kStages); j < u; ++j)
      if (!mbar_wait(kWaitLimitNs, &sm.full[j % kStages], static_cast<uint32_t>(j / kStages) & 1u)) break;
  }
}

__device__ __forceinline__ void store_out(int dtype, void* out, int64_t i, float v) {
  if (dtype == DT_BF16) Elem<__nv_bfloat16>::store1(out, i, v);
  else Elem<__half>::store1(out, i, v);
}

__device__ __forceinline__ void consumer_barrier() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory"); }

// kBoxes: fed by TMA boxes, else row by row. kWindow: a part of each sequence.
template <int DP, int HG, bool kBoxes, bool kWindow>
__global__ void __launch_bounds__(kThreads, 2)
    attention_split_kernel(const __grid_constant__ Maps maps, const __grid_constant__ SplitArgs a) {
  using S = Shape<DP>;
  using Sm = Shared<DP, HG>;
  constexpr int kSlabs = Item<DP, HG>::kSlabs;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // The swizzles repeat every 1024 bytes: align the ring to 1024.
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const PagedArgs& p = a.p;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  pdl_trigger();
  if (kBoxes && threadIdx.x == kConsumers) {
    if (S::kA > 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k128)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v128)) : "memory");
    }
    if (S::kB > 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.k64)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.v64)) : "memory");
    }
  }
  if (threadIdx.x < Sm::kStages) {
    // full: lane 0 of a producer for its masks and boxes, and each lane's own copies where there are any
    mbar_init(&sm.full[threadIdx.x], kBoxes ? (a.bulk_scales != 0 ? 1 : 33) : 33 * kProducers);
    mbar_init(&sm.empty[threadIdx.x], kWarps);
    fence_barrier_init();
  }

  pdl_wait();
  // Bring the page table to the L2 cache while the lengths are on their way: one line per thread of the grid,
  // as far as that goes.
  if (p.max_len > 0) {
    const uint32_t width = static_cast<uint32_t>((p.max_len - 1) / p.cache.page_size) + 1u;
    const uint32_t i = (blockIdx.x * kThreads + threadIdx.x) * 32u, b = i / width;  // 32 entries per 128-byte line
    if (b < static_cast<uint32_t>(p.B))
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + b * p.table_stride + (i - b * width)));
  }
  // This CTA's places [begin, end) of all, and its first unit. (block_scan's barriers also publish the mbarriers.)
  int64_t total = 0, incl = 0, mine = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
    mine = extent_of<DP, HG, kWindow>(a, b0 + static_cast<int32_t>(threadIdx.x));
    int64_t sum;
    incl = block_scan(mine, sm.scan, &sum);
    total += sum;
  }
  const int32_t n = min(static_cast<int32_t>(gridDim.x), units_in(total));  // CTAs with places
  const int32_t cta = blockIdx.x;
  if (cta >= n) {
    if (threadIdx.x == 0 && a.meta != nullptr) a.meta[cta].b = -1;
    write_empty(p, kThreads);
    return;
  }
  const Share share(places_in(total), n);
  const int32_t begin = share.begin(cta), end = share.begin(cta + 1);
  int64_t carry = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
    if (p.B > kThreads) {  // else the scan above is this one
      mine = extent_of<DP, HG, kWindow>(a, b);
      int64_t sum;
      incl = block_scan(mine, sm.scan, &sum) + carry;
      carry += sum;
    }
    const int32_t from = places_in(incl - mine), to = places_in(incl);
    const bool has_begin = from <= begin && begin < to, has_end = from < end && end <= to;
    if (has_begin || has_end) {
      const int32_t tiles = tiles_of<DP, HG, kWindow>(p, length_of(p, b));
      auto units_before = [&](int32_t place, int32_t& item, int32_t& tile) {
        item = (place - from) / (tiles + 1);
        tile = place - from - item * (tiles + 1);
        return units_in(incl - mine) + item * tiles + tile;
      };
      int32_t item, tile;
      if (has_end) sm.before_end = units_before(end, item, tile);
      if (has_begin) {
        sm.before_begin = units_before(begin, item, tile);
        sm.start_b = b;
        sm.start_item = item;
        sm.start_tile = tile;
      }
    }
  }
  __syncthreads();
  Place<DP, HG, kWindow> use;
  use.b = sm.start_b;
  use.item = sm.start_item;
  use.len = length_of(p, use.b);
  const int32_t nt = tiles_of<DP, HG, kWindow>(p, use.len);
  int32_t t = sm.start_tile;
  const int32_t units = sm.before_end - sm.before_begin;
  const int32_t first = begin - t;  // the head's first place
  use.left = nt - t;
  if (units > 0 && use.left == 0) {  // the place behind a head
    use.next_head(a);
    t = 0;
  }
  if (units == 0) {
    if (threadIdx.x == 0 && a.meta != nullptr) a.meta[cta].b = -1;
    write_empty(p, kThreads);
    return;
  }
  if (warp >= kWarps) {
    if constexpr (!kBoxes) produce_rows<DP, HG, kWindow>(a, sm, use, units, warp - kWarps);
    else if (warp == kWarps) produce_boxes<DP, HG, kWindow>(a, maps, sm, use, units);
    return;
  }
  if (threadIdx.x == 0 && a.meta != nullptr) {
    // The head's first part is the first thing its CTA does if that begins at the head's first place, or one before
    // it, behind the head before.
    Meta m;
    m.b = t > 0 ? use.b : -1;
    m.item = use.item;
    m.first = share.owner(first);
    m.last = share.owner(first + nt - 1);
    m.slot = share.begin(m.first) >= first - 1 ? 0 : 1;
    a.meta[cta] = m;
  }

  // --------------------------------------------------------------------------- the heads
  // This warp's tokens of a unit, columns and heads of an item.
  constexpr int CG = Item<DP, HG>::CG;
  const int slab = warp % kSlabs, cols = CG == 1 ? 0 : warp / kSlabs % CG, group = warp / (kSlabs * CG);
  // Query fragments (fp16): word j of piece i of head g.
  constexpr bool kQueryHeld = DP <= 128;
  uint4 q[kQueryHeld ? DP / 32 : 1];
  // Of heads 2c and 2c + 1, the same in the eight threads that share them (l: of this thread's tokens only).
  float qf[2] = {0.f, 0.f}, m[2], mo[2], l[2];
  // Output tiles of 16 columns x 8 heads: o[n][2h + e] is column 16g + .. + h of head 2c + e.
  constexpr int kN = DP == 64 ? 4 : 8;
  float o[kN][4];
  bool first_segment = true;
  bool fresh = true, from_start = false;
  int32_t rows = 0, head0 = 0;  // query heads of the item, and the first of them
  int stage = 0;
  uint32_t phase = 0;
  bool arrived = true;  // false once a wait gave up: the rest runs through without waiting, its tokens left out

  for (int32_t u = 0; u < units; ++u) {
    if (fresh) {
      fresh = false;
      from_start = use.left == tiles_of<DP, HG, kWindow>(p, use.len);
      const int32_t head = use.item / a.chunks, chunk = use.item - head * a.chunks;
      rows = min(Item<DP, HG>::kRows, a.G - Item<DP, HG>::kRows * chunk);
      head0 = head * a.G + Item<DP, HG>::kRows * chunk;
      const int32_t h = kHeads * group + g;
      const uint8_t* src = p.q + static_cast<int64_t>(use.b) * p.q_stride + static_cast<int64_t>(head0 + h) * p.D;
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        const int d = i < 2 * S::kA ? 128 * (i >> 1) + 16 * (2 * c + (i & 1)) : 128 * S::kA + 16 * c;
        const uint4 v = h < rows && d < p.D ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0u, 0u, 0u, 0u);
        uint4 lo, hi;
        codes_f16(v.x, lo.x, lo.y);
        codes_f16(v.y, lo.z, lo.w);
        codes_f16(v.z, hi.x, hi.y);
        codes_f16(v.w, hi.z, hi.w);
        if constexpr (kQueryHeld) {
          q[2 * i] = lo;
          q[2 * i + 1] = hi;
        } else if (slab == 0 && cols == 0) {  // the last head's readers have passed its join
          sm.query[group][2 * i][lane] = lo;
          sm.query[group][2 * i + 1][lane] = hi;
        }
      }
      if constexpr (!kQueryHeld) consumer_barrier();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int32_t he = kHeads * group + 2 * c + e;
        qf[e] = he < rows ? p.q_scale[static_cast<int64_t>(use.b) * p.q_scale_stride + head0 + he] * p.scale_log2 : 0.f;
        m[e] = mo[e] = kLowest;
        l[e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    // one verdict for the whole warp: the products and shuffles below are collective
    if (arrived && !__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &sm.full[stage], phase))) {
      flag_failure(a.status);
      arrived = false;
    }
    const uint32_t live = arrived ? sm.live[stage][slab] : 0u;  // a stage that has not landed may change while it is read
    if (live != 0u) {
      const unsigned char* kt = sm.codes[stage][0];
      // Scores of tokens g (0, 1) and g + 8 (2, 3) with heads 2c and 2c + 1; two chains of sums.
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll kQueryHeld ? DP / 64 : 1  // loads of more than one iteration at a time spill above head size 128
      for (int i = 0; i < DP / 64; ++i) {
        const int at = i < 2 * S::kA ? 128 * Sm::kUnit * (i >> 1) + 2048 * slab + spot128(g, 2 * c + (i & 1))
                                     : 128 * Sm::kUnit * S::kA + 1024 * slab + spot64(g, c);
        const uint4 k0 = *reinterpret_cast<const uint4*>(kt + at);
        const uint4 k1 = *reinterpret_cast<const uint4*>(kt + at + (i < 2 * S::kA ? 1024 : 512));  // row g + 8
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4 qi;
          if constexpr (kQueryHeld) qi = q[2 * i + j];
          else qi = sm.query[group][2 * i + j][lane];
          uint32_t a0, a1, a2, a3;
          codes_f16(word(k0, 2 * j), a0, a2);
          codes_f16(word(k1, 2 * j), a1, a3);
          mma_f16(s0, a0, a1, a2, a3, qi.x, qi.y);
          codes_f16(word(k0, 2 * j + 1), a0, a2);
          codes_f16(word(k1, 2 * j + 1), a1, a3);
          mma_f16(s1, a0, a1, a2, a3, qi.z, qi.w);
        }
      }
      const float* sk = &sm.scales[stage][0][kStep * slab + g];
      const float* sv = &sm.scales[stage][1][kStep * slab + g];
      const float ks[2] = {sk[0], sk[8]}, lv[2] = {lg2_all(sv[0]), lg2_all(sv[8])};
      float x[2][2], w[2][2];  // [token][head]
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[t][e] = (s0[2 * t + e] + s1[2 * t + e]) * (qf[e] * ks[t]);
          w[t][e] = x[t][e] + lv[t];
        }
      if (live != 0xffffu) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (!((live >> (g + 8 * t)) & 1u)) x[t][0] = x[t][1] = w[t][0] = w[t][1] = -CUDART_INF_F;
      }
      bool above = false;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        above = above || fmaxf(x[0][e], x[1][e]) > m[e] + kSlack || fmaxf(w[0][e], w[1][e]) > mo[e] + (kRoom + kSlack);
      if (__any_sync(0xffffffffu, above)) {
        float keep[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(m[e], column_max(fmaxf(x[0][e], x[1][e])));
          const float on = fmaxf(mo[e], column_max(fmaxf(w[0][e], w[1][e])) - kRoom);
          l[e] *= ex2(m[e] - mn);
          keep[e] = ex2(mo[e] - on);
          m[e] = mn;
          mo[e] = on;
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          o[i][0] *= keep[0];
          o[i][1] *= keep[1];
          o[i][2] *= keep[0];
          o[i][3] *= keep[1];
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += ex2(x[0][e] - m[e]) + ex2(x[1][e] - m[e]);
      // Weights: (tokens x heads) pairs of heads -> B fragments, pairs of tokens of head g.
      const uint32_t p0 = transpose8(pack_f16(ex2(w[0][0] - mo[0]), ex2(w[0][1] - mo[1])));
      const uint32_t p1 = transpose8(pack_f16(ex2(w[1][0] - mo[0]), ex2(w[1][1] - mo[1])));
      const unsigned char* vt = sm.codes[stage][1];
      if (S::kA > 0 && (S::kA == CG || cols == 0)) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = *reinterpret_cast<const uint4*>(vt + 128 * Sm::kUnit * cols + 2048 * slab +
                                                 spot128(2 * c + (e & 1) + 8 * (e >> 1), g));
        if (live != 0xffffu) {  // codes of tokens that do not count may be NaN: 0 * NaN must not reach the sum
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((live >> (2 * c + (e & 1) + 8 * (e >> 1))) & 1u)) v[e] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kN / 2; ++k) {
          uint32_t lo[4], hi[4];
          pair_f16(word(v[0], k), word(v[1], k), lo);
          pair_f16(word(v[2], k), word(v[3], k), hi);
          mma_f16(o[2 * k], lo[0], lo[1], hi[0], hi[1], p0, p1);
          mma_f16(o[2 * k + 1], lo[2], lo[3], hi[2], hi[3], p0, p1);
        }
      } else if constexpr (S::kB > 0) {
        uint2 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = *reinterpret_cast<const uint2*>(vt + 128 * Sm::kUnit * S::kA + 1024 * slab +
                                                 spot64(2 * c + (e & 1) + 8 * (e >> 1), g >> 1) + 8 * (g & 1));
        if (live != 0xffffu) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((live >> (2 * c + (e & 1) + 8 * (e >> 1))) & 1u)) v[e] = make_uint2(0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t lo[4], hi[4];
          pair_f16(k == 0 ? v[0].x : v[0].y, k == 0 ? v[1].x : v[1].y, lo);
          pair_f16(k == 0 ? v[2].x : v[2].y, k == 0 ? v[3].x : v[3].y, hi);
          mma_f16(o[2 * k], lo[0], lo[1], hi[0], hi[1], p0, p1);
          mma_f16(o[2 * k + 1], lo[2], lo[3], hi[2], hi[3], p0, p1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[stage]);
    if (++stage == Sm::kStages) {
      stage = 0;
      phase ^= 1u;
    }

    // ------------------------------------------------------------------- the end of a head
    const bool done = --use.left == 0;
    if (done || u + 1 == units) {
      const bool whole = done && from_start;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], d);
        if (g == 0) {
          sm.stat[warp][2 * c + e][0] = m[e];
          sm.stat[warp][2 * c + e][1] = mo[e];
          sm.stat[warp][2 * c + e][2] = l[e];
        }
      }
      consumer_barrier();
      float f[2];  // brings heads 2c and 2c + 1 to the largest M of the warps that share them
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < kSlabs; ++w) top = fmaxf(top, sm.stat[group * (CG * kSlabs) + w][2 * c + e][1]);
        f[e] = ex2(mo[e] - top);
      }
      // Thread (warp, lane) finishes head 8r + warp of the item, column `lane` of each piece of 32.
      const int64_t slot = 2 * static_cast<int64_t>(cta) + (first_segment ? 0 : 1);
      first_segment = false;
      Norm norm[HG];
#pragma unroll
      for (int r = 0; r < HG; ++r) {
        float top = kLowest, topo = kLowest, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kSlabs; ++w) {
          top = fmaxf(top, sm.stat[r * (CG * kSlabs) + w][warp][0]);
          topo = fmaxf(topo, sm.stat[r * (CG * kSlabs) + w][warp][1]);
        }
#pragma unroll
        for (int w = 0; w < kSlabs; ++w)
          sum = fmaf(sm.stat[r * (CG * kSlabs) + w][warp][2], ex2(sm.stat[r * (CG * kSlabs) + w][warp][0] - top), sum);
        norm[r] = norm_of(top, topo, sum);
        const int row = kHeads * r + warp;
        if (row < rows && lane == 0) {
          if (!whole)
            *reinterpret_cast<float4*>(a.stats + (slot * Item<DP, HG>::kRows + row) * 4) = make_float4(top, topo, sum, 0.f);
          else if (p.lse != nullptr)
            p.lse[static_cast<int64_t>(use.b) * p.Hq + head0 + row] =
                sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.693147180559945309f;
        }
      }
      // Piece k: each thread's columns 4k..4k+3 of its two heads.
#pragma unroll
      for (int k = 0; k < kN / 2; ++k) {
        const bool narrow = S::kA < CG && (S::kA == 0 || cols > 0);  // 8 columns a thread, not 16
        if (!narrow || k < 2) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(&sm.join[warp][2 * c + e][4 * g]) =
                make_float4(o[2 * k][e] * f[e], o[2 * k][2 + e] * f[e], o[2 * k + 1][e] * f[e], o[2 * k + 1][2 + e] * f[e]);
        }
        consumer_barrier();
#pragma unroll
        for (int r = 0; r < HG; ++r)
#pragma unroll
          for (int y = 0; y < CG; ++y) {
            const bool slim = y >= S::kA;
            if (slim && k >= 2) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kSlabs; ++w) v += sm.join[(r * CG + y) * kSlabs + w][warp][lane];
            const int row = kHeads * r + warp, d = 128 * y + (slim ? 8 : 16) * (lane >> 2) + 4 * k + (lane & 3);
            if (row < rows && d < p.D) {
              if (whole) store_out(a.dtype, p.out, (static_cast<int64_t>(use.b) * p.Hq + head0 + row) * p.D + d, norm[r](v));
              else a.part[(slot * Item<DP, HG>::kRows + row) * DP + d] = v;
            }
          }
        consumer_barrier();
      }
      fresh = true;
      if (u + 1 < units) use.next_head(a);
    }
  }
  write_empty(p, kConsumers);
}

// Joins partial results. Every CTA of the first kernel but a head's first has a counterpart here, and these share the
// head's rows: CTA k takes each (parts - 1)-th. A head of few parts takes a warp per row, one of many (it then has as
// many CTAs here) the whole CTA, whose warps share the parts, each in a fixed order. What bounds it is its start and
// two dependent loads (which head; statistics and values): 3 us behind the 47 us of one sequence of 131072 tokens,
// 2.5 to 4.7 us elsewhere; with a CTA for each row of each head, most of them idle, it took 5 to 9.5 us.
constexpr int kJoinWarps = 8;

// Running maxima, sum and values of parts `from`, `from + step`, ... of a row; lane l has columns 2l, 2l + 1, 2l + 64, ...
// Statistics and values of kAhead parts are on their way at the same time.
template <int DP>
struct JoinRow {
  static constexpr int kV = DP / 64;
  float top = kLowest, topo = kLowest, l = 0.f;
  float2 v[kV];

  template <int kAhead, typename Slot>
  __device__ __forceinline__ void add(const SplitArgs& a, int rows, int row, int from, int step, int parts, Slot slot_of) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = make_float2(0.f, 0.f);
    for (int i0 = from; i0 < parts; i0 += step * kAhead) {
      float4 st[kAhead];
      float2 x[kAhead][kV];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const bool have = i0 + step * e < parts;
        const int64_t at = slot_of(have ? i0 + step * e : i0) * rows + row;
        st[e] = have ? *reinterpret_cast<const float4*>(a.stats + at * 4) : make_float4(kLowest, kLowest, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
          const int d = 2 * (lane + 32 * j);
          x[e][j] = have && d < a.p.D ? *reinterpret_cast<const float2*>(a.part + at * DP + d) : make_float2(0.f, 0.f);
        }
      }
      float mn = top, on = topo;
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        mn = fmaxf(mn, st[e].x);
        on = fmaxf(on, st[e].y);
      }
      l *= ex2(top - mn);
      const float keep = ex2(topo - on);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[j] = mul2(v[j], splat2(keep));
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        l = fmaf(st[e].z, ex2(st[e].x - mn), l);
        const float f = ex2(st[e].y - on);
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = fma2(x[e][j], splat2(f), v[j]);
      }
      top = mn;
      topo = on;
    }
  }
};

__device__ __forceinline__ float lse_of(float top, float l) {
  return l == 0.f ? -CUDART_INF_F : (top + log2f(l)) * 0.693147180559945309f;
}

__device__ __forceinline__ void store_pair(const SplitArgs& a, int64_t row, int pair, float2 y) {
  static_cast<uint32_t*>(a.p.out)[row * (a.p.D / 2) + pair] =
      a.dtype == DT_BF16 ? Elem<__nv_bfloat16>::pack(y) : Elem<__half>::pack(y);
}

template <int DP, int HG>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const __grid_constant__ SplitArgs a) {
  constexpr int kRows = Item<DP, HG>::kRows, kV = DP / 64;
  // Parts of a warp at a time where a head has many: 4 took 51.0 us for one sequence of 131072 tokens, 8 50.1 (heads of
  // 256 slow down by the registers).
  constexpr int kMany = DP <= 128 ? 8 : 4;
  __shared__ float2 sum[kJoinWarps][DP / 2];
  __shared__ float4 stat[kJoinWarps];
  pdl_trigger();
  pdl_wait();
  const int64_t k = blockIdx.x + 1;
  const Meta me = a.meta[k];
  const PagedArgs& p = a.p;
  if (me.b < 0) return;
  const int chunk = me.item % a.chunks, rows = min(kRows, a.G - kRows * chunk);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = me.last - me.first + 1, others = parts - 1;
  auto slot_of = [&](int i) { return i == 0 ? 2 * static_cast<int64_t>(me.first) + me.slot : 2 * static_cast<int64_t>(me.first + i); };
  const int64_t orow0 = static_cast<int64_t>(me.b) * p.Hq + me.item / a.chunks * a.G + kRows * chunk;
  const int first = static_cast<int>(k) - me.first - 1;  // this CTA's first row
  JoinRow<DP> r;
  if (parts <= kJoinWarps) {
    for (int row = first + others * warp; row < rows; row += others * kJoinWarps) {
      r = JoinRow<DP>();
      r.template add<4>(a, kRows, row, 0, 1, parts, slot_of);
      const Norm norm = norm_of(r.top, r.topo, r.l);
#pragma unroll
      for (int j = 0; j < kV; ++j)
        if (2 * (lane + 32 * j) < p.D) store_pair(a, orow0 + row, lane + 32 * j, norm(r.v[j]));
      if (p.lse != nullptr && lane == 0) p.lse[orow0 + row] = lse_of(r.top, r.l);
    }
    return;
  }
  for (int row = first; row < rows; row += others) {
    r = JoinRow<DP>();
    r.template add<kMany>(a, kRows, row, warp, kJoinWarps, parts, slot_of);
    if (lane == 0) stat[warp] = make_float4(r.top, r.topo, r.l, 0.f);
#pragma unroll
    for (int j = 0; j < kV; ++j) sum[warp][lane + 32 * j] = r.v[j];
    __syncthreads();
    float mj = kLowest, oj = kLowest, lj = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      mj = fmaxf(mj, stat[w].x);
      oj = fmaxf(oj, stat[w].y);
    }
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) lj = fmaf(stat[w].z, ex2(stat[w].x - mj), lj);
    const Norm norm = norm_of(mj, oj, lj);
    for (int d = threadIdx.x; 2 * d < p.D; d += kJoinWarps * 32) {
      float2 y = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) y = fma2(sum[w][d], splat2(ex2(stat[w].y - oj)), y);
      store_pair(a, orow0 + row, d, norm(y));
    }
    if (p.lse != nullptr && threadIdx.x == 0) p.lse[orow0 + row] = lse_of(mj, lj);
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------------- host side
inline int padded(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

struct Plan {
  int64_t grid, units, chunks;  // units: at most
  int hg;                       // warps that share a step's tokens
  bool join;
};

// `seen`: the most tokens of a sequence that take part, in `parts` runs.
inline Plan plan_of(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len, int64_t seen, int64_t parts) {
  Plan q;
  const int64_t G = Hq / Hk;
  q.hg = G > kHeads ? 2 : 1;
  const int64_t unit = kStep * kWarps / (q.hg * (padded(D) > 128 ? 2 : 1)), rows = kHeads * q.hg;
  const int64_t all = (max_len + unit - 1) / unit, some = (seen + unit - 1) / unit + parts;
  const int64_t tiles = some < all ? some : all;
  q.chunks = (G + rows - 1) / rows;
  const int64_t resident = static_cast<int64_t>(sm_count()) * 2;  // two CTAs per SM
  const __int128 units = static_cast<__int128>(B) * Hk * q.chunks * tiles;
  q.units = units < 0x7fffffffLL ? static_cast<int64_t>(units) : 0x7fffffffLL;
  q.grid = units < resident ? static_cast<int64_t>(units) : resident;
  if (q.grid < 1) q.grid = 1;
  q.join = tiles > 1 && q.grid > 1;
  return q;
}

template <int DP, int HG, bool kBoxes, bool kWindow>
bool launch_fed(const SplitArgs& a, const Maps& maps, const Plan& plan, cudaStream_t s) {
  auto kern = attention_split_kernel<DP, HG, kBoxes, kWindow>;
  constexpr size_t smem = sizeof(Shared<DP, HG>) + 1024;
  static_assert(smem <= 227 * 1024 && (smem + 1024) * 2 <= 228 * 1024, "the ring fits the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  launch_overlapped(kern, dim3(static_cast<unsigned>(plan.grid)), kThreads, smem, 1, s, maps, a);
  if (plan.join)
    launch_overlapped(attention_join_kernel<DP, HG>, dim3(static_cast<unsigned>(plan.grid - 1)), kJoinWarps * 32, 0, 1, s, a);
  return true;
}

// Maps of the cache for the TMA feed; false where its layout has none (the rows are then copied one by one).
template <int DP>
bool cache_maps(const PagedArgs& p, int box_rows, Maps* m) {
  const CacheView& c = p.cache;
  const uint64_t dims[4] = {static_cast<uint64_t>(p.D), static_cast<uint64_t>(c.page_size), static_cast<uint64_t>(p.Hk),
                            static_cast<uint64_t>(c.pages)};
  // the stride of a dimension of one element is never used, but has to be a valid one
  auto stride = [](int64_t extent, int64_t s) { return static_cast<uint64_t>(extent > 1 ? s : 256); };
  const uint64_t strides[3] = {stride(c.page_size, c.token_stride), stride(p.Hk, c.head_stride), stride(c.pages, c.page_stride)};
  for (uint64_t s : strides)
    if (s >= (1ull << 40)) return false;
  const uint32_t wide[4] = {128, static_cast<uint32_t>(box_rows), 1, 1}, narrow[4] = {64, static_cast<uint32_t>(box_rows), 1, 1};
  bool ok = true;
  if constexpr (Shape<DP>::kA > 0)
    ok = ok && byte_tensor_map(&m->k128, 4, c.k, dims, strides, wide, CU_TENSOR_MAP_SWIZZLE_128B) &&
         byte_tensor_map(&m->v128, 4, c.v, dims, strides, wide, CU_TENSOR_MAP_SWIZZLE_128B);
  if constexpr (Shape<DP>::kB > 0)
    ok = ok && byte_tensor_map(&m->k64, 4, c.k, dims, strides, narrow, CU_TENSOR_MAP_SWIZZLE_64B) &&
         byte_tensor_map(&m->v64, 4, c.v, dims, strides, narrow, CU_TENSOR_MAP_SWIZZLE_64B);
  return ok;
}

template <int DP, int HG, bool kWindow>
bool launch_dp(SplitArgs a, const Plan& plan, cudaStream_t s) {
  const CacheView& c = a.p.cache;
  Maps maps{};
  // Rows per box: the largest power of two that divides a page, at most a unit.
  a.box_shift = 0;
  while ((2 << a.box_shift) <= Item<DP, HG>::kUnit && c.page_size % (2 << a.box_shift) == 0) ++a.box_shift;
  // Small boxes cost the TMA unit as much as large ones (about 30 clocks each): below 1 KB rows are copied one by one.
  if (a.box_shift < 3 || (DP << a.box_shift) < 1024 || !cache_maps<DP>(a.p, 1 << a.box_shift, &maps)) return launch_fed<DP, HG, false, kWindow>(a, maps, plan, s);
  auto quad = [](int64_t extent, int64_t s) { return extent <= 1 || s % 4 == 0; };
  a.bulk_scales = c.s_token_stride == 1 && quad(a.p.Hk, c.s_head_stride) && quad(c.pages, c.s_page_stride) &&
                  (reinterpret_cast<uintptr_t>(c.k_scale) | reinterpret_cast<uintptr_t>(c.v_scale)) % 16 == 0;
  return launch_fed<DP, HG, true, kWindow>(a, maps, plan, s);
}

template <int HG, bool kWindow>
bool launch_hg(const SplitArgs& a, const Plan& plan, cudaStream_t s) {
  switch (padded(a.p.D)) {
    case 64: return launch_dp<64, HG, kWindow>(a, plan, s);
    case 128: return launch_dp<128, HG, kWindow>(a, plan, s);
    case 192: return launch_dp<192, HG, kWindow>(a, plan, s);
    default: return launch_dp<256, HG, kWindow>(a, plan, s);
  }
}

template <bool kWindow>
bool launch_split(const PagedArgs& p, int dtype, cudaStream_t s) {
  const int64_t seen = static_cast<int64_t>(p.window) + p.sinks;
  const Plan plan = plan_of(p.B, p.Hq, p.Hk, p.D, p.max_len, kWindow ? seen : p.max_len, kWindow ? 2 : 0);
  if (plan.units > 0x3fffffffLL) return false;  // units, and places up to twice as many, are counted in 32 bits
  // A warp passes over sequences without tokens one by one while others wait for it, in waits of a second at most
  // (20 sequences of 1000 tokens take 14.2 us alone, 14.5 spread over 128 places, 17.7 over 512, 30.5 over 2048).
  if (p.B > 65536) return false;
  SplitArgs a{};
  a.p = p;
  a.G = p.Hq / p.Hk;
  a.chunks = static_cast<int32_t>(plan.chunks);
  a.slots = static_cast<int32_t>(2 * plan.grid);
  a.status = device_status_ptr();
  int lg = 0;
  while ((1LL << lg) < p.cache.page_size) ++lg;
  a.page_magic_shift = 31 + lg;
  a.page_magic = static_cast<uint32_t>(((1ull << a.page_magic_shift) + p.cache.page_size - 1) / p.cache.page_size);
  if (plan.join) {
    a.meta = reinterpret_cast<Meta*>(p.partial);
    a.stats = reinterpret_cast<float*>(a.meta + plan.grid);
    a.part = a.stats + static_cast<int64_t>(a.slots) * kHeads * plan.hg * 4;
  }
  a.dtype = dtype;
  return plan.hg == 2 ? launch_hg<2, kWindow>(a, plan, s) : launch_hg<1, kWindow>(a, plan, s);
}

}  // namespace

// Compiled twice, side by side, since the instances are many: here for whole sequences, and by fq_attention_window.cu for
// windows.
#ifdef FQ_ATTENTION_WINDOW
bool launch_attention_window(const PagedArgs& p, int dtype, cudaStream_t s) { return launch_split<true>(p, dtype, s); }
#else
size_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  const Plan plan = plan_of(B, Hq, Hk, D, max_len, max_len, 0);
  if (!plan.join) return 0;
  return static_cast<size_t>(plan.grid) * (sizeof(Meta) + 2 * kHeads * plan.hg * (4 + padded(D)) * sizeof(float));
}

bool launch_attention_split(const PagedArgs& p, int dtype, cudaStream_t s) {
  return p.window < p.max_len ? launch_attention_window(p, dtype, s) : launch_split<false>(p, dtype, s);
}
#endif

}  // namespace fq
