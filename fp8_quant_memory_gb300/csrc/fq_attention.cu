// fq_attention.cu -- attention of one new token per sequence over a paged FP8 key-value cache, the work
// split over the caches' length and joined.
//
// Mathematics. For a query head with codes q, key rows k_j and value rows v_j (codes), in base 2:
//   x_j = (q . k_j) * (q_scale * softmax_scale * log2 e * k_scale_j),  m = max x,  l = sum 2^(x_j - m),
//   out = (sum 2^(x_j - m) v_scale_j v_j) / l,  lse = (m + log2 l) * ln 2.
// One pass with running m and l. The value sum has a running maximum of its own, M = max (x_j + log2
// v_scale_j): its weights 2^(x_j + log2 v_scale_j - M) are at most 1 whatever the scales of the rows are,
// so they fit fp16 for the tensor cores (rounded by 2^-11 of themselves, or 2^-25 of the largest), and
// partial results (m, l, M, O) join exactly: out = O * 2^(M - m) / l.
//
// What bounds it: every key and value byte is read once and used Hq/Hk <= 16 times, so HBM. The products
// are legacy-shape warp matrix instructions on purpose: the 16 rows of one m16n8 tile hold all query heads
// of a key head, and one step of 16 tokens per warp issues 8 e4m3 products (4.25 clocks each and
// scheduler) and 16 fp16 products (8 clocks), about 230 of the ~700 clocks its 4 KB take to arrive at
// 6.8 TB/s; tcgen05 would need the value tile transposed through shared memory and 128 rows to fill.
//
// Layout. Nothing is exchanged between threads on the way in. Both products contract over an index whose
// order is free as long as both operands agree: thread (g, c) = (lane / 4, lane % 4) takes bytes 64i + 16c
// .. +15 of key rows as the k indices that its B fragments hold, and bytes 16g .. +15 of value rows
// 4c..4c+3, so every cp.async of 16 bytes lands in the thread's own slots of a ring in shared memory, is
// read back by the same thread, and covers whole 64- or 128-byte runs of global memory per row. The score
// tile's columns are numbered so that its accumulators are the weights' A fragment without a shuffle.
//
// Split. The work is a list of units (128 tokens of one sequence and key head, 16 per warp) in the order
// sequence, head, tokens; CTA i of n takes units [i*U/n, (i+1)*U/n). The lengths are on the device, so each
// CTA finds its range itself. A run of units of one head that is not the whole head goes to the workspace
// as a partial result, at most two per CTA (its first and its last), and a second kernel joins them in
// order: no atomics, and the same bits on every run.
#include <math_constants.h>

#include "fq_device.cuh"
#include "fq_serving.h"
#include "fq_sync.cuh"

namespace fq {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 16;                // tokens of one warp per unit
constexpr int kUnit = kStep * kWarps;    // tokens per unit
constexpr int kRows = 16;                // query heads per work item (rows of the score tile)
constexpr float kLowest = -3.402823466e38f;  // below every score: a maximum before the first token

// Ring depth and CTAs per SM by padded head size: two CTAs where the output accumulators (DP/2 registers a
// thread) leave room, and as deep a ring as their shared memory holds.
template <int DP>
struct Shape {
  static constexpr int kCtas = DP <= 128 ? 2 : 1;
  static constexpr int kStages = DP == 64 ? 6 : DP == 128 ? 3 : DP == 192 ? 4 : 3;
  static constexpr int kStageBytes = 2 * kStep * DP;  // codes of one warp's step
  static constexpr int kV16 = DP / 128;               // 16-byte pieces of a value row per lane
  static constexpr int kV8 = (DP % 128) / 64;         // 8-byte pieces
};

constexpr int kJoinStride = 36;  // floats per joined row of 32: float4 stores without bank conflicts

template <int DP>
struct Shared {
  alignas(16) unsigned char codes[kWarps][Shape<DP>::kStages][Shape<DP>::kStageBytes];
  alignas(16) float scales[kWarps][Shape<DP>::kStages][2 * kStep];  // K then V
  uint32_t live[kWarps][Shape<DP>::kStages];                        // bit t: token t of the step counts
  alignas(16) float join[kWarps][8][kJoinStride];
  float stat[kWarps][kRows][3];  // m, M, l
  int64_t scan[kWarps];
  int64_t start_unit;
  int32_t start_b;
};

// What a CTA that begins inside a head leaves for the join of that head.
struct Meta {
  int32_t b, item, last, slot;  // b < 0: nothing to join here; slot: which partial of CTA (this - 1)
};

struct SplitArgs {
  PagedArgs p;
  int32_t G;       // query heads per key head
  int32_t chunks;  // work items per key head: ceil(G / 16)
  int32_t slots;   // 2 * the first kernel's grid
  Meta* meta;      // [grid]
  float* stats;    // [slots][16][4]: m, M, l
  float* part;     // [slots][16][DP]
};

__device__ __forceinline__ int32_t length_of(const PagedArgs& p, int32_t b) {
  return static_cast<int32_t>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(__ldg(p.lens + b)), p.max_len)));
}

__device__ __forceinline__ int32_t tiles_of(int32_t len) { return (len + kUnit - 1) / kUnit; }

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float lg2(float v) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Copies of `bytes` (or zeros in their place) into shared memory.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, bool live) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0)
                 : "memory");
}

__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// A place in the list of units: tile t of work item `item` (key head item / chunks, query heads from
// 16 * (item % chunks)) of sequence b, which has `len` tokens.
struct Place {
  int32_t b, item, t, len;

  __device__ __forceinline__ void step(const SplitArgs& a) {
    if (++t < tiles_of(len)) return;
    t = 0;
    if (++item < a.p.Hk * a.chunks) return;
    item = 0;
    len = 0;
    while (len == 0 && ++b < a.p.B) len = length_of(a.p, b);
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
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  *total = all;
  return v + before;
}

template <typename T, int DP, bool kWide>
__global__ void __launch_bounds__(kThreads, Shape<DP>::kCtas) attention_split_kernel(const SplitArgs a) {
  using S = Shape<DP>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared<DP>& sm = *reinterpret_cast<Shared<DP>*>(smem_raw);
  const PagedArgs& p = a.p;
  const CacheView& cache = p.cache;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // This CTA's units [begin, end) of all U, and the place of the first.
  const int64_t per_tile = static_cast<int64_t>(p.Hk) * a.chunks;
  int64_t total = 0;
  int64_t incl = 0, mine = 0;
  for (int32_t b0 = 0; b0 < p.B; b0 += kThreads) {
    const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
    const int32_t len = b < p.B ? length_of(p, b) : 0;
    mine = tiles_of(len) * per_tile;
    int64_t sum;
    incl = block_scan(mine, sm.scan, &sum);
    total += sum;
    // Sequences without tokens: zeros and -inf, spread over the CTAs.
    if (b < p.B && len == 0 && b % gridDim.x == blockIdx.x) {
      T* o = static_cast<T*>(p.out) + static_cast<int64_t>(b) * p.Hq * p.D;
      for (int64_t i = 0; i < static_cast<int64_t>(p.Hq) * p.D; i += 8)
        *reinterpret_cast<uint4*>(o + i) = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse != nullptr)
        for (int32_t h = 0; h < p.Hq; ++h) p.lse[static_cast<int64_t>(b) * p.Hq + h] = -CUDART_INF_F;
    }
  }
  const int64_t n = min(static_cast<int64_t>(gridDim.x), total);  // CTAs with work
  const int64_t cta = blockIdx.x;
  const int64_t begin = cta < n ? cta * total / n : 0, end = cta < n ? (cta + 1) * total / n : 0;
  if (begin == end) {
    if (threadIdx.x == 0 && a.meta != nullptr) a.meta[cta].b = -1;
    return;
  }
  if (p.B <= kThreads) {
    if (incl - mine <= begin && begin < incl) {
      sm.start_b = threadIdx.x;
      sm.start_unit = begin - (incl - mine);
    }
  } else {
    int64_t carry = 0;
    for (int32_t b0 = 0; b0 < p.B && carry <= begin; b0 += kThreads) {
      const int32_t b = b0 + static_cast<int32_t>(threadIdx.x);
      mine = b < p.B ? tiles_of(length_of(p, b)) * per_tile : 0;
      int64_t sum;
      incl = block_scan(mine, sm.scan, &sum) + carry;
      if (incl - mine <= begin && begin < incl) {
        sm.start_b = b;
        sm.start_unit = begin - (incl - mine);
      }
      carry += sum;
    }
  }
  __syncthreads();
  Place use;
  use.b = sm.start_b;
  use.len = length_of(p, use.b);
  {
    const int32_t nt = tiles_of(use.len);
    use.item = static_cast<int32_t>(sm.start_unit / nt);
    use.t = static_cast<int32_t>(sm.start_unit - static_cast<int64_t>(use.item) * nt);
    if (threadIdx.x == 0 && a.meta != nullptr) {
      // The head this CTA begins inside is joined by the second CTA that has a part of it.
      const int64_t first = begin - use.t;                       // the head's first unit
      const int64_t i0 = ((first + 1) * n - 1) / total;          // the CTA that has it
      const int64_t i1 = ((first + nt) * n - 1) / total;         // the CTA that has its last unit
      Meta m;
      m.b = use.t > 0 && i0 == cta - 1 ? use.b : -1;
      m.item = use.item;
      m.last = static_cast<int32_t>(i1);
      m.slot = i0 * total / n == first ? 0 : 1;
      a.meta[cta] = m;
    }
  }
  const int64_t units = end - begin;

  // ------------------------------------------------------------------------------- way in
  Place next = use;
  int64_t issued = 0;
  // The page of this lane's token of the next unit to be issued, loaded one unit ahead.
  auto page_of = [&](const Place& at) {
    const int32_t tok = at.t * kUnit + warp * kStep + (lane & 15);
    if (tok >= at.len) return -1;
    const int32_t i = cache.page_shift >= 0 ? tok >> cache.page_shift : tok / cache.page_size;
    return __ldg(p.table + static_cast<int64_t>(at.b) * p.table_stride + i);
  };
  int32_t page = page_of(next);
  auto issue = [&](int stage) {
    if (issued < units) {
      const int32_t tok = next.t * kUnit + warp * kStep + (lane & 15);
      const int32_t off = cache.page_shift >= 0 ? tok & (cache.page_size - 1) : tok % cache.page_size;
      const int32_t head = next.item / a.chunks;
      const bool live = page >= 0 && page < cache.pages;
      const int64_t row = live ? page * cache.page_stride + head * cache.head_stride + off * cache.token_stride : -1;
      const int64_t srow = page * cache.s_page_stride + head * cache.s_head_stride + off * cache.s_token_stride;
      const uint32_t mask = __ballot_sync(0xffffffffu, live) & 0xffffu;
      if (lane == 0) sm.live[warp][stage] = mask;
      if (mask != 0u) {
        const uint32_t dst = smem_addr(sm.codes[warp][stage]);
        const float* sbase = lane < 16 ? cache.k_scale : cache.v_scale;
        cp_async<4>(smem_addr(&sm.scales[warp][stage][lane]), live ? sbase + srow : sbase, live);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t r = __shfl_sync(0xffffffffu, row, 4 * (g >> 1) + (g & 1) + 2 * u);
#pragma unroll
          for (int i = 0; i < DP / 64; ++i) {
            const bool ok = r >= 0 && 64 * i + 16 * c < p.D;
            cp_async<16>(dst + ((u * (DP / 64) + i) * 32 + lane) * 16, cache.k + (ok ? r + 64 * i + 16 * c : 0), ok);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t r = __shfl_sync(0xffffffffu, row, 4 * c + e);
#pragma unroll
          for (int i = 0; i < S::kV16; ++i) {
            const bool ok = r >= 0 && 128 * i + 16 * g < p.D;
            cp_async<16>(dst + kStep * DP + (i * 4 + e) * 512 + lane * 16, cache.v + (ok ? r + 128 * i + 16 * g : 0), ok);
          }
          if constexpr (S::kV8 > 0) {
            constexpr int d0 = 128 * S::kV16;
            const bool ok = r >= 0 && d0 + 8 * g < p.D;
            cp_async<8>(dst + kStep * DP + S::kV16 * 2048 + e * 256 + lane * 8, cache.v + (ok ? r + d0 + 8 * g : 0), ok);
          }
        }
      }
      next.step(a);
      if (++issued < units) page = page_of(next);
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < S::kStages - 1; ++s) issue(s);

  // --------------------------------------------------------------------------- the heads
  constexpr int kN = DP / 8;  // output tiles of 8 columns
  uint4 qa[DP / 64], qb[kWide ? DP / 64 : 1];
  float qf[2], m[2], mo[2], l[2];
  float o[kN][4];
  bool first_segment = true;
  bool fresh = true;
  int32_t t0 = use.t;
  int stage = 0, fill = S::kStages - 1;

  for (int64_t u = 0; u < units; ++u) {
    const int32_t rows = min(kRows, a.G - kRows * (use.item % a.chunks));
    const int32_t head0 = use.item / a.chunks * a.G + kRows * (use.item % a.chunks);  // first query head
    if (fresh) {
      fresh = false;
      t0 = use.t;
      const uint8_t* q = p.q + static_cast<int64_t>(use.b) * p.q_stride + static_cast<int64_t>(head0) * p.D;
      const float* qs = p.q_scale + static_cast<int64_t>(use.b) * p.q_scale_stride + head0;
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        const int d = 64 * i + 16 * c;
        qa[i] = g < rows && d < p.D ? __ldg(reinterpret_cast<const uint4*>(q + g * p.D + d)) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (kWide)
          qb[i] = g + 8 < rows && d < p.D ? __ldg(reinterpret_cast<const uint4*>(q + (g + 8) * p.D + d))
                                          : make_uint4(0u, 0u, 0u, 0u);
      }
      qf[0] = g < rows ? __ldg(qs + g) * p.scale_log2 : 0.f;
      qf[1] = kWide && g + 8 < rows ? __ldg(qs + g + 8) * p.scale_log2 : 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[r] = mo[r] = kLowest;
        l[r] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kN; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    }
    cp_wait<S::kStages - 2>();
    __syncwarp();  // the scales and the mask come from other lanes
    issue(fill);
    if (++fill == S::kStages) fill = 0;

    const uint32_t live = sm.live[warp][stage];
    if (live != 0u) {
      const unsigned char* st = sm.codes[warp][stage];
      float s[2][4] = {};
#pragma unroll
      for (int i = 0; i < DP / 64; ++i) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(st + (i * 32 + lane) * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(st + ((DP / 64 + i) * 32 + lane) * 16);
        const uint4 b8 = kWide ? qb[kWide ? i : 0] : make_uint4(0u, 0u, 0u, 0u);
        mma_e4m3(s[0], qa[i].x, b8.x, qa[i].y, b8.y, k0.x, k0.y);
        mma_e4m3(s[1], qa[i].x, b8.x, qa[i].y, b8.y, k1.x, k1.y);
        mma_e4m3(s[0], qa[i].z, b8.z, qa[i].w, b8.w, k0.z, k0.w);
        mma_e4m3(s[1], qa[i].z, b8.z, qa[i].w, b8.w, k1.z, k1.w);
      }
      const float4 ks4 = *reinterpret_cast<const float4*>(&sm.scales[warp][stage][4 * c]);
      const float4 vs4 = *reinterpret_cast<const float4*>(&sm.scales[warp][stage][kStep + 4 * c]);
      const float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w};
      const float lv[4] = {lg2(vs4.x), lg2(vs4.y), lg2(vs4.z), lg2(vs4.w)};
      constexpr int kR = kWide ? 2 : 1;
      uint32_t pa[4] = {0u, 0u, 0u, 0u};
      float keep[2] = {1.f, 1.f};
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        float x[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float v = s[e >> 1][2 * r + (e & 1)] * (qf[r] * ks[e]);
          x[e] = (live >> (4 * c + e)) & 1u ? v : -CUDART_INF_F;
          w[e] = x[e] + lv[e];
          if (!((live >> (4 * c + e)) & 1u)) w[e] = -CUDART_INF_F;
        }
        const float mn = quad_max(fmaxf(fmaxf(m[r], fmaxf(x[0], x[1])), fmaxf(x[2], x[3])));
        const float on = quad_max(fmaxf(fmaxf(mo[r], fmaxf(w[0], w[1])), fmaxf(w[2], w[3])));
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += ex2(x[e] - mn);
        l[r] = fmaf(l[r], ex2(m[r] - mn), sum);
        keep[r] = ex2(mo[r] - on);
        m[r] = mn;
        mo[r] = on;
        pa[r] = pack_f16(ex2(w[0] - on), ex2(w[1] - on));
        pa[2 + r] = pack_f16(ex2(w[2] - on), ex2(w[3] - on));
      }
      if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          o[i][0] *= keep[0];
          o[i][1] *= keep[0];
          o[i][2] *= keep[1];
          o[i][3] *= keep[1];
        }
      }
      const unsigned char* vt = st + kStep * DP;
#pragma unroll
      for (int i = 0; i < S::kV16; ++i) {
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint4*>(vt + (i * 4 + e) * 512 + lane * 16);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t b0[4], b1[4];
          pair_f16(word(v[0], k), word(v[1], k), b0);
          pair_f16(word(v[2], k), word(v[3], k), b1);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(o[i * 16 + 4 * k + j], pa, b0[j], b1[j]);
        }
      }
      if constexpr (S::kV8 > 0) {
        uint2 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint2*>(vt + S::kV16 * 2048 + e * 256 + lane * 8);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t b0[4], b1[4];
          pair_f16(k == 0 ? v[0].x : v[0].y, k == 0 ? v[1].x : v[1].y, b0);
          pair_f16(k == 0 ? v[2].x : v[2].y, k == 0 ? v[3].x : v[3].y, b1);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma_f16(o[S::kV16 * 16 + 4 * k + j], pa, b0[j], b1[j]);
        }
      }
    }
    if (++stage == S::kStages) stage = 0;

    // ------------------------------------------------------------------- the end of a head
    const int32_t nt = tiles_of(use.len);
    const bool done = use.t + 1 == nt;
    if (done || u + 1 == units) {
      const bool whole = done && t0 == 0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (c == 0) {
          sm.stat[warp][g + 8 * r][0] = m[r];
          sm.stat[warp][g + 8 * r][1] = mo[r];
          sm.stat[warp][g + 8 * r][2] = l[r];
        }
      }
      __syncthreads();
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float top = kLowest;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm.stat[w][g + 8 * r][1]);
        f[r] = ex2(mo[r] - top);
      }
      const int64_t slot = 2 * cta + (first_segment ? 0 : 1);
      first_segment = false;
#pragma unroll
      for (int r = 0; r < (kWide ? 2 : 1); ++r) {
        // Thread (warp, lane) finishes row 8*r + warp, column `lane` of each piece of 32.
        const int row = 8 * r + warp;
        float top = kLowest, topo = kLowest, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          top = fmaxf(top, sm.stat[w][row][0]);
          topo = fmaxf(topo, sm.stat[w][row][1]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum = fmaf(sm.stat[w][row][2], ex2(sm.stat[w][row][0] - top), sum);
        const float norm = sum == 0.f ? 0.f : ex2(topo - top) / sum;
        const bool live_row = row < rows;
        const int64_t orow = static_cast<int64_t>(use.b) * p.Hq + head0 + row;
        if (live_row && lane == 0) {
          if (whole) {
            if (p.lse != nullptr) p.lse[orow] = sum == 0.f ? -CUDART_INF_F : (top + log2f(sum)) * 0.693147180559945309f;
          } else {
            float* st = a.stats + (slot * kRows + row) * 4;
            st[0] = top;
            st[1] = topo;
            st[2] = sum;
          }
        }
        auto piece = [&](int n0, int d) {  // output tiles n0..n0+3; d: the column this thread finishes
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float4*>(&sm.join[warp][g][8 * c + 4 * h]) =
                make_float4(o[n0][2 * r + h] * f[r], o[n0 + 1][2 * r + h] * f[r], o[n0 + 2][2 * r + h] * f[r],
                            o[n0 + 3][2 * r + h] * f[r]);
          __syncthreads();
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) v += sm.join[w][warp][lane];
          if (live_row && d < p.D) {
            if (whole) Elem<T>::store1(p.out, orow * p.D + d, v * norm);
            else a.part[(slot * kRows + row) * DP + d] = v;
          }
          __syncthreads();
        };
        // Column `lane` of a piece is (c, h, j) = (lane / 8, lane / 4 % 2, lane % 4).
#pragma unroll
        for (int i = 0; i < S::kV16; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            piece(i * 16 + 4 * k, 128 * i + 16 * (2 * (lane >> 3) + ((lane >> 2) & 1)) + 4 * k + (lane & 3));
        if constexpr (S::kV8 > 0)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            piece(S::kV16 * 16 + 4 * k, 128 * S::kV16 + 8 * (2 * (lane >> 3) + ((lane >> 2) & 1)) + 4 * k + (lane & 3));
      }
      fresh = true;
    }
    use.step(a);
  }
  cp_wait<0>();
}

// Joins the partial results of one head: CTA (k, row) takes the head that CTA k of the first kernel began
// inside. The warps share the parts, each in a fixed order.
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads) attention_join_kernel(const SplitArgs a) {
  constexpr int kV = DP / 64;  // float2 per lane
  __shared__ float2 sum[kWarps][DP / 2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t k = blockIdx.x + 1;
  const Meta me = a.meta[k];
  const PagedArgs& p = a.p;
  if (me.b < 0) return;
  const int32_t row = blockIdx.y;
  const int32_t rows = min(kRows, a.G - kRows * (me.item % a.chunks));
  if (row >= rows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = static_cast<int>(me.last - k + 2);
  auto slot_of = [&](int i) { return i == 0 ? 2 * (k - 1) + me.slot : 2 * (k - 1 + i); };
  float top = kLowest, topo = kLowest;
  for (int i = lane; i < parts; i += 32) {
    const float4 st = *reinterpret_cast<const float4*>(a.stats + (slot_of(i) * kRows + row) * 4);
    top = fmaxf(top, st.x);
    topo = fmaxf(topo, st.y);
  }
  top = group_max<32>(top);
  topo = group_max<32>(topo);
  float l = 0.f;
  for (int i = lane; i < parts; i += 32) {
    const float4 st = *reinterpret_cast<const float4*>(a.stats + (slot_of(i) * kRows + row) * 4);
    l = fmaf(st.z, ex2(st.x - top), l);
  }
  l = group_sum<32>(l);
  float2 v[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) v[i] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < parts; i += kWarps) {
    const int64_t at = slot_of(i) * kRows + row;
    const float f = ex2(a.stats[at * 4 + 1] - topo);
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      const int d = 2 * (lane + 32 * j);
      const float2 x = d < p.D ? *reinterpret_cast<const float2*>(a.part + at * DP + d) : make_float2(0.f, 0.f);
      v[j] = fma2(x, splat2(f), v[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kV; ++j) sum[warp][lane + 32 * j] = v[j];
  __syncthreads();
  const float norm = l == 0.f ? 0.f : ex2(topo - top) / l;
  const int64_t orow = static_cast<int64_t>(me.b) * p.Hq + me.item / a.chunks * a.G + kRows * (me.item % a.chunks) + row;
  for (int d = threadIdx.x; 2 * d < p.D; d += kThreads) {
    float2 r = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) r = add2(r, sum[w][d]);
    static_cast<uint32_t*>(p.out)[(orow * p.D) / 2 + d] = Elem<T>::pack(make_float2(r.x * norm, r.y * norm));
  }
  if (p.lse != nullptr && threadIdx.x == 0)
    p.lse[orow] = l == 0.f ? -CUDART_INF_F : (top + log2f(l)) * 0.693147180559945309f;
}

// ---------------------------------------------------------------------------------- host side
int padded(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

struct Plan {
  int64_t grid, items_per_seq;
  bool join;
};

Plan plan_of(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  Plan q;
  const int64_t G = Hq / Hk, tiles = (max_len + kUnit - 1) / kUnit;
  q.items_per_seq = Hk * ((G + kRows - 1) / kRows);
  const int64_t resident = static_cast<int64_t>(sm_count()) * (padded(D) <= 128 ? 2 : 1);
  const __int128 units = static_cast<__int128>(B) * q.items_per_seq * tiles;
  q.grid = units < resident ? static_cast<int64_t>(units) : resident;
  if (q.grid < 1) q.grid = 1;
  q.join = tiles > 1 && q.grid > 1;
  return q;
}

template <typename T, int DP, bool kWide>
bool launch_dp(const SplitArgs& a, const Plan& plan, cudaStream_t s) {
  auto kern = attention_split_kernel<T, DP, kWide>;
  constexpr size_t smem = sizeof(Shared<DP>);
  static_assert(smem <= 227 * 1024 && (smem + 1024) * Shape<DP>::kCtas <= 228 * 1024, "the ring fits the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  kern<<<static_cast<unsigned>(plan.grid), kThreads, smem, s>>>(a);
  if (!plan.join) return true;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(plan.grid - 1), a.G < kRows ? a.G : kRows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, attention_join_kernel<T, DP>, a);  // a failure is reported by the caller's check
  return true;
}

template <typename T, bool kWide>
bool launch_t(const SplitArgs& a, const Plan& plan, cudaStream_t s) {
  switch (padded(a.p.D)) {
    case 64: return launch_dp<T, 64, kWide>(a, plan, s);
    case 128: return launch_dp<T, 128, kWide>(a, plan, s);
    case 192: return launch_dp<T, 192, kWide>(a, plan, s);
    default: return launch_dp<T, 256, kWide>(a, plan, s);
  }
}

}  // namespace

size_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len) {
  const Plan plan = plan_of(B, Hq, Hk, D, max_len);
  if (!plan.join) return 0;
  return static_cast<size_t>(plan.grid) * (sizeof(Meta) + 2 * kRows * (4 + padded(D)) * sizeof(float));
}

bool launch_attention_split(const PagedArgs& p, int dtype, cudaStream_t s) {
  const Plan plan = plan_of(p.B, p.Hq, p.Hk, p.D, p.max_len);
  if (plan.items_per_seq > 0x7fffffffLL) return false;
  SplitArgs a{};
  a.p = p;
  a.G = p.Hq / p.Hk;
  a.chunks = (a.G + kRows - 1) / kRows;
  a.slots = static_cast<int32_t>(2 * plan.grid);
  if (plan.join) {
    a.meta = reinterpret_cast<Meta*>(p.partial);
    a.stats = reinterpret_cast<float*>(a.meta + plan.grid);
    a.part = a.stats + static_cast<int64_t>(a.slots) * kRows * 4;
  }
  const bool wide = a.G > 8;
  if (dtype == DT_BF16) return wide ? launch_t<__nv_bfloat16, true>(a, plan, s) : launch_t<__nv_bfloat16, false>(a, plan, s);
  return wide ? launch_t<__half, true>(a, plan, s) : launch_t<__half, false>(a, plan, s);
}

}  // namespace fq
