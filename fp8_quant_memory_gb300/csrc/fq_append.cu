// fq_append.cu -- the QK-Norm + RoPE + FP8 prologue on whole QKV rows, K and V placed in a paged FP8 cache.
//
// Mathematics: q and k rows as the prologue (fq_rows.cuh, MODE_QK: norm, rotation, one scale per row, all in fp32);
// v rows are quantised as they are. What bounds it: HBM, 2 bytes read and 1 written per element. One pass: every
// element is read once, held in registers through norm, rotation and row maximum, and leaves as a code in its place
// in the cache, so nothing is written and read again between the prologue and the cache.
//
// Two kernels. Heads of 128 columns, all rotated, in packed QKV rows (the usual shape) stream through a ring of shared
// memory (append_stream_kernel); other shapes take a register kernel (append_kernel).
//
// append_kernel: a group of LPR lanes owns a (token, head) row, as in fq_rows.cu; consecutive groups take consecutive rows,
// so loads cover whole contiguous runs of the QKV row. Rows of q and k and rows of v meet in a warp only where the
// head counts are not multiples of its rows; such a warp runs both bodies, each with its own rows live.
#include <math_constants.h>

#include "fq_device.cuh"
#include "fq_rows.cuh"
#include "fq_serving.h"
#include "fq_sync.cuh"

namespace fq {
namespace {

using namespace rows;

constexpr int kThreads = 256;
// Rows from which the streaming kernel is the faster one (48 rows a token: 256 tokens take 3.41 us in it and 3.25 in the
// register kernel, 512 take 4.27 and 4.95, 2048 take 9.1 and 13.1).
constexpr int64_t kStreamRows = 16384;

// Page and offset of a slot.
__device__ __forceinline__ void locate(const CacheView& c, int64_t slot, int64_t* page, int64_t* off) {
  if (c.page_shift >= 0) {
    *page = slot >> c.page_shift;
    *off = slot & (c.page_size - 1);
  } else if (slot <= 0xffffffffll) {
    const uint32_t p = static_cast<uint32_t>(slot) / static_cast<uint32_t>(c.page_size);
    *page = p;
    *off = static_cast<uint32_t>(slot) - p * static_cast<uint32_t>(c.page_size);
  } else {
    *page = slot / c.page_size;
    *off = slot - *page * c.page_size;
  }
}

// The divisor in div2_by's correction. A row that holds an infinity has an infinite scale, whose reciprocal is 0: its
// finite values' quotients are their products with that, 0, and a correction by infinity times 0 would make them NaN.
__device__ __forceinline__ float corrected_by(float scale) { return scale == CUDART_INF_F ? 0.f : scale; }

template <typename T, typename TT, int LPR, int HS, int TS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs p) {
  constexpr int kRowsPerCta = kThreads / LPR;
  constexpr int kV = HS + 2 * TS;
  const RowArgs& a = p.rows;
  const int lane = threadIdx.x & (LPR - 1), grp = threadIdx.x / LPR;
  const int N = a.N, nv = N >> 3, hv = (N - a.R) >> 3, th = a.R >> 4, half = a.R >> 1;
  const int32_t rows = static_cast<int32_t>(a.rows);
  pdl_trigger();
  pdl_wait();
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kRowsPerCta; base < rows; base += static_cast<int64_t>(gridDim.x) * kRowsPerCta) {
    const bool inside = base + grp < rows;
    const int32_t r = inside ? static_cast<int32_t>(base) + grp : 0;
    const int32_t t = inside ? r / a.H : 0, h = inside ? r - t * a.H : 0;
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + p.Hk;
    const T* x = static_cast<const T*>(a.x) + (static_cast<int64_t>(t) * a.token_stride + static_cast<int64_t>(h) * N);
    // Vector s of a lane: in the order of the rotation's halves for q and k, plain order for v.
    uint4 xv[kV];
#pragma unroll
    for (int s = 0; s < kV; ++s) {
      const bool ok = is_v ? lane + s * LPR < nv : slot_ok<LPR, HS, TS>(s, lane, hv, th);
      const int col = is_v ? 8 * (lane + s * LPR) : slot_col<LPR, HS, TS>(s, lane, hv, th);
      xv[s] = inside && ok ? ld_stream16(x + col) : make_uint4(0u, 0u, 0u, 0u);
    }
    uint8_t* codes = a.q + (static_cast<int64_t>(t) * a.Hq + h) * N;
    float* scale = a.scale + static_cast<int64_t>(t) * a.Hq + h;
    bool live = inside;
    if (!is_q) {
      const int64_t slot = p.slots[t];
      live = inside && slot >= 0 && slot < p.cache.pages * p.cache.page_size;
      int64_t page = 0, off = 0;
      if (live) locate(p.cache, slot, &page, &off);
      const int32_t head = is_v ? h - a.Hq - p.Hk : h - a.Hq;
      codes = (is_v ? p.cache.v : p.cache.k) + page * p.cache.page_stride + head * p.cache.head_stride + off * p.cache.token_stride;
      scale = (is_v ? p.cache.v_scale : p.cache.k_scale) + page * p.cache.s_page_stride + head * p.cache.s_head_stride +
              off * p.cache.s_token_stride;
    }
    if (__any_sync(0xffffffffu, inside && !is_v)) {
      RowArgs row = a;  // row 0 of these outputs is this row's place
      row.q = codes;
      row.scale = scale;
      row_body<T, TT, MODE_QK, LPR, HS, TS, false, false, true>(row, 0, live && !is_v, h, xv, lane, hv, th, static_cast<float>(N), a.cos,
                                                   a.sin, static_cast<int64_t>(t) * half);
    }
    if (__any_sync(0xffffffffu, inside && is_v)) {
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < kV; ++s)
#pragma unroll
        for (int k = 0; k < 4; k += 2) amax = absmax4(amax, Elem<T>::unpack(word(xv[s], k)), Elem<T>::unpack(word(xv[s], k + 1)));
      amax = fmaxf(group_max<LPR>(amax), 1e-4f);
      const float sc = __fdiv_rn(amax, a.fp8_max), rc = __frcp_rn(sc), by = corrected_by(sc);
      const bool clamp = a.fp8_max != 448.0f;
      if (live && is_v) {
#pragma unroll
        for (int s = 0; s < kV; ++s) {
          if (lane + s * LPR >= nv) continue;
          float2 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = div2_by(Elem<T>::unpack(word(xv[s], k)), by, rc);
            if (clamp) v[k] = make_float2(clamp_or_nan(v[k].x, a.fp8_max), clamp_or_nan(v[k].y, a.fp8_max));
          }
          st_stream8(codes + 8 * (lane + s * LPR), pack_e4m3x8(v[0], v[1], v[2], v[3]));
        }
        if (lane == 0) *scale = sc;
      }
    }
  }
}

template <typename T, typename TT, int LPR, int HS, int TS>
bool launch_shape(const AppendArgs& p, cudaStream_t s) {
  auto kern = append_kernel<T, TT, LPR, HS, TS>;
  constexpr int kRowsPerCta = kThreads / LPR;
  const int64_t need = (p.rows.rows + kRowsPerCta - 1) / kRowsPerCta, cap = static_cast<int64_t>(sm_count()) * 8;
  launch_overlapped(kern, dim3(static_cast<unsigned>(need < cap ? need : cap)), kThreads, 0, 1, s, p);
  return true;
}

// (LPR, HS, TS) covers hv = (D - R) / 8 <= LPR*HS head vectors, th = R / 16 <= LPR*TS rotated pairs of vectors and
// D / 8 <= LPR*(HS + 2*TS) vectors of a v row.
template <typename T, typename TT>
bool launch_typed(const AppendArgs& p, cudaStream_t s) {
  const int hv = (p.rows.N - p.rows.R) / 8, th = p.rows.R / 16;
  if (hv == 0 && th <= 8) return launch_shape<T, TT, 8, 0, 1>(p, s);
  if (hv <= 16 && th <= 8) return launch_shape<T, TT, 8, 2, 1>(p, s);
  if (hv <= 32 && th <= 16) return launch_shape<T, TT, 16, 2, 1>(p, s);
  if (hv <= 64 && th <= 32) return launch_shape<T, TT, 32, 2, 1>(p, s);
  return false;
}

// ------------------------------------------------------------------------------------ stream
// Rows of 128 columns, all rotated. A producer warp brings chunks of 32 consecutive (token, head) rows, the cos and
// sin rows of their tokens and the tokens' slots into a ring of stages (1-D bulk copies); four consumer
// warps take a chunk, eight rows each, four lanes to a row, two such groups taking alternate chunks. Lane j of a row
// holds the NeoX pairs 16j..16j+15, so the rotation needs no exchange. The weights stay in shared memory: in registers
// they spill. A lane walks its two sub-chunks of eight pairs in an order that depends on j and on the row, which spreads
// the eight lanes of a 16-byte access phase over all banks for the rows and for the tables.
//
// Arithmetic (q and k): u = x*w exactly in fp32 (two 8- or 11-bit significands), z = rope(u), rstd = 1/sqrt(sum x^2
// / 128 + eps); the definition's y equals rstd * z up to rounding, and so do amax = rstd * max |z| and the codes
// e4m3(z * m) with m = rstd / scale. rstd and m come from the hardware's approximations with one Newton step each,
// which brings them within an ulp: the codes sit as near to the 64-bit definition as those of fp32 steps, though a few in
// a million, at ties, are not the other kernel's. The scale is amax / fp8_max correctly rounded, by Markstein's
// correction of a quotient from a correctly rounded reciprocal. v rows are divided by their scale exactly, as everywhere.
constexpr int kSD = 128;
constexpr int kSRows = 32;                         // rows per stage
constexpr int kSWarps = 8;                         // consumer warps
constexpr int kSThreads = (kSWarps + 1) * 32;
constexpr int kSRowBytes = kSD * 2;

struct StreamArgs {
  AppendArgs p;
  uint32_t magic;  // t = (r * magic) >> shift == r / H for r < 2^31
  int32_t shift, stages, stage_bytes, tab_block, chunks;
  float rcp_fp8_max;
  unsigned int* status;
};

__device__ __forceinline__ uint32_t token_of(uint32_t r, const StreamArgs& a) {
  return static_cast<uint32_t>((static_cast<uint64_t>(r) * a.magic) >> a.shift);
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Eight table entries in shared memory -> 4 pairs.
template <typename TT>
__device__ __forceinline__ void lds_table8(uint32_t addr, float2 (&v)[4]) {
  if constexpr (sizeof(TT) == 4) {
    const uint4 a = lds16(addr), b = lds16(addr + 16);
    v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
    v[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
    v[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
  } else {
    const uint4 u = lds16(addr);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = Elem<TT>::unpack(word(u, e));
  }
}

// Sixteen codes of each half of the row, the lane's two sub-chunks put back into column order.
__device__ __forceinline__ void store_codes(uint8_t* row, int j, int flip, const uint2 (&lo)[2], const uint2 (&hi)[2]) {
  const uint2 l0 = flip ? lo[1] : lo[0], l1 = flip ? lo[0] : lo[1], h0 = flip ? hi[1] : hi[0], h1 = flip ? hi[0] : hi[1];
  st_stream16(row + 16 * j, make_uint4(l0.x, l0.y, l1.x, l1.y));
  st_stream16(row + kSD / 2 + 16 * j, make_uint4(h0.x, h0.y, h1.x, h1.y));
}

// The codes of a row whose sum of squares left fp32 (rstd = 0), where x*w or its rotation may have left it too: by the
// definition's order y = rope((x * 0) * w), zeros, and NaN where one of a pair is not finite.
template <typename T>
__device__ __noinline__ void store_zero_row(uint32_t xrow, uint32_t w, int j, uint8_t* codes) {
  uint2 c[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t at = xrow + (2 * j + m) * 16, wat = w + (2 * j + m) * 16;
    const uint4 xl = lds16(at), xh = lds16(at + kSRowBytes / 2), wl = lds16(wat), wh = lds16(wat + kSRowBytes / 2);
    float2 z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      z[e] = add2(mul2(mul2(Elem<T>::unpack(word(xl, e)), splat2(0.f)), Elem<T>::unpack(word(wl, e))),
                  mul2(mul2(Elem<T>::unpack(word(xh, e)), splat2(0.f)), Elem<T>::unpack(word(wh, e))));
    c[m] = pack_e4m3x8(z[0], z[1], z[2], z[3]);
  }
  store_codes(codes, j, 0, c, c);
}

// One q or k row by its four lanes; `xrow`, `tab` and `w` are shared-memory addresses (cos row, sin is one block
// further; the head type's weight row).
template <typename T, typename TT, bool kClamp>
__device__ __forceinline__ void stream_qk(const StreamArgs& a, uint32_t xrow, uint32_t tab, int j, int flip, uint32_t w,
                                          uint8_t* codes, float* scale, bool live) {
  const RowArgs& r = a.p.rows;
  float2 zl[2][4], zh[2][4], acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
  float am = 0.f;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int sub = m ^ flip;
    const uint32_t at = xrow + (2 * j + sub) * 16;
    const uint4 xl = lds16(at), xh = lds16(at + kSRowBytes / 2);
    const uint4 wl = lds16(w + (2 * j + sub) * 16), wh = lds16(w + (2 * j + sub) * 16 + kSRowBytes / 2);
    float2 c[4], s[4];
    const uint32_t t8 = tab + (2 * j + sub) * 8 * static_cast<int>(sizeof(TT));
    lds_table8<TT>(t8, c);
    lds_table8<TT>(t8 + a.tab_block, s);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc0 = Mixed<T>::sq_add(word(xl, e), acc0);
      acc1 = Mixed<T>::sq_add(word(xh, e), acc1);
      const float2 ul = Mixed<T>::mul(word(xl, e), word(wl, e)), uh = Mixed<T>::mul(word(xh, e), word(wh, e));
      zl[m][e] = fma2(neg2(uh), s[e], mul2(ul, c[e]));
      zh[m][e] = fma2(ul, s[e], mul2(uh, c[e]));
    }
    am = absmax4(absmax4(am, zl[m][0], zh[m][0]), zl[m][1], zh[m][1]);
    am = absmax4(absmax4(am, zl[m][2], zh[m][2]), zl[m][3], zh[m][3]);
  }
  const float2 a01 = add2(acc0, acc1);
  float ss = a01.x + a01.y;
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  }
  const float v = __fadd_rn(__fmul_rn(ss, 0.0078125f), r.eps);
  const float r0 = rsqrtf(v);
  // r0 + r0/2 * (1 - v r0^2); where v is 0 or not finite the approximation is the answer
  const float e0 = __fmaf_rn(-v * r0, r0, 1.0f);
  const float rstd = fabsf(e0) < 0.5f ? __fmaf_rn(0.5f * r0, e0, r0) : r0;
  const float amax = fmaxf(__fmul_rn(rstd, am), 1e-4f);
  const float s0 = __fmul_rn(amax, a.rcp_fp8_max);
  const float sc = __fmaf_rn(__fmaf_rn(-s0, r.fp8_max, amax), a.rcp_fp8_max, s0);  // amax / fp8_max (Markstein)
  float rc;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc) : "f"(sc));
  rc = __fmaf_rn(rc, __fmaf_rn(-sc, rc, 1.0f), rc);
  const float2 m2 = splat2(__fmul_rn(rstd, rc));
  uint2 lo[2], hi[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float2 l[4], h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      l[e] = mul2(zl[m][e], m2);
      h[e] = mul2(zh[m][e], m2);
      if constexpr (kClamp) {
        l[e] = make_float2(clamp_or_nan(l[e].x, r.fp8_max), clamp_or_nan(l[e].y, r.fp8_max));
        h[e] = make_float2(clamp_or_nan(h[e].x, r.fp8_max), clamp_or_nan(h[e].y, r.fp8_max));
      }
    }
    lo[m] = pack_e4m3x8(l[0], l[1], l[2], l[3]);
    hi[m] = pack_e4m3x8(h[0], h[1], h[2], h[3]);
  }
  if (live) {
    store_codes(codes, j, flip, lo, hi);
    if (j == 0) *scale = sc;
    if (rstd == 0.f) store_zero_row<T>(xrow, w, j, codes);
  }
}

// One v row.
template <typename T, bool kClamp>
__device__ __forceinline__ void stream_v(const StreamArgs& a, uint32_t xrow, int j, int flip, uint8_t* codes, float* scale, bool live) {
  const float fp8_max = a.p.rows.fp8_max;
  uint4 xl[2], xh[2];
  float am = 0.f;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const uint32_t at = xrow + (2 * j + (m ^ flip)) * 16;
    xl[m] = lds16(at);
    xh[m] = lds16(at + kSRowBytes / 2);
#pragma unroll
    for (int e = 0; e < 4; ++e) am = absmax4(am, Elem<T>::unpack(word(xl[m], e)), Elem<T>::unpack(word(xh[m], e)));
  }
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
  const float sc = __fdiv_rn(fmaxf(am, 1e-4f), fp8_max), rc = __frcp_rn(sc), by = corrected_by(sc);
  uint2 lo[2], hi[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    float2 l[4], h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      l[e] = div2_by(Elem<T>::unpack(word(xl[m], e)), by, rc);
      h[e] = div2_by(Elem<T>::unpack(word(xh[m], e)), by, rc);
      if constexpr (kClamp) {
        l[e] = make_float2(clamp_or_nan(l[e].x, fp8_max), clamp_or_nan(l[e].y, fp8_max));
        h[e] = make_float2(clamp_or_nan(h[e].x, fp8_max), clamp_or_nan(h[e].y, fp8_max));
      }
    }
    lo[m] = pack_e4m3x8(l[0], l[1], l[2], l[3]);
    hi[m] = pack_e4m3x8(h[0], h[1], h[2], h[3]);
  }
  if (live) {
    store_codes(codes, j, flip, lo, hi);
    if (j == 0) *scale = sc;
  }
}

__host__ __device__ constexpr size_t stream_smem(int stages, int stage_bytes) {
  return static_cast<size_t>(stages) * stage_bytes + 2 * stages * sizeof(uint64_t) + 2 * kSRowBytes;
}

template <typename T, typename TT, bool kClamp>
__global__ void __launch_bounds__(kSThreads, 2) append_stream_kernel(const __grid_constant__ StreamArgs a) {
  constexpr int kTabRow = (kSD / 2) * static_cast<int>(sizeof(TT));
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + static_cast<size_t>(a.stages) * a.stage_bytes);
  uint64_t* empty = full + a.stages;
  unsigned char* weights = reinterpret_cast<unsigned char*>(empty + a.stages);  // q's row, then k's
  const RowArgs& r = a.p.rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t rows = static_cast<int32_t>(r.rows);
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&full[s], 33);            // lane 0 for the bulk copies, and each lane's slot
      mbar_init(&empty[s], kSWarps / 2);  // a chunk is one half of the consumers'
    }
    fence_barrier_init();
  }
  pdl_trigger();
  pdl_wait();
  if (threadIdx.x < 32)
    *reinterpret_cast<uint4*>(weights + 16 * threadIdx.x) =
        ld_cached16(static_cast<const T*>(threadIdx.x < 16 ? r.wq : r.wk) + 8 * (threadIdx.x & 15));
  __syncthreads();
  const int32_t mine = (a.chunks - static_cast<int32_t>(blockIdx.x) + static_cast<int32_t>(gridDim.x) - 1) / static_cast<int32_t>(gridDim.x);

  if (warp == kSWarps) {
    // ------------------------------------------------------------------------ producer
    int s = 0;
    uint32_t phase = 1;
    int32_t k = 0;
    for (; k < mine; ++k) {
      if (k >= a.stages && !__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &empty[s], phase))) break;
      const int32_t rs = (static_cast<int32_t>(blockIdx.x) + k * static_cast<int32_t>(gridDim.x)) * kSRows, re = min(rs + kSRows, rows);
      const uint32_t tf = token_of(rs, a), tl = token_of(re - 1, a), tokens = tl - tf + 1;
      unsigned char* st = smem + static_cast<size_t>(s) * a.stage_bytes;
      if (lane < static_cast<int>(tokens))  // the tokens' slots, copied: waiting for them here would cost a load per chunk
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(st + kSRows * kSRowBytes + 2 * a.tab_block) + 8 * lane),
                     "l"(a.p.slots + tf + lane)
                     : "memory");
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&full[s])) : "memory");
      if (lane == 0) {
        const uint32_t xbytes = static_cast<uint32_t>(re - rs) * kSRowBytes;
        mbar_arrive_expect_tx(&full[s], xbytes + 2u * tokens * kTabRow);
        bulk_g2s(st, static_cast<const unsigned char*>(r.x) + static_cast<int64_t>(rs) * kSRowBytes, xbytes, &full[s]);
        unsigned char* tab = st + kSRows * kSRowBytes;
        bulk_g2s(tab, static_cast<const unsigned char*>(r.cos) + static_cast<int64_t>(tf) * kTabRow, tokens * kTabRow, &full[s]);
        bulk_g2s(tab + a.tab_block, static_cast<const unsigned char*>(r.sin) + static_cast<int64_t>(tf) * kTabRow, tokens * kTabRow,
                 &full[s]);
      }
      if (++s == a.stages) {
        s = 0;
        phase ^= 1u;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (k < mine) {
      flag_failure(a.status);
      // Let the copies already issued land before this CTA's shared memory goes away.
      for (int32_t i = max(0, k - a.stages); i < k; ++i)
        if (!mbar_wait(kWaitLimitNs, &full[i % a.stages], static_cast<uint32_t>(i / a.stages) & 1u)) break;
    }
    return;
  }

  // -------------------------------------------------------------------------- consumers
  const int g = lane >> 2, j = lane & 3;
  const int half = warp / (kSWarps / 2), l = (warp % (kSWarps / 2)) * 8 + g;  // the lane group's row of a chunk
  const int flip = (j >> 1) ^ (g & 1);
  for (int32_t k = half; k < mine; k += 2) {
    const int s = k % a.stages;
    if (!__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &full[s], static_cast<uint32_t>(k / a.stages) & 1u))) {
      flag_failure(a.status);
      return;
    }
    const unsigned char* st = smem + static_cast<size_t>(s) * a.stage_bytes;
    const int32_t rs = (static_cast<int32_t>(blockIdx.x) + k * static_cast<int32_t>(gridDim.x)) * kSRows;
    const bool inside = rs + l < rows;
    const uint32_t row = static_cast<uint32_t>(inside ? rs + l : rs);  // a lane group without a row reads the chunk's first
    const uint32_t t = token_of(row, a), tf = token_of(rs, a);
    const int32_t h = static_cast<int32_t>(row - t * static_cast<uint32_t>(r.H));
    const bool is_q = h < r.Hq, is_v = h >= r.Hq + a.p.Hk;
    const uint32_t base = smem_addr(st), xrow = base + static_cast<uint32_t>(row - rs) * kSRowBytes;
    const uint32_t tab = base + kSRows * kSRowBytes + (t - tf) * kTabRow;
    uint8_t* codes = r.q + (static_cast<int64_t>(t) * r.Hq + h) * kSD;
    float* scale = r.scale + static_cast<int64_t>(t) * r.Hq + h;
    bool live = inside;
    if (!is_q) {
      const CacheView& c = a.p.cache;
      const int64_t slot = *reinterpret_cast<const int64_t*>(st + kSRows * kSRowBytes + 2 * a.tab_block + 8 * (t - tf));
      live = inside && slot >= 0 && slot < c.pages * c.page_size;
      int64_t page = 0, off = 0;
      if (live) locate(c, slot, &page, &off);
      const int32_t head = is_v ? h - r.Hq - a.p.Hk : h - r.Hq;
      codes = (is_v ? c.v : c.k) + page * c.page_stride + off * c.token_stride + head * c.head_stride;
      scale = (is_v ? c.v_scale : c.k_scale) + page * c.s_page_stride + off * c.s_token_stride + head * c.s_head_stride;
    }
    const uint32_t vmask = __ballot_sync(0xffffffffu, is_v);
    const uint32_t w = smem_addr(weights) + (is_q ? 0 : kSRowBytes);
    if (vmask != 0xffffffffu) stream_qk<T, TT, kClamp>(a, xrow, tab, j, flip, w, codes, scale, live && !is_v);
    if (vmask != 0u) stream_v<T, kClamp>(a, xrow, j, flip, codes, scale, live && is_v);
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
  }
}

template <typename T, typename TT>
bool launch_stream(const AppendArgs& p, cudaStream_t s) {
  StreamArgs a{};
  a.p = p;
  a.status = device_status_ptr();
  a.rcp_fp8_max = static_cast<float>(1.0 / static_cast<double>(p.rows.fp8_max));
  const int32_t H = p.rows.H;
  int lg = 0;
  while ((1LL << lg) < H) ++lg;
  a.shift = 31 + lg;
  const uint64_t magic = static_cast<uint64_t>(((static_cast<unsigned __int128>(1) << a.shift) + H - 1) / H);
  if (magic > 0xffffffffull) return false;
  a.magic = static_cast<uint32_t>(magic);
  const int tokens = (kSRows - 1) / H + 2;  // a chunk touches at most
  if (tokens > 32) return false;
  a.tab_block = (tokens * (kSD / 2) * static_cast<int>(sizeof(TT)) + 15) & ~15;
  a.stage_bytes = (kSRows * kSRowBytes + 2 * a.tab_block + tokens * 8 + 127) & ~127;
  a.stages = 110 * 1024 / a.stage_bytes;  // two CTAs per SM
  if (a.stages > 12) a.stages = 12;
  // Even, so that a stage always belongs to the same half of the consumers: waiting for chunk k by parity is sound only
  // once the stage's previous chunk has landed, which the half that consumed it knows.
  a.stages &= ~1;
  if (a.stages < 4) return false;
  a.chunks = static_cast<int32_t>((p.rows.rows + kSRows - 1) / kSRows);
  const size_t smem = stream_smem(a.stages, a.stage_bytes);
  auto kern = p.rows.fp8_max != 448.0f ? append_stream_kernel<T, TT, true> : append_stream_kernel<T, TT, false>;
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  const int32_t resident = 2 * sm_count();
  launch_overlapped(kern, dim3(static_cast<unsigned>(a.chunks < resident ? a.chunks : resident)), kSThreads, smem, 1, s, a);
  return true;
}

}  // namespace

bool launch_append_vector(const AppendArgs& p, int dtype, int table_dtype, cudaStream_t s) {
  if (p.rows.N == kSD && p.rows.R == kSD && p.rows.token_stride == static_cast<int64_t>(p.rows.H) * kSD &&
      p.rows.rows >= kStreamRows) {
    const bool done = table_dtype == DT_FP32
                          ? (dtype == DT_BF16 ? launch_stream<__nv_bfloat16, float>(p, s) : launch_stream<__half, float>(p, s))
                          : (dtype == DT_BF16 ? launch_stream<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_stream<__half, __half>(p, s));
    if (done) return true;
  }
  if (p.rows.R > 0 && table_dtype == DT_FP32)
    return dtype == DT_BF16 ? launch_typed<__nv_bfloat16, float>(p, s) : launch_typed<__half, float>(p, s);
  return dtype == DT_BF16 ? launch_typed<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_typed<__half, __half>(p, s);
}

}  // namespace fq
