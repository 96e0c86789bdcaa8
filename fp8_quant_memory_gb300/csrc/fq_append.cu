// fq_append.cu -- the QK-Norm + RoPE + FP8 prologue on whole QKV rows, K and V placed in a paged FP8 cache.
//
// Mathematics: q and k rows as the prologue (fq_rows.cuh, MODE_QK: norm, rotation, one scale per row, all in fp32);
// v rows are quantised as they are. What bounds it: HBM, 2 bytes read and 1 written per element. One pass: every
// element is read once, held in registers through norm, rotation and row maximum, and leaves as a code in its place
// in the cache, so nothing is written and read again between the prologue and the cache.
//
// Layout: a warp takes a token, or a part of its heads where there are few tokens, and walks over its rows 32 / LPR at
// a time, LPR lanes to a row. A lane holds the same columns of every row, so the token's cos and sin entries and the
// norm weight of the current head type stay in its registers, and the next rows' loads are issued before the current
// rows are computed. Each NeoX pair sits in one lane (slot_col in fq_rows.cuh). Rows of different types meet in a
// warp step only where the head counts are not multiples of its rows; such a step runs both bodies, each with its own
// rows live.
#include "fq_device.cuh"
#include "fq_rows.cuh"
#include "fq_serving.h"

namespace fq {
namespace {

using namespace rows;

constexpr int kThreads = 256;

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

// y of a q or k row from its vectors: normalised, the tail rotated, all in fp32, each step rounded as the definition's.
template <typename T, int LPR, int HS, int TS>
__device__ __forceinline__ void norm_rope(const uint4 (&xv)[HS + 2 * TS], const uint4 (&wv)[HS + 2 * TS],
                                          const float2 (&c)[TS][4], const float2 (&s)[TS][4], float fN, float eps,
                                          float2 (&y)[HS + 2 * TS][4]) {
  float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < HS + 2 * TS; ++v) {
    acc0 = Mixed<T>::sq_add(xv[v].x, acc0);
    acc1 = Mixed<T>::sq_add(xv[v].y, acc1);
    acc0 = Mixed<T>::sq_add(xv[v].z, acc0);
    acc1 = Mixed<T>::sq_add(xv[v].w, acc1);
  }
  const float2 acc = add2(acc0, acc1);
  const float2 rstd = splat2(rstd_from_ss(group_sum<LPR>(acc.x + acc.y), fN, eps));
#pragma unroll
  for (int v = 0; v < HS; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      y[v][k] = mul2(mul2(Elem<T>::unpack(word(xv[v], k)), rstd), Elem<T>::unpack(word(wv[v], k)));
#pragma unroll
  for (int v = 0; v < TS; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int l = HS + v, h = HS + TS + v;
      const float2 lo = mul2(mul2(Elem<T>::unpack(word(xv[l], k)), rstd), Elem<T>::unpack(word(wv[l], k)));
      const float2 hi = mul2(mul2(Elem<T>::unpack(word(xv[h], k)), rstd), Elem<T>::unpack(word(wv[h], k)));
      y[l][k] = sub2(mul2(lo, c[v][k]), mul2(hi, s[v][k]));
      y[h][k] = add2(mul2(hi, c[v][k]), mul2(lo, s[v][k]));
    }
}

template <typename T, typename TT, int LPR, int HS, int TS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs p, const int32_t steps,
                                                          const int32_t parts) {
  constexpr int kRows = 32 / LPR;  // rows of a warp step
  constexpr int kV = HS + 2 * TS;
  const RowArgs& a = p.rows;
  const int lane = threadIdx.x & (LPR - 1), g = (threadIdx.x & 31) / LPR;
  const int N = a.N, nv = N >> 3, hv = (N - a.R) >> 3, th = a.R >> 4, half = a.R >> 1;
  const float fN = static_cast<float>(N);
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);  // one warp's
  const int32_t t = static_cast<int32_t>(item / parts), part = static_cast<int32_t>(item - static_cast<int64_t>(t) * parts);
  if (static_cast<int64_t>(t) * a.H >= a.rows) return;
  const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(t) * a.token_stride;

  // The token's place in the cache and its table entries.
  const int64_t slot = __ldg(p.slots + t);
  const bool kept = slot >= 0 && slot < p.cache.pages * p.cache.page_size;
  int64_t place = 0, splace = 0;
  if (kept) {
    int64_t page, off;
    locate(p.cache, slot, &page, &off);
    place = page * p.cache.page_stride + off * p.cache.token_stride;
    splace = page * p.cache.s_page_stride + off * p.cache.s_token_stride;
  }
  float2 c[TS][4], s[TS][4];
#pragma unroll
  for (int v = 0; v < TS; ++v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c[v][k] = s[v][k] = make_float2(0.f, 0.f);
    if (lane + v * LPR < th) {
      const int64_t at = static_cast<int64_t>(t) * half + 8 * (lane + v * LPR);
      load_table8<TT, false>(a.cos, at, c[v]);
      load_table8<TT, false>(a.sin, at, s[v]);
    }
  }

  // Vector v of this lane of row h: the rotation's halves for q and k, plain order for v rows.
  auto fetch = [&](int32_t h, uint4 (&xv)[kV]) {
    const bool is_v = h >= a.Hq + p.Hk;
    const T* row = x + static_cast<int64_t>(h) * N;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const bool ok = h < a.H && (is_v ? lane + v * LPR < nv : slot_ok<LPR, HS, TS>(v, lane, hv, th));
      const int col = is_v ? 8 * (lane + v * LPR) : slot_col<LPR, HS, TS>(v, lane, hv, th);
      xv[v] = ok ? ld_stream16(row + col) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  const int32_t first = part * steps * kRows + g;
  uint4 next[kV], wv[kV];
  fetch(first, next);
  int held = -1;  // whose weight wv is: 0 q, 1 k
  const bool clamp = a.fp8_max != 448.0f;
  for (int32_t i = 0; i < steps; ++i) {
    const int32_t h = first + i * kRows;
    if (h - g >= a.H) break;  // warp-uniform
    uint4 xv[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) xv[v] = next[v];
    if (i + 1 < steps) fetch(h + kRows, next);
    const bool inside = h < a.H, is_q = h < a.Hq, is_v = h >= a.Hq + p.Hk;
    float2 y[kV][4];
    if (__any_sync(0xffffffffu, inside && !is_v)) {
      const int type = is_q ? 0 : 1;
      if (held != type) {
        held = type;
        const T* w = static_cast<const T*>(is_q ? a.wq : a.wk);
#pragma unroll
        for (int v = 0; v < kV; ++v)
          wv[v] = slot_ok<LPR, HS, TS>(v, lane, hv, th) ? ld_cached16(w + slot_col<LPR, HS, TS>(v, lane, hv, th))
                                                       : make_uint4(0u, 0u, 0u, 0u);
      }
      norm_rope<T, LPR, HS, TS>(xv, wv, c, s, fN, a.eps, y);
    }
    if (is_v) {
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int k = 0; k < 4; ++k) y[v][k] = Elem<T>::unpack(word(xv[v], k));
    }
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) amax = absmax4(absmax4(amax, y[v][0], y[v][1]), y[v][2], y[v][3]);
    amax = fmaxf(group_max<LPR>(amax), 1e-4f);
    const float sc = __fdiv_rn(amax, a.fp8_max), rc = __frcp_rn(sc);
    const int32_t head = is_v ? h - a.Hq - p.Hk : h - a.Hq;
    uint8_t* codes = is_q ? a.q + (static_cast<int64_t>(t) * a.Hq + h) * N
                          : (is_v ? p.cache.v : p.cache.k) + place + head * p.cache.head_stride;
    if (inside && (is_q || kept)) {
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        if (!(is_v ? lane + v * LPR < nv : slot_ok<LPR, HS, TS>(v, lane, hv, th))) continue;
        float2 d[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          d[k] = div2_by(y[v][k], sc, rc);
          if (clamp) d[k] = make_float2(clamp_abs(d[k].x, a.fp8_max), clamp_abs(d[k].y, a.fp8_max));
        }
        st_stream8(codes + (is_v ? 8 * (lane + v * LPR) : slot_col<LPR, HS, TS>(v, lane, hv, th)),
                   pack_e4m3x8(d[0], d[1], d[2], d[3]));
      }
      if (lane == 0) {
        float* scale = is_q ? a.scale + static_cast<int64_t>(t) * a.Hq + h
                            : (is_v ? p.cache.v_scale : p.cache.k_scale) + splace + head * p.cache.s_head_stride;
        *scale = sc;
      }
    }
  }
}

template <typename T, typename TT, int LPR, int HS, int TS>
bool launch_shape(const AppendArgs& p, cudaStream_t s) {
  auto kern = append_kernel<T, TT, LPR, HS, TS>;
  // Warp steps per token, and into how many parts they are split: as many as the GPU has room for warps (32 per SM)
  // beside the tokens, one step each at most.
  const int64_t tokens = p.rows.rows / p.rows.H, all = (static_cast<int64_t>(p.rows.H) * LPR + 31) / 32;
  int64_t parts = 32 * static_cast<int64_t>(sm_count()) / tokens;
  parts = parts < 1 ? 1 : parts > all ? all : parts;
  const int64_t steps = (all + parts - 1) / parts;
  parts = (all + steps - 1) / steps;
  const int64_t grid = (tokens * parts + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7fffffffLL) return false;
  kern<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p, static_cast<int32_t>(steps), static_cast<int32_t>(parts));
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

}  // namespace

bool launch_append_vector(const AppendArgs& p, int dtype, int table_dtype, cudaStream_t s) {
  if (p.rows.R > 0 && table_dtype == DT_FP32)
    return dtype == DT_BF16 ? launch_typed<__nv_bfloat16, float>(p, s) : launch_typed<__half, float>(p, s);
  return dtype == DT_BF16 ? launch_typed<__nv_bfloat16, __nv_bfloat16>(p, s) : launch_typed<__half, __half>(p, s);
}

}  // namespace fq
