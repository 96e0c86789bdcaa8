// fq_append.cu -- the QK-Norm + RoPE + FP8 prologue on whole QKV rows, K and V placed in a paged FP8 cache.
//
// Mathematics: q and k rows as the prologue (fq_rows.cuh, MODE_QK: norm, rotation, one scale per row, all in fp32);
// v rows are quantised as they are. What bounds it: HBM, 2 bytes read and 1 written per element. One pass: every
// element is read once, held in registers through norm, rotation and row maximum, and leaves as a code in its place
// in the cache, so nothing is written and read again between the prologue and the cache.
//
// Layout: a group of LPR lanes owns a (token, head) row, as in fq_rows.cu; consecutive groups take consecutive rows,
// so loads cover whole contiguous runs of the QKV row. Rows of q and k and rows of v meet in a warp only where the
// head counts are not multiples of its rows; such a warp runs both bodies, each with its own rows live.
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

template <typename T, typename TT, int LPR, int HS, int TS>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs p) {
  constexpr int kRowsPerCta = kThreads / LPR;
  constexpr int kV = HS + 2 * TS;
  const RowArgs& a = p.rows;
  const int lane = threadIdx.x & (LPR - 1), grp = threadIdx.x / LPR;
  const int N = a.N, nv = N >> 3, hv = (N - a.R) >> 3, th = a.R >> 4, half = a.R >> 1;
  const int32_t rows = static_cast<int32_t>(a.rows);
  for (int32_t base = blockIdx.x * kRowsPerCta; base < rows; base += gridDim.x * kRowsPerCta) {
    const int32_t r = base + grp;
    const bool inside = r < rows;
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
      const int64_t slot = __ldg(p.slots + t);
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
      row_body<T, TT, MODE_QK, LPR, HS, TS, false>(row, 0, live && !is_v, h, xv, lane, hv, th, static_cast<float>(N), a.cos,
                                                   a.sin, static_cast<int64_t>(t) * half);
    }
    if (__any_sync(0xffffffffu, inside && is_v)) {
      float amax = 0.f;
#pragma unroll
      for (int s = 0; s < kV; ++s)
#pragma unroll
        for (int k = 0; k < 4; k += 2) amax = absmax4(amax, Elem<T>::unpack(word(xv[s], k)), Elem<T>::unpack(word(xv[s], k + 1)));
      amax = fmaxf(group_max<LPR>(amax), 1e-4f);
      const float sc = __fdiv_rn(amax, a.fp8_max), rc = __frcp_rn(sc);
      const bool clamp = a.fp8_max != 448.0f;
      if (live && is_v) {
#pragma unroll
        for (int s = 0; s < kV; ++s) {
          if (lane + s * LPR >= nv) continue;
          float2 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = div2_by(Elem<T>::unpack(word(xv[s], k)), sc, rc);
            if (clamp) v[k] = make_float2(clamp_abs(v[k].x, a.fp8_max), clamp_abs(v[k].y, a.fp8_max));
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
  kern<<<static_cast<unsigned>(need < cap ? need : cap), kThreads, 0, s>>>(p);
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
