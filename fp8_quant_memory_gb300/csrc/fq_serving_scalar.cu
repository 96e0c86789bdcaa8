// fq_serving_scalar.cu -- any-layout kernels of the FP8 serving operators: any width, alignment and
// stride. One thread per output (matrix product), one warp per row (append) and one block per query
// row (attention), element-wise loads, fp32 sums. The layouts that the vectorised kernels take go there;
// these keep the same results for the others.
#include <math_constants.h>

#include "fq_device.cuh"
#include "fq_epilogue.cuh"
#include "fq_serving.h"

namespace fq {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

__device__ __forceinline__ float ld_any(int dt, const void* p, int64_t i) {
  if (dt == DT_BF16) return Elem<__nv_bfloat16>::load1(p, i);
  if (dt == DT_FP16) return Elem<__half>::load1(p, i);
  return Elem<float>::load1(p, i);
}

__device__ __forceinline__ void st_any(int dt, void* p, int64_t i, float v) {
  if (dt == DT_BF16) Elem<__nv_bfloat16>::store1(p, i, v);
  else Elem<__half>::store1(p, i, v);
}

// ------------------------------------------------------------------------------ matrix product
__global__ void __launch_bounds__(kThreads) matmul_scalar_kernel(const MatmulArgs a, int dt) {
  const int64_t total = a.M * a.N;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int64_t i = e / a.N, j = e - i * a.N;
    const uint8_t* ar = a.a + i * a.a_stride;
    const uint8_t* br = a.b + j * a.b_stride;
    float acc = 0.f;
    for (int64_t g = 0; g < a.groups; ++g) {
      const int64_t end = min((g + 1) * kScaleBlock, a.K);
      float s = 0.f;
      for (int64_t k = g * kScaleBlock; k < end; ++k) s = __fmaf_rn(e4m3_value(ar[k]), e4m3_value(br[k]), s);
      const float sc = __fmul_rn(a.a_scale[i * a.a_scale_stride + g], a.b_scale[j / kScaleBlock * a.b_scale_stride + g]);
      acc = __fmaf_rn(s, sc, acc);
    }
    if (a.bias != nullptr) acc = __fadd_rn(acc, ld_any(dt, a.bias, j));
    float2 y[1] = {make_float2(acc, 0.f)};
    activate_each(a.activation, y);
    acc = y[0].x;
    if (a.residual != nullptr) acc = __fadd_rn(acc, ld_any(dt, a.residual, i * a.residual_stride + j));
    st_any(dt, a.out, i * a.out_stride + j, acc);
  }
}

// -------------------------------------------------------------------------------------- append
__global__ void __launch_bounds__(kThreads) append_scalar_kernel(const AppendArgs p, int dt, int tdt) {
  const RowArgs& a = p.rows;
  const int lane = threadIdx.x & 31;
  const int N = a.N, half = a.R / 2, tail = a.N - a.R;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); r < a.rows;
       r += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t t = r / a.H;
    const int32_t h = static_cast<int32_t>(r - t * a.H);
    const char* x = static_cast<const char*>(a.x) + (t * a.token_stride + static_cast<int64_t>(h) * N) * 2;
    const bool is_q = h < a.Hq, is_v = h >= a.Hq + p.Hk;
    uint8_t* codes;
    float* scale;
    if (is_q) {
      codes = a.q + (t * a.Hq + h) * N;
      scale = a.scale + t * a.Hq + h;
    } else {
      const int64_t slot = p.slots[t];
      if (slot < 0 || slot >= p.cache.pages * p.cache.page_size) continue;
      const int64_t page = slot / p.cache.page_size, off = slot - page * p.cache.page_size;
      const int32_t head = (h - a.Hq) % p.Hk;
      codes = (is_v ? p.cache.v : p.cache.k) + page * p.cache.page_stride + head * p.cache.head_stride +
              off * p.cache.token_stride;
      scale = (is_v ? p.cache.v_scale : p.cache.k_scale) + page * p.cache.s_page_stride +
              head * p.cache.s_head_stride + off * p.cache.s_token_stride;
    }
    float rstd = 0.f;
    if (!is_v) {
      float ss = 0.f;
      for (int j = lane; j < N; j += 32) {
        const float v = ld_any(dt, x, j);
        ss = __fmaf_rn(v, v, ss);
      }
      rstd = rstd_from_ss(group_sum<32>(ss), static_cast<float>(N), a.eps);
    }
    const void* w = is_q ? a.wq : a.wk;
    auto normed = [&](int j) { return __fmul_rn(__fmul_rn(ld_any(dt, x, j), rstd), ld_any(dt, w, j)); };
    auto value = [&](int j) {
      if (is_v) return ld_any(dt, x, j);
      if (j < tail) return normed(j);
      const bool first = j - tail < half;
      const int i = first ? j - tail : j - tail - half;
      const float lo = normed(tail + i), hi = normed(tail + half + i);
      const float c = ld_any(tdt, a.cos, t * half + i), s = ld_any(tdt, a.sin, t * half + i);
      return first ? __fsub_rn(__fmul_rn(lo, c), __fmul_rn(hi, s)) : __fadd_rn(__fmul_rn(hi, c), __fmul_rn(lo, s));
    };
    float amax = 0.f;
    for (int j = lane; j < N; j += 32) amax = fmaxf(amax, fabsf(value(j)));
    const float sc = __fdiv_rn(fmaxf(group_max<32>(amax), 1e-4f), a.fp8_max);
    for (int j = lane; j < N; j += 32)
      codes[j] = static_cast<uint8_t>(e4m3x2(make_float2(clamp_or_nan(__fdiv_rn(value(j), sc), a.fp8_max), 0.f)));
    if (lane == 0) *scale = sc;
  }
}

// ----------------------------------------------------------------------------------- attention
// One block per (sequence, query head). Every warp takes each kWarps-th token with its own running
// maximum, sum and output (dimension lane + 32*i in register i), joined in shared memory.
constexpr int kMaxD = 256;

__global__ void __launch_bounds__(kThreads) attention_scalar_kernel(const PagedArgs a, int dt) {
  __shared__ float part[kWarps][kMaxD + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int64_t b = row / a.Hq;
  const int32_t h = static_cast<int32_t>(row - b * a.Hq);
  const int32_t hk = h / (a.Hq / a.Hk);
  const CacheView& c = a.cache;
  const int64_t len = max(static_cast<int64_t>(0), static_cast<int64_t>(min(a.lens[b], a.max_len)));
  const float qs = a.q_scale[b * a.q_scale_stride + h] * a.scale_log2;
  float q[kMaxD / 32], o[kMaxD / 32];
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) {
    const int d = lane + 32 * i;
    q[i] = d < a.D ? e4m3_value(a.q[b * a.q_stride + static_cast<int64_t>(h) * a.D + d]) : 0.f;
    o[i] = 0.f;
  }
  float m = -CUDART_MAX_NORMAL_F, l = 0.f;
  // the visible tokens: [0, sunk) and [start, len)
  const int64_t start = max(len - a.window, static_cast<int64_t>(0)), sunk = min(static_cast<int64_t>(a.sinks), start);
  for (int64_t v = warp; v < len - start + sunk; v += kWarps) {
    const int64_t t = v < sunk ? v : v - sunk + start;
    const int64_t at = t / c.page_size, off = t - at * c.page_size;
    const int64_t page = a.table[b * a.table_stride + at];
    if (page < 0 || page >= c.pages) continue;  // absent page: its tokens take no part
    const int64_t base = page * c.page_stride + hk * c.head_stride + off * c.token_stride;
    const int64_t sbase = page * c.s_page_stride + hk * c.s_head_stride + off * c.s_token_stride;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i)
      if (lane + 32 * i < a.D) s = __fmaf_rn(q[i], e4m3_value(c.k[base + lane + 32 * i]), s);
    s = group_sum<32>(s) * (qs * c.k_scale[sbase]);
    const float mn = fmaxf(m, s);
    const float keep = exp2f(m - mn), p = exp2f(s - mn);
    const float pv = p * c.v_scale[sbase];
    l = l * keep + p;
    m = mn;
#pragma unroll
    for (int i = 0; i < kMaxD / 32; ++i)
      if (lane + 32 * i < a.D) o[i] = __fmaf_rn(pv, e4m3_value(c.v[base + lane + 32 * i]), o[i] * keep);
  }
#pragma unroll
  for (int i = 0; i < kMaxD / 32; ++i) part[warp][lane + 32 * i] = o[i];
  if (lane == 0) {
    part[warp][kMaxD] = m;
    part[warp][kMaxD + 1] = l;
  }
  __syncthreads();
  float mj = part[0][kMaxD];
  for (int w = 1; w < kWarps; ++w) mj = fmaxf(mj, part[w][kMaxD]);
  float lj = 0.f;
  for (int w = 0; w < kWarps; ++w) lj += part[w][kMaxD + 1] * exp2f(part[w][kMaxD] - mj);
  for (int d = threadIdx.x; d < a.D; d += kThreads) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v = __fmaf_rn(part[w][d], exp2f(part[w][kMaxD] - mj), v);
    st_any(dt, a.out, row * a.D + d, lj == 0.f ? 0.f : v / lj);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[row] = lj == 0.f ? -CUDART_INF_F : (mj + log2f(lj)) * 0.693147180559945309f;
}

}  // namespace

void launch_matmul_scalar(const MatmulArgs& a, int dtype, cudaStream_t s) {
  const int64_t need = (a.M * a.N + kThreads - 1) / kThreads, cap = static_cast<int64_t>(sm_count()) * 64;
  matmul_scalar_kernel<<<static_cast<unsigned>(need < cap ? need : cap), kThreads, 0, s>>>(a, dtype);
}

void launch_append_scalar(const AppendArgs& a, int dtype, int table_dtype, cudaStream_t s) {
  const int64_t need = (a.rows.rows + kWarps - 1) / kWarps, cap = static_cast<int64_t>(sm_count()) * 16;
  append_scalar_kernel<<<static_cast<unsigned>(need < cap ? need : cap), kThreads, 0, s>>>(a, dtype, table_dtype);
}

void launch_attention_scalar(const PagedArgs& a, int dtype, cudaStream_t s) {
  attention_scalar_kernel<<<static_cast<unsigned>(static_cast<int64_t>(a.B) * a.Hq), kThreads, 0, s>>>(a, dtype);
}

}  // namespace fq
