// fq_sample.cu -- the next token of each row of logits: temperature, top-k, top-p, min-p and a given uniform number.
//
// Mathematics. A row of 16-bit logits is, but for the order of equal ones, how often each value occurs in it. With the
// values in falling order (bin i is the i-th below the largest), counts c_i and weights w_i = exp((x_i - max) / T), every
// cut keeps a prefix of the sorted tokens: top-k the first k, top-p those before which the running sum is below top_p
// times the sum, min-p the bins with w_i >= min_p. So nothing is sorted: a histogram, running sums over it, and the
// search for the bin in which a running sum passes a border. The token is then the n-th of the row with that value.
//
// Borders are met by random numbers, and results have to be those of exact arithmetic: weights are computed in two fp32
// words each (2^-44 of themselves), held as integers in units of 2^-62 of the largest, and summed in 128 bits, without
// rounding and in any order. fp64 instructions would cost more than everything else here (2 a clock and SM).
#include <cmath>

#include "fq_device.cuh"
#include "fq_serving.h"
#include "fq_sync.cuh"

namespace fq {
namespace {

using u128 = unsigned __int128;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 49152;  // 192 KB; values further below the largest take a second round
constexpr int kOne = 62;      // weights are integers, 2^62 the largest

// ------------------------------------------------------------------------------------- weights
// 2^(-j / 1024) as a sum of two floats, j in [0, 1024].
struct PowerTable {
  float hi[1025], lo[1025];
};

constexpr double half_power(int k) {  // 2^(-1 / 2^k), square roots by Newton's iteration
  double v = 0.5;
  for (int i = 0; i < k; ++i) {
    double r = 0.5 * (v + 1.0);
    for (int n = 0; n < 6; ++n) r = 0.5 * (r + v / r);
    v = r;
  }
  return v;
}

constexpr PowerTable make_powers() {
  PowerTable t{};
  double root[11] = {};
  for (int b = 0; b <= 10; ++b) root[b] = half_power(10 - b);  // 2^(-2^b / 1024)
  for (int j = 0; j <= 1024; ++j) {
    double v = 1.0;
    for (int b = 0; b <= 10; ++b)
      if ((j >> b) & 1) v *= root[b];
    t.hi[j] = static_cast<float>(v);
    t.lo[j] = static_cast<float>(v - static_cast<double>(t.hi[j]));
  }
  return t;
}

__device__ const PowerTable kPowers = make_powers();

// What a row's weights depend on: its largest value, and log2(e) / T / unit as two floats. Values are taken in halves
// (unit 1/2) from a temperature of 1 on, so that the difference of any two is finite.
struct Heat {
  float top, unit, hi, lo;
};

// 2^62 * exp((x - top) / T), x <= top, to 2^-41 of itself or 1.
//
// d = top - x is exact in two floats, y = d * log2(e) / T but for 2^-47 of it; with n = floor(y), y = n + j / 1024 + r, the
// weight is 2^-n * table[j] * (1 + z + z^2 / 2 + z^3 / 6), z = -r ln 2, |z| < 2^-11.5, whose square fits one float.
__device__ __forceinline__ uint64_t weight_of(const Heat& h, float x) {
  if (x == h.top) return 1ull << kOne;
  const float t = h.top * h.unit;
  x *= h.unit;
  const float d = __fsub_rn(t, x);
  // the rounding of d (the sum of two floats and its error, by their six operations)
  const float bx = __fsub_rn(t, d), err = __fadd_rn(__fsub_rn(t, __fadd_rn(d, bx)), __fsub_rn(bx, x));
  const float p = __fmul_rn(d, h.hi);
  if (!(p < 126.f)) return 0;  // also where the largest is infinite
  const float e = fmaf(d, h.hi, -p) + (d * h.lo + err * h.hi);
  const float n = floorf(p), f = __fsub_rn(p, n);              // exact
  const float j = rintf(f * 1024.f), r = fmaf(j, -0.0009765625f, f);  // exact, |r| <= 2^-11
  const int at = static_cast<int>(j);
  const float th = __ldg(&kPowers.hi[at]), tl = __ldg(&kPowers.lo[at]);
  constexpr float kLn2 = 0.693147182464599609f, kLn2Lo = -1.90465429995776e-9f;
  const float z = __fmul_rn(r, -kLn2);
  const float zl = fmaf(r, -kLn2, -z) - fmaf(r, kLn2Lo, e * kLn2);
  const float q = z * z * fmaf(z, 0.166666667f, 0.5f);
  // th + tl + (th + tl)(z + zl + q), the large parts with their errors
  const float a = __fmul_rn(th, z), al = fmaf(th, z, -a);
  const float s = __fadd_rn(th, a), sl = __fsub_rn(a, __fsub_rn(s, th));  // |a| < th
  const float lo = sl + (al + fmaf(th, zl + q, fmaf(tl, z, tl)));
  const float scale = __int_as_float((127 + kOne - static_cast<int>(n)) << 23);
  return static_cast<uint64_t>(__float2ll_rn(s * scale) + __float2ll_rn(lo * scale));
}

__device__ __forceinline__ float to_float(u128 v) {
  return fmaf(__ull2float_rn(static_cast<uint64_t>(v >> 64)), 18446744073709551616.f, __ull2float_rn(static_cast<uint64_t>(v)));
}

__device__ __forceinline__ u128 lesser(u128 a, u128 b) { return a < b ? a : b; }

// floor (or ceil) of v * total for v in [0, 1], total < 2^94.
__device__ __forceinline__ u128 share_of(float v, u128 total, bool up) {
  if (v <= 0.f) return 0;
  const int bits = __float_as_int(v), expo = bits >> 23;
  const uint32_t mant = expo == 0 ? bits & 0x7fffffu : (bits & 0x7fffffu) | 0x800000u;
  const int shift = 150 - (expo == 0 ? 1 : expo);  // v = mant * 2^-shift, shift >= 23
  const u128 prod = total * mant;
  if (shift >= 128) return up ? 1 : 0;
  const u128 down = prod >> shift;
  return up && (down << shift) != prod ? down + 1 : down;
}

// ---------------------------------------------------------------------------------------- keys
// 16-bit logits as whole numbers in the order of their values. Keys in (kFloor, kTop] are numbers and +inf; -inf and
// the NaNs are outside. -0 has a key of its own below that of 0 and counts as 0.
template <typename T>
struct Keys;
template <>
struct Keys<__nv_bfloat16> {
  static constexpr uint32_t kFloor = 0x007f, kTop = 0xff80;
};
template <>
struct Keys<__half> {
  static constexpr uint32_t kFloor = 0x03ff, kTop = 0xfc00;
};
constexpr uint32_t kZero = 0x8000, kMinusZero = 0x7fff;

__device__ __forceinline__ uint32_t two_keys(uint32_t raw) {  // of two packed values
  uint32_t sign;  // 0xffff where the sign bit is set
  asm("prmt.b32 %0, %1, 0, 0xbb99;" : "=r"(sign) : "r"(raw));
  return raw ^ (sign | 0x80008000u);
}

template <typename T>
__device__ __forceinline__ float value_of(uint32_t key) {
  const uint32_t raw = key & 0x8000u ? key & 0x7fffu : ~key & 0xffffu;
  return Elem<T>::unpack(raw).x;
}

// The least key that x or a larger value may have.
template <typename T>
__device__ __forceinline__ uint32_t key_from(float x);
template <>
__device__ __forceinline__ uint32_t key_from<__nv_bfloat16>(float x) {
  const uint32_t raw = __bfloat16_as_ushort(__float2bfloat16_rd(x));
  return two_keys(raw) & 0xffffu;
}
template <>
__device__ __forceinline__ uint32_t key_from<__half>(float x) {
  const uint32_t raw = __half_as_ushort(__float2half_rd(x));
  return two_keys(raw) & 0xffffu;
}

// A row as 16-byte vectors: vector v holds elements 8v - skip .. 8v - skip + 7, those outside the row as NaN.
struct Row {
  const uint16_t* x;
  int32_t V, skip, vectors;

  __device__ __forceinline__ uint4 operator()(int32_t v) const {
    const int64_t from = 8 * static_cast<int64_t>(v) - skip;
    if (from >= 0 && from + 8 <= V) return __ldg(reinterpret_cast<const uint4*>(x + from));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t a = from + 2 * i;
      const uint32_t lo = a >= 0 && a < V ? x[a] : 0xffffu, hi = a + 1 >= 0 && a + 1 < V ? x[a + 1] : 0xffffu;
      w[i] = lo | (hi << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

template <typename F>
__device__ __forceinline__ void each_key(const uint4& v, F f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t k = two_keys(w[i]);
    f(k & 0xffffu, 2 * i);
    f(k >> 16, 2 * i + 1);
  }
}

// ----------------------------------------------------------------------------------- the block
__device__ __forceinline__ u128 shfl_up(u128 v, int o) {
  const uint64_t lo = __shfl_up_sync(0xffffffffu, static_cast<uint64_t>(v), o);
  const uint64_t hi = __shfl_up_sync(0xffffffffu, static_cast<uint64_t>(v >> 64), o);
  return (static_cast<u128>(hi) << 64) | lo;
}

template <typename N>
__device__ __forceinline__ N warp_scan(N v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    N u;
    if constexpr (sizeof(N) == 16) u = shfl_up(v, o);
    else u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The block's exclusive sum of v, and the total.
template <typename N>
__device__ __forceinline__ N block_scan(N v, N* part, N* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const N incl = warp_scan(v);
  __syncthreads();
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) part[lane] = warp_scan(part[lane]);
  __syncthreads();
  *total = part[kWarps - 1];
  return (warp == 0 ? N(0) : part[warp - 1]) + incl - v;
}

struct Shared {
  uint32_t bin[kBins];
  u128 wide[kWarps];
  uint32_t narrow[kWarps];
  // the thread's bins in which a border lies
  u128 before;
  int32_t rank, first;
  // found there
  u128 sum;
  int32_t key, nth;
};

struct Cuts {
  Heat heat;
  uint32_t top_k;
  uint64_t min_weight;
};

// The first bin of [first, first + n) up to and with which the running sum, `before` and `rank` tokens ahead of it, is
// above `border`; one warp. Returns the bin, the sum before it and its weight.
template <typename T>
__device__ __forceinline__ int find_bin(const Shared& sm, const Cuts& c, uint32_t top, int first, int n, u128 before, uint32_t rank,
                                        u128 border, u128* sum_before, uint64_t* weight) {
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int i = first + i0 + lane;
    const uint32_t count = i0 + lane < n ? sm.bin[i] : 0u;
    const uint32_t ahead = rank + warp_scan(count) - count;
    const uint32_t in = ahead >= c.top_k ? 0u : min(count, c.top_k - ahead);
    const uint64_t w = in != 0u ? weight_of(c.heat, value_of<T>(top - i)) : 0;
    const u128 incl = before + warp_scan(static_cast<u128>(w) * in);
    const uint32_t hit = __ballot_sync(0xffffffffu, incl > border);
    if (hit != 0u) {
      const int l = __ffs(hit) - 1;
      const u128 from = incl - static_cast<u128>(w) * in;
      *sum_before = (static_cast<u128>(__shfl_sync(0xffffffffu, static_cast<uint64_t>(from >> 64), l)) << 64) |
                    __shfl_sync(0xffffffffu, static_cast<uint64_t>(from), l);
      *weight = __shfl_sync(0xffffffffu, w, l);
      return first + i0 + l;
    }
    before = (static_cast<u128>(__shfl_sync(0xffffffffu, static_cast<uint64_t>(incl >> 64), 31)) << 64) |
             __shfl_sync(0xffffffffu, static_cast<uint64_t>(incl), 31);
    rank += __shfl_sync(0xffffffffu, warp_scan(count), 31);
  }
  return -1;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_trigger();
  pdl_wait();
  for (int32_t b = blockIdx.x; b < a.B; b += gridDim.x) {
    Row row;
    row.x = a.logits + b * a.stride;
    row.V = a.V;
    row.skip = static_cast<int32_t>((reinterpret_cast<uintptr_t>(row.x) & 15u) / 2);
    row.vectors = static_cast<int32_t>((static_cast<int64_t>(a.V) + row.skip + 7) / 8);
    const float temperature = a.temperature == nullptr ? 1.f : a.temperature[b];
    const int32_t k = a.top_k == nullptr ? 0 : a.top_k[b];
    const float top_p = a.top_p == nullptr ? 1.f : a.top_p[b], min_p = a.min_p == nullptr ? 0.f : a.min_p[b];

    // ------------------------------------------------------------------- the largest value
    uint32_t top = 0;
    for (int32_t v = threadIdx.x; v < row.vectors; v += kThreads)
      each_key(row(v), [&](uint32_t s, int) {
        if (s > Keys<T>::kFloor && s <= Keys<T>::kTop) top = max(top, s);
      });
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();  // the last row's readers are through
    if (lane == 0) sm.narrow[warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, sm.narrow[lane]);
    if (top == kMinusZero) top = kZero;
    if (top == 0u) {  // nothing is left of the row
      if (threadIdx.x == 0) {
        a.token[b] = -1;
        if (a.logprob != nullptr) a.logprob[b] = -INFINITY;
      }
      continue;
    }

    uint32_t key = top;
    int32_t nth = 0;
    float logprob = 0.f;
    if (temperature >= 1.17549435e-38f && k != 1) {
      Cuts c;
      c.heat.top = value_of<T>(top);
      c.heat.unit = temperature >= 1.f ? 0.5f : 1.f;
      const double heat = 1.4426950408889634074 / (static_cast<double>(temperature) * c.heat.unit);
      c.heat.hi = static_cast<float>(heat);
      c.heat.lo = static_cast<float>(heat - static_cast<double>(c.heat.hi));
      c.top_k = k <= 0 ? 0xffffffffu : static_cast<uint32_t>(k);
      c.min_weight = min_p > 0.f ? static_cast<uint64_t>(share_of(fminf(min_p, 1.f), static_cast<u128>(1) << kOne, true)) : 0;
      // Weights below exp(-45) of the largest are 0 in units of 2^-62.
      const float least = c.heat.top - 45.f * temperature;
      uint32_t floor_key = Keys<T>::kFloor + 1;
      if (least == least) floor_key = max(floor_key, key_from<T>(least));
      const int bins = static_cast<int>(top - floor_key) + 1, rounds = (bins + kBins - 1) / kBins;

      u128 sum_before = 0, sum_mine = 0, border = 0, kept = 0;
      uint32_t rank_before = 0;
      int from = 0, per = 0, base = 0;
      // Round r: bins kBins * r ... Their counts, and this thread's bins [from, from + per) with the tokens and the sum
      // before them.
      auto count = [&](int r, uint32_t& rank_carry, u128& sum_carry, u128& floor_sum) {
        base = kBins * r;
        __syncthreads();  // the last round's readers are through
        const int here = min(kBins, bins - base);
        for (int i = threadIdx.x; i < here; i += kThreads) sm.bin[i] = 0u;
        __syncthreads();
        const uint32_t first_key = top - base;
        for (int32_t v = threadIdx.x; v < row.vectors; v += kThreads)
          each_key(row(v), [&](uint32_t s, int) {
            if (s == kMinusZero) s = kZero;
            const uint32_t i = first_key - s;  // larger keys (NaN, and the last round's) wrap around
            if (i < static_cast<uint32_t>(here)) atomicAdd(&sm.bin[i], 1u);
          });
        __syncthreads();
        per = ((here + kThreads - 1) / kThreads) | 1;  // odd: the threads' bins are in different banks
        from = min(here, static_cast<int>(threadIdx.x) * per);
        const int to = min(here, from + per);
        uint32_t mine = 0, all;
        for (int i = from; i < to; ++i) mine += sm.bin[i];
        const uint32_t rank = rank_carry + block_scan(mine, sm.narrow, &all);
        rank_carry += all;
        rank_before = rank;
        u128 sum = 0, above = 0;
        uint32_t ahead = rank;
        for (int i = from; i < to && ahead < c.top_k; ++i) {
          const uint32_t n = sm.bin[i];
          if (n == 0u) continue;
          const uint64_t w = weight_of(c.heat, value_of<T>(first_key - i));
          const u128 add = static_cast<u128>(w) * min(n, c.top_k - ahead);
          sum += add;
          if (w >= c.min_weight) above += add;
          ahead += n;
        }
        u128 total;
        sum_mine = sum;
        sum_before = sum_carry + block_scan(sum, sm.wide, &total);
        sum_carry += total;
        u128 total_above;
        block_scan(above, sm.wide, &total_above);
        floor_sum += total_above;
      };
      // The bin of the round in which the running sum passes `border`, if it does; every thread.
      auto search = [&](u128 border_at, bool crossing, uint64_t* w, u128* ahead, int* bin) {
        __syncthreads();
        if (threadIdx.x == 0) sm.first = -1;
        __syncthreads();
        if (crossing) {
          sm.first = from;
          sm.before = sum_before;
          sm.rank = static_cast<int32_t>(rank_before);
        }
        __syncthreads();
        if (sm.first < 0) return false;
        const int here = min(kBins, bins - base);
        *bin = find_bin<T>(sm, c, top - base, sm.first, min(per, here - sm.first), sm.before, static_cast<uint32_t>(sm.rank),
                           border_at, ahead, w);
        return *bin >= 0;
      };
      auto redo = [&](int r, uint32_t& rank_carry, u128& sum_carry) {
        u128 unused = 0;
        if (rounds > 1) count(r, rank_carry, sum_carry, unused);
      };
      uint32_t ranks = 0;
      u128 total = 0, above = 0;
      for (int r = 0; r < rounds; ++r) count(r, ranks, total, above);
      kept = lesser(total, above);
      if (top_p < 1.f) {
        // The first running sum that reaches the border: tokens before which it is below are kept.
        u128 reach = share_of(fmaxf(top_p, 0.f), total, true);
        if (reach == 0) reach = 1;
        uint32_t rc = 0;
        u128 sc = 0;
        for (int r = 0; r < rounds; ++r) {
          redo(r, rc, sc);
          uint64_t w;
          u128 ahead;
          int bin;
          if (search(reach - 1, sum_before < reach && sum_before + sum_mine >= reach, &w, &ahead, &bin)) {
            const u128 n = (reach - ahead + w - 1) / w;
            kept = lesser(kept, ahead + n * w);
            break;
          }
        }
      }
      const float u = a.u[b];
      border = share_of(u > 0.f ? fminf(u, 0.999999940395355225f) : 0.f, kept, false);
      uint32_t rc = 0;
      u128 sc = 0;
      for (int r = 0; r < rounds; ++r) {
        redo(r, rc, sc);
        uint64_t w;
        u128 ahead;
        int bin;
        if (search(border, sum_before <= border && sum_before + sum_mine > border, &w, &ahead, &bin)) {
          key = top - base - bin;
          nth = static_cast<int32_t>((border - ahead) / w);
          const float whole = to_float(kept), rest = to_float(kept - w);
          logprob = rest < 0.5f * whole ? log1pf(-rest / whole) : logf(to_float(w) / whole);
          break;
        }
      }
    }

    // ------------------------------------------------------- the nth element of that value
    // Each warp takes an equal run of vectors: how many it has, then the run with the nth.
    const uint32_t twin = key == kZero ? kMinusZero : key;
    const int32_t run = (row.vectors + kWarps - 1) / kWarps, v0 = min(row.vectors, warp * run), v1 = min(row.vectors, v0 + run);
    uint32_t mine = 0;
    for (int32_t v = v0 + lane; v < v1; v += 32) each_key(row(v), [&](uint32_t s, int) { mine += s == key || s == twin; });
    mine = __reduce_add_sync(0xffffffffu, mine);
    __syncthreads();
    if (lane == 0) sm.narrow[warp] = mine;
    __syncthreads();
    const uint32_t upto = warp_scan(sm.narrow[lane]), all_before = __shfl_sync(0xffffffffu, upto - sm.narrow[lane], warp);
    if (all_before <= static_cast<uint32_t>(nth) && static_cast<uint32_t>(nth) < all_before + mine) {
      uint32_t left = nth - all_before;
      for (int32_t v = v0; v < v1; v += 32) {
        uint32_t bits = 0;  // of this lane's eight
        if (v + lane < v1) each_key(row(v + lane), [&](uint32_t s, int i) { bits |= static_cast<uint32_t>(s == key || s == twin) << i; });
        const uint32_t has = __popc(bits), incl = warp_scan(has), all = __shfl_sync(0xffffffffu, incl, 31);
        if (left < all) {
          if (incl - has <= left && left < incl) {
            for (uint32_t n = left - (incl - has); n > 0; --n) bits &= bits - 1;
            a.token[b] = 8 * static_cast<int64_t>(v + lane) - row.skip + (__ffs(bits) - 1);
            if (a.logprob != nullptr) a.logprob[b] = logprob;
          }
          break;
        }
        left -= all;
      }
    }
  }
}

template <typename T>
bool launch(const SampleArgs& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(Shared);
  static_assert(smem <= 227 * 1024, "the bins fit the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(sample_kernel<T>), smem)) return false;
  const int64_t rows = a.B, sms = sm_count();
  launch_overlapped(sample_kernel<T>, dim3(static_cast<unsigned>(rows < sms ? rows : sms)), kThreads, smem, 1, s, a);
  return true;
}

}  // namespace

bool launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
  return dtype == DT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace fq
