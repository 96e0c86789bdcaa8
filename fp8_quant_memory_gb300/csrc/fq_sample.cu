// fq_sample.cu -- the next token of each row of logits: temperature, top-k, top-p, min-p and a given uniform number.
//
// Mathematics. A row of 16-bit logits is, but for the order of equal ones, how often each value occurs in it. With the
// values in falling order (bin i is the i-th below the largest), counts c_i and weights w_i = exp((x_i - max) / T), every
// cut keeps a prefix of the sorted tokens: top-k the first k, top-p those before which the running sum is below top_p
// times the sum, min-p the bins with w_i >= min_p. So nothing is sorted: a histogram, running sums over it, and the
// search for the bin in which a running sum passes a border. The token is then the n-th of the row with that value.
//
// Borders are met by random numbers, and results have to be those of exact arithmetic: weights are computed in two fp32
// words each (2^-41 of themselves), held as integers in units of 2^-62 of the largest, and summed in 128 bits. (A bin's, which is
// the product of two such, is right to 2^-40 or four units: one for each factor's rounding, two for the product's.) fp64
// instructions would cost more than everything else here (2 a clock and SM: a division by every thread was 6 us).
//
// A block takes a row in three ways. A row's largest alone (temperature 0, top-k 1): one pass. Few tokens (a top-k, a min-p
// without top-p): the k-th largest of the threads' own largest bounds the k-th token; the threads that hold one as large are
// looked at again, by all, and what they list is sorted by counting. Else every token counts: bins of 32-bit counts, 192 KB,
// over the keys from the largest down to where weights are 0, filled while the largest is still being looked for: that of the
// first 8192 tells where the bins have to lie, but for rows whose largest is far above it, which take a second pass.
//
// What bounds it. 256 x 151936 bf16, a third of the rows whole: 41 us, the bytes 11.5. A whole row takes an SM 22 us, 28 with
// all SMs reading (its bytes at an SM's share of the memory: 6.7): 12 us the bins (22 thousand clocks for 4.8 thousand
// warp-wide additions: banks that 32 lanes meet at random, 3.7 clocks each by the conflict counter, a plain store is no
// faster), 5 us sums and searches, 3 us the token's place: phases that hand over at the block's barriers, where warps wait most
// of all (8.6 to an issue slot, 2.4 for shared memory; 31% of the slots issue). Other rows take 8 to 12 us, of the memory's
// latency and barriers. 1 x 32000, top-k 50 and top-p: 6.7 us, 2.5 of them launch and first loads.
//
// Tried and left: the largest first, then the bins (256 x 151936 whole: 70 us against 59; rows of few tokens 0.5 us less, whose
// loads need not wait for the row's settings); the largest of 32768 instead of 8192, kept in registers (63 us); a cluster of
// blocks for a row (1 x 151936 whole: 26 us where a block took 25; a barrier of 8 x 1024 threads costs 1.2 us, and the bins pass
// through distributed shared memory); counts of 16 bits with two blocks an SM (256 x 151936: 82 us against 66 then: additions
// are the SM's bound, not the block's); rows through bulk copies (1 x 151936 with top-k: 10.5 against 8.1).
#include <cmath>

#include "fq_device.cuh"
#include "fq_serving.h"
#include "fq_sync.cuh"

namespace fq {
namespace {

using u128 = unsigned __int128;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 49152;          // 192 KB; values further below the largest take a second round
constexpr int kGroups = kBins / 32;   // a warp's bins at a time
constexpr int kPer = 2;               // groups of a thread in the sums over them
static_assert(kPer * kThreads >= kGroups, "every group has a thread");
constexpr int kBatches = kGroups / 32;  // of 32 groups, one to a lane; two of them to a warp at most
static_assert(kBatches <= 2 * kWarps && kBatches > kWarps, "two batches a warp");
constexpr int kExponents = 32;        // below the largest of a row, whose steps are in a table
constexpr int kFew = 256;             // threads whose part of the row is looked at again
constexpr int kListed = 256;          // tokens that are sorted where few count
constexpr int kOne = 62;              // weights are integers, 2^62 the largest

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
// (unit 1/2) from a temperature of 1 on, so that the difference of any two is finite, and in smaller units at temperatures
// whose reciprocal leaves fp32's normal range.
struct Heat {
  float top, unit, hi, lo;
};

// hi = L / t rounded, lo what it lacks: the remainder L - hi * t is exact.
__device__ __forceinline__ Heat heat_of(float top, float temperature) {
  constexpr float kL = 1.44269502162933349609f, kLLo = 1.92596299112661746e-8f;  // log2(e)
  Heat h;
  h.top = top;
  h.unit = temperature >= 1.8446744e19f ? 1.3552527e-20f : temperature >= 1.f ? 0.5f : 1.f;  // 2^64: 2^-66
  const float t = temperature * h.unit;
  if (t < INFINITY) {
    h.hi = __fdiv_rn(kL, t);
    h.lo = __fdiv_rn(fmaf(-h.hi, t, kL) + kLLo, t);
  } else {
    h.hi = h.lo = 0.f;
  }
  return h;
}

// 2^62 * 2^-((d + err) * log2(e) / T), d >= 0 and err its error, in the heat's unit, to 2^-41 of itself or 1.
//
// y = (d + err) * log2(e) / T in two floats, to 2^-47 of it; with n = floor(y), y = n + j / 1024 + r, the weight is
// 2^-n * table[j] * (1 + z + z^2 / 2 + z^3 / 6), z = -r ln 2, |z| < 2^-11.5, whose square fits one float.
__device__ __forceinline__ uint64_t falling(const Heat& h, float d, float err) {
  const float p = __fmul_rn(d, h.hi);
  if (!(p < 126.f)) return 0;  // also where the largest is infinite
  const float e = fmaf(d, h.hi, -p) + (d * h.lo + err * h.hi);
  const float n = floorf(p), f = __fsub_rn(p, n);                     // exact
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

// 2^62 * exp((x - top) / T), x <= top. top - x is exact as a float and its error (the six operations of an exact sum).
__device__ __forceinline__ uint64_t weight_of(const Heat& h, float x) {
  if (x == h.top) return 1ull << kOne;
  const float t = h.top * h.unit;
  x *= h.unit;
  const float d = __fsub_rn(t, x), bx = __fsub_rn(t, d);
  return falling(h, d, __fadd_rn(__fsub_rn(t, __fadd_rn(d, bx)), __fsub_rn(bx, x)));
}

__device__ __forceinline__ float to_float(u128 v) {
  return fmaf(__ull2float_rn(static_cast<uint64_t>(v >> 64)), 18446744073709551616.f, __ull2float_rn(static_cast<uint64_t>(v)));
}

// floor(n / d) of a quotient below 2^31: float estimates of what is left, each 2^-21 of the last at most, or one unit.
__device__ __forceinline__ int64_t quotient(u128 n, uint64_t d) {
  const float inv = __fdividef(1.f, to_float(d));
  int64_t q = static_cast<int64_t>(to_float(n) * inv);
  for (;;) {
    const __int128 left = static_cast<__int128>(n) - static_cast<__int128>(d) * q;
    if (left >= 0 && left < static_cast<__int128>(d)) return q;
    const int64_t part = max(static_cast<int64_t>(to_float(left < 0 ? -left : left) * inv), static_cast<int64_t>(1));
    q += left < 0 ? -part : part;
  }
}

__device__ __forceinline__ u128 lesser(u128 a, u128 b) { return a < b ? a : b; }

// log(w / kept), w <= kept.
__device__ __forceinline__ float log_share(uint64_t w, u128 kept) {
  const float whole = to_float(kept), rest = to_float(kept - w);
  return rest < 0.5f * whole ? log1pf(-rest / whole) : logf(to_float(w) / whole);
}

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
// Step of a value to its neighbours: 2^(exponent - kBias) with the raw exponent field, 1 for those without one.
template <>
struct Keys<__nv_bfloat16> {
  static constexpr uint32_t kFloor = 0x007f, kTop = 0xff80;
  static constexpr int kFraction = 7, kBias = 134;
};
template <>
struct Keys<__half> {
  static constexpr uint32_t kFloor = 0x03ff, kTop = 0xfc00;
  static constexpr int kFraction = 10, kBias = 25;
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

// The exponent field of a key's value, at least 1; the same for the 32 keys of a group, which differ in their last five bits.
template <typename T>
__device__ __forceinline__ int exponent_of(uint32_t key) {
  const uint32_t raw = (key & 0x8000u ? key : ~key) & 0x7fffu;
  return max(static_cast<int>(raw >> Keys<T>::kFraction), 1);
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

// A row as 16-byte vectors: vector v holds elements 8v - skip .. 8v - skip + 7. Vectors [first, last) are whole; there may
// be one before and one behind, whose places outside the row are NaN.
struct Row {
  const uint16_t* x;
  int32_t V, skip, vectors, first, last;

  __device__ __forceinline__ Row(const uint16_t* from, int32_t n) : x(from), V(n) {
    skip = static_cast<int32_t>((reinterpret_cast<uintptr_t>(x) & 15u) / 2);
    vectors = static_cast<int32_t>((static_cast<int64_t>(V) + skip + 7) / 8);
    first = skip > 0 ? 1 : 0;
    last = max(first, static_cast<int32_t>((static_cast<int64_t>(V) + skip) / 8));
  }
  __device__ __forceinline__ uint4 whole(int32_t v) const {
    return ld_stream16(x + (8 * static_cast<int64_t>(v) - skip));
  }
  __device__ __forceinline__ uint4 part(int32_t v) const {
    uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t a = 8 * static_cast<int64_t>(v) - skip + i;
      if (a >= 0 && a < V) w[i / 2] = (i & 1) ? (w[i / 2] & 0xffffu) | (static_cast<uint32_t>(x[a]) << 16) : (w[i / 2] & 0xffff0000u) | x[a];
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// f(vector, its number) for vectors from, from + step, ... below `to`; kAhead loads on their way at a time.
template <int kAhead, typename F>
__device__ __forceinline__ void each_vector(const Row& row, int32_t from, int32_t to, int32_t step, F f) {
  if (from < row.first && from < to) f(row.part(from), from);
  int32_t v = from < row.first ? from + step : from;
  const int32_t end = min(to, row.last);
  for (; v + (kAhead - 1) * static_cast<int64_t>(step) < end; v += kAhead * step) {
    uint4 x[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = row.whole(v + i * step);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f(x[i], v + i * step);
  }
  // the rest, in one go
  uint4 x[kAhead - 1];
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i)
    if (v + i * step < end) x[i] = row.whole(v + i * step);
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i)
    if (v + i * step < end) f(x[i], v + i * step);
  if (row.last < to && row.last >= from && (row.last - from) % step == 0 && row.last < row.vectors) f(row.part(row.last), row.last);
}

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

__device__ __forceinline__ u128 broadcast(u128 v, int lane) {
  return (static_cast<u128>(__shfl_sync(0xffffffffu, static_cast<uint64_t>(v >> 64), lane)) << 64) |
         __shfl_sync(0xffffffffu, static_cast<uint64_t>(v), lane);
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
  // of a group of 32 bins: tokens before it (x, by its number), and the number of the n-th that has any (y, by n)
  uint2 group[kGroups];
  u128 batch[kBatches];  // sums of 32 filled groups
  u128 wide[kWarps];
  uint64_t scan[kWarps];
  uint32_t narrow[kWarps];
  union {
    // few tokens: key and complement of the index of each, and, in their order, that and the weight
    struct {
      uint64_t listed[kListed], sorted[kListed], weight[kListed];
      uint32_t place[kListed];
    };
    // else: what a value's weight loses in 0 to 31 steps of an exponent, in two limbs of 31 bits
    uint2 steps[kExponents][32];
  };
  uint16_t ids[kFew];
  int32_t list_size, id_count;
  // the border to find, the batch in which it lies and the sum before that, and what was found, by one thread for all
  u128 border, kept, upto;
  int32_t found;
  uint32_t key;
  int32_t nth;
  float logprob;
  int32_t index;
};

struct Cuts {
  Heat heat;
  uint32_t top;  // the largest key
  uint32_t top_k;
  uint64_t min_weight;
};

// The warp's sum of v < 2^108, whole in every lane: limbs of 27 bits, whose sums over 32 lanes fit 32 bits.
__device__ __forceinline__ u128 warp_sum(u128 v) {
  u128 sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    sum += static_cast<u128>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(v >> (27 * i)) & 0x7ffffffu)) << (27 * i);
  return sum;
}

// A sum of weights times counts (together below 2^31), in two limbs: weights have 62 bits, and one instruction multiplies
// 32 and adds 64.
struct Sum {
  uint64_t lo = 0, hi = 0;
  __device__ __forceinline__ u128 whole() const { return (static_cast<u128>(hi) << 31) + lo; }
};

// a * b / 2^62 of numbers up to 2^62, less 2 at most: the low limbs' product, below 1, is left out, and the rest rounded down.
__device__ __forceinline__ uint64_t product62(uint64_t a, uint64_t b) {
  const uint32_t a0 = static_cast<uint32_t>(a) & 0x7fffffffu, a1 = static_cast<uint32_t>(a >> 31);
  const uint32_t b0 = static_cast<uint32_t>(b) & 0x7fffffffu, b1 = static_cast<uint32_t>(b >> 31);
  const uint64_t cross = static_cast<uint64_t>(a1) * b0 + static_cast<uint64_t>(a0) * b1;
  return static_cast<uint64_t>(a1) * b1 + (cross >> 31);
}

// This lane's tokens of a group (`count` in its bin, `rank` before the group) that are among the first top_k.
__device__ __forceinline__ uint32_t among_first(uint32_t count, uint32_t rank, uint32_t top_k) {
  if (rank >= top_k) return 0;
  const uint32_t ahead = warp_scan(count) - count, left = top_k - rank;
  return ahead >= left ? 0u : min(count, left - ahead);
}

// The counts of a round, bins 0 .. bins - 1 for keys first_key - bin, and their sums: over groups of 32 bins, of which
// those that hold any tokens are shared out, in order, a group to a lane.
//
// first_key ends in five ones, so that a group's keys differ in their last five bits alone: its values are evenly spaced,
// and their weights the group's first one times powers of one factor, which the groups of an exponent share. A lane so adds
// up counts times steps, two instructions a bin, and multiplies by the group's first weight once. (A weight for each bin by
// itself took 90 instructions of each lane, 20 of the 29 thousand clocks of a row of 151936 fp16 logits.) Bins are taken
// one by one where that does not do: in the first group, whose first values may be above the largest of the row, in one that
// top-k or min-p cuts, and at exponents 2^-32 of the largest. A group's sum, rounded down twice, and the sum over its bins may
// differ by a unit or two a token.
template <typename T>
struct Round {
  uint32_t first_key;
  int at;               // place of its bin
  int bins;
  int least;            // the lowest exponent in the table
  int32_t filled;       // groups with tokens
  u128 before, mine[2];  // sum before the round (in the first warp), and of this lane's groups

  __device__ __forceinline__ uint32_t group_key(uint32_t g) const { return first_key - 32 * g; }
  __device__ __forceinline__ bool even(const Cuts& c, uint32_t g) const {
    return group_key(g) <= c.top && exponent_of<T>(group_key(g)) >= least;
  }
  // Weight of bin `i` of a group with that first weight.
  __device__ __forceinline__ uint64_t weight(const Shared& sm, const Cuts& c, uint32_t g, int i, uint64_t first) const {
    if (even(c, g)) {
      const uint2 step = sm.steps[exponent_of<T>(group_key(g)) - least][i];
      return product62(first, (static_cast<uint64_t>(step.y) << 31) + step.x);
    }
    const uint32_t key = group_key(g) - i;
    return key <= c.top ? weight_of(c.heat, value_of<T>(key)) : 0;
  }
  __device__ __forceinline__ uint64_t first_weight(const Cuts& c, uint32_t g) const {
    return even(c, g) ? weight_of(c.heat, value_of<T>(group_key(g))) : 0;
  }

  // The sum of a group's weights, `rank` tokens before it, and that of the weights of at least min_weight; for a lane's
  // group each, or, where a lane's is to be taken bin by bin, by the warp. To be called by whole warps.
  __device__ __forceinline__ u128 sum_of(const Shared& sm, const Cuts& c, bool any, uint32_t g, uint32_t rank, u128* above) const {
    const int lane = threadIdx.x & 31;
    const uint32_t* count = sm.bin + at + 32 * g;
    const uint64_t first = any ? first_weight(c, g) : 0;
    any = any && rank < c.top_k;
    bool apart = any && !even(c, g);
    if (c.top_k != 0xffffffffu && any && !apart) {
      uint32_t n = 0;
      for (int i = 0; i < 32; ++i) n += count[(i + lane) & 31];
      apart = n > c.top_k - rank;
    }
    const bool low = first < c.min_weight;  // none reaches min_weight
    if (c.min_weight > 0 && any && !apart && !low) apart = weight(sm, c, g, 31, first) < c.min_weight;
    u128 total = 0;
    if (any && !apart) {
      const uint2* step = sm.steps[exponent_of<T>(group_key(g)) - least];
      Sum sum;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) {
        const int at = (i + lane) & 31;  // lanes read different banks
        const uint32_t n = count[at];
        const uint2 s = step[at];
        sum.lo += static_cast<uint64_t>(s.x) * n;
        sum.hi += static_cast<uint64_t>(s.y) * n;
      }
      // first * (hi * 2^31 + lo) / 2^62, in limbs of 31 bits of the first: 2^62 * 2^31 a product at most
      const uint32_t f0 = static_cast<uint32_t>(first) & 0x7fffffffu, f1 = static_cast<uint32_t>(first >> 31);
      const u128 whole = sum.whole();
      total = (whole * f1 + ((whole * f0) >> 31)) >> 31;
      if (!low) *above += total;
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, apart); todo != 0u; todo &= todo - 1) {
      const int who = __ffs(todo) - 1;
      const uint32_t its = __shfl_sync(0xffffffffu, g, who), ahead = __shfl_sync(0xffffffffu, rank, who);
      const uint32_t held = sm.bin[at + 32 * its + lane], n = c.top_k != 0xffffffffu ? among_first(held, ahead, c.top_k) : held;
      const uint64_t w = n != 0u ? weight(sm, c, its, lane, first_weight(c, its)) : 0;
      const u128 part = static_cast<u128>(w) * n, all = warp_sum(part), some = warp_sum(w >= c.min_weight ? part : 0);
      if (lane == who) {
        total = all;
        *above += some;
      }
    }
    return total;
  }

  // Adds the round's tokens, weights, and weights of at least min_weight to the three sums, the latter two in the first warp
  // alone: sums of 128 bits take it 60 instructions, and all warps 32 times that.
  __device__ __forceinline__ void add_up(Shared& sm, const Cuts& c, uint32_t& ranks, u128& total, u128& above) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, groups = (bins + 31) / 32;
    // tokens in the low half, filled groups in the high half
    uint64_t size[kPer], own = 0, all;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * threadIdx.x + i;
      uint32_t n = 0;
      if (g < groups) {
        const uint4* in = reinterpret_cast<const uint4*>(sm.bin + at + 32 * g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 v = in[(j + lane) & 7];  // eight lanes read different banks
          n += v.x + v.y + v.z + v.w;
        }
      }
      size[i] = n == 0u ? 0 : (1ull << 32) + n;
      own += size[i];
    }
    uint64_t place = block_scan(own, sm.scan, &all);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = kPer * threadIdx.x + i;
      if (size[i] != 0) {
        sm.group[g].x = ranks + static_cast<uint32_t>(place);
        sm.group[place >> 32].y = g;
      }
      place += size[i];
    }
    filled = static_cast<int32_t>(all >> 32);
    ranks += static_cast<uint32_t>(all);
    before = total;
    __syncthreads();
    u128 own_above = 0;
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      const int batch = warp + kWarps * i, n = 32 * batch + lane;
      if (batch >= kBatches) break;
      if (32 * batch >= filled) {
        if (lane == 0) sm.batch[batch] = 0;
        continue;
      }
      const uint32_t g = n < filled ? sm.group[n].y : 0u;
      u128 sum = sum_of(sm, c, n < filled, g, sm.group[g].x, &own_above);
      if (i == 0) mine[0] = sum;
      else mine[1] = sum;
      sum = warp_sum(sum);
      if (lane == 0) sm.batch[batch] = sum;
    }
    __syncthreads();
    if (warp == 0) total += warp_sum(sm.batch[lane] + (lane + kWarps < kBatches ? sm.batch[lane + kWarps] : 0));
    if (c.min_weight > 0) {
      own_above = warp_sum(own_above);
      if (lane == 0) sm.wide[warp] = own_above;
      __syncthreads();
      if (warp == 0) above += warp_sum(sm.wide[lane]);
    }
  }

  // Whether the running sum passes sm.border in this round; one thread then has called found(bin, its weight, its tokens, the
  // sum before it).
  template <typename F>
  __device__ __forceinline__ bool find(Shared& sm, const Cuts& c, F found) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp == 0) {
      const u128 border = sm.border;
      u128 upto = before;
      int batch = -1;
#pragma unroll 1
      for (int i = 0; i < 2 && batch < 0; ++i) {
        const u128 s = lane + kWarps * i < kBatches ? sm.batch[lane + kWarps * i] : 0, incl = upto + warp_scan(s);
        const uint32_t hit = __ballot_sync(0xffffffffu, incl > border);
        if (hit != 0u) {
          batch = __ffs(hit) - 1 + kWarps * i;
          upto = broadcast(incl - s, __ffs(hit) - 1);
        } else {
          upto = broadcast(incl, 31);
        }
      }
      if (lane == 0) {
        sm.found = batch;
        sm.upto = upto;
      }
    }
    __syncthreads();
    const int batch = sm.found;
    if (batch < 0) {
      __syncthreads();  // read by all before the next round's search
      return false;
    }
    if (warp == (batch & (kWarps - 1))) {
      const u128 border = sm.border;
      u128 upto = sm.upto;
      const u128 s = batch < kWarps ? mine[0] : mine[1], incl = upto + warp_scan(s);
      const int who = __ffs(__ballot_sync(0xffffffffu, incl > border)) - 1;
      upto = broadcast(incl - s, who);
      const uint32_t g = sm.group[32 * batch + who].y;
      const uint32_t held = sm.bin[at + 32 * g + lane], count = c.top_k != 0xffffffffu ? among_first(held, sm.group[g].x, c.top_k) : held;
      const uint64_t w = weight(sm, c, g, lane, first_weight(c, g));
      const u128 part = static_cast<u128>(w) * count, to = upto + warp_scan(part);
      // the last bin with tokens where the sum over the bins falls short of the group's
      uint32_t hit = __ballot_sync(0xffffffffu, to > border);
      if (hit == 0u) hit = 0x80000000u >> __clz(__ballot_sync(0xffffffffu, count > 0 && w > 0));
      if (lane == __ffs(hit) - 1) found(32 * static_cast<int>(g) + lane, w, count, to - part);
    }
    __syncthreads();
    return true;
  }
};

// The whole of the choice among n tokens that are listed, n <= kListed.
template <typename T>
__device__ __forceinline__ void sample_listed(Shared& sm, const Cuts& c, int n, float top_p, float u, int64_t* token, float* logprob) {
  const int tid = threadIdx.x, lane = tid & 31;
  // Each token's place is the number of those ahead of it, counted by teams of threads that share the others.
  int wide = 32;
  while (wide < n) wide *= 2;
  const int parts = kThreads / wide, me = tid & (wide - 1), part = tid / wide;
  if (me < n) {
    const uint64_t mine = sm.listed[me];
    int ahead = 0;
    for (int j = part; j < n; j += parts) ahead += sm.listed[j] > mine;
    atomicAdd(&sm.place[me], ahead);
  }
  __syncthreads();
  if (tid < n) {
    const uint64_t mine = sm.listed[tid];
    const uint32_t at = sm.place[tid];
    sm.sorted[at] = mine;
    sm.weight[at] = at < c.top_k ? weight_of(c.heat, value_of<T>(static_cast<uint32_t>(mine >> 32))) : 0;
  }
  __syncthreads();
  if (tid >= 32) return;
  // Each lane a run of the order.
  constexpr int kRun = kListed / 32;
  const int run = (n + 31) / 32, first = lane * run, last = min(first + run, n);
  uint64_t w[kRun];
  u128 mine = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    w[i] = i < run && first + i < last ? sm.weight[first + i] : 0;
    mine += w[i];
  }
  const u128 upto = warp_scan(mine), total = broadcast(upto, 31), before = upto - mine;
  u128 kept = total;
  if (c.min_weight > 0) {
    u128 above = 0;
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (w[i] >= c.min_weight) above += w[i];
    kept = warp_sum(above);
  }
  // The running sum up to and with the token that passes `border`; its place, weight.
  int at = 0;
  uint64_t weight = 0;
  auto pass = [&](u128 border) {
    const int who = __ffs(__ballot_sync(0xffffffffu, before <= border && border < upto)) - 1;
    u128 sum = before;
    int found = -1;
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (found < 0) {
        sum += w[i];
        if (sum > border) found = i;
      }
    at = __shfl_sync(0xffffffffu, first + max(found, 0), who);
    weight = sm.weight[at];
    return broadcast(sum, who);
  };
  if (top_p < 1.f) {
    const u128 goal = share_of(fmaxf(top_p, 0.f), total, true);
    kept = lesser(kept, pass(goal > 0 ? goal - 1 : 0));
  }
  pass(share_of(u, kept, false));
  if (lane == 0) {
    *token = static_cast<int64_t>(~static_cast<uint32_t>(sm.sorted[at]));
    if (logprob != nullptr) *logprob = log_share(weight, kept);
  }
}

// f(vector, its number) for the vectors of the threads for which `mine` is true (n of them, at most kFew), spread over all
// threads. To be called by every thread.
template <typename F>
__device__ __forceinline__ void each_of_few(Shared& sm, const Row& row, bool mine, int n, F f) {
  const int tid = threadIdx.x;
  const uint32_t in = __ballot_sync(0xffffffffu, mine);
  int at = 0;
  if ((tid & 31) == 0 && in != 0u) at = atomicAdd(&sm.id_count, __popc(in));
  at = __shfl_sync(0xffffffffu, at, 0) + __popc(in & ((1u << (tid & 31)) - 1u));
  if (mine) sm.ids[at] = static_cast<uint16_t>(tid);
  __syncthreads();
  const int rounds = (row.vectors + kThreads - 1) / kThreads;
  for (int32_t j = tid; j < n * rounds; j += kThreads) {  // 256 * 2^18 at most
    const int32_t i = j / n, v = sm.ids[j - i * n] + kThreads * i;
    if (v < row.vectors) f(v >= row.first && v < row.last ? row.whole(v) : row.part(v), v);
  }
}

// Settings of a row.
struct Setting {
  float temperature, top_p, min_p;
  int32_t k;
  __device__ __forceinline__ Setting(const SampleArgs& a, int32_t b)
      : temperature(a.temperature == nullptr ? 1.f : a.temperature[b]), top_p(a.top_p == nullptr ? 1.f : a.top_p[b]),
        min_p(a.min_p == nullptr ? 0.f : a.min_p[b]), k(a.top_k == nullptr ? 0 : a.top_k[b]) {}
  // Whether the largest alone is asked for.
  __device__ __forceinline__ bool greedy() const { return !(temperature >= 1.17549435e-38f) || k == 1; }
  // Whether every token counts (no top-k that a list holds, nor a min-p alone): such a row takes longer than others. The list
  // for a top-k has some more tokens than that: 230 for 200. (256 x 151936, top-k 200: 37 us listed; 256, the list too short
  // and then the bins: 69; 300, straight into the bins: 60.)
  __device__ __forceinline__ bool all() const { return !greedy() && (k <= 0 || k > kListed * 7 / 8) && (top_p < 1.f || !(min_p > 0.f)); }
};

// The least key whose weight is not 0 in units of 2^-62 of that of the largest (which is below exp(-45)), or that `reach`
// temperatures below it.
template <typename T>
__device__ __forceinline__ uint32_t floor_of(float top, float temperature, float reach) {
  const float least = top - reach * temperature;
  uint32_t key = Keys<T>::kFloor + 1;
  if (least == least) key = max(key, key_from<T>(least));
  return key == kZero ? kMinusZero : key;
}

// The i-th row and the then-th (-1: there is none), the long ones first. For at most kThreads rows.
__device__ __forceinline__ int2 rows_of(const SampleArgs& a, Shared& sm, int32_t i, int32_t then) {
  const int tid = threadIdx.x, lane = tid & 31;
  const bool slow = tid < a.B && Setting(a, tid).all();
  const uint32_t in = __ballot_sync(0xffffffffu, slow);
  if (lane == 0) sm.narrow[tid >> 5] = __popc(in);
  __syncthreads();
  const uint32_t mine = sm.narrow[lane], upto = warp_scan(mine), all = __shfl_sync(0xffffffffu, upto, 31);
  const int32_t ahead = __shfl_sync(0xffffffffu, upto - mine, tid >> 5) + __popc(in & ((1u << lane) - 1u));
  const int32_t place = slow ? ahead : static_cast<int32_t>(all) + tid - ahead;
  if (tid == 0) sm.nth = -1;
  __syncthreads();
  if (tid < a.B && place == i) sm.index = tid;
  if (tid < a.B && place == then) sm.nth = tid;
  __syncthreads();
  return make_int2(sm.index, sm.nth);
}

// Brings a row to the L2 cache; one warp.
__device__ __forceinline__ void prefetch_row(const SampleArgs& a, int32_t b) {
  constexpr uint32_t kPiece = 8192;
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.logits + b * a.stride), from = (at + 15) & ~static_cast<uintptr_t>(15);
  const uintptr_t to = (at + 2 * static_cast<uintptr_t>(a.V)) & ~static_cast<uintptr_t>(15);
  for (uintptr_t p = from + kPiece * (threadIdx.x & 31); p < to; p += 32 * kPiece)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(static_cast<uint32_t>(to - p < kPiece ? to - p : kPiece)) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a, bool ordered, int32_t ahead) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Shared& sm = *reinterpret_cast<Shared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  int2 rows = make_int2(static_cast<int32_t>(blockIdx.x), static_cast<int64_t>(blockIdx.x) + ahead < a.B ? static_cast<int32_t>(blockIdx.x) + ahead : -1);
  if (ordered) rows = rows_of(a, sm, rows.x, rows.y);
  const int32_t b = rows.x;
  const Row row(a.logits + b * a.stride, a.V);
  const Setting set(a, b);
  const float given = a.u[b], u = given > 0.f ? fminf(given, 0.999999940395355225f) : 0.f;
  auto block_max = [&](uint32_t v) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) sm.narrow[warp] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, sm.narrow[lane]);
  };

  // ------------------------------------------------------------------- the largest value
  // Where every token counts, they go into the bins on the same pass: those from the floor below the largest of the first
  // 8192 up to `end`, as many as there are bins for. They do for the whole row unless its largest is above that.
  uint32_t two = 0, own, end = 0, low = 0;  // of this thread's vectors tid, tid + 1024, ...
  auto largest_two = [](const uint4& v) { return __vmaxu2(__vmaxu2(two_keys(v.x), two_keys(v.y)), __vmaxu2(two_keys(v.z), two_keys(v.w))); };
  const int32_t rest = tid + kThreads;
  uint4 head;  // the first of them
  if (tid >= row.first && tid < row.last) head = row.whole(tid);
  else head = tid < row.vectors ? row.part(tid) : make_uint4(~0u, ~0u, ~0u, ~0u);  // NaN
  const bool all = set.all();
  two = __vmaxu2(two, largest_two(head));
  if (all) {
    uint32_t some = max(two & 0xffffu, two >> 16);
    if (some > Keys<T>::kTop) {
      some = 0;
      each_key(head, [&](uint32_t s, int) {
        if (s <= Keys<T>::kTop) some = max(some, s);
      });
    }
    some = block_max(some);
    if (some > Keys<T>::kFloor) {
      low = floor_of<T>(value_of<T>(some), set.temperature, 45.f);
      end = min((low & ~31u) + kBins, 0x10000u);
      if (some >= end) end = 0;
    }
  }
  if (end != 0) {
    const uint32_t last_key = end - 1, n = end - low;
    for (uint32_t i = tid; i < (n + 31) / 32 * 8; i += kThreads) reinterpret_cast<uint4*>(sm.bin)[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    auto put = [&](uint32_t s, int) {
      if (last_key - s < n) atomicAdd(&sm.bin[last_key - s], 1u);
    };
    each_key(head, put);
    each_vector<4>(row, rest, row.vectors, kThreads, [&](const uint4& v, int32_t) {
      two = __vmaxu2(two, largest_two(v));
      each_key(v, put);
    });
  } else {
    each_vector<4>(row, rest, row.vectors, kThreads, [&](const uint4& v, int32_t) { two = __vmaxu2(two, largest_two(v)); });
  }
  own = max(two & 0xffffu, two >> 16);
  if (own > Keys<T>::kTop) {  // NaN among them
    own = 0;
    each_vector<4>(row, tid, row.vectors, kThreads, [&](const uint4& v, int32_t) {
      each_key(v, [&](uint32_t s, int) {
        if (s <= Keys<T>::kTop) own = max(own, s);
      });
    });
  }
  if (own == kMinusZero) own = kZero;
  const uint32_t top = block_max(own);
  if (tid == 0) {
    sm.list_size = 0;
    sm.id_count = 0;
    sm.index = 0x7fffffff;
  }
  const bool counted = top < end;
  // The row of the block that follows on this SM, now that this one has been read.
  if (ahead > 0 && rows.y >= 0 && warp == 0) prefetch_row(a, rows.y);
  if (top <= Keys<T>::kFloor) {  // nothing is left of the row
    if (tid == 0) {
      a.token[b] = -1;
      if (a.logprob != nullptr) a.logprob[b] = -INFINITY;
    }
    return;
  }

  uint32_t key = top;
  int32_t nth = 0;
  float logprob = 0.f;
  if (!set.greedy()) {
    const float top_p = set.top_p, min_p = set.min_p;
    Cuts c;
    c.heat = heat_of(value_of<T>(top), set.temperature);
    c.top = top;
    c.top_k = set.k <= 0 ? 0xffffffffu : static_cast<uint32_t>(set.k);
    // (above 1 as 1: the largest and its equals)
    c.min_weight = min_p > 0.f ? static_cast<uint64_t>(share_of(fminf(min_p, 1.f), static_cast<u128>(1) << kOne, true)) : 0;
    // Which keys count at all. Those below min_p matter to the sum that top_p is a part of, but without top_p to nothing.
    float reach = 45.f;
    if (min_p > 0.f && !(top_p < 1.f)) reach = fminf(reach, -logf(fminf(min_p, 1.f)) * 1.001f + 1e-5f);
    uint32_t floor_key = floor_of<T>(c.heat.top, set.temperature, reach);
    if (c.top_k <= kThreads && !counted) {
      // At least k tokens are as large as the k-th largest of the threads' own largest, so none below it counts. It is
      // looked for in the first bins, else by bisection.
      constexpr int kNear = kPer * kThreads;
      reinterpret_cast<uint2*>(sm.bin)[tid] = make_uint2(0u, 0u);
      __syncthreads();
      if (top - own < kNear) atomicAdd(&sm.bin[top - own], 1u);
      __syncthreads();
      const uint2 n = reinterpret_cast<const uint2*>(sm.bin)[tid];
      uint32_t all, upto = block_scan(n.x + n.y, sm.narrow, &all);
      if (all >= c.top_k) {
        if (upto < c.top_k && upto + n.x + n.y >= c.top_k) sm.key = top - (kPer * tid + (upto + n.x >= c.top_k ? 0 : 1));
        __syncthreads();
        floor_key = max(floor_key, sm.key);
      } else {
        uint32_t lo = 0, hi = 0x10000;  // count(own >= lo) >= k > count(own >= hi)
        while (hi - lo > 1) {
          const uint32_t mid = (lo + hi) / 2;
          if (static_cast<uint32_t>(__syncthreads_count(own >= mid)) >= c.top_k) lo = mid;
          else hi = mid;
        }
        floor_key = max(floor_key, lo);
      }
    }
    if (counted) floor_key = max(floor_key, low);
    if (floor_key == kZero) floor_key = kMinusZero;  // the k-th largest
    const uint32_t first_bin = top | 31u;
    const int bins = static_cast<int>(first_bin - floor_key) + 1, rounds = (bins + kBins - 1) / kBins;
    const int looked_at = __syncthreads_count(own >= floor_key);
    if (looked_at <= kFew && !counted) {
      if (tid < kListed) sm.place[tid] = 0;
      each_of_few(sm, row, own >= floor_key, looked_at, [&](const uint4& v, int32_t at) {
        const uint32_t most = __vmaxu2(__vmaxu2(two_keys(v.x), two_keys(v.y)), __vmaxu2(two_keys(v.z), two_keys(v.w)));
        if (max(most & 0xffffu, most >> 16) < floor_key) return;
        each_key(v, [&](uint32_t s, int i) {
          if (s == kMinusZero) s = kZero;
          if (s < floor_key || s > top) return;  // above the largest: NaN
          const int place = atomicAdd(&sm.list_size, 1);
          if (place < kListed) sm.listed[place] = (static_cast<uint64_t>(s) << 32) | ~static_cast<uint32_t>(8 * at - row.skip + i);
        });
      });
      __syncthreads();
      if (sm.list_size <= kListed) {
        sample_listed<T>(sm, c, sm.list_size, top_p, u, a.token + b, a.logprob == nullptr ? nullptr : a.logprob + b);
        return;
      }
    }

    Round<T> round;
    {
      // The table of steps, an exponent to a warp.
      round.least = max(exponent_of<T>(top), exponent_of<T>(floor_key)) - (kExponents - 1);
      __syncthreads();  // the list is over
      const float step = ldexpf(static_cast<float>(lane), round.least + warp - Keys<T>::kBias) * c.heat.unit;
      const uint64_t w = falling(c.heat, step, 0.f);
      sm.steps[warp][lane] = make_uint2(static_cast<uint32_t>(w) & 0x7fffffffu, static_cast<uint32_t>(w >> 31));
    }
    auto count = [&](int r) {
      round.first_key = first_bin - kBins * r;
      round.bins = min(kBins, bins - kBins * r);
      round.at = counted ? static_cast<int>(end - 1 - first_bin) : 0;
      __syncthreads();  // the last round's readers are through
      if (!counted) {
        for (int i = tid; i < (round.bins + 31) / 32 * 8; i += kThreads) reinterpret_cast<uint4*>(sm.bin)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
      }
      const uint32_t first_key = round.first_key, n = static_cast<uint32_t>(round.bins);
      uint32_t* const bin = sm.bin + round.at;
      if (counted) {  // on the first pass
      } else if (own >= floor_key && rounds == 1) {
        each_vector<4>(row, tid, row.vectors, kThreads, [&](const uint4& v, int32_t) {
          each_key(v, [&](uint32_t s, int) {
            if (first_key - s < n) atomicAdd(&sm.bin[first_key - s], 1u);
          });
        });
      } else if (own >= floor_key) {
        each_vector<2>(row, tid, row.vectors, kThreads, [&](const uint4& v, int32_t) {
          each_key(v, [&](uint32_t s, int) {
            if (s == kMinusZero) s = kZero;
            if (first_key - s < n)  // keys of the rounds before wrap around
              atomicAdd(&sm.bin[first_key - s], 1u);
          });
        });
      }
      __syncthreads();
      if (rounds == 1 && top >= kZero && first_key - kMinusZero < n) {  // in one round -0 is counted on its own
        if (tid == 0) {
          bin[first_key - kZero] += bin[first_key - kMinusZero];
          bin[first_key - kMinusZero] = 0;
        }
        __syncthreads();
      }
      if (r == 0 && first_bin > Keys<T>::kTop) {  // bins above the largest are those of NaN
        if (tid < static_cast<int>(first_bin - top)) bin[tid] = 0u;
        __syncthreads();
      }
    };
    uint32_t ranks = 0;
    u128 total = 0, above = 0;
    for (int r = 0; r < rounds; ++r) {
      count(r);
      round.add_up(sm, c, ranks, total, above);
    }
    // Again, round by round, where one does not hold them all; true once f is.
    auto again = [&](auto f) {
      uint32_t rc = 0;
      u128 sc = 0, unused = 0;
      for (int r = 0; r < rounds; ++r) {
        if (rounds > 1) {
          count(r);
          round.add_up(sm, c, rc, sc, unused);
        }
        if (f()) return;
      }
    };
    // Borders and what lies at them: 128-bit arithmetic, by one thread.
    auto aim = [&] {
      sm.border = share_of(u, sm.kept, false);
    };
    if (tid == 0) {
      sm.kept = c.min_weight > 0 ? lesser(total, above) : total;
      if (top_p < 1.f) {
        // Tokens before which the running sum is below the border are kept: up to the first sum that reaches it.
        const u128 goal = share_of(fmaxf(top_p, 0.f), total, true);
        sm.border = goal > 0 ? goal - 1 : 0;
      } else {
        aim();
      }
    }
    __syncthreads();
    if (top_p < 1.f)
      again([&] {
        return round.find(sm, c, [&](int, uint64_t w, uint32_t n, u128 ahead) {
          sm.kept = lesser(sm.kept, ahead + static_cast<u128>(min(quotient(sm.border - ahead, w) + 1, static_cast<int64_t>(n))) * w);
          aim();
        });
      });
    again([&] {
      return round.find(sm, c, [&](int bin, uint64_t w, uint32_t n, u128 ahead) {
        sm.key = round.first_key - bin;
        sm.nth = static_cast<int32_t>(min(quotient(sm.border - ahead, w), static_cast<int64_t>(n) - 1));
        sm.logprob = log_share(w, sm.kept);
      });
    });
    key = sm.key;
    nth = sm.nth;
    logprob = sm.logprob;
  }

  // ------------------------------------------------------- the nth element of that value
  const uint32_t twin = key == kZero ? kMinusZero : key;
  // Vectors without that value are passed by: the least of (x ^ value) over a vector's low and high halves is not 0.
  // (The zeros of both signs differ in a bit that is left out.)
  const uint32_t pair = (key & 0x8000u ? key & 0x7fffu : ~key & 0xffffu) * 0x10001u, bits_used = key == kZero ? 0x7fff7fffu : 0xffffffffu;
  auto holds = [&](const uint4& v) {
    const uint32_t x = __vminu2(__vminu2((v.x ^ pair) & bits_used, (v.y ^ pair) & bits_used), __vminu2((v.z ^ pair) & bits_used, (v.w ^ pair) & bits_used));
    return (x & 0xffffu) == 0u || x < 0x10000u;
  };
  if (key == top && nth == 0) {
    // The least index of those threads that have it, if they are few.
    const int n = __syncthreads_count(own == top);
    if (n <= kFew) {
      __syncthreads();
      if (tid == 0) sm.id_count = 0;
      __syncthreads();
      each_of_few(sm, row, own == top, n, [&](const uint4& v, int32_t at) {
        int32_t least = 0x7fffffff;
        each_key(v, [&](uint32_t s, int i) {
          if (s == key || s == twin) least = min(least, 8 * at - row.skip + i);
        });
        if (least != 0x7fffffff) atomicMin(&sm.index, least);
      });
      __syncthreads();
      if (tid == 0) {
        a.token[b] = sm.index;
        if (a.logprob != nullptr) a.logprob[b] = logprob;
      }
      return;
    }
  }
  // Each warp takes an equal run of vectors: how many it has; then the block takes the run with the nth, a vector to a thread.
  // (A warp by itself searched its run up to 7 us: 256 x 151936 with mixed settings 50 us, 44.5 so.)
  const int32_t run = (row.vectors + kWarps - 1) / kWarps, v0 = min(row.vectors, warp * run), v1 = min(row.vectors, v0 + run);
  uint32_t mine = 0;
  each_vector<4>(row, v0 + lane, v1, 32, [&](const uint4& v, int32_t) {
    if (holds(v)) each_key(v, [&](uint32_t s, int) { mine += s == key || s == twin; });
  });
  mine = __reduce_add_sync(0xffffffffu, mine);
  __syncthreads();
  if (lane == 0) sm.narrow[warp] = mine;
  __syncthreads();
  const uint32_t its = sm.narrow[lane], upto = warp_scan(its);
  const int who = __ffs(__ballot_sync(0xffffffffu, upto > static_cast<uint32_t>(nth))) - 1;
  uint32_t left = nth - __shfl_sync(0xffffffffu, upto - its, who);
  const int32_t last = min(row.vectors, (who + 1) * run);
  for (int32_t from = who * run; from < last; from += kThreads) {
    const int32_t v = from + tid;
    uint32_t bits = 0, all;  // of this thread's eight
    if (v < last) each_key(v >= row.first && v < row.last ? row.whole(v) : row.part(v), [&](uint32_t s, int i) { bits |= static_cast<uint32_t>(s == key || s == twin) << i; });
    const uint32_t has = __popc(bits), before = block_scan(has, sm.narrow, &all);
    if (before <= left && left < before + has) {
      for (uint32_t n = left - before; n > 0; --n) bits &= bits - 1;
      a.token[b] = 8 * static_cast<int64_t>(v) - row.skip + (__ffs(bits) - 1);
      if (a.logprob != nullptr) a.logprob[b] = logprob;
    }
    if (left < all) break;
    left -= all;
  }
}

template <typename T>
bool launch(const SampleArgs& a, cudaStream_t s) {
  constexpr size_t smem = sizeof(Shared);
  static_assert(smem <= 227 * 1024, "the bins fit the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(sample_kernel<T>), smem)) return false;
  // More rows than SMs: the long ones go first, or the last of them is waited for.
  const int sms = sm_count();
  const bool ordered = a.B > sms && a.B <= kThreads;
  launch_overlapped(sample_kernel<T>, dim3(static_cast<unsigned>(a.B)), kThreads, smem, 1, s, a, ordered, a.B > sms ? sms : 0);
  return true;
}

}  // namespace

bool launch_sample(const SampleArgs& a, int dtype, cudaStream_t s) {
  return dtype == DT_BF16 ? launch<__nv_bfloat16>(a, s) : launch<__half>(a, s);
}

}  // namespace fq
