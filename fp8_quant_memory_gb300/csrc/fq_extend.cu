// fq_extend.cu -- block tables and slot maps of one step from the requests' lengths.
//
// All of it follows from three running sums over the sequences: tokens added, pages needed (of the sequences that fit),
// pages returned. A sequence is granted its pages if the sum up to and with its own is at most the free pages: so those
// granted any are the first ones that need some, the pages taken are the first of the ring, and the j-th of them belongs
// to the sequence whose sums enclose j. Tokens and returned pages find their sequence the same way.
//
// What bounds it: one launch and two dependent rounds of loads (lengths; table and ring entries), not bytes: a step of 64
// tokens moves 3.6 KB, one of 65536 1 MB. One cluster does the whole step: every CTA sums all lengths itself (a few
// per thread, in L2), then takes its share of the tokens and pages. Lengths and pool may be updated in place, so they are
// written behind a barrier of the cluster, after every CTA has read them.
#include "fq_serving.h"
#include "fq_sync.cuh"
#include "fq_tcgen05.cuh"

namespace fq {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kRefused = 0x80000000u;  // flag in `need`'s sums

__device__ __forceinline__ int32_t cut(int64_t v) { return v > 0x7fffffffLL ? 0x7fffffff : static_cast<int32_t>(v); }

// The block's exclusive sum of v over its threads, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scan, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int64_t w = scan[lane];  // kWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
  return before + incl - v;
}

// The last i in [0, n) with first[i] <= x; first[0] <= x.
__device__ __forceinline__ int32_t owner(const uint32_t* first, int32_t n, uint32_t mask, uint32_t x) {
  int32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if ((first[mid] & mask) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Lengths, pool, table and ring are read through L2: this call writes them, and a kernel that starts on the same SM
// before this one ends must not find their old lines in L1.
__device__ __forceinline__ int32_t held_tokens(const ExtendArgs& a, int32_t b) { return max(__ldcg(a.lens + b), 0); }

// Pages of n < 2^31 tokens.
__device__ __forceinline__ uint32_t pages_of(const ExtendArgs& a, int64_t n) {
  return (static_cast<uint32_t>(n) + a.page_size - 1u) / static_cast<uint32_t>(a.page_size);
}

__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const ExtendArgs a) {
  extern __shared__ uint32_t sums[];
  uint32_t* tokens = sums;             // [B + 1], running sums before each sequence
  uint32_t* taken = sums + a.B + 1;    // with kRefused where a sequence is not granted its tokens
  uint32_t* given = taken + a.B + 1;   // returned pages
  __shared__ int64_t scan[kWarps];
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const int32_t per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, static_cast<int32_t>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  pdl_trigger();
  pdl_wait();
  const int64_t F = a.places;
  int64_t front = __ldcg(a.pool) % F;
  if (front < 0) front += F;
  const int64_t free_count = min(max(static_cast<int64_t>(__ldcg(a.pool + 1)), static_cast<int64_t>(0)), F);
  auto place = [&](int64_t i) { return a.ring + (front + i < F ? front + i : front + i - F); };  // 0 <= i <= F

  int64_t sum = 0, all_tokens, all_taken, all_given;
  for (int32_t b = b0; b < b1; ++b) sum += max(__ldcg(a.added + b), 0);
  int64_t at = block_scan(sum, scan, &all_tokens);
  int64_t need = 0, back = 0;
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = __ldcg(a.added + b), len = held_tokens(a, b);
    tokens[b] = cut(at);
    at += max(n, 0);
    const uint32_t held = pages_of(a, len);
    const int64_t then = static_cast<int64_t>(len) + n;
    const bool fits = n >= 0 && then <= static_cast<int64_t>(a.width) * a.page_size && at <= a.tokens;
    taken[b] = fits ? pages_of(a, then) - held : kRefused;
    given[b] = n < 0 ? min(held, static_cast<uint32_t>(a.width)) : 0u;
    need += taken[b] & ~kRefused;
    back += given[b];
  }
  int64_t off = block_scan(need, scan, &all_taken), off_back = block_scan(back, scan, &all_given);
  for (int32_t b = b0; b < b1; ++b) {
    const uint32_t own = taken[b] & ~kRefused, returned = given[b];
    const bool granted = (taken[b] & kRefused) == 0u && (own == 0u || off + own <= free_count);
    taken[b] = static_cast<uint32_t>(cut(off)) | (granted ? 0u : kRefused);
    given[b] = cut(off_back);
    off += own;
    off_back += returned;
  }
  if (threadIdx.x == 0) {
    tokens[a.B] = cut(all_tokens);
    taken[a.B] = cut(all_taken);
    given[a.B] = cut(all_given);
  }
  __syncthreads();
  // Pages taken: those of the granted ones, whose sums end where the free pages do, or at the last sum that is no more.
  int64_t last = min(all_taken, free_count);
  if (all_taken > free_count && a.B > 0) {
    const int32_t b = owner(taken, a.B + 1, ~kRefused, static_cast<uint32_t>(free_count));
    last = taken[b] & ~kRefused;  // the sequence whose pages would pass the border is refused
  }
  const int64_t room = F - free_count, returned = min(all_given, room);

  const uint32_t first = threadIdx.x + kThreads * rank, step = kThreads * ctas;
  for (int64_t t = first; t < a.tokens; t += step) {
    int64_t slot = -1;
    int32_t pos = 0;
    if (t < all_tokens) {
      const int32_t b = owner(tokens, a.B, ~0u, static_cast<uint32_t>(t));
      const int32_t len = held_tokens(a, b);
      pos = cut(len + (t - tokens[b]));
      const uint32_t own = taken[b];
      if ((own & kRefused) == 0u) {
        const int32_t at_page = pos / a.page_size, held = static_cast<int32_t>(pages_of(a, len));
        const int32_t id = at_page < held ? __ldcg(a.table + b * a.table_stride + at_page)
                                          : __ldcg(place(static_cast<int64_t>(own) + (at_page - held)));
        if (id >= 0) slot = static_cast<int64_t>(id) * a.page_size + (pos - at_page * a.page_size);
      }
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
  for (int64_t j = first; j < last; j += step) {
    const int32_t b = owner(taken, a.B, ~kRefused, static_cast<uint32_t>(j));
    const int64_t held = pages_of(a, held_tokens(a, b));
    a.table[b * a.table_stride + held + (j - (taken[b] & ~kRefused))] = __ldcg(place(j));
  }
  for (int64_t j = first; j < returned; j += step) {
    const int32_t b = owner(given, a.B, ~0u, static_cast<uint32_t>(j));
    *place(free_count + j) = __ldcg(a.table + b * a.table_stride + (j - given[b]));
  }
  // Every CTA has read the lengths and the pool.
  __syncthreads();
  if (ctas > 1) cluster_barrier();
  for (int32_t b = first; b <= a.B; b += step) {
    a.starts[b] = static_cast<int32_t>(tokens[b]);
    if (b == a.B) break;
    const int32_t n = __ldcg(a.added + b), len = held_tokens(a, b);
    a.lens_out[b] = (taken[b] & kRefused) == 0u ? len + n : n < 0 ? 0 : len;
  }
  if (first == 0) {
    a.pool_out[0] = static_cast<int32_t>(place(last) - a.ring);
    a.pool_out[1] = static_cast<int32_t>(free_count - last + returned);
    a.pool_out[2] = cut(all_taken - last);
  }
}

}  // namespace

bool launch_extend(const ExtendArgs& a, cudaStream_t s) {
  const size_t smem = 3 * (static_cast<size_t>(a.B) + 1) * sizeof(uint32_t);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(extend_kernel), smem)) return false;
  unsigned cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(cluster) * kThreads < a.tokens) cluster *= 2;
  launch_overlapped(extend_kernel, dim3(cluster), kThreads, smem, cluster, s, a);
  return true;
}

}  // namespace fq
