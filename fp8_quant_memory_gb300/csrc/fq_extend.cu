// fq_extend.cu -- block tables and slot maps of one step from the requests' lengths.
//
// All of it follows from three running sums over the sequences: tokens added, pages needed (of the sequences that fit),
// pages returned. A sequence is granted its pages if the sum up to and with its own is at most the free pages: so those
// granted any are the first ones that need some, the pages taken are the first of the ring, and the j-th of them belongs
// to the sequence whose sums enclose j. Tokens and returned pages find their sequence the same way.
//
// What bounds it: one launch and two dependent rounds of loads (lengths; table and ring entries), not bytes: a step of 64
// tokens moves 3.6 KB, one of 65536 1 MB. They take 3.6 and 8.0 us. Every CTA sums all lengths itself (a few per thread), then takes its share of the
// tokens and pages, so that none waits for another (returned pages that go to places which this step's pages leave, in a ring
// smaller than the pages, are one CTA's, with all that is to be read there first); only where lengths or pool are updated in place, the CTAs are one
// cluster and write them behind its barrier, after every CTA has read them.
#include "fq_serving.h"
#include "fq_sync.cuh"
#include "fq_tcgen05.cuh"

namespace fq {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kSmall = 256;                  // tokens and sequences of a step that one small block takes
constexpr uint32_t kRefused = 0x80000000u;  // flag in the sums of pages taken

__device__ __forceinline__ int32_t cut(int64_t v) { return v > 0x7fffffffLL ? 0x7fffffff : static_cast<int32_t>(v); }

// The block's exclusive sums of kN numbers over its threads, and the totals.
template <int kThreads, int kN>
__device__ __forceinline__ void block_scan(int64_t (&v)[kN], int64_t (*scan)[kThreads / 32], int64_t (&total)[kN]) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) incl[i] = v[i];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t u = __shfl_up_sync(0xffffffffu, incl[i], o);
      if (lane >= o) incl[i] += u;
    }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < kN; ++i) scan[i][warp] = incl[i];
  __syncthreads();
  int64_t w[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) w[i] = lane < kWarps ? scan[i][lane] : 0;
#pragma unroll
  for (int o = 1; o < kWarps; o <<= 1)
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int64_t u = __shfl_up_sync(0xffffffffu, w[i], o);
      if (lane >= o) w[i] += u;
    }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    total[i] = __shfl_sync(0xffffffffu, w[i], kWarps - 1);
    const int64_t before = __shfl_sync(0xffffffffu, w[i], warp == 0 ? 0 : warp - 1);
    v[i] = (warp == 0 ? 0 : before) + incl[i] - v[i];
  }
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

// Page of position t < 2^31; pages of n < 2^31 tokens.
__device__ __forceinline__ uint32_t page_of(const ExtendArgs& a, uint32_t t) {
  return static_cast<uint32_t>((static_cast<uint64_t>(t) * a.page_magic) >> a.page_magic_shift);
}
__device__ __forceinline__ uint32_t pages_of(const ExtendArgs& a, int64_t n) { return n == 0 ? 0u : page_of(a, static_cast<uint32_t>(n) - 1u) + 1u; }

// kRun: tokens that a thread takes at a time. A small step's block shares its warps out: half of them take tokens, a
// quarter the pages taken, a quarter those returned, each of which is a chain of loads.
template <int kThreads, int kRun, bool kSmallStep>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const ExtendArgs a) {
  extern __shared__ uint32_t sums[];
  uint32_t* tokens = sums;             // [B + 1], running sums before each sequence
  uint32_t* taken = sums + a.B + 1;    // with kRefused where a sequence is not granted its tokens
  uint32_t* given = taken + a.B + 1;   // returned pages
  uint32_t* lens = given + a.B + 1;    // tokens held
  __shared__ int64_t scan[2][kThreads / 32];
  const uint32_t ctas = gridDim.x, rank = blockIdx.x;
  const int32_t per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, static_cast<int32_t>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  pdl_trigger();
  pdl_wait();
  const int64_t F = a.places;
  int64_t front = __ldcg(a.pool);
  const int64_t free_count = min(max(static_cast<int64_t>(__ldcg(a.pool + 1)), static_cast<int64_t>(0)), F);
  int64_t sum[1] = {0}, all[2], all_tokens[1];
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = __ldcg(a.added + b);
    lens[b] = max(__ldcg(a.lens + b), 0);
    given[b] = n;  // for the moment
    sum[0] += max(n, 0);
  }
  if (front < 0 || front >= F) {
    front %= F;
    if (front < 0) front += F;
  }
  auto place = [&](int64_t i) { return a.ring + (front + i < F ? front + i : front + i - F); };  // 0 <= i <= F
  block_scan<kThreads>(sum, scan, all_tokens);
  int64_t at = sum[0], need[2] = {0, 0};  // pages taken, returned
  for (int32_t b = b0; b < b1; ++b) {
    const int32_t n = static_cast<int32_t>(given[b]), len = static_cast<int32_t>(lens[b]);
    tokens[b] = cut(at);
    at += max(n, 0);
    const uint32_t held = pages_of(a, len);
    const int64_t then = static_cast<int64_t>(len) + n;
    const bool fits = n >= 0 && then <= static_cast<int64_t>(a.width) * a.page_size && at <= a.tokens;
    taken[b] = fits ? pages_of(a, then) - held : kRefused;
    given[b] = n < 0 ? min(held, static_cast<uint32_t>(a.width)) : 0u;
    if (n < 0) lens[b] = 0;  // from here on, the length without the step's tokens
    need[0] += taken[b] & ~kRefused;
    need[1] += given[b];
  }
  block_scan<kThreads>(need, scan, all);
  const int64_t all_taken = all[0], all_given = all[1];
  int64_t off = need[0], off_back = need[1];
  for (int32_t b = b0; b < b1; ++b) {
    const uint32_t own = taken[b] & ~kRefused, returned = given[b];
    const bool granted = (taken[b] & kRefused) == 0u && (own == 0u || off + own <= free_count);
    taken[b] = static_cast<uint32_t>(cut(off)) | (granted ? 0u : kRefused);
    given[b] = cut(off_back);
    off += own;
    off_back += returned;
  }
  if (threadIdx.x == 0) {
    tokens[a.B] = cut(all_tokens[0]);
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
  // Places for returned pages: those behind the last free page, then those that this step's pages leave.
  const int64_t room = F - free_count, returned = min(all_given, room + last), refilled = max(returned - room, static_cast<int64_t>(0));
  // The first places are then written over: what is to be read there, tokens' pages among it, is left to the CTA that does so,
  // behind a barrier of its own.
  const uint32_t apart = ctas > 1 ? static_cast<uint32_t>(refilled) : 0u;
  const int passes = apart > 0u && rank == 0u ? 2 : 1;

  // This thread and how many there are for the tokens, the pages taken and those returned.
  constexpr uint32_t kPart = kThreads / 4;
  const uint32_t warps_of = kSmallStep ? threadIdx.x / kPart : 0u;
  const uint32_t first = threadIdx.x + kThreads * rank, step = kThreads * ctas;
  if (!kSmallStep || warps_of < 2) {
    const uint32_t step_t = kSmallStep ? 2 * kPart : step;
    const uint32_t live = static_cast<uint32_t>(min(all_tokens[0], static_cast<int64_t>(a.tokens)));
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll 1
    for (int pass = 0; pass < passes; ++pass) {
      const uint32_t from = pass == 0 ? first : threadIdx.x, by = pass == 0 ? step_t : kThreads;
      // A warp takes 32 * kRun tokens in a row: their first and last sequence, then each token's between those.
      for (uint32_t base = (from - lane) * kRun; base < live; base += by * kRun) {
        int32_t b_first, b_last;
        if constexpr (kRun > 1) {
          // one search by each half of the warp
          const int32_t found = owner(tokens, a.B, ~0u, lane < 16 ? base : min(base + 32 * kRun, live) - 1);
          b_first = __shfl_sync(0xffffffffu, found, 0);
          b_last = __shfl_sync(0xffffffffu, found, 31);
        } else {
          b_first = 0;
          b_last = a.B - 1;
        }
        int32_t b[kRun], end[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          b[i] = b_first;
          end[i] = b_last + 1;
        }
        for (int32_t n = b_last - b_first; n > 0; n >>= 1) {  // owner(tokens, ..) of each, side by side
#pragma unroll
          for (int i = 0; i < kRun; ++i) {
            const int32_t mid = (b[i] + end[i]) >> 1;
            if (end[i] - b[i] > 1) {
              if (tokens[mid] <= base + 32 * i + lane) b[i] = mid;
              else end[i] = mid;
            }
          }
        }
        int32_t pos[kRun], id[kRun];  // a negative position: not of this pass
        uint32_t in_page[kRun];
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          const uint32_t t = base + 32 * i + lane;
          pos[i] = -1;
          id[i] = -1;
          in_page[i] = 0;
          if (t >= live) continue;
          const uint32_t len = lens[b[i]], own = taken[b[i]], held = pages_of(a, len);
          const int32_t at_t = cut(static_cast<int64_t>(len) + (t - tokens[b[i]]));
          const uint32_t p = page_of(a, at_t), nth = own + (p - held);  // of the pages taken, if p is one
          const bool granted = (own & kRefused) == 0u, late = granted && p >= held && nth < apart;
          if (late != (pass == 1)) continue;
          pos[i] = at_t;
          if (!granted) continue;
          in_page[i] = at_t - p * a.page_size;
          id[i] = __ldcg(p < held ? a.table + b[i] * a.table_stride + p : place(nth));
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i) {
          const uint32_t t = base + 32 * i + lane;
          if (pos[i] < 0) continue;
          a.slots[t] = id[i] >= 0 ? static_cast<int64_t>(id[i]) * a.page_size + in_page[i] : -1;
          a.positions[t] = pos[i];
        }
      }
    }
    for (uint32_t t = live + first; t < static_cast<uint32_t>(a.tokens); t += step_t) {
      a.slots[t] = -1;
      a.positions[t] = 0;
    }
  }
  if (!kSmallStep || warps_of == 2) {
    const uint32_t first_p = kSmallStep ? threadIdx.x - 2 * kPart : first, step_p = kSmallStep ? kPart : step;
    auto take = [&](int64_t j) {
      const int32_t b = owner(taken, a.B, ~kRefused, static_cast<uint32_t>(j));
      const int64_t held = pages_of(a, lens[b]);
      a.table[b * a.table_stride + held + (j - (taken[b] & ~kRefused))] = __ldcg(place(j));
    };
    for (int64_t j = static_cast<int64_t>(apart) + first_p; j < last; j += step_p) take(j);
    if (passes == 2)
      for (int64_t j = threadIdx.x; j < apart; j += kThreads) take(j);
  }
  if (!kSmallStep || warps_of == 3) {
    const uint32_t first_p = kSmallStep ? threadIdx.x - 3 * kPart : first, step_p = kSmallStep ? kPart : step;
    constexpr int kAtOnce = 4;
    for (int64_t j0 = first_p; j0 < returned - refilled; j0 += kAtOnce * static_cast<int64_t>(step_p)) {
      int32_t id[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t j = j0 + i * static_cast<int64_t>(step_p);
        if (j >= returned - refilled) continue;
        const int32_t b = owner(given, a.B, ~0u, static_cast<uint32_t>(j));
        id[i] = __ldcg(a.table + b * a.table_stride + (j - given[b]));
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t j = j0 + i * static_cast<int64_t>(step_p);
        if (j < returned - refilled) *place(free_count + j) = id[i];
      }
    }
  }
  __syncthreads();
  if (refilled > 0 && rank == 0u)  // all that lay there has been read, by this CTA
    for (int64_t j = room + threadIdx.x; j < returned; j += kThreads) {
      const int32_t b = owner(given, a.B, ~0u, static_cast<uint32_t>(j));
      *place(j - room) = __ldcg(a.table + b * a.table_stride + (j - given[b]));
    }
  // In place: every CTA has read the lengths and the pool.
  if (a.in_place != 0 && ctas > 1) cluster_barrier();
  for (int32_t b = first; b <= a.B; b += step) {
    a.starts[b] = static_cast<int32_t>(tokens[b]);
    if (b == a.B) break;
    // Tokens granted fit the step, so their sums are whole.
    a.lens_out[b] = static_cast<int32_t>(lens[b] + ((taken[b] & kRefused) == 0u ? tokens[b + 1] - tokens[b] : 0u));
  }
  if (first == 0) {
    a.pool_out[0] = static_cast<int32_t>(place(last) - a.ring);
    a.pool_out[1] = static_cast<int32_t>(free_count - last + returned);
    a.pool_out[2] = cut(all_taken - last);
  }
}

template <int kThreads, int kRun, bool kSmallStep>
bool launch(const ExtendArgs& a, int64_t ctas, cudaStream_t s) {
  auto kern = extend_kernel<kThreads, kRun, kSmallStep>;
  const size_t smem = 4 * (static_cast<size_t>(a.B) + 1) * sizeof(uint32_t);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), kThreads, smem, a.in_place != 0 ? static_cast<unsigned>(ctas) : 1, s, a);
  return true;
}

}  // namespace

bool launch_extend(const ExtendArgs& given, cudaStream_t s) {
  ExtendArgs a = given;
  int lg = 0;
  while ((1LL << lg) < a.page_size) ++lg;
  a.page_magic_shift = 31 + lg;
  a.page_magic = static_cast<uint32_t>(((1ull << a.page_magic_shift) + a.page_size - 1) / a.page_size);
  a.in_place = a.lens_out == a.lens || a.pool_out == a.pool;
  if (a.tokens <= kSmall && a.B <= kSmall) return launch<2 * kSmall, 1, true>(a, 1, s);
  // A CTA for each 1024 tokens, up to one for each SM or, where lengths or pool are written over, up to a cluster; their
  // threads take several tokens at a time where there are more. 65536 tokens: 8.0 us, in place 15.
  const int64_t want = (static_cast<int64_t>(a.tokens) + 1023) / 1024, most = a.in_place != 0 ? kMaxCluster : sm_count();
  int64_t ctas = 1;
  if (a.in_place != 0)
    while (ctas < most && ctas < want) ctas *= 2;
  else
    ctas = want < 1 ? 1 : want < most ? want : most;
  return want > ctas ? launch<1024, 8, false>(a, ctas, s) : launch<1024, 1, false>(a, ctas, s);
}

}  // namespace fq
