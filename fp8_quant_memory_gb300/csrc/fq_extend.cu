// fq_extend.cu -- block tables and slot maps of one step from the requests' lengths.
//
// All of it follows from three running sums over the sequences: tokens added, pages needed (of the sequences that fit),
// pages returned. A sequence is granted its pages if the sum up to and with its own is at most the free pages: so those
// granted any are the first ones that need some, the pages taken are the first of the ring, and the j-th of them belongs
// to the sequence whose sums enclose j. Tokens and returned pages find their sequence the same way.
//
// What bounds it: one launch and two dependent rounds of loads (lengths; table and ring entries), not bytes: a step of 64
// tokens moves 3.6 KB, one of 65536 1 MB. They take 3.8 and 9.3 us. Every CTA sums all lengths itself (a few per thread), then
// takes its share of the tokens and pages, so that none waits for another. Returned pages are a
// cluster's: absent ones are left out, so that each one's place depends on those before it; and in a ring smaller than the pages
// they go to places which this step's pages leave, with all that is to be read there first. (Spread over all CTAs as they
// stand, absent ones too, they took 1.3 us less of the 9.3, and 18 more of 19 where 170 thousand return in a step of 4096
// tokens; a single CTA took 13 more.) Where lengths or pool are updated in place, that cluster is the only one and writes them
// behind its barrier, after every CTA has read them.
#include "fq_serving.h"
#include "fq_sync.cuh"
#include "fq_tcgen05.cuh"

namespace fq {
namespace {

constexpr int kTeam = 8;                     // CTAs that share the returned pages, one cluster
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

// owner() of base + 32 * i + lane, i < kN, below `limit`, for a warp, side by side; kBetween: between the owners of the first
// and the last, which half of the warp looks for each.
template <bool kBetween, int kN>
__device__ __forceinline__ void owners(const uint32_t* first, int32_t n, uint32_t base, uint32_t limit, int32_t (&b)[kN]) {
  const uint32_t lane = threadIdx.x & 31;
  int32_t b_first = 0, b_last = n - 1, end[kN];
  if constexpr (kBetween) {
    const int32_t found = owner(first, n, ~0u, lane < 16 ? base : min(base + 32 * kN, limit) - 1);
    b_first = __shfl_sync(0xffffffffu, found, 0);
    b_last = __shfl_sync(0xffffffffu, found, 31);
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    b[i] = b_first;
    end[i] = b_last + 1;
  }
  for (int32_t m = b_last - b_first; m > 0; m >>= 1) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int32_t mid = (b[i] + end[i]) >> 1;
      if (end[i] - b[i] > 1) {
        if (first[mid] <= base + 32 * i + lane) b[i] = mid;
        else end[i] = mid;
      }
    }
  }
}

// Lengths, pool, table and ring are read through L2: other CTAs of this call write them, and no line of L1 is left with what
// they held before.

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
  __shared__ uint32_t present[kThreads / 32], present_in[kTeam];  // returned pages of each warp, each CTA of the team
  const uint32_t ctas = gridDim.x, rank = blockIdx.x, team = a.team;
  const int32_t per = (a.B + kThreads - 1) / kThreads, b0 = min(a.B, static_cast<int32_t>(threadIdx.x) * per), b1 = min(a.B, b0 + per);
  pdl_trigger();
  pdl_wait();
  if (team > 1 && rank < team) cluster_arrive();  // waited for before the first access to another CTA: it runs by then
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
  // Places for returned pages: those behind the last free page, then those that this step's pages leave, of which `refilled`
  // at most are written over. What is to be read there, tokens' pages among it, is left to the CTAs that do so, before they do.
  const int64_t room = F - free_count, refilled = min(max(all_given - room, static_cast<int64_t>(0)), last);
  const bool returns = rank < team, works = rank >= ctas - a.workers;  // the latter take tokens and pages
  const uint32_t apart = ctas > 1 ? static_cast<uint32_t>(refilled) : 0u;
  const int pass0 = works ? 0 : 1, passes = apart > 0u && returns ? 2 : 1;

  // This thread and how many there are for the tokens, the pages taken and those returned.
  constexpr uint32_t kPart = kThreads / 4;
  const uint32_t warps_of = kSmallStep ? threadIdx.x / kPart : 0u;
  const uint32_t first = threadIdx.x + kThreads * (rank - (ctas - a.workers)), step = kThreads * a.workers;
  const uint32_t first_back = threadIdx.x + kThreads * rank, step_back = kThreads * team;  // in the team
  if (!kSmallStep || warps_of < 2) {
    const uint32_t step_t = kSmallStep ? 2 * kPart : step;
    const uint32_t live = static_cast<uint32_t>(min(all_tokens[0], static_cast<int64_t>(a.tokens)));
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll 1
    for (int pass = pass0; pass < passes; ++pass) {
      const uint32_t from = pass == 0 ? first : first_back, by = pass == 0 ? step_t : step_back;
      // A warp takes 32 * kRun tokens in a row.
      for (uint32_t base = (from - lane) * kRun; base < live; base += by * kRun) {
        int32_t b[kRun];
        owners<(kRun > 1)>(tokens, a.B, base, live, b);
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
    for (uint32_t t = live + first; works && t < static_cast<uint32_t>(a.tokens); t += step_t) {
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
    for (int64_t j = static_cast<int64_t>(apart) + first_p; works && j < last; j += step_p) take(j);
    if (passes == 2)
      for (int64_t j = first_back; j < apart; j += step_back) take(j);
  }
  // The pages of sequences that end, but for absent ones: each warp of the team counts those of its run, then writes them
  // behind the others'.
  int64_t kept = 0;
  if (kSmallStep && refilled > 0) __syncthreads();  // all that lay there has been read
  if (kSmallStep ? warps_of == 3 : returns && all_given > 0) {
    constexpr int kOwn = kSmallStep ? 4 : 8, kWarps = kSmallStep ? kPart / 32 : kThreads / 32;
    const int64_t most = room + last;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x / 32 & (kWarps - 1), warps = kWarps * team;
    const uint32_t limit = static_cast<uint32_t>(cut(all_given)), run = (limit / warps + 32) & ~31u;
    const uint32_t from = min(limit, run * (kWarps * rank + warp)), to = min(limit, from + run);
    int32_t id[kOwn];
    auto load = [&](uint32_t at) {
      int32_t b[kOwn];
      if constexpr (kSmallStep) {
        owners<false>(given, a.B, at, to, b);
      } else {
        // First and last sequence of each 32, which are often one, then each page's between those. (All side by side between
        // the run's first and last: 0.7 us more for 25 thousand pages, by its instructions.)
        const int32_t found = owner(given, a.B, ~0u, min(at + 32 * (lane / 2 & (kOwn - 1)) + 31 * (lane & 1), to - 1));
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          b[i] = __shfl_sync(0xffffffffu, found, 2 * i);
          int32_t end = __shfl_sync(0xffffffffu, found, 2 * i + 1) + 1;
          for (int32_t n = end - b[i] - 1; n > 0; n >>= 1) {
            const int32_t mid = (b[i] + end) >> 1;
            if (end - b[i] > 1) {
              if (given[mid] <= at + 32 * i + lane) b[i] = mid;
              else end = mid;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const uint32_t j = at + 32 * i + lane;
        id[i] = -1;
        if (j < to) id[i] = __ldcg(a.table + b[i] * a.table_stride + (j - given[b[i]]));
      }
    };
    uint32_t count = 0;
    for (uint32_t at = from; at < to; at += 32 * kOwn) {
      load(at);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) count += __popc(__ballot_sync(0xffffffffu, id[i] >= 0));
    }
    if (lane == 0) present[warp] = count;
    __syncwarp();
    if constexpr (kSmallStep) asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
    else __syncthreads();
    const uint32_t its = lane < kWarps ? present[lane] : 0u;
    uint32_t spot = __reduce_add_sync(0xffffffffu, lane < warp ? its : 0u), total = __reduce_add_sync(0xffffffffu, its);
    if (!kSmallStep && team > 1) {
      cluster_wait();
      if (warp == 0 && lane < team)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(&present_in[rank], lane)), "r"(total) : "memory");
      __syncwarp();
      cluster_barrier();  // in place, too: every CTA has read the lengths and the pool
      const uint32_t of = lane < team ? present_in[lane] : 0u;
      spot += __reduce_add_sync(0xffffffffu, lane < rank ? of : 0u);
      total = __reduce_add_sync(0xffffffffu, of);
    }
    kept = min(static_cast<int64_t>(total), most);
    for (uint32_t at = from; at < to && spot < kept; at += 32 * kOwn) {
      if (run > 32 * kOwn) load(at);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const uint32_t mask = __ballot_sync(0xffffffffu, id[i] >= 0);
        const int64_t k = spot + __popc(mask & ((1u << lane) - 1u));
        if (id[i] >= 0 && k < kept) *place(k < room ? free_count + k : k - room) = id[i];
        spot += __popc(mask);
      }
    }
  } else if (!kSmallStep && team > 1 && returns) {
    __syncwarp();  // whole warps, which the loops above have split
    cluster_wait();
    if (a.in_place != 0) cluster_barrier();
  }
  __syncthreads();
  for (int32_t b = threadIdx.x + kThreads * rank; b <= a.B; b += kThreads * ctas) {
    a.starts[b] = static_cast<int32_t>(tokens[b]);
    if (b == a.B) break;
    // Tokens granted fit the step, so their sums are whole.
    a.lens_out[b] = static_cast<int32_t>(lens[b] + ((taken[b] & kRefused) == 0u ? tokens[b + 1] - tokens[b] : 0u));
  }
  if (rank == 0 && threadIdx.x == (kSmallStep ? 3 * kPart : 0u)) {
    a.pool_out[0] = static_cast<int32_t>(place(last) - a.ring);
    a.pool_out[1] = static_cast<int32_t>(free_count - last + kept);
    a.pool_out[2] = cut(all_taken - last);
  }
}

template <int kThreads, int kRun, bool kSmallStep>
bool launch(const ExtendArgs& a, int64_t ctas, cudaStream_t s) {
  auto kern = extend_kernel<kThreads, kRun, kSmallStep>;
  const size_t smem = 4 * (static_cast<size_t>(a.B) + 1) * sizeof(uint32_t);
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), kThreads, smem, static_cast<unsigned>(a.team), s, a);
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
  a.team = a.workers = 1;
  if (a.tokens <= kSmall && a.B <= kSmall) return launch<2 * kSmall, 1, true>(a, 1, s);
  // A CTA for each 1024 tokens, in clusters, up to one for each SM behind that of the returned pages, or, where lengths or pool
  // are written over, that cluster alone; their threads take several tokens at a time where there are more. 65536 tokens:
  // 9.3 us, in place 16.
  const int64_t want = (static_cast<int64_t>(a.tokens) + 1023) / 1024;
  if (a.in_place != 0) {
    while (a.team < kTeam && a.team < want) a.team *= 2;
    a.workers = a.team;
  } else {
    a.team = kTeam;
    const int64_t most = sm_count() / kTeam * kTeam - kTeam, whole = (want + kTeam - 1) / kTeam * kTeam;
    a.workers = static_cast<int32_t>(whole < kTeam || most < kTeam ? kTeam : whole < most ? whole : most);
  }
  const int64_t ctas = a.in_place != 0 ? a.team : a.team + a.workers;
  return want > a.workers ? launch<1024, 8, false>(a, ctas, s) : launch<1024, 1, false>(a, ctas, s);
}

}  // namespace fq
