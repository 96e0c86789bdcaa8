// fq_matmul.cuh -- the block-scaled FP8 matrix product on the 5th-generation tensor cores.
//
// Mathematics: out[i, j] = sum over blocks g of 128 k of sa[i, g] sb[j/128, g] P_g[i, j], P_g = sum of a[i, k]
// b[j, k] over the block. A block is one 128-byte swizzled row of a tile, four tcgen05.mma of 32 k; its product
// P_g is complete in tensor memory, so the epilogue warps read it once per block and add it, scaled, to fp32
// accumulators in registers: one FMA per output and block, against 128 products on the tensor cores.
//
// What bounds it. Per SM and clock the tensor cores take 8192 e4m3 products; a 128 x 256 block of 128 k is 512
// clocks. The epilogue of the same block is 128 clocks of FMA pairs and 128 of tensor-memory reads per warp, two
// warps per scheduler, under the products of the next block (two accumulator buffers). With few rows the weights'
// bytes bound it: HBM.
//
// Two kernels:
//   wide   (many rows): CTA pairs, tiles of 256 x 256 outputs, rows of `a` on the tensor-memory lanes, so a
//          thread owns an output row and its scale of `a` is one register; persistent, outputs staged in shared
//          memory and stored by TMA.
//   narrow (few rows): weight rows on the lanes, NT rows of `a` as columns, so that the weights stream through
//          the large operand whatever the number of rows; the k range is split over the CTAs of a cluster, which
//          add their partial sums through distributed shared memory in rank order (no workspace, no atomics, the
//          same bits every time).
//
// Waits are bounded (fq_sync.cuh): a role that gives up flags the device status word and leaves its loop, the
// others follow when their own waits run out, and tensor memory is freed either way.
#pragma once

#include <type_traits>

#include "fq_device.cuh"
#include "fq_epilogue.cuh"
#include "fq_serving.h"
#include "fq_tcgen05.cuh"
#include "fq_tensormap.h"

namespace fq {
namespace {

constexpr int kBK = 128;  // k per stage: one scale block, one swizzled row

struct MmArgs {
  const float* sa;
  const float* sb;
  int64_t sa_stride, sb_stride;
  void* out;
  int64_t out_stride;
  unsigned int* status;
  int32_t M, N, nkb;
  int32_t tiles_m, tiles_n;
  int32_t dtype;
  // wide: whole tiles, column ranges that each of the others is cut into, pieces of work in all; whether out has
  // a tensor map
  int32_t whole, parts, pieces, tma_store;
  // fused epilogue (kernels with kFused): out = dtype(activation(product + bias) + residual)
  const void* bias;      // nullable
  const void* residual;  // nullable
  int64_t residual_stride;
  int32_t activation;
  int32_t bias_vec, residual_vec;  // wide: may be read 16 bytes at a time
};

__device__ __forceinline__ uint32_t pack_out(int dtype, float2 v) {
  return dtype == DT_BF16 ? Elem<__nv_bfloat16>::pack(v) : Elem<__half>::pack(v);
}

__device__ __forceinline__ void store_out(int dtype, void* out, int64_t i, float v) {
  if (dtype == DT_BF16) Elem<__nv_bfloat16>::store1(out, i, v);
  else Elem<__half>::store1(out, i, v);
}

__device__ __forceinline__ float load_in(int dtype, const void* p, int64_t i) {
  return dtype == DT_BF16 ? Elem<__nv_bfloat16>::load1(p, i) : Elem<__half>::load1(p, i);
}

__device__ __forceinline__ float2 unpack_in(int dtype, uint32_t v) {
  return dtype == DT_BF16 ? Elem<__nv_bfloat16>::unpack(v) : Elem<__half>::unpack(v);
}

inline MmArgs device_args(const MatmulArgs& a, int dtype) {
  MmArgs p{};
  p.sa = a.a_scale;
  p.sb = a.b_scale;
  p.sa_stride = a.a_scale_stride;
  p.sb_stride = a.b_scale_stride;
  p.out = a.out;
  p.out_stride = a.out_stride;
  p.status = device_status_ptr();
  p.M = static_cast<int32_t>(a.M);
  p.N = static_cast<int32_t>(a.N);
  p.nkb = static_cast<int32_t>(a.groups);
  p.dtype = dtype;
  p.bias = a.bias;
  p.residual = a.residual;
  p.residual_stride = a.residual_stride;
  p.activation = a.activation;
  p.bias_vec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
  p.residual_vec = reinterpret_cast<uintptr_t>(a.residual) % 16 == 0 && (a.M == 1 || a.residual_stride % 8 == 0);
  return p;
}

// A single row's stride is never used, but has to be a valid one for a tensor map.
inline MatmulArgs valid_strides(MatmulArgs a) {
  if (a.M == 1) a.a_stride = (a.K + 15) / 16 * 16;
  if (a.N == 1) a.b_stride = (a.K + 15) / 16 * 16;
  return a;
}

// ================================================================================= narrow
// Epilogue warps in G groups of four, then the producer's and the products' warp. A block costs an epilogue warp a
// chain of latencies (barrier, tensor memory, scales) with nothing else on its scheduler. Two groups take the blocks in
// turn and add their sums at the end, 0.3 us. Measured at 64 columns: 64 x 8192 x 4096 (16 blocks a CTA) takes 11.3 us
// with two and 11.6 with one, 64 x 8192 x 8320 (33) 17.9 and 21.3, but 333 x 1111 x 1968 (8) 7.7 and 7.4. Fewer columns
// gain nothing (24 x 6144 x 8192: 15.1 and 15.2) and 128 leave no registers for it.
constexpr int kTwoGroupBlocks = 12;  // blocks of k per CTA

template <int G>
constexpr int kNarrowThreads = 32 * (4 * G + 2);

// One CTA per SM with as deep a ring as fits: a few CTAs then keep HBM busy (90 KB in flight on each of 48 SMs
// moved 2 TB/s), and no cluster larger than a pair is needed to occupy the GPU (clusters of 4 to 8 CTAs started
// in several rounds: 1 x 6144 x 4096 took 13.5 us split six ways and 8.4 us split in two).
constexpr int kMaxSplit = 4;

template <int NT>
struct Narrow {
  static constexpr int kStageBytes = (128 + NT) * kBK;
  static constexpr int kStages = NT == 16 ? 11 : NT == 32 ? 10 : NT == 64 ? 8 : 5;
  static constexpr int kBufs = 4;
  static constexpr uint32_t kCols = NT * kBufs;  // 64 to 512
};

template <int NT>
struct NarrowShared {
  alignas(1024) unsigned char ring[Narrow<NT>::kStages][Narrow<NT>::kStageBytes];  // weights, then rows of a
  float part[NT / 4 * 3][128];                                                    // partial sums from the cluster's others
  alignas(16) float scale[NT == 64 ? 8 : 4][2][NT];                               // per epilogue warp, two blocks
  alignas(8) uint64_t full[Narrow<NT>::kStages];
  uint64_t empty[Narrow<NT>::kStages];
  uint64_t done[Narrow<NT>::kBufs];   // a block's products are in tensor memory
  uint64_t free_[Narrow<NT>::kBufs];  // and have been read
  uint32_t tmem;
};

// Residuals of rows col0 .. col0 + N - 1 of column `row`, two in a word. Through L2, as in the wide kernel: they may be the
// output, whose old values no line of L1 should hold when the next kernel starts beside this one.
template <int N>
__device__ __forceinline__ void narrow_residual(const MmArgs& p, int col0, int row, uint32_t (&r)[N / 2]) {
  const uint16_t* from = static_cast<const uint16_t*>(p.residual) + static_cast<int64_t>(col0) * p.residual_stride + row;
  const int n = p.residual != nullptr && row < p.N ? p.M - col0 : 0;
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    uint32_t lo = 0, hi = 0;
    if (j < n) lo = __ldcg(from);
    from += p.residual_stride;
    if (j + 1 < n) hi = __ldcg(from);
    from += p.residual_stride;
    r[j / 2] = lo | (hi << 16);
  }
}

// The fused epilogue and the stores of N outputs of column `row`, whose sums and residuals the thread itself has put into
// `sums` and `words`, and the cluster's others into `part`: added in rank order, `mine` being this CTA's. A loop over
// shared memory and not over registers: unrolled, as registers want it, it was 30 KB of instructions that every launch
// fetches anew (333 x 1111 x 1968: 13.0 us with gelu, 11.3 with a bias alone, 7.5 without).
template <int N, int SPLIT>
__device__ __forceinline__ void narrow_finish(const MmArgs& p, int col0, int row, int t, const float (*sums)[128],
                                              const float (*part)[128], int mine, const uint32_t (*words)[128]) {
  const bool in_row = row < p.N;
  const float bias = p.bias != nullptr && in_row ? load_in(p.dtype, p.bias, row) : -0.f;  // y + -0 is y
  int64_t at = static_cast<int64_t>(col0) * p.out_stride + row;
  constexpr int kGroup = N < 8 ? N : 8;
#pragma unroll 1
  for (int j = 0; j < N && col0 + j < p.M; j += kGroup) {
    float2 v[kGroup / 2];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      float x = 0.f;
#pragma unroll
      for (int q = 0; q < SPLIT; ++q) x += q == mine ? sums[j + i][t] : part[N * (q < mine ? q : q - 1) + j + i][t];
      const float y = __fadd_rn(SPLIT == 1 ? sums[j + i][t] : x, bias);
      if (i & 1) v[i / 2].y = y;
      else v[i / 2].x = y;
    }
    activate_each(p.activation, v);
    if (p.residual != nullptr) {
#pragma unroll
      for (int i = 0; i < kGroup / 2; ++i) v[i] = add2(v[i], unpack_in(p.dtype, words[j / 2 + i][t]));
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i, at += p.out_stride)
      if (in_row && col0 + j + i < p.M) store_out(p.dtype, p.out, at, i & 1 ? v[i / 2].y : v[i / 2].x);
  }
}

template <int NT, int SPLIT, int G, bool kFused>
__global__ void __launch_bounds__(kNarrowThreads<G>, 1)
    matmul_narrow_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap,
                         const __grid_constant__ MmArgs p) {
  using C = Narrow<NT>;
  constexpr int kProducer = 4 * G, kProducts = kProducer + 1;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // The swizzle repeats every 1024 bytes: align the ring to 1024.
  NarrowShared<NT>& sm = *reinterpret_cast<NarrowShared<NT>*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x;  // the cluster is the whole x axis
  const int n0 = blockIdx.y * 128, t0 = blockIdx.z * NT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.nkb) * rank / SPLIT);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.nkb) * (rank + 1) / SPLIT);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&sm.done[b], 1);
      mbar_init(&sm.free_[b], 4);
    }
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&amap)) : "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (warp == kProducts) tmem_alloc<1>(&sm.tmem, C::kCols);
  tc_fence_before();
  __syncthreads();
  if (SPLIT > 1) cluster_arrive();  // waited for before the first access to another CTA: it runs by then
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp == kProducer) {
    // ------------------------------------------------------------------------ producer
    if (lane == 0) {
      int s = 0;
      uint32_t phase = 1;
      int k = kb0;
      for (; k < kb1; ++k) {
        if (k - kb0 >= C::kStages && !mbar_wait(kWaitLimitNs, &sm.empty[s], phase)) break;
        mbar_arrive_expect_tx(&sm.full[s], C::kStageBytes);
        tma_load_2d(sm.ring[s], &wmap, k * kBK, n0, &sm.full[s]);
        tma_load_2d(sm.ring[s] + 128 * kBK, &amap, k * kBK, t0, &sm.full[s]);
        if (++s == C::kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (k < kb1) {
        flag_failure(p.status);
        // Let the copies already issued land before this CTA's shared memory goes away.
        for (int j = max(0, k - kb0 - C::kStages); j < k - kb0; ++j)
          if (!mbar_wait(kWaitLimitNs, &sm.full[j % C::kStages], static_cast<uint32_t>(j / C::kStages) & 1u)) break;
      }
    }
  } else if (warp == kProducts) {
    // ------------------------------------------------------------------------ products
    if (lane == 0) {
      constexpr uint32_t idesc = e4m3_idesc(128, NT);
      int s = 0, b = 0;
      uint32_t phase = 0, bphase = 1;
      bool ok = true;
      for (int k = kb0; k < kb1 && ok; ++k) {
        ok = (k - kb0 < C::kBufs || mbar_wait(kWaitLimitNs, &sm.free_[b], bphase)) &&
             mbar_wait(kWaitLimitNs, &sm.full[s], phase);
        if (!ok) {
          flag_failure(p.status);
          break;
        }
        tc_fence_after();
        const uint64_t wd = tile_desc(smem_addr(sm.ring[s])), ad = tile_desc(smem_addr(sm.ring[s] + 128 * kBK));
#pragma unroll
        for (int i = 0; i < kBK / 32; ++i) mma_e4m3_tile<1>(tmem + b * NT, wd + 2 * i, ad + 2 * i, idesc, i > 0);
        mma_commit<1>(&sm.empty[s]);
        mma_commit<1>(&sm.done[b]);
        if (++s == C::kStages) {
          s = 0;
          phase ^= 1u;
        }
        if (++b == C::kBufs) {
          b = 0;
          bphase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------------ epilogue
    // Thread (quarter, lane) of a group owns weight row n0 + 32*quarter + lane; acc[j] is row t0 + j of a.
    const int quarter = warp & 3, group = warp >> 2;
    float2 acc[NT / 2];
#pragma unroll
    for (int j = 0; j < NT / 2; ++j) acc[j] = make_float2(0.f, 0.f);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float* sb = p.sb + static_cast<int64_t>(blockIdx.y) * p.sb_stride;
    constexpr int kL = (NT + 31) / 32;  // scales of a that a lane brings per block
    float next[kL];
    auto fetch = [&](int k) {
      const float b = sb[k];
#pragma unroll
      for (int i = 0; i < kL; ++i) {
        const int j = lane + 32 * i;
        next[i] = j < NT && t0 + j < p.M ? p.sa[static_cast<int64_t>(t0 + j) * p.sa_stride + k] * b : 0.f;
      }
    };
    // The residuals of the outputs that this thread will finish are on their way during the products, as far as there
    // are registers for it.
    constexpr int kOwn = NT / SPLIT;
    constexpr bool kEarly = kFused && kOwn <= 64;
    uint32_t residual[kFused ? kOwn / 2 : 1];
    if constexpr (kEarly)
      if (group == 0) narrow_residual<kOwn>(p, t0 + kOwn * rank, n0 + 32 * quarter + lane, residual);
    const int first = kb0 + group;
    if (first < kb1) fetch(first);
    int b = group, turn = 0;
    uint32_t phase = 0;
    for (int k = first; k < kb1; k += G, turn ^= 1) {
      float* sc = sm.scale[warp][turn];
#pragma unroll
      for (int i = 0; i < kL; ++i)
        if (lane + 32 * i < NT) sc[lane + 32 * i] = next[i];
      __syncwarp();  // the other buffer's readers have passed the last block's barrier
      if (k + G < kb1) fetch(k + G);
      // one verdict for the whole warp: the loads below are collective
      if (!__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &sm.done[b], phase))) {
        flag_failure(p.status);
        break;
      }
      tc_fence_after();
      uint32_t d[NT < 32 ? 16 : 32];
#pragma unroll
      for (int c = 0; c < (NT + 31) / 32; ++c) {
        if constexpr (NT < 32) tmem_ld16(lanes + b * NT, d);
        else tmem_ld32(lanes + b * NT + 32 * c, d);
        tmem_wait_ld();
        if (c == (NT + 31) / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.free_[b]);
        }
#pragma unroll
        for (int j = 0; j < (NT < 32 ? 16 : 32); j += 4) {
          const float4 s4 = *reinterpret_cast<const float4*>(sc + 32 * c + j);
          float2& lo = acc[16 * c + j / 2];
          float2& hi = acc[16 * c + j / 2 + 1];
          lo = fma2(make_float2(__uint_as_float(d[j]), __uint_as_float(d[j + 1])), make_float2(s4.x, s4.y), lo);
          hi = fma2(make_float2(__uint_as_float(d[j + 2]), __uint_as_float(d[j + 3])), make_float2(s4.z, s4.w), hi);
        }
      }
      b += G;
      if (b >= C::kBufs) {
        b = group;
        phase ^= 1u;
      }
    }
    if constexpr (G == 2) {
      // Once both groups have seen their last block, nothing uses the ring: the second group's sums pass through it.
      float (*sums)[128] = reinterpret_cast<float (*)[128]>(sm.ring);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (group == 1) {
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          sums[2 * j][32 * quarter + lane] = acc[j].x;
          sums[2 * j + 1][32 * quarter + lane] = acc[j].y;
        }
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          acc[j].x += sums[2 * j][32 * quarter + lane];
          acc[j].y += sums[2 * j + 1][32 * quarter + lane];
        }
      }
    }
    if (group == 0) {
      // Each CTA of the cluster finishes NT / SPLIT of the columns: the others push their partial sums of these into
      // its shared memory, and it adds them in rank order.
      const int row = 32 * quarter + lane;
      auto value = [&](int j) { return j & 1 ? acc[j / 2].y : acc[j / 2].x; };
      if constexpr (kFused) {
        // Nothing uses the ring any more: this thread's own outputs and residuals lie there, in its own column.
        if constexpr (!kEarly) narrow_residual<kOwn>(p, t0 + kOwn * rank, n0 + row, residual);
        float (*sums)[128] = reinterpret_cast<float (*)[128]>(sm.ring);
        uint32_t (*words)[128] = reinterpret_cast<uint32_t (*)[128]>(sums + kOwn);
#pragma unroll
        for (int r = 0; r < SPLIT; ++r)
          if (r == rank) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) sums[j][row] = value(kOwn * r + j);
          }
#pragma unroll
        for (int j = 0; j < kOwn / 2; ++j) words[j][row] = residual[j];
      }
      if constexpr (SPLIT == 1 && kFused) {
        narrow_finish<NT, 1>(p, t0, n0 + row, row, reinterpret_cast<float (*)[128]>(sm.ring), sm.part, 0,
                             reinterpret_cast<uint32_t (*)[128]>(sm.ring) + NT);
      } else if constexpr (SPLIT == 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (t0 + j < p.M && n0 + row < p.N) store_out(p.dtype, p.out, static_cast<int64_t>(t0 + j) * p.out_stride + n0 + row, value(j));
      } else {
        cluster_wait();
#pragma unroll
        for (int r = 0; r < SPLIT; ++r)
          if (r != rank) {
            // the part of rank q lies at (q < r ? q : q - 1) of rank r's
            const uint32_t to = in_cta(&sm.part[kOwn * (rank < r ? rank : rank - 1)][row], r);
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + j * 512), "f"(value(kOwn * r + j)) : "memory");
          }
        cluster_barrier();
        if constexpr (kFused) {
          narrow_finish<kOwn, SPLIT>(p, t0 + kOwn * rank, n0 + row, row, reinterpret_cast<float (*)[128]>(sm.ring), sm.part, rank,
                                     reinterpret_cast<uint32_t (*)[128]>(sm.ring) + kOwn);
        } else {
#pragma unroll
          for (int r = 0; r < SPLIT; ++r)
            if (r == rank) {
#pragma unroll
              for (int j = 0; j < kOwn; ++j) {
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < SPLIT; ++q) v += q == r ? value(kOwn * r + j) : sm.part[kOwn * (q < r ? q : q - 1) + j][row];
                const int col = t0 + kOwn * r + j;
                if (col < p.M && n0 + row < p.N) store_out(p.dtype, p.out, static_cast<int64_t>(col) * p.out_stride + n0 + row, v);
              }
            }
        }
      }
    }
  }
  if (SPLIT > 1 && warp >= 4) {
    __syncwarp();
    cluster_wait();
    cluster_barrier();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProducts) tmem_free<1>(tmem, C::kCols);
}

template <int NT, bool kFused>
bool launch_narrow(const MatmulArgs& a, MmArgs p, const MatmulPlan& plan, cudaStream_t s) {
  CUtensorMap wmap, amap;
  const uint64_t wd[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.N)}, ws[1] = {static_cast<uint64_t>(a.b_stride)};
  const uint64_t ad[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.M)}, as[1] = {static_cast<uint64_t>(a.a_stride)};
  const uint32_t wb[2] = {kBK, 128}, ab[2] = {kBK, NT};
  if (!byte_tensor_map(&wmap, 2, a.b, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !byte_tensor_map(&amap, 2, a.a, ad, as, ab, CU_TENSOR_MAP_SWIZZLE_128B))
    return false;
  p.tiles_n = static_cast<int32_t>((a.N + 127) / 128);
  p.tiles_m = static_cast<int32_t>((a.M + NT - 1) / NT);
  const int split = plan.split;
  auto kern = split == 1   ? matmul_narrow_kernel<NT, 1, 1, kFused>
              : split == 2 ? matmul_narrow_kernel<NT, 2, 1, kFused>
                           : matmul_narrow_kernel<NT, 4, 1, kFused>;
  int threads = kNarrowThreads<1>;
  if constexpr (NT == 64) {
    if (plan.groups == 2) {
      kern = split == 1   ? matmul_narrow_kernel<NT, 1, 2, kFused>
             : split == 2 ? matmul_narrow_kernel<NT, 2, 2, kFused>
                          : matmul_narrow_kernel<NT, 4, 2, kFused>;
      threads = kNarrowThreads<2>;
    }
  }
  constexpr size_t smem = sizeof(NarrowShared<NT>) + 1024;
  static_assert(smem <= 227 * 1024, "the ring fits the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem)) return false;
  launch_overlapped(kern, dim3(static_cast<unsigned>(split), static_cast<unsigned>(p.tiles_n), static_cast<unsigned>(p.tiles_m)),
                    threads, smem, static_cast<unsigned>(split), s, wmap, amap, p);
  return true;
}

// =================================================================================== wide
// Warpgroup 0: producer (warp 0), products (warp 1), two idle warps; warpgroups 1 and 2: epilogue. The epilogue's
// registers come from warpgroup 0: 384 x 168 at launch = 128 x 72 + 256 x 216.
constexpr int kWideThreads = 384;
constexpr int kIdleRegs = 72, kEpiRegs = 216;
constexpr int kPlain = -1;  // no fused epilogue

constexpr int kTileM = 256, kTileN = 256;  // outputs of a CTA pair
constexpr int kWideStageBytes = 256 * kBK; // one CTA's half of the pair's operands
// With a fused epilogue a stage less, for staging rows of all a warp's columns: their residuals arrive there during the
// products (half of them loaded at the end took 12 us more: 4096 x 8192 x 4096 with bias and residual, 127 us).
template <bool kFused>
struct WideShared {
  static constexpr int kWideStages = kFused ? 5 : 6;
  alignas(1024) unsigned char ring[kWideStages][kWideStageBytes];  // 128 rows of a, then 128 weight rows
  alignas(1024) unsigned char out[8][kFused ? 2 : 1][32 * 128];    // per epilogue warp: 32 rows x 64 columns
  alignas(8) uint64_t full[kWideStages];  // leader: both CTAs' operands have landed
  uint64_t empty[kWideStages];            // both: the products have read them
  uint64_t done[2];                       // both: a block's products are in tensor memory
  uint64_t free_[2];                      // leader: all sixteen epilogue warps have read them
  uint32_t tmem;
};

// Columns n0.. of tile row m, `width` of them (256, 128 or 64).
struct Tile {
  int m, n0, width;
};

// The t-th piece of work: whole tiles, eight tile rows at a time so that CTA pairs that run together share operand
// rows in L2; then the tiles that do not fill a last round, cut into `parts` column ranges. (Narrow products take
// as long as wide ones per instruction, which is why only the last round is cut.)
__device__ __forceinline__ Tile tile_at(const MmArgs& p, int t) {
  constexpr int kRowsAtATime = 8;
  int sub = 0, width = kTileN;
  if (t >= p.whole) {
    const int extra = t - p.whole;
    t = p.whole + extra / p.parts;
    sub = extra - extra / p.parts * p.parts;
    width = kTileN / p.parts;
  }
  const int per = kRowsAtATime * p.tiles_n, group = t / per, in = t - group * per;
  const int rows = min(kRowsAtATime, p.tiles_m - group * kRowsAtATime);
  const int n = in / rows;
  return {group * kRowsAtATime + in - n * rows, n * kTileN + sub * width, width};
}

// A warp's part of a piece: 32 rows x 32*kChunks columns over every block of k; `b` and `phase` are the next
// accumulator buffer and its parity, a_next and b_next the first block's scales. False if a wait gave up.
template <int kChunks, typename Sm>
__device__ __forceinline__ bool wide_accumulate(const MmArgs& p, Sm& sm, const float* sa, const float* sb, float a_next,
                                                float b_next, uint32_t from, uint32_t free0, uint32_t free1, int& b,
                                                uint32_t& phase, float2 (&acc)[16 * kChunks]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16 * kChunks; ++j) acc[j] = make_float2(0.f, 0.f);
  for (int kb = 0; kb < p.nkb; ++kb) {
    const float2 s2 = splat2(a_next * b_next);
    if (kb + 1 < p.nkb) {
      a_next = ld_f32(sa + kb + 1);
      b_next = ld_f32(sb + kb + 1);
    }
    // one verdict for the whole warp: the loads below are collective
    if (!__all_sync(0xffffffffu, mbar_wait(kWaitLimitNs, &sm.done[b], phase))) return false;
    tc_fence_after();
    uint32_t d[2][16];
    tmem_ld16(from + 256 * b, d[0]);
#pragma unroll
    for (int c = 0; c < 2 * kChunks; ++c) {
      tmem_wait_ld();
      if (c + 1 < 2 * kChunks) {
        tmem_ld16(from + 256 * b + 16 * (c + 1), d[(c + 1) & 1]);
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(b == 0 ? free0 : free1);
      }
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        float2& x = acc[8 * c + j / 2];
        x = fma2(make_float2(__uint_as_float(d[c & 1][j]), __uint_as_float(d[c & 1][j + 1])), s2, x);
      }
    }
    b ^= 1;
    if (b == 0) phase ^= 1u;
  }
  return true;
}

// 64 columns of the warp's outputs out of its staging rows: by a TMA box, or row by row with neighbouring lanes on
// neighbouring columns where the output has no tensor map (rows that are not whole 16-byte pieces).
__device__ __forceinline__ void send_staged(const MmArgs& p, const CUtensorMap* omap, unsigned char* stage, int row0, int col) {
  const int lane = threadIdx.x & 31;
  if (p.tma_store) {
    fence_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (row0 < p.M && col < p.N) tma_store_2d(omap, col, row0, stage);
      bulk_commit();
    }
  } else {
    __syncwarp();
    const int rows = min(32, p.M - row0);
    uint16_t* out = static_cast<uint16_t*>(p.out) + static_cast<int64_t>(row0) * p.out_stride + col;
#pragma unroll 1
    for (int r = 0; r < rows; ++r, out += p.out_stride)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int x = lane + 32 * h;
        if (col + x < p.N) out[x] = *reinterpret_cast<const uint16_t*>(stage + r * 128 + (((x >> 3) ^ (r & 7)) << 4) + 2 * (x & 7));
      }
    __syncwarp();
  }
}

// The warp's outputs from (row0, col0), 64 columns at a time through staging rows of 128 bytes (16-byte pieces
// swizzled).
template <int kChunks>
__device__ __forceinline__ void wide_store(const MmArgs& p, const CUtensorMap* omap, unsigned char* stage, int row0, int col0,
                                           const float2 (&acc)[16 * kChunks]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < kChunks / 2; ++c) {
    if (lane == 0) bulk_wait_read();  // the last box has left the staging rows
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2* v = &acc[32 * c + 4 * e];
      *reinterpret_cast<uint4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) =
          make_uint4(pack_out(p.dtype, v[0]), pack_out(p.dtype, v[1]), pack_out(p.dtype, v[2]), pack_out(p.dtype, v[3]));
    }
    send_staged(p, omap, stage, row0, col0 + 64 * c);
  }
}

__device__ __forceinline__ const uint16_t* residual_at(const MmArgs& p, int row, int col) {
  return static_cast<const uint16_t*>(p.residual) + static_cast<int64_t>(row) * p.residual_stride + col;
}

// 64 columns from `col` of the warp's residual rows into staging rows, as wide_store lays them out.
__device__ __forceinline__ void copy_residual(const MmArgs& p, unsigned char* stage, int row0, int col) {
  const int lane = threadIdx.x & 31, rows = min(32, p.M - row0);
  if (p.residual_vec != 0 && col + 64 <= p.N) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3), e = lane & 7;
      if (r < rows)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(stage + r * 128 + ((e ^ (r & 7)) << 4))),
                     "l"(residual_at(p, row0 + r, col + 8 * e))
                     : "memory");
    }
    return;
  }
#pragma unroll 4
  for (int r = 0; r < rows; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = lane + 32 * h;
      if (col + x < p.N) *reinterpret_cast<uint16_t*>(stage + r * 128 + (((x >> 3) ^ (r & 7)) << 4) + 2 * (x & 7)) = __ldcg(residual_at(p, row0 + r, col + x));
    }
}

// What a piece's epilogue needs, on its way from the piece's start: the residuals, to the staging rows, and 4 columns'
// biases of each lane (-0 where there are none: y + -0 is y), these before the residuals, behind which they would be waited
// for (5 us of 4096 x 8192 x 4096).
template <int kChunks>
__device__ __forceinline__ uint2 wide_prepare(const MmArgs& p, unsigned char* stage, int row0, int col0) {
  const int lane = threadIdx.x & 31, col = col0 + 4 * lane;
  uint2 b = make_uint2(0x80008000u, 0x80008000u);
  if (p.bias != nullptr && lane < 8 * kChunks) {
    const uint16_t* from = static_cast<const uint16_t*>(p.bias) + col;
    if (p.bias_vec != 0 && col + 4 <= p.N) {
      b = *reinterpret_cast<const uint2*>(from);
    } else {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = col + i < p.N ? from[i] : 0x8000u;
      b = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
    }
  }
  if (p.residual != nullptr) {
    if (lane == 0) bulk_wait_read();  // the last boxes have left the staging rows
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kChunks / 2; ++c) copy_residual(p, stage + 4096 * c, row0, col0 + 64 * c);
  }
  return b;
}

// wide_store with the fused epilogue: residuals come through the staging rows, whose pieces each lane replaces by its
// outputs.
template <int kChunks, int kAct, typename T>
__device__ __forceinline__ void wide_store_fused(const MmArgs& p, const CUtensorMap* omap, unsigned char* stage, int row0, int col0,
                                                 uint2 bias, const float2 (&acc)[16 * kChunks]) {
  constexpr int kAtOnce = 4;  // pieces of 8 columns
  const int lane = threadIdx.x & 31;
  if (p.residual == nullptr) {
    if (lane == 0) bulk_wait_read();
  } else {
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kChunks / 2; ++c) {
#pragma unroll
    for (int e0 = 0; e0 < 8; e0 += kAtOnce) {
      uint4 res[kAtOnce];  // before the stores of these pieces, which the compiler cannot tell apart from them
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        res[i] = p.residual != nullptr ? *reinterpret_cast<const uint4*>(stage + 4096 * c + lane * 128 + (((e0 + i) ^ (lane & 7)) << 4))
                                       : make_uint4(0u, 0u, 0u, 0u);
      float2 y[4 * kAtOnce];
#pragma unroll
      for (int i = 0; i < 2 * kAtOnce; ++i) {
        const int owner = 16 * c + 2 * e0 + i;  // the lane with these four columns' biases
        y[2 * i] = add2(acc[32 * c + 4 * e0 + 2 * i], Elem<T>::unpack(__shfl_sync(0xffffffffu, bias.x, owner)));
        y[2 * i + 1] = add2(acc[32 * c + 4 * e0 + 2 * i + 1], Elem<T>::unpack(__shfl_sync(0xffffffffu, bias.y, owner)));
      }
      activate_pairs<kAct>(y);
      if (p.residual != nullptr) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          y[4 * i] = add2(y[4 * i], Elem<T>::unpack(res[i].x));
          y[4 * i + 1] = add2(y[4 * i + 1], Elem<T>::unpack(res[i].y));
          y[4 * i + 2] = add2(y[4 * i + 2], Elem<T>::unpack(res[i].z));
          y[4 * i + 3] = add2(y[4 * i + 3], Elem<T>::unpack(res[i].w));
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        *reinterpret_cast<uint4*>(stage + 4096 * c + lane * 128 + (((e0 + i) ^ (lane & 7)) << 4)) =
            make_uint4(Elem<T>::pack(y[4 * i]), Elem<T>::pack(y[4 * i + 1]), Elem<T>::pack(y[4 * i + 2]), Elem<T>::pack(y[4 * i + 3]));
    }
    send_staged(p, omap, stage + 4096 * c, row0, col0 + 64 * c);
  }
}

// kAct: the activation of the fused epilogue, or kPlain.
template <int kAct, typename T>
__global__ void __launch_bounds__(kWideThreads, 1)
    matmul_wide_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap omap, const __grid_constant__ MmArgs p) {
  constexpr bool kFused = kAct != kPlain;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // The swizzle repeats every 1024 bytes: align to 1024 (the same offset in both CTAs).
  using Sm = WideShared<kFused>;
  constexpr int kWideStages = Sm::kWideStages;
  Sm& sm = *reinterpret_cast<Sm*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pairs = gridDim.x / 2, first = blockIdx.x / 2;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kWideStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.done[b], 1);
      mbar_init(&sm.free_[b], 16);
    }
    fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&amap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&wmap)) : "memory");
  }
  pdl_trigger();
  pdl_wait();
  if (warp == 1) tmem_alloc<2>(&sm.tmem, 512);
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIdleRegs));
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------------- producer
      int s = 0;
      uint32_t phase = 1;
      int64_t k = 0;  // stages issued
      bool ok = true;
      for (int t = first; t < p.pieces && ok; t += pairs) {
        const Tile at = tile_at(p, t);
        const int arow = at.m * kTileM + 128 * static_cast<int>(rank);
        const int wrow = at.n0 + at.width / 2 * static_cast<int>(rank);  // of a narrow piece the box's first rows count
        for (int kb = 0; kb < p.nkb; ++kb, ++k) {
          if (k >= kWideStages && !mbar_wait(kWaitLimitNs, &sm.empty[s], phase)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * kWideStageBytes);
          const uint32_t bar = in_cta(&sm.full[s], 0);
          tma_load_2d_pair(sm.ring[s], &amap, kb * kBK, arow, bar);
          tma_load_2d_pair(sm.ring[s] + 128 * kBK, &wmap, kb * kBK, wrow, bar);
          if (++s == kWideStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {
        flag_failure(p.status);
        // Let the copies already issued land before this CTA's shared memory goes away: the leader sees both
        // CTAs' on its barriers; the cluster barrier at the end keeps the peer.
        if (rank == 0)
          for (int64_t j = max(static_cast<int64_t>(0), k - kWideStages); j < k; ++j)
            if (!mbar_wait(kWaitLimitNs, &sm.full[j % kWideStages], static_cast<uint32_t>(j / kWideStages) & 1u)) break;
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------------------------------------------------------------- products
      int s = 0, b = 0;
      uint32_t phase = 0, bphase = 1;
      bool ok = true;
      int64_t k = 0;
      for (int t = first; t < p.pieces && ok; t += pairs) {
        const int width = tile_at(p, t).width;
        const uint32_t idesc = width == 256 ? e4m3_idesc(256, 256) : width == 128 ? e4m3_idesc(256, 128) : e4m3_idesc(256, 64);
        for (int kb = 0; kb < p.nkb; ++kb, ++k) {
          ok = (k < 2 || mbar_wait(kWaitLimitNs, &sm.free_[b], bphase)) && mbar_wait(kWaitLimitNs, &sm.full[s], phase);
          if (!ok) {
            flag_failure(p.status);
            break;
          }
          tc_fence_after();
          const uint64_t ad = tile_desc(smem_addr(sm.ring[s])), wd = tile_desc(smem_addr(sm.ring[s] + 128 * kBK));
#pragma unroll
          for (int i = 0; i < kBK / 32; ++i) mma_e4m3_tile<2>(tmem + b * 256, ad + 2 * i, wd + 2 * i, idesc, i > 0);
          mma_commit<2>(&sm.empty[s]);
          mma_commit<2>(&sm.done[b]);
          if (++s == kWideStages) {
            s = 0;
            phase ^= 1u;
          }
          b ^= 1;
          if (b == 0) bphase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------------ epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3, half = (warp - 4) >> 2;  // lanes 32*quarter.., which half of the columns
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    unsigned char* stage = sm.out[warp - 4][0];
    const uint32_t free0 = in_cta(&sm.free_[0], 0), free1 = in_cta(&sm.free_[1], 0);
    int b = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = first; t < p.pieces && ok; t += pairs) {
      const Tile at = tile_at(p, t);
      // 128 or 64 columns of a warp; a piece of 64 leaves the second half without any, but its barriers are kept.
      const bool both = at.width == 256, none = at.width == 64 && half == 1;
      const int row0 = at.m * kTileM + 128 * static_cast<int>(rank) + 32 * quarter, col0 = at.n0 + (both ? 128 : 64) * half;
      const uint32_t from = lanes + (both ? 128 : 64) * half;
      const float* sa = p.sa + static_cast<int64_t>(min(row0 + lane, p.M - 1)) * p.sa_stride;
      // The columns start at a multiple of their number, so they lie in one scale block.
      const float* sb = p.sb + static_cast<int64_t>(min(col0, p.N - 1) / kScaleBlock) * p.sb_stride;
      // Of a piece of 64 columns the second half has none: it reads what is there and keeps the barriers going.
      auto piece = [&](auto chunks) {
        constexpr int kChunks = decltype(chunks)::value;
        const float a0 = ld_f32(sa), b0 = ld_f32(sb);
        uint2 bias = make_uint2(0u, 0u);
        if (kFused && !none) bias = wide_prepare<kChunks>(p, stage, row0, col0);
        float2 acc[16 * kChunks];
        ok = wide_accumulate<kChunks>(p, sm, sa, sb, a0, b0, from, free0, free1, b, phase, acc);
        if (!ok || none) return;
        if constexpr (kFused) wide_store_fused<kChunks, kAct, T>(p, &omap, stage, row0, col0, bias, acc);
        else wide_store<kChunks>(p, &omap, stage, row0, col0, acc);
      };
      if (both) piece(std::integral_constant<int, 4>());
      else piece(std::integral_constant<int, 2>());
      if (!ok) flag_failure(p.status);
    }
    if (kFused) asm volatile("cp.async.wait_all;" ::: "memory");  // of a piece whose products never came
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  cluster_barrier();  // no CTA leaves while its peer's products, arrivals or copies refer to it
  tc_fence_after();
  if (warp == 1) tmem_free<2>(tmem, 512);
}

template <int kAct, typename T>
bool launch_wide(const MatmulArgs& a, MmArgs p, const MatmulPlan& plan, cudaStream_t s) {
  CUtensorMap amap, wmap, omap{};
  const uint64_t ad[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.M)}, as[1] = {static_cast<uint64_t>(a.a_stride)};
  const uint64_t wd[2] = {static_cast<uint64_t>(a.K), static_cast<uint64_t>(a.N)}, ws[1] = {static_cast<uint64_t>(a.b_stride)};
  const uint32_t ab[2] = {kBK, 128}, wb[2] = {kBK, 128};
  if (!byte_tensor_map(&amap, 2, a.a, ad, as, ab, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !byte_tensor_map(&wmap, 2, a.b, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B))
    return false;
  // Output boxes of 64 columns, 128 bytes. The map counts 16-bit elements: coordinates are 32-bit, and as bytes those of
  // columns from 2^30 on would not fit. Rows that are not whole 16-byte pieces are stored directly, by their stride and
  // by their length: a box store cut off by the end of a row writes zeros up to the next 16-byte boundary (measured: 4
  // elements behind rows of 2300), which in an output whose rows are further apart is not the call's to write.
  const uint64_t od[2] = {static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.M)}, os[1] = {static_cast<uint64_t>(a.out_stride) * 2};
  const uint32_t ob[2] = {64, 32};
  p.tma_store = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && os[0] % 16 == 0 && a.N % 8 == 0 &&
                half_tensor_map(&omap, 2, a.out, od, os, ob, CU_TENSOR_MAP_SWIZZLE_128B);
  p.tiles_m = static_cast<int32_t>((a.M + kTileM - 1) / kTileM);
  p.tiles_n = static_cast<int32_t>((a.N + kTileN - 1) / kTileN);
  const int64_t tiles = static_cast<int64_t>(p.tiles_m) * p.tiles_n;
  if (tiles > 0x0fffffff) return false;
  const int64_t pairs = sm_count() / 2, rest = tiles % pairs;
  p.whole = static_cast<int32_t>(tiles - rest);
  p.parts = plan.parts;
  p.pieces = static_cast<int32_t>(p.whole + rest * p.parts);
  constexpr size_t smem = sizeof(WideShared<kAct != kPlain>) + 1024;
  static_assert(smem <= 227 * 1024, "the ring and the staging rows fit the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(matmul_wide_kernel<kAct, T>), smem)) return false;
  launch_overlapped(matmul_wide_kernel<kAct, T>, dim3(static_cast<unsigned>(2 * (p.pieces < pairs ? p.pieces : pairs))), kWideThreads, smem, 2, s,
                    amap, wmap, omap, p);
  return true;
}

}  // namespace
}  // namespace fq
