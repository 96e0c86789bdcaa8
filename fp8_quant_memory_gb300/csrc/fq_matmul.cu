// fq_matmul.cu -- the block-scaled FP8 matrix product on the 5th-generation tensor cores.
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
#include <cmath>

#include "fq_device.cuh"
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
};

__device__ __forceinline__ uint32_t pack_out(int dtype, float2 v) {
  return dtype == DT_BF16 ? Elem<__nv_bfloat16>::pack(v) : Elem<__half>::pack(v);
}

__device__ __forceinline__ void store_out(int dtype, void* out, int64_t i, float v) {
  if (dtype == DT_BF16) Elem<__nv_bfloat16>::store1(out, i, v);
  else Elem<__half>::store1(out, i, v);
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

template <int NT, int SPLIT, int G>
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
      const float b = __ldg(sb + k);
#pragma unroll
      for (int i = 0; i < kL; ++i) {
        const int j = lane + 32 * i;
        next[i] = j < NT && t0 + j < p.M ? __ldg(p.sa + static_cast<int64_t>(t0 + j) * p.sa_stride + k) * b : 0.f;
      }
    };
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
      if constexpr (SPLIT == 1) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (t0 + j < p.M && n0 + row < p.N) store_out(p.dtype, p.out, static_cast<int64_t>(t0 + j) * p.out_stride + n0 + row, value(j));
      } else {
        constexpr int kOwn = NT / SPLIT;
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
  if (SPLIT > 1 && warp >= 4) {
    __syncwarp();
    cluster_wait();
    cluster_barrier();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProducts) tmem_free<1>(tmem, C::kCols);
}

template <int NT>
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
  auto kern = split == 1 ? matmul_narrow_kernel<NT, 1, 1> : split == 2 ? matmul_narrow_kernel<NT, 2, 1> : matmul_narrow_kernel<NT, 4, 1>;
  int threads = kNarrowThreads<1>;
  if constexpr (NT == 64) {
    if (plan.groups == 2) {
      kern = split == 1 ? matmul_narrow_kernel<NT, 1, 2> : split == 2 ? matmul_narrow_kernel<NT, 2, 2> : matmul_narrow_kernel<NT, 4, 2>;
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

constexpr int kTileM = 256, kTileN = 256;  // outputs of a CTA pair
constexpr int kWideStageBytes = 256 * kBK; // one CTA's half of the pair's operands
constexpr int kWideStages = 6;

struct WideShared {
  alignas(1024) unsigned char ring[kWideStages][kWideStageBytes];  // 128 rows of a, then 128 weight rows
  alignas(1024) unsigned char out[8][32 * 128];                    // per epilogue warp: 32 rows x 64 columns
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
// accumulator buffer and its parity. False if a wait gave up.
template <int kChunks>
__device__ __forceinline__ bool wide_accumulate(const MmArgs& p, WideShared& sm, const float* sa, const float* sb, uint32_t from,
                                                uint32_t free0, uint32_t free1, int& b, uint32_t& phase,
                                                float2 (&acc)[16 * kChunks]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 16 * kChunks; ++j) acc[j] = make_float2(0.f, 0.f);
  float a_next = __ldg(sa), b_next = __ldg(sb);
  for (int kb = 0; kb < p.nkb; ++kb) {
    const float2 s2 = splat2(a_next * b_next);
    if (kb + 1 < p.nkb) {
      a_next = __ldg(sa + kb + 1);
      b_next = __ldg(sb + kb + 1);
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

// The warp's outputs from (row0, col0), 64 columns at a time through staging rows of 128 bytes (16-byte pieces
// swizzled): by a TMA box, or row by row with neighbouring lanes on neighbouring columns where the output has no
// tensor map (rows that are not whole 16-byte pieces).
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
    const int col = col0 + 64 * c;
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
}

__global__ void __launch_bounds__(kWideThreads, 1)
    matmul_wide_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap omap, const __grid_constant__ MmArgs p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  // The swizzle repeats every 1024 bytes: align to 1024 (the same offset in both CTAs).
  WideShared& sm = *reinterpret_cast<WideShared*>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
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
    unsigned char* stage = sm.out[warp - 4];
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
      if (both) {
        float2 acc[64];
        ok = wide_accumulate<4>(p, sm, sa, sb, from, free0, free1, b, phase, acc);
        if (ok) wide_store<4>(p, &omap, stage, row0, col0, acc);
      } else {
        // Of a piece of 64 columns the second half has none: it reads what is there and keeps the barriers going.
        float2 acc[32];
        ok = wide_accumulate<2>(p, sm, sa, sb, from, free0, free1, b, phase, acc);
        if (ok && !none) wide_store<2>(p, &omap, stage, row0, col0, acc);
      }
      if (!ok) flag_failure(p.status);
    }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  cluster_barrier();  // no CTA leaves while its peer's products, arrivals or copies refer to it
  tc_fence_after();
  if (warp == 1) tmem_free<2>(tmem, 512);
}

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
  constexpr size_t smem = sizeof(WideShared) + 1024;
  static_assert(smem <= 227 * 1024, "the ring and the staging rows fit the SM");
  if (!ensure_dynamic_smem(reinterpret_cast<const void*>(matmul_wide_kernel), smem)) return false;
  launch_overlapped(matmul_wide_kernel, dim3(static_cast<unsigned>(2 * (p.pieces < pairs ? p.pieces : pairs))), kWideThreads, smem, 2, s,
                    amap, wmap, omap, p);
  return true;
}

}  // namespace

MatmulPlan matmul_plan(int64_t M, int64_t N, int64_t K, int sm_total) {
  const int64_t nkb = (K + kBK - 1) / kBK;
  const double blocks = static_cast<double>(nkb), sms = sm_total, pairs = sm_total / 2;
  // CTAs that share a tile's k: as many as occupy SMs that would be idle.
  auto narrow_tiles = [&](int nt) { return ((N + 127) / 128) * ((M + nt - 1) / nt); };
  auto split_of = [&](int nt) {
    int split = 1;
    while (split < kMaxSplit && 2 * split * narrow_tiles(nt) <= sm_total && 2 * split <= nkb) split *= 2;
    return split;
  };
  // The kernel with the least estimated time. A CTA of the narrow kernel costs a start and a time per block of k,
  // which grow with its columns; the wide kernel a start and a time per block for each round of CTA pairs. In us,
  // fitted to a sweep over M of 1 to 2048 and (N, K) of (1111, 1968) to (8192, 8192), where the choice is the fastest
  // or within 15% of it: at 4096 x 4096 for example M = 16 takes 6.2 us with 16 columns and 7.8 with 64, M = 64 takes
  // 12.8 and 7.9, M = 256 takes 16.9 with 64, 16.4 with 128 and 18.8 wide, M = 512 26.1 with 128 and 19.5 wide.
  // It counts starts and blocks, no bytes, and was not fitted beyond these sizes: 1 x 28672 x 8192 goes to the CTA pairs
  // by an estimate of 60 us and takes 81 there (16 rows 59), 1 x 151936 x 4096 takes 177 (16 rows 134; the weights
  // alone, at the copy rate, 35 and 92 us); 64 x 8192 x 28672 takes 45 (35).
  auto narrow = [&](int nt, double start, double block) {
    // its tiles are the y and z axes of its grid, 65535 at most
    if ((N + 127) / 128 > 65535 || (M + nt - 1) / nt > 65535) return static_cast<double>(INFINITY);
    const int split = split_of(nt);
    return std::ceil(narrow_tiles(nt) * split / sms) * (start + std::ceil(blocks / split) * block);
  };
  const double t16 = narrow(16, 2.8, 0.43), t32 = narrow(32, 3.0, 0.43), t64 = narrow(64, 4.0, 0.47), t128 = narrow(128, 6.0, 0.67);
  const double tiles = static_cast<double>((M + kTileM - 1) / kTileM) * static_cast<double>((N + kTileN - 1) / kTileN);
  const double rest = std::fmod(tiles, pairs);
  const double wide = 4.5 + blocks * 0.47 * (std::floor(tiles / pairs) + (rest * 2 <= pairs ? 0.85 : 1.0));
  const double best = std::fmin(std::fmin(std::fmin(t16, t32), std::fmin(t64, t128)), wide);
  // Of the wide kernel, whole rounds of the CTA pairs first; the rest cut in two or four if one round takes all the
  // cuts (a narrow piece costs about 0.85 of a whole one).
  if (best == wide) return {kTileM, 1, 1, rest == 0 ? 1 : rest * 4 <= pairs ? 4 : rest * 2 <= pairs ? 2 : 1};
  const int rows = best == t16 ? 16 : best == t32 ? 32 : best == t64 ? 64 : 128, split = split_of(rows);
  return {rows, split, rows == 64 && nkb / split >= kTwoGroupBlocks ? 2 : 1, 1};
}

bool launch_matmul_tc(const MatmulArgs& a, int dtype, cudaStream_t s) {
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
  MatmulArgs b = a;
  // a single row's stride is never used, but has to be a valid one
  if (b.M == 1) b.a_stride = (b.K + 15) / 16 * 16;
  if (b.N == 1) b.b_stride = (b.K + 15) / 16 * 16;
  const MatmulPlan plan = matmul_plan(a.M, a.N, a.K, sm_count());
  switch (plan.rows) {
    case 16: return launch_narrow<16>(b, p, plan, s);
    case 32: return launch_narrow<32>(b, p, plan, s);
    case 64: return launch_narrow<64>(b, p, plan, s);
    case 128: return launch_narrow<128>(b, p, plan, s);
    default: return launch_wide(b, p, plan, s);
  }
}

}  // namespace fq
