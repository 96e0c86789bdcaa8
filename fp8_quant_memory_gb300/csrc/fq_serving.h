// fq_serving.h -- host-side launch interface of the FP8 serving operators: the block-scaled matrix
// product, the QKV prologue that appends to a paged cache, and paged attention of one new token.
#pragma once

#include "fq_internal.h"

namespace fq {

constexpr int kScaleBlock = 128;  // columns (and weight rows) per scale of the matrix product

// out[i, j] = dtype(sum_g a_scale[i, g] * b_scale[j / 128, g] * sum_{k in block g} a[i, k] * b[j, k]).
// Strides are in elements; `groups` = ceil(K / 128).
struct MatmulArgs {
  const uint8_t* a;
  const uint8_t* b;
  const float* a_scale;
  const float* b_scale;
  void* out;
  int64_t a_stride, b_stride, a_scale_stride, b_scale_stride, out_stride;
  int64_t M, N, K, groups;
};

// The cache as the kernels see it: row (page, head, slot) of K starts at k + page*page_stride +
// head*head_stride + slot*token_stride (bytes: e4m3 codes), its scale likewise with the s_* strides.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, head_stride, token_stride;
  int64_t s_page_stride, s_head_stride, s_token_stride;
  int64_t pages;
  int32_t page_size;
  int32_t page_shift;  // log2(page_size), or -1 when it is no power of two
};

struct AppendArgs {
  RowArgs rows;  // x = qkv, H = Hq + 2*Hk, rows = T*H, q and scale = the q outputs
  const int64_t* slots;
  CacheView cache;
  int32_t Hk;
};

struct PagedArgs {
  const uint8_t* q;
  const float* q_scale;
  int64_t q_stride, q_scale_stride;
  CacheView cache;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  void* out;
  float* lse;  // nullable
  float* partial;
  int32_t B, Hq, Hk, D;
  int32_t max_len;  // lengths are cut to this (the caller's bound and what the page table holds)
  float scale_log2;  // softmax_scale * log2(e)
};

// Launches `kern` so that its set-up overlaps the tail of the previous kernel in the stream (it calls pdl_wait before
// its first global access), in clusters of `cluster` CTAs along x. A failure is reported by the caller's check.
template <typename... P, typename... A>
void launch_overlapped(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                       const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaLaunchKernelEx(&cfg, kern, args...);
}

// How the tensor cores take a product on a GPU of `sms` SMs: rows of `a` per tile (16 to 128: the narrow kernel, 256: the
// wide one); narrow: CTAs that share a tile's k, and groups of epilogue warps; wide: column ranges that each tile of
// the last round is cut into.
struct MatmulPlan {
  int rows, split, groups, parts;
};
MatmulPlan matmul_plan(int64_t M, int64_t N, int64_t K, int sms);

// tcgen05 kernels: 16-byte aligned operands and strides. False (nothing launched) otherwise.
bool launch_matmul_tc(const MatmulArgs& a, int dtype, cudaStream_t s);
void launch_matmul_scalar(const MatmulArgs& a, int dtype, cudaStream_t s);

bool launch_append_vector(const AppendArgs& a, int dtype, int table_dtype, cudaStream_t s);
void launch_append_scalar(const AppendArgs& a, int dtype, int table_dtype, cudaStream_t s);

// Partial results of split sequences: what launch_attention_split needs in its workspace.
size_t attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_len);
bool launch_attention_split(const PagedArgs& a, int dtype, cudaStream_t s);
void launch_attention_scalar(const PagedArgs& a, int dtype, cudaStream_t s);

// Launch result of an entry point (and the strict-mode check), as every entry point reports it.
int finish_launch(const char* fn, cudaStream_t s);
// Drops a stale error that an unrelated earlier call left behind.
void drop_stale_error();
int succeed();

}  // namespace fq
