// fq_serving_api.cu -- the extern "C" entry points of the FP8 serving operators declared in
// include/fq.h: argument validation on the host (before any CUDA call), the choice between the
// tensor-core / vectorised and the any-layout kernels, launch and error reporting.
#include <cmath>

#include "fq.h"
#include "fq_serving.h"

namespace {

constexpr int64_t kMaxDim = 0x7fffffffLL - 1024;  // rows and columns: tile arithmetic stays in int32
constexpr int64_t kMaxWidth = 1LL << 24;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int check_dtype(const char* fn, int dtype) {
  if (dtype != FQ_BF16 && dtype != FQ_FP16)
    return fq::set_error(FQ_ERR_UNSUPPORTED, "%s: dtype %d is not FQ_BF16 or FQ_FP16", fn, dtype);
  return FQ_OK;
}

struct Axis {
  int64_t extent, stride;
};

// Whether rows of `inner` elements laid out over the three axes neither overlap nor leave 63 bits.
bool disjoint(Axis x, Axis y, Axis z, int64_t inner) {
  Axis ax[3] = {x, y, z};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (ax[j].extent > 1 && (ax[j + 1].extent <= 1 || ax[j].stride > ax[j + 1].stride)) {
        const Axis t = ax[j];
        ax[j] = ax[j + 1];
        ax[j + 1] = t;
      }
  // axes of extent 1 first (their stride is never used), then by growing stride
  __int128 span = inner;
  for (const Axis& a : ax) {
    if (a.extent <= 1) continue;
    if (a.stride < span) return false;
    span += static_cast<__int128>(a.stride) * (a.extent - 1);
  }
  return span < (static_cast<__int128>(1) << 62);
}

int cache_view(const char* fn, const fq_paged_cache* c, int64_t Hk, int64_t D, fq::CacheView* v) {
  if (c == nullptr) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: cache is null", fn);
  if (c->pages < 0 || c->pages > kMaxDim || c->page_size < 1 || c->page_size > kMaxDim)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need 0 <= pages < 2^31 and 1 <= page_size < 2^31", fn);
  if (c->pages > 0 && Hk > 0) {
    if (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr)
      return fq::set_error(FQ_ERR_INVALID_ARG, "%s: null cache pointer", fn);
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
      return fq::set_error(FQ_ERR_INVALID_ARG, "%s: the cache's scales must be 4-byte aligned", fn);
    if (!disjoint({c->pages, c->page_stride}, {Hk, c->head_stride}, {c->page_size, c->token_stride}, D) ||
        !disjoint({c->pages, c->scale_page_stride}, {Hk, c->scale_head_stride}, {c->page_size, c->scale_token_stride}, 1))
      return fq::set_error(FQ_ERR_INVALID_ARG, "%s: the cache's strides make rows overlap", fn);
  }
  v->k = c->k;
  v->v = c->v;
  v->k_scale = c->k_scale;
  v->v_scale = c->v_scale;
  v->page_stride = c->page_stride;
  v->head_stride = c->head_stride;
  v->token_stride = c->token_stride;
  v->s_page_stride = c->scale_page_stride;
  v->s_head_stride = c->scale_head_stride;
  v->s_token_stride = c->scale_token_stride;
  v->pages = c->pages;
  v->page_size = static_cast<int32_t>(c->page_size);
  v->page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c->page_size == (1LL << i)) v->page_shift = i;
  return FQ_OK;
}

// 16-byte loads of a row of codes: base and every stride that is used a multiple of 16.
bool cache_vec16(const fq::CacheView& c, int64_t Hk) {
  auto ok = [](int64_t extent, int64_t stride) { return extent <= 1 || stride % 16 == 0; };
  return aligned(c.k, 16) && aligned(c.v, 16) && ok(c.pages, c.page_stride) && ok(Hk, c.head_stride) &&
         ok(c.page_size, c.token_stride);
}

}  // namespace

extern "C" {

int fq_fp8_matmul(const uint8_t* a, int64_t a_stride, const float* a_scale, int64_t a_scale_stride, const uint8_t* b,
                  int64_t b_stride, const float* b_scale, int64_t b_scale_stride, void* out, int64_t out_stride,
                  int64_t M, int64_t N, int64_t K, int dtype, cudaStream_t stream) {
  const char* fn = "fq_fp8_matmul";
  if (int rc = check_dtype(fn, dtype)) return rc;
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim || K < 1 || K > kMaxDim)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need 0 <= M, N < 2^31 - 1024 and 1 <= K < 2^31 - 1024", fn);
  if (M == 0 || N == 0) return fq::succeed();
  if (a == nullptr || a_scale == nullptr || b == nullptr || b_scale == nullptr || out == nullptr)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: null pointer", fn);
  const int64_t groups = (K + fq::kScaleBlock - 1) / fq::kScaleBlock;
  constexpr int64_t kMaxStride = 1LL << 40;
  // a, b and their scales are only read: any stride, 0 (a broadcast row) among them, names valid rows
  if (a_stride < 0 || b_stride < 0 || a_scale_stride < 0 || b_scale_stride < 0 || a_stride > kMaxStride ||
      b_stride > kMaxStride || a_scale_stride > kMaxStride || b_scale_stride > kMaxStride || out_stride > kMaxStride ||
      (M > 1 && out_stride < N))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40], out_stride >= N", fn);
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(out, 2))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: scales must be 4-byte and out 2-byte aligned", fn);
  fq::MatmulArgs m{};
  m.a = a;
  m.b = b;
  m.a_scale = a_scale;
  m.b_scale = b_scale;
  m.out = out;
  m.a_stride = a_stride;
  m.b_stride = b_stride;
  m.a_scale_stride = a_scale_stride;
  m.b_scale_stride = b_scale_stride;
  m.out_stride = out_stride;
  m.M = M;
  m.N = N;
  m.K = K;
  m.groups = groups;
  // The tensor maps need 16-byte aligned operands and row strides, and rows that do not overlap.
  const bool tc = aligned(a, 16) && aligned(b, 16) && (M == 1 || (a_stride % 16 == 0 && a_stride >= K)) &&
                  (N == 1 || (b_stride % 16 == 0 && b_stride >= K));
  fq::drop_stale_error();
  if (!(tc && fq::launch_matmul_tc(m, dtype, stream))) fq::launch_matmul_scalar(m, dtype, stream);
  return fq::finish_launch(fn, stream);
}

int fq_fp8_matmul_plan(int64_t M, int64_t N, int64_t K, int sms, int* plan) {
  const char* fn = "fq_fp8_matmul_plan";
  if (plan == nullptr) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: plan is null", fn);
  if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim || sms < 2)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need 1 <= M, N, K < 2^31 - 1024 and at least 2 SMs", fn);
  const fq::MatmulPlan p = fq::matmul_plan(M, N, K, sms);
  plan[0] = p.rows;
  plan[1] = p.split;
  plan[2] = p.groups;
  plan[3] = p.parts;
  return fq::succeed();
}

int fq_qkv_norm_rope_append(const void* qkv, int64_t token_stride, const void* wq, const void* wk, const void* cos,
                            const void* sin, const int64_t* slots, uint8_t* q_out, float* q_scale,
                            const fq_paged_cache* cache, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                            int64_t rope_dim, int dtype, int table_dtype, float eps, float fp8_max,
                            cudaStream_t stream) {
  const char* fn = "fq_qkv_norm_rope_append";
  if (int rc = check_dtype(fn, dtype)) return rc;
  if (table_dtype != FQ_BF16 && table_dtype != FQ_FP16 && table_dtype != FQ_FP32)
    return fq::set_error(FQ_ERR_UNSUPPORTED, "%s: table dtype %d is not FQ_BF16, FQ_FP16 or FQ_FP32", fn, table_dtype);
  if (!(eps >= 0.0f) || !std::isfinite(eps))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (!(fp8_max > 0.0f && fp8_max <= 448.0f))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: fp8_max must be in (0, 448], got %g", fn, static_cast<double>(fp8_max));
  if (T < 0 || Hq < 0 || Hk < 1 || D < 1 || D > kMaxWidth || Hq > kMaxWidth || Hk > kMaxWidth)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need T >= 0, Hq >= 0, Hk >= 1, D >= 1", fn);
  if (rope_dim < 0 || rope_dim % 2 != 0 || rope_dim > D)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: rope_dim must be even and in [0, %lld], got %lld", fn,
                         static_cast<long long>(D), static_cast<long long>(rope_dim));
  const int64_t H = Hq + 2 * Hk;
  if (token_stride < H * D && T > 1)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: token_stride %lld < (Hq+2*Hk)*D = %lld", fn,
                         static_cast<long long>(token_stride), static_cast<long long>(H * D));
  if (T > kMaxDim / H) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: T*(Hq+2*Hk) must be < 2^31 - 1024", fn);
  fq::AppendArgs p{};
  if (int rc = cache_view(fn, cache, Hk, D, &p.cache)) return rc;
  if (T == 0) return fq::succeed();
  if (qkv == nullptr || wk == nullptr || slots == nullptr || (Hq > 0 && (wq == nullptr || q_out == nullptr || q_scale == nullptr)))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (rope_dim > 0 && (cos == nullptr || sin == nullptr))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: cos/sin are null", fn);
  const unsigned tsize = table_dtype == FQ_FP32 ? 4 : 2;
  if (!aligned(qkv, 2) || !aligned(wk, 2) || (Hq > 0 && (!aligned(wq, 2) || !aligned(q_scale, 4))) ||
      !aligned(slots, 8) || (rope_dim > 0 && (!aligned(cos, tsize) || !aligned(sin, tsize))))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
  p.rows.x = qkv;
  p.rows.wq = Hq > 0 ? wq : wk;
  p.rows.wk = wk;
  p.rows.cos = cos;
  p.rows.sin = sin;
  p.rows.q = q_out;
  p.rows.scale = q_scale;
  p.rows.rows = T * H;
  p.rows.token_stride = token_stride;
  p.rows.H = static_cast<int32_t>(H);
  p.rows.Hq = static_cast<int32_t>(Hq);
  p.rows.N = static_cast<int32_t>(D);
  p.rows.R = static_cast<int32_t>(rope_dim);
  p.rows.eps = eps;
  p.rows.fp8_max = fp8_max;
  p.slots = slots;
  p.Hk = static_cast<int32_t>(Hk);
  const bool vec = D % 16 == 0 && rope_dim % 16 == 0 && aligned(qkv, 16) && aligned(p.rows.wq, 16) && aligned(wk, 16) &&
                   (T == 1 || token_stride % 8 == 0) && aligned(q_out, 16) && cache_vec16(p.cache, Hk) &&
                   (rope_dim == 0 || (aligned(cos, 16) && aligned(sin, 16) && (rope_dim / 2 * tsize) % 16 == 0 &&
                                      (table_dtype == FQ_FP32 || table_dtype == dtype)));
  fq::drop_stale_error();
  if (!(vec && fq::launch_append_vector(p, dtype, table_dtype, stream)))
    fq::launch_append_scalar(p, dtype, table_dtype, stream);
  return fq::finish_launch(fn, stream);
}

size_t fq_paged_attention_workspace_bytes(int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_seq_len) {
  if (B <= 0 || Hk <= 0 || Hq <= 0 || D <= 0 || D > 256 || max_seq_len <= 0 || Hq % Hk != 0) return 0;
  // a larger bound is no bound: no call takes longer sequences
  return fq::attention_workspace_bytes(B, Hq, Hk, D, max_seq_len < kMaxDim ? max_seq_len : kMaxDim);
}

int fq_paged_attention(const uint8_t* q, int64_t q_stride, const float* q_scale, int64_t q_scale_stride,
                       const fq_paged_cache* cache, const int32_t* page_table, int64_t table_stride,
                       const int32_t* seq_lens, void* out, float* lse, void* workspace, size_t workspace_bytes,
                       int64_t B, int64_t Hq, int64_t Hk, int64_t D, int64_t max_pages, int64_t max_seq_len,
                       float softmax_scale, int dtype, cudaStream_t stream) {
  const char* fn = "fq_paged_attention";
  if (int rc = check_dtype(fn, dtype)) return rc;
  if (!std::isfinite(softmax_scale)) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: softmax_scale must be finite", fn);
  if (B < 0 || Hq < 1 || Hk < 1 || Hq > 65536 || Hq % Hk != 0 || B > kMaxDim / Hq)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need B >= 0, Hk >= 1, Hq a multiple of Hk up to 65536, B*Hq < 2^31 - 1024", fn);
  if (D < 1) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need D >= 1", fn);
  if (D > 256) return fq::set_error(FQ_ERR_UNSUPPORTED, "%s: head_dim %lld is above 256", fn, static_cast<long long>(D));
  constexpr int64_t kMaxStride = 1LL << 40;
  if (max_pages < 0 || max_seq_len < 0 || max_pages > kMaxDim)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: need 0 <= max_pages < 2^31 - 1024 and max_seq_len >= 0", fn);
  if (table_stride < 0 || q_stride < 0 || q_scale_stride < 0 || table_stride > kMaxStride || q_stride > kMaxStride ||
      q_scale_stride > kMaxStride)
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: strides must be in [0, 2^40]", fn);
  fq::PagedArgs p{};
  if (int rc = cache_view(fn, cache, Hk, D, &p.cache)) return rc;
  if (B == 0) return fq::succeed();
  int64_t max_len = max_seq_len;
  if (max_pages == 0 || p.cache.pages == 0) max_len = 0;
  else if (max_len > max_pages * p.cache.page_size) max_len = max_pages * p.cache.page_size;
  if (max_len > kMaxDim) return fq::set_error(FQ_ERR_INVALID_ARG, "%s: lengths must be < 2^31 - 1024", fn);
  if (q == nullptr || q_scale == nullptr || seq_lens == nullptr || out == nullptr || (max_len > 0 && page_table == nullptr))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned(q_scale, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(out, 2) || !aligned(lse, 4))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: a pointer is not aligned to its element", fn);
  const size_t need = max_len > 0 ? fq::attention_workspace_bytes(B, Hq, Hk, D, max_len) : 0;
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                         workspace == nullptr ? static_cast<size_t>(0) : workspace_bytes);
  if (need > 0 && !aligned(workspace, 16))
    return fq::set_error(FQ_ERR_INVALID_ARG, "%s: workspace must be 16-byte aligned", fn);
  p.q = q;
  p.q_scale = q_scale;
  p.q_stride = q_stride;
  p.q_scale_stride = q_scale_stride;
  p.table = page_table;
  p.table_stride = table_stride;
  p.lens = seq_lens;
  p.out = out;
  p.lse = lse;
  p.partial = static_cast<float*>(workspace);
  p.B = static_cast<int32_t>(B);
  p.Hq = static_cast<int32_t>(Hq);
  p.Hk = static_cast<int32_t>(Hk);
  p.D = static_cast<int32_t>(D);
  p.max_len = static_cast<int32_t>(max_len);
  p.scale_log2 = softmax_scale * 1.44269504088896341f;
  const bool vec = D % 16 == 0 && aligned(q, 16) && (B == 1 || q_stride % 16 == 0) && cache_vec16(p.cache, Hk) &&
                   aligned(out, 16);
  fq::drop_stale_error();
  if (!(vec && fq::launch_attention_split(p, dtype, stream))) fq::launch_attention_scalar(p, dtype, stream);
  return fq::finish_launch(fn, stream);
}

}  // extern "C"
