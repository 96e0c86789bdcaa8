// fq_matmul.cu -- the choice of the matrix product's kernel, and the products without an epilogue (fq_matmul_fused.cu has
// those with one: the instances are many and compile side by side).
#include <cmath>

#include "fq_matmul.cuh"

namespace fq {
namespace {

bool launch_product(const MatmulArgs& a, const MmArgs& p, const MatmulPlan& plan, cudaStream_t s) {
  switch (plan.rows) {
    case 16: return launch_narrow<16, false>(a, p, plan, s);
    case 32: return launch_narrow<32, false>(a, p, plan, s);
    case 64: return launch_narrow<64, false>(a, p, plan, s);
    case 128: return launch_narrow<128, false>(a, p, plan, s);
    default: return launch_wide<kPlain, void>(a, p, plan, s);
  }
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
  const MatmulPlan plan = matmul_plan(a.M, a.N, a.K, sm_count());
  if (a.fused()) return launch_matmul_fused(a, plan, dtype, s);
  return launch_product(valid_strides(a), device_args(a, dtype), plan, s);
}

}  // namespace fq
