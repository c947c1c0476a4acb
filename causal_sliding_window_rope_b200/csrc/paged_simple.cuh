// paged_simple.cuh -- first form of the accumulated weights: one warp per
// cached row, float32 throughout.
#pragma once
#include "paged.cuh"

namespace cswattn {
namespace paged {

struct WeighParams {
  View v;
  float scale;
  const __nv_bfloat16 *q, *k_pages;
  const float* lse;
  float* weight;
};

// Warp = cached row of one KV head: sum over the tokens that see it.
template <int D>
__global__ void __launch_bounds__(256) weigh_simple_kernel(const WeighParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const View& v = p.v;
  const int b = blockIdx.y, lane = lane_id();
  Seq s;
  if (!seq_load(v, b, blockIdx.x == 0 && threadIdx.x == 0, s) || s.n == 0) return;
  const int lo = max(0, s.L - v.W + 1), rows = s.L + s.n - lo;
  for (int w = blockIdx.x * 8 + warp_id(); w < rows * v.Hk; w += gridDim.x * 8) {
    const int r = lo + w / v.Hk, hk = w % v.Hk;
    const int page = page_at(v, b, r / v.page_size);
    if (page < 0) continue;
    const size_t at = kv_index(v, page, r % v.page_size, hk) * D;
    float k[D / 32], sum = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) k[e] = __bfloat162float(p.k_pages[at + e * 32 + lane]);
    // token i sees rows (L + i - W, L + i]
    for (int i = max(0, r - s.L); i < s.n && s.L + i - v.W < r; ++i)
      for (int h = 0; h < v.g; ++h) {
        const size_t row = static_cast<size_t>(s.tok0 + i) * v.H + hk * v.g + h;
        float d = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) d = fmaf(k[e], __bfloat162float(p.q[row * D + e * 32 + lane]), d);
        sum += expf(row_sum<32>(d) * p.scale - p.lse[row]);
      }
    if (lane == 0) p.weight[term_index(v, page, r % v.page_size, hk)] += sum;
  }
}

}  // namespace paged
}  // namespace cswattn
