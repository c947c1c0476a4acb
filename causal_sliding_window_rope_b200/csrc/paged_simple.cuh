// paged_simple.cuh -- first forms of the paged attention and of the
// accumulated weights: one warp per output row, float32 throughout.
#pragma once
#include "paged.cuh"

namespace cswattn {
namespace paged {

struct AttendParams {
  View v;
  float scale;
  int min_rows;
  const __nv_bfloat16 *q, *k_pages, *v_pages;
  __nv_bfloat16* O;
  float* lse;
};

// Warp = (token, head): online softmax over the rows the token sees.
template <int D>
__global__ void __launch_bounds__(256) attend_simple_kernel(const AttendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const View& v = p.v;
  const int b = blockIdx.y, lane = lane_id();
  Seq s;
  if (!seq_load(v, b, blockIdx.x == 0 && threadIdx.x == 0, s) || s.n * v.g < p.min_rows) return;
  for (int w = blockIdx.x * 8 + warp_id(); w < s.n * v.H; w += gridDim.x * 8) {
    const int i = w / v.H, h = w % v.H, hk = h / v.g;
    const size_t row = static_cast<size_t>(s.tok0 + i) * v.H + h;
    float q[D / 32], o[D / 32], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      q[e] = __bfloat162float(p.q[row * D + e * 32 + lane]);
      o[e] = 0.f;
    }
    const int last = s.L + i;
    for (int r = max(0, last - v.W + 1); r <= last; ++r) {
      const int page = page_at(v, b, r / v.page_size);
      if (page < 0) continue;
      const size_t at = kv_index(v, page, r % v.page_size, hk) * D;
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) d = fmaf(q[e], __bfloat162float(p.k_pages[at + e * 32 + lane]), d);
      d = row_sum<32>(d) * p.scale;
      const float mn = fmaxf(m, d), a = expf(m - mn), x = expf(d - mn);
      l = l * a + x;
      m = mn;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        o[e] = fmaf(x, __bfloat162float(p.v_pages[at + e * 32 + lane]), o[e] * a);
    }
#pragma unroll
    for (int e = 0; e < D / 32; ++e) p.O[row * D + e * 32 + lane] = __float2bfloat16_rn(o[e] / l);
    if (lane == 0) p.lse[row] = m + logf(l);
  }
}

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
