// paged_evict.cuh -- a budget of cached rows: which rows a sequence keeps
// (select) and the moves that bring them together (move).
//
// Each KV head of a sequence keeps n_keep of its L rows: those whose position
// is one of the n_recent newest, then the ones of largest accumulated weight,
// of equal weights the lowest row. The kept rows at or past n_keep move into
// the evicted rows below it (equally many), both in ascending order: no row
// moves that need not, every move's source lies past every target, so all
// moves are independent. A row keeps the key that was rotated to its
// position, and attention over rows that are all visible does not depend on
// their order.
#pragma once
#include "paged.cuh"

namespace cswattn {
namespace paged {

constexpr int kSelectThreads = 1024;
constexpr int kSelectMaxKeys = 48 << 10;  // keys held in shared memory; further rows are read again

struct SelectParams {
  View v;
  const float* weight;
  const int *position, *next_pos;
  int n_keep, n_recent;
  int smem_keys;
  int *n_moves, *src, *dst, *new_len;
};

// Order of a row: the recent ones first, then by weight; a NaN is below
// every number, and the zeros of both signs are equal.
__device__ __forceinline__ uint32_t weight_order(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[2048];
  __shared__ int s_warp[3][32];
  __shared__ uint32_t s_pick[2];
  const View& v = p.v;
  const int hk = blockIdx.x, b = blockIdx.y;
  const int warp = warp_id(), lane = lane_id();
  pdl_launch_dependents();
  pdl_wait();
  const int L = v.cache_len[b];
  const size_t head = static_cast<size_t>(b) * v.Hk + hk;
  if (L < 0 || L > v.T) {
    if (hk == 0 && threadIdx.x == 0) atomicOr(&g_status, kStatusRange);
    return;
  }
  if (hk == 0 && threadIdx.x == 0) p.new_len[b] = min(L, p.n_keep);
  int* src = p.src + head * p.n_keep;
  int* dst = p.dst + head * p.n_keep;
  if (L <= p.n_keep) {
    if (threadIdx.x == 0) p.n_moves[head] = 0;
    for (int i = threadIdx.x; i < p.n_keep; i += kSelectThreads) src[i] = dst[i] = -1;
    return;
  }
  // 64 bits: next_pos - n_recent may pass the smallest int
  const long long recent = static_cast<long long>(p.next_pos[b]) - p.n_recent;
  auto compute = [&](int r) -> uint32_t {
    const int page = page_at(v, b, r / v.page_size);
    if (page < 0) return 0u;
    const size_t at = term_index(v, page, r % v.page_size, hk);
    return p.position[at] >= recent ? 0xFFFFFFFFu : weight_order(p.weight[at]);
  };
  const int held = min(L, p.smem_keys);
  for (int r = threadIdx.x; r < held; r += kSelectThreads) s_key[r] = compute(r);
  auto key = [&](int r) { return r < held ? s_key[r] : compute(r); };

  // Radix selection of the n_keep-th largest key: digits of 11, 11 and 10
  // bits from the top. `want` keys are still to be found below the prefix.
  uint32_t prefix = 0u;
  int want = p.n_keep;
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    const int bins = d == 2 ? 1024 : 2048;
    for (int i = threadIdx.x; i < 2048; i += kSelectThreads) s_hist[i] = 0u;
    __syncthreads();
    for (int r0 = 0; r0 < L; r0 += kSelectThreads) {
      const int r = r0 + threadIdx.x;
      const uint32_t k = r < L ? key(r) : 0u;
      const bool in = r < L && (d == 0 || (k >> (d == 1 ? 21 : 10)) == prefix);
      const uint32_t digit = in ? ((k >> shift) & (bins - 1)) : 0xFFFFFFFFu;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&s_hist[digit], __popc(same));
    }
    __syncthreads();
    // Suffix sums from the top bin: thread t holds bins 2t and 2t + 1.
    const uint32_t h0 = s_hist[2 * threadIdx.x], h1 = s_hist[2 * threadIdx.x + 1];
    uint32_t inc = h0 + h1;  // inclusive suffix sum over threads t .. 1023
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_down_sync(0xffffffffu, inc, o);
      if (lane + o < 32) inc += t;
    }
    if (lane == 0) s_warp[0][warp] = static_cast<int>(inc);
    __syncthreads();
    for (int w = warp + 1; w < 32; ++w) inc += static_cast<uint32_t>(s_warp[0][w]);
    const uint32_t above = inc - h0 - h1;  // keys in bins over 2t + 1
    if (above < static_cast<uint32_t>(want) && inc >= static_cast<uint32_t>(want)) {
      const bool top = above + h1 >= static_cast<uint32_t>(want);
      s_pick[0] = 2 * threadIdx.x + (top ? 1 : 0);
      s_pick[1] = static_cast<uint32_t>(want) - above - (top ? 0u : h1);
    }
    __syncthreads();
    prefix = d == 0 ? s_pick[0] : ((prefix << (d == 1 ? 11 : 10)) | s_pick[0]);
    want = static_cast<int>(s_pick[1]);
  }
  // Kept: keys above `prefix`, and the first `want` rows equal to it. Each
  // warp takes a run of consecutive rows and counts before it writes.
  const int seg = ((L + 31) / 32 + 31) / 32 * 32;
  const int r_lo = min(L, warp * seg), r_hi = min(L, r_lo + seg);
  auto warp_prefix = [&](int which, int mine, int& before) {
    if (lane == 0) s_warp[which][warp] = mine;
    __syncthreads();
    const int x = s_warp[which][lane];
    before = 0;
    int total = 0;
    for (int w = 0; w < 32; ++w) {
      const int y = __shfl_sync(0xffffffffu, x, w);
      if (w < warp) before += y;
      total += y;
    }
    return total;
  };
  int eq = 0;
  for (int r0 = r_lo; r0 < r_hi; r0 += 32)
    eq += __popc(__ballot_sync(0xffffffffu, r0 + lane < r_hi && key(r0 + lane) == prefix));
  int eq_before;
  warp_prefix(0, eq, eq_before);
  const uint32_t below = (1u << lane) - 1u;
  int holes = 0, movers = 0, hole_at = 0, mover_at = 0, total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int e = eq_before;
    int nh = hole_at, nm = mover_at;
    for (int r0 = r_lo; r0 < r_hi; r0 += 32) {
      const int r = r0 + lane;
      const bool in = r < r_hi;
      const uint32_t k = in ? key(r) : 0u;
      const uint32_t tie = __ballot_sync(0xffffffffu, in && k == prefix);
      const bool kept = in && (k > prefix || (k == prefix && e + __popc(tie & below) < want));
      e += __popc(tie);
      const bool hole = in && !kept && r < p.n_keep, mover = kept && r >= p.n_keep;
      const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
      if (pass == 1) {
        if (hole) dst[nh + __popc(mh & below)] = r;
        if (mover) src[nm + __popc(mm & below)] = r;
      }
      nh += __popc(mh);
      nm += __popc(mm);
    }
    if (pass == 0) {
      holes = nh;
      movers = nm;
      warp_prefix(1, holes, hole_at);
      total = warp_prefix(2, movers, mover_at);
    }
  }
  if (threadIdx.x == 0) p.n_moves[head] = total;
  for (int i = total + threadIdx.x; i < p.n_keep; i += kSelectThreads) src[i] = dst[i] = -1;
}

struct MoveParams {
  View v;
  const int *n_moves, *src, *dst;
  int stride;  // entries of src and dst per head
  __nv_bfloat16 *k_pages, *v_pages;
  float* weight;
  int* position;
};

constexpr int kMoveThreads = 256;

// D / 8 lanes copy one row of K and of V, 16 bytes each.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  constexpr int LPR = D / 8, RPP = kMoveThreads / LPR;
  const View& v = p.v;
  const int hk = blockIdx.y, b = blockIdx.z;
  pdl_launch_dependents();
  pdl_wait();
  const size_t head = static_cast<size_t>(b) * v.Hk + hk;
  const int n = p.n_moves[head];
  if (n < 0 || n > p.stride) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_status, kStatusRange);
    return;
  }
  const int sub = threadIdx.x % LPR;
  for (int i = blockIdx.x * RPP + threadIdx.x / LPR; i < n; i += gridDim.x * RPP) {
    const int from = p.src[head * p.stride + i], to = p.dst[head * p.stride + i];
    if (from < 0 || from >= v.T || to < 0 || to >= v.T) {
      if (sub == 0) atomicOr(&g_status, kStatusRange);
      continue;
    }
    const int pf = page_at(v, b, from / v.page_size), pt = page_at(v, b, to / v.page_size);
    if (pf < 0 || pt < 0) continue;
    const size_t a = kv_index(v, pf, from % v.page_size, hk) * D + sub * 8;
    const size_t z = kv_index(v, pt, to % v.page_size, hk) * D + sub * 8;
    const uint4 kk = *reinterpret_cast<const uint4*>(p.k_pages + a);
    const uint4 vv = *reinterpret_cast<const uint4*>(p.v_pages + a);
    *reinterpret_cast<uint4*>(p.k_pages + z) = kk;
    *reinterpret_cast<uint4*>(p.v_pages + z) = vv;
    if (sub == 0) {
      const size_t ta = term_index(v, pf, from % v.page_size, hk), tz = term_index(v, pt, to % v.page_size, hk);
      p.weight[tz] = p.weight[ta];
      p.position[tz] = p.position[ta];
    }
  }
}

}  // namespace paged
}  // namespace cswattn
