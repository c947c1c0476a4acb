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
constexpr int kSelectMaxKeys = 48 << 10;   // keys a CTA holds in shared memory; further rows are read again
constexpr int kSelectMaxCluster = 8;       // CTAs that share one head's rows
constexpr int kSelectRows = 2048;          // rows worth a CTA of their own
constexpr int kBins = 2048;                // bins of one radix pass

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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Two words of shared memory of the cluster's CTA `rank` at the place of p.
__device__ __forceinline__ uint2 peer_load2(const void* p, int rank) {
  uint32_t a;
  uint2 y;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(y.x), "=r"(y.y) : "r"(a) : "memory");
  return y;
}

// A cluster of gridDim.x CTAs = (sequence, KV head), each with a run of
// consecutive rows. The n_keep-th largest key comes from three radix passes
// (11, 11, 10 bits): each CTA counts its rows' digits, the counts of all
// CTAs are read through the cluster's shared memory. Bound by latency, so the
// rows are read once (keys stay in shared memory) and long heads are spread
// over up to 8 SMs. Every path of a cluster's CTAs meets the same barriers.
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) uint32_t s_hist[2][kBins];  // two, so that a pass needs one meeting of the cluster
  __shared__ uint32_t s_warp[32];
  __shared__ uint32_t s_pick[2];
  __shared__ __align__(8) uint2 s_count[2];  // this CTA's ties; its holes and movers
  __shared__ uint2 s_before, s_all;          // ... of the CTAs before it, and of all
  const View& v = p.v;
  const int rank = blockIdx.x, ranks = gridDim.x, hk = blockIdx.y, b = blockIdx.z;
  const int warp = warp_id(), lane = lane_id(), tid = threadIdx.x;
  pdl_launch_dependents();
  for (int i = tid; i < 2 * kBins; i += kSelectThreads) (&s_hist[0][0])[i] = 0u;
  pdl_wait();
  const int L = v.cache_len[b];
  const size_t head = static_cast<size_t>(b) * v.Hk + hk;
  const bool lead = rank == 0;
  if (L < 0 || L > v.T) {
    if (lead && hk == 0 && tid == 0) atomicOr(&g_status, kStatusRange);
    return;
  }
  if (lead && hk == 0 && tid == 0) p.new_len[b] = min(L, p.n_keep);
  int* src = p.src + head * p.n_keep;
  int* dst = p.dst + head * p.n_keep;
  if (L <= p.n_keep) {
    if (lead && tid == 0) p.n_moves[head] = 0;
    for (int i = rank * kSelectThreads + tid; i < p.n_keep; i += ranks * kSelectThreads) src[i] = dst[i] = -1;
    return;
  }
  // This CTA's rows [base, base + mine).
  const int per = (L + ranks - 1) / ranks;
  const int base = min(L, rank * per), mine = min(L - base, per);
  // 64 bits: next_pos - n_recent may pass the smallest int
  const long long recent = static_cast<long long>(p.next_pos[b]) - p.n_recent;
  auto compute = [&](int i) -> uint32_t {
    const int r = base + i;
    const int page = page_at(v, b, page_entry(v, r));
    if (page < 0) return 0u;
    const size_t at = term_index(v, page, page_slot(v, r), hk);
    const float w = p.weight[at];
    return p.position[at] >= recent ? 0xFFFFFFFFu : weight_order(w);
  };
  const int held = min(mine, p.smem_keys);
#pragma unroll 4
  for (int i = tid; i < held; i += kSelectThreads) s_key[i] = compute(i);
  auto key = [&](int i) { return i < held ? s_key[i] : compute(i); };
  __syncthreads();

  // `want` keys are still to be found among those that start with `prefix`.
  uint32_t prefix = 0u;
  int want = p.n_keep;
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : (d == 1 ? 10 : 0);
    uint32_t* hist = s_hist[d & 1];
    for (int i0 = 0; i0 < mine; i0 += kSelectThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < mine ? key(i) : 0u;
      const bool in = i < mine && (d == 0 || (k >> (d == 1 ? 21 : 10)) == prefix);
      const uint32_t digit = (k >> shift) & (d == 2 ? 1023u : 2047u);
      // Equal weights (rows never attended to) are common: the lanes that
      // agree with the first counting one add once.
      const uint32_t m = __ballot_sync(0xffffffffu, in);
      if (m == 0u) continue;
      const int head_lane = __ffs(m) - 1;
      const uint32_t first_digit = __shfl_sync(0xffffffffu, digit, head_lane);
      const uint32_t same = __ballot_sync(0xffffffffu, in && digit == first_digit);
      if (lane == head_lane) atomicAdd(&hist[digit], __popc(same));
      else if (in && !((same >> lane) & 1u)) atomicAdd(&hist[digit], 1u);
    }
    cluster_sync();
    // Thread t holds bins 2t and 2t + 1 of all CTAs; suffix sums from the top.
    // (each CTA starts with its own counts, so that not all read the same one)
    uint32_t h0 = hist[2 * tid], h1 = hist[2 * tid + 1];
#pragma unroll
    for (int j = 1; j < kSelectMaxCluster; ++j) {
      if (j >= ranks) break;
      const uint2 h = peer_load2(&hist[2 * tid], (rank + j) % ranks);
      h0 += h.x;
      h1 += h.y;
    }
    uint32_t inc = h0 + h1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_down_sync(0xffffffffu, inc, o);
      if (lane + o < 32) inc += t;
    }
    if (lane == 0) s_warp[warp] = inc;
    __syncthreads();
    uint32_t later = s_warp[lane];  // of the warps behind this one
    later = lane > warp ? later : 0u;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) later += __shfl_xor_sync(0xffffffffu, later, o);
    inc += later;
    const uint32_t above = inc - h0 - h1;  // keys in bins over 2t + 1
    if (above < static_cast<uint32_t>(want) && inc >= static_cast<uint32_t>(want)) {
      const bool top = above + h1 >= static_cast<uint32_t>(want);
      s_pick[0] = 2 * tid + (top ? 1 : 0);
      s_pick[1] = static_cast<uint32_t>(want) - above - (top ? 0u : h1);
    }
    __syncthreads();
    prefix = d == 0 ? s_pick[0] : ((prefix << (d == 1 ? 11 : 10)) | s_pick[0]);
    want = static_cast<int>(s_pick[1]);
    // The buffer of pass 0 serves pass 2: cleared here, while no CTA reads it
    // any more (all have passed the meeting of pass 1).
    if (d == 1) {
      for (int i = tid; i < kBins; i += kSelectThreads) s_hist[0][i] = 0u;
      __syncthreads();
    }
  }
  // Kept: keys above `prefix`, and the first `want` rows equal to it. Each
  // warp takes a run of consecutive rows and counts before it writes; a
  // count's place is what the warps and the CTAs before it have.
  const int seg = ((mine + 31) / 32 + 31) / 32 * 32;
  const int i_lo = min(mine, warp * seg), i_hi = min(mine, i_lo + seg);
  auto before_warp = [&](uint32_t count, uint32_t& total) -> uint32_t {
    __syncthreads();
    if (lane == 0) s_warp[warp] = count;
    __syncthreads();
    const uint32_t x = s_warp[lane];
    uint32_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    total = __shfl_sync(0xffffffffu, inc, 31);
    return __shfl_sync(0xffffffffu, inc - x, warp);
  };
  auto exchange = [&](int which) {  // the cluster's counts: lane k of warp 0 reads CTA k's
    cluster_sync();
    if (warp == 0) {
      uint2 x = lane < ranks ? peer_load2(&s_count[which], lane) : make_uint2(0u, 0u);
      uint2 b = lane < rank ? x : make_uint2(0u, 0u);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        b.x += __shfl_xor_sync(0xffffffffu, b.x, o);
        b.y += __shfl_xor_sync(0xffffffffu, b.y, o);
      }
      if (lane == 0) {
        s_before = b;
        s_all = x;
      }
    }
    __syncthreads();
  };
  const uint32_t below = (1u << lane) - 1u;
  uint32_t eq = 0u, cta_total;
  for (int i0 = i_lo; i0 < i_hi; i0 += 32)
    eq += __popc(__ballot_sync(0xffffffffu, i0 + lane < i_hi && key(i0 + lane) == prefix));
  uint32_t eq_before = before_warp(eq, cta_total);
  if (tid == 0) s_count[0] = make_uint2(cta_total, 0u);
  exchange(0);
  eq_before += s_before.x;
  uint32_t hole_at = 0u, mover_at = 0u, total = 0u;
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t e = eq_before, nh = hole_at, nm = mover_at;
    for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
      const int i = i0 + lane, r = base + i;
      const bool in = i < i_hi;
      const uint32_t k = in ? key(i) : 0u;
      const uint32_t tie = __ballot_sync(0xffffffffu, in && k == prefix);
      const bool kept =
          in && (k > prefix || (k == prefix && e + __popc(tie & below) < static_cast<uint32_t>(want)));
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
      uint32_t cta_movers;
      hole_at = before_warp(nh, cta_total);
      mover_at = before_warp(nm, cta_movers);
      if (tid == 0) s_count[1] = make_uint2(cta_total, cta_movers);
      exchange(1);
      hole_at += s_before.x;
      mover_at += s_before.y;
      total = s_all.y;
    }
  }
  if (lead && tid == 0) p.n_moves[head] = static_cast<int>(total);
  for (int i = static_cast<int>(total) + rank * kSelectThreads + tid; i < p.n_keep; i += ranks * kSelectThreads)
    src[i] = dst[i] = -1;
  cluster_sync();  // no CTA leaves while another may still read its counts
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
constexpr int kMoveMaxCtas = 256;    // of a head: its moves are spread over them
constexpr int kMoveBatch = 4;        // moves a group of lanes has in flight

// D / 8 lanes copy one row of K and of V, 16 bytes each, kMoveBatch rows at a
// time: the rows lie anywhere, so what counts is how many loads are in
// flight behind the three dependent ones (move, page, row).
template <int D>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveParams p) {
  constexpr int LPR = D / 8, GPC = kMoveThreads / LPR;
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
  for (int i0 = (blockIdx.x * GPC + threadIdx.x / LPR) * kMoveBatch; i0 < n; i0 += gridDim.x * GPC * kMoveBatch) {
    int from[kMoveBatch], to[kMoveBatch], pf[kMoveBatch], pt[kMoveBatch];
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j) {
      const bool in = i0 + j < n;
      from[j] = in ? p.src[head * p.stride + i0 + j] : 0;
      to[j] = in ? p.dst[head * p.stride + i0 + j] : 0;
    }
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j) {
      pf[j] = pt[j] = -1;
      if (i0 + j >= n) continue;
      if (from[j] < 0 || from[j] >= v.T || to[j] < 0 || to[j] >= v.T) {
        atomicOr(&g_status, kStatusRange);
        continue;
      }
      pf[j] = page_at(v, b, page_entry(v, from[j]));
      pt[j] = page_at(v, b, page_entry(v, to[j]));
    }
    uint4 kk[kMoveBatch], vv[kMoveBatch];
    float w[kMoveBatch];
    int pos[kMoveBatch];
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j) {
      if (pf[j] < 0 || pt[j] < 0) continue;
      const int slot = page_slot(v, from[j]);
      const size_t a = kv_index(v, pf[j], slot, hk) * D + sub * 8;
      kk[j] = *reinterpret_cast<const uint4*>(p.k_pages + a);
      vv[j] = *reinterpret_cast<const uint4*>(p.v_pages + a);
      if (sub == 0) {
        w[j] = p.weight[term_index(v, pf[j], slot, hk)];
        pos[j] = p.position[term_index(v, pf[j], slot, hk)];
      }
    }
#pragma unroll
    for (int j = 0; j < kMoveBatch; ++j) {
      if (pf[j] < 0 || pt[j] < 0) continue;
      const int slot = page_slot(v, to[j]);
      const size_t z = kv_index(v, pt[j], slot, hk) * D + sub * 8;
      *reinterpret_cast<uint4*>(p.k_pages + z) = kk[j];
      *reinterpret_cast<uint4*>(p.v_pages + z) = vv[j];
      if (sub == 0) {
        p.weight[term_index(v, pt[j], slot, hk)] = w[j];
        p.position[term_index(v, pt[j], slot, hk)] = pos[j];
      }
    }
  }
}

}  // namespace paged
}  // namespace cswattn
