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
// One or two words of shared memory of the cluster's CTA `rank` at the place of p.
__device__ __forceinline__ uint32_t peer_load(const void* p, int rank) {
  uint32_t a, y;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(y) : "r"(a) : "memory");
  return y;
}
__device__ __forceinline__ uint2 peer_load2(const void* p, int rank) {
  uint32_t a;
  uint2 y;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(y.x), "=r"(y.y) : "r"(a) : "memory");
  return y;
}

// A cluster of gridDim.x CTAs = (sequence, KV head), each with a run of
// consecutive rows. The n_keep-th largest key comes from three radix passes
// (11, 11, 10 bits): each CTA counts its rows' digits, the sums of 32 bins
// are read from all CTAs' shared memory, then the 32 bins of the one that
// holds the key. Bound by latency, so the rows are read once (keys stay in
// shared memory), long heads are spread over up to 8 SMs, and what the
// others have to know of a CTA's rows is exchanged once. Every path of a
// cluster's CTAs meets the same barriers. Measured: 128 heads of 1025 rows 8.5
// us; 16 heads of up to 40000 rows 22.2 us (111 with one CTA a head).
// A lone CTA (CLUSTER false) meets itself at the block's barrier and reads its
// own counts.
template <bool CLUSTER>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const SelectParams p) {
  const int ranks = CLUSTER ? gridDim.x : 1;
  auto meet = [] {
    if constexpr (CLUSTER) cluster_sync();
    else __syncthreads();
  };
  auto load1 = [](const uint32_t* x, int k) { return CLUSTER ? peer_load(x, k) : *x; };
  auto load2 = [](const void* x, int k) { return CLUSTER ? peer_load2(x, k) : *static_cast<const uint2*>(x); };
  extern __shared__ uint32_t s_key[];
  __shared__ uint32_t s_hist[2][kBins];          // two, so that a pass needs one meeting of the cluster
  __shared__ __align__(8) uint32_t s_sum[2][64];  // of 32 bins each
  __shared__ uint32_t s_pick[2];
  __shared__ uint32_t s_warp[4][32];             // of each warp's rows: ties and larger keys, below n_keep and past it
  __shared__ __align__(8) uint2 s_count[2];      // the same of this CTA
  __shared__ uint32_t s_before[3], s_total;      // ties, holes, movers of the CTAs before it; movers of all
  const View& v = p.v;
  const int rank = CLUSTER ? blockIdx.x : 0, hk = blockIdx.y, b = blockIdx.z;
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
  auto order = [&](float w, int pos) { return pos >= recent ? 0xFFFFFFFFu : weight_order(w); };
  const int held = min(mine, p.smem_keys);
  constexpr int kBatch = 8;  // rows a thread has in flight: a page, then a weight and a position each
  for (int i0 = tid; i0 < held; i0 += kBatch * kSelectThreads) {
    int page[kBatch], pos[kBatch];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kSelectThreads;
      page[j] = i < held ? page_at(v, b, page_entry(v, base + i)) : -1;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (page[j] < 0) continue;
      const size_t at = term_index(v, page[j], page_slot(v, base + i0 + j * kSelectThreads), hk);
      w[j] = p.weight[at];
      pos[j] = p.position[at];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kSelectThreads;
      if (i < held) s_key[i] = page[j] < 0 ? 0u : order(w[j], pos[j]);
    }
  }
  auto key = [&](int i) -> uint32_t {
    if (i < held) return s_key[i];
    const int page = page_at(v, b, page_entry(v, base + i));
    if (page < 0) return 0u;
    const size_t at = term_index(v, page, page_slot(v, base + i), hk);
    return order(p.weight[at], p.position[at]);
  };
  __syncthreads();

  // Of 32 values, the one that holds the want-th from the top (lane 31 first): its lane, and what is wanted of it.
  auto pick = [&](uint32_t x, uint32_t want, int& at, uint32_t& rest) {
    uint32_t inc = x;  // of this lane and those above
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_down_sync(0xffffffffu, inc, o);
      if (lane + o < 32) inc += t;
    }
    at = 31 - __clz(__ballot_sync(0xffffffffu, inc >= want));
    rest = want - __shfl_sync(0xffffffffu, inc - x, at);
  };
  // `want` keys are still to be found among those that start with `prefix`.
  uint32_t prefix = 0u, want = static_cast<uint32_t>(p.n_keep);
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
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = __reduce_add_sync(0xffffffffu, hist[(2 * warp + j) * 32 + lane]);
      if (lane == 0) s_sum[d & 1][2 * warp + j] = x;
    }
    meet();
    if (warp == 0) {
      uint2 x = make_uint2(0u, 0u);  // sums 2 lane and 2 lane + 1 of all CTAs
      uint32_t y = 0u;               // then a bin
#pragma unroll
      for (int j = 0; j < kSelectMaxCluster; ++j) {
        if (j >= ranks) break;
        const uint2 t = load2(&s_sum[d & 1][2 * lane], (rank + j) % ranks);
        x.x += t.x;
        x.y += t.y;
      }
      int at, bin;
      uint32_t rest;
      pick(x.x + x.y, want, at, rest);
      const uint32_t top = __shfl_sync(0xffffffffu, x.y, at);
      const bool second = top >= rest;
      at = 2 * at + (second ? 1 : 0);
      if (!second) rest -= top;
#pragma unroll
      for (int j = 0; j < kSelectMaxCluster; ++j) {
        if (j >= ranks) break;
        y += load1(&hist[at * 32 + lane], (rank + j) % ranks);
      }
      pick(y, rest, bin, rest);
      if (lane == 0) {
        s_pick[0] = static_cast<uint32_t>(at * 32 + bin);
        s_pick[1] = rest;
      }
    }
    __syncthreads();
    prefix = d == 0 ? s_pick[0] : ((prefix << (d == 1 ? 11 : 10)) | s_pick[0]);
    want = s_pick[1];
    // The buffer of pass 0 serves pass 2: cleared here, while no CTA reads it
    // any more (all have passed the meeting of pass 1).
    if (d == 1) {
      for (int i = tid; i < kBins; i += kSelectThreads) s_hist[0][i] = 0u;
      __syncthreads();
    }
  }
  // Kept: keys above `prefix`, and the first `want` rows equal to it. Each
  // warp counts the ties and the larger keys of its run of rows, those below
  // n_keep apart. Ties are taken in row order, so from these counts follow,
  // for every warp and every CTA, the ties taken (want less the ties before),
  // the holes and the movers, and where its own begin.
  const int seg = ((mine + 31) / 32 + 31) / 32 * 32;
  const int i_lo = min(mine, warp * seg), i_hi = min(mine, i_lo + seg);
  uint32_t c[4] = {0u, 0u, 0u, 0u};  // ties below n_keep, ties past it, larger below, larger past
  for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < i_hi ? key(i) : 0u;
    const uint32_t tie = __ballot_sync(0xffffffffu, i < i_hi && k == prefix);
    const uint32_t more = __ballot_sync(0xffffffffu, i < i_hi && k > prefix);
    const uint32_t low = __ballot_sync(0xffffffffu, base + i < p.n_keep);
    c[0] += __popc(tie & low);
    c[1] += __popc(tie & ~low);
    c[2] += __popc(more & low);
    c[3] += __popc(more & ~low);
  }
  if (lane < 4) s_warp[lane][warp] = lane == 0 ? c[0] : (lane == 1 ? c[1] : (lane == 2 ? c[2] : c[3]));
  __syncthreads();
  // Holes and movers among `rows_low` rows below n_keep and those past it.
  auto places = [&](uint32_t ties_before, uint32_t t_low, uint32_t t_high, uint32_t m_low, uint32_t m_high,
                    uint32_t rows_low, uint32_t& holes, uint32_t& movers) {
    const uint32_t taken = min(t_low + t_high, want - min(want, ties_before));
    holes = rows_low - m_low - min(taken, t_low);
    movers = m_high + (taken - min(taken, t_low));
  };
  auto rows_below = [&](int first, int last) {  // rows of [first, last) below n_keep
    return static_cast<uint32_t>(max(0, min(last, p.n_keep) - min(first, p.n_keep)));
  };
  auto before_lane = [&](uint32_t x) {  // sum over the lanes before this one
    uint32_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    return inc - x;
  };
  if (warp == 0) {
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = __reduce_add_sync(0xffffffffu, s_warp[j][lane]);
    if (lane == 0) {
      s_count[0] = make_uint2(t[0], t[1]);
      s_count[1] = make_uint2(t[2], t[3]);
    }
  }
  meet();
  if (warp == 0) {  // lane k: CTA k
    uint2 ties = make_uint2(0u, 0u), more = make_uint2(0u, 0u);
    uint32_t holes = 0u, movers = 0u;
    if (lane < ranks) {
      ties = load2(&s_count[0], lane);
      more = load2(&s_count[1], lane);
    }
    const uint32_t ties_before = before_lane(ties.x + ties.y);
    const int first = min(L, lane * per), last = min(L, first + per);
    if (lane < ranks)
      places(ties_before, ties.x, ties.y, more.x, more.y, rows_below(first, last), holes, movers);
    const uint32_t holes_before = before_lane(holes), movers_before = before_lane(movers);
    const uint32_t all = __reduce_add_sync(0xffffffffu, movers);
    if (lane == rank) {
      s_before[0] = ties_before;
      s_before[1] = holes_before;
      s_before[2] = movers_before;
      s_total = all;
    }
  }
  __syncthreads();
  uint32_t e, nh, nm;  // ties, holes, movers before this warp's rows
  {
    const uint32_t t_low = s_warp[0][lane], t_high = s_warp[1][lane];  // lane k: warp k
    const uint32_t ties_before = s_before[0] + before_lane(t_low + t_high);
    const int first = base + min(mine, lane * seg), last = base + min(mine, (lane + 1) * seg);
    uint32_t holes, movers;
    places(ties_before, t_low, t_high, s_warp[2][lane], s_warp[3][lane], rows_below(first, last), holes, movers);
    e = __shfl_sync(0xffffffffu, ties_before, warp);
    nh = s_before[1] + __shfl_sync(0xffffffffu, before_lane(holes), warp);
    nm = s_before[2] + __shfl_sync(0xffffffffu, before_lane(movers), warp);
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i0 = i_lo; i0 < i_hi; i0 += 32) {
    const int i = i0 + lane, r = base + i;
    const bool in = i < i_hi;
    const uint32_t k = in ? key(i) : 0u;
    const uint32_t tie = __ballot_sync(0xffffffffu, in && k == prefix);
    const bool kept = in && (k > prefix || (k == prefix && e + __popc(tie & below) < want));
    e += __popc(tie);
    const bool hole = in && !kept && r < p.n_keep, mover = kept && r >= p.n_keep;
    const uint32_t mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole) dst[nh + __popc(mh & below)] = r;
    if (mover) src[nm + __popc(mm & below)] = r;
    nh += __popc(mh);
    nm += __popc(mm);
  }
  const int total = static_cast<int>(s_total);
  if (lead && tid == 0) p.n_moves[head] = total;
  for (int i = total + rank * kSelectThreads + tid; i < p.n_keep; i += ranks * kSelectThreads) src[i] = dst[i] = -1;
  if constexpr (CLUSTER) cluster_sync();  // no CTA leaves while another may still read its counts
}

struct MoveParams {
  View v;
  const int *n_moves, *src, *dst;
  int stride;  // entries of src and dst per head
  __nv_bfloat16 *k_pages, *v_pages;
  float* weight;
  int* position;
};

constexpr int kMoveThreads = 256;    // moves of a CTA's step, too
constexpr int kMoveMaxCtas = 64;     // of a head
constexpr int kMoveBatch = 4;        // moves a group of lanes has in flight

// The rows lie anywhere, so what counts is how many loads are in flight. A
// CTA takes kMoveThreads moves at a time (67 thousand rows of 16 sequences
// 19.4 us = 3.6 TB/s, and 25 with a group of lanes per move all the way):
// first a thread per move follows move and page to the two rows' places (three
// dependent loads, paid once), then D / 8 lanes copy a row of K and of V,
// kMoveBatch moves at a time.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 4) move_kernel(const MoveParams p) {
  constexpr int LPR = D / 8, GPC = kMoveThreads / LPR;
  __shared__ long long s_from[kMoveThreads], s_to[kMoveThreads];  // row of a pool of K or V rows; -1: none
  const View& v = p.v;
  const int hk = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  pdl_launch_dependents();
  pdl_wait();
  const size_t head = static_cast<size_t>(b) * v.Hk + hk;
  const int n = p.n_moves[head], L = v.cache_len[b];
  for (int i0 = blockIdx.x * kMoveThreads; i0 < p.stride; i0 += gridDim.x * kMoveThreads) {
    const bool in = i0 + tid < p.stride;
    const int from = in ? p.src[head * p.stride + i0 + tid] : 0;  // (beside n: one latency less)
    const int to = in ? p.dst[head * p.stride + i0 + tid] : 0;
    if (n < 0 || n > p.stride || L < 0 || L > v.T) {  // (select writes nothing for a length that does not fit)
      if (blockIdx.x == 0 && tid == 0) atomicOr(&g_status, kStatusRange);
      return;
    }
    if (i0 >= n) return;
    long long a = -1, z = -1;
    if (i0 + tid < n) {
      if (from < 0 || from >= v.T || to < 0 || to >= v.T) {
        atomicOr(&g_status, kStatusRange);
      } else {
        const int pf = page_at(v, b, page_entry(v, from)), pt = page_at(v, b, page_entry(v, to));
        if (pf >= 0 && pt >= 0) {
          a = static_cast<long long>(kv_index(v, pf, page_slot(v, from), hk));
          z = static_cast<long long>(kv_index(v, pt, page_slot(v, to), hk));
          const size_t ta = term_index(v, pf, page_slot(v, from), hk), tz = term_index(v, pt, page_slot(v, to), hk);
          const float w = p.weight[ta];
          const int pos = p.position[ta];
          p.weight[tz] = w;
          p.position[tz] = pos;
        }
      }
    }
    s_from[tid] = a;
    s_to[tid] = z;
    __syncthreads();
    const int count = min(n - i0, kMoveThreads), sub = tid % LPR;
    for (int m0 = tid / LPR; m0 < count; m0 += GPC * kMoveBatch) {
      uint4 kk[kMoveBatch], vv[kMoveBatch];
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int m = m0 + j * GPC;
        if (m >= count || s_from[m] < 0) continue;
        const size_t at = static_cast<size_t>(s_from[m]) * D + sub * 8;
        kk[j] = *reinterpret_cast<const uint4*>(p.k_pages + at);
        vv[j] = *reinterpret_cast<const uint4*>(p.v_pages + at);
      }
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int m = m0 + j * GPC;
        if (m >= count || s_from[m] < 0) continue;
        const size_t at = static_cast<size_t>(s_to[m]) * D + sub * 8;
        *reinterpret_cast<uint4*>(p.k_pages + at) = kk[j];
        *reinterpret_cast<uint4*>(p.v_pages + at) = vv[j];
      }
    }
    __syncthreads();
  }
}

}  // namespace paged
}  // namespace cswattn
