// paged_weigh.cuh -- accumulated attention weight of cached rows:
//   weight[row] += sum over tokens i that see the row, heads h of the group,
//                  of exp(c q_ih . k_row - lse_ih).
//
// The sums run over queries, so the products are taken transposed (a cached
// row is a row of S^T = K Q^T) and each sum stays inside one thread, or four
// lanes. Every cached row belongs to one CTA (or one cluster) of a call, which
// adds in a fixed order and updates the row without atomics: the same call
// gives the same bits.
//
// Two kernels, by a sequence's query rows (new tokens x heads of the group):
//   weigh_rows_kernel   few rows (<= 32): bound by reading K once. Blocks of 64
//     cached rows, dealt out evenly as in the attention of few rows; mma.sync
//     with K as the first operand, the query rows as columns (8 per product).
//   weigh_tile_kernel   many rows: tcgen05, 128 cached rows x 128 query rows
//     per product, thread = cached row; bound by the exponentials.
#pragma once
#include "paged_tile.cuh"

namespace cswattn {
namespace paged {

// ---------------------------------------------------------------- few query rows

struct WeighRowsParams {
  View v;
  float scale_log2;
  int unit, max_rows;
  const __nv_bfloat16* q;
  const float* lse;
  float* weight;
  unsigned long long wait_ns;
};

template <int D>
struct WeighRowsSmem {
  static constexpr int kPanel = kBlk * 128;
  static constexpr int kStage = (D / 64) * kPanel;   // a block of K
  static constexpr int kStages = D == 128 ? 10 : 16;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kOffPre = kOffBar + 8 * (2 * kStages + 2);
  static constexpr int kBytes = kOffPre + 1024;      // and 4 (B + 1) more
  static_assert(kBytes + 4 * (kMaxSeqs + 1) <= 232448, "shared memory per block");
};

constexpr int kWeighGroups = 2;  // groups of 4 warps that take alternate blocks: two blocks' latencies overlap

// NT: products of 8 query rows (max_rows <= 8 NT).
template <int D, int NT>
__global__ void __launch_bounds__(32 * (4 * kWeighGroups + 1), 1)
    weigh_rows_kernel(const __grid_constant__ CUtensorMap tmK, const WeighRowsParams p) {
  using SM = WeighRowsSmem<D>;
  constexpr int NS = SM::kStages, NP = D / 64, kWarps = 4 * kWeighGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* empty = full + NS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NS);
  int* pre = reinterpret_cast<int*>(smem + SM::kOffPre);
  const View& v = p.v;
  const int warp = warp_id(), lane = lane_id(), c = blockIdx.x;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  fill_prefix(v, pre, p.max_rows, c == 0);
  const Deal deal(static_cast<long long>(pre[v.B]) * v.Hk, gridDim.x);
  if (c >= deal.ctas) return;
  Walk w(pre, v.B, v.Hk, deal.begin(c), deal.begin(c + 1));
  const WaitCtx wc{abort_flag, p.wait_ns};

  if (warp == kWarps) {
    // ---------------------------------------------------- producer
    if (lane == 0) prefetch_tmap(&tmK);
    const int boxes = (kBlk / p.unit) * NP;
    const int my_unit = lane / NP, my_panel = lane % NP;
    uint8_t* my_dst = smem + my_panel * SM::kPanel + my_unit * p.unit * 128;
    int stage = 0, use = 0, issued = 0;
    bool ok = true;
    for (; ok && w.valid(); w.next()) {
      Seq s;
      int first;
      seq_load(v, w.b, false, s);
      visible_blocks(v, s, p.max_rows, first);
      const int lo = max(0, s.L - v.W + 1), end = s.L + s.n;
      auto lookup = [&](int t) -> int {
        const int r = (first + t) * kBlk + my_unit * p.unit;
        if (lane >= boxes || r >= end || r + p.unit <= lo) return v.n_pages;
        const int page = page_at(v, w.b, r / v.page_size);
        return page < 0 ? v.n_pages : page;
      };
      int page = lookup(w.t0);
      for (int t = w.t0; t < w.t1; ++t) {
        const int next = t + 1 < w.t1 ? lookup(t + 1) : 0;
        if (use > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], (use - 1) & 1, wc));
          if (!ok) break;
        }
        if (lane == 0) mbar_expect_tx(&full[stage], SM::kStage);
        __syncwarp();
        if (lane < boxes)
          tma_load_4d(&tmK, &full[stage], my_dst + stage * SM::kStage, 64 * my_panel, w.hk,
                      ((first + t) * kBlk + my_unit * p.unit) % v.page_size, page);
        ++issued;
        page = next;
        if (++stage == NS) {
          stage = 0;
          ++use;
        }
      }
    }
    if (lane == 0)
      for (int s = 0; s < NS && s < issued; ++s) drain_wait(&full[s], ((issued - 1 - s) / NS) & 1);
    return;
  }

  // ------------------------------------------------------ sums
  const int group = warp >> 2, key_w = (warp & 3) * 16;  // this warp's 16 rows of a block
  const uint32_t s_base = smem_u32(smem);
  // ldmatrix row and chunk of this lane: matrices (rows 0-7, 8-15) x (chunk, chunk + 1)
  const int a_row = key_w + (lane & 7) + ((lane >> 3) & 1) * 8;
  int at = 0;  // blocks of the CTA so far
  for (; w.valid(); w.next()) {
    Seq s;
    int first;
    seq_load(v, w.b, false, s);
    visible_blocks(v, s, p.max_rows, first);
    const int rows = s.n * v.g, end = s.L + s.n;
    // Query rows as B fragments (column = row), their log-sum-exp and the cached rows they see.
    uint32_t qb[NT][D / 16][2];
    float l2[NT][2];
    int hi[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + (lane >> 2);
      const bool in = r < rows;
      const __nv_bfloat16* src = p.q + (static_cast<size_t>(s.tok0 + (in ? r / v.g : 0)) * v.H + w.hk * v.g +
                                        (in ? r % v.g : 0)) * D + (lane & 3) * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qb[nt][kk][0] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
        qb[nt][kk][1] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = nt * 8 + (lane & 3) * 2 + e;
        const bool on = col < rows;
        const int i = on ? col / v.g : 0;
        hi[nt][e] = on ? s.L + i : -1;  // -1: no row is seen
        l2[nt][e] = on ? p.lse[static_cast<size_t>(s.tok0 + i) * v.H + w.hk * v.g + col % v.g] * 1.4426950408889634f
                       : 0.f;
      }
    }
    for (int t = w.t0; t < w.t1; ++t, ++at) {
      if (at % kWeighGroups != group) continue;
      const int stage = at % NS, use = at / NS;
      const int key0 = (first + t) * kBlk + key_w;
      // The row this lane updates (lanes 0 and 1 of each four), ahead of the products.
      const int key = key0 + (lane >> 2) + (lane & 1) * 8;
      const bool mine = (lane & 3) < 2 && key < end && key > s.L - v.W;
      float* dst = nullptr;
      float old = 0.f;
      if (mine) {
        const int page = page_at(v, w.b, key / v.page_size);
        if (page >= 0) {
          dst = p.weight + term_index(v, page, key % v.page_size, w.hk);
          old = *dst;
        }
      }
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], use & 1, wc))) return;
      const uint32_t kb = s_base + stage * SM::kStage;
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const int chunk = 2 * kk + (lane >> 4);
        uint32_t a[4];
        ldmatrix4<false>(kb + (chunk >> 3) * SM::kPanel + a_row * 128 + (((chunk & 7) ^ (a_row & 7)) << 4), a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(sc[nt], a, qb[nt][kk][0], qb[nt][kk][1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = key0 + (lane >> 2) + (e >> 1) * 8, h = hi[nt][e & 1];
          const float x = ex2(fmaf(sc[nt][e], p.scale_log2, -l2[nt][e & 1]));
          sum[e >> 1] += (k <= h && k > h - v.W) ? x : 0.f;  // a select: what lies in unseen rows does not matter
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
        sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      }
      if (dst) *dst = old + ((lane & 1) ? sum[1] : sum[0]);
    }
  }
}

// ---------------------------------------------------------------- many query rows

struct WeighTileParams {
  View v;
  float scale_log2;
  int unit, tpt, short_rows;
  const float* lse;
  float* weight;
  unsigned long long wait_ns;
};

constexpr int kWeighThreads = 320;  // producer, MMA issuer, 8 warps of sums
constexpr int kWeighCluster = 4;    // CTAs that may share a unit's query tiles
constexpr int kWeighCtas = 2 * kSMs;  // two per SM: one's products and copies under the other's sums
constexpr int kWeighWhole = 6;      // units per CTA from which each takes whole ones

template <int D>
struct WeighTileSmem {
  static constexpr int kPanel = 128 * 128;
  static constexpr int kOp = (D / 64) * kPanel;
  static constexpr int kOffQ = kOp;                 // 2 slots
  static constexpr int kOffLse = 3 * kOp;           // [2][128] float
  static constexpr int kOffSum = kOffLse + 1024;    // [2][kWeighCluster - 1][128] float: the other CTAs' sums
  static constexpr int kOffHalf = kOffSum + 2 * (kWeighCluster - 1) * 512;  // [128] float: the second half's sums
  static constexpr int kOffBar = kOffHalf + 512;
  static constexpr int kOffPre = kOffBar + 8 * 18;  // int [B + 1]
  static constexpr int kBytes = kOffPre + 1024;     // and 4 (B + 1) more; two CTAs fit an SM
  static_assert(kBytes + 4 * (kMaxSeqs + 1) <= 232448, "shared memory per block");
};

// Shared memory of another CTA of the cluster: address, store, arrival; and
// the wait that sees what was stored before the arrivals.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, const WaitCtx& w) {
  if (!mbar_wait(bar, parity, w)) return false;
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
  return true;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// CTA (or cluster of kWeighCluster) = one 128-row tile of cached rows after
// another; the query tiles that see it stream past. With a cluster, CTA `rank`
// takes every kWeighCluster-th query tile; the others write their sums into
// rank 0's shared memory (two buffers, handed back by an arrival), which adds
// them in the order of the ranks. All threads meet at the cluster's barrier
// once at the start (barriers set up) and once at the end (no CTA leaves
// while another may still reach its shared memory); no path skips either.
template <int D>
__global__ void __launch_bounds__(kWeighThreads, 2) __cluster_dims__(kWeighCluster, 1, 1)
    weigh_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ WeighTileParams p) {
  using SM = WeighTileSmem<D>;
  constexpr int NP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  float* s_lse = reinterpret_cast<float*>(smem + SM::kOffLse);
  float* s_sum = reinterpret_cast<float*>(smem + SM::kOffSum);  // [2][kWeighCluster - 1][128]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* k_empty = k_full + 1;
  uint64_t* q_full = k_full + 2;    // [2]
  uint64_t* q_empty = k_full + 4;   // [2]
  uint64_t* s_full = k_full + 6;    // [2] S^T buffers
  uint64_t* s_empty = k_full + 8;   // [2] (256 arrivals)
  uint64_t* mma_done = k_full + 10;
  uint64_t* sum_full = k_full + 11;  // [2] rank 0: the others' sums have come
  uint64_t* sum_free = k_full + 13;  // [2] the others: rank 0 has read the buffer
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(k_full + 16);
  int* pre = reinterpret_cast<int*>(smem + SM::kOffPre);
  const View& v = p.v;
  const int warp = warp_id(), lane = lane_id();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 256);
      mbar_init(&sum_full[i], 128 * (kWeighCluster - 1));
      mbar_init(&sum_free[i], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  pdl_wait();
  // Tiles of cached rows of each long sequence, and their running sum.
  for (int b = threadIdx.x; b < v.B; b += kWeighThreads) {
    Seq s;
    seq_load(v, b, blockIdx.x == 0, s);
    int lo, hi, n = 0;
    if (is_long(v, s, p.short_rows)) {
      token_blocks(v, s, 0, s.n, lo, hi);
      n = hi - lo + 1;
    }
    pre[b + 1] = n;
  }
  if (threadIdx.x == 0) pre[0] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) {
    int run = 0;
    for (int b0 = 0; b0 < v.B; b0 += 32) {
      const int b = b0 + lane;
      int x = b < v.B ? pre[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < v.B) pre[b + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  cluster_sync();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.wait_ns};
  const long long units = static_cast<long long>(pre[v.B]) * v.Hk;
  const bool shared = units < static_cast<long long>(kWeighWhole) * gridDim.x;
  const int rank = shared ? blockIdx.x % kWeighCluster : 0, ranks = shared ? kWeighCluster : 1;
  const long long first_unit = shared ? blockIdx.x / kWeighCluster : blockIdx.x;
  const long long stride = shared ? gridDim.x / kWeighCluster : gridDim.x;

  // Unit u: sequence b, KV head hk, tile of cached rows [k0, k0 + 128); this
  // CTA's query tiles are q0, q0 + ranks, ... <= q1 (of tpt tokens each).
  struct Unit {
    int b, hk, k0, q0, q1;
    Seq s;
  };
  auto unit_at = [&](long long u) -> Unit {
    int lo = 0, hi = v.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (static_cast<long long>(pre[mid]) * v.Hk <= u) lo = mid;
      else hi = mid;
    }
    Unit x;
    x.b = lo;
    seq_load(v, lo, false, x.s);
    const int rem = static_cast<int>(u - static_cast<long long>(pre[lo]) * v.Hk), cnt = pre[lo + 1] - pre[lo];
    x.hk = rem / cnt;
    x.k0 = ((max(0, x.s.L - v.W + 1) >> 7) + rem % cnt) * 128;
    // tokens i with k <= L + i and L + i - W < k for some k of the tile
    const int i_lo = max(0, x.k0 - x.s.L);
    const long long i_hi = min(static_cast<long long>(x.s.n) - 1, static_cast<long long>(x.k0) + 127 - x.s.L + v.W - 1);
    x.q0 = i_lo / p.tpt + rank;
    x.q1 = i_hi < i_lo ? -1 : static_cast<int>(i_hi) / p.tpt;
    return x;
  };
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
    }
    const int boxes = (128 / p.unit) * NP;
    const int my_unit = lane / NP, my_panel = lane % NP;
    int nk = 0, nq = 0;
    for (long long u = first_unit; ok && u < units; u += stride) {
      const Unit x = unit_at(u);
      if (x.q0 > x.q1) continue;
      const int lo = max(0, x.s.L - v.W + 1), end = x.s.L + x.s.n;
      int page = v.n_pages;
      const int r = x.k0 + my_unit * p.unit;
      if (lane < boxes && r < end && r + p.unit > lo) {
        page = page_at(v, x.b, r / v.page_size);
        if (page < 0) page = v.n_pages;
      }
      if (nk > 0) ok = __all_sync(0xffffffffu, mbar_wait(k_empty, (nk - 1) & 1, wc));
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(k_full, SM::kOp);
      __syncwarp();
      if (lane < boxes)
        tma_load_4d(&tmK, k_full, smem + my_panel * SM::kPanel + my_unit * p.unit * 128, 64 * my_panel, x.hk,
                    r % v.page_size, page);
      ++nk;
      if (lane == 0) {
        for (int q = x.q0; ok && q <= x.q1; q += ranks, ++nq) {
          const int slot = nq & 1;
          if (nq > 1) ok = mbar_wait(&q_empty[slot], ((nq >> 1) - 1) & 1, wc);
          if (!ok) break;
          mbar_expect_tx(&q_full[slot], p.tpt * v.g * 128 * NP);
          for (int pn = 0; pn < NP; ++pn)
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem + SM::kOffQ + slot * SM::kOp + pn * SM::kPanel)),
                "l"(reinterpret_cast<uint64_t>(&tmQ)), "r"(smem_u32(&q_full[slot])), "r"(64 * pn), "r"(x.hk * v.g),
                "r"(x.s.tok0 + q * p.tpt)
                : "memory");
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    if (lane == 0) {  // every issued copy has landed
      if (nk > 0) drain_wait(k_full, (nk - 1) & 1);
      for (int i = 0; i < 2 && i < nq; ++i) drain_wait(&q_full[i], ((nq - 1 - i) >> 1) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // -------------------------------------------------- S^T = K Q^T
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      const uint64_t dK = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + SM::kOffQ), 16, 1024);
      int nk = 0, nq = 0;
      for (long long u = first_unit; ok && u < units; u += stride) {
        const Unit x = unit_at(u);
        if (x.q0 > x.q1) continue;
        ok = mbar_wait(k_full, nk & 1, wc);
        ++nk;
        for (int q = x.q0; ok && q <= x.q1; q += ranks, ++nq) {
          const int buf = nq & 1;
          ok = mbar_wait(&q_full[buf], (nq >> 1) & 1, wc) &&
               (nq < 2 || mbar_wait(&s_empty[buf], ((nq >> 1) - 1) & 1, wc));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t off = static_cast<uint64_t>(((kk >> 2) * SM::kPanel + (kk & 3) * 32) >> 4);
            mma_ss(tmem + buf * 128u, dK + off, dQ + static_cast<uint64_t>((buf * SM::kOp) >> 4) + off, idS,
                   kk > 0 ? 1u : 0u);
          }
          mma_commit(&q_empty[buf]);
          mma_commit(&s_full[buf]);
        }
        if (ok) mma_commit(k_empty);
      }
      mma_commit(mma_done);
      drain_wait(mma_done, 0);
    }
  } else {
    // ---------------------------------------------------- sums: two threads per cached row
    // Warps 2-5 take columns 0-63 of each tile, warps 6-9 columns 64-127.
    const int quad = warp & 3, r = quad * 32 + lane, half = warp >= 6 ? 1 : 0;
    float* s_half = reinterpret_cast<float*>(smem + SM::kOffHalf);
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const float c2 = p.scale_log2;
    int nq = 0, nu = 0;
    for (long long u = first_unit; ok && u < units; u += stride, ++nu) {
      const Unit x = unit_at(u);
      const int key = x.k0 + r, end = x.s.L + x.s.n;
      const bool mine = key < end && key > x.s.L - v.W;
      float total = 0.f;
      // Row r of query tile q: its log-sum-exp in log2 units, negated.
      auto row_term = [&](int q) -> float {
        const int i = q * p.tpt + r / v.g;
        return q <= x.q1 && r < p.tpt * v.g && i < x.s.n
                   ? p.lse[static_cast<size_t>(x.s.tok0 + i) * v.H + x.hk * v.g + r % v.g] * -1.4426950408889634f
                   : 0.f;
      };
      float term = half == 0 ? row_term(x.q0) : 0.f;
      for (int q = x.q0; ok && q <= x.q1; q += ranks, ++nq) {
        const int buf = nq & 1, i0 = q * p.tpt;
        if (half == 0) {
          s_lse[buf * 128 + r] = term;
          term = row_term(q + ranks);  // the next tile's, under this one's sums
        }
        ok = named_bar_and(1, 256, mbar_wait(&s_full[buf], (nq >> 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        // Columns [a, b] are the query rows that see this cached row:
        // key - L <= token < key - L + W.
        const int cols = min(p.tpt, x.s.n - i0) * v.g;
        const long long lo_col = (static_cast<long long>(key) - x.s.L - i0) * v.g;
        const long long hi_col = (static_cast<long long>(key) - x.s.L + v.W - i0) * v.g - 1;
        const int a = static_cast<int>(max(0ll, lo_col));
        const int b = static_cast<int>(min(static_cast<long long>(cols) - 1, hi_col));
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const int h = 2 * half + h2;
          if (!__any_sync(0xffffffffu, a <= 32 * h + 31 && b >= 32 * h)) continue;  // nobody sees these
          uint32_t sv[32];
          tmem_ld32(tmem + lane_off + buf * 128 + h * 32, sv);
          tmem_ld_wait();
          const bool all = __all_sync(0xffffffffu, a <= 32 * h && b >= 32 * h + 31);
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 l4 = *reinterpret_cast<const float4*>(&s_lse[buf * 128 + h * 32 + e4 * 4]);
            const float x0 = ex2(fmaf(__uint_as_float(sv[4 * e4]), c2, l4.x));
            const float x1 = ex2(fmaf(__uint_as_float(sv[4 * e4 + 1]), c2, l4.y));
            const float x2 = ex2(fmaf(__uint_as_float(sv[4 * e4 + 2]), c2, l4.z));
            const float x3 = ex2(fmaf(__uint_as_float(sv[4 * e4 + 3]), c2, l4.w));
            if (all) {
              part[0] += x0;
              part[1] += x1;
              part[2] += x2;
              part[3] += x3;
            } else {  // a select: what lies in unseen places does not matter
              const int e = 32 * h + 4 * e4;
              part[0] += (e >= a && e <= b) ? x0 : 0.f;
              part[1] += (e + 1 >= a && e + 1 <= b) ? x1 : 0.f;
              part[2] += (e + 2 >= a && e + 2 <= b) ? x2 : 0.f;
              part[3] += (e + 3 >= a && e + 3 <= b) ? x3 : 0.f;
            }
          }
        }
        total += (part[0] + part[1]) + (part[2] + part[3]);
        tc_fence_before();
        mbar_arrive(&s_empty[buf]);
      }
      if (!ok) break;
      // The two halves of a row meet; warps 2-5 go on with its sum.
      if (half == 1) s_half[r] = total;
      named_bar(1, 256);
      if (half == 0) {
        total += s_half[r];
        const int buf = nu & 1;
        float* slot = s_sum + buf * (kWeighCluster - 1) * 128 + r;
        if (shared && rank > 0) {
          ok = named_bar_and(2, 128, nu < 2 || mbar_wait(&sum_free[buf], ((nu >> 1) - 1) & 1, wc));
          if (ok) {
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(slot + (rank - 1) * 128, 0)), "f"(total)
                         : "memory");
            cluster_arrive(cluster_addr(&sum_full[buf], 0));
          }
        } else if (shared) {
          ok = named_bar_and(2, 128, cluster_wait(&sum_full[buf], (nu >> 1) & 1, wc));
          if (ok) {
#pragma unroll
            for (int k = 0; k < kWeighCluster - 1; ++k) total += slot[k * 128];
            named_bar(2, 128);  // every thread has read the buffer
            if (r > 0 && r < kWeighCluster) cluster_arrive(cluster_addr(&sum_free[buf], r));
          }
        }
        if (ok && rank == 0 && mine) {
          const int page = page_at(v, x.b, key / v.page_size);
          if (page >= 0) p.weight[term_index(v, page, key % v.page_size, x.hk)] += total;
        }
      }
      ok = named_bar_and(1, 256, ok);  // all leave together when a wait ran out
    }
  }
  __syncwarp();
  cluster_sync();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

}  // namespace paged
}  // namespace cswattn
