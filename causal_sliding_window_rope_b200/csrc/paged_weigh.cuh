// paged_weigh.cuh -- accumulated attention weight of cached rows:
//   weight[row] += sum over tokens i that see the row, heads h of the group,
//                  of exp(c q_ih . k_row - lse_ih).
//
// The sums run over queries, so the products are taken transposed (a cached
// row is a row of S^T = K Q^T) and each sum stays inside one thread, or four
// lanes. Every cached row belongs to one CTA of a call (the shares of a unit
// that is cut are added by a kernel of their own), which adds in a fixed order
// and updates the row without atomics: the same call gives the same bits.
//
// Two kernels, by the most query rows a sequence of the call may have (new
// tokens x heads of the group):
//   weigh_rows_kernel   few (<= 32): bound by reading K once and by the start
//     of a CTA. Blocks of 64 cached rows, dealt out evenly as in the attention
//     of few rows; mma.sync with K as the first operand, the query rows as
//     columns (8 per product). 32 ragged sequences of up to 2048 rows 12.5 us.
//   weigh_tile_kernel   many: tcgen05, 128 cached rows x 128 query rows per
//     product, two threads per cached row; no unit is saturated (the exponentials',
//     one per score, is 55 % busy and would take 33 us alone, issue slots 46 %,
//     the tensor pipe 24 %): a tile's chain of waits bounds it. 2213 tokens of 16 heads on 4 over
//     11081 rows 64 us = 530 TFLOP/s. A call with a chunk runs it for its
//     single tokens too.
#pragma once
#include "paged_tile.cuh"

namespace cswattn {
namespace paged {

// ---------------------------------------------------------------- few query rows

struct WeighRowsParams {
  View v;
  float scale_log2;
  int unit;
  const __nv_bfloat16* q;
  const float* lse;
  float* weight;
  unsigned long long wait_ns;
};

constexpr int kWeighRuns = 2 * kSMs;  // CTAs of weigh_tile_kernel, two per SM

template <int D>
struct WeighRowsSmem {
  static constexpr int kPanel = kBlk * 128;
  static constexpr int kStage = (D / 64) * kPanel;   // a block of K
  // (128 KB in flight on an SM; 12 slots at head_dim 128: step 12.5 -> 13.0 us,
  // 32 sequences of 8192 rows alike)
  static constexpr int kStages = D == 128 ? 8 : 16;
  static constexpr int kOffBar = kStages * kStage;
  static constexpr int kOffPre = kOffBar + 8 * (2 * kStages + 2);
  static constexpr int kBytes = kOffPre + 1024;      // and 4 (B + 1) more
  static_assert(kBytes + 4 * (kMaxSeqs + 1) <= 232448, "shared memory per block");
};

// Groups of 4 warps that take the blocks in turn, so that the latencies of
// several blocks (page, old weight) overlap: as many as the registers allow.
template <int NT>
struct WeighGroups {
  static constexpr int value = NT <= 2 ? 4 : 2;
};

// NT: products of 8 query rows; a sequence has at most 8 NT (max_new times the heads of a group).
template <int D, int NT>
__global__ void __launch_bounds__(32 * (4 * WeighGroups<NT>::value + 1), 1)
    weigh_rows_kernel(const __grid_constant__ CUtensorMap tmK, const WeighRowsParams p) {
  using SM = WeighRowsSmem<D>;
  constexpr int NS = SM::kStages, NP = D / 64, kGroups = WeighGroups<NT>::value, kWarps = 4 * kGroups;
  // A wait for a slot's phase parity returns too while the phase before it is
  // still open. A group waits for its own blocks only, so a slot's uses must
  // all be one group's: that of its next block has then seen its last one land.
  static_assert(NS % kGroups == 0, "a slot's blocks belong to one group of warps");
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
  fill_prefix(v, pre, c == 0);
  const Deal deal = deal_out(v, pre, gridDim.x, c, nullptr);
  if (deal.at >= deal.end) return;
  Walk w(deal);
  const WaitCtx wc{abort_flag, p.wait_ns};

  if (warp == kWarps) {
    // ---------------------------------------------------- producer
    if (lane == 0) prefetch_tmap(&tmK);
    const int boxes = kBlk / p.unit * NP;  // as in rows_kernel
    const int my_unit = lane / NP, my_panel = lane % NP;
    uint8_t* my_dst = smem + my_panel * SM::kPanel + my_unit * p.unit * 128;
    int stage = 0, use = 0, issued = 0;
    bool ok = true;
    for (; ok && w.valid(); w.next()) {
      Seq s;
      int first;
      seq_load(v, w.b, false, s);
      visible_blocks(v, s, first);
      UnitPages up(v, w.b, s, first * kBlk + my_unit * p.unit, kBlk, p.unit);
      for (int t = w.t0; t < w.t1; ++t) {
        const int page = up.page(t, lane < boxes);
        if (use > 0) ok = __all_sync(0xffffffffu, mbar_wait(&empty[stage], (use - 1) & 1, wc));
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&full[stage], SM::kStage);
        __syncwarp();
        if (lane < boxes)
          tma_load_4d(&tmK, &full[stage], my_dst + stage * SM::kStage, 64 * my_panel, w.hk, up.slot(t), page);
        ++issued;
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
    // Pairs of fewer blocks than there are groups: only the groups that have
    // one load the query rows, the others go on to the next pair.
    if ((group - at % kGroups + kGroups) % kGroups >= w.t1 - w.t0) {
      at += w.t1 - w.t0;
      continue;
    }
    Seq s;
    int first;
    seq_load(v, w.b, false, s);
    visible_blocks(v, s, first);
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
      if (at % kGroups != group) continue;
      const int stage = at % NS, use = at / NS;
      const int key0 = (first + t) * kBlk + key_w;
      // The row this lane updates (lanes 0 and 1 of each four), ahead of the products.
      const int key = key0 + (lane >> 2) + (lane & 1) * 8;
      const bool mine = (lane & 3) < 2 && key < end && key > s.L - v.W;
      float* dst = nullptr;
      float old = 0.f;
      if (mine) {
        const int page = page_at(v, w.b, page_entry(v, key));
        if (page >= 0) {
          dst = p.weight + term_index(v, page, page_slot(v, key), w.hk);
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
  int unit, tpt;
  Plan* plan;
  int* seqs;
  const float* lse;
  float* weight;
  float* part;  // (2 kWeighRuns, 128): sums of cut units
  unsigned long long wait_ns;
};

constexpr int kWeighThreads = 320;  // producer, MMA issuer, 8 warps of sums

template <int D>
struct WeighTileSmem {
  static constexpr int kPanel = 128 * 128;
  static constexpr int kOp = (D / 64) * kPanel;
  static constexpr int kTerms = 8;                   // buffers of the query rows' terms
  static constexpr int kOffQ = kOp;                  // 2 slots
  static constexpr int kOffTerm = 3 * kOp;           // [kTerms][128] float
  static constexpr int kOffHalf = kOffTerm + kTerms * 512;   // [2][128] float: the second half's sums
  static constexpr int kOffBar = kOffHalf + 1024;
  static constexpr int kBytes = kOffBar + 8 * (18 + kTerms) + 1024;
  static_assert(2 * (kBytes + 1024) <= 233472, "two blocks per SM");
};

// The deal's units are tiles of 128 cached rows, their blocks the query tiles
// that see them. K stays, the query tiles stream past: S^T = K Q^T in one of
// two TMEM buffers, and two threads per cached row add up 64 columns each.
// Two CTAs per SM, so that one's products, copies and ends of units run under
// the other's sums. The sums of a cut unit go to `part`.
template <int D>
__global__ void __launch_bounds__(kWeighThreads, 2)
    weigh_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ WeighTileParams p) {
  using SM = WeighTileSmem<D>;
  constexpr int NP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  float* s_term = reinterpret_cast<float*>(smem + SM::kOffTerm);
  float* s_half = reinterpret_cast<float*>(smem + SM::kOffHalf);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* k_empty = k_full + 1;
  uint64_t* q_full = k_full + 2;     // [2]
  uint64_t* q_empty = k_full + 4;    // [2]
  uint64_t* s_full = k_full + 6;     // [2] S^T buffers
  uint64_t* s_empty = k_full + 8;    // [2] read by all sums (256 arrivals)
  uint64_t* h_full = k_full + 10;    // [2] the second half's sums written (128 arrivals)
  uint64_t* h_empty = k_full + 12;   // [2] ... and read (128 arrivals)
  uint64_t* mma_done = k_full + 14;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(k_full + 15);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(k_full + 16);
  uint64_t* t_full = k_full + 17;    // [kTerms] -lse log2(e) of a tile's query rows written (32 arrivals)
  const View& v = p.v;
  const int warp = warp_id(), lane = lane_id(), c = blockIdx.x;
  if (threadIdx.x == 0) {
    mbar_init(k_full, 1);
    mbar_init(k_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 256);
      mbar_init(&h_full[i], 128);
      mbar_init(&h_empty[i], 128);
    }
    for (int i = 0; i < SM::kTerms; ++i) mbar_init(&t_full[i], 32);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __shared__ Run run;
  static_assert(kPlanSmem <= SM::kOffTerm, "the plan's scratch lies where the tiles will");
  pdl_wait();
  find_run(v, RowUnits{p.tpt}, gridDim.x, c, p.plan, p.seqs, smem, &run);
  if (run.left == 0) return;  // uniform over the CTA, before TMEM is taken
  fence_proxy_async_smem();   // the scratch is written, the copies of the tiles come next
  if (warp == 1) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Not before: a successor that takes tensor memory ahead of its wait for this
  // kernel, beside a CTA that has not taken its own yet, would block it.
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{abort_flag, p.wait_ns};
  UnitWalk<RowUnits> w(v, RowUnits{p.tpt}, run, p.seqs);
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------- producer
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
    }
    const int boxes = (128 / p.unit) * NP;
    const int my_unit = lane / NP, my_panel = lane % NP;
    int q_tok[4], q_head[4];  // token of the tile and head of the group of this lane's query rows
    bool q_in[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int qr = lane + 32 * e;
      q_tok[e] = qr / v.g;
      q_head[e] = qr % v.g;
      q_in[e] = qr < p.tpt * v.g;
    }
    int nk = 0, nq = 0;
    for (; ok && w.valid(); w.next()) {
      UnitPages up(v, w.seq(), w.s, w.units.first_row(v, w.s, w.u) + my_unit * p.unit, 128, p.unit);
      const int page = up.page(0, lane < boxes);
      if (nk > 0) ok = __all_sync(0xffffffffu, mbar_wait(k_empty, (nk - 1) & 1, wc));
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(k_full, SM::kOp);
      __syncwarp();
      if (lane < boxes)
        tma_load_4d(&tmK, k_full, smem + my_panel * SM::kPanel + my_unit * p.unit * 128, 64 * my_panel, w.hk,
                    up.slot(0), page);
      ++nk;
      // Terms of the query rows lane, lane + 32, ... of a tile: loaded one tile
      // ahead, written behind the wait for the tile's slot, which needs no
      // barrier of their own: tile nq - 2 has been multiplied, so the sums had
      // taken tile nq - 4 before, and had left the terms up to tile nq - 5.
      static_assert(SM::kTerms >= 5, "terms' buffers");
      float term[4];
      auto load_terms = [&](int t) {
        const int i0 = (w.first + t) * p.tpt;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool in = q_in[e] && i0 + q_tok[e] < w.s.n;
          term[e] = in ? p.lse[static_cast<size_t>(w.s.tok0 + i0 + q_tok[e]) * v.H + w.hk * v.g + q_head[e]] : 0.f;
        }
      };
      load_terms(w.t0);
      for (int t = w.t0; t < w.t1; ++t, ++nq) {
        const int slot = nq & 1, tb = nq % SM::kTerms;
        if (nq > 1) ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[slot], ((nq >> 1) - 1) & 1, wc));
        if (!ok) break;
        if (lane == 0) {
          mbar_expect_tx(&q_full[slot], p.tpt * v.g * 128 * NP);
          for (int pn = 0; pn < NP; ++pn)
            tma_load_3d(&tmQ, &q_full[slot], smem + SM::kOffQ + slot * SM::kOp + pn * SM::kPanel, 64 * pn, w.hk * v.g,
                        w.s.tok0 + (w.first + t) * p.tpt);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) s_term[tb * 128 + lane + 32 * e] = term[e] * -1.4426950408889634f;
        mbar_arrive(&t_full[tb]);
        if (t + 1 < w.t1) load_terms(t + 1);
      }
    }
    if (lane == 0) {  // every issued copy has landed
      if (nk > 0) drain_wait(k_full, (nk - 1) & 1);
      for (int i = 0; i < 2 && i < nq; ++i) drain_wait(&q_full[i], ((nq - 1 - i) >> 1) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------- S^T = K Q^T
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);
      const uint64_t dK = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + SM::kOffQ), 16, 1024);
      int nk = 0, nq = 0;
      for (; ok && w.valid(); w.next(), ++nk) {
        ok = mbar_wait(k_full, nk & 1, wc);
        for (int t = w.t0; ok && t < w.t1; ++t, ++nq) {
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
    __syncwarp();
  } else {
    // ---------------------------------------------------- sums: two threads per cached row
    // Warps 2-5 take columns 0-63 of each tile, warps 6-9 columns 64-127.
    const int quad = warp & 3, r = quad * 32 + lane, half = warp >= 6 ? 1 : 0;
    const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + 64u * half;
    const float c2 = p.scale_log2;
    int nq = 0, nu = 0;
    for (; ok && w.valid(); w.next(), ++nu) {
      const int key = w.units.first_row(v, w.s, w.u) + r, end = w.s.L + w.s.n;
      const bool whole = w.whole();
      // The row this thread updates: its place and old weight, under the first products.
      float* place = nullptr;
      float old = 0.f;
      if (half == 0) {
        if (!whole) {
          place = p.part + static_cast<size_t>(2 * c + (nu == 0 ? 0 : 1)) * 128 + r;
        } else if (key < end && key > w.s.L - v.W) {
          const int page = page_at(v, w.seq(), page_entry(v, key));
          if (page >= 0) {
            place = p.weight + term_index(v, page, page_slot(v, key), w.hk);
            old = *place;
          }
        }
      }
      float total = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++nq) {
        const int buf = nq & 1, i0 = (w.first + t) * p.tpt;
        // Columns [a, b] of this half are the query rows that see this cached
        // row: key - L <= token < key - L + W.
        // (rows and windows are below 2^20, g at most 128: 32 bits hold the products)
        const int past = key - w.s.L - i0;
        const int a = max(0, past * v.g) - 64 * half;
        const int b = min(min(p.tpt, w.s.n - i0) * v.g, (past + v.W) * v.g) - 1 - 64 * half;
        ok = __all_sync(0xffffffffu, mbar_wait(&t_full[nq % SM::kTerms], (nq / SM::kTerms) & 1, wc) &&
                                         mbar_wait(&s_full[buf], (nq >> 1) & 1, wc));
        if (!ok) break;
        tc_fence_after();
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t sv[2][32];
        tmem_ld32(tS + buf * 128, sv[0]);
        tmem_ld32(tS + buf * 128 + 32, sv[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(&s_empty[buf]);  // the scores are in registers: the next product may overwrite them
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!__any_sync(0xffffffffu, a <= 32 * h + 31 && b >= 32 * h)) continue;  // nobody sees these
          const bool all = __all_sync(0xffffffffu, a <= 32 * h && b >= 32 * h + 31);
#pragma unroll
          for (int e4 = 0; e4 < 8; ++e4) {
            const float4 l4 = *reinterpret_cast<const float4*>(&s_term[nq % SM::kTerms * 128 + 64 * half + h * 32 + e4 * 4]);
            const float x0 = ex2(fmaf(__uint_as_float(sv[h][4 * e4]), c2, l4.x));
            const float x1 = ex2(fmaf(__uint_as_float(sv[h][4 * e4 + 1]), c2, l4.y));
            const float x2 = ex2(fmaf(__uint_as_float(sv[h][4 * e4 + 2]), c2, l4.z));
            const float x3 = ex2(fmaf(__uint_as_float(sv[h][4 * e4 + 3]), c2, l4.w));
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
      }
      if (!ok) break;
      // The second half hands its sum over; the first adds and writes.
      const int hb = nu & 1;
      if (half == 1) {
        ok = __all_sync(0xffffffffu, nu < 2 || mbar_wait(&h_empty[hb], ((nu >> 1) - 1) & 1, wc));
        if (!ok) break;
        s_half[hb * 128 + r] = total;
        mbar_arrive(&h_full[hb]);
      } else {
        ok = __all_sync(0xffffffffu, mbar_wait(&h_full[hb], (nu >> 1) & 1, wc));
        if (!ok) break;
        total += s_half[hb * 128 + r];
        mbar_arrive(&h_empty[hb]);
        if (place) *place = whole ? old + total : total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// CTA = a boundary between two CTAs' runs: the unit cut there gets its shares
// in the order of the CTAs that have them.
__global__ void __launch_bounds__(128) weigh_join_kernel(const __grid_constant__ WeighTileParams p) {
  pdl_launch_dependents();
  pdl_wait();
  Cut cut;
  if (!cut.find(p.plan, blockIdx.x + 1) || cut.nth != 0) return;
  const View& v = p.v;
  const Seq& s = cut.s;
  const int key = RowUnits{p.tpt}.first_row(v, s, cut.st.unit) + threadIdx.x;
  if (key >= s.L + s.n || key <= s.L - v.W) return;
  const int page = page_at(v, cut.b, page_entry(v, key));
  if (page < 0) return;
  float total = 0.f;
#pragma unroll 4
  for (int k = 0; k < cut.n; ++k) total += p.part[static_cast<size_t>(cut.slot(k)) * 128 + threadIdx.x];
  p.weight[term_index(v, page, page_slot(v, key), cut.st.hk)] += total;
}

}  // namespace paged
}  // namespace cswattn
