// paged_tile.cuh -- paged attention of calls in which some sequence has many
// query rows (a prompt's chunk): tcgen05 tensor cores, 128-row tiles.
//
// A tile's 128 rows are tokens x heads of one KV head's group (row = token in
// the tile * g + head in the group; 128 / g tokens), so every head that reads
// a K or V row shares the one copy of it; a unit of work is two consecutive
// tiles of one (sequence, KV head), which share the blocks of 128 cached rows
// too. The units' blocks in a row are dealt out evenly to one CTA per SM, as
// in the kernel of few rows (a unit is cut where a CTA's run ends; its
// partial outputs go to the workspace and join_kernel joins them), so
// neither ragged chunks nor the causal edge nor a last wave leave SMs idle.
//
// Roles (12 warps), as in the dense forward:
//   warp 0      producer: the units' Q tiles and their K and V blocks, through
//               one 5-slot ring; every lane copies one box (a page unit of
//               rows x 64 columns); units that no token sees are read past the
//               pool's end, which fills zeros
//   warp 1      TMEM owner, MMA issuer
//   warps 4-7   softmax of tile 0, warps 8-11 of tile 1: thread = query row
// TMEM (512 columns): S0 | S1 | O0 | O1. Per block: S = Q K^T, P (bf16) over
// the S columns, O += P V, in the order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
// so that one tile's softmax overlaps the other's products. The barriers'
// phases run on from unit to unit, and the next unit's first S is issued
// while the last one's output is still being written.
// Bound by the chain of a tile (S, softmax, P V, next S: about 3200 cycles a
// block, the products 2050 of them) and, in long runs, by the power limit
// (1.6 GHz): 2 x 2048 tokens of 16 heads on 4 over 8192 rows 245 us = 980
// TFLOP/s (0.60 of the burst, 0.70 of the sustained rate of a matrix product).
// Short chunks are bound by latency: lengths, page table, first copy and first
// block, 18 thousand cycles of the 33 of a CTA with four blocks.
// Two warps that issue, one per tile, let the tiles fall into step: 302 us.
#pragma once
#include "paged_rows.cuh"

namespace cswattn {
namespace paged {

constexpr int kTileThreads = 384;
constexpr int kTileRegLo = 80, kTileRegHi = 208;
static_assert(128 * kTileRegLo + 256 * kTileRegHi <= kTileThreads * 168, "register budget");

struct TileParams {
  View v;
  float scale_log2;
  int unit;        // rows of a K or V box
  int tpt;         // tokens per tile: 128 / g
  Plan* plan;
  int* seqs;
  __nv_bfloat16* O;
  float* lse;
  float* part_o;     // (2 kSMs, 256, D)
  float2* part_ml;   // (2 kSMs, 256)
  unsigned long long wait_ns;
};

// The walk, with the blocks [lo, hi] of the segment that tile X (0 or 1) of the unit has.
struct TileWalk : UnitWalk<TokenUnits> {
  __device__ TileWalk(const TileParams& p, const Run& run)
      : UnitWalk<TokenUnits>(p.v, TokenUnits{p.tpt}, run, p.seqs) {}
  __device__ bool tokens(int X) const { return (2 * u + X) * units.tpt < s.n; }
  __device__ bool tile(int X, int& lo, int& hi) const {
    const int i0 = (2 * u + X) * units.tpt;
    if (i0 >= s.n) return false;
    token_blocks(v, s, i0, min(s.n, i0 + units.tpt), lo, hi);
    lo = max(lo, first + t0);
    hi = min(hi, first + t1 - 1);
    return lo <= hi;
  }
};

template <int D>
struct TileSmem {
  static constexpr int kPanel = 128 * 128;       // 128 rows x 64 columns
  static constexpr int kOp = (D / 64) * kPanel;  // a Q tile, a block of K or V
  static constexpr int kSlots = D == 128 ? 5 : 8;
  static constexpr int kOffKV = 2 * kOp;
  static constexpr int kOffBar = kOffKV + kSlots * kOp;
  static constexpr int kBytes = kOffBar + 8 * (2 * kSlots + 12) + 1024;
  static_assert(kBytes <= 232448, "shared memory per block");
};

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TileParams p) {
  using SM = TileSmem<D>;
  constexpr int NS = SM::kSlots, NP = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);  // [NS]
  uint64_t* kv_empty = kv_full + NS;                                    // [NS]
  uint64_t* q_full = kv_empty + NS;   // the unit's Q tiles have landed
  uint64_t* q_empty = q_full + 1;     // ... and every S of the segment is complete
  uint64_t* s_full = q_full + 2;      // [2] per tile
  uint64_t* p_full = q_full + 4;      // [2]
  uint64_t* o_full = q_full + 6;      // [2]
  uint64_t* mma_done = q_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 9);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(q_full + 10);
  const View& v = p.v;
  const int warp = warp_id(), lane = lane_id(), c = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int X = 0; X < 2; ++X) {
      mbar_init(&s_full[X], 1);
      mbar_init(&p_full[X], 128);
      mbar_init(&o_full[X], 1);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __shared__ Run run;
  static_assert(kPlanSmem <= SM::kOffBar, "the plan's scratch lies where the tiles will");
  pdl_wait();
  find_run(v, TokenUnits{p.tpt}, gridDim.x, c, p.plan, p.seqs, smem, &run);
  if (run.left == 0) return;  // uniform over the CTA, before TMEM is taken
  fence_proxy_async_smem();   // the scratch is written, the copies of the tiles come next
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
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

  if (warp < 4) {
    regs_dec<kTileRegLo>();
    if (warp == 0) {
      // ------------------------------------------------ producer
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
      }
      const int boxes = (128 / p.unit) * NP;  // <= 16 per operand
      const int my_unit = lane / NP, my_panel = lane % NP;
      uint8_t* my_dst = smem + SM::kOffKV + my_panel * SM::kPanel + my_unit * p.unit * 128;
      int slot = 0, use = 0, issued = 0, segs = 0, q_issued = 0;
      bool ok = true;
      auto load_q = [&](const TileWalk& w) {
        if (lane == 0) {
          const uint32_t bytes = p.tpt * v.g * 128 * NP;
          mbar_expect_tx(q_full, w.tokens(1) ? 2 * bytes : bytes);
          for (int X = 0; X < 2; ++X) {
            if (!w.tokens(X)) continue;
            for (int pn = 0; pn < NP; ++pn)
              tma_load_3d(&tmQ, q_full, smem + X * SM::kOp + pn * SM::kPanel, 64 * pn, w.hk * v.g,
                          w.s.tok0 + (2 * w.u + X) * p.tpt);
          }
        }
        ++q_issued;
        __syncwarp();
      };
      for (TileWalk w(p, run); ok && w.valid(); w.next(), ++segs) {
        // The first Q tiles go out before the page table is read, later ones
        // behind their unit's first block: their buffer frees last.
        if (segs == 0) load_q(w);
        UnitPages up(v, w.seq(), w.s, w.first * 128 + my_unit * p.unit, 128, p.unit);
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const int page = up.page(t, lane < boxes), row_slot = up.slot(t);
#pragma unroll
          for (int kind = 0; kind < 2; ++kind) {
            if (use > 0) ok = ok && __all_sync(0xffffffffu, mbar_wait(&kv_empty[slot], (use - 1) & 1, wc));
            if (!ok) break;
            if (lane == 0) mbar_expect_tx(&kv_full[slot], SM::kOp);
            __syncwarp();
            if (lane < boxes)
              tma_load_4d(kind ? &tmV : &tmK, &kv_full[slot], my_dst + slot * SM::kOp, 64 * my_panel, w.hk, row_slot,
                          page);
            ++issued;
            if (++slot == NS) {
              slot = 0;
              ++use;
            }
          }
          if (ok && segs > 0 && t == w.t0) {
            ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (segs - 1) & 1, wc));
            if (!ok) break;
            load_q(w);
          }
        }
        if (!ok) break;
      }
      // Every issued copy has landed before the CTA may exit.
      if (lane == 0) {
        for (int s = 0; s < NS && s < issued; ++s) drain_wait(&kv_full[s], ((issued - 1 - s) / NS) & 1);
        if (q_issued > 0) drain_wait(q_full, (q_issued - 1) & 1);
      }
    } else if (warp == 1) {
      // ------------------------------------------------ MMA issuer (the whole warp, one lane of which issues)
      constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);  // Q K^T: both K-major
      constexpr uint32_t idPV = idesc_bf16(128, D, 0, 1);   // P V: V MN-major
      const uint32_t leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t dQ0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dK0 = sdesc_sw128(smem_u32(smem + SM::kOffKV), 16, 1024);
      const uint64_t dV0 = sdesc_sw128(smem_u32(smem + SM::kOffKV), SM::kPanel, 1024);
      int ks = 0, ku = 0;  // ring position of the block's K; its V is the next one
      int segs = 0, np[2] = {0, 0};  // segments; P tiles taken, per tile
      bool ok = true;
      auto wait = [&](uint64_t* bar, int parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, static_cast<uint32_t>(parity), wc));
      };
      auto after = [&](int& slot, int& use) {
        if (++slot == NS) {
          slot = 0;
          ++use;
        }
      };
      auto issue_S = [&](int X, int slot) {
        const uint64_t qd = dQ0 + static_cast<uint64_t>((X * SM::kOp) >> 4);
        const uint64_t kd = dK0 + static_cast<uint64_t>(__shfl_sync(0xffffffffu, slot, 0) * (SM::kOp >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = static_cast<uint64_t>(((kk >> 2) * SM::kPanel + (kk & 3) * 32) >> 4);
          mma_ss_warp(tm + static_cast<uint32_t>(X) * 128u, qd + off, kd + off, idS, kk > 0 ? 1u : 0u, leader);
        }
        mma_commit_warp(&s_full[X], leader);
      };
      auto issue_PV = [&](int X, int slot, uint32_t add) {
        const uint64_t vd = dV0 + static_cast<uint64_t>(__shfl_sync(0xffffffffu, slot, 0) * (SM::kOp >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts_warp(tm + 256u + static_cast<uint32_t>(X) * 128u, tm + static_cast<uint32_t>(X) * 128u + kk * 8,
                      vd + static_cast<uint64_t>((kk * 2048) >> 4), idPV, kk > 0 ? 1u : add, leader);
      };
      for (TileWalk w(p, run); ok && w.valid(); w.next(), ++segs) {
        const int lo = w.first + w.t0, hi = w.first + w.t1 - 1;
        int lo_t[2], hi_t[2];
        bool on[2];
#pragma unroll
        for (int X = 0; X < 2; ++X) on[X] = w.tile(X, lo_t[X], hi_t[X]);
        ok = wait(q_full, segs & 1) && wait(&kv_full[ks], ku & 1);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int X = 0; X < 2; ++X)
          if (on[X] && lo_t[X] == lo) issue_S(X, ks);
        mma_commit_warp(&kv_empty[ks], leader);
        if (lo == hi) mma_commit_warp(q_empty, leader);
        for (int j = lo; j <= hi; ++j) {
          int vs = ks, vu = ku;  // V_j, then K_j+1
          after(vs, vu);
          ks = vs;
          ku = vu;
          after(ks, ku);
          ok = wait(&kv_full[vs], vu & 1) && (j == hi || wait(&kv_full[ks], ku & 1));
          if (!ok) break;
#pragma unroll
          for (int X = 0; X < 2; ++X) {
            if (on[X] && j >= lo_t[X] && j <= hi_t[X]) {
              ok = ok && wait(&p_full[X], np[X] & 1);
              if (!ok) break;
              ++np[X];
              tc_fence_after();
              issue_PV(X, vs, j > lo_t[X] ? 1u : 0u);
              if (j == hi_t[X]) mma_commit_warp(&o_full[X], leader);
            }
            if (on[X] && j + 1 >= lo_t[X] && j + 1 <= hi_t[X]) issue_S(X, ks);
          }
          if (!ok) break;
          mma_commit_warp(&kv_empty[vs], leader);  // V_j consumed
          if (j < hi) mma_commit_warp(&kv_empty[ks], leader);  // K_j+1 consumed
          if (j + 1 == hi) mma_commit_warp(q_empty, leader);
        }
      }
      // All issued MMAs complete before TMEM is released.
      mma_commit_warp(mma_done, leader);
      if (leader) drain_wait(mma_done, 0);
      __syncwarp();
    }
  } else {
    regs_inc<kTileRegHi>();
    // -------------------------------------------------- softmax and output
    const int X = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;  // TMEM lane = row of the tile
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + static_cast<uint32_t>(X) * 128u;
    const uint32_t tO = tmem + lane_off + 256u + static_cast<uint32_t>(X) * 128u;
    const float c2 = p.scale_log2;
    int base = 0, ns = 0, no = 0;  // blocks of earlier segments; S and O tiles taken
    bool ok = true, first_seg = true;
    for (TileWalk w(p, run); ok && w.valid(); w.next(), first_seg = false) {
      int lo_t, hi_t;
      const bool on = w.tile(X, lo_t, hi_t);
      const int seg_lo = w.first + w.t0, end = w.s.L + w.s.n, lo_seq = max(0, w.s.L - v.W + 1);
      const int i0 = (2 * w.u + X) * p.tpt, i = i0 + r / v.g;
      const bool live = r < p.tpt * v.g && i < w.s.n;  // a row of the output
      const int qi = w.s.L + i;                        // the row's own cached row: the last it sees
      const int q_lo = w.s.L + i0, q_hi = q_lo + p.tpt - 1;  // bounds of qi over the tile
      float m2 = -INFINITY, l = 0.f;
      if (on) {
        for (int j = lo_t; j <= hi_t; ++j) {
          const bool got = mbar_wait(&s_full[X], ns & 1, wc);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          ++ns;
          tc_fence_after();
          uint32_t sv[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(tS + q * 32, sv[q]);
          tmem_ld_wait();
          const int k0 = j * 128;
          if (k0 + 127 > q_lo || q_hi - k0 >= v.W) {
            // Row r keeps the keys k0 + e with a <= e <= b (causal: key <= qi;
            // window: qi - key < W); an empty range keeps none.
            int a = max(qi - v.W + 1 - k0, 0);
            const int b = min(qi - k0, 127);
            unsigned span = static_cast<unsigned>(b - a);
            if (b < a) {
              a = 1 << 20;
              span = 0u;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (__all_sync(0xffffffffu, a <= 32 * q && 32 * q + 31 <= b)) continue;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (static_cast<unsigned>(32 * q + e - a) > span) sv[q][e] = __float_as_uint(-INFINITY);
            }
          }
          float mp[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float t[11];
#pragma unroll
            for (int k = 0; k < 10; ++k)
              t[k] = fmax3(__uint_as_float(sv[q][3 * k]), __uint_as_float(sv[q][3 * k + 1]),
                           __uint_as_float(sv[q][3 * k + 2]));
            t[10] = fmaxf(__uint_as_float(sv[q][30]), __uint_as_float(sv[q][31]));
            mp[q] = fmax3(fmax3(t[0], t[1], t[2]), fmax3(t[3], t[4], t[5]),
                          fmaxf(fmax3(t[6], t[7], t[8]), fmaxf(t[9], t[10])));
          }
          const float mx = fmax3(mp[0], mp[1], fmaxf(mp[2], mp[3])) * c2;
          float alpha = 1.f;
          bool rescale = false;
          if (j == lo_t) {
            m2 = mx;
          } else if (mx > m2 + 8.f) {  // lazily: only when the maximum grew by 2^8
            alpha = ex2(m2 - mx);
            m2 = mx;
            rescale = true;
          }
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t o[32];
              tmem_ld32(tO + q * 32, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(tO + q * 32, o);
            }
            tmem_st_wait();
          }
          const float mu = (m2 == -INFINITY) ? 0.f : m2;
          const uint64_t c2x2 = f2_pack(c2, c2), nmu2 = f2_pack(-mu, -mu);
          uint64_t ls2[4];
#pragma unroll
          for (int a = 0; a < 4; ++a) ls2[a] = f2_pack(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint64_t x2 = f2_fma(
                  f2_pack(__uint_as_float(sv[q][2 * e]), __uint_as_float(sv[q][2 * e + 1])), c2x2, nmu2);
              float x0, x1;
              f2_unpack(x2, x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              ls2[e & 3] = f2_add(ls2[e & 3], f2_pack(p0, p1));
              pk[e] = pack_bf16x2(p0, p1);  // half a bf16 step, 2^-8 of each weight
            }
            tmem_st16(tS + q * 16, pk);
          }
          float la, lb, lc, ld;
          f2_unpack(f2_add(ls2[0], ls2[1]), la, lb);
          f2_unpack(f2_add(ls2[2], ls2[3]), lc, ld);
          l = l * alpha + ((la + lb) + (lc + ld));
          // Rows of the block that no token sees may hold anything, and 0 * NaN
          // is not 0: thread r clears row r of V before its products.
          if (k0 < lo_seq || k0 + 128 > end) {
            const int slot_i = 2 * (base + j - seg_lo) + 1;
            const int slot = slot_i % NS;
            if (!__all_sync(0xffffffffu, mbar_wait(&kv_full[slot], (slot_i / NS) & 1, wc))) {
              ok = false;
              break;
            }
            if (k0 + r < lo_seq || k0 + r >= end) {
              uint8_t* z = smem + SM::kOffKV + slot * SM::kOp + r * 128;
#pragma unroll
              for (int pn = 0; pn < NP; ++pn)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4*>(z + pn * SM::kPanel + ((e ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&p_full[X]);
        }
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&o_full[X], no & 1, wc));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      base += w.t1 - w.t0;
      // The row's output, or its share of it.
      const bool whole = w.whole();
      const size_t orow = live ? static_cast<size_t>(w.s.tok0 + i) * v.H + w.hk * v.g + r % v.g : 0;
      const size_t prow = static_cast<size_t>(2 * c + (first_seg ? 0 : 1)) * 256 + X * 128 + r;
      if (live) {
        if (whole) p.lse[orow] = (m2 + log2f(l)) * 0.69314718055994531f;
        else p.part_ml[prow] = make_float2(m2, l);
      }
      if (on) {
        const float inv_l = 1.f / l;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          tmem_ld32(tO + q * 32, o);
          tmem_ld_wait();
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint4 x;
              x.x = pack_bf16x2(__uint_as_float(o[8 * e + 0]) * inv_l, __uint_as_float(o[8 * e + 1]) * inv_l);
              x.y = pack_bf16x2(__uint_as_float(o[8 * e + 2]) * inv_l, __uint_as_float(o[8 * e + 3]) * inv_l);
              x.z = pack_bf16x2(__uint_as_float(o[8 * e + 4]) * inv_l, __uint_as_float(o[8 * e + 5]) * inv_l);
              x.w = pack_bf16x2(__uint_as_float(o[8 * e + 6]) * inv_l, __uint_as_float(o[8 * e + 7]) * inv_l);
              *reinterpret_cast<uint4*>(p.O + orow * D + q * 32 + e * 8) = x;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              *reinterpret_cast<uint4*>(p.part_o + prow * D + q * 32 + e * 4) =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
      }
      tc_fence_before();  // the next unit's products overwrite O only after p_full
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct JoinParams {
  View v;
  int rows, tpt;     // query rows of a share; tokens of a tile
  const float* part_o;
  const float2* part_ml;
  const int2* info;  // of rows_kernel
  const Plan* plan;  // of tile_kernel
  __nv_bfloat16* O;
  float* lse;
};

constexpr int kJoinWarps = 8;
constexpr int kJoinRows = 4;                                   // rows of a warp where units of few shares are joined
constexpr int kJoinFew = 8;                                    // shares
constexpr int kJoinUnitCtas = 256 / (kJoinWarps * kJoinRows);  // CTAs of a unit's cut

// R output rows by one warp, rows row0 .. of n partials (maximum, sum,
// output): O = sum 2^(m - M) O_i / sum 2^(m - M) l_i; at(i) is the i-th one's
// place, live a bit per row, to(j) the j-th row's place in O and lse. 32 / R
// lanes have a row's maxima and sums, all of them its output, of which R E
// loads are in flight.
template <int D, int R, int E, class At, class To>
__device__ __forceinline__ void join_rows(const float* part_o, const float2* part_ml, int n, const At& at, int row0,
                                          uint32_t live, const To& to, __nv_bfloat16* O, float* lse) {
  constexpr int W = 32 / R, C = D / 32;
  const int lane = lane_id(), mine = lane / W, k_mine = lane % W;
  const bool on = (live >> mine) & 1u;
  float M = -INFINITY;
  for (int k = k_mine; k < n; k += W)
    if (on) M = fmaxf(M, part_ml[at(k) + row0 + mine].x);
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, a[R][C];
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int e = 0; e < C; ++e) a[j][e] = 0.f;
  for (int k0 = 0; k0 < n; k0 += W) {
    const float2 x = on && k0 + k_mine < n ? part_ml[at(k0 + k_mine) + row0 + mine] : make_float2(-INFINITY, 0.f);
    const float f = x.x == -INFINITY ? 0.f : ex2(x.x - M);  // 0: no key of this share, its output may not be written
    L = fmaf(x.y, f, L);
    const int m = min(W, n - k0);
#pragma unroll 1
    for (int kk = 0; kk < m; kk += E) {
      float y[E][R][C], g[E][R];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float* src = part_o + (at(k0 + kk + i) + row0) * D + lane * C;
#pragma unroll
        for (int j = 0; j < R; ++j) {
          g[i][j] = __shfl_sync(0xffffffffu, f, j * W + kk + i);  // 0 past the last share
#pragma unroll
          for (int e = 0; e < C; ++e) y[i][j][e] = 0.f;
          if (g[i][j] != 0.f) {
            if constexpr (C == 4) {
              const float4 t = *reinterpret_cast<const float4*>(src + j * D);
              y[i][j][0] = t.x, y[i][j][1] = t.y, y[i][j][2] = t.z, y[i][j][3] = t.w;
            } else {
              const float2 t = *reinterpret_cast<const float2*>(src + j * D);
              y[i][j][0] = t.x, y[i][j][1] = t.y;
            }
          }
        }
      }
#pragma unroll
      for (int i = 0; i < E; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int e = 0; e < C; ++e) a[j][e] = fmaf(y[i][j][e], g[i][j], a[j][e]);
    }
  }
#pragma unroll
  for (int o = W / 2; o >= 1; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const float inv = 1.f / __shfl_sync(0xffffffffu, L, j * W);
    if (!((live >> j) & 1u)) continue;
    __nv_bfloat16* dst = O + to(j) * D + lane * C;
#pragma unroll
    for (int e = 0; e < C; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(a[j][e] * inv, a[j][e + 1] * inv);
  }
  if (on && k_mine == 0) lse[to(mine)] = (M + log2f(L)) * 0.69314718055994531f;
}

// CTA = a (sequence, KV head) pair, joined if rows_kernel cut it; or, with
// TILES, a cut between two CTAs' runs of tile_kernel and rows of the unit that
// lies there: 32 of its 256, by the CTAs of its first cut, or, of a unit in
// more than kJoinFew shares, 8 by those of each of its first kJoinRows cuts (a
// chunk of 64 tokens over 20000 rows, 37 shares: 36 us, 70 with the former).
template <int D, bool TILES>
__global__ void __launch_bounds__(32 * kJoinWarps, TILES ? 4 : 1) join_kernel(const JoinParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const View& v = p.v;
  if constexpr (!TILES) {
    const int b = blockIdx.x / v.Hk, hk = blockIdx.x % v.Hk;
    // Unspecified for a sequence without tokens, and where a wait of
    // rows_kernel has run out: what does not name slots is not followed.
    const int2 inf = p.info[blockIdx.x];
    int first;
    Seq s;
    seq_load(v, b, false, s);
    if (visible_blocks(v, s, first) == 0 || inf.y <= 1) return;
    if (inf.x < 0 || inf.x >= 2 * kSMs || inf.y > kSMs - (inf.x >> 1)) return;
    for (int r = warp_id(); r < s.n * v.g; r += kJoinWarps)
      join_rows<D, 1, 8>(
          p.part_o, p.part_ml, inf.y,
          [&](int k) { return static_cast<size_t>(k == 0 ? inf.x : 2 * ((inf.x >> 1) + k)) * p.rows; }, r, 1u,
          [&](int) { return static_cast<size_t>(s.tok0 + r / v.g) * v.H + hk * v.g + r % v.g; }, p.O, p.lse);
  } else {
    Cut cut;
    if (!cut.find(p.plan, blockIdx.x / kJoinUnitCtas + 1)) return;
    const bool many = cut.n > kJoinFew;
    if (cut.nth >= (many ? kJoinRows : 1)) return;
    const int w = blockIdx.x % kJoinUnitCtas * kJoinWarps + warp_id();
    // Rows of the unit's two tiles.
    const int row0 = many ? kJoinRows * w + cut.nth : kJoinRows * w, rows = many ? 1 : kJoinRows;
    const int r0 = row0 & 127, i0 = (2 * cut.st.unit + (row0 >> 7)) * p.tpt;
    uint32_t live = 0u;
#pragma unroll
    for (int j = 0; j < kJoinRows; ++j)
      if (j < rows && r0 + j < p.tpt * v.g && i0 + (r0 + j) / v.g < cut.s.n) live |= 1u << j;
    if (live == 0u) return;
    auto at = [&](int k) { return static_cast<size_t>(cut.slot(k)) * 256; };
    auto to = [&](int j) {
      return static_cast<size_t>(cut.s.tok0 + i0 + (r0 + j) / v.g) * v.H + cut.st.hk * v.g + (r0 + j) % v.g;
    };
    // As many loads as 64 registers hold: four CTAs on an SM are worth more
    // (2 x 2048 tokens over 8192 rows 245 us, 250 with twice the loads).
    constexpr int kLoads = D == 128 ? 4 : 8;
    if (many) join_rows<D, 1, kLoads>(p.part_o, p.part_ml, cut.n, at, row0, live, to, p.O, p.lse);
    else join_rows<D, kJoinRows, kLoads / kJoinRows>(p.part_o, p.part_ml, cut.n, at, row0, live, to, p.O, p.lse);
  }
}

}  // namespace paged
}  // namespace cswattn
