// paged_tile.cuh -- paged attention of sequences with many query rows (a
// prompt's chunk): tcgen05 tensor cores, 128-row tiles.
//
// A tile's 128 rows are tokens x heads of one KV head's group (row = token in
// the tile * g + head in the group; 128 / g tokens), so every head that reads
// a K or V row shares the one copy of it; a unit of work is two consecutive
// tiles of one (sequence, KV head), which share the blocks of 128 cached rows
// too. The units' blocks in a row are dealt out evenly to one CTA per SM, as
// in the kernel of few rows (a unit is cut where a CTA's run ends; its
// partial outputs go to the workspace and tile_combine_kernel joins them), so
// neither ragged chunks nor the causal edge nor a last wave leave SMs idle.
// plan_kernel computes the deal once: where each CTA's run starts.
//
// Roles (12 warps), as in the dense forward:
//   warp 0      producer: the units' Q tiles and their K and V blocks, through
//               one 5-slot ring; every lane copies one box (a page unit of
//               rows x 64 columns); units that no token sees are read past the
//               pool's end, which fills zeros
//   warp 1      TMEM owner, single-thread MMA issuer
//   warps 4-7   softmax of tile 0, warps 8-11 of tile 1: thread = query row
// TMEM (512 columns): S0 | S1 | O0 | O1. Per block: S = Q K^T, P (bf16) over
// the S columns, O += P V, in the order PV_0(j), S_0(j+1), PV_1(j), S_1(j+1)
// so that one tile's softmax overlaps the other's products. The barriers'
// phases run on from unit to unit, and the next unit's first S is issued
// while the last one's output is still being written.
// Bound by the softmax (one exponential per score) and the tensor pipe.
#pragma once
#include "paged_rows.cuh"

namespace cswattn {
namespace paged {

constexpr int kTileThreads = 384;
constexpr int kTileMinBlocks = 2;  // fewest blocks worth a CTA of their own
constexpr int kTileRegLo = 80, kTileRegHi = 208;
static_assert(128 * kTileRegLo + 256 * kTileRegHi <= kTileThreads * 168, "register budget");

// Where a CTA's run starts: the k-th long sequence, KV head, unit, block of the unit.
struct Start {
  int k, hk, unit, t0;
};

struct Plan {
  int ctas, n_long;
  long long total;
  Start start[kSMs];
};

struct TileParams {
  View v;
  float scale_log2;
  int unit;        // rows of a K or V box
  int tpt;         // tokens per tile: 128 / g
  int short_rows;  // sequences with more query rows than this are this kernel's
  const Plan* plan;
  const int* longs;  // the long sequences, in order
  __nv_bfloat16* O;
  float* lse;
  float* part_o;     // (2 kSMs, 256, D)
  float2* part_ml;   // (2 kSMs, 256)
  unsigned long long wait_ns;
};

__device__ __forceinline__ bool is_long(const View& v, const Seq& s, int short_rows) {
  return static_cast<long long>(s.n) * v.g > short_rows;
}

// Blocks of 128 cached rows that the tokens [i0, i1) of a sequence see.
__device__ __forceinline__ void token_blocks(const View& v, const Seq& s, int i0, int i1, int& lo, int& hi) {
  lo = max(0, s.L + i0 - v.W + 1) >> 7;
  hi = (s.L + i1 - 1) >> 7;
}
__device__ __forceinline__ int unit_blocks(const View& v, const Seq& s, int tpt, int u) {
  int lo, hi;
  token_blocks(v, s, u * 2 * tpt, min(s.n, (u + 1) * 2 * tpt), lo, hi);
  return hi - lo + 1;
}
__device__ __forceinline__ int unit_count(const Seq& s, int tpt) { return (s.n + 2 * tpt - 1) / (2 * tpt); }

constexpr int kPlanThreads = 1024;

// One CTA: the blocks of every long sequence, their running sum, and the
// start of each CTA's run (a warp per sequence, then a warp per start).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const View v, int tpt, int short_rows, Plan* plan,
                                                            int* longs) {
  __shared__ long long pre[kMaxSeqs + 1];  // per long sequence: blocks of one KV head before it
  __shared__ int s_total[33];
  const int warp = warp_id(), lane = lane_id();
  pdl_launch_dependents();
  pdl_wait();
  // The long sequences, in order.
  int n_long = 0;
  for (int b0 = 0; b0 < v.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    bool yes = false;
    if (b < v.B) {
      Seq s;
      yes = seq_load(v, b, true, s) && is_long(v, s, short_rows);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, yes);
    if (lane == 0) s_total[warp] = __popc(m);
    __syncthreads();
    int before = n_long;
    for (int w = 0; w < warp; ++w) before += s_total[w];
    if (yes) longs[before + __popc(m & ((1u << lane) - 1u))] = b;
    for (int w = 0; w < 32; ++w) n_long += s_total[w];
    __syncthreads();
  }
  for (int k = warp; k < n_long; k += 32) {
    Seq s;
    seq_load(v, longs[k], false, s);
    long long sum = 0;
    for (int u = lane; u < unit_count(s, tpt); u += 32) sum += unit_blocks(v, s, tpt, u);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) pre[k + 1] = sum;
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  if (warp == 0) {
    long long run = 0;
    for (int k0 = 0; k0 < n_long; k0 += 32) {
      long long x = k0 + lane < n_long ? pre[k0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (k0 + lane < n_long) pre[k0 + lane + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  const long long total = pre[n_long] * v.Hk;
  const long long most = (total + kTileMinBlocks - 1) / kTileMinBlocks;
  const int ctas = static_cast<int>(most < kSMs ? most : kSMs);
  if (threadIdx.x == 0) {
    plan->ctas = ctas;
    plan->n_long = n_long;
    plan->total = total;
  }
  for (int c = warp; c < ctas; c += 32) {
    const long long at = total * c / ctas;
    int lo = 0, hi = n_long;  // the last k with pre[k] * Hk <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] * v.Hk <= at) lo = mid;
      else hi = mid;
    }
    Seq s;
    seq_load(v, longs[lo], false, s);
    const long long cnt = pre[lo + 1] - pre[lo], rem = at - pre[lo] * v.Hk;
    long long left = rem % cnt;
    const int nu = unit_count(s, tpt);
    for (int u0 = 0; u0 < nu; u0 += 32) {  // 32 units at a time: the one that holds block `left`
      const int u = u0 + lane;
      const int mine = u < nu ? unit_blocks(v, s, tpt, u) : 0;
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      const bool here = u < nu && left >= inc - mine && left < inc;
      if (here) plan->start[c] = Start{lo, static_cast<int>(rem / cnt), u, static_cast<int>(left) - (inc - mine)};
      if (__any_sync(0xffffffffu, here)) break;
      left -= __shfl_sync(0xffffffffu, inc, 31);
    }
  }
}

// A CTA's walk over its run: one segment (blocks [t0, t1) of a unit) at a time.
struct TileWalk {
  const TileParams& p;
  long long left;
  int k, hk, u, t0, t1, cnt, units, first;
  Seq s;
  __device__ TileWalk(const TileParams& p_, int c) : p(p_) {
    const Start st = p.plan->start[c];
    const long long total = p.plan->total;
    const int ctas = p.plan->ctas;
    left = total * (c + 1) / ctas - total * c / ctas;
    k = st.k;
    hk = st.hk;
    u = st.unit;
    t0 = st.t0;
    load();
    set();
  }
  __device__ void load() {
    seq_load(p.v, p.longs[k], false, s);
    units = unit_count(s, p.tpt);
  }
  __device__ void set() {
    int hi;
    token_blocks(p.v, s, u * 2 * p.tpt, min(s.n, (u + 1) * 2 * p.tpt), first, hi);
    cnt = hi - first + 1;
    t1 = left < cnt - t0 ? t0 + static_cast<int>(left) : cnt;
  }
  __device__ bool valid() const { return left > 0; }
  __device__ void next() {
    left -= t1 - t0;
    t0 = 0;
    if (left <= 0) return;
    if (++u == units) {
      u = 0;
      if (++hk == p.v.Hk) {
        hk = 0;
        ++k;
        load();
      }
    }
    set();
  }
  // Blocks [lo, hi] of the segment that tile X (0 or 1) of the unit has; false if none.
  __device__ bool tile(int X, int& lo, int& hi) const {
    const int i0 = (2 * u + X) * p.tpt;
    if (i0 >= s.n) return false;
    token_blocks(p.v, s, i0, min(s.n, i0 + p.tpt), lo, hi);
    lo = max(lo, first + t0);
    hi = min(hi, first + t1 - 1);
    return lo <= hi;
  }
  __device__ bool tokens(int X) const { return (2 * u + X) * p.tpt < s.n; }
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
  pdl_launch_dependents();
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
  pdl_wait();
  if (c >= p.plan->ctas) return;  // uniform over the CTA, before TMEM is taken
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
      for (TileWalk w(p, c); ok && w.valid(); w.next(), ++segs) {
        const int b = p.longs[w.k];
        const int lo = max(0, w.s.L - v.W + 1), end = w.s.L + w.s.n;
        auto lookup = [&](int t) -> int {  // page of this lane's unit, or past the pool
          const int r = (w.first + t) * 128 + my_unit * p.unit;
          if (lane >= boxes || r >= end || r + p.unit <= lo) return v.n_pages;
          const int page = page_at(v, b, r / v.page_size);
          return page < 0 ? v.n_pages : page;
        };
        int page = lookup(w.t0);
        for (int t = w.t0; ok && t < w.t1; ++t) {
          const int next = t + 1 < w.t1 ? lookup(t + 1) : 0;
          const int row_slot = ((w.first + t) * 128 + my_unit * p.unit) % v.page_size;
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
          if (ok && t == w.t0) {  // the Q tiles, behind the first block: their buffer frees last
            if (segs > 0) ok = __all_sync(0xffffffffu, mbar_wait(q_empty, (segs - 1) & 1, wc));
            if (!ok) break;
            if (lane == 0) {
              const uint32_t bytes = p.tpt * v.g * 128 * NP;
              mbar_expect_tx(q_full, w.tokens(1) ? 2 * bytes : bytes);
              for (int X = 0; X < 2; ++X) {
                if (!w.tokens(X)) continue;
                for (int pn = 0; pn < NP; ++pn) {
                  asm volatile(
                      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem + X * SM::kOp + pn * SM::kPanel)),
                      "l"(reinterpret_cast<uint64_t>(&tmQ)), "r"(smem_u32(q_full)), "r"(64 * pn), "r"(w.hk * v.g),
                      "r"(w.s.tok0 + (2 * w.u + X) * p.tpt)
                      : "memory");
                }
              }
            }
            ++q_issued;
            __syncwarp();
          }
          page = next;
        }
        if (!ok) break;
      }
      // Every issued copy has landed before the CTA may exit.
      if (lane == 0) {
        for (int s = 0; s < NS && s < issued; ++s) drain_wait(&kv_full[s], ((issued - 1 - s) / NS) & 1);
        if (q_issued > 0) drain_wait(q_full, (q_issued - 1) & 1);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // ---------------------------------------------- MMA issuer
        constexpr uint32_t idS = idesc_bf16(128, 128, 0, 0);  // Q K^T: both K-major
        constexpr uint32_t idPV = idesc_bf16(128, D, 0, 1);   // P V: V MN-major
        const uint64_t dQ0 = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t dK0 = sdesc_sw128(smem_u32(smem + SM::kOffKV), 16, 1024);
        const uint64_t dV0 = sdesc_sw128(smem_u32(smem + SM::kOffKV), SM::kPanel, 1024);
        int base = 0, segs = 0;  // blocks of earlier segments; segments
        int np[2] = {0, 0};      // P tiles taken, per tile
        bool ok = true;
        for (TileWalk w(p, c); ok && w.valid(); w.next(), ++segs) {
          const int lo = w.first + w.t0, hi = w.first + w.t1 - 1;
          int lo_t[2], hi_t[2];
          bool on[2];
          for (int X = 0; X < 2; ++X) on[X] = w.tile(X, lo_t[X], hi_t[X]);
          auto ring = [&](int j, int kind, int& slot, int& use) {
            const int i = 2 * (base + j - lo) + kind;
            slot = i % NS;
            use = i / NS;
          };
          auto issue_S = [&](int X, int j) -> bool {
            int s, use;
            ring(j, 0, s, use);
            if (!mbar_wait(&kv_full[s], use & 1, wc)) return false;
            tc_fence_after();
            const uint64_t qd = dQ0 + static_cast<uint64_t>((X * SM::kOp) >> 4);
            const uint64_t kd = dK0 + static_cast<uint64_t>((s * SM::kOp) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint64_t off = static_cast<uint64_t>(((kk >> 2) * SM::kPanel + (kk & 3) * 32) >> 4);
              mma_ss(tmem + static_cast<uint32_t>(X) * 128u, qd + off, kd + off, idS, kk > 0 ? 1u : 0u);
            }
            mma_commit(&s_full[X]);
            return true;
          };
          auto issue_PV = [&](int X, int j) -> bool {
            int s, use;
            ring(j, 1, s, use);
            if (!mbar_wait(&kv_full[s], use & 1, wc)) return false;
            if (!mbar_wait(&p_full[X], np[X] & 1, wc)) return false;
            ++np[X];
            tc_fence_after();
            const uint64_t vd = dV0 + static_cast<uint64_t>((s * SM::kOp) >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + 256u + static_cast<uint32_t>(X) * 128u, tmem + static_cast<uint32_t>(X) * 128u + kk * 8,
                     vd + static_cast<uint64_t>((kk * 2048) >> 4), idPV, (j > lo_t[X] || kk > 0) ? 1u : 0u);
            return true;
          };
          int rs, ru;
          ok = mbar_wait(q_full, segs & 1, wc);
          if (ok) tc_fence_after();
          for (int X = 0; X < 2 && ok; ++X)
            if (on[X] && lo_t[X] == lo) ok = issue_S(X, lo);
          if (!ok) break;
          ring(lo, 0, rs, ru);
          mma_commit(&kv_empty[rs]);
          if (lo == hi) mma_commit(q_empty);
          for (int j = lo; ok && j <= hi; ++j) {
            for (int X = 0; X < 2 && ok; ++X) {
              if (!on[X]) continue;
              if (j >= lo_t[X] && j <= hi_t[X]) {
                ok = issue_PV(X, j);
                if (ok && j == hi_t[X]) mma_commit(&o_full[X]);
              }
              if (ok && j + 1 >= lo_t[X] && j + 1 <= hi_t[X]) ok = issue_S(X, j + 1);
            }
            if (!ok) break;
            ring(j, 1, rs, ru);
            mma_commit(&kv_empty[rs]);  // V_j consumed
            if (j + 1 <= hi) {
              ring(j + 1, 0, rs, ru);
              mma_commit(&kv_empty[rs]);  // K_j+1 consumed
              if (j + 1 == hi) mma_commit(q_empty);
            }
          }
          base += hi - lo + 1;
        }
        // All issued MMAs complete before TMEM is released.
        mma_commit(mma_done);
        drain_wait(mma_done, 0);
      }
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
    for (TileWalk w(p, c); ok && w.valid(); w.next(), first_seg = false) {
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
              pk[e] = pack_bf16x2(p0, p1);  // half a bf16 step, 2^-9 of each weight
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
      const bool whole = w.t0 == 0 && w.t1 == w.cnt;
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

constexpr int kTileCombineRows = 8;  // rows (warps) of a CTA

// CTA = (boundary between two CTAs' runs, 8 rows): the unit cut there, if the
// boundary is its first, from the shares of all CTAs that had a part of it.
template <int D>
__global__ void __launch_bounds__(32 * kTileCombineRows) tile_combine_kernel(const __grid_constant__ TileParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x + 1, lane = lane_id();
  const Plan* plan = p.plan;
  if (c >= plan->ctas) return;
  const View& v = p.v;
  const Start st = plan->start[c], before = plan->start[c - 1];
  auto same = [&](const Start& a) { return a.k == st.k && a.hk == st.hk && a.unit == st.unit; };
  if (st.t0 == 0 || (same(before) && before.t0 > 0)) return;
  int last = c;
  while (last + 1 < plan->ctas && same(plan->start[last + 1])) ++last;
  const int slot0 = 2 * (c - 1) + (same(before) ? 0 : 1);
  Seq s;
  seq_load(v, p.longs[st.k], false, s);
  const int row = blockIdx.y * kTileCombineRows + warp_id();  // of the unit's two tiles
  const int r = row & 127, i = (2 * st.unit + (row >> 7)) * p.tpt + r / v.g;
  if (r >= p.tpt * v.g || i >= s.n) return;
  auto at = [&](int k) { return static_cast<size_t>(k < c ? slot0 : 2 * k) * 256 + row; };
  float M = -INFINITY;
  for (int k = c - 1; k <= last; ++k) M = fmaxf(M, p.part_ml[at(k)].x);
  float L = 0.f, a[D / 32];
#pragma unroll
  for (int e = 0; e < D / 32; ++e) a[e] = 0.f;
  for (int k = c - 1; k <= last; ++k) {
    const float2 x = p.part_ml[at(k)];
    if (x.x == -INFINITY) continue;  // no key of this share: its output may not be written
    const float f = ex2(x.x - M);
    L = fmaf(x.y, f, L);
    const float* src = p.part_o + at(k) * D + lane * (D / 32);
#pragma unroll
    for (int e = 0; e < D / 32; e += 2) {
      const float2 y = *reinterpret_cast<const float2*>(src + e);
      a[e] = fmaf(y.x, f, a[e]);
      a[e + 1] = fmaf(y.y, f, a[e + 1]);
    }
  }
  const size_t orow = static_cast<size_t>(s.tok0 + i) * v.H + st.hk * v.g + r % v.g;
  const float inv = 1.f / L;
#pragma unroll
  for (int e = 0; e < D / 32; e += 2)
    *reinterpret_cast<uint32_t*>(p.O + orow * D + lane * (D / 32) + e) = pack_bf16x2(a[e] * inv, a[e + 1] * inv);
  if (lane == 0) p.lse[orow] = (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace paged
}  // namespace cswattn
