// paged_rows.cuh -- paged attention of calls with few query rows a sequence
// (new tokens x heads of a group at most 16 MB): a generation step, a few
// speculated tokens. The step reads every visible K and V row once, so it is
// bound by HBM; the products need 16 x 8 tiles, not 128 x 128 ones. Measured
// with its join: 32 sequences of 2048 rows, 12 heads on 4 of 128, 28.0 us =
// 4.8 TB/s (0.73 of a copy's rate), about 3 us of it the CTAs' start (lengths,
// page table, first copy: dependent loads) and 3 the launches; one sequence of
// 1000 rows, 6 heads, 9.1 us.
//
// Work is cut by bytes, not by sequence: the 64-row blocks of all (sequence,
// KV head) pairs in a row are dealt out evenly to one CTA per SM, so ragged
// lengths and any number of sequences load the SMs alike. A CTA's run covers
// whole pairs, whose output it writes itself, and at most two cut ones (its
// first and its last), whose partial maximum, sum and float32 output go to
// the workspace; join_kernel joins those.
//
// CTA: one producer warp streams 64-row blocks of K and V through a ring (one
// TMA box per page unit and 64-column panel, 128B swizzle, straight on from
// one pair to the next), and 4 MB warps compute: warp (m, k) takes the 16
// query rows 16 m .. and the 16 cached rows 16 k .. of each block, with its
// own running maximum, sum and output, so no barrier stands between warps
// until a pair ends. S = Q K^T and O += P V are m16n8k16 products of mma.sync:
// a tile of 128 rows would leave 9 of 10 rows of tcgen05's idle here, and its
// way through TMEM costs more than the product.
// Units of a block that hold no visible row are not read: their box lies past
// the pool's last page, and TMA fills it with zeros.
#pragma once
#include "paged_plan.cuh"

namespace cswattn {
namespace paged {

constexpr int kBlk = 64;         // cached rows of a block
constexpr int kKeyGroups = 4;    // warps that share a block, 16 rows each
// Fewest blocks worth a CTA of their own (one chat over 1000 rows: 1 9.0 us, 2
// 9.1, 4 10.5; 2 leaves half the shares to join).
constexpr int kMinBlocks = 2;

struct RowsParams {
  View v;
  float scale_log2;  // softmax scale * log2(e)
  int unit;          // rows of a TMA box: divides the page and the block
  const __nv_bfloat16* q;
  __nv_bfloat16* O;
  float* lse;
  float* part_o;     // (2 kSMs, 16 MB, D)
  float2* part_ml;   // (2 kSMs, 16 MB): maximum (log2 units) and sum
  int2* info;        // (B, Hk): first slot of a pair and its number of slots
  unsigned long long wait_ns;
};

__device__ __forceinline__ void mma_bf16_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Blocks of the rows that sequence s's tokens see; 0 when it has none.
__device__ __forceinline__ int visible_blocks(const View& v, const Seq& s, int& first) {
  first = max(0, s.L - v.W + 1) / kBlk;
  if (s.n == 0) return 0;
  return (s.L + s.n - 1) / kBlk - first + 1;
}

// The deal: pair (sequence, KV head) blocks in a row, CTA c of n takes
// [total c / n, total (c + 1) / n), or, with `whole`, the pairs that begin there.
struct Deal {
  const int* pre;  // blocks of one KV head before each sequence
  int B, Hk;
  long long total;
  int ctas;
  bool whole;
  long long at, end;  // this CTA's run
  int b;              // the sequence that holds its first block

  __device__ int owner(long long x) const {
    return total < (1 << 23) ? static_cast<int>((static_cast<uint32_t>(x + 1) * ctas - 1) / static_cast<uint32_t>(total))
                             : static_cast<int>(((x + 1) * ctas - 1) / total);
  }
  // The last b with pre[b] * Hk <= x.
  __device__ int sequence(long long x) const {
    const int y = total < (1 << 23) ? static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(Hk))
                                    : static_cast<int>(x / Hk);
    int lo = 0, hi = B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (pre[mid] <= y) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

struct DealShared {
  long long begin[kSMs + 1], pair[kSMs + 1];  // of each run: its block, and the first pair that begins there or later
  int b[kSMs + 1], pair_b[kSMs + 1];
};

// All threads call. With sh (in shared memory), whole pairs
// where no run then exceeds the average by a quarter: the SMs share HBM, so
// the others' runs are read no slower, and nothing is left to join
// (32 sequences of 2048 rows on 4 KV heads, 128 pairs: 29.6 -> 28.1 us); runs
// of twice the average would leave most SMs idle behind the longest.
// Without it (sh null) each thread works its CTA's run out for itself.
__device__ __forceinline__ Deal deal_out(const View& v, const int* pre, int grid, int c, DealShared* sh) {
  Deal d;
  d.pre = pre;
  d.B = v.B;
  d.Hk = v.Hk;
  d.total = static_cast<long long>(pre[v.B]) * v.Hk;
  const long long most = (d.total + kMinBlocks - 1) / kMinBlocks;
  d.ctas = static_cast<int>(most < grid ? most : grid);
  d.whole = false;
  d.at = d.end = 0;
  d.b = 0;
  if (!sh) {
    if (c < d.ctas) {
      d.at = share_of(d.total, c, d.ctas);
      d.end = share_of(d.total, c + 1, d.ctas);
      d.b = d.sequence(d.at);
    }
    return d;
  }
  for (int i = threadIdx.x; i <= d.ctas && d.ctas > 0; i += blockDim.x) {
    const long long x = share_of(d.total, i, d.ctas);
    long long y = x;
    int b = v.B, pb = v.B;
    if (i < d.ctas) {
      b = pb = d.sequence(x);
      const int cnt = pre[b + 1] - pre[b], rem = static_cast<int>(x - static_cast<long long>(pre[b]) * v.Hk);
      const int up = (rem + cnt - 1) / cnt * cnt;
      y = x - rem + up;
      if (up == cnt * v.Hk) {  // the next sequence's first pair
        do ++pb;
        while (pb < v.B && pre[pb + 1] == pre[pb]);
      }
    }
    sh->begin[i] = x;
    sh->pair[i] = y;
    sh->b[i] = b;
    sh->pair_b[i] = pb;
  }
  __syncthreads();
  bool uneven = false;
  for (int i = threadIdx.x; i < d.ctas; i += blockDim.x)
    uneven = uneven || 4 * (sh->pair[i + 1] - sh->pair[i]) * d.ctas > 5 * d.total;
  d.whole = !__syncthreads_or(uneven);
  if (c < d.ctas) {
    d.at = d.whole ? sh->pair[c] : sh->begin[c];
    d.end = d.whole ? sh->pair[c + 1] : sh->begin[c + 1];
    d.b = d.whole ? sh->pair_b[c] : sh->b[c];
  }
  return d;
}

template <int D, int MB>
struct RowsSmem {
  static constexpr int kStages = D == 64 ? 8 : (MB == 1 ? 5 : 4);
  static constexpr int kPanel = kBlk * 128;           // 64 rows x 64 columns
  static constexpr int kOp = (D / 64) * kPanel;       // a block of K or V
  static constexpr int kStage = 2 * kOp;
  static constexpr int kStride = D + 8;               // floats of a staged output row: no bank conflicts
  static constexpr int kOffMerge = kStages * kStage;  // [MB][4][16][kStride] float
  static constexpr int kOffMl = kOffMerge + MB * kKeyGroups * 16 * kStride * 4;
  static constexpr int kOffBar = kOffMl + MB * kKeyGroups * 16 * 8;
  static constexpr int kOffPre = kOffBar + 8 * (3 * kStages + 2);  // int [B + 1]
  static constexpr int kBytes = kOffPre + 1024;       // and 4 (B + 1) more
  static_assert(kBytes + 4 * (kMaxSeqs + 1) <= 232448, "shared memory per block");
};

// A CTA's walk over its run of blocks: one segment per pair.
struct Walk {
  const int* pre;
  int B, Hk;
  long long at, end;
  int b, hk, t0, t1, cnt;
  __device__ explicit Walk(const Deal& deal)
      : pre(deal.pre), B(deal.B), Hk(deal.Hk), at(deal.at), end(deal.end), b(deal.b) {
    set();
  }
  __device__ void set() {
    cnt = pre[b + 1] - pre[b];
    const int rem = static_cast<int>(at - static_cast<long long>(pre[b]) * Hk);
    hk = rem / cnt;
    t0 = rem % cnt;
    const long long left = end - at;
    t1 = left < cnt - t0 ? t0 + static_cast<int>(left) : cnt;
  }
  __device__ bool valid() const { return at < end; }
  __device__ void next() {
    at += t1 - t0;
    if (at >= end) return;
    while (static_cast<long long>(pre[b + 1]) * Hk <= at) ++b;
    set();
  }
};

// Sum of the blocks before each sequence, in shared memory; all threads call.
__device__ __forceinline__ void fill_prefix(const View& v, int* pre, bool report) {
  for (int b = threadIdx.x; b < v.B; b += blockDim.x) {
    Seq s;
    int first;
    seq_load(v, b, report, s);
    pre[b + 1] = visible_blocks(v, s, first);
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  if (warp_id() == 0) {
    int run = 0;
    for (int b0 = 0; b0 < v.B; b0 += 32) {
      const int b = b0 + lane_id();
      int x = b < v.B ? pre[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane_id() >= o) x += y;
      }
      if (b < v.B) pre[b + 1] = run + x;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
}

template <int D, int MB>
__global__ void __launch_bounds__(32 * (kKeyGroups * MB + 1), 1)
    rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const RowsParams p) {
  using SM = RowsSmem<D, MB>;
  constexpr int NS = SM::kStages, NP = D / 64;
  constexpr int kWarps = kKeyGroups * MB;  // compute warps; warp kWarps streams
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align1024(smem_raw);
  uint64_t* full_k = reinterpret_cast<uint64_t*>(smem + SM::kOffBar);
  uint64_t* full_v = full_k + NS;
  uint64_t* empty = full_v + NS;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + NS);
  int* pre = reinterpret_cast<int*>(smem + SM::kOffPre);
  const View& v = p.v;
  const int warp = warp_id(), lane = lane_id();
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full_k[s], 1);
      mbar_init(&full_v[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  const int c = blockIdx.x;
  fill_prefix(v, pre, c == 0);
  __shared__ DealShared s_deal;
  const Deal deal = deal_out(v, pre, gridDim.x, c, &s_deal);
  if (deal.at >= deal.end) return;
  Walk w(deal);
  const WaitCtx wc{abort_flag, p.wait_ns};

  if (warp == kWarps) {
    // ---------------------------------------------------- producer: K and V blocks
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    const int boxes = kBlk / p.unit * NP;  // <= 8 per operand; lane: unit and panel
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
        if (lane == 0) {
          mbar_expect_tx(&full_k[stage], SM::kOp);
          mbar_expect_tx(&full_v[stage], SM::kOp);
        }
        __syncwarp();
        if (lane < boxes) {
          const int slot = up.slot(t);
          uint8_t* dst = my_dst + stage * SM::kStage;
          tma_load_4d(&tmK, &full_k[stage], dst, 64 * my_panel, w.hk, slot, page);
          tma_load_4d(&tmV, &full_v[stage], dst + SM::kOp, 64 * my_panel, w.hk, slot, page);
        }
        ++issued;
        if (++stage == NS) {
          stage = 0;
          ++use;
        }
      }
    }
    // Every issued copy has landed before the CTA may exit.
    if (lane == 0)
      for (int s = 0; s < NS && s < issued; ++s) {
        const int last = (issued - 1 - s) / NS;  // last use of the slot
        drain_wait(&full_k[s], last & 1);
        drain_wait(&full_v[s], last & 1);
      }
    return;
  }

  // ------------------------------------------------------ compute warps
  const int m = warp / kKeyGroups, kg = warp % kKeyGroups;
  const int r0 = m * 16 + (lane >> 2);  // query rows r0 and r0 + 8
  float* merge = reinterpret_cast<float*>(smem + SM::kOffMerge) + m * kKeyGroups * 16 * SM::kStride;
  float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl) + m * kKeyGroups * 16;
  // This lane's row addresses of ldmatrix: K (rows = n, 4 x 8 columns of k) and V (transposed: rows = k).
  const int k_row = kg * 16 + (lane & 7);                          // + 8 for the second n tile; matrix lane >> 3 = chunk
  const int v_row = kg * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;  // matrices 0, 1: rows 0-7, 8-15; 2, 3: next chunk
  const uint32_t s_base = smem_u32(smem);
  int stage = 0, use = 0;
  for (bool first_seg = true; w.valid(); w.next(), first_seg = false) {
    Seq s;
    int first;
    seq_load(v, w.b, false, s);
    visible_blocks(v, s, first);
    const int rows = s.n * v.g;
    const int lo_seq = max(0, s.L - v.W + 1), end_seq = s.L + s.n;
    // Q rows as A fragments; a row past the last is zero.
    uint32_t qa[D / 16][4];
    int hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + 8 * e;
      const bool in = r < rows;
      const int i = in ? r / v.g : 0, h = in ? r % v.g : 0;
      hi[e] = in ? s.L + i : -1;
      lo[e] = max(0, s.L + i - v.W + 1);
      const __nv_bfloat16* src = p.q + (static_cast<size_t>(s.tok0 + i) * v.H + w.hk * v.g + h) * D + (lane & 3) * 2;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qa[kk][e] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
        qa[kk][e + 2] = in ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
      }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    bool ok = true;
    for (int t = w.t0; t < w.t1; ++t) {
      const uint32_t kb = s_base + stage * SM::kStage, vb = kb + SM::kOp;
      ok = __all_sync(0xffffffffu, mbar_wait(&full_k[stage], use & 1, wc));
      if (!ok) break;
      const int key0 = (first + t) * kBlk;
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
        const int row = k_row + nt * 8;
#pragma unroll
        for (int k2 = 0; k2 < D / 32; ++k2) {  // 32 columns: two k steps
          const int chunk = k2 * 4 + (lane >> 3);
          uint32_t b[4];
          ldmatrix4<false>(kb + (chunk >> 3) * SM::kPanel + row * 128 + (((chunk & 7) ^ (row & 7)) << 4), b);
          mma_bf16_16816(sc[nt], qa[2 * k2], b[0], b[1]);
          mma_bf16_16816(sc[nt], qa[2 * k2 + 1], b[2], b[3]);
        }
      }
      // Mask (a select: what lies in unseen rows does not matter), maximum, exponentials.
      const bool edge = key0 + kBlk > s.L || key0 < lo_seq + s.n;  // some row does not see the whole block
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nt][e] *= p.scale_log2;
          if (edge) {
            const int key = key0 + kg * 16 + nt * 8 + (lane & 3) * 2 + (e & 1);
            if (key > hi[e >> 1] || key < lo[e >> 1]) sc[nt][e] = -INFINITY;
          }
        }
      float top[2];
      bool grow = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(sc[0][2 * e], sc[0][2 * e + 1]), fmaxf(sc[1][2 * e], sc[1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
        top[e] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
        grow = grow || top[e] > mx[e] + 8.f;  // rescale only when a row's maximum grew by 2^8 (or from -inf)
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float mn = fmaxf(mx[e], top[e]);
          const float a = mn == -INFINITY ? 1.f : ex2(mx[e] - mn);
          mx[e] = mn;
          sum[e] *= a;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][2 * e] *= a;
            o[i][2 * e + 1] *= a;
          }
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mu = mx[e] == -INFINITY ? 0.f : mx[e];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float p0 = ex2(sc[nt][2 * e] - mu), p1 = ex2(sc[nt][2 * e + 1] - mu);
          sum[e] += p0 + p1;
          pa[nt * 2 + e] = pack_bf16x2(p0, p1);  // bf16 operand of the second product: half a step, 2^-8 of each weight
        }
      }
      ok = __all_sync(0xffffffffu, mbar_wait(&full_v[stage], use & 1, wc));
      if (!ok) break;
      // Rows of the block that no token sees may hold anything, and 0 * NaN is
      // not 0: this warp's are cleared first.
      if (key0 < lo_seq || key0 + kBlk > end_seq) {
        const int row = kg * 16 + (lane & 15);
        if (key0 + row < lo_seq || key0 + row >= end_seq) {
          uint8_t* z = smem + stage * SM::kStage + SM::kOp + row * 128 + (lane >> 4) * 64;
#pragma unroll
          for (int pn = 0; pn < NP; ++pn)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(z + pn * SM::kPanel + ((i ^ (row & 3)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();  // before the slot's next copy
        __syncwarp();
      }
#pragma unroll
      for (int d2 = 0; d2 < D / 16; ++d2) {  // 16 columns of V: two n tiles
        const int chunk = d2 * 2 + (lane >> 4);
        uint32_t b[4];
        ldmatrix4<true>(vb + (chunk >> 3) * SM::kPanel + v_row * 128 + (((chunk & 7) ^ (v_row & 7)) << 4), b);
        mma_bf16_16816(o[2 * d2], pa, b[0], b[1]);
        mma_bf16_16816(o[2 * d2 + 1], pa, b[2], b[3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == NS) {
        stage = 0;
        ++use;
      }
    }
    // ---- the segment's end: join the four key groups of the row block
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 1);
      sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], 2);
      const int row = (lane >> 2) + 8 * e;
      if ((lane & 3) == 0) ml[kg * 16 + row] = make_float2(mx[e], sum[e]);
      float* dst = merge + (kg * 16 + row) * SM::kStride + (lane & 3) * 2;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(dst + i * 8) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
    }
    // A wait that ran out ends the row block's four warps together.
    if (!named_bar_and(1 + m, 32 * kKeyGroups, ok)) return;
    const int tid = kg * 32 + lane;  // 8 threads per row, D / 8 columns each
    const int row = tid >> 3, r = m * 16 + row;
    if (r < rows) {
      float M = -INFINITY, L = 0.f, f[kKeyGroups];
#pragma unroll
      for (int k = 0; k < kKeyGroups; ++k) M = fmaxf(M, ml[k * 16 + row].x);
#pragma unroll
      for (int k = 0; k < kKeyGroups; ++k) {
        const float2 x = ml[k * 16 + row];
        f[k] = x.x == -INFINITY ? 0.f : ex2(x.x - M);
        L = fmaf(x.y, f[k], L);
      }
      const bool whole = w.t0 == 0 && w.t1 == w.cnt;
      const float inv = whole ? 1.f / L : 1.f;
      const size_t orow = static_cast<size_t>(s.tok0 + r / v.g) * v.H + w.hk * v.g + r % v.g;
      const int slot = 2 * c + (first_seg ? 0 : 1);
      const size_t prow = static_cast<size_t>(slot) * (16 * MB) + r;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {  // 4 columns at a time, the row's 8 threads side by side
        const int col = i * 32 + (tid & 7) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kKeyGroups; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(merge + (k * 16 + row) * SM::kStride + col);
          a.x = fmaf(x.x, f[k], a.x);
          a.y = fmaf(x.y, f[k], a.y);
          a.z = fmaf(x.z, f[k], a.z);
          a.w = fmaf(x.w, f[k], a.w);
        }
        if (whole)
          *reinterpret_cast<uint2*>(p.O + orow * D + col) =
              make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
        else
          *reinterpret_cast<float4*>(p.part_o + prow * D + col) = a;
      }
      if ((tid & 7) == 0) {
        if (whole) p.lse[orow] = (M + log2f(L)) * 0.69314718055994531f;
        else p.part_ml[prow] = make_float2(M, L);
      }
    }
    if (w.t0 == 0 && tid == 0 && m == 0) {  // the pair's first segment names its slots
      const int slots = deal.whole ? 1 : deal.owner(w.at + w.cnt - 1) - c + 1;
      p.info[static_cast<size_t>(w.b) * v.Hk + w.hk] = make_int2(2 * c + (first_seg ? 0 : 1), slots);
    }
    named_bar(1 + m, 32 * kKeyGroups);  // the staging area is free again
  }
}

}  // namespace paged
}  // namespace cswattn
