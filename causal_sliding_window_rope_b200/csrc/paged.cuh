// paged.cuh -- what the paged-cache kernels share: the batch as the device
// sees it, the lookup of a token's sequence and of a row's page.
//
// Page "5만원으로 나만의 ChatGPT 훈련하는 방법", section "6. 추론 엔진
// (nanochat/engine.py)": generation over a pre-filled KV cache. Here the
// cache rows of a sequence lie in pages of `page_size` rows, in any order of
// pages, and a call takes any number of new tokens per sequence.
//
// Sequence b has L = cache_len[b] rows before the call and the tokens
// new_start[b] .. new_start[b + 1] of the call; token i of it is row L + i.
// The lengths live on the device, so the host cannot check them: each kernel
// checks a sequence before it touches it (seq_load) and reports one that does
// not fit through the status word; such a sequence is left alone.
#pragma once
#include <climits>

#include "prologue.cuh"
#include "decode.cuh"

namespace cswattn {
namespace paged {

// 3-D tile load global -> shared, completing on an mbarrier (no multicast).
__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* dst, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// mma_ss, mma_ts and mma_commit for a warp whose 32 lanes run the issuing code together:
// only the lane with `leader` set (elect_one) issues. Loop counters and
// descriptors are then the same in all lanes and can live in the registers
// that a warp shares, which the instruction takes its operands from; a lone
// thread moves every operand there first, and is slower than the product.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_ss_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_commit_warp(uint64_t* bar, uint32_t leader) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(leader)
      : "memory");
}


constexpr int kMaxSeqs = 4096;   // sequences of one call (the kernels scan their lengths)
constexpr int kUnit = 16;        // rows: a page holds whole units, so a unit never straddles pages

struct View {
  int B, T, H, Hk, g, W;
  int page_size, n_pages, pages_per_seq;
  int page_shift;  // log2(page_size), or -1
  int n_tokens, max_new;
  const int *page_table, *cache_len, *new_start;
};

struct Seq {
  int L, n, tok0;  // rows before the call, new tokens, first of them
};

// False (and reported, by the thread that `report` selects) when the lengths
// of sequence b do not fit the call; the sequence then counts as empty.
__device__ __forceinline__ bool seq_load(const View& v, int b, bool report, Seq& s) {
  s.L = v.cache_len[b];
  s.tok0 = v.new_start[b];
  const int end = v.new_start[b + 1];
  const bool ok = s.L >= 0 && s.tok0 >= 0 && end >= s.tok0 && end <= v.n_tokens && end - s.tok0 <= v.max_new &&
                  s.L <= v.T - (end - s.tok0);
  s.n = ok ? end - s.tok0 : 0;
  if (!ok) {
    s.L = 0;
    if (report) atomicOr(&g_status, kStatusRange);
  }
  return ok;
}

// Page of a row of sequence b; -1 (and reported) when the table's entry is
// not a page of the pool. row < T <= pages_per_seq * page_size.
__device__ __forceinline__ int page_at(const View& v, int b, int entry) {
  const int p = v.page_table[static_cast<size_t>(b) * v.pages_per_seq + entry];
  if (p >= 0 && p < v.n_pages) return p;
  atomicOr(&g_status, kStatusRange);
  return -1;
}

// A row's entry of the page table and its slot in the page: shifts where the
// page is a power of two (a division costs some 20 instructions).
__device__ __forceinline__ int page_entry(const View& v, int row) {
  return v.page_shift >= 0 ? row >> v.page_shift : row / v.page_size;
}
__device__ __forceinline__ int page_slot(const View& v, int row) {
  return v.page_shift >= 0 ? row & (v.page_size - 1) : row % v.page_size;
}

// Pages of a producer warp's units: lane l's unit is rows [row, row + unit) of
// block 0, and the same of every `step` rows. The warp holds 32 entries of the
// page table, one per lane, so the table's latency is paid once in 32 pages;
// entries of rows that no token sees are not read, and the box of such a unit
// lies past the pool, which reads as zeros.
struct UnitPages {
  const View& v;
  const int* table;  // the sequence's row of the page table
  int row, step, unit, lo, end, held, base;
  static constexpr int kNone = INT_MIN;
  __device__ UnitPages(const View& v_, int b, const Seq& s, int row_, int step_, int unit_)
      : v(v_), table(v_.page_table + static_cast<size_t>(b) * v_.pages_per_seq), row(row_), step(step_), unit(unit_),
        lo(max(0, s.L - v_.W + 1)), end(s.L + s.n), held(kNone), base(INT_MIN / 2) {}
  // All lanes call; those with `mine` get their unit's page of block t.
  __device__ int page(int t, bool mine) {
    const int r = row + t * step, e = page_entry(v, r);
    if (__any_sync(0xffffffffu, mine && (e < base || e >= base + 32))) {  // a block's units have at most 8 pages
      base = __shfl_sync(0xffffffffu, e, 0);
      const int mine_e = base + lane_id();
      held = mine_e >= page_entry(v, lo) && mine_e <= page_entry(v, end - 1) ? table[mine_e] : kNone;
    }
    const int p = __shfl_sync(0xffffffffu, held, e - base);
    if (!mine || r >= end || r + unit <= lo) return v.n_pages;
    if (p >= 0 && p < v.n_pages) return p;
    atomicOr(&g_status, kStatusRange);
    return v.n_pages;
  }
  __device__ int slot(int t) const { return page_slot(v, row + t * step); }
};

// Row of a (pages, page_size, Hk) pool of K or V rows (in units of head_dim
// elements) and of a (pages, Hk, page_size) pool of row terms.
__device__ __forceinline__ size_t kv_index(const View& v, int page, int slot, int hk) {
  return (static_cast<size_t>(page) * v.page_size + slot) * v.Hk + hk;
}
__device__ __forceinline__ size_t term_index(const View& v, int page, int slot, int hk) {
  return (static_cast<size_t>(page) * v.Hk + hk) * v.page_size + slot;
}

}  // namespace paged
}  // namespace cswattn
