// paged_plan.cuh -- how work on many query rows is dealt out. A sequence that
// has new tokens is a row of units per KV head, each of some blocks; the units
// of all of them follow one another, and CTA c of n takes the blocks
// [total c / n, total (c + 1) / n): whole units, and at most two cut ones.
// Each CTA finds its own run (find_run: all its threads add up the units of
// all sequences, which is quicker than a launch that does it for everybody)
// and leaves its start in the workspace for the kernel that joins cut units.
#pragma once
#include "paged.cuh"

namespace cswattn {
namespace paged {

constexpr int kSMs = 148;
constexpr int kMaxRuns = 2 * kSMs;  // CTAs that work may be dealt to
constexpr int kPlanMinBlocks = 2;   // fewest blocks worth a CTA of their own

// total c / n, in 32 bits where they hold the product (a 64-bit division costs
// a few hundred cycles, and a CTA's start is a tenth of a generation step).
static_assert(kMaxRuns < 512, "share_of in 32 bits");
__device__ __forceinline__ long long share_of(long long total, int c, int n) {
  if (total < (1 << 23)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(n);
  return total * c / n;
}

// Where a CTA's run starts: the k-th sequence that has tokens, KV head, unit, block of the unit.
struct Start {
  int k, hk, unit, t0;
};

// ... and with it what the join needs of the sequence, which is then one load away.
struct Begin {
  Start st;
  Seq s;
  int b;
};

struct Plan {
  Begin begin[kMaxRuns];
  int ctas;
};

// A CTA's run: `left` blocks from st on (in sequence s); none when left is 0.
struct Run {
  Start st;
  long long left;
  Seq s;
};

// Tiles of 128 cached rows that the tokens [i0, i1) of a sequence see.
__device__ __forceinline__ void token_blocks(const View& v, const Seq& s, int i0, int i1, int& lo, int& hi) {
  lo = max(0, s.L + i0 - v.W + 1) >> 7;
  hi = (s.L + i1 - 1) >> 7;
}

// Units of the attention: two tiles of tpt tokens; blocks: tiles of cached rows they see.
struct TokenUnits {
  int tpt;
  __device__ int count(const View&, const Seq& s) const { return (s.n + 2 * tpt - 1) / (2 * tpt); }
  __device__ void range(const View& v, const Seq& s, int u, int& lo, int& hi) const {
    token_blocks(v, s, u * 2 * tpt, min(s.n, (u + 1) * 2 * tpt), lo, hi);
  }
};

// Units of the row weights: a tile of 128 cached rows; blocks: tiles of tpt
// tokens that see it (tokens i with k <= L + i and L + i - W < k for a row k).
struct RowUnits {
  int tpt;
  __device__ int count(const View& v, const Seq& s) const {
    int lo, hi;
    token_blocks(v, s, 0, s.n, lo, hi);
    return hi - lo + 1;
  }
  __device__ int first_row(const View& v, const Seq& s, int u) const {
    return ((max(0, s.L - v.W + 1) >> 7) + u) * 128;
  }
  __device__ void range(const View& v, const Seq& s, int u, int& lo, int& hi) const {
    const long long k0 = first_row(v, s, u);
    lo = static_cast<int>(max(0ll, k0 - s.L)) / tpt;
    hi = static_cast<int>(min(s.n - 1ll, k0 + 126 - s.L + v.W)) / tpt;
  }
};

constexpr int kPlanSmem = 8 * (kMaxSeqs + 1) + 4 * 36 + 2 * kMaxSeqs;

// All threads of a CTA (a multiple of 32, at most 1024) call; `smem` is
// kPlanSmem bytes of scratch; `seqs` (the sequences that have tokens, in
// order) is written alike by every CTA. The result is in *run, in shared
// memory.
template <class Units>
__device__ __forceinline__ void find_run(const View& v, const Units& units, int runs, int c, Plan* plan,
                                         int* seqs, void* smem, Run* run) {
  long long* pre = static_cast<long long*>(smem);  // per such sequence: blocks of one KV head before it
  int* s_total = reinterpret_cast<int*>(pre + kMaxSeqs + 1);
  uint16_t* s_seqs = reinterpret_cast<uint16_t*>(s_total + 36);  // `seqs`, at hand
  static_assert(kMaxSeqs <= 1 << 16, "sequences in 16 bits");
  const int warp = warp_id(), lane = lane_id(), warps = blockDim.x >> 5;
  auto blocks = [&](const Seq& s, int u) -> int {
    int lo, hi;
    units.range(v, s, u, lo, hi);
    return hi - lo + 1;
  };
  int n_seqs = 0;
  for (int b0 = 0; b0 < v.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    bool yes = false;
    Seq s;
    if (b < v.B) yes = seq_load(v, b, c == 0, s) && s.n > 0;
    const uint32_t m = __ballot_sync(0xffffffffu, yes);
    if (lane == 0) s_total[warp] = __popc(m);
    __syncthreads();
    int before = n_seqs;
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += s_total[w];
      n_seqs += s_total[w];
    }
    if (yes) {
      const int k = before + __popc(m & ((1u << lane) - 1u)), n = units.count(v, s);
      seqs[k] = b;
      s_seqs[k] = static_cast<uint16_t>(b);
      long long sum = -1;  // few units: this thread adds them up; else a warp does
      if (n <= 8) {
        sum = 0;
        for (int u = 0; u < n; ++u) sum += blocks(s, u);
      }
      pre[k + 1] = sum;
    }
    __syncthreads();
  }
  for (int k = warp; k < n_seqs; k += warps) {
    if (pre[k + 1] >= 0) continue;
    Seq s;
    seq_load(v, s_seqs[k], false, s);
    const int n = units.count(v, s);
    long long sum = 0;
    for (int u = lane; u < n; u += 32) sum += blocks(s, u);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncwarp();
    if (lane == 0) pre[k + 1] = sum;
  }
  if (threadIdx.x == 0) {
    pre[0] = 0;
    run->left = 0;
  }
  __syncthreads();
  if (warp == 0) {
    long long sum = 0;
    for (int k0 = 0; k0 < n_seqs; k0 += 32) {
      long long x = k0 + lane < n_seqs ? pre[k0 + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (k0 + lane < n_seqs) pre[k0 + lane + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    __syncwarp();
    const long long total = sum * v.Hk;
    const long long most = (total + kPlanMinBlocks - 1) / kPlanMinBlocks;
    const int ctas = static_cast<int>(most < runs ? most : runs);
    if (c == 0 && lane == 0) plan->ctas = ctas;
    if (c < ctas) {
      const long long at = share_of(total, c, ctas);
      int lo = 0, hi = n_seqs;  // the last k with pre[k] * Hk <= at
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] * v.Hk <= at) lo = mid;
        else hi = mid;
      }
      Seq s;
      seq_load(v, s_seqs[lo], false, s);
      const long long cnt = pre[lo + 1] - pre[lo], rem = at - pre[lo] * v.Hk;
      const int hk = total < INT_MAX ? static_cast<int>(rem) / static_cast<int>(cnt) : static_cast<int>(rem / cnt);
      long long left = rem - hk * cnt;
      const int n = units.count(v, s);
      for (int u0 = 0; u0 < n; u0 += 32) {  // 32 units at a time: the one that holds block `left`
        const int u = u0 + lane;
        const int mine = u < n ? blocks(s, u) : 0;
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += y;
        }
        const bool here = u < n && left >= inc - mine && left < inc;
        if (here) {
          const Start st{lo, hk, u, static_cast<int>(left) - (inc - mine)};
          plan->begin[c] = Begin{st, s, s_seqs[lo]};
          run->st = st;
          run->s = s;
          run->left = share_of(total, c + 1, ctas) - at;
        }
        if (__any_sync(0xffffffffu, here)) break;
        left -= __shfl_sync(0xffffffffu, inc, 31);
      }
    }
  }
  __syncthreads();
}

// A CTA's walk over its run: one segment (blocks [first + t0, first + t1) of a unit) at a time.
template <class Units>
struct UnitWalk {
  const View& v;
  const Units units;
  const int* seqs;
  long long left;
  int k, hk, u, t0, t1, cnt, n_units, first;
  Seq s;
  __device__ UnitWalk(const View& v_, const Units& units_, const Run& run, const int* seqs_)
      : v(v_), units(units_), seqs(seqs_), left(run.left), k(run.st.k), hk(run.st.hk), u(run.st.unit), t0(run.st.t0),
        s(run.s) {
    n_units = units.count(v, s);
    set();
  }
  __device__ int seq() const { return seqs[k]; }
  __device__ void load() {
    seq_load(v, seqs[k], false, s);
    n_units = units.count(v, s);
  }
  __device__ void set() {
    int hi;
    units.range(v, s, u, first, hi);
    cnt = hi - first + 1;
    t1 = left < cnt - t0 ? t0 + static_cast<int>(left) : cnt;
  }
  __device__ bool valid() const { return left > 0; }
  __device__ bool whole() const { return t0 == 0 && t1 == cnt; }
  __device__ void next() {
    left -= t1 - t0;
    t0 = 0;
    if (left <= 0) return;
    if (++u == n_units) {
      u = 0;
      if (++hk == v.Hk) {
        hk = 0;
        ++k;
        load();
      }
    }
    set();
  }
};

// The unit that is cut at the start of CTA c's run: its n shares lie with
// consecutive CTAs, share k at slot(k) (a CTA has two slots, one for its first
// segment and one for a later one), and c is the nth-th of its n - 1 cuts. All
// lanes of a warp call find, which reads the starts of 32 CTAs to either side
// at once.
struct Cut {
  Start st;
  Seq s;
  int b, n, nth, slot0, slot1;
  __device__ bool find(const Plan* plan, int c) {
    const int lane = lane_id();
    auto start = [&](int i) { return i >= 0 && i < kMaxRuns ? plan->begin[i].st : Start{-1, -1, -1, -1}; };
    Start back = start(c - 1 - lane), on = start(c + 1 + lane);
    const Begin mine = plan->begin[c];
    const int ctas = plan->ctas;
    if (c >= ctas || mine.st.t0 == 0) return false;
    st = mine.st;
    s = mine.s;
    b = mine.b;
    auto within = [&](const Start& x) { return x.k == st.k && x.hk == st.hk && x.unit == st.unit; };
    int first = c, last = c;  // of the CTAs that start in the unit, past its beginning
    bool same;                // the CTA before those starts at its beginning
    for (;;) {
      const bool in = within(back);
      const uint32_t m = __ballot_sync(0xffffffffu, in && back.t0 > 0);
      const int t = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      first -= t;
      if (t < 32) {
        same = __shfl_sync(0xffffffffu, in, t);
        break;
      }
      back = start(first - 1 - lane);
    }
    for (;;) {
      const uint32_t m = __ballot_sync(0xffffffffu, last + 1 + lane < ctas && within(on));
      const int t = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      last += t;
      if (t < 32) break;
      on = start(last + 1 + lane);
    }
    n = last - first + 2;
    nth = c - first;
    slot0 = 2 * (first - 1) + (same ? 0 : 1);
    slot1 = 2 * first;
    return true;
  }
  __device__ int slot(int k) const { return k == 0 ? slot0 : slot1 + 2 * (k - 1); }
};

}  // namespace paged
}  // namespace cswattn
