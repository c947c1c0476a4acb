// paged_append.cuh -- the prologue of new tokens into a paged cache:
// q~ = RoPE(n(q)) to q_out, k~ = RoPE(n(k)) and v_eff = v + 3 sigmoid(gate) ve
// to their rows of the pages, the rows' accumulated weight to 0 and their
// position to the token's.
//
// RoPE in its usual forms: pairs (i, i + R/2) or (2i, 2i + 1) of the first R
// elements of a head (the rest passes through), each pair with its own
// frequency (so that stretched contexts are a choice of frequencies), cos and
// sin times a common factor. The angle pos * omega_i is a product in float64,
// reduced to a fraction of a turn before it is rounded to float32: far
// positions lose nothing (in float32 the product alone is off by 0.03 rad at
// position 2^19).
//
// Bound by HBM (one read and one write per element): 8150 tokens of 16 + 4
// heads 28.9 us = 3.8 TB/s (a copy of a kernel this short reaches 4.5); 25
// tokens 7.4 us. Staging the tokens in shared memory by bulk copies took 33.8
// us, holding rows in registers ahead of the setup 30 to 41: both cost CTAs in
// flight. A CTA takes kAppendTok consecutive tokens: its threads find the
// tokens' sequences by one coalesced pass over new_start, fill a cos/sin table,
// then walk the rows. A row of D elements belongs to D / 16 lanes, 16 elements
// each as two 16-byte vectors: with the half layout lane l < R/16 holds
// [8l, 8l + 8) of both halves of the rotary part, so each pair is inside one
// lane; all others hold 16 consecutive elements.
#pragma once
#include "paged.cuh"

namespace cswattn {
namespace paged {

constexpr int kAppendThreads = 256;
constexpr int kAppendTok = 8;

struct AppendParams {
  View v;
  int has_ve, rotary_pairs;
  float eps, factor;
  double turns[kMaxHalfD];  // omega_i / 2 pi: turns per position
  const __nv_bfloat16 *q, *k, *val, *ve, *gate;
  const int* positions;  // (n_tokens), or null: a token's position is its row
  __nv_bfloat16 *q_out, *k_pages, *v_pages;
  float* weight;   // (n_pages, Hk, page_size), or null
  int* position;   // likewise
};

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 16;                       // lanes per row
  constexpr int RPP = kAppendThreads / LPR;         // rows per pass
  using V8 = Vec16<__nv_bfloat16>;
  __shared__ __align__(16) float s_cos[kAppendTok][D / 2], s_sin[kAppendTok][D / 2];
  __shared__ int s_seq[kAppendTok], s_pos[kAppendTok];
  __shared__ int s_page[kAppendTok], s_slot[kAppendTok];
  const View& v = p.v;
  const int t0 = blockIdx.x * kAppendTok;
  const int ntt = min(kAppendTok, v.n_tokens - t0);
  pdl_launch_dependents();
  if (threadIdx.x < kAppendTok) s_seq[threadIdx.x] = -1;
  __syncthreads();
  pdl_wait();
  for (int b = threadIdx.x; b < v.B; b += kAppendThreads) {
    const int lo = v.new_start[b], hi = v.new_start[b + 1];
    // Only a sequence whose lengths fit has tokens: the range of one that does
    // not may lie over another's. One CTA reports them.
    const bool here = lo < t0 + ntt && hi > t0;
    Seq s;
    if (!(here || blockIdx.x == 0) || !seq_load(v, b, blockIdx.x == 0, s)) continue;
    for (int tt = max(0, s.tok0 - t0); tt < min(ntt, s.tok0 + s.n - t0); ++tt) s_seq[tt] = b;
  }
  __syncthreads();
  if (threadIdx.x < ntt) {
    const int tt = threadIdx.x, b = s_seq[tt];
    int page = -1;
    if (b >= 0) {
      Seq s;
      seq_load(v, b, false, s);
      const int row = s.L + (t0 + tt - s.tok0);
      page = page_at(v, b, page_entry(v, row));
      s_slot[tt] = page_slot(v, row);
      s_pos[tt] = p.positions ? p.positions[t0 + tt] : row;
    }
    s_page[tt] = page;  // -1: the token belongs to nobody, or has no place
  }
  __syncthreads();
  for (int e = threadIdx.x; e < ntt * p.rotary_pairs; e += kAppendThreads) {
    const int tt = e / p.rotary_pairs, i = e % p.rotary_pairs;
    if (s_page[tt] < 0) continue;
    const double turn = static_cast<double>(s_pos[tt]) * p.turns[i];
    float sn, cs;
    sincospif(2.f * static_cast<float>(turn - rint(turn)), &sn, &cs);
    s_cos[tt][i] = cs * p.factor;
    s_sin[tt][i] = sn * p.factor;
  }
  if (p.weight)
    for (int e = threadIdx.x; e < ntt * v.Hk; e += kAppendThreads) {
      const int tt = e / v.Hk, hk = e % v.Hk;
      if (s_page[tt] < 0) continue;
      const size_t at = term_index(v, s_page[tt], s_slot[tt], hk);
      p.weight[at] = 0.f;
      p.position[at] = s_pos[tt];
    }
  __syncthreads();

  const int rows_per_tok = v.H + 2 * v.Hk;
  const int total = ntt * rows_per_tok;
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const bool rotates = sub * 8 < p.rotary_pairs;  // rotary_pairs is a multiple of 8
  const int lo = (!INTERLEAVED && rotates) ? 8 * sub : 16 * sub;
  const int hi = (!INTERLEAVED && rotates) ? p.rotary_pairs + 8 * sub : 16 * sub + 8;
  RowCursor cur{0, 0};
  cur.advance(grp, rows_per_tok);
  for (int base = 0; base < total; base += RPP) {  // every lane takes part in every shuffle
    const bool in = base + grp < total;
    const int tt = in ? cur.tt : 0, kr = in ? cur.kind_row : 0;
    cur.advance(RPP, rows_per_tok);
    const int page = s_page[tt];
    const bool valid = in && page >= 0;
    const int kind = kr < v.H ? 0 : (kr < v.H + v.Hk ? 1 : 2);
    const int head = kind == 0 ? kr : (kind == 1 ? kr - v.H : kr - v.H - v.Hk);
    const size_t src = (static_cast<size_t>(t0 + tt) * (kind == 0 ? v.H : v.Hk) + head) * D;
    const __nv_bfloat16* x = kind == 0 ? p.q : (kind == 1 ? p.k : p.val);
    float a[8], b[8];
    if (valid) {
      V8::load(x + src + lo, a);
      V8::load(x + src + hi, b);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    ss = row_sum<LPR>(ss);
    if (!valid) continue;
    __nv_bfloat16* out;
    if (kind == 2) {
      if (p.has_ve) {
        float ea[8], eb[8];
        V8::load(p.ve + src + lo, ea);
        V8::load(p.ve + src + hi, eb);
        const float gl = __bfloat162float(p.gate[static_cast<size_t>(t0 + tt) * v.Hk + head]);
        const float coef = 3.0f / (1.0f + expf(-gl));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = fmaf(coef, ea[i], a[i]);
          b[i] = fmaf(coef, eb[i], b[i]);
        }
      }
      out = p.v_pages + kv_index(v, page, s_slot[tt], head) * D;
    } else {
      const float rstd = rsqrtf(ss / static_cast<float>(D) + p.eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= rstd;
        b[i] *= rstd;
      }
      if (rotates) {
        const float *cs = &s_cos[tt][8 * sub], *sn = &s_sin[tt][8 * sub];
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
            a[2 * i] = a0 * cs[i] - a1 * sn[i];
            a[2 * i + 1] = a0 * sn[i] + a1 * cs[i];
            b[2 * i] = b0 * cs[4 + i] - b1 * sn[4 + i];
            b[2 * i + 1] = b0 * sn[4 + i] + b1 * cs[4 + i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x0 = a[i], x1 = b[i];
            a[i] = x0 * cs[i] - x1 * sn[i];
            b[i] = x0 * sn[i] + x1 * cs[i];
          }
        }
      }
      out = kind == 0 ? p.q_out + src : p.k_pages + kv_index(v, page, s_slot[tt], head) * D;
    }
    V8::store(out + lo, a);
    V8::store(out + hi, b);
  }
}

}  // namespace paged
}  // namespace cswattn
