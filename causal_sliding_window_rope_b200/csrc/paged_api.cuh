// paged_api.cuh -- C ABI of the paged cache: host-side validation and
// launches. Included by cswattn.cu, whose helpers it uses.
#pragma once

namespace {

constexpr int kMaxPagedGroup = 128;  // query heads per KV head: one token's rows fit one tile

// Checks the layer and the batch's sizes; needs_tokens: the call reads the
// new tokens (n_tokens, max_new, new_start).
cswattn_status check_paged(const cswattn_layer* layer, const cswattn_paged* pg, bool needs_tokens, Shape* s,
                           paged::View* v) {
  if (!layer) return fail(CSWATTN_ERR_INVALID_ARG, "layer is NULL");
  if (!pg) return fail(CSWATTN_ERR_INVALID_ARG, "paged is NULL");
  if (layer->B < 1) return fail(CSWATTN_ERR_INVALID_ARG, "B must be >= 1");
  cswattn_layer one = *layer;  // T is a bound on each sequence, not B dense ones
  one.B = 1;
  cswattn_status st = check_layer(&one, s);
  if (st != CSWATTN_OK) return st;
  s->B = layer->B;
  if (!s->bf16) return fail(CSWATTN_ERR_UNSUPPORTED, "the paged cache supports bf16 layers only");
  if (s->g > kMaxPagedGroup)
    return fail(CSWATTN_ERR_UNSUPPORTED, "the paged cache supports up to %d query heads per KV head (got %d)",
                kMaxPagedGroup, s->g);
  if (s->B > paged::kMaxSeqs)
    return fail(CSWATTN_ERR_UNSUPPORTED, "the paged cache supports up to %d sequences (got %d)", paged::kMaxSeqs,
                s->B);
  if (pg->page_size < 1 || pg->n_pages < 1 || pg->pages_per_seq < 1)
    return fail(CSWATTN_ERR_INVALID_ARG, "page_size, n_pages and pages_per_seq must be >= 1");
  if (pg->page_size % paged::kUnit != 0)
    return fail(CSWATTN_ERR_UNSUPPORTED, "page_size must be a multiple of %d (got %d)", paged::kUnit,
                pg->page_size);
  if (static_cast<long long>(pg->pages_per_seq) * pg->page_size < s->T)
    return fail(CSWATTN_ERR_INVALID_ARG, "T = %d rows do not fit %d pages of %d", s->T, pg->pages_per_seq,
                pg->page_size);
  // The pools' byte strides are those of a tensor map (below 2^40).
  if (static_cast<double>(pg->page_size) * s->Hk * s->D >= 5e11)
    return fail(CSWATTN_ERR_UNSUPPORTED, "page too large");
  CHECK_PTR(pg->page_table, 4);
  CHECK_PTR(pg->cache_len, 4);
  if (needs_tokens) {
    CHECK_PTR(pg->new_start, 4);
    if (pg->n_tokens < 0) return fail(CSWATTN_ERR_INVALID_ARG, "n_tokens must be >= 0 (got %d)", pg->n_tokens);
    if (pg->max_new < 1 || pg->max_new > s->T)
      return fail(CSWATTN_ERR_INVALID_ARG, "max_new must be in [1, T = %d] (got %d)", s->T, pg->max_new);
  }
  v->B = s->B;
  v->T = s->T;
  v->H = s->H;
  v->Hk = s->Hk;
  v->g = s->g;
  v->W = s->W;
  v->page_size = pg->page_size;
  v->page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (pg->page_size == 1 << i) v->page_shift = i;
  v->n_pages = pg->n_pages;
  v->pages_per_seq = pg->pages_per_seq;
  v->n_tokens = pg->n_tokens;
  v->max_new = pg->max_new;
  v->page_table = pg->page_table;
  v->cache_len = pg->cache_len;
  v->new_start = pg->new_start;
  return CSWATTN_OK;
}

// Rows of a TMA box: the largest power of two that divides the page, at most
// `most`; a block of rows is read as boxes that lie in one page each.
int page_unit(int page_size, int most) {
  int u = paged::kUnit;
  while (u < most && page_size % (2 * u) == 0) u *= 2;
  return u;
}

// A call whose sequences have at most 32 query rows (new tokens x heads of a
// group) each runs rows_kernel; any other runs tile_kernel for all of its
// sequences: few rows leave most of a tile empty there, but it reads the
// cache as fast, and one launch of each kind fewer counts (31 single tokens
// over 2000 rows beside a chunk of 512 tokens 61 us, 71 with rows_kernel for
// the 31; 200 over 300 rows beside a chunk of 64 63 us, 74).
struct PagedWorkspace {
  bool tiles;
  int rows;  // query rows of a share: 16 or 32, or a unit's 256
  float* part_o;
  float2* part_ml;
  int2* info;          // rows_kernel: the pairs' shares
  paged::Plan* plan;   // tile_kernel: the CTAs' runs, and the sequences in order
  int* seqs;
  size_t bytes;
};

PagedWorkspace carve_paged(const Shape& s, const paged::View& v, void* base) {
  uint8_t* p = static_cast<uint8_t*>(base);
  PagedWorkspace w;
  const long long most = static_cast<long long>(v.max_new) * s.g;
  w.tiles = most > 32;
  w.rows = w.tiles ? 256 : (most > 16 ? 32 : 16);
  const size_t rows = static_cast<size_t>(2 * paged::kSMs) * w.rows;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void* at = p + off;
    off += pad256(bytes);
    return at;
  };
  w.part_o = static_cast<float*>(take(rows * s.D * 4));
  w.part_ml = static_cast<float2*>(take(rows * 8));
  w.info = nullptr;
  w.plan = nullptr;
  w.seqs = nullptr;
  if (w.tiles) {
    w.plan = static_cast<paged::Plan*>(take(sizeof(paged::Plan)));
    w.seqs = static_cast<int*>(take(static_cast<size_t>(s.B) * 4));
  } else {
    w.info = static_cast<int2*>(take(static_cast<size_t>(s.B) * s.Hk * 8));
  }
  w.bytes = off;
  return w;
}

// Tensor map of q (n_tokens, H, D) whose box is one 64-column panel of `tpt`
// tokens x g heads: the 128 rows (or fewer) of a tile, tokens outermost.
cswattn_status make_map_group(CUtensorMap* map, const void* base, int n_tokens, int H, int D, int g, int tpt) {
  EncodeTiledFn enc;
  cswattn_status s = get_encoder(&enc);
  if (s != CSWATTN_OK) return s;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                              static_cast<cuuint64_t>(n_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(g), static_cast<cuuint32_t>(tpt)};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(CSWATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return CSWATTN_OK;
}

template <int D, int MB>
cswattn_status prepare_rows_kernel() {
  return set_smem(paged::rows_kernel<D, MB>, paged::RowsSmem<D, MB>::kBytes + 4 * (paged::kMaxSeqs + 1));
}
template <int D, int MB>
void launch_rows_kernel(const paged::RowsParams& rp, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  launch_pdl(paged::rows_kernel<D, MB>, dim3(paged::kSMs), dim3(32 * (paged::kKeyGroups * MB + 1)),
             static_cast<size_t>(paged::RowsSmem<D, MB>::kBytes) + 4 * (rp.v.B + 1), st, mk, mv, rp);
}

// The attention of few query rows or that of many, and the join of what it
// has cut. With prepare_only, sets what the launches need: a call that may
// fail is made before anything of an entry point is enqueued.
template <int D>
cswattn_status launch_paged(const paged::RowsParams& rp, const paged::TileParams& tp, const paged::JoinParams& jp,
                            bool tiles, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mq,
                            cudaStream_t st, bool prepare_only) {
  const bool wide = jp.rows > 16;
  if (prepare_only) {
    if (tiles) return set_smem(paged::tile_kernel<D>, paged::TileSmem<D>::kBytes);
    return wide ? prepare_rows_kernel<D, 2>() : prepare_rows_kernel<D, 1>();
  }
  if (tiles)
    launch_pdl(paged::tile_kernel<D>, dim3(paged::kSMs), dim3(paged::kTileThreads), paged::TileSmem<D>::kBytes, st,
               mq, mk, mv, tp);
  else if (wide)
    launch_rows_kernel<D, 2>(rp, mk, mv, st);
  else
    launch_rows_kernel<D, 1>(rp, mk, mv, st);
  const dim3 grid(tiles ? (paged::kSMs - 1) * paged::kJoinUnitCtas : static_cast<unsigned>(rp.v.B) * rp.v.Hk);
  launch_pdl(tiles ? paged::join_kernel<D, true> : paged::join_kernel<D, false>, grid, dim3(32 * paged::kJoinWarps), 0,
             st, jp);
  return CSWATTN_OK;
}

struct WeighWorkspace {
  paged::Plan* plan;
  int* seqs;
  float* part;
  int max_rows;  // query rows of a sequence that the kernel of few is compiled for
  bool tiles;    // a sequence may have more
  size_t bytes;
};

// A call whose sequences have at most 32 query rows (new tokens x heads of a
// group) runs weigh_rows_kernel, one with more runs weigh_tile_kernel for all
// of its sequences, single tokens too. Both launched, each for its sequences,
// is the slower for 31 single tokens over 2000 rows beside a chunk of 512
// tokens (38.2 us, 36.3) and for 8 sequences of 64 tokens (12.8, 10.8), the
// faster for 63 single tokens over 4000 rows beside a chunk of 64 (79.9, 90.6)
// and for 31 over 2000 beside one of 20 (30.8, 32.5): many long caches beside
// a short chunk lose by it, short caches and long chunks gain, and the host,
// which knows max_new alone, cannot tell them apart.
WeighWorkspace carve_weigh(const Shape& s, const paged::View& v, void* base) {
  uint8_t* p = static_cast<uint8_t*>(base);
  WeighWorkspace w;
  const long long rows = static_cast<long long>(v.max_new) * s.g;
  w.max_rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : 32);
  w.tiles = rows > w.max_rows;
  w.plan = nullptr;
  w.seqs = nullptr;
  w.part = nullptr;
  w.bytes = 0;
  if (!w.tiles) return w;
  size_t off = 0;
  w.plan = reinterpret_cast<paged::Plan*>(p + off);
  off += pad256(sizeof(paged::Plan));
  w.seqs = reinterpret_cast<int*>(p + off);
  off += pad256(static_cast<size_t>(s.B) * 4);
  w.part = reinterpret_cast<float*>(p + off);
  off += pad256(static_cast<size_t>(2 * paged::kWeighRuns) * 128 * 4);
  w.bytes = off;
  return w;
}

template <int D, int NT>
cswattn_status launch_weigh_rows(const paged::WeighRowsParams& rp, const CUtensorMap& mk, cudaStream_t st,
                                 bool prepare_only) {
  using SM = paged::WeighRowsSmem<D>;
  if (prepare_only) return set_smem(paged::weigh_rows_kernel<D, NT>, SM::kBytes + 4 * (paged::kMaxSeqs + 1));
  launch_pdl(paged::weigh_rows_kernel<D, NT>, dim3(paged::kSMs), dim3(32 * (4 * paged::WeighGroups<NT>::value + 1)),
             static_cast<size_t>(SM::kBytes) + 4 * (rp.v.B + 1), st, mk, rp);
  return CSWATTN_OK;
}

// As launch_paged, for the row weights.
template <int D>
cswattn_status launch_weigh(const paged::WeighRowsParams& rp, const paged::WeighTileParams& tp, bool tiles,
                            int max_rows, const CUtensorMap& mk, const CUtensorMap& mq, cudaStream_t st,
                            bool prepare_only) {
  if (!tiles)
    return max_rows == 8    ? launch_weigh_rows<D, 1>(rp, mk, st, prepare_only)
           : max_rows == 16 ? launch_weigh_rows<D, 2>(rp, mk, st, prepare_only)
                            : launch_weigh_rows<D, 4>(rp, mk, st, prepare_only);
  if (prepare_only) return set_smem(paged::weigh_tile_kernel<D>, paged::WeighTileSmem<D>::kBytes);
  launch_pdl(paged::weigh_tile_kernel<D>, dim3(paged::kWeighRuns), dim3(paged::kWeighThreads),
             paged::WeighTileSmem<D>::kBytes, st, mq, mk, tp);
  launch_pdl(paged::weigh_join_kernel, dim3(paged::kWeighRuns - 1), dim3(128), 0, st, tp);
  return CSWATTN_OK;
}

}  // namespace

extern "C" {

cswattn_status attn_paged_append(const cswattn_layer* layer, const cswattn_paged* paged, const cswattn_rope* rope,
                                 const void* q, const void* k, const void* v, const void* ve, const void* gate,
                                 const int* positions, void* q_out, void* k_pages, void* v_pages, float* weight,
                                 int* position, void* stream) {
  const NvtxRange nvtx_range("attn_paged_append");
  Shape s;
  paged::AppendParams ap;
  cswattn_status st = check_paged(layer, paged, true, &s, &ap.v);
  if (st != CSWATTN_OK) return st;
  ap.rotary_pairs = s.D / 2;
  ap.factor = 1.f;
  bool interleaved = false;
  const double* freq = nullptr;
  if (rope) {
    if (rope->rotary_dim < 1 || rope->rotary_dim > s.D || (rope->interleaved != 0 && rope->interleaved != 1))
      return fail(CSWATTN_ERR_INVALID_ARG, "rotary_dim must be in [1, head_dim], interleaved 0 or 1");
    if (rope->rotary_dim % 16 != 0)
      return fail(CSWATTN_ERR_UNSUPPORTED, "rotary_dim must be a multiple of 16 (got %d)", rope->rotary_dim);
    if (!(rope->factor > 0.f) || !std::isfinite(rope->factor))
      return fail(CSWATTN_ERR_INVALID_ARG, "rope factor must be finite and > 0");
    ap.rotary_pairs = rope->rotary_dim / 2;
    ap.factor = rope->factor;
    interleaved = rope->interleaved != 0;
    freq = rope->frequencies;
  }
  for (int i = 0; i < ap.rotary_pairs; ++i) {
    const double w = freq ? freq[i] : std::pow(static_cast<double>(layer->rope_base), -1.0 * i / ap.rotary_pairs);
    if (!std::isfinite(w)) return fail(CSWATTN_ERR_INVALID_ARG, "rope frequency %d is not finite", i);
    ap.turns[i] = w / 6.283185307179586476925;
  }
  if (paged->n_tokens == 0) return CSWATTN_OK;
  CHECK_PTR(q, 16);
  CHECK_PTR(k, 16);
  CHECK_PTR(v, 16);
  CHECK_PTR(q_out, 16);
  CHECK_PTR(k_pages, 16);
  CHECK_PTR(v_pages, 16);
  if (layer->has_ve) {
    CHECK_PTR(ve, 16);
    CHECK_PTR(gate, 2);
  }
  if (positions) CHECK_PTR(positions, 4);
  if ((weight == nullptr) != (position == nullptr))
    return fail(CSWATTN_ERR_INVALID_ARG, "weight and position must be given both or neither");
  if (weight) {
    CHECK_PTR(weight, 4);
    CHECK_PTR(position, 4);
  }
  if (k_pages == v_pages) return fail(CSWATTN_ERR_INVALID_ARG, "k_pages and v_pages must differ");
  if (q_out == q || q_out == k || q_out == v || q_out == ve)
    return fail(CSWATTN_ERR_INVALID_ARG, "q_out must not alias an input");
  ap.has_ve = layer->has_ve;
  ap.eps = layer->eps;
  ap.q = static_cast<const __nv_bfloat16*>(q);
  ap.k = static_cast<const __nv_bfloat16*>(k);
  ap.val = static_cast<const __nv_bfloat16*>(v);
  ap.ve = static_cast<const __nv_bfloat16*>(ve);
  ap.gate = static_cast<const __nv_bfloat16*>(gate);
  ap.positions = positions;
  ap.q_out = static_cast<__nv_bfloat16*>(q_out);
  ap.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  ap.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  ap.weight = weight;
  ap.position = position;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const dim3 grid((paged->n_tokens + paged::kAppendTok - 1) / paged::kAppendTok);
  {
    ScopedTiming tm(CSWATTN_K_PROLOGUE, cs);
    if (s.D == 64)
      launch_pdl(interleaved ? paged::append_kernel<64, true> : paged::append_kernel<64, false>, grid,
                 dim3(paged::kAppendThreads), 0, cs, ap);
    else
      launch_pdl(interleaved ? paged::append_kernel<128, true> : paged::append_kernel<128, false>, grid,
                 dim3(paged::kAppendThreads), 0, cs, ap);
  }
  return launched("paged append launch");
}

size_t attn_paged_workspace_bytes(const cswattn_layer* layer, const cswattn_paged* paged) {
  Shape s;
  paged::View v;
  if (check_paged(layer, paged, true, &s, &v) != CSWATTN_OK) return 0;
  return carve_paged(s, v, nullptr).bytes;
}

cswattn_status attn_paged(const cswattn_layer* layer, const cswattn_paged* paged, const void* q_out,
                          const void* k_pages, const void* v_pages, void* O, float* lse, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const NvtxRange nvtx_range("attn_paged");
  Shape s;
  paged::View v;
  cswattn_status st = check_paged(layer, paged, true, &s, &v);
  if (st != CSWATTN_OK) return st;
  if (paged->n_tokens == 0) return CSWATTN_OK;
  CHECK_PTR(q_out, 16);
  CHECK_PTR(k_pages, 16);
  CHECK_PTR(v_pages, 16);
  CHECK_PTR(O, 16);
  CHECK_PTR(lse, 4);
  CHECK_PTR(workspace, 256);
  if (O == q_out) return fail(CSWATTN_ERR_INVALID_ARG, "O must not alias q_out");
  const PagedWorkspace w = carve_paged(s, v, workspace);
  if (workspace_bytes < w.bytes)
    return fail(CSWATTN_ERR_INVALID_ARG, "paged workspace too small: %zu < %zu bytes", workspace_bytes, w.bytes);
  const int unit = page_unit(v.page_size, w.tiles ? 128 : paged::kBlk);
  paged::RowsParams rp;
  rp.v = v;
  rp.scale_log2 = s.scale * 1.4426950408889634f;
  rp.unit = unit;
  rp.q = static_cast<const __nv_bfloat16*>(q_out);
  rp.O = static_cast<__nv_bfloat16*>(O);
  rp.lse = lse;
  rp.part_o = w.part_o;
  rp.part_ml = w.part_ml;
  rp.info = w.info;
  rp.wait_ns = g_wait_ns.load();
  paged::TileParams tp;
  tp.v = v;
  tp.scale_log2 = rp.scale_log2;
  tp.unit = unit;
  tp.tpt = 128 / s.g;
  tp.plan = w.plan;
  tp.seqs = w.seqs;
  tp.O = rp.O;
  tp.lse = lse;
  tp.part_o = w.part_o;
  tp.part_ml = w.part_ml;
  tp.wait_ns = rp.wait_ns;
  paged::JoinParams jp;
  jp.v = v;
  jp.rows = w.rows;
  jp.tpt = tp.tpt;
  jp.part_o = w.part_o;
  jp.part_ml = w.part_ml;
  jp.info = w.info;
  jp.plan = w.plan;
  jp.O = rp.O;
  jp.lse = lse;
  // What may fail is done before anything is enqueued.
  CUtensorMap mk, mv, mq;
  if ((st = make_map(&mk, k_pages, v.n_pages, v.page_size, s.Hk, unit, s.D)) != CSWATTN_OK) return st;
  if ((st = make_map(&mv, v_pages, v.n_pages, v.page_size, s.Hk, unit, s.D)) != CSWATTN_OK) return st;
  if (w.tiles && (st = make_map_group(&mq, q_out, v.n_tokens, s.H, s.D, s.g, tp.tpt)) != CSWATTN_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const auto launch = s.D == 64 ? launch_paged<64> : launch_paged<128>;
  if ((st = launch(rp, tp, jp, w.tiles, mk, mv, mq, cs, true)) != CSWATTN_OK) return st;
  {
    ScopedTiming tm(CSWATTN_K_DECODE, cs);
    launch(rp, tp, jp, w.tiles, mk, mv, mq, cs, false);
  }
  return launched("paged attention launch");
}

size_t attn_paged_weigh_workspace_bytes(const cswattn_layer* layer, const cswattn_paged* paged) {
  Shape s;
  paged::View v;
  if (check_paged(layer, paged, true, &s, &v) != CSWATTN_OK) return 0;
  return carve_weigh(s, v, nullptr).bytes;
}

cswattn_status attn_paged_weigh(const cswattn_layer* layer, const cswattn_paged* paged, const void* q_out,
                                const void* k_pages, const float* lse, float* weight, void* workspace,
                                size_t workspace_bytes, void* stream) {
  const NvtxRange nvtx_range("attn_paged_weigh");
  Shape s;
  paged::View v;
  cswattn_status st = check_paged(layer, paged, true, &s, &v);
  if (st != CSWATTN_OK) return st;
  if (paged->n_tokens == 0) return CSWATTN_OK;
  CHECK_PTR(q_out, 16);
  CHECK_PTR(k_pages, 16);
  CHECK_PTR(lse, 4);
  CHECK_PTR(weight, 4);
  const WeighWorkspace w = carve_weigh(s, v, workspace);
  if (w.bytes > 0) CHECK_PTR(workspace, 256);
  if (workspace_bytes < w.bytes)
    return fail(CSWATTN_ERR_INVALID_ARG, "weights workspace too small: %zu < %zu bytes", workspace_bytes, w.bytes);
  paged::WeighRowsParams rp;
  rp.v = v;
  rp.scale_log2 = s.scale * 1.4426950408889634f;
  rp.unit = page_unit(v.page_size, w.tiles ? 128 : paged::kBlk);
  rp.q = static_cast<const __nv_bfloat16*>(q_out);
  rp.lse = lse;
  rp.weight = weight;
  rp.wait_ns = g_wait_ns.load();
  paged::WeighTileParams tp;
  tp.v = v;
  tp.scale_log2 = rp.scale_log2;
  tp.unit = rp.unit;
  tp.tpt = 128 / s.g;
  tp.plan = w.plan;
  tp.seqs = w.seqs;
  tp.lse = lse;
  tp.weight = weight;
  tp.part = w.part;
  tp.wait_ns = rp.wait_ns;
  CUtensorMap mk, mq;
  if ((st = make_map(&mk, k_pages, v.n_pages, v.page_size, s.Hk, rp.unit, s.D)) != CSWATTN_OK) return st;
  if (w.tiles && (st = make_map_group(&mq, q_out, v.n_tokens, s.H, s.D, s.g, tp.tpt)) != CSWATTN_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const auto launch = s.D == 64 ? launch_weigh<64> : launch_weigh<128>;
  if ((st = launch(rp, tp, w.tiles, w.max_rows, mk, mq, cs, true)) != CSWATTN_OK) return st;
  {
    ScopedTiming tm(CSWATTN_K_DECODE, cs);
    launch(rp, tp, w.tiles, w.max_rows, mk, mq, cs, false);
  }
  return launched("paged weights launch");
}

cswattn_status attn_paged_select(const cswattn_layer* layer, const cswattn_paged* paged, const float* weight,
                                 const int* position, const int* next_pos, int n_keep, int n_recent, int* n_moves,
                                 int* src, int* dst, int* new_len, void* stream) {
  const NvtxRange nvtx_range("attn_paged_select");
  Shape s;
  paged::SelectParams sp;
  cswattn_status st = check_paged(layer, paged, false, &s, &sp.v);
  if (st != CSWATTN_OK) return st;
  if (n_keep < 1 || n_keep > s.T)
    return fail(CSWATTN_ERR_INVALID_ARG, "n_keep must be in [1, T = %d] (got %d)", s.T, n_keep);
  if (n_recent < 0 || n_recent > n_keep)
    return fail(CSWATTN_ERR_INVALID_ARG, "n_recent must be in [0, n_keep = %d] (got %d)", n_keep, n_recent);
  CHECK_PTR(weight, 4);
  CHECK_PTR(position, 4);
  CHECK_PTR(next_pos, 4);
  CHECK_PTR(n_moves, 4);
  CHECK_PTR(src, 4);
  CHECK_PTR(dst, 4);
  CHECK_PTR(new_len, 4);
  if (new_len == paged->cache_len) return fail(CSWATTN_ERR_INVALID_ARG, "new_len must not alias cache_len");
  sp.weight = weight;
  sp.position = position;
  sp.next_pos = next_pos;
  sp.n_keep = n_keep;
  sp.n_recent = n_recent;
  // CTAs per head: enough rows for each, and no more CTAs than the SMs hold at once.
  int ranks = 1;
  while (ranks < paged::kSelectMaxCluster && s.T > ranks * paged::kSelectRows &&
         2ll * ranks * s.B * s.Hk <= paged::kSMs)
    ranks *= 2;
  sp.smem_keys = std::min((s.T + ranks - 1) / ranks, paged::kSelectMaxKeys);
  sp.n_moves = n_moves;
  sp.src = src;
  sp.dst = dst;
  sp.new_len = new_len;
  const auto kernel = ranks > 1 ? paged::select_kernel<true> : paged::select_kernel<false>;
  if ((st = set_smem(kernel, paged::kSelectMaxKeys * 4)) != CSWATTN_OK) return st;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  {
    ScopedTiming tm(CSWATTN_K_DECODE, cs);
    launch_pdl_cluster(kernel, dim3(ranks, s.Hk, s.B), dim3(paged::kSelectThreads),
                       static_cast<size_t>(sp.smem_keys) * 4, static_cast<unsigned>(ranks), cs, sp);
  }
  return launched("paged select launch");
}

cswattn_status attn_paged_move(const cswattn_layer* layer, const cswattn_paged* paged, const int* n_moves,
                               const int* src, const int* dst, int n_keep, void* k_pages, void* v_pages,
                               float* weight, int* position, void* stream) {
  const NvtxRange nvtx_range("attn_paged_move");
  Shape s;
  paged::MoveParams mp;
  cswattn_status st = check_paged(layer, paged, false, &s, &mp.v);
  if (st != CSWATTN_OK) return st;
  if (n_keep < 1 || n_keep > s.T)
    return fail(CSWATTN_ERR_INVALID_ARG, "n_keep must be in [1, T = %d] (got %d)", s.T, n_keep);
  CHECK_PTR(n_moves, 4);
  CHECK_PTR(src, 4);
  CHECK_PTR(dst, 4);
  CHECK_PTR(k_pages, 16);
  CHECK_PTR(v_pages, 16);
  CHECK_PTR(weight, 4);
  CHECK_PTR(position, 4);
  if (k_pages == v_pages) return fail(CSWATTN_ERR_INVALID_ARG, "k_pages and v_pages must differ");
  mp.n_moves = n_moves;
  mp.src = src;
  mp.dst = dst;
  mp.stride = n_keep;
  mp.k_pages = static_cast<__nv_bfloat16*>(k_pages);
  mp.v_pages = static_cast<__nv_bfloat16*>(v_pages);
  mp.weight = weight;
  mp.position = position;
  // At most min(n_keep, T - n_keep) rows move per head.
  const int most = std::min(n_keep, s.T - n_keep);
  if (most == 0) return CSWATTN_OK;
  const int per = paged::kMoveThreads;
  const dim3 grid(std::min(paged::kMoveMaxCtas, (most + per - 1) / per), s.Hk, s.B);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  {
    ScopedTiming tm(CSWATTN_K_DECODE, cs);
    launch_pdl(s.D == 64 ? paged::move_kernel<64> : paged::move_kernel<128>, grid, dim3(paged::kMoveThreads), 0, cs,
               mp);
  }
  return launched("paged move launch");
}

}  // extern "C"
