// dense_api.cuh -- host side of the paged append and the dense attention
// (qsa_append_kv, qsa_paged_attn_fwd, qsa_prompt_attn_fwd, qsa_prompt_attn_bwd):
// argument checks, work tables, launches.  Included once, by qsa_api.cu.
#pragma once
#include "append.cuh"
#include "dense.cuh"
#include "dense_simt.cuh"
#include "dense_tc.cuh"
#include "dense_decode.cuh"
#include "dense_bwd_tc.cuh"

namespace qsa {
namespace {

// ------------------------------------------------------------------ checks
qsa_status_t check_pages(const qsa_config_t* c, const qsa_pages_t* p) {
  if (!p || !p->k || !p->v || !p->table || !aligned16(p->k) || !aligned16(p->v) || ((uintptr_t)p->table & 3u))
    return QSA_ERR_INVALID_ARG;
  if (p->n_pages <= 0 || p->page_tokens <= 0 || p->n_rows <= 0 || p->max_pages <= 0) return QSA_ERR_INVALID_ARG;
  if (p->page_tokens % 16 != 0) return QSA_ERR_UNSUPPORTED;
  // cache rows are TMA coordinates (int32, with room for a box behind the last)
  if ((int64_t)p->n_pages * c->n_kv_groups > (INT32_MAX - 512) / p->page_tokens) return QSA_ERR_UNSUPPORTED;
  return QSA_OK;
}

// Segments within the table and the token arrays, and no token row in two of them.
qsa_status_t check_dense_segments(const qsa_segment_t* segs, int32_t n_segs, int32_t n_tokens,
                                  const qsa_pages_t* pages, bool prompt) {
  if (n_segs < 0 || n_tokens < 0 || (n_segs > 0 && !segs)) return QSA_ERR_INVALID_ARG;
  bool sorted = true;
  int64_t end = 0;
  for (int i = 0; i < n_segs; ++i) {
    const qsa_segment_t& s = segs[i];
    if (s.q_len < 0 || s.q_offset < 0 || s.pos0 < 0) return QSA_ERR_INVALID_ARG;
    if ((int64_t)s.q_offset + s.q_len > n_tokens) return QSA_ERR_INVALID_ARG;
    if ((int64_t)s.pos0 + s.q_len > INT32_MAX) return QSA_ERR_INVALID_ARG;
    if (prompt && s.pos0 != 0) return QSA_ERR_INVALID_ARG;
    if (pages && (s.slot < 0 || s.slot >= pages->n_rows ||
                  (int64_t)s.pos0 + s.q_len > (int64_t)pages->max_pages * pages->page_tokens))
      return QSA_ERR_INVALID_ARG;
    if (s.q_len == 0) continue;
    if (s.q_offset < end) sorted = false;
    end = (int64_t)s.q_offset + s.q_len;
  }
  if (sorted) return QSA_OK;
  std::vector<std::pair<int32_t, int32_t>> r;
  for (int i = 0; i < n_segs; ++i)
    if (segs[i].q_len > 0) r.emplace_back(segs[i].q_offset, segs[i].q_len);
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if ((int64_t)r[i - 1].first + r[i - 1].second > r[i].first) return QSA_ERR_INVALID_ARG;
  return QSA_OK;
}

// An array of a call (p null: not given).
struct Span {
  const void* p;
  int64_t bytes;
};
// No output shares memory with an input or another output: the kernels of a call
// read their inputs while others of it write results, and some read them twice.
bool spans_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  auto meet = [](const Span& a, const Span& b) {
    return a.p && b.p && (const char*)a.p < (const char*)b.p + b.bytes && (const char*)b.p < (const char*)a.p + a.bytes;
  };
  for (const Span& o : outs) {
    for (const Span& i : ins)
      if (meet(o, i)) return false;
    for (const Span& other : outs)
      if (&other != &o && meet(o, other)) return false;
  }
  return true;
}

// ------------------------------------------------------------------ plan
// Shape of one kind of launch.  For levelling: a unit's fixed cost (loading Q,
// the epilogue) in chunks, and the fewest chunks a CTA takes of the tail, below
// which a piece's partial result costs more than the chunks it saves.
struct DenseKind {
  int rows, kc, grid;
  bool by_keys;
  int cost = 2, min_tail = 4;
  int part_rows = 0;                     // rows of a partial result, where they are not the unit's rows
  bool level = true;                     // false: whole units in turn, for launches that hardly ever have work
};

// Fills rounds, cut and the list of cut units of a table whose segments are set.
void cut_table(DenseTable& t, DenseSplits& sp, const DenseKind& kind) {
  const int64_t kUnitCost = kind.cost, kMinTail = kind.min_tail;
  const int grid = t.grid;
  const int n_units = t.item0[t.n] * t.G;
  sp.n = 0;
  if (!kind.level) {
    t.rounds = n_units / grid;
    for (int c = 0; c <= grid; ++c) t.cut[c] = {std::min(t.rounds * grid + c, n_units), 0};
    return;
  }
  std::vector<int32_t> chunks((size_t)n_units);
  int64_t total = 0;
  for (int u = 0; u < n_units; ++u) {
    chunks[u] = dense_unit(t, u).nchunks;
    total += chunks[u] + kUnitCost;
  }
  // the most whole rounds after which no CTA has more than its share of everything
  std::vector<int64_t> load((size_t)grid, 0), best = load;
  t.rounds = 0;
  for (int r = 0; (r + 1) * grid <= n_units; ++r) {
    int64_t mx = 0;
    for (int c = 0; c < grid; ++c) {
      load[c] += chunks[r * grid + ((r & 1) ? grid - 1 - c : c)] + kUnitCost;
      mx = std::max(mx, load[c]);
    }
    if (mx * grid <= total + (int64_t)grid * kUnitCost) {
      t.rounds = r + 1;
      best = load;
    }
  }
  const int tail0 = t.rounds * grid;
  int64_t tail = 0, whole = 0;
  for (int u = tail0; u < n_units; ++u) tail += chunks[u] + kUnitCost;
  for (int c = 0; c < grid; ++c) whole += best[c];
  // cuts for CTAs filled up to `share`, never leaving less than kMinTail chunks on
  // either side of a cut; true if that holds everything
  auto lay = [&](int64_t share) -> bool {
    int u = tail0;
    int64_t at = 0;                     // chunks of unit u already taken
    for (int c = 0; c < grid; ++c) {
      t.cut[c] = {u, (int32_t)at};
      int64_t want = share - best[c];
      while (u < n_units) {
        const int64_t left = chunks[u] - at;
        if (left + kUnitCost <= want) {
          want -= left + kUnitCost;
          ++u;
          at = 0;
          continue;
        }
        const int64_t take = std::min(want - kUnitCost, left - kMinTail);
        if (take >= kMinTail) at += take;
        break;
      }
    }
    return u >= n_units;
  };
  // the smallest share that holds everything: a unit cut in n pieces costs n times kUnitCost
  int64_t lo = cdiv(whole + tail, grid), hi = lo + (kMinTail + 2 * kUnitCost);
  while (!lay(hi)) {
    lo = hi;
    hi += hi - cdiv(whole + tail, grid);
  }
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    if (lay(mid)) hi = mid; else lo = mid;
  }
  lay(hi);
  t.cut[grid] = {n_units, 0};
  // a unit is cut iff some CTA's stretch starts inside it
  for (int c = 1; c < grid; ++c) {
    if (t.cut[c].chunk == 0) continue;
    const int unit = t.cut[c].unit;
    if (sp.n > 0 && sp.unit[sp.n - 1] == unit) {
      sp.last[sp.n - 1] = (int16_t)c;
      continue;
    }
    int first = c - 1;                  // the CTA that holds the unit's first chunk
    while (first > 0 && (t.cut[first].unit == unit && t.cut[first].chunk > 0)) --first;
    sp.unit[sp.n] = unit;
    sp.first[sp.n] = (int16_t)first;
    sp.last[sp.n] = (int16_t)c;
    ++sp.n;
  }
}

// Calls launch(table, splits) for batches of at most kMaxSegs of the non-empty
// segments, longest first.
template <typename Launch>
qsa_status_t for_each_dense(const Geo& g, std::vector<qsa_segment_t> segs, const DenseKind& kind, Launch launch) {
  segs.erase(std::remove_if(segs.begin(), segs.end(), [](const qsa_segment_t& s) { return s.q_len <= 0; }), segs.end());
  std::stable_sort(segs.begin(), segs.end(), [](const qsa_segment_t& a, const qsa_segment_t& b) {
    return (int64_t)a.pos0 + a.q_len > (int64_t)b.pos0 + b.q_len;
  });
  size_t i = 0;
  while (i < segs.size()) {
    DenseTable t;
    DenseSplits sp;
    memset(&t, 0, sizeof t);
    memset(&sp, 0, sizeof sp);
    t.G = g.G;
    t.hpg = g.hpg;
    t.rows = kind.rows;
    t.kc = kind.kc;
    t.grid = kind.grid;
    t.by_keys = kind.by_keys;
    int64_t tiles = 0, most = 0;
    for (; i < segs.size() && t.n < kMaxSegs; ++i) {
      const qsa_segment_t& s = segs[i];
      // a unit's rows, keys and positions are int32, with room for the last tile and chunk
      if ((int64_t)s.q_len * g.hpg > INT32_MAX - 512 || (int64_t)s.pos0 + s.q_len > INT32_MAX - 512)
        return QSA_ERR_UNSUPPORTED;
      const int64_t rows = (int64_t)s.q_len * (kind.by_keys ? 1 : g.hpg), it = cdiv(rows, kind.rows);
      if (t.n > 0 && (tiles + it) * g.G > INT32_MAX / 4) break;
      if ((tiles + it) * g.G > INT32_MAX / 4) return QSA_ERR_UNSUPPORTED;
      t.q_offset[t.n] = s.q_offset;
      t.q_len[t.n] = s.q_len;
      t.pos0[t.n] = s.pos0;
      t.slot[t.n] = s.slot;
      tiles += it;
      t.item0[++t.n] = (int32_t)tiles;
      most = std::max(most, std::min<int64_t>(rows, kind.rows));
    }
    t.prows = kind.part_rows > 0 ? kind.part_rows : (int32_t)most;
    cut_table(t, sp, kind);
    const qsa_status_t r = launch(t, sp);
    if (r != QSA_OK) return r;
  }
  return QSA_OK;
}

// One launch's table with its cut units.
struct DenseLaunch {
  DenseTable t;
  DenseSplits sp;
  size_t part;                           // offset of its partial results
};

// Bytes of a table's partial results.
size_t partial_bytes(const DenseTable& t, const DenseSplits& sp) {
  return sp.n > 0 ? (size_t)2 * t.grid * t.prows * dense::kPartFloats * 4 : 0;
}

// The launches of one kind for the segments; `part` grows by their partial results.
qsa_status_t plan_launches(const Geo& g, const std::vector<qsa_segment_t>& segs, const DenseKind& kind,
                           std::vector<DenseLaunch>& out, size_t& part) {
  return for_each_dense(g, segs, kind, [&](const DenseTable& t, const DenseSplits& sp) {
    out.push_back({t, sp, part});
    part += align_up(partial_bytes(t, sp), 256);
    return QSA_OK;
  });
}

// A forward call's segments by the kernel that takes them, in launch order.
enum class DenseForm { kWide, kNarrow, kDecode };
struct DenseGroup {
  DenseForm form;
  DenseKind kind;
  std::vector<qsa_segment_t> segs;
  std::vector<DenseLaunch> launches;
};

// Single tokens over a cache go to the decode kernels.  bf16: other segments of
// at most 128 rows go to single CTAs unless larger ones are there, whose pairs then
// take them too (one launch and its tail, 15 us, for a few half-empty tiles).
std::vector<DenseGroup> dense_groups(const Geo& g, bool tc, bool paged, const qsa_segment_t* segs, int n) {
  DenseGroup wide{DenseForm::kWide, {}, {}, {}}, narrow{DenseForm::kNarrow, {}, {}, {}},
      decode{DenseForm::kDecode, {}, {}, {}};
  if (tc) {
    using N = dense_tc::Shape<1>;
    using W = dense_tc::Shape<2>;
    narrow.kind = {N::kRows, N::kKeys, N::kGrid, false};
    wide.kind = {W::kRows, W::kKeys, W::kGrid, false, 4, 4};      // a unit's 5.5 us in chunks of 1.4 us
  } else {
    narrow.kind = {dense_simt::kRowsNarrow, dense_simt::kKeys, kNumSms, false};
    wide.kind = {dense_simt::kRowsWide, dense_simt::kKeys, kNumSms, false};
  }
  decode.kind = {dense_decode::kRows, dense_decode::kKeys, kNumSms, false, 1, 1};
  for (int i = 0; i < n; ++i) {
    if (segs[i].q_len <= 0) continue;
    const bool few = (int64_t)segs[i].q_len * g.hpg <= narrow.kind.rows;
    (paged && segs[i].q_len == 1 ? decode : few ? narrow : wide).segs.push_back(segs[i]);
  }
  if (tc && !wide.segs.empty()) {
    wide.segs.insert(wide.segs.end(), narrow.segs.begin(), narrow.segs.end());
    narrow.segs.clear();
  }
  std::vector<DenseGroup> out;
  for (DenseGroup* d : {&wide, &narrow, &decode})
    if (!d->segs.empty()) out.push_back(std::move(*d));
  return out;
}

// The groups with their launches, and the bytes of workspace they need.
qsa_status_t plan_dense_fwd(const Geo& g, bool tc, bool paged, const qsa_segment_t* segs, int n,
                            std::vector<DenseGroup>& out, size_t& ws) {
  out = dense_groups(g, tc, paged, segs, n);
  ws = 0;
  for (DenseGroup& d : out) {
    const qsa_status_t r = plan_launches(g, d.segs, d.kind, d.launches, ws);
    if (r != QSA_OK) return r;
  }
  return QSA_OK;
}

size_t dense_fwd_ws(const Geo& g, bool tc, bool paged, const qsa_segment_t* segs, int n) {
  std::vector<DenseGroup> groups;
  size_t ws = 0;
  return plan_dense_fwd(g, tc, paged, segs, n, groups, ws) == QSA_OK ? ws : SIZE_MAX;
}

// ------------------------------------------------------------------ forward
template <int ROWS, bool PAGED>
cudaError_t launch_dense_simt(const Geo& g, const DenseTable& t, const KvSource& kv, const void* q, void* o,
                              float* lse, float* part, cudaStream_t st) {
  const int smem = dense_simt::fwd_smem(ROWS);
  cudaError_t e = cudaFuncSetAttribute(dense_fwd_simt_kernel<ROWS, PAGED>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_chained(dense_fwd_simt_kernel<ROWS, PAGED>, dim3(t.grid), dim3(dense_simt::kThreads), smem, st, t,
                        kv, (const float*)q, (float*)o, lse, part, g.H, g.scale);
}

// Map over rows of 256 dims (paged: every cache row; packed: a token's groups
// side by side), in boxes of `box` rows x 64 dims, 128-byte swizzled.
bool make_dense_map(CUtensorMap* m, const void* base, int64_t rows, int groups, int box) {
  if (rows > INT32_MAX - 512) return false;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)kHeadDim * groups, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)kHeadDim * groups * 2};
  cuuint32_t boxes[2] = {64, (cuuint32_t)box};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, boxes, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int CG, bool PAGED>
cudaError_t launch_dense_tc(const DenseTable& t, const CUtensorMap (&m)[4], const DenseTcArgs& a, cudaStream_t st) {
  auto kernel = dense_fwd_tc_kernel<CG, PAGED>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dense_tc::kSmemBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(t.grid * CG);
  cfg.blockDim = dim3(dense_tc::kThreads);
  cfg.dynamicSmemBytes = dense_tc::kSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kernel, m[0], m[1], m[2], m[3], t, a);
}

cudaError_t launch_dense_decode(const DenseTable& t, const DenseTcArgs& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(dense_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             dense_decode::kSmemBytes);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_chained(dense_decode_kernel, dim3(t.grid), dim3(dense_decode::kThreads), dense_decode::kSmemBytes, st,
                        t, a);
}

template <int HP>
cudaError_t launch_decode_f32(const DenseTable& t, const DenseDecodeF32Args& a, cudaStream_t st) {
  const cudaError_t e = cudaFuncSetAttribute(dense_decode_f32_kernel<HP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             dense_decode::kSmemBytes32);
  if (e != cudaSuccess) return e;
  count_launch();
  return launch_chained(dense_decode_f32_kernel<HP>, dim3(t.grid), dim3(dense_decode::kThreads),
                        dense_decode::kSmemBytes32, st, t, a);
}
cudaError_t launch_dense_decode(const DenseTable& t, const DenseDecodeF32Args& a, cudaStream_t st) {
  if (t.hpg <= 4) return launch_decode_f32<4>(t, a, st);
  if (t.hpg <= 8) return launch_decode_f32<8>(t, a, st);
  return t.hpg <= 12 ? launch_decode_f32<12>(t, a, st) : launch_decode_f32<16>(t, a, st);
}

template <typename T>
cudaError_t launch_dense_combine(const Geo& g, const DenseTable& t, const DenseSplits& sp, const float* part, void* o,
                                 float* lse, cudaStream_t st) {
  count_launch();
  int most = 0;
  for (int i = 0; i < sp.n; ++i) most = std::max(most, sp.last[i] - sp.first[i] + 1);
  if (most > kFewPieces)                 // a warp per row adds four pieces in the time of a barrier or two
    return launch_chained(dense_combine_many_kernel<T>, dim3(sp.n, (unsigned)t.prows), dim3(256), 0, st, t, sp, part,
                          (T*)o, lse, g.H);
  return launch_chained(dense_combine_kernel<T>, dim3(sp.n, (unsigned)cdiv(t.prows, 4)), dim3(128), 0, st, t, sp,
                        part, (T*)o, lse, g.H);
}

// kv_rows, kv_groups: the shape of the tensor map over K and V (make_dense_map).
template <bool PAGED>
qsa_status_t run_dense_fwd(const Geo& g, bool tc, const qsa_segment_t* segs, int n, const KvSource& kv,
                           int64_t kv_rows, int kv_groups, int32_t n_tokens, const void* q, void* o, float* lse,
                           void* ws, size_t ws_bytes, cudaStream_t st) {
  std::vector<DenseGroup> groups;
  size_t need = 0;
  const qsa_status_t r = plan_dense_fwd(g, tc, PAGED, segs, n, groups, need);
  if (r != QSA_OK) return r;
  if (need > 0 && (!ws || ws_bytes < need)) return QSA_ERR_WORKSPACE;
  if (need > 0 && !aligned16(ws)) return QSA_ERR_INVALID_ARG;
  const int64_t row = kHeadDim * (tc ? 2 : 4), q_bytes = (int64_t)n_tokens * g.H * row;
  const int64_t kv_bytes = kv_rows * kv_groups * row;
  if (!spans_apart({{o, q_bytes}, {lse, (int64_t)n_tokens * g.H * 4}},
                   {{q, q_bytes}, {kv.k, kv_bytes}, {kv.v, kv_bytes}}))
    return QSA_ERR_INVALID_ARG;
  CUtensorMap m[4];                      // K, V, Q by whole tokens, Q by parts of one
  DenseTcArgs a;
  if (tc) {
    if ((int64_t)n_tokens * g.H > INT32_MAX - 512) return QSA_ERR_UNSUPPORTED;      // TMA row coordinates
    a = {kv, (const __nv_bfloat16*)q, (__nv_bfloat16*)o, lse, nullptr, g.H, PAGED ? dense_box(kv.page_tokens) : 64,
         g.scale, false};
    if ((groups.size() > 1 || groups[0].form != DenseForm::kDecode) &&      // decode takes no maps
        (!make_dense_map(&m[0], kv.k, kv_rows, kv_groups, a.box) ||
         !make_dense_map(&m[1], kv.v, kv_rows, kv_groups, a.box) ||
         !make_dense_map(&m[2], q, (int64_t)n_tokens * g.H, 1, g.hpg) ||
         !make_dense_map(&m[3], q, (int64_t)n_tokens * g.H, 1, g.hpg & -g.hpg)))
      return QSA_ERR_CUDA;
  }
  // every launch's kernel, each after the first beside the one before; then the joins
  auto part_of = [&](const DenseLaunch& x) { return (float*)((char*)ws + x.part); };
  a.late = false;
  for (const DenseGroup& d : groups)
    for (const DenseLaunch& x : d.launches) {
      const bool is_wide = d.form == DenseForm::kWide;
      a.part = part_of(x);
      cudaError_t e;
      if (d.form == DenseForm::kDecode)
        e = tc ? launch_dense_decode(x.t, a, st)
               : launch_dense_decode(x.t,
                                     DenseDecodeF32Args{kv, (const float*)q, (float*)o, lse, part_of(x), g.H, g.scale,
                                                        false},
                                     st);
      else if (tc)
        e = is_wide ? launch_dense_tc<2, PAGED>(x.t, m, a, st) : launch_dense_tc<1, PAGED>(x.t, m, a, st);
      else
        e = is_wide ? launch_dense_simt<dense_simt::kRowsWide, PAGED>(g, x.t, kv, q, o, lse, a.part, st)
                    : launch_dense_simt<dense_simt::kRowsNarrow, PAGED>(g, x.t, kv, q, o, lse, a.part, st);
      if (e != cudaSuccess) return QSA_ERR_CUDA;
      a.late = true;
    }
  for (const DenseGroup& d : groups)
    for (const DenseLaunch& x : d.launches) {
      if (x.sp.n == 0) continue;
      const cudaError_t e = tc ? launch_dense_combine<__nv_bfloat16>(g, x.t, x.sp, part_of(x), o, lse, st)
                               : launch_dense_combine<float>(g, x.t, x.sp, part_of(x), o, lse, st);
      if (e != cudaSuccess) return QSA_ERR_CUDA;
    }
  return QSA_OK;
}

// ------------------------------------------------------------------ backward
// Workspace of the gradient: delta by token; for bf16 also the statistics by
// head (segments padded to whole tiles) and the segments' flags; the partial
// results of the cut units, the keys' launches' twice (dv, dk).
struct DenseBwdPlan {
  std::vector<qsa_segment_t> segs;       // non-empty; slot: the segment's first statistics tile
  std::vector<DenseLaunch> rows, keys;   // launches by rows (dq) and by keys (dk, dv)
  int64_t stat_rows = 0;
  size_t off_lse2 = 0, off_delta_h = 0, off_flags = 0, off_part = 0, off_part2 = 0, bytes = 0;
};

DenseKind dense_bwd_kind(bool tc, bool by_keys) {
  if (tc) return {dense_bwd::kRows, dense_bwd::kKeys, dense_bwd::kGrid, by_keys, 3, 4};      // 6 us, 2.1 us
  using namespace dense_simt;
  return by_keys ? DenseKind{kBKeys, kBRows, kNumSms, true, 1, 1, 2 * kBKeys}
                 : DenseKind{kBRows, kBKeys, kNumSms, false, 1, 1};
}

qsa_status_t plan_dense_bwd(const Geo& g, bool tc, const qsa_segment_t* segs, int n, int32_t n_tokens,
                            DenseBwdPlan& p) {
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (segs[i].q_len <= 0) continue;
    p.segs.push_back(segs[i]);
    p.segs.back().slot = (int32_t)tiles;
    tiles += cdiv(segs[i].q_len, dense_bwd::kStatTile);
  }
  size_t at = align_up((size_t)n_tokens * g.H * 4, 256);
  if (tc) {
    p.stat_rows = tiles * dense_bwd::kStatTile;
    const size_t stats = align_up((size_t)p.stat_rows * g.H * 4, 256);
    p.off_lse2 = at;
    p.off_delta_h = at + stats;
    p.off_flags = at + 2 * stats;
    at = p.off_flags + align_up((size_t)tiles * (dense_bwd::kStatTile / 4), 256);
  }
  p.off_part = at;
  size_t part = 0;
  qsa_status_t r = plan_launches(g, p.segs, dense_bwd_kind(tc, false), p.rows, part);
  const size_t part_rows = part;
  if (r == QSA_OK) r = plan_launches(g, p.segs, dense_bwd_kind(tc, true), p.keys, part);
  p.off_part2 = at + part - part_rows;   // the keys' offsets start behind the rows'
  p.bytes = at + part + (tc ? part - part_rows : 0);
  return r;
}

size_t dense_bwd_ws(const Geo& g, bool tc, const qsa_segment_t* segs, int n, int32_t n_tokens) {
  DenseBwdPlan p;
  return plan_dense_bwd(g, tc, segs, n, n_tokens, p) == QSA_OK ? p.bytes : SIZE_MAX;
}

// Joins the cut units of every launch's gradients: dq's from `parts`, dk's and
// dv's from `dk_parts` and `dv_parts`, dv's partial rows `dv_row` behind dk's.
template <typename T>
cudaError_t launch_bwd_joins(const Geo& g, const DenseBwdPlan& p, const DenseBwdArgs& a, const char* parts,
                             const char* dk_parts, const char* dv_parts, int dv_row, const uint8_t* flags,
                             cudaStream_t st) {
  for (size_t i = 0; i < std::max(p.rows.size(), p.keys.size()); ++i) {
    static const DenseLaunch kNone{};
    const DenseLaunch& r = i < p.rows.size() ? p.rows[i] : kNone;
    const DenseLaunch& k = i < p.keys.size() ? p.keys[i] : kNone;
    if (r.sp.n == 0 && k.sp.n == 0) continue;
    auto rows_of = [](const DenseLaunch& x) { return x.sp.n ? std::min(x.t.prows, x.t.rows) : 0; };
    const DenseBwdJoins<T> joins{{{(const float*)(parts + r.part), (T*)a.dq, g.scale, 0, 0},
                                  {(const float*)(dk_parts + k.part), (T*)a.dk, g.scale, 0, 1},
                                  {(const float*)(dv_parts + k.part), (T*)a.dv, 1.f, dv_row, 1}},
                                 flags,
                                 g.H};
    count_launch();
    const cudaError_t e = launch_chained(
        dense_bwd_combine_kernel<T>,
        dim3(std::max(r.sp.n, k.sp.n), (unsigned)cdiv(std::max(rows_of(r), rows_of(k)), 4), 3), dim3(128), 0, st, r.t,
        r.sp, k.t, k.sp, joins);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

qsa_status_t run_dense_bwd_f32(const Geo& g, const DenseBwdPlan& p, const DenseBwdArgs& a, const void* o, char* ws,
                               cudaStream_t st) {
  const qsa_status_t r = for_each_table(
      p.segs.data(), (int)p.segs.size(), [&](const qsa_segment_t& s) { return (int64_t)s.q_len; },
      [&](const SegTable& t) -> cudaError_t {
        count_launch();
        return launch_chained(dense_delta_kernel<float>, dim3((unsigned)cdiv((int64_t)t.item0[t.n] * g.H, 8)),
                              dim3(256), 0, st, t, (const float*)o, (const float*)a.dout, (float*)ws, g.H);
      });
  if (r != QSA_OK) return r;
  cudaError_t e = cudaFuncSetAttribute(dense_dq_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       dense_simt::kBwdSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(dense_dkv_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dense_simt::kBwdSmem);
  char* const parts = ws + p.off_part;
  for (const bool keys : {false, true})
    for (const DenseLaunch& x : keys ? p.keys : p.rows) {
      if (e != cudaSuccess) break;
      count_launch();
      e = launch_chained(keys ? dense_dkv_simt_kernel : dense_dq_simt_kernel, dim3(x.t.grid),
                         dim3(dense_simt::kThreads), dense_simt::kBwdSmem, st, x.t, a, (float*)(parts + x.part));
    }
  if (e == cudaSuccess) e = launch_bwd_joins<float>(g, p, a, parts, parts, parts, dense_simt::kBKeys, nullptr, st);
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

// One gradient on the tensor cores; partial results from `parts` on.
template <dense_bwd::Grad M>
qsa_status_t run_dense_grad_tc(const DenseBwdPlan& p, const DenseBwdMaps& m, DenseBwdTcArgs a, char* parts,
                               cudaStream_t st) {
  auto kernel = dense_bwd_tc_kernel<M>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, dense_bwd::kSmemBytes);
  for (const DenseLaunch& x : M == dense_bwd::kDq ? p.rows : p.keys) {
    if (e != cudaSuccess) break;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(x.t.grid * 2);
    cfg.blockDim = dim3(dense_bwd::kThreads);
    cfg.dynamicSmemBytes = dense_bwd::kSmemBytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    a.part = (float*)(parts + x.part);
    count_launch();
    e = cudaLaunchKernelEx(&cfg, kernel, m, x.t, a);
    a.late = true;
  }
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

qsa_status_t run_dense_bwd_bf16(const Geo& g, const DenseBwdPlan& p, DenseBwdArgs a, const void* o, char* ws,
                                int32_t n_tokens, cudaStream_t st) {
  using B = __nv_bfloat16;
  float* delta = (float*)ws;
  float* lse2_h = (float*)(ws + p.off_lse2);
  float* delta_h = (float*)(ws + p.off_delta_h);
  uint8_t* flags = (uint8_t*)(ws + p.off_flags);
  CUtensorMap mq, mo, mk, mv, tq, to, rq, ro;      // boxes of 64 rows; Q and dO by whole tokens and parts of one
  const int64_t rows = (int64_t)n_tokens * g.H;
  if (rows > INT32_MAX - 512) return QSA_ERR_UNSUPPORTED;
  if (!make_dense_map(&mq, a.q, n_tokens, g.H, 64) || !make_dense_map(&mo, a.dout, n_tokens, g.H, 64) ||
      !make_dense_map(&mk, a.k, n_tokens, g.G, 64) || !make_dense_map(&mv, a.v, n_tokens, g.G, 64) ||
      !make_dense_map(&tq, a.q, rows, 1, g.hpg) || !make_dense_map(&to, a.dout, rows, 1, g.hpg) ||
      !make_dense_map(&rq, a.q, rows, 1, g.hpg & -g.hpg) || !make_dense_map(&ro, a.dout, rows, 1, g.hpg & -g.hpg))
    return QSA_ERR_CUDA;
  // launches for the flagged segments, not levelled; rows and keys split alike, by the
  // number of segments (n_tokens * H in 31 bits is far from the limit on units)
  std::vector<DenseLaunch> rows_l, keys_l;
  size_t part = 0;
  DenseKind kr = dense_bwd_kind(false, false), kk = dense_bwd_kind(false, true);
  kr.level = kk.level = false;
  qsa_status_t r = plan_launches(g, p.segs, kr, rows_l, part);
  if (r == QSA_OK) r = plan_launches(g, p.segs, kk, keys_l, part);
  if (r != QSA_OK) return r;
  r = for_each_table(
      p.segs.data(), (int)p.segs.size(),
      [&](const qsa_segment_t& s) { return cdiv(s.q_len, dense_bwd::kStatTile) * dense_bwd::kStatTile; },
      [&](const SegTable& t) -> cudaError_t {
        count_launch();
        return launch_chained(dense_stats_kernel, dim3((unsigned)(t.item0[t.n] / 4)), dim3(256), 0,
                              st, t, (const B*)o, (const B*)a.dout, a.lse, (const B*)a.k, (const B*)a.v, delta, lse2_h,
                              delta_h, flags, p.stat_rows, g.H, g.G);
      });
  if (r != QSA_OK) return r;
  // dq, beside its end dv, then dk (which reads delta as dq leaves it); then the
  // joins of their cut units
  char* const parts = ws + p.off_part;
  char* const parts2 = ws + p.off_part2;
  DenseBwdTcArgs b{lse2_h, delta_h, flags, (B*)a.dq, nullptr, p.stat_rows, g.H, g.scale, false};
  if ((r = run_dense_grad_tc<dense_bwd::kDq>(p, {mk, mv, mk, tq, to, rq, ro}, b, parts, st)) != QSA_OK) return r;
  b.late = true;
  b.out = (B*)a.dv;
  if ((r = run_dense_grad_tc<dense_bwd::kDv>(p, {mq, mq, mo, mk, mv, mk, mv}, b, parts, st)) != QSA_OK) return r;
  b.late = false;
  b.out = (B*)a.dk;
  if ((r = run_dense_grad_tc<dense_bwd::kDk>(p, {mq, mo, mq, mk, mv, mk, mv}, b, parts2, st)) != QSA_OK) return r;
  cudaError_t e = launch_bwd_joins<B>(g, p, a, parts, parts2, parts, 0, flags, st);
  a.flags = flags;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(dense_bwd_flagged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             dense_simt::kBwdSmem);
  for (size_t i = 0; i < rows_l.size() && e == cudaSuccess; ++i) {
    count_launch();
    e = launch_chained(dense_bwd_flagged_kernel, dim3(rows_l[i].t.grid), dim3(dense_simt::kThreads),
                       dense_simt::kBwdSmem, st, rows_l[i].t, keys_l[i].t, a);
  }
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}

// Runs an entry point's body; host memory that runs out is an error code, not
// an exception through the C interface.
template <typename Body>
qsa_status_t guarded(Body body) {
  try {
    return body();
  } catch (...) {
    return QSA_ERR_CUDA;
  }
}

}  // namespace
}  // namespace qsa

using namespace qsa;

QSA_API qsa_status_t qsa_append_kv(const qsa_config_t* cfg, const qsa_pages_t* pages, const qsa_segment_t* segs,
                                   int32_t n_segs, int32_t n_tokens, const void* k, int64_t ld_k, const void* v,
                                   int64_t ld_v, const void* q, int64_t ld_q, void* q_out, void* stream) {
  return guarded([&]() -> qsa_status_t {
    qsa_status_t s = check_cfg(cfg, false);
    if (s != QSA_OK) return s;
    if ((s = check_pages(cfg, pages)) != QSA_OK) return s;
    if ((s = check_dense_segments(segs, n_segs, n_tokens, pages, false)) != QSA_OK) return s;
    if (seg_rows(segs, n_segs) == 0) return QSA_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v) || (!q) != (!q_out) || !aligned16(q) || !aligned16(q_out))
      return QSA_ERR_INVALID_ARG;
    const int64_t per16 = cfg->dtype == QSA_DTYPE_BF16 ? 8 : 4;
    auto bad_ld = [&](int64_t ld, int heads) { return ld < (int64_t)heads * kHeadDim || ld % per16 != 0; };
    if (bad_ld(ld_k, cfg->n_kv_groups) || bad_ld(ld_v, cfg->n_kv_groups) || (q && bad_ld(ld_q, cfg->n_q_heads)))
      return QSA_ERR_INVALID_ARG;
    if (q && q == q_out && ld_q != (int64_t)cfg->n_q_heads * kHeadDim) return QSA_ERR_INVALID_ARG;
    const Geo g = make_geo(cfg, nullptr);
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.k = k;
    a.v = v;
    a.q = q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.ld_q = ld_q;
    a.q_out = q_out;
    a.kp = pages->k;
    a.vp = pages->v;
    a.table = pages->table;
    a.n_pages = pages->n_pages;
    a.page_tokens = pages->page_tokens;
    a.max_pages = pages->max_pages;
    int rd = (int)floor((double)cfg->head_dim * (double)cfg->rope_fraction);
    rd -= rd & 1;
    a.half = rd / 2;
    for (int i = 0; i < a.half; ++i) a.theta[i] = pow(cfg->rope_base, -(2.0 * (double)i) / (double)rd);
    return for_each_table(
        segs, n_segs, [&](const qsa_segment_t& sg) { return (int64_t)sg.q_len; },
        [&](const SegTable& t) -> cudaError_t {
          count_launch();
          // one warp per token once that fills the GPU's warp slots about once
          const int n = t.item0[t.n];
          const bool many = n >= 16 * kNumSms;
          const dim3 grid((unsigned)(many ? cdiv(n, append::kWarps) : n)), block(append::kThreads);
          const cudaStream_t s0 = (cudaStream_t)stream;
          if (cfg->dtype == QSA_DTYPE_BF16)
            return many ? launch_chained(append_kernel<__nv_bfloat16, 1>, grid, block, 0, s0, g, t, a)
                        : launch_chained(append_kernel<__nv_bfloat16, append::kWarps>, grid, block, 0, s0, g, t, a);
          return many ? launch_chained(append_kernel<float, 1>, grid, block, 0, s0, g, t, a)
                      : launch_chained(append_kernel<float, append::kWarps>, grid, block, 0, s0, g, t, a);
        });
  });
}

QSA_API qsa_status_t qsa_paged_attn_fwd(const qsa_config_t* cfg, const qsa_pages_t* pages, const qsa_segment_t* segs,
                                        int32_t n_segs, int32_t n_tokens, const void* q, void* o, float* lse,
                                        void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> qsa_status_t {
    qsa_status_t s = check_cfg(cfg, false);
    if (s != QSA_OK) return s;
    if ((s = check_pages(cfg, pages)) != QSA_OK) return s;
    if ((s = check_dense_segments(segs, n_segs, n_tokens, pages, false)) != QSA_OK) return s;
    if (seg_rows(segs, n_segs) == 0) return QSA_OK;
    if (!q || !o || !aligned16(q) || !aligned16(o) || ((uintptr_t)lse & 3u)) return QSA_ERR_INVALID_ARG;
    const Geo g = make_geo(cfg, nullptr);
    const KvSource kv{pages->k, pages->v, pages->table, pages->n_pages, pages->page_tokens, pages->max_pages};
    return run_dense_fwd<true>(g, cfg->dtype == QSA_DTYPE_BF16, segs, n_segs, kv,
                               (int64_t)pages->n_pages * cfg->n_kv_groups * pages->page_tokens, 1, n_tokens, q, o, lse,
                               workspace, ws_bytes, (cudaStream_t)stream);
  });
}

QSA_API qsa_status_t qsa_prompt_attn_fwd(const qsa_config_t* cfg, const qsa_segment_t* segs, int32_t n_segs,
                                         int32_t n_tokens, const void* q, const void* k, const void* v, void* o,
                                         float* lse, void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> qsa_status_t {
    qsa_status_t s = check_cfg(cfg, false);
    if (s != QSA_OK) return s;
    if ((s = check_dense_segments(segs, n_segs, n_tokens, nullptr, true)) != QSA_OK) return s;
    if (seg_rows(segs, n_segs) == 0) return QSA_OK;
    if (!q || !k || !v || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        ((uintptr_t)lse & 3u))
      return QSA_ERR_INVALID_ARG;
    const Geo g = make_geo(cfg, nullptr);
    const KvSource kv{k, v, nullptr, 0, 0, 0};
    return run_dense_fwd<false>(g, cfg->dtype == QSA_DTYPE_BF16, segs, n_segs, kv, n_tokens, cfg->n_kv_groups, n_tokens,
                                q, o, lse, workspace, ws_bytes, (cudaStream_t)stream);
  });
}

QSA_API qsa_status_t qsa_prompt_attn_bwd(const qsa_config_t* cfg, const qsa_segment_t* segs, int32_t n_segs,
                                         int32_t n_tokens, const void* q, const void* k, const void* v, const void* o,
                                         const float* lse, const void* dout, void* dq, void* dk, void* dv,
                                         void* workspace, size_t ws_bytes, void* stream) {
  return guarded([&]() -> qsa_status_t {
    qsa_status_t s = check_cfg(cfg, false);
    if (s != QSA_OK) return s;
    if ((s = check_dense_segments(segs, n_segs, n_tokens, nullptr, true)) != QSA_OK) return s;
    if (seg_rows(segs, n_segs) == 0) return QSA_OK;
    for (const void* p : {q, k, v, o, dout, (const void*)dq, (const void*)dk, (const void*)dv})
      if (!p || !aligned16(p)) return QSA_ERR_INVALID_ARG;
    if (!lse || ((uintptr_t)lse & 3u)) return QSA_ERR_INVALID_ARG;
    const Geo g = make_geo(cfg, nullptr);
    const bool tc = cfg->dtype == QSA_DTYPE_BF16;
    DenseBwdPlan p;
    if ((s = plan_dense_bwd(g, tc, segs, n_segs, n_tokens, p)) != QSA_OK) return s;
    if (!workspace || ws_bytes < p.bytes) return QSA_ERR_WORKSPACE;
    if (!aligned16(workspace)) return QSA_ERR_INVALID_ARG;
    const int64_t row = kHeadDim * (tc ? 2 : 4), q_bytes = (int64_t)n_tokens * g.H * row;
    const int64_t kv_bytes = (int64_t)n_tokens * g.G * row;
    if (!spans_apart({{dq, q_bytes}, {dk, kv_bytes}, {dv, kv_bytes}},
                     {{q, q_bytes}, {k, kv_bytes}, {v, kv_bytes}, {o, q_bytes}, {dout, q_bytes},
                      {lse, (int64_t)n_tokens * g.H * 4}}))
      return QSA_ERR_INVALID_ARG;
    const DenseBwdArgs a{q, k, v, lse, (const float*)workspace, dout, dq, dk, dv, g.H, g.scale, nullptr};
    return tc ? run_dense_bwd_bf16(g, p, a, o, (char*)workspace, n_tokens, (cudaStream_t)stream)
              : run_dense_bwd_f32(g, p, a, o, (char*)workspace, (cudaStream_t)stream);
  });
}
