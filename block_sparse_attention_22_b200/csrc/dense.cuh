// dense.cuh -- work tables of the dense causal attention kernels (over a paged
// cache and over packed prompts): units, their order, and the split of the
// last units over the grid.
//
// A unit is (tile, KV group): `rows` consecutive query rows of one segment and
// group, row r = token r / hpg, head r % hpg of the group, against the keys
// 0 .. position of the tile's last token, in chunks of `kc` keys.  Units are
// ordered longest first (segments by length, a segment's tiles from its end).
// Whole rounds of units are dealt to the grid back and forth; the units left
// over form one flat sequence of chunks that is cut so that every CTA ends
// with the same number of chunks.  A unit cut between CTAs is computed in
// pieces, each leaving an unnormalised fp32 partial result, which
// dense_combine_kernel joins in a fixed order.  Units with few rows (decode)
// are nothing but such a sequence: keys split over the GPU.
//
// With by_keys the roles are exchanged (gradients of keys and values): a unit
// is `rows` consecutive keys of one segment and group, against the group's
// heads of every token from the unit's first key on, a chunk being `kc` tokens
// of one head (heads innermost).  A segment's first keys have the most.
#pragma once
#include "qsa_internal.cuh"

namespace qsa {
namespace dense {
constexpr int kMaxGrid = 148;              // CTAs (or CTA pairs) a table is cut for
constexpr int kPartFloats = kHeadDim + 4;  // a row's partial: 256 sums, maximum and sum of its softmax, 2 unused
constexpr float kNan = __builtin_nanf("");
}  // namespace dense

// A kernel that needs nothing from the one launched before it, only what that
// one itself waited for, runs beside its last CTAs: it waits for it at its end
// instead of its start (`late`), so that the kernels after it may rely on both.
__device__ __forceinline__ void dense_wait_first(bool late) {
  if (!late) pdl_wait();
  pdl_trigger();
}
__device__ __forceinline__ void dense_wait_last(bool late) {
  if (late) pdl_wait();
}

struct DensePoint {
  int32_t unit, chunk;
};

struct DenseTable {
  int32_t n;
  int32_t q_offset[kMaxSegs];
  int32_t q_len[kMaxSegs];
  int32_t pos0[kMaxSegs];
  int32_t slot[kMaxSegs];
  int32_t item0[kMaxSegs + 1];             // tiles of the segments before
  int32_t G, hpg;
  int32_t rows, kc;                        // query rows per tile, keys per chunk
  int32_t grid;                            // CTAs (or pairs)
  int32_t rounds;                          // whole units per CTA; unit rounds*grid is the first of the tail
  int32_t prows;                           // rows of a partial result
  int32_t by_keys;
  DensePoint cut[dense::kMaxGrid + 1];     // CTA c takes the tail from cut[c] up to cut[c+1]
};

// Units cut into pieces: the CTAs first..last each may hold one.
struct DenseSplits {
  int32_t n;
  int32_t unit[dense::kMaxGrid];
  int16_t first[dense::kMaxGrid], last[dense::kMaxGrid];
};

// Rows and positions of a segment fit 32 bits (checked on the host): 64-bit
// divisions by the group size cost more than a chunk's products.
struct DenseUnit {
  int si;                // segment
  int grp;
  int32_t row0;          // first row of the tile in the segment's rows (by_keys: first key)
  int nrows;             // valid rows (>= 1)
  int32_t kv_len;        // keys 0 .. kv_len-1 are those of the tile's last token (by_keys: the segment's tokens)
  int nchunks;
};

__host__ __device__ __forceinline__ DenseUnit dense_unit(const DenseTable& t, int u) {
  DenseUnit x;
  const int tile = u / t.G;
  x.grp = u - tile * t.G;
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.item0[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  x.si = lo;
  if (t.by_keys) {
    x.row0 = (tile - t.item0[lo]) * t.rows;
    x.kv_len = t.q_len[lo];
    const int32_t left = x.kv_len - x.row0;
    x.nrows = left < t.rows ? left : t.rows;
    x.nchunks = (left + t.kc - 1) / t.kc * t.hpg;
    return x;
  }
  x.row0 = (t.item0[lo + 1] - 1 - tile) * t.rows;     // tiles from the segment's end
  const int32_t left = t.q_len[lo] * t.hpg - x.row0;
  x.nrows = left < t.rows ? left : t.rows;
  x.kv_len = t.pos0[lo] + (x.row0 + x.nrows - 1) / t.hpg + 1;
  x.nchunks = (x.kv_len + t.kc - 1) / t.kc;
  return x;
}

// Row `row` of the unit's segment and group in the token-major arrays, in heads.
__device__ __forceinline__ int64_t dense_q_row(const DenseTable& t, const DenseUnit& x, int32_t row, int H) {
  const int32_t tok = row / t.hpg;
  return (int64_t)(t.q_offset[x.si] + tok) * H + x.grp * t.hpg + (row - tok * t.hpg);
}

// One piece of work of a CTA: chunks c0 .. c1-1 of a unit.  part < 0: the
// whole unit; else the slot of its partial result.
struct DensePiece {
  int unit, c0, c1, part;
};

// Walks a CTA's pieces: its whole units, then its stretch of the tail.
struct DenseWalk {
  int cta, round, unit;
  __host__ __device__ __forceinline__ void init(const DenseTable& t, int c) {
    cta = c;
    round = 0;
    unit = t.cut[c].unit;
  }
  // Fills p and, for the caller, the unit; false at the end.
  __host__ __device__ __forceinline__ bool next(const DenseTable& t, DensePiece& p, DenseUnit& x) {
    if (round < t.rounds) {
      p.unit = round * t.grid + ((round & 1) ? t.grid - 1 - cta : cta);
      ++round;
      x = dense_unit(t, p.unit);
      p.c0 = 0;
      p.c1 = x.nchunks;
      p.part = -1;
      return true;
    }
    const DensePoint a = t.cut[cta], b = t.cut[cta + 1];
    while (unit < b.unit || (unit == b.unit && b.chunk > 0)) {
      x = dense_unit(t, unit);
      p.unit = unit;
      p.c0 = unit == a.unit ? a.chunk : 0;
      p.c1 = unit == b.unit ? b.chunk : x.nchunks;
      p.part = (p.c0 == 0 && p.c1 == x.nchunks) ? -1 : 2 * cta + (unit == a.unit ? 0 : 1);
      ++unit;
      if (p.c0 < p.c1) return true;
    }
    return false;
  }
};

// Slot of the partial result that CTA c holds of the cut unit u; -1: none.
__device__ __forceinline__ int dense_piece_slot(const DenseTable& t, int u, int c) {
  const DensePoint a = t.cut[c], b = t.cut[c + 1];
  if (a.unit > u || b.unit < u || (b.unit == u && b.chunk == 0) || (a.unit == b.unit && a.chunk == b.chunk)) return -1;
  return 2 * c + (a.unit == u ? 0 : 1);
}

// Joins the pieces of each cut unit: with m the largest of the pieces' maxima
// (log2 units), l = sum l_p 2^(m_p - m), o = sum o_p 2^(m_p - m) / l.  A piece
// without a key of a row has m_p = -inf and l_p = 0 and counts nothing (scores that
// are all NaN: m_p = -inf, l_p = NaN; all -inf: l_p = -1, which counts nothing beside
// other scores and makes the row NaN, 0 / 0, without them).  One warp per row,
// 8 dims per lane, for units in kFewPieces or fewer, all read at once; pieces are
// added in the order of their keys.
constexpr int kFewPieces = 4;
__device__ __forceinline__ void store4(float* dst, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(dst) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* dst, float a, float b, float c, float d) {
  __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&x), *reinterpret_cast<uint32_t*>(&y));
}
template <typename T>
__global__ void __launch_bounds__(128)
    dense_combine_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseSplits sp,
                         const float* part, T* o, float* lse, int H) {
  const int i = blockIdx.x;
  const int u = sp.unit[i];
  const DenseUnit x = dense_unit(t, u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = blockIdx.y * 4 + warp;
  if (r >= x.nrows) return;
  const int64_t at = dense_q_row(t, x, x.row0 + r, H) * kHeadDim + lane * 4;
  const float* p[kFewPieces];                      // null: no such piece
#pragma unroll
  for (int k = 0; k < kFewPieces; ++k) {
    const int c = sp.first[i] + k, slot = c <= sp.last[i] ? dense_piece_slot(t, u, c) : -1;
    p[k] = slot < 0 ? nullptr : part + ((int64_t)slot * t.prows + r) * dense::kPartFloats;
  }
  pdl_wait();                                      // so far only the launch's own tables
  pdl_trigger();
  float2 ml[kFewPieces];
  float4 v[kFewPieces][2];
#pragma unroll
  for (int k = 0; k < kFewPieces; ++k) {
    ml[k] = make_float2(-INFINITY, 0.f);
    if (p[k]) {
      ml[k] = *reinterpret_cast<const float2*>(p[k] + kHeadDim);
      v[k][0] = reinterpret_cast<const float4*>(p[k])[lane];
      v[k][1] = reinterpret_cast<const float4*>(p[k])[lane + 32];
    }
  }
  float m = -INFINITY, l = 0.f, acc[8] = {};
#pragma unroll
  for (int k = 0; k < kFewPieces; ++k) m = fmaxf(m, ml[k].x);
#pragma unroll
  for (int k = 0; k < kFewPieces; ++k) {
    const float w = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - m);
    l += w * ml[k].y;                              // NaN if the piece's scores are all NaN
    if (w == 0.f) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      acc[4 * h] += w * v[k][h].x;
      acc[4 * h + 1] += w * v[k][h].y;
      acc[4 * h + 2] += w * v[k][h].z;
      acc[4 * h + 3] += w * v[k][h].w;
    }
  }
  float inv = l != 0.f ? 1.f / l : 0.f;           // l = 0: no key at all, or scores of -inf only
#pragma unroll
  for (int k = 0; k < kFewPieces; ++k)
    if (l == 0.f && ml[k].y < 0.f) inv = dense::kNan;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    store4(o + at + 128 * h, acc[4 * h] * inv, acc[4 * h + 1] * inv, acc[4 * h + 2] * inv, acc[4 * h + 3] * inv);
  if (lse && lane == 0) lse[at / kHeadDim] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// The same by a block of eight warps per row, for units in many pieces (decode
// of a long sequence: 74 of them): the pieces' statistics are read at once, the
// warps add up every eighth piece and then join in order.
template <typename T>
__global__ void __launch_bounds__(256, 1)
    dense_combine_many_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseSplits sp,
                              const float* part, T* o, float* lse, int H) {
  __shared__ float w_s[dense::kMaxGrid], red[8], acc_s[8][kHeadDim];
  __shared__ int64_t at_s[dense::kMaxGrid];
  const int u = sp.unit[blockIdx.x], c0 = sp.first[blockIdx.x], n = sp.last[blockIdx.x] - c0 + 1;
  const DenseUnit x = dense_unit(t, u);
  const int r = blockIdx.y;
  if (r >= x.nrows) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto block_reduce = [&](float v, bool is_max) {
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const float y = __shfl_xor_sync(0xffffffffu, v, off);
      v = is_max ? fmaxf(v, y) : v + y;
    }
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) v = is_max ? fmaxf(v, red[k]) : v + red[k];
    return v;
  };
  const int slot = threadIdx.x < n ? dense_piece_slot(t, u, c0 + (int)threadIdx.x) : -1;
  const int64_t at_part = ((int64_t)slot * t.prows + r) * dense::kPartFloats;
  if (threadIdx.x < n) at_s[threadIdx.x] = at_part;
  const int64_t at = dense_q_row(t, x, x.row0 + r, H);
  pdl_wait();                                            // so far only the launch's own tables
  pdl_trigger();
  float mp = -INFINITY, lp = 0.f;
  if (slot >= 0) {
    const float2 ml = *reinterpret_cast<const float2*>(part + at_part + kHeadDim);
    mp = ml.x;
    lp = ml.y;
  }
  const float m = block_reduce(mp, true);
  const float w = mp == -INFINITY ? 0.f : exp2f(mp - m);
  if (threadIdx.x < n) w_s[threadIdx.x] = w;
  const float l = block_reduce(w * lp, false);          // its barriers also order w_s, at_s
  // l = 0 (the same in every thread): no key at all, or scores of -inf only
  const bool all_inf = l == 0.f && __syncthreads_or(lp < 0.f);
  float acc[8] = {};
  constexpr int kBatch = 5;                              // pieces in flight: 74 of a long row are two batches
  for (int k0 = warp; k0 < n; k0 += 8 * kBatch) {
    float f[kBatch];
    float4 v[kBatch][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int k = k0 + 8 * b;
      f[b] = k < n ? w_s[k] : 0.f;
      v[b][0] = v[b][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f[b] != 0.f) {
        const float4* p = reinterpret_cast<const float4*>(part + at_s[k]);
        v[b][0] = p[lane];
        v[b][1] = p[lane + 32];
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        acc[4 * h] = fmaf(f[b], v[b][h].x, acc[4 * h]);
        acc[4 * h + 1] = fmaf(f[b], v[b][h].y, acc[4 * h + 1]);
        acc[4 * h + 2] = fmaf(f[b], v[b][h].z, acc[4 * h + 2]);
        acc[4 * h + 3] = fmaf(f[b], v[b][h].w, acc[4 * h + 3]);
      }
  }
  reinterpret_cast<float4*>(acc_s[warp])[lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  reinterpret_cast<float4*>(acc_s[warp])[lane + 32] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  __syncthreads();
  float v = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v += acc_s[k][threadIdx.x];
  o[at * kHeadDim + threadIdx.x] = IO<T>::from_f(l != 0.f ? v / l : all_inf ? dense::kNan : 0.f);
  if (lse && threadIdx.x == 0) lse[at] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace qsa
