// dense_simt.cuh -- dense causal GQA attention in fp32 on CUDA cores: forward
// over a paged cache or packed prompts, and the gradient over packed prompts.
//
// The formulas are those of qsa_paged_attn_fwd, qsa_prompt_attn_fwd and
// qsa_prompt_attn_bwd (qsa.h).  fp32 products have no tensor-core form of the
// same precision, so the work is FFMA on tiles held in shared memory, rows
// padded by 4 floats so that the 16-byte reads of neighbouring rows fall into
// different banks.  A thread owns R query rows x 4 keys of a 64-key chunk's
// scores and the same R rows x 16 dims of the result; the 16 threads of a row
// are half a warp, so the softmax exchanges by shuffles.  cp.async brings the
// next chunk's K during the softmax and products of this one and its V during
// the next scores.  At two warps per scheduler FMA and shared-memory reads hardly
// overlap, so what counts is reads per product and instructions: packed f32x2
// products, tiles as large as the registers allow.  Measured: the training step of
// prompts of 256, 700 and 33 tokens (24 heads, 2 groups, 24 GFLOP) 1.04 ms,
// the FMA pipe half busy, shared-memory reads two thirds.
//
// Masked places may hold anything: keys past the sequence are filled with
// zeros instead of being read, scores of keys after the row's position are
// replaced, and in a chunk that holds such keys their V rows are skipped
// row by row (0 * NaN would spread).
#pragma once
#include <type_traits>

#include "qsa_internal.cuh"
#include "sm100.cuh"
#include "dense.cuh"

namespace qsa {
namespace dense_simt {
constexpr int kThreads = 256;
constexpr int kKeys = 64;
constexpr int kLd = kHeadDim + 4;
constexpr int kPLd = kKeys + 4;
constexpr int kRowsWide = 64, kRowsNarrow = 16;
constexpr int fwd_smem(int rows) { return (rows * kLd + 2 * kKeys * kLd + rows * kPLd + kKeys) * 4; }
// gradient kernels: 64 rows (Q, dO) and 32 keys (K, V)
constexpr int kBRows = 64, kBKeys = 32, kBLd = kBKeys + 4;
constexpr int kBwdSmem = (2 * kBRows * kLd + 2 * kBKeys * kLd + 2 * kBRows * kBLd + 2 * kBRows) * 4;
}  // namespace dense_simt

// Where keys and values lie: paged, or packed token rows.
struct KvSource {
  const void* k;
  const void* v;
  const int32_t* table;      // paged only
  int32_t n_pages, page_tokens, max_pages;
};

// Element offset of the row of position j (-1: its page is out of range).
template <bool PAGED>
__device__ __forceinline__ int64_t kv_row(const KvSource& s, const DenseTable& t, int si, int grp, int32_t j) {
  if (PAGED) {
    const int32_t pi = j / s.page_tokens;
    const int32_t page = s.table[(int64_t)t.slot[si] * s.max_pages + pi];
    if (page < 0 || page >= s.n_pages) return -1;
    return (((int64_t)page * t.G + grp) * s.page_tokens + (j - pi * s.page_tokens)) * kHeadDim;
  }
  return ((int64_t)(t.q_offset[si] + j) * t.G + grp) * kHeadDim;
}

// Whether any of the keys j0 .. j1 of a segment is there to be attended, for rows
// whose softmax sum is 0: true means that all their scores are -inf.
template <bool PAGED>
__device__ __noinline__ bool any_key(const KvSource& s, const DenseTable& t, int si, int32_t j0, int32_t j1) {
  if (j1 < j0) return false;
  if (!PAGED) return true;
  const int32_t* pages = s.table + (int64_t)t.slot[si] * s.max_pages;
  for (int32_t pi = j0 / s.page_tokens; pi <= j1 / s.page_tokens; ++pi)
    if (pages[pi] >= 0 && pages[pi] < s.n_pages) return true;
  return false;
}

// Copies `rows` rows of 256 floats into shared memory (stride kLd); row r from
// src(r), zeros where src(r) is null.
template <typename T, typename Src>
__device__ __forceinline__ void simt_load_rows(float* dst, int rows, const T* any, Src src) {
  for (int i = threadIdx.x; i < rows * (kHeadDim / 4); i += dense_simt::kThreads) {
    const int r = i / (kHeadDim / 4), c = (i % (kHeadDim / 4)) * 4;
    const T* p = src(r);
    float* to = dst + r * dense_simt::kLd + c;
    if constexpr (sizeof(T) == 4) {
      sm100::cp_async16(sm100::smem_u32(to), p ? p + c : any, p ? 16u : 0u);
    } else {
      uint2 x = p ? *reinterpret_cast<const uint2*>(p + c) : make_uint2(0, 0);
      const float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x.x));
      const float2 b = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&x.y));
      *reinterpret_cast<float4*>(to) = make_float4(a.x, a.y, b.x, b.y);
    }
  }
}

// Two fp32 products and sums in one instruction: the FMA pipe's rate is the
// same, but at two warps per scheduler its issue slots are what runs short.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 lo2(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4& x) { return make_float2(x.z, x.w); }

// out[i][j] = a row (ra + i) . b row (rb + 16 j), rows of 256 floats (sums of the
// even and odd dims, then of both)
template <int R, int N>
__device__ __forceinline__ void simt_dots(const float* a, const float* b, int ra, int rb, float (&out)[R][N]) {
  using dense_simt::kLd;
  float2 acc[R][N];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 8
  for (int d = 0; d < kHeadDim; d += 4) {
    float4 x[R], y[N];
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ra + i) * kLd + d);
#pragma unroll
    for (int j = 0; j < N; ++j) y[j] = *reinterpret_cast<const float4*>(b + (rb + 16 * j) * kLd + d);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        acc[i][j] = fma2(lo2(x[i]), lo2(y[j]), acc[i][j]);
        acc[i][j] = fma2(hi2(x[i]), hi2(y[j]), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) out[i][j] = acc[i][j].x + acc[i][j].y;
}

// acc[i][16] += sum over n keys of p[row ra + i][key] * b[key][dims]; the
// thread's dims are 4 tx + 64 jj.  With limit[i] < n only the first limit[i]
// keys of row i are added.
template <int R, bool kLimited>
__device__ __forceinline__ void simt_accumulate_as(const float* p, int ldp, const float* b, int ra, int tx, int n,
                                                   const int (&limit)[R], float (&acc)[R][16]) {
  using dense_simt::kLd;
#pragma unroll 2
  for (int k = 0; k < n; k += 4) {
    float4 w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) w[i] = *reinterpret_cast<const float4*>(p + (ra + i) * ldp + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float4 y[4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) y[jj] = *reinterpret_cast<const float4*>(b + (k + kk) * kLd + 4 * tx + 64 * jj);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float f = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
        if (kLimited && k + kk >= limit[i]) continue;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          float2* d = reinterpret_cast<float2*>(&acc[i][4 * jj]);
          d[0] = fma2(make_float2(f, f), lo2(y[jj]), d[0]);
          d[1] = fma2(make_float2(f, f), hi2(y[jj]), d[1]);
        }
      }
    }
  }
}

template <int R>
__device__ __forceinline__ void simt_accumulate(const float* p, int ldp, const float* b, int ra, int tx, int n,
                                                bool limited, const int (&limit)[R], float (&acc)[R][16]) {
  if (limited)                                     // a copy of the loop: its comparisons are a fifth of its instructions
    simt_accumulate_as<R, true>(p, ldp, b, ra, tx, n, limit, acc);
  else
    simt_accumulate_as<R, false>(p, ldp, b, ra, tx, n, limit, acc);
}

template <int ROWS, bool PAGED>
__global__ void __launch_bounds__(dense_simt::kThreads, 1)
    dense_fwd_simt_kernel(const __grid_constant__ DenseTable t, KvSource kv, const float* q, float* o, float* lse,
                          float* part, int H, float scale) {
  using namespace dense_simt;
  constexpr int R = ROWS / 16;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + ROWS * kLd;
  float* Vs = Ks + kKeys * kLd;
  float* Ps = Vs + kKeys * kLd;
  int* ok = reinterpret_cast<int*>(Ps + ROWS * kPLd);         // key of the chunk can be attended
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, ra = ty * R;
  const float s2 = scale * 1.4426950408889634f;
  pdl_wait();
  pdl_trigger();
  DenseWalk walk;
  walk.init(t, blockIdx.x);
  DensePiece p;
  DenseUnit x;
  while (walk.next(t, p, x)) {
    const int si = x.si;
    auto q_at = [&](int r) { return dense_q_row(t, x, x.row0 + r, H); };
    auto load_kv = [&](float* dst, const void* base, int c, bool note) {
      simt_load_rows(dst, kKeys, (const float*)base, [&](int r) -> const float* {
        const int32_t j = c * kKeys + r;
        const int64_t off = j < x.kv_len ? kv_row<PAGED>(kv, t, si, x.grp, j) : -1;
        if (PAGED && j < x.kv_len && off < 0) report_error(kErrBadIndex);
        return off < 0 ? nullptr : (const float*)base + off;
      });
      if (note && threadIdx.x < kKeys) {
        const int32_t j = c * kKeys + (int)threadIdx.x;
        ok[threadIdx.x] = j < x.kv_len && kv_row<PAGED>(kv, t, si, x.grp, j) >= 0;
      }
      sm100::cp_async_commit();
    };
    simt_load_rows(Qs, ROWS, q, [&](int r) -> const float* { return r < x.nrows ? q + q_at(r) * kHeadDim : nullptr; });
    load_kv(Ks, kv.k, p.c0, true);
    load_kv(Vs, kv.v, p.c0, false);
    int64_t pos[R];
    float m[R], l[R], acc[R][16];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      pos[i] = t.pos0[si] + (x.row0 + ra + i) / t.hpg;
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][k] = 0.f;
    }
    const int64_t first_pos = t.pos0[si] + x.row0 / t.hpg;
    for (int c = p.c0; c < p.c1; ++c) {
      const int64_t j0 = (int64_t)c * kKeys;
      sm100::cp_async_wait<1>();
      __syncthreads();
      float s[R][4];
      simt_dots<R, 4>(Qs, Ks, ra, tx, s);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float mc = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = tx + 16 * j;
          s[i][j] = (j0 + key <= pos[i] && ok[key]) ? s[i][j] * s2 : -INFINITY;
          mc = fmaxf(mc, s[i][j]);
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, off));
        const float mn = fmaxf(m[i], mc), mb = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[i] - mb);          // 0 while the row has no key yet
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(s[i][j] - mb);
          sum += e;
          Ps[(ra + i) * kPLd + tx + 16 * j] = e;
        }
#pragma unroll
        for (int off = 8; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        l[i] = l[i] * f + sum;
        m[i] = mn;
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[i][k] *= f;
      }
      __syncthreads();                             // K and ok read, P written
      if (c + 1 < p.c1) load_kv(Ks, kv.k, c + 1, true); else sm100::cp_async_commit();
      sm100::cp_async_wait<1>();
      __syncthreads();
      int limit[R];
#pragma unroll
      for (int i = 0; i < R; ++i) limit[i] = (int)min((int64_t)kKeys, pos[i] - j0 + 1);
      simt_accumulate<R>(Ps, kPLd, Vs, ra, tx, kKeys, j0 + kKeys - 1 > first_pos, limit, acc);
      __syncthreads();
      if (c + 1 < p.c1) load_kv(Vs, kv.v, c + 1, false); else sm100::cp_async_commit();
    }
    sm100::cp_async_wait_all();
    __syncthreads();                               // shared memory free for the next piece
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (ra + i >= x.nrows) continue;
      const bool all_inf =
          l[i] == 0.f && any_key<PAGED>(kv, t, si, p.c0 * kKeys, min((int32_t)pos[i], p.c1 * kKeys - 1));
      if (p.part < 0) {
        const float inv = all_inf ? dense::kNan : l[i] != 0.f ? 1.f / l[i] : 0.f;
        const int64_t at = q_at(ra + i);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          store4(o + at * kHeadDim + 4 * tx + 64 * jj, acc[i][4 * jj] * inv, acc[i][4 * jj + 1] * inv,
                      acc[i][4 * jj + 2] * inv, acc[i][4 * jj + 3] * inv);
        if (lse && tx == 0) lse[at] = l[i] != 0.f ? (m[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
      } else {
        float* dst = part + ((int64_t)p.part * t.prows + ra + i) * dense::kPartFloats;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          *reinterpret_cast<float4*>(dst + 4 * tx + 64 * jj) =
              make_float4(acc[i][4 * jj], acc[i][4 * jj + 1], acc[i][4 * jj + 2], acc[i][4 * jj + 3]);
        if (tx == 0) {
          dst[kHeadDim] = m[i];
          dst[kHeadDim + 1] = all_inf ? -1.f : l[i];
        }
      }
    }
  }
}

// ------------------------------------------------------------------ gradient
struct DenseBwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* lse;        // [T][H]
  const float* delta;      // [T][H]
  const void* dout;
  void* dq;
  void* dk;
  void* dv;
  int H;
  float scale;
  const uint8_t* flags;    // null: every segment; else the flagged ones (segment_flagged)
};

// delta[i][h] = dout[i][h] . o[i][h], one warp per row of the segments.
template <typename T>
__global__ void __launch_bounds__(256)
    dense_delta_kernel(SegTable st, const T* o, const T* dout, float* delta, int H) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int item = (int)(w / H);
  if (item >= st.item0[st.n]) return;
  const int si = find_segment(st, item);
  const int64_t at = (int64_t)(st.q_offset[si] + item - st.item0[si]) * H + w % H;
  Vec8<T> a, b;
  a.load(o + at * kHeadDim + lane * 8);
  b.load(dout + at * kHeadDim + lane * 8);
  float fa[8], fb[8], s = 0.f;
  a.get(fa);
  b.get(fb);
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(fa[i], fb[i], s);
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (lane == 0) delta[at] = s;
}

// The gradient's products of 64 rows of a with 32 rows of b: a thread adds up 8 x 4
// of them over a quarter of the dims (every fourth group of four), so that 12
// shared-memory reads feed 128 products (4 x 2 over all dims: 6 for 32); the four
// quarters, in the lanes 8 apart, then meet by exchanging halves.  out[i][j] is
// that of row simt_row0() + i and key simt_key0() + j.
__device__ __forceinline__ int simt_row0() {
  const int lane = threadIdx.x & 31;
  return (threadIdx.x >> 6) * 16 + 4 * ((lane >> 2) & 1) + 8 * ((lane >> 3) & 1);
}
__device__ __forceinline__ int simt_key0() {
  const int lane = threadIdx.x & 31;
  return ((threadIdx.x >> 5) & 1) * 16 + 4 * (lane & 3) + 2 * (lane >> 4);
}
__device__ __forceinline__ void simt_dots_64x32(const float* a, const float* b, float (&out)[4][2]) {
  using dense_simt::kLd;
  const int lane = threadIdx.x & 31, quarter = lane >> 3;
  const float* pa = a + ((threadIdx.x >> 6) * 16 + 4 * ((lane >> 2) & 1)) * kLd + 4 * quarter;
  const float* pb = b + (((threadIdx.x >> 5) & 1) * 16 + 4 * (lane & 3)) * kLd + 4 * quarter;
  float2 acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int d = 0; d < kHeadDim; d += 16) {
    float4 x[8], y[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const float4*>(pa + ((i & 3) + 8 * (i >> 2)) * kLd + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(pb + j * kLd + d);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(lo2(x[i]), lo2(y[j]), acc[i][j]);
        acc[i][j] = fma2(hi2(x[i]), hi2(y[j]), acc[i][j]);
      }
  }
  const bool odd = quarter & 1, high = quarter & 2;
  float half[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v0 = acc[i][j].x + acc[i][j].y, v1 = acc[i + 4][j].x + acc[i + 4][j].y;
      half[i][j] = (odd ? v1 : v0) + __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 8);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
      out[i][j] = (high ? half[i][j + 2] : half[i][j]) +
                  __shfl_xor_sync(0xffffffffu, high ? half[i][j] : half[i][j + 2], 16);
}

// From a thread's scores and dP of 64 rows x 32 keys, P (if Ps) and dS into shared
// memory ([row][key]); row statistics in st_lse (log2 units) and st_delta; masked
// entries are zero.  row0: the tile's first row, in rows of the segment.
__device__ __forceinline__ void simt_p_ds(const float (&s)[4][2], const float (&dp)[4][2], float* Ps, float* Ds,
                                          const float* st_lse, const float* st_delta, int32_t row0, int nrows, int hpg,
                                          int32_t j0, int32_t n_keys, float s2) {
  using namespace dense_simt;
  const int ra = simt_row0(), ka = simt_key0();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ra + i;
    const int32_t pos = (row0 + r) / hpg;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int key = ka + j;
      const bool seen = r < nrows && j0 + key <= pos && j0 + key < n_keys;
      const float p = seen ? exp2f(fmaf(s[i][j], s2, -st_lse[r])) : 0.f;
      if (Ps) Ps[r * kBLd + key] = p;
      Ds[r * kBLd + key] = seen ? p * (dp[i][j] - st_delta[r]) : 0.f;
    }
  }
}

// Flags of the bf16 gradient: 32 bytes for each 128 tokens of a segment (from its
// first statistics tile on), one per 4 tokens; nonzero: they hold what is not
// finite.  True if any of the segment's is; called by whole warps.
__device__ __forceinline__ bool segment_flagged(const uint8_t* flags, int32_t tile, int32_t n) {
  const uint4* f = reinterpret_cast<const uint4*>(flags) + 2 * (int64_t)tile;
  uint32_t any = 0;
  for (int i = threadIdx.x & 31; i < (n + 127) / 128 * 2; i += 32) {
    const uint4 v = f[i];
    any |= v.x | v.y | v.z | v.w;
  }
  return __any_sync(0xffffffffu, any != 0);
}

// dq of tiles of 64 rows, in chunks of 32 keys (dense.cuh); a piece of a cut
// unit leaves its unscaled sum.
template <typename T>
__device__ __forceinline__ void simt_dq(const DenseTable& t, const DenseBwdArgs& a, float* part) {
  using namespace dense_simt;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Os = Qs + kBRows * kLd;
  float* Ks = Os + kBRows * kLd;
  float* Vs = Ks + kBKeys * kLd;
  float* Ps = Vs + kBKeys * kLd;
  float* Ds = Ps + kBRows * kBLd;
  float* st_lse = Ds + kBRows * kBLd;
  float* st_delta = st_lse + kBRows;
  const float s2 = a.scale * 1.4426950408889634f;
  const int tx = threadIdx.x & 15, ra = (threadIdx.x >> 4) * 4;
  DenseWalk walk;
  walk.init(t, blockIdx.x);
  DensePiece p;
  DenseUnit x;
  while (walk.next(t, p, x)) {
    const int si = x.si;
    if (a.flags && !segment_flagged(a.flags, t.slot[si], t.q_len[si])) continue;
    __syncthreads();
    auto q_at = [&](int r) { return dense_q_row(t, x, x.row0 + r, a.H); };
    auto rows_of = [&](const void* base) {
      return [&, base](int r) -> const T* {
        return r < x.nrows ? (const T*)base + q_at(r) * kHeadDim : nullptr;
      };
    };
    simt_load_rows(Qs, kBRows, (const T*)a.q, rows_of(a.q));
    simt_load_rows(Os, kBRows, (const T*)a.dout, rows_of(a.dout));
    if (threadIdx.x < kBRows) {
      const bool v = threadIdx.x < x.nrows;
      st_lse[threadIdx.x] = v ? a.lse[q_at(threadIdx.x)] * 1.4426950408889634f : 0.f;
      st_delta[threadIdx.x] = v ? a.delta[q_at(threadIdx.x)] : 0.f;
    }
    auto load_keys = [&](float* dst, const void* base, int c) {
      simt_load_rows(dst, kBKeys, (const T*)base, [&](int r) -> const T* {
        const int32_t j = c * kBKeys + r;
        return j < x.kv_len ? (const T*)base + ((int64_t)(t.q_offset[si] + j) * t.G + x.grp) * kHeadDim : nullptr;
      });
    };
    load_keys(Vs, a.v, p.c0);
    sm100::cp_async_commit();
    load_keys(Ks, a.k, p.c0);
    sm100::cp_async_commit();
    float acc[4][16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][k] = 0.f;
    const int32_t first_pos = x.row0 / t.hpg;
    // V of the next chunk loads under this one's sum, K under the next one's dP
    for (int c = p.c0; c < p.c1; ++c) {
      const int32_t j0 = c * kBKeys;
      float sc[4][2], dp[4][2];
      sm100::cp_async_wait<1>();
      __syncthreads();
      simt_dots_64x32(Os, Vs, dp);
      sm100::cp_async_wait<0>();
      __syncthreads();
      simt_dots_64x32(Qs, Ks, sc);
      simt_p_ds(sc, dp, nullptr, Ds, st_lse, st_delta, x.row0, x.nrows, t.hpg, j0, x.kv_len, s2);
      __syncthreads();
      if (c + 1 < p.c1) load_keys(Vs, a.v, c + 1);
      sm100::cp_async_commit();
      int limit[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) limit[i] = min(kBKeys, (x.row0 + ra + i) / t.hpg - j0 + 1);
      simt_accumulate<4>(Ds, kBLd, Ks, ra, tx, kBKeys, j0 + kBKeys - 1 > first_pos, limit, acc);
      __syncthreads();
      if (c + 1 < p.c1) load_keys(Ks, a.k, c + 1);
      sm100::cp_async_commit();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (ra + i >= x.nrows) continue;
      if (p.part < 0) {
        T* dst = (T*)a.dq + q_at(ra + i) * kHeadDim;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          store4(dst + 4 * tx + 64 * jj, acc[i][4 * jj] * a.scale, acc[i][4 * jj + 1] * a.scale,
                      acc[i][4 * jj + 2] * a.scale, acc[i][4 * jj + 3] * a.scale);
      } else {
        float* dst = part + ((int64_t)p.part * t.prows + ra + i) * dense::kPartFloats;
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
          store4(dst + 4 * tx + 64 * jj, acc[i][4 * jj], acc[i][4 * jj + 1], acc[i][4 * jj + 2],
                      acc[i][4 * jj + 3]);
      }
    }
  }
}

// dk and dv of tiles of 32 keys, by keys (dense.cuh): a chunk is 64 tokens of
// one head.  A thread owns 4 keys x 8 dims of both.  A piece of a cut unit leaves
// its unscaled sums, dv's rows kBKeys behind dk's.  (One block per unit held 64 of
// 148 SMs at 989 tokens x 2 groups, and the longest of them 3.5 ms.)
template <typename T>
__device__ __forceinline__ void simt_dkv(const DenseTable& t, const DenseBwdArgs& a, float* part) {
  using namespace dense_simt;
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Os = Qs + kBRows * kLd;
  float* Ks = Os + kBRows * kLd;
  float* Vs = Ks + kBKeys * kLd;
  float* Ps = Vs + kBKeys * kLd;
  float* Ds = Ps + kBRows * kBLd;
  float* st_lse = Ds + kBRows * kBLd;
  float* st_delta = st_lse + kBRows;
  const float s2 = a.scale * 1.4426950408889634f;
  const int kq = (threadIdx.x >> 5) * 4, dl = (threadIdx.x & 31) * 4;
  DenseWalk walk;
  walk.init(t, blockIdx.x);
  DensePiece p;
  DenseUnit x;
  while (walk.next(t, p, x)) {
    if (a.flags && !segment_flagged(a.flags, t.slot[x.si], t.q_len[x.si])) continue;
    __syncthreads();
    const int32_t j0 = x.row0, n = x.kv_len;
    const int64_t q0 = t.q_offset[x.si];
    auto key_at = [&](int r) -> int64_t { return ((q0 + j0 + r) * t.G + x.grp) * kHeadDim; };
    auto keys_of = [&](const void* base) {
      return [&, base](int r) -> const T* { return j0 + r < n ? (const T*)base + key_at(r) : nullptr; };
    };
    simt_load_rows(Ks, kBKeys, (const T*)a.k, keys_of(a.k));
    simt_load_rows(Vs, kBKeys, (const T*)a.v, keys_of(a.v));
    float dk[4][8], dv[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) dk[i][k] = dv[i][k] = 0.f;
    // rows of chunk c: 64 tokens of one head
    auto load_chunk = [&](float* dst, const void* base, int c, bool stats) {
      const int32_t i0 = j0 + c / t.hpg * kBRows;
      const int nrows = min(kBRows, n - i0);
      const int64_t at = (q0 + i0) * a.H + x.grp * t.hpg + c % t.hpg;
      simt_load_rows(dst, kBRows, (const T*)base, [&](int r) -> const T* {
        return r < nrows ? (const T*)base + (at + (int64_t)r * a.H) * kHeadDim : nullptr;
      });
      if (stats && threadIdx.x < kBRows) {
        const bool v = threadIdx.x < nrows;
        const int64_t row = at + (int64_t)threadIdx.x * a.H;
        st_lse[threadIdx.x] = v ? a.lse[row] * 1.4426950408889634f : 0.f;
        st_delta[threadIdx.x] = v ? a.delta[row] : 0.f;
      }
    };
    load_chunk(Os, a.dout, p.c0, true);
    sm100::cp_async_commit();
    load_chunk(Qs, a.q, p.c0, false);
    sm100::cp_async_commit();
    // dO of the next chunk loads under this one's dk, Q under the next one's dP
    for (int c = p.c0; c < p.c1; ++c) {
      const int32_t i0 = j0 + c / t.hpg * kBRows;
      const int nrows = min(kBRows, n - i0);
      float sc[4][2], dp[4][2];
      sm100::cp_async_wait<1>();
      __syncthreads();
      simt_dots_64x32(Os, Vs, dp);
      sm100::cp_async_wait<0>();
      __syncthreads();
      simt_dots_64x32(Qs, Ks, sc);
      simt_p_ds(sc, dp, Ps, Ds, st_lse, st_delta, i0, nrows, 1, j0, n, s2);
      __syncthreads();
      // sums over the chunk's rows of w[row][key] times the row, for this thread's
      // keys; a row before a key does not touch it
      const bool limited = j0 + kBKeys - 1 > i0;
      auto add_rows = [&](auto is_limited, const float* w, const float* rows, float (&g)[4][8]) {
#pragma unroll 4
        for (int r = 0; r < nrows; ++r) {
          const float4 wr = *reinterpret_cast<const float4*>(w + r * kBLd + kq);
          const float ww[4] = {wr.x, wr.y, wr.z, wr.w};
          const float4 x0 = *reinterpret_cast<const float4*>(rows + r * kLd + dl);
          const float4 x1 = *reinterpret_cast<const float4*>(rows + r * kLd + dl + 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (decltype(is_limited)::value && j0 + kq + i > i0 + r) continue;
            float2* d = reinterpret_cast<float2*>(g[i]);
            const float2 f = make_float2(ww[i], ww[i]);
            d[0] = fma2(f, lo2(x0), d[0]);
            d[1] = fma2(f, hi2(x0), d[1]);
            d[2] = fma2(f, lo2(x1), d[2]);
            d[3] = fma2(f, hi2(x1), d[3]);
          }
        }
      };
      if (limited) add_rows(std::true_type{}, Ps, Os, dv); else add_rows(std::false_type{}, Ps, Os, dv);
      __syncthreads();
      if (c + 1 < p.c1) load_chunk(Os, a.dout, c + 1, true);
      sm100::cp_async_commit();
      if (limited) add_rows(std::true_type{}, Ds, Qs, dk); else add_rows(std::false_type{}, Ds, Qs, dk);
      __syncthreads();
      if (c + 1 < p.c1) load_chunk(Qs, a.q, c + 1, false);
      sm100::cp_async_commit();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (kq + i >= x.nrows) continue;
      const int64_t at = key_at(kq + i) + dl;
      float* pk = part + ((int64_t)p.part * t.prows + kq + i) * dense::kPartFloats + dl;
      float* pv = pk + kBKeys * dense::kPartFloats;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (p.part < 0) {
          store4((T*)a.dk + at + 128 * h, dk[i][4 * h] * a.scale, dk[i][4 * h + 1] * a.scale,
                      dk[i][4 * h + 2] * a.scale, dk[i][4 * h + 3] * a.scale);
          store4((T*)a.dv + at + 128 * h, dv[i][4 * h], dv[i][4 * h + 1], dv[i][4 * h + 2], dv[i][4 * h + 3]);
        } else {
          store4(pk + 128 * h, dk[i][4 * h], dk[i][4 * h + 1], dk[i][4 * h + 2], dk[i][4 * h + 3]);
          store4(pv + 128 * h, dv[i][4 * h], dv[i][4 * h + 1], dv[i][4 * h + 2], dv[i][4 * h + 3]);
        }
      }
    }
  }
}

// fp32: dq, or dk and dv, of a launch.
__global__ void __launch_bounds__(dense_simt::kThreads, 1)
    dense_dq_simt_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseBwdArgs a, float* part) {
  pdl_wait();
  pdl_trigger();
  simt_dq<float>(t, a, part);
}
__global__ void __launch_bounds__(dense_simt::kThreads, 1)
    dense_dkv_simt_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseBwdArgs a, float* part) {
  pdl_wait();
  pdl_trigger();
  simt_dkv<float>(t, a, part);
}
// bf16: all gradients of the flagged segments, of which there are hardly ever
// any; no unit of the tables is cut.
__global__ void __launch_bounds__(dense_simt::kThreads, 1)
    dense_bwd_flagged_kernel(const __grid_constant__ DenseTable rows, const __grid_constant__ DenseTable keys,
                             const __grid_constant__ DenseBwdArgs a) {
  pdl_wait();
  pdl_trigger();
  bool any = false;
  for (int i = threadIdx.x >> 5; i < rows.n; i += dense_simt::kThreads / 32)
    any |= segment_flagged(a.flags, rows.slot[i], rows.q_len[i]);
  if (!__syncthreads_or(any)) return;
  simt_dq<__nv_bfloat16>(rows, a, nullptr);
  simt_dkv<__nv_bfloat16>(keys, a, nullptr);
}

// Adds up the pieces of each cut unit in the order of their chunks, scales and
// rounds.  blockIdx.z: an output of the call; one warp per stationary row.  With
// flags: not the units of flagged segments.
template <typename T>
struct DenseBwdJoin {
  const float* part;
  T* out;
  float factor;
  int row;                 // of a unit's partial result, for its first stationary row
  int keys;                // which table
};
template <typename T>
struct DenseBwdJoins {
  DenseBwdJoin<T> join[3];
  const uint8_t* flags;    // or null
  int H;
};
template <typename T>
__global__ void __launch_bounds__(128)
    dense_bwd_combine_kernel(const __grid_constant__ DenseTable rows, const __grid_constant__ DenseSplits srows,
                             const __grid_constant__ DenseTable keys, const __grid_constant__ DenseSplits skeys,
                             const __grid_constant__ DenseBwdJoins<T> joins) {
  const DenseBwdJoin<T>& w = joins.join[blockIdx.z];
  const DenseTable& t = w.keys ? keys : rows;
  const DenseSplits& sp = w.keys ? skeys : srows;
  const int i = blockIdx.x;
  if (i >= sp.n) return;
  const int u = sp.unit[i];
  const DenseUnit x = dense_unit(t, u);
  const int lane = threadIdx.x & 31, r = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (r >= x.nrows) return;
  pdl_wait();                                      // so far only the launch's own tables
  pdl_trigger();
  if (joins.flags && segment_flagged(joins.flags, t.slot[x.si], t.q_len[x.si])) return;
  float acc[8] = {};
  for (int c0 = sp.first[i]; c0 <= sp.last[i]; c0 += 32) {
    const int my = c0 + lane <= sp.last[i] ? dense_piece_slot(t, u, c0 + lane) : -1;
    const int n = min(32, sp.last[i] - c0 + 1);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
      const int slot = __shfl_sync(0xffffffffu, my, k);
      const float4* p =
          reinterpret_cast<const float4*>(w.part + ((int64_t)max(slot, 0) * t.prows + w.row + r) * dense::kPartFloats);
      const float4 v0 = slot >= 0 ? p[2 * lane] : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 v1 = slot >= 0 ? p[2 * lane + 1] : make_float4(0.f, 0.f, 0.f, 0.f);
      acc[0] += v0.x; acc[1] += v0.y; acc[2] += v0.z; acc[3] += v0.w;
      acc[4] += v1.x; acc[5] += v1.y; acc[6] += v1.z; acc[7] += v1.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] *= w.factor;
  const int32_t row = x.row0 + r;
  const int64_t at =
      t.by_keys ? (int64_t)(t.q_offset[x.si] + row) * t.G + x.grp : dense_q_row(t, x, row, joins.H);
  Vec8<T> v;
  v.set(acc);
  v.store(w.out + at * kHeadDim + lane * 8);
}

}  // namespace qsa
