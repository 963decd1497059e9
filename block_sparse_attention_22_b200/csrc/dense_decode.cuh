// dense_decode.cuh -- dense attention of single new tokens over a paged cache,
// bf16: one token's heads of a KV group against all its keys.
//
// The work is the HBM read of K and V once: 12 heads make 12 flop per byte and
// operand, beyond what CUDA cores add up at HBM rate, a fifth of what
// mma.sync gives.  tcgen05 tiles would be a tenth full and tie the SM's loads
// to one chain of barriers (a chunk's products, softmax and the slots' reuse took
// 1.8 us for 64 KiB on them: 2.9 TB/s); here eight warps each stream keys of
// their own, 16 at a time, through three 8 KiB slots, with no barrier between
// them, so that 128 KiB are in flight per SM all the time:
//   S[16 heads, 16 keys] = Q K^T   32 mma.m16n8k16, K by ldmatrix
//   O[16 heads, 256]    += P V     32 mma.m16n8k16, V by ldmatrix.trans
// A warp keeps its own maximum (moved only when a tile exceeds it by more than 8 in
// log2 units), sum and O (128 registers); at the end of a piece the warps join
// through shared memory.  P is rounded to bf16 for its product, the row sum
// adds the unrounded values.  Tables, pieces and their join: dense.cuh, rows =
// 16 and a chunk of 128 keys, 16 for each warp.  Measured: 32 sequences of 16K to
// 50K keys (2.1 GB) 342 us with the join, 0.97 of the HBM rate; one row at 256K 95
// us, 0.87.
//
// A token's keys are all visible to it, so nothing is masked but keys beyond
// the sequence and of pages out of range: neither is read (zeros are filled
// in), their scores are -inf.
#pragma once
#include "dense.cuh"
#include "dense_simt.cuh"
#include "dense_tc.cuh"

namespace qsa {
namespace dense_decode {
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kTile = 16;                             // keys of a warp's step
constexpr int kRows = 16, kKeys = kWarps * kTile;     // of a unit, of a chunk
constexpr int kSlotBytes = kTile * kHeadDim * 2, kSlots = 3;
constexpr int kOffQ = kWarps * kSlots * kSlotBytes;
constexpr int kOffStat = kOffQ + kRows * kHeadDim * 2;       // maxima and sums of the warps' rows
constexpr int kSmemBytes = kOffStat + 2 * kWarps * kRows * 4;
constexpr int kOLd = kHeadDim + 8;                    // floats between a warp's O rows in shared memory
static_assert(kRows * kOLd * 4 <= kSlots * kSlotBytes, "O of a warp over its slots");
}  // namespace dense_decode

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_m16n8k16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Joins the warps' maxima, sums and O (in shared memory, a warp's over its slots)
// of a piece: a whole unit's result, or the piece's partial one.  Eight lanes
// make a row's factors first, in place of the maxima; then a thread joins four
// dims of every fourth row.
template <typename T>
__device__ __forceinline__ void decode_join(const DenseTable& t, const KvSource& kv, const DenseUnit& x,
                                            const DensePiece& p, int64_t head0, const unsigned char* smem, float* m_s,
                                            float* l_s, T* o, float* lse, float* part) {
  using namespace dense_decode;
  static_assert(kWarps == 8 && kRows * kWarps <= kThreads && kThreads == kHeadDim, "thread layouts below");
  float* const dst = part + (int64_t)p.part * t.prows * dense::kPartFloats;      // used by a cut unit's piece only
  if (threadIdx.x < kRows * kWarps) {
    const int r = threadIdx.x >> 3, at = (threadIdx.x & 7) * kRows + r;
    const float m = m_s[at];
    float mr = m, l;
#pragma unroll
    for (int off = 4; off; off >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, off));
    const float f = m == -INFINITY ? 0.f : exp2f(m - mr);
    l = f * l_s[at];
#pragma unroll
    for (int off = 4; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    m_s[at] = f;
    if ((threadIdx.x & 7) == 0) {
      const bool all_inf = r < x.nrows && l == 0.f &&
                           any_key<true>(kv, t, x.si, p.c0 * kKeys, min(x.kv_len, p.c1 * kKeys) - 1);
      l_s[at] = all_inf ? dense::kNan : l;
      if (r < x.nrows && p.part >= 0)
        *reinterpret_cast<float2*>(dst + r * dense::kPartFloats + kHeadDim) = make_float2(mr, all_inf ? -1.f : l);
      else if (r < x.nrows && lse)
        lse[head0 + r] = l != 0.f ? (mr + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  const int d = (threadIdx.x & 63) * 4;
#pragma unroll 2
  for (int r = threadIdx.x >> 6; r < x.nrows; r += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = m_s[w * kRows + r];
      const float4 y =
          *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * kSlots * kSlotBytes) + r * kOLd + d);
      v.x = fmaf(f, y.x, v.x);
      v.y = fmaf(f, y.y, v.y);
      v.z = fmaf(f, y.z, v.z);
      v.w = fmaf(f, y.w, v.w);
    }
    if (p.part >= 0) {
      *reinterpret_cast<float4*>(dst + r * dense::kPartFloats + d) = v;
    } else {
      const float l = l_s[r], inv = l != 0.f ? 1.f / l : 0.f;
      store4(o + (head0 + r) * kHeadDim + d, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
  }
}

__global__ void __launch_bounds__(dense_decode::kThreads, 1)
    dense_decode_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseTcArgs a) {
  using namespace dense_decode;
  using namespace sm100;
  extern __shared__ __align__(1024) unsigned char smem_1k[];
  unsigned char* const smem = smem_1k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = smem_u32(smem) + warp * kSlots * kSlotBytes, q_addr = smem_u32(smem + kOffQ);
  float* const o_s = reinterpret_cast<float*>(smem + warp * kSlots * kSlotBytes);
  float* const m_s = reinterpret_cast<float*>(smem + kOffStat);        // [warp][row]
  float* const l_s = m_s + kWarps * kRows;
  const float tau2 = a.scale * 1.4426950408889634f;
  // 16-byte piece `piece` of line r of a tile, swizzled so that eight lines of one piece hit all banks
  auto at = [](int r, int piece) { return (uint32_t)(r * (kHeadDim * 2) + ((piece ^ (r & 7)) << 4)); };
  const int mi = lane >> 3, ml = lane & 7;              // this lane's matrix and line of an ldmatrix.x4
  dense_wait_first(a.late);
  DenseWalk walk;
  walk.init(t, blockIdx.x);
  DensePiece p;
  DenseUnit x;
  while (walk.next(t, p, x)) {
    const int64_t head0 = (int64_t)t.q_offset[x.si] * a.H + x.grp * t.hpg;
    // Q, rows beyond the group's heads zero; it arrives with the first tile's K
    for (int i = threadIdx.x; i < kRows * 32; i += kThreads) {
      const int r = i >> 5, c = i & 31;
      cp_async16(q_addr + at(r, c), a.q + (head0 + (r < x.nrows ? r : 0)) * kHeadDim + c * 8, r < x.nrows ? 16u : 0u);
    }
    // this warp's tiles: keys (p.c0 + i) * 128 + 16 warp, of those that hold a key
    const int32_t key0 = p.c0 * kKeys + warp * kTile;
    const int n = min(p.c1 - p.c0, max(0, (x.kv_len - key0 + kKeys - 1) / kKeys));
    // rows of the tiles, looked up for 32 tiles at a time (-1: page out of range)
    int32_t look0 = -32;
    int64_t my_row = -1;
    auto tile_row = [&](int i) -> int64_t {               // first cache row of tile i (lanes agree)
      if (i - look0 >= 32) {
        look0 = i;
        const int32_t key = key0 + (i + lane) * kKeys;
        my_row = -1;
        if (i + lane < n) {
          const int32_t pi = key / a.kv.page_tokens;
          const int32_t page = a.kv.table[(int64_t)t.slot[x.si] * a.kv.max_pages + pi];
          if (page >= 0 && page < a.kv.n_pages)
            my_row = ((int64_t)page * t.G + x.grp) * a.kv.page_tokens + (key - pi * a.kv.page_tokens);
          else
            report_error(kErrBadIndex);
        }
      }
      return __shfl_sync(0xffffffffu, my_row, i - look0);
    };
    // item 2 i: K of tile i, 2 i + 1: V; slot = item % 3.  The row of a tile
    // is kept for its V and (below) its scores.
    int64_t row_k = -1, row_v = -1;                       // of the last K / V issued
    auto load = [&](int item) {
      const int i = item >> 1;
      if (i < n) {
        const bool is_v = item & 1;
        const int64_t row = is_v ? row_v : tile_row(i);
        if (!is_v) row_k = row;
        const __nv_bfloat16* base = (const __nv_bfloat16*)(is_v ? a.kv.v : a.kv.k);
        const int valid = row < 0 ? 0 : min(kTile, x.kv_len - (key0 + i * kKeys));
        const __nv_bfloat16* src = base + (valid > 0 ? row : 0) * kHeadDim + lane * 8;
        const uint32_t dst = ring + (item % kSlots) * kSlotBytes;
#pragma unroll
        for (int r = 0; r < kTile; ++r)
          cp_async16(dst + at(r, lane), r < valid ? src + r * kHeadDim : src, r < valid ? 16u : 0u);
      }
      cp_async_commit();
    };
    float o[32][4];
#pragma unroll
    for (int j = 0; j < 32; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[j][k] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};      // rows lane/4 and lane/4 + 8
    load(0);
    row_v = row_k;
    load(1);
    int64_t row_now = row_k;
    load(2);
    cp_async_wait<2>();
    __syncthreads();                                      // Q written
    for (int i = 0; i < n; ++i) {
      // ---- S of tile i
      cp_async_wait<2>();
      __syncwarp();
      float s[2][2][4] = {};                              // [k-step parity][keys 0-7, 8-15]
      const uint32_t ks = ring + ((2 * i) % kSlots) * kSlotBytes;
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        uint32_t qa[4], kb[4];
        ldmatrix_x4(q_addr + at((mi & 1) * 8 + ml, 2 * kk + (mi >> 1)), qa);
        ldmatrix_x4(ks + at((mi >> 1) * 8 + ml, 2 * kk + (mi & 1)), kb);
        mma_m16n8k16(s[kk & 1][0], qa, kb[0], kb[1]);
        mma_m16n8k16(s[kk & 1][1], qa, kb[2], kb[3]);
      }
      __syncwarp();
      row_v = row_k;                                      // of tile i + 1
      const bool bad = row_now < 0;
      row_now = row_k;
      load(2 * i + 3);                                    // V of tile i + 1 over K of tile i
      // ---- softmax: this thread's keys are 8 j + 2 (lane % 4), + 1
      const int left = bad ? 0 : x.kv_len - (key0 + i * kKeys);
      uint32_t pa[4];
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float v = s[0][j][k] + s[1][j][k];
          s[0][j][k] = 8 * j + 2 * (lane & 3) + (k & 1) < left ? v * tau2 : -INFINITY;
          mx[k >> 1] = fmaxf(mx[k >> 1], s[0][j][k]);
        }
      float f[2] = {1.f, 1.f};
      bool need = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        if (mx[r] > m[r] + 8.f) {                         // false while both are -inf
          if (m[r] != -INFINITY) {
            f[r] = exp2f(m[r] - mx[r]);
            need = true;
          }
          m[r] = mx[r];
        }
      }
      if (__any_sync(0xffffffffu, need)) {
        l[0] *= f[0];
        l[1] *= f[1];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          o[j][0] *= f[0];
          o[j][1] *= f[0];
          o[j][2] *= f[1];
          o[j][3] *= f[1];
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float e[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float mb = m[k >> 1] == -INFINITY ? 0.f : m[k >> 1];
          e[k] = ex2_approx(s[0][j][k] - mb);
          l[k >> 1] += e[k];
        }
        pa[2 * j] = pack_bf16x2(e[0], e[1]);
        pa[2 * j + 1] = pack_bf16x2(e[2], e[3]);
      }
      // ---- O += P V of tile i
      cp_async_wait<2>();
      __syncwarp();
      const uint32_t vs = ring + ((2 * i + 1) % kSlots) * kSlotBytes;
#pragma unroll
      for (int jj = 0; jj < 16; ++jj) {
        uint32_t vb[4];
        ldmatrix_x4_trans(vs + at((mi & 1) * 8 + ml, 2 * jj + (mi >> 1)), vb);
        mma_m16n8k16(o[2 * jj], pa, vb[0], vb[1]);
        mma_m16n8k16(o[2 * jj + 1], pa, vb[2], vb[3]);
      }
      __syncwarp();
      load(2 * i + 4);                                    // K of tile i + 2 over V of tile i
    }
    // ---- join the warps
    cp_async_wait_all();
    __syncwarp();
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        m_s[warp * kRows + 8 * r + (lane >> 2)] = m[r];
        l_s[warp * kRows + 8 * r + (lane >> 2)] = l[r];
      }
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float* dst = o_s + (lane >> 2) * kOLd + 8 * j + 2 * (lane & 3);
      *reinterpret_cast<float2*>(dst) = make_float2(o[j][0], o[j][1]);
      *reinterpret_cast<float2*>(dst + 8 * kOLd) = make_float2(o[j][2], o[j][3]);
    }
    __syncthreads();
    decode_join(t, a.kv, x, p, head0, smem, m_s, l_s, a.o, a.lse, a.part);
    __syncthreads();                                      // shared memory free for the next piece
  }
  dense_wait_last(a.late);
}

// ------------------------------------------------------------------ fp32
// The same for fp32, on CUDA cores: 12 heads make 6 products per byte, half of
// what the FMA pipe does at HBM rate.  A warp takes 16 keys of a chunk four at a
// time through six 4 KiB slots (K, V, K, V, ...); a lane holds 8 dims of the four
// rows and of every head's O, reads each head's q from shared memory (two reads
// for 32 products), and the 4 x HP sums over the lanes are reduced together, halving
// their number with each exchange.  Lane h then does head h's softmax.  HP: heads,
// rounded up to 4.  Bound by the instructions per key, not HBM, from 12 heads on: 16
// sequences of 8000 keys take 110 us with 24 heads in two groups (0.74 of the HBM
// rate) and 142 us with 32 (0.57), 8 of 2000 keys 25 us; 8 heads in 8 groups read at
// the HBM rate.
namespace dense_decode {
constexpr int kStep = 4;                              // keys
constexpr int kF32Slots = 6, kF32SlotBytes = kStep * kHeadDim * 4;
static_assert(kF32Slots * kF32SlotBytes == kSlots * kSlotBytes, "a warp's slots as in the bf16 kernel");
constexpr int kOffQ32 = kWarps * kSlots * kSlotBytes;
constexpr int kOffStat32 = kOffQ32 + kRows * kHeadDim * 4;
constexpr int kOffP32 = kOffStat32 + 2 * kWarps * kRows * 4;         // per warp: scores or P [16][4], factors [16]
constexpr int kSmemBytes32 = kOffP32 + kWarps * (kRows * kStep + kRows) * 4;
}  // namespace dense_decode

struct DenseDecodeF32Args {
  KvSource kv;
  const float* q;           // [T][H][D]
  float* o;
  float* lse;               // [T][H] or null
  float* part;
  int H;
  float scale;
  bool late;                // dense_wait_first
};

// Sums of v[0 .. N-1] over the warp's lanes, the number of values halved at each of
// the first exchanges (MASK = 16, 8, ..) while it is even; `base` ends as the index
// of the first sum that the lane is left with.
template <int N, int MASK>
__device__ __forceinline__ void reduce_halving(float* v, int& base) {
  if constexpr (MASK >= 1) {
    const bool up = threadIdx.x & MASK;
    if constexpr (N % 2 == 0) {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float keep = up ? v[i + N / 2] : v[i], send = up ? v[i] : v[i + N / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, MASK);
      }
      base += up ? N / 2 : 0;
      reduce_halving<N / 2, MASK / 2>(v, base);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], MASK);
      reduce_halving<N, MASK / 2>(v, base);
    }
  }
}
constexpr int reduce_left(int n, int mask) {
  return mask < 1 ? n : n % 2 == 0 ? reduce_left(n / 2, mask / 2) : reduce_left(n, mask / 2);
}

template <int HP>
__global__ void __launch_bounds__(dense_decode::kThreads, 1)
    dense_decode_f32_kernel(const __grid_constant__ DenseTable t, const __grid_constant__ DenseDecodeF32Args a) {
  using namespace dense_decode;
  using namespace sm100;
  constexpr int kHeads = HP == 16 ? 8 : HP;             // whose scores are formed together: 16 would spill
  extern __shared__ __align__(1024) unsigned char smem_1k[];
  unsigned char* const smem = smem_1k;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* const ring = smem + warp * kF32Slots * kF32SlotBytes;
  float* const q_s = reinterpret_cast<float*>(smem + kOffQ32);
  float* const m_s = reinterpret_cast<float*>(smem + kOffStat32);
  float* const l_s = m_s + kWarps * kRows;
  float* const p_s = reinterpret_cast<float*>(smem + kOffP32) + warp * (kRows * kStep + kRows);
  float* const f_s = p_s + kRows * kStep;
  const float tau2 = a.scale * 1.4426950408889634f;
  dense_wait_first(a.late);
  DenseWalk walk;
  walk.init(t, blockIdx.x);
  DensePiece p;
  DenseUnit x;
  while (walk.next(t, p, x)) {
    auto head0 = [&]() { return (int64_t)t.q_offset[x.si] * a.H + x.grp * t.hpg; };
    for (int i = threadIdx.x; i < kRows * (kHeadDim / 4); i += kThreads) {     // rows beyond the heads zero
      const bool in = i / (kHeadDim / 4) < x.nrows;
      cp_async16(smem_u32(q_s) + i * 16, a.q + head0() * kHeadDim + (in ? i * 4 : 0), in ? 16u : 0u);
    }
    // this warp's keys: 16 of each chunk, in steps of 4 (step j: chunk j / 4)
    const int32_t key0 = p.c0 * kKeys + warp * kTile;
    const int nc = min(p.c1 - p.c0, max(0, (x.kv_len - key0 + kKeys - 1) / kKeys)), n = nc * (kTile / kStep);
    int32_t look0 = -32;
    int32_t my_row = -1;                                  // cache rows fit 32 bits (they are TMA coordinates elsewhere)
    auto chunk_row = [&](int c) -> int32_t {              // first cache row of this warp's 16 keys of chunk c
      if (c - look0 >= 32) {
        look0 = c;
        const int32_t key = key0 + (c + lane) * kKeys;
        my_row = -1;
        if (c + lane < nc) {
          const int32_t pi = key / a.kv.page_tokens;
          const int32_t page = a.kv.table[(int64_t)t.slot[x.si] * a.kv.max_pages + pi];
          if (page >= 0 && page < a.kv.n_pages)
            my_row = (page * t.G + x.grp) * a.kv.page_tokens + (key - pi * a.kv.page_tokens);
          else
            report_error(kErrBadIndex);
        }
      }
      return __shfl_sync(0xffffffffu, my_row, c - look0);
    };
    auto load = [&](int j) -> uint32_t {                  // K and V of step j, one group each; 1: no page
      int32_t row = -1;
      int valid = 0;
      if (j < n) {
        row = chunk_row(j / (kTile / kStep));
        valid = row < 0 ? 0 : max(0, min(kStep, x.kv_len - (key0 + j / (kTile / kStep) * kKeys + j % (kTile / kStep) * kStep)));
        if (valid > 0) row += j % (kTile / kStep) * kStep;
      }
#pragma unroll
      for (int is_v = 0; is_v < 2; ++is_v) {
        if (j < n) {
          const int64_t at = (int64_t)(valid > 0 ? row : 0) * kHeadDim + lane * 4;
          const float* src = (const float*)(is_v ? a.kv.v : a.kv.k) + at;
          const uint32_t dst = smem_u32(ring + (2 * j + is_v) % kF32Slots * kF32SlotBytes) + lane * 16;
#pragma unroll
          for (int r = 0; r < kStep; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              cp_async16(dst + r * (kHeadDim * 4) + h * 512, r < valid ? src + r * kHeadDim + h * 128 : src,
                         r < valid ? 16u : 0u);
        }
        cp_async_commit();
      }
      return row < 0 ? 1u : 0u;
    };
    float2 o[HP][4];                                      // dims 4 lane .. +3 and 128 + 4 lane .. +3
#pragma unroll
    for (int h = 0; h < HP; ++h)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[h][k] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;                         // of head `lane`
    uint32_t bad_ahead = 0;                               // bit per step in flight, the oldest in bit 0
#pragma unroll
    for (int j = 0; j < 3; ++j) bad_ahead |= load(j) << j;
    cp_async_wait<5>();
    __syncthreads();                                      // q written
    for (int j = 0; j < n; ++j) {
      const bool bad = bad_ahead & 1;
      // ---- scores
      cp_async_wait<5>();
      __syncwarp();
      {
        const float4* ks = reinterpret_cast<const float4*>(ring + (2 * j) % kF32Slots * kF32SlotBytes) + lane;
        float4 k0[kStep], k1[kStep];
#pragma unroll
        for (int r = 0; r < kStep; ++r) {
          k0[r] = ks[r * 64];
          k1[r] = ks[r * 64 + 32];
        }
#pragma unroll
        for (int h0 = 0; h0 < HP; h0 += kHeads) {
          float dots[kHeads * kStep];
#pragma unroll
          for (int h = 0; h < kHeads; ++h) {
            const float4 q0 = reinterpret_cast<const float4*>(q_s + (h0 + h) * kHeadDim)[lane];
            const float4 q1 = reinterpret_cast<const float4*>(q_s + (h0 + h) * kHeadDim)[lane + 32];
#pragma unroll
            for (int r = 0; r < kStep; ++r) {
              float2 s = fma2(lo2(q0), lo2(k0[r]), make_float2(0.f, 0.f));
              s = fma2(hi2(q0), hi2(k0[r]), s);
              s = fma2(lo2(q1), lo2(k1[r]), s);
              s = fma2(hi2(q1), hi2(k1[r]), s);
              dots[h * kStep + r] = s.x + s.y;
            }
          }
          int base = h0 * kStep;
          reduce_halving<kHeads * kStep, 16>(dots, base);
#pragma unroll
          for (int i = 0; i < reduce_left(kHeads * kStep, 16); ++i) p_s[base + i] = dots[i];
        }
      }
      __syncwarp();
      // ---- softmax of head `lane`
      bool need = false;
      if (lane < HP) {
        const int left = bad ? 0 : x.kv_len - (key0 + j / (kTile / kStep) * kKeys + j % (kTile / kStep) * kStep);
        float4 s4 = reinterpret_cast<const float4*>(p_s)[lane];
        float s[kStep] = {s4.x, s4.y, s4.z, s4.w}, mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < kStep; ++r) {
          s[r] = r < left ? s[r] * tau2 : -INFINITY;
          mx = fmaxf(mx, s[r]);
        }
        float f = 1.f;
        if (mx > m + 8.f) {                               // false while both are -inf
          if (m != -INFINITY) {
            f = exp2f(m - mx);
            need = true;
          }
          m = mx;
        }
        f_s[lane] = f;
        l *= f;
        const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int r = 0; r < kStep; ++r) {
          s[r] = exp2f(s[r] - mb);
          l += s[r];
        }
        reinterpret_cast<float4*>(p_s)[lane] = make_float4(s[0], s[1], s[2], s[3]);
      }
      __syncwarp();
      if (__any_sync(0xffffffffu, need)) {
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float f = f_s[h];
#pragma unroll
          for (int k = 0; k < 4; ++k) o[h][k] = make_float2(o[h][k].x * f, o[h][k].y * f);
        }
      }
      // ---- O += P V
      cp_async_wait<4>();
      __syncwarp();
      {
        const float4* vs = reinterpret_cast<const float4*>(ring + (2 * j + 1) % kF32Slots * kF32SlotBytes) + lane;
        float4 v0[kStep], v1[kStep];
#pragma unroll
        for (int r = 0; r < kStep; ++r) {
          v0[r] = vs[r * 64];
          v1[r] = vs[r * 64 + 32];
        }
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float4 p4 = reinterpret_cast<const float4*>(p_s)[h];
          const float pr[kStep] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int r = 0; r < kStep; ++r) {
            const float2 f = make_float2(pr[r], pr[r]);
            o[h][0] = fma2(f, lo2(v0[r]), o[h][0]);
            o[h][1] = fma2(f, hi2(v0[r]), o[h][1]);
            o[h][2] = fma2(f, lo2(v1[r]), o[h][2]);
            o[h][3] = fma2(f, hi2(v1[r]), o[h][3]);
          }
        }
      }
      __syncwarp();                                       // the step's slots and P are read
      bad_ahead = bad_ahead >> 1 | load(j + 3) << 2;
    }
    // ---- join the warps
    cp_async_wait_all();
    __syncwarp();
    if (lane < kRows) {
      m_s[warp * kRows + lane] = lane < HP ? m : -INFINITY;
      l_s[warp * kRows + lane] = lane < HP ? l : 0.f;
    }
    float* const o_s = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      reinterpret_cast<float4*>(o_s + h * kOLd)[lane] = make_float4(o[h][0].x, o[h][0].y, o[h][1].x, o[h][1].y);
      reinterpret_cast<float4*>(o_s + h * kOLd)[lane + 32] = make_float4(o[h][2].x, o[h][2].y, o[h][3].x, o[h][3].y);
    }
    __syncthreads();
    decode_join(t, a.kv, x, p, head0(), smem, m_s, l_s, a.o, a.lse, a.part);
    __syncthreads();                                      // shared memory free for the next piece
  }
  dense_wait_last(a.late);
}

}  // namespace qsa
