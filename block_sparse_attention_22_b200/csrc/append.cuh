// append.cuh -- new tokens' keys and values into a paged K/V cache, keys (and
// queries) rotated to their positions on the way.
//
// Miles docs "Qwen3.8-Flash-Next", section 1: rotary base 1e7 at rotary
// percent 0.25 of the 256 head dims.  For a token at position t and a rotated
// pair (i, i + half): (a, b) -> (a cos - b sin, b cos + a sin) at the angle
// t * theta_i, formed in fp64 (positions reach 2^20), cos and sin rounded to
// fp32, products in fp32, one rounding to the I/O dtype; the other dims and V
// are copied.
#pragma once
#include "qsa_internal.cuh"

namespace qsa {
namespace append {
constexpr int kThreads = 256;
constexpr int kMaxHalf = kHeadDim / 2;      // rotated pairs at rope_fraction 1
constexpr int kUnroll = 4;                  // vectors a warp loads before it stores the first
}  // namespace append

struct AppendArgs {
  const void* k;            // row (i, g) at k + i*ld_k + g*D elements
  const void* v;
  const void* q;            // or null
  int64_t ld_k, ld_v, ld_q;
  void* q_out;              // [T][H][D]
  void* kp;                 // [n_pages][G][page_tokens][D]
  void* vp;
  const int32_t* table;     // [n_rows][max_pages]
  int32_t n_pages, page_tokens, max_pages;
  int32_t half;             // rotated pairs
  double theta[append::kMaxHalf];
};

// Eight consecutive elements of a lane.
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
  uint4 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = x; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  }
};
template <> struct Vec8<float> {
  float4 x, y;
  __device__ __forceinline__ void load(const float* p) {
    x = reinterpret_cast<const float4*>(p)[0];
    y = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = x;
    reinterpret_cast<float4*>(p)[1] = y;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    x = make_float4(f[0], f[1], f[2], f[3]);
    y = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// One block per token.  A token's G keys, H queries (when given) and G values
// are vectors of 256 dims, one warp each, 8 dims per lane; warp w takes
// vectors w, w + 8, ...  The first loads are in flight while the block's first
// `half` threads form the token's cosines and sines.
template <typename T>
__global__ void __launch_bounds__(append::kThreads)
    append_kernel(Geo g, SegTable st, AppendArgs a) {
  using namespace append;
  __shared__ float cs[kMaxHalf], sn[kMaxHalf];
  __shared__ float row[kThreads / 32][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kThreads / 32;
  const int si = find_segment(st, (int)blockIdx.x);
  const int j = (int)blockIdx.x - st.item0[si];
  const int64_t tok = (int64_t)st.q_offset[si] + j;
  const int64_t pos = (int64_t)st.pos0[si] + j;
  pdl_wait();
  pdl_trigger();
  const int nq = a.q ? g.H : 0;
  const int n_rot = g.G + nq, n_vec = n_rot + g.G;
  const int32_t page = a.table[(int64_t)st.slot[si] * a.max_pages + pos / a.page_tokens];
  const bool stored = page >= 0 && page < a.n_pages;
  if (!stored && threadIdx.x == 0) report_error(kErrBadIndex);
  const int64_t cache_row = (int64_t)page * g.G * a.page_tokens + pos % a.page_tokens;   // of group 0
  auto src = [&](int v) -> const T* {
    if (v < g.G) return (const T*)a.k + tok * a.ld_k + (int64_t)v * kHeadDim;
    if (v < n_rot) return (const T*)a.q + tok * a.ld_q + (int64_t)(v - g.G) * kHeadDim;
    return (const T*)a.v + tok * a.ld_v + (int64_t)(v - n_rot) * kHeadDim;
  };
  auto dst = [&](int v) -> T* {          // null: not stored
    if (v >= g.G && v < n_rot) return (T*)a.q_out + (tok * g.H + (v - g.G)) * kHeadDim;
    if (!stored) return nullptr;
    const bool is_k = v < g.G;
    const int64_t r = cache_row + (int64_t)(is_k ? v : v - n_rot) * a.page_tokens;
    return (T*)(is_k ? a.kp : a.vp) + r * kHeadDim;
  };
  bool angles = false;
  for (int v0 = warp; v0 < n_vec || !angles; v0 += kWarps * kUnroll) {
    Vec8<T> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (v0 + u * kWarps < n_vec) x[u].load(src(v0 + u * kWarps) + lane * 8);
    if (!angles) {
      if (threadIdx.x < a.half) {
        double s, c;
        sincos((double)pos * a.theta[threadIdx.x], &s, &c);
        cs[threadIdx.x] = (float)c;
        sn[threadIdx.x] = (float)s;
      }
      __syncthreads();
      angles = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int v = v0 + u * kWarps;
      if (v >= n_vec) break;
      T* out = dst(v);
      if (v < n_rot) {                   // rotate: a pair's halves may sit in different lanes
        float f[8];
        x[u].get(f);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) row[warp][lane * 8 + i] = f[i];
        __syncwarp();
        if (lane * 8 < 2 * a.half) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = lane * 8 + i;
            float oa, ob;
            if (d < a.half) {
              rope_pair(f[i], row[warp][d + a.half], cs[d], sn[d], oa, ob);
              f[i] = oa;
            } else if (d < 2 * a.half) {
              rope_pair(row[warp][d - a.half], f[i], cs[d - a.half], sn[d - a.half], oa, ob);
              f[i] = ob;
            }
          }
          x[u].set(f);
        }
      }
      if (out) x[u].store(out + lane * 8);
    }
  }
}

}  // namespace qsa
