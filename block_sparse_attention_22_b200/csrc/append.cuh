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
constexpr int kTokens = 8;                  // tokens of a block, when there are enough for every SM
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

// A block takes TPB tokens.  A token's G keys, H queries (when given) and G
// values are vectors of 256 dims, one warp each, 8 dims per lane.  The kernel
// is a copy, bound by HBM; what it waits for is the fp64 sine and cosine, so with
// eight tokens at 32 rotated pairs every thread forms one of them while the
// warps' first loads are in flight.  (One token per block left seven of eight warps
// idle meanwhile: 44 us for a 4096-token chunk of 24 + 2 + 2 heads, 117 MB.)  Few
// tokens take a block each, for the latency.  A pair's halves are `half` / 8 lanes
// apart; where that is no whole number they meet in shared memory.
template <typename T, int TPB>
__global__ void __launch_bounds__(append::kThreads)
    append_kernel(Geo g, const __grid_constant__ SegTable st, const __grid_constant__ AppendArgs a) {
  using namespace append;
  constexpr int kWarps = kThreads / 32;
  __shared__ float cs[TPB][kMaxHalf], sn[TPB][kMaxHalf];
  __shared__ float row[kWarps][kHeadDim];
  __shared__ int64_t tok_s[TPB], pos_s[TPB], cache_s[TPB];      // cache row of group 0; -1: not stored
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = (int)blockIdx.x * TPB, ntok = min(TPB, st.item0[st.n] - first);
  pdl_wait();
  pdl_trigger();
  if (threadIdx.x < ntok) {
    const int item = first + (int)threadIdx.x;
    const int si = find_segment(st, item);
    const int j = item - st.item0[si];
    const int32_t pos = st.pos0[si] + j, pi = pos / a.page_tokens;
    const int32_t page = a.table[(int64_t)st.slot[si] * a.max_pages + pi];
    const bool ok = page >= 0 && page < a.n_pages;
    if (!ok) report_error(kErrBadIndex);
    tok_s[threadIdx.x] = (int64_t)st.q_offset[si] + j;
    pos_s[threadIdx.x] = pos;
    cache_s[threadIdx.x] = ok ? (int64_t)page * g.G * a.page_tokens + (pos - pi * a.page_tokens) : -1;
  }
  __syncthreads();
  const int nq = a.q ? g.H : 0;
  const int n_rot = g.G + nq, n_vec = n_rot + g.G, total = ntok * n_vec;
  auto src = [&](int i, int v) -> const T* {
    const int64_t tok = tok_s[i];
    if (v < g.G) return (const T*)a.k + tok * a.ld_k + (int64_t)v * kHeadDim;
    if (v < n_rot) return (const T*)a.q + tok * a.ld_q + (int64_t)(v - g.G) * kHeadDim;
    return (const T*)a.v + tok * a.ld_v + (int64_t)(v - n_rot) * kHeadDim;
  };
  auto dst = [&](int i, int v) -> T* {   // null: not stored
    if (v >= g.G && v < n_rot) return (T*)a.q_out + (tok_s[i] * g.H + (v - g.G)) * kHeadDim;
    if (cache_s[i] < 0) return nullptr;
    const bool is_k = v < g.G;
    const int64_t r = cache_s[i] + (int64_t)(is_k ? v : v - n_rot) * a.page_tokens;
    return (T*)(is_k ? a.kp : a.vp) + r * kHeadDim;
  };
  const bool by_lane = (a.half & 7) == 0;
  const int apart = a.half >> 3;         // lanes between a pair's halves
  bool angles = false;
  for (int w0 = warp; w0 < total || !angles; w0 += kWarps * kUnroll) {
    Vec8<T> x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int w = w0 + u * kWarps, i = w / n_vec;
      if (w < total) x[u].load(src(i, w - i * n_vec) + lane * 8);
    }
    if (!angles) {
      for (int k = threadIdx.x; k < ntok * a.half; k += kThreads) {
        const int i = k / a.half, p = k - i * a.half;
        double s, c;
        sincos((double)pos_s[i] * a.theta[p], &s, &c);
        cs[i][p] = (float)c;
        sn[i][p] = (float)s;
      }
      __syncthreads();
      angles = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int w = w0 + u * kWarps;
      if (w >= total) break;
      const int i = w / n_vec, v = w - i * n_vec;
      T* out = dst(i, v);
      if (v < n_rot) {
        float f[8], y[8];                // this lane's dims and their partners
        x[u].get(f);
        if (by_lane) {
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = __shfl_sync(0xffffffffu, f[k], lane < apart ? lane + apart : lane - apart);
        } else {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) row[warp][lane * 8 + k] = f[k];
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int d = lane * 8 + k;
            y[k] = d < a.half ? row[warp][d + a.half] : d < 2 * a.half ? row[warp][d - a.half] : 0.f;
          }
        }
        if (lane * 8 < 2 * a.half) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int d = lane * 8 + k;
            float oa, ob;
            if (d < a.half) {
              rope_pair(f[k], y[k], cs[i][d], sn[i][d], oa, ob);
              f[k] = oa;
            } else if (d < 2 * a.half) {
              rope_pair(y[k], f[k], cs[i][d - a.half], sn[i][d - a.half], oa, ob);
              f[k] = ob;
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
