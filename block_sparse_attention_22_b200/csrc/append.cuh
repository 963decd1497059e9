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
constexpr int kWarps = kThreads / 32;
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

// WPT warps take a token (one, or the block's eight when there are too few
// tokens to fill the GPU).  A token's G keys, H queries (when given) and G values
// are vectors of 256 dims; the rotated dims are a part of the first 16-byte pieces
// of each.  The kernel is a copy, bound by HBM as long as it stays short of
// instructions: pieces that are only copied go lane by lane down the vectors, and
// the rotated ones are taken pairwise, a lane holding eight dims and their eight
// partners, so no lane converts what it does not rotate.  A warp forms its own
// token's sines and cosines while its first loads are in flight.  (With a vector
// per warp and step, partners by shuffle, and the pointers formed per vector, a
// 4096-token chunk of 24 + 2 + 2 heads took 44 us, bound by instruction issue.)
template <typename T, int WPT>
__global__ void __launch_bounds__(append::kThreads)
    append_kernel(Geo g, const __grid_constant__ SegTable st, const __grid_constant__ AppendArgs a) {
  using namespace append;
  __shared__ float cs_s[kWarps][kMaxHalf], sn_s[kWarps][kMaxHalf];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPT;
  const int item = (int)blockIdx.x * (kWarps / WPT) + warp / WPT;
  float* const cs = cs_s[warp];
  float* const sn = sn_s[warp];
  pdl_wait();
  pdl_trigger();
  if (item >= st.item0[st.n]) return;
  const int si = find_segment(st, item);
  const int j = item - st.item0[si];
  const int64_t tok = (int64_t)st.q_offset[si] + j;
  const int32_t pos = st.pos0[si] + j, pi = pos / a.page_tokens;
  const int32_t page = a.table[(int64_t)st.slot[si] * a.max_pages + pi];
  const bool stored = page >= 0 && page < a.n_pages;
  if (!stored && lane == 0 && sub == 0) report_error(kErrBadIndex);
  const T* const k = (const T*)a.k + tok * a.ld_k;
  const T* const v = (const T*)a.v + tok * a.ld_v;
  const T* const q = (const T*)a.q + tok * a.ld_q;
  T* const qo = (T*)a.q_out + tok * g.H * kHeadDim;
  const int64_t at = stored ? ((int64_t)page * g.G * a.page_tokens + (pos - pi * a.page_tokens)) * kHeadDim : 0;
  T* const kp = (T*)a.kp + at;
  T* const vp = (T*)a.vp + at;
  const int64_t ld_p = (int64_t)a.page_tokens * kHeadDim;      // between a page's groups
  const int half = a.half, nq = a.q ? g.H : 0, n_rot = g.G + nq;
  // vector w: keys, then queries, then values (which are not rotated)
  auto from = [&](int w) { return w < g.G ? k + w * kHeadDim : w < n_rot ? q + (w - g.G) * kHeadDim : v + (w - n_rot) * kHeadDim; };
  auto to = [&](int w) { return w < g.G ? kp + w * ld_p : w < n_rot ? qo + (w - g.G) * kHeadDim : vp + (w - n_rot) * ld_p; };
  auto wanted = [&](int w) { return stored || (w >= g.G && w < n_rot); };
  // values, and the pieces of the rotated vectors behind the rotation; kUnroll
  // loads before the first store, which may alias them (q in place)
  constexpr int kUnroll = sizeof(T) == 2 ? 6 : 4;
  const int mixed = (2 * half + 7) >> 3;                        // pieces with rotated dims
  auto form_angles = [&]() {
    for (int p = lane; p < half; p += 32) {
      double s, c;
      sincos((double)pos * a.theta[p], &s, &c);
      cs[p] = (float)c;
      sn[p] = (float)s;
    }
  };
  bool angles = false;
  for (int w0 = sub; w0 < n_rot + g.G; w0 += kUnroll * WPT) {
    Vec8<T> x[kUnroll];
    auto mine = [&](int w) { return w < n_rot + g.G && (w >= n_rot || lane >= mixed) && wanted(w); };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (mine(w0 + u * WPT)) x[u].load(from(w0 + u * WPT) + lane * 8);
    if (!angles) form_angles();
    angles = true;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (mine(w0 + u * WPT)) x[u].store(to(w0 + u * WPT) + lane * 8);
  }
  if (!angles) form_angles();                                   // a warp without vectors may have rotations
  __syncwarp();
  if ((half & 7) == 0) {
    const int per = half >> 3, tasks = n_rot * per;             // lane tasks of a vector, of the token
    constexpr int kPairs = 2;
    for (int i0 = sub * 32 + lane; i0 < tasks; i0 += kPairs * WPT * 32) {
      Vec8<T> x[kPairs], y[kPairs];
      int w[kPairs], d[kPairs];
#pragma unroll
      for (int u = 0; u < kPairs; ++u) {
        const int i = i0 + u * WPT * 32;
        w[u] = i / per;
        d[u] = (i - w[u] * per) * 8;
        if (i >= tasks || !wanted(w[u])) w[u] = -1;
        if (w[u] >= 0) {
          x[u].load(from(w[u]) + d[u]);
          y[u].load(from(w[u]) + half + d[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kPairs; ++u) {
        if (w[u] < 0) continue;
        float fx[8], fy[8];
        x[u].get(fx);
        y[u].get(fy);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float oa, ob;
          rope_pair(fx[e], fy[e], cs[d[u] + e], sn[d[u] + e], oa, ob);
          fx[e] = oa;
          fy[e] = ob;
        }
        x[u].set(fx);
        y[u].set(fy);
        x[u].store(to(w[u]) + d[u]);
        y[u].store(to(w[u]) + half + d[u]);
      }
    }
  } else {                                                      // pairs, then the dims that share their pieces
    const int rest = mixed * 8 - 2 * half, per = half + rest;
    for (int i = sub * 32 + lane; i < n_rot * per; i += WPT * 32) {
      const int w = i / per, d = i - w * per;
      if (!wanted(w)) continue;
      if (d < half) {
        float oa, ob;
        rope_pair(IO<T>::to_f(from(w)[d]), IO<T>::to_f(from(w)[half + d]), cs[d], sn[d], oa, ob);
        to(w)[d] = IO<T>::from_f(oa);
        to(w)[half + d] = IO<T>::from_f(ob);
      } else {
        to(w)[half + d] = from(w)[half + d];
      }
    }
  }
}

}  // namespace qsa
