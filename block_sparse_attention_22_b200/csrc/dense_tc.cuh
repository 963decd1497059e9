// dense_tc.cuh -- dense causal GQA attention, bf16, on tcgen05 tensor cores:
// forward over a paged cache and over packed prompts.
//
// A unit (dense.cuh) is a tile of query rows of one KV group -- row = token *
// hpg + head, so the heads of a group share every key and value that is
// loaded -- against keys 0 .. the last token's position, in chunks:
//   S[row, key] = Q[row, :] . K[key, :]        (K = 256 dims)
//   O[row, :]  += P[row, key] V[key, :]        (N = 256 dims)
// with one pass over the keys: a row's reference maximum moves only when a
// chunk's maximum exceeds it by more than 8 (log2 units), then O and the row's
// sum so far are rescaled in tensor memory; P stays below 2^8 in between.  P
// is rounded to bf16 for its product (relative error 2^-8 of each weight, as
// in the sparse kernels); the row sum adds the unrounded values in fp32.
//
// Two forms (CG = CTAs per unit):
//   CG = 1  128 rows, chunks of 64 keys, one CTA: segments of 2 to 128 rows
//           (a few tokens each; prompts of one), where no longer ones are in the
//           call.  Single tokens over a cache have kernels of their own
//           (dense_decode.cuh).
//   CG = 2  256 rows, chunks of 128 keys, a CTA pair (cta_group::2): each CTA
//           owns 128 rows, loads half of K's keys and half of V's dims, and
//           the pair's MMAs read both halves, so a key crosses L2 once per
//           256 rows.  A lone CTA would need 64 bytes per cycle and SM at full
//           tensor rate (17 TB/s over the GPU), a pair needs half.
//
// Per CTA 12 warps: eight softmax warps (two per TMEM lane quadrant, each
// thread one row and half of a chunk's keys and dims), one TMA producer that
// fills two 32 KiB slots each of K and V in the order the MMAs consume them
// (K0, K1, V0, K2, V1, ...), one warp that issues the MMAs (in rank 0), one
// that loads Q of the next unit and one that checks V of the unit's own tokens.
// K completes on rank 0's barrier, V on each CTA's own, where the softmax warps
// wait for it before they hand over P, so the MMA warp waits once per product and
// needs no fence.  That rank 1's V has landed is released to it by rank 1's own
// MMA warp, which issues nothing: the softmax warps release their P, which is in
// tensor memory, without holding up for a release at cluster scope (by them it
// cost 14 % of a long chunk's time), but for rows they zeroed.  A product is
// committed to one barrier, which its readers and its slot's producer share.
// TMEM: two S buffers (each half's P overwrites its own S columns), O in
// columns 256..511.
//
// Keys that do not count -- beyond the sequence, on a page out of range, after
// a row's position -- may hold anything: their scores are replaced by -inf;
// V rows beyond the sequence and of bad pages are zeroed in shared memory
// before the product (0 * NaN would spread).  Values of the tile's own tokens
// (visible to some rows only) are checked for infinities and NaN while Q is
// loaded; such a key's V row is zeroed too and its contribution added in the
// epilogue to the rows that attend it.
// Every mbarrier wait is bounded; a timeout records an error and the CTA
// drains and returns.
//
// Measured (24 heads, 2 groups): a 4096-token chunk over 128K keys 10.0 ms, 1.30
// PFLOP/s, 0.94 of sustained cuBLAS under the same power cap; two prompts of 8192
// 1.30 ms, where the softmax (2400 cycles a chunk, its exponentials 1024 on
// MUFU) outlasts the products' 2048 and a unit's change costs 5 us.
#pragma once
#include "qsa_internal.cuh"
#include "sm100.cuh"
#include "attn_tc.cuh"
#include "attn_union_tc.cuh"
#include "dense.cuh"
#include "dense_simt.cuh"

namespace qsa {
namespace dense_tc {
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kSoftmaxWarps = 8;
constexpr int kProducerWarp = 8, kMmaWarp = 9, kQWarp = 10, kNfWarp = 11;
constexpr int kSlots = 4, kKSlots = 2, kVSlots = 2;   // K's as many as S buffers, V's as P: they share barriers
constexpr int kSlotBytes = 32768;
constexpr int kQBytes = 65536;                        // 128 rows x 256 dims, 4 slabs of 16 KiB
constexpr int kOffV = kKSlots * kSlotBytes;
constexpr int kOffQ = kSlots * kSlotBytes;            // 131072
constexpr int kOffCtl = kOffQ + kQBytes;              // 196608
constexpr int kCtlBytes = 3 * 1024;
constexpr int kSmemBytes = kOffCtl + kCtlBytes;       // 199680: the base itself is 1024-byte aligned
constexpr uint32_t kTmemCols = 512, kTmemO = 256;
constexpr int kNfBufs = 4;                            // units whose non-finite lists may be in use at once, or made ahead
template <int CG> struct Shape {
  static constexpr int kRows = 128 * CG;
  static constexpr int kKeys = 64 * CG;
  static constexpr int kGrid = 148 / CG;
  static constexpr uint32_t kIdescS = sm100::idesc_bf16(128 * CG, kKeys, false, false);
  static constexpr uint32_t kIdescPV = sm100::idesc_bf16(128 * CG, 256, false, true);
};
}  // namespace dense_tc

struct DenseTcArgs {
  KvSource kv;
  const __nv_bfloat16* q;   // [T][H][D]
  __nv_bfloat16* o;
  float* lse;               // [T][H] or null
  float* part;
  int H;
  int box;                  // rows of a TMA box: keys that are contiguous in the cache
  float scale;
  bool late;                // dense_wait_first
};

struct DenseTcCtl {
  uint64_t k_full[dense_tc::kKSlots];     // rank 0's: both CTAs' halves
  uint64_t v_full[dense_tc::kVSlots];     // this CTA's half
  uint64_t q_full, q_empty;
  uint64_t s_done[2], p_full[2], pv_done[2];          // by chunk parity
  uint64_t o_full, o_free;
  uint64_t nf_full[dense_tc::kNfBufs], nf_free[dense_tc::kNfBufs];
  uint64_t mma_done;
  float red[2][2][128];                   // by chunk parity: row maxima / sums of the two warps of a row
  uint32_t nf[dense_tc::kNfBufs][8];   // keys first_pos+1+i whose V is not finite
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(DenseTcCtl) <= dense_tc::kCtlBytes, "control block");

// Largest power of two that divides page_tokens, at most 64: a run of that
// many keys, starting at a multiple of it, lies in one page.
inline int dense_box(int page_tokens) {
  int b = 16;
  while (b < 64 && page_tokens % (2 * b) == 0) b *= 2;
  return b;
}

// Loads rows row0 .. row0+n-1 (n <= 128) of a unit's segment and group into a
// 128-byte swizzled tile, completing n * 512 bytes on rank 0's barrier: a token's
// heads are consecutive rows of the token-major array, so a whole token is one
// box per 64 dims; tokens cut by the tile's ends come in boxes of as many rows as
// divide both 128 and the group's heads.  By TMA, since the tensor cores' operand reads leave other shared-memory
// writes little room: cp.async took 25 us for 128 KiB under them.  (The swizzle
// goes by address bits, so boxes may start at any 128-byte line.)
template <int CG>
__device__ __forceinline__ void load_q_rows(unsigned char* tile, const CUtensorMap* tokens, const CUtensorMap* rows,
                                            const DenseTable& t, const DenseUnit& x, int32_t row0, int n, int H,
                                            int lane, uint64_t* bar) {
  const int32_t tok0 = row0 / t.hpg;
  const int h0 = row0 - tok0 * t.hpg;
  const int lead = h0 == 0 ? 0 : min(t.hpg - h0, n), whole = (n - lead) / t.hpg, tail = n - lead - whole * t.hpg;
  const int32_t y0 = (t.q_offset[x.si] + tok0) * H + x.grp * t.hpg;      // head 0 of the first row's token
  const int32_t y1 = h0 == 0 ? y0 : y0 + H;                              // of the first whole token
  const int slab = lane & 3;
#pragma unroll 1
  for (int k = lane >> 2; k < whole; k += 8)
    sm100::tma_load_2d_leader<CG>(tile + slab * 16384 + (lead + k * t.hpg) * 128, tokens, slab * 64, y1 + k * H, bar);
  const int step = t.hpg & -t.hpg;
#pragma unroll 1
  for (int e = (lane >> 2) * step; e < lead + tail; e += 8 * step) {
    const bool first = e < lead;
    const int r = first ? e : n - tail + (e - lead);
    sm100::tma_load_2d_leader<CG>(tile + slab * 16384 + r * 128, rows, slab * 64,
                                  first ? y0 + h0 + e : y1 + whole * H + (e - lead), bar);
  }
}

// Four lanes' 4 x 4 blocks of 16 bytes transposed: lane k of a quad then holds
// piece k of the four lanes' rows.
__device__ __forceinline__ void quad_transpose(uint4 (&v)[4], int lane) {
  auto swap = [&](uint4& lo, uint4& hi, int bit) {
    const bool up = lane & bit;
    uint4 s = up ? lo : hi;
    s.x = __shfl_xor_sync(0xffffffffu, s.x, bit);
    s.y = __shfl_xor_sync(0xffffffffu, s.y, bit);
    s.z = __shfl_xor_sync(0xffffffffu, s.z, bit);
    s.w = __shfl_xor_sync(0xffffffffu, s.w, bit);
    if (up) lo = s; else hi = s;
  };
  swap(v[0], v[1], 1);
  swap(v[2], v[3], 1);
  swap(v[0], v[2], 2);
  swap(v[1], v[3], 2);
}

// Stores 32 result columns (from `col` on) of the warp's 32 rows: out != null:
// times f, rounded, to the rows at[] (of this lane's quad, in heads; < 0: not
// stored); else as they are to the partial rows from `part` (the quad's first).
// Transposed first, so that a store instruction touches 8 rows, not 32: the
// epilogue's stores took 10 cycles per row and instruction under the MMAs.
__device__ __forceinline__ void store_cols32(const float (&o)[32], float f, __nv_bfloat16* out, float* part,
                                             const int64_t (&at)[4], int col, int lane) {
  uint4 v[4];
  if (out) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      v[c] = make_uint4(pack_bf16x2(o[8 * c] * f, o[8 * c + 1] * f), pack_bf16x2(o[8 * c + 2] * f, o[8 * c + 3] * f),
                        pack_bf16x2(o[8 * c + 4] * f, o[8 * c + 5] * f),
                        pack_bf16x2(o[8 * c + 6] * f, o[8 * c + 7] * f));
    quad_transpose(v, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (at[j] >= 0) *reinterpret_cast<uint4*>(out + at[j] * kHeadDim + col + 8 * (lane & 3)) = v[j];
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        v[c] = make_uint4(__float_as_uint(o[16 * h + 4 * c]), __float_as_uint(o[16 * h + 4 * c + 1]),
                          __float_as_uint(o[16 * h + 4 * c + 2]), __float_as_uint(o[16 * h + 4 * c + 3]));
      quad_transpose(v, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at[j] >= 0)
          *reinterpret_cast<uint4*>(part + j * dense::kPartFloats + col + 16 * h + 4 * (lane & 3)) = v[j];
    }
  }
}

// mbar_wait_fast by a whole warp, with one answer.
template <bool kPair = false>
__device__ __forceinline__ bool warp_wait_fast(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, sm100::mbar_wait_fast<kPair>(bar, parity, abort_flag));
}

// After an abort: copies in flight land within microseconds; the CTA stays for
// about a millisecond.
__device__ __forceinline__ void drain_copies() {
  const long long t0 = clock64();
  while (clock64() - t0 < 2000000) {
  }
}

template <int CG, bool PAGED>
__global__ void __launch_bounds__(dense_tc::kThreads, 1)
    dense_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_tok, const __grid_constant__ CUtensorMap tm_row,
                        const __grid_constant__ DenseTable t, const __grid_constant__ DenseTcArgs a) {
  using namespace dense_tc;
  using namespace sm100;
  constexpr int KC = Shape<CG>::kKeys, NK = KC / 2;          // keys of a chunk, of a softmax thread
  extern __shared__ __align__(1024) unsigned char smem_1k[];
  unsigned char* const smem = smem_1k;
  DenseTcCtl& ctl = *reinterpret_cast<DenseTcCtl*>(smem + kOffCtl);
  volatile int* abort_flag = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0;
  const int cta = blockIdx.x / CG;

  // ---------------------------------------------------------------- set-up
  // The swizzled tiles need the alignment that smem_1k asks for; the same in every CTA.
  // Without it there is no result, which is what a wait that gave up tells the host.
  if (smem_u32(smem) & 1023u) {
    report_error(kErrWaitTimeout);
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.k_full[i], CG);
      mbar_init(&ctl.v_full[i], 1);
      mbar_init(&ctl.s_done[i], 1);
      mbar_init(&ctl.p_full[i], CG == 1 ? kSoftmaxWarps : kSoftmaxWarps * 2 + 1);
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (int i = 0; i < kNfBufs; ++i) {
      mbar_init(&ctl.nf_full[i], 1);
      mbar_init(&ctl.nf_free[i], kSoftmaxWarps);
    }
    mbar_init(&ctl.q_full, CG);
    mbar_init(&ctl.q_empty, 1);
    mbar_init(&ctl.o_full, 1);
    mbar_init(&ctl.o_free, kSoftmaxWarps * CG);
    mbar_init(&ctl.mma_done, 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_cg<CG>(&ctl.tmem_base, kTmemCols);
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  dense_wait_first(a.late);

  DenseWalk walk;
  walk.init(t, cta);
  DensePiece p = {};
  DenseUnit x = {};
  if (warp == kProducerWarp) {
    // ============================================================ TMA producer
    // A slot is 256 / box boxes of `box` keys x 64 dims, one per lane.  A chunk's
    // cache rows are formed once, a run of `box` keys per lane, a chunk ahead of
    // their use: a product's time is 500 of this warp's instructions.
    constexpr int kSlabsV = CG == 2 ? 2 : 4;
    const int nbox = 256 / a.box, runs = KC / a.box;
    // this lane's box: K keys run_k.. of this CTA's 64, V all keys x this CTA's dims
    const int slab_k = lane & 3, run_k = (lane >> 2) + (CG == 2 ? (int)rank * 64 / a.box : 0);
    const int slab_v = lane % kSlabsV, run_v = lane / kSlabsV;
    const int off_k = slab_k * 8192 + (lane >> 2) * a.box * 128;
    const int off_v = slab_v * (256 / kSlabsV) * 128 + run_v * a.box * 128;
    const int x_v = slab_v * 64 + (CG == 2 ? (int)rank * 128 : 0);
    const bool has_box = lane < nbox;
    uint32_t gk = 0, gv = 0;                                 // chunks of K and V so far
    bool ok = true;
    // cache row of run `lane` of chunk c (of the piece); < 0: not loaded
    auto rows_of = [&](int c) -> int32_t {
      const int32_t key = (p.c0 + c) * KC + lane * a.box;
      if (lane >= runs || c >= p.c1 - p.c0 || key >= x.kv_len) return -1;
      if (!PAGED) return t.q_offset[x.si] + key;
      const int32_t pi = key / a.kv.page_tokens;
      const int32_t page = a.kv.table[(int64_t)t.slot[x.si] * a.kv.max_pages + pi];
      if (page < 0 || page >= a.kv.n_pages) {
        report_error(kErrBadIndex);
        return -1;
      }
      return (page * t.G + x.grp) * a.kv.page_tokens + (key - pi * a.kv.page_tokens);
    };
    auto put = [&](bool is_v, int32_t rows, int32_t x0) -> bool {
      uint32_t& g = is_v ? gv : gk;
      const uint32_t slot = g & 1, phase = (g >> 1) & 1;
      ++g;
      const int32_t y = __shfl_sync(0xffffffffu, rows, is_v ? run_v : run_k);
      const uint32_t live = __ballot_sync(0xffffffffu, has_box && y >= 0);
      const uint32_t bytes = (uint32_t)__popc(live) * (uint32_t)(a.box * 128);
      if (!warp_wait_fast(is_v ? &ctl.pv_done[slot] : &ctl.s_done[slot], phase ^ 1, abort_flag)) return false;
      if (is_v) {
        if (lane == 0) mbar_expect_tx(&ctl.v_full[slot], bytes);
        __syncwarp();
        if (has_box && y >= 0)
          tma_load_2d(smem + kOffV + slot * kSlotBytes + off_v, &tm_v, x0 + x_v, y, &ctl.v_full[slot]);
      } else {
        if (lane == 0) mbar_expect_tx_leader<CG>(&ctl.k_full[slot], bytes);
        __syncwarp();
        if (has_box && y >= 0)
          tma_load_2d_leader<CG>(smem + slot * kSlotBytes + off_k, &tm_k, x0 + slab_k * 64, y, &ctl.k_full[slot]);
      }
      return true;
    };
    while (ok && walk.next(t, p, x)) {
      const int n = p.c1 - p.c0;
      const int32_t x0 = PAGED ? 0 : x.grp * kHeadDim;
      int32_t cur = rows_of(0), next = rows_of(1);
      ok = put(false, cur, x0);
      for (int c = 0; c < n && ok; ++c) {
        const int32_t after = rows_of(c + 2);
        if (c + 1 < n) ok = put(false, next, x0);
        ok = ok && put(true, cur, x0);
        cur = next;
        next = after;
      }
    }
    if (!ok) drain_copies();                                 // no copy outlives the CTA
  } else if (warp == kMmaWarp && rank == 0) {
    // ============================================================ MMA issuer
    int64_t gc = 0, uc = 0;                                  // chunks and pieces so far
    const uint32_t sb = smem_u32(smem), leader = elect_one();
    // what both CTAs' threads arrive on
    auto wait = [&](uint64_t* bar, int64_t phase) {
      return mbar_wait_fast<CG == 2>(bar, (uint32_t)(phase & 1), abort_flag);
    };
    auto pv = [&](int cx, int n) -> bool {
      const int64_t xg = gc + cx;
      const int b = (int)(xg & 1);
      if (!wait(&ctl.p_full[b], xg >> 1)) return false;      // P, and both halves of V
      if (cx == 0 && !wait(&ctl.o_free, uc ^ 1)) return false;
      tc_fence_after();
      const uint64_t db = desc_sw128(sb + kOffV + b * kSlotBytes, KC * 128, 1024);
#pragma unroll
      for (int kk = 0; kk < KC / 16; ++kk)                   // k-steps of 16 keys; each half's P in its S columns
        umma_ts_warp<CG>(leader, tmem + kTmemO, tmem + b * KC + (kk / (KC / 32)) * NK + (kk % (KC / 32)) * 8,
                         db + kk * 128, Shape<CG>::kIdescPV, (cx | kk) != 0);
      umma_commit_warp<CG>(leader, &ctl.pv_done[b]);
      if (cx == n - 1) umma_commit_warp<CG>(leader, &ctl.o_full);
      return true;
    };
    const uint64_t da = desc_sw128(sb + kOffQ, 16, 1024);
    bool ok = true;
    while (ok && walk.next(t, p, x)) {
      if (!(ok = wait(&ctl.q_full, uc))) break;
      const int n = p.c1 - p.c0;
      for (int c = 0; c < n && ok; ++c) {
        const int64_t xg = gc + c;
        const int b = (int)(xg & 1);
        // S buffer b: P of chunk c-2 (of this or the last piece) was read by a product issued before
        if (!(ok = wait(&ctl.k_full[b], xg >> 1))) break;
        tc_fence_after();
        const uint64_t db = desc_sw128(sb + b * kSlotBytes, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)                      // k-steps of 16 dims: 32 bytes of a slab's 128-byte lines
          umma_ss_warp<CG>(leader, tmem + b * KC, da + (kk >> 2) * 1024 + (kk & 3) * 2,
                           db + (kk >> 2) * 512 + (kk & 3) * 2, Shape<CG>::kIdescS, kk != 0);
        umma_commit_warp<CG>(leader, &ctl.s_done[b]);
        if (c == n - 1) umma_commit_warp<CG>(leader, &ctl.q_empty);
        if (c > 0) ok = pv(c - 1, n);
      }
      if (!ok) break;
      ok = pv(n - 1, n);
      gc += n;
      ++uc;
    }
    // every MMA issued above has finished before TMEM is freed
    if (leader) {
      if constexpr (CG == 1) umma_commit(&ctl.mma_done); else umma_commit_pair_local(&ctl.mma_done);
      volatile int never = 0;
      mbar_wait(&ctl.mma_done, 0, &never);
    }
    __syncwarp();
  } else if (CG == 2 && warp == kMmaWarp) {
    // ============================================================ rank 1's V handed to rank 0
    int64_t gc = 0;
    for (bool ok = true; ok && walk.next(t, p, x);)
      for (int c = p.c0; c < p.c1 && ok; ++c, ++gc) {
        ok = warp_wait_fast(&ctl.v_full[gc % kVSlots], (uint32_t)((gc / kVSlots) & 1), abort_flag);
        if (ok && lane == 0) mbar_arrive_cluster(&ctl.p_full[gc & 1], 0);
        __syncwarp();
      }
  } else if (warp == kQWarp) {
    // ============================================================ Q of the next unit
    int64_t uc = 0;
    bool ok = true;
    while (ok && walk.next(t, p, x)) {
      if (!(ok = !warp_aborted(abort_flag) &&
                 warp_wait_sleep(&ctl.q_empty, (uint32_t)((uc & 1) ^ 1), abort_flag))) break;
      const int n = max(0, min(x.nrows - (int)rank * 128, 128));             // rows of this CTA
      if (lane == 0) mbar_expect_tx_leader<CG>(&ctl.q_full, (uint32_t)n * (kHeadDim * 2));
      __syncwarp();
      load_q_rows<CG>(smem + kOffQ, &tm_tok, &tm_row, t, x, x.row0 + (int)rank * 128, n, a.H, lane, &ctl.q_full);
      ++uc;
    }
    if (!ok) drain_copies();
  } else if (warp == kNfWarp) {
    // ============================================================ V of the unit's own tokens checked
    int64_t uc = 0;
    while (walk.next(t, p, x)) {
      if (warp_aborted(abort_flag)) break;
      // A list is free once every softmax warp has taken the one kNfBufs units before.
      // Those warps take each unit's, so neither side can be two phases behind the
      // other and mistake one for the next by its parity (paced by q_empty, which
      // nothing held back for this warp, that was possible in units of a chunk or two).
      if (!warp_wait_sleep(&ctl.nf_free[uc % kNfBufs], (uint32_t)((uc / kNfBufs & 1) ^ 1), abort_flag)) break;
      // keys that only some rows see (at most 255), 32 at a time; none in a piece that ends before them
      const int32_t first = t.pos0[x.si] + x.row0 / t.hpg;   // position of the unit's first row
      const int own = p.c1 * KC - 1 > first ? x.kv_len - 1 - first : 0;
      uint32_t word = 0;
      for (int i0 = 0; i0 < own; i0 += 32) {
        const int64_t my_off = i0 + lane < own ? kv_row<PAGED>(a.kv, t, x.si, x.grp, first + 1 + i0 + lane) : -1;
        const int rows = min(32, own - i0);
        uint32_t bits = 0;                                   // rows whose 8 dims of this lane hold one
#pragma unroll 4
        for (int i = 0; i < rows; ++i) {
          const int64_t off = __shfl_sync(0xffffffffu, my_off, i);
          uint4 v = make_uint4(0, 0, 0, 0);
          if (off >= 0) v = *reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.kv.v + off + lane * 8);
          // an exponent of all ones carries into the sign bit
          const uint32_t c = ((v.x & 0x7f807f80u) + 0x00800080u) | ((v.y & 0x7f807f80u) + 0x00800080u) |
                             ((v.z & 0x7f807f80u) + 0x00800080u) | ((v.w & 0x7f807f80u) + 0x00800080u);
          bits |= (c & 0x80008000u ? 1u : 0u) << i;
        }
        bits = __reduce_or_sync(0xffffffffu, bits);
        if (lane == (i0 >> 5)) word = bits;
      }
      if (lane < 8) ctl.nf[uc % kNfBufs][lane] = word;
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.nf_full[uc % kNfBufs]);
      ++uc;
    }
  } else if (warp < kSoftmaxWarps) {
    // ============================================================ softmax + epilogue
    const int quad = warp & 3, half = warp >> 2;
    const int li = quad * 32 + lane;                         // TMEM lane: row of this CTA
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const float tau2 = a.scale * 1.4426950408889634f;
    int64_t gc = 0, uc = 0;
    // No early exit: the two warps of a quadrant meet at a named barrier per chunk.
    // The next piece is looked up while this one's last product runs.
    DensePiece p_next;
    DenseUnit x_next;
    for (bool more = walk.next(t, p, x); more; p = p_next, x = x_next) {
      const int n = p.c1 - p.c0;
      const int valid = x.nrows - (int)rank * 128;
      const bool active = li < valid, warp_active = quad * 32 < valid;
      const int32_t row = x.row0 + (active ? (int)rank * 128 + li : 0);
      const int32_t pos = t.pos0[x.si] + row / t.hpg;
      const int64_t at = dense_q_row(t, x, row, a.H);
      const int32_t first = t.pos0[x.si] + x.row0 / t.hpg;               // of the unit
      const int32_t first_cta = t.pos0[x.si] + (x.row0 + (int)rank * 128) / t.hpg;
      const int32_t kv_len = x.kv_len;
      // the unit's list of values that are not finite, taken before its first own key,
      // or at the end of a piece without one (empty then)
      bool nf_taken = false, any_nf = false;
      uint32_t my_nf = 0;
      auto take_nf = [&]() {
        nf_taken = true;
        mbar_wait_fast(&ctl.nf_full[uc % kNfBufs], (uint32_t)((uc / kNfBufs) & 1), abort_flag);
        my_nf = lane < 8 ? ctl.nf[uc % kNfBufs][lane] : 0u;
        any_nf = __any_sync(0xffffffffu, my_nf != 0);
        if (lane == 0) mbar_arrive(&ctl.nf_free[uc % kNfBufs]);
      };
      // the page of run `lane` of 16 keys of a chunk; 0 where nothing is looked up
      auto page_of_run = [&](int c) -> int32_t {
        const int32_t key = c * KC + lane * 16;
        if (!PAGED || lane >= KC / 16 || c >= p.c1 || key >= kv_len) return 0;
        return a.kv.table[(int64_t)t.slot[x.si] * a.kv.max_pages + key / a.kv.page_tokens];
      };
      int32_t next_page = page_of_run(p.c0);
      float m = -INFINITY, l = 0.f;
      for (int c = 0; c < n; ++c, ++gc) {
        const int b = (int)(gc & 1);
        const int32_t j0 = (p.c0 + c) * KC;
        // bit per run of 16 keys of the chunk: its page is out of range
        const uint32_t bad =
            PAGED ? __ballot_sync(0xffffffffu, next_page < 0 || next_page >= a.kv.n_pages) : 0u;
        next_page = page_of_run(p.c0 + c + 1);
        if (!nf_taken && j0 + KC - 1 > first) take_nf();
        mbar_wait_fast(&ctl.s_done[b], (uint32_t)((gc >> 1) & 1), abort_flag);
        tc_fence_after();
        const bool clear = j0 + KC > kv_len || bad || (any_nf && j0 + KC - 1 > first);
        if (clear) {
          // V rows that must not reach the product become zero in shared memory
          mbar_wait_fast(&ctl.v_full[gc % kVSlots], (uint32_t)((gc / kVSlots) & 1), abort_flag);
          unsigned char* vs = smem + kOffV + (gc % kVSlots) * kSlotBytes;
          constexpr int kPieces = 2048 / KC;                 // 16-byte pieces of a key's row here: 32 or 16
          for (int i = threadIdx.x; i < KC * kPieces; i += kSoftmaxWarps * 32) {
            const int key = i / kPieces, piece = i % kPieces;     // a warp covers one or two keys
            const int32_t rel = j0 + key - first - 1;
            const uint32_t w = __shfl_sync(0xffffffffu, my_nf, rel >= 0 ? (rel >> 5) & 7 : 0);
            const bool zero = j0 + key >= kv_len || ((bad >> (key >> 4)) & 1u) ||
                              (rel >= 0 && ((w >> (rel & 31)) & 1u));
            if (zero)
              *reinterpret_cast<uint4*>(vs + (piece >> 3) * (KC * 128) + key * 128 + ((piece & 7) << 4)) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (warp_active) {
          float s[NK];                                       // raw scores
#pragma unroll
          for (int k = 0; k < NK; k += 16) {
            float v[16];
            tmem_ld16(lane_addr + b * KC + half * NK + k, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[k + i] = v[i];
          }
          tmem_wait_ld();
          if (j0 + KC - 1 > first_cta || bad) {              // keys this row does not attend: -inf
            const int32_t lim = pos - j0 - half * NK;
#pragma unroll
            for (int i = 0; i < NK; ++i)
              if (i > lim || ((bad >> ((half * NK + i) >> 4)) & 1u)) s[i] = -INFINITY;
          }
          float pm4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int i = 4; i < NK; i += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) pm4[k] = fmaxf(pm4[k], s[i + k]);
          }
          ctl.red[b][half][li] = fmaxf(fmaxf(pm4[0], pm4[1]), fmaxf(pm4[2], pm4[3])) * tau2;
          named_bar_sync(1 + quad, 64);
          const float mc = fmaxf(ctl.red[b][0][li], ctl.red[b][1][li]);
          float f = 1.f;
          bool need = false;
          if (mc > m + 8.f) {                                // false while both are -inf
            if (m != -INFINITY) {
              f = exp2f(m - mc);
              need = true;
            }
            m = mc;
          }
          l *= f;
          if (__any_sync(0xffffffffu, need)) {
            // O holds chunks 0..c-1 (c >= 1 here): wait for the last of their products
            const int64_t xp = gc - 1;
            mbar_wait_fast(&ctl.pv_done[xp & 1], (uint32_t)((xp >> 1) & 1), abort_flag);
            tc_fence_after();
#pragma unroll 1
            for (int piece = 0; piece < 8; ++piece) {
              float o[16];
              const uint32_t addr = lane_addr + kTmemO + half * 128 + piece * 16;
              tmem_ld16(addr, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tmem_st16(addr, o);
            }
            tmem_wait_st();
          }
          const float mb = m == -INFINITY ? 0.f : m;
          float l4[4] = {l, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < NK; k += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p0 = ex2_approx(fmaf(s[k + 2 * i], tau2, -mb));
              const float p1 = ex2_approx(fmaf(s[k + 2 * i + 1], tau2, -mb));
              l4[i & 3] += p0 + p1;
              pk[i] = pack_bf16x2(p0, p1);
            }
            tmem_st16u(lane_addr + b * KC + half * NK + k / 2, pk);   // over this thread's own scores
          }
          l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        mbar_wait_fast(&ctl.v_full[gc % kVSlots], (uint32_t)((gc / kVSlots) & 1), abort_flag);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_leader<CG>(&ctl.p_full[b], clear);
      }
      if (!nf_taken) take_nf();
      float lt = 0.f;
      if (warp_active) {                                     // the row's sum: both warps' parts
        ctl.red[gc & 1][half][li] = l;                       // the last chunk's buffer is the other one
        named_bar_sync(1 + quad, 64);
        lt = ctl.red[gc & 1][0][li] + ctl.red[gc & 1][1][li];
        named_bar_sync(1 + quad, 64);                        // the next piece's first chunk writes this buffer
      }
      more = walk.next(t, p_next, x_next);
      mbar_wait_fast(&ctl.o_full, (uint32_t)(uc & 1), abort_flag);
      tc_fence_after();
      if (warp_active) {
        const bool whole = p.part < 0;
        // lt = 0: no key at all, or scores of -inf only
        const bool all_inf = active && lt == 0.f && any_key<PAGED>(a.kv, t, x.si, p.c0 * KC, min(pos, p.c1 * KC - 1));
        __syncwarp();
        const float inv = !whole ? 1.f : all_inf ? dense::kNan : lt != 0.f ? 1.f / lt : 0.f;
        const int row_q = (int)rank * 128 + quad * 32 + (lane & ~3);   // first row of this lane's quad
        float* part_q = whole ? nullptr : a.part + ((int64_t)p.part * t.prows + row_q) * dense::kPartFloats;
        int64_t at_q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) at_q[j] = __shfl_sync(0xffffffffu, active ? at : -1, (lane & ~3) + j);
#pragma unroll 1
        for (int piece = 0; piece < 4; ++piece) {
          float o[32];
#pragma unroll
          for (int k = 0; k < 32; k += 16) {
            float v[16];
            tmem_ld16(lane_addr + kTmemO + half * 128 + piece * 32 + k, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) o[k + i] = v[i];
          }
          tmem_wait_ld();
          if (any_nf) {                                      // keys kept out of the product
#pragma unroll 1
            for (int w = 0; w < 8; ++w) {
              uint32_t bits = __shfl_sync(0xffffffffu, my_nf, w);
              while (bits) {
                const int32_t key = first + 1 + w * 32 + __ffs(bits) - 1;
                bits &= bits - 1;
                if (!active || key > pos || key < p.c0 * KC || key >= p.c1 * KC) continue;
                const int64_t off = kv_row<PAGED>(a.kv, t, x.si, x.grp, key);
                if (off < 0) continue;
                const __nv_bfloat16* kr = (const __nv_bfloat16*)a.kv.k + off;
                const __nv_bfloat16* vr = (const __nv_bfloat16*)a.kv.v + off + half * 128 + piece * 32;
                float sc = 0.f;
#pragma unroll 1
                for (int d = 0; d < kHeadDim; ++d)
                  sc = fmaf(__bfloat162float(a.q[at * kHeadDim + d]), __bfloat162float(kr[d]), sc);
                const float pw = ex2_approx(fmaf(sc, tau2, m == -INFINITY ? 0.f : -m));
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = fmaf(pw, __bfloat162float(vr[i]), o[i]);
              }
            }
            __syncwarp();
          }
          store_cols32(o, inv, whole ? a.o : nullptr, part_q, at_q, half * 128 + piece * 32, lane);
        }
        if (active && half == 0) {
          if (!whole) {
            float* st = part_q + (lane & 3) * dense::kPartFloats + kHeadDim;
            st[0] = m;
            st[1] = all_inf ? -1.f : lt;
          } else if (a.lse) {
            a.lse[at] = lt != 0.f ? (m + log2f(lt)) * 0.6931471805599453f : -INFINITY;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader<CG>(&ctl.o_free);
      ++uc;
    }
  }
  tc_fence_before();
  if constexpr (CG == 2) cluster_sync_all(); else __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem, kTmemCols);
  }
  dense_wait_last(a.late);
}

}  // namespace qsa
