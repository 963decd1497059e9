// dense_bwd_tc.cuh -- gradient of the packed prompts' causal GQA attention,
// bf16, on tcgen05 tensor cores.
//
// With s the softmax scale, lse and delta_i = dout_i . o_i of the forward:
//   P = exp(s Q K^T - lse),  dP = dO V^T,  dS = P (dP - delta),
//   dV = P^T dO,  dK = s dS^T Q,  dQ = s dS K.
// At 256 dims one tile's dK and dV fill tensor memory (2 x 256 columns), so
// each gradient has a kernel of its own that keeps its sums in 256 columns
// and S and dP in the other 256:
//   dV  keys stay (K), rows stream: S^T = K Q^T, dV += P^T dO      2 products
//   dK  keys stay (K, V), rows stream: S^T, dP^T, dK += dS^T Q     3 products
//   dQ  rows stay (Q, dO), keys stream: S, dP, dQ += dS K          3 products
// Eight products where five would do with all sums in one place; none needs
// atomics, so the same inputs give the same bits.  (Keys on 64-row tiles that
// hold dK and dV together would stream Q and dO at 64 bytes per cycle and SM,
// beyond L2; 128 keys per CTA of a pair need 32.)
//
// A unit is a tile of 256 stationary rows on a CTA pair (cta_group::2, 128
// each): for dQ rows (token, head) of a KV group as in the forward, for dK and
// dV keys, whose chunks are the group's heads x tiles of 128 tokens from the
// unit's first key on.  Chunks are 128 wide; the streamed operand of S and dP
// is split between the CTAs by rows, that of the gradient's product by dims.
// P and dS are rounded to bf16 for the products, once each, and written over the
// columns they were computed from, so no warp waits for another's reads.  A rounded
// dS makes the error of dq and dk 1.42 times that of rounding the result alone, as
// P's does dv's.  (Its remainders could be multiplied too, from the columns that dS
// leaves free: 1.00 times, but 8.33 ms instead of 7.29, in the same minute, for the
// two prompts below with their forward.)  Rows of few keys have an o as large as v, and the error of
// delta = dout . o, o rounded, is then several times dS's: for rows whose keys are
// all in the first chunk (positions below 128) the dQ kernel forms delta as the sum
// of P dP instead and leaves it for the dK kernel.
//
// Roles per CTA (12 warps): eight softmax warps (two per lane quadrant, each
// thread one lane and 64 of a chunk's columns), one TMA producer, one warp that
// issues the MMAs (in rank 0), one that loads the stationary tiles.  MMA order with three products:
//   S0 dP0 | S1 D0 dP1 | S2 D1 dP2 | ...
// so that the exponentials of chunk c+1 run under D(c) and dP(c+1), and dS(c+1)
// under S(c+2); one buffer each for S and dP is enough.  With two products (dV)
// S is double-buffered as in the forward.
//
// Segments whose lse, delta, K or V hold infinities or NaN are left to the
// CUDA-core kernels (dense_simt.cuh), which skip masked pairs one by one; here
// masked pairs are multiplied by zero.  Rows behind a segment's end may be
// anything: their scores are replaced and their operand rows zeroed in shared
// memory.  Every mbarrier wait is bounded.
//
// Measured (two prompts of 8192, 24 heads, 2 groups): dQ 1.62 ms, dV 1.34, dK 2.05,
// 6.6 TFLOP issued in 5.0 ms, the tensor pipe 72 to 80 % active at the 1.3 to 1.5
// GHz that the power cap leaves.
#pragma once
#include <type_traits>

#include "dense_tc.cuh"

namespace qsa {
namespace dense_bwd {
using dense_tc::kThreads;
using dense_tc::kSoftmaxWarps;
using dense_tc::kProducerWarp;
using dense_tc::kMmaWarp;
using dense_tc::kQWarp;
using dense_tc::kSlotBytes;
using dense_tc::kQBytes;
enum Grad { kDv, kDk, kDq };
constexpr int kRows = 256, kKeys = 128, kGrid = 74;
constexpr int kStatTile = 128;                        // tokens of a row of the statistics
template <Grad M> struct Ring {
  static constexpr int kProducts = M == kDv ? 2 : 3;
  static constexpr int kTiles = M == kDv ? 1 : 2;     // stationary tiles of 64 KiB
  // 32 KiB slots of the three streamed operands
  static constexpr int kN0 = M == kDv ? 2 : 1, kN1 = M == kDv ? 0 : 1, kN2 = M == kDv ? 3 : 1;
  static constexpr int kSlots = kN0 + kN1 + kN2;
  __device__ static constexpr int slots(int kind) { return kind == 0 ? kN0 : kind == 1 ? kN1 : kN2; }
  __device__ static constexpr int offset(int kind) { return (kind == 0 ? 0 : kind == 1 ? kN0 : kN0 + kN1) * kSlotBytes; }
  static constexpr int kBufs = M == kDv ? 2 : 1;      // S buffers
  static constexpr int kStats = M == kDv ? 4 : 2;     // buffers of row statistics
};
constexpr int kOffCtl = 3 * kSlotBytes + 2 * kQBytes; // 229376; dV: 5 slots and one tile
constexpr int kCtlBytes = 3 * 1024;
constexpr int kSmemBytes = kOffCtl + kCtlBytes;       // 232448: the base itself is 1024-byte aligned
constexpr uint32_t kTmemP = 128, kTmemD = 256;
using Pair = dense_tc::Shape<2>;
}  // namespace dense_bwd

// Tensor maps of one gradient's kernel: streamed operands of S, dP and the
// gradient's product; the stationary tiles (dQ: Q and dO by token and by row;
// dK, dV: K and V).
struct DenseBwdMaps {
  CUtensorMap s, p, d, fix0, fix1, row0, row1;
};

struct DenseBwdTcArgs {
  const float* lse2;          // [H][stat rows] lse * log2 e, +inf behind a segment's end
  float* delta;               // [H][stat rows]; those of positions below kKeys are rewritten by dQ
  const uint8_t* flags;       // segment_flagged: not for these kernels
  __nv_bfloat16* out;
  float* part;
  int64_t stat_rows;
  int H;
  float scale;
  bool late;                  // dense_wait_first
};

struct DenseBwdTcCtl {
  uint64_t full[2][2];                                // of S's and dP's operand, rank 0's: both CTAs' halves
  uint64_t d_full[3];                                 // of the gradient's operand: this CTA's half
  uint64_t s_done[2], dp_done, d_done[3];             // products: for their readers, and their operand's slot is free
  uint64_t fix_full, fix_empty;
  uint64_t s_free, w_full[2];                         // S read; P (dV) or dS written
  uint64_t o_full, o_free;
  uint64_t st_full[4], st_free[4];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};
constexpr int kBwdStatOff = 1024;                     // of the control block: lse2[128] by buffer, then delta[128] (dK)
static_assert(sizeof(DenseBwdTcCtl) <= kBwdStatOff, "control block");
static_assert(kBwdStatOff + 2 * 1024 <= dense_bwd::kCtlBytes, "control block");

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          sm100::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
      : "memory");
}

template <dense_bwd::Grad M>
__global__ void __launch_bounds__(dense_bwd::kThreads, 1)
    dense_bwd_tc_kernel(const __grid_constant__ DenseBwdMaps tm, const __grid_constant__ DenseTable t,
                        const __grid_constant__ DenseBwdTcArgs a) {
  using namespace dense_bwd;
  using namespace sm100;
  using R = Ring<M>;
  constexpr bool kByKeys = M != kDq;
  constexpr int kProducts = R::kProducts, kBufs = R::kBufs;
  extern __shared__ __align__(1024) unsigned char smem_1k[];
  unsigned char* const smem = smem_1k;
  constexpr int kOffFix = R::kSlots * kSlotBytes;
  DenseBwdTcCtl& ctl = *reinterpret_cast<DenseBwdTcCtl*>(smem + kOffCtl);
  float* stats = reinterpret_cast<float*>(smem + kOffCtl + kBwdStatOff);
  volatile int* abort_flag = &ctl.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int cta = blockIdx.x / 2;

  // ---------------------------------------------------------------- set-up
  if (smem_u32(smem) & 1023u) {                      // as in the forward
    report_error(kErrWaitTimeout);
    pdl_wait();
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.full[0][i], 2);
      mbar_init(&ctl.full[1][i], 2);
      mbar_init(&ctl.s_done[i], 1);
      mbar_init(&ctl.w_full[i], kSoftmaxWarps * 2 + 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&ctl.d_full[i], 1);
      mbar_init(&ctl.d_done[i], 1);
    }
    for (int i = 0; i < R::kStats; ++i) {
      mbar_init(&ctl.st_full[i], 1);
      mbar_init(&ctl.st_free[i], kSoftmaxWarps);
    }
    mbar_init(&ctl.s_free, kSoftmaxWarps * 2);
    mbar_init(&ctl.dp_done, 1);
    mbar_init(&ctl.fix_full, 2);
    mbar_init(&ctl.fix_empty, 1);
    mbar_init(&ctl.o_full, 1);
    mbar_init(&ctl.o_free, kSoftmaxWarps * 2);
    mbar_init(&ctl.mma_done, 1);
    ctl.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc_cg<2>(&ctl.tmem_base, dense_tc::kTmemCols);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  dense_wait_first(a.late);

  DenseWalk walk;
  walk.init(t, cta);
  DensePiece p;
  DenseUnit x;
  // the next piece of a segment that is not flagged (the same in every role and CTA)
  int seen = -1;                                     // the segment looked up last
  bool flagged = false;
  auto next_of = [&](DensePiece& np, DenseUnit& nx) -> bool {
    while (walk.next(t, np, nx)) {
      if (nx.si != seen) {
        seen = nx.si;
        flagged = segment_flagged(a.flags, t.slot[nx.si], t.q_len[nx.si]);
      }
      if (!flagged) return true;
    }
    return false;
  };
  auto next = [&]() { return next_of(p, x); };
  // a stationary row in its token-major array
  auto unit_row = [&](int32_t row) -> int64_t {
    return kByKeys ? (int64_t)(t.q_offset[x.si] + row) * t.G + x.grp : dense_q_row(t, x, row, a.H);
  };
  if (warp == kProducerWarp) {
    // ============================================================ TMA producer
    // A slot is four boxes of 64 lines x 64 dims, one per lane: rows of this
    // CTA's half x 256 dims (S, dP), or 128 rows x this CTA's half of the dims.
    const int off_s = (lane & 3) * 8192, x_s = (lane & 3) * 64, y_s = (int)rank * 64;
    const int off_d = (lane & 1) * 16384 + ((lane >> 1) & 1) * 8192;
    const int x_d = (lane & 1) * 64 + (int)rank * 128, y_d = ((lane >> 1) & 1) * 64;
    uint32_t slot[3] = {0, 0, 0}, phase[3] = {0, 0, 0}, st_buf = 0, st_phase = 0;
    bool ok = true;
    // a chunk's first row of the segment and its head (dQ: KV group)
    struct Chunk {
      int32_t r0, head, left;                        // left: heads until the next rows
    };
    auto advance = [&](Chunk& c) {
      if (!kByKeys) {
        c.r0 += kKeys;
      } else if (--c.left > 0) {
        ++c.head;
      } else {
        c.r0 += kKeys;
        c.head -= t.hpg - 1;
        c.left = t.hpg;
      }
    };
    auto put = [&](auto kind_c, const Chunk& c) -> bool {
      constexpr int kind = decltype(kind_c)::value;
      constexpr uint32_t kN = R::slots(kind);
      const uint32_t b = slot[kind], ph = phase[kind];
      slot[kind] = b + 1 == kN ? 0 : b + 1;
      if (b + 1 == kN) phase[kind] ^= 1;
      unsigned char* to = smem + R::offset(kind) + b * kSlotBytes;
      const int32_t cx = c.head * kHeadDim, cy = t.q_offset[x.si] + c.r0;
      uint64_t* const free_bar = kind == 0 ? &ctl.s_done[b] : kind == 1 ? &ctl.dp_done : &ctl.d_done[b];
      if (!warp_wait_fast(free_bar, ph ^ 1, abort_flag)) return false;
      if constexpr (kind == 2) {
        if (lane == 0) mbar_expect_tx(&ctl.d_full[b], kSlotBytes);
        __syncwarp();
        if (lane < 4) tma_load_2d(to + off_d, &tm.d, cx + x_d, cy + y_d, &ctl.d_full[b]);
      } else {
        if (lane == 0) mbar_expect_tx_leader<2>(&ctl.full[kind][b], kSlotBytes);
        __syncwarp();
        if (lane < 4)
          tma_load_2d_leader<2>(to + off_s, kind == 0 ? &tm.s : &tm.p, cx + x_s, cy + y_s, &ctl.full[kind][b]);
      }
      // The chunk's row statistics, behind a load whose slot was freed after
      // the softmax that held the buffer: this wait does not hold up the ring.
      if constexpr (kByKeys && kind == kProducts - 2) {
        if (!warp_wait_fast(&ctl.st_free[st_buf], st_phase ^ 1, abort_flag)) return false;
        if (lane == 0) {
          const int64_t at = (int64_t)c.head * a.stat_rows + t.slot[x.si] * kStatTile + c.r0;
          mbar_expect_tx(&ctl.st_full[st_buf], M == kDv ? 512 : 1024);
          bulk_load(stats + st_buf * 128, a.lse2 + at, 512, &ctl.st_full[st_buf]);
          if (M != kDv) bulk_load(stats + (R::kStats + st_buf) * 128, a.delta + at, 512, &ctl.st_full[st_buf]);
        }
        __syncwarp();
        st_buf = st_buf + 1 == R::kStats ? 0 : st_buf + 1;
        if (st_buf == 0) st_phase ^= 1;
      }
      return true;
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0> kPutS{};
    constexpr integral_constant<int, kProducts == 3 ? 1 : 0> kPutP{};
    constexpr integral_constant<int, 2> kPutD{};
    while (ok && next()) {
      const int n = p.c1 - p.c0;
      Chunk cur;
      if (kByKeys) {
        const int tile = p.c0 / t.hpg, hl = p.c0 - tile * t.hpg;
        cur = {x.row0 + tile * kKeys, x.grp * t.hpg + hl, t.hpg - hl};
      } else {
        cur = {p.c0 * kKeys, x.grp, 0};
      }
      Chunk nxt = cur;
      advance(nxt);
      ok = put(kPutS, cur);
      if (kProducts == 3) ok = ok && put(kPutP, cur);
      for (int c = 0; c < n && ok; ++c) {
        if (c + 1 < n) ok = put(kPutS, nxt);
        ok = ok && put(kPutD, cur);
        if (kProducts == 3 && c + 1 < n) ok = ok && put(kPutP, nxt);
        cur = nxt;
        advance(nxt);
      }
    }
    if (!ok) drain_copies();                         // no copy outlives the CTA
  } else if (warp == kMmaWarp && rank == 0) {
    // ============================================================ MMA issuer
    int64_t gc = 0, uc = 0;                          // chunks and pieces so far
    const uint32_t sb = smem_u32(smem), leader = elect_one();
    // what both CTAs' threads arrive on
    auto wait = [&](uint64_t* bar, int64_t phase) {
      return warp_wait_fast<true>(bar, (uint32_t)(phase & 1), abort_flag);
    };
    // S (kind 0) or dP (kind 1) of the piece's chunk c
    auto scores = [&](int kind, int c, int n) -> bool {
      const int64_t xg = gc + c;
      const int slot = (int)(xg % R::slots(kind));
      // with one S buffer: the softmax has read the last chunk's.  With two, P of
      // chunk c-2 was read by a product issued before.
      if (kBufs == 1 && kind == 0 && !wait(&ctl.s_free, xg ^ 1)) return false;
      if (!wait(&ctl.full[kind][slot], xg / R::slots(kind))) return false;
      tc_fence_after();
      const uint64_t da = desc_sw128(sb + kOffFix + kind * kQBytes, 16, 1024);
      const uint64_t db = desc_sw128(sb + R::offset(kind) + slot * kSlotBytes, 16, 1024);
      const uint32_t d = tmem + (kind == 1 ? kTmemP : (uint32_t)slot * 128);
#pragma unroll
      for (int kk = 0; kk < 16; ++kk)                // k-steps of 16 dims: 32 bytes of a slab's 128-byte lines
        umma_ss_warp<2>(leader, d, da + (kk >> 2) * 1024 + (kk & 3) * 2, db + (kk >> 2) * 512 + (kk & 3) * 2,
                        Pair::kIdescS, kk != 0);
      umma_commit_warp<2>(leader, kind == 0 ? &ctl.s_done[slot] : &ctl.dp_done);
      if (c == n - 1 && kind == kProducts - 2) umma_commit_warp<2>(leader, &ctl.fix_empty);
      return true;
    };
    auto grad = [&](int c, int n) -> bool {
      const int64_t xg = gc + c;
      const int b = (int)(xg % kBufs), slot = (int)(xg % R::kN2);
      if (!wait(&ctl.w_full[b], xg / kBufs)) return false;        // P or dS, and both halves of the operand
      if (c == 0 && !wait(&ctl.o_free, uc ^ 1)) return false;
      tc_fence_after();
      const uint64_t db = desc_sw128(sb + R::offset(2) + slot * kSlotBytes, 16384, 1024);
      const uint32_t w = tmem + (M == kDv ? (uint32_t)b * 128 : kTmemP);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)                 // k-steps of 16 chunk columns; each half's start at its columns
        umma_ts_warp<2>(leader, tmem + kTmemD, w + (kk >> 2) * 64 + (kk & 3) * 8, db + kk * 128, Pair::kIdescPV,
                        (c | kk) != 0);
      umma_commit_warp<2>(leader, &ctl.d_done[slot]);
      if (c == n - 1) umma_commit_warp<2>(leader, &ctl.o_full);
      return true;
    };
    bool ok = true;
    while (ok && next()) {
      if (!(ok = wait(&ctl.fix_full, uc))) break;
      const int n = p.c1 - p.c0;
      ok = scores(0, 0, n);
      if (kProducts == 3) ok = ok && scores(1, 0, n);
      for (int c = 0; c < n && ok; ++c) {
        if (c + 1 < n) ok = scores(0, c + 1, n);
        ok = ok && grad(c, n);
        if (kProducts == 3 && c + 1 < n) ok = ok && scores(1, c + 1, n);
      }
      gc += n;
      ++uc;
    }
    // every MMA issued above has finished before TMEM is freed
    if (leader) {
      umma_commit_pair_local(&ctl.mma_done);
      volatile int never = 0;
      mbar_wait(&ctl.mma_done, 0, &never);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ============================================================ rank 1's operand handed to rank 0
    // That of the gradient's product, as the forward's V.  A chunk's arrival waits for
    // the product that used the same w_full before: with more slots than buffers the
    // operand may be a chunk too early.
    uint32_t gc = 0;
    for (bool ok = true; ok && next();)
      for (int c = p.c0; c < p.c1 && ok; ++c, ++gc) {
        const uint32_t last = gc - kBufs;
        if (R::kN2 > kBufs && gc >= kBufs)
          ok = warp_wait_fast(&ctl.d_done[last % R::kN2], last / R::kN2 & 1, abort_flag);
        ok = ok && warp_wait_fast(&ctl.d_full[gc % R::kN2], gc / R::kN2 & 1, abort_flag);
        if (ok && lane == 0) mbar_arrive_cluster(&ctl.w_full[gc % kBufs], 0);
        __syncwarp();
      }
  } else if (warp == kQWarp) {
    // ============================================================ stationary tiles of the next unit
    int64_t uc = 0;
    bool ok = true;
    while (ok && next()) {
      if (!(ok = !warp_aborted(abort_flag) &&
                 warp_wait_sleep(&ctl.fix_empty, (uint32_t)((uc & 1) ^ 1), abort_flag))) break;
      const int n = kByKeys ? 128 : max(0, min(x.nrows - (int)rank * 128, 128));   // rows of this CTA that are loaded
      if (lane == 0) mbar_expect_tx_leader<2>(&ctl.fix_full, (uint32_t)(n * kHeadDim * 2 * R::kTiles));
      __syncwarp();
      if constexpr (kByKeys) {                       // boxes of 64 keys x 64 dims
        if (lane < 8 * R::kTiles) {
          const int tile = lane >> 3, slab = lane & 3, run = (lane >> 2) & 1;
          tma_load_2d_leader<2>(smem + kOffFix + tile * kQBytes + slab * 16384 + run * 8192,
                                tile == 0 ? &tm.fix0 : &tm.fix1, x.grp * kHeadDim + slab * 64,
                                t.q_offset[x.si] + x.row0 + (int)rank * 128 + run * 64, &ctl.fix_full);
        }
      } else {
        const int32_t r0 = x.row0 + (int)rank * 128;
        load_q_rows<2>(smem + kOffFix, &tm.fix0, &tm.row0, t, x, r0, n, a.H, lane, &ctl.fix_full);
        load_q_rows<2>(smem + kOffFix + kQBytes, &tm.fix1, &tm.row1, t, x, r0, n, a.H, lane, &ctl.fix_full);
      }
      ++uc;
    }
    if (!ok) drain_copies();
  } else if (warp < kSoftmaxWarps) {
    // ============================================================ P, dS and the epilogue
    const int quad = warp & 3, half = warp >> 2;
    const int li = quad * 32 + lane;                 // TMEM lane: stationary row of this CTA
    const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
    const float tau2 = a.scale * 1.4426950408889634f;
    int64_t gc = 0, uc = 0;
    // No early exit: after an abort every wait returns at once.  The next piece is
    // looked up while this one's last product runs.
    DensePiece p_next;
    DenseUnit x_next;
    for (bool more = next(); more; p = p_next, x = x_next) {
      const int n = p.c1 - p.c0;
      const int valid = x.nrows - (int)rank * 128;
      const bool active = li < valid;
      const int32_t row = x.row0 + (active ? (int)rank * 128 + li : 0);
      const int32_t seg_n = t.q_len[x.si];
      const int32_t own = kByKeys ? x.row0 + (int)rank * 128 + li : row / t.hpg;   // position
      const int64_t at = unit_row(row);
      float lse2 = 0.f, delta = 0.f;                 // of this thread's row (dQ)
      int64_t sat = 0;
      if (!kByKeys) {
        sat = (int64_t)(x.grp * t.hpg + row - own * t.hpg) * a.stat_rows +
                            (int64_t)t.slot[x.si] * kStatTile + own;
        lse2 = a.lse2[sat];
        delta = a.delta[sat];
      }
      // first position of this CTA's stationary rows (dQ: below it no key is masked), last one (dK, dV)
      const int32_t edge = kByKeys ? x.row0 + (int)rank * 128 + 127 : (x.row0 + (int)rank * 128) / t.hpg;
      // Rows behind the segment's end become zero in the operand of the chunk's product.
      auto clear_tail = [&](int32_t j0) {
        unsigned char* ds = smem + R::offset(2) + (gc % R::kN2) * kSlotBytes;
        for (int i = threadIdx.x + (seg_n - j0) * 16; i < kKeys * 16; i += kSoftmaxWarps * 32)
          *reinterpret_cast<uint4*>(ds + ((i >> 3) & 1) * 16384 + (i >> 4) * 128 + ((i & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
      };
      // first position of a chunk's columns; by keys, `left` heads until the next tokens
      const int tile0 = kByKeys ? p.c0 / t.hpg : 0;
      int left = kByKeys ? t.hpg - (p.c0 - tile0 * t.hpg) : 0;
      int32_t j0 = kByKeys ? x.row0 + tile0 * kKeys : p.c0 * kKeys;
      for (int c = 0; c < n; ++c, ++gc) {
        const int b = (int)(gc % kBufs);
        const int sbuf = (int)(gc % R::kStats);
        const float* st_l = stats + sbuf * 128 + half * 64;
        const float* st_d = st_l + R::kStats * 128;
        if (kByKeys) mbar_wait_fast(&ctl.st_full[sbuf], (uint32_t)((gc / R::kStats) & 1), abort_flag);
        mbar_wait_fast(&ctl.s_done[b], (uint32_t)((gc / kBufs) & 1), abort_flag);
        tc_fence_after();
        float w[64];
#pragma unroll
        for (int k = 0; k < 64; k += 16) {
          float v[16];
          tmem_ld16(lane_addr + b * 128 + half * 64 + k, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) w[k + i] = v[i];
        }
        tmem_wait_ld();
        if (kBufs == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_leader<2>(&ctl.s_free);
        }
        // columns lo .. hi-1 of this thread's 64 count
        int lo = 0, hi = 64;
        bool cut = j0 + kKeys > seg_n;
        if (kByKeys) {
          cut |= j0 < edge;
          lo = own - j0 - half * 64;
          hi = min(64, seg_n - j0 - half * 64);
        } else {
          cut |= j0 + kKeys - 1 > edge;
          hi = own - j0 - half * 64 + 1;
        }
#pragma unroll
        for (int k = 0; k < 64; k += 4) {
          float4 l = make_float4(lse2, lse2, lse2, lse2);
          if (kByKeys) l = *reinterpret_cast<const float4*>(st_l + k);
          w[k] = ex2_approx(fmaf(w[k], tau2, -l.x));
          w[k + 1] = ex2_approx(fmaf(w[k + 1], tau2, -l.y));
          w[k + 2] = ex2_approx(fmaf(w[k + 2], tau2, -l.z));
          w[k + 3] = ex2_approx(fmaf(w[k + 3], tau2, -l.w));
        }
        uint32_t dst = lane_addr + b * 128 + half * 64;
        if (M == kDv) {
          if (cut) {
#pragma unroll
            for (int i = 0; i < 64; ++i) w[i] = (i >= lo && i < hi) ? w[i] : 0.f;
          }
        } else {
          dst = lane_addr + kTmemP + half * 64;
          mbar_wait_fast(&ctl.dp_done, (uint32_t)(gc & 1), abort_flag);
          tc_fence_after();
          // Delta from the row's own P and dP, for rows without keys in later chunks.  (edge:
          // of the CTA, so that both warps of a row meet here.)
          if (M == kDq && j0 == 0 && edge < kKeys) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 64; k += 16) {
              float v[16];
              tmem_ld16(dst + k, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) sum += k + i < hi ? w[k + i] * v[i] : 0.f;
            }
            stats[half * 128 + li] = sum;
            named_bar_sync(1 + quad, 64);
            if (own < kKeys) {
              delta = stats[li] + stats[128 + li];
              if (active && half == 0) a.delta[sat] = delta;
            }
            named_bar_sync(1 + quad, 64);            // read before the next unit's sums
          }
          float v[4][16];                            // one wait for all: dS is what the next products wait for
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld16(dst + 16 * k, v[k]);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            float4 d = make_float4(delta, delta, delta, delta);
            if (kByKeys) d = *reinterpret_cast<const float4*>(st_d + i);
            w[i] *= v[i >> 4][i & 15] - d.x;
            w[i + 1] *= v[i >> 4][(i & 15) + 1] - d.y;
            w[i + 2] *= v[i >> 4][(i & 15) + 2] - d.z;
            w[i + 3] *= v[i >> 4][(i & 15) + 3] - d.w;
          }
          if (cut) {
#pragma unroll
            for (int i = 0; i < 64; ++i) w[i] = (i >= lo && i < hi) ? w[i] : 0.f;
          }
        }
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = pack_bf16x2(w[k + 2 * i], w[k + 2 * i + 1]);
          tmem_st16u(dst + k / 2, pk);
        }
        tmem_wait_st();
        const bool clear = j0 + kKeys > seg_n;
        mbar_wait_fast(&ctl.d_full[gc % R::kN2], (uint32_t)((gc / R::kN2) & 1), abort_flag);
        if (clear) clear_tail(j0);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_leader<2>(&ctl.w_full[b], clear);
          if (kByKeys) mbar_arrive(&ctl.st_free[sbuf]);
        }
        if (!kByKeys || --left == 0) {
          j0 += kKeys;
          left = t.hpg;
        }
      }
      more = next_of(p_next, x_next);
      mbar_wait_fast(&ctl.o_full, (uint32_t)(uc & 1), abort_flag);
      tc_fence_after();
      const bool whole = p.part < 0;
      const float f = whole && M != kDv ? a.scale : 1.f;
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
          tmem_ld16(lane_addr + kTmemD + half * 128 + piece * 32 + k, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) o[k + i] = v[i];
        }
        tmem_wait_ld();
        store_cols32(o, f, whole ? a.out : nullptr, part_q, at_q, half * 128 + piece * 32, lane);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_leader<2>(&ctl.o_free);
      ++uc;
    }
  }
  tc_fence_before();
  cluster_sync_all();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_cg<2>(tmem, dense_tc::kTmemCols);
  }
  dense_wait_last(a.late);
}

// Row statistics for the gradient kernels, a block per 4 tokens (a segment's
// tokens rounded up to 128): delta = dout . o, by token for the CUDA-core kernel
// and, with lse in log2 units, by head and statistics row for the tensor-core
// kernels; rows behind a segment's end get lse +inf (P = 0).  The block's flag: an
// lse, delta, key or value of its tokens is not finite.  A warp takes a head's four
// rows at once and reduces them together (6 exchanges instead of 20); bound by the
// HBM read of o and dout.
__global__ void __launch_bounds__(256)
    dense_stats_kernel(const __grid_constant__ SegTable st, const __nv_bfloat16* o, const __nv_bfloat16* dout,
                       const float* lse, const __nv_bfloat16* k, const __nv_bfloat16* v, float* delta, float* lse2_h,
                       float* delta_h, uint8_t* flags, int64_t stat_rows, int H, int G) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item0 = (int)blockIdx.x * 4;
  const int si = find_segment(st, item0);            // padded to 128: the four tokens are of one segment
  const int j0 = item0 - st.item0[si], left = st.q_len[si] - j0;
  const int64_t tok0 = (int64_t)st.q_offset[si] + j0;
  const int64_t stat0 = (int64_t)st.slot[si] * dense_bwd::kStatTile + j0;
  const int mine = ((lane >> 4) & 1) + ((lane >> 2) & 2);      // the token whose sum this lane's group of 8 ends with
  bool bad = false;
  for (int h = warp; h < H + G; h += 8) {
    const bool is_kv = h >= H;
    const int64_t ld = (int64_t)(is_kv ? G : H) * kHeadDim;
    const int64_t at = tok0 * ld + (int64_t)(is_kv ? h - H : h) * kHeadDim + lane * 8;
    const __nv_bfloat16* pa = (is_kv ? k : o) + at;
    const __nv_bfloat16* pb = (is_kv ? v : dout) + at;
    Vec8<__nv_bfloat16> a[4], b[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      a[q].x = b[q].x = make_uint4(0, 0, 0, 0);
      if (q < left) {
        a[q].load(pa + q * ld);
        b[q].load(pb + q * ld);
      }
    }
    if (is_kv) {                                     // an exponent of all ones carries into the sign bit
      uint32_t c = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t u[8] = {a[q].x.x, a[q].x.y, a[q].x.z, a[q].x.w, b[q].x.x, b[q].x.y, b[q].x.z, b[q].x.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) c |= (u[e] & 0x7f807f80u) + 0x00800080u;
      }
      bad |= (c & 0x80008000u) != 0;
      continue;
    }
    const float l = mine < left ? lse[(tok0 + mine) * H + h] : 0.f;
    float s[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float fa[8], fb[8];
      a[q].get(fa);
      b[q].get(fb);
      s[q] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s[q] = fmaf(fa[e], fb[e], s[q]);
    }
    const bool up = lane & 16, up8 = lane & 8;
    const float s01 = (up ? s[1] : s[0]) + __shfl_xor_sync(0xffffffffu, up ? s[0] : s[1], 16);
    const float s23 = (up ? s[3] : s[2]) + __shfl_xor_sync(0xffffffffu, up ? s[2] : s[3], 16);
    float d = (up8 ? s23 : s01) + __shfl_xor_sync(0xffffffffu, up8 ? s01 : s23, 8);
#pragma unroll
    for (int off = 4; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
    bad |= !isfinite(d) || !isfinite(l);
    if ((lane & 7) == 0) {
      if (mine < left) delta[(tok0 + mine) * H + h] = d;
      lse2_h[h * stat_rows + stat0 + mine] = mine < left ? l * 1.4426950408889634f : INFINITY;
      delta_h[h * stat_rows + stat0 + mine] = d;
    }
  }
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) flags[stat0 / 4] = any != 0;
}

}  // namespace qsa
