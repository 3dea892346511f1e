// tcgen05 latent attention of trees of drafted tokens (tree.cuh has the rule
// of visibility, mla_draft.h the formulas; bf16 layers, entries 512 + 64).
//
// Work unit: 128 consecutive rows (node, head) of a block, over a range of its
// keys in tiles of 128, by a cluster of two CTAs, one per half of the 512 value
// dims: a 128 x 512 fp32 accumulator alone would fill an SM's tensor memory,
// so each CTA keeps O for 256 dims and computes the 576-wide scores itself
// (3328 tensor cycles a tile instead of 2176: at most 65% of the peak on the
// algorithm's flops).
//
// What a tile costs beyond its MMAs is hidden by running the scores one tile
// ahead: the tensor pipe executes S(0), S(1), PV(0), S(2), PV(1), ..., and
// softmax(t) has PV(t - 1) and S(t + 1) to finish in.  That needs S free as
// soon as the softmax has read it, so P has tensor memory of its own (O 256
// columns, S 128, P 64, two of the nine Q chunks 64) and every operand streams:
// the cache chunks that a CTA reads as values come a second time for PV, from
// L2.  The stream of a CTA is, per tile, four pairs of 64-dim key chunks and two
// pairs of value chunks, through a ring of three 32 KB slots, each refilled by
// a warp of its own (a copy holds its thread for about 550 cycles), and the
// 16 KB rope chunk in a slot of its own, read last.
//
// Softmax: warps 0-3 and 8-11, two threads a row (64 keys and 128 value
// columns each) that exchange their half maxima; fp32, exp2 domain, O rescaled
// only when the running maximum grows by more than 2^8.  P is rounded to bf16
// as it meets the bf16 values (one kind::f16 MMA takes one type; its sum keeps
// the unrounded weights).  Tiles wholly inside the context need no mask without
// a window; the others test 64 bits a thread (tree::key_bits).  Entries that
// no row of the unit sees may hold anything: their scores are masked, and the
// refilling warp clears their rows of the value chunks before PV reads them.
//
// When the units do not fill the GPU their key range is cut in `splits` parts
// (grid y); a part writes its normalised rows in fp32 and their log2-sum-exp to
// the workspace and tree_merge_kernel joins them in split order.
#include "tree_tc.cuh"

#include <math.h>

#include <mutex>

#include "gemm_tc.cuh"
#include "tc_ptx.cuh"

namespace mla {
namespace tc {
namespace {

constexpr int QROWS = 128, KT = 128, NCH = 9;
constexpr int CH_BYTES = 128 * 64 * 2;                    // a 64-dim chunk of 128 rows
constexpr int NQT = 2, NQS = NCH - NQT;                   // Q chunks in tensor / shared memory
constexpr int SLOTS = 3, SLOT_BYTES = 2 * CH_BYTES;
constexpr int THREADS = 416;                              // softmax x4, MMA, ring x3, softmax x4, Q and rope
constexpr int W_MMA = 4, W_RING = 5, W_ROPE = 12;
constexpr int OFF_Q = 0, OFF_RING = OFF_Q + NQS * CH_BYTES, OFF_ROPE = OFF_RING + SLOTS * SLOT_BYTES;
constexpr int OFF_BAR = OFF_ROPE + CH_BYTES, OFF_SEEN = OFF_BAR + 256, OFF_XM = OFF_SEEN + tree::MAX_NODES / 8;
constexpr int SMEM_BYTES = 1024 + OFF_XM + 2 * QROWS * 4;
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr uint32_t TMEM_COLS = 512, TM_O = 0, TM_S = 256, TM_P = 384, TM_Q = 448;
constexpr float RESCALE_LOG2 = 8.f, kLn2 = 0.6931471805599453f;

struct Bars {
  uint64_t q_full, q_tmem;            // Q in shared memory (TMA) / in tensor memory
  uint64_t full[SLOTS], empty[SLOTS], clean[SLOTS];
  uint64_t rope_full, rope_empty;
  uint64_t s_full, s_free;            // S(t) complete / read
  uint64_t p_full, o_done;            // P(t) written / P(t) V(t) complete
  uint64_t drain;
  uint32_t tmem_slot;
  int abort, z_lo, any;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__device__ __forceinline__ bool wait_bar(Bars* B, uint64_t* bar, uint32_t parity, uint32_t* st) {
  if (*(volatile int*)&B->abort) return false;
  if (mbar_wait(bar, parity, st)) return true;
  B->abort = 1;
  return false;
}
// 2^x by the hardware approximation (relative error about 2^-22); 2^-inf = 0.
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The 64 threads of a row group (warps w and w + 8).
__device__ __forceinline__ void pair_sync(int w) { asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory"); }

// What use u of the ring holds: keys (pair 0..3) or values (pair 0..1) of a tile.
struct Item {
  int tile, pair;
  bool value;
};
__device__ __forceinline__ Item item_of(int u, int nt) {
  if (u < 4) return Item{0, u, false};
  const int g = (u - 4) / 6, i = (u - 4) % 6;
  if (g < nt - 1) return i < 4 ? Item{g + 1, i, false} : Item{g, i - 4, true};
  return Item{nt - 1, i, true};
}

struct Unit {
  int b, qt, half, n, W, ctx, j_lo, nt, z_lo;
  long row0;
};

// Tiles whose value rows need clearing: those that reach the block's own keys
// or the end, and those that reach below the first key that a row sees.
__device__ __forceinline__ bool dirty_tile(const Unit& U, int t) {
  const int j0 = U.j_lo + t * KT;
  return j0 + KT > U.ctx || j0 < U.z_lo;
}

__device__ __forceinline__ void softmax_role(const TreeParams& P, Bars* B, uint8_t* smem, uint32_t tmem,
                                             const Unit& U) {
  const int r = threadIdx.x & (QROWS - 1), kh = threadIdx.x >= 256 ? 1 : 0, w = r / 32;
  constexpr int KH = KT / 2;
  const uint32_t lane_base = (uint32_t)(w * 32) << 16;
  float* xm = (float*)(smem + OFF_XM);                    // [2][128]
  const tree::Rule& R = P.rule;
  const int row_in_block = U.qt * QROWS + r;
  const bool live = row_in_block < R.T * R.H;
  const int node = live ? row_in_block / R.H : 0;
  const long m = (long)U.b * R.T + node;
  const int32_t* parent = R.parent + (long)U.b * R.T;
  const bool ok = live && U.n > 0 && (R.q_visible ? R.q_visible[m] != 0 : true) &&
                  tree::in_tree(R, parent, node, false);
  // rows that see nothing are computed like their neighbours and written as
  // zeros, so that they do not take a warp off the unmasked path
  const int lo = U.W > 0 ? max(0, R.positions[m] - U.W + 1) : 0;
  float mrun = -INFINITY, lsum = 0.f;
  if (U.nt > 0) {
    // Q dims 0..127 of this row -> tensor memory (bf16 pairs), 64 dims a thread
    const uint4* src = reinterpret_cast<const uint4*>(P.q_abs + (U.row0 + r) * 576 + 64 * kh);
    uint32_t q[32];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
      q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
    }
    tmem_st32_u(tmem + TM_Q + 32 * kh + lane_base, q);
    tc_fence_before();
    mbar_arrive(&B->q_tmem);
  }
  for (int t = 0; t < U.nt; ++t) {
    const int jh = U.j_lo + t * KT + KH * kh;             // first key of this thread's half
    float s[KH];
    wait_bar(B, &B->s_full, t & 1, P.rule.status);
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < KH; c += 32) tmem_ld32_nowait(tmem + TM_S + KH * kh + c + lane_base, s + c);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < KH; c += 32) tmem_reg_fence32(s + c);
    tc_fence_before();
    mbar_arrive(&B->s_free);                              // S(t + 1) may overwrite it
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (__all_sync(0xffffffffu, !ok || (jh >= lo && jh + KH <= U.ctx))) {
#pragma unroll
      for (int i = 0; i < KH; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
    } else {
      const unsigned long long vis = tree::key_bits(R, U.b, node, ok, U.n, U.W, U.ctx, jh);
      const uint32_t v0 = (uint32_t)vis, v1 = (uint32_t)(vis >> 32);
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        s[i] = ((i < 32 ? v0 >> i : v1 >> (i - 32)) & 1u) ? s[i] : -INFINITY;
        mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
      }
    }
    // the row's maximum from both halves, in the exp2 domain (the scale is positive)
    const float hmax = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
    xm[kh * QROWS + r] = hmax;
    pair_sync(w);
    const float tmax = fmaxf(hmax, xm[(1 - kh) * QROWS + r]) * P.scale_log2;
    pair_sync(w);                                         // both read before the next write
    const bool grow = tmax > mrun + RESCALE_LOG2;
    const float m_new = grow ? tmax : mrun;
    const float mref = m_new == -INFINITY ? 0.f : m_new;  // nothing seen so far: P = 0
    float ps4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KH; ++i) {
      s[i] = fast_exp2(fmaf(s[i], P.scale_log2, -mref));
      ps4[i & 3] += s[i];
    }
    const float alpha = (grow && mrun != -INFINITY) ? exp2f(mrun - m_new) : 1.f;
    lsum = lsum * alpha + ((ps4[0] + ps4[1]) + (ps4[2] + ps4[3]));
    mrun = m_new;
    uint32_t pw[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      __nv_bfloat162 h2 = __floats2bfloat162_rn(s[2 * i], s[2 * i + 1]);
      pw[i] = *reinterpret_cast<uint32_t*>(&h2);
    }
    // P(t - 1) V(t - 1) is done with P and O
    if (t > 0) {
      wait_bar(B, &B->o_done, (t - 1) & 1, P.rule.status);
      tc_fence_after();
      if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
        for (int c = 128 * kh; c < 128 * kh + 128; c += 32) {
          float o[32];
          tmem_ld32(tmem + TM_O + lane_base + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= alpha;
          tmem_st32(tmem + TM_O + lane_base + c, o);
        }
      }
    }
    tmem_st32_u(tmem + TM_P + 32 * kh + lane_base, pw);
    tc_fence_before();
    mbar_arrive(&B->p_full);
  }
  // the row sum from both halves
  xm[kh * QROWS + r] = lsum;
  pair_sync(w);
  lsum += xm[(1 - kh) * QROWS + r];
  if (U.nt > 0) wait_bar(B, &B->o_done, (U.nt - 1) & 1, P.rule.status);
  tc_fence_after();
  const bool any = ok && U.nt > 0 && lsum > 0.f;
  const float inv = any ? 1.f / lsum : 0.f;
  const int col = U.half * 256 + 128 * kh;
  const long row = U.row0 + r;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float o[32];
    if (U.nt > 0) tmem_ld32(tmem + TM_O + lane_base + 128 * kh + c, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] = any ? o[i] * inv : 0.f;
    if (!live) continue;
    if (P.splits == 1) {
      uint4* dst = reinterpret_cast<uint4*>(P.o_lat + row * 512 + col + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __half2 h2[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) h2[k] = __floats2half2_rn(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
        dst[i] = *reinterpret_cast<uint4*>(h2);
      }
    } else if (any) {
      float4* dst = reinterpret_cast<float4*>(P.part + ((long)blockIdx.y * P.rows + row) * 512 + col + c);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
    }
  }
  if (!live || U.half || kh) return;
  const float l2 = any ? mrun + log2f(lsum) : -INFINITY;
  if (P.splits == 1) {
    if (P.lse) P.lse[row] = any ? l2 * kLn2 : -INFINITY;
  } else {
    P.part_lse[(long)blockIdx.y * P.rows + row] = l2;
  }
  if (P.vis_stats && blockIdx.y == 0 && row_in_block % R.H == 0) {
    int cnt = 0, first = -1, last = -1;
    if (ok) {
      if (lo < U.ctx) { cnt = U.ctx - lo; first = lo; last = U.ctx - 1; }
      const int32_t* pos = R.positions + (long)U.b * R.T;
      int low = -1, high = -1;
      for (int k = node; k >= 0; k = parent[k])
        if (U.W == 0 || pos[node] - pos[k] < U.W) {
          ++cnt;
          low = k;
          high = max(high, k);
        }
      if (high >= 0) {
        if (first < 0) first = U.ctx + low;
        last = U.ctx + high;
      }
    }
    P.vis_stats[m * 3 + 0] = cnt;
    P.vis_stats[m * 3 + 1] = first;
    P.vis_stats[m * 3 + 2] = last;
  }
}

__global__ void __launch_bounds__(THREADS, 1) tree_attn_tc_kernel(const __grid_constant__ TreeParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Bars* B = (Bars*)(smem + OFF_BAR);
  uint32_t* seen = (uint32_t*)(smem + OFF_SEEN);         // nodes that a row of this unit sees
  const tree::Rule& R = P.rule;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int unit = blockIdx.x >> 1;
  Unit U;
  U.half = blockIdx.x & 1;
  U.b = unit / P.tiles_per_block;
  U.qt = unit % P.tiles_per_block;
  U.row0 = ((long)U.b * R.T) * R.H + (long)U.qt * QROWS;

  if (tid == 0) {
    mbar_init(&B->q_full, 1);
    mbar_init(&B->q_tmem, 2 * QROWS);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
      mbar_init(&B->clean[i], 1);
    }
    mbar_init(&B->rope_full, 1);
    mbar_init(&B->rope_empty, 1);
    mbar_init(&B->s_full, 1);
    mbar_init(&B->s_free, 2 * QROWS);
    mbar_init(&B->p_full, 2 * QROWS);
    mbar_init(&B->o_done, 1);
    mbar_init(&B->drain, 1);
    B->abort = 0;
    B->z_lo = 0x7fffffff;
    B->any = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) tmem_alloc(&B->tmem_slot, TMEM_COLS);
  for (int i = tid; i < tree::MAX_NODES / 32; i += THREADS) seen[i] = 0;
  if (tid == 0) pdl_trigger();
  pdl_wait();                  // Q_abs and the nodes' own entries come from the kernels before
  U.n = tree::block_keys(R, U.b, &U.W, &U.ctx, tid == 0 && U.half == 0 && U.qt == 0 && blockIdx.y == 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_slot;
  // what the unit's rows see: the first context key and the nodes on their paths
  {
    const int t0 = U.qt * QROWS / R.H, t1 = min(R.T - 1, (U.qt * QROWS + QROWS - 1) / R.H);
    const int32_t* parent = R.parent + (long)U.b * R.T;
    const int32_t* pos = R.positions + (long)U.b * R.T;
    for (int i = t0 + tid; i <= t1; i += THREADS) {
      if (U.n <= 0 || (R.q_visible && !R.q_visible[(long)U.b * R.T + i])) continue;
      if (!tree::in_tree(R, parent, i, U.half == 0 && blockIdx.y == 0)) continue;
      B->any = 1;
      atomicMin(&B->z_lo, U.W > 0 ? max(0, min(pos[i] - U.W + 1, U.ctx)) : 0);
      for (int k = i; k >= 0; k = parent[k])
        if (U.W == 0 || pos[i] - pos[k] < U.W) atomicOr(&seen[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    U.z_lo = B->any ? B->z_lo : 0;
    U.j_lo = U.z_lo / KT * KT;
    const int all = B->any ? (U.n - U.j_lo + KT - 1) / KT : 0;
    const int tb = (int)((long)blockIdx.y * all / P.splits), te = (int)((long)(blockIdx.y + 1) * all / P.splits);
    U.j_lo += tb * KT;
    U.nt = te - tb;
  }

  if (warp >= W_RING && warp < W_RING + SLOTS) {
    // ---- ring slot `s`: uses s, s + 3, ... ----
    const int s = warp - W_RING;
    const int ps = R.page_size, past_end = R.num_pages * ps, seg = P.seg_rows, nseg = KT / seg;
    uint8_t* slot = smem + OFF_RING + s * SLOT_BYTES;
    if (lane == 0) { prefetch_tmap(&P.tmC); prefetch_tmap(&P.tmK); }
    int k = 0;
    for (int u = s; u < 6 * U.nt; u += SLOTS, ++k) {
      const Item it = item_of(u, U.nt);
      const int j0 = U.j_lo + it.tile * KT;
      const int ch = it.value ? 4 * U.half + 2 * it.pair : 2 * it.pair;
      // cache row of this lane's page segment (past the end: the copy fills zeros)
      int y = past_end;
      if (lane < nseg && j0 + lane * seg < U.n) {
        const int j = j0 + lane * seg;
        const int pg = R.block_table[(long)U.b * R.max_pages + j / ps];
        if (pg >= 0 && pg < R.num_pages) y = pg * ps + j % ps;
        else set_status(R.status, MLA_DEV_BAD_PAGE);
      }
      if (!wait_bar(B, &B->empty[s], (k & 1) ^ 1, R.status)) break;
      if (nseg == 1) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&B->full[s], SLOT_BYTES);
          tma_load_3d(slot, &P.tmC, &B->full[s], 0, y, ch);
        }
      } else {
        if (lane == 0) mbar_arrive_expect_tx(&B->full[s], SLOT_BYTES);
        __syncwarp();
        if (lane < nseg) {
          tma_load_3d(slot + lane * seg * 128, &P.tmK, &B->full[s], ch * 64, y, 0);
          tma_load_3d(slot + CH_BYTES + lane * seg * 128, &P.tmK, &B->full[s], ch * 64 + 64, y, 0);
        }
      }
      __syncwarp();
      if (it.value && dirty_tile(U, it.tile)) {
        // rows nobody sees become zeros: 0 x NaN is not 0
        if (!wait_bar(B, &B->full[s], k & 1, R.status)) { ++k; break; }
        for (int key = lane; key < KT; key += 32) {
          const int j = j0 + key, node = j - U.ctx;
          const bool need = j < U.n && j >= U.z_lo && (node < 0 || ((seen[node >> 5] >> (node & 31)) & 1u));
          if (!need) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              *reinterpret_cast<uint4*>(slot + key * 128 + q * 16) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(slot + CH_BYTES + key * 128 + q * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->clean[s]);
      }
    }
    // every copy into this CTA has landed before it may exit
    if (k > 0) mbar_wait(&B->full[s], (k - 1) & 1, R.status);
  } else if (warp == W_ROPE) {
    // ---- Q once, then the rope chunk of every tile ----
    if (U.nt > 0) {
      const int ps = R.page_size, past_end = R.num_pages * ps, seg = P.seg_rows, nseg = KT / seg;
      if (lane == 0) {
        prefetch_tmap(&P.tmQ);
        mbar_arrive_expect_tx(&B->q_full, NQS * CH_BYTES);
        tma_load_3d(smem + OFF_Q, &P.tmQ, &B->q_full, 0, (int)U.row0, NQT);
      }
      __syncwarp();
      int t = 0;
      for (; t < U.nt; ++t) {
        int y = past_end;
        const int j = U.j_lo + t * KT + lane * seg;
        if (lane < nseg && j < U.n) {
          const int pg = R.block_table[(long)U.b * R.max_pages + j / ps];
          if (pg >= 0 && pg < R.num_pages) y = pg * ps + j % ps;
        }
        if (!wait_bar(B, &B->rope_empty, (t & 1) ^ 1, R.status)) break;
        if (lane == 0) mbar_arrive_expect_tx(&B->rope_full, CH_BYTES);
        __syncwarp();
        if (lane < nseg)
          tma_load_3d(smem + OFF_ROPE + lane * seg * 128, &P.tmK, &B->rope_full, 512, y, 0);
        __syncwarp();
      }
      mbar_wait(&B->q_full, 0, R.status);
      if (t > 0) mbar_wait(&B->rope_full, (t - 1) & 1, R.status);
    }
  } else if (warp == W_MMA) {
    if (lane == 0 && U.nt > 0) {
      const uint32_t idesc_qk = idesc_f16(QROWS, KT, false), idesc_pv = idesc_f16_bmn(QROWS, 128, false);
      constexpr uint64_t U_CH = CH_BYTES / 16, U_SLOT = SLOT_BYTES / 16, U_KSTEP = 16 * 128 / 16;
      const uint64_t dQ = smem_desc_sw128(smem + OFF_Q), dR = smem_desc_sw128(smem + OFF_RING);
      const uint64_t dRope = smem_desc_sw128(smem + OFF_ROPE);
      const uint64_t dV = smem_desc_sw128_mn(smem + OFF_RING, CH_BYTES);
      const uint32_t tS = tmem + TM_S, tQ = tmem + TM_Q, tO = tmem + TM_O, tP = tmem + TM_P;
      int s = 0;                                          // slot of the next use of the ring
      uint32_t par = 0, cpar = 0;                         // its parity; bit i: parity of clean[i]
      bool ok = wait_bar(B, &B->q_full, 0, R.status) && wait_bar(B, &B->q_tmem, 0, R.status);
      auto next = [&]() { if (++s == SLOTS) { s = 0; par ^= 1; } };
      auto scores = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!ok || !(ok = wait_bar(B, &B->full[s], par, R.status))) return;
          tc_fence_after();
          const uint64_t db = dR + s * U_SLOT;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              if (i == 0)
                mma_f16_ts(tS, tQ + 32 * c + 8 * d, db + c * U_CH + 2 * d, idesc_qk, (c | d) ? 1u : 0u);
              else
                mma_f16(tS, dQ + (2 * i - 2 + c) * U_CH + 2 * d, db + c * U_CH + 2 * d, idesc_qk, 1u);
            }
          mma_commit(&B->empty[s]);
          next();
        }
        if (!(ok = wait_bar(B, &B->rope_full, t & 1, R.status))) return;
        tc_fence_after();
#pragma unroll
        for (int d = 0; d < 4; ++d) mma_f16(tS, dQ + (NQS - 1) * U_CH + 2 * d, dRope + 2 * d, idesc_qk, 1u);
        mma_commit(&B->rope_empty);
        mma_commit(&B->s_full);
      };
      scores(0);
      for (int t = 0; t < U.nt && ok; ++t) {
        if (t + 1 < U.nt) {
          if (!(ok = wait_bar(B, &B->s_free, t & 1, R.status))) break;
          tc_fence_after();
          scores(t + 1);
          if (!ok) break;
        }
        if (!(ok = wait_bar(B, &B->p_full, t & 1, R.status))) break;
        tc_fence_after();
        const bool dirty = dirty_tile(U, t);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (dirty) {
            ok = ok && wait_bar(B, &B->clean[s], (cpar >> s) & 1, R.status);
            cpar ^= 1u << s;
          }
          if (!ok || !(ok = wait_bar(B, &B->full[s], par, R.status))) break;
          tc_fence_after();
          const uint64_t db = dV + s * U_SLOT;
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_f16_ts(tO + 128 * p, tP + 8 * k, db + U_KSTEP * k, idesc_pv, (t | k) ? 1u : 0u);
          mma_commit(&B->empty[s]);
          next();
        }
        mma_commit(&B->o_done);
      }
      mma_commit(&B->drain);
      mbar_wait(&B->drain, 0, R.status);
    }
  } else {
    softmax_role(P, B, smem, tmem, U);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc(tmem, TMEM_COLS);
}

// One warp per row: sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s - max), in
// split order; a row that no split saw is zero.
__global__ void __launch_bounds__(256) tree_merge_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ part_lse, long rows,
                                                         int splits, __half* __restrict__ o_lat,
                                                         float* __restrict__ lse) {
  pdl_wait();
  const long row = (long)blockIdx.x * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  float mx = -INFINITY;
  for (int s = 0; s < splits; ++s) mx = fmaxf(mx, part_lse[s * rows + row]);
  float acc[16], den = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  if (mx != -INFINITY) {
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float l = part_lse[s * rows + row];
      if (l == -INFINITY) continue;                      // nothing was written for it
      const float w = exp2f(l - mx);
      den += w;
      const float4* src = reinterpret_cast<const float4*>(part + (s * rows + row) * 512) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[32 * i];
        acc[4 * i] += w * v.x; acc[4 * i + 1] += w * v.y; acc[4 * i + 2] += w * v.z; acc[4 * i + 3] += w * v.w;
      }
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 h2[2] = {__floats2half2_rn(acc[4 * i] * inv, acc[4 * i + 1] * inv),
                     __floats2half2_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv)};
    *reinterpret_cast<uint2*>(o_lat + row * 512 + 128 * i + 4 * lane) = *reinterpret_cast<uint2*>(h2);
  }
  if (lse && lane == 0) lse[row] = den > 0.f ? (mx + log2f(den)) * kLn2 : -INFINITY;
}

}  // namespace

// Parts of a unit's key range.  Cost in tiles: the waves of CTA pairs that one
// split count needs, each of FIXED tiles' time beyond its share of the keys, and
// the merge.  Keys are bounded by the page table; shorter sequences only split
// finer than they need.
int tree_splits(const mla_handle* h, const mla_attn_desc_t& d) {
  constexpr double FIXED = 5.0, MERGE = 4.0, MERGE_PART = 0.02;
  const long units = (long)d.num_blocks * (((long)d.block_len * h->lay.H + QROWS - 1) / QROWS);
  const long tiles = ((long)d.max_pages * h->cfg.page_size + KT - 1) / KT, pairs = h->num_sms / 2;
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= 64 && s <= tiles; ++s) {
    const double waves = (double)((units * s + pairs - 1) / pairs);
    const double c = waves * (FIXED + (double)((tiles + s - 1) / s)) +
                     (s > 1 ? MERGE + MERGE_PART * units * s : 0.0);
    if (c < cost) { cost = c; best = s; }
    if (units * s > 8 * pairs) break;
  }
  return best;
}

size_t tree_attention_ws(const mla_handle* h, const mla_attn_desc_t& d) {
  const int s = tree_splits(h, d);
  if (s == 1) return 0;
  const long rows = (long)d.num_blocks * d.block_len * h->lay.H;
  return align256((size_t)s * rows * 512 * 4) + align256((size_t)s * rows * 4);
}

mla_status_t tree_attention(cudaStream_t st, mla_handle* h, const tree::Rule& r,
                            const mla_attn_desc_t& d, const __nv_bfloat16* q_abs,
                            const __nv_bfloat16* cache, __half* o_lat, float* lse, void* ws, bool pdl) {
  const Layout& l = h->lay;
  const long rows = (long)d.num_blocks * d.block_len * l.H, slots = (long)r.num_pages * r.page_size;
  if (slots > 0x7fffffffL) return fail(MLA_ERR_UNSUPPORTED, "tree attention: num_pages * page_size < 2^31");
  TreeParams P;
  P.seg_rows = r.page_size < KT ? r.page_size : KT;
  if (!make_tmap_chunked(&P.tmQ, false, q_abs, rows, l.L, l.L, QROWS, NQS) ||
      !make_tmap_chunked(&P.tmC, false, cache, slots, l.L, l.L, KT, 2) ||
      !make_tmap_2d(&P.tmK, false, cache, slots, l.L, l.L, P.seg_rows))
    return fail(MLA_ERR_CUDA, "tree attention: cuTensorMapEncodeTiled failed");
  P.rule = r;
  P.q_abs = q_abs;
  P.o_lat = o_lat;
  P.lse = lse;
  P.vis_stats = d.vis_stats;
  P.rows = rows;
  P.splits = tree_splits(h, d);
  P.part = (float*)ws;
  P.part_lse = P.splits > 1 ? (float*)((char*)ws + align256((size_t)P.splits * rows * 512 * 4)) : nullptr;
  P.tiles_per_block = (int)(((long)d.block_len * l.H + QROWS - 1) / QROWS);
  P.scale_log2 = h->scale * 1.4426950408889634f;
  const long units = (long)d.num_blocks * P.tiles_per_block;
  if (units > 0x3fffffffL) return fail(MLA_ERR_INVALID_ARG, "tree attention: too many rows");
  static std::once_flag once;
  std::call_once(once, [] {
    cudaFuncSetAttribute(tree_attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  Launch L(dim3((unsigned)(2 * units), (unsigned)P.splits), dim3(THREADS), SMEM_BYTES, st, pdl, dim3(2, 1, 1));
  cudaError_t e = cudaLaunchKernelEx(&L.cfg, tree_attn_tc_kernel, P);
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  h->launches += 1;
  if (P.splits > 1) {
    Launch M(dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, st, false);
    e = cudaLaunchKernelEx(&M.cfg, tree_merge_kernel, (const float*)P.part, (const float*)P.part_lse, rows,
                           P.splits, o_lat, lse);
    if (e != cudaSuccess) return cuda_fail(e, "tree attention merge launch");
    h->launches += 1;
  }
  return MLA_OK;
}

}  // namespace tc
}  // namespace mla
