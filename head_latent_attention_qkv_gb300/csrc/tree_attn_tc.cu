// tcgen05 latent attention of trees of drafted tokens (tree.cuh has the rule
// of visibility, mla_draft.h the formulas; bf16 layers, entries 512 + 64).
//
// A 128 x 512 fp32 accumulator alone would fill an SM's tensor memory, so a
// CTA keeps O for 128 rows (node, head) and 256 of the value dims and computes
// the 576-wide scores of its rows itself: 3328 tensor cycles per tile of 128
// keys instead of 2176, at most 65% of the peak on the algorithm's flops.  A
// cluster works on one range of a block's keys:
//  - tree_attn_pair_kernel, blocks of more than 128 rows: two row tiles and one
//    value half; their MMAs run as one over the pair (cta_group::2), so each
//    CTA fetches and reads half of the keys' and values' bytes (2560 cycles of
//    shared-memory traffic a tile against 3328 of MMAs).  8192 rows x 6-8 k keys x
//    4 sequences: 457 us, 1.1 PFLOP/s on the algorithm's flops, at an SM clock of
//    2.07 GHz (462 at the 1.93 GHz of a second of such calls);
//  - tree_attn_tc_kernel, blocks of at most 128 rows: one row tile, a CTA per
//    value half (4224 cycles of shared-memory traffic a tile, and a slot's next
//    copy waits for P V, 2 k cycles from L2: 6 to 7 k cycles a tile).  Blocks of at
//    most 64 and 32 rows give the space of the rows that they lack to a fourth and
//    a fifth slot: 64 sequences x 32 rows x 4 k keys 127 us with three, 108 with
//    five; x 64 rows 127 and, with four, 114.
//
// What a tile costs beyond its MMAs is hidden by running the scores one tile
// ahead: the tensor pipe executes S(0), S(1), PV(0), S(2), PV(1), ..., and
// softmax(t) has PV(t - 1) and S(t + 1) to finish in.  That needs S free as
// soon as the softmax has read it, so P has tensor memory of its own (O 256
// columns, S 128, P 64, two of the nine Q chunks 64) and every operand streams:
// the cache chunks that a CTA reads as values come a second time for PV, from
// L2.  Per tile the stream has four pairs of 64-dim key chunks, two pairs of
// value chunks and the rope chunk.  Scores and P V are issued by two threads,
// and each looks at its next barrier before it issues the MMAs of the one at
// hand (a look takes 100 to 340 cycles, a commit 125, the eight MMAs of a pair
// 512, so barriers are shared where the operands allow it).  P V(t) is held back
// until S(t + 1) is in the pipe: it then fills the 1.1 k cycles until the softmax
// has read S(t + 1), instead of delaying it (5.7 k -> 4.9 k cycles a tile).
//
// A cluster's fixed cost is about 13 us (set-up, Q and the first keys, the first
// scores, the last P V, the join and the store), which is what small calls take.
//
// Softmax: warps 0-3 and 8-11, two threads a row (64 keys and 128 value
// columns each) that exchange their half maxima; fp32, exp2 domain, O rescaled
// only when the running maximum grows by more than 2^8.  P is rounded to bf16
// as it meets the bf16 values (one kind::f16 MMA takes one type; its sum keeps
// the unrounded weights).  Tiles wholly inside the context need no mask without
// a window; the others test 64 bits a thread (tree::key_bits).  Entries that
// no row of the cluster sees may hold anything: their scores are masked, and
// the refilling warps clear their rows of the value chunks before PV reads them.
//
// When the units do not fill the GPU their key range is cut in parts (grid y).
// Up to four neighbouring parts share a cluster and are joined through its
// shared memory; what is left of them writes its rows in fp32 and their
// log2-sum-exp to the workspace, and tree_merge_kernel joins them in order.
#include "tree_tc.cuh"

#include <math.h>
#include <stddef.h>

#include <mutex>

#include "gemm_tc.cuh"
#include "pair_ptx.cuh"

namespace mla {
namespace tc {
namespace {

constexpr int QROWS = 128, KT = 128, NCH = 9;
constexpr int CH_BYTES = 128 * 64 * 2;                    // a 64-dim chunk of 128 rows
constexpr int NQT = 2, NQS = NCH - NQT;                   // Q chunks in tensor / shared memory
constexpr int SLOT_BYTES = 2 * CH_BYTES, MAX_SLOTS = 5;
constexpr int THREADS = 448;                              // softmax x4, S, loads x3, softmax x4, PV, Q and rope
constexpr int W_S = 4, W_RING = 5, W_PV = 12, W_ROPE = 13;
constexpr int OFF_Q = 0, OFF_RING = OFF_Q + NQS * CH_BYTES, OFF_ROPE = OFF_RING + 3 * SLOT_BYTES;
constexpr int OFF_BAR = OFF_ROPE + CH_BYTES, OFF_SEEN = OFF_BAR + 320, OFF_XM = OFF_SEEN + tree::MAX_NODES / 8;
constexpr int SMEM_BYTES = 1024 + OFF_XM + 2 * QROWS * 4;
// the pair kernel's slots (a CTA's halves): four key pairs and two value pairs of 16 KB
constexpr int PK = 4, PV = 2, PSLOT_BYTES = CH_BYTES, OFF_PK = OFF_RING, OFF_PV = OFF_PK + PK * PSLOT_BYTES;
static_assert(OFF_PV + PV * PSLOT_BYTES <= OFF_ROPE, "slots");
static_assert(NQT == 2 && PV * PSLOT_BYTES == NQT * CH_BYTES && SLOT_BYTES == NQT * CH_BYTES, "Q's way through a slot");
// The other kernel, for blocks of up to QR rows: Q's chunks take QR rows each (the MMAs
// read 128; what follows them is scores of rows that do not exist), which leaves
// space for more slots, each with a warp of its own.
template <int QR>
struct Ring {
  static constexpr int SLOTS = QR == 128 ? 3 : QR == 64 ? 4 : 5, QCH = QR * 128;
  static constexpr int OFF_RING = OFF_Q + NQS * QCH, OFF_ROPE = OFF_RING + SLOTS * SLOT_BYTES;
  static constexpr int OFF_Q01 = OFF_RING + (SLOTS - 1) * SLOT_BYTES;       // Q passes through the last slot
  static constexpr int NT = THREADS + 32 * (SLOTS - 3);
  static_assert(SLOTS <= MAX_SLOTS && OFF_ROPE + CH_BYTES <= OFF_BAR, "ring");
};
// the epilogue's rows, over Q and the slots: fp32, 256 dims, padded against bank
// conflicts, then their log2-sum-exps
constexpr int STG_PITCH = 260, OFF_STG_LSE = QROWS * STG_PITCH * 4;
static_assert(OFF_STG_LSE + QROWS * 4 <= OFF_BAR, "staging");
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr uint32_t TMEM_COLS = 512, TM_O = 0, TM_S = 256, TM_P = 384, TM_Q = 448;
constexpr int MAX_PARTS = 64;                             // partials of a row that the merge joins
constexpr float RESCALE_LOG2 = 8.f, kLn2 = 0.6931471805599453f;

struct Bars {
  uint64_t q_full, q_tmem;            // Q in shared memory (TMA) / in tensor memory
  uint64_t q01_full, q01_read;        // its first two chunks, on their way through a value or ring slot
  // keys and values land on barriers of their own: each has one consumer, which
  // never falls two phases behind (a parity tells only two apart)
  uint64_t k_full[MAX_SLOTS], k_empty[MAX_SLOTS], v_full[MAX_SLOTS], clean[MAX_SLOTS], land;
  uint64_t rope_full;
  uint64_t s_full, s_free;            // S(t) complete (the rope chunk is free) / read
  uint64_t p_full, o_done;            // P(t) written / P(t) V(t) complete
  uint64_t seen_full;                 // z_lo and the nodes' bits are known
  uint64_t drain[2];
  uint32_t tmem_slot;
  int abort, z_lo;
  int issued;                         // tiles whose scores are in the tensor pipe
};
static_assert(sizeof(Bars) <= OFF_SEEN - OFF_BAR, "barrier block");

__device__ __forceinline__ bool wait_bar(Bars* B, uint64_t* bar, uint32_t parity, uint32_t* st,
                                         bool ready = false) {
  if (ready) return true;
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
// The 64 threads of a row group (warps w and w + 8), each warp converged.
__device__ __forceinline__ void pair_sync(int w) { asm volatile("bar.sync %0, 64;" ::"r"(1 + w) : "memory"); }

// What use u of the ring holds: keys (pair 0..3) or values (pair 0..1) of a
// tile.  The order is that of the tensor pipe: S(0), S(1), PV(0), S(2), ...
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
__device__ __forceinline__ int first_key_use(int t) { return t == 0 ? 0 : 6 * t - 2; }
__device__ __forceinline__ int first_value_use(int t, int nt) { return 6 * t + (t < nt - 1 ? 8 : 4); }

// Lets the scores of `tiles` tiles into the tensor pipe first: P V then fills
// the gap until the softmax has read them, instead of delaying them.  Only an
// order is at stake, so it gives up early.
__device__ __forceinline__ void behind_scores(Bars* B, int tiles) {
  for (int i = 0; i < 1024 && *(volatile int*)&B->issued < tiles; ++i) {}
}

struct Unit {
  int b, qt, half, n, W, ctx, j_lo, nt;
  int tiles;             // row tiles of the cluster: 1, or 2 (this CTA's and its peer's)
  uint32_t lead;         // rank of the CTA whose barriers the issuing threads wait on
  bool first;            // reports and statistics of the block's rows are this CTA's
  long row0;
};

// First key of the t-th tile.  The tiles run from the end of the range down:
// the ones whose value rows need clearing (the block's own keys) come first,
// while the pipeline fills.
__device__ __forceinline__ int tile_key(const Unit& U, int t) { return U.j_lo + (U.nt - 1 - t) * KT; }

// Tiles whose value rows need clearing: those that reach the block's own keys
// or the end, and those that reach below the first key that a row sees.
__device__ __forceinline__ bool dirty_tile(const Unit& U, int z_lo, int t) {
  const int j0 = tile_key(U, t);
  return j0 + KT > U.ctx || j0 < z_lo;
}

template <bool PAIR>
__device__ __forceinline__ void softmax_role(const TreeParams& P, Bars* B, uint8_t* smem, uint32_t tmem,
                                             const Unit& U, const uint8_t* q01, int q01_bytes) {
  const int r = threadIdx.x & (QROWS - 1), kh = threadIdx.x >= 256 ? 1 : 0, w = r / 32, lane = r % 32;
  constexpr int KH = KT / 2;
  const uint32_t lane_base = (uint32_t)(w * 32) << 16;
  float* xm = (float*)(smem + OFF_XM);                    // [2][128]
  const tree::Rule& R = P.rule;
  const int row_in_block = U.qt * QROWS + r;
  const bool live = row_in_block < R.T * R.H;
  const int node = live ? row_in_block / R.H : 0;
  const long m = (long)U.b * R.T + node;
  const int32_t* parent = R.parent + (long)U.b * R.T;
  const uint32_t s_free = mapa(smem_u32(&B->s_free), U.lead), p_full = mapa(smem_u32(&B->p_full), U.lead);
  if (U.nt > 0) {
    // Q dims 0..127 of this row -> tensor memory (bf16 pairs), 64 dims a thread,
    // by way of shared memory (row by row from global memory they took 2 us)
    uint32_t q[32];
    wait_bar(B, &B->q01_full, 0, P.rule.status);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(q01 + kh * q01_bytes + r * 128 + ((i ^ (r & 7)) * 16));
      q[4 * i] = v.x; q[4 * i + 1] = v.y; q[4 * i + 2] = v.z; q[4 * i + 3] = v.w;
    }
    mbar_arrive(&B->q01_read);
    tmem_st32_u(tmem + TM_Q + 32 * kh + lane_base, q);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(mapa(smem_u32(&B->q_tmem), U.lead));
  }
  // The walks over the tree run while the first scores are on their way.  Up to
  // 64 nodes fit one word, found in one walk: a row's first thread takes its
  // own node and its second the peer's (both CTAs of a pair need to know what
  // either's rows see); deeper trees walk again for every tile of nodes' keys.
  // Rows that see nothing are computed like their neighbours and written as
  // zeros, so that they do not take a warp off the unmasked path.
  const int lo = U.W > 0 ? tree::window_start(R.positions[m], U.W) : 0;
  float mrun = -INFINITY, lsum = 0.f;
  const bool small = R.T <= 64;
  unsigned long long mine = 0;                            // (small) the nodes that this row sees
  bool ok;
  {
    uint32_t* seen = (uint32_t*)(smem + OFF_SEEN);
    const int32_t* pos = R.positions + (long)U.b * R.T;
    const int other = (kh ? U.qt ^ 1 : U.qt) * QROWS + r, nd = other / R.H;
    const bool walks = kh < U.tiles && other < R.T * R.H && U.n > 0 &&
                       (R.q_visible ? R.q_visible[(long)U.b * R.T + nd] != 0 : true);
    const bool first_row = other % R.H == 0 || r == 0;     // one row of a node speaks for all
    bool sound = false;
    if (small) {
      if (walks) mine = tree::walk_bits(R, U.b, nd, U.W, 0, &sound, U.first && kh == 0);
      if (sound && first_row) {
        atomicOr(&seen[0], (uint32_t)mine);
        atomicOr(&seen[1], (uint32_t)(mine >> 32));
      }
      // through the row's own two places of xm: other rows' belong to other warps,
      // which may be in the loop already
      uint32_t* word = (uint32_t*)xm;
      if (!kh) {
        word[r] = (uint32_t)mine;
        word[QROWS + r] = (uint32_t)(mine >> 32);
      }
      __syncwarp();                                        // the walks may have parted the warp
      pair_sync(w);
      mine = word[r] | (unsigned long long)word[QROWS + r] << 32;
      pair_sync(w);
      ok = live && mine != 0;
    } else {
      sound = walks && tree::in_tree(R, parent, nd, U.first && kh == 0);
      if (sound && first_row)
        for (int k = nd; k >= 0; k = parent[k])
          if (U.W == 0 || pos[nd] - pos[k] < U.W) atomicOr(&seen[k >> 5], 1u << (k & 31));
      if (!kh) xm[r] = sound ? 1.f : 0.f;
      __syncwarp();
      pair_sync(w);
      ok = live && xm[r] != 0.f;
      pair_sync(w);
    }
    if (sound && first_row) atomicMin(&B->z_lo, U.W > 0 ? min(tree::window_start(pos[nd], U.W), U.ctx) : 0);
  }
  mbar_arrive(&B->seen_full);
  __syncwarp();
  // a warp without rows: its P stays undefined.  (Not in pairs, where it is rare and
  // the test alone made the loop of 128 heads x 64 nodes 2.5% slower)
  const bool dead = U.qt * QROWS + 32 * w >= R.T * R.H;
  for (int t = 0; t < U.nt; ++t) {
    const int jh = tile_key(U, t) + KH * kh;              // first key of this thread's half
    float s[KH];
    wait_bar(B, &B->s_full, t & 1, P.rule.status);
    if (!PAIR && dead) {
      if (lane == 0) mbar_arrive_pair(s_free);
      if (t > 0) wait_bar(B, &B->o_done, (t - 1) & 1, P.rule.status);   // (no phase of p_full ahead of the others)
      if (lane == 0) mbar_arrive_pair(p_full);
      __syncwarp();
      continue;
    }
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < KH; c += 32) tmem_ld32_nowait(tmem + TM_S + KH * kh + c + lane_base, s + c);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < KH; c += 32) tmem_reg_fence32(s + c);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(s_free);              // S(t + 1) may overwrite it
    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (__all_sync(0xffffffffu, !ok || (jh >= lo && jh + KH <= U.ctx))) {
#pragma unroll
      for (int i = 0; i < KH; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
    } else {
      const unsigned long long vis =
          !small ? tree::key_bits(R, U.b, node, ok, U.n, U.W, U.ctx, jh)
          : ok   ? tree::context_bits(R, U.b, node, U.n, U.W, U.ctx, jh) | tree::place_bits(mine, U.ctx, jh)
                 : 0ull;
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
    __syncwarp();
    if (lane == 0) mbar_arrive_pair(p_full);
  }
  // the row sum from both halves
  xm[kh * QROWS + r] = lsum;
  pair_sync(w);
  lsum += xm[(1 - kh) * QROWS + r];
  if (U.nt > 0) wait_bar(B, &B->o_done, (U.nt - 1) & 1, P.rule.status);
  tc_fence_after();
  const bool any = ok && U.nt > 0 && lsum != 0.f;         // (a NaN that a row sees reaches its output)
  const float inv = any ? 1.f / lsum : 0.f;
  float* prow = (float*)smem + r * STG_PITCH + 128 * kh;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float o[32];
    if (U.nt > 0) tmem_ld32(tmem + TM_O + lane_base + 128 * kh + c, o);
#pragma unroll
    for (int i = 0; i < 32; i += 4)
      *reinterpret_cast<float4*>(prow + c + i) =
          any ? make_float4(o[i] * inv, o[i + 1] * inv, o[i + 2] * inv, o[i + 3] * inv)
              : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (kh) return;
  ((float*)(smem + OFF_STG_LSE))[r] = any ? mrun + log2f(lsum) : -INFINITY;
  if (live && P.vis_stats && U.first && row_in_block % R.H == 0) {
    int cnt = 0, first = -1, last = -1;
    if (ok) {
      if (lo < U.ctx) { cnt = U.ctx - lo; first = lo; last = U.ctx - 1; }
      const int32_t* pos = R.positions + (long)U.b * R.T;
      int low = -1, high = -1;
      if (small) {
        cnt += __popcll(mine);
        low = __ffsll(mine) - 1;
        high = 63 - __clzll(mine);
      } else {
        for (int k = node; k >= 0; k = parent[k])
          if (U.W == 0 || pos[node] - pos[k] < U.W) {
            ++cnt;
            low = k;
            high = max(high, k);
          }
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

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}

// The staged rows of the cluster's parts, joined and written whole: part y of
// the cluster takes rows [128 y / CS, 128 (y + 1) / CS), a warp per row, 4 and
// 4 dims a lane (no bank conflicts), parts in order; a row that no part saw is zero.
template <int CS>
__device__ __forceinline__ void store_rows(const TreeParams& P, const uint8_t* smem, const Unit& U) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int rows = min(QROWS, P.rule.T * P.rule.H - U.qt * QROWS);
  const int y = CS > 1 ? (int)(blockIdx.y % CS) : 0, x = (int)(blockIdx.x & 1);
  const uint32_t stg = smem_u32(smem), lse_a = stg + OFF_STG_LSE;
#pragma unroll(CS == 4 ? 2 : 4)
  for (int r = y * (QROWS / CS) + warp; r < min(rows, (y + 1) * (QROWS / CS)); r += blockDim.x / 32) {
    float l[CS];
    float4 a[CS], c[CS];
#pragma unroll
    for (int s = 0; s < CS; ++s) {
      const uint32_t rank = (uint32_t)(x + 2 * s), at = stg + (uint32_t)(r * STG_PITCH + 4 * lane) * 4;
      if (CS == 1 || s == y) {                            // this CTA's own
        l[s] = ((const float*)(smem + OFF_STG_LSE))[r];
        a[s] = *(const float4*)((const float*)smem + r * STG_PITCH + 4 * lane);
        c[s] = *(const float4*)((const float*)smem + r * STG_PITCH + 4 * lane + 128);
      } else {
        l[s] = ld_cluster_f32(mapa(lse_a + 4 * r, rank));
        a[s] = ld_cluster_v4(mapa(at, rank));
        c[s] = ld_cluster_v4(mapa(at + 512, rank));
      }
    }
    float mx = l[0];
#pragma unroll
    for (int s = 1; s < CS; ++s) mx = fmaxf(mx, l[s]);
    float v[8] = {a[0].x, a[0].y, a[0].z, a[0].w, c[0].x, c[0].y, c[0].z, c[0].w}, l2 = l[0];
    if (CS > 1) {
      float den = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
      for (int s = 0; s < CS; ++s) {
        const float w = l[s] == -INFINITY ? 0.f : exp2f(l[s] - mx);
        den += w;
        v[0] += w * a[s].x; v[1] += w * a[s].y; v[2] += w * a[s].z; v[3] += w * a[s].w;
        v[4] += w * c[s].x; v[5] += w * c[s].y; v[6] += w * c[s].z; v[7] += w * c[s].w;
      }
      const float inv = den != 0.f ? 1.f / den : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= inv;
      l2 = den != 0.f ? mx + log2f(den) : -INFINITY;
    }
    const long row = U.row0 + r;
    const int parts = gridDim.y / CS;
    if (parts == 1) {
      __half2 h2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h2[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      uint2* dst = reinterpret_cast<uint2*>(P.o_lat + row * 512 + U.half * 256 + 4 * lane);
      dst[0] = *reinterpret_cast<uint2*>(h2);
      dst[32] = *reinterpret_cast<uint2*>(h2 + 2);
      if (P.lse && U.half == 0 && lane == 0) P.lse[row] = l2 == -INFINITY ? l2 : l2 * kLn2;
    } else {
      const long at = (long)(blockIdx.y / CS) * P.rows + row;
      float4* dst = reinterpret_cast<float4*>(P.part + at * 512 + U.half * 256 + 4 * lane);
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[32] = make_float4(v[4], v[5], v[6], v[7]);
      if (U.half == 0 && lane == 0) P.part_lse[at] = l2;
    }
  }
}
__device__ __forceinline__ void join_and_store(const TreeParams& P, const uint8_t* smem, const Unit& U) {
  if (P.cluster_parts == 1) store_rows<1>(P, smem, U);
  else if (P.cluster_parts == 2) store_rows<2>(P, smem, U);
  else store_rows<4>(P, smem, U);
}

// Barriers and, while the cluster meets, the unit's keys and this part's share
// of their tiles; every warp.
__device__ __forceinline__ void set_up(const TreeParams& P, Bars* B, uint8_t* smem, Unit& U) {
  const tree::Rule& R = P.rule;
  const int tid = threadIdx.x, lane = tid % 32;
  uint32_t* seen = (uint32_t*)(smem + OFF_SEEN);          // nodes that a row of the cluster sees
  // the loads that the unit depends on first, their answers (1.5 k cycles) after
  // the barriers are set: the block's length, and this lane's first node
  const int q0 = U.tiles == 2 ? U.qt & ~1 : U.qt;
  const int t0 = q0 * QROWS / R.H, t1 = min(R.T - 1, ((q0 + U.tiles) * QROWS - 1) / R.H);
  auto load_node = [&](int i, int* parent, int* pos, bool* shown) {
    const long m = (long)U.b * R.T + i;
    *parent = R.parent[m];
    *pos = R.positions[m];
    *shown = R.q_visible ? R.q_visible[m] != 0 : true;
  };
  int parent = -2, pos = 0;
  bool shown = false;
  if (t0 + lane <= t1) load_node(t0 + lane, &parent, &pos, &shown);
  const int kv_len = R.kv_len[U.b], window = R.window ? R.window[U.b] : 0;
  // a thread a barrier (one thread for all of them: about 1 k cycles)
  constexpr int NBAR = (int)(offsetof(Bars, tmem_slot) / 8);
  static_assert(NBAR <= THREADS, "a barrier a thread");
  if (tid < NBAR) {
    uint64_t* bar = (uint64_t*)B + tid;
    const uint32_t count = bar == &B->q_tmem || bar == &B->s_free || bar == &B->p_full ? 8 * U.tiles
                           : bar >= B->clean && bar < B->clean + MAX_SLOTS                  ? U.tiles
                           : bar == &B->seen_full || bar == &B->q01_read                ? 2 * QROWS
                                                                                         : 1;
    mbar_init(bar, count);
    fence_mbar_init();
  }
  if (tid == 32) {
    B->abort = 0;
    B->issued = 0;
    B->z_lo = 0x7fffffff;
    pdl_trigger();
  }
  for (int i = tid; i < tree::MAX_NODES / 32; i += THREADS) seen[i] = 0;
  tc_fence_before();           // (the tensor memory's address)
  __syncthreads();
  // the peers need the barriers only, which their own fence has published (a release
  // of everything took 800 cycles)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // whether a row may see anything (padding and masked rows left out), and the
  // first tile that a row's window reaches
  bool any = false;
  int pmin = 0x7fffffff;
  for (int i = t0 + lane; i <= t1; i += 32) {
    if (i >= t0 + 32) load_node(i, &parent, &pos, &shown);
    const bool in = parent >= -1 && shown;
    any |= in;
    if (in) pmin = min(pmin, pos);
  }
  U.W = window;
  U.n = tree::checked_keys(R, kv_len, &U.W, &U.ctx, tid == 0 && U.first && U.qt == 0);
  any = __any_sync(0xffffffffu, any);
  pmin = __reduce_min_sync(0xffffffffu, pmin);
  U.j_lo = U.W > 0 ? min(tree::window_start(pmin, U.W), U.ctx) / KT * KT : 0;
  const int all = any && U.n > 0 ? (U.n - U.j_lo + KT - 1) / KT : 0;
  const int tb = (int)((long)blockIdx.y * all / gridDim.y), te = (int)((long)(blockIdx.y + 1) * all / gridDim.y);
  U.j_lo += tb * KT;
  U.nt = te - tb;
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
}

// Cache row of logical key j (past the end of the keys or on a bad page: past
// the cache, where a copy reads zeros).
__device__ __forceinline__ int cache_row(const tree::Rule& R, const Unit& U, int j, bool report) {
  const int past_end = R.num_pages * R.page_size;
  if (j >= U.n) return past_end;
  const int pg = R.block_table[(long)U.b * R.max_pages + j / R.page_size];
  if (pg >= 0 && pg < R.num_pages) return pg * R.page_size + j % R.page_size;
  if (report) set_status(R.status, MLA_DEV_BAD_PAGE);
  return past_end;
}

// Clears the rows of `nch` value chunks whose keys nobody sees (0 x NaN is not
// 0); a warp.
__device__ __forceinline__ void clear_unseen(const Unit& U, const uint8_t* smem, uint8_t* chunks, int nch,
                                             int j0, int z_lo) {
  const uint32_t* seen = (const uint32_t*)(smem + OFF_SEEN);
  for (int key = threadIdx.x % 32; key < KT; key += 32) {
    const int j = j0 + key, node = j - U.ctx;
    if (j < U.n && j >= z_lo && (node < 0 || ((seen[node >> 5] >> (node & 31)) & 1u))) continue;
    for (int c = 0; c < nch; ++c)
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(chunks + c * CH_BYTES + key * 128 + q * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int QR>
__global__ void __launch_bounds__(Ring<QR>::NT, 1) tree_attn_tc_kernel(const __grid_constant__ TreeParams P) {
  using G = Ring<QR>;
  constexpr int SLOTS = G::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Bars* B = (Bars*)(smem + OFF_BAR);
  const tree::Rule& R = P.rule;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int unit = (int)(blockIdx.x >> 1) + P.group0;
  Unit U;
  U.half = blockIdx.x & 1;
  U.tiles = 1;
  U.lead = cluster_ctarank();
  U.first = U.half == 0 && blockIdx.y == 0;
  U.b = unit / P.tiles_per_block;
  U.qt = unit % P.tiles_per_block;
  U.row0 = ((long)U.b * R.T) * R.H + (long)U.qt * QROWS;
  if (warp == W_ROPE && lane == 0) { prefetch_tmap(&P.tmQ01); prefetch_tmap(&P.tmK); prefetch_tmap(&P.tmC); prefetch_tmap(&P.tmQ); }
  if (warp == W_S) tmem_alloc(&B->tmem_slot, TMEM_COLS);
  // Q_abs and the nodes' own entries come from the kernels before; a launch of the
  // rest starts after every CTA of the first has seen their end
  if (!P.rest) pdl_wait();
  set_up(P, B, smem, U);
  const uint32_t tmem = B->tmem_slot;
  const int seg = P.seg_rows, nseg = KT / seg;

  const int s_of = warp > W_ROPE ? warp - W_ROPE + 2 : warp - W_RING;        // a load warp's slot
  if (warp > W_ROPE || (warp >= W_RING && warp < W_RING + 3)) {
    // ---- ring slot `s`: uses s, s + SLOTS, ... ----
    const int s = s_of;
    uint8_t* slot = smem + G::OFF_RING + s * SLOT_BYTES;
    int nk = 0, nv = 0;                                   // key and value uses issued
    int z_lo = -1;                                        // known from seen_full on
    for (int u = s; u < 6 * U.nt; u += SLOTS) {
      const Item it = item_of(u, U.nt);
      const int j0 = tile_key(U, it.tile);
      const int ch = it.value ? 4 * U.half + 2 * it.pair : 2 * it.pair;
      uint64_t* full = it.value ? &B->v_full[s] : &B->k_full[s];
      const int y = lane < nseg ? cache_row(R, U, j0 + lane * seg, true) : 0;
      if (u == SLOTS - 1 && !wait_bar(B, &B->q01_read, 0, R.status)) break;   // Q passes through it first
      if (!wait_bar(B, &B->k_empty[s], ((u / SLOTS) & 1) ^ 1, R.status)) break;
      if (lane == 0) mbar_arrive_expect_tx(full, SLOT_BYTES);
      __syncwarp();
      if (nseg == 1) {
        if (lane == 0) tma_load_3d(slot, &P.tmC, full, 0, y, ch);
      } else if (lane < nseg) {
        tma_load_3d(slot + lane * seg * 128, &P.tmK, full, ch * 64, y, 0);
        tma_load_3d(slot + CH_BYTES + lane * seg * 128, &P.tmK, full, ch * 64 + 64, y, 0);
      }
      __syncwarp();
      if (!it.value) {
        ++nk;
        continue;
      }
      ++nv;
      if (z_lo < 0) {
        if (!wait_bar(B, &B->seen_full, 0, R.status)) break;
        z_lo = B->z_lo;
      }
      if (dirty_tile(U, z_lo, it.tile)) {
        if (!wait_bar(B, full, (nv - 1) & 1, R.status)) break;
        clear_unseen(U, smem, slot, 2, j0, z_lo);
        if (lane == 0) mbar_arrive(&B->clean[s]);
      }
    }
    // every copy into this CTA has landed before its shared memory is used again
    if (nk > 0) mbar_wait(&B->k_full[s], (nk - 1) & 1, R.status);
    if (nv > 0) mbar_wait(&B->v_full[s], (nv - 1) & 1, R.status);
  } else if (warp == W_ROPE) {
    // ---- Q once, then the rope chunk of every tile ----
    if (U.nt > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(&B->q01_full, NQT * G::QCH);
        tma_load_3d(smem + G::OFF_Q01, &P.tmQ01, &B->q01_full, 0, (int)U.row0, 0);
        mbar_arrive_expect_tx(&B->q_full, NQS * G::QCH);
        tma_load_3d(smem + OFF_Q, &P.tmQ, &B->q_full, 0, (int)U.row0, NQT);
      }
      __syncwarp();
      int t = 0;
      for (; t < U.nt; ++t) {
        const int y = lane < nseg ? cache_row(R, U, tile_key(U, t) + lane * seg, false) : 0;
        if (!wait_bar(B, &B->s_full, (t & 1) ^ 1, R.status)) break;
        if (lane == 0) mbar_arrive_expect_tx(&B->rope_full, CH_BYTES);
        __syncwarp();
        if (lane < nseg) tma_load_3d(smem + G::OFF_ROPE + lane * seg * 128, &P.tmK, &B->rope_full, 512, y, 0);
        __syncwarp();
      }
      mbar_wait(&B->q01_full, 0, R.status);
      mbar_wait(&B->q_full, 0, R.status);
      if (t > 0) mbar_wait(&B->rope_full, (t - 1) & 1, R.status);
    }
  } else if (warp == W_S) {
    if (lane == 0 && U.nt > 0) {
      // ---- S(t) = Q K(t)^T ----
      const uint32_t idesc = idesc_f16(QROWS, KT, false), tS = tmem + TM_S, tQ = tmem + TM_Q;
      constexpr uint64_t U_Q = G::QCH / 16, U_CH = CH_BYTES / 16, U_SLOT = SLOT_BYTES / 16;
      const uint64_t dQ = smem_desc_sw128(smem + OFF_Q), dR = smem_desc_sw128(smem + G::OFF_RING);
      const uint64_t dRope = smem_desc_sw128(smem + G::OFF_ROPE);
      bool ok = wait_bar(B, &B->q_full, 0, R.status) && wait_bar(B, &B->q_tmem, 0, R.status);
      tc_fence_after();
      uint32_t par = 0;                                   // bit i: parity of k_full[i]
      for (int t = 0; t < U.nt && ok; ++t) {
        int s = first_key_use(t) % SLOTS;
        bool ready = mbar_test_wait(&B->k_full[s], (par >> s) & 1);
        if (t > 0) {
          if (!(ok = wait_bar(B, &B->s_free, (t - 1) & 1, R.status))) break;
          tc_fence_after();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!(ok = ok && wait_bar(B, &B->k_full[s], (par >> s) & 1, R.status, ready))) break;
          par ^= 1u << s;
          const int s1 = s + 1 < SLOTS ? s + 1 : 0;
          // a look at the next barrier, its answer used after these MMAs
          ready = i < 3 ? mbar_test_wait(&B->k_full[s1], (par >> s1) & 1) : mbar_test_wait(&B->rope_full, t & 1);
          const uint64_t db = dR + s * U_SLOT;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              if (i == 0)
                mma_f16_ts(tS, tQ + 32 * c + 8 * d, db + c * U_CH + 2 * d, idesc, (c | d) ? 1u : 0u);
              else
                mma_f16(tS, dQ + (2 * i - 2 + c) * U_Q + 2 * d, db + c * U_CH + 2 * d, idesc, 1u);
            }
          mma_commit(&B->k_empty[s]);
          s = s1;
        }
        if (!(ok = ok && wait_bar(B, &B->rope_full, t & 1, R.status, ready))) break;
#pragma unroll
        for (int d = 0; d < 4; ++d) mma_f16(tS, dQ + (NQS - 1) * U_Q + 2 * d, dRope + 2 * d, idesc, 1u);
        mma_commit(&B->s_full);
        *(volatile int*)&B->issued = t + 1;
      }
      mma_commit(&B->drain[0]);
      mbar_wait(&B->drain[0], 0, R.status);
    }
  } else if (warp == W_PV) {
    if (lane == 0 && U.nt > 0) {
      // ---- O += P(t) V(t) ----
      const uint32_t idesc = idesc_f16_bmn(QROWS, 128, false), tO = tmem + TM_O, tP = tmem + TM_P;
      constexpr uint64_t U_SLOT = SLOT_BYTES / 16, U_KSTEP = 16 * 128 / 16;
      const uint64_t dV = smem_desc_sw128_mn(smem + G::OFF_RING, CH_BYTES);
      uint32_t par = 0, cpar = 0;                         // bit i: parity of v_full[i], clean[i]
      bool ok = wait_bar(B, &B->seen_full, 0, R.status);
      const int z_lo = B->z_lo;
      for (int t = 0; t < U.nt && ok; ++t) {
        int s = first_value_use(t, U.nt) % SLOTS;
        const bool dirty = dirty_tile(U, z_lo, t);
        if (!(ok = wait_bar(B, &B->p_full, t & 1, R.status))) break;
        tc_fence_after();
        bool ready = mbar_test_wait(&B->v_full[s], (par >> s) & 1);
        behind_scores(B, min(t + 2, U.nt));
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (dirty) {
            ok = ok && wait_bar(B, &B->clean[s], (cpar >> s) & 1, R.status);
            cpar ^= 1u << s;
          }
          if (!(ok = ok && wait_bar(B, &B->v_full[s], (par >> s) & 1, R.status, ready))) break;
          par ^= 1u << s;
          const int s1 = s + 1 < SLOTS ? s + 1 : 0;
          if (p == 0) ready = mbar_test_wait(&B->v_full[s1], (par >> s1) & 1);
          const uint64_t db = dV + s * U_SLOT;
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_f16_ts(tO + 128 * p, tP + 8 * k, db + U_KSTEP * k, idesc, (t | k) ? 1u : 0u);
          mma_commit(&B->k_empty[s]);
          s = s1;
        }
        mma_commit(&B->o_done);
      }
      mma_commit(&B->drain[1]);
      mbar_wait(&B->drain[1], 0, R.status);
    }
  } else {
    softmax_role<false>(P, B, smem, tmem, U, smem + G::OFF_Q01, G::QCH);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (P.cluster_parts > 1) cluster_sync_all();            // every part has staged its rows
  tc_fence_after();
  join_and_store(P, smem, U);
  if (warp == W_S) tmem_dealloc(tmem, TMEM_COLS);
  if (P.cluster_parts > 1) cluster_sync_all();            // nobody leaves while its rows may be read
  if (P.rest) pdl_wait();
}

__global__ void __launch_bounds__(THREADS, 1) tree_attn_pair_kernel(const __grid_constant__ TreeParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Bars* B = (Bars*)(smem + OFF_BAR);
  const tree::Rule& R = P.rule;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int group = (int)(blockIdx.x >> 1) + P.group0, unit = group >> 1, p = blockIdx.x & 1;
  const int units = (P.tiles_per_block + 1) / 2;
  const uint32_t rank = cluster_ctarank();
  Unit U;
  U.half = group & 1;
  U.tiles = 2;
  U.lead = rank & ~1u;
  U.first = U.half == 0 && blockIdx.y == 0;
  U.b = unit / units;
  U.qt = 2 * (unit % units) + p;
  U.row0 = ((long)U.b * R.T) * R.H + (long)U.qt * QROWS;
  if (warp == W_ROPE && lane == 0) { prefetch_tmap(&P.tmQ01); prefetch_tmap(&P.tmK); prefetch_tmap(&P.tmQ); }
  if (warp == W_S) tmem_alloc_pair(&B->tmem_slot, TMEM_COLS);
  // Q_abs and the nodes' own entries come from the kernels before; a launch of the
  // rest starts after every CTA of the first has seen their end
  if (!P.rest) pdl_wait();
  set_up(P, B, smem, U);
  const uint32_t tmem = B->tmem_slot, both = 3u << U.lead;
  // segments: rows of a page, at most this CTA's 64 keys of a tile
  const int seg = P.seg_rows, nkseg = 64 / seg, nvseg = KT / seg;

  if (warp == W_RING || warp == W_RING + 1) {
    // ---- keys: this CTA's 64 of every tile, chunk pairs 2 w and 2 w + 1 (and
    // the rope chunk): one barrier and one release for both, each costing the
    // issuing thread 100 to 200 cycles ----
    const int w = warp - W_RING, c = lane / nkseg, sg = lane % nkseg;
    const uint32_t bar = mapa(smem_u32(&B->k_full[w]), U.lead);
    uint64_t* freed = w == 0 ? &B->k_empty[0] : &B->s_full;
    int t = 0;
    bool ok = true;
    for (; t < U.nt && ok; ++t) {
      const int y = lane < 2 * nkseg ? cache_row(R, U, tile_key(U, t) + 64 * p + sg * seg, true) : 0;
      if (!(ok = wait_bar(B, freed, (t & 1) ^ 1, R.status))) break;
      if (p == 0 && lane == 0) mbar_arrive_expect_tx(&B->k_full[w], 4 * PSLOT_BYTES + (w ? CH_BYTES : 0));
      __syncwarp();
      if (lane < 2 * nkseg) {
        for (int i = 2 * w; i < 2 * w + 2; ++i)
          tma_load_3d_pair(smem + OFF_PK + i * PSLOT_BYTES + c * (CH_BYTES / 2) + sg * seg * 128, &P.tmK, bar,
                           (2 * i + c) * 64, y, 0);
        if (w == 1 && c == 0) tma_load_3d_pair(smem + OFF_ROPE + sg * seg * 128, &P.tmK, bar, 512, y, 0);
      }
      __syncwarp();
    }
    // every copy of the pair has landed before its shared memory is used again
    if (p == 0 && ok && t > 0) mbar_wait(&B->k_full[w], (t - 1) & 1, R.status);
  } else if (warp == W_RING + 2) {
    // ---- values: chunks 2 p and 2 p + 1 of this half ----
    bool ok = U.nt > 0 && wait_bar(B, &B->q01_read, 0, R.status);   // Q passes through the slots first
    int z_lo = -1;                                        // known from seen_full on
    uint32_t nd = 0;                                      // tiles cleared so far
    auto know_seen = [&]() {
      if (z_lo < 0 && (ok = ok && wait_bar(B, &B->seen_full, 0, R.status))) z_lo = B->z_lo;
    };
    for (int t = 0; t < U.nt && ok; ++t) {
      const int j0 = tile_key(U, t);
      const int y = lane < nvseg ? cache_row(R, U, j0 + lane * seg, true) : 0;
      bool dirty = j0 + KT > U.ctx;                       // whatever is seen: loaded at once
      if (!dirty) {
        know_seen();
        if (!ok) break;
        dirty = dirty_tile(U, z_lo, t);
      }
      if (!(ok = wait_bar(B, &B->o_done, (t & 1) ^ 1, R.status))) break;
      // a tile to be cleared lands on a barrier of this CTA's own
      const uint32_t bar = dirty ? smem_u32(&B->land) : mapa(smem_u32(&B->v_full[0]), U.lead);
      if (lane == 0) {
        if (dirty) mbar_arrive_expect_tx(&B->land, PV * PSLOT_BYTES);
        else if (p == 0) mbar_arrive_expect_tx(&B->v_full[0], 2 * PV * PSLOT_BYTES);
      }
      __syncwarp();
      if (lane < nvseg)
        for (int i = 0; i < PV; ++i)
          tma_load_3d_pair(smem + OFF_PV + i * PSLOT_BYTES + lane * seg * 128, &P.tmK, bar,
                           (4 * U.half + 2 * p + i) * 64, y, 0);
      __syncwarp();
      if (dirty) {
        know_seen();
        if (!(ok = ok && wait_bar(B, &B->land, nd & 1, R.status))) break;
        clear_unseen(U, smem, smem + OFF_PV, PV, j0, z_lo);
        if (lane == 0) mbar_arrive_pair(mapa(smem_u32(&B->clean[0]), U.lead));
      }
      nd += dirty;
    }
  } else if (warp == W_ROPE) {
    if (U.nt > 0 && lane == 0) {
      mbar_arrive_expect_tx(&B->q01_full, NQT * CH_BYTES);
      tma_load_3d(smem + OFF_PV, &P.tmQ01, &B->q01_full, 0, (int)U.row0, 0);
      if (p == 0) mbar_arrive_expect_tx(&B->q_full, 2 * NQS * CH_BYTES);
      tma_load_3d_pair(smem + OFF_Q, &P.tmQ, mapa(smem_u32(&B->q_full), U.lead), 0, (int)U.row0, NQT);
      mbar_wait(&B->q01_full, 0, R.status);
      if (p == 0) mbar_wait(&B->q_full, 0, R.status);
    }
  } else if (warp == W_S) {
    if (p == 0 && lane == 0 && U.nt > 0) {
      // ---- S(t) = Q K(t)^T of both row tiles ----
      const uint32_t idesc = idesc_f16(2 * QROWS, KT, false), tS = tmem + TM_S, tQ = tmem + TM_Q;
      constexpr uint64_t U_CH = CH_BYTES / 16, U_SLOT = PSLOT_BYTES / 16;
      const uint64_t dQ = smem_desc_sw128(smem + OFF_Q), dK = smem_desc_sw128(smem + OFF_PK);
      const uint64_t dRope = smem_desc_sw128(smem + OFF_ROPE);
      bool ok = wait_bar(B, &B->q_full, 0, R.status) && wait_bar(B, &B->q_tmem, 0, R.status);
      tc_fence_after();
      for (int t = 0; t < U.nt && ok; ++t) {
        const uint32_t par = t & 1;
        bool ready = mbar_test_wait(&B->k_full[0], par);
        if (t > 0) {
          if (!(ok = wait_bar(B, &B->s_free, par ^ 1, R.status))) break;
          tc_fence_after();
        }
#pragma unroll
        for (int i = 0; i < PK; ++i) {
          if (i % 2 == 0) {
            if (!(ok = ok && wait_bar(B, &B->k_full[i / 2], par, R.status, ready))) break;
            // a look at the next barrier, its answer used after these MMAs
            if (i == 0) ready = mbar_test_wait(&B->k_full[1], par);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int d = 0; d < 4; ++d) {
              const uint64_t db = dK + i * U_SLOT + c * (U_CH / 2) + 2 * d;
              if (i == 0)
                mma_f16_ts_pair(tS, tQ + 32 * c + 8 * d, db, idesc, (c | d) ? 1u : 0u);
              else
                mma_f16_pair(tS, dQ + (2 * i - 2 + c) * U_CH + 2 * d, db, idesc, 1u);
            }
          if (i == 1) mma_commit_pair(&B->k_empty[0], both);
        }
        if (!ok) break;
#pragma unroll
        for (int d = 0; d < 4; ++d) mma_f16_pair(tS, dQ + (NQS - 1) * U_CH + 2 * d, dRope + 2 * d, idesc, 1u);
        mma_commit_pair(&B->s_full, both);          // keys 2 and 3 and the rope chunk are free, too
        *(volatile int*)&B->issued = t + 1;
      }
      mma_commit_pair(&B->drain[0], both);
      mbar_wait(&B->drain[0], 0, R.status);
    }
  } else if (warp == W_PV) {
    if (p == 0 && lane == 0 && U.nt > 0) {
      // ---- O += P(t) V(t) of both row tiles ----
      const uint32_t idesc = idesc_f16_bmn(2 * QROWS, 256, false), tO = tmem + TM_O, tP = tmem + TM_P;
      constexpr uint64_t U_KSTEP = 16 * 128 / 16;
      const uint64_t dV = smem_desc_sw128_mn(smem + OFF_PV, CH_BYTES);
      uint32_t nd = 0, nf = 0;                            // tiles cleared / not cleared so far
      bool ok = wait_bar(B, &B->seen_full, 0, R.status);
      const int z_lo = B->z_lo;
      for (int t = 0; t < U.nt && ok; ++t) {
        const bool dirty = dirty_tile(U, z_lo, t);
        uint64_t* bar = dirty ? &B->clean[0] : &B->v_full[0];     // (both CTAs have cleared their halves)
        if (!(ok = wait_bar(B, bar, (dirty ? nd : nf) & 1, R.status))) break;
        if (!(ok = wait_bar(B, &B->p_full, t & 1, R.status))) break;
        tc_fence_after();
        behind_scores(B, min(t + 2, U.nt));
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          mma_f16_ts_pair(tO, tP + 8 * k, dV + U_KSTEP * k, idesc, (t | k) ? 1u : 0u);
        mma_commit_pair(&B->o_done, both);
        if (dirty) ++nd; else ++nf;
      }
      mma_commit_pair(&B->drain[1], both);
      mbar_wait(&B->drain[1], 0, R.status);
    }
  } else {
    softmax_role<true>(P, B, smem, tmem, U, smem + OFF_PV, CH_BYTES);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (P.cluster_parts > 1) cluster_sync_all();            // every part has staged its rows
  join_and_store(P, smem, U);
  cluster_sync_all();          // nobody leaves while its rows, or its half of an MMA, may be read
  tc_fence_after();
  if (warp == W_S) tmem_dealloc_pair(tmem, TMEM_COLS);
  if (P.rest) pdl_wait();
}

// A row and quarter of its dims: sum_s w_s o_s / sum_s w_s with w_s = 2^(lse_s -
// max); a row that no part saw is zero.  WPI warps share the parts (w, w + WPI,
// ...; up to eight loads in flight each) and their sums are added in warp
// order: one warp for few parts, eight for many, whose chain of loads would
// otherwise be the kernel's time (52 parts of 128 rows: 32 us with one warp a
// whole row).  The lanes hold the parts' log-sum-exps (at most MAX_PARTS).
template <int WPI>
__global__ void __launch_bounds__(256) tree_merge_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ part_lse, long rows,
                                                         int parts, __half* __restrict__ o_lat,
                                                         float* __restrict__ lse) {
  __shared__ float4 sums[8][32];
  pdl_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long item = ((long)blockIdx.x * 8 + warp) / WPI;
  const long row = item >> 2;
  const int quarter = (int)(item & 3), w = warp % WPI;
  const bool live = row < rows;
  float w0 = 0.f, w1 = 0.f, den = 0.f, mx = -INFINITY;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) {
    const float l0 = lane < parts ? part_lse[lane * rows + row] : -INFINITY;
    const float l1 = lane + 32 < parts ? part_lse[(lane + 32) * rows + row] : -INFINITY;
    mx = fmaxf(l0, l1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    w0 = l0 == -INFINITY ? 0.f : exp2f(l0 - mx);
    w1 = l1 == -INFINITY ? 0.f : exp2f(l1 - mx);
    den = w0 + w1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float4* src = reinterpret_cast<const float4*>(part + row * 512) + quarter * 32 + lane;
#pragma unroll 8
    for (int s = w; s < parts; s += WPI) {
      const float x = __shfl_sync(0xffffffffu, s < 32 ? w0 : w1, s & 31);
      const float4 v = src[(long)s * rows * 128];         // (rows of parts that saw nothing are zero)
      acc.x += x * v.x; acc.y += x * v.y; acc.z += x * v.z; acc.w += x * v.w;
    }
  }
  if (WPI > 1) {
    sums[warp][lane] = acc;
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int k = 1; k < WPI; ++k) {
      const float4 v = sums[warp + k][lane];
      acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
    }
  }
  if (!live) return;
  const float inv = den != 0.f ? 1.f / den : 0.f;
  __half2 h2[2] = {__floats2half2_rn(acc.x * inv, acc.y * inv), __floats2half2_rn(acc.z * inv, acc.w * inv)};
  *reinterpret_cast<uint2*>(o_lat + row * 512 + quarter * 128 + 4 * lane) = *reinterpret_cast<uint2*>(h2);
  if (lse && lane == 0 && quarter == 0) lse[row] = den != 0.f ? (mx + log2f(den)) * kLn2 : -INFINITY;
}

}  // namespace

// Row tiles in pairs, parts of a unit's key range (a multiple of the parts of a
// cluster).  Cost in tiles (about 2.5 us) of the waves of CTAs that a choice
// needs: FIXED beyond a part's share of the keys, JOIN for a cluster's join,
// MERGE and MERGE_PART for the second kernel.  Measured, us: 512 rows x 2064
// keys x 8 sequences 45 whole, 39 in two parts merged, 35 in two joined; 8192
// rows x 6-8 k keys x 4 sequences 468, 513, 528; 128 rows x 32 k keys 45 in 32
// parts, 37 in 48, 35 in 56 or 64, 37 in 60 joined by fours.  The lengths and
// windows are on the device: keys are bounded by the page table and, when windows
// are given, taken as at most 16 tiles (800 rows x 5 sequences with a window of 512
// keys 28 us whole, 37 in three parts).  Both can be far off.  A table much wider
// than its sequences splits them too finely (512 rows x 2064 keys x 8 sequences
// under a table of 131072 keys: 16 parts, 147 us for 35, and a workspace of 135 MB),
// and long ranges beside windows, or windows of 0, too coarsely (128 rows x 32 k
// keys with a window tensor of zeros: 65 us for 35).
//
// Clusters of whole units that do not fill their last wave have that wave's
// units cut in parts of a second launch, joined in clusters: 256 clusters, of
// which the GPU holds 76, 457 us in two launches (28 of them in two parts), 484 in
// one; 80 clusters 61 and 75, both at 2.07 GHz and in turns.
struct Plan {
  bool pair;
  int parts, cluster_parts;
  long groups, rest;       // clusters of one part; those of them in the second launch
  int rest_parts;          // their parts
};
Plan tree_plan(const mla_handle* h, const mla_attn_desc_t& d) {
  constexpr double FIXED = 4.0, JOIN = 2.8, MERGE = 3.5, MERGE_PART = 0.05;
  const long rows = (long)d.block_len * h->lay.H, tpb = (rows + QROWS - 1) / QROWS;
  long tiles = ((long)d.max_pages * h->cfg.page_size + KT - 1) / KT;
  if (d.window && tiles > 16) tiles = 16;
  Plan best{tpb > 1, 1, 1, 0, 0, 1};
  const long groups = best.groups = (long)d.num_blocks * (best.pair ? 2 * ((tpb + 1) / 2) : tpb);
  // clusters of 2 cs CTAs that the GPU holds at once (GPCs are not a multiple of 8)
  auto held = [&](int cs) -> long {
    const long n = cs == 1 ? h->num_sms / 2 : cs == 2 ? h->num_sms / 4 - 2 : h->num_sms / 8 - 4;
    return n > 0 ? n : 1;
  };
  double cost = 1e300;
  for (int cs = 1; cs <= 4; cs *= 2) {
    const long hold = held(cs);
    for (const int g : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 56, MAX_PARTS}) {
      if ((long)g * cs > (tiles > cs ? tiles : cs)) break;
      const double waves = (double)((groups * g + hold - 1) / hold);
      const double c = waves * (FIXED + (cs > 1 ? JOIN : 0.0) + (double)((tiles + g * cs - 1) / (g * cs))) +
                       (g > 1 ? MERGE + MERGE_PART * groups * g : 0.0);
      if (c < cost) { cost = c; best.parts = g * cs; best.cluster_parts = cs; }
      if (groups * g > 8 * hold) break;
    }
  }
  const long rest = groups % held(1);
  if (best.parts == 1 && rest && groups > rest)
    for (int cs = 2; cs <= 4 && cs <= tiles; cs *= 2) {
      const double c = (double)(groups / held(1)) * (FIXED + (double)tiles) +
                       (double)((rest + held(cs) - 1) / held(cs)) * (FIXED + JOIN + (double)((tiles + cs - 1) / cs));
      if (c < cost) { cost = c; best.rest = rest; best.rest_parts = cs; }
    }
  return best;
}

size_t tree_attention_ws(const mla_handle* h, const mla_attn_desc_t& d) {
  const Plan p = tree_plan(h, d);
  const int parts = p.parts / p.cluster_parts;
  if (parts == 1) return 0;
  const long rows = (long)d.num_blocks * d.block_len * h->lay.H;
  return align256((size_t)parts * rows * 512 * 4) + align256((size_t)parts * rows * 4);
}

mla_status_t tree_attention(cudaStream_t st, mla_handle* h, const tree::Rule& r,
                            const mla_attn_desc_t& d, const __nv_bfloat16* q_abs,
                            const __nv_bfloat16* cache, __half* o_lat, float* lse, void* ws, bool pdl) {
  const Layout& l = h->lay;
  const long rows = (long)d.num_blocks * d.block_len * l.H, slots = (long)r.num_pages * r.page_size;
  if (slots > 0x7fffffffL || rows > 0x7ffffc00L)
    return fail(MLA_ERR_UNSUPPORTED, "tree attention: num_pages * page_size and rows below 2^31 - 1023");
  const Plan plan = tree_plan(h, d);
  const int parts = plan.parts / plan.cluster_parts;      // that reach the workspace when more than one
  TreeParams P;
  const int max_seg = plan.pair ? KT / 2 : KT;
  P.seg_rows = r.page_size < max_seg ? r.page_size : max_seg;
  const long block_rows = (long)d.block_len * l.H;
  const int q_rows = block_rows <= 32 ? 32 : block_rows <= 64 ? 64 : QROWS;      // pairs have more than 128
  if (!make_tmap_chunked(&P.tmQ, false, q_abs, rows, l.L, l.L, q_rows, NQS) ||
      !make_tmap_chunked(&P.tmQ01, false, q_abs, rows, l.L, l.L, q_rows, NQT) ||
      (!plan.pair && !make_tmap_chunked(&P.tmC, false, cache, slots, l.L, l.L, KT, 2)) ||
      !make_tmap_2d(&P.tmK, false, cache, slots, l.L, l.L, P.seg_rows))
    return fail(MLA_ERR_CUDA, "tree attention: cuTensorMapEncodeTiled failed");
  P.rule = r;
  P.o_lat = o_lat;
  P.lse = lse;
  P.vis_stats = d.vis_stats;
  P.rows = rows;
  P.cluster_parts = plan.cluster_parts;
  P.part = (float*)ws;
  P.part_lse = parts > 1 ? (float*)((char*)ws + align256((size_t)parts * rows * 512 * 4)) : nullptr;
  P.tiles_per_block = (int)(((long)d.block_len * l.H + QROWS - 1) / QROWS);
  P.scale_log2 = h->scale * 1.4426950408889634f;
  if (2 * plan.groups > 0x7fffffffL) return fail(MLA_ERR_INVALID_ARG, "tree attention: too many rows");
  static std::once_flag once;
  std::call_once(once, [] {
    for (auto* k : {tree_attn_tc_kernel<32>, tree_attn_tc_kernel<64>, tree_attn_tc_kernel<128>, tree_attn_pair_kernel})
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  auto launch = [&](long groups, int key_parts, bool dependent) {
    const int threads = plan.pair || q_rows == 128 ? THREADS : q_rows == 64 ? Ring<64>::NT : Ring<32>::NT;
    Launch L(dim3((unsigned)(2 * groups), (unsigned)key_parts), dim3((unsigned)threads), SMEM_BYTES, st, dependent,
             dim3(2, (unsigned)P.cluster_parts, 1));
    h->launches += 1;
    return cudaLaunchKernelEx(&L.cfg, plan.pair       ? tree_attn_pair_kernel
                                      : q_rows == 32  ? tree_attn_tc_kernel<32>
                                      : q_rows == 64  ? tree_attn_tc_kernel<64>
                                                      : tree_attn_tc_kernel<128>, P);
  };
  P.group0 = 0;
  P.rest = 0;
  cudaError_t e = launch(plan.groups - plan.rest, plan.parts, pdl);
  if (e == cudaSuccess && plan.rest) {
    P.group0 = (int)(plan.groups - plan.rest);
    P.rest = 1;
    P.cluster_parts = plan.rest_parts;
    e = launch(plan.rest, plan.rest_parts, true);
  }
  if (e != cudaSuccess) return cuda_fail(e, "tree attention launch");
  if (parts > 1) {
    const int wpi = parts > 8 ? 8 : 1;
    const long blocks = (rows * 4 * wpi + 7) / 8;
    if (blocks > 0x7fffffffL) return fail(MLA_ERR_INVALID_ARG, "tree attention: too many rows");
    Launch M(dim3((unsigned)blocks), dim3(256), 0, st, true);
    e = cudaLaunchKernelEx(&M.cfg, wpi == 8 ? tree_merge_kernel<8> : tree_merge_kernel<1>, (const float*)P.part,
                           (const float*)P.part_lse, rows, parts, o_lat, lse);
    if (e != cudaSuccess) return cuda_fail(e, "tree attention merge launch");
    h->launches += 1;
  }
  return MLA_OK;
}

}  // namespace tc
}  // namespace mla
