// tcgen05 key weights (mla_draft.h has the formula, tree.cuh the rule of
// visibility; bf16 layers, entries 512 + 64): per cached key the sum over the
// block's rows of exp(scale <q, e> - lse).
//
// The keys are the MMA's M: S^T = E Q^T puts a key on a tensor-memory lane and
// its rows on the columns, so a key's sum over the rows stays in the registers
// of its two threads and nothing crosses lanes.  Two CTAs work on one MMA
// (cta_group::2): each holds 128 keys (nine 64-dim chunks, 144 KB, all of its
// shared memory's worth) and half of the rows of Q, which streams past in
// 16 KB chunks of 128 rows; a pair's MMA of 256 keys x 256 rows x 64 dims takes
// 512 cycles, in which each SM has 16 KB of Q to fetch (64 dims of 128 keys
// alone would need 32 KB).  The keys are read from HBM once; a chunk trio is
// refilled for the next key tile as soon as the last rows are done with it, so
// for few rows (decode) the kernel is a stream over the cache.
//
// Persistent: the (block, 256-key tile, row part) items are dealt out to the
// pairs in turn.  The scores of one row tile are summed while the next are
// computed (two accumulators of 256 columns).  exp2 by the hardware
// approximation (2^-22), the arguments in fp32.  Keys wholly inside the context
// of rows without a window need no mask; otherwise every lane works out the 32
// keys of its warp for four columns (tree::key_bits) and the words are
// broadcast.  A step of the issuing thread (a barrier, four MMAs, a commit)
// takes about 530 cycles however few the columns, so blocks of at most 64 rows
// bring Q in three chunks a slot (64 sequences x 32 rows x 1-4 k keys: 53 us
// against 57 with one, 43 with the items looked up by the key warp, 41 with the
// log-sum-exps read ahead: 4.6 TB/s of cache).  2048 rows x 8 k keys x 4 sequences:
// 65 us, the tensor pipe active half of the cycles: Q's slots (80 KB in flight a
// CTA) turn over in 2.5 k cycles.  When the key tiles alone do not fill the GPU
// the rows are cut in parts whose sums a second kernel adds in order.
#include <math.h>

#include <mutex>

#include "gemm_tc.cuh"
#include "pair_ptx.cuh"
#include "tree_tc.cuh"

namespace mla {
namespace tc {
namespace {

constexpr int KT = 128, PAIR_KT = 2 * KT, NCH = 9, TRIO = 3, NMAX = 256;
constexpr int CH_BYTES = 128 * 64 * 2, QSLOTS = 5;
constexpr int THREADS = 384;                              // sums x4, MMA, keys, Q x2, sums x4
constexpr int W_MMA = 4, W_KEYS = 5, W_Q = 6;
constexpr int OFF_K = 0, OFF_Q = OFF_K + NCH * CH_BYTES, OFF_BAR = OFF_Q + QSLOTS * CH_BYTES;
constexpr int OFF_LSE = OFF_BAR + 256, SMEM_BYTES = 1024 + OFF_LSE + NMAX * 4;
static_assert(SMEM_BYTES <= 232448, "shared memory");
constexpr uint32_t TMEM_COLS = 512;

struct Bars {
  uint64_t k_full[TRIO], k_empty[TRIO];
  uint64_t q_full[QSLOTS], q_empty[QSLOTS];
  uint64_t s_full[2], s_free[2];
  uint64_t drain;
  // row tiles [first, end) of the item whose keys k_full[0] announces, by its
  // parity; end < 0: no more.  The key warp looks items up (2 k cycles) under its waits; the
  // issuing thread, which has no time to spare, reads them here.
  int first[2], end[2];
  uint32_t tmem_slot;
  int abort;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

__device__ __forceinline__ bool wait_bar(Bars* B, uint64_t* bar, uint32_t parity, uint32_t* st,
                                         bool ready = false) {
  if (ready) return true;
  if (*(volatile int*)&B->abort) return false;
  if (mbar_wait(bar, parity, st)) return true;
  B->abort = 1;
  return false;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sum_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// One (block, 256-key tile, row part) item; every role of both CTAs walks the
// same items.  Called by whole warps; the lanes hold 32 blocks at a time (loading
// and scanning them anew for every item took 3.6 k cycles of a decode item's
// 9.6 k).  num_blocks * key tiles * parts < 2^31 (2^35 keys, 256 a tile, 16 parts).
struct Items {
  const WeightParams& P;
  uint32_t id, step;
  int b0 = -32;               // first block of the group at hand
  uint32_t before = 0, total = 0;     // key tiles of the blocks before the group, of the group
  int l_n0 = 0, l_W = 0, l_ctx = 0;   // this lane's block
  uint32_t l_tiles = 0, l_end = 0;    // its tiles, and those up to and with it
  // the item at hand
  int b, n, n0, W, ctx, kt, sp, qt0, qt1;
  bool skip;                  // no row of the block reaches the tile (windows)

  const uint32_t splits;
  const int tiles, block_rows, cap;   // row tiles and rows of a block, columns of the output

  __device__ Items(const WeightParams& p)
      : P(p), id(blockIdx.x >> 1), step(gridDim.x >> 1), splits((uint32_t)p.splits),
        tiles((p.rule.T * p.rule.H + NMAX - 1) / NMAX), block_rows(p.rule.T * p.rule.H),
        cap((int)min(p.ldw, 0x7fffffffL)) {}

  __device__ bool next() {
    const tree::Rule& R = P.rule;
    const int lane = threadIdx.x % 32;
    const uint32_t tile = splits == 1 ? id : id / splits;
    sp = (int)(id - tile * splits);
    id += step;
    while (tile >= before + total) {
      before += total;
      b0 += 32;
      if (b0 >= P.num_blocks) return false;
      l_tiles = 0;
      if (b0 + lane < P.num_blocks) {
        l_n0 = tree::block_keys(R, b0 + lane, &l_W, &l_ctx, false);
        l_tiles = (uint32_t)(min(l_n0, cap) + PAIR_KT - 1) / PAIR_KT;
      }
      l_end = l_tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, l_end, o);
        if (lane >= o) l_end += y;
      }
      total = __shfl_sync(0xffffffffu, l_end, 31);
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, tile < before + l_end)) - 1;
    b = b0 + l;
    kt = (int)(tile - before - __shfl_sync(0xffffffffu, l_end - l_tiles, l));
    n0 = __shfl_sync(0xffffffffu, l_n0, l);
    W = __shfl_sync(0xffffffffu, l_W, l);
    ctx = __shfl_sync(0xffffffffu, l_ctx, l);
    n = min(n0, cap);
    // (at most 2^31 rows a block: the product stays below 2^32)
    qt0 = splits == 1 ? 0 : (int)((uint32_t)sp * tiles / splits);
    qt1 = splits == 1 ? tiles : (int)((uint32_t)(sp + 1) * tiles / splits);
    skip = qt0 == qt1;
    if (W > 0 && (kt + 1) * PAIR_KT <= ctx) {
      int pmin = 0x7fffffff;
      for (int i = lane; i < R.T; i += 32) pmin = min(pmin, R.positions[(long)b * R.T + i]);
      pmin = __reduce_min_sync(0xffffffffu, pmin);
      skip |= (kt + 1) * PAIR_KT <= tree::window_start(pmin, W);
    }
    return true;
  }
  __device__ int rows(int qt) const { return min(NMAX, block_rows - qt * NMAX); }
  // columns of row tile qt's MMA (each CTA holds half of them)
  __device__ int cols(int qt) const { return (rows(qt) + 31) & ~31; }
};

__device__ __forceinline__ void sum_role(const WeightParams& P, Bars* B, uint8_t* smem, uint32_t tmem,
                                         int rank) {
  const tree::Rule& R = P.rule;
  const int key = threadIdx.x & (KT - 1), half = threadIdx.x >= 256 ? 1 : 0;
  const int w = key / 32, lane = threadIdx.x % 32, col_id = half * 128 + key;
  const uint32_t lane_base = (uint32_t)(w * 32) << 16;
  float* lses = (float*)(smem + OFF_LSE);
  // exp(scale s - lse): the difference first, so that the factor log2(e) rounds a
  // small number (rounding lse log2(e) of each row instead cost ten times the error)
  auto weight = [&](float s, float lse) { return fast_exp2(fmaf(s, P.scale, -lse) * 1.4426950408889634f); };
  const uint32_t s_free0 = mapa(smem_u32(&B->s_free[0]), 0), s_free1 = mapa(smem_u32(&B->s_free[1]), 0);
  uint32_t tile = 0;                                      // row tiles so far, over all items
  Items it(P);
  while (it.next()) {
    const int j = it.kt * PAIR_KT + rank * KT + key;
    const int jw = j - lane;                              // the warp's first key
    float sum = 0.f;
    if (!it.skip) {
      // the context's keys among the warp's 32 (without a window), alike for all rows
      const uint32_t context = (uint32_t)tree::context_bits(R, it.b, 0, it.n0, 0, it.ctx, jw);
      // this thread's column of a row tile: its row's log-sum-exp, -inf for none
      auto load_lse = [&](int qt) {
        const int c = qt * NMAX + col_id;
        if (c >= R.T * R.H) return -INFINITY;
        if (R.q_visible && !R.q_visible[(long)it.b * R.T + c / R.H]) return -INFINITY;
        return P.lse[(long)it.b * R.T * R.H + c];
      };
      float l = load_lse(it.qt0);
      for (int qt = it.qt0; qt < it.qt1; ++qt, ++tile) {
        const int cols = it.cols(qt);
        sum_sync();                                       // the last tile's values have been read
        lses[col_id] = l;
        sum_sync();
        if (qt + 1 < it.qt1) l = load_lse(qt + 1);        // on its way while this tile is summed
        // the warp's 32 keys as this lane's four columns see them; where nodes'
        // keys are among them, a lane walks from one node for all its rows
        uint32_t word[4];
        bool all = true;
        const bool own = R.parent && jw + 32 > it.ctx && jw < it.n0;
        const int node0 = (qt * NMAX + half * 128) / R.H;
        const bool shared = own && (qt * NMAX + half * 128 + 127) / R.H - node0 < 32;
        uint32_t walked = 0;
        bool sound = true;
        if (shared && node0 + lane < R.T) walked = (uint32_t)tree::walk_bits(R, it.b, node0 + lane, it.W, jw - it.ctx, &sound, true);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = half * 128 + 32 * q + lane;
          const bool ok = lses[c] != -INFINITY;           // (rows outside the tree have lse = -inf)
          word[q] = ok ? context : 0u;
          if (it.W > 0 || own) {
            const int node = (qt * NMAX + c) / R.H;
            if (it.W > 0 && ok) word[q] = (uint32_t)tree::context_bits(R, it.b, node, it.n0, it.W, it.ctx, jw);
            if (shared) {
              const uint32_t w1 = __shfl_sync(0xffffffffu, walked, node - node0);
              const bool s1 = __shfl_sync(0xffffffffu, (int)sound, node - node0) != 0;
              word[q] = ok && s1 ? word[q] | w1 : 0u;
            } else if (own && ok) {
              bool s1;
              const uint32_t w1 = (uint32_t)tree::walk_bits(R, it.b, node, it.W, jw - it.ctx, &s1, true);
              word[q] = s1 ? word[q] | w1 : 0u;
            }
          }
          all = all && (word[q] == 0xffffffffu || c >= cols);
        }
        all = __all_sync(0xffffffffu, all);
        __syncwarp();                                     // the walks may have parted the warp
        const int buf = tile & 1;
        wait_bar(B, &B->s_full[buf], (tile >> 1) & 1, R.status);
        tc_fence_after();
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c0 = half * 128 + 32 * q;
          if (c0 < cols) {
            float s[32];
            tmem_ld32(tmem + buf * NMAX + c0 + lane_base, s);
            if (all) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 l = *reinterpret_cast<const float4*>(lses + c0 + i);
                part[0] += weight(s[i], l.x);
                part[1] += weight(s[i + 1], l.y);
                part[2] += weight(s[i + 2], l.z);
                part[3] += weight(s[i + 3], l.w);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const uint32_t m = __shfl_sync(0xffffffffu, word[q], i);
                const float p = weight(s[i], lses[c0 + i]);
                part[i & 3] += ((m >> lane) & 1u) ? p : 0.f;
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_pair(buf ? s_free1 : s_free0);
        sum += (part[0] + part[1]) + (part[2] + part[3]);
      }
    }
    // the key's two halves; half 0 writes
    sum_sync();
    if (half) lses[key] = sum;
    sum_sync();
    if (!half && j < it.n) {
      const float t = sum + lses[key];
      if (P.splits > 1) {
        P.part[((long)it.sp * P.num_blocks + it.b) * P.ldp + j] = t;
      } else {
        const long at = (long)it.b * P.ldw + j;
        P.out[at] = P.prior ? fmaf(P.decay, P.prior[at], t) : t;
      }
    }
  }
}

// QC: chunks of Q a slot holds.
template <int QC>
__global__ void __launch_bounds__(THREADS, 1) key_weights_tc_kernel(const __grid_constant__ WeightParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Bars* B = (Bars*)(smem + OFF_BAR);
  const tree::Rule& R = P.rule;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = (int)cluster_ctarank();
  if (tid == 0) {
    for (int i = 0; i < TRIO; ++i) { mbar_init(&B->k_full[i], 1); mbar_init(&B->k_empty[i], 1); }
    for (int i = 0; i < QSLOTS; ++i) { mbar_init(&B->q_full[i], 1); mbar_init(&B->q_empty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&B->s_full[i], 1); mbar_init(&B->s_free[i], 16); }
    mbar_init(&B->drain, 1);
    B->abort = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) tmem_alloc_pair(&B->tmem_slot, TMEM_COLS);
  if (blockIdx.x == 0)
    for (int b = tid; b < P.num_blocks; b += THREADS) {
      int w, c;
      if (tree::block_keys(R, b, &w, &c, true) > P.ldw) set_status(R.status, MLA_DEV_BAD_LENGTH);
    }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // both CTAs' barriers are up
  tc_fence_after();
  const uint32_t tmem = B->tmem_slot;

  if (warp == W_KEYS) {
    // ---- the CTA's 128 keys of every item, in three trios of chunks ----
    const int ps = R.page_size, past_end = R.num_pages * ps, seg = P.seg_rows, nseg = KT / seg;
    if (lane == 0) prefetch_tmap(&P.tmC);
    uint32_t use = 0;
    bool ok = true;
    Items it(P);
    // the next item that loads keys, and the cache row of this lane's segment
    auto look = [&](int* y) {
      do {
        if (!it.next()) return false;
      } while (it.skip);
      *y = past_end;
      const int j = it.kt * PAIR_KT + rank * KT + lane * seg;
      if (lane < nseg && j < it.n) {
        const int pg = R.block_table[(long)it.b * R.max_pages + j / ps];
        if (pg >= 0 && pg < R.num_pages) *y = pg * ps + j % ps;
        else set_status(R.status, MLA_DEV_BAD_PAGE);
      }
      return true;
    };
    int y = 0;
    bool more = look(&y);
    while (ok && more) {
      const int y0 = y;
      const int first = it.qt0, end = it.qt1;
      for (int c3 = 0; c3 < TRIO; ++c3) {
        if (c3 == TRIO - 1) more = look(&y);              // under the wait for the last trio
        if (!(ok = wait_bar(B, &B->k_empty[c3], (use & 1) ^ 1, R.status))) break;
        if (rank == 0 && lane == 0) {
          if (c3 == 0) {
            B->first[use & 1] = first;
            B->end[use & 1] = end;
          }
          mbar_arrive_expect_tx(&B->k_full[c3], 2 * 3 * CH_BYTES);
        }
        __syncwarp();
        const uint32_t bar = mapa(smem_u32(&B->k_full[c3]), 0);
        uint8_t* dst = smem + OFF_K + 3 * c3 * CH_BYTES;
        if (nseg == 1) {
          if (lane == 0) tma_load_3d_pair(dst, &P.tmC, bar, 0, y0, 3 * c3);
        } else if (lane < nseg) {
          for (int c = 0; c < 3; ++c)
            tma_load_3d_pair(dst + c * CH_BYTES + lane * seg * 128, &P.tmK, bar, (3 * c3 + c) * 64, y0, 0);
        }
        __syncwarp();
      }
      ++use;
    }
    // the end, once the last item's first keys are done with (its other copies land
    // before the pair may exit: the barriers are the even CTA's)
    if (rank == 0 && ok && wait_bar(B, &B->k_empty[0], (use & 1) ^ 1, R.status)) {
      if (lane == 0) {
        B->end[use & 1] = -1;
        mbar_arrive(&B->k_full[0]);
      }
      if (use > 0)
        for (int i = 1; i < TRIO; ++i) mbar_wait(&B->k_full[i], (use - 1) & 1, R.status);
    }
  } else if (warp == W_Q || warp == W_Q + 1) {
    // ---- this CTA's half of the rows, chunk by chunk; the two warps take turns ----
    if (lane == 0) prefetch_tmap(&P.tmQ);
    uint32_t u = 0;                                       // slots used so far
    int last = -1;
    bool ok = true;
    Items it(P);
    while (ok && it.next()) {
      if (it.skip) continue;
      for (int qt = it.qt0; qt < it.qt1 && ok; ++qt) {
        const int y = (int)((long)it.b * R.T * R.H + (long)qt * NMAX + rank * (it.cols(qt) / 2));
        for (int c = 0; c < NCH; c += QC, ++u) {
          if ((u & 1) != (uint32_t)(warp - W_Q)) continue;
          const int s = u % QSLOTS;
          ok = wait_bar(B, &B->q_empty[s], ((u / QSLOTS) & 1) ^ 1, R.status);
          if (!ok) break;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&B->q_full[s], 2 * QC * P.q_box_rows * 128);
            tma_load_3d_pair(smem + OFF_Q + s * CH_BYTES, &P.tmQ, mapa(smem_u32(&B->q_full[s]), 0), 0, y, c);
          }
          __syncwarp();
          last = (int)u;
        }
      }
    }
    if (rank == 0 && last >= 0)
      mbar_wait(&B->q_full[last % QSLOTS], (last / QSLOTS) & 1, R.status);
  } else if (warp == W_MMA && rank == 0) {
    // ---- MMA issue for the pair (the even CTA) ----
    constexpr uint64_t U_CH = CH_BYTES / 16;
    const uint64_t dK = smem_desc_sw128(smem + OFF_K), dQ = smem_desc_sw128(smem + OFF_Q);
    if (lane == 0) {
      const int block_rows = R.T * R.H;
      uint32_t use = 0, tile = 0, qpar = 0;
      int s = 0;
      for (bool ok = true; ok; ++use) {
        if (!(ok = wait_bar(B, &B->k_full[0], use & 1, R.status))) break;
        const int first = *(volatile int*)&B->first[use & 1], end = *(volatile int*)&B->end[use & 1];
        if (end < 0) break;
        for (int qt = first; qt < end && ok; ++qt, ++tile) {
          const int buf = tile & 1, cols = (min(NMAX, block_rows - qt * NMAX) + 31) & ~31;
          const uint32_t d = tmem + buf * NMAX, idesc = idesc_f16(256, cols, false);
          bool ready = mbar_test_wait(&B->q_full[s], qpar);
          if (!(ok = wait_bar(B, &B->s_free[buf], ((tile >> 1) & 1) ^ 1, R.status))) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < NCH; c += QC) {
            if (qt == first && c > 0 && c % 3 == 0 && ok) ok = wait_bar(B, &B->k_full[c / 3], use & 1, R.status);
            if (!ok || !(ok = wait_bar(B, &B->q_full[s], qpar, R.status, ready))) break;
            // a look at the next slot, its answer used after these MMAs
            ready = s + 1 == QSLOTS ? mbar_test_wait(&B->q_full[0], qpar ^ 1) : mbar_test_wait(&B->q_full[s + 1], qpar);
#pragma unroll
            for (int x = 0; x < QC; ++x) {
              const uint64_t db = dQ + s * U_CH + (uint64_t)x * P.q_box_rows * 8;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_pair(d, dK + (c + x) * U_CH + 2 * k, db + 2 * k, idesc, (c | x | k) ? 1u : 0u);
            }
            mma_commit_pair(&B->q_empty[s]);
            if (qt == end - 1 && (c + QC) % 3 == 0) mma_commit_pair(&B->k_empty[c / 3]);
            if (++s == QSLOTS) { s = 0; qpar ^= 1; }
          }
          mma_commit_pair(&B->s_full[buf]);
        }
      }
      mma_commit_pair(&B->drain);
      mbar_wait(&B->drain, 0, R.status);
    }
  } else if (warp != W_MMA) {
    sum_role(P, B, smem, tmem, rank);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();          // the pair's MMAs and copies are done in both CTAs
  tc_fence_after();
  if (warp == W_MMA) tmem_dealloc_pair(tmem, TMEM_COLS);
}

// out = decay * prior + the row parts' sums, in order.
__global__ void __launch_bounds__(256) weights_finish_kernel(const WeightParams P) {
  const long t = blockIdx.x * 256L + threadIdx.x;
  const int b = (int)(t / P.ldp);
  const long j = t % P.ldp;
  if (b >= P.num_blocks) return;
  int W, ctx;
  const long n = min((long)tree::block_keys(P.rule, b, &W, &ctx, false), P.ldw);
  if (j >= n) return;
  float sum = 0.f;
  for (int s = 0; s < P.splits; ++s) sum += P.part[((long)s * P.num_blocks + b) * P.ldp + j];
  const long at = (long)b * P.ldw + j;
  P.out[at] = P.prior ? fmaf(P.decay, P.prior[at], sum) : sum;
}

long key_tiles(const mla_handle* h, const mla_attn_desc_t& d, long ldw) {
  const long cap = (long)d.max_pages * h->cfg.page_size;
  return ((ldw < cap ? ldw : cap) + PAIR_KT - 1) / PAIR_KT;
}

// Parts of a block's rows, so that the last round of items leaves few pairs of
// SMs idle: the cost is rounds times an item's row tiles and a load of its keys
// (about half a row tile), by the page table's bound on the keys; a second
// kernel weighs as much as a row tile.
int weight_splits(const mla_handle* h, const mla_attn_desc_t& d, long ldw) {
  const long rows = (long)d.block_len * h->lay.H, row_tiles = (rows + NMAX - 1) / NMAX;
  const long items = (long)d.num_blocks * key_tiles(h, d, ldw), pairs = h->num_sms / 2;
  int best = 1;
  double cost = 1e300;
  for (long s = 1; s <= row_tiles && s <= 16 && items * s <= 32 * pairs; ++s) {
    const double rounds = (double)((items * s + pairs - 1) / pairs);
    const double c = rounds * ((double)((row_tiles + s - 1) / s) + 0.5) + (s > 1 ? 1.0 : 0.0);
    if (c < cost) { cost = c; best = (int)s; }
  }
  return best;
}

}  // namespace

size_t key_weights_ws(const mla_handle* h, const mla_attn_desc_t& d, long ldw) {
  const int s = weight_splits(h, d, ldw);
  return s == 1 ? 0 : align256((size_t)s * d.num_blocks * key_tiles(h, d, ldw) * PAIR_KT * 4);
}

mla_status_t key_weights(cudaStream_t st, mla_handle* h, const tree::Rule& r, const mla_attn_desc_t& d,
                         const __nv_bfloat16* q_abs, const __nv_bfloat16* cache, const float* lse,
                         float decay, const float* prior, float* out, long ldw, void* ws) {
  const Layout& l = h->lay;
  const long rows = (long)d.num_blocks * r.T * r.H, slots = (long)r.num_pages * r.page_size;
  if (slots > 0x7fffffffL) return fail(MLA_ERR_UNSUPPORTED, "key weights: num_pages * page_size < 2^31");
  WeightParams P;
  const long block_rows = (long)r.T * r.H;
  P.q_box_rows = (int)((block_rows < NMAX ? (block_rows + 31) & ~31L : NMAX) / 2);
  P.seg_rows = r.page_size < KT ? r.page_size : KT;
  // up to 64 rows: 3 chunks of at most 32 rows a CTA (rows go up to whole 16s a CTA, the
  // next, 48, would take 18 KB) fit a slot of 16 KB
  const int qc = 3 * P.q_box_rows * 128 <= CH_BYTES ? 3 : 1;
  if (!make_tmap_chunked(&P.tmQ, false, q_abs, rows, l.L, l.L, P.q_box_rows, qc) ||
      !make_tmap_chunked(&P.tmC, false, cache, slots, l.L, l.L, KT, 3) ||
      !make_tmap_2d(&P.tmK, false, cache, slots, l.L, l.L, P.seg_rows))
    return fail(MLA_ERR_CUDA, "key weights: cuTensorMapEncodeTiled failed");
  P.rule = r;
  P.lse = lse;
  P.prior = prior;
  P.out = out;
  P.part = (float*)ws;
  P.ldw = ldw;
  P.ldp = key_tiles(h, d, ldw) * PAIR_KT;
  P.num_blocks = d.num_blocks;
  P.splits = weight_splits(h, d, ldw);
  P.decay = decay;
  P.scale = h->scale;
  static std::once_flag once;
  std::call_once(once, [] {
    for (auto* k : {key_weights_tc_kernel<1>, key_weights_tc_kernel<3>})
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  const long items = (long)d.num_blocks * key_tiles(h, d, ldw) * P.splits, pairs = h->num_sms / 2;
  Launch L(dim3((unsigned)(2 * (items < pairs ? items : pairs))), dim3(THREADS), SMEM_BYTES, st, false,
           dim3(2, 1, 1));
  cudaError_t e = cudaLaunchKernelEx(&L.cfg, qc == 3 ? key_weights_tc_kernel<3> : key_weights_tc_kernel<1>, P);
  if (e != cudaSuccess) return cuda_fail(e, "key weights launch");
  h->launches += 1;
  if (P.splits > 1) {
    weights_finish_kernel<<<(unsigned)((d.num_blocks * P.ldp + 255) / 256), 256, 0, st>>>(P);
    h->launches += 1;
  }
  return MLA_OK;
}

}  // namespace tc
}  // namespace mla
