// Latent attention over the 8-bit cache (mla_latent_attention8), on the tensor cores.
//
// Mathematics.  128 keys fill the MMA's M, and 32 query rows its N, twice:
//   S^T = K8 [Qhi | Qlo]^T     (e4m3, M = 128 keys, N = 64, K = 512 dims; 16 MMAs)
//   R^T = Kpe Qpe^T            (bf16, N = 32, K = 64; 4 MMAs)
//   O^T += V8^T [Phi | Plo]^T  (e4m3, M = 128 value dims x 4, N = 64, K = 128 keys; 16 MMAs)
// so the cache's own bytes are the operands of both products: nothing is widened, a
// tile is read from memory once and from shared memory twice, by dims and, MN-major, by
// keys.  A bf16 number has 8 significant bits and e4m3 4: q / 2^k is hi + lo exactly
// (down to 2^-10 where the row's largest is 224 or more), and the halves' products are added in
// fp32.  The score of key j is then
//   t_j = c 2^k s_j (S_hi + S_lo) + c R + log2 s_j        (c = scale log2 e, s_j the key's scale)
// whose maximum is the softmax's reference: w_j = 2^(t_j - M) <= 2^1.75 is the weight times
// the key's scale, what meets the codes.  2^7 w_j is split like q, its rest by 2^4 more:
// e4m3 spans 2^17, and a weight is off by 2^-8 of itself and 2^-21 of 2^M.  The smallest
// weights round to nothing, so that n of them may lose n 2^-21: after 64 tiles a piece is
// put away and joined by its log-sum-exp.  The sum of the softmax, l = sum w_j / s_j, is fp32.
//
// Work split.  One persistent CTA per SM.  The 128-key tiles of all units (a block's groups
// of 32 rows), in order, are cut into equal ranges, or, where there are fewer units than CTAs,
// into equal pieces that start with their unit; a (unit, CTA) piece writes its
// normalised partial to one of the CTA's two slots, or the output itself where the unit lies in one CTA; the
// join kernel adds the pieces by log-sum-exp in order.
//   warps 0-7  : softmax, two groups of 128 threads, thread = key, 16 rows each; between
//                segments the next one's queries are split before the last one's output is
//                stored, so that its first S runs meanwhile
//   warps 8, 9 : the scores' and the outputs' MMAs (warp 8 holds the tensor memory)
//   warps 10-11: copies; a tile is five 16 KB chunks, each refilled once its product is done
// Warps 8 to 11 run converged with one elected thread that issues: operands of MMAs and copies lie in
// uniform registers, and what a loop of one thread would move there for each MMA took 80-100 cycles of
// issue for 48 of work (128 heads x 16 tokens: 207 -> 171 us).
//
// What bounds it.  Two tiles of 80 KB are all that fits beside the queries, so a tile's place goes
// round in copy (1.0 k cycles from L2, up to 4 k from HBM) - scores (1.2 k) - softmax (0.8 k) - output
// (0.8-1.0 k) and the hand-overs between them, 5.6 k: one tile in 2.8 k cycles, where the products'
// operands alone pass shared memory in 1.75 k (an MMA of N = 64 takes 48 cycles, the time of
// its 6 KB).  A raised reference waits for the output before it and costs 1.2 k: all rows' are raised to
// their largest score so far when one has to be, which halves how often.  Widened to bf16 the same tile would not
// fit twice.  Code is the other bound: with the MMA loops unrolled, or more of it elsewhere, the roles' loops
// do not fit the instruction cache together (8% misses as it is), and what runs once in a segment runs cold: the step
// from a unit to the next (queries, sums, output) takes 10 k cycles.  128 heads x 16 tokens over 4 x 8 k
// keys 166 us (816 TFLOP/s of the bf16 operation), 128 heads x 1 token over 131 k keys 57 us, 64 sequences x 32
// heads over 1-4 k keys 36 us (3.0 TB/s: first tiles of a cold SM at 6 us, eleven tiles, a store, the
// join).  The softmax's arithmetic is in pairs of fp32 and its maxima are warp reductions of one instruction.
#include "cache8.cuh"
#include "gemm_tc.cuh"
#include "tc_ptx.cuh"

#include <math.h>

#include <algorithm>
#include <mutex>

namespace mla {
namespace cache8 {
namespace {

using namespace tc;

constexpr int KT = 128, NR = 32, HALF = 16;          // keys a tile, rows a unit, rows a softmax thread
// Units whose join is shared by 16 CTAs, not 4 (32 heads x 1 over 1-2 k and 8-16 k keys, with 16 and with 4: 8 units
// 15.6 and 17.0 us, 24.0 and 25.9; 16 units 16.4 and 17.0, 36.3 and 37.6; 20 units 18.3 and 16.8, 35.0 and 33.8;
// 24 units 18.7 and 17.0, 47.3 and 44.7; 64 units 30.8 and 24.4, 100 and 92).
constexpr int FEW_UNITS = 16;
constexpr int SEG_TILES = 64;                        // tiles after which a piece is put away
constexpr int JOIN_TILES = 3;                        // what cutting units costs, in tiles
constexpr int THREADS = 384, SM_THREADS = 256;
constexpr int STAGES = 2, CHUNKS = 5;                // 4 chunks of 128 latent dims, one of 64 rotary ones
constexpr int CH_BYTES = KT * 128;                   // 16 KB
constexpr int STAGE_BYTES = CHUNKS * CH_BYTES;
constexpr int Q_CH_BYTES = 2 * NR * 128;             // [hi rows | lo rows] x 128 dims
constexpr int QR_BYTES = NR * 128;
constexpr int P_BYTES = KT * 2 * NR;                 // [key][hi | lo], 64 bytes a key
constexpr int OFF_Q = STAGES * STAGE_BYTES;
constexpr int OFF_QR = OFF_Q + 4 * Q_CH_BYTES;
constexpr int OFF_P = OFF_QR + QR_BYTES;
constexpr int OFF_RED = OFF_P + 2 * P_BYTES;
constexpr int Q_ROWS = NR / (SM_THREADS / 32), Q_BATCH = 2;
static_assert(Q_ROWS == 2 * Q_BATCH, "two rounds of a warp's rows");
// TMEM: S of tile g at column 128 (g % 2): hi 0-31, lo 32-63, rotary 64-95; O at 256: 4 x (hi | lo)
constexpr uint32_t TMEM_COLS = 512, TM_O = 256;
constexpr float SLACK_LOG2 = 1.75f;                  // 2^7 2^1.75 < 448
constexpr float P_LOG2 = 7.f, LO_UP = 16.f;

struct Params {
  CUtensorMap tmL;    // the latents' bytes as [slots, 256] 16-bit numbers, chunked, box seg_rows x 1 chunk
  CUtensorMap tmR;    // rotary dims [slots, 64], box seg_rows
  tree::Rule rule;
  const float* scale;
  const __nv_bfloat16* q;
  __half* o_lat;      // [rows, 512]
  float* lse;         // [rows] or NULL
  float* part;        // [slots][4 quarters][8 x 4 rows][128 dims][4 rows] normalised partial outputs
  float* part_lse;    // [slots, 32]
  int* first_tile;    // [blocks + 1] tiles of a group's worth of keys before each block, [1] tiles of a piece or 0
  int num_blocks, groups, seg_rows;
  bool whole;         // every unit in one CTA: nothing to join
  float scale_log2;
};

// The scales of entries that are no page's (their dims are copied as zeros): such a key counts as zeros whatever
// the cache holds.
struct Ones {
  float of[KT];
  constexpr Ones() : of() {
    for (int i = 0; i < KT; ++i) of[i] = 1.f;
  }
};
__device__ __align__(16) const Ones no_page_scales;

struct Bars {
  uint64_t full[STAGES];            // a tile landed
  uint64_t empty[STAGES][CHUNKS];   // the products of a chunk are done
  uint64_t q_full;
  uint64_t s_full[2];               // S(g) done (and all before it), by g % 2
  uint64_t p_full[2];               // P(g) in shared memory
  uint64_t o_done;                  // O(g) done (waited on for a rescale only)
  uint64_t o_seg;                   // the segment's last O done
  uint64_t drain, drain_o;
  uint32_t tmem_slot;
  int abort;
};

// A bounded wait in few instructions: a CTA's code competes for the instruction cache.
__device__ __forceinline__ bool wait_bar(Bars* B, uint64_t* bar, uint32_t parity, uint32_t* st) {
  if (mbar_test_wait(bar, parity)) return true;
  uint32_t rounds = 0;
  while (!mbar_try_wait(bar, parity))
    if (++rounds > kWaitBudget || *(volatile int*)&B->abort) {
      if (!atomicExch(&B->abort, 1)) set_status(st, MLA_DEV_TIMEOUT);
      return false;
    }
  return true;
}
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / x, off by one unit in the last place (the sums and their parts lie in 2^-120 .. 2^100).
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(2 + g) : "memory"); }
__device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 4, 256;" ::: "memory"); }

// D[tmem] (+)= A B^T, e4m3 operands, fp32 sums.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// Instruction descriptor of kind::f8f6f4: fp32 D, e4m3 A and B.
constexpr uint32_t idesc_f8(int M, int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24); }
// MN-major operand of 64 MN bytes a row with 64-byte swizzle: 8-row groups of K 512 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw64_mn(const void* tile) {
  uint64_t d = (smem_u32(tile) & 0x3FFFFull) >> 4;
  d |= (uint64_t)(512 >> 4) << 16;
  d |= (uint64_t)(512 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)4 << 61;
  return d;
}

// An untiled copy (addresses and size multiples of 16 bytes) that completes on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
// 16-byte global store with an L2 eviction policy.
__device__ __forceinline__ void st_global_hint4(float4* p, float4 v, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.f32 [%0], {%1, %2, %3, %4}, %5;"
               ::"l"(p), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "l"(policy) : "memory");
}

// 16 consecutive fp32 columns of this thread's TMEM lane, no wait.
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_reg_fence16(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]),
                 "+f"(v[15]));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
        "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void lds16(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < HALF; i += 4) *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(p + i);
}

// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
// The largest over the warp's lanes (a NaN is left out).
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Lane l ends with the sum over the warp's lanes of x[l % 16] (x[0 .. 15] per lane).
__device__ __forceinline__ float transpose_sum16(float* x, int lane) {
#pragma unroll
  for (int s = 8; s >= 1; s >>= 1) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float send = upper ? x[i] : x[i + s], keep = upper ? x[i + s] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

// Keys of block b: [j_lo, n) in nt tiles, j_lo the first key that any row's window reaches,
// rounded down to a tile.  Not behind the context: a window counts the nodes' own positions, which
// may lie anywhere ahead of their keys' indices.
struct Keys {
  int n, W, ctx, j_lo, nt;
};
__device__ __forceinline__ Keys keys_of(const Params& P, int b, bool report) {
  Keys k;
  k.n = tree::block_keys(P.rule, b, &k.W, &k.ctx, report);
  k.j_lo = 0;
  if (k.W > 0 && k.n > 0) {
    int p = 0x7fffffff;
    for (int t = 0; t < P.rule.T; ++t) p = min(p, P.rule.positions[(long)b * P.rule.T + t]);
    k.j_lo = min(tree::window_start(p, k.W), k.ctx) / KT * KT;
  }
  k.nt = k.n > k.j_lo ? (k.n - k.j_lo + KT - 1) / KT : 0;
  return k;
}

// The U tiles in G ranges (G <= U), the first U % G of them one tile longer.  (In 32 bits: the host
// refuses more tiles.)
struct Ranges {
  int len, longer;                         // U / G, U % G
  __device__ __forceinline__ int begin(int c) const { return c * len + min(c, longer); }
  __device__ __forceinline__ int cta_of(int u) const {
    const int head = longer * (len + 1);
    return u < head ? u / (len + 1) : longer + (u - head) / len;
  }
};

// One lane of a converged warp, always the same.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p;
}
// Lane 0's number: the compiler then knows that the warp's lanes agree.
__device__ __forceinline__ int warp_same(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ uint64_t desc(uint32_t hi, uint32_t lo) { return (uint64_t)hi << 32 | lo; }
// wait_bar() of a whole warp.
__device__ __forceinline__ bool warp_wait(Bars* B, uint64_t* bar, uint32_t parity, uint32_t* st) {
  return __all_sync(0xffffffffu, wait_bar(B, bar, parity, st));
}

// Where CTA c leaves what it has of a unit that others share: of one begun before its range, or of the
// last one of its range (which also puts away the segments of units of its own, before).
__device__ __forceinline__ long slot_of(int c, bool begun, int ctas) { return begun ? c : ctas + c; }

// A CTA's pieces, in order: tiles [t0, t0 + n) of a unit, its keys.  The first MAX_PIECES are worked
// out once, before the copies start: what a role reads from memory later comes behind 160 KB of tiles.
constexpr int MAX_PIECES = 32;
struct Piece {
  int unit, b, t0, n;
  Keys k;
};
// Where a role stands in its CTA's range: a segment is at most SEG_TILES of a piece.
struct Seg {
  int unit, b, t0, n;
  bool first, last;                        // of the piece
  Keys k;
};
struct SegIter {
  int piece;                               // next one
  int unit, left;                          // behind the listed pieces: the next unit, tiles to hand out
  int rest;                                // tiles of the current piece not yet handed out
};

struct __align__(128) Shared {
  float scale[STAGES][KT];          // the keys' scales of a tile
  float wpart[2][2][4][HALF];       // by tile parity, group, warp: row maxima
  float m[NR];                      // reference of each row (log2), at a segment's end
  float inv[NR], keep[NR];          // factors of a segment's O and of what its piece has put away
  float q_scale[NR];                // c 2^k of each row
  int lo[NR], hi[NR];               // context keys that each row sees
  float sum[2][4][HALF];
  float run_lse[NR];                // log2-sum-exp of what a piece has put away
  uint32_t seen[2][NR][4];          // by group: which keys of a tile each row sees
  int fast_lo, fast_hi, any_lo, any_hi;
  uint32_t alive;
  int first_unit, first_tile, pieces, more_unit, more_left;
  uint32_t empty;                   // of whole units: those without a key
  Piece piece[MAX_PIECES];
  int scan[THREADS / 32];
  Bars bars;
};

constexpr int SMEM_BYTES = 1024 + OFF_RED + (int)sizeof(Shared);
static_assert(SMEM_BYTES <= 232448, "shared memory");

// The next segment of a CTA's range.
__device__ __forceinline__ bool next_seg(const Params& P, const Shared* sh, SegIter& it, Seg& s) {
  if (it.rest > 0) {                       // goes on with the piece
    s.t0 += s.n;
    s.first = false;
  } else if (it.piece < sh->pieces) {
    const Piece p = sh->piece[it.piece++];
    s.unit = p.unit;
    s.b = p.b;
    s.t0 = p.t0;
    s.k = p.k;
    s.first = true;
    it.rest = p.n;
  } else {
    if (it.piece++ == sh->pieces) {
      it.unit = sh->more_unit;
      it.left = sh->more_left;
    }
    while (true) {                         // (small blocks: more of them than the list holds)
      if (it.left <= 0) return false;
      s.unit = it.unit++;
      s.b = s.unit / P.groups;
      s.k = keys_of(P, s.b, false);
      if (s.k.nt > 0) break;
    }
    s.t0 = 0;
    s.first = true;
    it.rest = min(s.k.nt, it.left);
    it.left -= it.rest;
  }
  s.n = min(it.rest, SEG_TILES);
  it.rest -= s.n;
  s.last = it.rest == 0;
  return true;
}

__global__ void __launch_bounds__(THREADS, 1) attn8_kernel(const __grid_constant__ Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  Shared* sh = (Shared*)(smem + OFF_RED);
  Bars* B = &sh->bars;
  uint32_t* status = P.rule.status;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int c = blockIdx.x, nb = P.num_blocks;

  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&B->full[s], 1);
      for (int q = 0; q < CHUNKS; ++q) mbar_init(&B->empty[s][q], 1);
    }
    mbar_init(&B->q_full, SM_THREADS / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s_full[i], 1);
      mbar_init(&B->p_full[i], SM_THREADS);
    }
    mbar_init(&B->o_done, 1);
    mbar_init(&B->o_seg, 1);
    mbar_init(&B->drain, 1);
    mbar_init(&B->drain_o, 1);
    B->abort = 0;
    sh->first_unit = nb * P.groups;
    sh->first_tile = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(&B->tmem_slot, TMEM_COLS);

  // ---- schedule: the tiles of one group before each block, then this CTA's first unit and tile
  // (from the same numbers when every block has a thread); of whole units their numbers will do
  int nt = 0, excl = 0;
  auto total = [&](int x) {                // over the CTA's threads
    x = __reduce_add_sync(0xffffffffu, x);
    if (lane == 0) sh->scan[warp] = x;
    __syncthreads();
    x = __reduce_add_sync(0xffffffffu, lane < THREADS / 32 ? sh->scan[lane] : 0);
    __syncthreads();
    return x;
  };
  auto scan = [&](int run) {
    int x = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sh->scan[warp] = x;
    __syncthreads();
    const int of = lane < THREADS / 32 ? sh->scan[lane] : 0;
    const int before = run + __reduce_add_sync(0xffffffffu, lane < warp ? of : 0);
    const int all = run + __reduce_add_sync(0xffffffffu, of);
    __syncthreads();
    excl = before + x - nt;
    return all;
  };
  auto keys = [&](int base, bool report) { nt = base + tid < nb ? keys_of(P, base + tid, report).nt : 0; };
  const int units = nb * P.groups;
  int run = 0, piece_tiles = 0;
  if (!P.whole)
    for (int base = 0; base < nb; base += THREADS) {
      keys(base, c == 0);
      // Where there are fewer units than CTAs, pieces of L tiles that start with their unit, one a CTA, if an
      // L of the even share to three tiles more gives few enough of them: a CTA's second unit costs it as
      // much as four tiles (5 x 25 units behind a window 29.7 -> 25.7 us, 128 heads over 131 k keys 60 -> 56; 32 heads
      // over 1-2 k and 8-16 k keys, even ranges and pieces: 2 units 14.0 and 14.2, 23.0 and 21.1; 8 units 15.2 and 15.6,
      // 26.4 and 24.0; 16 units 20.3 and 16.4, 38.2 and 36.3; 32 units 22.2 and 18.3, 56.1 and 55.8; 48 units 23.6 and
      // 20.8, 74.4 and 75.2; 64 units 26.7 and 24.4, 92.2 and 92.5).  The units count as padded to whole pieces.
      if (units <= (int)gridDim.x) {
        const int even = (total(nt) * P.groups + gridDim.x - 1) / gridDim.x;
        if (even > 1) {
#pragma unroll 1
          for (int L = even; L <= even + 3 && !piece_tiles; ++L)
            if (total(nt > 0 ? (nt - 1) / L + 1 : 0) * P.groups <= (int)gridDim.x) piece_tiles = L;
          if (piece_tiles && nt > 0) nt = ((nt - 1) / piece_tiles + 1) * piece_tiles;
        }
      }
      run = scan(run);
    }
  // the first min(gridDim, U) CTAs take one range each, so none is empty
  const int U = P.whole ? units : run * P.groups;
  const int G = piece_tiles ? U / piece_tiles : min((int)gridDim.x, max(U, 1));
  const Ranges ranges = piece_tiles ? Ranges{piece_tiles, 0} : Ranges{U / G, U % G};
  const int u0 = c < G ? ranges.begin(c) : U, u1 = c < G ? ranges.begin(c + 1) : U;
  if (!P.whole) {
    run = 0;
    for (int base = 0; base < nb; base += THREADS) {
      if (nb > THREADS) {
        keys(base, false);
        run = scan(run);
      }
      const int b = base + tid;
      if (b < nb) {
        if (nt > 0 && u1 > u0 && u0 >= excl * P.groups && u0 < (excl + nt) * P.groups) {
          const int in = u0 - excl * P.groups;
          sh->first_unit = b * P.groups + in / nt;
          sh->first_tile = in % nt;
        }
        if (c == 0) {
          pdl_wait();                      // the workspace may still be read by the kernel before
          P.first_tile[b] = excl;
          if (b == nb - 1) {
            P.first_tile[nb] = excl + nt;
            P.first_tile[nb + 1] = piece_tiles;
          }
        }
      }
    }
  }
  __syncthreads();
  if (warp == 11) {
    // lane i: the i-th unit from the first one on
    const int first = P.whole ? u0 : sh->first_unit, unit = first + lane;
    Piece p{};
    if (u1 > u0 && unit < (P.whole ? u1 : units)) {
      p.unit = unit;
      p.b = unit / P.groups;
      p.k = keys_of(P, p.b, P.whole && unit % P.groups == 0);
      p.t0 = lane ? 0 : sh->first_tile;
    }
    const int have = p.k.nt - p.t0;
    int upto = have;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    p.n = P.whole ? have : max(min(have, u1 - u0 - (upto - have)), 0);
    if (piece_tiles && lane > 0) p.n = 0;
    const uint32_t mine = __ballot_sync(0xffffffffu, p.n > 0);
    if (p.n > 0) sh->piece[__popc(mine & ((1u << lane) - 1u))] = p;
    const uint32_t none = __ballot_sync(0xffffffffu, P.whole && unit < u1 && p.n == 0);
    if (lane == 31) {
      sh->pieces = __popc(mine);
      sh->more_unit = first + 32;
      sh->more_left = P.whole || piece_tiles ? 0 : u1 - u0 - upto;
      sh->empty = none;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem_slot;
  const SegIter start{};
  const bool work = sh->pieces > 0;
  // (lengths, windows, positions and page rows are inputs of the call; what the kernel
  // before wrote, queries and entries, is read behind pdl_wait only)

  // Two warps issue: the scores, as soon as a tile is there, and the outputs, as soon as its weights
  // are; a commit and the look at a barrier cost 40 and 200 cycles, which pass while the
  // other's products run.  (S(g) comes behind O(g - 2), which frees its tile's place, and behind the
  // reading of S(g - 2), which P(g - 2) follows.)
  if (warp == 8) {
    if (work) {
      const uint32_t one = elect_one();
      const uint32_t id_s = idesc_f8(KT, 2 * NR);                            // K-major A and B
      const uint32_t id_r = idesc_f16(KT, NR, false);
      const uint32_t hi = (uint32_t)(smem_desc_sw128(smem) >> 32);
      const uint32_t dK = (uint32_t)smem_desc_sw128(smem);
      const uint32_t dQ = (uint32_t)smem_desc_sw128(smem + OFF_Q), dR = (uint32_t)smem_desc_sw128(smem + OFF_QR);
      constexpr uint32_t U_STAGE = STAGE_BYTES / 16, U_CH = CH_BYTES / 16, U_Q = Q_CH_BYTES / 16;
      SegIter it = start;
      Seg s{};
      uint32_t g = 0, kseg = 0;
      bool ok = true;
      while (ok && warp_same(next_seg(P, sh, it, s))) {
        const int n = warp_same(s.n);
        ok = warp_wait(B, &B->q_full, kseg & 1, status);
        for (int t = 0; ok && t < n; ++t, ++g) {
          const uint32_t st = g % STAGES, d = tmem + 128 * (g & 1);
          if (g >= 2 && !(ok = warp_wait(B, &B->p_full[g & 1], ((g >> 1) - 1) & 1, status))) break;
          if (!(ok = warp_wait(B, &B->full[st], (g / STAGES) & 1, status))) break;
          tc_fence_after();
          const uint32_t a = dK + st * U_STAGE;
          if (one) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_f16(d + 64, desc(hi, a + 4 * U_CH + 2 * i), desc(hi, dR + 2 * i), id_r, i > 0);
            mma_commit(&B->empty[st][4]);
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
#pragma unroll
              for (int i = 0; i < 4; ++i) mma_f8(d, desc(hi, a + q * U_CH + 2 * i), desc(hi, dQ + q * U_Q + 2 * i), id_s, q + i > 0);
            }
            mma_commit(&B->s_full[g & 1]);
          }
          __syncwarp();
        }
        ++kseg;
      }
      if (one) {
        mma_commit(&B->drain);
        mbar_wait(&B->drain, 0, status);
      }
    }
  } else if (warp == 9) {
    if (work) {
      const uint32_t one = elect_one();
      const uint32_t id_o = idesc_f8(KT, 2 * NR) | (1u << 15) | (1u << 16);  // A and B MN-major
      const uint32_t hv = (uint32_t)(smem_desc_sw128_mn(smem, CH_BYTES) >> 32), dV = (uint32_t)smem_desc_sw128_mn(smem, CH_BYTES);
      const uint32_t hp = (uint32_t)(smem_desc_sw64_mn(smem + OFF_P) >> 32), dP = (uint32_t)smem_desc_sw64_mn(smem + OFF_P);
      constexpr uint32_t U_STAGE = STAGE_BYTES / 16, U_CH = CH_BYTES / 16;
      constexpr uint32_t U_P = P_BYTES / 16, U_VSTEP = 32 * 128 / 16, U_PSTEP = 32 * 64 / 16;
      SegIter it = start;
      Seg s{};
      uint32_t g = 0;
      bool ok = true;
      while (ok && warp_same(next_seg(P, sh, it, s))) {
        const int n = warp_same(s.n);
        for (int t = 0; t < n; ++t, ++g) {
          const uint32_t st = g % STAGES;
          // (the tile itself, whose scores the other warp issued, and its weights)
          if (!(ok = warp_wait(B, &B->full[st], (g / STAGES) & 1, status))) break;
          if (!(ok = warp_wait(B, &B->p_full[g & 1], (g >> 1) & 1, status))) break;
          tc_fence_after();
          const uint32_t a = dV + st * U_STAGE, p = dP + (g & 1) * U_P;
          if (one) {
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma_f8(tmem + TM_O + 64 * q, desc(hv, a + q * U_CH + i * U_VSTEP), desc(hp, p + i * U_PSTEP), id_o, t > 0 || i > 0);
              mma_commit(&B->empty[st][q]);
            }
            mma_commit(&B->o_done);
            if (t == n - 1) mma_commit(&B->o_seg);
          }
          __syncwarp();
        }
      }
      if (one) {
        mma_commit(&B->drain_o);
        mbar_wait(&B->drain_o, 0, status);
      }
    }
  } else if (warp >= 10) {
    if (work) {
      uint32_t g = 0;
      bool ok = true;
      // ---- copies: the rotary chunk, chunks 0 and 2 here, 1, 3 and the scales in the other warp, each
      // as its place comes free; lane i takes page segment i of a chunk, and holds the number of page
      // `base + i` and of the 32 behind them ----
      const int ps = P.rule.page_size, past_end = P.rule.num_pages * ps, segs = KT / P.seg_rows;
      const uint32_t scale_bytes = P.seg_rows * 4;
      const uint32_t one = elect_one();
      if (one) {
        prefetch_tmap(&P.tmL);
        prefetch_tmap(&P.tmR);
      }
      SegIter it = start;
      Seg s{};
      bool have = next_seg(P, sh, it, s);
      const int32_t* table = P.rule.block_table + (long)s.b * P.rule.max_pages;
      auto pages = [&](const int32_t* t, int at) { return t[min(at + lane, P.rule.max_pages - 1)]; };
      // page and row of a tile's first key
      int page = (s.k.j_lo + s.t0 * KT) / ps, row = s.k.j_lo + s.t0 * KT - page * ps;
      int base = page, cur = pages(table, base), ahead = pages(table, base + 32);
      pdl_wait();
      while (ok && have) {
        const Seg was = s;
        for (int t = 0; t < was.n && ok; ++t, ++g) {
          const uint32_t st = g % STAGES, ph = (g / STAGES) & 1;
          const int j0 = was.k.j_lo + (was.t0 + t) * KT;
          uint8_t* dst = smem + st * STAGE_BYTES;
          if (t == was.n - 1) {
            // the next segment's pages are on their way while this one's last tile waits for its place
            have = next_seg(P, sh, it, s);
          }
          if (page >= base + 32) {
            base += 32;
            cur = ahead;
            ahead = pages(table, base + 32);
          }
          // (32 pages are whole tiles: a tile's segments lie in one lot)
          const int pg = __shfl_sync(0xffffffffu, cur, page - base + min(lane, segs - 1));
          int y = past_end;                              // (zeros)
          if (lane < segs && j0 + lane * P.seg_rows < was.k.n) {
            if (pg >= 0 && pg < P.rule.num_pages) y = pg * ps + row;
            else set_status(status, MLA_DEV_BAD_PAGE);
          }
          if (segs > 1) {
            page += segs;
          } else if ((row += KT) == ps) {
            row = 0;
            ++page;
          }
          auto copy = [&](int chunk) {
            ok = ok && warp_wait(B, &B->empty[st][chunk], ph ^ 1, status);
            if (!ok) return;
            if (one && chunk == 4) mbar_arrive_expect_tx(&B->full[st], STAGE_BYTES + KT * 4);
#pragma unroll 1
            for (int i = 0; i < segs; ++i) {
              const int yi = __shfl_sync(0xffffffffu, y, i);
              uint8_t* to = dst + chunk * CH_BYTES + i * P.seg_rows * 128;
              if (one) {
                if (chunk < 4) tma_load_3d(to, &P.tmL, &B->full[st], 0, yi, chunk);
                else tma_load_3d(to, &P.tmR, &B->full[st], 0, yi, 0);
                // the scales with a chunk that is freed behind their use
                if (chunk == 1)
                  bulk_load(&sh->scale[st][i * P.seg_rows], yi == past_end ? no_page_scales.of : P.scale + yi, scale_bytes,
                            &B->full[st]);
              }
            }
          };
          if (warp == 10) {
            copy(4);
            copy(0);
            copy(2);
          } else {
            copy(1);
            copy(3);
          }
        }
        if (have && s.first) {
          table = P.rule.block_table + (long)s.b * P.rule.max_pages;
          page = (s.k.j_lo + s.t0 * KT) / ps;
          row = s.k.j_lo + s.t0 * KT - page * ps;
          base = page;
          cur = pages(table, base);
          ahead = pages(table, base + 32);
        }
      }
      // the copies in flight land before the CTA exits (after a wait that gave up, a part of
      // one tile more; that wait gives up, too)
      if (!ok) ++g;
      for (uint32_t i = g > STAGES ? g - STAGES : 0; lane == 0 && i < g; ++i)
        mbar_wait(&B->full[i % STAGES], (i / STAGES) & 1, status);
    }
  } else if (work) {
    // ---- softmax: thread = key (TMEM lane), rows 16 grp .. 16 grp + 15.  After a wait
    // that gave up everything runs on to its end (the barriers below count every thread). ----
    const int grp = warp / 4, wq = warp % 4, key = tid % 128;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    const int r0 = grp * HALF, live = P.rule.T * P.rule.H;
    const float c2 = P.scale_log2;
    SegIter it = start;
    Seg s{};
    uint32_t g = 0, kseg = 0;
    int u_seg = u0;                  // global index of the segment's first tile
    pdl_wait();
    uint32_t alive = 0;
    float l[HALF], m[HALF];
    Seg done{};                            // the segment whose tiles are done
    bool have = next_seg(P, sh, it, s), ended = false;
    while (true) {
      const int grp0 = (s.unit % P.groups) * NR;         // the unit's first row in its block
      if (have) {
        // ---- queries: four rows a warp, each split in two e4m3 numbers over a power of two (the
        // S of the segment before are done: its last tile's weights have been made); all four are on their way
        // at once, since what comes later waits behind the tiles' copies ----
        uint4 v[Q_ROWS][2];
        uint32_t vr[Q_ROWS];
#pragma unroll
        for (int i = 0; i < Q_ROWS; ++i) {
          const int r = warp * Q_ROWS + i;
          const bool in = grp0 + r < live;
          const uint4* src = reinterpret_cast<const uint4*>(P.q + ((long)s.b * live + (in ? grp0 + r : 0)) * ENTRY);
          v[i][0] = in ? src[2 * lane] : make_uint4(0, 0, 0, 0);
          v[i][1] = in ? src[2 * lane + 1] : make_uint4(0, 0, 0, 0);
          vr[i] = in ? reinterpret_cast<const uint32_t*>(src + RANK / 8)[lane] : 0u;
        }
#pragma unroll 1
        for (int i0 = 0; i0 < Q_ROWS; i0 += Q_BATCH) {
          if (i0 > 0) {
#pragma unroll
            for (int i = 0; i < Q_BATCH; ++i) {
              v[i][0] = v[Q_BATCH + i][0];
              v[i][1] = v[Q_BATCH + i][1];
              vr[i] = vr[Q_BATCH + i];
            }
          }
#pragma unroll
          for (int i = 0; i < Q_BATCH; ++i) {
            const int r = warp * Q_ROWS + i0 + i;
            const uint32_t u[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, max(u[e] & 0x7fffu, (u[e] >> 16) & 0x7fffu));
            top = __reduce_max_sync(0xffffffffu, top);
            const int k = max((int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 96u ? 1 : 0), -100);
            const float inv = pow2(-k);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float f[4] = {__uint_as_float(u[2 * e] << 16) * inv, __uint_as_float(u[2 * e] & 0xffff0000u) * inv,
                                  __uint_as_float(u[2 * e + 1] << 16) * inv,
                                  __uint_as_float(u[2 * e + 1] & 0xffff0000u) * inv};
              const uint32_t h0 = e4m3x2(f[0], f[1]), h1 = e4m3x2(f[2], f[3]);
              const float2 g0 = from_e4m3x2(h0), g1 = from_e4m3x2(h1);
              hi[e] = h0 | h1 << 16;
              lo[e] = e4m3x2(f[0] - g0.x, f[1] - g0.y) | e4m3x2(f[2] - g1.x, f[3] - g1.y) << 16;
            }
            uint8_t* q = smem + OFF_Q + (lane / 8) * Q_CH_BYTES + (((lane % 8) ^ (r & 7)) << 4);
            *reinterpret_cast<uint4*>(q + r * 128) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(q + (NR + r) * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<uint32_t*>(smem + OFF_QR + r * 128 + (((lane / 4) ^ (r & 7)) << 4) + (lane % 4) * 4) = vr[i];
            // (a query that is no number makes its row none, whatever its bytes became)
            if (lane == 0) sh->q_scale[r] = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : pow2(k) * c2;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B->q_full);
      }
      if (ended) {
        // ---- end of a segment: its sums, then the output or the piece's slot ----
        const int row0 = (done.unit % P.groups) * NR;
        const int unit0 = u_seg - done.t0;              // the unit's first tile
        const bool direct = P.whole || ranges.cta_of(unit0) == ranges.cta_of(unit0 + done.k.nt - 1);
        const long slot = slot_of(c, unit0 < u0, gridDim.x);
        {
          const float sum = transpose_sum16(l, lane);
          if (lane < HALF) sh->sum[grp][wq][lane] = sum;
        }
        softmax_sync();
        if (warp == 0) {
          const int h = lane / HALF, r = lane % HALF;
          const float sum = (sh->sum[h][0][r] + sh->sum[h][1][r]) + (sh->sum[h][2][r] + sh->sum[h][3][r]);
          const bool dead = !((alive >> lane) & 1) || sum == 0.f;
          const float l2 = dead ? -INFINITY : sh->m[lane] - P_LOG2 + __log2f(sum);
          float inv = dead ? 0.f : fast_rcp(sum), keep = 0.f, all = l2;
          if (!done.first) {
            const float old = sh->run_lse[lane], top = fmaxf(old, l2);
            const float a = old == -INFINITY ? 0.f : fast_exp2(old - top), b = l2 == -INFINITY ? 0.f : fast_exp2(l2 - top);
            const float part = a + b == 0.f ? 0.f : fast_rcp(a + b);
            keep = a * part;
            inv = dead ? 0.f : inv * b * part;
            all = a + b == 0.f ? -INFINITY : top + __log2f(a + b);
          }
          sh->run_lse[lane] = all;
          sh->inv[lane] = inv;
          sh->keep[lane] = keep;
          if (done.last) {
            if (!direct) P.part_lse[slot * NR + lane] = all;
            else if (P.lse && row0 + lane < live)
              P.lse[(long)done.b * live + row0 + lane] = all == -INFINITY ? all : all * 0.6931471805599453f;
          }
        }
        softmax_sync();
        wait_bar(B, &B->o_seg, kseg & 1, status);
        tc_fence_after();
        float inv[HALF];
        lds16(sh->inv + r0, inv);
        const uint64_t stay = l2_policy_evict_last();
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float o[HALF], e[HALF];
          const uint32_t at = tmem + TM_O + 2 * NR * q + r0 + lanes;
          tmem_ld16_nowait(at, o);
          tmem_ld16_nowait(at + NR, e);
          tmem_ld_wait();
          tmem_reg_fence16(o);
          tmem_reg_fence16(e);
          // partials lie [quarter][four rows][dim][row]: a thread's four rows of a dim are one store
          float4* part = reinterpret_cast<float4*>(P.part + slot * NR * RANK) + (q * (NR / 4) + r0 / 4) * 128 + key;
#pragma unroll
          for (int r = 0; r < HALF; ++r) {
            const float v = fmaf(e[r], 1.f / LO_UP, o[r]);
            o[r] = inv[r] == 0.f ? 0.f : v * inv[r];
          }
          if (!done.first) {
#pragma unroll
            for (int r = 0; r < HALF; r += 4) {
              const float4 old = part[r / 4 * 128], k = *reinterpret_cast<const float4*>(sh->keep + r0 + r);
              if (k.x != 0.f) o[r] = fmaf(old.x, k.x, o[r]);
              if (k.y != 0.f) o[r + 1] = fmaf(old.y, k.y, o[r + 1]);
              if (k.z != 0.f) o[r + 2] = fmaf(old.z, k.z, o[r + 2]);
              if (k.w != 0.f) o[r + 3] = fmaf(old.w, k.w, o[r + 3]);
            }
          }
          if (done.last && direct) {
            // neighbouring lanes' dims in one store: the even lane takes the first 8 rows
            const bool odd = lane & 1;
            __half* out = P.o_lat + ((long)done.b * live + row0 + r0 + (odd ? HALF / 2 : 0)) * RANK + 128 * q + (key & ~1);
#pragma unroll
            for (int r = 0; r < HALF / 2; ++r) {
              const float mine = odd ? o[r + HALF / 2] : o[r], give = odd ? o[r] : o[r + HALF / 2];
              const float got = __shfl_xor_sync(0xffffffffu, give, 1);
              if (row0 + r0 + (odd ? HALF / 2 : 0) + r < live)
                *reinterpret_cast<__half2*>(out + (long)r * RANK) =
                    odd ? __floats2half2_rn(got, mine) : __floats2half2_rn(mine, got);
            }
          } else {
            // (kept in L2 for the join: the cache's stream would push them out)
#pragma unroll
            for (int r = 0; r < HALF; r += 4)
              st_global_hint4(part + r / 4 * 128, make_float4(o[r], o[r + 1], o[r + 2], o[r + 3]), stay);
          }
        }
        tc_fence_before();
        u_seg += done.n;
        g += done.n;
        ++kseg;
      }
      if (!have) break;
      const int k_begin = s.k.j_lo + s.t0 * KT;
      softmax_sync();                      // the segment before is done with the rows' state
      if (warp == 0) {
        const int row = grp0 + lane, i = row / P.rule.H;
        int lo = 0, hi = 0;
        bool see = row < live;
        if (see) {
          see = !P.rule.q_visible || P.rule.q_visible[(long)s.b * P.rule.T + i] != 0;
          if (P.rule.parent)
            see = tree::in_tree(P.rule, P.rule.parent + (long)s.b * P.rule.T, i, true) && see;
          if (see) {
            lo = s.k.W > 0 ? min(tree::window_start(P.rule.positions[(long)s.b * P.rule.T + i], s.k.W), s.k.n) : 0;
            hi = s.k.ctx;
          }
        }
        sh->lo[lane] = lo;
        sh->hi[lane] = hi;
        if (s.first) sh->run_lse[lane] = -INFINITY;
        const int fl = __reduce_max_sync(0xffffffffu, see ? lo : 0);
        const int fh = __reduce_min_sync(0xffffffffu, see ? hi : 0x7fffffff);
        const int al = __reduce_min_sync(0xffffffffu, see ? lo : 0x7fffffff);
        const int ah = __reduce_max_sync(0xffffffffu, see ? hi : 0);
        const uint32_t sees = __ballot_sync(0xffffffffu, see);
        if (lane == 0) {
          sh->fast_lo = fl;
          sh->fast_hi = sees ? fh : 0;
          sh->any_lo = al;
          sh->any_hi = ah;
          sh->alive = sees;
        }
      }
      softmax_sync();
      alive = sh->alive;
      const int fast_lo = sh->fast_lo, fast_hi = sh->fast_hi, any_lo = sh->any_lo, any_hi = sh->any_hi;
#pragma unroll
      for (int r = 0; r < HALF; ++r) {
        l[r] = 0.f;
        m[r] = 0.f;                        // P_LOG2 less the references (0 before the first)
      }
      float m_lane = -INFINITY, top = -INFINITY;   // row lane % 16: its reference, its largest so far
#pragma unroll 1
      for (int t = 0; t < s.n; ++t) {
        asm volatile("" : "+r"(t));        // (one copy of the loop's code, none peeled off)
        const uint32_t gg = g + t, buf = gg & 1;
        const int j0 = k_begin + t * KT, j = j0 + key;
        const bool fast = j0 >= fast_lo && j0 + KT <= fast_hi;
        const bool bits = !fast && P.rule.parent && j0 + KT > s.k.ctx;
        if (__builtin_expect(bits, 0)) {
          // which keys each row sees: the group's first 64 threads take half a tile of a row each
          group_sync(grp);                 // (the tile before is done with the words)
          if (key < 2 * NR) {
            const int r = key / 2, h = key % 2;
            unsigned long long m = 0;
            if ((alive >> r) & 1)
              m = tree::key_bits(P.rule, s.b, (grp0 + r) / P.rule.H, true, s.k.n, s.k.W, s.k.ctx, j0 + 64 * h);
            sh->seen[grp][r][2 * h] = (uint32_t)m;
            sh->seen[grp][r][2 * h + 1] = (uint32_t)(m >> 32);
          }
          group_sync(grp);
        }
        wait_bar(B, &B->full[gg % STAGES], (gg / STAGES) & 1, status);       // (for the scales; long done)
        wait_bar(B, &B->s_full[buf], (gg >> 1) & 1, status);
        tc_fence_after();
        float ks = sh->scale[gg % STAGES][key];
        // what is below takes a scale by its exponent: another number is as NaN, and reported where a row sees the key
        bool odd = false;
        if (__builtin_expect(!sound_scale(ks), 0)) {
          odd = !isnan(ks);
          ks = __uint_as_float(0x7fc00000u);
        }
        float x[HALF];
        {
          float y[HALF], z[HALF];
          const uint32_t ts = tmem + 128 * buf + lanes;
          tmem_ld16_nowait(ts + r0, x);
          tmem_ld16_nowait(ts + NR + r0, y);
          tmem_ld16_nowait(ts + 2 * NR + r0, z);
          tmem_ld_wait();
          tmem_reg_fence16(x);
          tmem_reg_fence16(y);
          tmem_reg_fence16(z);
          float qs[HALF];
          lds16(sh->q_scale + r0, qs);
          const float kexp = (float)((int)(__float_as_uint(ks) >> 23) - 127);    // log2 of a power of two
          const float2 ks2 = make_float2(ks, ks), c22 = make_float2(c2, c2), kexp2 = make_float2(kexp, kexp);
#pragma unroll
          for (int r = 0; r < HALF; r += 2) {
            const float2 v = fma2(add2(make_float2(x[r], x[r + 1]), make_float2(y[r], y[r + 1])),
                                  mul2(make_float2(qs[r], qs[r + 1]), ks2),
                                  fma2(make_float2(z[r], z[r + 1]), c22, kexp2));
            x[r] = v.x;
            x[r + 1] = v.y;
          }
        }
        if (__builtin_expect(!fast, 0)) {
          bool seen = false;
          if (bits) {
#pragma unroll
            for (int r = 0; r < HALF; ++r)
              if (!((sh->seen[grp][r0 + r][wq] >> lane) & 1)) x[r] = -INFINITY;
            for (int r = 0; r < NR; ++r) seen |= (sh->seen[grp][r][wq] >> lane) & 1;
          } else {
            seen = j >= any_lo && j < any_hi;
            if (fast_lo == any_lo && fast_hi == any_hi) {      // (the rows that see anything see the same: little code)
              if (!seen)
#pragma unroll
                for (int r = 0; r < HALF; ++r) x[r] = -INFINITY;
            } else {
#pragma unroll
              for (int r = 0; r < HALF; ++r)
                if (j < sh->lo[r0 + r] || j >= sh->hi[r0 + r]) x[r] = -INFINITY;
            }
          }
          // a key that no row of the unit sees may hold any bytes: its latent becomes zero before
          // it meets its weights, which are zero (S is done with it, and O waits for P)
          if (!seen) {
            odd = false;
            uint8_t* row = smem + (gg % STAGES) * STAGE_BYTES + 2 * grp * CH_BYTES + key * 128;
#pragma unroll 1
            for (int q = 0; q < 2; ++q)
#pragma unroll 1
              for (int i = 0; i < 8; ++i)      // (neighbouring lanes' rows in different banks)
                *reinterpret_cast<uint4*>(row + q * CH_BYTES + ((i ^ lane) & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        if (__builtin_expect(odd, 0)) set_status(status, MLA_DEV_BAD_SCALE);
        {
          float y[HALF];
#pragma unroll
          for (int r = 0; r < HALF; ++r) y[r] = warp_max(x[r]);
          if (lane == 0) {
#pragma unroll
            for (int r = 0; r < HALF; r += 4)
              *reinterpret_cast<float4*>(&sh->wpart[buf][grp][wq][r]) = make_float4(y[r], y[r + 1], y[r + 2], y[r + 3]);
          }
          group_sync(grp);
          const float* part = &sh->wpart[buf][grp][0][lane % HALF];
          top = fmaxf(top, fmaxf(fmaxf(part[0], part[HALF]), fmaxf(part[2 * HALF], part[3 * HALF])));
          const bool up = top > m_lane + SLACK_LOG2;
          if (__builtin_expect(__any_sync(0xffffffffu, up), 0)) {               // (the same for every warp of the group)
            const float m_new = fmaxf(m_lane, ceilf(top));
            const float f = m_lane == -INFINITY ? 1.f : fast_exp2(m_lane - m_new);
            m_lane = m_new;
#pragma unroll
            for (int r = 0; r < HALF; ++r) {
              m[r] = __shfl_sync(0xffffffffu, m_new == -INFINITY ? 0.f : P_LOG2 - m_new, r);
              y[r] = __shfl_sync(0xffffffffu, f, r);
              l[r] *= y[r];
            }
            if (t > 0) {
              // O(g - 1) is issued behind S(g), and O(g) only behind this tile's P
              wait_bar(B, &B->o_done, (gg - 1) & 1, status);
              tc_fence_after();
#pragma unroll 1
              for (int q = 0; q < 8; ++q) {
                float o[HALF];
                const uint32_t at = tmem + TM_O + NR * q + r0 + lanes;
                tmem_ld16_nowait(at, o);
                tmem_ld_wait();
                tmem_reg_fence16(o);
#pragma unroll
                for (int r = 0; r < HALF; ++r) o[r] *= y[r];
                tmem_st16(at, o);
              }
            }
          }
        }
        // weights 2^7 w and their split; the sum takes them over the key's scale
        // (finite also for the scale of an entry that holds nothing, whose weights are 0 or NaN)
        const uint32_t ks_exp = __float_as_uint(ks) >> 23;
        const float inv_ks = ks_exp - 1u < 253u ? __uint_as_float((254u - ks_exp) << 23) : 1.f;
        uint32_t hi[HALF / 4], lo[HALF / 4];
#pragma unroll
        for (int r = 0; r < HALF; r += 2) {
          const float2 d = add2(make_float2(x[r], x[r + 1]), make_float2(m[r], m[r + 1]));
          const float2 w = make_float2(fast_exp2(d.x), fast_exp2(d.y));
          const float2 sum = fma2(w, make_float2(inv_ks, inv_ks), make_float2(l[r], l[r + 1]));
          l[r] = sum.x;
          l[r + 1] = sum.y;
          const uint32_t h = e4m3x2(w.x, w.y);
          const float2 f = from_e4m3x2(h);
          // (exact: the difference, and a power of two times it)
          const float2 rest = mul2(fma2(f, make_float2(-1.f, -1.f), w), make_float2(LO_UP, LO_UP));
          const uint32_t e = e4m3x2(rest.x, rest.y);
          if (r % 4 == 0) {
            hi[r / 4] = h;
            lo[r / 4] = e;
          } else {
            hi[r / 4] |= h << 16;
            lo[r / 4] |= e << 16;
          }
        }
        uint8_t* p = smem + OFF_P + buf * P_BYTES + key * 64;
        const int sw = (key >> 1) & 3;
        *reinterpret_cast<uint4*>(p + ((grp ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(p + (((2 + grp) ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&B->p_full[buf]);
      }
      if (wq == 0 && lane < HALF) sh->m[r0 + lane] = m_lane;
      done = s;
      ended = true;
      have = next_seg(P, sh, it, s);
    }
  }
  // (here, not earlier: a join that waits on every SM from the start costs the long cases a tenth)
  if (tid == 0) pdl_trigger();
  pdl_wait();        // (a no-op for the threads that waited already)
  for (uint32_t none = sh->empty; none; none &= none - 1) {      // (other than of whole units: the join's)
    const int unit = u0 + __ffs(none) - 1, rows = P.rule.T * P.rule.H;
    const int n = min(NR, rows - unit % P.groups * NR);
    const long row = (long)(unit / P.groups) * rows + unit % P.groups * NR;
    for (int i = tid; i < n * (RANK / 8); i += THREADS)
      reinterpret_cast<uint4*>(P.o_lat + row * RANK)[i] = make_uint4(0, 0, 0, 0);
    if (P.lse && tid < n) P.lse[row + tid] = -INFINITY;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, TMEM_COLS);
}

// Grid (unit, 32 DIMS value dims): the pieces of each row added by log-sum-exp in CTA order.  Thread
// i: rows 4 (i / 32) .. + 3 of dims i % 32 + 32 j; 16 / DIMS pieces' numbers are in flight at once.
// Few units are shared by more CTAs (DIMS = 1), since each has many pieces then.
constexpr int JOIN_THREADS = 256;
template <int DIMS>
__global__ void __launch_bounds__(JOIN_THREADS, 2) join8_kernel(const __grid_constant__ Params P, int ctas) {
  constexpr int JOIN_LOADS = 16 / DIMS;
  extern __shared__ float w_s[];           // [pieces][32]
  __shared__ float lse_s[NR];
  pdl_trigger();
  pdl_wait();
  const int unit = blockIdx.x, part = blockIdx.y, tid = threadIdx.x;
  const int b = unit / P.groups, grp0 = (unit % P.groups) * NR, live = P.rule.T * P.rule.H;
  const int t0 = P.first_tile[b], nt = P.first_tile[b + 1] - t0, U = P.first_tile[P.num_blocks] * P.groups;
  const long first_row = (long)b * live + grp0;
  const int ra = 4 * (tid / 32), da = tid % 32;
  float acc[DIMS][4];                      // [j][row]
#pragma unroll
  for (int j = 0; j < DIMS; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  if (nt > 0) {
    const int G = min(ctas, U), u = t0 * P.groups + (unit % P.groups) * nt;
    const int piece_tiles = P.first_tile[P.num_blocks + 1];
    const Ranges ranges = piece_tiles ? Ranges{piece_tiles, 0} : Ranges{U / G, U % G};
    const int f = ranges.cta_of(u), cnt = ranges.cta_of(u + nt - 1) - f + 1;
    if (cnt == 1) return;
    for (int i = tid; i < cnt * NR; i += JOIN_THREADS) w_s[i] = P.part_lse[slot_of(f + i / NR, i >= NR, ctas) * NR + i % NR];
    __syncthreads();
    {
      const int r = tid / 8, sl = tid % 8;
      float mx = -INFINITY, den = 0.f;
      bool nan = false;
      for (int s = sl; s < cnt; s += 8) {
        mx = fmaxf(mx, w_s[s * NR + r]);
        nan |= isnan(w_s[s * NR + r]);
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      for (int s = sl; s < cnt; s += 8) {
        const float l = w_s[s * NR + r];
        const float w = l == -INFINITY ? 0.f : exp2f(l - mx);
        w_s[s * NR + r] = w;
        den += w;
      }
      if (nan) den = __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      const float inv = den == 0.f ? 0.f : 1.f / den;
      for (int s = sl; s < cnt; s += 8) w_s[s * NR + r] *= inv;
      if (sl == 0) lse_s[r] = den == 0.f ? -INFINITY : mx + log2f(den);
    }
    __syncthreads();
    for (int s0 = 0; s0 < cnt; s0 += JOIN_LOADS) {
      float4 v[JOIN_LOADS][DIMS];
#pragma unroll
      for (int i = 0; i < JOIN_LOADS; ++i)
        if (s0 + i < cnt) {
          const float4* src = reinterpret_cast<const float4*>(P.part + slot_of(f + s0 + i, s0 + i > 0, ctas) * NR * RANK) +
                              (part * DIMS / 4 * (NR / 4) + ra / 4) * 128 + part * DIMS % 4 * 32 + da;
#pragma unroll
          for (int j = 0; j < DIMS; ++j) v[i][j] = src[32 * j];
        }
#pragma unroll
      for (int i = 0; i < JOIN_LOADS; ++i)
        if (s0 + i < cnt) {
          const float4 w = *reinterpret_cast<const float4*>(w_s + (s0 + i) * NR + ra);
#pragma unroll
          for (int j = 0; j < DIMS; ++j) {
            acc[j][0] = fmaf(w.x, v[i][j].x, acc[j][0]);
            acc[j][1] = fmaf(w.y, v[i][j].y, acc[j][1]);
            acc[j][2] = fmaf(w.z, v[i][j].z, acc[j][2]);
            acc[j][3] = fmaf(w.w, v[i][j].w, acc[j][3]);
          }
        }
    }
  } else if (tid < NR) {
    lse_s[tid] = -INFINITY;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (grp0 + ra + r < live) {
      __half* out = P.o_lat + (first_row + ra + r) * RANK + 32 * DIMS * part + da;
#pragma unroll
      for (int j = 0; j < DIMS; ++j) out[32 * j] = __float2half_rn(acc[j][r]);
    }
  if (part == 0 && tid < NR && grp0 + tid < live && P.lse) {
    const float l2 = lse_s[tid];
    P.lse[first_row + tid] = l2 == -INFINITY ? l2 : l2 * 0.6931471805599453f;
  }
}

// The keys that each query sees, counted with the kernel's own rule: a warp a token.
__global__ void __launch_bounds__(128) seen8_kernel(const tree::Rule a, long tokens, int32_t* stats) {
  const long m = blockIdx.x * 4L + threadIdx.x / 32;
  if (m >= tokens) return;
  const long b = m / a.T;
  const int i = (int)(m % a.T), lane = threadIdx.x % 32;
  int W, ctx, count = 0, first = 0x7fffffff, last = -1;
  const int n = tree::block_keys(a, (int)b, &W, &ctx, false);
  bool ok = !a.q_visible || a.q_visible[m] != 0;
  if (a.parent && n > 0) ok = tree::in_tree(a, a.parent + b * a.T, i, false) && ok;
  for (int j = 64 * lane; j < n; j += 64 * 32) {
    const unsigned long long bits = tree::key_bits(a, b, i, ok, n, W, ctx, j);
    if (!bits) continue;
    count += __popcll(bits);
    first = min(first, j + __ffsll((long long)bits) - 1);
    last = max(last, j + 63 - __clzll((long long)bits));
  }
  count = __reduce_add_sync(0xffffffffu, count);
  first = __reduce_min_sync(0xffffffffu, first);
  last = __reduce_max_sync(0xffffffffu, last);
  if (lane == 0) {
    stats[m * 3] = count;
    stats[m * 3 + 1] = count ? first : -1;
    stats[m * 3 + 2] = last;
  }
}

int groups_of(const mla_handle* h, const mla_attn_desc_t& d) {
  return (int)(((long)d.block_len * h->lay.H + NR - 1) / NR);
}
// Whether no unit is cut.  By the table's width, since the lengths are on the device: the fullest CTA
// then has `rounds` units of `tiles` tiles, and with cuts an even share of all, whose join (a launch,
// about 4 us of the GPU and 3 of the host) and second segment a CTA cost as much as JOIN_TILES tiles (a call
// from Python, 16 rows over 300 keys: 15 us whole, 20 cut; over 640: 18.5 and 19.5, of the GPU 16.4 and 12.7;
// 64 sequences of 500 keys, 4 x 32 rows: 29 and 39; 152 of 2000 keys, 32 rows: 44 and 49).
bool whole_units(const mla_handle* h, const mla_attn_desc_t& d) {
  const long units = (long)d.num_blocks * groups_of(h, d), sms = h->num_sms;
  const long tiles = ((long)d.max_pages * h->cfg.page_size + KT - 1) / KT;
  // (what a piece of several segments puts away needs a slot)
  return tiles <= SEG_TILES && units <= 32 * sms &&
         (units + sms - 1) / sms * tiles <= (units * tiles + sms - 1) / sms + JOIN_TILES;
}
// Workspace: two slots a CTA, whatever the number of units (20 MB; a slot for each unit and CTA made 128 heads x 1
// over 131 k keys 0.5 us faster and took 64 KB a unit); none of whole units.
size_t ws_layout(const mla_handle* h, const mla_attn_desc_t& d, size_t* off_lse, size_t* off_first) {
  *off_lse = *off_first = 0;
  if (whole_units(h, d)) return 0;
  const long slots = 2L * h->num_sms;
  size_t o = align256((size_t)slots * NR * RANK * 4);
  *off_lse = o;
  o += align256((size_t)slots * NR * 4);
  *off_first = o;
  return o + align256((size_t)(d.num_blocks + 2) * 4);
}

}  // namespace

size_t attention_ws(const mla_handle* h, const mla_attn_desc_t& d) {
  size_t a, b;
  return ws_layout(h, d, &a, &b);
}

mla_status_t attention(cudaStream_t st, mla_handle* h, const tree::Rule& r, const mla_attn_desc_t& d,
                       const __nv_bfloat16* q_abs, const mla_cache8_t& c, __half* o_lat, float* lse,
                       void* ws, bool pdl) {
  const int ps = h->cfg.page_size;
  const long slots = (long)r.num_pages * ps;
  Params P;
  P.seg_rows = ps < KT ? ps : KT;
  if (!make_tmap_chunked(&P.tmL, false, c.latent, slots, RANK / 2, RANK / 2, P.seg_rows, 1) ||
      !make_tmap_2d(&P.tmR, false, c.rope, slots, ROPE, ROPE, P.seg_rows))
    return fail(MLA_ERR_CUDA, "attention8: cuTensorMapEncodeTiled failed");
  size_t off_lse, off_first;
  ws_layout(h, d, &off_lse, &off_first);
  P.rule = r;
  P.scale = c.scale;
  P.q = q_abs;
  P.o_lat = o_lat;
  P.lse = lse;
  P.part = (float*)ws;
  P.part_lse = (float*)((char*)ws + off_lse);
  P.first_tile = (int*)((char*)ws + off_first);
  P.num_blocks = d.num_blocks;
  P.groups = groups_of(h, d);
  P.whole = whole_units(h, d);
  P.scale_log2 = h->scale * 1.4426950408889634f;
  if ((double)P.num_blocks * P.groups * (((long)d.max_pages * ps + KT - 1) / KT) > 2147483647.0)
    return fail(MLA_ERR_INVALID_ARG, "attention8: too many rows and keys (2^31 tiles of 32 x 128)");
  const long units = (long)P.num_blocks * P.groups;
  static std::once_flag once;
  static cudaError_t room = cudaSuccess;
  std::call_once(once, [] {
    room = cudaFuncSetAttribute(attn8_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  });
  if (room != cudaSuccess) return cuda_fail(room, "attention8: shared memory");
  Launch L(dim3((unsigned)std::min<long>(h->num_sms, P.whole ? units : h->num_sms)), dim3(THREADS), SMEM_BYTES, st, pdl);
  MLA_CUDA_TRY(cudaLaunchKernelEx(&L.cfg, attn8_kernel, P));
  h->launches += 1;
  if (!P.whole) {
    const bool few = units <= FEW_UNITS;
    Launch J(dim3((unsigned)units, few ? 16 : 4), dim3(JOIN_THREADS), (size_t)h->num_sms * NR * 4, st, true);
    MLA_CUDA_TRY(cudaLaunchKernelEx(&J.cfg, few ? join8_kernel<1> : join8_kernel<4>, P, h->num_sms));
    h->launches += 1;
  }
  if (d.vis_stats) {
    const long tokens = (long)d.num_blocks * d.block_len;
    seen8_kernel<<<(unsigned)((tokens + 3) / 4), 128, 0, st>>>(r, tokens, d.vis_stats);
    MLA_CUDA_TRY(cudaGetLastError());
    h->launches += 1;
  }
  return MLA_OK;
}

}  // namespace cache8
}  // namespace mla
