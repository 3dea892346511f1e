// Eviction from the latent cache: which keys of a sequence stay
// (mla_cache_select) and moving their entries together (mla_cache_compact).
//
// Selection.  Per sequence of n keys with weights w: the first `sink` and the
// last `recent` keys stay, and of the others the budget - sink - recent
// heaviest (ties: the lower index).  The weights map to unsigned integers of
// the same order (NaN lowest, -0 equal to +0) and the k-th largest is found
// by three counting passes over 11, 11 and 10 bits: a pass counts the keys
// that share the digits found so far per next digit, and the digit at which
// the count from above reaches k is the next one.  After it `need` of the keys
// equal to the threshold stay.  Every warp owns a contiguous run of keys, so
// the ascending list follows from ballots and one prefix over the warps, with
// no sort.  A cluster of up to 8 CTAs shares one sequence (their counts meet
// through distributed shared memory, every CTA adding the same counts in rank
// order).  4 bytes read per key and 4 written per kept one: the work is a chain
// of latencies, not of bytes (64 sequences of 1-4 k keys 10.4 us, 2 of 131 k 24).
//
// Compaction.  Row d of the result is row src(d) >= d of the sequence (src
// ascending).  A CTA moves a chunk of rows through registers: every load of
// the chunk is issued before its first store.  In place, the rows a chunk
// overwrites may be sources of earlier chunks only (src(d') >= d' for the
// later ones), so a chunk announces its loads with a flag and waits for the
// flags of the earlier chunks that read its destination.  Chunks are numbered
// by a ticket taken when a CTA starts: whoever is waited for has started, and
// loading waits for nobody, so every wait ends.  Which chunks to wait for is read
// from the list, which has to ascend for that: a first kernel, which also clears
// the flags, looks at every list, and a sequence whose list does not ascend is
// left alone.  2 entry rows of traffic per moved row: HBM bound (64 sequences to 1024 entries of 1152 bytes, 151 MB: 31
// us, 4.9 TB/s; 16 rows a CTA, 33 us with 32).  In place the same takes 53 us: the
// lists' kernel, the tickets and the waits for earlier chunks' loads.
#include "cache8.cuh"
#include "common.cuh"
#include "tc_ptx.cuh"

#include <math.h>

#include <mutex>

namespace mla {
namespace evict {
namespace {

// ---------------------------------------------------------------------------
// Selection
// ---------------------------------------------------------------------------
constexpr int SEL_THREADS = 1024, SEL_WARPS = SEL_THREADS / 32, BINS = 2048;
constexpr int SEL_SMEM_KEYS = 32768;      // keys of a CTA held in shared memory

struct SelectArgs {
  const float* weights;
  const int32_t* kv_len;
  int32_t* keep;
  int32_t* keep_len;
  long ldw;
  int budget, sink, recent;
  uint32_t* status;
};

// Unsigned integer of the same order as the weight (larger = heavier).
__device__ __forceinline__ uint32_t order_key(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;        // NaN: lighter than anything
  if ((u << 1) == 0u) u = 0u;                             // -0 == +0
  return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int ld_cluster_int(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int2 ld_cluster_int2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ int lane_prefix(int x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if ((int)(threadIdx.x % 32) >= o) x += y;
  }
  return x;
}

// Warp w gets the sum of v (uniform in a warp) over warps 0 .. w - 1, and
// *total the sum over all.
__device__ __forceinline__ int warp_prefix(int v, int* buf, int* total) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) buf[warp] = v;
  __syncthreads();
  const int x = lane_prefix(buf[lane]);
  *total = __shfl_sync(0xffffffffu, x, 31);
  const int before = __shfl_sync(0xffffffffu, x, warp) - v;
  __syncthreads();
  return before;
}

// HELD: a CTA's keys stay in shared memory (at most SEL_SMEM_KEYS), so that two
// counts fit a word: the peers' counts are most of what crosses the cluster (8
// CTAs: 4.2 k cycles a pass with a word a count).
template <int CL, bool HELD>
__global__ void __launch_bounds__(SEL_THREADS) select_kernel(const SelectArgs a) {
  extern __shared__ uint32_t keys[];                     // this CTA's keys (HELD)
  constexpr int WORDS = HELD ? BINS / 2 : BINS;
  __shared__ __align__(8) uint32_t hist[2][WORDS];
  __shared__ int buf[32], buf2[32], found[2];
  __shared__ __align__(8) int cta_counts[2];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = CL > 1 ? (int)tc::cluster_ctarank() : 0;
  const long seq = blockIdx.x / CL;
  int n = a.kv_len[seq];
  if (n < 0 || n > a.ldw) {
    if (tid == 0 && rank == 0) set_status(a.status, MLA_DEV_BAD_LENGTH);
    n = n < 0 ? 0 : (int)a.ldw;
  }
  int32_t* keep = a.keep + seq * a.budget;
  const int kept = min(n, a.budget);
  if (rank == 0 && tid == 0) a.keep_len[seq] = kept;
  // (a step behind a budget near 2^31 passes it)
  for (long i = (long)kept + rank * SEL_THREADS + tid; i < a.budget; i += CL * SEL_THREADS) keep[i] = -1;
  if (n <= a.budget) {                                   // uniform over the cluster
    for (int i = rank * SEL_THREADS + tid; i < n; i += CL * SEL_THREADS) keep[i] = i;
    return;
  }
  const float* w = a.weights + seq * a.ldw;
  const int mid_lo = a.sink, mid_hi = n - a.recent;       // keys that compete
  int k = a.budget - a.sink - a.recent;                   // of which k stay
  // this warp's run of keys
  const int nw = CL * SEL_WARPS;
  const int wlen = ((n + nw - 1) / nw + 31) & ~31;
  const int i0 = (int)min((long)(rank * SEL_WARPS + warp) * wlen, (long)n);   // (n < 2^30)
  uint32_t* mine = keys + warp * wlen;
  if (HELD)
#pragma unroll 8
    for (int o = lane; o < wlen; o += 32) {
      const int i = i0 + o;
      mine[o] = i < n ? order_key(w[i]) : 0u;
    }
  auto key_at = [&](int o) -> uint32_t {
    return HELD ? mine[o] : (i0 + o < n ? order_key(w[i0 + o]) : 0u);
  };
  uint32_t prefix = 0, mask = 0;
  for (int i = tid; i < WORDS; i += SEL_THREADS) hist[0][i] = 0;
  __syncthreads();
  // k == 0: only the protected keys stay
  if (k > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t dmask = (1u << bits) - 1u;
      uint32_t* hp = hist[pass & 1];
#pragma unroll 8
      for (int o = lane; o < wlen; o += 32) {
        const int i = i0 + o;
        const uint32_t u = key_at(o);
        const bool in = i >= mid_lo && i < mid_hi && (u & mask) == prefix;
        const uint32_t digit = (u >> shift) & dmask;
        if (in) atomicAdd(&hp[HELD ? digit >> 1 : digit], HELD && (digit & 1) ? 0x10000u : 1u);
      }
      if (CL > 1) tc::cluster_sync_all(); else __syncthreads();
      // every CTA is done with the other array (pass - 1): clear it for pass + 1
      for (int i = tid; i < WORDS; i += SEL_THREADS) hist[(pass + 1) & 1][i] = 0;
      // counts of this thread's two bins, from the top: bins B - 1 - 2 tid, B - 2 - 2 tid
      const int bin = BINS - 1 - 2 * tid;
      int c0 = 0, c1 = 0;
      int2 from[CL];                                     // every CTA's counts, all loads in flight
#pragma unroll
      for (int r = 0; r < CL; ++r) {
        if (HELD) {
          const uint32_t v = CL == 1 ? hp[bin >> 1] : (uint32_t)ld_cluster_int(tc::mapa(tc::smem_u32(&hp[bin >> 1]), (uint32_t)r));
          from[r] = make_int2((int)(v & 0xffffu), (int)(v >> 16));
        } else {
          from[r] = CL == 1 ? *reinterpret_cast<const int2*>(&hp[bin - 1])
                            : ld_cluster_int2(tc::mapa(tc::smem_u32(&hp[bin - 1]), (uint32_t)r));
        }
      }
#pragma unroll
      for (int r = 0; r < CL; ++r) { c0 += from[r].y; c1 += from[r].x; }
      const int x = lane_prefix(c0 + c1);
      if (lane == 31) buf[warp] = x;
      __syncthreads();
      const int b = lane_prefix(buf[lane]);
      const int before = __shfl_sync(0xffffffffu, b, max(warp - 1, 0));
      const int above = (warp ? before : 0) + x - c0 - c1;   // keys in higher bins than this thread's
      if (above < k && above + c0 + c1 >= k) {
        const bool second = above + c0 < k;
        found[0] = second ? bin - 1 : bin;
        found[1] = k - above - (second ? c0 : 0);
      }
      __syncthreads();
      prefix |= (uint32_t)found[0] << shift;
      mask |= dmask << shift;
      k = found[1];
    }
  }
  const uint32_t thr = prefix;
  const int need = k;                                    // keys equal to thr that stay
  const bool none = a.budget == a.sink + a.recent;
  // 2: stays, 1: equals the threshold, 0: goes
  auto klass = [&](int o) -> int {
    const int i = i0 + o;
    if (i >= n) return 0;
    if (i < mid_lo || i >= mid_hi) return 2;
    if (none) return 0;
    const uint32_t u = key_at(o);
    return u > thr ? 2 : u == thr ? 1 : 0;
  };
  int cnt2 = 0, cnt1 = 0;
  uint32_t held2 = 0, held1 = 0;                         // (HELD) lane i: the votes of step i
#pragma unroll 4
  for (int o = lane; o < wlen; o += 32) {
    const int c = klass(o);
    const uint32_t b2 = __ballot_sync(0xffffffffu, c == 2), b1 = __ballot_sync(0xffffffffu, c == 1);
    cnt2 += __popc(b2);
    cnt1 += __popc(b1);
    if (o / 32 == lane) { held2 = b2; held1 = b1; }
  }
  int tot2, tot1;
  int before2 = warp_prefix(cnt2, buf, &tot2);
  int before1 = warp_prefix(cnt1, buf2, &tot1);
  if (CL > 1) {
    if (tid == 0) { cta_counts[0] = tot2; cta_counts[1] = tot1; }
    tc::cluster_sync_all();
    int2 from[CL];
#pragma unroll
    for (int r = 0; r < CL; ++r) from[r] = ld_cluster_int2(tc::mapa(tc::smem_u32(cta_counts), (uint32_t)r));
#pragma unroll
    for (int r = 0; r < CL; ++r)
      if (r < rank) { before2 += from[r].x; before1 += from[r].y; }
  }
  const uint32_t lt = (1u << lane) - 1u;
#pragma unroll 4
  for (int o = lane; o < wlen; o += 32) {
    uint32_t b2, b1;
    if (HELD) {
      b2 = __shfl_sync(0xffffffffu, held2, o / 32);
      b1 = __shfl_sync(0xffffffffu, held1, o / 32);
    } else {
      const int c = klass(o);
      b2 = __ballot_sync(0xffffffffu, c == 2);
      b1 = __ballot_sync(0xffffffffu, c == 1);
    }
    const int r2 = before2 + __popc(b2 & lt), r1 = before1 + __popc(b1 & lt);
    if (((b2 >> lane) & 1u) || (((b1 >> lane) & 1u) && r1 < need)) keep[r2 + min(r1, need)] = i0 + o;
    before2 += __popc(b2);
    before1 += __popc(b1);
  }
  if (CL > 1) tc::cluster_sync_all();                    // no CTA leaves while its counts may be read
}

// CTAs that share a sequence of at most ldw keys: one up to 8192 keys (8 per
// thread); beyond it the passes over a CTA's keys cost more than the cluster's
// barriers.
int select_cluster(long ldw) { return ldw <= 8192 ? 1 : ldw <= 16384 ? 2 : ldw <= 32768 ? 4 : 8; }

// ---------------------------------------------------------------------------
// Compaction
// ---------------------------------------------------------------------------
constexpr int MV_THREADS = 128, MV_UPT = 9;              // units a thread holds
constexpr int MV_UNITS = MV_THREADS * MV_UPT;            // 1152: 16 rows of 576 bf16
constexpr int MV_MAX_ROWS = 128;
constexpr int ZERO_ROWS = 4096;                          // weights a tail chunk clears
constexpr int LIST_THREADS = 256, LIST_PART = 4096;      // entries of a list that a CTA looks at
constexpr uint32_t FLAG_BUDGET = 1u << 24;

struct CompactArgs {
  char* cache;
  const int32_t *block_table, *kv_len, *keep, *keep_len, *first, *dst_table;
  const float* weights;
  float* weights_out;
  long ldk, ldw;
  long row_cap;               // longest sequence that the caller's weights have room for
  int num_pages, page_size, max_pages, dst_pages;
  int units, rows;            // 16- or 4-byte units of an entry; rows of a chunk
  int data_chunks, chunks;    // per sequence: chunks that may move rows; with those that clear weights
  int in_place;
  // in place, more than one chunk: the ticket, a flag per sequence and data chunk, and
  // per sequence and LIST_PART of its list whether that is out of order; else NULL
  int* ticket;
  int list_parts;             // parts of a list (0 without a ticket)
  int num_seqs;
  uint32_t* status;
};

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(int* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t fold(uint32_t v) { return v; }
__device__ __forceinline__ uint32_t fold(uint4 v) { return v.x ^ v.y ^ v.z ^ v.w; }

// Slot of logical key j through a page table, -1 (status set) for a bad page.
__device__ __forceinline__ long slot_of(const CompactArgs& a, const int32_t* table, int max_pages, int j) {
  const int p = j / a.page_size;
  const int pg = p < max_pages ? table[p] : -1;
  if (pg < 0 || pg >= a.num_pages) {
    set_status(a.status, MLA_DEV_BAD_PAGE);
    return -1;
  }
  return (long)pg * a.page_size + j % a.page_size;
}

// Ahead of a compaction in place: clears the ticket and the flags, and notes for
// part `blockIdx.x` (of list_parts a sequence) of the lists whether every entry lies
// above the one before it and inside the sequence.
__global__ void __launch_bounds__(LIST_THREADS) compact_lists_kernel(const CompactArgs a) {
  pdl_trigger();
  const long flags = 1 + (long)a.num_seqs * a.data_chunks;
  for (long i = blockIdx.x * (long)LIST_THREADS + threadIdx.x; i < flags; i += (long)gridDim.x * LIST_THREADS)
    a.ticket[i] = 0;
  if (a.list_parts == 0) return;
  const int seq = blockIdx.x / a.list_parts, part = blockIdx.x % a.list_parts;
  const int32_t* keep = a.keep + (long)seq * a.ldk;
  const int n = a.kv_len[seq], first = a.first ? a.first[seq] : 0;
  const int end = (int)min((long)a.keep_len[seq], a.ldk);
  int bad = 0;
#pragma unroll
  for (int k = 0; k < LIST_PART / LIST_THREADS; ++k) {
    const int i = part * LIST_PART + k * LIST_THREADS + threadIdx.x;
    if (i < end) {
      const int s = keep[i];
      bad |= s >= n || (i ? s <= keep[i - 1] : s < first);
    }
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) a.ticket[flags + blockIdx.x] = bad;
}

template <typename V>
__global__ void __launch_bounds__(MV_THREADS) compact_kernel(const CompactArgs a) {
  __shared__ long src_slot[MV_MAX_ROWS], dst_slot[MV_MAX_ROWS];
  __shared__ int s_ticket, s_ok;
  const int tid = threadIdx.x;
  pdl_wait();                                            // (in place: compact_lists_kernel)
  if (tid == 0) {
    s_ticket = a.ticket ? atomicAdd(a.ticket, 1) : (int)blockIdx.x;
    s_ok = 1;
  }
  __syncthreads();
  const int seq = s_ticket / a.chunks, c = s_ticket % a.chunks;
  const int cap = (int)min((long)a.max_pages * a.page_size, a.row_cap);
  const int n = a.kv_len[seq];
  if (n < 0 || n > cap) {
    if (tid == 0 && c == 0) set_status(a.status, MLA_DEV_BAD_LENGTH);
    return;                                              // the sequence is left as it was
  }
  const int first = a.first ? a.first[seq] : 0, nk = a.keep_len[seq];
  if (first < 0 || first > n || nk < 0 || nk > a.ldk || nk > n - first) {
    if (tid == 0 && c == 0) set_status(a.status, MLA_DEV_BAD_KEEP);
    return;                                              // as above
  }
  const int total = first + nk;
  const int base = a.in_place ? first : 0;               // rows before it are where they belong
  const int32_t* keep = a.keep + (long)seq * a.ldk;
  auto src_of = [&](int d) { return d < first ? d : keep[d - first]; };
  int* flags = a.ticket ? a.ticket + 1 + (long)seq * a.data_chunks : nullptr;
  int out_of_order = 0;                                  // in place: the list is
  for (int i = tid; i < a.list_parts; i += MV_THREADS)
    out_of_order |= a.ticket[1 + (long)a.num_seqs * a.data_chunks + (long)seq * a.list_parts + i];
  const bool data = c < a.data_chunks;
  const int d0 = data ? base + c * a.rows : 0;
  const int rows = data ? min(a.rows, total - d0) : 0;
  int w0 = 0, wn = 0;                                    // weights a tail chunk clears
  if (!data) {
    w0 = total + (c - a.data_chunks) * ZERO_ROWS;
    wn = min(ZERO_ROWS, n - w0);
    if (wn <= 0) return;
  } else if (rows <= 0) {
    return;
  }
  V hold[MV_UPT] = {};
  float wt = 0.f;
  bool wt_ok = false;
  if (data) {
    if (tid < rows) {                                    // rows <= MV_THREADS
      const int d = d0 + tid, s = src_of(d), prev = d > 0 ? src_of(d - 1) : -1;
      long ss = -1, ds = -1;
      if (s < 0 || s >= n || s < d || s <= prev) {
        set_status(a.status, MLA_DEV_BAD_KEEP);          // not ascending within the sequence: skipped
        out_of_order = 1;
      } else {
        const bool moves = !a.in_place || s != d;
        if (moves) {
          ss = slot_of(a, a.block_table + (long)seq * a.max_pages, a.max_pages, s);
          ds = a.in_place ? slot_of(a, a.block_table + (long)seq * a.max_pages, a.max_pages, d)
                          : slot_of(a, a.dst_table + (long)seq * a.dst_pages, a.dst_pages, d);
        }
        if (a.weights_out && (!moves || (ss >= 0 && ds >= 0))) {   // a weight goes with its entry
          wt = a.weights[(long)seq * a.ldw + s];
          wt_ok = true;
        }
      }
      src_slot[tid] = ds < 0 ? -1 : ss;
      dst_slot[tid] = ds;
    }
  }
  if (__syncthreads_or(out_of_order) && a.in_place) {    // (uniform over the sequence's chunks)
    if (tid == 0) set_status(a.status, MLA_DEV_BAD_KEEP);
    return;                                              // the sequence is left as it was
  }
  if (data) {
    const int live = rows * a.units;
#pragma unroll
    for (int i = 0; i < MV_UPT; ++i) {
      const int u = tid + i * MV_THREADS;
      if (u < live) {
        const long s = src_slot[u / a.units];
        if (s >= 0) hold[i] = *(reinterpret_cast<const V*>(a.cache) + s * a.units + u % a.units);
      }
    }
  }
  if (flags) {
    if (data) {
      // the flag is raised after every load of the chunk has returned: the
      // barrier's vote depends on the loaded words
      uint32_t x = __float_as_uint(wt);
#pragma unroll
      for (int i = 0; i < MV_UPT; ++i) x ^= fold(hold[i]);
      const int vote = __syncthreads_or(x == 0x9e3779b9u);
      if (tid == 0) {
        __threadfence();
        st_release(&flags[c], 1 + (vote != 0));
      }
    }
    // earlier chunks whose last source lies at or behind this chunk's first
    // destination read rows that it is about to overwrite
    const int lo = data ? d0 : w0;
    const int nchunks = (total - base + a.rows - 1) / a.rows;
    for (int e = (data ? c : nchunks) - 1 - tid; e >= 0; e -= MV_THREADS) {
      if (src_of(min(base + (e + 1) * a.rows, total) - 1) < lo) break;
      uint32_t round = 0;
      while (ld_acquire(&flags[e]) == 0) {
        if (++round > FLAG_BUDGET) {
          set_status(a.status, MLA_DEV_TIMEOUT);
          s_ok = 0;
          break;
        }
        __nanosleep(32);
      }
    }
    __syncthreads();
    if (!s_ok) return;
  } else {
    __syncthreads();                                     // in place: a row stored may be another thread's source
  }
  if (!data) {
    for (int i = tid; i < wn; i += MV_THREADS) a.weights_out[(long)seq * a.ldw + w0 + i] = 0.f;
    return;
  }
  const int live = rows * a.units;
#pragma unroll
  for (int i = 0; i < MV_UPT; ++i) {
    const int u = tid + i * MV_THREADS;
    if (u < live) {
      const int r = u / a.units;
      if (src_slot[r] >= 0)
        *(reinterpret_cast<V*>(a.cache) + dst_slot[r] * a.units + u % a.units) = hold[i];
    }
  }
  if (wt_ok) a.weights_out[(long)seq * a.ldw + d0 + tid] = wt;
}

// Unit size and rows a chunk moves for entries of `bytes` bytes.
void chunk_shape(size_t bytes, bool wide, int* units, int* rows) {
  *units = (int)(bytes / (wide ? 16 : 4));
  const int r = MV_UNITS / *units;
  *rows = r < 1 ? 1 : r > MV_MAX_ROWS ? MV_MAX_ROWS : r;
}

}  // namespace
}  // namespace evict
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_cache_select(mla_handle_t* h, const float* weights, int64_t ldw,
                                         const int32_t* kv_len, int32_t num_seqs, int32_t budget,
                                         int32_t sink, int32_t recent, int32_t* keep,
                                         int32_t* keep_len, void* stream) {
  if (!h) return fail(MLA_ERR_INVALID_ARG, "select: null handle");
  if (num_seqs < 0) return fail(MLA_ERR_INVALID_ARG, "select: num_seqs < 0");
  if (budget <= 0 || sink < 0 || recent < 0 || (long)sink + recent > budget)
    return fail(MLA_ERR_INVALID_ARG, "select: budget > 0, sink and recent >= 0, sink + recent <= budget");
  if (ldw <= 0 || ldw > 0x3fffffffL) return fail(MLA_ERR_INVALID_ARG, "select: 0 < ldw < 2^30");
  if (num_seqs == 0) return MLA_OK;
  if (!weights || !kv_len || !keep || !keep_len) return fail(MLA_ERR_INVALID_ARG, "select: null pointer");
  const int cl = evict::select_cluster(ldw);
  if ((long)num_seqs * cl > 0x7fffffffL) return fail(MLA_ERR_INVALID_ARG, "select: too many sequences");
  const long nw = (long)cl * evict::SEL_WARPS;
  const long wlen = ((ldw + nw - 1) / nw + 31) & ~31L;
  const long keys = evict::SEL_WARPS * wlen;              // of a CTA, at most
  const bool held = keys <= evict::SEL_SMEM_KEYS;
  evict::SelectArgs a{weights, kv_len, keep, keep_len, (long)ldw, budget, sink, recent, h->status};
  static std::once_flag once;
  std::call_once(once, [] {
    for (auto* k : {evict::select_kernel<1, true>, evict::select_kernel<2, true>, evict::select_kernel<4, true>,
                    evict::select_kernel<8, true>})
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, evict::SEL_SMEM_KEYS * 4);
  });
  Launch L(dim3((unsigned)(num_seqs * cl)), dim3(evict::SEL_THREADS), held ? (size_t)keys * 4 : 0,
           (cudaStream_t)stream, false, dim3((unsigned)cl, 1, 1));
  // (only clusters of 8 share more keys than fit)
  MLA_CUDA_TRY(cudaLaunchKernelEx(&L.cfg, !held      ? evict::select_kernel<8, false>
                                          : cl == 1  ? evict::select_kernel<1, true>
                                          : cl == 2  ? evict::select_kernel<2, true>
                                          : cl == 4  ? evict::select_kernel<4, true>
                                                     : evict::select_kernel<8, true>, a));
  h->launches += 1;
  return MLA_OK;
}

namespace {

// Workspace of a compaction of rows of `bytes` bytes in place.
size_t compact_ws(size_t bytes, int num_seqs, int64_t ldk) {
  int units, rows;
  evict::chunk_shape(bytes, false, &units, &rows);       // the smaller chunks
  const size_t parts = (size_t)((ldk + evict::LIST_PART - 1) / evict::LIST_PART);
  return align256(((size_t)num_seqs * ((ldk + rows - 1) / rows + parts) + 1) * sizeof(int));
}

// Longest sequence that weights [num_seqs, ldw] (or none) have room for.
long weights_cap(const float* weights, int64_t ldw) { return weights ? (long)ldw : 0x7fffffffL; }

// mla_cache_compact of an array of rows of `bytes` bytes, page by page, of sequences of at most row_cap rows.
mla_status_t compact_rows(mla_handle_t* h, void* cache, size_t bytes, int32_t num_pages,
                          const int32_t* block_table, int32_t max_pages, const int32_t* kv_len,
                          int32_t num_seqs, const int32_t* keep, int64_t ldk, const int32_t* keep_len,
                          const int32_t* first, const int32_t* dst_block_table, int32_t dst_max_pages,
                          const float* weights, float* weights_out, int64_t ldw, long row_cap, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!h) return fail(MLA_ERR_INVALID_ARG, "compact: null handle");
  if (num_seqs < 0 || max_pages <= 0 || num_pages <= 0 || ldk < 0 || ldk > 0x3fffffffL)
    return fail(MLA_ERR_INVALID_ARG, "compact: num_seqs >= 0, max_pages and num_pages > 0, 0 <= ldk < 2^30");
  if (num_seqs == 0) return MLA_OK;
  if (!cache || !block_table || !kv_len || !keep_len || (!keep && ldk > 0))
    return fail(MLA_ERR_INVALID_ARG, "compact: null pointer");
  if ((uintptr_t)cache % 4) return fail(MLA_ERR_INVALID_ARG, "compact: cache must be 4-byte aligned");
  if (dst_block_table && dst_max_pages <= 0)
    return fail(MLA_ERR_INVALID_ARG, "compact: dst_max_pages > 0 with a destination table");
  const long cap = (long)max_pages * h->cfg.page_size;
  if (cap > 0x3fffffffL) return fail(MLA_ERR_INVALID_ARG, "compact: max_pages * page_size < 2^30");
  const bool in_place = dst_block_table == nullptr;
  if ((weights == nullptr) != (weights_out == nullptr))
    return fail(MLA_ERR_INVALID_ARG, "compact: weights and weights_out go together");
  if (weights && ldw <= 0) return fail(MLA_ERR_INVALID_ARG, "compact: ldw > 0");
  if (weights && (weights == weights_out) != in_place)
    return fail(MLA_ERR_INVALID_ARG, "compact: weights_out == weights exactly when the cache is compacted in place");
  const bool wide = bytes % 16 == 0 && (uintptr_t)cache % 16 == 0;
  evict::CompactArgs a{};
  evict::chunk_shape(bytes, wide, &a.units, &a.rows);
  const long max_rows = in_place || !first ? ldk : cap;
  const long dc = (max_rows + a.rows - 1) / a.rows;
  const long wcap = weights ? (ldw < cap ? (long)ldw : cap) : 0;
  const long zc = (wcap + evict::ZERO_ROWS - 1) / evict::ZERO_ROWS;
  if (dc + zc == 0) return MLA_OK;
  if ((dc + zc) * num_seqs > 0x7fffffffL) return fail(MLA_ERR_INVALID_ARG, "compact: too many rows");
  a.cache = (char*)cache; a.block_table = block_table; a.kv_len = kv_len; a.keep = keep;
  a.keep_len = keep_len; a.first = first; a.dst_table = dst_block_table; a.weights = weights;
  a.weights_out = weights_out; a.ldk = ldk; a.ldw = ldw; a.row_cap = row_cap; a.num_pages = num_pages;
  a.page_size = h->cfg.page_size; a.max_pages = max_pages; a.dst_pages = dst_max_pages;
  a.data_chunks = (int)dc; a.chunks = (int)(dc + zc); a.in_place = in_place; a.status = h->status;
  cudaStream_t st = (cudaStream_t)stream;
  a.num_seqs = num_seqs;
  if (in_place && a.chunks > 1) {
    const size_t need = compact_ws(bytes, num_seqs, ldk);
    if (!workspace || workspace_bytes < need || (uintptr_t)workspace % 256)
      return fail(MLA_ERR_INVALID_ARG,
                  "compact: workspace smaller than mla_cache_compact_workspace_bytes() or not 256-byte aligned");
    a.ticket = (int*)workspace;
    a.list_parts = (int)((ldk + evict::LIST_PART - 1) / evict::LIST_PART);
    const long parts = (long)num_seqs * a.list_parts;     // (at most as many as there are data chunks)
    evict::compact_lists_kernel<<<(unsigned)(parts ? parts : 1), evict::LIST_THREADS, 0, st>>>(a);
    MLA_CUDA_TRY(cudaGetLastError());
    h->launches += 1;
  }
  const unsigned grid = (unsigned)((dc + zc) * num_seqs);
  Launch L(dim3(grid), dim3(evict::MV_THREADS), 0, st, a.ticket != nullptr);
  MLA_CUDA_TRY(cudaLaunchKernelEx(&L.cfg, wide ? evict::compact_kernel<uint4> : evict::compact_kernel<uint32_t>, a));
  h->launches += 1;
  return MLA_OK;
}

}  // namespace

extern "C" size_t mla_cache_compact_workspace_bytes(const mla_handle_t* h, int32_t num_seqs,
                                                    int64_t ldk) {
  return h && num_seqs >= 0 && ldk >= 0 ? compact_ws((size_t)h->lay.L * h->lay.elt, num_seqs, ldk) : 0;
}

extern "C" mla_status_t mla_cache_compact(mla_handle_t* h, void* cache, int32_t num_pages,
                                          const int32_t* block_table, int32_t max_pages,
                                          const int32_t* kv_len, int32_t num_seqs,
                                          const int32_t* keep, int64_t ldk, const int32_t* keep_len,
                                          const int32_t* first, const int32_t* dst_block_table,
                                          int32_t dst_max_pages, const float* weights,
                                          float* weights_out, int64_t ldw, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  return compact_rows(h, cache, h ? (size_t)h->lay.L * h->lay.elt : 0, num_pages, block_table, max_pages, kv_len,
                      num_seqs, keep, ldk, keep_len, first, dst_block_table, dst_max_pages, weights, weights_out,
                      ldw, weights_cap(weights, ldw), workspace, workspace_bytes, stream);
}

// The three arrays of an 8-bit cache one after the other; in place the calls share the workspace (each
// clears its flags behind the one before).  The weights move with the first; all three take the same sequences:
// an entry is worth nothing without its scale.  64 sequences of 4 k entries to 1024: 23.7 us into other pages (29.3 for
// the bf16 cache, 1.8 times the bytes), 48.6 in place (54.3); 5 of 16 nodes of each: 10.9 us in place (3.9), three launches.
extern "C" size_t mla_cache8_compact_workspace_bytes(const mla_handle_t* h, int32_t num_seqs, int64_t ldk) {
  return h && num_seqs >= 0 && ldk >= 0 ? compact_ws(cache8::RANK, num_seqs, ldk) : 0;
}

extern "C" mla_status_t mla_cache8_compact(mla_handle_t* h, const mla_cache8_t* cache, int32_t num_pages,
                                           const int32_t* block_table, int32_t max_pages,
                                           const int32_t* kv_len, int32_t num_seqs, const int32_t* keep,
                                           int64_t ldk, const int32_t* keep_len, const int32_t* first,
                                           const int32_t* dst_block_table, int32_t dst_max_pages,
                                           const float* weights, float* weights_out, int64_t ldw,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  mla_status_t s = cache8::check_cache(h, cache, num_pages, "cache8 compact");
  if (s != MLA_OK) return s;
  void* const array[3] = {cache->latent, cache->rope, cache->scale};
  const size_t bytes[3] = {cache8::RANK, 2 * cache8::ROPE, sizeof(float)};
  for (int i = 0; i < 3 && s == MLA_OK; ++i)
    s = compact_rows(h, array[i], bytes[i], num_pages, block_table, max_pages, kv_len, num_seqs, keep, ldk, keep_len,
                     first, dst_block_table, dst_max_pages, i ? nullptr : weights, i ? nullptr : weights_out, ldw,
                     weights_cap(weights, ldw), workspace, workspace_bytes, stream);
  return s;
}
