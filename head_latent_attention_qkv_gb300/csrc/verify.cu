// Verification of drafted tokens against the target's probabilities (mla_verify_drafts).
//
// A sequence stands at a node with what is left of the target's row there, w, and
// its mass s; a node drafted after it is taken when u s q(x) < w(x), else w
// becomes max(w - s q, 0).  w is never stored: after k refusals at a node it
// follows from the rows and the k masses, element by element, so the walk reads two
// numbers a node until something is refused, and one pass over the rows (of the
// target and the draft) gives each new mass.  The token behind the path needs
// the sums of w by parts of the vocabulary, which the last pass leaves.
//
// Borders.  A token's share of a large vocabulary is about 2^-17, and 10^5
// shares add up to the number that the last uniform is held against: fp32 sums
// would move it over a border in one draw of seven.  w and the sums are pairs of floats
// (a value and what its rounding left, together 2^-40 or better), whose operations run at
// the fp32 rate (this GPU adds doubles 64 times slower).
//
// A cluster of CL CTAs shares a sequence's rows: every warp owns a contiguous run
// of the vocabulary, and every CTA walks the same nodes and adds the same sums in the
// same order, so nobody has to be told what was decided.  The token behind the path is looked
// up by the CTA whose warp's run holds it, a run at a time in shared memory.
//
// Bound by the two rows of the node at which a sequence stops (64 chains of 15 over 152 k
// tokens, fp32: 78 MB, 19.8 us in a graph of calls, 3.9 TB/s: 1 us until the first probabilities are
// there, 11 for the pass, 3 for its sums and 3.5 for the token).  A refusal costs a pass of
// 1.8 us (8 trees of 32 nodes over 129 k, bf16: 19 us); one chain of 5 over 32 k takes 7.
#include "common.cuh"
#include "tc_ptx.cuh"
#include "tree.cuh"

#include <math.h>

#include <mutex>

namespace mla {
namespace verify {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAX_NODES = tree::MAX_NODES;
constexpr int STAGED = 5 * MAX_NODES / 2;  // elements (pairs) in the place of the five numbers a node has
constexpr int GROUP = 16;                  // elements a lane has in flight in a pass
constexpr int LOOK = 5;                    // and of a staged run

struct Args {
  const void* target;
  const void* draft;                       // may be NULL
  const int32_t* tokens;
  const int32_t* parent;                   // may be NULL
  const float* uniforms;
  const int32_t* first;                    // may be NULL
  int32_t* accepted;
  int32_t* num_accepted;
  int32_t* next_token;
  long ldt, ldd;
  int T, V;
  bool wide;                               // rows start at 16-byte boundaries
  uint32_t* status;
};

// A value and what is left of its rounding (at most half a step of hi).
struct __align__(8) Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair quick_sum(float a, float b) {     // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Pair add(Pair x, Pair y) {
  const Pair s = two_sum(x.hi, y.hi);
  return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(x.lo, y.lo)));
}
__device__ __forceinline__ Pair times(Pair s, float q) {
  const float h = __fmul_rn(s.hi, q);
  return quick_sum(h, __fmaf_rn(s.lo, q, __fmaf_rn(s.hi, q, -h)));
}
__device__ __forceinline__ Pair minus(Pair x, Pair y) { return add(x, Pair{-y.hi, -y.lo}); }
__device__ __forceinline__ bool above(Pair x, Pair y) { return x.hi > y.hi || (x.hi == y.hi && x.lo > y.lo); }
__device__ __forceinline__ Pair shfl_xor(Pair x, int o) {
  return {__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)};
}
// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ Pair lane_sums(Pair x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y{__shfl_up_sync(0xffffffffu, x.hi, o), __shfl_up_sync(0xffffffffu, x.lo, o)};
    if (lane >= o) x = add(x, y);
  }
  return x;
}
// A probability: 0 where it is no number that counts.
__device__ __forceinline__ float prob(float p) { return p > 0.f && p < INFINITY ? p : 0.f; }
// What k > 0 refusals with masses s[0] = 1, s[1] .. s[k - 1] leave of an element.
__device__ __forceinline__ Pair left_of(float p, float q, const Pair* s, int k) {
  Pair w = two_sum(p, -q);
  if (!(w.hi > 0.f)) return Pair{0.f, 0.f};
  for (int j = 1; j < k; ++j) {
    w = minus(w, times(s[j], q));
    if (!(w.hi > 0.f)) return Pair{0.f, 0.f};
  }
  return w;
}

// Where a walk stands.
struct State {
  int node;                                // -1: the context
  int next;                                // next node to look at
  int refused;                             // refusals here
  int kept;                                // nodes taken
  bool over;                               // no node is left to look at
};

__device__ __forceinline__ Pair ld_cluster_pair(uint32_t addr) {
  Pair v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(addr) : "memory");
  return v;
}

// What the sums are taken over: the target's row, its difference to the draft's, that
// after several refusals, or the row without the tokens refused.
enum Mode { ROW, DIFF, DIFFS, WITHOUT };

template <typename T>
struct Rest {
  const T* p;
  const T* q;
  const Pair* mass;
  const int* banned;
  int k;
  template <int MODE>
  __device__ __forceinline__ Pair of(float pv, float qv, int x) const {
    if (MODE == ROW) return Pair{pv, 0.f};
    if (MODE == WITHOUT) {
      bool out = false;
      for (int j = 0; j < k; ++j) out |= banned[j] == x;
      return Pair{out ? 0.f : pv, 0.f};
    }
    return left_of(pv, qv, mass, MODE == DIFF ? 1 : k);
  }
  // What is left of element x, from its numbers in the rows.
  __device__ __forceinline__ Pair left(float pv, float qv, int x) const {
    return !k ? Pair{pv, 0.f} : q ? left_of(pv, qv, mass, k) : of<WITHOUT>(pv, 0.f, x);
  }
  // One more element into a running sum; the roundings gather in `tail`.  CLEAN: as left(); else an
  // infinity makes the sum no finite number (the draft's by way of tail: 0 times it).
  template <int MODE, bool CLEAN>
  __device__ __forceinline__ void take(Pair& acc, float& tail, float pv, float qv, int x) const {
    const Pair w = CLEAN ? of<MODE>(prob(pv), prob(qv), x) : of<MODE>(fmaxf(pv, 0.f), fmaxf(qv, 0.f), x);
    const Pair s = two_sum(acc.hi, w.hi);
    acc.hi = s.hi;
    tail = __fadd_rn(tail, __fadd_rn(s.lo, w.lo));
    if (!CLEAN && (MODE == DIFF || MODE == DIFFS)) tail = __fmaf_rn(fmaxf(qv, 0.f), 0.f, tail);
  }
  // A lane's share of the elements lo .. hi - 1 (lo a multiple of 32); `wide`: rows are 16-byte aligned.
  template <int MODE>
  __device__ __forceinline__ Pair sum(int lo, int hi, int lane, bool wide) const {
    const Pair s = sum_of<MODE, false>(lo, hi, lane, wide);
    return s.hi < INFINITY ? s : sum_of<MODE, true>(lo, hi, lane, false);
  }
  template <int MODE, bool CLEAN>
  __device__ __forceinline__ Pair sum_of(int lo, int hi, int lane, bool wide) const {
    constexpr bool TWO = MODE == DIFF || MODE == DIFFS;
    constexpr int NV = 16 / sizeof(T), LOADS = GROUP / NV;
    Pair acc{0.f, 0.f};
    int x0 = lo;
    if (wide)
      for (; x0 + 32 * GROUP <= hi; x0 += 32 * GROUP) {
        uint4 pv[LOADS], qv[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          pv[i] = *reinterpret_cast<const uint4*>(p + x0 + (32 * i + lane) * NV);
          if (TWO) qv[i] = *reinterpret_cast<const uint4*>(q + x0 + (32 * i + lane) * NV);
        }
        if (MODE == WITHOUT) {             // (a refused token is in few of these)
          for (int j = 0; j < k; ++j) {
            const int x = banned[j] - x0, at = x / NV;
            if ((unsigned)x < 32u * GROUP && at % 32 == lane) {
#pragma unroll
              for (int i = 0; i < LOADS; ++i)
                if (i == at / 32) {
                  uint32_t* word = reinterpret_cast<uint32_t*>(&pv[i]);
                  const int e = x % NV, bits = 8 * sizeof(T), per = 32 / bits;
#pragma unroll
                  for (int w = 0; w < 4; ++w)
                    if (w == e / per) word[w] &= per == 1 ? 0u : e % per ? 0xffffu : 0xffff0000u;
                }
            }
          }
        }
        float tail = 0.f;
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
#pragma unroll
          for (int e = 0; e < NV; ++e)
            take<MODE == WITHOUT ? ROW : MODE, CLEAN>(acc, tail, to_f32(reinterpret_cast<const T*>(&pv[i])[e]),
                TWO ? to_f32(reinterpret_cast<const T*>(&qv[i])[e]) : 0.f, 0);
        acc = quick_sum(acc.hi, __fadd_rn(acc.lo, tail));
      }
    for (x0 += lane; x0 < hi; x0 += 32 * GROUP) {
      float pv[GROUP], qv[GROUP];
#pragma unroll
      for (int i = 0; i < GROUP; ++i) {
        const int x = x0 + 32 * i;
        pv[i] = x < hi ? to_f32(p[x]) : 0.f;
        qv[i] = TWO && x < hi ? to_f32(q[x]) : 0.f;
      }
      float tail = 0.f;
#pragma unroll
      for (int i = 0; i < GROUP; ++i) take<MODE, CLEAN>(acc, tail, pv[i], qv[i], x0 + 32 * i);
      acc = quick_sum(acc.hi, __fadd_rn(acc.lo, tail));
    }
    return acc;
  }
};

template <typename T, int CL>
__global__ void __launch_bounds__(THREADS) verify_kernel(const Args a) {
  constexpr int SUMS = CL * WARPS, PER_LANE = (SUMS + 31) / 32;
  __shared__ __align__(8) uint32_t pool[5 * MAX_NODES];
  float *px = reinterpret_cast<float*>(pool), *qx = px + MAX_NODES, *u = qx + MAX_NODES;
  int *par = reinterpret_cast<int*>(u + MAX_NODES), *tok = par + MAX_NODES;
  __shared__ int path[MAX_NODES];
  __shared__ bool takes[MAX_NODES];
  __shared__ Pair mass[MAX_NODES + 1];     // s after j refusals here
  __shared__ int banned[MAX_NODES];        // draft NULL: tokens refused here
  __shared__ State st;
  __shared__ Pair parts[WARPS];
  __shared__ int found, fallback;
  __shared__ Pair sums[2][WARPS];          // of this CTA's warps, by pass parity
  __shared__ Pair runs[SUMS], before[SUMS + 1];   // sums of the warps' runs, of those in front of each, of all
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = CL > 1 ? (int)tc::cluster_ctarank() : 0;
  const long b = blockIdx.x / CL;
  const int nodes = a.T, V = a.V;
  const T* target = (const T*)a.target + b * (nodes + 1) * a.ldt;
  const T* draft = a.draft ? (const T*)a.draft + b * nodes * a.ldd : nullptr;

  for (int i = tid; i < nodes; i += THREADS) {
    const int x = a.tokens[b * nodes + i], p = a.parent ? a.parent[b * nodes + i] : i - 1;
    const bool in = p >= -1 && p < i, known = x >= 0 && x < V;
    if (rank == 0 && (p >= i || (in && !known)))
      set_status(a.status, p >= i ? MLA_DEV_BAD_TREE : MLA_DEV_BAD_DRAFT);
    par[i] = in ? p : -2;
    tok[i] = known ? x : -1;
    u[i] = a.uniforms[b * (nodes + 1) + i];
    const bool read = in && known;
    px[i] = read ? prob(to_f32(target[(p + 1) * a.ldt + x])) : 0.f;
    qx[i] = read && draft ? prob(to_f32(draft[(p + 1) * a.ldd + x])) : 1.f;
    takes[i] = above(Pair{px[i], 0.f}, times(Pair{qx[i], 0.f}, u[i]));    // with nothing refused before it
  }
  if (tid == 0) {
    st = State{-1, 0, 0, 0, false};
    found = fallback = -1;
    mass[0] = Pair{1.f, 0.f};
  }
  __syncthreads();

  const int slice = ((V + SUMS - 1) / SUMS + 31) & ~31;
  const int lo = (int)min((long)(rank * WARPS + warp) * slice, (long)V), hi = min(lo + slice, V);
  int parity = 0;
  bool whole = false;                      // nothing was left: the target's row itself
  Rest<T> rest{nullptr, nullptr, mass, banned, 0};
  int summed_node = -2, summed_k = 0;
  while (true) {
    if (tid == 0 && !st.over) {
      State s = st;
      s.over = true;
      for (; s.next < nodes; ++s.next) {
        const int i = s.next;
        if (par[i] != s.node || tok[i] < 0) continue;
        Pair w{px[i], 0.f};
        const Pair m = mass[s.refused];
        bool take = takes[i];
        if (s.refused) {
          if (draft) {
            w = left_of(px[i], qx[i], mass, s.refused);
          } else {
            for (int j = 0; j < s.refused; ++j)
              if (banned[j] == tok[i]) w.hi = 0.f;
          }
          take = above(w, times(times(m, qx[i]), u[i]));
        }
        if (take) {
          path[s.kept++] = i;
          s.node = i;
          s.refused = 0;
          continue;
        }
        ++s.refused;
        if (!draft) {
          banned[s.refused - 1] = tok[i];
          mass[s.refused] = minus(m, w);
          continue;
        }
        ++s.next;
        s.over = false;                    // the mass that is left decides about the next one
        break;
      }
      st = s;
    }
    __syncthreads();
    const State s = st;
    rest.k = whole ? 0 : s.refused;
    if (s.node != summed_node || rest.k != summed_k || whole) {
      rest.p = target + (long)(s.node + 1) * a.ldt;
      rest.q = rest.k && draft ? draft + (long)(s.node + 1) * a.ldd : nullptr;
      const Mode mode = rest.k == 0 ? ROW : !draft ? WITHOUT : rest.k == 1 ? DIFF : DIFFS;
      Pair x = mode == ROW ? rest.template sum<ROW>(lo, hi, lane, a.wide)
               : mode == DIFF ? rest.template sum<DIFF>(lo, hi, lane, a.wide)
               : mode == DIFFS ? rest.template sum<DIFFS>(lo, hi, lane, a.wide)
                               : rest.template sum<WITHOUT>(lo, hi, lane, a.wide);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x = add(x, shfl_xor(x, o));
      if (lane == 0) sums[parity][warp] = x;
      if (CL > 1) tc::cluster_sync_all();
      else __syncthreads();
      if (warp == 0) {
        Pair v[PER_LANE], own{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
          const int w = lane * PER_LANE + i;
          v[i] = w >= SUMS ? Pair{0.f, 0.f}
                 : CL > 1 ? ld_cluster_pair(tc::mapa(tc::smem_u32(&sums[parity][w % WARPS]), (uint32_t)(w / WARPS)))
                          : sums[parity][w];
          own = add(own, v[i]);
        }
        const Pair incl = lane_sums(own, lane);
        Pair run{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
        if (lane == 0) run = Pair{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
          const int w = lane * PER_LANE + i;
          if (w < SUMS) {
            runs[w] = v[i];
            before[w] = run;
          }
          run = add(run, v[i]);
        }
        if (lane == 31) {
          before[SUMS] = run;
          if (!s.over) mass[s.refused] = run;
        }
      }
      __syncthreads();
      parity ^= 1;
      summed_node = s.node;
      summed_k = rest.k;
    }
    if (!s.over) continue;
    if (before[SUMS].hi > 0.f || whole || rest.k == 0) break;
    whole = true;
  }

  // The token: the least x whose sum is above the goal lies in the run of the last warp
  // that has anything and whose sum in front is not above it.
  const Pair total = before[SUMS];
  const Pair goal = times(total, fmaxf(a.uniforms[b * (nodes + 1) + nodes], 0.f));
  int owner = -1;
  for (int i0 = 0; i0 < SUMS; i0 += 32) {
    const int i = i0 + lane;
    const bool mine = i < SUMS && runs[i].hi > 0.f && !above(before[i], goal);
    const uint32_t some = __ballot_sync(0xffffffffu, mine);
    if (some) owner = i0 + 31 - __clz(some);
  }
  if (owner >= 0 && owner / WARPS == rank) {
    // Its CTA takes that run STAGED elements at a time: into shared memory, a contiguous part to
    // each thread, and the thread whose part the goal falls into looks it up.
    const int run_lo = (int)min((long)owner * slice, (long)V), run_hi = min(run_lo + slice, V);
    Pair* el = reinterpret_cast<Pair*>(pool);
    const T* row2 = rest.q ? rest.q : rest.p;
    Pair front = before[owner];
    int top = -1;                          // (where rounding leaves nothing above the goal)
    for (int x0 = run_lo; x0 < run_hi; x0 += STAGED) {
      const int n = min(STAGED, run_hi - x0), part = (n + THREADS - 1) / THREADS;
      __syncthreads();                     // (the buffer is free; the last part's answer is known)
      if (found >= 0) break;
      for (int i = tid; i < n; i += THREADS * LOOK) {
        float pv[LOOK], qv[LOOK];
#pragma unroll
        for (int e = 0; e < LOOK; ++e) {
          const int x = x0 + min(i + e * THREADS, n - 1);
          pv[e] = to_f32(rest.p[x]);
          qv[e] = to_f32(row2[x]);
        }
#pragma unroll
        for (int e = 0; e < LOOK; ++e)
          if (i + e * THREADS < n) el[i + e * THREADS] = rest.left(prob(pv[e]), prob(qv[e]), x0 + i + e * THREADS);
      }
      __syncthreads();
      const int i0 = min(tid * part, n), i1 = min(i0 + part, n);
      Pair own{0.f, 0.f};
      for (int i = i0; i < i1; ++i) own = add(own, el[i]);
      const Pair incl = lane_sums(own, lane);
      if (lane == 31) parts[warp] = incl;
      const Pair lower{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
      __syncthreads();
      Pair cum = front;
      for (int w = 0; w < WARPS; ++w) {
        if (w == warp) cum = front;
        front = add(front, parts[w]);
      }
      if (lane > 0) cum = add(cum, lower);
      if (own.hi > 0.f && !above(cum, goal)) {
        int last = -1, hit = -1;
        for (int i = i0; i < i1 && hit < 0; ++i) {
          cum = add(cum, el[i]);
          if (el[i].hi > 0.f) {
            last = x0 + i;
            if (above(cum, goal)) hit = last;
          }
        }
        if (hit >= 0) atomicMin(reinterpret_cast<unsigned*>(&found), (unsigned)hit);   // (-1: none yet)
        top = last;
      }
      if (top >= 0) atomicMax(&fallback, top);
    }
    __syncthreads();
    if (tid == 0) a.next_token[b] = found >= 0 ? found : fallback;
  }
  if (rank == 0) {
    if (owner < 0 && tid == 0) {
      a.next_token[b] = -1;
      set_status(a.status, MLA_DEV_BAD_DRAFT);
    }
    const int f = a.first ? a.first[b] : 0, kept = st.kept;
    for (int i = tid; i < nodes; i += THREADS) a.accepted[b * nodes + i] = i < kept ? path[i] + f : -1;
    if (tid == 0) a.num_accepted[b] = kept;
  }
  if (CL > 1) tc::cluster_sync_all();      // a peer may still read this CTA's sums
}

// Whether the GPU runs clusters of 16 (more than 8 have to be asked for, and may be refused: a part of a GPU may have
// no 16 SMs that can form one).
template <typename T>
bool wide_clusters() {
  static std::once_flag once;
  static bool wide = false;
  std::call_once(once, [] {
    Launch L(dim3(16), dim3(THREADS), 0, nullptr, false, dim3(16, 1, 1));
    int clusters = 0;
    wide = cudaFuncSetAttribute(verify_kernel<T, 16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
           cudaOccupancyMaxActiveClusters(&clusters, verify_kernel<T, 16>, &L.cfg) == cudaSuccess && clusters > 0;
    if (!wide) cudaGetLastError();         // (the refusal is dealt with)
  });
  return wide;
}

template <typename T>
cudaError_t launch(const Args& a, int num_seqs, int cl, cudaStream_t st) {
  if (cl == 16 && !wide_clusters<T>()) cl = 8;
  Launch L(dim3((unsigned)(num_seqs * cl)), dim3(THREADS), 0, st, false, dim3((unsigned)cl, 1, 1));
  return cudaLaunchKernelEx(&L.cfg, cl == 1   ? verify_kernel<T, 1>
                                    : cl == 2 ? verify_kernel<T, 2>
                                    : cl == 4 ? verify_kernel<T, 4>
                                    : cl == 8 ? verify_kernel<T, 8>
                                              : verify_kernel<T, 16>, a);
}

// CTAs that share a sequence: 16, fewer where the sequences fill the GPU (four CTAs an SM) without
// them, so that all of a batch's clusters run at once, and fewer for a small vocabulary, whose passes are
// shorter than what a wider cluster's barriers cost (16 for 8: 20 trees of 8 over 129 k tokens 42 -> 27 us,
// one chain over 152 k 11.0 -> 9.2; 30 chains over 32 k 8.1 -> 10.3).
int cluster_size(int num_seqs, int vocab, int num_sms) {
  int cl = 16;
  while (cl > 1 && ((long)num_seqs * cl > 4L * num_sms || vocab <= 2048 * cl)) cl /= 2;
  return cl;
}

}  // namespace
}  // namespace verify
}  // namespace mla

using namespace mla;

extern "C" mla_status_t mla_verify_drafts(mla_handle_t* h, const void* target, int64_t ldt, const void* draft,
                                          int64_t ldd, int32_t dtype, const int32_t* tokens,
                                          const int32_t* parent, const float* uniforms, const int32_t* first,
                                          int32_t num_seqs, int32_t num_nodes, int32_t vocab,
                                          int32_t* accepted, int32_t* num_accepted, int32_t* next_token,
                                          void* stream) {
  if (!h) return fail(MLA_ERR_INVALID_ARG, "verify: null handle");
  if (num_seqs < 0 || num_nodes < 0 || vocab <= 0 || vocab > 0x3fffffff)
    return fail(MLA_ERR_INVALID_ARG, "verify: num_seqs and num_nodes >= 0, 0 < vocab < 2^30");
  if (num_seqs == 0) return MLA_OK;
  if (num_seqs > 0xfffffff) return fail(MLA_ERR_INVALID_ARG, "verify: too many sequences");
  if (num_nodes > verify::MAX_NODES) return fail(MLA_ERR_UNSUPPORTED, "verify: at most 1024 nodes a sequence");
  if (dtype != MLA_FP32 && dtype != MLA_BF16 && dtype != MLA_FP16)
    return fail(MLA_ERR_INVALID_ARG, "verify: dtype MLA_FP32, MLA_BF16 or MLA_FP16");
  if (!target || !uniforms || !num_accepted || !next_token || (num_nodes > 0 && (!tokens || !accepted)))
    return fail(MLA_ERR_INVALID_ARG, "verify: null pointer");
  if (ldt < vocab || (draft && ldd < vocab)) return fail(MLA_ERR_INVALID_ARG, "verify: ldt and ldd >= vocab");
  const size_t e = dtype == MLA_FP32 ? 4 : 2;
  if ((uintptr_t)target % e || (uintptr_t)draft % e)
    return fail(MLA_ERR_INVALID_ARG, "verify: target and draft must be aligned to their elements");
  const bool wide = ((uintptr_t)target | (uintptr_t)draft | (size_t)ldt * e | (draft ? (size_t)ldd * e : 0)) % 16 == 0;
  const verify::Args a{target, num_nodes ? draft : nullptr, tokens, parent, uniforms, first, accepted,
                       num_accepted, next_token, (long)ldt, (long)ldd, num_nodes, vocab, wide, h->status};
  const int cl = verify::cluster_size(num_seqs, vocab, h->num_sms);
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t err = dtype == MLA_FP32   ? verify::launch<float>(a, num_seqs, cl, st)
                          : dtype == MLA_BF16 ? verify::launch<__nv_bfloat16>(a, num_seqs, cl, st)
                                              : verify::launch<__half>(a, num_seqs, cl, st);
  MLA_CUDA_TRY(err);
  MLA_CUDA_TRY(cudaGetLastError());
  h->launches += 1;
  return MLA_OK;
}
