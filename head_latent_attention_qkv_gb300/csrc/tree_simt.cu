// Tree attention and key weights on the CUDA cores (tree.cuh has the rule of
// visibility, mla_draft.h the formulas): the fp32 layers, whose tolerance the
// tensor cores' TF32 would not meet.
//
// Tree attention: one CTA per (block, 16 rows of (node, head)); 32 cache
// entries at a time are staged in shared memory, the next ones by asynchronous
// copies while these meet an online softmax.  Key weights: one CTA per (block,
// 32 keys) holds its keys and walks the block's rows 16 at a time; a key's sum
// is kept by the 16 threads that share it and added in a fixed order at the
// end, so repeated calls agree bit for bit.  Rows are read 16 bytes at a time
// with an odd number of 16-byte units between them, which keeps eight threads
// on eight rows off one another's banks.  Such layers and their calls are
// small: what counts is the chain of latencies (4 heads x 8 nodes, 64 keys: 12.4
// us; 22.9 with scalar loads and one buffer).
#include "simt.cuh"
#include "tree.cuh"

#include <math.h>

#include <mutex>

namespace mla {
namespace simt {
namespace {

constexpr int RT = 16, KT = 32, THREADS = 256, MAX_OUT = 8;   // rkv <= 64 * MAX_OUT
constexpr int MAX_SMEM = 227 * 1024;

__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Floats between rows of L in shared memory: a whole, odd number of 16-byte units.
__host__ __device__ __forceinline__ int pitch_of(int L) { return (((L + 3) / 4) | 1) * 4; }

// Copies N = 8 or 16 bytes asynchronously, zeros when !ok.
template <int N>
__device__ __forceinline__ void copy_async(float* dst, const float* src, bool ok) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = ok ? N : 0;
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// A row of L floats (L even) by threads part, part + step, ...; the unit after
// an L that is no multiple of 4 is cleared.
__device__ __forceinline__ void copy_row(float* dst, const float* src, int L, int part, int step, bool ok) {
  if (L % 4 == 0) {
    for (int u = part; u < L / 4; u += step) copy_async<16>(dst + 4 * u, src + 4 * u, ok);
  } else {
    for (int u = part; u < L / 2; u += step) copy_async<8>(dst + 2 * u, src + 2 * u, ok);
    if (part == 0) *reinterpret_cast<float2*>(dst + L) = make_float2(0.f, 0.f);
  }
}

// Entries j0 .. j0 + 31 of block b (zeros past the end or on a bad page).
__device__ __forceinline__ void stage_keys(const tree::Rule& a, const float* cache, int b, int j0, int n,
                                           int L, float* Es) {
  const int part = threadIdx.x % 8, kk = threadIdx.x / 8, j = j0 + kk;
  long slot = -1;
  if (j < n) {
    const int page = a.block_table[(long)b * a.max_pages + j / a.page_size];
    if (page >= 0 && page < a.num_pages) slot = (long)page * a.page_size + j % a.page_size;
    else if (part == 0) set_status(a.status, MLA_DEV_BAD_PAGE);
  }
  copy_row(Es + kk * pitch_of(L), cache + max(slot, 0L) * L, L, part, 8, slot >= 0);
}
// Rows row0 .. row0 + 15 of Q_abs (zeros past the last of `rows`).
__device__ __forceinline__ void stage_rows(const float* q, long row0, int rows, int L, float* Qs) {
  const int part = threadIdx.x % 16, r = threadIdx.x / 16;
  copy_row(Qs + r * pitch_of(L), q + (row0 + (r < rows ? r : 0)) * L, L, part, 16, r < rows);
}

// <q, k0> and <q, k1> over `units` 16-byte units.
__device__ __forceinline__ float2 dot2(const float* q, const float* k0, const float* k1, int units) {
  float4 s0 = make_float4(0.f, 0.f, 0.f, 0.f), s1 = s0;
#pragma unroll 10
  for (int u = 0; u < units; ++u) {
    const float4 x = reinterpret_cast<const float4*>(q)[u];
    const float4 y = reinterpret_cast<const float4*>(k0)[u], z = reinterpret_cast<const float4*>(k1)[u];
    s0.x = fmaf(x.x, y.x, s0.x); s0.y = fmaf(x.y, y.y, s0.y); s0.z = fmaf(x.z, y.z, s0.z); s0.w = fmaf(x.w, y.w, s0.w);
    s1.x = fmaf(x.x, z.x, s1.x); s1.y = fmaf(x.y, z.y, s1.y); s1.z = fmaf(x.z, z.z, s1.z); s1.w = fmaf(x.w, z.w, s1.w);
  }
  return make_float2((s0.x + s0.y) + (s0.z + s0.w), (s1.x + s1.y) + (s1.z + s1.w));
}

__global__ void __launch_bounds__(THREADS)
tree_attn_kernel(const tree::Rule a, const float* __restrict__ q_abs, const float* __restrict__ cache,
                 int rkv, int L, int tiles, int buffers, float scale, float* __restrict__ o_lat,
                 float* __restrict__ lse, int32_t* __restrict__ vis_stats) {
  extern __shared__ __align__(16) float sm[];
  const int pitch = pitch_of(L), units = (L + 3) / 4;
  float* Qs = sm;                               // [RT] rows
  float* Ps = Qs + RT * pitch;                  // [RT][KT]
  float* Es = Ps + RT * KT;                     // [buffers][KT] rows
  const int b = blockIdx.x / tiles, r0 = blockIdx.x % tiles * RT;
  const int tid = threadIdx.x, r = tid / 16, c0 = tid % 16;
  const int rows = min(RT, a.T * a.H - r0);
  const long row0 = (long)b * a.T * a.H + r0;
  stage_rows(q_abs, row0, rows, L, Qs);
  int W, ctx;
  const int n = tree::block_keys(a, b, &W, &ctx, tid == 0 && r0 == 0);
  // first key that any of these rows can see
  int j_lo = 0;
  if (W > 0) {
    int pmin = 0x7fffffff;
    for (int t = r0 / a.H; t <= (r0 + rows - 1) / a.H; ++t) pmin = min(pmin, a.positions[(long)b * a.T + t]);
    // own nodes are held against the nodes' positions: none of them is skipped
    j_lo = min(min(n, tree::window_start(pmin, W)), ctx) / KT * KT;
  }
  if (j_lo < n) stage_keys(a, cache, b, j_lo, n, L, Es);
  copy_commit();
  const bool live = r < rows;
  const int i = live ? (r0 + r) / a.H : 0;
  const long m = (long)b * a.T + i, row = row0 + r;
  bool ok = live && n > 0 && (a.q_visible ? a.q_visible[m] != 0 : true);
  if (ok && a.parent) ok = tree::in_tree(a, a.parent + (long)b * a.T, i, c0 == 0);
  const int nout = (rkv + 63) / 64;             // groups of 4 dims of this thread: 4 c0 + 64 k
  float4 o[MAX_OUT];
#pragma unroll
  for (int k = 0; k < MAX_OUT; ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  float mrow = -INFINITY, lrow = 0.f;
  int cnt = 0, last = -1, first = -1, buf = 0;
  for (int j0 = j_lo; j0 < n; j0 += KT) {
    const float* E = Es + buf * KT * pitch;
    if (buffers == 2 && j0 + KT < n) {          // (its readers passed the barrier below)
      stage_keys(a, cache, b, j0 + KT, n, L, Es + (buf ^ 1) * KT * pitch);
      copy_commit();
      copy_wait<1>();
    } else {
      copy_wait<0>();
    }
    const unsigned vis = (unsigned)tree::key_bits(a, b, i, ok, n, W, ctx, j0);
    __syncthreads();
    if (vis) {
      cnt += __popc(vis);
      if (first < 0) first = j0 + __ffs(vis) - 1;
      last = j0 + 31 - __clz(vis);
    }
    const float2 d = dot2(Qs + r * pitch, E + c0 * pitch, E + (c0 + 16) * pitch, units);
    const float s0 = (vis >> c0) & 1u ? d.x * scale : -INFINITY;
    const float s1 = (vis >> (c0 + 16)) & 1u ? d.y * scale : -INFINITY;
    const float m_new = fmaxf(mrow, max16(fmaxf(s0, s1)));
    const float alpha = mrow == -INFINITY ? 0.f : expf(mrow - m_new);
    const float p0 = s0 == -INFINITY ? 0.f : expf(s0 - m_new);
    const float p1 = s1 == -INFINITY ? 0.f : expf(s1 - m_new);
    lrow = lrow * alpha + sum16(p0 + p1);
    mrow = m_new;
    Ps[r * KT + c0] = p0;
    Ps[r * KT + c0 + 16] = p1;
    __syncwarp();                               // a row's 16 threads share a warp
    // unseen keys (weight 0) are taken as zeros: their entries may hold anything.  A
    // select, not a branch: the two rows of a warp see different keys, and
    // branching took 3.4 k cycles a tile
    const bool whole = __all_sync(0xffffffffu, vis == 0xffffffffu);
#pragma unroll
    for (int k = 0; k < MAX_OUT; ++k) {
      const int c = 4 * c0 + 64 * k;
      if (k < nout && c < rkv) {
        float4 acc = make_float4(o[k].x * alpha, o[k].y * alpha, o[k].z * alpha, o[k].w * alpha);
#pragma unroll 2
        for (int k4 = 0; k4 < KT; k4 += 4) {
          const float4 p4 = *reinterpret_cast<const float4*>(Ps + r * KT + k4);
          const float p[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float4 v = *reinterpret_cast<const float4*>(E + (k4 + u) * pitch + c);
            if (!whole) {
              const bool seen = (vis >> (k4 + u)) & 1u;
              v.x = seen ? v.x : 0.f; v.y = seen ? v.y : 0.f; v.z = seen ? v.z : 0.f; v.w = seen ? v.w : 0.f;
            }
            acc.x = fmaf(p[u], v.x, acc.x); acc.y = fmaf(p[u], v.y, acc.y);
            acc.z = fmaf(p[u], v.z, acc.z); acc.w = fmaf(p[u], v.w, acc.w);
          }
        }
        o[k] = acc;
      }
    }
    __syncthreads();                            // the tile has been read
    if (buffers == 2) {
      buf ^= 1;
    } else if (j0 + KT < n) {
      stage_keys(a, cache, b, j0 + KT, n, L, Es);
      copy_commit();
    }
  }
  copy_wait<0>();
  if (live) {
    const bool any = lrow != 0.f;                // (a NaN that a row sees reaches its output)
    const float inv = 1.f / lrow;
#pragma unroll
    for (int k = 0; k < MAX_OUT; ++k) {
      const int c = 4 * c0 + 64 * k;
      if (k < nout && c < rkv)
        *reinterpret_cast<float4*>(o_lat + row * rkv + c) =
            any ? make_float4(o[k].x * inv, o[k].y * inv, o[k].z * inv, o[k].w * inv)
                : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (lse && c0 == 0) lse[row] = any ? mrow + logf(lrow) : -INFINITY;
    if (vis_stats && (r0 + r) % a.H == 0 && c0 == 0) {
      vis_stats[m * 3 + 0] = cnt;
      vis_stats[m * 3 + 1] = first;
      vis_stats[m * 3 + 2] = last;
    }
  }
}

__global__ void __launch_bounds__(THREADS)
key_weights_kernel(const tree::Rule a, const float* __restrict__ q_abs, const float* __restrict__ cache,
                   int L, int tiles, int buffers, float scale, const float* __restrict__ lse, float decay,
                   const float* prior, float* out, long ldw) {
  extern __shared__ __align__(16) float sm[];
  const int pitch = pitch_of(L), units = (L + 3) / 4;
  float* Es = sm;                               // [KT] rows
  float* Ps = Es + KT * pitch;                  // [RT][KT]
  float* Qs = Ps + RT * KT;                     // [buffers][RT] rows
  const int b = blockIdx.x / tiles, j0 = blockIdx.x % tiles * KT;
  const int tid = threadIdx.x, r = tid / 16, c0 = tid % 16, all = a.T * a.H;
  const long row0 = (long)b * all;
  int W, ctx;
  const int n0 = tree::block_keys(a, b, &W, &ctx, tid == 0 && j0 == 0);
  const int n = (int)min((long)n0, ldw);
  if (n < n0 && tid == 0 && j0 == 0) set_status(a.status, MLA_DEV_BAD_LENGTH);
  if (j0 >= n) return;
  stage_keys(a, cache, b, j0, n, L, Es);
  stage_rows(q_abs, row0, min(RT, all), L, Qs);
  copy_commit();
  float sum[2] = {0.f, 0.f};
  int buf = 0;
  for (int r0 = 0; r0 < all; r0 += RT) {
    const float* Q = Qs + buf * RT * pitch;
    if (buffers == 2 && r0 + RT < all) {
      stage_rows(q_abs, row0 + r0 + RT, min(RT, all - r0 - RT), L, Qs + (buf ^ 1) * RT * pitch);
      copy_commit();
      copy_wait<1>();
    } else {
      copy_wait<0>();
    }
    const bool live = r0 + r < all;
    const int i = live ? (r0 + r) / a.H : 0;
    const float l = live ? lse[row0 + r0 + r] : -INFINITY;
    bool ok = live && l != -INFINITY && (a.q_visible ? a.q_visible[(long)b * a.T + i] != 0 : true);
    // rows outside the tree have lse = -inf; only tiles with nodes' keys walk
    if (ok && a.parent && j0 + KT > ctx) ok = tree::in_tree(a, a.parent + (long)b * a.T, i, c0 == 0);
    const unsigned vis = (unsigned)tree::key_bits(a, b, i, ok, n0, W, ctx, j0);
    __syncthreads();
    const float2 d = dot2(Q + r * pitch, Es + c0 * pitch, Es + (c0 + 16) * pitch, units);
    if ((vis >> c0) & 1u) sum[0] += expf(d.x * scale - l);
    if ((vis >> (c0 + 16)) & 1u) sum[1] += expf(d.y * scale - l);
    __syncthreads();                            // the rows have been read
    if (buffers == 2) {
      buf ^= 1;
    } else if (r0 + RT < all) {
      stage_rows(q_abs, row0 + r0 + RT, min(RT, all - r0 - RT), L, Qs);
      copy_commit();
    }
  }
  copy_wait<0>();
  Ps[r * KT + c0] = sum[0];
  Ps[r * KT + c0 + 16] = sum[1];
  __syncthreads();
  if (tid < KT && j0 + tid < n) {
    float t = 0.f;
    for (int k = 0; k < RT; ++k) t += Ps[k * KT + tid];
    const long at = (long)b * ldw + j0 + tid;
    out[at] = prior ? fmaf(decay, prior[at], t) : t;
  }
}

// Shared memory with `once` rows held once and `buffers` times `per` rows.
size_t smem_bytes(int L, int once, int per, int buffers) {
  return sizeof(float) * ((size_t)pitch_of(L) * (once + per * buffers) + RT * KT);
}

template <typename K>
void allow_smem(K* kernel) {
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
}

}  // namespace

void tree_attention(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                    const float* q_abs, const float* cache, float* o_lat, float* lse, int32_t* vis_stats) {
  const Layout& l = h->lay;
  static std::once_flag once;
  std::call_once(once, [] { allow_smem(tree_attn_kernel); });
  const int tiles = (r.T * r.H + RT - 1) / RT;
  const int buffers = smem_bytes(l.L, RT, KT, 2) <= MAX_SMEM ? 2 : 1;
  tree_attn_kernel<<<(unsigned)num_blocks * tiles, THREADS, smem_bytes(l.L, RT, KT, buffers), st>>>(
      r, q_abs, cache, l.rkv, l.L, tiles, buffers, h->scale, o_lat, lse, vis_stats);
}

void key_weights(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                 const float* q_abs, const float* cache, const float* lse, float decay,
                 const float* prior, float* out, long ldw) {
  const Layout& l = h->lay;
  static std::once_flag once;
  std::call_once(once, [] { allow_smem(key_weights_kernel); });
  const long keys = min((long)r.max_pages * r.page_size, ldw);
  const int tiles = (int)((keys + KT - 1) / KT);
  const int buffers = smem_bytes(l.L, KT, RT, 2) <= MAX_SMEM ? 2 : 1;
  key_weights_kernel<<<(unsigned)num_blocks * tiles, THREADS, smem_bytes(l.L, KT, RT, buffers), st>>>(
      r, q_abs, cache, l.L, tiles, buffers, h->scale, lse, decay, prior, out, ldw);
}

}  // namespace simt
}  // namespace mla
