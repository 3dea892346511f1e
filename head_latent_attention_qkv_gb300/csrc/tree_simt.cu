// Tree attention and key weights on the CUDA cores (tree.cuh has the rule of
// visibility, mla_draft.h the formulas): the path of the fp32 layers.
//
// Tree attention: one CTA per (block, 16 rows of (node, head)); 32 cache
// entries at a time are staged in shared memory as fp32 and meet an online
// softmax.  Key weights: one CTA per (block, 32 keys) holds its keys and walks
// the block's rows 16 at a time; a key's sum is kept by the 16 threads that
// share it and added in a fixed order at the end, so repeated calls agree bit
// for bit.
#include "simt.cuh"
#include "tree.cuh"

#include <math.h>

#include <mutex>

namespace mla {
namespace simt {
namespace {

constexpr int RT = 16, KT = 32, THREADS = 256, MAX_OUT = 32;   // rkv <= 16 * MAX_OUT

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

// 32 entries from key j0 on into Es [32][L + 1] (0 past the end or on a bad page).
template <typename TC>
__device__ __forceinline__ void stage_keys(const tree::Rule& a, const TC* cache, int b, int j0, int n,
                                           int L, float* Es) {
  const int part = threadIdx.x % 8, kk = threadIdx.x / 8, j = j0 + kk;
  long slot = -1;
  if (j < n) {
    const int page = a.block_table[(long)b * a.max_pages + j / a.page_size];
    if (page >= 0 && page < a.num_pages) slot = (long)page * a.page_size + j % a.page_size;
    else if (part == 0) set_status(a.status, MLA_DEV_BAD_PAGE);
  }
  for (int d = part; d < L; d += 8) Es[kk * (L + 1) + d] = slot >= 0 ? to_f32(cache[slot * L + d]) : 0.f;
}

template <typename TC, typename TO>
__global__ void __launch_bounds__(THREADS)
tree_attn_kernel(const tree::Rule a, const TC* __restrict__ q_abs, const TC* __restrict__ cache,
                 int rkv, int L, int tiles, float scale, TO* __restrict__ o_lat, float* __restrict__ lse,
                 int32_t* __restrict__ vis_stats) {
  extern __shared__ float sm[];
  float* Qs = sm;                      // [RT][L]
  float* Es = Qs + RT * L;             // [KT][L + 1]
  float* Ps = Es + KT * (L + 1);       // [RT][KT]
  const int b = blockIdx.x / tiles, r0 = blockIdx.x % tiles * RT;
  const int tid = threadIdx.x, r = tid / 16, c0 = tid % 16;
  const int rows = min(RT, a.T * a.H - r0);
  int W, ctx;
  const int n = tree::block_keys(a, b, &W, &ctx, tid == 0 && r0 == 0);
  const bool live = r < rows;
  const int i = live ? (r0 + r) / a.H : 0;
  const long m = (long)b * a.T + i, row = (long)b * a.T * a.H + r0 + r;
  bool ok = live && n > 0 && (a.q_visible ? a.q_visible[m] != 0 : true);
  if (ok && a.parent) ok = tree::in_tree(a, a.parent + (long)b * a.T, i, c0 == 0);
  // first key that any of these rows can see
  int j_lo = 0;
  if (W > 0) {
    int pmin = 0x7fffffff;
    for (int t = r0 / a.H; t <= (r0 + rows - 1) / a.H; ++t) pmin = min(pmin, a.positions[(long)b * a.T + t]);
    // own nodes are held against the nodes' positions: none of them is skipped
    j_lo = max(0, min(min(n, pmin - W + 1), ctx)) / KT * KT;
  }
  for (int idx = tid; idx < RT * L; idx += THREADS) {
    const int rr = idx / L;
    Qs[idx] = rr < rows ? to_f32(q_abs[((long)b * a.T * a.H + r0 + rr) * L + idx % L]) : 0.f;
  }
  const int nout = rkv / 16;
  float o[MAX_OUT];
#pragma unroll
  for (int k = 0; k < MAX_OUT; ++k) o[k] = 0.f;
  float mrow = -INFINITY, lrow = 0.f;
  int cnt = 0, last = -1, first = -1;
  for (int j0 = j_lo; j0 < n; j0 += KT) {
    __syncthreads();
    stage_keys(a, cache, b, j0, n, L, Es);
    const unsigned vis = (unsigned)tree::key_bits(a, b, i, ok, n, W, ctx, j0);
    __syncthreads();
    if (vis) {
      cnt += __popc(vis);
      if (first < 0) first = j0 + __ffs(vis) - 1;
      last = j0 + 31 - __clz(vis);
    }
    float s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int kk = c0 + 16 * u;
      s[u] = -INFINITY;
      if ((vis >> kk) & 1u) {
        float acc = 0.f;
        const float* qr = Qs + r * L;
        const float* kr = Es + kk * (L + 1);
        for (int d = 0; d < L; ++d) acc = fmaf(qr[d], kr[d], acc);
        s[u] = acc * scale;
      }
    }
    const float m_new = fmaxf(mrow, max16(fmaxf(s[0], s[1])));
    const float alpha = mrow == -INFINITY ? 0.f : expf(mrow - m_new);
    const float p0 = s[0] == -INFINITY ? 0.f : expf(s[0] - m_new);
    const float p1 = s[1] == -INFINITY ? 0.f : expf(s[1] - m_new);
    lrow = lrow * alpha + sum16(p0 + p1);
    mrow = m_new;
    Ps[r * KT + c0] = p0;
    Ps[r * KT + c0 + 16] = p1;
    __syncthreads();
    // unseen keys are left out of the sum: their entries may hold anything
#pragma unroll
    for (int k = 0; k < MAX_OUT; ++k) {
      if (k < nout) {
        const int c = c0 + 16 * k;
        float acc = o[k] * alpha;
        for (int kk = 0; kk < KT; ++kk)
          if ((vis >> kk) & 1u) acc = fmaf(Ps[r * KT + kk], Es[kk * (L + 1) + c], acc);
        o[k] = acc;
      }
    }
  }
  if (live) {
    const bool any = lrow > 0.f;
#pragma unroll
    for (int k = 0; k < MAX_OUT; ++k)
      if (k < nout) o_lat[row * rkv + c0 + 16 * k] = from_f32<TO>(any ? o[k] / lrow : 0.f);
    if (lse && c0 == 0) lse[row] = any ? mrow + logf(lrow) : -INFINITY;
    if (vis_stats && (r0 + r) % a.H == 0 && c0 == 0) {
      vis_stats[m * 3 + 0] = cnt;
      vis_stats[m * 3 + 1] = first;
      vis_stats[m * 3 + 2] = last;
    }
  }
}

template <typename TC>
__global__ void __launch_bounds__(THREADS)
key_weights_kernel(const tree::Rule a, const TC* __restrict__ q_abs, const TC* __restrict__ cache,
                   int L, int tiles, float scale, const float* __restrict__ lse, float decay,
                   const float* prior, float* out, long ldw) {
  extern __shared__ float sm[];
  float* Qs = sm;                      // [RT][L]
  float* Es = Qs + RT * L;             // [KT][L + 1]
  float* Ps = Es + KT * (L + 1);       // [RT][KT]
  const int b = blockIdx.x / tiles, j0 = blockIdx.x % tiles * KT;
  const int tid = threadIdx.x, r = tid / 16, c0 = tid % 16;
  int W, ctx;
  const int n0 = tree::block_keys(a, b, &W, &ctx, tid == 0 && j0 == 0);
  const int n = (int)min((long)n0, ldw);
  if (n < n0 && tid == 0 && j0 == 0) set_status(a.status, MLA_DEV_BAD_LENGTH);
  if (j0 >= n) return;
  stage_keys(a, cache, b, j0, n, L, Es);
  float sum[2] = {0.f, 0.f};
  for (int r0 = 0; r0 < a.T * a.H; r0 += RT) {
    const int rows = min(RT, a.T * a.H - r0);
    __syncthreads();
    for (int idx = tid; idx < RT * L; idx += THREADS) {
      const int rr = idx / L;
      Qs[idx] = rr < rows ? to_f32(q_abs[((long)b * a.T * a.H + r0 + rr) * L + idx % L]) : 0.f;
    }
    const bool live = r < rows;
    const int i = live ? (r0 + r) / a.H : 0;
    const float l = live ? lse[(long)b * a.T * a.H + r0 + r] : -INFINITY;
    bool ok = live && l != -INFINITY && (a.q_visible ? a.q_visible[(long)b * a.T + i] != 0 : true);
    if (ok && a.parent) ok = tree::in_tree(a, a.parent + (long)b * a.T, i, c0 == 0);
    const unsigned vis = (unsigned)tree::key_bits(a, b, i, ok, n0, W, ctx, j0);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int kk = c0 + 16 * u;
      if ((vis >> kk) & 1u) {
        float acc = 0.f;
        const float* qr = Qs + r * L;
        const float* kr = Es + kk * (L + 1);
        for (int d = 0; d < L; ++d) acc = fmaf(qr[d], kr[d], acc);
        sum[u] += expf(acc * scale - l);
      }
    }
  }
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

size_t smem_bytes(int L) { return sizeof(float) * (RT * L + KT * (L + 1) + RT * KT); }

template <typename K>
void allow_smem(K* kernel) {
  cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
}

}  // namespace

void tree_attention(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                    const void* q_abs, const void* cache, void* o_lat, float* lse, int32_t* vis_stats) {
  const Layout& l = h->lay;
  static std::once_flag once;
  std::call_once(once, [] {
    allow_smem(tree_attn_kernel<float, float>);
    allow_smem(tree_attn_kernel<__nv_bfloat16, __half>);
  });
  const int tiles = (r.T * r.H + RT - 1) / RT;
  const unsigned grid = (unsigned)num_blocks * tiles;
  if (h->cfg.dtype == MLA_BF16)
    tree_attn_kernel<__nv_bfloat16, __half><<<grid, THREADS, smem_bytes(l.L), st>>>(
        r, (const __nv_bfloat16*)q_abs, (const __nv_bfloat16*)cache, l.rkv, l.L, tiles, h->scale,
        (__half*)o_lat, lse, vis_stats);
  else
    tree_attn_kernel<float, float><<<grid, THREADS, smem_bytes(l.L), st>>>(
        r, (const float*)q_abs, (const float*)cache, l.rkv, l.L, tiles, h->scale, (float*)o_lat, lse, vis_stats);
}

void key_weights(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                 const void* q_abs, const void* cache, const float* lse, float decay,
                 const float* prior, float* out, long ldw) {
  const Layout& l = h->lay;
  static std::once_flag once;
  std::call_once(once, [] {
    allow_smem(key_weights_kernel<float>);
    allow_smem(key_weights_kernel<__nv_bfloat16>);
  });
  const long keys = min((long)r.max_pages * r.page_size, ldw);
  const int tiles = (int)((keys + KT - 1) / KT);
  const unsigned grid = (unsigned)num_blocks * tiles;
  if (h->cfg.dtype == MLA_BF16)
    key_weights_kernel<__nv_bfloat16><<<grid, THREADS, smem_bytes(l.L), st>>>(
        r, (const __nv_bfloat16*)q_abs, (const __nv_bfloat16*)cache, l.L, tiles, h->scale, lse, decay, prior, out, ldw);
  else
    key_weights_kernel<float><<<grid, THREADS, smem_bytes(l.L), st>>>(
        r, (const float*)q_abs, (const float*)cache, l.L, tiles, h->scale, lse, decay, prior, out, ldw);
}

}  // namespace simt
}  // namespace mla
