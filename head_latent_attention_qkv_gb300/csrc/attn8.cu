// Latent attention over the 8-bit cache (mla_latent_attention8), a plain kernel: one
// CTA per query row, chunks of 32 keys, online softmax in fp32.
#include "cache8.cuh"

#include <math.h>

namespace mla {
namespace cache8 {
namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32, CHUNK = 32;

struct Attn8Args {
  tree::Rule rule;
  const uint8_t* latent;
  const __nv_bfloat16* rope;
  const float* scale;
  const __nv_bfloat16* q;
  __half* o_lat;
  float* lse;
  int32_t* vis_stats;
  float softmax_scale;
};

__global__ void __launch_bounds__(THREADS) attn8_kernel(const Attn8Args a) {
  __shared__ float q[ENTRY], p[CHUNK], key_scale[CHUNK];
  __shared__ long slots[CHUNK];
  const long row = blockIdx.x, token = row / a.rule.H;
  const long b = token / a.rule.T;
  const int i = (int)(token % a.rule.T), tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  for (int d = tid; d < ENTRY; d += THREADS) q[d] = __bfloat162float(a.q[row * ENTRY + d]);
  int W, ctx;
  const bool lead = row % ((long)a.rule.T * a.rule.H) == 0 && tid == 0;
  const int n = tree::block_keys(a.rule, (int)b, &W, &ctx, lead);
  bool ok = !a.rule.q_visible || a.rule.q_visible[token] != 0;
  if (a.rule.parent && n > 0)
    ok = tree::in_tree(a.rule, a.rule.parent + b * a.rule.T, i, tid == 0 && row % a.rule.H == 0) && ok;
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
  int seen = 0, first = -1, last = -1;
  for (int j0 = 0; j0 < n; j0 += CHUNK) {
    const unsigned long long bits = tree::key_bits(a.rule, b, i, ok, n, W, ctx, j0) & 0xffffffffull;
    if (!bits) continue;
    __syncthreads();
    if (tid < CHUNK) {
      const int j = j0 + tid;
      long slot = -1;
      if ((bits >> tid) & 1) {
        const int pg = a.rule.block_table[b * a.rule.max_pages + j / a.rule.page_size];
        if (pg < 0 || pg >= a.rule.num_pages) set_status(a.rule.status, MLA_DEV_BAD_PAGE);
        else slot = (long)pg * a.rule.page_size + j % a.rule.page_size;
      }
      slots[tid] = slot;
      key_scale[tid] = slot >= 0 ? a.scale[slot] : 0.f;
    }
    __syncthreads();
    for (int k = warp; k < CHUNK; k += WARPS) {
      const long slot = slots[k];
      float s = 0.f;
      if (slot >= 0) {
        float x = 0.f;
        for (int d = 2 * lane; d < RANK; d += 64) {
          const float2 f = from_e4m3x2(*reinterpret_cast<const uint16_t*>(a.latent + slot * RANK + d));
          x = fmaf(q[d], f.x, fmaf(q[d + 1], f.y, x));
        }
        s = x * key_scale[k];
        for (int d = lane; d < ROPE; d += 32) s = fmaf(q[RANK + d], __bfloat162float(a.rope[slot * ROPE + d]), s);
      }
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) p[k] = ((bits >> k) & 1) ? s * a.softmax_scale : -INFINITY;
    }
    __syncthreads();
    float mx = m;
    for (int k = 0; k < CHUNK; ++k) mx = fmaxf(mx, p[k]);
    const float f = m == -INFINITY ? 0.f : expf(m - mx);
    l *= f; o0 *= f; o1 *= f;
    m = mx;
    for (int k = 0; k < CHUNK; ++k) {
      if (!((bits >> k) & 1)) continue;
      const float w = expf(p[k] - m), ws = w * key_scale[k];
      l += w;
      if (slots[k] >= 0) {
        const float2 v = from_e4m3x2(*reinterpret_cast<const uint16_t*>(a.latent + slots[k] * RANK + 2 * tid));
        o0 = fmaf(ws, v.x, o0);
        o1 = fmaf(ws, v.y, o1);
      }
    }
    seen += __popcll(bits);
    if (first < 0) first = j0 + __ffsll((long long)bits) - 1;
    last = j0 + 63 - __clzll((long long)bits);
  }
  const float inv = seen ? 1.f / l : 0.f;
  a.o_lat[row * RANK + 2 * tid] = __float2half_rn(seen ? o0 * inv : 0.f);
  a.o_lat[row * RANK + 2 * tid + 1] = __float2half_rn(seen ? o1 * inv : 0.f);
  if (tid == 0) {
    if (a.lse) a.lse[row] = seen ? m + logf(l) : -INFINITY;
    if (a.vis_stats && row % a.rule.H == 0) {
      a.vis_stats[token * 3] = seen;
      a.vis_stats[token * 3 + 1] = first;
      a.vis_stats[token * 3 + 2] = last;
    }
  }
}

}  // namespace

size_t attention_ws(const mla_handle* h, const mla_attn_desc_t& d) { return 0; }

mla_status_t attention(cudaStream_t st, mla_handle* h, const tree::Rule& r, const mla_attn_desc_t& d,
                       const __nv_bfloat16* q_abs, const mla_cache8_t& c, __half* o_lat, float* lse,
                       void* ws, bool pdl) {
  const Attn8Args a{r, (const uint8_t*)c.latent, (const __nv_bfloat16*)c.rope, c.scale, q_abs, o_lat, lse,
                    d.vis_stats, h->scale};
  attn8_kernel<<<(unsigned)(d.num_blocks * (long)d.block_len * h->lay.H), THREADS, 0, st>>>(a);
  MLA_CUDA_TRY(cudaGetLastError());
  h->launches += 1;
  return MLA_OK;
}

}  // namespace cache8
}  // namespace mla
