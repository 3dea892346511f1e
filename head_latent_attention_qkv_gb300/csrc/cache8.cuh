// The latent cache in 8 bits: one entry's form, and the launchers of the kernels that
// write it and attend it (cache8.cu, attn8_tc.cu).
//
// An entry is 512 latent dims in e4m3 over a scale 2^k of its own, 64 rotary dims in
// bf16, and the scale.  A power of two, so that every number the cache holds is a
// bf16 number (4 significant bits at any exponent) and reading back rounds nothing; one for the
// whole latent, since e4m3 itself spans 2^17 and a normalised latent far less.
// The rotary dims stay in bf16: their error would rotate into the scores of far keys.
#pragma once

#include <cuda.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "tree.cuh"

namespace mla {
namespace cache8 {

constexpr int RANK = 512, ROPE = 64, ENTRY = RANK + ROPE;
constexpr int K_MIN = -64, K_MAX = 119;    // least exponent of a scale, and that of a latent just below 2^127

// Exponent of an entry's scale from the largest |bits| of its latent's bf16 numbers: the
// least k >= K_MIN with amax <= 448 2^k (448 = 1.75 2^8).
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  return max((int)(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 96u ? 1 : 0), K_MIN);
}
__device__ __forceinline__ float pow2(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }
// Whether a scale is one that a store writes for an entry that it holds: 2^K_MIN .. 2^K_MAX.  (The bits above those
// of 2^K_MIN, turned so that a power of two is its exponent and every other number large.)
__device__ __forceinline__ bool sound_scale(float s) {
  const uint32_t above = __float_as_uint(s) - ((uint32_t)(K_MIN + 127) << 23);
  return __funnelshift_l(above, above, 9) <= (uint32_t)(K_MAX - K_MIN);
}
// An entry that 8 bits do not hold: something NaN or infinite, or a latent of 2^127 or more.
__device__ __forceinline__ bool poisoned(uint32_t amax_latent_bits, uint32_t amax_rope_bits) {
  return amax_latent_bits >= 0x7f00u || amax_rope_bits >= 0x7f80u;
}
// Two e4m3 numbers, `a` in the low byte (rounded to nearest even).
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// The numbers that two e4m3 bytes stand for.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t x) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)x, __NV_E4M3)));
}

// Entries from their raw fp32 rows (row stride ld), as simt::kv_finish, into the 8-bit cache.
void kv_finish8(cudaStream_t st, const mla_handle* h, const float* kv, long ld, int n,
                const int32_t* positions, const int64_t* slots, const mla_cache8_t& c, long num_slots,
                bool pdl);

// What every entry point asks of a cache (`who` opens the message).
mla_status_t check_cache(const mla_handle* h, const mla_cache8_t* c, int num_pages, const char* who);

size_t attention_ws(const mla_handle* h, const mla_attn_desc_t& d);
mla_status_t attention(cudaStream_t st, mla_handle* h, const tree::Rule& r, const mla_attn_desc_t& d,
                       const __nv_bfloat16* q_abs, const mla_cache8_t& c, __half* o_lat, float* lse,
                       void* ws, bool pdl);

}  // namespace cache8
}  // namespace mla
