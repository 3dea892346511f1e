// Launchers of the tensor-core kernels over trees (tree_attn_tc.cu, key_weights_tc.cu).
#pragma once

#include <cuda.h>

#include "tree.cuh"

namespace mla {
namespace tc {

struct TreeParams {
  CUtensorMap tmQ;    // Q_abs bf16 [rows, 576], chunked view, box 128 rows x 7 chunks
  CUtensorMap tmQ01;  // the same, box 128 rows x 2 chunks
  CUtensorMap tmC;    // the cache, chunked view, box 128 rows x 2 chunks (not for pairs)
  CUtensorMap tmK;    // the cache, box 64 dims x seg_rows
  tree::Rule rule;
  __half* o_lat;      // [rows, 512]
  float* lse;         // [rows] or NULL
  int32_t* vis_stats;
  float* part;        // [parts, rows, 512] when the parts do not all meet in a cluster
  float* part_lse;    // [parts, rows] log2-sum-exp
  long rows;
  int cluster_parts;  // parts of a key range that share a cluster: 1, 2, 4
  int group0, rest;   // first cluster's number; whether this is the launch of the last wave's units
  int seg_rows, tiles_per_block;
  float scale_log2;
};

struct WeightParams {
  CUtensorMap tmQ;    // Q_abs, chunked view, box q_box_rows rows x 1 or 3 chunks
  CUtensorMap tmC;    // the cache, chunked view, box 128 rows x 3 chunks
  CUtensorMap tmK;    // the cache, box 64 dims x seg_rows
  tree::Rule rule;
  const float* lse;
  const float* prior; // may be NULL
  float* out;         // [num_blocks, ldw]
  float* part;        // [splits, num_blocks, ldp] when splits > 1
  long ldw, ldp;
  int num_blocks, splits, seg_rows, q_box_rows;
  float decay, scale;
};

size_t tree_attention_ws(const mla_handle* h, const mla_attn_desc_t& d);
mla_status_t tree_attention(cudaStream_t st, mla_handle* h, const tree::Rule& r,
                            const mla_attn_desc_t& d, const __nv_bfloat16* q_abs,
                            const __nv_bfloat16* cache, __half* o_lat, float* lse, void* ws, bool pdl);


size_t key_weights_ws(const mla_handle* h, const mla_attn_desc_t& d, long ldw);
mla_status_t key_weights(cudaStream_t st, mla_handle* h, const tree::Rule& r, const mla_attn_desc_t& d,
                         const __nv_bfloat16* q_abs, const __nv_bfloat16* cache, const float* lse,
                         float decay, const float* prior, float* out, long ldw, void* ws);

}  // namespace tc
}  // namespace mla
