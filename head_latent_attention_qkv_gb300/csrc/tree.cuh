// Which keys a query sees when its block's own keys form a tree, and the
// launchers of the kernels built on it (tree attention, key weights).
//
// A block of T nodes over a context: logical keys 0 .. kv_len - T - 1 are the
// context, key kv_len - T + k is node k's own.  parent[i] is -1 (a child of
// the context) or an earlier node; any other value takes the node, and the
// nodes below it, out of the tree: their rows see nothing and nobody sees
// their keys.  Node i sees the context and the nodes on its path from the
// root, itself among them; a window W > 0 keeps the keys less than W positions
// before it (a context key's position is its index, a node's its own
// positions[] entry).  Without parents the rule of mla_attn_desc_t applies.
#pragma once

#include "common.cuh"

namespace mla {
namespace tree {

constexpr int MAX_NODES = 1024;

struct Rule {
  const int32_t* block_table; const int32_t* kv_len; const int32_t* window;
  const uint8_t* q_visible; const int32_t* positions;
  const int32_t* parent;        // NULL: the block rule
  int num_pages, page_size, max_pages, T, H;
  uint32_t* status;
};

// Keys of a block of length n and window *W (0 when one of them is rejected)
// and, with a tree, the context length.
__device__ __forceinline__ int checked_keys(const Rule& a, int n, int* W, int* ctx, bool report) {
  const int cap = a.max_pages * a.page_size;
  if (n < 0 || n > cap || (a.parent && n < a.T)) {
    if (report) set_status(a.status, MLA_DEV_BAD_LENGTH);
    n = a.parent ? 0 : max(0, min(n, cap));
  }
  if (*W < 0) {
    if (report) set_status(a.status, MLA_DEV_BAD_WINDOW);
    n = 0;
  }
  *ctx = a.parent ? max(0, n - a.T) : n;
  return n;
}
// Those of block b, and its window.
__device__ __forceinline__ int block_keys(const Rule& a, int b, int* W, int* ctx, bool report) {
  *W = a.window ? a.window[b] : 0;
  return checked_keys(a, a.kv_len[b], W, ctx, report);
}

// First context key that a window W > 0 leaves to position p.  The least position of
// a block's rows is taken over padding, too, whose entries may hold anything: a
// difference that wraps would hide keys from the other rows.
__device__ __forceinline__ int window_start(int p, int W) { return p < W ? 0 : p - W + 1; }

// Whether node i's path to the context is sound (its ancestors and itself in
// the tree).  `parent` points at the block's T entries; every step goes to an
// earlier node, so the walk ends.
__device__ __forceinline__ bool in_tree(const Rule& a, const int32_t* parent, int i, bool report) {
  while (true) {
    const int p = parent[i];
    if (p == -1) return true;
    if (p < -1) return false;
    if (p >= i) {
      if (report) set_status(a.status, MLA_DEV_BAD_TREE);
      return false;
    }
    i = p;
  }
}

// Bits of the nodes k0 .. k0 + 63 (k0 >= 0) that node i sees (i in the tree;
// the walk ends at a parent that is no earlier node, too).
__device__ __forceinline__ unsigned long long path_bits(const int32_t* parent, const int32_t* pos,
                                                        int W, int i, int k0) {
  unsigned long long m = 0;
  const int pi = pos[i];
  for (int k = i; k >= k0;) {
    const bool near = W == 0 || pi - pos[k] < W;
    if (near && k < k0 + 64) m |= 1ull << (k - k0);
    const int p = parent[k];
    if (p >= k) break;
    k = p;
  }
  return m;
}

// Bits of the context's keys (the whole block's without parents) among j0 .. j0 +
// 63 that query i of block b sees.  n, W and ctx are block_keys()'s.
__device__ __forceinline__ unsigned long long context_bits(const Rule& a, long b, int i, int n, int W,
                                                           int ctx, int j0) {
  const int lo = W > 0 ? max(0, min(n, window_start(a.positions[b * a.T + i], W)) - j0) : 0, hi = min(ctx - j0, 64);
  if (hi <= lo) return 0ull;
  return (hi >= 64 ? ~0ull : (1ull << hi) - 1ull) & (~0ull << lo);
}

// Bits of keys j0 .. j0 + 63 that query i of block b sees; `ok`: the row sees
// anything at all (visible, in the tree).
__device__ __forceinline__ unsigned long long key_bits(const Rule& a, long b, int i, bool ok, int n,
                                                       int W, int ctx, int j0) {
  if (!ok || j0 >= n) return 0ull;
  unsigned long long m = context_bits(a, b, i, n, W, ctx, j0);
  if (a.parent && j0 + 64 > ctx) {
    const int k0 = j0 - ctx;                          // node of bit 0 (negative: still context)
    const unsigned long long t = path_bits(a.parent + b * a.T, a.positions + b * a.T, W, i, max(k0, 0));
    m |= k0 >= 0 ? t : t << (-k0);
  }
  return m;
}

// in_tree() and the bits of nodes k0 .. k0 + 63 that node i sees in one walk: 0 when
// it is not in the tree.  Its own bit is set otherwise (if it is among them).
__device__ __forceinline__ unsigned long long walk_bits(const Rule& a, long b, int i, int W, int k0,
                                                        bool* sound, bool report) {
  const int32_t *parent = a.parent + b * a.T, *pos = a.positions + b * a.T;
  const int pi = W > 0 ? pos[i] : 0;
  unsigned long long m = 0;
  while (true) {
    const uint32_t rel = (uint32_t)(i - k0);
    if (rel < 64u && (W == 0 || pi - pos[i] < W)) m |= 1ull << rel;
    const int p = parent[i];
    if (p < 0 || p >= i) {
      if (p >= i && report) set_status(a.status, MLA_DEV_BAD_TREE);
      *sound = p == -1;
      return p == -1 ? m : 0ull;
    }
    i = p;
  }
}
// Bits of nodes 0 .. 63 moved to keys j0 .. j0 + 63.
__device__ __forceinline__ unsigned long long place_bits(unsigned long long nodes, int ctx, int j0) {
  const int sh = ctx - j0;
  return sh >= 64 || sh <= -64 ? 0ull : sh >= 0 ? nodes << sh : nodes >> (-sh);
}

}  // namespace tree

namespace simt {
// Tree attention and key weights of the fp32 layers, on the CUDA cores (q_abs and
// cache 16-byte aligned).
void tree_attention(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                    const float* q_abs, const float* cache, float* o_lat, float* lse, int32_t* vis_stats);
void key_weights(cudaStream_t st, const mla_handle* h, const tree::Rule& r, int num_blocks,
                 const float* q_abs, const float* cache, const float* lse, float decay,
                 const float* prior, float* out, long ldw);
}  // namespace simt
}  // namespace mla
