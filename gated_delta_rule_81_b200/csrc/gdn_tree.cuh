// Trees of drafted tokens: the device-side reading of a sequence's parent array, and the launch
// parameters of the tree kernels (internal to libgdn.so).
#pragma once

#include "../../include/gdn.h"
#include "gdn_kernels.cuh"

namespace gdn {

constexpr int kMaxNodes = GDN_MAX_TREE_NODES;
constexpr int kMaxHeads = 8;          // value heads per key head
constexpr int kDevErrCacheFull = 16;  // a sequence's KV cache has no row for a new token
constexpr int kDevErrCacheLen = 32;   // a cache_len outside [0, cap]
constexpr int kDevErrBadIndex = 128;  // a tree parent, an accepted node or a cache row outside its range

struct Tree {
  int parent[kMaxNodes];                // -1: child of the committed prefix; only meaningful for nodes that are there
  unsigned long long mask[kMaxNodes];   // bit j: node j is an ancestor of this node or the node itself; 0: absent
  int up[kMaxNodes];                    // (scratch) the node 1, 2, 4, .. steps up, -1 past the root, -2 absent
};

// One warp (all lanes) reads sequence n's T parents and forms the ancestor masks by pointer
// doubling: after round i a node's mask holds its 2^i nearest ancestors (itself included), so
// 64 nodes take 6 rounds, whatever the depth.
__device__ __forceinline__ void tree_load(Tree& tr, const int* parent, long long n, int T, int* err) {
  const int lane = threadIdx.x & 31;
  for (int t = lane; t < kMaxNodes; t += 32) {
    int p = -2;
    if (t < T) {
      p = parent ? parent[n * T + t] : t - 1;
      if (p >= t) {
        if (err) atomicOr(err, kDevErrBadIndex);
        p = -2;
      }
      if (p < -2) p = -2;
    }
    tr.parent[t] = p;
    tr.up[t] = p;
    tr.mask[t] = 1ull << t;
  }
  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < 6; ++i) {
    int u[2];
    unsigned long long m[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = lane + 32 * e, p = tr.up[t];
      m[e] = tr.mask[t] | (p >= 0 ? tr.mask[p] : 0ull);
      u[e] = p >= 0 ? tr.up[p] : p;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      tr.up[lane + 32 * e] = u[e];
      tr.mask[lane + 32 * e] = m[e];
    }
    __syncwarp();
  }
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (tr.up[lane + 32 * e] != -1) tr.mask[lane + 32 * e] = 0ull;  // absent, or below an absent node
  __syncwarp();
}

// The accepted path's mask: 0 when nothing is accepted, or the entry is out of range or absent (reported).
__device__ __forceinline__ unsigned long long tree_accepted(const Tree& tr, int accepted, int T, int* err) {
  if (accepted == -1) return 0ull;
  const unsigned long long m = accepted >= 0 && accepted < T ? tr.mask[accepted] : 0ull;
  if (m == 0ull && err) atomicOr(err, kDevErrBadIndex);
  return m;
}

struct TreeParams {
  const bf16 *q, *k, *v, *a, *b, *z;  // node t of sequence n is token n * T + t
  long long sq, sk, sv, sz, sa, sb;   // token strides (elements)
  const bf16* conv_w;
  const float* A_log;
  const bf16* norm_w;
  float scale;
  int H_k, H_v, N, T;
  const int* parent;      // [N][T] or null (a chain)
  const int* accepted;    // [N] (commit)
  const int* state_slot;  // [N] or null (slot n)
  int n_slots;
  const float* state_in;  // [n_slots][H_v][128][128]
  float* state_out;       // (commit) may be state_in
  const bf16* conv_in;    // [n_slots][3][C_conv]
  bf16* conv_out;         // (commit) may be conv_in
  bf16* out;              // [N * T][H_v][128] (verification)
  int* err;
};

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream, void* const* events);
cudaError_t launch_tree_commit(const TreeParams& p, cudaStream_t stream);

struct RopeParams {
  const bf16 *q, *k, *v;
  long long ld_q, ld_k, ld_v;
  const bf16 *q_norm_w, *k_norm_w;
  int H_q, H_kv;
  long long n_tok;
  const int* positions;     // [n_tok], or null: the token's index, or (tree_T > 0) from the tree
  const long long* rows;    // [n_tok] or null (row = token)
  long long n_rows;
  int tree_T;               // > 0: token n * tree_T + t is node t of sequence n, at position base[n] + its depth
  const int* parent;        // [n_tok] or null (a chain); with tree_T > 0
  const int* base;          // [n_tok / tree_T]
  bf16 *q_out, *k_out, *v_out;
  long long ld_qo, ld_ko, ld_vo;
  int* err;
};

cudaError_t launch_qk_norm_rope(const gdn_rope& rope, const RopeParams& p, cudaStream_t stream);

struct AttnTreeParams {
  const bf16* q;          // [N * T][ld_q]
  long long ld_q;
  const bf16 *k_tree, *v_tree;
  long long ld_kt, ld_vt;
  const bf16 *k_cache, *v_cache;  // [N][cap][H_kv][D]
  int cap;
  const int* cache_len;   // [N]
  const int* parent;      // [N][T] or null
  const bf16* g;          // [N * T][ld_g] or null
  long long ld_g;
  int H_q, H_kv, D, N, T;
  float scale;
  bf16* out;              // [N * T][H_q][D]
  void* workspace;
  int* err;
};

size_t attention_tree_workspace(int H_q, int H_kv, int D, int N, int T);
cudaError_t launch_attention_tree(const AttnTreeParams& p, cudaStream_t stream);

struct AttnCommitParams {
  const bf16 *k_tree, *v_tree;
  long long ld_kt, ld_vt;
  int H_kv, D, N, T;
  const int *parent, *accepted;
  bf16 *k_cache, *v_cache;
  int cap;
  const int* cache_len;
  int* cache_len_out;
  int* err;
};

cudaError_t launch_attn_tree_commit(const AttnCommitParams& p, cudaStream_t stream);

}  // namespace gdn
