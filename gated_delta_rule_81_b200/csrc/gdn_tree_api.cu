// C ABI of tree decoding: argument validation, workspace layout and kernel launches of the calls that
// verify a tree of drafted tokens and commit its accepted path.  Declared in include/gdn.h.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "gdn_checks.cuh"
#include "gdn_tree.cuh"

using namespace gdn;

namespace {

constexpr int kMaxGridYZ = 65535;  // sequences per call: a grid's y extent

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// bytes from the first element of rows x ld to the end of the last row's `width` elements
size_t extent(long long rows, long long ld, long long width) {
  if (rows <= 0 || width <= 0) return 0;
  return sizeof(bf16) * (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(width));
}

bool inputs_overlap(const gdn_inputs* in, long long T_tot, const void* p, size_t bytes) {
  const long long qk = static_cast<long long>(in->H_k) * GDN_HEAD_DIM, vz = static_cast<long long>(in->H_v) * GDN_HEAD_DIM;
  const size_t conv_w = static_cast<size_t>(2 * in->H_k + in->H_v) * GDN_HEAD_DIM * GDN_CONV_TAPS * sizeof(bf16);
  return overlap(p, bytes, in->q, extent(T_tot, in->stride_q, qk)) ||
         overlap(p, bytes, in->k, extent(T_tot, in->stride_k, qk)) ||
         overlap(p, bytes, in->v, extent(T_tot, in->stride_v, vz)) ||
         overlap(p, bytes, in->z, extent(T_tot, in->stride_z, vz)) ||
         overlap(p, bytes, in->a, extent(T_tot, in->stride_a, in->H_v)) ||
         overlap(p, bytes, in->b, extent(T_tot, in->stride_b, in->H_v)) || overlap(p, bytes, in->conv_w, conv_w) ||
         overlap(p, bytes, in->A_log, static_cast<size_t>(in->H_v) * sizeof(float)) ||
         overlap(p, bytes, in->norm_w, GDN_HEAD_DIM * sizeof(bf16));
}

size_t state_bytes(int H_v, int n) {
  return static_cast<size_t>(n) * H_v * GDN_HEAD_DIM * GDN_HEAD_DIM * sizeof(float);
}

size_t conv_bytes(int H_k, int H_v, int n) {
  return static_cast<size_t>(n) * 3 * (2 * H_k + H_v) * GDN_HEAD_DIM * sizeof(bf16);
}

TreeParams tree_params(const gdn_inputs* in, int N, int T, const int* parent, const int* state_slot, int n_slots,
                       int* err) {
  TreeParams p = {};
  p.q = static_cast<const bf16*>(in->q);
  p.k = static_cast<const bf16*>(in->k);
  p.v = static_cast<const bf16*>(in->v);
  p.a = static_cast<const bf16*>(in->a);
  p.b = static_cast<const bf16*>(in->b);
  p.z = static_cast<const bf16*>(in->z);
  p.sq = in->stride_q; p.sk = in->stride_k; p.sv = in->stride_v; p.sz = in->stride_z;
  p.sa = in->stride_a; p.sb = in->stride_b;
  p.conv_w = static_cast<const bf16*>(in->conv_w);
  p.A_log = in->A_log;
  p.norm_w = static_cast<const bf16*>(in->norm_w);
  p.scale = in->scale;
  p.H_k = in->H_k;
  p.H_v = in->H_v;
  p.N = N;
  p.T = T;
  p.parent = parent;
  p.state_slot = state_slot;
  p.n_slots = n_slots;
  p.err = err;
  return p;
}

// the counts common to the tree calls
gdn_status check_tree_counts(int N, int T) {
  if (N < 0 || T < 1 || T > GDN_MAX_TREE_NODES) return GDN_ERR_INVALID_ARG;
  if (N > kMaxGridYZ) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn_status check_decode_tree(const gdn_inputs* in, int N, int T, const int* parent, const float* state,
                             const void* conv_state, const int* state_slot, int n_slots, const void* out) {
  gdn_status st = check_tree_counts(N, T);
  if (st != GDN_OK) return st;
  if (n_slots < 0) return GDN_ERR_INVALID_ARG;
  const long long T_tot = static_cast<long long>(N) * T;
  if ((st = check_inputs(in, T_tot)) != GDN_OK || N == 0) return st;
  if (!state || !conv_state || !out) return GDN_ERR_INVALID_ARG;
  if (!state_slot && n_slots < N) return GDN_ERR_INVALID_ARG;
  if (!aligned16(state) || !aligned16(conv_state) || !aligned16(out) || !aligned4(state_slot) || !aligned4(parent))
    return GDN_ERR_MISALIGNED;
  const size_t ob = static_cast<size_t>(T_tot) * in->H_v * GDN_HEAD_DIM * sizeof(bf16);
  if (inputs_overlap(in, T_tot, out, ob) || overlap(out, ob, state, state_bytes(in->H_v, n_slots)) ||
      overlap(out, ob, conv_state, conv_bytes(in->H_k, in->H_v, n_slots)) ||
      overlap(out, ob, state_slot, sizeof(int) * static_cast<size_t>(N)) ||
      overlap(out, ob, parent, sizeof(int) * static_cast<size_t>(T_tot)))
    return GDN_ERR_ALIAS;
  return GDN_OK;
}

gdn_status check_tree_commit(const gdn_inputs* in, int N, int T, const int* parent, const int* accepted,
                             const float* state_in, const float* state_out, const void* conv_in, const void* conv_out,
                             const int* state_slot, int n_slots) {
  gdn_status st = check_tree_counts(N, T);
  if (st != GDN_OK) return st;
  if (n_slots < 0) return GDN_ERR_INVALID_ARG;
  const long long T_tot = static_cast<long long>(N) * T;
  if ((st = check_inputs(in, T_tot)) != GDN_OK || N == 0) return st;
  if (!accepted || !state_in || !state_out || !conv_in || !conv_out) return GDN_ERR_INVALID_ARG;
  if (!state_slot && n_slots < N) return GDN_ERR_INVALID_ARG;
  if (!aligned16(state_in) || !aligned16(state_out) || !aligned16(conv_in) || !aligned16(conv_out) ||
      !aligned4(state_slot) || !aligned4(parent) || !aligned4(accepted))
    return GDN_ERR_MISALIGNED;
  const size_t sb = state_bytes(in->H_v, n_slots), cb = conv_bytes(in->H_k, in->H_v, n_slots);
  const size_t nb = sizeof(int) * static_cast<size_t>(N), tb = sizeof(int) * static_cast<size_t>(T_tot);
  if ((state_in != state_out && overlap(state_in, sb, state_out, sb)) ||
      (conv_in != conv_out && overlap(conv_in, cb, conv_out, cb)) || overlap(state_out, sb, conv_out, cb) ||
      overlap(state_out, sb, conv_in, cb) || overlap(state_in, sb, conv_out, cb))
    return GDN_ERR_ALIAS;
  if (inputs_overlap(in, T_tot, state_out, sb) || inputs_overlap(in, T_tot, conv_out, cb)) return GDN_ERR_ALIAS;
  for (const int* idx : {parent, accepted, state_slot}) {
    const size_t ib = idx == parent ? tb : nb;
    if (overlap(idx, ib, state_out, sb) || overlap(idx, ib, conv_out, cb)) return GDN_ERR_ALIAS;
  }
  return GDN_OK;
}

gdn_status check_layer(const gdn_layer* L) {
  if (!L || L->H_k <= 0 || L->H_v <= 0 || L->hidden <= 0 || L->H_v % L->H_k != 0) return GDN_ERR_INVALID_ARG;
  if (L->hidden % 64 != 0) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

// a projection's operands, as gdn_gemm_bf16 wants them, checked before the layer's first launch
gdn_status check_gemm(const void* A, long long lda, const void* B, long long ldb, const void* C, long long ldc,
                      long long M, long long N, long long K) {
  if (!A || !B || !C || lda < K || ldb < K || ldc < N) return GDN_ERR_INVALID_ARG;
  if (!aligned16(A) || !aligned16(B) || !aligned16(C) || ((lda | ldb | ldc) & 7)) return GDN_ERR_MISALIGNED;
  if (overlap(C, extent(M, ldc, N), A, extent(M, lda, K)) || overlap(C, extent(M, ldc, N), B, extent(N, ldb, K)))
    return GDN_ERR_ALIAS;
  return GDN_OK;
}

// The tree step's workspace of the attention layer, each part from a 1 KiB boundary: the projection
// (q | g | k | v of each node), q_hat, the nodes' normalised, rotated keys, the attention output, the attention's scratch.
struct AttnTreeLayout {
  size_t q_hat, k_tree, att, scratch, end;
};

constexpr long long kAttnQ = static_cast<long long>(GDN_ATTN_Q_HEADS) * GDN_ATTN_HEAD_DIM;
constexpr long long kAttnKv = static_cast<long long>(GDN_ATTN_KV_HEADS) * GDN_ATTN_HEAD_DIM;

AttnTreeLayout attn_tree_layout(int N, int T) {
  const size_t T_tot = static_cast<size_t>(N) * T;
  AttnTreeLayout L;
  L.q_hat = round_up(T_tot * GDN_ATTN_N_IN * 2, 1024);
  L.k_tree = L.q_hat + round_up(T_tot * kAttnQ * 2, 1024);
  L.att = L.k_tree + round_up(T_tot * kAttnKv * 2, 1024);
  L.scratch = L.att + round_up(T_tot * kAttnQ * 2, 1024);
  L.end = L.scratch + attention_tree_workspace(GDN_ATTN_Q_HEADS, GDN_ATTN_KV_HEADS, GDN_ATTN_HEAD_DIM, N, T);
  return L;
}

// the attention layer's rotation: the first 64 dims of each head, pairs (i, i + 32), base 1e7, eps 1e-6
const gdn_rope& attn_layer_rope() {
  static const gdn_rope rope = [] {
    gdn_rope r;
    gdn_rope_init(&r, GDN_ATTN_HEAD_DIM, 64, GDN_ROPE_HALF, GDN_ROPE_NONE, 1e7, 1.0, 0, 0.0, 0.0, 1e-6f);
    return r;
  }();
  return rope;
}

gdn_status check_cache(const void* k_cache, const void* v_cache, size_t kv_bytes) {
  if (!k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return GDN_ERR_MISALIGNED;
  return overlap(k_cache, kv_bytes, v_cache, kv_bytes) ? GDN_ERR_ALIAS : GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_decode_tree(const gdn_inputs* in, int N, int T, const int* parent, const float* state,
                           const void* conv_state, const int* state_slot, int n_slots, void* out, int* err,
                           void* stream) {
  const NvtxRange nvtx_range("gdn_decode_tree");
  const gdn_status st = check_decode_tree(in, N, T, parent, state, conv_state, state_slot, n_slots, out);
  if (st != GDN_OK || N == 0) return st;
  TreeParams p = tree_params(in, N, T, parent, state_slot, n_slots, err);
  p.state_in = state;
  p.conv_in = static_cast<const bf16*>(conv_state);
  p.out = static_cast<bf16*>(out);
  return launch_decode_tree(p, static_cast<cudaStream_t>(stream), in->events) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_decode_tree_commit(const gdn_inputs* in, int N, int T, const int* parent, const int* accepted,
                                  const float* state_in, float* state_out, const void* conv_in, void* conv_out,
                                  const int* state_slot, int n_slots, int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_decode_tree_commit");
  const gdn_status st = check_tree_commit(in, N, T, parent, accepted, state_in, state_out, conv_in, conv_out,
                                          state_slot, n_slots);
  if (st != GDN_OK || N == 0) return st;
  TreeParams p = tree_params(in, N, T, parent, state_slot, n_slots, err);
  p.accepted = accepted;
  p.state_in = state_in;
  p.state_out = state_out;
  p.conv_in = static_cast<const bf16*>(conv_in);
  p.conv_out = static_cast<bf16*>(conv_out);
  return launch_tree_commit(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_layer_tree_workspace_size(int H_k, int H_v, int N, int T) {
  if (H_k <= 0 || H_v <= 0 || N < 0 || T < 1 || T > GDN_MAX_TREE_NODES) return 0;
  const size_t T_tot = static_cast<size_t>(N) * T;
  return round_up(T_tot * layer_ld_proj(H_k, H_v) * 2, 1024) +
         round_up(T_tot * static_cast<size_t>(H_v) * GDN_HEAD_DIM * 2, 1024);
}

gdn_status gdn_layer_decode_tree(const gdn_layer* L, int N, int T, const int* parent, const void* x, long long ldx,
                                 const float* state, const void* conv_state, const int* state_slot, int n_slots,
                                 void* y, long long ldy, void* workspace, size_t workspace_bytes, int* err,
                                 void* stream) {
  const NvtxRange nvtx_range("gdn_layer_decode_tree");
  gdn_status s = check_layer(L);
  if (s == GDN_OK) s = check_tree_counts(N, T);
  if (s != GDN_OK || N == 0) return s;
  const long long T_tot = static_cast<long long>(N) * T;
  const size_t need = gdn_layer_tree_workspace_size(L->H_k, L->H_v, N, T);
  if (!x || !y || !L->w_in || !L->w_out) return GDN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  const long long n_in = gdn_layer_n_in(L->H_k, L->H_v), ld_p = layer_ld_proj(L->H_k, L->H_v);
  const long long d_v = static_cast<long long>(L->H_v) * GDN_HEAD_DIM;
  bf16* proj = static_cast<bf16*>(workspace);
  bf16* mix = reinterpret_cast<bf16*>(static_cast<uint8_t*>(workspace) + round_up(static_cast<size_t>(T_tot) * ld_p * 2, 1024));
  const gdn_inputs in = layer_mixer_inputs(L, proj, ld_p);
  // everything a later call would reject is rejected here, before the first launch
  const int slots = state_slot ? n_slots : N;
  if ((s = check_decode_tree(&in, N, T, parent, state, conv_state, state_slot, slots, mix)) != GDN_OK) return s;
  if ((s = check_gemm(x, ldx, L->w_in, L->ld_w_in, proj, ld_p, T_tot, n_in, L->hidden)) != GDN_OK) return s;
  if ((s = check_gemm(mix, d_v, L->w_out, L->ld_w_out, y, ldy, T_tot, L->hidden, d_v)) != GDN_OK) return s;
  const size_t yb = extent(T_tot, ldy, L->hidden);
  const size_t sb = state_bytes(L->H_v, slots), cb = conv_bytes(L->H_k, L->H_v, slots);
  if (overlap(y, yb, workspace, need) || overlap(x, extent(T_tot, ldx, L->hidden), workspace, need) ||
      overlap(state, sb, workspace, need) || overlap(conv_state, cb, workspace, need) || overlap(y, yb, state, sb) ||
      overlap(y, yb, conv_state, cb) || overlap(parent, sizeof(int) * static_cast<size_t>(T_tot), workspace, need) ||
      overlap(state_slot, sizeof(int) * static_cast<size_t>(N), workspace, need))
    return GDN_ERR_ALIAS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto mark = [&](int i) {
    if (L->events) cudaEventRecord(static_cast<cudaEvent_t>(L->events[i]), st);
  };
  mark(0);
  s = gdn_gemm_bf16(x, ldx, L->w_in, L->ld_w_in, proj, ld_p, static_cast<int>(T_tot), static_cast<int>(n_in), L->hidden,
                    err, stream);
  if (s != GDN_OK) return s;
  mark(1);
  s = gdn_decode_tree(&in, N, T, parent, state, conv_state, state_slot, slots, mix, err, stream);
  if (s != GDN_OK) return s;
  mark(2);
  s = gdn_gemm_bf16(mix, d_v, L->w_out, L->ld_w_out, y, ldy, static_cast<int>(T_tot), L->hidden, static_cast<int>(d_v),
                    err, stream);
  if (s != GDN_OK) return s;
  mark(3);
  return GDN_OK;
}

gdn_status gdn_layer_tree_commit(const gdn_layer* L, int N, int T, const int* parent, const int* accepted,
                                 float* state, void* conv_state, const int* state_slot, int n_slots,
                                 const void* workspace, size_t workspace_bytes, int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_layer_tree_commit");
  gdn_status s = check_layer(L);
  if (s == GDN_OK) s = check_tree_counts(N, T);
  if (s != GDN_OK || N == 0) return s;
  if (!workspace || workspace_bytes < gdn_layer_tree_workspace_size(L->H_k, L->H_v, N, T)) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  const gdn_inputs in = layer_mixer_inputs(L, static_cast<const bf16*>(workspace), layer_ld_proj(L->H_k, L->H_v));
  return gdn_decode_tree_commit(&in, N, T, parent, accepted, state, state, conv_state, conv_state, state_slot,
                                state_slot ? n_slots : N, err, stream);
}

gdn_status gdn_qk_norm_rope(const gdn_rope* rope, long long n_tok, int H_q, int H_kv, const void* q, long long ld_q,
                            const void* k, long long ld_k, const void* v, long long ld_v, const void* q_norm_w,
                            const void* k_norm_w, const int* positions, const long long* rows, long long n_rows,
                            void* q_out, long long ld_qo, void* k_out, long long ld_ko, void* v_out, long long ld_vo,
                            int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_qk_norm_rope");
  if (!rope || n_tok < 0 || H_q < 0 || H_kv < 0 || n_rows < 0) return GDN_ERR_INVALID_ARG;
  const int D = rope->head_dim, R = rope->rotary_dim;
  if (D < 8 || D > GDN_ROPE_MAX_HEAD_DIM || D % 8 != 0 || R < 0 || R > D || R % 16 != 0 ||
      (rope->layout != GDN_ROPE_HALF && rope->layout != GDN_ROPE_INTERLEAVED))
    return GDN_ERR_INVALID_ARG;  // not a struct gdn_rope_init has filled
  if (n_tok > INT_MAX) return GDN_ERR_UNSUPPORTED;
  const long long wq = static_cast<long long>(H_q) * D, wk = static_cast<long long>(H_kv) * D;
  if (wq + 2 * wk > INT_MAX) return GDN_ERR_UNSUPPORTED;
  if (n_tok == 0 || (H_q == 0 && H_kv == 0)) return GDN_OK;
  if (H_q > 0 && (!q || !q_out || ld_q < wq || ld_qo < wq)) return GDN_ERR_INVALID_ARG;
  if (H_kv > 0 && (!k || !k_out || ld_k < wk || ld_ko < wk)) return GDN_ERR_INVALID_ARG;
  if ((v == nullptr) != (v_out == nullptr) || (v && (H_kv == 0 || ld_v < wk || ld_vo < wk))) return GDN_ERR_INVALID_ARG;
  if (H_kv > 0 && !rows && n_rows < n_tok) return GDN_ERR_INVALID_ARG;
  long long lds = 0;
  if (H_q > 0) lds |= ld_q | ld_qo;
  if (H_kv > 0) lds |= ld_k | ld_ko;
  if (v) lds |= ld_v | ld_vo;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(v_out) ||
      !aligned16(q_norm_w) || !aligned16(k_norm_w) || !aligned4(positions) || (reinterpret_cast<uintptr_t>(rows) & 7u) ||
      (lds & 7))
    return GDN_ERR_MISALIGNED;
  // what is written may meet nothing that is read or written beside it, but for the two in-place forms
  struct Buf {
    const void* p;
    size_t bytes;
  };
  const Buf written[3] = {{H_q > 0 ? q_out : nullptr, extent(n_tok, ld_qo, wq)},
                          {H_kv > 0 ? k_out : nullptr, extent(n_rows, ld_ko, wk)},
                          {v_out, extent(n_rows, ld_vo, wk)}};
  const Buf read[7] = {{H_q > 0 ? q : nullptr, extent(n_tok, ld_q, wq)},
                       {H_kv > 0 ? k : nullptr, extent(n_tok, ld_k, wk)},
                       {v, extent(n_tok, ld_v, wk)},
                       {q_norm_w, static_cast<size_t>(D) * 2},
                       {k_norm_w, static_cast<size_t>(D) * 2},
                       {positions, sizeof(int) * static_cast<size_t>(n_tok)},
                       {rows, sizeof(long long) * static_cast<size_t>(n_tok)}};
  // rows of one strided buffer (columns of a projection) interleave with their neighbours' without sharing an element
  auto apart = [&](const void* a, long long lda, long long wa, const void* b, long long ldb, long long wb) {
    if (lda != ldb) return false;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    const uintptr_t lo = pa < pb ? pa : pb, hi = pa < pb ? pb : pa;
    const uintptr_t w_lo = static_cast<uintptr_t>(pa < pb ? wa : wb) * 2, w_hi = static_cast<uintptr_t>(pa < pb ? wb : wa) * 2;
    const uintptr_t row = static_cast<uintptr_t>(lda) * 2, d = (hi - lo) % row;
    return d >= w_lo && d + w_hi <= row;
  };
  const long long w_ld[3] = {ld_qo, ld_ko, ld_vo}, w_w[3] = {wq, wk, wk}, r_ld[3] = {ld_q, ld_k, ld_v}, r_w[3] = {wq, wk, wk};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 7; ++j) {
      if (!overlap(written[i].p, written[i].bytes, read[j].p, read[j].bytes)) continue;
      const bool in_place = i == j && i < 2 && written[i].p == read[j].p && w_ld[i] == r_ld[j] && (i == 0 || !rows);
      if (in_place || (j < 3 && apart(written[i].p, w_ld[i], w_w[i], read[j].p, r_ld[j], r_w[j]))) continue;
      return GDN_ERR_ALIAS;
    }
    for (int j = i + 1; j < 3; ++j)
      if (overlap(written[i].p, written[i].bytes, written[j].p, written[j].bytes) &&
          !apart(written[i].p, w_ld[i], w_w[i], written[j].p, w_ld[j], w_w[j]))
        return GDN_ERR_ALIAS;
  }
  RopeParams p = {};
  p.q = static_cast<const bf16*>(q);
  p.k = static_cast<const bf16*>(k);
  p.v = static_cast<const bf16*>(v);
  p.ld_q = ld_q; p.ld_k = ld_k; p.ld_v = ld_v;
  p.q_norm_w = static_cast<const bf16*>(q_norm_w);
  p.k_norm_w = static_cast<const bf16*>(k_norm_w);
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.n_tok = n_tok;
  p.positions = positions;
  p.rows = rows;
  p.n_rows = n_rows;
  p.q_out = static_cast<bf16*>(q_out);
  p.k_out = static_cast<bf16*>(k_out);
  p.v_out = static_cast<bf16*>(v_out);
  p.ld_qo = ld_qo; p.ld_ko = ld_ko; p.ld_vo = ld_vo;
  p.err = err;
  return launch_qk_norm_rope(*rope, p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_attention_tree_workspace_size(int H_q, int H_kv, int head_dim, int N, int T) {
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || H_q / H_kv > 16 || (head_dim != 128 && head_dim != 256) || N < 0 ||
      T < 1 || T > GDN_MAX_TREE_NODES)
    return 0;
  return attention_tree_workspace(H_q, H_kv, head_dim, N, T);
}

gdn_status gdn_attention_tree(const void* q_hat, long long ld_q, const void* k_tree, long long ld_kt,
                              const void* v_tree, long long ld_vt, const void* k_cache, const void* v_cache,
                              int cache_cap, const int* cache_len, const int* parent, const void* g, long long ld_g,
                              int H_q, int H_kv, int head_dim, float scale, int N, int T, void* out, void* workspace,
                              size_t workspace_bytes, int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_attention_tree");
  gdn_status st = check_tree_counts(N, T);
  if (st != GDN_OK) return st;
  if (H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || cache_cap < 1 || !(scale > 0.f) || !isfinite(scale))
    return GDN_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || H_q / H_kv > 16 || H_kv > 4096) return GDN_ERR_UNSUPPORTED;
  // a sequence's cache is one dimension of a TMA tensor map: its stride stays below 2^40 bytes
  if (2LL * H_kv * head_dim * cache_cap >= (1LL << 40) || (ld_kt | ld_vt) >= (1LL << 32)) return GDN_ERR_UNSUPPORTED;
  if (N == 0) return GDN_OK;
  const long long T_tot = static_cast<long long>(N) * T;
  const long long wq = static_cast<long long>(H_q) * head_dim, wk = static_cast<long long>(H_kv) * head_dim;
  if (!q_hat || !k_tree || !v_tree || !cache_len || !out) return GDN_ERR_INVALID_ARG;
  if (ld_q < wq || ld_kt < wk || ld_vt < wk || (g && ld_g < wq)) return GDN_ERR_INVALID_ARG;
  const size_t kv_bytes = static_cast<size_t>(N) * cache_cap * wk * 2;
  if (!k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
  if (!aligned16(q_hat) || !aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(g) || !aligned16(out) || !aligned16(workspace) || !aligned4(cache_len) || !aligned4(parent) ||
      ((ld_q | ld_kt | ld_vt | (g ? ld_g : 0)) & 7))
    return GDN_ERR_MISALIGNED;
  const size_t need = attention_tree_workspace(H_q, H_kv, head_dim, N, T);
  if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  const size_t ob = static_cast<size_t>(T_tot) * wq * 2;
  struct Buf {
    const void* p;
    size_t bytes;
  };
  const Buf read[8] = {{q_hat, extent(T_tot, ld_q, wq)},   {k_tree, extent(T_tot, ld_kt, wk)}, {v_tree, extent(T_tot, ld_vt, wk)},
                       {k_cache, kv_bytes},                {v_cache, kv_bytes},                {g, extent(T_tot, ld_g, wq)},
                       {cache_len, sizeof(int) * static_cast<size_t>(N)}, {parent, sizeof(int) * static_cast<size_t>(T_tot)}};
  for (const Buf& b : read)
    if (overlap(out, ob, b.p, b.bytes) || overlap(workspace, need, b.p, b.bytes)) return GDN_ERR_ALIAS;
  if (overlap(out, ob, workspace, need)) return GDN_ERR_ALIAS;
  AttnTreeParams p = {};
  p.q = static_cast<const bf16*>(q_hat);
  p.ld_q = ld_q;
  p.k_tree = static_cast<const bf16*>(k_tree);
  p.v_tree = static_cast<const bf16*>(v_tree);
  p.ld_kt = ld_kt;
  p.ld_vt = ld_vt;
  p.k_cache = static_cast<const bf16*>(k_cache);
  p.v_cache = static_cast<const bf16*>(v_cache);
  p.cap = cache_cap;
  p.cache_len = cache_len;
  p.parent = parent;
  p.g = static_cast<const bf16*>(g);
  p.ld_g = ld_g;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.D = head_dim;
  p.N = N;
  p.T = T;
  p.scale = scale;
  p.out = static_cast<bf16*>(out);
  p.workspace = workspace;
  p.err = err;
  return launch_attention_tree(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_attn_tree_commit(const void* k_tree, long long ld_kt, const void* v_tree, long long ld_vt, int H_kv,
                                int head_dim, int N, int T, const int* parent, const int* accepted, void* k_cache,
                                void* v_cache, int cache_cap, const int* cache_len, int* cache_len_out, int* err,
                                void* stream) {
  const NvtxRange nvtx_range("gdn_attn_tree_commit");
  gdn_status st = check_tree_counts(N, T);
  if (st != GDN_OK) return st;
  if (H_kv <= 0 || cache_cap < 1) return GDN_ERR_INVALID_ARG;
  if ((head_dim != 128 && head_dim != 256) || H_kv > 4096) return GDN_ERR_UNSUPPORTED;
  if (N == 0) return GDN_OK;
  const long long T_tot = static_cast<long long>(N) * T, wk = static_cast<long long>(H_kv) * head_dim;
  if (!k_tree || !v_tree || !accepted || !cache_len || !cache_len_out || ld_kt < wk || ld_vt < wk)
    return GDN_ERR_INVALID_ARG;
  const size_t kv_bytes = static_cast<size_t>(N) * cache_cap * wk * 2;
  if ((st = check_cache(k_cache, v_cache, kv_bytes)) != GDN_OK) return st;
  if (!aligned16(k_tree) || !aligned16(v_tree) || ((ld_kt | ld_vt) & 7) || !aligned4(parent) || !aligned4(accepted) ||
      !aligned4(cache_len) || !aligned4(cache_len_out))
    return GDN_ERR_MISALIGNED;
  const size_t nb = sizeof(int) * static_cast<size_t>(N), tb = sizeof(int) * static_cast<size_t>(T_tot);
  struct Buf {
    const void* p;
    size_t bytes;
  };
  const Buf read[4] = {{k_tree, extent(T_tot, ld_kt, wk)}, {v_tree, extent(T_tot, ld_vt, wk)}, {parent, tb}, {accepted, nb}};
  const Buf written[3] = {{k_cache, kv_bytes}, {v_cache, kv_bytes}, {cache_len_out, nb}};
  for (const Buf& w : written)
    for (const Buf& r : read)
      if (overlap(w.p, w.bytes, r.p, r.bytes)) return GDN_ERR_ALIAS;
  if (overlap(cache_len_out, nb, k_cache, kv_bytes) || overlap(cache_len_out, nb, v_cache, kv_bytes) ||
      overlap(cache_len, nb, k_cache, kv_bytes) || overlap(cache_len, nb, v_cache, kv_bytes) ||
      (cache_len != cache_len_out && overlap(cache_len, nb, cache_len_out, nb)))
    return GDN_ERR_ALIAS;
  AttnCommitParams p = {};
  p.k_tree = static_cast<const bf16*>(k_tree);
  p.v_tree = static_cast<const bf16*>(v_tree);
  p.ld_kt = ld_kt;
  p.ld_vt = ld_vt;
  p.H_kv = H_kv;
  p.D = head_dim;
  p.N = N;
  p.T = T;
  p.parent = parent;
  p.accepted = accepted;
  p.k_cache = static_cast<bf16*>(k_cache);
  p.v_cache = static_cast<bf16*>(v_cache);
  p.cap = cache_cap;
  p.cache_len = cache_len;
  p.cache_len_out = cache_len_out;
  p.err = err;
  return launch_attn_tree_commit(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_attn_layer_tree_workspace_size(int N, int T) {
  if (N < 0 || T < 1 || T > GDN_MAX_TREE_NODES) return 0;
  return attn_tree_layout(N, T).end;
}

gdn_status gdn_attn_layer_decode_tree(const gdn_attn_layer* L, int N, int T, const int* parent, const void* x,
                                      long long ldx, const void* k_cache, const void* v_cache, int cache_cap,
                                      const int* cache_len, void* y, long long ldy, void* workspace,
                                      size_t workspace_bytes, int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_attn_layer_decode_tree");
  if (!L || L->hidden <= 0 || cache_cap < 1) return GDN_ERR_INVALID_ARG;
  if (L->hidden % 64 != 0) return GDN_ERR_UNSUPPORTED;
  gdn_status s = check_tree_counts(N, T);
  if (s != GDN_OK || N == 0) return s;
  if (!x || !y || !cache_len || !L->w_in || !L->w_out || !L->q_norm_w || !L->k_norm_w) return GDN_ERR_INVALID_ARG;
  const long long T_tot = static_cast<long long>(N) * T;
  const AttnTreeLayout ws = attn_tree_layout(N, T);
  if (!workspace || workspace_bytes < ws.end) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace) || !aligned16(L->q_norm_w) || !aligned16(L->k_norm_w) || !aligned4(cache_len) || !aligned4(parent))
    return GDN_ERR_MISALIGNED;
  const size_t kv_bytes = static_cast<size_t>(N) * cache_cap * kAttnKv * 2;
  if (!k_cache || !v_cache) return GDN_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return GDN_ERR_MISALIGNED;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  bf16* proj = reinterpret_cast<bf16*>(w);
  bf16* q_hat = reinterpret_cast<bf16*>(w + ws.q_hat);
  bf16* k_tree = reinterpret_cast<bf16*>(w + ws.k_tree);
  bf16* att = reinterpret_cast<bf16*>(w + ws.att);
  if ((s = check_gemm(x, ldx, L->w_in, L->ld_w_in, proj, GDN_ATTN_N_IN, T_tot, GDN_ATTN_N_IN, L->hidden)) != GDN_OK) return s;
  if ((s = check_gemm(att, kAttnQ, L->w_out, L->ld_w_out, y, ldy, T_tot, L->hidden, kAttnQ)) != GDN_OK) return s;
  const size_t yb = extent(T_tot, ldy, L->hidden), nb = sizeof(int) * static_cast<size_t>(N);
  const size_t tb = sizeof(int) * static_cast<size_t>(T_tot);
  if (overlap(y, yb, w, ws.end) || overlap(x, extent(T_tot, ldx, L->hidden), w, ws.end) || overlap(k_cache, kv_bytes, w, ws.end) ||
      overlap(v_cache, kv_bytes, w, ws.end) || overlap(y, yb, k_cache, kv_bytes) || overlap(y, yb, v_cache, kv_bytes) ||
      overlap(cache_len, nb, w, ws.end) || overlap(parent, tb, w, ws.end) || overlap(cache_len, nb, y, yb) ||
      overlap(parent, tb, y, yb))
    return GDN_ERR_ALIAS;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto mark = [&](int i) {
    if (L->events) cudaEventRecord(static_cast<cudaEvent_t>(L->events[i]), st);
  };
  mark(0);
  s = gdn_gemm_bf16(x, ldx, L->w_in, L->ld_w_in, proj, GDN_ATTN_N_IN, static_cast<int>(T_tot), GDN_ATTN_N_IN, L->hidden,
                    err, stream);
  if (s != GDN_OK) return s;
  mark(1);
  RopeParams rp = {};
  rp.q = proj;
  rp.k = proj + 2 * kAttnQ;
  rp.ld_q = rp.ld_k = GDN_ATTN_N_IN;
  rp.q_norm_w = static_cast<const bf16*>(L->q_norm_w);
  rp.k_norm_w = static_cast<const bf16*>(L->k_norm_w);
  rp.H_q = GDN_ATTN_Q_HEADS;
  rp.H_kv = GDN_ATTN_KV_HEADS;
  rp.n_tok = rp.n_rows = T_tot;
  rp.tree_T = T;
  rp.parent = parent;
  rp.base = cache_len;
  rp.q_out = q_hat;
  rp.k_out = k_tree;
  rp.ld_qo = kAttnQ;
  rp.ld_ko = kAttnKv;
  rp.err = err;
  if (launch_qk_norm_rope(attn_layer_rope(), rp, st) != cudaSuccess) return GDN_ERR_CUDA;
  s = gdn_attention_tree(q_hat, kAttnQ, k_tree, kAttnKv, proj + 2 * kAttnQ + kAttnKv, GDN_ATTN_N_IN, k_cache, v_cache,
                         cache_cap, cache_len, parent, proj + kAttnQ, GDN_ATTN_N_IN, GDN_ATTN_Q_HEADS, GDN_ATTN_KV_HEADS,
                         GDN_ATTN_HEAD_DIM, 0.0625f, N, T, att, w + ws.scratch, ws.end - ws.scratch, err, stream);
  if (s != GDN_OK) return s;
  mark(2);
  s = gdn_gemm_bf16(att, kAttnQ, L->w_out, L->ld_w_out, y, ldy, static_cast<int>(T_tot), L->hidden,
                    static_cast<int>(kAttnQ), err, stream);
  if (s != GDN_OK) return s;
  mark(3);
  return GDN_OK;
}

gdn_status gdn_attn_layer_tree_commit(int N, int T, const int* parent, const int* accepted, void* k_cache,
                                      void* v_cache, int cache_cap, int* cache_len, const void* workspace,
                                      size_t workspace_bytes, int* err, void* stream) {
  const NvtxRange nvtx_range("gdn_attn_layer_tree_commit");
  const gdn_status s = check_tree_counts(N, T);
  if (s != GDN_OK || N == 0) return s;
  const AttnTreeLayout ws = attn_tree_layout(N, T);
  if (!workspace || workspace_bytes < ws.end) return GDN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return GDN_ERR_MISALIGNED;
  const uint8_t* w = static_cast<const uint8_t*>(workspace);
  return gdn_attn_tree_commit(w + ws.k_tree, kAttnKv, reinterpret_cast<const bf16*>(w) + 2 * kAttnQ + kAttnKv,
                              GDN_ATTN_N_IN, GDN_ATTN_KV_HEADS, GDN_ATTN_HEAD_DIM, N, T, parent, accepted, k_cache, v_cache,
                              cache_cap, cache_len, cache_len, err, stream);
}

}  // extern "C"
