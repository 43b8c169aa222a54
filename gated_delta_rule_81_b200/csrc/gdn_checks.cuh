// Host-side argument checks and buffer layouts shared by the C ABI's entry points.
#pragma once

#include <stdint.h>
#include <stdlib.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/gdn.h"
#include "gdn_kernels.cuh"

namespace gdn {

// NVTX ranges named after the entry points, when GDN_NVTX is set (to anything but 0) in the
// environment; read once.  NVTX3 is header-only and loads nothing unless a profiler injects it.
inline bool nvtx_on() {
  static const bool on = [] {
    const char* e = getenv("GDN_NVTX");
    return e && *e && !(e[0] == '0' && e[1] == 0);
  }();
  return on;
}

struct NvtxRange {
  bool on;
  explicit NvtxRange(const char* name) : on(nvtx_on()) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxRange() {
    if (on) nvtxRangePop();
  }
};

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

inline size_t round_up(size_t x, size_t m) { return (x + m - 1) / m * m; }

// leading dimension of the layer's projection buffer: n_in rounded up to 8 (16-byte rows)
inline long long layer_ld_proj(int H_k, int H_v) {
  return (2LL * H_k * GDN_HEAD_DIM + 2LL * H_v * GDN_HEAD_DIM + 2LL * H_v + 7) / 8 * 8;
}

// chunk_base[N+1] and seq_order[N] (ints) after the 1 KiB header
inline size_t chunk_base_bytes(int N) { return round_up(sizeof(int) * (2 * static_cast<size_t>(N) + 1), 1024); }

// Common checks of the per-token inputs; T_tot tokens.
inline gdn_status check_inputs(const gdn_inputs* in, long long T_tot) {
  if (!in) return GDN_ERR_INVALID_ARG;
  if (in->H_k <= 0 || in->H_v <= 0 || in->H_v % in->H_k != 0) return GDN_ERR_INVALID_ARG;
  if (in->H_v / in->H_k > 8) return GDN_ERR_UNSUPPORTED;
  if (T_tot == 0) return GDN_OK;
  if (!in->q || !in->k || !in->v || !in->a || !in->b || !in->z || !in->conv_w || !in->A_log || !in->norm_w)
    return GDN_ERR_INVALID_ARG;
  const long long qk = static_cast<long long>(in->H_k) * GDN_HEAD_DIM, vz = static_cast<long long>(in->H_v) * GDN_HEAD_DIM;
  if (in->stride_q < qk || in->stride_k < qk || in->stride_v < vz || in->stride_z < vz || in->stride_a < in->H_v ||
      in->stride_b < in->H_v)
    return GDN_ERR_INVALID_ARG;
  if (!aligned16(in->q) || !aligned16(in->k) || !aligned16(in->v) || !aligned16(in->z) || !aligned16(in->conv_w))
    return GDN_ERR_MISALIGNED;
  if ((in->stride_q | in->stride_k | in->stride_v | in->stride_z) & 7) return GDN_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(in->a) | reinterpret_cast<uintptr_t>(in->b) |
       reinterpret_cast<uintptr_t>(in->norm_w)) & 1u)
    return GDN_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(in->A_log) & 3u) return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

// `out` must not overlap any input read by the same call
// bytes from the first element of a [T_tot] x stride input to the end of its last row's `width` channels
inline size_t input_extent(long long T_tot, long long stride, long long width) {
  return sizeof(bf16) * (static_cast<size_t>(T_tot - 1) * static_cast<size_t>(stride) + static_cast<size_t>(width));
}

inline gdn_status check_out_alias(const gdn_inputs* in, long long T_tot, const void* out) {
  const size_t ob = static_cast<size_t>(T_tot) * in->H_v * GDN_HEAD_DIM * sizeof(bf16);
  const long long qk = static_cast<long long>(in->H_k) * GDN_HEAD_DIM, vz = static_cast<long long>(in->H_v) * GDN_HEAD_DIM;
  if (overlap(out, ob, in->q, input_extent(T_tot, in->stride_q, qk)) ||
      overlap(out, ob, in->k, input_extent(T_tot, in->stride_k, qk)) ||
      overlap(out, ob, in->v, input_extent(T_tot, in->stride_v, vz)) ||
      overlap(out, ob, in->z, input_extent(T_tot, in->stride_z, vz)) ||
      overlap(out, ob, in->a, input_extent(T_tot, in->stride_a, in->H_v)) ||
      overlap(out, ob, in->b, input_extent(T_tot, in->stride_b, in->H_v)))
    return GDN_ERR_ALIAS;
  return GDN_OK;
}

// The mixer's inputs as columns of the layer's projection buffer [T_tot][ld_p]:
// q | k | v | z | a | b, read through the row stride ld_p (no copy).
inline gdn_inputs layer_mixer_inputs(const gdn_layer* L, const bf16* proj, long long ld_p) {
  const long long HkD = static_cast<long long>(L->H_k) * GDN_HEAD_DIM;
  const long long d_v = static_cast<long long>(L->H_v) * GDN_HEAD_DIM;
  gdn_inputs in = {};
  in.q = proj;
  in.k = proj + HkD;
  in.v = proj + 2 * HkD;
  in.z = proj + 2 * HkD + d_v;
  in.a = proj + 2 * HkD + 2 * d_v;
  in.b = proj + 2 * HkD + 2 * d_v + L->H_v;
  in.stride_q = in.stride_k = in.stride_v = in.stride_z = in.stride_a = in.stride_b = ld_p;
  in.conv_w = L->conv_w;
  in.A_log = L->A_log;
  in.norm_w = L->norm_w;
  in.H_k = L->H_k;
  in.H_v = L->H_v;
  in.scale = L->scale;
  in.schedule = L->schedule;
  return in;
}

// The aliasing rule of every prefill entry point, in one place: among the state and conv
// buffers and the output (out_bytes of it; nullptr when the call has none), a buffer the call
// writes (state_out, conv_out, out) overlaps no other one, except that state_out may be
// exactly state_in (the state is updated in place, each row by the one CTA that reads it).
inline gdn_status check_state_aliases(int H_k, int H_v, int n, const float* state_in, const float* state_out,
                               const void* conv_in, const void* conv_out, const void* out, size_t out_bytes) {
  const size_t state_bytes = static_cast<size_t>(n) * H_v * GDN_HEAD_DIM * GDN_HEAD_DIM * sizeof(float);
  const size_t conv_bytes = static_cast<size_t>(n) * 3 * (2 * H_k + H_v) * GDN_HEAD_DIM * sizeof(bf16);
  struct Buf {
    const void* p;
    size_t bytes;
    bool written;
  };
  const Buf b[5] = {{state_in, state_bytes, false}, {state_out, state_bytes, true}, {conv_in, conv_bytes, false},
                    {conv_out, conv_bytes, true}, {out, out_bytes, true}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j) {
      if (!b[i].written && !b[j].written) continue;
      if (i == 0 && j == 1 && state_in == state_out) continue;
      if (overlap(b[i].p, b[i].bytes, b[j].p, b[j].bytes)) return GDN_ERR_ALIAS;
    }
  return GDN_OK;
}

// The layer entry points check the states the mixer will take before their first launch, so
// that a rejected call launches nothing: alignment, and the aliasing rules of the mixer calls.
inline gdn_status check_layer_states(int H_k, int H_v, int n, const float* state_in, const float* state_out,
                              const void* conv_in, const void* conv_out) {
  if (!aligned16(state_in) || !aligned16(state_out) || !aligned16(conv_in) || !aligned16(conv_out))
    return GDN_ERR_MISALIGNED;
  return check_state_aliases(H_k, H_v, n, state_in, state_out, conv_in, conv_out, nullptr, 0);
}

// None of the state and conv buffers of a layer call may lie in its workspace (the projection,
// the mixer output and the mixer's scratch are written there).
inline bool states_in_workspace(int H_k, int H_v, int n, const void* s0, const void* s1, const void* c0, const void* c1,
                         const void* ws, size_t ws_bytes) {
  const size_t state_bytes = static_cast<size_t>(n) * H_v * GDN_HEAD_DIM * GDN_HEAD_DIM * sizeof(float);
  const size_t conv_bytes = static_cast<size_t>(n) * 3 * (2 * H_k + H_v) * GDN_HEAD_DIM * sizeof(bf16);
  return overlap(s0, state_bytes, ws, ws_bytes) || overlap(s1, state_bytes, ws, ws_bytes) ||
         overlap(c0, conv_bytes, ws, ws_bytes) || overlap(c1, conv_bytes, ws, ws_bytes);
}

}  // namespace gdn
