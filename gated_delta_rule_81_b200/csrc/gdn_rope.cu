// gdn_qk_norm_rope: RMS norm of each head of q and k, rotary positions, and the placement of k
// and v into cache rows, in one pass.
//
// Per head x of D dims: y = x / sqrt(mean x^2 + eps) * w, then pair i of the first R dims turns by
// the angle position * theta_i: (y1, y2) -> (y1 c - y2 s, y2 c + y1 s).
//
// Angles: the table holds theta_i / 2 pi in units of 2^-64 turns, and position * turns[i] in 64-bit
// integers wraps modulo one turn by itself, so the reduction is exact at any position; the top 32
// bits go to sincospif.  The rest is fp32 with one rounding to bf16.
#include <cmath>

#include "gdn_tree.cuh"

namespace gdn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTok = 4;   // tokens per CTA at most
constexpr int kRopeItems = 4; // heads whose loads a lane group has in flight

__device__ __forceinline__ void unpack8(uint4 u, float* f) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}

// A group of W lanes (8, 16 or 32: the power of two that holds D / 8) takes a head, lane l its dims 8l .. 8l + 7
// (one 16-byte load).  A CTA takes `tok` tokens: its threads first form the tokens' cosines and sines in
// shared memory, R / 2 per token shared by all heads; then the groups walk the heads, kRopeItems at a time.
template <int W, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const __grid_constant__ gdn_rope rope, RopeParams p, int tok) {
  __shared__ float2 cs_s[kRopeTok][GDN_ROPE_MAX_HEAD_DIM / 2];
  __shared__ int tree_s[kRopeTok][kMaxNodes];
  const int tid = threadIdx.x;
  const int D = rope.head_dim, R = rope.rotary_dim, half = R / 2;
  const long long t0 = static_cast<long long>(blockIdx.x) * tok;
  const int n_here = static_cast<int>(min(static_cast<long long>(tok), p.n_tok - t0));
  if (p.tree_T > 0) {  // the parents of each token's sequence, for the walk to its root
    for (int x = tid; x < n_here * p.tree_T; x += kRopeThreads) {
      const int i = x / p.tree_T, j = x % p.tree_T;
      tree_s[i][j] = p.parent ? p.parent[(t0 + i) / p.tree_T * p.tree_T + j] : j - 1;
    }
    __syncthreads();
  }
  for (int x = tid; x < n_here * half; x += kRopeThreads) {
    const int i = x / half, f = x % half;
    long long pos = t0 + i;
    if (p.tree_T > 0) {
      const int j = static_cast<int>(pos % p.tree_T);
      pos = p.base[pos / p.tree_T];
      // one step per ancestor; a parent that is no earlier node ends the walk
      for (int node = j, up = tree_s[i][j]; up >= 0 && up < node; node = up, up = tree_s[i][up]) ++pos;
    } else if (p.positions) {
      pos = p.positions[pos];
    }
    const unsigned long long turn = static_cast<unsigned long long>(pos) * rope.turns[f];
    float sn, cn;
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: in half turns
    cs_s[i][f] = make_float2(cn * rope.amplitude, sn * rope.amplitude);
  }
  __syncthreads();

  constexpr int kGroups = kRopeThreads / W;
  const int grp = tid / W, l = tid % W;
  const bool on = 8 * l < D;
  const bool turned = 8 * l < R;
  const int H = p.H_q + p.H_kv + (p.v ? p.H_kv : 0);
  float wq[8], wk[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) wq[e] = wk[e] = 1.f;
  if (on && p.q_norm_w) unpack8(reinterpret_cast<const uint4*>(p.q_norm_w)[l], wq);
  if (on && p.k_norm_w) unpack8(reinterpret_cast<const uint4*>(p.k_norm_w)[l], wk);
  const float inv_D = 1.0f / static_cast<float>(D);
  // half layout: lanes 0 .. R/16 - 1 hold the first of each pair, the next R/16 lanes the second
  const bool first = l < R / 16;
  const int partner = !turned ? l : first ? l + R / 16 : l - R / 16;

  for (int i = 0; i < n_here; ++i) {
    const long long t = t0 + i;
    float c8[8], s8[8];  // per dim (half) or the first four per pair (interleaved)
    if (turned) {
      const float4* src = reinterpret_cast<const float4*>(&cs_s[i][kInterleaved ? 4 * l : 8 * (first ? l : l - R / 16)]);
#pragma unroll
      for (int e = 0; e < (kInterleaved ? 2 : 4); ++e) {
        const float4 x = src[e];
        c8[2 * e] = x.x; s8[2 * e] = x.y; c8[2 * e + 1] = x.z; s8[2 * e + 1] = x.w;
      }
    }
    long long row = p.rows ? p.rows[t] : t;
    if (row >= p.n_rows) {
      if (tid == 0 && p.H_kv > 0 && p.err) atomicOr(p.err, kDevErrBadIndex);
      row = -1;
    }
    for (int h0 = 0; h0 < H; h0 += kRopeItems * kGroups) {
      uint4 raw[kRopeItems];
#pragma unroll
      for (int u = 0; u < kRopeItems; ++u) {
        const int h = h0 + u * kGroups + grp;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (on && h < H) {
          const bf16* src = h < p.H_q            ? p.q + t * p.ld_q + static_cast<long long>(h) * D
                            : h < p.H_q + p.H_kv ? p.k + t * p.ld_k + static_cast<long long>(h - p.H_q) * D
                                                 : p.v + t * p.ld_v + static_cast<long long>(h - p.H_q - p.H_kv) * D;
          raw[u] = reinterpret_cast<const uint4*>(src)[l];
        }
      }
#pragma unroll
      for (int u = 0; u < kRopeItems; ++u) {
        if (h0 + u * kGroups >= H) break;  // the same for the whole CTA
        const int h = h0 + u * kGroups + grp;
        const bool is_q = h < p.H_q, is_v = h >= p.H_q + p.H_kv;
        float x[8];
        unpack8(raw[u], x);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const bool norm = is_q ? p.q_norm_w != nullptr : p.k_norm_w != nullptr;
        const float inv = norm ? rsqrtf(fmaf(ss, inv_D, rope.eps)) : 1.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * (is_q ? wq[e] : wk[e]);
        if (kInterleaved) {
          if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = x[2 * e], b = x[2 * e + 1];
              x[2 * e] = fmaf(a, c8[e], -(b * s8[e]));
              x[2 * e + 1] = fmaf(b, c8[e], a * s8[e]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float other = __shfl_sync(0xffffffffu, x[e], partner, W);
            if (turned) x[e] = first ? fmaf(x[e], c8[e], -(other * s8[e])) : fmaf(x[e], c8[e], other * s8[e]);
          }
        }
        if (!on || h >= H || (!is_q && row < 0)) continue;
        if (is_v) {
          reinterpret_cast<uint4*>(p.v_out + row * p.ld_vo + static_cast<long long>(h - p.H_q - p.H_kv) * D)[l] = raw[u];
        } else {
          bf16* dst = is_q ? p.q_out + t * p.ld_qo + static_cast<long long>(h) * D
                           : p.k_out + row * p.ld_ko + static_cast<long long>(h - p.H_q) * D;
          reinterpret_cast<uint4*>(dst)[l] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                        pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        }
      }
    }
  }
}

template <int W>
void rope_launch(const gdn_rope& rope, const RopeParams& p, int tok, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((p.n_tok + tok - 1) / tok);
  if (rope.layout == GDN_ROPE_INTERLEAVED)
    qk_norm_rope_kernel<W, true><<<grid, kRopeThreads, 0, stream>>>(rope, p, tok);
  else
    qk_norm_rope_kernel<W, false><<<grid, kRopeThreads, 0, stream>>>(rope, p, tok);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const gdn_rope& rope, const RopeParams& p, cudaStream_t stream) {
  if (p.n_tok == 0 || p.H_q + p.H_kv == 0) return cudaSuccess;
  // several tokens per CTA share its set-up once there are CTAs enough for all SMs either way
  const int tok = p.n_tok >= 4096 ? 4 : p.n_tok >= 1024 ? 2 : 1;
  if (rope.head_dim <= 64) rope_launch<8>(rope, p, tok, stream);
  else if (rope.head_dim <= 128) rope_launch<16>(rope, p, tok, stream);
  else rope_launch<32>(rope, p, tok, stream);
  return cudaGetLastError();
}

}  // namespace gdn

extern "C" gdn_status gdn_rope_init(gdn_rope* rope, int head_dim, int rotary_dim, int layout, int scaling, double base,
                                    double factor, int original_len, double beta_fast, double beta_slow, float eps) {
  if (!rope || head_dim <= 0 || rotary_dim < 0 || rotary_dim > head_dim) return GDN_ERR_INVALID_ARG;
  if (layout != GDN_ROPE_HALF && layout != GDN_ROPE_INTERLEAVED) return GDN_ERR_INVALID_ARG;
  if (scaling < GDN_ROPE_NONE || scaling > GDN_ROPE_YARN) return GDN_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base) || !(factor >= 1.0) || !std::isfinite(factor) || !(eps >= 0.f) ||
      !std::isfinite(eps))
    return GDN_ERR_INVALID_ARG;
  if (scaling == GDN_ROPE_YARN && (original_len < 1 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast)))
    return GDN_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > GDN_ROPE_MAX_HEAD_DIM || rotary_dim % 16 != 0) return GDN_ERR_UNSUPPORTED;
  const long double kTwoPi = 6.283185307179586476925286766559005768L;
  const int half = rotary_dim / 2;
  long double b = base;
  if (scaling == GDN_ROPE_NTK && rotary_dim > 0) b *= powl(factor, static_cast<long double>(rotary_dim) / (rotary_dim - 2));
  double lo = 0, hi = 0;
  if (scaling == GDN_ROPE_YARN && half > 0) {
    // the (fractional) pair that turns `beta` times within original_len positions
    auto pair = [&](double beta) {
      return rotary_dim * std::log(original_len / (beta * static_cast<double>(kTwoPi))) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair(beta_slow)), half - 1.0);
  }
  *rope = gdn_rope{};
  rope->head_dim = head_dim;
  rope->rotary_dim = rotary_dim;
  rope->layout = layout;
  rope->eps = eps;
  rope->amplitude = scaling == GDN_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  for (int i = 0; i < half; ++i) {
    long double theta = powl(b, -static_cast<long double>(i) / half);
    if (scaling == GDN_ROPE_LINEAR) theta /= factor;
    if (scaling == GDN_ROPE_YARN) {
      const long double ramp = std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0);
      theta = theta * (1 - ramp) + theta / factor * ramp;
    }
    rope->turns[i] = static_cast<unsigned long long>(roundl(ldexpl(theta / kTwoPi, 64)));
  }
  return GDN_OK;
}
