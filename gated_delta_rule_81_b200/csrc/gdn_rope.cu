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
constexpr int kRopeFlight = 4;  // heads whose loads a lane group has in flight

__device__ __forceinline__ void unpack8(uint4 u, float2 (&f)[4]) {
  f[0] = make_float2(bf16_lo(u.x), bf16_hi(u.x));
  f[1] = make_float2(bf16_lo(u.y), bf16_hi(u.y));
  f[2] = make_float2(bf16_lo(u.z), bf16_hi(u.z));
  f[3] = make_float2(bf16_lo(u.w), bf16_hi(u.w));
}

// A group of W lanes (8, 16 or 32: the power of two that holds D / 8) takes `per` heads of one token, lane l their dims
// 8l .. 8l + 7 (one 16-byte load each).  Cosines, sines and norm weights stay in registers over the heads, so that a head
// costs little more than its own arithmetic in packed fp32: with them fetched per head, and q, k and v told apart per
// load, the kernel spent 180 instructions per 8 elements and was bound by issuing them (179 us for 32,768 tokens of 48 heads of
// 128; the bytes take 123 us); now 151 us, 5.3 TB/s, at 39% of the issue slots.  Few tokens are split into
// many items of few heads: items below `whole` are whole tokens, the others `per` heads of one, `splits` to a token.
template <int W, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4)
    qk_norm_rope_kernel(const __grid_constant__ gdn_rope rope, const __grid_constant__ RopeParams p, long long whole, int splits, int per) {
  constexpr int kGroups = kRopeThreads / W;
  __shared__ int tree_s[kGroups][kMaxNodes];
  // frequencies: from parameter memory lanes read one after the other, which a long call is spared (154 -> 151 us for 32,768 tokens)
  // and a short one would pay the barrier for (4.2 -> 4.5 us for 21)
  __shared__ unsigned long long turns_s[GDN_ROPE_MAX_HEAD_DIM / 2];
  if (whole > 0) {
    for (int i = threadIdx.x; i < rope.rotary_dim / 2; i += kRopeThreads) turns_s[i] = rope.turns[i];
    __syncthreads();
  }
  const int grp = threadIdx.x / W, l = threadIdx.x % W;
  const unsigned mask = W == 32 ? 0xffffffffu : ((1u << (W & 31)) - 1u) << ((threadIdx.x & 31) / W * W);
  const long long item = static_cast<long long>(blockIdx.x) * kGroups + grp;
  const long long t = item < whole ? item : whole + (item - whole) / splits;
  if (t >= p.n_tok) return;  // whole groups
  const int D = rope.head_dim, R = rope.rotary_dim;
  const bool on = 8 * l < D, turned = 8 * l < R;
  long long pos = t;
  if (p.tree_T > 0) {  // the walk to the node's root, through a copy of its sequence's parents
    const long long n = t / p.tree_T;
    const int node = static_cast<int>(t % p.tree_T);
    for (int j = l; j < p.tree_T; j += W) tree_s[grp][j] = p.parent ? p.parent[n * p.tree_T + j] : j - 1;
    pos = p.base[n];
    __syncwarp(mask);
    for (int at = node, up = tree_s[grp][at]; up >= 0 && up < at; at = up, up = tree_s[grp][at]) ++pos;
  } else if (p.positions) {
    pos = p.positions[t];
  }
  long long row = p.rows ? p.rows[t] : t;
  if (row >= p.n_rows) {
    if (l == 0 && p.H_kv > 0 && p.err) atomicOr(p.err, kDevErrBadIndex);
    row = -1;
  }

  // half layout: lanes 0 .. R/16 - 1 hold the first of each pair, the next R/16 lanes the second
  const bool first = l < R / 16;
  const int partner = !turned ? l : first ? l + R / 16 : l - R / 16;
  // factors of this lane's dims 2 e, 2 e + 1 and of the dims they are paired with
  float2 c2[4], s2[4];
  {
    // four frequencies per lane: its own pairs' (interleaved), or half of those it shares with its partner
    const int f0 = !turned ? 0 : kInterleaved ? 4 * l : first ? 8 * l : 8 * (l - R / 16) + 4;
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned long long turn = static_cast<unsigned long long>(pos) * (whole > 0 ? turns_s[f0 + i] : rope.turns[f0 + i]);
      sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &s[i], &c[i]);  // 2^-31: in half turns
      c[i] *= rope.amplitude;
      s[i] *= rope.amplitude;
    }
    if (kInterleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c2[e] = make_float2(c[e], c[e]);
        s2[e] = make_float2(-s[e], s[e]);
      }
    } else {
      const float sign = first ? -1.f : 1.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 cm = make_float2(c[2 * e], c[2 * e + 1]), sm = make_float2(s[2 * e], s[2 * e + 1]);
        const float2 co = make_float2(__shfl_sync(mask, cm.x, partner, W), __shfl_sync(mask, cm.y, partner, W));
        const float2 so = make_float2(__shfl_sync(mask, sm.x, partner, W), __shfl_sync(mask, sm.y, partner, W));
        c2[e] = first ? cm : co;
        c2[e + 2] = first ? co : cm;
        const float2 a = first ? sm : so, b = first ? so : sm;
        s2[e] = make_float2(sign * a.x, sign * a.y);
        s2[e + 2] = make_float2(sign * b.x, sign * b.y);
      }
    }
    if (!turned) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        c2[e] = make_float2(1.f, 1.f);
        s2[e] = make_float2(0.f, 0.f);
      }
    }
  }
  const float inv_D = 1.0f / static_cast<float>(D);

  // heads h0 .. h1 - 1 of src (and dst), normed by w and turned
  auto heads = [&](const bf16* src, bf16* dst, const bf16* w, int h0, int h1) {
    float2 w2[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w2[e] = make_float2(1.f, 1.f);
    if (w && on) unpack8(reinterpret_cast<const uint4*>(w)[l], w2);
    const uint4* s4 = reinterpret_cast<const uint4*>(src) + static_cast<long long>(h0) * (D / 8) + l;
    uint4* d4 = reinterpret_cast<uint4*>(dst) + static_cast<long long>(h0) * (D / 8) + l;
    for (int h = h0; h < h1; h += kRopeFlight, s4 += kRopeFlight * (D / 8), d4 += kRopeFlight * (D / 8)) {
      uint4 raw[kRopeFlight];
#pragma unroll
      for (int u = 0; u < kRopeFlight; ++u) {
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (on && h + u < h1) raw[u] = __ldcs(s4 + u * (D / 8));
      }
#pragma unroll
      for (int u = 0; u < kRopeFlight; ++u) {
        if (h + u >= h1) break;  // the same for the group
        float2 x[4];
        unpack8(raw[u], x);
        if (w) {
          float2 q = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e) q = __ffma2_rn(x[e], x[e], q);
          float ss = q.x + q.y;
#pragma unroll
          for (int o = W / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
          const float inv = rsqrtf(fmaf(ss, inv_D, rope.eps));
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = __fmul2_rn(__fmul2_rn(x[e], make_float2(inv, inv)), w2[e]);
        }
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 other = kInterleaved ? make_float2(x[e].y, x[e].x)
                                            : make_float2(__shfl_sync(mask, x[e].x, partner, W), __shfl_sync(mask, x[e].y, partner, W));
          y[e] = turned ? __ffma2_rn(x[e], c2[e], __fmul2_rn(other, s2[e])) : x[e];  // (0 times an infinity left out)
        }
        if (on)
          d4[u * (D / 8)] = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y), pack_bf16x2(y[2].x, y[2].y),
                                       pack_bf16x2(y[3].x, y[3].y));
      }
    }
  };
  // this item's heads among q | k | v
  const int k0 = p.H_q, v0 = p.H_q + p.H_kv, end = v0 + (p.v ? p.H_kv : 0);
  const int b = item < whole ? 0 : static_cast<int>((item - whole) % splits) * per, e = item < whole ? end : b + per;
  if (b < k0) heads(p.q + t * p.ld_q, p.q_out + t * p.ld_qo, p.q_norm_w, b, min(e, k0));
  if (row < 0) return;
  if (b < v0 && e > k0) heads(p.k + t * p.ld_k, p.k_out + row * p.ld_ko, p.k_norm_w, max(b, k0) - k0, min(e, v0) - k0);
  if (e > v0 && b < end) {
    const int h0 = max(b, v0) - v0, n16 = (min(e, end) - v0 - h0) * (D / 8);
    const uint4* src = reinterpret_cast<const uint4*>(p.v + t * p.ld_v) + static_cast<long long>(h0) * (D / 8);
    uint4* dst = reinterpret_cast<uint4*>(p.v_out + row * p.ld_vo) + static_cast<long long>(h0) * (D / 8);
#pragma unroll 4
    for (int x = l; x < n16; x += W) dst[x] = __ldcs(src + x);
  }
}

template <int W>
void rope_launch(const gdn_rope& rope, const RopeParams& p, cudaStream_t stream) {
  constexpr int kGroups = kRopeThreads / W;
  const int H = p.H_q + p.H_kv + (p.v ? p.H_kv : 0);
  // Tokens whole while they fill the GPU round by round; left over ones that fill no more than a third of a round are split into
  // items of so few heads, in rounds of kRopeFlight, that they take one short round.  An item forms its token's factors again, which
  // more of them would not gain back (20,000 tokens of 48 heads, 2.11 rounds: 94 us split, 105 whole; 16,384, 1.73 rounds: 95 and 78;
  // 32,768, 3.46 rounds: 152 and 151, and 190 with all tokens in halves).
  const long long want = 148LL * 4 * kGroups;  // groups resident at once
  long long whole = p.n_tok / want * want;
  if ((p.n_tok - whole) * 3 > want && whole > 0) whole = p.n_tok;
  const long long rest = p.n_tok - whole;
  long long per = (rest * H + want - 1) / want;
  per = (per + kRopeFlight - 1) / kRopeFlight * kRopeFlight;
  if (per > H) per = H;
  if (per < 1) per = 1;
  const int splits = static_cast<int>((H + per - 1) / per);
  const unsigned grid = static_cast<unsigned>((whole + rest * splits + kGroups - 1) / kGroups);
  if (rope.layout == GDN_ROPE_INTERLEAVED)
    qk_norm_rope_kernel<W, true><<<grid, kRopeThreads, 0, stream>>>(rope, p, whole, splits, static_cast<int>(per));
  else
    qk_norm_rope_kernel<W, false><<<grid, kRopeThreads, 0, stream>>>(rope, p, whole, splits, static_cast<int>(per));
}

}  // namespace

cudaError_t launch_qk_norm_rope(const gdn_rope& rope, const RopeParams& p, cudaStream_t stream) {
  if (p.n_tok == 0 || p.H_q + p.H_kv == 0) return cudaSuccess;
  if (rope.head_dim <= 64) rope_launch<8>(rope, p, stream);
  else if (rope.head_dim <= 128) rope_launch<16>(rope, p, stream);
  else rope_launch<32>(rope, p, stream);
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
    // the (fractional) pair that turns `beta` times within original_len positions; the one of beta_slow may lie beyond the last
    // pair, half - 1, and the ramp then does not reach 1
    auto pair = [&](double beta) {
      return rotary_dim * std::log(original_len / (beta * static_cast<double>(kTwoPi))) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(pair(beta_fast)), 0.0);
    hi = std::fmin(std::ceil(pair(beta_slow)), rotary_dim - 1.0);
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
