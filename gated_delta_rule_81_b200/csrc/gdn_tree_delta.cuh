// What the three kernels of gdn_decode_tree share (gdn_tree.cu up to 32 nodes, gdn_tree_small.cu up to 8 with several value heads
// per CTA, gdn_tree_wide.cu beyond 32).
#pragma once

#include "gdn_tree.cuh"

namespace gdn {

constexpr int kWorkers = 256;            // threads of warps 0-7
constexpr int kVRow = 132;               // floats of a node's v (then o): lanes (g, c) read bank 8 c + g

__device__ __forceinline__ void bar_arrive(int id, int n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// hi and lo words of two values
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - bf16_lo(hi), y - bf16_hi(hi));
}

// d += A B^T with A = ah + al and B's words b = (hi0, hi1, lo0, lo1)
__device__ __forceinline__ void mma_split(float (&d)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], const uint4& b) {
  mma_16816(d, ah, b.x, b.y);
  mma_16816(d, ah, b.z, b.w);
  mma_16816(d, al, b.x, b.y);
}

// conv weights of CH channels from their staged copy: w[i] holds the four taps of channel i
template <int CH>
__device__ __forceinline__ void load_taps(const uint8_t* staged, float4 (&w)[CH]) {
#pragma unroll
  for (int i = 0; i < CH / 2; ++i) {
    const uint4 u = reinterpret_cast<const uint4*>(staged)[i];
    w[2 * i] = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
    w[2 * i + 1] = make_float4(bf16_lo(u.z), bf16_hi(u.z), bf16_lo(u.w), bf16_hi(u.w));
  }
}

// the causal conv and SiLU of CH channels of a node: x[3] its own raw row (CH / 2 words), x[0 .. 2] the three before it on its
// path, oldest first
template <int CH>
__device__ __forceinline__ void conv_silu(const uint32_t (&x)[kTaps][CH / 2], const float4 (&w)[CH], float (&y)[CH]) {
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    auto at = [&](int tap) { return e & 1 ? bf16_hi(x[tap][e >> 1]) : bf16_lo(x[tap][e >> 1]); };
    y[e] = silu_fast(fmaf(w[e].w, at(3), fmaf(w[e].z, at(2), fmaf(w[e].y, at(1), w[e].x * at(0)))));
  }
}

// a slot out of range: zero rows, reported once per sequence
__device__ __forceinline__ void zero_rows(const TreeParams& p, int n, int T, int HP, int hv0, bool leader, int tid, int threads) {
  if (tid == 0 && leader && p.err) atomicOr(p.err, kDevErrBadSlot);
  for (int x = tid; x < T * HP * (kD / 8); x += threads) {
    const int t = x / (HP * (kD / 8)), y = x % (HP * (kD / 8));
    reinterpret_cast<uint4*>(p.out + ((static_cast<long long>(n) * T + t) * p.H_v + hv0) * kD)[y] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// A node's log decay from its logit, rate = -e^{A_log}; not below -128, whose decay is zero in fp32 like every smaller one.  Without
// the limit one infinite or huge term takes the path sums of all nodes behind it (infinite, or too large to hold the other terms)
// and with them the differences that are the decays between those nodes.  NaN stays NaN.
__device__ __forceinline__ float log_decay(float rate, float a) {
  const float g = rate * softplus_f(a);
  return g < -128.f ? -128.f : g;
}

// Sums of log decays up each node's path, by pointer doubling: lane l holds nodes l and l + 32, `up` their parents (-1 at a root
// and for absent nodes).
__device__ __forceinline__ void path_sums(double (&acc)[2], int (&up)[2]) {
#pragma unroll 1
  while (__any_sync(0xffffffffu, up[0] >= 0 || up[1] >= 0)) {
    double add[2];
    int nu[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {  // the node `up` steps above, in whichever lane holds it
      const int src = max(up[e], 0);
      const double a0 = __shfl_sync(0xffffffffu, acc[0], src & 31), a1 = __shfl_sync(0xffffffffu, acc[1], src & 31);
      const int u0 = __shfl_sync(0xffffffffu, up[0], src & 31), u1 = __shfl_sync(0xffffffffu, up[1], src & 31);
      add[e] = up[e] >= 0 ? (src < 32 ? a0 : a1) : 0.0;
      nu[e] = up[e] >= 0 ? (src < 32 ? u0 : u1) : -1;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      acc[e] += add[e];
      up[e] = nu[e];
    }
  }
}

// The MMA operand A of two neighbouring 8-column accumulator tiles (or of one, the other zero).
__device__ __forceinline__ void split_tiles(const float (&m0)[4], const float (&m1)[4], bool two, uint32_t (&ah)[4], uint32_t (&al)[4]) {
  split2(m0[0], m0[1], ah[0], al[0]);
  split2(m0[2], m0[3], ah[1], al[1]);
  if (two) {
    split2(m1[0], m1[1], ah[2], al[2]);
    split2(m1[2], m1[3], ah[3], al[3]);
  } else {
    ah[2] = ah[3] = al[2] = al[3] = 0u;
  }
}

// The gate's rows of nodes t0, t0 + step, ... of value head h, 4 dims a lane.
template <int kNodes>
__device__ __forceinline__ void load_z(uint2 (&zz)[kNodes], const TreeParams& p, long long tok0, int T, int h, int lane, int t0, int step) {
#pragma unroll
  for (int i = 0; i < kNodes; ++i) {
    const int t = t0 + step * i;
    zz[i] = t < T ? *reinterpret_cast<const uint2*>(p.z + (tok0 + t) * p.sz + static_cast<long long>(h) * kD + 4 * lane)
                    : make_uint2(0u, 0u);
  }
}

// Gated RMS norm of those nodes by one warp: o / sqrt(mean o^2 + 1e-6) norm_w SiLU(z); zeros for absent nodes, NaN for those whose
// path holds a poisoned node.  o: rows of kVRow floats.
template <int kNodes>
__device__ __forceinline__ void norm_rows(const uint2 (&zz)[kNodes], const float* o, const float (&nw)[4], const TreeParams& p,
                                          const Tree& tree, unsigned long long poison, long long tok0, int T, int h, int lane, int t0,
                                          int step) {
  float4 ov[kNodes];
  float ss[kNodes];
#pragma unroll
  for (int i = 0; i < kNodes; ++i) {
    ov[i] = *reinterpret_cast<const float4*>(o + (t0 + step * i) * kVRow + 4 * lane);
    ss[i] = fmaf(ov[i].x, ov[i].x, fmaf(ov[i].y, ov[i].y, fmaf(ov[i].z, ov[i].z, ov[i].w * ov[i].w)));
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1)
#pragma unroll
    for (int i = 0; i < kNodes; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], x);
#pragma unroll
  for (int i = 0; i < kNodes; ++i) {
    const int t = t0 + step * i;
    const unsigned long long mask = tree.mask[t];
    const float inv = rsqrtf(ss[i] * (1.0f / kD) + 1e-6f);
    float f[4] = {ov[i].x * inv * nw[0] * silu_fast(bf16_lo(zz[i].x)), ov[i].y * inv * nw[1] * silu_fast(bf16_hi(zz[i].x)),
                  ov[i].z * inv * nw[2] * silu_fast(bf16_lo(zz[i].y)), ov[i].w * inv * nw[3] * silu_fast(bf16_hi(zz[i].y))};
    if (poison & mask) f[0] = f[1] = f[2] = f[3] = __int_as_float(0x7fffffff);
    const uint2 y = mask ? make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])) : make_uint2(0u, 0u);
    if (t < T) *reinterpret_cast<uint2*>(p.out + ((tok0 + t) * p.H_v + h) * kD + 4 * lane) = y;
  }
}

// x_t = e_t - sum_{i < t} A_ti x_i: column `col` of the inverse of I + A for one block of up to 16 nodes, A's rows 20 floats apart
template <int kRows>
__device__ __forceinline__ void invert_column(const float* ab, int col, float (&x)[kRows]) {
#pragma unroll
  for (int t = 0; t < kRows; ++t) {
    float s = col == t ? 1.f : 0.f;
#pragma unroll
    for (int i4 = 0; i4 < (t + 3) / 4; ++i4) {
      const float4 av = *reinterpret_cast<const float4*>(ab + t * 20 + 4 * i4);
      if (4 * i4 < t) s = fmaf(-av.x, x[4 * i4], s);
      if (4 * i4 + 1 < t) s = fmaf(-av.y, x[4 * i4 + 1], s);
      if (4 * i4 + 2 < t) s = fmaf(-av.z, x[4 * i4 + 2], s);
      if (4 * i4 + 3 < t) s = fmaf(-av.w, x[4 * i4 + 3], s);
    }
    x[t] = s;
  }
}

cudaError_t launch_decode_tree_small(const TreeParams& p, cudaStream_t stream);            // up to 8 nodes
cudaError_t launch_decode_tree_wide(const TreeParams& p, int parts, cudaStream_t stream);  // 33 to 64 nodes

}  // namespace gdn
