// gdn_attention_tree: attention of a tree's nodes over a KV cache and their ancestors.
#include "gdn_tree.cuh"

namespace gdn {

namespace {

constexpr int kTaThreads = 128;

// One CTA per (node, query head, sequence): keys in blocks of 128, one per thread, with a running maximum and sum.
__global__ void __launch_bounds__(kTaThreads) attention_tree_kernel(AttnTreeParams p) {
  const int t = blockIdx.x, h = blockIdx.y, n = blockIdx.z, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = p.D, kvh = h / (p.H_q / p.H_kv);
  __shared__ Tree tree;
  __shared__ float q_s[256], p_s[kTaThreads], red[4];
  if (warp == 0) tree_load(tree, p.parent, n, p.T, t == 0 && h == 0 ? p.err : nullptr);
  const long long tok = static_cast<long long>(n) * p.T + t;
  for (int d = tid; d < D; d += kTaThreads) q_s[d] = __bfloat162float(p.q[tok * p.ld_q + static_cast<long long>(h) * D + d]) * p.scale;
  __syncthreads();
  const int len = p.cache_len[n];
  const unsigned long long mask = tree.mask[t];
  bf16* out = p.out + (tok * p.H_q + h) * D;
  if (len < 0 || len > p.cap || mask == 0) {
    if ((len < 0 || len > p.cap) && tid == 0 && p.err) atomicOr(p.err, kDevErrCacheLen);
    for (int d = tid; d < D; d += kTaThreads) out[d] = __float2bfloat16(0.f);
    return;
  }
  const long long row_el = static_cast<long long>(p.H_kv) * D;
  const bf16* kc = p.k_cache + static_cast<long long>(n) * p.cap * row_el + kvh * D;
  const bf16* vc = p.v_cache + static_cast<long long>(n) * p.cap * row_el + kvh * D;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int j0 = 0; j0 < len + p.T; j0 += kTaThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j < len || (j < len + p.T && ((mask >> (j - len)) & 1))) {
      const bf16* k = j < len ? kc + j * row_el : p.k_tree + (static_cast<long long>(n) * p.T + j - len) * p.ld_kt + kvh * D;
      s = 0.f;
      for (int d = 0; d < D; ++d) s = fmaf(q_s[d], __bfloat162float(k[d]), s);
    }
    float mx = s;
    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = mx == -INFINITY ? 0.f : mx;
    const float e = s == -INFINITY ? 0.f : expf(s - base);
    const float f = expf(m - base);
    m = mx;
    float sum = e;
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    p_s[tid] = e;
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    l = l * f + (red[0] + red[1] + red[2] + red[3]);
    o[0] *= f;
    o[1] *= f;
    for (int i = 0; i < kTaThreads && j0 + i < len + p.T; ++i) {
      const int jj = j0 + i;
      if (jj >= len && !((mask >> (jj - len)) & 1)) continue;
      const bf16* v = jj < len ? vc + jj * row_el : p.v_tree + (static_cast<long long>(n) * p.T + jj - len) * p.ld_vt + kvh * D;
      o[0] = fmaf(p_s[i], __bfloat162float(v[tid]), o[0]);
      if (D > kTaThreads) o[1] = fmaf(p_s[i], __bfloat162float(v[kTaThreads + tid]), o[1]);
    }
    __syncthreads();
  }
  for (int i = 0; i < D / kTaThreads; ++i) {
    const int d = i * kTaThreads + tid;
    float y = o[i] / l;
    if (p.g) y *= sigmoid_f(__bfloat162float(p.g[tok * p.ld_g + static_cast<long long>(h) * D + d]));
    out[d] = __float2bfloat16(y);
  }
}

}  // namespace

size_t attention_tree_workspace(int, int, int, int, int) { return 16; }

cudaError_t launch_attention_tree(const AttnTreeParams& p, cudaStream_t stream) {
  attention_tree_kernel<<<dim3(p.T, p.H_q, p.N), kTaThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
