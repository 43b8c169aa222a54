// gdn_decode_tree: the delta-rule mixer's outputs of every node of a tree of drafted tokens.
#include "gdn_tree.cuh"

namespace gdn {

namespace {

constexpr int kTreeThreads = 128;  // thread = state row (d_v)

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// One CTA per (value head, sequence).  Shared: q, k, u f32 [T][128] and K K^T, Q K^T f32 [T][T].
__global__ void __launch_bounds__(kTreeThreads) decode_tree_kernel(TreeParams p) {
  const int h = blockIdx.x, n = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = p.T, kh = h / (p.H_v / p.H_k);
  const long long C_conv = static_cast<long long>(2 * p.H_k + p.H_v) * kD;
  extern __shared__ __align__(16) float tree_sm[];
  float* q_s = tree_sm;
  float* k_s = q_s + T * kD;
  float* u_s = k_s + T * kD;
  float* kk_s = u_s + T * kD;
  float* qk_s = kk_s + T * T;
  __shared__ Tree tree;
  __shared__ float alpha_s[kMaxNodes], beta_s[kMaxNodes], start_s[kMaxNodes];
  const int slot = p.state_slot ? p.state_slot[n] : n;
  const bool bad = slot < 0 || slot >= p.n_slots;
  if (warp == 0) tree_load(tree, p.parent, n, T, h == 0 ? p.err : nullptr);
  if (bad) {
    if (tid == 0 && h == 0 && p.err) atomicOr(p.err, kDevErrBadSlot);
    for (int t = 0; t < T; ++t)
      p.out[((static_cast<long long>(n) * T + t) * p.H_v + h) * kD + tid] = __float2bfloat16(0.f);
    return;
  }
  __syncthreads();
  // conv of each node along its path, one channel of q, k and v per thread
  const bf16* hist = p.conv_in + static_cast<long long>(slot) * 3 * C_conv;
#pragma unroll 1
  for (int part = 0; part < 3; ++part) {
    const bf16* x = part == 0 ? p.q : part == 1 ? p.k : p.v;
    const long long ld = part == 0 ? p.sq : part == 1 ? p.sk : p.sv;
    const long long c0 = static_cast<long long>(part == 2 ? h : kh) * kD + tid;
    const long long ch = c0 + static_cast<long long>(part) * p.H_k * kD;
    float* dst = part == 0 ? q_s : part == 1 ? k_s : u_s;
    for (int t = 0; t < T; ++t) {
      float y = 0.f;
      int at = t;  // a node, or -1, -2, -3: history, latest first
      if (tree.mask[t]) {
#pragma unroll
        for (int tap = kTaps - 1; tap >= 0; --tap) {
          const float xv = __bfloat162float(at >= 0 ? x[(static_cast<long long>(n) * T + at) * ld + c0]
                                                    : hist[(3 + at) * C_conv + ch]);
          y = fmaf(__bfloat162float(p.conv_w[ch * kTaps + tap]), xv, y);
          at = at >= 0 ? tree.parent[at] : at - 1;
        }
      }
      dst[t * kD + tid] = silu_f(y);
    }
  }
  if (tid < T) {
    const long long tok = static_cast<long long>(n) * T + tid;
    alpha_s[tid] = tree.mask[tid] ? expf(-expf(p.A_log[h]) * softplus_f(__bfloat162float(p.a[tok * p.sa + h]))) : 0.f;
    beta_s[tid] = tree.mask[tid] ? sigmoid_f(__bfloat162float(p.b[tok * p.sb + h])) : 0.f;
  }
  __syncthreads();
  for (int x = warp; x < 2 * T; x += kTreeThreads / 32) {
    float* row = (x & 1 ? k_s : q_s) + (x >> 1) * kD;
    float ss = 0.f;
    for (int j = lane; j < kD; j += 32) ss = fmaf(row[j], row[j], ss);
    const float f = rsqrtf(warp_sum(ss) + 1e-6f) * (x & 1 ? 1.f : p.scale);
    for (int j = lane; j < kD; j += 32) row[j] *= f;
  }
  __syncthreads();
  for (int x = tid; x < T * T; x += kTreeThreads) {
    const int t = x / T, j = x % T;
    float kk = 0.f, qk = 0.f;
    if ((tree.mask[t] >> j) & 1) {
      for (int i = 0; i < kD; ++i) {
        kk = fmaf(k_s[j * kD + i], k_s[t * kD + i], kk);
        qk = fmaf(k_s[j * kD + i], q_s[t * kD + i], qk);
      }
    }
    kk_s[x] = kk;
    qk_s[x] = qk;
  }
  __syncthreads();
  const float4* S = reinterpret_cast<const float4*>(p.state_in + ((static_cast<long long>(slot) * p.H_v + h) * kD + tid) * kD);
  for (int t = 0; t < T; ++t) {
    if (tree.mask[t] == 0) {
      p.out[((static_cast<long long>(n) * T + t) * p.H_v + h) * kD + tid] = __float2bfloat16(0.f);
      continue;
    }
    float sk = 0.f, sq = 0.f;
    for (int i = 0; i < kD / 4; ++i) {
      const float4 s = S[i];
      const float4 kv = reinterpret_cast<const float4*>(k_s + t * kD)[i], qv = reinterpret_cast<const float4*>(q_s + t * kD)[i];
      sk = fmaf(s.x, kv.x, fmaf(s.y, kv.y, fmaf(s.z, kv.z, fmaf(s.w, kv.w, sk))));
      sq = fmaf(s.x, qv.x, fmaf(s.y, qv.y, fmaf(s.z, qv.z, fmaf(s.w, qv.w, sq))));
    }
    // up the path: w = e^{G_t - G_j}
    float w = alpha_s[t], su = 0.f, so = 0.f;
    for (int j = tree.parent[t]; j >= 0; j = tree.parent[j]) {
      const float wu = w * u_s[j * kD + tid];
      su = fmaf(kk_s[t * T + j], wu, su);
      so = fmaf(qk_s[t * T + j], wu, so);
      w *= alpha_s[j];
    }
    const float u = beta_s[t] * (u_s[t * kD + tid] - w * sk - su);
    const float o = fmaf(w, sq, fmaf(qk_s[t * T + t], u, so));
    u_s[t * kD + tid] = u;  // v_t made room for u_t: only this thread reads this column
    // gated RMS norm over the 128 rows
    start_s[warp] = 0.f;
    __syncthreads();
    const float ss = warp_sum(o * o);
    if (lane == 0) start_s[warp] = ss;
    __syncthreads();
    const float inv = rsqrtf((start_s[0] + start_s[1] + start_s[2] + start_s[3]) * (1.0f / kD) + 1e-6f);
    const long long tok = static_cast<long long>(n) * T + t;
    const float z = __bfloat162float(p.z[tok * p.sz + static_cast<long long>(h) * kD + tid]);
    p.out[(tok * p.H_v + h) * kD + tid] = __float2bfloat16(o * inv * __bfloat162float(p.norm_w[tid]) * silu_f(z));
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream, void* const* events) {
  const int smem = (3 * p.T * kD + 2 * p.T * p.T) * 4;
  const cudaError_t e = cudaFuncSetAttribute(decode_tree_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (events) cudaEventRecord(static_cast<cudaEvent_t>(events[0]), stream);
  decode_tree_kernel<<<dim3(p.H_v, p.N), kTreeThreads, smem, stream>>>(p);
  const cudaError_t e2 = cudaGetLastError();
  if (events) cudaEventRecord(static_cast<cudaEvent_t>(events[1]), stream);
  return e2;
}

}  // namespace gdn
