// The commits of tree decoding: the delta rule's state advanced along each sequence's accepted path,
// and the accepted nodes' keys and values appended to the attention layer's caches.
//
// State: the accepted tokens' updates in path order, with the arithmetic of the decode kernel
//   sk = s_r . k_t,  delta = beta_t (v_{t,r} - alpha_t sk),  s_r <- alpha_t s_r + delta k_t
// (same products, same order of every sum), so that the committed state is bitwise that of decoding the
// path token by token.  A state row is read once and written once for up to kCommitPass tokens, which
// covers a usual accepted path; a longer one goes over the rows again, from the output state.  8 rows per warp at a time keep
// 64 registers and four CTAs on an SM: 256 sequences of 48 heads, paths of up to 8, take 280 us, 91% of the copy
// bandwidth (16 rows and two CTAs: 313 us).  One sequence takes 7 us, bound by latency.
#include "gdn_tree.cuh"

namespace gdn {

namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitPass = 8;     // path tokens per pass over the state
constexpr int kRowsPerIter = 8;    // state rows per warp and block (4 KiB, contiguous)

__device__ __forceinline__ float4 lds4_again(const float4* p) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(smem_u32(p)));
  return v;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// channel j of the CTA (q head kh | k head kh | its value heads from hv0 on) among the C_conv channels
__device__ __forceinline__ long long conv_channel(int j, int kh, int H_k, int hv0) {
  return j < kD       ? static_cast<long long>(kh) * kD + j
         : j < 2 * kD ? static_cast<long long>(H_k + kh) * kD + (j - kD)
                      : static_cast<long long>(2 * H_k + hv0) * kD + (j - 2 * kD);
}

// Dynamic shared memory for G value heads per CTA (n_ch = (2 + G) 128): feat f32 [pass][n_ch - 128] (k, then v,
// after the conv), raw bf16 [pass][n_ch], history bf16 [3][n_ch], taps bf16 [n_ch][4].
__host__ __device__ inline int commit_smem(int G) {
  const int n_ch = (2 + G) * kD;
  return kCommitPass * ((n_ch - kD) * 4 + n_ch * 2) + 3 * n_ch * 2 + n_ch * kTaps * 2;
}

__global__ void __launch_bounds__(kCommitThreads, 4) tree_commit_kernel(TreeParams p) {
  // grid (parts, H_k, N), parts CTAs of a key head in one cluster, as in decode
  const int part = blockIdx.x, parts = gridDim.x, kh = blockIdx.y, n = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int H_k = p.H_k, H_v = p.H_v, G = H_v / H_k / parts, T = p.T;
  const int hv0 = (kh * parts + part) * G;
  const long long C_conv = static_cast<long long>(2 * H_k + H_v) * kD;
  const int accepted = p.accepted[n];
  const int slot = p.state_slot ? p.state_slot[n] : n;
  if (slot < 0 || slot >= p.n_slots) {  // the same value in every thread of the cluster: its CTAs leave together
    if (tid == 0 && p.err) atomicOr(p.err, kDevErrBadSlot);
    return;
  }
  const int n_ch = (2 + G) * kD, n_kv = n_ch - kD, n_rows = G * kD;
  const float* S_in = p.state_in + (static_cast<long long>(slot) * H_v + hv0) * kD * kD;
  float* S_out = p.state_out + (static_cast<long long>(slot) * H_v + hv0) * kD * kD;
  if (lane == 0) prefetch_l2(S_in + static_cast<long long>(warp) * kRowsPerIter * kD, kRowsPerIter * kD * 4);

  extern __shared__ __align__(16) unsigned char dsm_raw[];
  float* feat = reinterpret_cast<float*>(dsm_raw);  // [pass][n_kv]
  bf16* xraw = reinterpret_cast<bf16*>(feat + kCommitPass * n_kv);
  bf16* hist = xraw + kCommitPass * n_ch;
  bf16* taps = hist + 3 * n_ch;
  __shared__ Tree tree;
  __shared__ int path_s[kMaxNodes];
  __shared__ int len_s;
  __shared__ float red[kCommitPass];
  __shared__ float alpha_s[kCommitPass * kMaxHeads], beta_s[kCommitPass * kMaxHeads];

  const int n_p16 = n_ch / 8;
  const bf16* cs_in = p.conv_in + static_cast<long long>(slot) * 3 * C_conv;
  for (int i = tid; i < 3 * n_p16; i += kCommitThreads) {
    const int row = i / n_p16, e = (i % n_p16) * 8;
    cp_async16(hist + row * n_ch + e, cs_in + row * C_conv + conv_channel(e, kh, H_k, hv0));
  }
  for (int i = tid; i < n_ch / 2; i += kCommitThreads) {
    const int e = 2 * i;
    cp_async16(taps + e * kTaps, p.conv_w + conv_channel(e, kh, H_k, hv0) * kTaps);
  }
  cp_async_commit();
  if (warp == 0) {
    int* err = part == 0 && kh == 0 ? p.err : nullptr;  // one report per sequence
    tree_load(tree, p.parent, n, T, err);
    const unsigned long long m = tree_accepted(tree, accepted, T, err);
    if (lane == 0) len_s = __popcll(m);
    for (int t = lane; t < kMaxNodes; t += 32)
      if ((m >> t) & 1) path_s[__popcll(m & ((1ull << t) - 1))] = t;
  }
  cp_async_wait_all();
  __syncthreads();
  if (parts > 1) cluster_barrier();  // every CTA of the key head holds the old q/k history now
  const int len = len_s;

  const int g = lane >> 3, c = lane & 7;
  const int u_me = c >> 2;  // the row of its two that this lane completes
  for (int i0 = 0; i0 < len; i0 += kCommitPass) {
    const int cnt = min(kCommitPass, len - i0);
    if (i0 > 0) __syncthreads();  // the last pass has read feat and the gates
    for (int i = tid; i < cnt * n_p16; i += kCommitThreads) {
      const int t = i / n_p16, e = (i % n_p16) * 8;
      const long long tok = static_cast<long long>(n) * T + path_s[i0 + t];
      const bf16* src = e < kD       ? p.q + tok * p.sq + static_cast<long long>(kh) * kD + e
                        : e < 2 * kD ? p.k + tok * p.sk + static_cast<long long>(kh) * kD + (e - kD)
                                     : p.v + tok * p.sv + static_cast<long long>(hv0) * kD + (e - 2 * kD);
      cp_async16(xraw + t * n_ch + e, src);
    }
    cp_async_commit();
    for (int x = tid; x < cnt * G; x += kCommitThreads) {
      const int t = x / G, jh = x % G, h = hv0 + jh;
      const long long tok = static_cast<long long>(n) * T + path_s[i0 + t];
      const float a = __bfloat162float(p.a[tok * p.sa + h]);
      const float b = __bfloat162float(p.b[tok * p.sb + h]);
      alpha_s[t * kMaxHeads + jh] = expf(-expf(p.A_log[h]) * softplus_f(a));
      beta_s[t * kMaxHeads + jh] = sigmoid_f(b);
    }
    cp_async_wait_all();
    __syncthreads();
    // the conv along the path; its history slides on in shared memory, each channel in its own thread
    for (int j = tid; j < n_ch; j += kCommitThreads) {
      float h0 = __bfloat162float(hist[j]);
      float h1 = __bfloat162float(hist[n_ch + j]);
      float h2 = __bfloat162float(hist[2 * n_ch + j]);
      const bf16* w = taps + j * kTaps;
      const float w0 = __bfloat162float(w[0]), w1 = __bfloat162float(w[1]), w2 = __bfloat162float(w[2]),
                  w3 = __bfloat162float(w[3]);
      for (int t = 0; t < cnt; ++t) {
        const float x = __bfloat162float(xraw[t * n_ch + j]);
        if (j >= kD) {
          float y = w0 * h0;
          y = fmaf(w1, h1, y);
          y = fmaf(w2, h2, y);
          y = fmaf(w3, x, y);
          feat[t * n_kv + (j - kD)] = silu_f(y);
        }
        h0 = h1;
        h1 = h2;
        h2 = x;
      }
      hist[j] = __float2bfloat16(h0);
      hist[n_ch + j] = __float2bfloat16(h1);
      hist[2 * n_ch + j] = __float2bfloat16(h2);
    }
    __syncthreads();
    if (warp < cnt) {  // the key's norm, one warp per token
      float ss = 0.f;
      for (int j = lane; j < kD; j += 32) {
        const float x = feat[warp * n_kv + j];
        ss = fmaf(x, x, ss);
      }
      ss = warp_sum(ss);
      if (lane == 0) red[warp] = rsqrtf(ss + 1e-6f);
    }
    __syncthreads();
    for (int x = tid; x < cnt * kD; x += kCommitThreads) {
      const int t = x / kD, j = x % kD;
      feat[t * n_kv + j] = feat[t * n_kv + j] * red[t];
    }
    __syncthreads();

    // the state rows, as in the decode kernel without its queries: a warp takes 8 contiguous rows, eight lanes
    // share a row, and a transposed butterfly (the decode kernel's pairs of lanes in its order) leaves lane c with s.k of row u =
    // c >> 2 of its two
    const float* S = i0 == 0 ? S_in : S_out;
    for (int r0 = warp * kRowsPerIter; r0 < n_rows; r0 += (kCommitThreads / 32) * kRowsPerIter) {
      const int jh = r0 >> 7;
      float4 s[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          s[u][m] = __ldcs(reinterpret_cast<const float4*>(S + static_cast<long long>(r0 + g + 4 * u) * kD) + c + 8 * m);
      const int r_next = r0 + (kCommitThreads / 32) * kRowsPerIter;
      if (lane == 0 && r_next < n_rows) prefetch_l2(S + static_cast<long long>(r_next) * kD, kRowsPerIter * kD * 4);
      for (int t = 0; t < cnt; ++t) {
        const float4* kt = reinterpret_cast<const float4*>(feat + t * n_kv);
        float2 ak[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) ak[u] = make_float2(0.f, 0.f);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float4 kk = kt[c + 8 * m];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            ak[u] = __ffma2_rn(make_float2(s[u][m].x, s[u][m].y), make_float2(kk.x, kk.y), ak[u]);
            ak[u] = __ffma2_rn(make_float2(s[u][m].z, s[u][m].w), make_float2(kk.z, kk.w), ak[u]);
          }
        }
        float d[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) d[u] = ak[u].x + ak[u].y;
        float sk = (u_me ? d[1] : d[0]) + __shfl_xor_sync(0xffffffffu, u_me ? d[0] : d[1], 4);
        sk = sk + __shfl_xor_sync(0xffffffffu, sk, 2);
        sk = sk + __shfl_xor_sync(0xffffffffu, sk, 1);
        const float al = alpha_s[t * kMaxHeads + jh], be = beta_s[t * kMaxHeads + jh];
        const int r_me = r0 + g + 4 * u_me;
        const float delta_me = be * (feat[t * n_kv + kD + r_me] - al * sk);
        const float2 al2 = make_float2(al, al);
        float2 d2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float delta = __shfl_sync(0xffffffffu, delta_me, (lane & ~7) + 4 * u);
          d2[u] = make_float2(delta, delta);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float4 kk = lds4_again(kt + c + 8 * m);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 lo = __ffma2_rn(al2, make_float2(s[u][m].x, s[u][m].y),
                                         __fmul2_rn(d2[u], make_float2(kk.x, kk.y)));
            const float2 hi = __ffma2_rn(al2, make_float2(s[u][m].z, s[u][m].w),
                                         __fmul2_rn(d2[u], make_float2(kk.z, kk.w)));
            s[u][m] = make_float4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          __stcs(reinterpret_cast<float4*>(S_out + static_cast<long long>(r0 + g + 4 * u) * kD) + c + 8 * m, s[u][m]);
    }
  }
  if (len == 0 && p.state_out != p.state_in) {  // nothing accepted: the state moves over as it is
    const float4* src = reinterpret_cast<const float4*>(S_in);
    float4* dst = reinterpret_cast<float4*>(S_out);
    for (int x = tid; x < n_rows * kD / 4; x += kCommitThreads) __stcs(dst + x, __ldcs(src + x));
  }
  if (len > 0 || p.conv_out != p.conv_in) {
    bf16* cs_out = p.conv_out + static_cast<long long>(slot) * 3 * C_conv;
    for (int j = tid; j < n_ch; j += kCommitThreads) {  // the thread that slid this channel's history
      if (part != 0 && j < 2 * kD) continue;            // q/k channels: the cluster's first CTA alone
      const long long ch = conv_channel(j, kh, H_k, hv0);
#pragma unroll
      for (int r = 0; r < 3; ++r) cs_out[r * C_conv + ch] = hist[r * n_ch + j];
    }
  }
}

// A CTA per sequence: 16-byte pieces of its path's K and V rows, four loads in flight per thread.  5 - 6 us, the latency of the
// index loads, one load and one store: a path of 8 rows of 4 heads of 256 is 64 KB.
constexpr int kAppendThreads = 256;
__global__ void __launch_bounds__(kAppendThreads) attn_tree_commit_kernel(AttnCommitParams p) {
  const int n = blockIdx.x, tid = threadIdx.x;
  __shared__ Tree tree;
  __shared__ int path_s[kMaxNodes];
  __shared__ int len_s, base_s;
  if (tid < 32) {
    const int accepted = p.accepted[n], base = p.cache_len[n];  // on their way beside the parents
    tree_load(tree, p.parent, n, p.T, p.err);
    const unsigned long long m = tree_accepted(tree, accepted, p.T, p.err);
    for (int t = tid; t < kMaxNodes; t += 32)
      if ((m >> t) & 1) path_s[__popcll(m & ((1ull << t) - 1))] = t;
    if (tid == 0) {
      int len = __popcll(m);
      if (base < 0 || base > p.cap) {
        if (p.err) atomicOr(p.err, kDevErrCacheLen);
        len = 0;
      } else if (len > p.cap - base) {
        if (p.err) atomicOr(p.err, kDevErrCacheFull);
        len = 0;
      }
      len_s = len;
      base_s = base;
      p.cache_len_out[n] = base + len;
    }
  }
  __syncthreads();
  const int row_p16 = p.H_kv * p.D / 8;  // pieces of one row of K (or V)
  const int total = len_s * 2 * row_p16;
  constexpr int kInFlight = 4;
  for (int x0 = tid; x0 < total; x0 += kInFlight * kAppendThreads) {
    uint4 piece[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int x = x0 + u * kAppendThreads;
      if (x < total) {
        const int i = x / (2 * row_p16), y = x % (2 * row_p16);
        const long long tok = static_cast<long long>(n) * p.T + path_s[i];
        const bf16* src = y < row_p16 ? p.k_tree + tok * p.ld_kt + 8LL * y : p.v_tree + tok * p.ld_vt + 8LL * (y - row_p16);
        piece[u] = *reinterpret_cast<const uint4*>(src);
      }
    }
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int x = x0 + u * kAppendThreads;
      if (x < total) {
        const int i = x / (2 * row_p16), y = x % (2 * row_p16);
        const long long row = static_cast<long long>(n) * p.cap + base_s + i;
        bf16* dst = (y < row_p16 ? p.k_cache : p.v_cache) + row * row_p16 * 8 + 8LL * (y < row_p16 ? y : y - row_p16);
        *reinterpret_cast<uint4*>(dst) = piece[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_tree_commit(const TreeParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  // as in decode: one CTA per key head, or per value head (clusters of G) while that grid would leave SMs idle
  int G = p.H_v / p.H_k, parts = 1, dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (static_cast<long long>(p.N) * p.H_k < n_sm) parts = G;
  const int smem = commit_smem(G / parts);
  // (the limit is the largest call's, the same in every call: two threads' calls may interleave here)
  if (smem > 48 * 1024 && (e = cudaFuncSetAttribute(tree_commit_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    commit_smem(kMaxHeads))) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts, p.H_k, p.N);
  cfg.blockDim = dim3(kCommitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, tree_commit_kernel, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_attn_tree_commit(const AttnCommitParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  attn_tree_commit_kernel<<<p.N, kAppendThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
