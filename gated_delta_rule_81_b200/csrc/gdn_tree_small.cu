// gdn_decode_tree for trees of up to 8 nodes where a CTA has several value heads.  The mathematics, the operands as pairs hi + lo and
// the treatment of what is not finite are those of gdn_tree.cu; what differs is the order of the work.
//
// The state's bytes bound the call, so nothing may stop their stream: the 8 x 8 systems of all the CTA's value heads are solved
// first, a warp per head, and then each warp runs its 16 state rows of one head after the other (v, X, U, O) without meeting the others
// until the norm at the end.  Eight warps of 64 registers, four CTAs per SM.
//
// Measured (B200, 16 / 48 heads, in a graph): 256 sequences x 8 nodes 180 - 189 us (5.0 TB/s of the 906 MB it cannot do without; the
// kernel of gdn_tree.cu 194), 256 x 1 152 us (172), 64 x 8 52 us (57).  Bringing the state into L2 ahead of the loads changed nothing at one
// head ahead and cost 10% at all heads; templates of 16 nodes this way took 99 against 75 us at 64 x 16.
#include "gdn_tree_delta.cuh"

namespace gdn {

namespace {

constexpr int TP = 8;                                  // nodes, padded
constexpr int kQkRow = 576;                            // bytes of one node's k (or q): 8 steps x 4 lanes x (4 hi | 4 lo), and 64 more so
                                                       // that a quarter-warp's 16-byte reads of two rows fall into different banks
constexpr int kAhead = 2;                              // 16-column steps of the state loaded ahead
constexpr int kMR = TP + 4;                            // floats of a row of the T x T products
constexpr int kIR = 64;                                // bytes of a row of an operand image (16 columns)
// shared memory: [k; q] operand rows | k . k, then k . q | per value head: T's image, P's image, A (f32 [8][20]), gamma and beta,
// G as hi + lo | raw v rows | conv weights of q, k and the value heads | v, then o, of each head, or at first raw q | k rows
constexpr int kOffKk = 2 * TP * kQkRow;
constexpr int kOffHead = kOffKk + 2 * TP * kMR * 4;
constexpr int kImg = TP * kIR, kHeadA = 2 * kImg, kHeadGate = kHeadA + TP * 20 * 4, kHeadSum = kHeadGate + 2 * TP * 4;
constexpr int kHead = kHeadSum + TP * 8;
constexpr int kVraw = 8 * (TP + 3) * 32;               // raw v rows of a head, 16 channels of each row per warp
constexpr int kO = TP * kVRow * 4;                     // v, then o, of a head
constexpr int kRaw = (TP + 3) * 512;                   // raw q | k rows
constexpr __host__ __device__ int off_vraw(int heads) { return kOffHead + heads * kHead; }
constexpr __host__ __device__ int off_taps(int heads) { return off_vraw(heads) + heads * kVraw; }
constexpr __host__ __device__ int off_o(int heads) { return off_taps(heads) + (2 + heads) * kD * kTaps * 2; }
constexpr int smem_bytes(int heads) { return off_o(heads) + (heads * kO > kRaw ? heads * kO : kRaw); }
static_assert(kOffHead % 16 == 0 && kHead % 16 == 0 && kHeadGate % 16 == 0, "layout");

// q or k of a node, 8 dims a lane, 16 lanes: divided by its norm, times `scale`
__device__ __forceinline__ void qk_norm(float (&y)[8], float scale) {
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float f = rsqrtf(ss + 1e-6f) * scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= f;
}

// dims 8 l .. + 7 of an operand row: step l / 2, lane slots c = 2 (l % 2) and + 1
__device__ __forceinline__ void store_qk_row(uint8_t* row, int l, const float (&y)[8]) {
  uint8_t* dst = row + (l >> 1) * 64 + (l & 1) * 32;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint4 v;
    split2(y[4 * u], y[4 * u + 1], v.x, v.z);
    split2(y[4 * u + 2], y[4 * u + 3], v.y, v.w);
    reinterpret_cast<uint4*>(dst)[u] = v;
  }
}

// element j of a row of an operand image, as its pair: 16-column blocks of 64 bytes, in them the four columns of a lane slot
// side by side, hi then lo
__device__ __forceinline__ void put_pair(uint8_t* row, int j, float v) {
  bf16* at = reinterpret_cast<bf16*>(row + (j >> 4) * 64 + ((j & 7) >> 1) * 16 + ((j & 15) >> 3) * 4 + (j & 1) * 2);
  const bf16 hi = __float2bfloat16(v);
  at[0] = hi;
  at[4] = __float2bfloat16(v - __bfloat162float(hi));
}

// a node's gated RMS norm, 4 dims a lane: o / sqrt(mean o^2 + 1e-6) norm_w SiLU(z); zeros for an absent node, NaN for one whose
// path holds a poisoned node
__device__ __forceinline__ uint2 norm_row(const float4& o, const float (&nw)[4], const uint2& z, bool there, bool poisoned) {
  float ss = fmaf(o.x, o.x, fmaf(o.y, o.y, fmaf(o.z, o.z, o.w * o.w)));
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, x);
  const float inv = rsqrtf(ss * (1.0f / kD) + 1e-6f);
  float f[4] = {o.x * inv * nw[0] * silu_fast(bf16_lo(z.x)), o.y * inv * nw[1] * silu_fast(bf16_hi(z.x)),
                o.z * inv * nw[2] * silu_fast(bf16_lo(z.y)), o.w * inv * nw[3] * silu_fast(bf16_hi(z.y))};
  if (poisoned) f[0] = f[1] = f[2] = f[3] = __int_as_float(0x7fffffff);
  return there ? make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])) : make_uint2(0u, 0u);
}

__global__ void __launch_bounds__(kWorkers, 4) decode_tree_small_kernel(const __grid_constant__ TreeParams p) {
  const int part = blockIdx.x, parts = gridDim.x, kh = blockIdx.y, n = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int T = p.T, HP = p.H_v / p.H_k / parts, hv0 = (kh * parts + part) * HP;
  const long long C_conv = static_cast<long long>(2 * p.H_k + p.H_v) * kD;
  const bool leader = part == 0 && kh == 0;
  __shared__ Tree tree;
  if (warp == 7) tree_load(tree, p.parent, n, T, leader ? p.err : nullptr);  // (its loads beside the slot's)
  const int slot = p.state_slot ? p.state_slot[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    zero_rows(p, n, T, HP, hv0, leader, tid, kWorkers);
    return;
  }
  extern __shared__ __align__(16) uint8_t tsm[];
  float* kk_s = reinterpret_cast<float*>(tsm + kOffKk);
  uint8_t* taps_sm = tsm + off_taps(HP);
  uint8_t* o_sm = tsm + off_o(HP);
  __shared__ int tap_s[TP][kTaps - 1];                // staged rows 3, 2, 1 before the node's own (t + 3) on its path
  __shared__ unsigned poison_s[kMaxHeads];            // nodes of each head whose A, R or U was not finite

  const float* S0 = p.state_in + (static_cast<long long>(slot) * p.H_v + hv0) * kD * kD + (16 * warp + g) * kD + 4 * c;
  float4 raw[kAhead][2];
  auto load_step = [&](int jh, int ks) {
    const float* src = S0 + static_cast<long long>(jh) * kD * kD + 16 * ks;
    raw[ks % kAhead][0] = __ldcs(reinterpret_cast<const float4*>(src));
    raw[ks % kAhead][1] = __ldcs(reinterpret_cast<const float4*>(src + 8 * kD));
  };
  const bf16* hist = p.conv_in + static_cast<long long>(slot) * 3 * C_conv;
  const long long tok0 = static_cast<long long>(n) * T;
  for (int x = tid; x < (T + 3) * 32; x += kWorkers) {  // conv history oldest first, then the nodes' rows: q | k
    const int i = x >> 5, l = x & 15;
    const bool is_k = x & 16;
    const long long off = static_cast<long long>(kh) * kD + 8 * l;
    const bf16* src = i < 3 ? hist + i * C_conv + (is_k ? static_cast<long long>(p.H_k) * kD : 0) + off
                            : (is_k ? p.k + (tok0 + i - 3) * p.sk : p.q + (tok0 + i - 3) * p.sq) + off;
    cp_async16(o_sm + x * 16, src);
  }
  for (int x = tid; x < (2 + HP) * 64; x += kWorkers) {  // conv weights, 64 pieces per 128 channels
    const long long head = x < 64 ? kh : x < 128 ? p.H_k + kh : 2LL * p.H_k + hv0 + (x >> 6) - 2;
    cp_async16(taps_sm + x * 16, p.conv_w + head * kD * kTaps + (x & 63) * 8);
  }
  for (int x = tid; x < HP * (T + 3) * 16; x += kWorkers) {  // v: piece x % 16 (warp, half) of row i of head jh
    const int jh = x / ((T + 3) * 16), i = x / 16 % (T + 3), l = x & 15;
    const long long off = static_cast<long long>(hv0 + jh) * kD + 8 * l;
    cp_async16(tsm + off_vraw(HP) + jh * kVraw + (l >> 1) * ((TP + 3) * 32) + i * 32 + (l & 1) * 16,
               i < 3 ? hist + i * C_conv + 2LL * p.H_k * kD + off : p.v + (tok0 + i - 3) * p.sv + off);
  }
  cp_async_commit();
#pragma unroll
  for (int ks = 0; ks < kAhead; ++ks) load_step(0, ks);
  if (warp == 7 && lane < T) {
    int at = lane;
#pragma unroll
    for (int i = kTaps - 2; i >= 0; --i) {
      at = at >= 0 ? max(tree.parent[at], -1) : at - 1;
      tap_s[lane][i] = max(at, -3) + 3;
    }
  }
  if (tid < kMaxHeads) poison_s[tid] = 0u;
  // the gates of warp jh's head: lane t its node's log decay and beta
  float gl = 0.f, be = 0.f;
  cp_async_wait_all();
  __syncthreads();
  if (warp < HP && lane < T && tree.mask[lane]) {
    gl = log_decay(-expf(p.A_log[hv0 + warp]), __bfloat162float(p.a[(tok0 + lane) * p.sa + hv0 + warp]));
    be = sigmoid_f(__bfloat162float(p.b[(tok0 + lane) * p.sb + hv0 + warp]));
  }
  {
    // ---- q (lanes 0-15) and k (16-31) of one node per warp: conv, SiLU, norm, split into the operand rows
    const bool is_k = lane >= 16;
    const int l = lane & 15;
    float4 cw[8];
    load_taps<8>(taps_sm + ((is_k ? kD : 0) + 8 * l) * kTaps * 2, cw);
    const uint8_t* rows = o_sm + lane * 16;
#pragma unroll 1
    for (int t = warp; t < TP; t += 8) {
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (t < T && tree.mask[t]) {  // the same for the whole warp
        uint32_t w[kTaps][4];
#pragma unroll
        for (int i = 0; i < kTaps; ++i) {
          const uint4 u = *reinterpret_cast<const uint4*>(rows + (i < kTaps - 1 ? tap_s[t][i] : t + 3) * 512);
          w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
        }
        conv_silu<8>(w, cw, y);
        qk_norm(y, is_k ? 1.f : p.scale);
      }
      store_qk_row(tsm + (is_k ? t : TP + t) * kQkRow, l, y);
    }
  }
  __syncthreads();
  if (warp == 7) {  // ---- [K; Q] K^T
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    const uint8_t* ar = tsm + g * kQkRow + c * 16;
#pragma unroll 4
    for (int ks = 0; ks < kD / 16; ++ks) {
      const uint4 k = *reinterpret_cast<const uint4*>(ar + ks * 64), q = *reinterpret_cast<const uint4*>(ar + TP * kQkRow + ks * 64);
      const uint32_t ah[4] = {k.x, q.x, k.y, q.y}, al[4] = {k.z, q.z, k.w, q.w};
      mma_split(d, ah, al, k);
    }
    *reinterpret_cast<float2*>(kk_s + g * kMR + 2 * c) = make_float2(d[0], d[1]);
    *reinterpret_cast<float2*>(kk_s + (TP + g) * kMR + 2 * c) = make_float2(d[2], d[3]);
  }
  if (warp < HP) {  // this warp's head: sums of log decays up each path by pointer doubling, gamma, beta
    uint8_t* hd = tsm + kOffHead + warp * kHead;
    double acc[2] = {static_cast<double>(gl), 0.0};
    int up[2] = {lane < T && tree.mask[lane] ? tree.parent[lane] : -1, -1};
    path_sums(acc, up);
    if (lane < TP) {
      const float hi = static_cast<float>(acc[0]);
      reinterpret_cast<float*>(hd + kHeadGate)[lane] = expf(hi);
      reinterpret_cast<float*>(hd + kHeadGate)[TP + lane] = be;
      reinterpret_cast<float2*>(hd + kHeadSum)[lane] = make_float2(hi, static_cast<float>(acc[0] - static_cast<double>(hi)));
    }
    for (int x = lane; x < kHeadGate / 16; x += 32) reinterpret_cast<uint4*>(hd)[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();
  if (warp < HP) {  // A, P and T = (I + A)^-1 of this warp's head
    uint8_t* hd = tsm + kOffHead + warp * kHead;
    float* a_s = reinterpret_cast<float*>(hd + kHeadA);
    const float2* sum = reinterpret_cast<const float2*>(hd + kHeadSum);
    const float* beta = reinterpret_cast<const float*>(hd + kHeadGate) + TP;
#pragma unroll
    for (int x = lane; x < TP * TP; x += 32) {
      const int t = x / TP, j = x % TP;
      const float2 gt = sum[t], gj = sum[j];
      const float dec = j == t ? 1.f : __expf((gt.x - gj.x) + (gt.y - gj.y));
      const float pv = dec * kk_s[(TP + t) * kMR + j];
      float av = beta[t] * dec * kk_s[t * kMR + j];
      if ((tree.mask[t] >> j) & 1) {
        put_pair(hd + kImg + t * kIR, j, pv);
        if (j < t) {
          if (!isfinite(av)) {
            atomicOr(&poison_s[warp], 1u << t);
            av = 0.f;
          }
          a_s[t * 20 + j] = av;
        }
      }
    }
    __syncwarp();
    if (lane < TP) {
      float x[TP];
      invert_column(a_s, lane, x);
#pragma unroll
      for (int t = 0; t < TP; ++t) put_pair(hd + t * kIR, lane, x[t]);
    }
  }
  __syncthreads();

  // ---- each warp its 16 rows of one value head after the other
#pragma unroll 1
  for (int jh = 0; jh < HP; ++jh) {
    const uint8_t* hd = tsm + kOffHead + jh * kHead;
    float* v_s = reinterpret_cast<float*>(o_sm + jh * kO);
    {  // v: a lane takes 4 channels of one node
      const int piece = lane & 3;
      float4 cw[4];
      load_taps<4>(taps_sm + ((2 + jh) * kD + 16 * warp + 4 * piece) * kTaps * 2, cw);
      const uint8_t* rows = tsm + off_vraw(HP) + jh * kVraw + warp * ((TP + 3) * 32) + piece * 8;
      {
        const int t = lane >> 2;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < T && tree.mask[t]) {
          uint32_t w[kTaps][2];
#pragma unroll
          for (int i = 0; i < kTaps; ++i) {
            const uint2 u = *reinterpret_cast<const uint2*>(rows + (i < kTaps - 1 ? tap_s[t][i] : t + 3) * 32);
            w[i][0] = u.x; w[i][1] = u.y;
          }
          conv_silu<4>(w, cw, y);
        }
        *reinterpret_cast<float4*>(v_s + t * kVRow + 16 * warp + 4 * piece) = make_float4(y[0], y[1], y[2], y[3]);
      }
    }
    float x_k[4] = {0.f, 0.f, 0.f, 0.f}, x_q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks) {
      uint32_t ah[4], al[4];
      const float4 r0 = raw[ks % kAhead][0], r1 = raw[ks % kAhead][1];
      split2(r0.x, r0.y, ah[0], al[0]);
      split2(r1.x, r1.y, ah[1], al[1]);
      split2(r0.z, r0.w, ah[2], al[2]);
      split2(r1.z, r1.w, ah[3], al[3]);
      if (ks + kAhead < kD / 16) load_step(jh, ks + kAhead);
      else if (jh + 1 < HP) load_step(jh + 1, ks + kAhead - kD / 16);
      const uint8_t* br = tsm + g * kQkRow + ks * 64 + c * 16;
      mma_split(x_k, ah, al, *reinterpret_cast<const uint4*>(br));
      mma_split(x_q, ah, al, *reinterpret_cast<const uint4*>(br + TP * kQkRow));
    }
    __syncwarp();  // this warp's columns of v
    auto clean = [&](float (&m)[4]) {  // non-finite entries: their nodes are poisoned, zeros stand in
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!isfinite(m[e])) {
          atomicOr(&poison_s[jh], 1u << (2 * c + (e & 1)));
          m[e] = 0.f;
        }
    };
    auto not_finite = [](const float (&m)[4]) { return fmaf(m[0], 0.f, fmaf(m[1], 0.f, fmaf(m[2], 0.f, m[3] * 0.f))) != 0.f; };
    // R^T = beta (v - gamma X_k), X_q *= gamma (the start of O^T)
    const float* gate = reinterpret_cast<const float*>(hd + kHeadGate);
    const float2 ga = *reinterpret_cast<const float2*>(gate + 2 * c), bt = *reinterpret_cast<const float2*>(gate + TP + 2 * c);
    float* v0 = v_s + 2 * c * kVRow + 16 * warp + g;
    x_k[0] = bt.x * fmaf(-ga.x, x_k[0], v0[0]);
    x_k[1] = bt.y * fmaf(-ga.y, x_k[1], v0[kVRow]);
    x_k[2] = bt.x * fmaf(-ga.x, x_k[2], v0[8]);
    x_k[3] = bt.y * fmaf(-ga.y, x_k[3], v0[kVRow + 8]);
    x_q[0] *= ga.x;
    x_q[1] *= ga.y;
    x_q[2] *= ga.x;
    x_q[3] *= ga.y;
    if (not_finite(x_k)) clean(x_k);
    // U^T = R^T T^T, O^T += U^T P^T, over this warp's own columns of v
    uint32_t ah[4], al[4];
    split_tiles(x_k, x_k, false, ah, al);
    float u[4] = {0.f, 0.f, 0.f, 0.f};
    mma_split(u, ah, al, *reinterpret_cast<const uint4*>(hd + g * kIR + c * 16));
    if (not_finite(u)) clean(u);
    split_tiles(u, u, false, ah, al);
    mma_split(x_q, ah, al, *reinterpret_cast<const uint4*>(hd + kImg + g * kIR + c * 16));
    v0[0] = x_q[0];
    v0[kVRow] = x_q[1];
    v0[8] = x_q[2];
    v0[kVRow + 8] = x_q[3];
  }

  // ---- gated RMS norm, a warp per (node, head), a few at a time.  Every warp's rows of o are awaited; a warp without a pair
  // only announces its own.
  if (warp >= T * HP) {
    bar_arrive(1, kWorkers);
    return;
  }
  float nw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) nw[e] = __bfloat162float(p.norm_w[4 * lane + e]);  // norm_w: aligned to 2 bytes only
  constexpr int kAtOnce = 3;
  for (int x0 = warp; x0 < T * HP; x0 += 8 * kAtOnce) {
    uint2 zz[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int x = min(x0 + 8 * i, T * HP - 1);
      zz[i] = *reinterpret_cast<const uint2*>(p.z + (tok0 + x / HP) * p.sz + static_cast<long long>(hv0 + x % HP) * kD + 4 * lane);
    }
    if (x0 == warp) named_bar_sync(1, kWorkers);  // (the first round's loads are on their way)
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int x = x0 + 8 * i, t = min(x, T * HP - 1) / HP, jh = min(x, T * HP - 1) % HP;
      const unsigned long long mask = tree.mask[t];
      const uint2 y = norm_row(*reinterpret_cast<const float4*>(o_sm + jh * kO + (t * kVRow + 4 * lane) * 4), nw, zz[i], mask != 0ull,
                               (poison_s[jh] & static_cast<unsigned>(mask)) != 0u);
      if (x < T * HP) *reinterpret_cast<uint2*>(p.out + ((tok0 + t) * p.H_v + hv0 + jh) * kD + 4 * lane) = y;
    }
  }
}

}  // namespace

cudaError_t launch_decode_tree_small(const TreeParams& p, cudaStream_t stream) {
  const int smem = smem_bytes(p.H_v / p.H_k);
  // (the limit is the largest call's, the same in every call: two threads' calls may interleave here)
  const cudaError_t e = cudaFuncSetAttribute(decode_tree_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem_bytes(kMaxHeads));
  if (e != cudaSuccess) return e;
  decode_tree_small_kernel<<<dim3(1, p.H_k, p.N), kWorkers, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
