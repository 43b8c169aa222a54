// gdn_decode_tree: the delta-rule mixer's outputs of every node of a tree of drafted tokens, from
// one read of the state.  This file: trees of up to 32 nodes (with several value heads per CTA, of 9 to 32; gdn_tree_small.cu
// below), the launch, and the mathematics of all three kernels; gdn_tree_wide.cu: 33 to 64 nodes.
//
// Per value head, with G_t the sum of the log decays on node t's path, gamma_t = e^{G_t}, D_tj = e^{G_t - G_j} for
// an ancestor j of t (or t itself), 0 otherwise:
//   A_tj = beta_t D_tj (k_j . k_t) for j < t,   P_tj = D_tj (k_j . q_t)
//   R_t = beta_t (v_t - gamma_t S k_t),   (I + A) U = R,   o_t = gamma_t S q_t + sum_j P_tj u_j
// A is strictly lower triangular whatever the tree, because a parent comes before its children.  In
// the kernel's orientation (rows = d_v of the state): X = S [K | Q]^T, U^T = R^T T^T with T = (I + A)^-1,
// O^T = X_q diag(gamma) + U^T P^T, so everything after X is local to 16 state rows and stays in one warp's registers.
//
// A CTA takes one key head of one sequence and its value heads in turn (one value head per CTA while
// there are few sequences).  Warps 0-7, 16 state rows each: the conv, norm and products of q and k at the start,
// then per value head the conv of v, X, U, O and the gated norm.  One to four more warps (kSolvers) form the next
// value head's A, P and the inverses T_b of I + A's 16 x 16 diagonal blocks meanwhile; the workers solve block by block,
//   U_b = T_b (R_b - sum over blocks b' < b of A_bb' U_b'),
// with the same number of products as a multiplication by the whole inverse, which would have to be formed row by row (a
// dependent chain of 60 rows took 30 to 200 thousand cycles per head).  The state goes from global
// memory straight into MMA operand registers, two of a head's eight 16-column steps ahead; raw
// q, k and v rows come through shared memory by asynchronous copies, the next head's v during this head's products.
//
// The products are m16n8k16 bf16 MMAs: the state's 128 rows meet 2 T <= 64 columns once, which is too little per CTA for a tcgen05
// tile to pay for moving the state through tensor memory as bf16 pairs (a tcgen05 X took 175 against 134 us for 64 sequences x 32
// nodes; from 33 nodes on the wide kernel uses it).
// Every operand is a pair hi + lo (hi hi + hi lo + lo hi, about 16 significant bits): the gated norm
// amplifies the rounding of a sum whose terms nearly cancel, and plain bf16 operands leave the
// mixer's bound.  Sums, gates and the solve are fp32, the sums of log decays fp64 (their differences over a
// long path would lose bits).
//
// Measured (B200, 16 / 48 heads, the kernel alone): 64 sequences x 16 nodes 75 us (3.3 TB/s of the 248 MB it cannot do
// without), 64 x 32 129 us, one sequence x 13 nodes 9 us; 256 x 8 nodes 194 us, where the small kernel takes 180.  Latency bounds it:
// a warp issues every 8 to 10 cycles, so the time falls with the warps per SM.
//
// A node whose inputs are not finite: zeros stand in for its row of R and U, so that no zero weight meets an
// infinity, and its own outputs and its descendants' become NaN; other nodes do not see it.
#include "gdn_tree_delta.cuh"

namespace gdn {

namespace {

constexpr int kQkRow = 576;              // bytes of one node's k (or q): 8 steps x 4 lanes x (4 hi | 4 lo), and 64 more so
                                         // that a quarter-warp's 16-byte reads of two rows fall into different banks

template <int NT>
struct TreeCfg {
  static_assert(NT == 1 || NT == 2 || NT == 4, "up to 32 nodes");
  static constexpr int TP = 8 * NT;                       // nodes, padded
  static constexpr int KT = (TP + 15) / 16;               // 16-node blocks
  static constexpr int kSolvers = NT <= 2 ? 1 : 2;
  static constexpr int kThreads = kWorkers + 32 * kSolvers;
  // CTAs per SM: the phases of a value head are latency-bound, so warps per SM count for more than loads ahead per warp (256
  // sequences x 8 nodes: 226 us with 4 steps ahead and 2 CTAs, 199 us with 2 and 3, 191 us with 2 and 4)
  static constexpr int kMinCtas = NT == 1 ? 4 : NT == 2 ? 3 : 2;
  static constexpr int kAhead = 2;                        // 16-column steps of the state loaded ahead
  static constexpr int MR = TP + 4;                       // floats of a row of the T x T products
  static constexpr int IR = KT * 64 + (KT % 2 ? 0 : 64);  // bytes of a row of an operand image
  // shared memory: [k; q] operand rows | k . k, then k . q | raw v rows | images and o, or at first raw q | k rows
  static constexpr int kOffKk = 2 * TP * kQkRow;
  static constexpr int kOffVraw = kOffKk + 2 * TP * MR * 4;
  static constexpr int kVrawWarp = (TP + 3) * 32;         // 16 channels of each row, per warp
  static constexpr int kOffM = kOffVraw + 8 * kVrawWarp;  // -A off the diagonal blocks, T_b in them
  static constexpr int kOffP = kOffM + TP * IR;
  static constexpr int kOffD = kOffP + TP * IR;           // A's diagonal blocks, f32 [KT][16][20]
  static constexpr int kOffV = kOffD + KT * 16 * 20 * 4;
  static constexpr int kEnd = kOffV + TP * kVRow * 4;
  static constexpr int kOffRaw = kOffM;                   // [3 + TP][q 128 | k 128], until q and k are formed
  static constexpr int kRawEnd = kOffRaw + (TP + 3) * 512;
  static constexpr int kOffTaps = ((kEnd > kRawEnd ? kEnd : kRawEnd) + 15) / 16 * 16;  // conv weights of q, k and the value heads
  static constexpr int smem(int heads) { return kOffTaps + (2 + heads) * kD * kTaps * 2; }
};

template <int NT>
__global__ void __launch_bounds__(TreeCfg<NT>::kThreads, TreeCfg<NT>::kMinCtas)
    decode_tree_kernel(const __grid_constant__ TreeParams p) {
  using C = TreeCfg<NT>;
  constexpr int TP = C::TP, KT = C::KT;
  const int part = blockIdx.x, parts = gridDim.x, kh = blockIdx.y, n = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int T = p.T, HP = p.H_v / p.H_k / parts, hv0 = (kh * parts + part) * HP;
  const long long C_conv = static_cast<long long>(2 * p.H_k + p.H_v) * kD;
  const bool leader = part == 0 && kh == 0;
  __shared__ Tree tree;
  if (warp == 8) tree_load(tree, p.parent, n, T, leader ? p.err : nullptr);  // (its loads beside the slot's)
  const int slot = p.state_slot ? p.state_slot[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    zero_rows(p, n, T, HP, hv0, leader, tid, C::kThreads);
    return;
  }
  extern __shared__ __align__(16) uint8_t tsm[];
  float* kk_s = reinterpret_cast<float*>(tsm + C::kOffKk);
  float* d_s = reinterpret_cast<float*>(tsm + C::kOffD);
  float* v_s = reinterpret_cast<float*>(tsm + C::kOffV);
  __shared__ int tap_s[kMaxNodes][kTaps - 1];         // staged rows 3, 2, 1 before the node's own (t + 3) on its path
  __shared__ float g_s[kMaxHeads][TP], beta_s[kMaxHeads][TP];
  __shared__ float gamma_s[TP];
  __shared__ float2 sum_s[TP];                        // G as hi + lo
  __shared__ unsigned long long poison_s[kMaxHeads];  // nodes of each head whose A, R or U was not finite

  // ---- this warp's state rows, 16-column step ks: lane (g, c) takes columns 16 ks + 4 c .. + 3 of rows g, g + 8
  const float* S0 = p.state_in + (static_cast<long long>(slot) * p.H_v + hv0) * kD * kD;
  float4 raw[C::kAhead][2];
  auto load_step = [&](int jh, int ks) {
    const float* src = S0 + static_cast<long long>(jh) * kD * kD + (16 * warp + g) * kD + 16 * ks + 4 * c;
    raw[ks % C::kAhead][0] = __ldcs(reinterpret_cast<const float4*>(src));
    raw[ks % C::kAhead][1] = __ldcs(reinterpret_cast<const float4*>(src + 8 * kD));
  };
  const bf16* hist = p.conv_in + static_cast<long long>(slot) * 3 * C_conv;
  const long long tok0 = static_cast<long long>(n) * T;
  // staged row i: conv history oldest first, then the nodes' raw rows
  for (int x = tid; x < (T + 3) * 32; x += C::kThreads) {
    const int i = x >> 5, l = x & 15;
    const bool is_k = x & 16;
    const long long off = static_cast<long long>(kh) * kD + 8 * l;
    const bf16* src = i < 3 ? hist + i * C_conv + (is_k ? static_cast<long long>(p.H_k) * kD : 0) + off
                            : (is_k ? p.k + (tok0 + i - 3) * p.sk : p.q + (tok0 + i - 3) * p.sq) + off;
    cp_async16(tsm + C::kOffRaw + x * 16, src);
  }
  for (int x = tid; x < (2 + HP) * 64; x += C::kThreads) {  // 64 pieces per 128 channels
    const long long head = x < 64 ? kh : x < 128 ? p.H_k + kh : 2LL * p.H_k + hv0 + (x >> 6) - 2;
    cp_async16(tsm + C::kOffTaps + x * 16, p.conv_w + head * kD * kTaps + (x & 63) * 8);
  }
  uint8_t* vraw = tsm + C::kOffVraw + (warp & 7) * C::kVrawWarp;  // this worker's own
  auto stage_v = [&](int jh) {
    const long long off = static_cast<long long>(hv0 + jh) * kD + 16 * warp + 8 * (lane & 1);
    for (int i = lane >> 1; i < T + 3; i += 16)
      cp_async16(vraw + i * 32 + (lane & 1) * 16,
                 i < 3 ? hist + i * C_conv + 2LL * p.H_k * kD + off : p.v + (tok0 + i - 3) * p.sv + off);
  };
  if (warp < 8) stage_v(0);
  cp_async_commit();
  if (warp < 8) {
#pragma unroll
    for (int ks = 0; ks < C::kAhead; ++ks) load_step(0, ks);
  }
  if (warp == 8) {
    for (int t = lane; t < T; t += 32) {
      int at = t;
#pragma unroll
      for (int i = kTaps - 2; i >= 0; --i) {
        at = at >= 0 ? max(tree.parent[at], -1) : at - 1;
        tap_s[t][i] = max(at, -3) + 3;
      }
    }
  }
  if (tid < kMaxHeads) poison_s[tid] = 0ull;
  cp_async_wait_all();
  __syncthreads();

  if (warp < 8) {
    // ---- q (lanes 0-15) and k (16-31) of one node per warp: conv, SiLU, norm, split into the operand rows
    const bool is_k = lane >= 16;
    const int l = lane & 15;
    float4 cw[8];
    load_taps<8>(tsm + C::kOffTaps + ((is_k ? kD : 0) + 8 * l) * kTaps * 2, cw);
    const uint8_t* rows = tsm + C::kOffRaw + lane * 16;
#pragma unroll(NT >= 4 ? 2 : 1)
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
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float f = rsqrtf(ss + 1e-6f) * (is_k ? 1.f : p.scale);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= f;
      }
      // dims 8 l .. + 7: step l / 2, lane slots c = 2 (l % 2) and + 1
      uint8_t* dst = tsm + (is_k ? t : TP + t) * kQkRow + (l >> 1) * 64 + (l & 1) * 32;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint4 v;
        split2(y[4 * u], y[4 * u + 1], v.x, v.z);
        split2(y[4 * u + 2], y[4 * u + 3], v.y, v.w);
        reinterpret_cast<uint4*>(dst)[u] = v;
      }
    }
  } else {
    for (int x = tid - kWorkers; x < HP * TP; x += 32 * C::kSolvers) {
      const int jh = x / TP, t = x % TP, h = hv0 + jh;
      float gl = 0.f, be = 0.f;
      if (t < T && tree.mask[t]) {
        gl = log_decay(-expf(p.A_log[h]), __bfloat162float(p.a[(tok0 + t) * p.sa + h]));
        be = sigmoid_f(__bfloat162float(p.b[(tok0 + t) * p.sb + h]));
      }
      g_s[jh][t] = gl;
      beta_s[jh][t] = be;
    }
  }
  __syncthreads();
  if (warp < 8) {
    // ---- [K; Q] K^T: 16-row tile m of the 2 TP operand rows against the nodes j that can be ancestors of its
    // nodes, the tiles j shared by 8 / NT warps
    const int m = warp % NT, jt0 = warp / NT;
    constexpr int kStep = 8 / NT, kMine = (NT + kStep - 1) / kStep;
    const int t_max = TP >= 16 ? (16 * m) % TP + 15 : TP - 1;
    float d[kMine][4];
#pragma unroll
    for (int i = 0; i < kMine; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i][e] = 0.f;
    if (jt0 < NT) {
      const uint8_t* ar = tsm + (16 * m + g) * kQkRow + c * 16;
      const uint8_t* br = tsm + (8 * jt0 + g) * kQkRow + c * 16;
#pragma unroll 2
      for (int ks = 0; ks < kD / 16; ++ks) {
        const uint4 r0 = *reinterpret_cast<const uint4*>(ar + ks * 64), r1 = *reinterpret_cast<const uint4*>(ar + 8 * kQkRow + ks * 64);
        const uint32_t ah[4] = {r0.x, r1.x, r0.y, r1.y}, al[4] = {r0.z, r1.z, r0.w, r1.w};
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (jt0 + i * kStep < NT && 8 * (jt0 + i * kStep) <= t_max)
            mma_split(d[i], ah, al, *reinterpret_cast<const uint4*>(br + 8 * i * kStep * kQkRow + ks * 64));
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        if (jt0 + i * kStep < NT) {
          float* dst = kk_s + (16 * m + g) * C::MR + 8 * (jt0 + i * kStep) + 2 * c;
          *reinterpret_cast<float2*>(dst) = make_float2(d[i][0], d[i][1]);
          *reinterpret_cast<float2*>(dst + 8 * C::MR) = make_float2(d[i][2], d[i][3]);
        }
    }
  } else {
    // what no node sees stays zero in the images
    for (int x = tid - kWorkers; x < (C::kOffV - C::kOffM) / 16; x += 32 * C::kSolvers)
      reinterpret_cast<uint4*>(tsm + C::kOffM)[x] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncthreads();

  if (warp >= 8) {
    // ------------------------------------------------ the solvers: A, P and the diagonal blocks' inverses of each value head
    constexpr int kSolve = 32 * C::kSolvers;
    const int sw = warp - 8;
    // byte offset of element (row t, column j) in an image: the four columns of a lane side by side, hi then lo
    auto img = [](int t, int j) { return t * C::IR + (j >> 4) * 64 + ((j & 7) >> 1) * 16 + ((j & 15) >> 3) * 4 + (j & 1) * 2; };
    auto put = [](uint8_t* at, float v) {
      const bf16 hi = __float2bfloat16(v);
      reinterpret_cast<bf16*>(at)[0] = hi;
      reinterpret_cast<bf16*>(at)[4] = __float2bfloat16(v - __bfloat162float(hi));
    };
    for (int jh = 0; jh < HP; ++jh) {
      if (sw == 0) {  // sums of log decays up each path, by pointer doubling
        double acc[2];
        int up[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = lane + 32 * e;
          acc[e] = t < TP ? static_cast<double>(g_s[jh][t]) : 0.0;
          up[e] = t < T && tree.mask[t] ? tree.parent[t] : -1;
        }
        path_sums(acc, up);
        if (jh > 0) named_bar_sync(2, C::kThreads - (kSolve - 32));  // the workers have read the last head's images
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = lane + 32 * e;
          if (t < TP) {
            const float hi = static_cast<float>(acc[e]);
            sum_s[t] = make_float2(hi, static_cast<float>(acc[e] - static_cast<double>(hi)));
            gamma_s[t] = expf(hi);
          }
        }
      }
      if (C::kSolvers > 1) named_bar_sync(4, kSolve); else __syncwarp();
      // a lane per (row t, column j): a warp takes 32 / TP rows at a time
      constexpr int kRowsAtOnce = 32 / TP;
#pragma unroll(TP < 32 ? 4 : 2)
      for (int t0 = sw * kRowsAtOnce; t0 < TP; t0 += C::kSolvers * kRowsAtOnce) {
        const int t = t0 + lane / TP, j = lane % TP;
        const unsigned long long mt = tree.mask[t];
        const float2 gt = sum_s[t], gj = sum_s[j];
        const float be = beta_s[jh][t];
        const float kk = kk_s[t * C::MR + j], qk = kk_s[(TP + t) * C::MR + j];
        const float dec = j == t ? 1.f : __expf((gt.x - gj.x) + (gt.y - gj.y));
        const float pv = dec * qk;
        float av = be * dec * kk;
        if ((mt >> j) & 1) {
          put(tsm + C::kOffP + img(t, j), pv);
          if (j < t) {
            if (!isfinite(av)) {
              atomicOr(&poison_s[jh], 1ull << t);
              av = 0.f;
            }
            if ((t >> 4) == (j >> 4)) d_s[(t >> 4) * 320 + (t & 15) * 20 + (j & 15)] = av;
            else put(tsm + C::kOffM + img(t, j), -av);
          }
        }
      }
      if (C::kSolvers > 1) named_bar_sync(4, kSolve); else __syncwarp();
      // T_b: a lane per column of a 16 x 16 block, x_t = e_t - sum_{i < t} A_ti x_i down the column in registers
      // (invert_column written out: as a call it spills more registers at NT = 2, 64 sequences x 16 nodes 84 -> 88 us)
      if (sw * 2 < KT) {
        const int b = 2 * sw + (lane >> 4), col = lane & 15;
        if (b < KT && 16 * b + col < TP) {
          const float* ab = d_s + b * 320;
          float x[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) {
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
#pragma unroll
          for (int t = 0; t < 16; ++t)
            if (16 * b + t < TP) put(tsm + C::kOffM + img(16 * b + t, 16 * b + col), x[t]);
        }
      }
      bar_arrive(3, C::kThreads);
    }
    return;
  }

  // ------------------------------------------------ the workers
  float nw[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) nw[e] = __bfloat162float(p.norm_w[4 * lane + e]);  // norm_w: aligned to 2 bytes only
  for (int jh = 0; jh < HP; ++jh) {
    const int h = hv0 + jh;
    // ---- v of this warp's 16 rows: a lane takes 4 channels of one node, 8 nodes at a time
    {
      const int piece = lane & 3;
      float4 cw[4];
      load_taps<4>(tsm + C::kOffTaps + ((2 + jh) * kD + 16 * warp + 4 * piece) * kTaps * 2, cw);
      if (jh > 0) {
        cp_async_wait_all();
        __syncwarp();
      }
      const uint8_t* rows = vraw + piece * 8;
#pragma unroll(NT >= 4 ? 4 : NT)
      for (int i8 = 0; i8 < NT; ++i8) {
        const int t = 8 * i8 + (lane >> 2);
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
      __syncwarp();  // this warp's v_s columns; its raw rows are free
      if (jh + 1 < HP) {
        stage_v(jh + 1);
        cp_async_commit();
      }
    }
    // ---- X = S [K | Q]^T; tile i < NT: nodes' keys, i >= NT: queries
    float acc[2 * NT][4];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < kD / 16; ++ks) {
      uint32_t ah[4], al[4];
      const float4 r0 = raw[ks % C::kAhead][0], r1 = raw[ks % C::kAhead][1];
      split2(r0.x, r0.y, ah[0], al[0]);
      split2(r1.x, r1.y, ah[1], al[1]);
      split2(r0.z, r0.w, ah[2], al[2]);
      split2(r1.z, r1.w, ah[3], al[3]);
      if (ks < kD / 16 - C::kAhead) load_step(jh, ks + C::kAhead);
      const uint8_t* br = tsm + g * kQkRow + ks * 64 + c * 16;
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) mma_split(acc[i], ah, al, *reinterpret_cast<const uint4*>(br + 8 * i * kQkRow));
    }
    if (jh + 1 < HP) {
#pragma unroll
      for (int ks = 0; ks < C::kAhead; ++ks) load_step(jh + 1, ks);
    }
    named_bar_sync(3, C::kThreads);  // images and gamma of this head
    // non-finite entries: their nodes are poisoned, zeros stand in
    auto clean = [&](float (&m)[4], int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!isfinite(m[e])) {
          atomicOr(&poison_s[jh], 1ull << (8 * i + 2 * c + (e & 1)));
          m[e] = 0.f;
        }
    };
    // ---- R^T = beta (v - gamma X_k), X_q *= gamma (the start of O^T)
    float chk = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = 8 * i + 2 * c;
      const float2 be = *reinterpret_cast<const float2*>(&beta_s[jh][t]), ga = *reinterpret_cast<const float2*>(&gamma_s[t]);
      const float* v0 = v_s + t * kVRow + 16 * warp + g;
      acc[i][0] = be.x * fmaf(-ga.x, acc[i][0], v0[0]);
      acc[i][1] = be.y * fmaf(-ga.y, acc[i][1], v0[kVRow]);
      acc[i][2] = be.x * fmaf(-ga.x, acc[i][2], v0[8]);
      acc[i][3] = be.y * fmaf(-ga.y, acc[i][3], v0[kVRow + 8]);
      acc[NT + i][0] *= ga.x;
      acc[NT + i][1] *= ga.y;
      acc[NT + i][2] *= ga.x;
      acc[NT + i][3] *= ga.y;
#pragma unroll
      for (int e = 0; e < 4; ++e) chk = fmaf(acc[i][e], 0.f, chk);
    }
    if (chk != 0.f) {
#pragma unroll
      for (int i = 0; i < NT; ++i) clean(acc[i], i);
    }
    // the gate's rows this warp will norm, on their way during the products
    uint2 zz[NT];
    load_z(zz, p, tok0, T, h, lane, warp, 8);
    // ---- block by block: U_b^T = R_b^T T_b^T, then its part of the later blocks' R and of O
#pragma unroll
    for (int b = 0; b < KT; ++b) {
      constexpr bool kTwo = NT > 1;
      const int i1 = kTwo ? 2 * b + 1 : 0;
      const uint8_t* mb = tsm + C::kOffM + g * C::IR + b * 64 + c * 16;
      const uint8_t* pb = tsm + C::kOffP + g * C::IR + b * 64 + c * 16;
      uint32_t ah[4], al[4];
      split_tiles(acc[2 * b], acc[i1], kTwo, ah, al);
      float u[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      mma_split(u[0], ah, al, *reinterpret_cast<const uint4*>(mb + 16 * b * C::IR));
      if (kTwo) mma_split(u[1], ah, al, *reinterpret_cast<const uint4*>(mb + (16 * b + 8) * C::IR));
      chk = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) chk = fmaf(u[0][e], 0.f, fmaf(u[1][e], 0.f, chk));
      if (chk != 0.f) {
        clean(u[0], 2 * b);
        if (kTwo) clean(u[1], i1);
      }
      split_tiles(u[0], u[1], kTwo, ah, al);
#pragma unroll
      for (int i = 2 * b + 2; i < NT; ++i) mma_split(acc[i], ah, al, *reinterpret_cast<const uint4*>(mb + 8 * i * C::IR));
#pragma unroll
      for (int i = 2 * b; i < NT; ++i) mma_split(acc[NT + i], ah, al, *reinterpret_cast<const uint4*>(pb + 8 * i * C::IR));
    }
    if (jh + 1 < HP) bar_arrive(2, kWorkers + 32);  // images and gamma are free
    // ---- O^T into shared memory, over this warp's own columns of v
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float* dst = v_s + (8 * i + 2 * c) * kVRow + 16 * warp + g;
      dst[0] = acc[NT + i][0];
      dst[kVRow] = acc[NT + i][1];
      dst[8] = acc[NT + i][2];
      dst[kVRow + 8] = acc[NT + i][3];
    }
    named_bar_sync(1, kWorkers);
    // ---- gated RMS norm, a warp per node
    norm_rows(zz, v_s, nw, p, tree, poison_s[jh], tok0, T, h, lane, warp, 8);
    if (jh + 1 < HP) named_bar_sync(1, kWorkers);  // the next head's v overwrites o
  }
}

template <int NT>
cudaError_t launch_nt(const TreeParams& p, int parts, cudaStream_t stream) {
  using C = TreeCfg<NT>;
  const int smem = C::smem(p.H_v / p.H_k / parts);
  // (the limit is the largest call's, the same in every call: two threads' calls may interleave here)
  const cudaError_t e = cudaFuncSetAttribute(decode_tree_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(kMaxHeads));
  if (e != cudaSuccess) return e;
  decode_tree_kernel<NT><<<dim3(parts, p.H_k, p.N), C::kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeParams& p, cudaStream_t stream, void* const* events) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // one CTA per value head while one per key head would leave SMs idle
  const int parts = static_cast<long long>(p.N) * p.H_k < n_sm ? p.H_v / p.H_k : 1;
  if (events) cudaEventRecord(static_cast<cudaEvent_t>(events[0]), stream);
  // up to 8 nodes: the small kernel, unless a CTA has one value head (16 / 16 heads, 64 x 8 nodes: 28.7 against 26.5 us; 16 / 48
  // heads, 64 x 8 nodes: 52 against 57 us, 10 x 8 17 against 19, 256 x 1 152 against 172)
  e = p.T <= 8 && parts == 1 && p.H_v > p.H_k ? launch_decode_tree_small(p, stream)
      : p.T <= 8 ? launch_nt<1>(p, parts, stream)
      : p.T <= 16 ? launch_nt<2>(p, parts, stream)
      : p.T <= 32 ? launch_nt<4>(p, parts, stream)
                  : launch_decode_tree_wide(p, parts, stream);
  if (events) cudaEventRecord(static_cast<cudaEvent_t>(events[1]), stream);
  return e;
}

}  // namespace gdn
