// gdn_decode_tree for trees of 33 to 64 nodes.  The mathematics, the operands as pairs hi + lo and the treatment of what is not
// finite are those of gdn_tree.cu; what differs is the division of the work.
//
// At 64 nodes a CTA's shared memory leaves room for one CTA per SM, so nothing hides one phase's latency but another phase
// of the same CTA.  Sixteen warps in two groups run at the same time, a value head apart:
//   workers (0-7, 16 state rows each)  the state into tensor memory as bf16 pairs, the conv of v, R, the block solve, O;
//   side (8-15)                        the gates, the next head's A, P and inverses, the gated norm of the last head's o.
// X = S [K | Q]^T is a tcgen05 product of 128 state rows with 128 columns, a head ahead of the solve: the state comes from global
// memory into registers in the order of MMA fragments (lane (g, c): columns 16 s + 4 c .. + 3 of rows g and g + 8), is split there and
// stored to tensor memory as operand A (16x128b fragments); B = [K; Q] lies in shared memory, its 16-column steps in the same order.
// X comes back as m16n8 accumulator fragments (16x256b), in which R and the solve go on as in gdn_tree.cu.  [K; Q] K^T
// is a product of the same operand with itself.
//
// Measured (B200, 16 / 48 heads): 64 sequences x 61 nodes 256 us (the kernel of gdn_tree.cu at 64 nodes, one group of workers and four
// solver warps, 321), 8 x 64 60 us (65); 64 x 33 with 16 / 32 heads 185 us (201).  A CTA takes 68 thousand cycles, 17 of them until the
// first product; a head takes the workers 12 to 15 thousand (R and the solve 5, v 4, splitting the state 3) and the side warps about as
// many, so neither waits long for the other and what is left is the latency inside the phases at 16 warps per SM.
#include "gdn_tree_delta.cuh"

namespace gdn {

namespace {

constexpr int kThreads = 512, kSide = kThreads - kWorkers;
constexpr int TP = 64, NT = TP / 8, KT = TP / 16;       // nodes padded, 8- and 16-node blocks
constexpr int kMR = TP + 1;                             // floats of a row of the T x T products
constexpr int kIR = KT * 64;                            // bytes of a row of an operand image: 16-node blocks of 64; in odd rows the
                                                        // two of a pair change places (bank conflicts)
// shared memory, from a 1 KiB boundary: [k; q] as operand, hi then lo, each in two halves of d with 128 rows of 128 bytes | k_j . k_t
// below the diagonal, k_j . q_t on and above it (row j) | raw v rows | images and v, then o, of two heads by turns, or at first
// raw q | k rows
constexpr int kHalf = 2 * TP * 128, kLo = 2 * kHalf;
constexpr int kOffKk = 2 * kLo;
constexpr int kOffVraw = kOffKk + TP * kMR * 4;
constexpr int kVrawWarp = (TP + 3) * 32;                // 16 channels of each row, per worker
constexpr int kOffM = kOffVraw + 8 * kVrawWarp;         // -A off the diagonal blocks, T_b in them
constexpr int kOffP = kOffM + TP * kIR;
constexpr int kOffD = kOffP + TP * kIR;                 // A's diagonal blocks, f32 [KT][16][20]
constexpr int kOffV = kOffD + KT * 16 * 20 * 4;
constexpr int kV = TP * kVRow * 4;
constexpr int kOffRaw = kOffM;                          // [3 + TP][q 128 | k 128], until q and k are formed
constexpr int kOffTaps = kOffV + 2 * kV;                // conv weights of q, k and the value heads
constexpr int smem_bytes(int heads) { return 1024 + kOffTaps + (2 + heads) * kD * kTaps * 2; }
static_assert(kOffRaw + (TP + 3) * 512 <= kOffV && kOffVraw % 16 == 0 && kOffV % 16 == 0, "layout");
// tensor memory columns: X of two heads by turns, the state hi and lo, [K; Q] K^T
constexpr uint32_t kColX = 0, kColHi = 256, kColLo = 320, kColKk = 384;
// named barriers: images ready, o complete, the state stored, among the side warps, a buffer of o normed (two)
constexpr int kBarImages = 1, kBarO = 2, kBarState = 3, kBarSide = 4, kBarNormed = 5;

struct Shared {
  Tree tree;
  int tap[TP][kTaps - 1];                  // staged rows 3, 2, 1 before the node's own (t + 3) on its path
  float2 sum[kMaxHeads][TP];               // G as hi + lo
  float gamma[kMaxHeads][TP], beta[kMaxHeads][TP];
  unsigned long long poison[kMaxHeads];    // nodes of each head whose A, R or U was not finite
  uint64_t x_full[2], kk_full, drain;
  uint32_t tmem;
  int abort, next;
};

// 16 lanes x 64 columns of fp32 as m16n8 accumulator fragments: v[4 i + ..] = rows g, g + 8, columns 8 i + 2 c, + 1
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// 32 bytes at once, read once
__device__ __forceinline__ void load8(float (&v)[8], const float* src) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(src));
}

// 16 lanes x 8 columns: words c and 4 + c of rows g and g + 8
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

// element (row t, column j) of an operand image: the four columns of a lane side by side, hi then lo 8 bytes on
__device__ __forceinline__ int image_at(int t, int j) {
  return t * kIR + (((j >> 4) ^ (t & 1)) * 64) + ((j & 7) >> 1) * 16 + ((j & 15) >> 3) * 4 + (j & 1) * 2;
}

// the 128 registers of each of 512 threads are dealt out as 152 for the workers and 104 for the others (168 and 88: 289 against 285 us)
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 152;"); }
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 104;"); }

// kAligned32: the state begins at a multiple of 32 bytes, so that a lane's 32 can be loaded at once (64 sequences x 61 nodes 255 us,
// else 272)
template <bool kAligned32>
__global__ void __launch_bounds__(kThreads, 1) decode_tree_wide_kernel(const __grid_constant__ TreeParams p) {
  extern __shared__ uint8_t tw_smem[];
  __shared__ __align__(16) Shared sh;
  uint8_t* tsm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tw_smem) + 1023) & ~uintptr_t(1023));
  const int part = blockIdx.x, parts = gridDim.x, kh = blockIdx.y, n = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int T = p.T, HP = p.H_v / p.H_k / parts, hv0 = (kh * parts + part) * HP;
  const long long C_conv = static_cast<long long>(2 * p.H_k + p.H_v) * kD, tok0 = static_cast<long long>(n) * T;
  const bool leader = part == 0 && kh == 0;
  float* kk_s = reinterpret_cast<float*>(tsm + kOffKk);
  float* d_s = reinterpret_cast<float*>(tsm + kOffD);
  const Tree& tree = sh.tree;
  const Abort ab{p.err, &sh.abort};
  // the worker's rows: those lanes of tensor memory that its warp may access
  const int vw = 2 * (warp & 3) + ((warp >> 2) & 1), r0 = 16 * vw;

  // ---- staged row i: conv history oldest first, then the nodes' raw rows; these first, they do not wait for the slot
  for (int x = tid + 3 * 32; x < (T + 3) * 32; x += kThreads) {
    const int i = x >> 5, l = x & 15;
    const bf16* src = x & 16 ? p.k + (tok0 + i - 3) * p.sk : p.q + (tok0 + i - 3) * p.sq;
    cp_async16(tsm + kOffRaw + x * 16, src + static_cast<long long>(kh) * kD + 8 * l);
  }
  for (int x = tid; x < (2 + HP) * 64; x += kThreads) {  // conv weights, 64 pieces per 128 channels
    const long long head = x < 64 ? kh : x < 128 ? p.H_k + kh : 2LL * p.H_k + hv0 + (x >> 6) - 2;
    cp_async16(tsm + kOffTaps + x * 16, p.conv_w + head * kD * kTaps + (x & 63) * 8);
  }
  if (warp == 8) tree_load(sh.tree, p.parent, n, T, leader ? p.err : nullptr);
  const int slot = p.state_slot ? p.state_slot[n] : n;
  if (slot < 0 || slot >= p.n_slots) {
    cp_async_commit();
    cp_async_wait_all();
    zero_rows(p, n, T, HP, hv0, leader, tid, kThreads);
    return;
  }
  const bf16* hist = p.conv_in + static_cast<long long>(slot) * 3 * C_conv;
  if (tid < 3 * 32) {
    const int i = tid >> 5, l = tid & 15;
    cp_async16(tsm + kOffRaw + tid * 16, hist + i * C_conv + (tid & 16 ? static_cast<long long>(p.H_k) * kD : 0) +
                                             static_cast<long long>(kh) * kD + 8 * l);
  }
  auto stage_v = [&](int jh) {
    const long long off = static_cast<long long>(hv0 + jh) * kD + r0 + 8 * (lane & 1);
    for (int i = lane >> 1; i < T + 3; i += 16)
      cp_async16(tsm + kOffVraw + vw * kVrawWarp + i * 32 + (lane & 1) * 16,
                 i < 3 ? hist + i * C_conv + 2LL * p.H_k * kD + off : p.v + (tok0 + i - 3) * p.sv + off);
    cp_async_commit();
  };
  if (warp < 8) stage_v(0);
  cp_async_commit();

  // ---- the state rows of a worker: lane (g, c) takes columns 32 s + 8 c .. + 7 of rows g, g + 8: four for each of two 16-column steps
  float raw[kD / 32][2][8];
  const float* S0 = p.state_in + (static_cast<long long>(slot) * p.H_v + hv0) * kD * kD + (r0 + g) * kD + 8 * c;
  auto load_state = [&](int jh) {
#pragma unroll
    for (int s = 0; s < kD / 32; ++s)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float* src = S0 + static_cast<long long>(jh) * kD * kD + 32 * s + 8 * r * kD;
        if (kAligned32) {
          load8(raw[s][r], src);
        } else {
          const float4 a = __ldcs(reinterpret_cast<const float4*>(src)), b = __ldcs(reinterpret_cast<const float4*>(src) + 1);
          raw[s][r][0] = a.x; raw[s][r][1] = a.y; raw[s][r][2] = a.z; raw[s][r][3] = a.w;
          raw[s][r][4] = b.x; raw[s][r][5] = b.y; raw[s][r][6] = b.z; raw[s][r][7] = b.w;
        }
      }
  };
  auto store_state = [&](uint32_t tm) {  // tm: the worker's lanes
#pragma unroll
    for (int s = 0; s < kD / 16; ++s) {
      const float *x0 = raw[s >> 1][0] + 4 * (s & 1), *x1 = raw[s >> 1][1] + 4 * (s & 1);
      uint32_t hi[4], lo[4];
      split2(x0[0], x0[1], hi[0], lo[0]);
      split2(x1[0], x1[1], hi[1], lo[1]);
      split2(x0[2], x0[3], hi[2], lo[2]);
      split2(x1[2], x1[3], hi[3], lo[3]);
      tmem_st_frag(tm + kColHi + 8 * s, hi);
      tmem_st_frag(tm + kColLo + 8 * s, lo);
    }
    tmem_wait_st();
    tc_fence_before();
  };
  auto ahead = [&](int jh) {  // a head's state on its way into L2, so that the loads do not all wait for memory at once
    if (tid == kThreads - 1 && jh < HP)
      prefetch_l2(p.state_in + (static_cast<long long>(slot) * p.H_v + hv0 + jh) * kD * kD, kD * kD * 4);
  };
  ahead(0);

  if (tid == 0) {
    sh.abort = 0;
    sh.next = 0;
    mbar_init(&sh.x_full[0], 1);
    mbar_init(&sh.x_full[1], 1);
    mbar_init(&sh.kk_full, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (tid < kMaxHeads) sh.poison[tid] = 0ull;
  if (warp == 9) tmem_alloc<512>(&sh.tmem);
  if (warp == 8) {
    for (int t = lane; t < TP; t += 32) {  // (in range for the rows past T too)
      int at = t;
#pragma unroll
      for (int i = kTaps - 2; i >= 0; --i) {
        at = at >= 0 ? max(tree.parent[at], -1) : at - 1;
        sh.tap[t][i] = max(at, -3) + 3;
      }
    }
  }
  const int gate_head = warp >= 8 && warp - 8 < HP ? warp - 8 : -1;  // the head whose gates this warp forms
  bf16 a_raw[2], b_raw[2];
  float a_log = 0.f;
  if (gate_head >= 0) {
    a_log = p.A_log[hv0 + gate_head];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const long long row = tok0 + min(lane + 32 * e, T - 1);
      a_raw[e] = p.a[row * p.sa + hv0 + gate_head];
      b_raw[e] = p.b[row * p.sb + hv0 + gate_head];
    }
  }
  cp_async_wait_all();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sh.tmem, trow = tmem_addr(tbase, r0, 0);
  if (warp < 8) {
    load_state(0);
    store_state(trow);
  }
  ahead(1);

  if (gate_head >= 0) {
    // ---- a head's gates, and the sums of its log decays up each path
    const float rate = -expf(a_log);
    double acc[2];
    int up[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int t = lane + 32 * e;
      const bool there = t < T && tree.mask[t];
      up[e] = there ? tree.parent[t] : -1;
      acc[e] = there ? static_cast<double>(log_decay(rate, __bfloat162float(a_raw[e]))) : 0.0;
      sh.beta[gate_head][t] = there ? sigmoid_f(__bfloat162float(b_raw[e])) : 0.f;
    }
    path_sums(acc, up);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float hi = static_cast<float>(acc[e]);
      sh.sum[gate_head][lane + 32 * e] = make_float2(hi, static_cast<float>(acc[e] - static_cast<double>(hi)));
      sh.gamma[gate_head][lane + 32 * e] = expf(hi);
    }
  }
  {
    // ---- q (lanes 0-15) and k (16-31) of two nodes at a time: conv, SiLU, norm, split into the operand rows
    const bool is_k = lane >= 16;
    const int l = lane & 15;
    float4 cw[8];
    load_taps<8>(tsm + kOffTaps + ((is_k ? kD : 0) + 8 * l) * kTaps * 2, cw);
    const uint8_t* rows = tsm + kOffRaw + lane * 16;
    constexpr int kBatch = 2;
    while (true) {  // whichever warp is free takes the next two nodes: some are later, with the state or the gates
      int t0 = 0;
      if (lane == 0) t0 = atomicAdd(&sh.next, kBatch);
      t0 = __shfl_sync(0xffffffffu, t0, 0);
      if (t0 >= TP) break;
      uint32_t w[kBatch][kTaps][4];
      float y[kBatch][8], ss[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i;
#pragma unroll
        for (int k = 0; k < kTaps; ++k) {
          const uint4 u = *reinterpret_cast<const uint4*>(rows + (k < kTaps - 1 ? sh.tap[t][k] : t + 3) * 512);
          w[i][k][0] = u.x; w[i][k][1] = u.y; w[i][k][2] = u.z; w[i][k][3] = u.w;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        conv_silu<8>(w[i], cw, y[i]);
        ss[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss[i] = fmaf(y[i][e], y[i][e], ss[i]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < kBatch; ++i) ss[i] += __shfl_xor_sync(0xffffffffu, ss[i], o);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = t0 + i;
        const float f = rsqrtf(ss[i] + 1e-6f) * (is_k ? 1.f : p.scale);
        const bool there = tree.mask[t] != 0ull;  // (rows past T were not staged: a selection, not a product)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] = there ? y[i][e] * f : 0.f;
        // dims 8 l .. + 7: four for each of the steps 2 (l / 4), + 1, there words l % 4 and 4 + l % 4
        const int r = is_k ? t : TP + t;
        uint8_t* row = tsm + (l >> 3) * kHalf + (l & 3) * 4;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          uint32_t hi, lo;
          split2(y[i][2 * u], y[i][2 * u + 1], hi, lo);
          const uint32_t at = sw128_off(r, 4 * ((l >> 2) & 1) + u);
          *reinterpret_cast<uint32_t*>(row + at) = hi;
          *reinterpret_cast<uint32_t*>(row + kLo + at) = lo;
        }
      }
    }
  }
  fence_proxy_async_smem();
  __syncthreads();

  // ---- one thread issues: hi hi + hi lo + lo hi over the eight 16-column steps
  const uint64_t kq = smem_desc(smem_u32(tsm), 16, 1024, Swz::k128);
  auto step_at = [](int s, bool lo) { return static_cast<uint64_t>(((s >> 2) * kHalf + (s & 3) * 32 + (lo ? kLo : 0)) >> 4); };
  auto issue_x = [&](int buf) {
    tc_fence_after();
    const uint32_t idesc = idesc_bf16(128, 2 * TP, false, false);
#pragma unroll 1
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
        umma_bf16_ts(tbase + kColX + 2 * TP * buf, tbase + (i == 2 ? kColLo : kColHi) + 8 * s, kq + step_at(s, i == 1), idesc,
                     i > 0 || s > 0);
    umma_commit(&sh.x_full[buf]);
  };
  if (tid == kWorkers) {
    tc_fence_after();
    const uint32_t idesc = idesc_bf16(128, TP, false, false);
#pragma unroll 1
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
        umma_bf16(tbase + kColKk, kq + step_at(s, i == 2), kq + step_at(s, i == 1), idesc, i > 0 || s > 0);
    umma_commit(&sh.kk_full);
  }
  if (tid == 0) issue_x(0);
  __syncwarp();

  bool ok = true;
  if (warp >= 8) {
    // ------------------------------------------------ side
    regs_down();
    const int sw = warp - 8;
    float nw[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) nw[e] = __bfloat162float(p.norm_w[4 * lane + e]);  // norm_w: aligned to 2 bytes only
    {
      float d[NT][4] = {};
      ok = mbar_wait_warp(&sh.kk_full, 0, ab);
      tc_fence_after();
      if (ok) {
        tmem_ld_frag(trow + kColKk, &d[0][0]);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = r0 + g + (e >> 1) * 8, j = 8 * i + 2 * c + (e & 1);
          if (row < TP && j < row) kk_s[row * kMR + j] = d[i][e];
          if (row >= TP && j <= row - TP) kk_s[j * kMR + row - TP] = d[i][e];
        }
    }
    named_bar_sync(kBarSide, kSide);

    // A, P and the diagonal blocks' inverses of a head.  A lane per columns j, j + 1, four rows at a time.
    auto solve = [&](int jh) {
      const int j = 2 * lane;
      const float4 gj = *reinterpret_cast<const float4*>(&sh.sum[jh][j]);
      constexpr int kBatch = 4;
#pragma unroll 1
      for (int t0 = sw; t0 < TP; t0 += 8 * kBatch) {
        float pv[kBatch][2], av[kBatch][2], chk = 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int t = t0 + 8 * i;
          const unsigned m2 = static_cast<unsigned>(tree.mask[t] >> j);
          const float2 gt = sh.sum[jh][t];
          const float be = sh.beta[jh][t];
          const float d0 = j == t ? 1.f : __expf((gt.x - gj.x) + (gt.y - gj.y));
          const float d1 = j + 1 == t ? 1.f : __expf((gt.x - gj.z) + (gt.y - gj.w));
          pv[i][0] = m2 & 1u ? d0 * kk_s[j * kMR + t] : 0.f;
          pv[i][1] = m2 & 2u ? d1 * kk_s[(j + 1) * kMR + t] : 0.f;
          av[i][0] = (m2 & 1u) && j < t ? be * d0 * kk_s[t * kMR + j] : 0.f;
          av[i][1] = (m2 & 2u) && j + 1 < t ? be * d1 * kk_s[t * kMR + j + 1] : 0.f;
          chk = fmaf(av[i][0], 0.f, fmaf(av[i][1], 0.f, chk));
        }
        if (chk != 0.f) {  // (NaN)
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!isfinite(av[i][e])) {
                atomicOr(&sh.poison[jh], 1ull << (t0 + 8 * i));
                av[i][e] = 0.f;
              }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int t = t0 + 8 * i;
          if ((j >> 4) > (t >> 4)) continue;  // the blocks above the diagonal are not read
          uint32_t hi, lo;
          split2(pv[i][0], pv[i][1], hi, lo);
          uint8_t* at = tsm + kOffP + image_at(t, j);
          *reinterpret_cast<uint32_t*>(at) = hi;
          *reinterpret_cast<uint32_t*>(at + 8) = lo;
          if ((j >> 4) == (t >> 4)) {
            *reinterpret_cast<float2*>(d_s + (t >> 4) * 320 + (t & 15) * 20 + (j & 15)) = make_float2(av[i][0], av[i][1]);
          } else {
            split2(-av[i][0], -av[i][1], hi, lo);
            at += kOffM - kOffP;
            *reinterpret_cast<uint32_t*>(at) = hi;
            *reinterpret_cast<uint32_t*>(at + 8) = lo;
          }
        }
      }
      named_bar_sync(kBarSide, kSide);
      if (sw * 2 < KT) {  // T_b: a lane per column of a block
        const int b = 2 * sw + (lane >> 4), col = lane & 15;
        float x[16];
        invert_column(d_s + b * 320, col, x);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          bf16* at = reinterpret_cast<bf16*>(tsm + kOffM + image_at(16 * b + t, 16 * b + col));
          const bf16 hi = __float2bfloat16(x[t]);
          at[0] = hi;
          at[4] = __float2bfloat16(x[t] - __bfloat162float(hi));
        }
      }
      bar_arrive(kBarImages, kThreads);
    };
    solve(0);
    for (int jh = 0; jh < HP; ++jh) {
      uint2 zz[NT];
      load_z(zz, p, tok0, T, hv0 + jh, lane, sw, 8);
      ahead(jh + 2);
      named_bar_sync(kBarO, kThreads);  // and the workers have read this head's images
      if (jh + 1 < HP) solve(jh + 1);   // first: the workers wait for it
      norm_rows(zz, reinterpret_cast<const float*>(tsm + kOffV + (jh & 1) * kV), nw, p, tree, sh.poison[jh], tok0, T, hv0 + jh,
                lane, sw, 8);
      // (a barrier of one parity is met again two heads later, which both groups reach only after the other has left it)
      if (jh + 2 < HP) bar_arrive(kBarNormed + (jh & 1), kThreads);
    }
  } else {
    // ------------------------------------------------ workers
    regs_up();
    if (HP > 1) load_state(1);
    for (int jh = 0; jh < HP; ++jh) {
      float* v_s = reinterpret_cast<float*>(tsm + kOffV + (jh & 1) * kV);
      if (jh >= 2) named_bar_sync(kBarNormed + (jh & 1), kThreads);  // v overwrites the o of two heads before
      {  // ---- v of this worker's 16 rows: a lane takes 4 channels of one node, 8 nodes at a time
        const int piece = lane & 3;
        if (jh > 0) {
          cp_async_wait_all();
          __syncwarp();
        }
        float4 cw[4];
        load_taps<4>(tsm + kOffTaps + ((2 + jh) * kD + r0 + 4 * piece) * kTaps * 2, cw);
        const uint8_t* rows = tsm + kOffVraw + vw * kVrawWarp + piece * 8;
        constexpr int kBatch = 2;
#pragma unroll 1
        for (int i0 = 0; i0 < NT; i0 += kBatch) {
          uint32_t w[kBatch][kTaps][2];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int t = 8 * (i0 + i) + (lane >> 2);
#pragma unroll
            for (int k = 0; k < kTaps; ++k) {
              const uint2 u = *reinterpret_cast<const uint2*>(rows + (k < kTaps - 1 ? sh.tap[t][k] : t + 3) * 32);
              w[i][k][0] = u.x; w[i][k][1] = u.y;
            }
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int t = 8 * (i0 + i) + (lane >> 2);
            float y[4];
            conv_silu<4>(w[i], cw, y);
            const bool there = tree.mask[t] != 0ull;
            *reinterpret_cast<float4*>(v_s + t * kVRow + r0 + 4 * piece) =
                make_float4(there ? y[0] : 0.f, there ? y[1] : 0.f, there ? y[2] : 0.f, there ? y[3] : 0.f);
          }
        }
        __syncwarp();  // this worker's v_s columns; its raw rows are free
        if (jh + 1 < HP) stage_v(jh + 1);
      }
      // ---- X of this head is there, and the state it read can be overwritten by the next head's
      ok = ok && mbar_wait_warp(&sh.x_full[jh & 1], (jh >> 1) & 1, ab);
      tc_fence_after();
      if (jh + 1 < HP) {
        if (ok) store_state(trow);
        named_bar_sync(kBarState, kWorkers);
        if (tid == 0 && ok) issue_x((jh + 1) & 1);
        __syncwarp();
      }
      float acc[2 * NT][4] = {};  // tile i < NT: nodes' keys, i >= NT: queries
      if (ok) {
        tmem_ld_frag(trow + kColX + 2 * TP * (jh & 1), &acc[0][0]);
        tmem_ld_frag(trow + kColX + 2 * TP * (jh & 1) + TP, &acc[NT][0]);
        tmem_wait_ld();
        tc_fence_before();
      }
      named_bar_sync(kBarImages, kThreads);
      // non-finite entries: their nodes are poisoned, zeros stand in
      auto clean = [&](float (&m)[4], int i) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!isfinite(m[e])) {
            atomicOr(&sh.poison[jh], 1ull << (8 * i + 2 * c + (e & 1)));
            m[e] = 0.f;
          }
      };
      // ---- R^T = beta (v - gamma X_k), X_q *= gamma (the start of O^T)
      float chk = 0.f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int t = 8 * i + 2 * c;
        const float2 be = *reinterpret_cast<const float2*>(&sh.beta[jh][t]), ga = *reinterpret_cast<const float2*>(&sh.gamma[jh][t]);
        const float* v0 = v_s + t * kVRow + r0 + g;
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
      // ---- block by block: U_b^T = R_b^T T_b^T, then its part of the later blocks' R and of O
#pragma unroll
      for (int b = 0; b < KT; ++b) {
        const int at = g * kIR + ((b ^ (g & 1)) * 64) + c * 16;
        const uint8_t *mb = tsm + kOffM + at, *pb = tsm + kOffP + at;
        uint32_t ah[4], al[4];
        split_tiles(acc[2 * b], acc[2 * b + 1], true, ah, al);
        float u[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        mma_split(u[0], ah, al, *reinterpret_cast<const uint4*>(mb + 16 * b * kIR));
        mma_split(u[1], ah, al, *reinterpret_cast<const uint4*>(mb + (16 * b + 8) * kIR));
        chk = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) chk = fmaf(u[0][e], 0.f, fmaf(u[1][e], 0.f, chk));
        if (chk != 0.f) {
          clean(u[0], 2 * b);
          clean(u[1], 2 * b + 1);
        }
        split_tiles(u[0], u[1], true, ah, al);
#pragma unroll
        for (int i = 2 * b + 2; i < NT; ++i) mma_split(acc[i], ah, al, *reinterpret_cast<const uint4*>(mb + 8 * i * kIR));
#pragma unroll
        for (int i = 2 * b; i < NT; ++i) mma_split(acc[NT + i], ah, al, *reinterpret_cast<const uint4*>(pb + 8 * i * kIR));
      }
      if (jh + 2 < HP) load_state(jh + 2);
      // ---- O^T into shared memory, over this worker's own columns of v
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float* dst = v_s + (8 * i + 2 * c) * kVRow + r0 + g;
        dst[0] = acc[NT + i][0];
        dst[kVRow] = acc[NT + i][1];
        dst[8] = acc[NT + i][2];
        dst[kVRow + 8] = acc[NT + i][3];
      }
      bar_arrive(kBarO, kThreads);
    }
    if (tid == 0 && !ok) {  // products still in flight end before their operands and tensor memory are given up
      int drain_flag = 0;
      const Abort drain{nullptr, &drain_flag};
      umma_commit(&sh.drain);
      mbar_wait(&sh.drain, 0, drain);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) tmem_dealloc<512>(tbase);
}

}  // namespace

template <bool kAligned32>
static cudaError_t launch(const TreeParams& p, int parts, cudaStream_t stream) {
  const int smem = smem_bytes(p.H_v / p.H_k / parts);
  // (the limit is the largest call's, the same in every call: two threads' calls may interleave here)
  const cudaError_t e = cudaFuncSetAttribute(decode_tree_wide_kernel<kAligned32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             smem_bytes(kMaxHeads));
  if (e != cudaSuccess) return e;
  decode_tree_wide_kernel<kAligned32><<<dim3(parts, p.H_k, p.N), kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_decode_tree_wide(const TreeParams& p, int parts, cudaStream_t stream) {
  return (reinterpret_cast<uintptr_t>(p.state_in) & 31) == 0 ? launch<true>(p, parts, stream) : launch<false>(p, parts, stream);
}

}  // namespace gdn
