// gdn_attention_tree: attention of a tree's nodes over a KV cache and their ancestors.
//
// For sequence n and KV head kvh, the T nodes times the G query heads that share kvh are T G query
// rows (row t G + g), all over the same keys: cache_len[n] cache rows, then the T nodes' own.  With
//   s_rj = scale q_r . k_j,  m_r = max_j s_rj,  o_r = sum_j e^{s_rj - m_r} v_j / sum_j e^{s_rj - m_r}
// over the keys row r sees, the keys are taken once, in tiles of 64, with a running maximum and sum.
//
// Work split.  A unit is one (sequence, KV head): its tiles are ceil(cache_len / 64) tiles of the cache and
// one tile of the tree.  The tiles of all units in a row are cut into W equal shares, one per
// worker, so that ragged lengths balance and a single long sequence still fills the GPU; a unit cut between
// workers leaves partial (o, m, l) that a second kernel joins.  Rows beyond 128 go to further CTAs (blockIdx.x)
// of the same worker, which read the same tiles at about the same time, from L2.
//
// A CTA: warps 0-3 softmax and epilogue (thread = query row = TMEM lane), warp 4 TMA, warp 5 tcgen05.mma.
// TMEM: O (D columns) | Q as bf16 pairs (D / 2) | S in two buffers of 64.  Q sits in tensor memory, so the
// whole shared memory is a ring of K and V tiles: 6 stages of 32 KiB at D = 256, 12 of 16 KiB at D = 128.  Per tile j
//   S_j = Q K_j^T (M 128, N 64, K = D, A from TMEM), P_j = exp2(S_j c - m) as bf16 over S_j's first
//   32 columns, O += P_j V_j (M 128, N = D, K 64, A = P from TMEM, V MN-major),
// with S_{j+1} issued before P_j is awaited.  O and l are rescaled only when a row's maximum has grown by more than
// 2^8; the final division by l makes the result the same.
//
// Whatever a row may not see contributes exactly nothing: masked scores become -inf by selection, so infinities
// and NaN in masked keys vanish; masked values meet a zero probability in the product, so the
// rows behind the cache's last one, absent nodes' rows and non-finite elements of nodes' values are zeroed in
// shared memory first, and a non-finite value is added back in the epilogue to the rows that see it.
#include <cmath>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "gdn_tree.cuh"

namespace gdn {

namespace {

constexpr int kBN = 64;              // keys per tile
constexpr int kRows = 128;           // query rows per CTA
constexpr int kTaThreads = 192;
constexpr int kTaWarpTma = 4, kTaWarpMma = 5;
constexpr int kTaSms = 148;          // CTAs of the launch: one per SM of the part
constexpr int kRingBytes = 192 * 1024;
constexpr float kRescale = 8.0f;     // log2 units
constexpr int kMaxMTiles = kMaxNodes * 16 / kRows;

__host__ __device__ inline int attn_m_tiles(int G, int T) { return (T * G + kRows - 1) / kRows; }
__host__ __device__ inline int attn_workers(int m_tiles) { return kTaSms / m_tiles; }
__host__ __device__ inline int attn_slot_rows(int G, int T) { return T * G < kRows ? T * G : kRows; }

struct TaParams {
  AttnTreeParams a;
  int G, m_tiles, workers, slot_rows;
  float scale_log2e;
  float* part_o;    // [workers][2][m_tiles][slot_rows][D]
  float2* part_ml;  // [workers][2][m_tiles][slot_rows]: maximum (log2 units) and sum
};

// tiles of one unit of sequence n: 0 when its length is out of range
__device__ __forceinline__ int unit_tiles(int len, int cap) {
  return len < 0 || len > cap ? 0 : (len + kBN - 1) / kBN + 1;
}

// the first tile of worker w's share
__device__ __forceinline__ long long share_begin(long long total, int w, int workers) {
  return total / workers * w + min(total % workers, static_cast<long long>(w));
}

// the worker that takes tile x
__device__ __forceinline__ int share_owner(long long total, long long x, int workers) {
  const long long q = total / workers, r = total % workers;
  return static_cast<int>(x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q);
}

// Where tile `x` of all lies: sums the units' tiles over the sequences.  Every thread of the block calls it;
// `chunk_s` has room for blockDim.x + 1 sums.  Returns the total number of tiles; *seq, *base: the sequence and the
// tile number its first unit begins at (seq = N past the end).  With want_seq >= 0 it finds that sequence's base instead.
__device__ long long locate(const int* cache_len, int N, int cap, int H_kv, int w, int workers, int want_seq,
                            long long* chunk_s, int* seq_s, long long* base_s) {
  const int tid = threadIdx.x, n_thr = blockDim.x;
  const int per = (N + n_thr - 1) / n_thr;
  const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
  long long sum = 0;
  for (int n = n0; n < n1; ++n) sum += unit_tiles(cache_len[n], cap);
  chunk_s[tid] = sum * H_kv;
  if (tid == 0) {
    *seq_s = N;
    *base_s = 0;
  }
  __syncthreads();
  if (tid < 32) {  // exclusive prefix sums
    const int lane_per = (n_thr + 31) / 32;
    long long mine = 0;
    for (int i = tid * lane_per; i < min(n_thr, (tid + 1) * lane_per); ++i) mine += chunk_s[i];
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (tid >= o) incl += up;
    }
    long long run = incl - mine;
    for (int i = tid * lane_per; i < min(n_thr, (tid + 1) * lane_per); ++i) {
      const long long c = chunk_s[i];
      chunk_s[i] = run;
      run += c;
    }
    if (tid == 31) chunk_s[n_thr] = incl;
  }
  __syncthreads();
  const long long total = chunk_s[n_thr];
  const long long x = want_seq < 0 ? share_begin(total, w, workers) : 0;
  long long at = chunk_s[tid];
  for (int n = n0; n < n1; ++n) {
    const long long next = at + static_cast<long long>(unit_tiles(cache_len[n], cap)) * H_kv;
    if (want_seq < 0 ? (at <= x && x < next) : n == want_seq) {
      *seq_s = n;
      *base_s = at;
    }
    at = next;
  }
  __syncthreads();
  return total;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void unpack8(uint4 u, float* f) {
  f[0] = bf16_lo(u.x); f[1] = bf16_hi(u.x); f[2] = bf16_lo(u.y); f[3] = bf16_hi(u.y);
  f[4] = bf16_lo(u.z); f[5] = bf16_hi(u.z); f[6] = bf16_lo(u.w); f[7] = bf16_hi(u.w);
}

// both bf16 halves of a word with all-ones exponents (infinities, NaN) cleared
__device__ __forceinline__ uint32_t finite_only(uint32_t u) {
  if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
  if ((u & 0x7f800000u) == 0x7f800000u) u &= 0x0000ffffu;
  return u;
}

// One stretch of a worker's share within one unit.
struct Segment {
  int n, kvh, len;   // sequence, KV head, its cache rows
  int t0, nj, nt;    // first tile, tiles here, tiles of the whole unit
};

// Walks a worker's share [x, end) segment by segment, from sequence `seq` whose units begin at `base`.
struct Walk {
  const int* cache_len;
  int cap, H_kv, N, seq;
  long long base, x, end;
  __device__ __forceinline__ bool next(Segment& s) {
    while (x < end && seq < N) {
      const int len = cache_len[seq], nt = unit_tiles(len, cap);
      const long long off = x - base;
      if (off >= static_cast<long long>(nt) * H_kv) {
        base += static_cast<long long>(nt) * H_kv;
        ++seq;
        continue;
      }
      s.n = seq;
      s.len = len;
      s.nt = nt;
      s.kvh = static_cast<int>(off / nt);
      s.t0 = static_cast<int>(off % nt);
      s.nj = static_cast<int>(min(static_cast<long long>(nt - s.t0), end - x));
      x += s.nj;
      return true;
    }
    return false;
  }
};

// Positions in the ring, in loads since the segment's first: K_0, K_1, V_0, K_2, V_1, .. , V_{nj-1},
// the order in which the products take them.
__device__ __forceinline__ uint32_t ring_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t ring_v(int j, int nj) { return j < nj - 1 ? 2 * j + 2 : 2 * nj - 1; }

template <int D>
__global__ void __launch_bounds__(kTaThreads, 1)
    attention_tree_kernel(const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                          const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                          const __grid_constant__ TaParams p) {
  constexpr int kTileBytes = kBN * D * 2;
  constexpr int kStages = kRingBytes / kTileBytes;
  constexpr uint32_t kColO = 0, kColQ = D, kColS = D + D / 2;
  static_assert(kColS + 2 * kBN <= 512, "tensor memory columns");
  extern __shared__ uint8_t ta_smem[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ta_smem) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kStages], empty[kStages], s_full[2], p_full[2], pv_done[2], q_full, drain_b;
  __shared__ uint32_t tmem_base_s;
  __shared__ int abort_s;
  __shared__ long long chunk_s[kTaThreads + 1];
  __shared__ int seq_s;
  __shared__ long long base_s;
  __shared__ Tree tree;
  __shared__ unsigned long long bad_v_s;  // nodes whose values here are not all finite
  const AttnTreeParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = blockIdx.x, worker = blockIdx.y;

  const Abort ab{a.err, &abort_s};
  if (threadIdx.x == 0) {
    abort_s = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&p_full[b], kRows);
      mbar_init(&pv_done[b], 1);
    }
    mbar_init(&q_full, kRows);
    mbar_init(&drain_b, 1);
    fence_mbar_init();
  }
  if (warp == kTaWarpMma) tmem_alloc<512>(&tmem_base_s);
  const long long total = locate(a.cache_len, a.N, a.cap, a.H_kv, worker, p.workers, -1, chunk_s, &seq_s, &base_s);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  Walk walk{a.cache_len, a.cap, a.H_kv, a.N, seq_s, base_s, share_begin(total, worker, p.workers),
            share_begin(total, worker + 1, p.workers)};
  Segment sg;

  if (warp == kTaWarpTma) {
    if (lane == 0) {
      // ------------------------------------------------ loads, in the order of use
      uint32_t i = 0;  // loads so far
      bool ok = true;
      while (ok && walk.next(sg)) {
        const int x0 = sg.kvh * D;
        for (int l = 0; l < 2 * sg.nj && ok; ++l) {
          // load l of the segment: K_j for l = 0, 1, 3, 5, .., V_j for l = 2, 4, .. and the last
          const bool is_k = l == 0 || ((l & 1) && l < 2 * sg.nj - 1);
          const int j = is_k ? (l + 1) / 2 : l == 2 * sg.nj - 1 ? sg.nj - 1 : l / 2 - 1;
          const uint32_t st = i % kStages, use = i / kStages;
          if (use > 0 && !mbar_wait(&empty[st], (use - 1) & 1, ab)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[st], kTileBytes);
          const bool in_tree = sg.t0 + j == sg.nt - 1;
          const CUtensorMap* map = in_tree ? (is_k ? &tm_kt : &tm_vt) : (is_k ? &tm_kc : &tm_vc);
          const int y = in_tree ? 0 : (sg.t0 + j) * kBN;
#pragma unroll
          for (int kb = 0; kb < D / 64; ++kb)
            tma_load_3d(ring + st * kTileBytes + kb * (kBN * 128), map, x0 + kb * 64, y, sg.n, &full[st]);
          ++i;
        }
      }
      // copies still in flight (only after an abort) land before the CTA exits
      int drain_flag = 0;
      const Abort drain{nullptr, &drain_flag};
      for (uint32_t k = i > kStages ? i - kStages : 0; k < i; ++k) mbar_wait(&full[k % kStages], (k / kStages) & 1, drain);
    }
  } else if (warp == kTaWarpMma) {
    if (lane == 0) {
      // ------------------------------------------------ products
      const uint32_t idesc_s = idesc_bf16(kRows, kBN, false, false);
      const uint32_t idesc_o = idesc_bf16(kRows, D, false, true);
      const uint32_t ring_a = smem_u32(ring);
      uint32_t rb = 0;  // loads before this segment
      uint32_t gt = 0;  // tiles before this segment
      bool ok = true;
      for (uint32_t seg = 0; ok && walk.next(sg); ++seg) {
        if (!mbar_wait(&q_full, seg & 1, ab)) break;
        auto issue_pv = [&](int j) -> bool {  // O += P_j V_j
          const uint32_t t = gt + j, ld = rb + ring_v(j, sg.nj), st = ld % kStages;
          if (!mbar_wait(&p_full[t & 1], (t >> 1) & 1, ab)) return false;
          if (!mbar_wait(&full[st], (ld / kStages) & 1, ab)) return false;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < kBN / 16; ++ks)
            umma_bf16_ts(tbase + kColO, tbase + kColS + kBN * (t & 1) + 8u * ks,
                         smem_desc(ring_a + st * kTileBytes + ks * 2048u, kBN * 128, 1024, Swz::k128), idesc_o,
                         j > 0 || ks > 0);
          umma_commit(&pv_done[t & 1]);
          umma_commit(&empty[st]);
          return true;
        };
        for (int j = 0; j < sg.nj; ++j) {
          const uint32_t t = gt + j, s = t & 1, ld = rb + ring_k(j), st = ld % kStages;
          ok = mbar_wait(&full[st], (ld / kStages) & 1, ab);
          // S buffer s held P of two tiles before: its product must have read it
          ok = ok && (t < 2 || mbar_wait(&pv_done[s], ((t - 2) >> 1) & 1, ab));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            umma_bf16_ts(tbase + kColS + kBN * s, tbase + kColQ + 8u * ks,
                         smem_desc(ring_a + st * kTileBytes + (ks >> 2) * (kBN * 128u) + (ks & 3) * 32u, 16, 1024, Swz::k128),
                         idesc_s, ks > 0);
          umma_commit(&s_full[s]);
          umma_commit(&empty[st]);
          if (j >= 1 && !(ok = issue_pv(j - 1))) break;
        }
        if (ok) ok = issue_pv(sg.nj - 1);
        rb += 2 * sg.nj;
        gt += sg.nj;
      }
      umma_commit(&drain_b);
      int drain_flag = 0;
      const Abort drain{nullptr, &drain_flag};
      mbar_wait(&drain_b, 0, drain);
    }
  } else {
    // ------------------------------------------------ softmax and epilogue: thread = query row
    const int r = 32 * warp + lane, row = mt * kRows + r;
    const int t = row / p.G;                                  // the row's node
    const bool valid = row < a.T * p.G;
    const bool warp_on = mt * kRows + 32 * warp < a.T * p.G;  // some row of this warp
    const uint32_t trow = tmem_addr(tbase, 32 * warp, 0);
    uint32_t rb = 0, gt = 0;
    int tree_of = -1;
    // no early exit: the warps meet at a named barrier, so after a failed wait a warp keeps its place in the
    // loops and only skips its tensor-memory work
    bool ok = true;
    for (bool first = true; walk.next(sg); first = false) {
      const int h = sg.kvh * p.G + row % p.G;
      const long long tok = static_cast<long long>(sg.n) * a.T + t;
      // Q rows into tensor memory (what an idle row holds there is never used)
      if (ok && warp_on) {
        const uint4* src = reinterpret_cast<const uint4*>(a.q + (valid ? tok * a.ld_q + static_cast<long long>(h) * D : 0));
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 qv[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) qv[u] = valid ? src[8 * c + u] : make_uint4(0u, 0u, 0u, 0u);
          tmem_st32(trow + kColQ + 32u * c, reinterpret_cast<const float*>(qv));
        }
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(&q_full);
      // the tree of this sequence, while the first tiles load
      if (!first) named_bar_sync(1, kRows);  // all have done with the last segment's tree and bad_v_s
      if (tree_of != sg.n) {
        tree_of = sg.n;
        if (warp == 0) tree_load(tree, a.parent, sg.n, a.T, mt == 0 && sg.kvh == 0 && sg.t0 == 0 ? a.err : nullptr);
      }
      if (threadIdx.x == 0) bad_v_s = 0ull;
      named_bar_sync(1, kRows);
      const unsigned long long mask = valid ? tree.mask[t] : 0ull;

      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < sg.nj; ++j) {
        const uint32_t tl = gt + j, s = tl & 1;
        const int tile = sg.t0 + j;
        const bool in_tree = tile == sg.nt - 1;
        ok = ok && mbar_wait_warp(&s_full[s], (tl >> 1) & 1, ab);
        tc_fence_after();
        if (ok && warp_on) {
          float sv[kBN];
          tmem_ld32(trow + kColS + kBN * s, sv);
          tmem_ld32(trow + kColS + kBN * s + 32u, sv + 32);
          tmem_wait_ld();
          if (in_tree) {
#pragma unroll
            for (int c = 0; c < kBN; ++c) sv[c] = (mask >> c) & 1 ? sv[c] : -INFINITY;
          } else if ((tile + 1) * kBN > sg.len) {
            const int lim = sg.len - tile * kBN;
#pragma unroll
            for (int c = 0; c < kBN; ++c) sv[c] = c < lim ? sv[c] : -INFINITY;
          }
          float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int c = 4; c < kBN; ++c) mx[c & 3] = fmaxf(mx[c & 3], sv[c]);
          const float mloc = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2e;
          // per warp: the wait and the tensor-memory accesses are warp-collective
          const bool grow = mloc > m + kRescale || (m == -INFINITY && mloc > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mloc : m;
            if (j >= 1) {
              ok = mbar_wait_warp(&pv_done[(tl - 1) & 1], ((tl - 1) >> 1) & 1, ab);
              if (ok) {
                tc_fence_after();
                const float f = grow ? ex2(m - m_new) : 1.f;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                  float o[32];
                  tmem_ld32(trow + kColO + 32u * c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] *= f;
                  tmem_st32(trow + kColO + 32u * c, o);
                }
                l *= f;
              }
            }
            m = m_new;
          }
          const float m_use = m == -INFINITY ? 0.f : m;  // nothing seen yet: every score is -inf
          uint32_t pk[kBN / 2];
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kBN / 2; ++c) {
            const float p0 = ex2(fmaf(sv[2 * c], p.scale_log2e, -m_use));
            const float p1 = ex2(fmaf(sv[2 * c + 1], p.scale_log2e, -m_use));
            ls[c & 3] += p0 + p1;
            pk[c] = pack_bf16x2(p0, p1);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          if (ok) {
            tmem_st16(trow + kColS + kBN * s, pk);
            tmem_st16(trow + kColS + kBN * s + 16u, pk + 16);
            tmem_wait_st();
          }
        }
        if (in_tree || (tile + 1) * kBN > sg.len) {
          // values that some row may not see: zero them in place before the product reads the tile
          const uint32_t ld = rb + ring_v(j, sg.nj), st = ld % kStages;
          ok = ok && mbar_wait_warp(&full[st], (ld / kStages) & 1, ab);
          if (ok) {
            uint8_t* vt = ring + st * kTileBytes;
            const int lim = in_tree ? 0 : sg.len - tile * kBN;
            for (int x = lim * (D / 8) + threadIdx.x; x < kBN * (D / 8); x += kRows) {
              const int vr = x / (D / 8), ch = x % (D / 8);
              uint4* at = reinterpret_cast<uint4*>(vt + (ch >> 3) * (kBN * 128) + sw128_off(vr, ch & 7));
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (in_tree && tree.mask[vr] != 0ull) {
                const uint4 u = *at;
                v = make_uint4(finite_only(u.x), finite_only(u.y), finite_only(u.z), finite_only(u.w));
                if (((u.x ^ v.x) | (u.y ^ v.y) | (u.z ^ v.z) | (u.w ^ v.w)) == 0u) continue;
                atomicOr(&bad_v_s, 1ull << vr);
              }
              *at = v;
            }
            fence_proxy_async_smem();
          }
        }
        tc_fence_before();
        if (ok) mbar_arrive(&p_full[s]);
      }
      rb += 2 * sg.nj;
      gt += sg.nj;

      // ---- epilogue: O is complete once the last product is
      ok = ok && mbar_wait_warp(&pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, ab);
      tc_fence_after();
      named_bar_sync(1, kRows);  // bad_v_s is complete
      if (ok && warp_on) {
        const bool whole = sg.nj == sg.nt;
        const bool live = mask != 0ull;
        const unsigned long long bad = bad_v_s & mask;
        const int slot = ((worker * 2 + (first ? 0 : 1)) * p.m_tiles + mt) * p.slot_rows + r;
        const float inv_l = 1.0f / l;
        bf16* orow = a.out + (tok * a.H_q + h) * D;
        float* prow = p.part_o + static_cast<long long>(slot) * D;
        if (!whole && live) p.part_ml[slot] = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(trow + kColO + 32u * c, o);
          tmem_wait_ld();
          if (valid) {
            for (unsigned long long b = bad; b; b &= b - 1) {  // a non-finite value of a node this row sees
              const int node = __ffsll(static_cast<long long>(b)) - 1;
              const uint4* src = reinterpret_cast<const uint4*>(
                  a.v_tree + (static_cast<long long>(sg.n) * a.T + node) * a.ld_vt + sg.kvh * D + 32 * c);
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float x[8];
                unpack8(src[u], x);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!isfinite(x[e])) o[8 * u + e] += x[e];
              }
            }
            if (whole) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = live ? o[8 * u + e] * inv_l : 0.f;
                if (a.g && live) {
                  float gf[8];
                  unpack8(reinterpret_cast<const uint4*>(a.g + tok * a.ld_g + static_cast<long long>(h) * D + 32 * c)[u], gf);
#pragma unroll
                  for (int e = 0; e < 8; ++e) y[e] = y[e] / (1.0f + __expf(-gf[e]));
                }
                reinterpret_cast<uint4*>(orow + 32 * c)[u] =
                    make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
              }
            } else if (live) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                reinterpret_cast<float4*>(prow + 32 * c)[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTaWarpMma) tmem_dealloc<512>(tbase);
}

// Joins the partial results of the units that were cut: o = sum_i o_i 2^{m_i - M} / sum_i l_i 2^{m_i - M} over the
// workers i that share a unit, in their order.  CTA (row group, KV head, sequence): a warp per row, a lane D / 32
// dims.  It also writes the zero rows of sequences whose length is out of range, and reports them.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 16;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attention_tree_join_kernel(const __grid_constant__ TaParams p) {
  const AttnTreeParams& a = p.a;
  __shared__ long long chunk_s[kJoinThreads + 1];
  __shared__ int seq_s;
  __shared__ long long base_s;
  __shared__ Tree tree;
  const int n = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = a.cache_len[n], nt = unit_tiles(len, a.cap);
  constexpr int kPer = D / 32;
  if (nt > 0) {
    const long long total = locate(a.cache_len, a.N, a.cap, a.H_kv, 0, p.workers, n, chunk_s, &seq_s, &base_s);
    const long long u0 = base_s + static_cast<long long>(kvh) * nt, u1 = u0 + nt;
    const int w0 = share_owner(total, u0, p.workers), w1 = share_owner(total, u1 - 1, p.workers);
    if (w0 == w1) return;  // one worker had the whole unit and wrote it
    if (warp == 0) tree_load(tree, a.parent, n, a.T, nullptr);
    __syncthreads();
    // worker w0's piece is its first when its share begins with this unit, else its last
    const int first0 = share_begin(total, w0, p.workers) == u0 ? 0 : 1;
    for (int i = warp; i < kJoinRows; i += kJoinThreads / 32) {
      const int row = blockIdx.x * kJoinRows + i;
      if (row >= a.T * p.G) break;
      const int t = row / p.G, h = kvh * p.G + row % p.G, mt = row / kRows, r = row % kRows;
      const long long tok = static_cast<long long>(n) * a.T + t;
      bf16* dst = a.out + (tok * a.H_q + h) * D + lane * kPer;
      float y[kPer];
#pragma unroll
      for (int e = 0; e < kPer; ++e) y[e] = 0.f;
      if (tree.mask[t] != 0ull) {
        auto slot_of = [&](int w) { return ((w * 2 + (w == w0 ? first0 : 0)) * p.m_tiles + mt) * p.slot_rows + r; };
        float M = -INFINITY;
        for (int w = w0 + lane; w <= w1; w += 32) M = fmaxf(M, p.part_ml[slot_of(w)].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float L = 0.f;
        for (int w = w0; w <= w1; ++w) {
          const int slot = slot_of(w);
          const float2 ml = p.part_ml[slot];
          const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
          const float4* src = reinterpret_cast<const float4*>(p.part_o + static_cast<long long>(slot) * D + lane * kPer);
          L = fmaf(ml.y, f, L);
#pragma unroll
          for (int e = 0; e < kPer / 4; ++e) {
            const float4 v = src[e];
            y[4 * e] = fmaf(v.x, f, y[4 * e]);
            y[4 * e + 1] = fmaf(v.y, f, y[4 * e + 1]);
            y[4 * e + 2] = fmaf(v.z, f, y[4 * e + 2]);
            y[4 * e + 3] = fmaf(v.w, f, y[4 * e + 3]);
          }
        }
        const float inv = 1.0f / L;
        const bf16* g = a.g ? a.g + tok * a.ld_g + static_cast<long long>(h) * D + lane * kPer : nullptr;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          y[e] *= inv;
          if (g) y[e] = y[e] / (1.0f + __expf(-__bfloat162float(g[e])));
        }
      }
#pragma unroll
      for (int e = 0; e < kPer; e += 4)
        *reinterpret_cast<uint2*>(dst + e) = make_uint2(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]));
    }
    return;
  }
  if (threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0 && a.err) atomicOr(a.err, kDevErrCacheLen);
  for (int i = warp; i < kJoinRows; i += kJoinThreads / 32) {
    const int row = blockIdx.x * kJoinRows + i;
    if (row >= a.T * p.G) break;
    const long long tok = static_cast<long long>(n) * a.T + row / p.G;
    bf16* dst = a.out + (tok * a.H_q + kvh * p.G + row % p.G) * D + lane * kPer;
#pragma unroll
    for (int e = 0; e < kPer; e += 4) *reinterpret_cast<uint2*>(dst + e) = make_uint2(0u, 0u);
  }
}

// bf16 rows of `cols` elements, `rows` of them for each of `outer` sequences, as 64 x 64 boxes with the 128-byte
// swizzle; rows past the sequence's last read as zeros
bool encode_rows(CUtensorMap* map, const void* base, long long cols, long long rows, long long outer, long long row_el,
                 long long outer_el) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      fn = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_el) * 2, static_cast<cuuint64_t>(outer_el) * 2};
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(kBN), 1u};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const AttnTreeParams& a, cudaStream_t stream) {
  TaParams p;
  p.a = a;
  p.G = a.H_q / a.H_kv;
  p.m_tiles = attn_m_tiles(p.G, a.T);
  p.workers = attn_workers(p.m_tiles);
  p.slot_rows = attn_slot_rows(p.G, a.T);
  p.scale_log2e = a.scale * 1.4426950408889634f;
  const size_t slots = static_cast<size_t>(p.workers) * 2 * p.m_tiles * p.slot_rows;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + slots * D);
  const long long wk = static_cast<long long>(a.H_kv) * D;
  CUtensorMap kc, vc, kt, vt;
  if (!encode_rows(&kc, a.k_cache, wk, a.cap, a.N, wk, wk * a.cap) ||
      !encode_rows(&vc, a.v_cache, wk, a.cap, a.N, wk, wk * a.cap) ||
      !encode_rows(&kt, a.k_tree, wk, a.T, a.N, a.ld_kt, a.ld_kt * a.T) ||
      !encode_rows(&vt, a.v_tree, wk, a.T, a.N, a.ld_vt, a.ld_vt * a.T))
    return cudaErrorInvalidValue;
  constexpr int smem = kRingBytes + 1024;
  cudaError_t e = cudaFuncSetAttribute(attention_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  attention_tree_kernel<D><<<dim3(p.m_tiles, p.workers), kTaThreads, smem, stream>>>(kc, vc, kt, vt, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int groups = (a.T * p.G + kJoinRows - 1) / kJoinRows;
  attention_tree_join_kernel<D><<<dim3(groups, a.H_kv, a.N), kJoinThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t attention_tree_workspace(int H_q, int H_kv, int D, int, int T) {
  const int G = H_q / H_kv, m_tiles = attn_m_tiles(G, T);
  const size_t slots = static_cast<size_t>(attn_workers(m_tiles)) * 2 * m_tiles * attn_slot_rows(G, T);
  return slots * (static_cast<size_t>(D) + 2) * sizeof(float);
}

cudaError_t launch_attention_tree(const AttnTreeParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  return p.D == 256 ? launch_d<256>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace gdn
