// gdn_attention_tree: attention of a tree's nodes over a KV cache and their ancestors.
//
// For sequence n and KV head kvh, the T nodes times the G query heads that share kvh are T G query
// rows (row t G + g), all over the same keys: cache_len[n] cache rows, then the T nodes' own.  With
//   s_rj = scale q_r . k_j,  m_r = max_j s_rj,  o_r = sum_j e^{s_rj - m_r} v_j / sum_j e^{s_rj - m_r}
// over the keys row r sees, the keys are taken once, in tiles of 128, with a running maximum and sum.
//
// Work split.  A unit is one (sequence, KV head): its tiles are ceil(cache_len / 128) tiles of the cache and
// one tile of the tree (64 keys).  The tiles of all units in a row, each unit's preceded by what its beginning and
// end cost (kUnitCost), are cut into W equal shares, one per worker, so that ragged lengths balance and a single long
// sequence still fills the GPU; a unit cut between workers leaves partial (o, m, l) that a second kernel joins.  Rows beyond
// 128 go to further CTAs (blockIdx.x) of the same worker, which read the same tiles at about the same time, from L2.
//
// A CTA: warps 0-7 softmax and epilogue (thread = query row = TMEM lane; warps w and w + 4 share a row's
// 128 scores and O's D columns in halves), warp 8 TMA, warp 9 tcgen05.mma.  TMEM: O (D columns) | S in two buffers of
// 128.  Shared memory: Q, and a ring of slots of 64 D elements (5 of 32 KiB at D = 256, 12 of 16 KiB at D = 128), which hold
// half a K tile (128 keys x D / 2 dims) or half a V tile (64 keys x D) and are refilled as soon as their own products
// have read them.  Per tile j
//   S_j = Q K_j^T (M 128, N 128, K = D), P_j = exp2(S_j c - m) as bf16 over S_j's first 64 columns,
//   O += P_j V_j (M 128, N = D, K 128, A = P from TMEM, V MN-major),
// with S_{j+1} issued before P_j is awaited.  O and l are rescaled only when a row's maximum has grown by more than
// 2^8; the final division by l makes the result the same.  Tiles of 64 keys with Q in TMEM (a ring of six 32 KiB tiles) took
// 2450 cycles per 64 keys: an N = 64 product runs at 45 cycles per K step instead of 32, and the latency of the
// S -> softmax -> P V round trip is paid twice as often.  The next unit's Q is fetched and its first S issued while
// this one's epilogue runs.
//
// Measured (B200, 24 / 4 heads of 256, in a graph): one sequence of 262,144 keys x 64 nodes 368 - 372 us after a pause (1.12
// PFLOP/s), 380 - 428 us in a long run, when the power cap holds the SM clock at 1.46 GHz; of a tile's 3200 cycles shared memory takes 2500 (64
// KB of Q, 64 + 64 KB of K and V read and 128 KB written), the products 2050, the rest is not explained.  64 ragged sequences of up to 8192
// keys x 16 nodes 230 us (5.4 TB/s over all, HBM's rate while tiles stream; 249 us in a long run at 1.43 GHz), x 1 node 197 us (6140
// GB/s); one token of 777 keys 15 us.
//
// P enters the products as bf16, within 2^-8, like the prefill attention's: a pair hi + lo would double the P V products, and the
// error against 64 bits (0.0023 of the output, 0.0017 of it the output's own rounding) does not call for it.
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

constexpr int kBN = 128;             // keys per tile of the cache
constexpr int kBT = kMaxNodes;       // keys of the tree's tile
constexpr int kRows = 128;           // query rows per CTA
constexpr int kSoftmax = 256;        // threads of the softmax warps
constexpr int kTaThreads = kSoftmax + 64;
constexpr int kTaWarpTma = 8, kTaWarpMma = 9;
constexpr int kTaSms = 148;          // CTAs of the launch: one per SM of the part
constexpr float kRescale = 8.0f;     // log2 units

__host__ __device__ inline int attn_m_tiles(int G, int T) { return (T * G + kRows - 1) / kRows; }
__host__ __device__ inline int attn_workers(int m_tiles) { return kTaSms / m_tiles; }
__host__ __device__ inline int attn_slot_rows(int G, int T) { return T * G < kRows ? T * G : kRows; }

struct TaParams {
  AttnTreeParams a;
  int G, m_tiles, workers, slot_rows;
  float scale_log2e;
  float4* part_o;   // [workers][2][m_tiles][D / 4][slot_rows]: rows side by side, as the lanes that write and read them
  float2* part_ml;  // [workers][2][m_tiles][slot_rows]: maximum (log2 units) and sum; an absent node's: -inf, -1 (no sum is negative)
  int4* cut;        // [workers]: the unit that begins in a worker's share and ends in a later one's: sequence
                    // (-1: none), KV head, which of the worker's partials, the last worker
};

// tiles of one unit of sequence n: 0 when its length is out of range
__device__ __forceinline__ int unit_tiles(int len, int cap) {
  return len < 0 || len > cap ? 0 : (len + kBN - 1) / kBN + 1;
}

// What a unit counts in the shares: its tiles and, before them, the time that its beginning and end cost, in tiles: loads that
// wait behind the tiles' copies (gate, tree, the next Q), the epilogue, the first products.  Without it the workers that get many
// short units end last (64 ragged sequences x 16 nodes: 280 us at a cost of 0 tiles, 264 at 2, 249 at 4, 236 at 6, 226 at 8 and 10, 227 at
// 16; x 64 nodes 623 at 0, 500 at 8; one sequence of 32,768 keys x 21 nodes 59 and 53; equal lengths and heads of 128: 2% or less from 6 on).
constexpr int kUnitCost = 8;
__device__ __forceinline__ int unit_weight(int len, int cap) {
  const int nt = unit_tiles(len, cap);
  return nt > 0 ? nt + kUnitCost : 0;
}

// the first position of worker w's share
__device__ __forceinline__ long long share_begin(long long total, int w, int workers) {
  return total / workers * w + min(total % workers, static_cast<long long>(w));
}

// the worker that takes position x
__device__ __forceinline__ int share_owner(long long total, long long x, int workers) {
  const long long q = total / workers, r = total % workers;
  return static_cast<int>(x < r * (q + 1) ? x / (q + 1) : r + (x - r * (q + 1)) / q);
}

// Where worker w's share begins: sums the units' tiles over the sequences.  Every thread of the block calls it;
// `chunk_s` has room for blockDim.x + 1 sums.  Returns the total number of tiles; *seq, *base: the sequence and the
// tile number its first unit begins at (seq = N for an empty share).
__device__ long long locate(const int* cache_len, int N, int cap, int H_kv, int w, int workers, long long* chunk_s,
                            int* seq_s, long long* base_s) {
  const int tid = threadIdx.x, n_thr = blockDim.x;
  const int per = (N + n_thr - 1) / n_thr;
  const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
  long long sum = 0;
  for (int n = n0; n < n1; ++n) sum += unit_weight(cache_len[n], cap);
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
  const long long x = share_begin(total, w, workers);
  long long at = chunk_s[tid];
  for (int n = n0; n < n1; ++n) {
    const long long next = at + static_cast<long long>(unit_weight(cache_len[n], cap)) * H_kv;
    if (at <= x && x < next) {
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

// the largest of three, NaN left out
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
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

// D[tmem] (+)= A B^T, A in tensor or shared memory, descriptors given as halves: the high half is constant for a layout
// and the low one starts with the address / 16, so that a step costs the issuing thread one addition.
template <bool kAccumulate>
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t desc_lo, uint32_t desc_hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(desc_lo), "r"(desc_hi), "r"(idesc), "n"(kAccumulate ? 1 : 0)
      : "memory");
}

template <bool kAccumulate>
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(kAccumulate ? 1 : 0)
      : "memory");
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
      const int len = cache_len[seq], w = unit_weight(len, cap);
      const long long off = x - base;
      if (off >= static_cast<long long>(w) * H_kv) {
        base += static_cast<long long>(w) * H_kv;
        ++seq;
        continue;
      }
      s.n = seq;
      s.len = len;
      s.nt = w - kUnitCost;
      s.kvh = static_cast<int>(off / w);
      const int at = static_cast<int>(off % w), n = static_cast<int>(min(static_cast<long long>(w - at), end - x));
      s.t0 = max(at - kUnitCost, 0);
      s.nj = max(at + n - kUnitCost, 0) - s.t0;
      x += n;
      if (s.nj > 0) return true;  // (else the share ends before the unit's first tile)
    }
    return false;
  }
};

// Positions in the ring, in slots since the segment's first: K_0, K_1, V_0, K_2, V_1, .. , V_{nj-1}, two slots each, the
// order in which the products take them; the tree's V has one slot.
__device__ __forceinline__ uint32_t ring_k(int j) { return j == 0 ? 0 : 4 * j - 2; }
__device__ __forceinline__ uint32_t ring_v(int j, int nj) { return j < nj - 1 ? 4 * j + 4 : 4 * nj - 2; }

template <int D>
struct TaCfg {
  static constexpr int kQBytes = kRows * D * 2;      // blocks of 64 dims x 128 rows
  static constexpr int kSlotBytes = 64 * D * 2;
  static constexpr int kSlots = (D == 256 ? 160 : 192) * 1024 / kSlotBytes;
  static constexpr uint32_t kColO = 0, kColS = D;    // tensor memory
};

template <int D>
struct TaShared {
  uint64_t full[TaCfg<D>::kSlots], empty[TaCfg<D>::kSlots], s_full[2], p_full[2], pv_done[2], q_full, drain;
  long long base, total;
  unsigned long long bad_v;              // nodes whose values here are not all finite
  unsigned long long mask[kMaxNodes];    // the tree of the current sequence
  union {
    Tree tree;                           // while the masks are formed
    float red[2][kRows];                 // partial row maxima (at the end sums), per column half
  };
  uint32_t tmem;
  int abort, seq;
};

template <int D>
constexpr int kTaSmem = TaCfg<D>::kQBytes + TaCfg<D>::kSlots * TaCfg<D>::kSlotBytes + static_cast<int>(sizeof(TaShared<D>)) + 1023;
static_assert(kTaSmem<256> <= 232448 && kTaSmem<128> <= 232448, "shared memory of an SM");

template <int D>
__global__ void __launch_bounds__(kTaThreads, 1)
    attention_tree_kernel(const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
                          const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt,
                          const __grid_constant__ TaParams p) {
  using C = TaCfg<D>;
  constexpr uint32_t kSlots = C::kSlots;
  extern __shared__ uint8_t ta_smem[];
  uint8_t* q_sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(ta_smem) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = q_sm + C::kQBytes;
  TaShared<D>& sh = *reinterpret_cast<TaShared<D>*>(ring + kSlots * C::kSlotBytes);
  const AttnTreeParams& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = blockIdx.x, worker = blockIdx.y;

  const Abort ab{a.err, &sh.abort};
  if (threadIdx.x == 32 * kTaWarpTma) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_kc) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_vc) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_kt) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&tm_vt) : "memory");
  }
  if (threadIdx.x == 0) {
    sh.abort = 0;
    for (uint32_t i = 0; i < kSlots; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.s_full[b], 1);
      mbar_init(&sh.p_full[b], kSoftmax);
      mbar_init(&sh.pv_done[b], 1);
    }
    mbar_init(&sh.q_full, kSoftmax);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == kTaWarpMma) tmem_alloc<512>(&sh.tmem);
  asm volatile("griddepcontrol.launch_dependents;");  // the join may be brought up; it waits for this grid's end
  const long long total = locate(a.cache_len, a.N, a.cap, a.H_kv, worker, p.workers,
                                 reinterpret_cast<long long*>(q_sm), &sh.seq, &sh.base);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sh.tmem;
  if (threadIdx.x == 0) sh.total = total;  // for this thread
  Walk walk{a.cache_len, a.cap, a.H_kv, a.N, sh.seq, sh.base, share_begin(total, worker, p.workers),
            share_begin(total, worker + 1, p.workers)};
  Segment sg;

  if (warp == kTaWarpTma) {
    if (lane == 0) {
      // ------------------------------------------------ loads, in the order of use
      uint32_t st = 0, use = 0, n_loads = 0;  // slot, times round the ring
      bool ok = true;
      // a slot's load: false once a wait has given up
      auto load = [&](const CUtensorMap* map, int x, int boxes, int box_rows, int row, int n, int stride) -> bool {
        if (use > 0 && !mbar_wait(&sh.empty[st], (use - 1) & 1, ab)) return false;
        mbar_arrive_expect_tx(&sh.full[st], static_cast<uint32_t>(boxes * box_rows * 128));
        for (int i = 0; i < boxes; ++i)
          tma_load_3d(ring + st * C::kSlotBytes + i * stride, map, x + 64 * i, row, n, &sh.full[st]);
        ++n_loads;
        if (++st == kSlots) {
          st = 0;
          ++use;
        }
        return true;
      };
      while (ok && walk.next(sg)) {
        const int x0 = sg.kvh * D;
        auto load_k = [&](int j) {
          const bool in_tree = sg.t0 + j == sg.nt - 1;
          for (int i = 0; i < 2 && ok; ++i)
            ok = in_tree ? load(&tm_kt, x0 + i * (D / 2), D / 128, kBT, 0, sg.n, kBN * 128)
                         : load(&tm_kc, x0 + i * (D / 2), D / 128, kBN, (sg.t0 + j) * kBN, sg.n, kBN * 128);
        };
        auto load_v = [&](int j) {
          const bool in_tree = sg.t0 + j == sg.nt - 1;
          if (in_tree) {
            if (ok) ok = load(&tm_vt, x0, D / 64, kBT, 0, sg.n, 64 * 128);
          } else {
            for (int i = 0; i < 2 && ok; ++i)
              ok = load(&tm_vc, x0, D / 64, 64, (sg.t0 + j) * kBN + 64 * i, sg.n, 64 * 128);
          }
        };
        for (int j = 0; j < sg.nj; ++j) {
          load_k(j);
          if (j > 0) load_v(j - 1);
        }
        load_v(sg.nj - 1);
      }
      // copies still in flight (only after an abort) land before the CTA exits
      int drain_flag = 0;
      const Abort drain{nullptr, &drain_flag};
      for (uint32_t k = n_loads > kSlots ? n_loads - kSlots : 0; k < n_loads; ++k)
        mbar_wait(&sh.full[k % kSlots], (k / kSlots) & 1, drain);
    }
  } else if (warp == kTaWarpMma) {
    if (lane == 0) {
      // ------------------------------------------------ products
      const uint32_t idesc_s = idesc_bf16(kRows, kBN, false, false), idesc_st = idesc_bf16(kRows, kBT, false, false);
      const uint32_t idesc_o = idesc_bf16(kRows, D, false, true);
      // K-major operands: rows of 128 B, 8-row groups 1 KiB apart; V MN-major: 64-wide blocks of d 8 KiB apart
      const uint64_t q_desc = smem_desc(smem_u32(q_sm), 16, 1024, Swz::k128);
      const uint64_t v_desc = smem_desc(smem_u32(ring), 64 * 128, 1024, Swz::k128);
      const uint32_t q_lo = static_cast<uint32_t>(q_desc), k_hi = static_cast<uint32_t>(q_desc >> 32);
      const uint32_t k_lo = q_lo + C::kQBytes / 16;
      const uint32_t v_lo = static_cast<uint32_t>(v_desc), v_hi = static_cast<uint32_t>(v_desc >> 32);
      uint32_t st = 0, use = 0;  // the next slot to be read, times round the ring
      uint32_t gt = 0;           // tiles before this segment
      bool ok = true;
      auto slot_wait = [&]() { return mbar_wait(&sh.full[st], use & 1, ab); };
      auto slot_next = [&]() {
        umma_commit(&sh.empty[st]);
        if (++st == kSlots) {
          st = 0;
          ++use;
        }
      };
      for (uint32_t seg = 0; ok && walk.next(sg); ++seg) {
        if (!mbar_wait(&sh.q_full, seg & 1, ab)) break;
        auto issue_pv = [&](int j) -> bool {  // O += P_j V_j
          const uint32_t t = gt + j;
          const int halves = sg.t0 + j == sg.nt - 1 ? 1 : 2;
          if (!mbar_wait(&sh.p_full[t & 1], (t >> 1) & 1, ab)) return false;
          for (int i = 0; i < halves; ++i) {
            if (!slot_wait()) return false;
            tc_fence_after();
            const uint32_t pa = tbase + C::kColS + kBN * (t & 1) + 32u * i, b = v_lo + st * (C::kSlotBytes / 16);
            if (j > 0 || i > 0) umma_ts<true>(tbase + C::kColO, pa, b, v_hi, idesc_o);
            else umma_ts<false>(tbase + C::kColO, pa, b, v_hi, idesc_o);
#pragma unroll
            for (int ks = 1; ks < 4; ++ks) umma_ts<true>(tbase + C::kColO, pa + 8u * ks, b + ks * 128u, v_hi, idesc_o);
            slot_next();
          }
          umma_commit(&sh.pv_done[t & 1]);
          return true;
        };
        for (int j = 0; j < sg.nj; ++j) {
          const uint32_t t = gt + j, s = t & 1;
          const uint32_t idesc = sg.t0 + j == sg.nt - 1 ? idesc_st : idesc_s;
          // S buffer s held P of two tiles before: its product must have read it
          ok = t < 2 || mbar_wait(&sh.pv_done[s], ((t - 2) >> 1) & 1, ab);
          for (int i = 0; i < 2 && ok; ++i) {  // the two halves of the dims
            if (!(ok = slot_wait())) break;
            tc_fence_after();
            const uint32_t qa = q_lo + i * (C::kQBytes / 32), b = k_lo + st * (C::kSlotBytes / 16);
            if (i > 0) umma_ss<true>(tbase + C::kColS + kBN * s, qa, b, k_hi, idesc);
            else umma_ss<false>(tbase + C::kColS + kBN * s, qa, b, k_hi, idesc);
#pragma unroll
            for (int ks = 1; ks < D / 32; ++ks)
              umma_ss<true>(tbase + C::kColS + kBN * s, qa + (ks >> 2) * (kRows * 8u) + (ks & 3) * 2u,
                            b + (ks >> 2) * (kBN * 8u) + (ks & 3) * 2u, k_hi, idesc);
            slot_next();
          }
          if (!ok) break;
          umma_commit(&sh.s_full[s]);
          if (j >= 1 && !(ok = issue_pv(j - 1))) break;
        }
        if (ok) ok = issue_pv(sg.nj - 1);
        gt += sg.nj;
      }
      umma_commit(&sh.drain);
      int drain_flag = 0;
      const Abort drain{nullptr, &drain_flag};
      mbar_wait(&sh.drain, 0, drain);
    }
  } else {
    // ------------------------------------------------ softmax and epilogue: thread = query row, column half hc
    const int q4 = warp & 3, hc = warp >> 2;
    const int r = 32 * q4 + lane, row = mt * kRows + r;
    const int t = row / p.G;                                // the row's node
    const bool valid = row < a.T * p.G;
    const bool warp_on = mt * kRows + 32 * q4 < a.T * p.G;  // some row of this warp
    const uint32_t trow = tmem_addr(tbase, 32 * q4, 0);
    uint32_t rb = 0, gt = 0;  // slots and tiles before this segment
    int tree_of = -1;
    // the segment's Q rows into shared memory; rows past the last node's are left as they are (no row reads another's)
    auto fetch_q = [&](const Segment& s) {
      const int rows = min(kRows, a.T * p.G - mt * kRows);
      for (int x = threadIdx.x; x < rows * (D / 8); x += kSoftmax) {
        const int i = x / (D / 8), ch = x % (D / 8), gr = mt * kRows + i;
        const bf16* src = a.q + (static_cast<long long>(s.n) * a.T + gr / p.G) * a.ld_q +
                          static_cast<long long>(s.kvh * p.G + gr % p.G) * D + 8 * ch;
        cp_async16(q_sm + (ch >> 3) * (kRows * 128) + sw128_off(i, ch & 7), src);
      }
      cp_async_commit();
    };
    auto publish_q = [&]() {
      cp_async_wait_all();
      fence_proxy_async_smem();
      mbar_arrive(&sh.q_full);
    };
    // no early exit: the warps meet at named barriers, so after a failed wait a warp keeps its place in the
    // loops and only skips its tensor-memory work
    bool ok = true, have = walk.next(sg);
    if (have) fetch_q(sg);
    if (threadIdx.x == 0 && mt == 0) p.cut[worker] = make_int4(-1, 0, 0, 0);
    // sequences whose length is out of range have no tiles: their rows are zeros
    for (int n = worker; n < a.N && mt == 0; n += p.workers) {
      if (unit_tiles(a.cache_len[n], a.cap) > 0) continue;
      if (threadIdx.x == 0 && a.err) atomicOr(a.err, kDevErrCacheLen);
      uint4* dst = reinterpret_cast<uint4*>(a.out + static_cast<long long>(n) * a.T * a.H_q * D);
      for (int x = threadIdx.x; x < a.T * a.H_q * (D / 8); x += kSoftmax) dst[x] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (have) publish_q();
    for (bool first = true; have; first = false) {
      const int h = sg.kvh * p.G + row % p.G;
      const long long tok = static_cast<long long>(sg.n) * a.T + t;
      if (!first) named_bar_sync(1, kSoftmax);  // all have done with the last segment's masks, sums and bad_v
      if (tree_of != sg.n) {  // the tree of this sequence, while the first tiles load
        tree_of = sg.n;
        if (warp == 0) {
          tree_load(sh.tree, a.parent, sg.n, a.T, mt == 0 && sg.kvh == 0 && sg.t0 == 0 ? a.err : nullptr);
          sh.mask[lane] = sh.tree.mask[lane];
          sh.mask[lane + 32] = sh.tree.mask[lane + 32];
        }
      }
      if (threadIdx.x == 0) sh.bad_v = 0ull;
      named_bar_sync(1, kSoftmax);
      const unsigned long long mask = valid ? sh.mask[t] : 0ull;

      float m = -INFINITY, l = 0.f;  // l: this half's partial sum
      for (int j = 0; j < sg.nj; ++j) {
        const uint32_t tl = gt + j, s = tl & 1;
        const int tile = sg.t0 + j;
        const bool in_tree = tile == sg.nt - 1;
        const int lim = in_tree ? 0 : sg.len - tile * kBN;  // keys of this tile in the cache
        ok = ok && mbar_wait_warp(&sh.s_full[s], (tl >> 1) & 1, ab);
        tc_fence_after();
        if (warp_on) {
          constexpr int kHalf = kBN / 2;
          const bool here = !(in_tree && hc == 1);  // the tree's tile has no second half
          float sv[kHalf];
          float mraw = -INFINITY;
          if (here) {
            if (ok) {
              tmem_ld32(trow + C::kColS + kBN * s + kHalf * hc, sv);
              tmem_ld32(trow + C::kColS + kBN * s + kHalf * hc + 32u, sv + 32);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int c = 0; c < kHalf; ++c) sv[c] = 0.f;
            }
            if (in_tree) {
#pragma unroll
              for (int c = 0; c < kHalf; ++c) sv[c] = (mask >> c) & 1 ? sv[c] : -INFINITY;
            } else if (lim < kBN) {
#pragma unroll
              for (int c = 0; c < kHalf; ++c) sv[c] = kHalf * hc + c < lim ? sv[c] : -INFINITY;
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx[c] = max3(sv[3 * c], sv[3 * c + 1], sv[3 * c + 2]);
#pragma unroll
            for (int c = 12; c + 1 < kHalf; c += 2) mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], sv[c], sv[c + 1]);
            mraw = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
          }
          // the row's maximum from both halves; both have read their scores before either writes P over them
          sh.red[hc][r] = mraw;
          named_bar_sync(2 + q4, 64);
          const float mloc = fmaxf(mraw, sh.red[hc ^ 1][r]) * p.scale_log2e;
          named_bar_sync(2 + q4, 64);
          // per warp (the wait and the tensor-memory accesses are warp-collective); both warps of a row see
          // the same maxima and decide alike
          const bool grow = mloc > m + kRescale || (m == -INFINITY && mloc > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mloc : m;
            if (j >= 1) {
              ok = ok && mbar_wait_warp(&sh.pv_done[(tl - 1) & 1], ((tl - 1) >> 1) & 1, ab);
              if (ok) {
                tc_fence_after();
                const float f = grow ? ex2(m - m_new) : 1.f;
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                  float o[32];
                  tmem_ld32(trow + C::kColO + (D / 2) * hc + 32u * c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] *= f;
                  tmem_st32(trow + C::kColO + (D / 2) * hc + 32u * c, o);
                }
                tmem_wait_st();  // (the tree's tile has no P of the second half to wait for)
                l *= f;
              }
            }
            m = m_new;
          }
          if (here) {
            const float m_use = m == -INFINITY ? 0.f : m;  // nothing seen yet: every score is -inf
            uint32_t pk[kHalf / 2];
            float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            const float2 c2 = make_float2(p.scale_log2e, p.scale_log2e), m2 = make_float2(-m_use, -m_use);
#pragma unroll
            for (int c = 0; c < kHalf / 2; ++c) {
              const float2 x = __ffma2_rn(make_float2(sv[2 * c], sv[2 * c + 1]), c2, m2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              ls[c & 1] = __fadd2_rn(ls[c & 1], e);
              pk[c] = pack_bf16x2(e.x, e.y);
            }
            l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
            if (ok) {
              tmem_st16(trow + C::kColS + kBN * s + 32u * hc, pk);
              tmem_st16(trow + C::kColS + kBN * s + 32u * hc + 16u, pk + 16);
              tmem_wait_st();
            }
          }
        }
        if (in_tree || lim < kBN) {
          // values that some row may not see: zero them in place before the product reads the tile.  A slot's wait tells its last
          // fill from the one two before by parity only, and the slot of V_j's second half held V_{j-1}'s first (ring of 5): that
          // must have been read, or the wait could end on the fill before and the wrong tile be zeroed.
          if (j >= 1) ok = ok && mbar_wait_warp(&sh.pv_done[(tl - 1) & 1], ((tl - 1) >> 1) & 1, ab);
          const uint32_t ld = rb + ring_v(j, sg.nj);
          for (int i = 0; i < (in_tree ? 1 : 2); ++i) {
            const uint32_t st = (ld + i) % kSlots;
            ok = ok && mbar_wait_warp(&sh.full[st], ((ld + i) / kSlots) & 1, ab);
            if (!ok) break;
            uint8_t* vt = ring + st * C::kSlotBytes;
            for (int x = max(0, lim - 64 * i) * (D / 8) + threadIdx.x; x < 64 * (D / 8); x += kSoftmax) {
              const int vr = x / (D / 8), ch = x % (D / 8);
              uint4* at = reinterpret_cast<uint4*>(vt + (ch >> 3) * (64 * 128) + sw128_off(vr, ch & 7));
              uint4 v = make_uint4(0u, 0u, 0u, 0u);
              if (in_tree && sh.mask[vr] != 0ull) {
                const uint4 u = *at;
                v = make_uint4(finite_only(u.x), finite_only(u.y), finite_only(u.z), finite_only(u.w));
                if (((u.x ^ v.x) | (u.y ^ v.y) | (u.z ^ v.z) | (u.w ^ v.w)) == 0u) continue;
                atomicOr(&sh.bad_v, 1ull << vr);
              }
              *at = v;
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        if (ok) mbar_arrive(&sh.p_full[s]);
      }
      const bool tree_end = sg.t0 + sg.nj == sg.nt;
      rb += 4 * sg.nj - (tree_end ? 1 : 0);
      gt += sg.nj;

      // ---- every S of this segment has been read: the next one's Q may take its place, and its first S run beside
      // the epilogue
      if (sg.t0 == 0 && !tree_end)  // the unit goes on in later shares
        if (threadIdx.x == 0 && mt == 0)
          p.cut[worker] = make_int4(sg.n, sg.kvh, first ? 0 : 1, share_owner(sh.total, walk.x - 1 + (sg.nt - sg.nj), p.workers));
      Segment nx;
      have = walk.next(nx);
      if (have) fetch_q(nx);
      const bool whole = sg.nj == sg.nt;
      const bool live = mask != 0ull;
      const int d0 = (D / 2) * hc;
      // the gate of this row's half, 32 dims ahead of their use
      const bool gated = whole && live && a.g != nullptr;
      const uint4* grow = reinterpret_cast<const uint4*>(a.g + (gated ? tok * a.ld_g + static_cast<long long>(h) * D + d0 : 0));
      uint4 gv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) gv[u] = gated ? grow[u] : make_uint4(0u, 0u, 0u, 0u);
      // O is complete once the last product is
      ok = ok && mbar_wait_warp(&sh.pv_done[(gt - 1) & 1], ((gt - 1) >> 1) & 1, ab);
      if (have) publish_q();
      tc_fence_after();
      if (warp_on) sh.red[hc][r] = l;
      named_bar_sync(1, kSoftmax);  // both halves' sums; bad_v is complete
      if (ok && warp_on) {
        const float l_row = l + sh.red[hc ^ 1][r];
        const unsigned long long bad = sh.bad_v & mask;
        const int slot = (worker * 2 + (first ? 0 : 1)) * p.m_tiles + mt;
        const float inv_l = 1.0f / l_row;
        if (!whole && valid && hc == 0) p.part_ml[slot * p.slot_rows + r] = live ? make_float2(m, l_row) : make_float2(-INFINITY, -1.f);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float o[32];
          tmem_ld32(trow + C::kColO + d0 + 32u * c, o);
          tmem_wait_ld();
          for (unsigned long long b = bad; b; b &= b - 1) {  // a non-finite value of a node this row sees
            const int node = __ffsll(static_cast<long long>(b)) - 1;
            const uint4* src = reinterpret_cast<const uint4*>(
                a.v_tree + (static_cast<long long>(sg.n) * a.T + node) * a.ld_vt + sg.kvh * D + d0 + 32 * c);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float x[8];
              unpack8(src[u], x);
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (!isfinite(x[e])) o[8 * u + e] += x[e];
            }
          }
          __syncwarp();
          if (whole && valid) {
            bf16* orow = a.out + (tok * a.H_q + h) * D + d0 + 32 * c;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              float y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = live ? o[8 * u + e] * inv_l : 0.f;
              if (gated) {
                float gf[8];
                unpack8(gv[u], gf);
                if (c + 1 < D / 64) gv[u] = grow[4 * (c + 1) + u];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __fdividef(y[e], 1.0f + __expf(-gf[e]));
              }
              reinterpret_cast<uint4*>(orow)[u] =
                  make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            }
          } else if (!whole && live) {
            float4* dst = p.part_o + (static_cast<long long>(slot) * (D / 4) + d0 / 4 + 8 * c) * p.slot_rows + r;
#pragma unroll
            for (int u = 0; u < 8; ++u)
              dst[static_cast<long long>(u) * p.slot_rows] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
          }
        }
      }
      tc_fence_before();
      sg = nx;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kTaWarpMma) tmem_dealloc<512>(tbase);
}

// Joins the partial results of the units that were cut: o = sum_i o_i 2^{m_i - M} / sum_i l_i 2^{m_i - M} over the
// workers i that share a unit, in their order, with a running maximum M.  CTA (rows and dims, worker, row tile): the unit that
// is cut at the end of that worker's share; a thread has 4 dims of a row, kFlight partials' loads in flight.  Rows run
// along the lanes, as the partials lie.  Bound by latency: 4 us of a small call, about 10 us where every worker's share cuts a unit.
// Four CTAs per SM: with the registers of three (76) the batch of 64 ragged sequences takes 248 us in all instead of 242.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 4) attention_tree_join_kernel(const __grid_constant__ TaParams p) {
  constexpr int kFlight = 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials and cuts are complete
  const AttnTreeParams& a = p.a;
  const int w0 = blockIdx.y, mt = blockIdx.z;
  const int4 cut = p.cut[w0];
  if (cut.x < 0) return;
  const int rows = min(kRows, a.T * p.G - mt * kRows);
  const int x = blockIdx.x * kJoinThreads + threadIdx.x, r = x % rows, c4 = x / rows;
  if (c4 >= D / 4) return;
  const int row = mt * kRows + r, h = cut.y * p.G + row % p.G, w1 = cut.w;
  const long long tok = static_cast<long long>(cut.x) * a.T + row / p.G;
  uint2 gate = make_uint2(0u, 0u);
  if (a.g) gate = reinterpret_cast<const uint2*>(a.g + tok * a.ld_g + static_cast<long long>(h) * D)[c4];
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  float M = -INFINITY, L = 0.f;
  bool live = true;
  for (int wb = w0; wb <= w1; wb += kFlight) {
    float2 ml[kFlight];
    float4 v[kFlight];
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      // worker w0's piece is its last (or only) one, the others' are their first
      const int w = min(wb + i, w1), slot = (w * 2 + (w == w0 ? cut.z : 0)) * p.m_tiles + mt;
      ml[i] = p.part_ml[slot * p.slot_rows + r];
      v[i] = p.part_o[(static_cast<long long>(slot) * (D / 4) + c4) * p.slot_rows + r];
    }
    live = !(ml[0].y < 0.f);
    if (!live) break;  // an absent node's row: its values were never written
    float top = M;
#pragma unroll
    for (int i = 0; i < kFlight; ++i) top = fmaxf(top, ml[i].x);
    // A piece whose scores are all NaN (or -inf) has no maximum either: its sum is NaN (or 0), and is taken like any other.
    const float at = top == -INFINITY ? 0.f : top;
    const float f0 = ex2(M - at);
    M = top;
    L *= f0;
    y = make_float4(y.x * f0, y.y * f0, y.z * f0, y.w * f0);
#pragma unroll
    for (int i = 0; i < kFlight; ++i) {
      if (wb + i > w1) break;
      const float f = ex2(ml[i].x - at);
      L = fmaf(ml[i].y, f, L);
      y = make_float4(fmaf(v[i].x, f, y.x), fmaf(v[i].y, f, y.y), fmaf(v[i].z, f, y.z), fmaf(v[i].w, f, y.w));
    }
  }
  uint2 out = make_uint2(0u, 0u);
  if (live) {
    const float inv = 1.0f / L;
    float o[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
    if (a.g) {
      o[0] = __fdividef(o[0], 1.0f + __expf(-bf16_lo(gate.x)));
      o[1] = __fdividef(o[1], 1.0f + __expf(-bf16_hi(gate.x)));
      o[2] = __fdividef(o[2], 1.0f + __expf(-bf16_lo(gate.y)));
      o[3] = __fdividef(o[3], 1.0f + __expf(-bf16_hi(gate.y)));
    }
    out = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
  }
  reinterpret_cast<uint2*>(a.out + (tok * a.H_q + h) * D)[c4] = out;
}

// bf16 rows of `cols` elements, `rows` of them for each of `outer` sequences, as boxes of 64 columns x box_rows with the
// 128-byte swizzle; rows past the sequence's last read as zeros
bool encode_rows(CUtensorMap* map, const void* base, long long cols, long long rows, long long outer, long long row_el,
                 long long outer_el, int box_rows) {
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
  const cuuint32_t box[3] = {64u, static_cast<cuuint32_t>(box_rows), 1u};
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
  p.part_o = static_cast<float4*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + slots * (D / 4));
  p.cut = reinterpret_cast<int4*>(p.part_ml + slots);
  const long long wk = static_cast<long long>(a.H_kv) * D;
  CUtensorMap kc, vc, kt, vt;
  if (!encode_rows(&kc, a.k_cache, wk, a.cap, a.N, wk, wk * a.cap, kBN) ||
      !encode_rows(&vc, a.v_cache, wk, a.cap, a.N, wk, wk * a.cap, 64) ||
      !encode_rows(&kt, a.k_tree, wk, a.T, a.N, a.ld_kt, a.ld_kt * a.T, kBT) ||
      !encode_rows(&vt, a.v_tree, wk, a.T, a.N, a.ld_vt, a.ld_vt * a.T, kBT))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attention_tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTaSmem<D>);
  if (e != cudaSuccess) return e;
  attention_tree_kernel<D><<<dim3(p.m_tiles, p.workers), kTaThreads, kTaSmem<D>, stream>>>(kc, vc, kt, vt, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.slot_rows * (D / 4) + kJoinThreads - 1) / kJoinThreads, p.workers, p.m_tiles);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_tree_join_kernel<D>, p);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace

size_t attention_tree_workspace(int H_q, int H_kv, int D, int, int T) {
  const int G = H_q / H_kv, m_tiles = attn_m_tiles(G, T);
  const size_t slots = static_cast<size_t>(attn_workers(m_tiles)) * 2 * m_tiles * attn_slot_rows(G, T);
  // slots is even, so the cuts start on a 16-byte boundary
  return slots * (static_cast<size_t>(D) + 2) * sizeof(float) + attn_workers(m_tiles) * sizeof(int4);
}

cudaError_t launch_attention_tree(const AttnTreeParams& p, cudaStream_t stream) {
  if (p.N == 0) return cudaSuccess;
  return p.D == 256 ? launch_d<256>(p, stream) : launch_d<128>(p, stream);
}

}  // namespace gdn
