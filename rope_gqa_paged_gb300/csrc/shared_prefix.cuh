// Attention of a whole batch over a prefix that all its sequences share, on the fifth-generation
// tensor cores, and the merge of its partials with those of the sequences' own tokens (own_tokens.cuh).
//
// Softmax over the tokens [0, n) splits at the prefix length P by log-sum-exp: with m_i, l_i, o_i
// the maximum, the sum and the unnormalised output over part i, out = sum 2^(m_i - M) o_i / sum
// 2^(m_i - M) l_i. The part [0, P) has the same K and V for every sequence, so for one KV head it is
// the attention of B x gamma x n_rep query rows over P keys: a pair of matrix products whose K and V
// are read once for all the rows. The part [P, n) is own_tokens_kernel's. Every part leaves
// (o, m, l) in a slot of the row; one warp per row, or four, merges the slots (shared_merge_kernel).
//
// A prefix CTA takes one or two tiles of 128 of those rows (M of the MMAs) and a chunk of the prefix, in
// key tiles. K and V tiles arrive by TMA through boxes of {64 dims, 8 rows, D / 64 halves, block rows /
// 8}: a block of 16 tokens is one 4 KB copy, and every 8-row group of the tile lies at the same
// stride whatever the block size, as the MMA descriptors want it. For row tile k and key tile j:
//   S_k = Q_k K_j^T   D / 16 MMAs (M 128, N kTile, K 16) into Tensor Memory
//   softmax           warpgroup k, one row per thread: the S row into registers, running max (moved only
//                     when it grows by more than 2^8), P as bf16 pairs over the S columns
//   O_k += P V_j      kTile / 16 MMAs (M 128, N D, K 16), P the A operand from Tensor Memory, V MN-major
// P is rounded to bf16 (half a step, 2^-8 of each weight); maxima, sums and O stay in float32. Sequences of so few
// tokens that such errors do not average out have their P held to 2^-16. Behind a prefix of up to kShortRow tokens that
// is a second P.V here (SPLIT_P), for every row, with the bf16 remainders of P, which lie over the second half of the S
// columns (300 sequences of up to 100 tokens behind 128 shared: 25 us, 23.5 without it, 34 with those sequences read one
// by one). Behind a longer one they end inside the prefix or just past it, are few, and own_tokens_kernel's alone (a
// choice between the two products in the loop over key tiles took 140 us instead of 137 for 512 sequences behind 16384).
//
// One lane issues the MMAs, PV(0, j - 1), S(0, j), PV(1, j - 1), S(1, j), ...; they run in issue order,
// so S may overwrite the P before it (assumed: the PTX documentation promises it for MMAs of one shape and
// accumulator; prefill_tc_kernel relies on the same), and one commit per S says that everything before it is
// complete: the softmax that waits for it may rescale O, and its thread gives K_j and V_(j-1) back to
// the producer. A row tile's chain is softmax, P.V, S, softmax, ...; the first parts of P.V run while
// the last of the softmax do. What this took, 512 rows x 8 heads x 16384 keys in two chunks
// (137 GFLOP, with the merge): 244 us with a lane chosen by its index, key tiles of 64 and three
// commits a tile; 164 us with tiles of 128 and one commit; 151 us with an elected lane (elect_one);
// 121 us with one ring of four slots and rows that leave by bulk copies; 109 us with P in two
// halves and paired float32 instructions (1263 TFLOP/s); 2 % less with P in four parts (6 % more in
// eight). Slower: a second MMA warp; three ring slots, with or without L2 prefetches; a part of the ex2 as
// polynomials on the FMA pipe; two threads per row (1.57 us per key tile of two row tiles, 1.42 so); the first
// part of P before the row's max is known.
//
// Two shapes of CTA:
// * NQ = 1 (up to 128 rows per KV head): key tiles of 64 (128 at head dim 64), Q in Tensor Memory, 256 of
//   its columns, two CTAs per SM: while one is in its softmax the other's MMAs run, and two
//   CTAs' copies together keep up with HBM, which bounds this case (the prefix is read once).
// * NQ = 2 (more rows): key tiles of 128, one CTA per SM, K and V serve 256 rows, Q in shared memory; one
//   row tile's MMAs run while the other is in its softmax. Bound: that chain, some 1300 clocks per row
//   tile and key tile, of which the MMAs are 1024 (S takes Q and K from shared memory at its full rate).
//
// Every wait is bounded (a timeout sets RRA_ERR_TIMEOUT and the roles drain), but for the allocation's, for columns
// that only CTAs already at work can hold; the MMA lane waits for
// its last commit and the producer for its last copies before Tensor Memory is released.
#pragma once

#include "decode_mma.cuh"
#include "tcgen05.cuh"

namespace rra {
namespace spx {

constexpr int kRows = kSharedPrefixRows;        // rows of a tile: M of every MMA
constexpr float kRescaleLog2 = 8.f;             // move the running max only when it grows by more

template <int D, int NQ>
struct Cfg {
  static constexpr int kTile = shared_prefix_tile(D, NQ);  // keys per tile
  static constexpr int kParts = kTile == 128 ? 4 : 2;      // of a P tile, each handed to the MMAs as soon as it is there
  static constexpr int kHalves = D / 64;
  static constexpr int kGroupBytes = 1024 * kHalves;       // 8 rows: their 64-dim halves, 1 KB each
  static constexpr int kTileBytes = kTile / 8 * kGroupBytes;
  static constexpr int kQHalfBytes = kRows * 128;          // NQ 2: Q tiles, K-major, 64-dim halves
  static constexpr int kQBytes = NQ == 2 ? NQ * kHalves * kQHalfBytes : 0;
  static constexpr int kRing = NQ == 2 && D == 128 ? 4 : 6;  // slots: K_0, V_0, K_1, V_1, ...
  // Tensor Memory columns
  static constexpr uint32_t kColO = 0;                     // O_k: D columns each
  static constexpr uint32_t kColS = NQ * D;                // S_k: kTile columns each, P over their first half
  static constexpr uint32_t kColQ = kColS + NQ * kTile;    // NQ 1: Q as bf16 pairs, D / 2 columns
  static constexpr uint32_t kTmemCols = NQ == 2 ? 512 : 256;
  // shared memory
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffBar = kOffRing + kRing * kTileBytes;
  // q_ready, ring_full[kRing], ring_empty[kRing], s_full[NQ], p_full[NQ][kParts], mma_done
  static constexpr int kNumBars = 1 + 2 * kRing + NQ + NQ * kParts + 1;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = 1024 + kOffTmemSlot + 16;
  static constexpr int kSoftmaxThreads = 128 * NQ;
  static constexpr int kThreads = kSoftmaxThreads + 64;    // + producer warp + MMA warp
  static constexpr int kCtasPerSm = NQ == 2 ? 1 : 2;
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kRows, kTile, false);  // Q (K-major) . K^T (K-major)
  static constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, true);      // P (K-major) . V (MN-major)
  static_assert((NQ == 2 ? kColQ : kColQ + D / 2) <= kTmemCols, "Tensor Memory columns");
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of the SM");
};

__device__ __forceinline__ void tma_g2s_5d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, int c3, int c4,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_addr(bar))
      : "memory");
}

// One lane of a converged warp. The compiler knows that a branch on elect.sync holds one thread and keeps the
// MMAs' operands in uniform registers there: 15 clocks an MMA, against some 80 behind a test of the lane.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ float ex2(float x) {  // 2^x on the special-function unit (2^-inf = 0)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 operations in one instruction, on pairs (lo, hi).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return static_cast<uint64_t>(__float_as_uint(lo)) | (static_cast<uint64_t>(__float_as_uint(hi)) << 32);
}
__device__ __forceinline__ float lo2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float hi2(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t z;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(z) : "l"(x), "l"(y));
  return z;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t c) {
  uint64_t z;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(z) : "l"(x), "l"(y), "l"(c));
  return z;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Eight columns of this thread's row times alpha.
__device__ __forceinline__ void scale_cols8(uint32_t taddr, float alpha) {
  uint32_t v[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// N (a multiple of 32) consecutive 32-bit columns of this thread's row.
template <int N>
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&s)[N]) {
  uint32_t v[N / 32][32];
#pragma unroll
  for (int c = 0; c < N / 32; ++c) tc::tmem_ld32(taddr + 32 * c, v[c]);
  tc::tmem_wait_ld();
#pragma unroll
  for (int c = 0; c < N / 32; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i) s[32 * c + i] = v[c][i];
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&s)[N]) {
  if constexpr (N == 16) {
    tc::tmem_st16(taddr, s);
  } else {
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      uint32_t t[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) t[i] = s[32 * c + i];
      tc::tmem_st32(taddr + 32 * c, t);
    }
  }
}

// Sequences whose first new token attends at most this many tokens (L the attended length) hold P to 2^-16, as
// the verify kernel's do. Where a longer prefix has a pass of its own, one unit of the own-token kernel reads all
// their tokens, at most kShortTokens - 1.
constexpr int kShortRow = 256;
constexpr int kShortTokens = kShortRow + 16;
__device__ __forceinline__ bool short_sequence(const DecodeArgs& a, int L) { return L - a.gamma < kShortRow; }
__device__ __forceinline__ bool read_alone(const DecodeArgs& a, int L) {
  return a.prefix_splits > 0 && a.prefix_len > kShortRow && short_sequence(a, L);
}

// Own tokens per unit of a sequence of attended length L.
__device__ __forceinline__ int own_chunk(const DecodeArgs& a, int L) {
  const int slots = a.num_splits - a.prefix_splits, tokens = L - a.first_token;
  if (tokens <= slots * a.chunk) return a.chunk;
  const int stages = (tokens + kOwnStage - 1) / kOwnStage;
  return (stages + slots - 1) / slots * kOwnStage;
}

// L_b of sequence b, cut to the cache; the caller flags what is out of range.
__device__ __forceinline__ int attended_length(const DecodeArgs& a, int b) {
  if (a.positions == nullptr) return min(max(__ldcg(a.seq_lens + b), 0), a.capacity);
  return min(max(min(__ldcg(a.positions + b), a.capacity) + a.gamma, 0), a.capacity);
}

template <int D, int NQ, bool SPLIT_P>
__global__ void __launch_bounds__(Cfg<D, NQ>::kThreads, Cfg<D, NQ>::kCtasPerSm)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                         const DecodeArgs a) {
  using C = Cfg<D, NQ>;
  constexpr int kTile = C::kTile, kRing = C::kRing, kParts = C::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  const int g = blockIdx.z, split = blockIdx.y;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kProducerWarp = 4 * NQ, kMmaWarp = 4 * NQ + 1;
  const int start = split * a.prefix_chunk;
  const int end = min(a.prefix_len, start + a.prefix_chunk);
  const int n_tiles = (end - start + kTile - 1) / kTile;
  const int last_valid = end - start - (n_tiles - 1) * kTile;  // keys of the last tile

  uint64_t* q_ready = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* ring_full = q_ready + 1;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* s_full = ring_empty + kRing;
  uint64_t* p_full = s_full + NQ;
  uint64_t* mma_done = p_full + NQ * kParts;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);

  if (threadIdx.x == 0) {
    mbar_init(q_ready, 4 * NQ);  // one arrival per softmax warp
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], NQ);  // every row tile gives a slot back
    }
    for (int k = 0; k < NQ; ++k) mbar_init(&s_full[k], 1);
    for (int k = 0; k < NQ * kParts; ++k) mbar_init(&p_full[k], 4);
    mbar_init(mma_done, 1);
    fence_barrier_init();
  }
  // The kernel after this one reads the same inputs without waiting for this one, so it may start
  // only when this wait is over: every kernel before this one has then completed.
  pdl_wait();
  pdl_launch_dependents();
  // Tensor Memory only now: a kernel before this one that lets it start early and then allocates (decode_tc_kernel,
  // prefill_tc_kernel) would wait for columns held here, while this CTA waits for that kernel. The two kernels
  // after this one use none.
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, C::kTmemCols);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // ring position r: K of tile r / 2 (r even) or its V (r odd)
  auto slot_of = [](int r) { return r % kRing; };
  auto phase_of = [](int r) { return static_cast<uint32_t>((r / kRing) & 1); };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
    const int log2_bs = a.log2_bs, bs = 1 << log2_bs;
    const int box = min(bs, kTile);  // rows per TMA box, as the tensor maps were encoded
    // group of 8 rows where this lane's box of tile j starts (the id loads a tile ahead of its use)
    auto block_of = [&](int j) {
      const int t = start + j * kTile + lane * box;
      return lane < kTile / box && t < end ? __ldcg(a.prefix_blocks + (t >> log2_bs)) : 0;
    };
    int issued = 0, next = block_of(0);
    for (int j = 0; j < n_tiles && issued == 2 * j; ++j) {
      const int tile0 = start + j * kTile, nbox = (min(kTile, end - tile0) + box - 1) / box;
      int id = next;
      next = block_of(j + 1);
      if (id < 0 || id >= a.num_blocks) {
        flag_error(a.err, RRA_ERR_BLOCK_ID);
        id = 0;
      }
      const int rows8 = (id << (log2_bs - 3)) + (((tile0 + lane * box) & (bs - 1)) >> 3);
      for (int p = 2 * j; p < 2 * j + 2; ++p) {
        const int s = slot_of(p);
        int ok = 1;
        if (lane == 0) {
          if (p >= kRing && !mbar_wait(&ring_empty[s], phase_of(p) ^ 1u))
            ok = 0;
          else
            mbar_arrive_expect_tx(&ring_full[s], static_cast<uint32_t>(nbox * box * 128 * C::kHalves));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) break;
        if (lane < nbox)  // one copy per lane (at most 16)
          tma_g2s_5d(smem + C::kOffRing + s * C::kTileBytes + lane * (box >> 3) * C::kGroupBytes, (p & 1) ? &v_map : &k_map,
                     0, 0, 0, rows8, g, &ring_full[s]);
        __syncwarp();
        issued = p + 1;
      }
    }
    if (lane == 0) {
      if (issued < 2 * n_tiles) flag_error(a.err, RRA_ERR_TIMEOUT);
      // no copy may still be landing when the CTA exits
      for (int p = max(issued - kRing, 0); p < issued; ++p) mbar_wait(&ring_full[slot_of(p)], phase_of(p));
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issue (one lane)
    if (elect_one()) {
      const uint32_t base = smem_addr(smem);
      bool ok = mbar_wait(q_ready, 0);
      tc::fence_after_sync();
      auto issue_s = [&](int k, int j) -> bool {
        const int s = slot_of(2 * j);
        if (k == 0) {
          if (!mbar_wait(&ring_full[s], phase_of(2 * j))) return false;
          tc::fence_after_sync();
        }
        const uint32_t k_base = base + C::kOffRing + s * C::kTileBytes, s_col = tmem + C::kColS + kTile * k;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t kd = tc::sw128_desc(k_base + (kk >> 2) * 1024 + (kk & 3) * 32, 1024, C::kGroupBytes);
          if constexpr (NQ == 2)
            tc::mma_bf16_ss(s_col, tc::sw128_desc(base + (k * C::kHalves + (kk >> 2)) * C::kQHalfBytes + (kk & 3) * 32,
                                                  1024, 1024),
                            kd, C::kIdescS, kk > 0 ? 1u : 0u);
          else
            tc::mma_bf16_ts(s_col, tmem + C::kColQ + 8 * kk, kd, C::kIdescS, kk > 0 ? 1u : 0u);
        }
        tc::commit(&s_full[k]);
        return true;
      };
#pragma unroll
      for (int k = 0; k < NQ; ++k) ok = ok && issue_s(k, 0);
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int s = slot_of(2 * j + 1);
        const uint32_t v_base = base + C::kOffRing + s * C::kTileBytes;
        ok = mbar_wait(&ring_full[s], phase_of(2 * j + 1));
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk) {
            if (kk % (kTile / 16 / kParts) == 0) {
              ok = ok && mbar_wait(&p_full[k * kParts + kk / (kTile / 16 / kParts)], j & 1);
              if (!ok) break;
              tc::fence_after_sync();
            }
            tc::mma_bf16_ts(tmem + C::kColO + D * k, tmem + C::kColS + kTile * k + 8 * kk,
                            tc::sw128_desc(v_base + kk * 2 * C::kGroupBytes, 1024, C::kGroupBytes), C::kIdescPV,
                            (j > 0 || kk > 0) ? 1u : 0u);
          }
          if constexpr (SPLIT_P) {
            if (ok) {
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                tc::mma_bf16_ts(tmem + C::kColO + D * k, tmem + C::kColS + kTile * k + kTile / 2 + 8 * kk,
                                tc::sw128_desc(v_base + kk * 2 * C::kGroupBytes, 1024, C::kGroupBytes), C::kIdescPV, 1u);
            }
          }
          if (ok && j + 1 < n_tiles) ok = issue_s(k, j + 1);
        }
      }
      if (!ok) flag_error(a.err, RRA_ERR_TIMEOUT);
      tc::commit(mma_done);  // every MMA issued above has completed once this arrives
      mbar_wait(mma_done, 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax: thread = query row
    const int k = warp >> 2;                               // row tile of this warpgroup
    const int r = static_cast<int>(threadIdx.x) & 127;     // row = TMEM lane
    const int n_rep = a.Hq / a.Hkv;
    const int row = (blockIdx.x * NQ + k) * kRows + r;
    const bool real = row < a.B * a.gamma * n_rep;
    const bool warp_real = __any_sync(0xffffffffu, real);
    const int bt = real ? row / n_rep : 0;                 // token bt = b * gamma + j of the batch
    const int i_head = real ? row - bt * n_rep : 0;        // head of the group
    const size_t out_row = static_cast<size_t>(bt) * a.Hq + g * n_rep + i_head;
    // keys of the prefix that the row attends
    int lim = a.prefix_len;
    if (real) {
      const int b = bt / a.gamma, j_new = bt - b * a.gamma;
      const int L = attended_length(a, b);
      lim = read_alone(a, L) ? 0 : min(L - a.gamma + 1 + j_new, a.prefix_len);
    }
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_col = tmem + lane_base + C::kColO + D * k;
    {  // the query row
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + out_row * D);
      uint4 qv[D / 8];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) qv[c] = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (NQ == 2) {  // into the Q tile (K-major, 128-byte swizzle)
        uint8_t* dst = smem + k * C::kHalves * C::kQHalfBytes + r * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kQHalfBytes + (((c & 7) ^ (r & 7)) << 4)) = qv[c];
        tc::fence_smem_to_async();
      } else {  // into Tensor Memory: dims (2c, 2c + 1) in column kColQ + c
        uint32_t qw[D / 2];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          qw[4 * c] = qv[c].x;
          qw[4 * c + 1] = qv[c].y;
          qw[4 * c + 2] = qv[c].z;
          qw[4 * c + 3] = qv[c].w;
        }
        st_cols<D / 2>(tmem + lane_base + C::kColQ, qw);
        tc::tmem_wait_st();
        tc::fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    }
    const float sl = a.scale_log2;
    float m_use = -INFINITY, l = 0.f;  // running max (log2 units) and sum
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      if (!warp_wait(&s_full[k], j & 1)) {  // S_k is there, and every MMA issued before it is complete
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) {
        mbar_arrive(&ring_empty[slot_of(2 * j)]);
        if (j > 0) mbar_arrive(&ring_empty[slot_of(2 * j - 1)]);
      }
      if (j == n_tiles - 1 && last_valid < kTile) {
        // keys past the prefix: their V rows are whatever the slot held; zeros keep 0 * V at 0 (both
        // row tiles' threads write them, each before its own P.V)
        if (!warp_wait(&ring_full[slot_of(2 * j + 1)], phase_of(2 * j + 1))) {
          ok = false;
          break;
        }
        if (r >= last_valid && r < kTile) {
          uint8_t* vrow = smem + C::kOffRing + slot_of(2 * j + 1) * C::kTileBytes + (r >> 3) * C::kGroupBytes + (r & 7) * 128;
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(vrow + h * 1024 + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_smem_to_async();
      }
      if (warp_real) {
        const uint32_t s_col = tmem + lane_base + C::kColS + kTile * k;
        uint32_t sv[kTile];
        ld_cols<kTile>(s_col, sv);
        const int vis = min(lim, end) - (start + j * kTile);  // columns this row attends
        if (__any_sync(0xffffffffu, vis < kTile)) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) sv[c] = c < vis ? sv[c] : __float_as_uint(-INFINITY);
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = fmaxf(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
#pragma unroll
        for (int c = 8; c < kTile; c += 2)
          mx[(c >> 1) & 3] = max3(mx[(c >> 1) & 3], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
        const float rmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float m_new = fmaxf(m_use, rmax * sl);
        const bool rescale = m_new > m_use + kRescaleLog2;  // also the first finite max
        float alpha = 1.f;
        if (rescale) {
          alpha = ex2(m_use - m_new);
          m_use = m_new;
        }
        if (j > 0 && __any_sync(0xffffffffu, rescale)) {  // O rows whose max moved (alpha = 1 elsewhere)
#pragma unroll 1
          for (int c = 0; c < D / 8; ++c) scale_cols8(o_col + 8 * c, alpha);  // (few registers: S is held)
        }
        const float mref = m_use == -INFINITY ? 0.f : m_use;
        const uint64_t sl2 = pack2(sl, sl), mref2 = pack2(-mref, -mref);
        uint64_t ls[2] = {0, 0};
#pragma unroll
        for (int h = 0; h < kParts; ++h) {
          uint32_t pw[kTile / 2 / kParts];
          [[maybe_unused]] uint32_t lw[kTile / 2 / kParts];
#pragma unroll
          for (int c = 0; c < kTile / 2 / kParts; ++c) {
            const int cc = h * (kTile / 2 / kParts) + c;
            const uint64_t x = fma2(pack2(__uint_as_float(sv[2 * cc]), __uint_as_float(sv[2 * cc + 1])), sl2, mref2);
            const float e0 = ex2(lo2(x)), e1 = ex2(hi2(x));
            ls[c & 1] = add2(ls[c & 1], pack2(e0, e1));
            if constexpr (SPLIT_P)
              split_bf16x2(e0, e1, pw[c], lw[c]);
            else
              pw[c] = pack_bf16x2(e0, e1);
          }
          st_cols<kTile / 2 / kParts>(s_col + h * (kTile / 2 / kParts), pw);
          if constexpr (SPLIT_P) st_cols<kTile / 2 / kParts>(s_col + kTile / 2 + h * (kTile / 2 / kParts), lw);
          tc::tmem_wait_st();
          if (h + 1 < kParts) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[k * kParts + h]);
          }
        }
        const uint64_t lsum = add2(ls[0], ls[1]);
        l = l * alpha + (lo2(lsum) + hi2(lsum));
      } else if (kParts > 1) {
        __syncwarp();
        if (lane == 0)
          for (int h = 0; h + 1 < kParts; ++h) mbar_arrive(&p_full[k * kParts + h]);
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[k * kParts + kParts - 1]);
    }
    // ------------------------------------------------------------------ epilogue: this chunk's partial rows
    if (ok && warp_wait(mma_done, 0)) {
      tc::fence_after_sync();
      const size_t ps = out_row * a.num_splits + split;
      // the row through shared memory (Q and the ring, which every MMA has read by now) and out in one
      // copy: 16-byte stores of 32 rows at a time cost 1.7 TB/s. Rows 16 bytes apart modulo the banks.
      constexpr int kPitch = D * 4 + 16;
      static_assert(NQ * kRows * kPitch <= C::kOffBar, "the rows fit");
      uint8_t* orow = smem + (k * kRows + r) * kPitch;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tc::tmem_ld32(o_col + 32 * c, v);
        tc::tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 8; ++x)
          *reinterpret_cast<uint4*>(orow + 128 * c + 16 * x) = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
      }
      tc::fence_smem_to_async();
      if (real)
        asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.ws_o + ps * D),
                     "r"(smem_addr(orow)), "n"(D * 4)
                     : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      if (real) *reinterpret_cast<float2*>(a.ws_ml + 2 * ps) = make_float2(m_use, l);
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // written before the CTA ends
    } else {
      flag_error(a.err, RRA_ERR_TIMEOUT);
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Output rows from the prefix_splits partials of the prefix and those of the sequence's own chunks that hold
// tokens; WARPS warps per row, each with every WARPS-th four partials. Rows of a sequence whose position is
// refused are not written.
// Bound: latency (length, then partials and maxima together, then the sums); partials come from L2, four at a
// time and the next four ahead. (One by one behind the maxima: 16 sequences of 8192 tokens with one KV head 23.3
// us instead of 20.3. Eight at a time: 19.5 us there, but 136 us instead of 133 for the 16384 rows of three partials
// of 512 sequences.)
constexpr int kMergeWarps = 4;

template <int D, int WARPS>
__global__ void __launch_bounds__(32 * kMergeWarps) shared_merge_kernel(const DecodeArgs a) {
  constexpr int E = D / 32;  // dims per lane
  constexpr int kBatch = 4;  // partials loaded at a time, the first before the maxima are known
  __shared__ float part[WARPS > 1 ? WARPS - 1 : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = WARPS > 1 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * kMergeWarps + warp;
  const int w0 = WARPS > 1 ? warp : 0;
  if (row >= static_cast<int64_t>(a.B) * a.gamma * a.Hq) return;
  const int b = static_cast<int>(row / (static_cast<int64_t>(a.gamma) * a.Hq));
  // (the lengths are older than the kernels that wrote the partials, which let this one start)
  const int L = attended_length(a, b);
  const int p0 = a.positions != nullptr ? __ldcg(a.positions + b) : a.prefix_len;
  const bool refused = a.positions != nullptr && (p0 < a.prefix_len || p0 > a.capacity - a.gamma);
  const int chunk = own_chunk(a, L);
  const int n = a.prefix_splits + (read_alone(a, L)
                                       ? min(L, 1)
                                       : (max(L - a.first_token, 0) + chunk - 1) / chunk);
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml) + row * a.num_splits;
  const float* o = a.ws_o + row * a.num_splits * D + lane * E;
  float next[kBatch][E];
  auto load = [&](int s) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const float* p = o + static_cast<size_t>(s + k) * D;
      if (s + k < n) {
        if constexpr (E == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
          next[k][0] = v.x, next[k][1] = v.y, next[k][2] = v.z, next[k][3] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(p));
          next[k][0] = v.x, next[k][1] = v.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) next[k][e] = 0.f;
      }
    }
  };
  pdl_wait();  // by every warp: what follows this kernel relies on the two before it being complete
  pdl_launch_dependents();
  if (refused) return;
  load(kBatch * w0);
  float M = -INFINITY, l = 0.f;  // over the partials of all warps so far
  float acc[E] = {};             // over this warp's
  for (int s0 = 0; s0 < n; s0 += 32) {
    const float2 x = s0 + lane < n ? __ldcg(ml + s0 + lane) : make_float2(-INFINITY, 0.f);
    float m = x.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fmaxf(m, M);
    const float mref = m == -INFINITY ? 0.f : m;
    const float w = ex2(x.x - mref), keep = ex2(M - mref);
    float ls = w * x.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    l = l * keep + ls;
    M = m;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= keep;
    for (int s = s0 + kBatch * w0; s < min(n, s0 + 32); s += kBatch * WARPS) {
      float v[kBatch][E];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = next[k][e];
      load(s + kBatch * WARPS);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float ws = __shfl_sync(0xffffffffu, w, s - s0 + k);  // (0 from n on)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(ws, v[k][e], acc[e]);
      }
    }
  }
  if constexpr (WARPS > 1) {  // (always added up in the same order)
    if (warp > 0) {
#pragma unroll
      for (int e = 0; e < E; ++e) part[warp - 1][lane * E + e] = acc[e];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < WARPS - 1; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += part[i][lane * E + e];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, int NQ, bool SPLIT_P>
cudaError_t launch_prefix(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using C = Cfg<D, NQ>;
  static int done[64] = {0};
  auto kern = shared_prefix_kernel<D, NQ, SPLIT_P>;
  cudaError_t e = ensure_smem(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // row tiles innermost: CTAs that read the same keys run side by side and share them through L2
  const int rows = a.B * a.gamma * (a.Hq / a.Hkv);
  const dim3 grid((rows + NQ * kRows - 1) / (NQ * kRows), a.prefix_splits, a.Hkv);
  return launch_pdl(kern, grid, dim3(C::kThreads), C::kSmemBytes, st, km, vm, a);
}

template <int D>
cudaError_t launch_merge(const DecodeArgs& a, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.gamma * a.Hq;
  // Four warps per row where one would go through more than two batches and the SMs hold all of the warps (384
  // rows of 72 partials: 15.6 us the call, 21.3 with one warp; 16384 rows of 9: 178 us, 166 with one).
  if (a.num_splits > 8 && rows * kMergeWarps <= int64_t(64) * current_sm_count())
    return launch_pdl(shared_merge_kernel<D, kMergeWarps>, dim3(static_cast<unsigned>(rows)), dim3(32 * kMergeWarps), 0, st, a);
  const dim3 grid(static_cast<unsigned>((rows + kMergeWarps - 1) / kMergeWarps));
  return launch_pdl(shared_merge_kernel<D, 1>, grid, dim3(32 * kMergeWarps), 0, st, a);
}

}  // namespace spx
}  // namespace rra
