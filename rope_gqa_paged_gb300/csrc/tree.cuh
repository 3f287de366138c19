// Attention of a tree of drafted tokens over each sequence's cache, on the fifth-generation tensor cores.
//
// Sequence b has p cached tokens and a tree of n nodes in cache slots p .. p + n - 1 (their keys rotated for position
// p + depth). Query row (node j, head i of a KV head's group) attends [0, p), its ancestors and itself: one
// softmax over p + depth + 1 tokens,
//   out = sum_t e^(s_t - m) V_t / sum_t e^(s_t - m),   s_t = scale q.K_t,   m = max s_t.
// For one KV head these are n x n_rep rows over the same p + n keys, so the rows are M of the MMAs and every K and V
// byte that comes from HBM serves all of them (a tree of 16 nodes with 4 heads per group: 64 flops per byte;
// 256 rows need as many clocks of the tensor cores as HBM needs for their keys). The mask is in the last tiles
// only: bit words of the row's ancestors, shifted to the tile.
//
// Work: the key tiles of all (sequence, KV head) units, in one line, cut into `ranges` runs of equal length; the
// CTAs of a range (one per kRows x NQ rows: they share its keys through L2) go through its units or parts of
// units. So the load is even whatever the sequences' lengths are, which the host does not know: every CTA adds up the
// lengths for itself. A unit that lies wholly in one range is written to the output; the parts of a cut one leave
// (o, m, l) for tree_merge_kernel. Those are the first and the last unit of a range at most.
//
// In a CTA the roles run through the same list of units: one or two producer warps (K and V tiles by TMA into a ring that
// goes on over unit borders), an MMA lane and a softmax warpgroup for each row tile. For row tile k and key tile j
//   S_k = Q_k K_j^T   D / 16 MMAs (M 128, N kTile, K 16) into Tensor Memory
//   softmax           one row per thread; running max, moved only when it grows by more than 2^8
//   O_k += P V_j      kTile / 16 MMAs, P (bf16) the A operand from Tensor Memory over the S columns
// as in shared_prefix.cuh, whose notes on issue order and on waits hold here too. At the end of a unit the next one's
// Q goes in before O is read, so that its first S runs meanwhile; its first P.V waits for the softmax of its first
// tile, which comes after that reading.
// P is rounded to bf16 (half a step, 2^-8 of each weight); in sequences of fewer than kShortRow cached tokens, where
// such errors do not average out, its remainders go through a second P.V (2^-16). Longer ones are within 0.0023 of 64 bits (root
// mean square, relative), 0.0017 of which is the output's own rounding. A second P.V for them too leaves those 0.0017, and
// takes 1 % more for 64 ragged sequences of 16 nodes (201 us from 199), 7 % for one user's 4000 tokens (16.8 from 15.8) and at head dim 64 (94
// from 88), 13 % for 16 x 16 nodes of 32 heads with one KV head (55 from 49), 16 to 21 % with two row tiles (168 from 144, 136 from 113).
// Maxima, sums and O are float32.
//
// Two shapes of CTA, by the rows of a KV head:
// * NQ = 1 (up to 128): two CTAs per SM, whose copies together keep up with HBM, which bounds it: 64 sequences of 500 to 8000
//   tokens with 16 nodes of 32 / 8 heads (1.15 GB) 199 us the step, 5.8 TB/s; under a profiler 16 of them read 1.00 times their
//   bytes, tensor pipe 32 % busy.
// * NQ = 2 (more): one CTA per SM, K and V serve 256 rows, key tiles of 128. No one part bounds it: a CTA's copies (boxes of one
//   block), its MMAs and its softmax follow one another in part, some 1.7 us per key tile, of which the MMAs are 1.07. One user's 131000
//   tokens with 64 nodes 113 us, 101 where no tile is copied, 105 without the softmax's arithmetic; 32 sequences with up to 60 nodes 144, 134
//   and 135; 16 of 64 nodes of 64 heads 163, 155 and 138. K and V have a producer warp each (with one 118 us for the first and 157 for the
//   second; V through cp.async by two warps of its own: 135 and 170). The first does 1.2 PFLOP/s over its three kernels.
// Few keys are latency: one user's 4000 tokens 16 us, of which the queries are there after 5.7, a CTA's four
// tiles take 3.3, its partial rows 1.6 and the merge of 16 partials 4.
#pragma once

#include <atomic>

#include "shared_prefix.cuh"

namespace rra {
namespace tree {

using spx::add2;
using spx::elect_one;
using spx::ex2;
using spx::fma2;
using spx::hi2;
using spx::kRescaleLog2;
using spx::kShortRow;
using spx::ld_cols;
using spx::lo2;
using spx::max3;
using spx::pack2;
using spx::scale_cols8;
using spx::st_cols;
using spx::tma_g2s_5d;
using spx::warp_wait;

constexpr int kRows = kTreeRows;

template <int D, int NQ, bool PAGED>
struct Cfg {
  static constexpr int kTile = tree_tile(D, NQ);             // keys per tile
  static constexpr int kParts = kTile == 128 ? 4 : 2;        // of a P tile, each handed to the MMAs as soon as it is there
  static constexpr int kHalves = D / 64;
  // paged: 8-row groups with their 64-dim halves side by side; contiguous: whole halves
  static constexpr int kGroupBytes = PAGED ? 1024 * kHalves : 1024;
  static constexpr int kHalfBytes = PAGED ? 1024 : kTile * 128;
  static constexpr int kTileBytes = kTile * 128 * kHalves;
  static constexpr int kQHalfBytes = kRows * 128;            // NQ 2: Q tiles, K-major, 64-dim halves
  static constexpr int kQBytes = NQ == 2 ? NQ * kHalves * kQHalfBytes : 0;
  static constexpr int kRing = NQ == 2 && D == 128 ? 4 : 5;  // slots: K_0, V_0, K_1, V_1, ...
  static constexpr int kWarps = 4 * NQ;                      // softmax warps
  static constexpr int kStagePitch = 80;                     // 64 bytes of a row and 16: eight rows in other banks
  static constexpr int kStageBytes = 32 * kStagePitch;       // per softmax warp: rows on their way out
  // Tensor Memory columns
  static constexpr uint32_t kColO = 0;                       // O_k: D columns each
  static constexpr uint32_t kColS = NQ * D;                  // S_k: kTile columns each, P over their first half
  static constexpr uint32_t kColQ = kColS + NQ * kTile;      // NQ 1: Q as bf16 pairs, D / 2 columns
  static constexpr uint32_t kTmemCols = NQ == 2 ? 512 : 256;
  // shared memory
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffStage = kOffRing + kRing * kTileBytes;
  static constexpr int kOffSees = kOffStage + kWarps * kStageBytes;  // 128 bits per row: the nodes that it attends
  static constexpr int kOffBar = kOffSees + NQ * kRows * kTreeMaxNodes / 8;
  // q_ready, ring_full[kRing], ring_empty[kRing], s_full[NQ], p_full[NQ][kParts], o_done
  static constexpr int kNumBars = 1 + 2 * kRing + NQ + NQ * kParts + 1;
  static constexpr int kOffStart = kOffBar + kNumBars * 8;   // Start
  static constexpr int kOffUnits = kOffStart + 160;          // Units, one per softmax warp
  static constexpr int kOffTmemSlot = kOffUnits + kWarps * 48;
  static constexpr int kSmemBytes = 1024 + kOffTmemSlot + 16;
  // + producer warp + MMA warp; NQ 2: and the producer of V and an idle one, a whole warpgroup, which gives registers to the
  // softmax (which spilled some without: 5 % of the step)
  static constexpr int kThreads = 32 * kWarps + (NQ == 2 ? 128 : 64);
  static constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // 256 x 216 + 128 x 72 = 384 x 168, the launch's
  static constexpr int kCtasPerSm = NQ == 2 ? 1 : 2;
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kRows, kTile, false);  // Q (K-major) . K^T (K-major)
  static constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, true);      // P (K-major) . V (MN-major)
  static_assert((NQ == 2 ? kColQ : kColQ + D / 2) <= kTmemCols, "Tensor Memory columns");
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of the SM");
  static_assert(kThreads <= 32 * 32, "the scan's warps");
};

// 32 bytes from L2. A load instruction takes a clock per line that its lanes touch, so rows of 256 bytes, one per lane, come in
// half the time of 16-byte loads (which tensors that start at an odd multiple of 16 bytes need).
__device__ __forceinline__ void ld_32_bytes(const uint4* p, uint32_t* r, bool aligned32) {
  if (!aligned32) {
    const uint4 x = __ldcg(p), y = __ldcg(p + 1);
    r[0] = x.x, r[1] = x.y, r[2] = x.z, r[3] = x.w;
    r[4] = y.x, r[5] = y.y, r[6] = y.z, r[7] = y.w;
    return;
  }
  asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}

// Sequence b: cached tokens, nodes, key tiles. Refused: no tiles, and nothing of it is written.
struct Seq {
  int p, n, tiles;
  bool refused;
};
struct Raw {
  int p, n;
};
__device__ __forceinline__ Raw raw_sequence(const TreeArgs& a, int b) {
  return {__ldcg(a.positions + b), a.lens != nullptr ? __ldcg(a.lens + b) : a.N};
}
__device__ __forceinline__ Seq sequence(const TreeArgs& a, const Raw& raw, int tile, bool flag = false) {
  Seq s{raw.p, raw.n, 0, false};
  if (s.n < 0 || s.n > a.N) {
    if (flag) flag_error(a.err, RRA_ERR_SEQ_LEN);
    s.n = min(max(s.n, 0), a.N);
  }
  s.refused = s.n > 0 && (s.p < 0 || s.p > a.capacity - s.n);
  if (flag && s.refused) flag_error(a.err, RRA_ERR_POSITION);
  s.tiles = s.refused || s.n == 0 ? 0 : (s.p + s.n - 1) / tile + 1;
  return s;
}
__device__ __forceinline__ Seq sequence(const TreeArgs& a, int b, int tile, bool flag = false) {
  return sequence(a, raw_sequence(a, b), tile, flag);
}

// The units in one line, each `extra` places (what a CTA takes for one more unit, in key tiles) and its key tiles, cut into
// `ranges` runs whose lengths differ by one at most. A border among the extra places is the start of the unit.
// Where the units are equally long and `ranges` is a multiple of their number, every unit starts with a run of its own.
struct Cut {
  int total, ranges, extra;
  __device__ __forceinline__ int border(int r) const {
    if (total < 1 << 21) return static_cast<int>(static_cast<uint32_t>(total) * r / static_cast<uint32_t>(ranges));  // (at most 1024 of them)
    return static_cast<int>(static_cast<int64_t>(total) * r / ranges);
  }
  __device__ __forceinline__ int range_of(int t) const {  // the last r with border(r) <= t
    return static_cast<int>((static_cast<int64_t>(t + 1) * ranges - 1) / total);
  }
};

// Where a range starts: places [t0, t1) of the line, from place `off` of sequence b's on.
struct Start {
  int t0, t1, b, off;
  Cut cut;
  Seq seq;        // of sequence b
  int sums[2][12];
};

// Adds up the sequences' tiles and finds the start of range r (all threads of the CTA; r past the ranges in use: t0 = t1).
// Ranges of at least min_tiles tiles, unless there are more units than such ranges; and a whole number of them per unit where
// that leaves no more than every ninth out (a CTA that goes from one unit to the next takes some 3 us longer: one user's
// 4000 tokens). So some of a.ranges may stay unused.
template <int THREADS>
__device__ void locate(const TreeArgs& a, int tile, int r, bool flag, Start* s) {
  const int per = (a.B + THREADS - 1) / THREADS, b0 = min(static_cast<int>(threadIdx.x) * per, a.B), b1 = min(b0 + per, a.B);
  Seq seq{0, 0, 0, false};
  int tiles = 0, seqs = 0;
  for (int b = b0; b < b1; ++b) {
    seq = sequence(a, b, tile, flag);
    tiles += seq.tiles;
    seqs += seq.tiles > 0;
  }
  int tiles_to = tiles, seqs_to = seqs;  // inclusive sums
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, tiles_to, d), y = __shfl_up_sync(0xffffffffu, seqs_to, d);
    if (lane >= d) {
      tiles_to += x;
      seqs_to += y;
    }
  }
  if (lane == 31) {
    s->sums[0][warp] = tiles_to;
    s->sums[1][warp] = seqs_to;
  }
  if (threadIdx.x == 0) s->t0 = s->t1 = 0;
  __syncthreads();
  int tiles_before = tiles_to - tiles, seqs_before = seqs_to - seqs, total = 0, units = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) {
      tiles_before += s->sums[0][w];
      seqs_before += s->sums[1][w];
    }
    total += s->sums[0][w] * a.Hkv;
    units += s->sums[1][w] * a.Hkv;
  }
  int ranges = min(a.ranges, max((total + a.min_tiles - 1) / a.min_tiles, max(units, 1))), extra = a.unit_tiles;
  if (units > 0 && units <= ranges) {
    const int up = (ranges + units - 1) / units * units, down = ranges / units;
    if (up <= min(a.ranges, total))  // (no range without tiles)
      ranges = up;
    else if (down >= 8)
      ranges = down * units;
    if (ranges % units == 0) extra = 0;
  }
  if (r < ranges && total > 0) {
    const Cut cut{total + units * extra, ranges, extra};
    int before = (tiles_before + seqs_before * extra) * a.Hkv;
    const int mine = (tiles + seqs * extra) * a.Hkv, t0 = cut.border(r), t1 = cut.border(r + 1);
    if (t0 < t1 && before <= t0 && t0 < before + mine) {  // one thread
      int b = b0;
      if (per > 1) {
        for (;; ++b) {
          seq = sequence(a, b, tile);
          const int span = seq.tiles > 0 ? (seq.tiles + extra) * a.Hkv : 0;
          if (t0 < before + span) break;
          before += span;
        }
      }
      s->t0 = t0;
      s->t1 = t1;
      s->cut = cut;
      s->b = b;
      s->seq = seq;
      s->off = t0 - before;
    }
  }
  __syncthreads();
}

// A range's units one after the other: key tiles [j0, j1) of KV head g of sequence b; `rest` of its places are left
// for later ranges.
struct Units {
  int b, g, j0, j1, rest, off, left, extra;
  Seq seq;
  __device__ __forceinline__ Units(const Start& s)
      : b(s.b), g(0), j0(0), j1(0), rest(0), off(s.off), left(s.t1 - s.t0), extra(s.cut.extra), seq(s.seq) {}
  // `ahead`: what is known of sequence b + 1, loaded when b began.
  __device__ __forceinline__ bool next(const TreeArgs& a, int tile, int first_row, Raw& ahead) {
    while (left > 0) {
      while (seq.tiles == 0 || off >= (seq.tiles + extra) * a.Hkv) {
        off = 0;
        ++b;
        seq = sequence(a, ahead, tile);
        ahead = raw_sequence(a, min(b + 1, a.B - 1));
      }
      const int span = seq.tiles + extra;
      g = off / span;
      const int from = off - g * span, take = min(span - from, left);
      j0 = max(from - extra, 0);
      j1 = max(from + take - extra, 0);
      rest = span - from - take;
      off += take;
      left -= take;
      if (j1 > j0 && seq.n * a.n_rep > first_row) return true;  // (a smaller tree leaves this CTA's rows empty)
    }
    return false;
  }
  __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == seq.tiles; }
};

// Rows of nodes that a tree does not have are zero, and a sequence without any has nothing to merge; by a warp or a CTA, for
// every gridDim.x-th sequence.
__device__ __forceinline__ void pad_rows(const TreeArgs& a, int D, int thread, int threads) {
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const Seq s = sequence(a, b, 1);
    if (s.tiles == 0 && a.headers_by_unit)
      for (int g = thread; g < a.Hkv; g += threads) a.headers[b * a.Hkv + g] = make_int4(0, 0, 0, 0);
    if (s.refused || s.n == a.N) continue;
    uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (static_cast<size_t>(b) * a.N + s.n) * a.Hq * D);
    const size_t vecs = static_cast<size_t>(a.N - s.n) * a.Hq * (D / 8);
    for (size_t i = thread; i < vecs; i += threads) o[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

template <int D, int NQ, bool PAGED>
__global__ void __launch_bounds__(Cfg<D, NQ, PAGED>::kThreads, Cfg<D, NQ, PAGED>::kCtasPerSm)
    tree_attn_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                     const TreeArgs a) {
  using C = Cfg<D, NQ, PAGED>;
  constexpr int kTile = C::kTile, kRing = C::kRing, kParts = C::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  const int range = blockIdx.x / a.row_ctas, first_row = (blockIdx.x - range * a.row_ctas) * NQ * kRows;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int kProducerWarp = C::kWarps, kMmaWarp = C::kWarps + 1;

  uint64_t* q_ready = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* ring_full = q_ready + 1;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* s_full = ring_empty + kRing;
  uint64_t* p_full = s_full + NQ;
  uint64_t* o_done = p_full + NQ * kParts;
  Start* start = reinterpret_cast<Start*>(smem + C::kOffStart);
  static_assert(sizeof(Start) <= 160 && sizeof(Units) <= 48 && sizeof(Units) % 4 == 0 && C::kOffSees % 16 == 0 && kTreeMaxNodes == 128, "layout");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);

  if (threadIdx.x == 0) {
    mbar_init(q_ready, C::kWarps);  // one arrival per softmax warp
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], NQ);  // every row tile gives a slot back
    }
    for (int k = 0; k < NQ; ++k) mbar_init(&s_full[k], 1);
    for (int k = 0; k < NQ * kParts; ++k) mbar_init(&p_full[k], 4);
    mbar_init(o_done, 1);
    fence_barrier_init();
  }
  // Behind the append of the same call (after_append) everything that it does not write is complete already: it lets
  // this kernel start only when its own wait is over. Queries and the tree's keys wait for it further down.
  if (!a.after_append) pdl_wait();
  locate<C::kThreads>(a, kTile, range, blockIdx.x == 0, start);

  if (start->t0 >= start->t1) {  // (the same for every thread)
    if (threadIdx.x == 0 && first_row == 0 && a.headers != nullptr && !a.headers_by_unit) a.headers[range] = make_int4(0, 0, 0, 0);
    pad_rows(a, D, threadIdx.x, C::kThreads);
    pdl_wait();
    return;
  }
  // Tensor Memory when every kernel that may hold some is complete, and the next kernel only when all CTAs have theirs.
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, C::kTmemCols);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  __syncthreads();
  tc::fence_after_sync();
  pdl_launch_dependents();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // ring position r: K of the CTA's tile r / 2 (r even) or its V (r odd)
  auto slot_of = [](uint32_t r) { return r % kRing; };
  auto phase_of = [](uint32_t r) { return (r / kRing) & 1u; };

  if (warp >= C::kWarps) {
   if constexpr (NQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
   Units u(*start);
   Raw ahead = raw_sequence(a, min(u.b + 1, a.B - 1));
   if (warp == kProducerWarp || (NQ == 2 && warp == kMmaWarp + 1)) {
    // ------------------------------------------------------------------ producer (NQ 2: one for K, one for V)
    constexpr int kCopied = NQ == 2 ? 1 : 2;
    const int kv0 = warp == kProducerWarp ? 0 : 1;
    const bool first_producer = warp == kProducerWarp;
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
    const int log2_bs = a.log2_bs, bs = 1 << log2_bs;
    const int box = PAGED ? min(bs, kTile) : kTile;  // rows per TMA box, as the tensor maps were encoded
    bool ok = true, waited = !a.after_append;
    uint32_t tiles = 0;  // of the CTA so far
    int4 h = make_int4(0, 0, 0, 0);
    while (ok && u.next(a, kTile, first_row, ahead)) {
      const int L = u.seq.p + u.seq.n;
      if (first_producer && first_row == 0 && lane == 0 && a.headers != nullptr) {
        // a unit that starts here and goes on in later ranges (it is this one's last) is merged for this header
        h = make_int4(0, 0, 0, 0);
        if (u.j0 == 0 && !u.whole()) {
          const int end = start->t1 + u.rest;  // the unit's end in the line
          h = make_int4(start->cut.range_of(end - 1) - range + 1, range, u.b * a.Hkv + u.g, u.seq.n * a.n_rep);
        }
        if (a.headers_by_unit && u.j0 == 0) a.headers[u.b * a.Hkv + u.g] = h;
      }
      const int32_t* row = a.block_table + static_cast<size_t>(u.b) * a.max_blocks_per_seq;
      // block where this lane's box of tile j starts (the id loads a tile ahead of its use)
      auto block_of = [&](int j) {
        const int t = j * kTile + lane * box;
        return PAGED && j < u.j1 && lane < kTile / box && t < L ? __ldcg(row + (t >> log2_bs)) : 0;
      };
      int next = block_of(u.j0);
      for (int j = u.j0; ok && j < u.j1; ++j) {
        const int tile0 = j * kTile, nbox = PAGED ? (min(kTile, L - tile0) + box - 1) / box : 1;
        int id = next;
        next = block_of(j + 1);
        if (PAGED && (id < 0 || id >= a.num_blocks)) {
          flag_error(a.err, RRA_ERR_BLOCK_ID);
          id = 0;
        }
        if (!waited && tile0 + kTile > u.seq.p) {  // the tree's keys and values
          pdl_wait();
          waited = true;
        }
        const int rows8 = PAGED ? (id << (log2_bs - 3)) + (((tile0 + lane * box) & (bs - 1)) >> 3) : 0;
        for (int kv = kv0; ok && kv < kv0 + kCopied; ++kv) {
          const uint32_t r = 2 * tiles + kv, s = slot_of(r);
          int good = 1;
          if (lane == 0) {
            if (r >= kRing && !mbar_wait(&ring_empty[s], phase_of(r) ^ 1u))
              good = 0;
            else
              mbar_arrive_expect_tx(&ring_full[s], static_cast<uint32_t>(nbox * box * 128 * C::kHalves));
          }
          ok = __shfl_sync(0xffffffffu, good, 0) != 0;
          if (!ok) break;
          uint8_t* dst = smem + C::kOffRing + s * C::kTileBytes;
          const CUtensorMap* map = kv ? &v_map : &k_map;
          if constexpr (PAGED) {
            if (lane < nbox)  // one copy per lane (at most 16)
              tma_g2s_5d(dst + lane * (box >> 3) * C::kGroupBytes, map, 0, 0, 0, rows8, u.g, &ring_full[s]);
          } else if (lane < C::kHalves) {
            tma_g2s_3d(dst + lane * C::kHalfBytes, map, 64 * lane, tile0, u.b * a.Hkv + u.g, &ring_full[s]);
          }
          __syncwarp();
        }
        if (ok) ++tiles;
      }
    }
    if (first_producer) {
      if (first_row == 0 && lane == 0 && a.headers != nullptr && !a.headers_by_unit) a.headers[range] = h;
      pad_rows(a, D, lane, 32);
    }
    if (lane == 0) {
      if (!ok) flag_error(a.err, RRA_ERR_TIMEOUT);
      // no copy may still be landing when the CTA exits
      const uint32_t issued = 2 * tiles;
      for (uint32_t r = issued > kRing ? issued - kRing : 0; r < issued; ++r)
        if (kCopied == 2 || (r & 1u) == static_cast<uint32_t>(kv0)) mbar_wait(&ring_full[slot_of(r)], phase_of(r));
      if (!ok && kCopied == 2) mbar_wait(&ring_full[slot_of(issued)], phase_of(issued));  // (K of the tile whose V found no place)
    }
   } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issue (one lane)
    if (elect_one()) {
      // Descriptors by additions to one per operand (addresses count 16 bytes in their low bits): worked out one by one
      // and kept, they take more registers than this warp has.
      auto opaque = [](uint64_t d) {
        asm volatile("" : "+l"(d));
        return d;
      };
      const uint32_t base = smem_addr(smem);
      const uint64_t q_desc = tc::sw128_desc(base, 1024, 1024);
      bool ok = true;
      uint32_t c = 0, units = 0;  // the CTA's tiles and units so far
      while (ok && u.next(a, kTile, first_row, ahead)) {
        const bool short_seq = u.seq.p < kShortRow;
        ok = mbar_wait(q_ready, units & 1u);
        tc::fence_after_sync();
        auto issue_s = [&](int k, uint32_t t) -> bool {
          const uint32_t s = slot_of(2 * t);
          if (k == 0) {
            if (!mbar_wait(&ring_full[s], phase_of(2 * t))) return false;
            tc::fence_after_sync();
          }
          const uint32_t s_col = tmem + C::kColS + kTile * k;
          const uint64_t kd = opaque(tc::sw128_desc(base + C::kOffRing + s * C::kTileBytes, 1024, C::kGroupBytes));
          const uint64_t qd = opaque(q_desc);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t kd_kk = kd + ((kk >> 2) * C::kHalfBytes + (kk & 3) * 32) / 16;
            if constexpr (NQ == 2)
              tc::mma_bf16_ss(s_col, qd + ((k * C::kHalves + (kk >> 2)) * C::kQHalfBytes + (kk & 3) * 32) / 16, kd_kk,
                              C::kIdescS, kk > 0 ? 1u : 0u);
            else
              tc::mma_bf16_ts(s_col, tmem + C::kColQ + 8 * kk, kd_kk, C::kIdescS, kk > 0 ? 1u : 0u);
          }
          tc::commit(&s_full[k]);
          return true;
        };
#pragma unroll
        for (int k = 0; k < NQ; ++k) ok = ok && issue_s(k, c);
        for (int j = u.j0; ok && j < u.j1; ++j, ++c) {
          const uint32_t s = slot_of(2 * c + 1);
          const uint64_t vd = opaque(tc::sw128_desc(base + C::kOffRing + s * C::kTileBytes, C::kHalfBytes, C::kGroupBytes));
          ok = mbar_wait(&ring_full[s], phase_of(2 * c + 1));
#pragma unroll
          for (int k = 0; k < NQ; ++k) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk) {
              if (kk % (kTile / 16 / kParts) == 0) {
                ok = ok && mbar_wait(&p_full[k * kParts + kk / (kTile / 16 / kParts)], c & 1u);
                if (!ok) break;
                tc::fence_after_sync();
              }
              tc::mma_bf16_ts(tmem + C::kColO + D * k, tmem + C::kColS + kTile * k + 8 * kk,
                              vd + kk * 2 * C::kGroupBytes / 16, C::kIdescPV, (j > u.j0 || kk > 0) ? 1u : 0u);
            }
            if (ok && short_seq) {  // the remainders of P
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                tc::mma_bf16_ts(tmem + C::kColO + D * k, tmem + C::kColS + kTile * k + kTile / 2 + 8 * kk,
                                vd + kk * 2 * C::kGroupBytes / 16, C::kIdescPV, 1u);
            }
            if (ok && j + 1 < u.j1) ok = issue_s(k, c + 1);
          }
        }
        tc::commit(o_done);  // every MMA issued above has completed once this arrives
        ++units;
      }
      if (!ok) flag_error(a.err, RRA_ERR_TIMEOUT);
      if (units > 0) mbar_wait(o_done, (units - 1) & 1u);
    }
   }
  } else {
    if constexpr (NQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    // ------------------------------------------------------------------ softmax: thread = query row
    const int k = warp >> 2;                               // row tile of this warpgroup
    const int r = static_cast<int>(threadIdx.x) & 127;     // row = TMEM lane
    const int row = first_row + k * kRows + r;             // node row / n_rep, head row % n_rep of the group
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t o_col = tmem + lane_base + C::kColO + D * k;
    uint8_t* stage = smem + C::kOffStage + warp * C::kStageBytes;
    const float sl = a.scale_log2;
    uint4* sees = reinterpret_cast<uint4*>(smem + C::kOffSees);
    // The warp's place in the list of units, in shared memory: S takes the registers.
    Units& u = *reinterpret_cast<Units*>(smem + C::kOffUnits + 48 * warp);
    Raw ahead = raw_sequence(a, min(start->b + 1, a.B - 1));  // (lane 0's counts)
    auto advance = [&]() -> bool {
      __syncwarp();
      const int more = __shfl_sync(0xffffffffu, lane == 0 && u.next(a, kTile, first_row, ahead) ? 1 : 0, 0);
      __syncwarp();
      return more != 0;
    };
    if (lane == 0) u = Units(*start);
    if (a.after_append) pdl_wait();  // the queries

    auto out_row_of = [&](int b, int g) {
      const int j = row / a.n_rep;
      return (static_cast<size_t>(b) * a.N + j) * a.Hq + g * a.n_rep + (row - j * a.n_rep);
    };
    auto load_q = [&]() {  // the unit's query rows
      const int live = u.seq.n * a.n_rep;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q));
      if constexpr (NQ == 2) {
        uint4 qv[D / 8];
        // Into the Q tile (K-major, 128-byte swizzle): this warp's rows, 16 lanes a row (8 at head dim 64), so that loads are
        // whole lines. (A row per thread: one user's 131000 tokens 1.3 us longer.)
        constexpr int kLanes = D / 8, kRowsPer = 32 / kLanes;  // lanes per row, rows per load
        const int x = lane % kLanes, row0 = first_row + k * kRows + (r & ~31) + lane / kLanes;
        int j = row0 / a.n_rep, i = row0 - j * a.n_rep;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          qv[c] = row0 + c * kRowsPer < live ? __ldcg(q + ((static_cast<size_t>(u.b) * a.N + j) * a.Hq + u.g * a.n_rep + i) * kLanes + x)
                                             : make_uint4(0u, 0u, 0u, 0u);
          for (i += kRowsPer; i >= a.n_rep; i -= a.n_rep) ++j;
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const int rr = (r & ~31) + c * kRowsPer + lane / kLanes;
          *reinterpret_cast<uint4*>(smem + (k * C::kHalves + (x >> 3)) * C::kQHalfBytes + rr * 128 + (((x & 7) ^ (rr & 7)) << 4)) = qv[c];
        }
        tc::fence_smem_to_async();
      } else {
        // Into Tensor Memory, a row per lane: dims (2c, 2c + 1) in column kColQ + c. (By lines and through shared
        // memory: 2 us longer.)
        const uint4* src = q + out_row_of(u.b, u.g) * (D / 8);
        const bool aligned32 = (reinterpret_cast<uintptr_t>(a.q) & 31) == 0;
        uint32_t qw[D / 2] = {};
        if (row < live) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) ld_32_bytes(src + 2 * c, qw + 8 * c, aligned32);
        }
        st_cols<D / 2>(tmem + lane_base + C::kColQ, qw);
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready);
    };

    uint32_t c = 0, units = 0;  // the CTA's tiles and units so far
    bool ok = true, more = advance();
    if (more) load_q();
    while (ok && more) {
      const int p = u.seq.p, j0 = u.j0, j1 = u.j1;
      const bool short_seq = p < kShortRow;
      const bool warp_real = first_row + k * kRows + (r & ~31) < u.seq.n * a.n_rep;  // any row of this warp
      // The row's node and its ancestors, one bit each: parents now, the bits when the first tile with nodes comes (the
      // parents then too where S takes 128 of 168 registers).
      constexpr bool kParentsAhead = NQ == 2 || kTile == 64;
      int up[kTreeMaxNodes / 32];  // parents of nodes lane, lane + 32, ...
      const bool has_nodes = warp_real && j1 * kTile > p;
      auto load_parents = [&]() {
#pragma unroll
        for (int w = 0; w < kTreeMaxNodes / 32; ++w) {
          const int n = 32 * w + lane;
          up[w] = n < u.seq.n ? __ldcg(a.parents + static_cast<size_t>(u.b) * a.N + n) : -1;
        }
      };
      if (kParentsAhead && has_nodes) load_parents();
      auto find_ancestors = [&]() {  // (kept in shared memory: every register counts below)
        if (!kParentsAhead) load_parents();
#pragma unroll
        for (int w = 0; w < kTreeMaxNodes / 32; ++w)
          if (up[w] < -1 || up[w] >= 32 * w + lane) {
            flag_error(a.err, RRA_ERR_TREE);
            up[w] = -1;
          }
        uint32_t s0 = 0, s1 = 0, s2 = 0, s3 = 0;
        int n = row < u.seq.n * a.n_rep ? row / a.n_rep : -1;
        while (__any_sync(0xffffffffu, n >= 0)) {  // (parents come before their children)
          const uint32_t bit = n >= 0 ? 1u << (n & 31) : 0u;
          const int x0 = __shfl_sync(0xffffffffu, up[0], n & 31), x1 = __shfl_sync(0xffffffffu, up[1], n & 31);
          const int x2 = __shfl_sync(0xffffffffu, up[2], n & 31), x3 = __shfl_sync(0xffffffffu, up[3], n & 31);
          const int w = n >> 5;  // (-1: none)
          s0 |= w == 0 ? bit : 0u;
          s1 |= w == 1 ? bit : 0u;
          s2 |= w == 2 ? bit : 0u;
          s3 |= w == 3 ? bit : 0u;
          n = w < 0 ? -1 : w == 0 ? x0 : w == 1 ? x1 : w == 2 ? x2 : x3;
        }
        sees[threadIdx.x] = make_uint4(s0, s1, s2, s3);
      };
      const int first_nodes = max(j0, p / kTile);  // the first tile of this part that may have nodes
      float m_use = -INFINITY, l = 0.f;  // running max (log2 units) and sum
      for (int j = j0; j < j1; ++j, ++c) {
        if (has_nodes && j == first_nodes) find_ancestors();
        if (!warp_wait(&s_full[k], c & 1u)) {  // S_k is there, and every MMA issued before it is complete
          ok = false;
          break;
        }
        tc::fence_after_sync();
        if (r == 0) {
          mbar_arrive(&ring_empty[slot_of(2 * c)]);
          if (j > j0) mbar_arrive(&ring_empty[slot_of(2 * c - 1)]);
        }
        if (j + 1 == j1 && p + u.seq.n - j * kTile < kTile) {
          // rows past the last token: their V is whatever the slot held; zeros keep 0 * V at 0 (both row
          // tiles' threads write them, each before its own P.V)
          if (!warp_wait(&ring_full[slot_of(2 * c + 1)], phase_of(2 * c + 1))) {
            ok = false;
            break;
          }
          if (r >= p + u.seq.n - j * kTile && r < kTile) {
            uint8_t* vrow = smem + C::kOffRing + slot_of(2 * c + 1) * C::kTileBytes + (r >> 3) * C::kGroupBytes + (r & 7) * 128;
#pragma unroll
            for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
              for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(vrow + h * C::kHalfBytes + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
          }
          tc::fence_smem_to_async();
        }
        if (warp_real) {
          const uint32_t s_col = tmem + lane_base + C::kColS + kTile * k;
          uint32_t sv[kTile];
          ld_cols<kTile>(s_col, sv);
          if ((j + 1) * kTile > p) {  // the tree begins in this tile, or before it
            const uint4 s = sees[threadIdx.x];
#pragma unroll
            for (int w = 0; w < kTile / 32; ++w) {
              const int first = j * kTile + 32 * w - p, at = first >> 5;  // node of the word's first token
              uint32_t see = 0xffffffffu;
              if (first > -32) {
                const uint32_t lo = at < 0 ? 0xffffffffu : at == 0 ? s.x : at == 1 ? s.y : at == 2 ? s.z : at == 3 ? s.w : 0u;
                const uint32_t hi = at == -1 ? s.x : at == 0 ? s.y : at == 1 ? s.z : at == 2 ? s.w : 0u;
                see = __funnelshift_r(lo, hi, first & 31);
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) sv[32 * w + i] = (see >> i) & 1u ? sv[32 * w + i] : __float_as_uint(-INFINITY);
            }
          }
          float mx[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) mx[x] = fmaxf(__uint_as_float(sv[2 * x]), __uint_as_float(sv[2 * x + 1]));
#pragma unroll
          for (int x = 8; x < kTile; x += 2)
            mx[(x >> 1) & 3] = max3(mx[(x >> 1) & 3], __uint_as_float(sv[x]), __uint_as_float(sv[x + 1]));
          const float rmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          const float m_new = fmaxf(m_use, rmax * sl);
          const bool rescale = m_new > m_use + kRescaleLog2;  // also the first finite max
          float alpha = 1.f;
          if (rescale) {
            alpha = ex2(m_use - m_new);
            m_use = m_new;
          }
          if (j > j0 && __any_sync(0xffffffffu, rescale)) {  // O rows whose max moved (alpha = 1 elsewhere)
#pragma unroll 1
            for (int x = 0; x < D / 8; ++x) scale_cols8(o_col + 8 * x, alpha);  // (few registers: S is held)
          }
          const float mref = m_use == -INFINITY ? 0.f : m_use;
          const uint64_t sl2 = pack2(sl, sl), mref2 = pack2(-mref, -mref);
          uint64_t ls[2] = {0, 0};
#pragma unroll
          for (int h = 0; h < kParts; ++h) {
            constexpr int kWords = kTile / 2 / kParts;
            uint32_t pw[kWords];
#pragma unroll
            for (int x = 0; x < kWords; ++x) {
              const int cc = h * kWords + x;
              const uint64_t y = fma2(pack2(__uint_as_float(sv[2 * cc]), __uint_as_float(sv[2 * cc + 1])), sl2, mref2);
              const float e0 = ex2(lo2(y)), e1 = ex2(hi2(y));
              ls[x & 1] = add2(ls[x & 1], pack2(e0, e1));
              pw[x] = pack_bf16x2(e0, e1);
            }
            st_cols<kWords>(s_col + h * kWords, pw);
            if (short_seq) {  // the remainders (worked out again: there is no room to keep them beside S)
#pragma unroll
              for (int x = 0; x < kWords; ++x) {
                const int cc = h * kWords + x;
                const uint64_t y = fma2(pack2(__uint_as_float(sv[2 * cc]), __uint_as_float(sv[2 * cc + 1])), sl2, mref2);
                uint32_t hi;
                split_bf16x2(ex2(lo2(y)), ex2(hi2(y)), hi, pw[x]);
              }
              st_cols<kWords>(s_col + kTile / 2 + h * kWords, pw);
            }
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
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's rows, the next one's Q before them
      const bool whole = u.whole();
      const int slot = j0 > 0 ? 0 : 1, unit_b = u.b, unit_g = u.g;
      const int live = u.seq.n * a.n_rep;
      more = advance();
      if (more) load_q();
      if (!warp_wait(o_done, units & 1u)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) mbar_arrive(&ring_empty[slot_of(2 * c - 1)]);
      ++units;
      if (warp_real) {
        const int rows_here = min(32, live - (first_row + k * kRows + 32 * (warp & 3)));  // of this warp
        if (whole) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const size_t out_row = out_row_of(unit_b, unit_g);
          const uint32_t out_lo = static_cast<uint32_t>(out_row), out_hi = static_cast<uint32_t>(out_row >> 32);
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t v[32];
            tc::tmem_ld32(o_col + 32 * x, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[z] = pack_bf16x2(__uint_as_float(v[8 * y + 2 * z]) * inv, __uint_as_float(v[8 * y + 2 * z + 1]) * inv);
              *reinterpret_cast<uint4*>(stage + lane * C::kStagePitch + 16 * y) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int y = 0; y < 4; ++y) {  // 64 bytes of 8 rows at a time
              const int rr = 8 * y + (lane >> 2);
              const size_t to = __shfl_sync(0xffffffffu, out_lo, rr) |
                                (static_cast<size_t>(__shfl_sync(0xffffffffu, out_hi, rr)) << 32);
              const uint4 val = *reinterpret_cast<const uint4*>(stage + rr * C::kStagePitch + 16 * (lane & 3));
              if (rr < rows_here)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + to * D + 32 * x + 8 * (lane & 3)) = val;
            }
            __syncwarp();
          }
        } else {
          const size_t part = (static_cast<size_t>(range) * 2 + slot) * a.rows + row - lane;  // of lane 0's row
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            uint32_t v[32];
            tc::tmem_ld32(o_col + 32 * x, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int y = 0; y < 4; ++y)
                *reinterpret_cast<uint4*>(stage + lane * C::kStagePitch + 16 * y) =
                    make_uint4(v[16 * h + 4 * y], v[16 * h + 4 * y + 1], v[16 * h + 4 * y + 2], v[16 * h + 4 * y + 3]);
              __syncwarp();
#pragma unroll
              for (int y = 0; y < 4; ++y) {  // 64 bytes of 8 rows at a time
                const int rr = 8 * y + (lane >> 2);
                const uint4 val = *reinterpret_cast<const uint4*>(stage + rr * C::kStagePitch + 16 * (lane & 3));
                if (rr < rows_here) *reinterpret_cast<uint4*>(a.ws_o + (part + rr) * D + 32 * x + 16 * h + 4 * (lane & 3)) = val;
              }
              __syncwarp();
            }
          }
          if (lane < rows_here) *reinterpret_cast<float2*>(a.ws_ml + 2 * (part + lane)) = make_float2(m_use, l);
        }
      }
      tc::fence_before_sync();  // (O is read before the next unit's first P.V, which waits for its first P)
    }
    if (!ok) flag_error(a.err, RRA_ERR_TIMEOUT);
    tc::fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Output rows of the units that several ranges share, from their partials. A range writes the unit that it starts
// with into its slot 0 and the one that it ends with into slot 1, so a unit's partials are slot 1 of its first range and
// slot 0 of the following ones.
// Bound: latency (header, then maxima and partials together, then the rows) and L2's bandwidth. ROWS rows per warp at a
// time, so that a warp has 8 loads in flight: of one row where a unit has many partials, of four rows where it
// has two or three.
constexpr int kMergeWarps = 8;

template <int D, int ROWS>
__global__ void __launch_bounds__(32 * kMergeWarps) tree_merge_kernel(const TreeArgs a) {
  constexpr int E = D / 32;           // dims per lane
  constexpr int kBatch = 8 / ROWS;    // partials of a row loaded at a time, the first before the maxima are known
  constexpr int kGroup = 32 / ROWS;   // partials whose (max, sum) a warp looks at together
  const int lane = threadIdx.x & 31, mine = lane / kGroup, at = lane % kGroup;  // this lane's row of (max, sum), its partial
  const int row0 = (blockIdx.y * kMergeWarps + (threadIdx.x >> 5)) * ROWS;
  pdl_wait();
  pdl_launch_dependents();
  const int4 h = __ldcg(a.headers + blockIdx.x);
  const int n = h.x, first = h.y, b = h.z / a.Hkv, g = h.z - b * a.Hkv, rows = min(h.w, a.rows);
  // (what a range whose waits ran out has not written may be anything)
  if (n < 2 || first < 0 || first >= a.ranges || n > a.ranges - first || b < 0 || b >= a.B || g < 0 || row0 >= rows) return;
  const float2* ml = reinterpret_cast<const float2*>(a.ws_ml);
  auto slot = [&](int i, int row) { return static_cast<size_t>(2 * (first + i) + (i == 0 ? 1 : 0)) * a.rows + row; };
  float next[kBatch][ROWS][E];
  auto load = [&](int s) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        if (s + k < n && row0 + q < rows) {
          const float* o = a.ws_o + slot(s + k, row0 + q) * D + lane * E;
          if constexpr (E == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(o));
            next[k][q][0] = t.x, next[k][q][1] = t.y, next[k][q][2] = t.z, next[k][q][3] = t.w;
          } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(o));
            next[k][q][0] = t.x, next[k][q][1] = t.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) next[k][q][e] = 0.f;
        }
      }
  };
  load(0);
  float M = -INFINITY, l = 0.f;  // of row `mine`
  float acc[ROWS][E] = {};
  for (int s0 = 0; s0 < n; s0 += kGroup) {
    const float2 x = s0 + at < n && row0 + mine < rows ? __ldcg(ml + slot(s0 + at, row0 + mine)) : make_float2(-INFINITY, 0.f);
    float m = x.x;
#pragma unroll
    for (int d = kGroup / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    m = fmaxf(m, M);
    const float mref = m == -INFINITY ? 0.f : m;
    const float w = ex2(x.x - mref), keep = ex2(M - mref);
    float ls = w * x.y;
#pragma unroll
    for (int d = kGroup / 2; d > 0; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
    l = l * keep + ls;
    M = m;
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      const float f = __shfl_sync(0xffffffffu, keep, q * kGroup);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[q][e] *= f;
    }
    for (int i = s0; i < min(n, s0 + kGroup); i += kBatch) {
      float v[kBatch][ROWS][E];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int q = 0; q < ROWS; ++q)
#pragma unroll
          for (int e = 0; e < E; ++e) v[k][q][e] = next[k][q][e];
      load(i + kBatch);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int q = 0; q < ROWS; ++q) {
          const float ws = __shfl_sync(0xffffffffu, w, q * kGroup + i - s0 + k);  // (0 from n on)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[q][e] = fmaf(ws, v[k][q][e], acc[q][e]);
        }
    }
  }
#pragma unroll
  for (int q = 0; q < ROWS; ++q) {
    const float sum = __shfl_sync(0xffffffffu, l, q * kGroup), inv = sum > 0.f ? 1.f / sum : 0.f;
    if (row0 + q >= rows) continue;
    const int j = (row0 + q) / a.n_rep, i = row0 + q - j * a.n_rep;
    const size_t out_row = (static_cast<size_t>(b) * a.N + j) * a.Hq + g * a.n_rep + i;
    uint32_t out[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[q][e] * inv, acc[q][e + 1] * inv);
    uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + out_row * D + lane * E);
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
    else
      *to = out[0];
  }
}

template <int D, int ROWS>
cudaError_t launch_merge(const TreeArgs& a, cudaStream_t st) {
  const int headers = a.headers_by_unit ? a.B * a.Hkv : a.ranges;
  return launch_pdl(tree_merge_kernel<D, ROWS>, dim3(headers, (a.rows + kMergeWarps * ROWS - 1) / (kMergeWarps * ROWS)),
                    dim3(32 * kMergeWarps), 0, st, a);
}

template <int D, int NQ, bool PAGED>
cudaError_t launch_attn(const TreeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using C = Cfg<D, NQ, PAGED>;
  static int done[64] = {0};
  auto kern = tree_attn_kernel<D, NQ, PAGED>;
  cudaError_t e = ensure_smem(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  if constexpr (NQ == 2) {  // a block that asks for more registers than it was launched with would wait for them without end
    static std::atomic<int> regs{0};
    if (regs.load(std::memory_order_relaxed) == 0) {
      cudaFuncAttributes attr{};
      e = cudaFuncGetAttributes(&attr, kern);
      if (e != cudaSuccess) return e;
      regs.store(attr.numRegs, std::memory_order_relaxed);
    }
    if (regs.load(std::memory_order_relaxed) * C::kThreads < 256 * C::kSoftmaxRegs + 128 * C::kOtherRegs) return cudaErrorInvalidKernelImage;
  }
  e = launch_pdl(kern, dim3(static_cast<unsigned>(a.ranges) * a.row_ctas), dim3(C::kThreads), C::kSmemBytes, st, km, vm, a);
  if (e != cudaSuccess || a.ranges == 1) return e;
  // partials of a cut unit: about ranges / units, two or three where there are more units
  return a.headers_by_unit && a.ranges >= 4 * a.B * a.Hkv ? launch_merge<D, 1>(a, st) : launch_merge<D, 4>(a, st);
}

}  // namespace tree
}  // namespace rra
