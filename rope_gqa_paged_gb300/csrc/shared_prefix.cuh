// Attention of a whole batch over a prefix that all its sequences share, on the fifth-generation
// tensor cores: the prefix part of rra_shared_prefix_attn.
//
// Softmax over the tokens [0, n) splits at the prefix length P by log-sum-exp: with m_i, l_i, o_i
// the maximum, the sum and the unnormalised output over part i, out = sum 2^(m_i - M) o_i / sum
// 2^(m_i - M) l_i. The part [0, P) has the same K and V for every sequence, so for one KV head it is
// the attention of B x gamma x n_rep query rows over P keys: a pair of matrix products whose K and V
// are read once for all the rows. The part [P, n) is decode_verify_kernel<SHARED> (verify.cuh),
// which also merges the partials.
//
// One CTA takes 128 of those rows (M of every MMA) and a chunk of the prefix. Q, S, P and O live in
// Tensor Memory, so shared memory holds nothing but a ring of K and V tiles of 16 KB (64 keys at
// head dim 128, 128 keys at 64; TMA, 128-byte swizzle, 64-dim halves) and two CTAs fit an SM. For
// key tile j:
//   S = Q K_j^T     D / 16 MMAs (M 128, N kTile, K 16), Q the A operand from Tensor Memory
//   softmax         warps 0-3, one row per thread: the S row into registers, running max (moved only
//                   when it grows by more than 2^8), P as bf16 pairs over the S columns
//   O += P V_j      kTile / 16 MMAs, P the A operand from Tensor Memory, V an MN-major operand
// One lane of warp 5 issues S_0, PV_0, S_1, PV_1, ...; the MMAs run in issue order, so S_(j+1) may
// overwrite P_j, and s_full(j + 1) also says that PV_j is complete and O may be rescaled. While one
// CTA of an SM is in its softmax the other's MMAs run. P is rounded to bf16 (2^-8 of each weight,
// below what the bf16 output keeps); maxima, sums and O stay in float32.
//
// Every wait is bounded (a timeout sets RRA_ERR_TIMEOUT and the roles drain); the MMA lane waits for
// its last commit and the producer for its last copies before Tensor Memory is released.
#pragma once

#include "decode_mma.cuh"
#include "tcgen05.cuh"
#include "verify.cuh"

namespace rra {
namespace spx {

constexpr int kRows = kSharedPrefixRows;        // M of every MMA
constexpr int kRing = 6;                        // K / V tile slots (K_0, V_0, K_1, V_1, ...)
constexpr uint32_t kTmemCols = 256;             // two CTAs per SM share its 512 columns
constexpr float kRescaleLog2 = 8.f;             // move the running max only when it grows by more
constexpr int kSoftmaxThreads = 128;
constexpr int kProducerWarp = 4, kMmaWarp = 5;
constexpr int kThreads = kSoftmaxThreads + 64;

template <int D>
struct Cfg {
  static constexpr int kTile = 8192 / D;                   // keys per tile
  static constexpr int kHalves = D / 64;
  static constexpr int kHalfBytes = kTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;  // 16 KB
  static constexpr uint32_t kColO = 0;                     // O: D columns
  static constexpr uint32_t kColS = D;                     // S: kTile columns; P over its first half
  static constexpr uint32_t kColQ = D + kTile;             // Q as bf16 pairs: D / 2 columns
  static constexpr int kOffBar = kRing * kTileBytes;
  // q_ready, ring_full[kRing], ring_empty[kRing], s_full, p_full, mma_done
  static constexpr int kNumBars = 1 + 2 * kRing + 3;
  static constexpr int kOffTmemSlot = kOffBar + kNumBars * 8;
  static constexpr int kOffTable = kOffTmemSlot + 16;
  static constexpr int kSmemBytes = 1024 + kOffTable + kSharedPrefixTableEntries * 4;
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(kRows, kTile, false);  // Q (K-major) . K^T (K-major)
  static constexpr uint32_t kIdescPV = tc::idesc_bf16_f32(kRows, D, true);      // P (K-major) . V (MN-major)
  static_assert(kColQ + D / 2 <= kTmemCols, "Tensor Memory columns");
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ float ex2(float x) {  // 2^x on the special-function unit (2^-inf = 0)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
#pragma unroll
  for (int c = 0; c < N / 32; ++c) {
    uint32_t t[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) t[i] = s[32 * c + i];
    tc::tmem_st32(taddr + 32 * c, t);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                         const DecodeArgs a) {
  using C = Cfg<D>;
  constexpr int kTile = C::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

  const int g = blockIdx.z, split = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int start = split * a.prefix_chunk;
  const int end = min(a.prefix_len, start + a.prefix_chunk);
  const int n_tiles = (end - start + kTile - 1) / kTile;
  const int last_valid = end - start - (n_tiles - 1) * kTile;  // keys of the last tile

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* q_ready = bars;
  uint64_t* ring_full = bars + 1;
  uint64_t* ring_empty = ring_full + kRing;
  uint64_t* s_full = ring_empty + kRing;
  uint64_t* p_full = s_full + 1;
  uint64_t* mma_done = p_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffTmemSlot);
  int32_t* tbl = reinterpret_cast<int32_t*>(smem + C::kOffTable);

  if (threadIdx.x == 0) {
    mbar_init(q_ready, kSoftmaxThreads);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, kSoftmaxThreads);
    mbar_init(mma_done, 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
    tc::fence_before_sync();
  }
  // The kernel after this one reads the same inputs without waiting for this one, so it may start
  // only when this wait is over: every kernel before this one has then completed.
  pdl_wait();
  pdl_launch_dependents();
  const int first_blk = start >> a.log2_bs;
  {
    const int n_blk = ((end - 1) >> a.log2_bs) - first_blk + 1;
    for (int i = threadIdx.x; i < n_blk; i += kThreads) {
      int id = a.prefix_blocks[first_blk + i];
      if (id < 0 || id >= a.num_blocks) {
        flag_error(a.err, RRA_ERR_BLOCK_ID);
        id = 0;
      }
      tbl[i] = id;
    }
  }
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  // ring position r: K of tile r / 2 (r even) or its V (r odd), in slot r % kRing
  auto slot_of = [](int r) { return r % kRing; };
  auto phase_of = [](int r) { return static_cast<uint32_t>((r / kRing) & 1); };

  if (warp == kProducerWarp) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
    const int bs = 1 << a.log2_bs;
    const int box = min(bs, kTile);  // rows per TMA box, as the tensor maps were encoded
    int issued = 0;
    for (int r = 0; r < 2 * n_tiles; ++r) {
      const int s = slot_of(r);
      const int tile0 = start + (r >> 1) * kTile;
      const int nbox = (min(kTile, end - tile0) + box - 1) / box;
      int ok = 1;
      if (lane == 0) {
        if (r >= kRing && !mbar_wait(&ring_empty[s], phase_of(r) ^ 1u))
          ok = 0;
        else
          mbar_arrive_expect_tx(&ring_full[s], static_cast<uint32_t>(nbox * box * 128 * C::kHalves));
      }
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const CUtensorMap* map = (r & 1) ? &v_map : &k_map;
      uint8_t* dst = smem + s * C::kTileBytes;
      for (int c = lane; c < C::kHalves * nbox; c += 32) {  // (box, half) copies, from all lanes at once
        const int bx = c / C::kHalves, hf = c % C::kHalves;
        const int t = tile0 + bx * box;
        tma_g2s_4d(dst + hf * C::kHalfBytes + bx * box * 128, map, 64 * hf, g, t & (bs - 1),
                   tbl[(t >> a.log2_bs) - first_blk], &ring_full[s]);
      }
      __syncwarp();
      issued = r + 1;
    }
    if (lane == 0) {
      if (issued < 2 * n_tiles) flag_error(a.err, RRA_ERR_TIMEOUT);
      // no copy may still be landing when the CTA exits
      for (int r = max(issued - kRing, 0); r < issued; ++r) mbar_wait(&ring_full[slot_of(r)], phase_of(r));
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------ MMA issue (one lane)
    if (lane == 0) {
      const uint32_t ring_base = smem_addr(smem);
      bool ok = mbar_wait(q_ready, 0);
      tc::fence_after_sync();
      auto issue_s = [&](int j) -> bool {
        const int r = 2 * j;
        if (!mbar_wait(&ring_full[slot_of(r)], phase_of(r))) return false;
        tc::fence_after_sync();
        const uint32_t k_base = ring_base + slot_of(r) * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_bf16_ts(tmem + C::kColS, tmem + C::kColQ + 8 * kk,
                          tc::sw128_desc(k_base + (kk >> 2) * C::kHalfBytes + (kk & 3) * 32, 1024, 1024), C::kIdescS,
                          kk > 0 ? 1u : 0u);
        tc::commit(s_full);
        tc::commit(&ring_empty[slot_of(r)]);
        return true;
      };
      if (ok) ok = issue_s(0);
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int rv = 2 * j + 1;
        if (!mbar_wait(&ring_full[slot_of(rv)], phase_of(rv)) || !mbar_wait(p_full, j & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t v_base = ring_base + slot_of(rv) * C::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          tc::mma_bf16_ts(tmem + C::kColO, tmem + C::kColS + 8 * kk,
                          tc::sw128_desc(v_base + kk * 2048, C::kHalfBytes, 1024), C::kIdescPV,
                          (j > 0 || kk > 0) ? 1u : 0u);
        tc::commit(&ring_empty[slot_of(rv)]);
        if (j + 1 < n_tiles) ok = issue_s(j + 1);
      }
      if (!ok) flag_error(a.err, RRA_ERR_TIMEOUT);
      tc::commit(mma_done);  // every MMA issued above has completed once this arrives
      mbar_wait(mma_done, 0);
    }
  } else {
    // ------------------------------------------------------------------ softmax: thread = query row
    const int n_rep = a.Hq / a.Hkv;
    const int row = blockIdx.x * kRows + static_cast<int>(threadIdx.x);
    const bool real = row < a.B * a.gamma * n_rep;
    const bool warp_real = __any_sync(0xffffffffu, real);
    const int bt = real ? row / n_rep : 0;                 // token bt = b * gamma + j of the batch
    const int i = real ? row - bt * n_rep : 0;             // head of the group
    const int b = bt / a.gamma, j_new = bt - b * a.gamma;
    // keys of the prefix that the row attends
    int lim = a.prefix_len;
    if (real) {
      int L = a.positions != nullptr ? a.positions[b] + a.gamma : a.seq_lens[b];
      L = min(max(L, 0), a.capacity);
      lim = min(max(L - a.gamma + 1 + j_new, 0), a.prefix_len);
    }
    const uint32_t lane_base = static_cast<uint32_t>(32 * warp) << 16;
    const uint32_t s_col = tmem + lane_base + C::kColS, o_col = tmem + lane_base + C::kColO;
    {  // the query row into Tensor Memory: dims (2c, 2c + 1) in column kColQ + c
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        (static_cast<size_t>(bt) * a.Hq + g * n_rep + i) * D);
      uint32_t qw[D / 2];
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
        qw[4 * c] = x.x;
        qw[4 * c + 1] = x.y;
        qw[4 * c + 2] = x.z;
        qw[4 * c + 3] = x.w;
      }
      st_cols<D / 2>(tmem + lane_base + C::kColQ, qw);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      mbar_arrive(q_ready);
    }
    const float sl = a.scale_log2;
    float m_use = -INFINITY, l = 0.f;  // running max (log2 units) and sum
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      if (!warp_wait(s_full, j & 1)) {  // S_j is there, and P.V of tile j - 1 is complete
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (j == n_tiles - 1 && last_valid < kTile) {
        // keys past the prefix: their V rows are whatever the slot held; zeros keep 0 * V at 0
        const int rv = 2 * j + 1;
        if (!warp_wait(&ring_full[slot_of(rv)], phase_of(rv))) {
          ok = false;
          break;
        }
        const int r = static_cast<int>(threadIdx.x);
        if (r >= last_valid && r < kTile) {
          uint8_t* vrow = smem + slot_of(rv) * C::kTileBytes + r * 128;
#pragma unroll
          for (int h = 0; h < C::kHalves; ++h)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4*>(vrow + h * C::kHalfBytes + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_smem_to_async();
      }
      if (warp_real) {
        uint32_t sv[kTile];
        ld_cols<kTile>(s_col, sv);
        const int vis = min(lim, end) - (start + j * kTile);  // columns this row attends
        if (__any_sync(0xffffffffu, vis < kTile)) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) sv[c] = c < vis ? sv[c] : __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) mx[c] = __uint_as_float(sv[c]);
#pragma unroll
        for (int c = 8; c < kTile; ++c) mx[c & 7] = fmaxf(mx[c & 7], __uint_as_float(sv[c]));
        const float rmax = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
        const float m_new = fmaxf(m_use, rmax * sl);
        const bool rescale = m_new > m_use + kRescaleLog2;  // also the first finite max
        float alpha = 1.f;
        if (rescale) {
          alpha = ex2(m_use - m_new);
          m_use = m_new;
        }
        const float mref = m_use == -INFINITY ? 0.f : m_use;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pw[kTile / 2];
#pragma unroll
        for (int c = 0; c < kTile / 2; ++c) {
          const float e0 = ex2(fmaf(__uint_as_float(sv[2 * c]), sl, -mref));
          const float e1 = ex2(fmaf(__uint_as_float(sv[2 * c + 1]), sl, -mref));
          ls[c & 3] += e0 + e1;
          pw[c] = pack_bf16x2(e0, e1);
        }
        st_cols<kTile / 2>(s_col, pw);
        l = l * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
        if (j > 0 && __any_sync(0xffffffffu, rescale)) {  // O rows whose max moved (alpha = 1 elsewhere)
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tc::tmem_ld32(o_col + 32 * c, v);
            tc::tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * alpha);
            tc::tmem_st32(o_col + 32 * c, v);
          }
        }
        tc::tmem_wait_st();
      }
      tc::fence_before_sync();
      mbar_arrive(p_full);
    }
    // ------------------------------------------------------------------ epilogue: this chunk's partial rows
    if (ok && warp_wait(mma_done, 0)) {
      tc::fence_after_sync();
      const SharedRows rows{a.Hkv, n_rep, a.hpc, a.gamma};
      const size_t ps = rows(b, g, i, j_new) * a.num_splits + split;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tc::tmem_ld32(o_col + 32 * c, v);
        tc::tmem_wait_ld();
        if (!real) continue;
        float4* po = reinterpret_cast<float4*>(a.ws_o + ps * D) + 8 * c;
#pragma unroll
        for (int x = 0; x < 8; ++x)
          po[x] = make_float4(__uint_as_float(v[4 * x]), __uint_as_float(v[4 * x + 1]), __uint_as_float(v[4 * x + 2]),
                              __uint_as_float(v[4 * x + 3]));
      }
      if (real) *reinterpret_cast<float2*>(a.ws_ml + 2 * ps) = make_float2(m_use, l);
    } else {
      flag_error(a.err, RRA_ERR_TIMEOUT);
    }
    tc::fence_before_sync();
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch_prefix(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  static int done[64] = {0};
  auto kern = shared_prefix_kernel<D>;
  cudaError_t e = ensure_smem(kern, Cfg<D>::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  // row tiles innermost: CTAs that read the same keys run side by side and share them through L2
  const int rows = a.B * a.gamma * (a.Hq / a.Hkv);
  const dim3 grid((rows + kRows - 1) / kRows, a.prefix_splits, a.Hkv);
  return launch_pdl(kern, grid, dim3(kThreads), Cfg<D>::kSmemBytes, st, km, vm, a);
}

}  // namespace spx
}  // namespace rra
