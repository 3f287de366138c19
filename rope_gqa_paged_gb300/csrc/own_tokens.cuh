// Attention of each sequence's own tokens, [first_token, L_b), in shared-prefix attention: partials of
// a few query rows over a chunk of one sequence's paged cache, on the warp-level tensor cores.
//
// A unit is (sequence, KV head, slice of its query heads, chunk): up to 16 rows (hpc heads x gamma new
// tokens) that read the same keys. One warp takes one unit, alone in its CTA: it issues its own TMA
// copies into a ring of stages of 32 tokens of K and V (two of 16 KB at head dim 128, three of 8 KB at 64;
// boxes of 8-row groups as in shared_prefix.cuh) and consumes them, so there is no producer to wake, no
// barrier between warps and no merge of warps at the end of a unit, which for units of a few
// hundred tokens cost as much as the streaming itself (512 sequences of 1 to 256 own tokens behind
// 16384 shared ones: the whole call took 162 us with the decode kernel, whose CTAs of five warps share a
// unit, and 151 us with one-warp CTAs of 16 tokens per stage). The small CTAs also fit beside a prefix
// CTA that is still at work.
//
// Per stage (rows on N, tokens on M, as in decode_mma.cuh):
//   S^T [32 tokens x 8 NT rows] = K Q^T, softmax online in base 2, O^T [D x 8 NT rows] += V^T P^T
// P is rounded to bf16 (half a step, 2^-8 of each weight); in sequences of about kShortRow tokens or fewer, where
// such errors do not average out, P enters as that and the bf16 of its remainder (2^-16), as in the verify
// kernel, and behind a prefix of more than that all their tokens are one unit's. Maxima, sums and O stay in float32.
//
// Bound: HBM where units fill the SMs (1216 units of 1536 tokens, 8 KV heads of 128 dims: 7.0 TB/s with 8 rows,
// 6.5 with 16); with one unit per SM the warp's chain of products, shuffles and exponentials (0.36
// us per 16 tokens with 8 rows, 0.44 with 16; stages of 16 tokens took 0.66). K and V of 32 tokens arrive
// together, so that the loads of V need not wait for the softmax: slots given back one by one took
// 0.45 and 0.60 us (and 5 % less time on full SMs, where 24 KB per CTA let eight of them fit instead of
// six); a ring of twice to four times the depth changed nothing.
//
// Every unit leaves (o, m, l) in slot prefix_splits + split of its rows, or writes the rows when there
// is one slot. The kernel before this one (shared_prefix.cuh) may still be computing the prefix's
// partials: this one reads only what that kernel's predecessors wrote (past L1; that kernel let it
// start after it had waited for them), and its first CTA waits for that kernel, so that the merge
// finds both complete. Assumed, since the documentation promises it to the grid that waits and not to one that this
// grid lets start: what was visible to the prefix kernel after its wait is so here, read from L2.
#pragma once

#include <type_traits>

#include "decode_mma.cuh"
#include "shared_prefix.cuh"

namespace rra {
namespace own {

template <int D>
struct Cfg {
  static constexpr int kTok = kOwnStage;                    // tokens per stage
  static constexpr int kHalves = D / 64;
  static constexpr int kGroupBytes = 1024 * kHalves;       // 8 rows: their 64-dim halves, 1 KB each
  static constexpr int kTileBytes = kTok / 8 * kGroupBytes;  // K (or V) of a stage
  static constexpr int kStages = D == 128 ? 2 : 3;
  static constexpr int kOffBar = kStages * 2 * kTileBytes;
  static constexpr int kSmemBytes = 1024 + kOffBar + kStages * 8;
  static constexpr int kIds = kOwnMaxBlocks / 32;          // block ids per lane
  // Stages of a segment of a long chunk, for blocks of 8 tokens (twice and four times as many for 16 and more): at most
  // kOwnMaxBlocks blocks, and whole turns of the ring with both phases of its barriers.
  static constexpr int kSegStages = D == 128 ? 32 : 30;
  static_assert(kSegStages % (2 * kStages) == 0 && kSegStages * kTok / 8 <= kOwnMaxBlocks, "segments");
};

// The kTok tokens of a stage for NT tiles of 8 rows. k / v: shared addresses of K and V (v_gen: V's generic
// address); tok0: the first token; lim[n][j]: the last token that row 8 n + 2 (lane % 4) + j attends.
// CHECK: tokens from tok0 + valid on are none of the chunk's (their V rows are zeroed, so that nothing stale
// reaches the tensor cores), and rows may not see all tokens. SPLIT_P: P as a bf16 part and its remainder's.
template <int D, int NT, bool CHECK, bool SPLIT_P>
__device__ __forceinline__ void step(MmaWarpState<D> (&st)[NT], const uint32_t (&qb)[NT][D / 16][2], uint32_t k, uint32_t v,
                                     uint8_t* v_gen, int tok0, int valid, const int (&lim)[NT][2], int lane,
                                     float scale_log2) {
  using C = Cfg<D>;
  constexpr int U = C::kTok / 16;
  if (CHECK && valid < C::kTok) {
    for (int i = lane; i < (C::kTok - valid) * C::kHalves * 8; i += 32) {
      const int r = valid + i / (C::kHalves * 8), h = (i / 8) % C::kHalves, c = i % 8;
      *reinterpret_cast<uint4*>(v_gen + (r >> 3) * C::kGroupBytes + h * 1024 + (r & 7) * 128 + 16 * c) =
          make_uint4(0u, 0u, 0u, 0u);
    }
    __syncwarp();
  }
  const int mat = lane >> 3, r8 = lane & 7;
  float s[NT][U][2][4];  // two accumulators: half the chain of dependent products
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[n][u][0][c] = s[n][u][1][c] = 0.f;
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t a[4];
      ldsm_x4(k + (2 * u + (mat & 1)) * C::kGroupBytes + (kk >> 2) * 1024 + swz(r8, ((kk & 3) << 1) + (mat >> 1)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_bf16(s[n][u][kk & 1], a, qb[n][kk][0], qb[n][kk][1]);
    }
  uint32_t b[NT][U][2], b_lo[NT][U][2];
  const int t_lane = lane >> 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float x[2][2 * U], mnew[2];
    bool grow = false;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float mx = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2 * U; ++h) {  // token 8 h + lane / 4
        const float sum = s[n][h >> 1][0][2 * (h & 1) + j] + s[n][h >> 1][1][2 * (h & 1) + j];
        const int t = 8 * h + t_lane;
        x[j][h] = !CHECK || (tok0 + t <= lim[n][j] && t < valid) ? sum * scale_log2 : -INFINITY;
        mx = fmaxf(mx, x[j][h]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      mnew[j] = fmaxf(st[n].m[j], mx);
      grow |= mnew[j] > st[n].m[j];
    }
    if (__any_sync(0xffffffffu, grow)) {
      float alpha[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        alpha[j] = mnew[j] > st[n].m[j] ? exp2f(st[n].m[j] - mnew[j]) : 1.f;
        st[n].l[j] *= alpha[j];
        st[n].m[j] = mnew[j];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        st[n].o[i][0] *= alpha[0];
        st[n].o[i][1] *= alpha[1];
        st[n].o[i][2] *= alpha[0];
        st[n].o[i][3] *= alpha[1];
      }
    }
    float p[2][2 * U];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float mref = st[n].m[j] == -INFINITY ? 0.f : st[n].m[j];
#pragma unroll
      for (int h = 0; h < 2 * U; ++h) {
        p[j][h] = exp2f(x[j][h] - mref);
        st[n].l[j] += p[j][h];
      }
    }
#pragma unroll
    for (int h = 0; h < 2 * U; ++h) {
      uint32_t hi, lo;
      split_bf16x2(p[0][h], p[1][h], hi, lo);
      b[n][h >> 1][h & 1] = movmatrix_trans(hi);
      if constexpr (SPLIT_P) b_lo[n][h >> 1][h & 1] = movmatrix_trans(lo);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      uint32_t a[4];
      ldsm_x4_trans(v + (2 * u + (mat >> 1)) * C::kGroupBytes + (i >> 2) * 1024 + swz(r8, ((i & 3) << 1) + (mat & 1)), a);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_bf16(st[n].o[i], a, b[n][u][0], b[n][u][1]);
        if constexpr (SPLIT_P) mma_bf16(st[n].o[i], a, b_lo[n][u][0], b_lo[n][u][1]);
      }
    }
}

// ALONE: of short sequences behind a prefix that has a pass of its own, all tokens are the first unit's.
template <int D, int NT, bool ALONE>
__global__ void __launch_bounds__(32) own_tokens_kernel(const __grid_constant__ CUtensorMap k_map,
                                                        const __grid_constant__ CUtensorMap v_map, const DecodeArgs a) {
  using C = Cfg<D>;
  constexpr int kTok = C::kTok;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);

  const int lane = threadIdx.x;
  const int n_rep = a.Hq / a.Hkv, gamma = a.gamma, hpc = a.hpc;
  const int slices = (n_rep + hpc - 1) / hpc;
  const int g = blockIdx.x / slices, slice = blockIdx.x - g * slices;  // KV heads innermost: neighbours in memory
  const int split = blockIdx.y, b = blockIdx.z;
  const int rows = min(hpc, n_rep - slice * hpc) * gamma;
  // output row of unit row r: new token r % gamma of head r / gamma of the slice
  auto out_row = [&](int r) {
    const int hh = r / gamma;
    return (static_cast<size_t>(b) * gamma + (r - hh * gamma)) * a.Hq + g * n_rep + slice * hpc + hh;
  };
  // This kernel does not end before the one before it: its first CTA waits for that.
  auto leave = [&]() {
    if (a.prefix_splits > 0 && blockIdx.x == 0 && split == 0 && b == 0) pdl_wait();
  };

  if (a.prefix_splits == 0) pdl_wait();
  pdl_launch_dependents();
  int start = a.first_token + split * a.chunk, chunk = a.chunk;
  int first_blk = start >> a.log2_bs;
  int32_t ids[C::kIds];  // lane's block ids of the chunk (of a segment of a long one), loaded before its length is known
  auto load_ids = [&]() {
    const int32_t* row = a.block_table + static_cast<size_t>(b) * a.max_blocks_per_seq;
    const int prefix_blks = a.prefix_len >> a.log2_bs;
    const int reach = min(((chunk - 1) >> a.log2_bs) + 2, a.max_blocks_per_seq - first_blk);
#pragma unroll
    for (int k = 0; k < C::kIds; ++k) {
      const int i = lane + 32 * k, blk = first_blk + i;
      ids[k] = i < reach ? __ldcg((blk < prefix_blks ? a.prefix_blocks : row) + blk) : 0;
    }
  };
  load_ids();
  int p0, L;  // row (j, head) attends [0, p0 + j]
  if (a.positions != nullptr) {
    p0 = __ldcg(a.positions + b);
    if (p0 < a.prefix_len || p0 > a.capacity - gamma) {
      if (lane == 0 && blockIdx.x == 0 && split == 0) flag_error(a.err, RRA_ERR_POSITION);
      leave();
      return;
    }
    L = p0 + gamma;
  } else {
    L = __ldcg(a.seq_lens + b);
    if (L < 0 || L > a.capacity) {
      if (lane == 0 && blockIdx.x == 0 && split == 0) flag_error(a.err, RRA_ERR_SEQ_LEN);
      L = min(max(L, 0), a.capacity);
    }
    p0 = L - gamma;
  }
  const bool short_seq = spx::short_sequence(a, L);
  const bool alone = ALONE && short_seq && a.prefix_splits > 0;
  const int fits = alone ? spx::kShortTokens : spx::own_chunk(a, L);
  const bool moved = fits != chunk;
  if (moved) {
    chunk = fits;
    start = (alone ? 0 : a.first_token) + split * chunk;
  }
  if (start >= L) {
    if (a.num_splits == 1)  // no merge: the empty sequence's rows are zero
      for (int i = lane; i < rows * D; i += 32)
        static_cast<__nv_bfloat16*>(a.out)[out_row(i / D) * D + i % D] = __float2bfloat16_rn(0.f);
    leave();
    return;
  }
  if (lane == 0) {
    prefetch_tensormap(&k_map);
    prefetch_tensormap(&v_map);
    for (int s = 0; s < C::kStages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  asm volatile("fence.proxy.async.global;" ::: "memory");  // the append's writes, for the copies
  __syncwarp();

  // one segment, or more of a chunk that has grown
  const int chunk_end = min(L, start + chunk);
  const int seg_tokens = moved && !alone ? kTok * C::kSegStages << min(a.log2_bs - 3, 2) : chunk;
  int end = 0, n_stages = 0, issued = 0;
  // stage st: tokens start + st kTok ..., one copy per box and lane, K in the even lanes and V in the odd ones
  const int bs = 1 << a.log2_bs, box = min(bs, kTok);
  auto issue = [&](int st) {
    const int s = st % C::kStages, tok0 = start + st * kTok;
    const int nbox = (min(kTok, end - tok0) + box - 1) / box;
    if (lane == 0) mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(2 * nbox * box * 128 * C::kHalves));
    const int t = tok0 + (lane >> 1) * box, i = (t >> a.log2_bs) - first_blk;
    int id = 0;
#pragma unroll
    for (int k = 0; k < C::kIds; ++k) {
      const int x = __shfl_sync(0xffffffffu, ids[k], i & 31);
      if ((i >> 5) == k) id = x;
    }
    __syncwarp();
    if (lane < 2 * nbox) {
      const int rows8 = (id << (a.log2_bs - 3)) + ((t & (bs - 1)) >> 3);
      uint8_t* dst = smem + (2 * s + (lane & 1)) * C::kTileBytes + (lane >> 1) * (box >> 3) * C::kGroupBytes;
      spx::tma_g2s_5d(dst, (lane & 1) ? &v_map : &k_map, 0, 0, 0, rows8, g, &full[s]);
    }
  };
  uint32_t qb[NT][D / 16][2];
  int lim[NT][2];
  MmaWarpState<D> st[NT];
  // Q^T as the B operand: tile n, lane holds row 8 n + lane / 4, dims 16 kk + 2 (lane % 4) + {0, 1} and (+ 8)
  auto load_rows = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 8 * n + (lane >> 2);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(a.q) + out_row(r < rows ? r : 0) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qb[n][kk][0] = r < rows ? __ldcg(q + kk * 8 + (lane & 3)) : 0u;
        qb[n][kk][1] = r < rows ? __ldcg(q + kk * 8 + 4 + (lane & 3)) : 0u;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int rr = 8 * n + 2 * (lane & 3) + j;
        lim[n][j] = rr < rows ? p0 + rr % gamma : -1;
        st[n].m[j] = -INFINITY;
        st[n].l[j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i) st[n].o[i][0] = st[n].o[i][1] = st[n].o[i][2] = st[n].o[i][3] = 0.f;
    }
  };
  bool ok = true;
  auto consume = [&](int it, auto split_p) {
    const int s = it % C::kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(&full[s], (it / C::kStages) & 1))) {
      ok = false;
      return;
    }
    uint8_t* kst = smem + 2 * s * C::kTileBytes;
    uint8_t* vst = kst + C::kTileBytes;
    const int tok0 = start + it * kTok;
    const int valid = min(end - tok0, kTok);
    if (!split_p.value && valid == kTok && tok0 + kTok - 1 <= p0)
      step<D, NT, false, split_p.value>(st, qb, smem_addr(kst), smem_addr(vst), vst, tok0, kTok, lim, lane, a.scale_log2);
    else
      step<D, NT, true, split_p.value>(st, qb, smem_addr(kst), smem_addr(vst), vst, tok0, valid, lim, lane, a.scale_log2);
    __syncwarp();  // every lane has read the stage
    if (issued < n_stages) {
      issue(issued);
      ++issued;
    }
  };
#pragma unroll 1
  for (bool again = false;; again = true) {
    end = min(chunk_end, start + seg_tokens);
    n_stages = (end - start + kTok - 1) / kTok;
    if (again || moved) {
      first_blk = start >> a.log2_bs;
      load_ids();
    }
    const int n_blk = ((end - 1) >> a.log2_bs) - first_blk + 1;
#pragma unroll
    for (int k = 0; k < C::kIds; ++k)
      if (lane + 32 * k < n_blk && (ids[k] < 0 || ids[k] >= a.num_blocks)) {
        flag_error(a.err, RRA_ERR_BLOCK_ID);
        ids[k] = 0;
      }
    for (issued = 0; issued < min(C::kStages, n_stages); ++issued) issue(issued);
    if (!again) load_rows();
    if (short_seq) {
#pragma unroll 1
      for (int it = 0; ok && it < n_stages; ++it) consume(it, std::true_type());
    } else {
#pragma unroll 1
      for (int it = 0; ok && it < n_stages; ++it) consume(it, std::false_type());
    }
    if (!ok || end == chunk_end) break;
    start = end;
  }
  if (!ok) {  // no copy may still be landing when the CTA exits
    if (lane == 0) {
      flag_error(a.err, RRA_ERR_TIMEOUT);
      for (int it = max(issued - C::kStages, 0); it < issued; ++it) mbar_wait(&full[it % C::kStages], (it / C::kStages) & 1);
    }
    __syncwarp();
  }

#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float l = st[n].l[j];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      const int r = 8 * n + 2 * (lane & 3) + j, d = lane >> 2;
      if (r >= rows) continue;
      const size_t row = out_row(r);
      if (a.num_splits == 1) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D + d;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          out[16 * i] = __float2bfloat16_rn(st[n].o[i][j] * inv);
          out[16 * i + 8] = __float2bfloat16_rn(st[n].o[i][2 + j] * inv);
        }
      } else {
        const size_t ps = row * a.num_splits + a.prefix_splits + split;
        float* o = a.ws_o + ps * D + d;  // eight lanes write 32 bytes of a row
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          o[16 * i] = st[n].o[i][j];
          o[16 * i + 8] = st[n].o[i][2 + j];
        }
        if (d == 0) *reinterpret_cast<float2*>(a.ws_ml + 2 * ps) = make_float2(st[n].m[j], l);
      }
    }
  leave();
}

template <int D, int NT, bool ALONE>
cudaError_t launch(const DecodeArgs& a, const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t st) {
  using C = Cfg<D>;
  static int done[64] = {0};
  auto kern = own_tokens_kernel<D, NT, ALONE>;
  cudaError_t e = ensure_smem(kern, C::kSmemBytes, done);
  if (e != cudaSuccess) return e;
  const int n_rep = a.Hq / a.Hkv;
  const dim3 grid(a.Hkv * ((n_rep + a.hpc - 1) / a.hpc), a.num_splits - a.prefix_splits, a.B);
  return launch_pdl(kern, grid, dim3(32), C::kSmemBytes, st, km, vm, a);
}

}  // namespace own
}  // namespace rra
