// Softmax cross entropy through a frozen output head, and its gradient, without a t x v matrix of
// logits: l = X.W^T (X t x h hidden states, W v x h head, both bf16),
//   lse_i = log sum_v exp(l_iv),  loss_i = lse_i - l_i[y_i]  (0 where y_i is not counted),
//   dX_i  = sum_v g_iv W_v,  g_iv = a_i p_iv - b_i [v = y_i],  p_iv = exp(l_iv - lse_i),
//   b_i   = dloss_i (0 where y_i is not counted),  a_i = b_i + dlse_i.
//
// vocab_gemm_kernel is one persistent tcgen05 GEMM with four epilogues. The vocabulary is walked in
// pieces of 128 columns: a CTA pair computes 256 tokens x 256 columns of logits into tensor memory
// (fp32) and its epilogue reduces them there:
//   kVocabStats   a token's reference point (its maximum) and sum of exp(l - reference) over the piece,
//                 and the target's logit
//   kVocabScaled  the same with the target's logit as the reference, and exp(l - reference) in bf16
//   kVocabProb    g in bf16 but for the target's term, lse being known
//   kVocabGrad    (the second product, dX = g.W) dX in bf16, or fp32 partial tiles of a split K
// Only statistics leave the first kernel: 8 bytes per token and piece instead of 512. The backward
// holds g (or the scaled exponentials) of a bounded run of tokens at a time in the workspace.
// vocab_narrow_kernel and vocab_narrow_grad_kernel do the same for few tokens, with the operands'
// roles exchanged.
//
// Loss and gradient in one call form the logits once: exp(l - l[y]) needs nothing that is not known
// when a piece's logits are, floating point keeps its relative precision whatever its scale, and the
// row's factor exp(l[y] - lse) and then its dloss are applied to the finished dX (their product may be
// too small for fp32 where the gradient is not). The logits l[y] come first, from a
// kernel of their own (t dot products). The target's own term is left out of g and added in fp32 as
// (a.p[y] - b).W[y] (with one call dloss.(exp(-loss) - 1).W[y]), so that a confident token's small
// difference is not one of two rounded numbers and the largest term is not rounded to bf16. Only where
// some logit exceeds its row's target by more than 60 (a loss above 60) could the sums overflow: the piece
// then raises a flag, and kVocabProb runs again over the run with its lse (otherwise that launch returns
// at once).
//
// Logits are accumulated 512 inputs at a time in tensor memory and summed in the epilogue's registers.
// The tensor core truncates its fp32 sum after every 16 inputs: over 4096 (8192) inputs a logit then
// comes out 5e-6 (1.1e-5) of itself too small, which the loss, an fp32 value, would show; by pieces of
// 512 it is 6e-7. The second product, whose operand g and result are bf16, is accumulated 8192 words at a
// time in the same way: 512 truncations of 2^-23 at most, 6e-5 of the terms' magnitudes.
//
// Bound: the tensor cores (2thv per product) for more than a few hundred tokens, reading W for few.
// The design follows from the first: cta_group::2 (256 x 256 x 16 per instruction, each CTA loading
// half of A and half of B), a TMA ring of three stages of two K-steps, and two accumulators in tensor
// memory, so that a tile's epilogue (eight warps) runs under the next tile's products. g is rounded to
// bf16 because it is an operand of a bf16 product: 2^-8 of each term at most, as dX's own rounding.
// Measured on 32000 x 4096, 4096 tokens: loss and gradient 1590 to 1690 us, two products at 1.27 to 1.35
// PFLOP/s, where the card is at its power limit (1.39 in a plain bf16 product); 1 token: loss 50 us, W read once.
//
// Every wait is bounded (qlora::mbar_wait); on expiry the CTA reports QLORA_DEV_TIMEOUT, stops
// issuing, waits for its own copies and MMAs in flight, frees TMEM and returns.
#pragma once

#include "nf4_gemm.cuh"

namespace qlora {

namespace vg {
constexpr int BM = 256, BN = 256, BK = 64;   // per CTA pair
constexpr int KS = 2;                        // K-steps of 64 per stage
constexpr int STAGES = 3;
constexpr int ATOM = 128 * BK * 2;           // this CTA's half of A, or of B, for one step
constexpr int A_BYTES = KS * ATOM;
constexpr int STAGE_BYTES = 2 * A_BYTES;
constexpr int CHUNK = 4;                     // stages per accumulation of logits (K = 512)
constexpr int GRAD_CHUNK = 64;               // and of dX (K = 8192 words)
constexpr int PIECE = 128;                   // columns of a tile that one epilogue warp reduces
constexpr int kEpiWarps = 8;                 // four for each half of a tile's columns
constexpr int kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 10 * 32;
constexpr int kStaging = kEpiWarps * 4096;   // a 32-row x 128-byte tile per epilogue warp
constexpr int kTmemCols = 512;
constexpr size_t smem_bytes() { return 1024 + STAGES * STAGE_BYTES + kStaging + 256; }
static_assert(smem_bytes() <= 232448, "fits the opt-in shared memory of one CTA");
constexpr float kLog2e = 1.4426950408889634f;
}  // namespace vg

enum VocabMode : int { kVocabStats = 0, kVocabScaled = 1, kVocabProb = 2, kVocabGrad = 3 };

struct VocabGemmArgs {
  int M, N;              // rows and columns of the product (N: v, or h for kVocabGrad)
  int num_kb;            // stages of 128 along K
  int m_tiles, n_tiles;
  int m_group;           // row tiles that are walked together, column tile by column tile
  int whole;             // tiles computed in one piece; the ones behind are split along K
  int splits, kb_per_split;
  int items;             // whole + (tiles - whole) * splits
  int ldp;               // columns of the stored g (v rounded up to 64)
  const int64_t* targets;
  int64_t ignore;
  float2* stats;         // M x pieces: (reference point, sum of exp(l - reference))
  float* target_logit;   // M: the targets' logits, from this product
  const float* ref;      // kVocabScaled: the same, known beforehand: the reference points
  const float* lse;      // kVocabProb
  const float* dloss;
  const float* dlse;     // or NULL
  unsigned* redo;        // kVocabScaled: raised by rows it cannot serve. kVocabProb: NULL, or the flag
                         // without which there is nothing to do. kVocabGrad: see row_factor
  const float* factor;   // kVocabGrad: NULL, or the rows' factors, by which (and by dloss) g is still to be multiplied
  float* target_factor;  // kVocabProb writes, kVocabGrad reads: the factors of the targets' W
  int v;                 // kVocabGrad: the vocabulary (N is h there)
  const uint16_t* W;
};

struct VocabItem {
  int m0, n0, nt, kb0, kb1, part;   // part: the partial tile's index, or -1
};
__device__ __forceinline__ VocabItem vocab_item(const VocabGemmArgs& a, int item) {
  VocabItem it;
  int tile = item;
  it.kb0 = 0;
  it.kb1 = a.num_kb;
  it.part = -1;
  if (item >= a.whole) {
    const int j = item - a.whole, sp = j % a.splits;
    tile = a.whole + j / a.splits;
    it.kb0 = sp * a.kb_per_split;
    it.kb1 = min(a.num_kb, it.kb0 + a.kb_per_split);
    if (a.splits > 1) it.part = j;
  }
  const int per = a.m_group * a.n_tiles, g = tile / per, rem = tile - g * per;
  const int gm = min(a.m_group, a.m_tiles - g * a.m_group);
  it.nt = rem / gm;
  it.m0 = (g * a.m_group + rem - it.nt * gm) * vg::BM;
  it.n0 = it.nt * vg::BN;
  return it;
}

// dX from the second product: a row's factor and dloss times it, plus its target's factor times W[target].
// Without factors, or after kVocabProb ran again (g is then complete), both are 1, or 0 for a row that counts
// for nothing: its g is zero, but zero times a word that is not finite is not.
struct RowFactor {
  float f, d, ft;
  __device__ __forceinline__ float times(float v, float t) const {   // a row that counts for nothing: exactly zero
    return f == 0.f ? 0.f : fmaf(v * f, d, ft * t);
  }
  const uint16_t* w;   // the target's row of W, or NULL
  // eight columns from `col` on (col < the row's length, a multiple of 8)
  __device__ __forceinline__ void apply(float (&v)[8], int col) const {
    float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (w) unpack8(ldg_vec(w, col >> 3), t);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = times(v[e], t[e]);
  }
};
__device__ __forceinline__ RowFactor row_factor(const VocabGemmArgs& a, int row) {
  RowFactor r;
  r.f = r.d = r.ft = 0.f;
  r.w = nullptr;
  if (row >= 0) {
    if (a.factor && *a.redo == 0u) {
      r.f = a.factor[row];   // (zero for a row that is not counted)
      r.d = a.dloss[row];
    } else {
      const int64_t y = a.targets[row];
      const bool counted = y >= 0 && y < a.v && y != a.ignore;
      r.f = (counted && a.dloss[row] != 0.f) || (a.dlse && a.dlse[row] != 0.f) ? 1.f : 0.f;
      r.d = 1.f;
    }
    r.ft = a.target_factor[row];
    if (r.ft != 0.f) r.w = a.W + a.targets[row] * a.N;   // (counted: inside the vocabulary)
  }
  return r;
}

// The reference point of a row's piece whose logits have maximum m: the target's logit c where it
// serves (kScaled, a counted row), the maximum itself else. An infinite one is no reference point:
// exp(l) itself then sums to 0 or to infinity (base).
struct RowRef {
  float ref, base;
  bool redo;
};
template <bool kScaled>
__device__ __forceinline__ RowRef row_ref(float m, float c, bool counted) {
  RowRef r;
  r.redo = kScaled && counted && m - c > 60.f;
  r.ref = kScaled && counted && !r.redo ? c : m;
  r.base = fabsf(r.ref) == INFINITY ? 0.f : r.ref;
  return r;
}

template <int kMode>
__global__ void __launch_bounds__(vg::kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmPart,
                      const VocabGemmArgs args) {
  using namespace vg;
  auto chunk_end = [](const VocabItem& it, int kc) {
    return min(it.kb1, kc + (kMode == kVocabGrad ? GRAD_CHUNK : CHUNK));
  };
  constexpr bool kBmn = kMode == kVocabGrad;   // W as the K-major operand (logits) or the MN-major one
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + STAGES * STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + kStaging);
  uint64_t* empty = full + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint64_t* acc_empty = acc_full + 2;      // even CTA: both CTAs have drained the accumulator
  uint64_t* drained = acc_empty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  pdl_launch_dependents();
  if (kMode == kVocabProb) {
    pdl_wait();
    if (args.redo && *args.redo == 0u) return;   // (the whole grid alike)
  }
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());   // 0: MMA issuer, 1: its peer
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(drained, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc2(tmem_holder, kTmemCols);
    tmem_relinquish2();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
  }
  if (kMode != kVocabProb) pdl_wait();   // (before anything is read that a kernel of the same call wrote)
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == kTmaWarp) {
    // both CTAs' copies count on the even CTA's barrier: the MMA issuer waits for one barrier, and
    // no thread of the odd CTA has to pass the news on (a relay cost 930 cycles a K-step of 512)
    const uint32_t full0 = cluster_smem_addr(full, 0);
    int g = 0;
    bool ok = true;
    for (int item = pair; ok && item < args.items; item += pairs) {
      const VocabItem it = vocab_item(args, item);
      for (int kb = it.kb0; kb < it.kb1; ++kb, ++g) {
        const int slot = g % STAGES;
        if (!mbar_wait_warp(&empty[slot], ((g / STAGES) & 1) ^ 1u, abort_flag)) { ok = false; break; }
        uint8_t* dst = smem + slot * STAGE_BYTES;
        const uint32_t bar = full0 + static_cast<uint32_t>(slot * sizeof(uint64_t));
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * STAGE_BYTES);
#pragma unroll
          for (int s = 0; s < KS; ++s) {   // (a step behind K's end is filled with zeros)
            const int k = (kb * KS + s) * BK;
            uint8_t *a_dst = dst + s * ATOM, *b_dst = dst + A_BYTES + s * ATOM;
            tma_load_2d_pair(a_dst, &tmA, bar, k, it.m0 + rank * 128);
            if (!kBmn) {
              tma_load_2d_pair(b_dst, &tmB, bar, k, it.n0 + rank * 128);
            } else {
              tma_load_2d_pair(b_dst, &tmB, bar, it.n0 + rank * 128, k);
              tma_load_2d_pair(b_dst + 8192, &tmB, bar, it.n0 + rank * 128 + 64, k);
            }
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0 && *abort_flag) {
      // no copy may still be writing shared memory when its CTA exits: the even CTA waits for its
      // stages (both CTAs' bytes); the odd one, whose copies count there, gives its own, at most
      // STAGES of them, a thousand times a copy's latency (and stays until the cluster's barrier)
      if (rank == 0)
        for (int j = (g > STAGES ? g - STAGES : 0); j < g; ++j) mbar_drain(&full[j % STAGES], (j / STAGES) & 1);
      else
        for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    }
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      constexpr uint32_t kIdesc = idesc_bf16(BM, BN, false, kBmn);
      const uint32_t a_lo0 = sw128_desc_lo(smem_addr(smem), 16);
      const uint32_t b_lo0 = sw128_desc_lo(smem_addr(smem) + A_BYTES, kBmn ? 8192 : 16);
      int g = 0, n = 0;
      bool ok = true;
      for (int item = pair; ok && item < args.items; item += pairs) {
        const VocabItem it = vocab_item(args, item);
        for (int kc = it.kb0, ke; ok && kc < it.kb1; kc = ke, ++n) {   // one accumulation
          const int buf = n & 1;
          ke = chunk_end(it, kc);
          if (!mbar_wait_warp(&acc_empty[buf], ((n >> 1) & 1) ^ 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          for (int kb = kc; kb < ke; ++kb, ++g) {
            const int slot = g % STAGES;
            const uint32_t ph = (g / STAGES) & 1;
            if (!mbar_wait_warp(&full[slot], ph, abort_flag)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_lo = a_lo0 + slot * (STAGE_BYTES >> 4), b_lo = b_lo0 + slot * (STAGE_BYTES >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < KS * (BK / 16); ++k) {
                const uint32_t s = (k / (BK / 16)) * (ATOM >> 4), kk = k % (BK / 16);
                umma2_bf16(tmem_base + buf * BN, sw128_desc_of(a_lo + s + kk * 2),
                           sw128_desc_of(b_lo + s + kk * (kBmn ? 128 : 2)), kIdesc, (kb > kc || k > 0) ? 1u : 0u);
              }
              umma2_commit_multicast(&empty[slot], 0x3);   // frees the stage in both CTAs
            }
            __syncwarp();
          }
          if (elect_one()) umma2_commit_multicast(&acc_full[buf], 0x3);
          __syncwarp();
        }
      }
      // every MMA has read its operands before the CTAs leave (elect picks the lane that issued them)
      if (elect_one()) {
        umma2_commit_multicast(drained, 0x1);
        mbar_drain(drained, 0);
      }
      __syncwarp();
    }
  } else {
    // -------- epilogue: warp w has accumulator rows 32 (w mod 4) .. of this CTA, a row per lane, and the
    // columns 128 (w / 4) .. of the tile --------
    uint8_t* stage = staging + warp * 4096;
    const int quad = warp & 3, half = warp >> 2;
    int n = 0;
    // Stores 32 rows x 128 bytes at (x, y) of `map`: each lane's row as eight 16-byte chunks, 128-byte
    // swizzled (eight lanes' stores hit eight bank groups), by one TMA store.
    auto store_tile = [&](const uint4 (&q)[8], const CUtensorMap* map, int x, int y, bool any) {
      if (lane == 0) bulk_wait_group_read<0>();   // the store before has read the tile
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) = q[k];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (any) tma_store_2d(map, stage, x, y);
        bulk_commit_group();
      }
    };
    // One lane polls, with pauses: 256 threads polling the barrier through a whole main loop take
    // shared-memory bandwidth that the MMAs read their operands with.
    auto wait_acc = [&]() {
      bool ready = true;
      if (lane == 0) {
        for (int i = 0; i < 16384 && !mbar_try_wait(&acc_full[n & 1], (n >> 1) & 1) && !*abort_flag; ++i) __nanosleep(32);
        ready = mbar_wait(&acc_full[n & 1], (n >> 1) & 1, abort_flag);
      }
      ready = __shfl_sync(0xFFFFFFFFu, ready, 0);
      tc_fence_after();
      return ready;
    };
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * PIECE);
    auto release_acc = [&]() {   // the last read of this accumulation is behind
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(&acc_empty[n & 1], 0);
      ++n;
    };
    bool ok = true;
    for (int item = pair; ok && item < args.items; item += pairs) {
      const VocabItem it = vocab_item(args, item);
      const int row0 = it.m0 + rank * 128 + quad * 32, row = row0 + lane;
      const int n0 = it.n0 + half * PIECE;   // this warp's first column
      const bool rok = row < args.M;
      RowFactor rf;
      if (kMode == kVocabGrad) rf = row_factor(args, it.part < 0 && rok ? row : -1);   // (loaded under the products)
      // the tile's sums over its accumulations: the first one as it comes, all of its columns in flight, the
      // others 16 columns at a time (the sums leave no room for more)
      float s[PIECE];
#pragma unroll 1
      for (int kc = it.kb0; kc < it.kb1; kc = chunk_end(it, kc)) {
        if (!wait_acc()) { ok = false; break; }
        const uint32_t acc = lane_addr + (n & 1) * BN;
        if (kc == it.kb0) {
#pragma unroll
          for (int c = 0; c < PIECE; c += 16) tmem_ld_16(acc + c, *reinterpret_cast<uint32_t(*)[16]>(&s[c]));
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int c = 0; c < PIECE; c += 16) {
            uint32_t v[16];
            tmem_ld_16(acc + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) s[c + e] += __uint_as_float(v[e]);
          }
        }
        release_acc();
      }
      if (!ok) break;
      if (kMode == kVocabGrad) {
#pragma unroll
        for (int c = 0; c < PIECE; c += 64) {
          uint4 q[8];
          if (it.part < 0) {
            if (n0 + c >= args.N) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float (&f)[8] = *reinterpret_cast<float(*)[8]>(&s[c + 8 * k]);
              if (n0 + c + 8 * k < args.N) rf.apply(f, n0 + c + 8 * k);
              q[k] = pack8(f);
            }
            store_tile(q, &tmOut, n0 + c, row0, row0 < args.M);
          } else {
#pragma unroll
            for (int part = 0; part < 2; ++part) {
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float* f = &s[c + 32 * part + 4 * k];
                q[k] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
              }
              store_tile(q, &tmPart, half * PIECE + c + 32 * part, it.part * BM + rank * 128 + quad * 32, true);
            }
          }
        }
        continue;
      }
      // ---- logits ----------------------------------------------------------------------------------
      const int vcols = args.N - n0;   // columns behind the vocabulary read as zero products and count as -inf
      if (vcols < PIECE) {
#pragma unroll
        for (int e = 0; e < PIECE; ++e) s[e] = e < vcols ? s[e] : -INFINITY;
      }
      const int64_t y = rok ? __ldg(args.targets + row) : -1;
      const bool counted = y >= 0 && y < args.N && y != args.ignore;
      const int tcol = counted && y >= n0 && y < n0 + PIECE ? static_cast<int>(y - n0) : -1;
      const bool any_target = __any_sync(0xFFFFFFFFu, tcol >= 0);   // few pieces hold a target of the warp's rows
      if (kMode == kVocabProb) {
        const float b = counted ? __ldg(args.dloss + row) : 0.f;
        const float a = b + (rok && args.dlse ? __ldg(args.dlse + row) : 0.f);
        const float nl = rok ? -__ldg(args.lse + row) * kLog2e : 0.f;
        // a row that counts for nothing is zero whatever its logits are
#pragma unroll
        for (int e = 0; e < PIECE; ++e) s[e] = a != 0.f ? a * ex2(fmaf(s[e], kLog2e, nl)) : 0.f;
        float ft = 0.f;
        if (any_target) {
#pragma unroll
          for (int e = 0; e < PIECE; ++e) {
            ft = e == tcol ? s[e] - b : ft;
            s[e] = e == tcol ? 0.f : s[e];
          }
        }
        if (rok && (tcol >= 0 || (!counted && n0 == 0))) args.target_factor[row] = ft;
      } else {
        constexpr bool kScaled = kMode == kVocabScaled;
        if (any_target) {
          float ty = 0.f;
#pragma unroll
          for (int e = 0; e < PIECE; ++e) ty = e == tcol ? s[e] : ty;
          if (tcol >= 0) args.target_logit[row] = ty;
        }
        float m = s[0];
#pragma unroll
        for (int e = 1; e < PIECE; ++e) m = fmaxf(m, s[e]);
        const RowRef rr = row_ref<kScaled>(m, kScaled && counted ? __ldg(args.ref + row) : 0.f, counted);
        if (kScaled && rr.redo) *args.redo = 1u;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int e = 0; e < PIECE; e += 2) {
          s[e] = ex2((s[e] - rr.base) * kLog2e);   // (exact near the reference, which a product with
          s[e + 1] = ex2((s[e + 1] - rr.base) * kLog2e);   // log2 e rounded first would not be)
          s0 += s[e];
          s1 += s[e + 1];
        }
        if (rok) args.stats[(static_cast<int64_t>(row) * args.n_tiles + it.nt) * (BN / PIECE) + half] = make_float2(rr.ref, s0 + s1);
        if (kScaled && any_target) {
#pragma unroll
          for (int e = 0; e < PIECE; ++e) s[e] = e == tcol ? 0.f : s[e];
        }
      }
      if (kMode != kVocabStats) {
#pragma unroll
        for (int c = 0; c < PIECE; c += 64) {
          if (n0 + c >= args.ldp) break;
          uint4 q[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) q[k] = pack8(*reinterpret_cast<const float(*)[8]>(&s[c + 8 * k]));
          store_tile(q, &tmOut, n0 + c, row0, row0 < args.M);
        }
      }
    }
    if (lane == 0) bulk_wait_group<0>();   // the output is written before the CTA retires
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may still signal it or read its TMEM slice
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc2(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------------------------------------
// Few tokens: bound by reading W. The operands change places, D^T = W.X^T, so that an instruction
// computes 128 words x N tokens with N the tokens rounded up to 16 instead of 256 of them, and the
// pipeline holds little but W. A CTA takes one contiguous run of the vocabulary in units of 32 words
// (a warp's rows of an accumulator), which balances the card to a unit whatever the vocabulary;
// statistics are kept per unit. A warp's lanes are words and its columns tokens: the maximum over a
// column is one reduction instruction, the sums of 16 columns 16 shuffles.
// ------------------------------------------------------------------------------------------
namespace vn {
constexpr int kMaxTokens = 80;    // an epilogue thread's sums: one register per token
constexpr int CHUNK = 4;          // stages per accumulation of logits (K = 512), as above
constexpr int GRAD_CHUNK = 64;    // and of dX (K = 8192 words)
constexpr int BM = 128, BK = 64;
constexpr int KS = 2;             // K-steps of 64 per stage: a stage's waits and copies cost some 700 cycles
                                  // whatever it holds, so that 16 KB of W each were not enough to keep up with HBM
constexpr int kUnit = 32;         // words per unit
constexpr int A_ATOM = BM * BK * 2;      // 128 words (or columns of h) x 64 K
constexpr int A_BYTES = KS * A_ATOM;
constexpr int MAX_STAGES = 6;
constexpr int kThreads = 6 * 32, kTmaWarp = 4, kMmaWarp = 5;
constexpr int kTokenBytes = kMaxTokens * 5 * 4;
constexpr int kRoom = 232448 - 1024 - kTokenBytes - 512;
__host__ __device__ constexpr int tokens16(int t) { return (t + 15) / 16 * 16; }
__host__ __device__ constexpr int stage_bytes(int n16) { return A_BYTES + KS * n16 * BK * 2; }
__host__ __device__ constexpr int stages(int n16) {
  return kRoom / stage_bytes(n16) < MAX_STAGES ? kRoom / stage_bytes(n16) : MAX_STAGES;
}
constexpr size_t smem_bytes(int n16) {
  return 1024 + static_cast<size_t>(stages(n16)) * stage_bytes(n16) + kTokenBytes + 512;
}
}  // namespace vn

struct VocabNarrowArgs {
  int t, n16;            // tokens, and rounded up to 16
  int v, h;
  int num_kb;            // stages of 128 along K: of h, or for the gradient of ldp
  int units;             // ldp / 32
  int ldp;
  int tiles;             // the gradient: 128-column tiles of h
  const int64_t* targets;
  int64_t ignore;
  float2* stats;         // t x units
  float* target_logit;
  const float* ref;
  const float* lse;
  const float* dloss;
  const float* dlse;
  float* target_factor;
  unsigned* redo;
  uint16_t* g;           // t x ldp
  float* part;           // the gradient's partial tiles: [slot][token][128]
};

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(x));
  return r;
}

// One CTA's shared memory, barriers and tensor memory, the same for both kernels below.
struct NarrowCta {
  uint8_t* stage;
  uint64_t *full, *empty, *acc_full, *acc_empty;
  uint32_t* tmem_holder;
  volatile uint32_t* abort_flag;
  float* token;          // 5 values per token
  int stages, stage_bytes;
  uint32_t tmem_cols, tmem;
};
__device__ __forceinline__ NarrowCta narrow_setup(uint8_t* smem_raw, int n16) {
  NarrowCta c;
  c.stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  c.stages = vn::stages(n16);
  c.stage_bytes = vn::stage_bytes(n16);
  c.token = reinterpret_cast<float*>(c.stage + c.stages * c.stage_bytes);
  c.full = reinterpret_cast<uint64_t*>(c.token + 5 * vn::kMaxTokens);
  c.empty = c.full + vn::MAX_STAGES;
  c.acc_full = c.empty + vn::MAX_STAGES;
  c.acc_empty = c.acc_full + 2;
  c.tmem_holder = reinterpret_cast<uint32_t*>(c.acc_empty + 2);
  c.abort_flag = c.tmem_holder + 1;
  c.tmem_cols = 32;
  while (c.tmem_cols < 2u * n16) c.tmem_cols *= 2;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < c.stages; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.acc_full[b], 1);
      mbar_init(&c.acc_empty[b], 4);
    }
    *c.abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == vn::kMmaWarp) {
    tmem_alloc(c.tmem_holder, c.tmem_cols);
    tmem_relinquish();
  }
  return c;
}
__device__ __forceinline__ void narrow_begin(NarrowCta& c) {
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = *c.tmem_holder;
}
__device__ __forceinline__ void narrow_end(const NarrowCta& c) {
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == vn::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(c.tmem, c.tmem_cols);
  }
}
// A position in the ring: kept by counting, since dividing by a ring size that is known only at run time
// takes hundreds of cycles, once or more per K-step.
struct RingPos {
  int slot = 0;
  uint32_t phase = 0;
  int done = 0;          // stages passed
  __device__ __forceinline__ void next(int stages) {
    ++done;
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
};
// The MMA warp's part of one accumulator: `steps` K-steps from the ring at position g.
template <bool kAmn>
__device__ __forceinline__ bool narrow_mma(const NarrowCta& c, int n16, int buf, int n, int steps, RingPos& g) {
  if (!mbar_wait_warp(&c.acc_empty[buf], ((n >> 1) & 1) ^ 1u, c.abort_flag)) return false;
  tc_fence_after();
  const uint32_t idesc = idesc_bf16(vn::BM, n16, kAmn, false);
  const uint32_t a_lo0 = sw128_desc_lo(smem_addr(c.stage), kAmn ? 8192 : 16);
  const uint32_t b_lo0 = sw128_desc_lo(smem_addr(c.stage) + vn::A_BYTES, 16);
  for (int k = 0; k < steps; ++k, g.next(c.stages)) {
    const int slot = g.slot;
    if (!mbar_wait_warp(&c.full[slot], g.phase, c.abort_flag)) return false;
    tc_fence_after();
    const uint32_t a_lo = a_lo0 + slot * (c.stage_bytes >> 4), b_lo = b_lo0 + slot * (c.stage_bytes >> 4);
    if (elect_one()) {
#pragma unroll
      for (int s = 0; s < vn::KS; ++s)
#pragma unroll
        for (int kk = 0; kk < vn::BK / 16; ++kk)
          umma_bf16(c.tmem + buf * (c.tmem_cols / 2),
                    sw128_desc_of(a_lo + s * (vn::A_ATOM >> 4) + kk * (kAmn ? 128 : 2)),
                    sw128_desc_of(b_lo + s * n16 * (vn::BK * 2 / 16) + kk * 2), idesc,
                    (k > 0 || s > 0 || kk > 0) ? 1u : 0u);
      umma_commit(&c.empty[slot]);
    }
    __syncwarp();
  }
  if (elect_one()) umma_commit(&c.acc_full[buf]);
  __syncwarp();
  return true;
}
// After an abort: no copy may still be writing shared memory, no MMA reading it, when the CTA exits.
__device__ __forceinline__ void narrow_drain_copies(const NarrowCta& c, const RingPos& g) {
  if (*c.abort_flag)
    for (int j = (g.done > c.stages ? g.done - c.stages : 0); j < g.done; ++j)
      mbar_drain(&c.full[j % c.stages], (j / c.stages) & 1);
}
__device__ __forceinline__ void narrow_drain_mma(const NarrowCta& c, const RingPos& g) {
  // (each stage's commit arrives on its `empty` barrier and covers all MMAs before it)
  if (*c.abort_flag && g.done > 0) mbar_drain(&c.empty[(g.done - 1) % c.stages], ((g.done - 1) / c.stages) & 1);
}

template <int kMode>
__global__ void __launch_bounds__(vn::kThreads, 1)
    vocab_narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmWu,
                        const __grid_constant__ CUtensorMap tmX, const VocabNarrowArgs args) {
  using namespace vn;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  if (kMode == kVocabProb) {
    pdl_wait();
    if (args.redo && *args.redo == 0u) return;   // (the whole grid alike)
  }
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  NarrowCta cta = narrow_setup(smem_raw, args.n16);
  if (kMode != kVocabProb) pdl_wait();
  // per token: what the epilogue needs of it (a word that is nobody's target: -1)
  float *t_ref = cta.token, *t_a = cta.token + kMaxTokens, *t_b = cta.token + 2 * kMaxTokens;
  int* t_word = reinterpret_cast<int*>(cta.token + 3 * kMaxTokens);
  for (int n = threadIdx.x; n < args.n16; n += kThreads) {
    const int64_t y = n < args.t ? args.targets[n] : -1;
    const bool counted = y >= 0 && y < args.v && y != args.ignore;
    t_word[n] = counted ? static_cast<int>(y) : -1;
    if (kMode == kVocabScaled) t_ref[n] = counted ? args.ref[n] : 0.f;
    if (kMode == kVocabProb) {
      const float b = counted ? args.dloss[n] : 0.f;
      t_b[n] = b;
      t_a[n] = b + (n < args.t && args.dlse ? args.dlse[n] : 0.f);
      t_ref[n] = n < args.t ? -args.lse[n] * vg::kLog2e : 0.f;
    }
  }
  narrow_begin(cta);
  const int u0 = unit_row(args.units, gridDim.x, blockIdx.x), u1 = unit_row(args.units, gridDim.x, blockIdx.x + 1);

  if (warp == kTmaWarp) {   // (warp-uniform, an elected lane issuing: one lane's branch takes hundreds of cycles a stage)
    RingPos g;
    bool ok = true;
    for (int u = u0; ok && u < u1; u += 4) {
      const int nu = min(4, u1 - u);
      for (int kb = 0; kb < args.num_kb; ++kb, g.next(cta.stages)) {
        const int slot = g.slot;
        if (!mbar_wait_warp(&cta.empty[slot], g.phase ^ 1u, cta.abort_flag)) { ok = false; break; }
        uint8_t* dst = cta.stage + slot * cta.stage_bytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&cta.full[slot], KS * (nu * (kUnit * BK * 2) + args.n16 * (BK * 2)));
#pragma unroll
          for (int s = 0; s < KS; ++s) {   // (a step behind h is filled with zeros)
            const int x = (kb * KS + s) * BK;
            if (nu == 4) {   // (one copy of 128 rows: four of 32 take longer)
              tma_load_2d(dst + s * A_ATOM, &tmW, &cta.full[slot], x, u * kUnit);
            } else {
              for (int i = 0; i < nu; ++i)
                tma_load_2d(dst + s * A_ATOM + i * (kUnit * BK * 2), &tmWu, &cta.full[slot], x, (u + i) * kUnit);
            }
            tma_load_2d(dst + A_BYTES + s * args.n16 * (BK * 2), &tmX, &cta.full[slot], x, 0);
          }
        }
        __syncwarp();
      }
    }
    if (lane == 0) narrow_drain_copies(cta, g);
  } else if (warp == kMmaWarp) {
    RingPos g;
    int n = 0;
    // (a last tile of fewer than four units leaves the other rows of its operand as they were: their
    // accumulator rows are not read)
    bool ok = true;
    for (int u = u0; ok && u < u1; u += 4)
      for (int kc = 0; ok && kc < args.num_kb; kc += CHUNK, ++n)
        ok = narrow_mma<false>(cta, args.n16, n & 1, n, min(CHUNK, args.num_kb - kc), g);
    narrow_drain_mma(cta, g);
  } else {
    int n = 0;
    bool ok = true;
    for (int u = u0; ok && u < u1; u += 4) {
      float s[kMaxTokens];
#pragma unroll
      for (int j = 0; j < kMaxTokens; ++j) s[j] = 0.f;
#pragma unroll 1
      for (int kc = 0; kc < args.num_kb; kc += CHUNK, ++n) {
        const int buf = n & 1;
        if (!mbar_wait_warp(&cta.acc_full[buf], (n >> 1) & 1, cta.abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t taddr = cta.tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * (cta.tmem_cols / 2);
        if (u + warp < u1) {
#pragma unroll
          for (int c = 0; c < kMaxTokens; c += 16) {
            if (c >= args.n16) break;
            uint32_t v[16];
            tmem_ld_16(taddr + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) s[c + j] += __uint_as_float(v[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cta.acc_empty[buf]);
      }
      const int unit = u + warp;
      if (ok && unit < u1) {
        const int word = unit * kUnit + lane;
        const bool wok = word < args.v;
#pragma unroll
        for (int c = 0; c < kMaxTokens; c += 16) {
          if (c >= args.n16) break;
          const float* v = &s[c];
          float p[16];
          if (kMode == kVocabProb) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float a = t_a[c + j];
              // a row that counts for nothing is zero whatever its logits are
              p[j] = wok && a != 0.f ? a * ex2(fmaf(v[j], vg::kLog2e, t_ref[c + j])) : 0.f;
              const int w = t_word[c + j];
              if (word == w) {
                args.target_factor[c + j] = p[j] - t_b[c + j];
                p[j] = 0.f;
              }
              if (w < 0 && word == 0 && c + j < args.t) args.target_factor[c + j] = 0.f;
            }
          } else {
            constexpr bool kScaled = kMode == kVocabScaled;
            float mine = 0.f;    // the reference of this lane's token (lane / 2) below
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float l = wok ? v[j] : -INFINITY;
              const int w = t_word[c + j];
              const RowRef rr = row_ref<kScaled>(warp_max(l), kScaled ? t_ref[c + j] : 0.f, w >= 0);
              if (kScaled && rr.redo && lane == 0) *args.redo = 1u;
              if (word == w) args.target_logit[c + j] = l;
              if ((lane >> 1) == j) mine = rr.ref;
              p[j] = wok ? ex2((l - rr.base) * vg::kLog2e) : 0.f;
            }
            float q[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) q[j] = p[j];
            // sums of 16 columns over the lanes: each exchange halves the columns a lane holds
#pragma unroll
            for (int o = 16; o > 1; o >>= 1) {
#pragma unroll
              for (int j = 0; j < o / 2; ++j) {
                const float keep = (lane & o) ? q[j + o / 2] : q[j], give = (lane & o) ? q[j] : q[j + o / 2];
                q[j] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
              }
            }
            q[0] += __shfl_xor_sync(0xFFFFFFFFu, q[0], 1);
            const int tok = c + (lane >> 1);
            if (!(lane & 1) && tok < args.t)
              args.stats[static_cast<int64_t>(tok) * args.units + unit] = make_float2(mine, q[0]);
            if (kScaled) {
#pragma unroll
              for (int j = 0; j < 16; ++j) p[j] = word == t_word[c + j] ? 0.f : p[j];
            }
          }
          if (kMode != kVocabStats) {
#pragma unroll
            for (int j = 0; j < 16; ++j)   // a token's 32 words: 64 contiguous bytes
              if (c + j < args.t)
                args.g[static_cast<int64_t>(c + j) * args.ldp + word] = __bfloat16_as_ushort(__float2bfloat16_rn(p[j]));
          }
        }
      }
    }
  }
  narrow_end(cta);
}

// The second product for few tokens, dX^T = W^T.g^T: the K-steps of all 128-column tiles of h in one
// line, an equal contiguous run of them to each CTA, whose share of a tile goes to a partial tile of
// its own (number CTA + tile); vocab_narrow_join_kernel adds a tile's shares in order.
__global__ void __launch_bounds__(vn::kThreads, 1)
    vocab_narrow_grad_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmG,
                             const VocabNarrowArgs args) {
  using namespace vn;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  NarrowCta cta = narrow_setup(smem_raw, args.n16);
  pdl_wait();
  narrow_begin(cta);
  const int total = args.tiles * args.num_kb;
  const int x0 = unit_row(total, gridDim.x, blockIdx.x), x1 = unit_row(total, gridDim.x, blockIdx.x + 1);
  auto share_end = [&](int x) { return min(x1, (x / args.num_kb + 1) * args.num_kb); };

  if (warp == kTmaWarp) {
    RingPos g;
    int tile = x0 / args.num_kb, kb = x0 - tile * args.num_kb;
    for (int x = x0; x < x1; ++x, g.next(cta.stages)) {
      const int slot = g.slot;
      if (!mbar_wait_warp(&cta.empty[slot], g.phase ^ 1u, cta.abort_flag)) break;
      uint8_t* dst = cta.stage + slot * cta.stage_bytes;
      if (elect_one()) {
        mbar_arrive_expect_tx(&cta.full[slot], cta.stage_bytes);
#pragma unroll
        for (int s = 0; s < KS; ++s) {   // (a step behind ldp is filled with zeros)
          const int k = (kb * KS + s) * BK;
          tma_load_2d(dst + s * A_ATOM, &tmW, &cta.full[slot], tile * BM, k);
          tma_load_2d(dst + s * A_ATOM + 8192, &tmW, &cta.full[slot], tile * BM + 64, k);
          tma_load_2d(dst + A_BYTES + s * args.n16 * (BK * 2), &tmG, &cta.full[slot], k, 0);
        }
      }
      __syncwarp();
      if (++kb == args.num_kb) {
        kb = 0;
        ++tile;
      }
    }
    if (lane == 0) narrow_drain_copies(cta, g);
  } else if (warp == kMmaWarp) {
    RingPos g;
    int n = 0;
    bool ok = true;
    for (int x = x0; ok && x < x1;)
      for (const int end = share_end(x); ok && x < end; x = min(end, x + GRAD_CHUNK), ++n)   // one accumulation
        ok = narrow_mma<true>(cta, args.n16, n & 1, n, min(end - x, GRAD_CHUNK), g);
    narrow_drain_mma(cta, g);
  } else {
    int n = 0;
    bool ok = true;
    for (int x = x0, end; ok && x < x1; x = end) {
      end = share_end(x);
      float* dst = args.part + static_cast<int64_t>(blockIdx.x + x / args.num_kb) * args.n16 * BM + warp * 32 + lane;
      for (int k = x; k < end; k += GRAD_CHUNK, ++n) {
        const int buf = n & 1;
        if (!mbar_wait_warp(&cta.acc_full[buf], (n >> 1) & 1, cta.abort_flag)) { ok = false; break; }
        tc_fence_after();
        const uint32_t taddr = cta.tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * (cta.tmem_cols / 2);
        // a share's later accumulations are added to what this thread stored of the ones before
        for (int c = 0; c < args.n16; c += 16) {
          uint32_t v[16];
          tmem_ld_16(taddr + c, v);
          tmem_ld_wait();
          float* d = dst + static_cast<int64_t>(c) * BM;
          if (k > x) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < args.t) v[j] = __float_as_uint(d[j * BM] + __uint_as_float(v[j]));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < args.t) d[j * BM] = __uint_as_float(v[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&cta.acc_empty[buf]);
      }
    }
  }
  narrow_end(cta);
}

// ------------------------------------------------------------------------------------------
// rows
// ------------------------------------------------------------------------------------------
struct VocabRowArgs {
  const float2* stats;        // t x pieces
  const float* target_logit;
  const float* ref;           // with dloss: what the stored exponentials are relative to
  const int64_t* targets;
  int64_t ignore;
  int t, v, pieces;
  float* loss;
  float* lse;
  const float* dloss;         // NULL, or: make the rows' factors
  float* factor;
  float* target_factor;
};

// Joins two pieces of a row: the larger reference point is the new one, as in any running softmax. A
// sum is zero or infinite only where all or some of its logits are infinite.
__device__ __forceinline__ float2 join_stats(float2 p, float2 q) {
  const float m = fmaxf(p.x, q.x);
  const float r = fabsf(m) == INFINITY ? 0.f : m;
  // a piece whose reference is infinite was summed against 0
  const float pr = fabsf(p.x) == INFINITY ? 0.f : p.x, qr = fabsf(q.x) == INFINITY ? 0.f : q.x;
  const float ps = p.y == 0.f ? 0.f : p.y * ex2((pr - r) * vg::kLog2e);
  const float qs = q.y == 0.f ? 0.f : q.y * ex2((qr - r) * vg::kLog2e);
  return make_float2(m, ps + qs);
}

// Loss, lse, and with dloss the factors of dX = dloss.factor.(g.W) + target_factor.W[y]. kWarps: a row's
// warps: one, or all eight of a CTA where there are few rows (its pieces then come in one go).
template <int kWarps>
__global__ void __launch_bounds__(256) vocab_rows_kernel(const VocabRowArgs a) {
  __shared__ float2 sh[8];
  pdl_launch_dependents();
  pdl_wait();
  const int row = blockIdx.x * (8 / kWarps) + (threadIdx.x >> 5) / kWarps, lane = threadIdx.x & 31;
  if (row >= a.t) return;   // (whole warps; with eight to a row no CTA is without one)
  float2 st = make_float2(-INFINITY, 0.f);
#pragma unroll 4
  for (int i = threadIdx.x % (32 * kWarps); i < a.pieces; i += 32 * kWarps)
    st = join_stats(st, a.stats[static_cast<int64_t>(row) * a.pieces + i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    float2 q;
    q.x = __shfl_xor_sync(0xFFFFFFFFu, st.x, o);
    q.y = __shfl_xor_sync(0xFFFFFFFFu, st.y, o);
    st = join_stats(st, q);
  }
  if (kWarps > 1) {
    if (lane == 0) sh[threadIdx.x >> 5] = st;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 1; w < kWarps; ++w) st = join_stats(st, sh[w]);
  }
  if (threadIdx.x % (32 * kWarps) != 0) return;
  const float lse = (fabsf(st.x) == INFINITY ? 0.f : st.x) + logf(st.y);
  const int64_t y = a.targets[row];
  const bool inside = y >= 0 && y < a.v, counted = inside && y != a.ignore;
  if (!inside && y != a.ignore) report(kDevTarget);
  const float loss = counted ? lse - a.target_logit[row] : 0.f;
  a.loss[row] = loss;
  a.lse[row] = lse;
  if (a.dloss) {
    const float d = counted ? a.dloss[row] : 0.f, ref = counted ? a.ref[row] : 0.f;
    // not zero for a counted row: its loss is at most 60 + log v where factors are used
    a.factor[row] = d != 0.f ? expf(ref - lse) : 0.f;
    a.target_factor[row] = counted ? d * expm1f(-loss) : 0.f;  // dloss . (p[y] - 1)
  }
}

// The counted rows' target logits, and the redo flag's clearing. kWarps: as above.
template <int kWarps>
__global__ void __launch_bounds__(256)
    vocab_target_kernel(const uint16_t* X, const uint16_t* W, const int64_t* targets, int64_t ignore, int t, int h,
                        int v, float* ref, unsigned* redo) {
  __shared__ float sh[8];
  pdl_launch_dependents();
  const int row = blockIdx.x * (8 / kWarps) + (threadIdx.x >> 5) / kWarps, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *redo = 0u;
  if (row >= t) return;
  const int64_t y = targets[row];
  if (y < 0 || y >= v || y == ignore) return;   // (the row's threads alike)
  const uint16_t *x = X + static_cast<int64_t>(row) * h, *w = W + y * h;
  float s = 0.f;
#pragma unroll 4
  for (int i = threadIdx.x % (32 * kWarps); i < (h >> 3); i += 32 * kWarps) {
    float a[8], b[8];
    unpack8(ldg_vec(x, i), a);
    unpack8(ldg_vec(w, i), b);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if (kWarps > 1) {
    if (lane == 0) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int w = 1; w < kWarps; ++w) s += sh[w];
  }
  if (threadIdx.x % (32 * kWarps) == 0) ref[row] = s;
}

// dX tiles whose K was split: the partial tiles are added in order and rounded once.
__global__ void __launch_bounds__(256)
    vocab_join_kernel(const float* part, uint16_t* dX, const VocabGemmArgs a) {
  pdl_wait();
  const int tile = blockIdx.x, r = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  VocabGemmArgs b = a;
  b.splits = 1;
  const VocabItem it = vocab_item(b, a.whole + tile);
  const int row = it.m0 + r, col = it.n0 + lane * 8;
  if (row >= a.M || col >= a.N) return;   // N % 8 == 0
  const RowFactor rf = row_factor(a, row);
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int p = 0; p < a.splits; ++p) {
    const float4* q = reinterpret_cast<const float4*>(
        part + ((static_cast<int64_t>(tile) * a.splits + p) * vg::BM + r) * vg::BN + lane * 8);
    const float4 u = __ldcg(q), w = __ldcg(q + 1);
    s[0] += u.x; s[1] += u.y; s[2] += u.z; s[3] += u.w;
    s[4] += w.x; s[5] += w.y; s[6] += w.z; s[7] += w.w;
  }
  rf.apply(s, col);
  *reinterpret_cast<uint4*>(dX + static_cast<int64_t>(row) * a.N + col) = pack8(s);
}

// The same for few tokens: grid x a 128-column tile of h, grid y two tokens.
__global__ void __launch_bounds__(256)
    vocab_narrow_join_kernel(const float* part, uint16_t* dX, const VocabNarrowArgs a, const VocabGemmArgs f, int ctas) {
  pdl_wait();
  const int tile = blockIdx.x, col = threadIdx.x & 127, tok = blockIdx.y * 2 + (threadIdx.x >> 7);
  if (tok >= a.t || tile * vn::BM + col >= a.h) return;
  const int total = a.tiles * a.num_kb, base = total / ctas, extra = total - base * ctas;
  auto cta_of = [&](int x) {   // the CTA whose run has K-step x (the inverse of unit_row)
    const int long_runs = extra * (base + 1);
    return x < long_runs ? x / (base + 1) : extra + (x - long_runs) / base;
  };
  const int first = cta_of(tile * a.num_kb), last = cta_of((tile + 1) * a.num_kb - 1);
  float s = 0.f;
#pragma unroll 4
  for (int i = first; i <= last; ++i)
    s += __ldcg(part + (static_cast<int64_t>(i + tile) * a.n16 + tok) * vn::BM + col);
  const RowFactor rf = row_factor(f, tok);
  const int hc = tile * vn::BM + col;
  s = rf.times(s, rf.w ? bf16_bits_to_float(rf.w[hc]) : 0.f);
  dX[static_cast<int64_t>(tok) * a.h + hc] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

}  // namespace qlora
