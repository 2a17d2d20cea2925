// tcgen05 (5th-generation tensor core) fused NF4 GEMM for the training-shape QLoRA linear on
// sm_100a.
//
// nf4_gemm_kernel<BWD>: the frozen-base product with the NF4 dequantization fused into the
//    producer stage and the LoRA product folded into the same TMEM accumulator:
//       forward  (BWD = false):  Y  = X  . W'   + sT . L2      (M = t, N = o, K = h)
//       backward (BWD = true):   dX = dY . W'^T + sU . L1^T    (M = t, N = h, K = o)
//    ("The algebra", mchromiak.github.io; "QLoRA in LLMs" sections 3-4; "The core move",
//    goodomens.studio: each 4-bit block is dequantized on the fly, used, discarded.)
//    A (X or dY) and the packed codes (a ring of their own, steps ahead) arrive by TMA; 8
//    producer warps, four on every other K-step, turn each 64-weight block into bf16 (w' = bf16(level * (q8 * s2)), the exact nf4_dequantize values, selected
//    by byte permutes from a 16-entry product table built in registers per block) and
//    write it straight into the 128-byte-swizzled operand layout the MMA reads: K-major for
//    the forward (rows of Wt are N), MN-major for the backward (rows of Wt are K). A pair of
//    CTAs (a cluster of 2) owns 512 tokens x 256 columns and issues tcgen05.mma.cta_group::2:
//    each CTA dequantizes only its 128 of the 256 columns, and two accumulators per CTA (all
//    512 TMEM columns) make every dequantized tile feed 512 tokens. The h/64 (or o/64) weight
//    K-steps run first, then the r/64 LoRA K-steps (A = sT or sU, B = L2 or L1, both by
//    TMA), so that the kernel can start, by programmatic dependent launch, while the kernel
//    that produces sT or sU is still running. The same 8 warps then drain TMEM to bf16, with
//    bias, activation and residual where they are asked for (epilogue.cuh), or leave fp32
//    shares of a split K that nf4_gemm_join_kernel finishes.
//    Bound: the tensor cores. Copies and dequantized tiles of both CTAs are counted on the even
//    CTA's barriers, so its issuing warp waits for no relay. Measured, 4096 tokens, 4096 -> 11008:
//    257 us plain (1.46 PFLOP/s), 287 with bias, SiLU and Z kept.
//
// (tc_gemm.cuh holds the plain tcgen05 GEMM for the rank-r products.)
//
// Every wait is bounded (qlora::mbar_wait); on expiry the CTA reports QLORA_DEV_TIMEOUT,
// stops issuing, waits for its own copies and MMAs in flight, frees TMEM and returns.
#pragma once

#include "epilogue.cuh"
#include "nf4_codec.cuh"

namespace qlora {
namespace tc {

// A CTA pair (thread-block cluster of 2) owns 512 tokens x 256 output columns. One
// tcgen05.mma.cta_group::2 computes 256 tokens x 256 columns: each CTA supplies 128 rows of A
// and 128 of the 256 columns of B from its own shared memory and holds its 128 x 256 fp32
// slice of the accumulator in its own tensor memory. Two such accumulators per CTA (all 512
// TMEM columns) cover the 512 tokens, so each dequantized half-tile feeds 512 tokens.
constexpr int PAIR_M = 512;
constexpr int BN = 256;        // output columns per pair
constexpr int BNH = BN / 2;    // columns of B held (and dequantized) by each CTA
constexpr int BK = 64;         // K per stage: one 128-byte swizzle row of bf16, one NF4 block
constexpr int STAGES = 4;
constexpr int A_HALF = 128 * BK * 2;       // 16 KB: this CTA's 128 rows of one accumulator
constexpr int A_BYTES = 2 * A_HALF;        // 32 KB
constexpr int B_BYTES = BNH * BK * 2;      // 16 KB
constexpr int P_BYTES = BNH * BK / 2;      // 4 KB of packed codes
constexpr int P_STAGES = 8;                // their own ring, filled by a warp of its own: codes are read into
                                           // registers and their slot is free long before the step's MMAs
constexpr int kWorkWarps = 8;              // warps 0-7: dequant producers, then epilogue
constexpr int kGroupWarps = 4;             // producers of one stage; the groups take K-steps in turn: warps
                                           // 0-3, 4-7, and with kThreadsFew 11-14 (which only produce)
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;                // even CTA: MMA issuer
constexpr int kCodeWarp = 10;              // TMA of the packed codes
constexpr int kThreads = 11 * 32;
constexpr int kThreadsFew = 15 * 32;       // for 256 tokens or fewer: a step of half the products leaves two groups
                                           // behind (16 tokens, 8192 x 8192: 38.7 -> 34.4 us; at 4096 tokens a
                                           // third one costs 0.7%)
inline int nf4_gemm_threads(int64_t tokens) { return tokens <= PAIR_M / 2 ? kThreadsFew : kThreads; }

constexpr int kTmemCols = 512;
constexpr int kEpiZTile = kWorkWarps * 8192;   // the staging tiles of Z lie behind those of Y
static_assert(2 * kEpiZTile <= STAGES * (A_BYTES + B_BYTES), "staging tiles in the drained stage buffers");

constexpr size_t nf4_gemm_smem_bytes() {
  return 1024 /* alignment slack */ + STAGES * (A_BYTES + B_BYTES) + P_STAGES * P_BYTES + 384;
}

}  // namespace tc

struct Nf4GemmArgs {
  const uint8_t* q8;
  const float* s2;
  int64_t h;        // in_features: row length of Wt
  int M;            // tokens
  int N;            // output columns: o (forward) or h (backward)
  int num_kb;       // weight K-steps: h/64 (forward) or o/64 (backward)
  int num_lkb;      // LoRA K-steps: ceil(r/64)
  uint16_t* out;    // M x N bf16, row stride N
  Nf4Table tab;
  const uint16_t* addend;  // NULL, or M x N bf16 added to the accumulator before the rounding;
                           // written by the previous kernel on the stream (waited for first)
  EpilogueArgs epi;        // kEpiFused only
  int kb_per_split;        // kEpiPartial: weight K-steps of each of gridDim.z shares of K
};

// What the epilogue does with the accumulator.
enum GemmEpi : int {
  kEpiNone = 0,     // bf16 (plus the addend)
  kEpiFused = 1,    // Z = accumulator + bias, Y = act(Z) + residual; Z stored through tmZ where it is kept
  kEpiPartial = 2,  // fp32 share of a split K (grid z), through tmZ: M x N x shares
};

// Wait for an mbarrier phase ignoring the abort flag (used only to drain in-flight copies
// after an abort), still bounded by the timeout.
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      report(kDevTimeout);
      return;
    }
  }
}

template <bool kBwd, int kEpi = kEpiNone>
__global__ void __launch_bounds__(tc::kThreadsFew, 1)
    nf4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmP,
                    const __grid_constant__ CUtensorMap tmA2,
                    const __grid_constant__ CUtensorMap tmB2,
                    const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmZ,
                    const __grid_constant__ CUtensorMap tmR, const Nf4GemmArgs args) {
  using namespace tc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * A_BYTES;
  uint8_t* sP = sB + STAGES * B_BYTES;
  uint64_t* full_a = reinterpret_cast<uint64_t*>(sP + P_STAGES * P_BYTES);  // even CTA: both CTAs' A (and LoRA B)
  uint64_t* full_p = full_a + STAGES;       // this CTA's packed codes
  uint64_t* empty_p = full_p + P_STAGES;
  uint64_t* full_b = empty_p + P_STAGES;    // even CTA: both CTAs' dequantized B
  uint64_t* empty = full_b + STAGES;
  uint64_t* acc_full = empty + STAGES;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile uint32_t* abort_flag = tmem_holder + 1;

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();             // 0: MMA issuer, 1: its peer
  // Grid x walks the column tiles (two CTAs each) and grid y the 512-token row blocks, so the
  // pairs resident at one time share a few row blocks of A (the larger operand) across all
  // column tiles rather than streaming all of A once per wave.
  const int n0 = (blockIdx.x >> 1) * BN;                 // the pair's 256 output columns
  const int nh0 = n0 + static_cast<int>(rank) * BNH;    // this CTA's 128 of them
  const int mrow = blockIdx.y * PAIR_M + static_cast<int>(rank) * 128;  // + a * 256
  // weight K-steps (those of this share of K), then the LoRA K-steps (with the last share)
  const int kb0 = kEpi == kEpiPartial ? static_cast<int>(blockIdx.z) * args.kb_per_split : 0;
  const int nk = kEpi == kEpiPartial ? min(args.num_kb - kb0, args.kb_per_split) : args.num_kb;
  const int total = nk + (kEpi != kEpiPartial || blockIdx.z + 1 == gridDim.z ? args.num_lkb : 0);
  // 256 rows or fewer fill one of the two accumulators
  const int nacc = args.M - static_cast<int>(blockIdx.y) * PAIR_M > 256 ? 2 : 1;
  const uint32_t a_bytes = static_cast<uint32_t>(nacc) * A_HALF;
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full_a[s], 1);
      mbar_init(&full_b[s], 2 * kGroupWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < P_STAGES; ++s) {
      mbar_init(&full_p[s], 1);
      mbar_init(&empty_p[s], kGroupWarps);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc2(tmem_holder, kTmemCols);
    tmem_relinquish2();
  }
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmA2);
    tma_prefetch_desc(&tmB2);
    tma_prefetch_desc(&tmOut);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before any cross-CTA arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == kTmaWarp) {
    // What the MMA reads is counted on barriers of the even CTA, whose warp issues it, for both CTAs: the
    // odd CTA's copies and dequantized tiles arrive there directly. (Warp-uniform code with an elected
    // issuer, as below: from a branch of one lane a step's copies took 640 cycles to issue, of the 820 of a
    // whole step at 256 rows or fewer.)
    const uint32_t full_a0 = cluster_smem_addr(full_a, 0);
    int issued = 0;   // K-steps whose copies were issued
    for (int i = 0; i < total; ++i) {
      const int slot = i % STAGES;
      const uint32_t ph = (i / STAGES) & 1;
      if (!mbar_wait_warp(&empty[slot], ph ^ 1u, abort_flag)) break;
      uint8_t* a_dst = sA + slot * A_BYTES;
      uint8_t* b_dst = sB + slot * B_BYTES;
      const uint32_t bar = full_a0 + static_cast<uint32_t>(slot * sizeof(uint64_t));
      // sT / sU come from the kernel launched just before this one, which may still be running
      // (programmatic dependent launch): wait for it before the first LoRA load
      if (i == nk) pdl_wait();
      if (elect_one()) {
        if (kEpi == kEpiFused && args.epi.residual && i == (total > 16 ? total - 16 : 0)) {
          for (int a = 0; a < nacc; ++a)       // this CTA's 128 rows of each accumulator, 256 columns
            for (int c = 0; c < BN && n0 + c < args.N; c += 64) tma_prefetch_2d(&tmR, n0 + c, mrow + a * 256);
        }
        if (i >= nk) {
          const int li = i - nk;
          if (rank == 0) mbar_arrive_expect_tx(&full_a[slot], 2 * (a_bytes + B_BYTES));
          tma_load_2d_pair(a_dst, &tmA2, bar, li * BK, mrow);
          if (nacc == 2) tma_load_2d_pair(a_dst + A_HALF, &tmA2, bar, li * BK, mrow + 256);
          if (!kBwd) {
            // L2 (r x o), MN-major B: this CTA's two 64-column atoms, 8 KB apart
            tma_load_2d_pair(b_dst, &tmB2, bar, nh0, li * BK);
            tma_load_2d_pair(b_dst + 8192, &tmB2, bar, nh0 + 64, li * BK);
          } else {
            // L1 (h x r), K-major B: this CTA's 128 rows of 64 ranks
            tma_load_2d_pair(b_dst, &tmB2, bar, li * BK, nh0);
          }
        } else {
          if (rank == 0) mbar_arrive_expect_tx(&full_a[slot], 2 * a_bytes);
          tma_load_2d_pair(a_dst, &tmA, bar, (kb0 + i) * BK, mrow);
          if (nacc == 2) tma_load_2d_pair(a_dst + A_HALF, &tmA, bar, (kb0 + i) * BK, mrow + 256);
        }
      }
      __syncwarp();
      issued = i + 1;
    }
    if (lane == 0 && *abort_flag) {
      // make sure no copy is still writing this CTA's shared memory before it exits: the odd
      // CTA's A copies count on its peer's barriers, so it gives them, at most STAGES of them, a
      // thousand times a copy's latency (and stays until the cluster's barrier below)
      if (rank == 0)
        for (int j = (issued > STAGES ? issued - STAGES : 0); j < issued; ++j)
          mbar_drain(&full_a[j % STAGES], (j / STAGES) & 1);
      else
        for (int j = 0; j < 2000; ++j) __nanosleep(1000);
    }
  } else if (warp == kCodeWarp) {
    int issued = 0;
    for (int kb = 0; kb < nk; ++kb) {
      const int slot = kb % P_STAGES;
      if (!mbar_wait_warp(&empty_p[slot], ((kb / P_STAGES) & 1) ^ 1u, abort_flag)) break;
      if (elect_one()) {
        uint8_t* dst = sP + slot * P_BYTES;
        mbar_arrive_expect_tx(&full_p[slot], P_BYTES);
        if (!kBwd) {
          tma_load_2d(dst, &tmP, &full_p[slot], (kb0 + kb) * (BK / 2), nh0);
        } else {
          tma_load_2d(dst, &tmP, &full_p[slot], nh0 / 2, (kb0 + kb) * BK);
          tma_load_2d(dst + 2048, &tmP, &full_p[slot], nh0 / 2 + 32, (kb0 + kb) * BK);
        }
      }
      __syncwarp();
      issued = kb + 1;
    }
    if (lane == 0 && *abort_flag)
      for (int j = (issued > P_STAGES ? issued - P_STAGES : 0); j < issued; ++j)
        mbar_drain(&full_p[j % P_STAGES], (j / P_STAGES) & 1);
  } else if (warp == kMmaWarp) {
    if (rank == 0) {
      // M = 256 per instruction (128 rows from each CTA), N = 256 (128 columns from each)
      constexpr uint32_t kIdescMain = idesc_bf16(256, BN, false, kBwd);
      constexpr uint32_t kIdescLora = idesc_bf16(256, BN, false, !kBwd);
      bool any = false;
      const uint32_t a_lo0 = sw128_desc_lo(smem_addr(sA), 16);
      const uint32_t b_lo_k = sw128_desc_lo(smem_addr(sB), 16), b_lo_mn = sw128_desc_lo(smem_addr(sB), 8192);
      for (int i = 0; i < total; ++i) {
        const int slot = i % STAGES;
        const uint32_t ph = (i / STAGES) & 1;
        if (!mbar_wait_warp(&full_a[slot], ph, abort_flag)) break;
        if (!mbar_wait_warp(&full_b[slot], ph, abort_flag)) break;
        tc_fence_after();
        // A is K-major; B (the weights forward, L1 backward) K-major or (L2 forward, the weights
        // backward) MN-major
        const uint32_t a_lo = a_lo0 + slot * (A_BYTES >> 4), b_off = slot * (B_BYTES >> 4);
        auto issue = [&](uint32_t b_lo, uint32_t b_step, uint32_t idesc) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t bd = sw128_desc_of(b_lo + kk * b_step);
            umma2_bf16(tmem_base, sw128_desc_of(a_lo + kk * 2), bd, idesc, (i > 0 || kk > 0) ? 1u : 0u);
            if (nacc == 2)
              umma2_bf16(tmem_base + BN, sw128_desc_of(a_lo + (A_HALF >> 4) + kk * 2), bd, idesc,
                         (i > 0 || kk > 0) ? 1u : 0u);
          }
        };
        if (elect_one()) {
          if ((i >= nk) == kBwd)
            issue(b_lo_k + b_off, 2, i >= nk ? kIdescLora : kIdescMain);
          else
            issue(b_lo_mn + b_off, 128, i >= nk ? kIdescLora : kIdescMain);
          umma2_commit_multicast(&empty[slot], 0x3);   // frees the stage in both CTAs
        }
        __syncwarp();
        any = true;
      }
      // completes in both CTAs once every MMA above has finished (also after an abort)
      // (elect picks the lane that issued them)
      if (elect_one()) {
        umma2_commit_multicast(acc_full, 0x3);
        if (*abort_flag && any) mbar_drain(acc_full, 0);
      }
      __syncwarp();
    }
  } else {
    // ---------------- warps 0-7: dequant producers (a 64-weight block per thread per stage: 128
    // blocks of this CTA's 128 columns), then the epilogue -----------------------------------
    // Groups of four warps take K-steps in turn: a step's chain of waits, table, selects and
    // stores is longer than its MMAs, so that one group alone, or all eight warps on every step,
    // would set the pace (and a thread builds a block's table once, not two threads each).
    uint64_t lv2[8];                 // the 16 fp32 levels as pairs (2i low, 2i+1 high)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm("mov.b64 %0, {%1, %2};" : "=l"(lv2[i]) : "f"(args.tab.level[2 * i]), "f"(args.tab.level[2 * i + 1]));
    const int groups = blockDim.x == kThreadsFew ? 3 : 2;
    const int group = warp < kWorkWarps ? warp / kGroupWarps : 2;
    const int blk = (threadIdx.x + (warp < kWorkWarps ? 0 : 32)) & (kGroupWarps * 32 - 1);   // 0..127
    const int64_t nblk_row = args.h / kBlock;
    int64_t qbase, qstep;       // q8 index of this thread's block at weight K-step kb: qbase + kb*qstep
    int out_off, pk_off, swz;
    bool valid;
    if (!kBwd) {
      // block row blk of this CTA's columns is Wt row nh0 + blk; its block kb is K-step kb
      const int64_t j = nh0 + blk;
      valid = j < args.N;
      qbase = j * nblk_row;
      qstep = 1;
      pk_off = blk * 32;
      out_off = (blk >> 3) * 1024 + (blk & 7) * 128;
      swz = blk & 7;
    } else {
      // K row jl of the stage is Wt row kb*64 + jl; local column atom a is blocks nh0/64 + a
      const int jl = blk & 63, a = blk >> 6;
      valid = (nh0 + a * 64) < args.N;
      qbase = static_cast<int64_t>(jl) * nblk_row + (nh0 / 64) + a;
      qstep = 64 * nblk_row;
      pk_off = a * 2048 + jl * 32;
      out_off = a * 8192 + (jl >> 3) * 1024 + (jl & 7) * 128;
      swz = jl & 7;
    }
    // 8-bit scale and second-level scale of this thread's block, fetched kPf of its steps ahead into
    // a ring of registers; the loop below is unrolled by kPf so that every ring index is a
    // compile-time constant and a load is waited for only when its step comes up
    constexpr int kPf = 4;
    uint32_t qr[kPf];
    float sr[kPf];
#pragma unroll
    for (int j = 0; j < kPf; ++j) {
      const int i = groups * j + group;
      qr[j] = 0u;
      sr[j] = 0.f;
      if (valid && i < nk) {
        const int64_t qi = qbase + static_cast<int64_t>(kb0 + i) * qstep;
        qr[j] = __ldg(args.q8 + qi);
        sr[j] = __ldg(args.s2 + (qi >> 8));
      }
    }
    bool ok = true;
    for (int i0 = group; i0 < total && ok; i0 += groups * kPf) {
#pragma unroll
      for (int j = 0; j < kPf; ++j) {
        const int i = i0 + groups * j;
        if (i >= total || !ok) break;
        const int slot = i % STAGES;
        const uint32_t ph = (i / STAGES) & 1;
        if (i < nk) {
          // codes and table first: they do not depend on the operand slot's MMAs
          const float k = __fmul_rn(static_cast<float>(qr[j]), sr[j]);
          if (valid && i + groups * kPf < nk) {
            const int64_t qi = qbase + static_cast<int64_t>(kb0 + i + groups * kPf) * qstep;
            qr[j] = __ldg(args.q8 + qi);
            sr[j] = __ldg(args.s2 + (qi >> 8));
          }
          const int pslot = i % P_STAGES;
          if (!mbar_wait_warp(&full_p[pslot], (i / P_STAGES) & 1, abort_flag)) { ok = false; break; }
          const uint4* cp = reinterpret_cast<const uint4*>(sP + pslot * P_BYTES + pk_off);
          const uint4 c0 = cp[0], c1 = cp[1];
          const ProdTab tab = build_prod_tab(lv2, k);
          // The slot is refilled by the async proxy, which an arrival alone does not hold back behind
          // loads that are still queued: without the fence a refill overtook them now and then.
          fence_proxy_async_smem();
          __syncwarp();   // every lane has its codes
          if (lane == 0) mbar_arrive(&empty_p[pslot]);
          if (!mbar_wait_warp(&empty[slot], ph ^ 1u, abort_flag)) { ok = false; break; }
          if (valid) {
            const uint32_t words[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
            uint8_t* dst = sB + slot * B_BYTES + out_off;
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)   // 16-byte chunk (8 weights) within the 128-byte row
              *reinterpret_cast<uint4*>(dst + ((ch ^ swz) << 4)) = dequant8_tab(words[ch], tab);
          }
          fence_proxy_async_smem();
        } else if (!mbar_wait_warp(&empty[slot], ph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        __syncwarp();   // (each lane has fenced its own writes)
        if (lane == 0) mbar_arrive_pair(&full_b[slot], 0);
      }
    }

    // ---------------- epilogue: TMEM -> registers -> bf16 -> shared -> TMA store -------------
    // Warp w drains 32 accumulator rows (TMEM lanes 32 (w mod 4) .., accumulator w / 4) in
    // rounds of 64 columns: four 16-column TMEM loads before one wait, the bf16 row (128 bytes
    // per lane) into a 32 x 64 staging tile, 128-byte swizzled as the output tensor map
    // expects (so the eight lanes of each quarter-warp write eight distinct bank groups), then
    // one TMA store of the tile: whole 128-byte lines instead of 32 scattered row pieces per
    // store instruction. Two staging tiles per warp (8 KB, in the drained stage buffers) let a
    // round's shared-memory writes overlap the previous round's store.
    // The fused epilogue walks 16 columns at a time in a loop that is not unrolled: its code runs a few
    // times per CTA, and 64 columns of straight-line code per activation took longer to fetch than to
    // execute. Bias and residual run one step ahead, the first ones ahead of the last products.
    const bool epi_warp = warp < kWorkWarps;
    const int epi_row0 = mrow + (warp >> 2) * 256 + (warp & 3) * 32, epi_row = epi_row0 + lane;
    uint4 rq[2], bq[2];
    auto epi_load = [&](int col) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (args.epi.bias) bq[k] = ldg_vec(args.epi.bias, (col >> 3) + k);
        if (args.epi.residual && epi_row < args.M)
          rq[k] = ldg_vec(args.epi.residual, ((static_cast<int64_t>(epi_row) * args.N + col) >> 3) + k);
      }
    };
    if (kEpi == kEpiFused && epi_warp && epi_row0 < args.M) epi_load(n0);
    const bool done = epi_warp && mbar_wait_warp(acc_full, 0, abort_flag);
    tc_fence_after();
    if (__all_sync(0xFFFFFFFFu, done && !*abort_flag)) {
      if (args.addend) pdl_wait();
      const int acc = warp >> 2, quad = warp & 3;
      const int row0 = mrow + acc * 256 + quad * 32;
      const int row = row0 + lane;
      const uint32_t lane_addr =
          tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * BN);
      uint8_t* stage_tile = smem + warp * 8192;
      const bool any_row = row0 < args.M && acc < nacc;   // warp-uniform: rows past M are not stored
      // N is a multiple of 64, so a round is either wholly inside the output or wholly past it
      if (kEpi == kEpiPartial) {
        // fp32 tiles of 32 x 32 (128-byte rows, swizzled alike), alternating the two staging tiles
        for (int c0 = 0; c0 < BN && any_row && n0 + c0 < args.N; c0 += 32) {
          uint8_t* buf = stage_tile + ((c0 >> 5) & 1) * 4096;
          if (c0 >= 64) {
            if (lane == 0) bulk_wait_group_read<1>();
            __syncwarp();
          }
          uint32_t v0[16], v1[16];
          tmem_ld_16(lane_addr + c0, v0);
          tmem_ld_16(lane_addr + c0 + 16, v1);
          tmem_ld_wait();
          uint8_t* rowp = buf + lane * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            *reinterpret_cast<uint4*>(rowp + ((k ^ (lane & 7)) << 4)) =
                make_uint4(v0[4 * k], v0[4 * k + 1], v0[4 * k + 2], v0[4 * k + 3]);
            *reinterpret_cast<uint4*>(rowp + (((k + 4) ^ (lane & 7)) << 4)) =
                make_uint4(v1[4 * k], v1[4 * k + 1], v1[4 * k + 2], v1[4 * k + 3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tmZ, buf, n0 + c0, row0, static_cast<int>(blockIdx.z));
            bulk_commit_group();
          }
        }
      }
      if (kEpi == kEpiFused && any_row) {
        const int cols = min(BN, args.N - n0);   // a multiple of 64
        uint32_t v[16];
        tmem_ld_16(lane_addr, v);
#pragma unroll 1
        for (int c = 0; c < cols; c += 16) {
          uint8_t* buf = stage_tile + ((c >> 6) & 1) * 4096;
          if (c >= 128 && (c & 63) == 0) {   // the stores issued from this tile two rounds ago have read it
            if (lane == 0) bulk_wait_group_read<1>();
            __syncwarp();
          }
          tmem_ld_wait();
          float z[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) z[k] = __uint_as_float(v[k]);
          const uint4 r0 = rq[0], r1 = rq[1], b0 = bq[0], b1 = bq[1];
          if (c + 16 < cols) {
            tmem_ld_16(lane_addr + c + 16, v);
            epi_load(n0 + c + 16);
          }
          uint8_t* at0 = buf + lane * 128 + ((((c >> 3) & 7) ^ (lane & 7)) << 4);   // swizzled 16-byte chunks
          uint8_t* at1 = buf + lane * 128 + (((((c >> 3) & 7) + 1) ^ (lane & 7)) << 4);
          float f[16];
          if (args.epi.bias) {
            unpack8(b0, *reinterpret_cast<float(*)[8]>(&f[0]));
            unpack8(b1, *reinterpret_cast<float(*)[8]>(&f[8]));
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] += f[k];
          }
          if (args.epi.z_out) {
            *reinterpret_cast<uint4*>(at0 + kEpiZTile) = pack8(*reinterpret_cast<const float(*)[8]>(&z[0]));
            *reinterpret_cast<uint4*>(at1 + kEpiZTile) = pack8(*reinterpret_cast<const float(*)[8]>(&z[8]));
          }
          act_apply(z, args.epi.act);
          if (args.epi.residual) {   // (rows behind M: not stored)
            unpack8(r0, *reinterpret_cast<float(*)[8]>(&f[0]));
            unpack8(r1, *reinterpret_cast<float(*)[8]>(&f[8]));
#pragma unroll
            for (int k = 0; k < 16; ++k) z[k] += f[k];
          }
          *reinterpret_cast<uint4*>(at0) = pack8(*reinterpret_cast<const float(*)[8]>(&z[0]));
          *reinterpret_cast<uint4*>(at1) = pack8(*reinterpret_cast<const float(*)[8]>(&z[8]));
          if ((c & 63) == 48) {   // a 64-column tile is complete
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tmOut, buf, n0 + c - 48, row0);
              if (args.epi.z_out) tma_store_2d(&tmZ, buf + kEpiZTile, n0 + c - 48, row0);
              bulk_commit_group();
            }
          }
        }
      }
      for (int c0 = 0; kEpi == kEpiNone && c0 < BN / 16; c0 += 4) {
        if (n0 + c0 * 16 >= args.N || !any_row) break;
        uint8_t* buf = stage_tile + ((c0 >> 2) & 1) * 4096;
        if (c0 >= 8) {   // the store issued from this tile two rounds ago has read it
          if (lane == 0) bulk_wait_group_read<1>();
          __syncwarp();
        }
        uint32_t vv[4][16];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_16(lane_addr + (c0 + q) * 16, vv[q]);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t (&v)[16] = vv[q];
          if (args.addend && row < args.M) {
            const int64_t off = static_cast<int64_t>(row) * args.N + n0 + (c0 + q) * 16;
            const uint4* ad = reinterpret_cast<const uint4*>(args.addend + off);
            const uint4 a0 = ad[0], a1 = ad[1];
            const uint32_t w[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {  // word k: column 2k in the low half, 2k + 1 high
              v[2 * k] = __float_as_uint(__uint_as_float(v[2 * k]) + __uint_as_float(w[k] << 16));
              v[2 * k + 1] = __float_as_uint(__uint_as_float(v[2 * k + 1]) +
                                             __uint_as_float(w[k] & 0xFFFF0000u));
            }
          }
          uint8_t* rowp = buf + lane * 128;
          uint4 o0, o1;
          o0.x = pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1]));
          o0.y = pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3]));
          o0.z = pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5]));
          o0.w = pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7]));
          o1.x = pack_bf16x2(__uint_as_float(v[8]), __uint_as_float(v[9]));
          o1.y = pack_bf16x2(__uint_as_float(v[10]), __uint_as_float(v[11]));
          o1.z = pack_bf16x2(__uint_as_float(v[12]), __uint_as_float(v[13]));
          o1.w = pack_bf16x2(__uint_as_float(v[14]), __uint_as_float(v[15]));
          *reinterpret_cast<uint4*>(rowp + (((2 * q) ^ (lane & 7)) << 4)) = o0;
          *reinterpret_cast<uint4*>(rowp + (((2 * q + 1) ^ (lane & 7)) << 4)) = o1;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmOut, buf, n0 + c0 * 16, row0);
          bulk_commit_group();
        }
      }
      if (lane == 0) bulk_wait_group<0>();   // the output is written before the CTA retires
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // no CTA leaves while its peer may still signal it or read its TMEM slice
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc2(tmem_base, kTmemCols);
  }
  // completion stays in stream order even when an abort skipped the wait before the LoRA steps
  if (threadIdx.x == 0) pdl_wait();
}

// The fused epilogue over a split K's shares (shares x M x N fp32, added in order): eight columns of a
// row per thread.
__global__ void __launch_bounds__(256)
    nf4_gemm_join_kernel(const float* part, int shares, uint16_t* Y, int64_t rows, int N, const EpilogueArgs epi) {
  pdl_wait();
  const int64_t vec = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, nvec = N >> 3;
  if (vec >= rows * nvec) return;
  float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int p = 0; p < shares; ++p) {
    const float4* q = reinterpret_cast<const float4*>(part + p * rows * N) + 2 * vec;
    const float4 u = __ldcg(q), w = __ldcg(q + 1);
    z[0] += u.x; z[1] += u.y; z[2] += u.z; z[3] += u.w;
    z[4] += w.x; z[5] += w.y; z[6] += w.z; z[7] += w.w;
  }
  float b[8];
  if (epi.bias) {
    unpack8(ldg_vec(epi.bias, vec % nvec), b);
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] += b[k];
  }
  if (epi.z_out) reinterpret_cast<uint4*>(epi.z_out)[vec] = pack8(z);
  act_apply(z, epi.act);
  if (epi.residual) {
    unpack8(ldg_vec(epi.residual, vec), b);
#pragma unroll
    for (int k = 0; k < 8; ++k) z[k] += b[k];
  }
  reinterpret_cast<uint4*>(Y)[vec] = pack8(z);
}

}  // namespace qlora
