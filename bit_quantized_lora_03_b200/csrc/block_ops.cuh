// Host side of the operators around the linear: the fused epilogue, the norms of a block with its
// gate and residual scale, the vocabulary loss. Included by qlora_nf4.cu, whose argument checks, device table and launch
// helpers it uses.
#pragma once

namespace {

constexpr int kMaxSms = 160;   // workspace sizes are host functions: sized for any B200

// ------------------------------------------------------------------------------------------
// the linear's epilogue
// ------------------------------------------------------------------------------------------
bool valid_act(int act) { return act >= QLORA_ACT_NONE && act <= QLORA_ACT_SILU; }
static_assert(kActNone == QLORA_ACT_NONE && kActRelu == QLORA_ACT_RELU && kActGelu == QLORA_ACT_GELU &&
              kActGeluTanh == QLORA_ACT_GELU_TANH && kActSilu == QLORA_ACT_SILU, "activation ids");

// Runs of rows of the epilogue's backward: one wave of CTAs over the card, each with at least four
// rounds of its warps' rows in flight, so that a short batch is not cut into runs whose partial sums
// cost more than they save. The workspace is sized for the most runs there can be (sms = 0).
constexpr int kMaxEpiRuns = 1024;
int epilogue_runs(int64_t t, int64_t o, int sms, int ctas) {
  const int64_t rows = 4 * ep::kUnroll * ep::kWarps;
  int64_t runs = std::min<int64_t>((t + rows - 1) / rows, kMaxEpiRuns);
  const int64_t blocks = (o + ep::kCols - 1) / ep::kCols;
  if (sms) runs = std::min(runs, std::max<int64_t>(1, static_cast<int64_t>(sms) * ctas / blocks));
  return static_cast<int>(runs);
}

int launch_finish(int prof_kind, const float* part_pre, const float* part_post, const float* part_gate, float* dw_pre,
                  float* dw_post, float* dgate, int t, int h, int rows_per_gate, int parts, int units, int grid_y,
                  cudaStream_t st) {
  dim3 grid(static_cast<unsigned>((h + nr::kFinishCols - 1) / nr::kFinishCols), static_cast<unsigned>(grid_y));
  return launch_after(prof_kind, norm_residual_finish_kernel, grid, nr::kFinishWarps * 32, st, 0, part_pre, part_post,
                      part_gate, dw_pre, dw_post, dgate, t, h, rows_per_gate, parts, units);
}

// ------------------------------------------------------------------------------------------
// norms
// ------------------------------------------------------------------------------------------
int check_norm_shape(int64_t t, int64_t h) {
  if (t < 1) return QLORA_ERR_INVALID_ARG;
  if (h < 8 || h % 8 != 0 || h > nr::kMaxH || t >= kMaxDim) return QLORA_ERR_BAD_SHAPE;
  return QLORA_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct NormBwdPlan {
  int threads, ctas, units;   // CTAs, and runs of rows (warps for short rows, else CTAs)
  size_t smem;
};
// Threads of a row at two vectors of 8 each.
unsigned norm_threads(int64_t h) { return static_cast<unsigned>(((h / 8 + 1) / 2 + 31) / 32 * 32); }

NormBwdPlan plan_norm_bwd(int64_t t, int64_t h, int sms) {
  NormBwdPlan p{};
  constexpr int wpc = nr::kWarpRowThreads / 32;
  const bool warp_row = h <= nr::kWarpRowH, wide = h > nr::kStayH;
  p.threads = warp_row ? nr::kWarpRowThreads : static_cast<int>(norm_threads(h));
  // CTAs that fit an SM by threads (128 registers each); their rings and sums take
  // 512 threads x (3 rows x 4 + 2) x 32 bytes = 224 KB of its shared memory together
  const int per_sm = std::max(1, std::min(8, 512 / p.threads));
  p.ctas = static_cast<int>(std::min<int64_t>(warp_row ? (t + wpc - 1) / wpc : t, static_cast<int64_t>(sms) * per_sm));
  p.units = warp_row ? p.ctas * wpc : p.ctas;
  p.smem = static_cast<size_t>(p.threads) * 64 * (wide ? 3 : 1 + 2 * nr::kBwdStages);
  return p;
}

// ------------------------------------------------------------------------------------------
// vocabulary loss
// ------------------------------------------------------------------------------------------
// Tokens whose g (or scaled exponentials; for the loss alone, statistics) the workspace holds at a time: as
// many as fit 256 MiB, at least one row of tiles. Few long runs keep the second product's tiles busy and
// read W seldom.
constexpr size_t kVocabRunBytes = size_t(256) << 20;
constexpr int64_t kVocabMaxV = int64_t(1) << 24;
constexpr int kVocabMaxParts = kMaxSms;   // partial tiles of a split K

// Up to this many tokens go through the kernels that stream W past them (one 256-token tile of the
// others is computed whole whatever it holds). Measured on 32000 x 4096, loss and
// gradient: 102 us at 16 tokens, 121 at 64, 130 at 80, against 134 at 81, 143 at 96 and 152 at 200.
constexpr int64_t kVocabNarrowTokens = vn::kMaxTokens;
constexpr int64_t kFewRows = 1024;   // rows that get a CTA each in the kernels over rows (a warp each above)

struct VocabPlan {
  bool narrow;
  int64_t run;      // tokens per run
  int64_t ldp;      // v rounded up to 64
  int64_t pieces;   // of the vocabulary
  size_t g_bytes, stats_bytes, row_bytes, part_bytes;   // row_bytes: one float per token of a run
};
VocabPlan plan_vocab(int64_t t, int64_t h, int64_t v, bool stats, bool grad) {
  VocabPlan p{};
  p.narrow = t <= kVocabNarrowTokens;
  p.ldp = (v + 63) / 64 * 64;
  p.pieces = p.narrow ? p.ldp / vn::kUnit : (v + vg::BN - 1) / vg::BN * (vg::BN / vg::PIECE);
  const int64_t fit = static_cast<int64_t>(kVocabRunBytes) / (grad ? p.ldp * 2 : p.pieces * 8);
  p.run = std::min<int64_t>(t, std::max<int64_t>(vg::BM, fit / vg::BM * vg::BM));
  if (grad) {
    p.g_bytes = align256(static_cast<size_t>(p.run) * p.ldp * 2);
    p.part_bytes = p.narrow ? static_cast<size_t>(kMaxSms + (h + vn::BM - 1) / vn::BM) * vn::BM *
                                  vn::tokens16(static_cast<int>(t)) * 4
                            : static_cast<size_t>(kVocabMaxParts) * vg::BM * vg::BN * 4;
  }
  if (stats) p.stats_bytes = align256(static_cast<size_t>(p.run) * p.pieces * 8);
  p.row_bytes = align256(static_cast<size_t>(p.run) * 4);
  return p;
}

int check_vocab_shape(int64_t t, int64_t h, int64_t v) {
  if (t < 1 || v < 1) return QLORA_ERR_INVALID_ARG;
  if (h < 8 || h % 8 != 0 || h >= kMaxDim || t >= kMaxDim || v > kVocabMaxV) return QLORA_ERR_BAD_SHAPE;
  return QLORA_OK;
}

size_t vocab_ws_bytes(int64_t t, int64_t h, int64_t v, bool stats, bool grad) {
  if (check_vocab_shape(t, h, v) != QLORA_OK) return 0;
  const VocabPlan p = plan_vocab(t, h, v, stats, grad);
  return p.g_bytes + p.part_bytes + p.stats_bytes + 4 * p.row_bytes + 256;
}

// Tiles, their order and their split. Pairs walk the list in steps; row tiles are walked in groups
// of 16 (4096 tokens) per column tile, so that a group's A and the column tiles in flight stay in L2.
// The tiles of the last, partly filled round are split along K (fp32 partial tiles, joined in order)
// into the number of pieces that ends the round soonest.
VocabGemmArgs plan_vocab_gemm(int64_t M, int64_t N, int64_t K, bool split, int pairs) {
  VocabGemmArgs a{};
  a.M = static_cast<int>(M);
  a.N = static_cast<int>(N);
  a.num_kb = static_cast<int>((K + vg::KS * vg::BK - 1) / (vg::KS * vg::BK));
  a.m_tiles = static_cast<int>((M + vg::BM - 1) / vg::BM);
  a.n_tiles = static_cast<int>((N + vg::BN - 1) / vg::BN);
  a.m_group = std::min(a.m_tiles, 16);
  const int64_t tiles = static_cast<int64_t>(a.m_tiles) * a.n_tiles;
  const int rest = static_cast<int>(tiles % pairs);
  a.splits = 1;
  double best = 1.0;
  for (int s = 2; split && rest && rest * s <= kVocabMaxParts && s <= a.num_kb / 2; ++s) {
    const double cost = static_cast<double>((rest * s + pairs - 1) / pairs) / s + 0.01 * s;
    if (cost < best) {
      best = cost;
      a.splits = s;
    }
  }
  a.kb_per_split = (a.num_kb + a.splits - 1) / a.splits;
  a.splits = (a.num_kb + a.kb_per_split - 1) / a.kb_per_split;   // no empty piece
  a.whole = static_cast<int>(a.splits > 1 ? tiles - rest : tiles);
  a.items = static_cast<int>(a.whole + (tiles - a.whole) * a.splits);
  return a;
}

template <int kMode>
int launch_vocab_gemm(const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap& mOut,
                      const CUtensorMap& mPart, const VocabGemmArgs& a, int pairs, bool first, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(pairs, a.items)), 1, 1);
  cfg.blockDim = dim3(vg::kThreads, 1, 1);
  cfg.dynamicSmemBytes = vg::smem_bytes();
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // (the kernels wait before they read)
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = first ? 1 : 2;   // a call's first kernel starts after all earlier work
  cudaError_t e;
  {
    prof::Scope ps(prof::kVocabGemm, st);
    e = cudaLaunchKernelEx(&cfg, vocab_gemm_kernel<kMode>, mA, mB, mOut, mPart, a);
  }
  if (e != cudaSuccess) {
    cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return launch_status();
}

template <typename Kernel, typename... Maps>
int launch_narrow(Kernel kernel, const VocabNarrowArgs& a, int ctas, bool first, cudaStream_t st, const Maps&... maps) {
  if (first) {   // a call's first kernel starts after all earlier work
    prof::Scope ps(prof::kVocabGemm, st);
    kernel<<<static_cast<unsigned>(ctas), vn::kThreads, vn::smem_bytes(a.n16), st>>>(maps..., a);
    return launch_status();
  }
  return launch_after(prof::kVocabGemm, kernel, dim3(static_cast<unsigned>(ctas)), vn::kThreads, st,
                      vn::smem_bytes(a.n16), maps..., a);
}

struct VocabCall {
  const uint16_t *X, *W;
  int64_t t, h, v;
  const int64_t* targets;
  int64_t ignore;
  float *loss, *lse;        // outputs (lse an input of the backward alone)
  const float *dloss, *dlse;
  uint16_t* dX;
};

// The loss (dX == NULL), the loss and its gradient (loss and dX), or the gradient alone.
int vocab_core(const VocabCall& c, void* workspace, cudaStream_t st) {
  int dev, rc;
  if ((rc = current_device(&dev))) return rc;
  if (sm_count(dev) > kMaxSms) return QLORA_ERR_UNSUPPORTED_DEVICE;
  const int pairs = sm_count(dev) / 2;
  const bool stats = c.loss != nullptr, grad = c.dX != nullptr;
  const VocabPlan p = plan_vocab(c.t, c.h, c.v, stats, grad);
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  uint16_t* g = reinterpret_cast<uint16_t*>(ws);
  float* part = reinterpret_cast<float*>(ws + p.g_bytes);
  float2* st2 = reinterpret_cast<float2*>(ws + p.g_bytes + p.part_bytes);
  uint8_t* rows = ws + p.g_bytes + p.part_bytes + p.stats_bytes;
  float* tl = reinterpret_cast<float*>(rows);
  float* factor = reinterpret_cast<float*>(rows + p.row_bytes);
  float* target_factor = reinterpret_cast<float*>(rows + 2 * p.row_bytes);
  float* ref = reinterpret_cast<float*>(rows + 3 * p.row_bytes);
  unsigned* redo = reinterpret_cast<unsigned*>(rows + 4 * p.row_bytes);
  const auto run_targets = [&](int64_t i0, int64_t n) {
    prof::Scope ps(prof::kVocabRows, st);
    const bool few = n <= kFewRows;
    (few ? vocab_target_kernel<8> : vocab_target_kernel<1>)<<<static_cast<unsigned>(few ? n : (n + 7) / 8), 256, 0, st>>>(
        c.X + i0 * c.h, c.W, c.targets + i0, c.ignore, static_cast<int>(n), static_cast<int>(c.h),
        static_cast<int>(c.v), ref, redo);
    return launch_status();
  };
  const auto run_rows = [&](int64_t i0, int64_t n) {
    VocabRowArgs r{};
    r.stats = st2;
    r.target_logit = tl;
    r.ref = ref;
    r.targets = c.targets + i0;
    r.ignore = c.ignore;
    r.t = static_cast<int>(n);
    r.v = static_cast<int>(c.v);
    r.pieces = static_cast<int>(p.pieces);
    r.loss = c.loss + i0;
    r.lse = c.lse + i0;
    if (grad) {
      r.dloss = c.dloss + i0;
      r.factor = factor;
      r.target_factor = target_factor;
    }
    const bool few = n <= kFewRows;
    return launch_after(prof::kVocabRows, few ? vocab_rows_kernel<8> : vocab_rows_kernel<1>,
                        dim3(static_cast<unsigned>(few ? n : (n + 7) / 8)), 256, st, 0, r);
  };
  if (p.narrow) {
    VocabNarrowArgs a{};
    a.t = static_cast<int>(c.t);
    a.n16 = vn::tokens16(a.t);
    a.v = static_cast<int>(c.v);
    a.h = static_cast<int>(c.h);
    a.num_kb = static_cast<int>((c.h + vn::KS * vn::BK - 1) / (vn::KS * vn::BK));
    a.ldp = static_cast<int>(p.ldp);
    a.units = a.ldp / vn::kUnit;
    a.targets = c.targets;
    a.ignore = c.ignore;
    a.stats = st2;
    a.target_logit = tl;
    a.ref = ref;
    a.lse = c.lse;
    a.dloss = c.dloss;
    a.dlse = c.dlse;
    a.target_factor = target_factor;
    a.redo = stats ? redo : nullptr;
    a.g = g;
    a.part = part;
    CUtensorMap mW, mWu, mX;
    if (!map_bf16(&mW, c.W, c.h, c.v, 64, vn::BM) || !map_bf16(&mWu, c.W, c.h, c.v, 64, vn::kUnit) ||
        !map_bf16(&mX, c.X, c.h, c.t, 64, static_cast<uint32_t>(a.n16)))
      return QLORA_ERR_CUDA;
    const int ctas = std::min(sm_count(dev), a.units);
    if (stats) {
      if (grad && (rc = run_targets(0, c.t))) return rc;
      if ((rc = grad ? launch_narrow(vocab_narrow_kernel<kVocabScaled>, a, ctas, false, st, mW, mWu, mX)
                     : launch_narrow(vocab_narrow_kernel<kVocabStats>, a, ctas, true, st, mW, mWu, mX)))
        return rc;
      if ((rc = run_rows(0, c.t))) return rc;
    }
    if (!grad) return QLORA_OK;
    if ((rc = launch_narrow(vocab_narrow_kernel<kVocabProb>, a, ctas, !stats, st, mW, mWu, mX))) return rc;
    CUtensorMap mWmn, mG;
    if (!map_bf16(&mWmn, c.W, c.h, c.v, 64, 64) ||
        !map_bf16(&mG, g, p.ldp, c.t, 64, static_cast<uint32_t>(a.n16)))
      return QLORA_ERR_CUDA;
    VocabNarrowArgs d = a;
    d.num_kb = (a.ldp + vn::KS * vn::BK - 1) / (vn::KS * vn::BK);
    d.tiles = static_cast<int>((c.h + vn::BM - 1) / vn::BM);
    const int gctas = static_cast<int>(std::min<int64_t>(sm_count(dev), static_cast<int64_t>(d.tiles) * d.num_kb));
    if ((rc = launch_narrow(vocab_narrow_grad_kernel, d, gctas, false, st, mWmn, mG))) return rc;
    VocabGemmArgs f{};
    f.N = d.h;
    f.v = d.v;
    f.targets = c.targets;
    f.ignore = c.ignore;
    f.dloss = c.dloss;
    f.dlse = c.dlse;
    f.W = c.W;
    f.target_factor = target_factor;
    if (stats) {
      f.redo = redo;
      f.factor = factor;
    }
    return launch_after(prof::kVocabRows, vocab_narrow_join_kernel,
                        dim3(static_cast<unsigned>(d.tiles), static_cast<unsigned>((c.t + 1) / 2)), 256, st, 0, part, c.dX,
                        d, f, gctas);
  }
  CUtensorMap mWk, mWmn, mPart;
  if (!map_bf16(&mWk, c.W, c.h, c.v, 64, 128) || !map_bf16(&mWmn, c.W, c.h, c.v, 64, 64)) return QLORA_ERR_CUDA;
  if (grad && !make_map_2d(&mPart, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, part, vg::BN, kVocabMaxParts * vg::BM,
                           vg::BN * 4, 32, 32, true))
    return QLORA_ERR_CUDA;
  for (int64_t i0 = 0; i0 < c.t; i0 += p.run) {
    const int64_t n = std::min(p.run, c.t - i0);
    CUtensorMap mX, mG, mGs, mD;
    if (!map_bf16(&mX, c.X + i0 * c.h, c.h, n, 64, 128)) return QLORA_ERR_CUDA;
    if (grad && (!map_bf16(&mG, g, p.ldp, n, 64, 128) || !map_bf16(&mGs, g, p.ldp, n, 64, 32) ||
                 !map_bf16(&mD, c.dX + i0 * c.h, c.h, n, 64, 32)))
      return QLORA_ERR_CUDA;
    VocabGemmArgs a = plan_vocab_gemm(n, c.v, c.h, false, pairs);
    a.ldp = static_cast<int>(p.ldp);
    a.targets = c.targets + i0;
    a.ignore = c.ignore;
    a.stats = st2;
    a.target_logit = tl;
    a.ref = ref;
    a.lse = c.lse + i0;
    if (grad) {
      a.dloss = c.dloss + i0;
      a.dlse = c.dlse ? c.dlse + i0 : nullptr;
      a.target_factor = target_factor;
    }
    if (stats) {
      if (grad) {
        a.redo = redo;
        if ((rc = run_targets(i0, n))) return rc;
      }
      rc = grad ? launch_vocab_gemm<kVocabScaled>(mX, mWk, mGs, mX, a, pairs, false, st)
                : launch_vocab_gemm<kVocabStats>(mX, mWk, mX, mX, a, pairs, true, st);
      if (rc) return rc;
      if ((rc = run_rows(i0, n))) return rc;
    }
    if (!grad) continue;
    // g from lse: the backward alone, or again for a run whose scaled exponentials do not serve
    if ((rc = launch_vocab_gemm<kVocabProb>(mX, mWk, mGs, mX, a, pairs, !stats, st))) return rc;
    VocabGemmArgs d = plan_vocab_gemm(n, c.h, c.v, true, pairs);
    d.v = a.N;
    d.targets = a.targets;
    d.ignore = a.ignore;
    d.dloss = a.dloss;
    d.dlse = a.dlse;
    d.W = c.W;
    d.target_factor = target_factor;
    if (stats) {
      d.redo = redo;
      d.factor = factor;
    }
    if ((rc = launch_vocab_gemm<kVocabGrad>(mG, mWmn, mD, mPart, d, pairs, false, st))) return rc;
    if (d.splits > 1) {
      const int tiles = d.m_tiles * d.n_tiles - d.whole;
      if ((rc = launch_after(prof::kVocabRows, vocab_join_kernel, dim3(static_cast<unsigned>(tiles), vg::BM / 8), 256, st, 0,
                             part, c.dX + i0 * c.h, d)))
        return rc;
    }
  }
  return QLORA_OK;
}

int check_vocab_args(const VocabCall& c, bool stats, bool grad, const void* workspace) {
  if (!c.X || !c.W || !c.targets || !c.lse || (stats && !c.loss) || (grad && (!c.dX || !c.dloss)))
    return QLORA_ERR_INVALID_ARG;
  int rc = check_vocab_shape(c.t, c.h, c.v);
  if (rc) return rc;
  if (!aligned16(c.X) || !aligned16(c.W) || (c.dX && !aligned16(c.dX)) || (workspace && !aligned16(workspace)) ||
      (reinterpret_cast<uintptr_t>(c.targets) & 7u) || !aligned4(c.loss) || !aligned4(c.lse) ||
      !aligned4(c.dloss) || !aligned4(c.dlse))
    return QLORA_ERR_MISALIGNED;
  return QLORA_OK;
}

}  // namespace

extern "C" {

int qlora_linear_fwd_epilogue(const uint16_t* X, int64_t t, const nf4_weight* W, const uint16_t* L1,
                              const uint16_t* L2, int64_t r, float s, const uint16_t* bias, int act,
                              const uint16_t* residual, uint16_t* Y, uint16_t* Z_out, uint16_t* sT_out,
                              void* workspace, size_t ws_bytes, qlora_stream_t stream) {
  int rc = check_fwd_args(X, t, W, L1, L2, r, s, Y, sT_out, workspace);
  if (rc) return rc;
  if (!valid_act(act)) return QLORA_ERR_INVALID_ARG;
  if ((bias && !aligned16(bias)) || (residual && !aligned16(residual)) || (Z_out && !aligned16(Z_out)))
    return QLORA_ERR_MISALIGNED;
  if (!workspace || ws_bytes < qlora_fwd_epilogue_workspace_bytes(t, W->in_features, W->out_features, r))
    return QLORA_ERR_WORKSPACE;
  EpilogueArgs e{};
  e.bias = bias;
  e.residual = residual;
  e.z_out = Z_out;
  e.act = act;
  return fwd_core(X, X, t, W, L1, L2, r, s, Y, sT_out, workspace, reinterpret_cast<cudaStream_t>(stream), &e);
}

size_t qlora_fwd_epilogue_workspace_bytes(int64_t t, int64_t h, int64_t o, int64_t r) {
  const size_t base = qlora_fwd_workspace_bytes(t, h, o, r);
  if (!base || !epilogue_uses_gemm(t, h, o, r)) return base;
  const int shares = plan_epilogue(t, h, o).shares;
  return lora_region_bytes(t, r) + (shares > 1 ? static_cast<size_t>(shares) * t * o * 4 : 0);
}

size_t qlora_epilogue_bwd_workspace_bytes(int64_t t, int64_t o) {
  if (t < 1 || t >= kMaxDim || o < 8 || o % 8 != 0 || o >= kMaxDim) return 0;
  return align256(static_cast<size_t>(epilogue_runs(t, o, 0, 0)) * o * 4);
}

int qlora_epilogue_bwd(const uint16_t* dY, const uint16_t* Z, int64_t t, int64_t o, int act, uint16_t* dZ,
                       float* dbias, void* workspace, size_t ws_bytes, qlora_stream_t stream) {
  if (!dY || !valid_act(act) || (!dZ && !dbias) || (act != QLORA_ACT_NONE && !Z) || t < 1)
    return QLORA_ERR_INVALID_ARG;
  if (o < 8 || o % 8 != 0 || o >= kMaxDim || t >= kMaxDim) return QLORA_ERR_BAD_SHAPE;
  if (!aligned16(dY) || (Z && !aligned16(Z)) || (dZ && !aligned16(dZ)) || (dbias && !aligned16(dbias)) ||
      (workspace && !aligned16(workspace)))
    return QLORA_ERR_MISALIGNED;
  if (dbias && (!workspace || ws_bytes < qlora_epilogue_bwd_workspace_bytes(t, o))) return QLORA_ERR_WORKSPACE;
  int dev, rc;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int runs = epilogue_runs(t, o, sm_count(dev), device_info(dev).epi_bwd_ctas);
  EpilogueBwdArgs a{};
  a.dY = dY;
  a.Z = Z;
  a.dZ = dZ;
  a.part = !dbias ? nullptr : (runs == 1 ? dbias : reinterpret_cast<float*>(workspace));
  a.t = t;
  a.o = static_cast<int>(o);
  dim3 grid(static_cast<unsigned>((o + ep::kCols - 1) / ep::kCols), static_cast<unsigned>(runs));
  {
    prof::Scope ps(prof::kEpilogueBwd, st);
    switch (act) {
      case QLORA_ACT_RELU: epilogue_bwd_kernel<kActRelu><<<grid, ep::kWarps * 32, 0, st>>>(a); break;
      case QLORA_ACT_GELU: epilogue_bwd_kernel<kActGelu><<<grid, ep::kWarps * 32, 0, st>>>(a); break;
      case QLORA_ACT_GELU_TANH: epilogue_bwd_kernel<kActGeluTanh><<<grid, ep::kWarps * 32, 0, st>>>(a); break;
      case QLORA_ACT_SILU: epilogue_bwd_kernel<kActSilu><<<grid, ep::kWarps * 32, 0, st>>>(a); break;
      default: epilogue_bwd_kernel<kActNone><<<grid, ep::kWarps * 32, 0, st>>>(a); break;
    }
  }
  if ((rc = launch_status())) return rc;
  if (!dbias || runs == 1) return QLORA_OK;
  return launch_finish(prof::kEpilogueBwd, a.part, nullptr, nullptr, dbias, nullptr, nullptr, static_cast<int>(t), a.o, 1, runs, 0, 1, st);
}

int qlora_norm_residual_fwd(const uint16_t* x, const uint16_t* y, int64_t t, int64_t h, const uint16_t* w_post,
                            const uint16_t* gate, int64_t rows_per_gate, float scale, const uint16_t* w_pre,
                            float eps, uint16_t* x_out, uint16_t* n_out, float* rstd_post, float* rstd_pre,
                            qlora_stream_t stream) {
  if (!x || (!y && (w_post || gate)) || !w_pre != !n_out || (!x_out && !n_out) || (rstd_post && !w_post) ||
      (rstd_pre && !w_pre) || (gate && rows_per_gate < 1) || !std::isfinite(scale) || !std::isfinite(eps) ||
      eps < 0.f)
    return QLORA_ERR_INVALID_ARG;
  int rc = check_norm_shape(t, h);
  if (rc) return rc;
  for (const void* p : {static_cast<const void*>(x), static_cast<const void*>(y), static_cast<const void*>(w_post),
                        static_cast<const void*>(gate), static_cast<const void*>(w_pre),
                        static_cast<const void*>(x_out), static_cast<const void*>(n_out)})
    if (p && !aligned16(p)) return QLORA_ERR_MISALIGNED;
  if (!aligned4(rstd_post) || !aligned4(rstd_pre)) return QLORA_ERR_MISALIGNED;
  int dev;
  if ((rc = current_device(&dev))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormFwdArgs a{};
  a.x = x;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.x_out = x_out;
  a.n_out = n_out;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.t = static_cast<int>(t);
  a.h = static_cast<int>(h);
  a.rows_per_gate = static_cast<int>(gate ? std::min(rows_per_gate, t) : t);
  a.scale = scale;
  a.eps = eps;
  {
    prof::Scope ps(prof::kNorm, st);
    const int sms = sm_count(dev);
    constexpr int wpc = nr::kWarpRowThreads / 32;
    const bool warp_row = h <= nr::kWarpRowH;
    const unsigned threads = warp_row ? nr::kWarpRowThreads : norm_threads(h);
    const int64_t rows = warp_row ? (t + wpc - 1) / wpc : t;   // CTAs' worth of rows
    // CTAs that fit an SM by threads (up to 128 registers each; the rings take 128 KB together). With two
    // rounds of rows for each they stay and prefetch; with fewer, a row's own latency is all there is,
    // and a row with one vector per thread is the shortest way through it.
    const int64_t wave = static_cast<int64_t>(sms) * std::max(1u, std::min(8u, 512u / threads));
    const size_t smem = static_cast<size_t>(nr::kFwdStages) * 2 * 2 * threads * 16;
    if (h <= nr::kStayH && rows >= 2 * wave) {
      const unsigned grid = static_cast<unsigned>(wave);
      if (warp_row)
        norm_residual_fwd_kernel<2, true, true><<<grid, threads, smem, st>>>(a);
      else if (y && w_post && w_pre && x_out && h == 16 * static_cast<int64_t>(threads))
        norm_residual_fwd_kernel<2, false, true, true><<<grid, threads, smem, st>>>(a);
      else
        norm_residual_fwd_kernel<2, false, true><<<grid, threads, smem, st>>>(a);
    } else if (warp_row) {
      norm_residual_fwd_kernel<2, true, false><<<static_cast<unsigned>(rows), threads, 0, st>>>(a);
    } else if (h <= 8192) {
      norm_residual_fwd_kernel<1, false, false>
          <<<static_cast<unsigned>(rows), static_cast<unsigned>((h / 8 + 31) / 32 * 32), 0, st>>>(a);
    } else {
      norm_residual_fwd_kernel<2, false, false><<<static_cast<unsigned>(rows), threads, 0, st>>>(a);
    }
  }
  return launch_status();
}

size_t qlora_norm_residual_bwd_workspace_bytes(int64_t t, int64_t h) {
  if (check_norm_shape(t, h) != QLORA_OK) return 0;
  const NormBwdPlan p = plan_norm_bwd(t, h, kMaxSms);
  return 2 * align256(static_cast<size_t>(p.ctas) * h * 4) + align256(2 * static_cast<size_t>(p.units) * h * 4);
}

int qlora_norm_residual_bwd(const uint16_t* dx_out, const uint16_t* dn, const uint16_t* x_out, const uint16_t* y,
                            int64_t t, int64_t h, const uint16_t* w_post, const uint16_t* gate,
                            int64_t rows_per_gate, float scale, const uint16_t* w_pre, const float* rstd_post,
                            const float* rstd_pre, uint16_t* dx, uint16_t* dy, float* dw_post, float* dgate,
                            float* dw_pre, void* workspace, size_t ws_bytes, qlora_stream_t stream) {
  if (!dx || (!dx_out && !dn) || !dn != !w_pre || !dn != !dw_pre || (dn && (!x_out || !rstd_pre)) || !y != !dy ||
      (!y && (w_post || gate)) || !w_post != !dw_post || (w_post && !rstd_post) || !gate != !dgate ||
      (gate && rows_per_gate < 1) || !std::isfinite(scale))
    return QLORA_ERR_INVALID_ARG;
  int rc = check_norm_shape(t, h);
  if (rc) return rc;
  for (const void* p :
       {static_cast<const void*>(dx_out), static_cast<const void*>(dn), static_cast<const void*>(x_out),
        static_cast<const void*>(y), static_cast<const void*>(w_post), static_cast<const void*>(gate),
        static_cast<const void*>(w_pre), static_cast<const void*>(dx), static_cast<const void*>(dy),
        static_cast<const void*>(dw_post), static_cast<const void*>(dgate), static_cast<const void*>(dw_pre),
        static_cast<const void*>(workspace)})
    if (p && !aligned16(p)) return QLORA_ERR_MISALIGNED;
  if (!aligned4(rstd_post) || !aligned4(rstd_pre)) return QLORA_ERR_MISALIGNED;
  if (!workspace || ws_bytes < qlora_norm_residual_bwd_workspace_bytes(t, h)) return QLORA_ERR_WORKSPACE;
  int dev;
  if ((rc = current_device(&dev))) return rc;
  if (sm_count(dev) > kMaxSms) return QLORA_ERR_UNSUPPORTED_DEVICE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const NormBwdPlan pl = plan_norm_bwd(t, h, sm_count(dev));
  uint8_t* ws = reinterpret_cast<uint8_t*>(workspace);
  const size_t part = align256(static_cast<size_t>(pl.ctas) * h * 4);
  NormBwdArgs a{};
  a.dx_out = dx_out;
  a.dn = dn;
  a.x_out = x_out;
  a.y = y;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.rstd_post = rstd_post;
  a.rstd_pre = rstd_pre;
  a.dx = dx;
  a.dy = dy;
  a.dw_post = dw_post;
  a.dgate = dgate;
  a.dw_pre = dw_pre;
  a.part_post = pl.ctas == 1 ? dw_post : reinterpret_cast<float*>(ws);
  a.part_pre = pl.ctas == 1 ? dw_pre : reinterpret_cast<float*>(ws + part);
  a.part_gate = reinterpret_cast<float*>(ws + 2 * part);
  a.t = static_cast<int>(t);
  a.h = static_cast<int>(h);
  a.rows_per_gate = static_cast<int>(gate ? std::min(rows_per_gate, t) : t);
  a.units = pl.units;
  a.scale = scale;
  {
    prof::Scope ps(prof::kNorm, st);
    const unsigned grid = static_cast<unsigned>(pl.ctas), threads = static_cast<unsigned>(pl.threads);
    if (h <= nr::kWarpRowH)
      norm_residual_bwd_kernel<true, false><<<grid, threads, pl.smem, st>>>(a);
    else if (h <= nr::kStayH && dx_out && dn && w_post && h == 16 * static_cast<int64_t>(threads))
      norm_residual_bwd_kernel<false, false, true><<<grid, threads, pl.smem, st>>>(a);
    else if (h <= nr::kStayH)
      norm_residual_bwd_kernel<false, false><<<grid, threads, pl.smem, st>>>(a);
    else
      norm_residual_bwd_kernel<false, true><<<grid, threads, pl.smem, st>>>(a);
  }
  if ((rc = launch_status())) return rc;
  // gate rows are shared between units unless every unit's run starts a new one
  const int gate_blocks =
      gate && a.rows_per_gate > 1 && pl.units > 1 ? std::min(64, (a.t - 1) / a.rows_per_gate + 1) : 0;
  float* pre = pl.ctas > 1 ? dw_pre : nullptr;
  float* post = pl.ctas > 1 ? dw_post : nullptr;
  if (!pre && !post && !gate_blocks) return QLORA_OK;
  return launch_finish(prof::kNorm, a.part_pre, a.part_post, a.part_gate, pre, post, dgate, a.t, a.h, a.rows_per_gate,
                       pl.ctas, pl.units, 2 + gate_blocks, st);
}

size_t qlora_vocab_loss_fwd_workspace_bytes(int64_t t, int64_t h, int64_t v) {
  return vocab_ws_bytes(t, h, v, true, false);
}
size_t qlora_vocab_loss_bwd_workspace_bytes(int64_t t, int64_t h, int64_t v) {
  return vocab_ws_bytes(t, h, v, false, true);
}
size_t qlora_vocab_loss_fwd_bwd_workspace_bytes(int64_t t, int64_t h, int64_t v) {
  return vocab_ws_bytes(t, h, v, true, true);
}

int qlora_vocab_loss_fwd(const uint16_t* X, const uint16_t* W, int64_t t, int64_t h, int64_t v,
                         const int64_t* targets, int64_t ignore_index, float* loss, float* lse, void* workspace,
                         size_t ws_bytes, qlora_stream_t stream) {
  const VocabCall c{X, W, t, h, v, targets, ignore_index, loss, lse, nullptr, nullptr, nullptr};
  const int rc = check_vocab_args(c, true, false, workspace);
  if (rc) return rc;
  if (!workspace || ws_bytes < qlora_vocab_loss_fwd_workspace_bytes(t, h, v)) return QLORA_ERR_WORKSPACE;
  return vocab_core(c, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int qlora_vocab_loss_bwd(const uint16_t* X, const uint16_t* W, int64_t t, int64_t h, int64_t v,
                         const int64_t* targets, int64_t ignore_index, const float* lse, const float* dloss,
                         const float* dlse, uint16_t* dX, void* workspace, size_t ws_bytes,
                         qlora_stream_t stream) {
  const VocabCall c{X, W, t, h, v, targets, ignore_index, nullptr, const_cast<float*>(lse), dloss, dlse, dX};
  const int rc = check_vocab_args(c, false, true, workspace);
  if (rc) return rc;
  if (!workspace || ws_bytes < qlora_vocab_loss_bwd_workspace_bytes(t, h, v)) return QLORA_ERR_WORKSPACE;
  return vocab_core(c, workspace, reinterpret_cast<cudaStream_t>(stream));
}

int qlora_vocab_loss_fwd_bwd(const uint16_t* X, const uint16_t* W, int64_t t, int64_t h, int64_t v,
                             const int64_t* targets, int64_t ignore_index, const float* dloss, float* loss,
                             float* lse, uint16_t* dX, void* workspace, size_t ws_bytes, qlora_stream_t stream) {
  const VocabCall c{X, W, t, h, v, targets, ignore_index, loss, lse, dloss, nullptr, dX};
  const int rc = check_vocab_args(c, true, true, workspace);
  if (rc) return rc;
  if (!workspace || ws_bytes < qlora_vocab_loss_fwd_bwd_workspace_bytes(t, h, v)) return QLORA_ERR_WORKSPACE;
  return vocab_core(c, workspace, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
