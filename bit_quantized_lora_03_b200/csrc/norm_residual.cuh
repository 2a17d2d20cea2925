// The norms before and after a block, fused with the block's gate and residual scale, for the
// residual stream that joins QLoRA linears:
//   u = y . rstd(y) . w_post            (u = y without w_post)
//   x' = x + scale . gate . u           (gate: one row of h values per rows_per_gate tokens)
//   n = x' . rstd(x') . w_pre           (the next block's input; left out without w_pre)
// with rstd(a) = 1 / sqrt(mean(a^2) + eps) over a row of h values, and the backward of all of it.
//
// One pass over HBM each way: a row lives in the registers of one CTA (or, for h <= 512, of one
// warp, so that short rows do not leave most of a CTA idle) between its loads and its stores.
// All sums, statistics and intermediate values are fp32; x', n, dx and dy are rounded once, to
// bf16, when they are stored (n is computed from the unrounded x').
//
// Backward, with xh = x'.rx, yh = y.ry, dh = dn.w_pre, d0 = dx' + rx.dh, k = scale.gate.w_post.yh:
//   S1 = sum dh.xh, S2 = sum k.d0, S3 = sum k.xh           (one reduction of three sums per row)
//   g  = d0 - rx.xh.S1/h                                     = dx, the gradient of x' and of x
//   dy = ry.(scale.gate.w_post.g - yh.(S2 - rx.S1/h.S3)/h)   (scale.gate.g without w_post)
//   q  = sum over a gate row's tokens of g.yh: dgate = scale.w_post.q, dw_post = scale.sum gate.q,
//   dw_pre = sum_t dn.xh
// The second norm's sum over g is formed from S2 and S3 so that a row needs one block reduction,
// not two in a row. Token sums: every CTA (or warp) takes one contiguous run of rows, keeps its
// columns' sums in registers, writes them once as partial rows, and norm_residual_finish_kernel
// adds the partials in a fixed order (no atomics: results repeat bit for bit).
//
// Bound: HBM, 2 bytes for each value of x, y, x', n (forward: 4 per element of a row's h) and of dx', dn,
// x', y, dx, dy (backward: 6). Measured: forward, 2048 x 8192, 24.3 us (5.5 TB/s); backward, 4096 x 4096,
// 39.9 us (5.0 TB/s) and 4.8 us for the partial rows; one row 2.5 us, the latency of two reductions.
#pragma once

#include "qlora_common.cuh"

namespace qlora {

namespace nr {
constexpr int kMaxH = 16384;
constexpr int kStayH = 8192;     // rows whose sums and parameters fit the registers of 512 threads
constexpr int kWarpRowH = 512;   // rows up to this long belong to one warp
constexpr int kWarpRowThreads = 256;
constexpr int kFinishCols = 128; // columns per block of the finish kernel
constexpr int kFinishWarps = 16;
constexpr int kBwdStages = 3, kFwdStages = 4;   // rows in a CTA's ring, the one in work among them
}  // namespace nr

struct NormFwdArgs {
  const uint16_t* x;
  const uint16_t* y;       // or NULL: x' = x
  const uint16_t* w_post;  // or NULL
  const uint16_t* gate;    // or NULL
  const uint16_t* w_pre;   // or NULL: no n
  uint16_t* x_out;
  uint16_t* n_out;
  float* rstd_post;        // or NULL
  float* rstd_pre;         // or NULL
  int t, h, rows_per_gate;
  float scale, eps;
};

struct NormBwdArgs {
  const uint16_t* dx_out;  // gradient of x', or NULL (zero)
  const uint16_t* dn;      // gradient of n, or NULL (no w_pre)
  const uint16_t* x_out;   // x' (read with dn)
  const uint16_t* y;       // or NULL
  const uint16_t* w_post;
  const uint16_t* gate;
  const uint16_t* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  uint16_t* dx;
  uint16_t* dy;            // or NULL
  float* dw_post;          // outputs of the token sums (NULL where there is no such input)
  float* dgate;
  float* dw_pre;
  float* part_post;        // partial rows, one of h per CTA (one CTA: the outputs themselves)
  float* part_pre;
  float* part_gate;        // 2 x units x h: a unit's share of the gate row it opens in / closes in
  int t, h, rows_per_gate; // rows_per_gate: t where one row (or none) serves all tokens
  int units;               // runs of rows: CTAs, or warps for short rows
  float scale;
};

__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Sums of N values over a row's threads: one warp, or the CTA through `red` (two halves used in
// turn, so that one barrier per reduction is enough).
template <int N, bool kWarpRow>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
  if (kWarpRow) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float* b = red + turn * (N * 32);
  turn ^= 1;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) b[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < warps ? b[i * 32 + lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], o);
}

__device__ __forceinline__ uint4 ldg_vec(const uint16_t* p, int64_t vec) {
  return __ldg(reinterpret_cast<const uint4*>(p) + vec);
}
// activations are read once: no reason to keep them in L1
__device__ __forceinline__ uint4 ldg_stream(const uint16_t* p, int64_t vec) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(reinterpret_cast<const uint4*>(p) + vec));
  return v;
}

// Two fp32 values in a register pair, for the packed fp32x2 instructions (one issue for two results).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
// bf16x2 -> fp32x2 (exact) and back (round to nearest even)
__device__ __forceinline__ F2 widen(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t narrow(F2 a) {
  const float2 f = split(a);
  return pack_bf16x2(f.x, f.y);
}
struct V8 {   // eight values
  F2 p[4];
};
__device__ __forceinline__ V8 widen8(const uint4& q) {
  V8 r;
  r.p[0] = widen(q.x);
  r.p[1] = widen(q.y);
  r.p[2] = widen(q.z);
  r.p[3] = widen(q.w);
  return r;
}
__device__ __forceinline__ uint4 narrow8(const V8& a) {
  return make_uint4(narrow(a.p[0]), narrow(a.p[1]), narrow(a.p[2]), narrow(a.p[3]));
}
__device__ __forceinline__ V8 fill8(float x) {
  V8 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r.p[e] = f2(x, x);
  return r;
}
__device__ __forceinline__ void store8(float* p, int64_t vec, const V8& a) {
  float4* q = reinterpret_cast<float4*>(p) + 2 * vec;
  const float2 f0 = split(a.p[0]), f1 = split(a.p[1]), f2_ = split(a.p[2]), f3 = split(a.p[3]);
  q[0] = make_float4(f0.x, f0.y, f1.x, f1.y);
  q[1] = make_float4(f2_.x, f2_.y, f3.x, f3.y);
}

// A thread's own ring of row pieces in shared memory, filled ahead of use by asynchronous copies:
// rows in flight cost no registers, and since a thread reads only what it copied itself, waiting
// for its own copies is all the synchronisation there is.
__device__ __forceinline__ void cp_async_16(void* dst, const uint16_t* src, int64_t vec) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)),
               "l"(reinterpret_cast<const uint4*>(src) + vec)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit_group() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {   // all but the newest N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// scale . w_post . gate for one vector (absent factors are 1)
__device__ __forceinline__ V8 branch_scale(const uint16_t* w_post, const uint16_t* gate, float scale, int v) {
  V8 c = fill8(scale);
  if (w_post) {
    const V8 w = widen8(ldg_vec(w_post, v));
#pragma unroll
    for (int e = 0; e < 4; ++e) c.p[e] = c.p[e] * w.p[e];
  }
  if (gate) {
    const V8 g = widen8(ldg_vec(gate, v));
#pragma unroll
    for (int e = 0; e < 4; ++e) c.p[e] = c.p[e] * g.p[e];
  }
  return c;
}

// Threads of a row hold VPT vectors of 8 each. kStay: the CTAs stay and walk the rows, kFwdStages - 1
// of them in flight in the ring, the parameters in registers; else one row per CTA or warp, loaded
// directly (few rows, where latency counts, or rows too long for the registers). kAll: every operand
// is there and the row fills its threads, which spares the checks (of the backward's 28.8 million
// warp instructions at 4096 x 4096 it leaves 19.9).
template <int VPT, bool kWarpRow, bool kStay, bool kAll = false>
__global__ void __launch_bounds__(kWarpRow ? nr::kWarpRowThreads : (kStay ? 512 : 1024))
    norm_residual_fwd_kernel(const NormFwdArgs a) {
  constexpr int S = nr::kFwdStages;
  extern __shared__ __align__(16) uint4 ring[];   // [stage][x, y][VPT][thread]
  __shared__ float red[2 * 32];
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int per_cta = kWarpRow ? nr::kWarpRowThreads / 32 : 1;
  const int row0 = blockIdx.x * per_cta + (kWarpRow ? threadIdx.x >> 5 : 0);
  const int64_t step = kStay ? static_cast<int64_t>(gridDim.x) * per_cta : a.t;
  const int nvec = a.h >> 3;
  const bool has_y = kAll || a.y, has_post = kAll || a.w_post, has_pre = kAll || a.w_pre;
  const float inv_h = 1.f / static_cast<float>(a.h);
  int turn = 0, stage = 0;
  auto inside = [&](int v) { return kAll || v < nvec; };
  auto piece = [&](int st, int which, int i) { return ring + ((st * 2 + which) * VPT + i) * blockDim.x + threadIdx.x; };
  auto request = [&](int64_t row, int st) {
    if (row < a.t) {
      const int64_t base = row * nvec;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nthr + tid;
        if (inside(v)) {
          if (has_y) cp_async_16(piece(st, 1, i), a.y, base + v);
          cp_async_16(piece(st, 0, i), a.x, base + v);
        }
      }
    }
    cp_async_commit_group();
  };
  if (kStay) {
#pragma unroll
    for (int k = 0; k < S - 1; ++k) request(row0 + k * step, k);
  }
  int cur = -1;         // the gate row that c holds
  V8 c[VPT], w[VPT];
  if (kStay && has_pre) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (inside(i * nthr + tid)) w[i] = widen8(ldg_vec(a.w_pre, i * nthr + tid));
  }
  // (whole warps or whole CTAs leave together)
  for (int64_t row = row0; row < a.t; row += step) {
    const int64_t base = row * nvec;
    uint4 xq[VPT], yq[VPT];
    if (kStay) {
      request(row + (S - 1) * step, stage == 0 ? S - 1 : stage - 1);   // the slot of the row before
      cp_async_wait_group<S - 1>();
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      xq[i] = yq[i] = make_uint4(0u, 0u, 0u, 0u);
      if (inside(v)) {
        if (has_y) yq[i] = kStay ? *piece(stage, 1, i) : ldg_stream(a.y, base + v);
        xq[i] = kStay ? *piece(stage, 0, i) : ldg_stream(a.x, base + v);
      }
    }
    if (kStay) stage = stage + 1 == S ? 0 : stage + 1;
    const int grow = a.gate && a.rows_per_gate < a.t ? static_cast<int>(row) / a.rows_per_gate : 0;
    if (has_y && grow != cur) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (inside(i * nthr + tid))
          c[i] = branch_scale(a.w_post, a.gate ? a.gate + static_cast<int64_t>(grow) * a.h : nullptr, a.scale, i * nthr + tid);
      cur = grow;
    }
    V8 x[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) x[i] = widen8(xq[i]);
    if (has_y) {
      V8 y[VPT];
#pragma unroll
      for (int i = 0; i < VPT; ++i) y[i] = widen8(yq[i]);
      F2 ry = f2(1.f, 1.f);
      if (has_post) {
        F2 q = f2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) q = fma2(y[i].p[e], y[i].p[e], q);
        float s[1] = {split(q).x + split(q).y};
        row_sum<1, kWarpRow>(s, red, turn);
        const float r = rsqrtf(fmaf(s[0], inv_h, a.eps));
        if (tid == 0 && a.rstd_post) a.rstd_post[row] = r;
        ry = f2(r, r);
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (inside(i * nthr + tid))
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i].p[e] = fma2(y[i].p[e] * ry, c[i].p[e], x[i].p[e]);
    }
    if (kAll || a.x_out) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (inside(i * nthr + tid)) reinterpret_cast<uint4*>(a.x_out)[base + i * nthr + tid] = narrow8(x[i]);
    }
    if (!has_pre) continue;
    F2 q = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) q = fma2(x[i].p[e], x[i].p[e], q);   // (zero behind the row's end)
    float s[1] = {split(q).x + split(q).y};
    if (!kStay) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (inside(i * nthr + tid)) w[i] = widen8(ldg_vec(a.w_pre, i * nthr + tid));
    }
    row_sum<1, kWarpRow>(s, red, turn);
    const float r = rsqrtf(fmaf(s[0], inv_h, a.eps));
    if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = r;
    const F2 rx = f2(r, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!inside(i * nthr + tid)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i].p[e] = x[i].p[e] * rx * w[i].p[e];
      reinterpret_cast<uint4*>(a.n_out)[base + i * nthr + tid] = narrow8(x[i]);
    }
  }
}

// The first row of unit u when t rows go to `units` contiguous runs.
__device__ __forceinline__ int unit_row(int t, int units, int u) {
  const int base = t / units, extra = t - base * units;
  return u * base + min(u, extra);
}

// Two vectors of 8 per thread. Over rows a thread sums, for its columns, dw_pre and
//   q = sum g.yh over the tokens of one gate row,
// from which dgate = scale.w_post.q and dw_post = scale.(sum over gate rows of gate.q): one product
// and one sum per element and row instead of two of each.
// kWide: rows too long for that many registers (1024 threads): the sums lie in shared memory, rows
// and parameters are loaded directly. Else rows come through the ring and sums and parameters stay in
// registers (dw_post, which changes once per gate row, in shared memory). kAll: as in the forward.
template <bool kWarpRow, bool kWide, bool kAll = false>
__global__ void __launch_bounds__(kWarpRow ? nr::kWarpRowThreads : (kWide ? 1024 : 512))
    norm_residual_bwd_kernel(const NormBwdArgs a) {
  constexpr int VPT = 2, S = nr::kBwdStages;
  pdl_launch_dependents();
  extern __shared__ __align__(16) float4 dyn[];
  __shared__ float red[2 * 3 * 32];
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int unit = kWarpRow ? blockIdx.x * (nr::kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int nvec = a.h >> 3;
  // (a CTA's last warps may have no rows: unit >= units, r0 == r1 == t)
  const int r0 = min(a.t, unit_row(a.t, a.units, unit)), r1 = min(a.t, unit_row(a.t, a.units, unit + 1));
  const float inv_h = 1.f / static_cast<float>(a.h);
  const bool has_dx = kAll || a.dx_out, has_n = kAll || a.dn, has_y = kAll || a.y, has_post = kAll || a.w_post;
  auto inside = [&](int v) { return kAll || v < nvec; };
  int turn = 0, stage = 0;

  // shared sums: [sum][VPT][half vector][thread], every word of one thread only
  float4* ssum = dyn;
  uint4* ring = reinterpret_cast<uint4*>(dyn + 2 * VPT * blockDim.x);   // [stage][array][VPT][thread]
  auto sref = [&](int k, int i, int half) -> float4& {
    return ssum[((k * VPT + i) * 2 + half) * blockDim.x + threadIdx.x];
  };
  auto sget = [&](int k, int i) {
    const float4 lo = sref(k, i, 0), hi = sref(k, i, 1);
    V8 r;
    r.p[0] = f2(lo.x, lo.y); r.p[1] = f2(lo.z, lo.w); r.p[2] = f2(hi.x, hi.y); r.p[3] = f2(hi.z, hi.w);
    return r;
  };
  auto sput = [&](int k, int i, const V8& v) {
    const float2 f0 = split(v.p[0]), f1 = split(v.p[1]), f2_ = split(v.p[2]), f3 = split(v.p[3]);
    sref(k, i, 0) = make_float4(f0.x, f0.y, f1.x, f1.y);
    sref(k, i, 1) = make_float4(f2_.x, f2_.y, f3.x, f3.y);
  };
  constexpr int kPost = 0, kPre = 1, kQ = 2;
  V8 pre[VPT], q[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    pre[i] = q[i] = fill8(0.f);
    sput(kPost, i, q[i]);
    if (kWide) {
      sput(kPre, i, q[i]);
      sput(kQ, i, q[i]);
    }
  }
  auto request = [&](int row, int st) {
    if (row < r1) {
      const int64_t base = static_cast<int64_t>(row) * nvec;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nthr + tid;
        if (!inside(v)) continue;
        uint4* p = ring + (st * 4 * VPT + i) * blockDim.x + threadIdx.x;
        const int next = VPT * blockDim.x;
        if (has_dx) cp_async_16(p, a.dx_out, base + v);
        if (has_n) {
          cp_async_16(p + next, a.dn, base + v);
          cp_async_16(p + 2 * next, a.x_out, base + v);
        }
        if (has_y) cp_async_16(p + 3 * next, a.y, base + v);
      }
    }
    cp_async_commit_group();
  };
  V8 w[VPT], c[VPT];   // w_pre; scale . w_post . gate
  if (!kWide) {
#pragma unroll
    for (int k = 0; k < S - 1; ++k) request(r0 + k, k);
    if (has_n) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (inside(i * nthr + tid)) w[i] = widen8(ldg_vec(a.w_pre, i * nthr + tid));
    }
  }
  int cur = -1;
  float rx_next = has_n && r0 < r1 ? __ldg(a.rstd_pre + r0) : 0.f;
  float ry_next = has_post && r0 < r1 ? __ldg(a.rstd_post + r0) : 1.f;
  int left = 0;     // rows until this gate row's sum is due
  for (int row = r0; row < r1; ++row) {
    const int64_t base = static_cast<int64_t>(row) * nvec;
    if (!kWide) {
      request(min(row + (S - 1), r1), stage == 0 ? S - 1 : stage - 1);   // the slot of the row before
      cp_async_wait_group<S - 1>();
    }
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    auto get = [&](int which, const uint16_t* src, int i) {   // (again behind the reduction: the raw row
      const int v = i * nthr + tid;                           // needs no registers meanwhile)
      if (!kAll && (!src || v >= nvec)) return zero;
      return kWide ? ldg_vec(src, base + v) : ring[((stage * 4 + which) * VPT + i) * blockDim.x + threadIdx.x];
    };
    if (left == 0) {   // a new gate row (or the first row)
      cur = row / a.rows_per_gate;
      const int64_t end = (static_cast<int64_t>(cur) + 1) * a.rows_per_gate;
      left = static_cast<int>(min(end, static_cast<int64_t>(r1)) - row);
      if (!kWide && has_y) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
          if (inside(i * nthr + tid))
            c[i] = branch_scale(a.w_post, a.gate ? a.gate + static_cast<int64_t>(cur) * a.h : nullptr, a.scale, i * nthr + tid);
      }
    }
    const uint16_t* gate = a.gate ? a.gate + static_cast<int64_t>(cur) * a.h : nullptr;
    const float rx1 = rx_next, ry1 = ry_next;
    if (row + 1 < r1) {   // (a row ahead: their latency is not the row's)
      if (has_n) rx_next = __ldg(a.rstd_pre + row + 1);
      if (has_post) ry_next = __ldg(a.rstd_post + row + 1);
    }
    const F2 rx = f2(rx1, rx1), ry = f2(ry1, ry1);
    F2 s0 = f2(0.f, 0.f), s1 = s0, s2 = s0;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (!inside(v)) continue;
      V8 d = widen8(get(0, a.dx_out, i)), x;
      if (has_n) {
        const V8 dn = widen8(get(1, a.dn, i));
        x = widen8(get(2, a.x_out, i));
        if (kWide) w[i] = widen8(ldg_vec(a.w_pre, v));
        V8 p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x.p[e] = x.p[e] * rx;
          p.p[e] = dn.p[e] * x.p[e];
          s0 = fma2(p.p[e], w[i].p[e], s0);
          d.p[e] = fma2(dn.p[e] * rx, w[i].p[e], d.p[e]);
        }
        if (kWide) {
          const V8 o = sget(kPre, i);
#pragma unroll
          for (int e = 0; e < 4; ++e) p.p[e] = p.p[e] + o.p[e];
          sput(kPre, i, p);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) pre[i].p[e] = pre[i].p[e] + p.p[e];
        }
      }
      if (has_post) {
        const V8 y = widen8(get(3, a.y, i));
        if (kWide) c[i] = branch_scale(a.w_post, gate, a.scale, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 k = c[i].p[e] * y.p[e];   // ry is common to the row: applied below
          s1 = fma2(k, d.p[e], s1);
          if (has_n) s2 = fma2(k, x.p[e], s2);
        }
      }
    }
    if (has_n || has_post) {
      float s[3] = {split(s0).x + split(s0).y, split(s1).x + split(s1).y, split(s2).x + split(s2).y};
      row_sum<3, kWarpRow>(s, red, turn);
      const float c1 = rx1 * s[0] * inv_h;
      const float c2 = ry1 * (s[1] - c1 * s[2]) * inv_h;
      s0 = f2(-c1, -c1);
      s1 = f2(-c2 * ry1, -c2 * ry1);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (!inside(v)) continue;
      V8 g = widen8(get(0, a.dx_out, i));
      if (has_n) {
        const V8 dn = widen8(get(1, a.dn, i)), x = widen8(get(2, a.x_out, i));
        if (kWide) w[i] = widen8(ldg_vec(a.w_pre, v));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          g.p[e] = fma2(s0, x.p[e] * rx, fma2(dn.p[e] * rx, w[i].p[e], g.p[e]));
      }
      reinterpret_cast<uint4*>(a.dx)[base + v] = narrow8(g);
      if (!has_y) continue;
      V8 y = widen8(get(3, a.y, i));
      if (kWide) c[i] = branch_scale(a.w_post, gate, a.scale, v);
      V8 o;
      if (kWide) o = sget(kQ, i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        y.p[e] = y.p[e] * ry;
        if (kWide)
          o.p[e] = fma2(g.p[e], y.p[e], o.p[e]);
        else
          q[i].p[e] = fma2(g.p[e], y.p[e], q[i].p[e]);
        g.p[e] = g.p[e] * c[i].p[e];
        if (has_post) g.p[e] = fma2(s1, y.p[e], g.p[e] * ry);
      }
      if (kWide) sput(kQ, i, o);
      reinterpret_cast<uint4*>(a.dy)[base + v] = narrow8(g);
    }
    if (!kWide) stage = stage + 1 == S ? 0 : stage + 1;
    // the gate row's sum ends with its last token here: written as the result where this unit had
    // all of its tokens, else as this unit's share of it
    if (--left == 0 && has_y && (gate || has_post)) {
      const int64_t g0 = static_cast<int64_t>(cur) * a.rows_per_gate;
      const int64_t g1 = min(g0 + a.rows_per_gate, static_cast<int64_t>(a.t));
      float* dst = g0 >= r0 && g1 <= r1
          ? a.dgate + static_cast<int64_t>(cur) * a.h
          : a.part_gate + (static_cast<int64_t>(g0 < r0 ? 0 : a.units) + unit) * a.h;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nthr + tid;
        if (!inside(v)) continue;
        V8 o = kWide ? sget(kQ, i) : q[i];
        if (gate) {
          const V8 k = branch_scale(a.w_post, nullptr, a.scale, v);
          V8 r;
#pragma unroll
          for (int e = 0; e < 4; ++e) r.p[e] = k.p[e] * o.p[e];
          store8(dst, v, r);
        }
        if (a.w_post) {
          const V8 k = branch_scale(nullptr, gate, a.scale, v);
          V8 r = sget(kPost, i);
#pragma unroll
          for (int e = 0; e < 4; ++e) r.p[e] = fma2(k.p[e], o.p[e], r.p[e]);
          sput(kPost, i, r);
        }
        q[i] = fill8(0.f);
        if (kWide) sput(kQ, i, q[i]);
      }
    }
  }
  if (!kWarpRow) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (!inside(v)) continue;
      if (a.w_post) store8(a.part_post + static_cast<int64_t>(unit) * a.h, v, sget(kPost, i));
      if (a.dn) store8(a.part_pre + static_cast<int64_t>(unit) * a.h, v, kWide ? sget(kPre, i) : pre[i]);
    }
    return;
  }
  // short rows: the warps' sums are added here, one partial row per CTA
  float* sf = reinterpret_cast<float*>(ring);
  cp_async_wait_group<0>();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* part = k == 0 ? (a.w_post ? a.part_post : nullptr) : (a.dn ? a.part_pre : nullptr);
    if (!part) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (inside(i * nthr + tid))
        store8(sf + (threadIdx.x >> 5) * a.h, i * nthr + tid, k == 0 ? sget(kPost, i) : pre[i]);
    __syncthreads();
    for (int col = threadIdx.x; col < a.h; col += nr::kWarpRowThreads) {
      float v = 0.f;
#pragma unroll
      for (int w8 = 0; w8 < nr::kWarpRowThreads / 32; ++w8) v += sf[w8 * a.h + col];
      part[static_cast<int64_t>(blockIdx.x) * a.h + col] = v;
    }
  }
}

// Adds the partial rows in order. grid y: 0 dw_pre, 1 dw_post, 2.. the gate rows whose tokens fell
// to more than one unit: one block each while there are few, else blocks share them. A block takes
// 128 columns; its warps take every kFinishWarps-th partial row and are added in shared memory.
__global__ void __launch_bounds__(nr::kFinishWarps * 32)
    norm_residual_finish_kernel(const float* part_pre, const float* part_post, const float* part_gate,
                                float* dw_pre, float* dw_post, float* dgate, int t, int h,
                                int rows_per_gate, int parts, int units) {
  __shared__ float4 sh[nr::kFinishWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * nr::kFinishCols + lane * 4;
  pdl_wait();
  const bool cv = col < h;   // h % 8 == 0
  // out[col..] = the sum of rows [0, n) at `first`, and of the row at `extra` if there is one
  auto sum_rows = [&](const float* first, int n, const float* extra, float* out) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) { s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w; };
    if (cv) {
      if (extra && warp == 0) add(__ldcg(reinterpret_cast<const float4*>(extra + col)));
#pragma unroll 8
      for (int p = warp; p < n; p += nr::kFinishWarps)
        add(__ldcg(reinterpret_cast<const float4*>(first + static_cast<int64_t>(p) * h + col)));
    }
    sh[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && cv) {
#pragma unroll
      for (int w = 1; w < nr::kFinishWarps; ++w) add(sh[w][lane]);
      *reinterpret_cast<float4*>(out + col) = s;
    }
    __syncthreads();
  };
  if (blockIdx.y < 2) {
    float* out = blockIdx.y == 0 ? dw_pre : dw_post;
    if (out) sum_rows(blockIdx.y == 0 ? part_pre : part_post, parts, nullptr, out);
    return;
  }
  const int used = min(units, t);   // the units behind have no rows
  const int base = t / used, extra = t - base * used;
  auto unit_of = [&](int row) {     // the unit that has a row (the inverse of unit_row)
    const int long_rows = extra * (base + 1);
    return row < long_rows ? row / (base + 1) : extra + (row - long_rows) / base;
  };
  const int groups = (t - 1) / rows_per_gate + 1;
  for (int g = blockIdx.y - 2; g < groups; g += gridDim.y - 2) {
    // a gate row's shares: the closing one of the unit it starts in (row units + b0), unless that
    // unit has all of it and wrote the result, and the opening ones of the units behind
    const int64_t g0 = static_cast<int64_t>(g) * rows_per_gate;
    const int last = static_cast<int>(min(g0 + rows_per_gate, static_cast<int64_t>(t))) - 1;
    const int b0 = unit_of(static_cast<int>(g0)), b1 = unit_of(last);
    if (b0 != b1)
      sum_rows(part_gate + static_cast<int64_t>(b0 + 1) * h, b1 - b0,
               part_gate + static_cast<int64_t>(units + b0) * h, dgate + static_cast<int64_t>(g) * h);
  }
}

}  // namespace qlora
