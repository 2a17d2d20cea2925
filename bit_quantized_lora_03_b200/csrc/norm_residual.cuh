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
//   dw_pre = sum_t dn.xh, dw_post = sum_t scale.gate.g.yh, dgate = sum over its rows scale.g.yh.w_post
// The second norm's sum over g is formed from S2 and S3 so that a row needs one block reduction,
// not two in a row. Token sums: every CTA (or warp) takes one contiguous run of rows, keeps its
// columns' sums in registers, writes them once as partial rows, and norm_residual_finish_kernel
// adds the partials in a fixed order (no atomics: results repeat bit for bit).
#pragma once

#include "qlora_common.cuh"

namespace qlora {

namespace nr {
constexpr int kMaxH = 16384;
constexpr int kWarpRowH = 512;   // rows up to this long belong to one warp
constexpr int kWarpRowThreads = 256;
constexpr int kFinishCols = 128; // columns per block of the finish kernel
constexpr int kFinishWarps = 8;
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

template <int VPT, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? nr::kWarpRowThreads : 1024)
    norm_residual_fwd_kernel(const NormFwdArgs a) {
  __shared__ float red[2 * 32];
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int row = kWarpRow ? blockIdx.x * (nr::kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.t) return;   // whole warps (short rows) or whole CTAs
  const int nvec = a.h >> 3;
  const int64_t base = static_cast<int64_t>(row) * nvec;
  int turn = 0;
  uint4 xq[VPT], yq[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    xq[i] = yq[i] = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) {
      if (a.y) yq[i] = ldg_stream(a.y, base + v);
      xq[i] = ldg_stream(a.x, base + v);
    }
  }
  float ry = 1.f;
  if (a.w_post) {
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float y[8];
      unpack8(yq[i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] = fmaf(y[e], y[e], s[0]);
    }
    row_sum<1, kWarpRow>(s, red, turn);
    ry = 1.f / sqrtf(s[0] / static_cast<float>(a.h) + a.eps);
    if (tid == 0 && a.rstd_post) a.rstd_post[row] = ry;
  }
  const uint16_t* gate = a.gate ? a.gate + static_cast<int64_t>(row / a.rows_per_gate) * a.h : nullptr;
  float x[VPT][8];
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    unpack8(xq[i], x[i]);
    if (v >= nvec) continue;
    if (a.y) {
      float u[8];
      unpack8(yq[i], u);
      if (a.w_post) {
        float w[8];
        unpack8(ldg_vec(a.w_post, v), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = u[e] * ry * w[e];
      }
      if (gate) {
        float g[8];
        unpack8(ldg_vec(gate, v), g);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = fmaf(a.scale, u[e], x[i][e]);
    }
    if (a.x_out) reinterpret_cast<uint4*>(a.x_out)[base + v] = pack8(x[i]);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(x[i][e], x[i][e], s[0]);
  }
  if (!a.w_pre) return;
  row_sum<1, kWarpRow>(s, red, turn);
  const float rx = 1.f / sqrtf(s[0] / static_cast<float>(a.h) + a.eps);
  if (tid == 0 && a.rstd_pre) a.rstd_pre[row] = rx;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * nthr + tid;
    if (v >= nvec) continue;
    float w[8];
    unpack8(ldg_vec(a.w_pre, v), w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * rx * w[e];
    reinterpret_cast<uint4*>(a.n_out)[base + v] = pack8(x[i]);
  }
}

// The first row of unit u when t rows go to `units` contiguous runs.
__device__ __forceinline__ int unit_row(int t, int units, int u) {
  const int base = t / units, extra = t - base * units;
  return u * base + min(u, extra);
}

__device__ __forceinline__ void store8f(float* p, int64_t vec, const float (&f)[8]) {
  float4* q = reinterpret_cast<float4*>(p) + 2 * vec;
  q[0] = make_float4(f[0], f[1], f[2], f[3]);
  q[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// A thread's column sums (w_post, gate, w_pre): in registers, or for rows too long for that
// (VPT > 1) in shared memory at [sum][half][vector] as float4, each word of one thread only.
template <int VPT, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? nr::kWarpRowThreads : 1024)
    norm_residual_bwd_kernel(const NormBwdArgs a) {
  constexpr bool kSmem = !kWarpRow && VPT > 1;
  extern __shared__ __align__(16) float4 sacc[];
  __shared__ float red[2 * 3 * 32];
  const int nthr = kWarpRow ? 32 : blockDim.x;
  const int tid = kWarpRow ? (threadIdx.x & 31) : threadIdx.x;
  const int unit = kWarpRow ? blockIdx.x * (nr::kWarpRowThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
  const int nvec = a.h >> 3;
  // (a CTA's last warps may have no rows: unit >= units, r0 == r1 == t)
  const int r0 = min(a.t, unit_row(a.t, a.units, unit)), r1 = min(a.t, unit_row(a.t, a.units, unit + 1));
  const float inv_h = 1.f / static_cast<float>(a.h);
  int turn = 0;
  float acc[kSmem ? 1 : VPT][3][8];
  auto clear = [&](int k) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (kSmem) {
        const int v = i * nthr + tid;
        if (v < nvec) {
          sacc[(2 * k) * nvec + v] = make_float4(0.f, 0.f, 0.f, 0.f);
          sacc[(2 * k + 1) * nvec + v] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[i][k][e] = 0.f;
      }
    }
  };
  auto add = [&](int k, int i, int v, const float (&f)[8]) {
    if (kSmem) {
      float4 lo = sacc[(2 * k) * nvec + v], hi = sacc[(2 * k + 1) * nvec + v];
      lo.x += f[0]; lo.y += f[1]; lo.z += f[2]; lo.w += f[3];
      hi.x += f[4]; hi.y += f[5]; hi.z += f[6]; hi.w += f[7];
      sacc[(2 * k) * nvec + v] = lo;
      sacc[(2 * k + 1) * nvec + v] = hi;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[i][k][e] += f[e];
    }
  };
  auto write = [&](int k, float* dst) {   // this thread's columns of sum k -> a row of h floats
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (v >= nvec) continue;
      if (kSmem) {
        float4* q = reinterpret_cast<float4*>(dst) + 2 * v;
        q[0] = sacc[(2 * k) * nvec + v];
        q[1] = sacc[(2 * k + 1) * nvec + v];
      } else {
        store8f(dst, v, acc[i][k]);
      }
    }
  };
  clear(0);
  clear(1);
  clear(2);
  for (int row = r0; row < r1; ++row) {
    const int64_t base = static_cast<int64_t>(row) * nvec;
    const int grow = row / a.rows_per_gate;
    const uint16_t* gate = a.gate ? a.gate + static_cast<int64_t>(grow) * a.h : nullptr;
    const float rx = a.dn ? __ldg(a.rstd_pre + row) : 0.f;
    const float ry = a.w_post ? __ldg(a.rstd_post + row) : 1.f;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    uint4 dq[VPT], nq[VPT], xq[VPT], yq[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      dq[i] = nq[i] = xq[i] = yq[i] = zero;
      if (v < nvec) {
        if (a.dx_out) dq[i] = ldg_stream(a.dx_out, base + v);
        if (a.dn) {
          nq[i] = ldg_stream(a.dn, base + v);
          xq[i] = ldg_stream(a.x_out, base + v);
        }
        if (a.y) yq[i] = ldg_stream(a.y, base + v);
      }
    }
    float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (v >= nvec || !a.dn) continue;
      float dn[8], x[8], w[8], p[8];
      unpack8(nq[i], dn);
      unpack8(xq[i], x);
      unpack8(ldg_vec(a.w_pre, v), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= rx;
        p[e] = dn[e] * x[e];
        s[0] = fmaf(p[e], w[e], s[0]);
      }
      add(2, i, v, p);
      if (a.w_post) {
        float y[8], d[8], wo[8];
        unpack8(yq[i], y);
        unpack8(dq[i], d);
        unpack8(ldg_vec(a.w_post, v), wo);
        if (gate) {
          float g[8];
          unpack8(ldg_vec(gate, v), g);
#pragma unroll
          for (int e = 0; e < 8; ++e) wo[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float k = wo[e] * y[e];   // scale and ry are common to the row: applied below
          s[1] = fmaf(k, fmaf(rx * dn[e], w[e], d[e]), s[1]);
          s[2] = fmaf(k, x[e], s[2]);
        }
      }
    }
    if (!a.dn && a.w_post) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = i * nthr + tid;
        if (v >= nvec) continue;
        float y[8], d[8], wo[8];
        unpack8(yq[i], y);
        unpack8(dq[i], d);
        unpack8(ldg_vec(a.w_post, v), wo);
        if (gate) {
          float g[8];
          unpack8(ldg_vec(gate, v), g);
#pragma unroll
          for (int e = 0; e < 8; ++e) wo[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[1] = fmaf(wo[e] * y[e], d[e], s[1]);
      }
    }
    row_sum<3, kWarpRow>(s, red, turn);
    const float c1 = rx * s[0] * inv_h;
    const float c2 = a.scale * ry * (s[1] - c1 * s[2]) * inv_h;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * nthr + tid;
      if (v >= nvec) continue;
      float g[8];
      unpack8(dq[i], g);
      if (a.dn) {
        float dn[8], x[8], w[8];
        unpack8(nq[i], dn);
        unpack8(xq[i], x);
        unpack8(ldg_vec(a.w_pre, v), w);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = fmaf(rx * dn[e], w[e], g[e]) - c1 * (x[e] * rx);
      }
      reinterpret_cast<uint4*>(a.dx)[base + v] = pack8(g);
      if (!a.y) continue;
      float y[8], wo[8], p[8];
      unpack8(yq[i], y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] *= ry;
        g[e] *= a.scale;
        wo[e] = 1.f;
      }
      if (a.w_post) unpack8(ldg_vec(a.w_post, v), wo);
      if (gate) {
        float gt[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = g[e] * y[e] * wo[e];
        add(1, i, v, p);
        unpack8(ldg_vec(gate, v), gt);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] *= gt[e];
      }
      if (a.w_post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = g[e] * y[e];
          g[e] = ry * fmaf(-c2, y[e], g[e] * wo[e]);
        }
        add(0, i, v, p);
      }
      reinterpret_cast<uint4*>(a.dy)[base + v] = pack8(g);
    }
    // the gate row's sum ends with its last token: written as the result where this unit had
    // all of its rows, else as this unit's share of it
    if (gate && (row + 1 == r1 || (row + 1) % a.rows_per_gate == 0)) {
      const int64_t g0 = static_cast<int64_t>(grow) * a.rows_per_gate;
      const int64_t g1 = min(g0 + a.rows_per_gate, static_cast<int64_t>(a.t));
      if (g0 >= r0 && g1 <= r1)
        write(1, a.dgate + static_cast<int64_t>(grow) * a.h);
      else
        write(1, a.part_gate + (static_cast<int64_t>(g0 < r0 ? 0 : a.units) + unit) * a.h);
      clear(1);
    }
  }
  if (!kWarpRow) {
    if (a.w_post) write(0, a.part_post + static_cast<int64_t>(unit) * a.h);
    if (a.dn) write(2, a.part_pre + static_cast<int64_t>(unit) * a.h);
    return;
  }
  // short rows: the warps' sums are added here, one partial row per CTA
  float* sf = reinterpret_cast<float*>(sacc);
#pragma unroll
  for (int k = 0; k < 3; k += 2) {
    float* part = k == 0 ? (a.w_post ? a.part_post : nullptr) : (a.dn ? a.part_pre : nullptr);
    if (!part) continue;
    write(k, sf + (threadIdx.x >> 5) * a.h);
    __syncthreads();
    for (int c = threadIdx.x; c < a.h; c += nr::kWarpRowThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < nr::kWarpRowThreads / 32; ++w) v += sf[w * a.h + c];
      part[static_cast<int64_t>(blockIdx.x) * a.h + c] = v;
    }
    __syncthreads();
  }
}

// Adds the partial rows in order. grid y: 0 dw_pre, 1 dw_post, 2.. the gate rows whose tokens fell
// to more than one unit. A block takes 128 columns; its eight warps take every eighth partial row
// and are added in shared memory.
__global__ void __launch_bounds__(nr::kFinishWarps * 32)
    norm_residual_finish_kernel(const float* part_pre, const float* part_post, const float* part_gate,
                                float* dw_pre, float* dw_post, float* dgate, int t, int h,
                                int rows_per_gate, int parts, int units) {
  __shared__ float4 sh[nr::kFinishWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * nr::kFinishCols + lane * 4;
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
  // unit b > 0 opening inside a gate row that unit b - 1 opened: the row's shares are unit
  // b - 1's closing one (row units + b - 1) and the opening ones of units b .. e - 1
  const int used = min(units, t);   // the units behind have no rows
  for (int b = blockIdx.y - 1; b < used; b += gridDim.y - 2) {
    const int r = unit_row(t, units, b);
    const int64_t g = r / rows_per_gate, g0 = g * rows_per_gate;
    const int64_t g1 = min(g0 + rows_per_gate, static_cast<int64_t>(t));
    if (g0 == r || unit_row(t, units, b - 1) > g0) continue;
    int e = b + 1;   // the first unit that starts behind the row's tokens
    if (g1 == t) {
      e = used;
    } else {
      while (e < used && unit_row(t, units, e) < g1) ++e;
    }
    sum_rows(part_gate + static_cast<int64_t>(b) * h, e - b,
             part_gate + static_cast<int64_t>(units + b - 1) * h, dgate + g * h);
  }
}

}  // namespace qlora
