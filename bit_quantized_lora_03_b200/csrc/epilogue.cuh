// The epilogue of the QLoRA linear, Z = X.W' + s.X.L1.L2 + b, Y = act(Z) + R, and its backward.
//
// Forward: the GEMM (nf4_gemm.cuh) and the decode GEMV (nf4_gemv.cuh) apply it to their fp32
// accumulators, so that Z, b and R meet in fp32 and Y is rounded once; this header holds the
// activations. Backward (epilogue_bwd_kernel): dZ = dY . act'(Z), db = sum_t dZ, from the saved
// bf16 Z; dR = dY needs no work. dZ then takes dY's place in qlora_linear_bwd.
//
// Activations: relu; gelu, z.Phi(z); gelu_tanh, z.(1 + tanh u)/2 with u = sqrt(2/pi).(z +
// 0.044715 z^3), computed as z.sigmoid(2u); silu, z.sigmoid(z). sigmoid(v) = 1 / (1 + exp(-v))
// with the exp2 and reciprocal instructions: their relative error of a few 2^-23 is far below the bf16
// rounding of Y and dZ and keeps db at fp32 accuracy (the tanh instruction, at 2^-11, would not).
// Phi(z) = 1 - q/2 (z >= 0) or q/2, q = erfc(|z|/sqrt 2) by Abramowitz and Stegun 7.1.26, a polynomial
// of fifth degree in 1/(1 + 0.3275911 |z|/sqrt 2) times exp(-z^2/2), off by at most 1.5e-7: one
// exponential and one division, and the same exponential serves gelu's derivative (erff took 1.8
// times the time of silu in the GEMM's epilogue, this 1.1). Relative to gelu's own negative tail that is
// 5e-5 at -3, 1.6e-3 at -5 and 3.6e-3 at -6, half a step of bf16; gelu is below 6e-9 behind that.
#pragma once

#include "norm_residual.cuh"

namespace qlora {

enum ActKind : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sigmoid_fast(float v) {
  return rcp(1.f + ex2(-1.44269504f * v));   // exp(-v) may overflow: 1 / inf is 0
}

// Phi(z), and e = exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf_fast(float z, float& e) {
  const float x = fabsf(z);
  const float t = rcp(fmaf(0.3275911f * 0.70710678f, x, 1.f));
  e = ex2(-0.72134752f * z * z);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * q * t * e;
  return z >= 0.f ? 1.f - q : q;
}

template <int kAct>
__device__ __forceinline__ float act_fwd(float z) {
  if (kAct == kActRelu) return z < 0.f ? 0.f : z;   // a NaN stays one
  if (kAct == kActGelu) {
    float e;
    return z * normal_cdf_fast(z, e);
  }
  if (kAct == kActGeluTanh) return z * sigmoid_fast(1.5957691f * z * fmaf(0.044715f * z, z, 1.f));
  if (kAct == kActSilu) return z * sigmoid_fast(z);
  return z;
}

template <int kAct>
__device__ __forceinline__ float act_bwd(float z) {   // act'(z)
  if (kAct == kActRelu) return z > 0.f ? 1.f : (z <= 0.f ? 0.f : z);
  if (kAct == kActGelu) {
    float e;
    const float c = normal_cdf_fast(z, e);
    return fmaf(z * 0.39894228f, e, c);
  }
  if (kAct == kActGeluTanh) {
    z = z > 30.f ? 30.f : (z < -30.f ? -30.f : z);   // act' is 1 and 0 there; z^2 must not overflow
    const float sg = sigmoid_fast(1.5957691f * z * fmaf(0.044715f * z, z, 1.f));
    return fmaf(z * sg * (1.f - sg) * 1.5957691f, fmaf(0.134145f * z, z, 1.f), sg);
  }
  if (kAct == kActSilu) {
    const float sg = sigmoid_fast(z);
    return fmaf(z * sg, 1.f - sg, sg);
  }
  return 1.f;
}

// act over N values, the branch taken once (the kind is the same for the whole launch).
template <int N>
__device__ __forceinline__ void act_apply(float (&z)[N], int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = act_fwd<kActRelu>(z[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = act_fwd<kActGelu>(z[i]);
      break;
    case kActGeluTanh:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = act_fwd<kActGeluTanh>(z[i]);
      break;
    case kActSilu:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = act_fwd<kActSilu>(z[i]);
      break;
    default: break;
  }
}

// What the linear's epilogue adds to its product (all but act optional).
struct EpilogueArgs {
  const uint16_t* bias;      // o bf16
  const uint16_t* residual;  // t x o bf16
  uint16_t* z_out;           // t x o bf16: Z, before the activation
  int act;
};

namespace ep {
constexpr int kWarps = 8;
constexpr int kCols = 256;    // columns per CTA: 32 lanes x 8
constexpr int kUnroll = 2;    // rows in flight per warp (4 take registers from warps: 53 against 47 us)
}  // namespace ep

struct EpilogueBwdArgs {
  const uint16_t* dY;
  const uint16_t* Z;       // or NULL (no activation)
  uint16_t* dZ;            // or NULL (the bias gradient alone)
  float* part;             // column sums, gridDim.y x o (gridDim.y == 1: db itself), or NULL
  int64_t t;
  int o;
};

// HBM-bound: dY and Z are read and dZ is written once, in 512-byte warp rows; a warp keeps two
// rows in flight. A CTA takes 256 columns of one run of rows and keeps their sums in registers;
// its eight warps add theirs in shared memory, and the runs' partial rows are added in order by
// norm_residual_finish_kernel (no atomics). The sums take the unrounded dZ.
template <int kAct>
__global__ void __launch_bounds__(ep::kWarps * 32)
    epilogue_bwd_kernel(const EpilogueBwdArgs a) {
  using namespace ep;
  __shared__ float sh[kWarps][kCols];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nvec = a.o >> 3;
  const int v = blockIdx.x * (kCols / 8) + lane;
  const bool cv = v < nvec;
  const int r0 = unit_row(static_cast<int>(a.t), gridDim.y, blockIdx.y);
  const int r1 = unit_row(static_cast<int>(a.t), gridDim.y, blockIdx.y + 1);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (cv) {
    for (int64_t r = r0 + warp; r < r1; r += kUnroll * kWarps) {
      uint4 dq[kUnroll], zq[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int64_t at = (r + u * kWarps) * nvec + v;
        if (r + u * kWarps < r1) {
          dq[u] = ldg_stream(a.dY, at);
          if (kAct != kActNone) zq[u] = ldg_stream(a.Z, at);
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (r + u * kWarps >= r1) break;
        float d[8], z[8];
        unpack8(dq[u], d);
        if (kAct != kActNone) {
          unpack8(zq[u], z);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[e] *= act_bwd<kAct>(z[e]);
        }
        if (a.dZ) reinterpret_cast<uint4*>(a.dZ)[(r + u * kWarps) * nvec + v] = pack8(d);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], d[e]);   // no fusion with the product: db does
                                                                        // not depend on whether dZ is stored
      }
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sh[warp][e * 32 + lane] = acc[e];   // column 8 lane + e
  __syncthreads();
  const int e = threadIdx.x & 7, l = threadIdx.x >> 3;   // thread c sums column c = 8 l + e
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += sh[w][e * 32 + l];
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kCols + threadIdx.x;
  if (col < a.o) a.part[static_cast<int64_t>(blockIdx.y) * a.o + col] = s;
}

}  // namespace qlora
