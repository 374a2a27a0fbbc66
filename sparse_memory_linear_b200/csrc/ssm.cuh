// ssm.cuh -- selective state-space scan, the dense counterpart of the sparse memory pass: every
// head keeps a state of N rows of d_v values that every token decays, writes and reads whole.
//
// Token t of a sequence, head h (group g = h / (H / G) of the H / G heads that share k and q):
//   d = softplus(dt[t, h] + dt_bias[h])        (or dt itself)
//   M = exp(d A[h]) M + d k[t, g] (x) v[t, h]
//   y[t, h] = (q[t, g]^T M + D[h] v[t, h]) * act(gate[t, h])
// This file: the step for one token, and the token-by-token scan that serves every shape.
#pragma once

#include "common.cuh"
#include "conv.cuh"

namespace sdm {

struct SsmArgs {
  const void *k, *q, *v, *dt, *gate;
  const float *A, *dt_bias, *D;
  float* M;
  void* y;
  SeqBounds seq;
  int H, G, N, P;
  int from_zero, softplus, act;
  long long k_stride, q_stride, v_stride, dt_stride, gate_stride;  // elements between tokens
};

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// The token's step size: softplus as max(x, 0) + log1p(exp(-|x|)), which neither overflows nor
// loses small results; without it, dt itself with negative values taken as 0.
__device__ __forceinline__ float ssm_step_size(float dt, int softplus) {
  if (softplus) return fmaxf(dt, 0.0f) + log1pf(expf(-fabsf(dt)));
  return dt < 0.0f ? 0.0f : dt;
}

// Token-by-token scan.  A block holds 16 of a head's d_v columns: four per warp, eight lanes to
// a column, each lane with the state rows 32 j + 4 l .. + 3 in registers.  Tokens come through
// shared memory 16 at a time.  The chain from token to token is one multiply-add per state
// value; the sum over the rows ends in three shuffles.
constexpr int SSM_TB = 16;    // tokens staged at a time
constexpr int SSM_COLS = 16;  // columns of a block

template <typename T, int NJ>
__global__ void __launch_bounds__(128) ssm_scan_kernel(SsmArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int NP = 32 * NJ;
  __shared__ __align__(16) float sk[SSM_TB][NP];
  __shared__ __align__(16) float sq[SSM_TB][NP];
  __shared__ float sv[SSM_TB][SSM_COLS], sy[SSM_TB][SSM_COLS];
  __shared__ float sd[SSM_TB], sa[SSM_TB];
  const int tid = threadIdx.x, lane = tid & 31, ln = lane & 7;
  const int col = (tid >> 5) * 4 + (lane >> 3);
  const int h = blockIdx.y, g = h / (a.H / a.G);
  const int p0 = blockIdx.z * SSM_COLS, p = p0 + col;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) a.seq.check();
  const T* kp = static_cast<const T*>(a.k) + (size_t)g * a.N;
  const T* qp = static_cast<const T*>(a.q) + (size_t)g * a.N;
  const T* vp = static_cast<const T*>(a.v) + (size_t)h * a.P + p0;
  const T* zp = a.gate ? static_cast<const T*>(a.gate) + (size_t)h * a.P + p0 : nullptr;
  const T* dp = static_cast<const T*>(a.dt) + h;
  T* yp = static_cast<T*>(a.y) + (size_t)h * a.P + p0;
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.0f, D = a.D ? a.D[h] : 0.0f;
  for (int b = blockIdx.x; b < a.seq.B; b += gridDim.x) {
    const long long s0 = a.seq.start(b), e0 = a.seq.end(b);
    float* Mp = a.M + ((size_t)b * a.H + h) * a.N * a.P;
    float s[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * j + 4 * ln + i;
        s[j][i] = !a.from_zero && n < a.N && p < a.P ? Mp[(size_t)n * a.P + p] : 0.0f;
      }
    for (long long t0 = s0; t0 < e0; t0 += SSM_TB) {
      const int nt = e0 - t0 < SSM_TB ? (int)(e0 - t0) : SSM_TB;
      __syncthreads();
      for (int i = tid; i < nt * NP; i += 128) {
        const int t = i / NP, n = i % NP;
        const bool in = n < a.N;
        sk[t][n] = in ? to_f32(kp[(t0 + t) * a.k_stride + n]) : 0.0f;
        sq[t][n] = in ? to_f32(qp[(t0 + t) * a.q_stride + n]) : 0.0f;
      }
      for (int i = tid; i < nt * SSM_COLS; i += 128) {
        const int t = i / SSM_COLS, c = i % SSM_COLS;
        sv[t][c] = p0 + c < a.P ? to_f32(vp[(t0 + t) * a.v_stride + c]) : 0.0f;
      }
      if (tid < nt) {
        const float d = ssm_step_size(to_f32(dp[(t0 + tid) * a.dt_stride]) + bias, a.softplus);
        sd[tid] = d;
        sa[tid] = expf(d * A);
      }
      __syncthreads();
#pragma unroll 2
      for (int t = 0; t < nt; ++t) {
        const float al = sa[t], dv = sd[t] * sv[t][col];
        float acc = 0.0f;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float4 k4 = *reinterpret_cast<const float4*>(&sk[t][32 * j + 4 * ln]);
          const float4 q4 = *reinterpret_cast<const float4*>(&sq[t][32 * j + 4 * ln]);
          s[j][0] = fmaf(s[j][0], al, dv * k4.x);
          s[j][1] = fmaf(s[j][1], al, dv * k4.y);
          s[j][2] = fmaf(s[j][2], al, dv * k4.z);
          s[j][3] = fmaf(s[j][3], al, dv * k4.w);
          acc = fmaf(q4.x, s[j][0], acc);
          acc = fmaf(q4.y, s[j][1], acc);
          acc = fmaf(q4.z, s[j][2], acc);
          acc = fmaf(q4.w, s[j][3], acc);
        }
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) acc += __shfl_xor_sync(FULL_MASK, acc, m);
        if (ln == 0) sy[t][col] = acc;
      }
      __syncthreads();
      for (int i = tid; i < nt * SSM_COLS; i += 128) {
        const int t = i / SSM_COLS, c = i % SSM_COLS;
        if (p0 + c >= a.P) continue;
        float y = sy[t][c];
        if (a.D) y = fmaf(D, sv[t][c], y);
        if (zp) y *= gate_act(to_f32(zp[(t0 + t) * a.gate_stride + c]), a.act);
        yp[(size_t)(t0 + t) * a.H * a.P + c] = from_f32<T>(y);
      }
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 32 * j + 4 * ln + i;
        if (n < a.N && p < a.P) Mp[(size_t)n * a.P + p] = s[j][i];
      }
  }
}

// One token.  A block per (sequence, head): the state's N x P values as float4 columns, row
// groups side by side, each thread walking its rows; the row groups' shares of the read meet in
// shared memory.
template <typename T>
__global__ void __launch_bounds__(256) ssm_step_kernel(SsmArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ __align__(16) float part[256 * 4];
  const int h = blockIdx.x % a.H, b = blockIdx.x / a.H, g = h / (a.H / a.G);
  const int cols = a.P / 4, groups = 256 / cols;
  const int c = threadIdx.x % cols, grp = threadIdx.x / cols;
  const T* kp = static_cast<const T*>(a.k) + b * a.k_stride + (size_t)g * a.N;
  const T* qp = static_cast<const T*>(a.q) + b * a.q_stride + (size_t)g * a.N;
  const T* vp = static_cast<const T*>(a.v) + b * a.v_stride + (size_t)h * a.P;
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  const float d = ssm_step_size(
      to_f32(static_cast<const T*>(a.dt)[b * a.dt_stride + h]) + bias, a.softplus);
  const float al = expf(d * a.A[h]);
  float4* Mp = reinterpret_cast<float4*>(a.M + ((size_t)b * a.H + h) * a.N * a.P);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (grp < groups) {
    float dv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) dv[i] = d * to_f32(vp[4 * c + i]);
#pragma unroll 8
    for (int n = grp; n < a.N; n += groups) {
      float4 m = Mp[(size_t)n * cols + c];
      const float kn = to_f32(kp[n]), qn = to_f32(qp[n]);
      m.x = fmaf(m.x, al, dv[0] * kn);
      m.y = fmaf(m.y, al, dv[1] * kn);
      m.z = fmaf(m.z, al, dv[2] * kn);
      m.w = fmaf(m.w, al, dv[3] * kn);
      acc.x = fmaf(qn, m.x, acc.x);
      acc.y = fmaf(qn, m.y, acc.y);
      acc.z = fmaf(qn, m.z, acc.z);
      acc.w = fmaf(qn, m.w, acc.w);
      Mp[(size_t)n * cols + c] = m;
    }
    *reinterpret_cast<float4*>(&part[(grp * cols + c) * 4]) = acc;
  }
  __syncthreads();
  for (int p = threadIdx.x; p < a.P; p += 256) {
    float y = 0.0f;
    for (int i = 0; i < groups; ++i) y += part[i * a.P + p];
    if (a.D) y = fmaf(a.D[h], to_f32(vp[p]), y);
    if (a.gate)
      y *= gate_act(to_f32(static_cast<const T*>(a.gate)[b * a.gate_stride + (size_t)h * a.P + p]),
                    a.act);
    static_cast<T*>(a.y)[((size_t)b * a.H + h) * a.P + p] = from_f32<T>(y);
  }
}

}  // namespace sdm
