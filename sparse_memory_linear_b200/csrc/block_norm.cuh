// block_norm.cuh -- the norms after and before a block of a residual stack, fused with the
// block's gate, its residual scale and the residual sum.
//
//   f = u * rsqrt(mean(u^2) + eps) * post_gamma      (post norm; f = u without it)
//   f = f * act(gate) * scale                        (each factor only where given)
//   r' = r + f
//   n = r' * rsqrt(mean(r'^2) + eps) * pre_gamma     (the next block's input)
// Both means and the sum are fp32; n is computed from the unrounded r'.
#pragma once

#include "common.cuh"
#include "conv.cuh"

namespace sdm {

struct BlockNormArgs {
  const void* u;
  const void* gate;
  const void* r;
  void* r_out;
  void* n;
  const float* post_gamma;
  const float* pre_gamma;
  const float* scale;
  long long rows;
  int D, act, post;
  float eps;
};

// Sum over the TPR threads of a row (TPR a multiple of 32; rows of a block side by side).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(FULL_MASK, v, s);
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    constexpr int WPR = TPR / 32;
    const int w0 = warp / WPR * WPR;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) v += part[w0 + i];
  }
  return v;
}

// TPR threads per row, each with up to NV groups of eight values in registers; 256 threads (or
// TPR, if more) to a block, blocks stride over the rows.
template <typename T, typename TR, int TPR, int NV>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256) block_norm_kernel(BlockNormArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int THREADS = TPR > 256 ? TPR : 256;
  constexpr int RPB = THREADS / TPR;
  __shared__ float part[2][THREADS / 32];
  const int lane = threadIdx.x % TPR;
  const int nvec = a.D / 8;
  for (long long row0 = (long long)blockIdx.x * RPB; row0 < a.rows;
       row0 += (long long)gridDim.x * RPB) {
    const long long row = row0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const size_t base = (size_t)row * a.D;
    float f[NV][8], r[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * TPR;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = r[i][e] = 0.0f;
      if (on && v < nvec) {
        Vec8<T> t;
        Vec8<TR> tr;
        t.load(static_cast<const T*>(a.u) + base + 8 * v);
        tr.load(static_cast<const TR*>(a.r) + base + 8 * v);
        t.get(f[i]);
        tr.get(r[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[i][e], f[i][e], ss);
      }
    }
    float inv = 1.0f;
    if (a.post) inv = rsqrtf(row_sum<TPR>(ss, part[0]) / (float)a.D + a.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * TPR;
      if (!on || v >= nvec) continue;
      if (a.post) {
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.0f;
        if (a.post_gamma) {
          Vec8<float> t;
          t.load(a.post_gamma + 8 * v);
          t.get(g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * inv * g[e];
      }
      if (a.gate) {
        Vec8<T> t;
        float g[8];
        t.load(static_cast<const T*>(a.gate) + base + 8 * v);
        t.get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] *= gate_act(g[e], a.act);
      }
      if (a.scale) {
        Vec8<float> t;
        float g[8];
        t.load(a.scale + 8 * v);
        t.get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] *= g[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[i][e] += f[i][e];
        ss = fmaf(r[i][e], r[i][e], ss);
      }
      Vec8<TR> tr;
      tr.set(r[i]);
      tr.store(static_cast<TR*>(a.r_out) + base + 8 * v);
    }
    if (a.n) {
      inv = rsqrtf(row_sum<TPR>(ss, part[1]) / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lane + i * TPR;
        if (!on || v >= nvec) continue;
        float g[8], o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.0f;
        if (a.pre_gamma) {
          Vec8<float> t;
          t.load(a.pre_gamma + 8 * v);
          t.get(g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = r[i][e] * inv * g[e];
        Vec8<T> t;
        t.set(o);
        t.store(static_cast<T*>(a.n) + base + 8 * v);
      }
    }
    if constexpr (TPR > 32) __syncthreads();  // part[] is free again
  }
}

}  // namespace sdm
