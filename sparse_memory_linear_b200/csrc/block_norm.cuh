// block_norm.cuh -- the norms after and before a block of a residual stack, fused with the
// block's gate, its residual scale and the residual sum.
//
//   f = u * rsqrt(mean(u^2) + eps) * post_gamma      (post norm; f = u without it)
//   f = f * act(gate) * scale                        (each factor only where given)
//   r' = r + f
//   n = r' * rsqrt(mean(r'^2) + eps) * pre_gamma     (the next block's input)
// Both means and the sum are fp32; n is computed from the unrounded r'.
//
// Bound by its bytes: 32768 rows of 2048, bf16 with a gate and an fp32 residual (14 bytes a value),
// take 161 us, 5.84 TB/s, 0.89 of the measured copy rate.  A first version that read the
// parameters for every row and waited for each row's values took 206 us.
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

// Sum over the TPR threads of a row (TPR a multiple of 32; rows of a block side by side).  `part`
// is written once per call: calls that may overlap need a part of their own.
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

// Eight values of a parameter, 1 where there is none.
__device__ __forceinline__ void load_param(const float* p, int v, float2 g[4]) {
  if (p) {
    Vec8<float> t;
    t.load(p + 8 * v);
    t.get2(g);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = make_float2(1.0f, 1.0f);
  }
}

// TPR threads per row, each with up to NV groups of eight values in registers; 256 threads (or
// TPR, if more) to a block, blocks stride over the rows.  With one group a thread (rows of up to
// 4096 values) the parameters stay in registers, 12 of the 26 bytes a value that would cross
// the L1 otherwise, and the next row is on its way while this one is summed.  The sums keep two
// sets of partial sums, so that two barriers a row are enough.
template <typename T, typename TR, int TPR, int NV>
__global__ void __launch_bounds__(TPR > 256 ? TPR : 256, NV == 1 ? (TPR > 256 ? 1 : 2) : 1)
    block_norm_kernel(BlockNormArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  constexpr int THREADS = TPR > 256 ? TPR : 256;
  constexpr int RPB = THREADS / TPR;
  constexpr bool KEEP = NV == 1;
  __shared__ float part[2][2][THREADS / 32];
  const int lane = threadIdx.x % TPR;
  const int nvec = a.D / 8;
  const float inv_d = 1.0f / (float)a.D;
  float2 gpost[4], gscale[4], gpre[4];
  if (KEEP && lane < nvec) {
    load_param(a.post ? a.post_gamma : nullptr, lane, gpost);
    load_param(a.scale, lane, gscale);
    load_param(a.pre_gamma, lane, gpre);
  }
  struct Row {  // as stored: a third of the registers that the values take
    Vec8<T> u[NV], z[NV];
    Vec8<TR> r[NV];
  };
  Row next;
  auto fetch = [&](long long row, Row& o) {
    if (row >= a.rows) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * TPR;
      if (v >= nvec) continue;
      const size_t at = (size_t)row * a.D + 8 * v;
      o.u[i].load(static_cast<const T*>(a.u) + at);
      o.r[i].load(static_cast<const TR*>(a.r) + at);
      if (a.gate) o.z[i].load(static_cast<const T*>(a.gate) + at);
    }
  };
  const long long step = (long long)gridDim.x * RPB;
  if (KEEP) fetch((long long)blockIdx.x * RPB + threadIdx.x / TPR, next);
  int turn = 0;
  for (long long row0 = (long long)blockIdx.x * RPB; row0 < a.rows; row0 += step, turn ^= 1) {
    const long long row = row0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const size_t base = (size_t)row * a.D;
    Row cur;
    if (KEEP) {
      cur = next;
      fetch(row + step, next);
    } else {
      fetch(row, cur);
    }
    float2 r[NV][4];
    float ss = 0.0f;
    if (a.post) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!on || lane + i * TPR >= nvec) continue;
        float2 f[4];
        cur.u[i].get2(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ss = fmaf(f[e].x, f[e].x, ss);
          ss = fmaf(f[e].y, f[e].y, ss);
        }
      }
    }
    float inv = 1.0f;
    if (a.post) inv = rsqrtf(row_sum<TPR>(ss, part[turn][0]) * inv_d + a.eps);
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = lane + i * TPR;
      if (!on || v >= nvec) continue;
      if (!KEEP) {
        load_param(a.post ? a.post_gamma : nullptr, v, gpost);
        load_param(a.scale, v, gscale);
      }
      float2 f[4], z[4];
      cur.u[i].get2(f);
      cur.r[i].get2(r[i]);
      if (a.gate) {
        cur.z[i].get2(z);
        pair_act<T, 4>(z, a.act);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 t = mul2(mul2(f[e], make_float2(inv, inv)), gpost[e]);
        if (a.gate) t = mul2(t, z[e]);
        r[i][e] = fma2(t, gscale[e], r[i][e]);
        ss = fmaf(r[i][e].x, r[i][e].x, ss);
        ss = fmaf(r[i][e].y, r[i][e].y, ss);
      }
      Vec8<TR> tr;
      tr.set2(r[i]);
      tr.store(static_cast<TR*>(a.r_out) + base + 8 * v);
    }
    if (a.n) {
      inv = rsqrtf(row_sum<TPR>(ss, part[turn][1]) * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = lane + i * TPR;
        if (!on || v >= nvec) continue;
        if (!KEEP) load_param(a.pre_gamma, v, gpre);
        float2 o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = mul2(mul2(r[i][e], make_float2(inv, inv)), gpre[e]);
        Vec8<T> t;
        t.set2(o);
        t.store(static_cast<T*>(a.n) + base + 8 * v);
      }
    }
  }
}

}  // namespace sdm
