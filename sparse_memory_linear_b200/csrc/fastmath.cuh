// fastmath.cuh -- short forms of the arithmetic that the dense-state layer's kernels do per value.
#pragma once

#include "common.cuh"

namespace sdm {

// 2^x by the hardware (relative error about 2^-22, results below 2^-126 are 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)),
        "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return fma2(b, make_float2(-1.0f, -1.0f), a);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// act(g) for values that were or will be bf16, from one exponential and one reciprocal of the
// hardware, against tens of instructions for expf and a division.  The error relative to act(g) is
// about 2^-21 (1 + |g| / 4) for g > -87, far below half a step of bf16, 2^-8; below that the
// result, at most 2e-36, is 0.
// The activation is chosen once for all of a thread's pairs: chosen value by value it cost as
// much again.
__device__ __forceinline__ float2 fast_sigmoid2(float2 g) {
  const float2 t = mul2(g, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  const float2 d = add2(make_float2(fast_exp2(t.x), fast_exp2(t.y)), make_float2(1.0f, 1.0f));
  float2 r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(d.y));
  return r;
}
// For fp32 values: good to 9 half steps (expf 2 ulp, the reciprocal of a number in 1 .. 2 1 ulp),
// and to the last denormal.  20011 x 2568 fp32 convolutions take 78.3 us, 79.5 with the short form.
__device__ __forceinline__ float act_f32(float g, bool silu) {
  const float e = expf(-fabsf(g));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  const float top = g < 0.0f ? e : 1.0f;
  return (silu ? g * top : top) * r;
}
template <typename T, int PAIRS>
__device__ __forceinline__ void pair_act(float2 g[PAIRS], int act) {
  if (act == SDM_GATE_IDENTITY) return;
  const bool silu = act == SDM_GATE_SILU;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    if constexpr (sizeof(T) == 2) {
      const float2 s = fast_sigmoid2(g[i]);
      g[i] = mul2(s, make_float2(silu ? g[i].x : 1.0f, silu ? g[i].y : 1.0f));
    } else {
      g[i] = make_float2(act_f32(g[i].x, silu), act_f32(g[i].y, silu));
    }
  }
}

}  // namespace sdm
