// conv.cuh -- causal short convolution over the channels of a recurrent layer (prompts and
// single tokens).
//
// y[t, c] = act(bias[c] + sum_j w[c, j] x[t - K + 1 + j, c]), j = 0..K-1, each channel on its
// own; inputs before a sequence's first token are the kept state (its last K - 1 inputs) or
// zero.
//
// Bound by its bytes, every input read and every output written once.  Measured on one B200:
// 4 x 8192 x 1280 bf16, K = 4, SiLU 36.0 us (4.66 TB/s, 0.71 of the measured copy rate; without
// the activation 33 us; a plain copy of x 28.8 us: a thread loads a group of rows and computes it in
// turn, with no load on its way meanwhile), 20011 x 2568 fp32 in 23 packed sequences 79 us
// (5.2 TB/s, 0.80).
#pragma once

#include "fastmath.cuh"

namespace sdm {

// Eight values of a 16-bit or 32-bit row: 16 or 32 bytes.
template <typename T>
struct Vec8;

template <>
struct Vec8<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void get2(float2 f[4]) const {
    f[0] = unpack_bf16(raw.x);
    f[1] = unpack_bf16(raw.y);
    f[2] = unpack_bf16(raw.z);
    f[3] = unpack_bf16(raw.w);
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    raw = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint4*>(p) = raw;
  }
  __device__ __forceinline__ void set2(const float2 f[4]) {
    raw = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                     pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
  }
};

template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void get2(float2 f[4]) const {
    f[0] = make_float2(a.x, a.y);
    f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y);
    f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void set2(const float2 f[4]) {
    a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};

// Row bounds of the sequences of a batch: B sequences of T rows each (cu == nullptr), or
// packed, sequence b holding rows cu[b] .. cu[b + 1] - 1 of R.  Offsets are clamped to [0, R]
// and an end below its start gives an empty sequence, so that no bad offset leaves the buffers.
struct SeqBounds {
  const int* cu;
  int B;
  long long T;  // uniform length (cu == nullptr)
  long long R;  // rows in all

  __device__ __forceinline__ long long start(int b) const {
    if (!cu) return (long long)b * T;
    const long long s = cu[b];
    return s < 0 ? 0 : s > R ? R : s;
  }
  __device__ __forceinline__ long long end(int b) const {
    if (!cu) return (long long)(b + 1) * T;
    const long long s = start(b), e = start(b + 1);
    return e < s ? s : e;
  }
  // The first sequence that starts at row r or later (B: none).
  __device__ __forceinline__ int first_from(long long r) const {
    if (!cu) {
      // 32-bit division where it serves: the 64-bit one costs as much as several rows
      const long long b = R < 0x7fffffffLL ? (long long)((unsigned)(r + T - 1) / (unsigned)T)
                                           : (r + T - 1) / T;
      return b > B ? B : (int)b;
    }
    int lo = 0, hi = B;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) < r) lo = mid + 1; else hi = mid;
    }
    return lo;
  }
  // Records offsets that are out of range or not ascending; called by one block.
  __device__ __forceinline__ void check() const {
    if (!cu) return;
    for (int b = threadIdx.x; b <= B; b += blockDim.x) {
      const int c = cu[b];
      if (c < 0 || c > R || (b > 0 && c < cu[b - 1])) record_status(STATUS_BAD_INDEX);
    }
  }
};

struct ConvArgs {
  const void* x;
  const float* w;
  const float* bias;
  void* state;  // [B, K - 1, C]; may be null when from_zero
  void* y;
  SeqBounds seq;
  int C, cv;  // channels, C / 4
  int from_zero, act, rows_per_thread;
  long long x_stride, tiles;
};

// Four values: 8 or 16 bytes.
template <typename T>
struct Vec4;

template <>
struct Vec4<__nv_bfloat16> {
  uint2 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    raw = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint2*>(p) = raw;
  }
  __device__ __forceinline__ void zero() { raw = make_uint2(0, 0); }
  __device__ __forceinline__ void get2(float2 f[2]) const {
    f[0] = unpack_bf16(raw.x);
    f[1] = unpack_bf16(raw.y);
  }
  __device__ __forceinline__ void set2(const float2 f[2]) {
    raw = make_uint2(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y));
  }
};

template <>
struct Vec4<float> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) {
    raw = *reinterpret_cast<const float4*>(p);
  }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get2(float2 f[2]) const {
    f[0] = make_float2(raw.x, raw.y);
    f[1] = make_float2(raw.z, raw.w);
  }
  __device__ __forceinline__ void set2(const float2 f[2]) {
    raw = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  }
};

// A thread's four channels: weights by tap, as pairs of channels, and the last K - 1 inputs.
// With eight channels a thread held 128 registers, and 512 threads a multiprocessor kept too few
// loads on their way: 48 us against 38 for 4 x 8192 x 1280 bf16.
template <typename T, int K>
struct ConvLane {
  float2 w[K][2], bias[2], win[K][2];
  __device__ __forceinline__ void load_weights(const float* wp, const float* bp, int c0) {
    float f[4 * K];  // [channel][tap], contiguous
#pragma unroll
    for (int i = 0; i < K; ++i) {
      const float4 t = __ldg(reinterpret_cast<const float4*>(wp + (size_t)c0 * K) + i);
      f[4 * i] = t.x;
      f[4 * i + 1] = t.y;
      f[4 * i + 2] = t.z;
      f[4 * i + 3] = t.w;
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) w[j][e] = make_float2(f[2 * e * K + j], f[(2 * e + 1) * K + j]);
    float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (bp) b = __ldg(reinterpret_cast<const float4*>(bp + c0));
    bias[0] = make_float2(b.x, b.y);
    bias[1] = make_float2(b.z, b.w);
  }
  // The next input: its output row, and the window moves up by one.
  __device__ __forceinline__ void row(const Vec4<T>& in, int act, T* out) {
    in.get2(win[K - 1]);
    float2 o[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float2 acc = bias[e];
#pragma unroll
      for (int j = 0; j < K; ++j) acc = fma2(w[j][e], win[j][e], acc);
      o[e] = acc;
    }
    pair_act<T, 2>(o, act);
#pragma unroll
    for (int j = 0; j + 1 < K; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) win[j][e] = win[j + 1][e];
    Vec4<T> r;
    r.set2(o);
    r.store(out);
  }
};

// One thread walks `rows_per_thread` rows of four channels with the last K - 1 inputs in
// registers.  The first K - 1 rows of a sequence need its kept state, and the state is
// rewritten in place; so the thread whose rows hold a sequence's first row also computes the
// rest of those K - 1 rows and writes the new state, and no other thread touches the state.
template <typename T, int K>
__global__ void __launch_bounds__(128, 7) conv_forward_kernel(ConvArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) a.seq.check();
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long tile =
      idx < 0xffffffffLL ? (long long)((unsigned)idx / (unsigned)a.cv) : idx / a.cv;
  if (tile >= a.tiles) return;
  const int c0 = (int)(idx - tile * a.cv) * 4;
  const T* x = static_cast<const T*>(a.x) + c0;
  T* y = static_cast<T*>(a.y) + c0;
  T* state = a.state ? static_cast<T*>(a.state) + c0 : nullptr;
  ConvLane<T, K> lane;
  lane.load_weights(a.w, a.bias, c0);
  const long long r0 = tile * a.rows_per_thread;
  const bool last_tile = tile == a.tiles - 1;
  const long long r1 = last_tile ? a.seq.R : r0 + a.rows_per_thread;

  auto walk = [&](long long r, long long end) {
    const T* xr = x + r * a.x_stride;
    T* yr = y + r * a.C;
    constexpr int CONV_ROWS = 16 / (int)sizeof(T);  // on their way at a time: 64 bytes
    for (; r + CONV_ROWS <= end; r += CONV_ROWS) {
      Vec4<T> nx[CONV_ROWS];
#pragma unroll
      for (int i = 0; i < CONV_ROWS; ++i) nx[i].load(xr + i * a.x_stride);
#pragma unroll
      for (int i = 0; i < CONV_ROWS; ++i) lane.row(nx[i], a.act, yr + (size_t)i * a.C);
      xr += CONV_ROWS * a.x_stride;
      yr += (size_t)CONV_ROWS * a.C;
    }
    for (; r < end; ++r) {
      Vec4<T> nx;
      nx.load(xr);
      lane.row(nx, a.act, yr);
      xr += a.x_stride;
      yr += a.C;
    }
  };

  int b = a.seq.first_from(r0);
  if (b > 0) {  // the sequence that runs on from an earlier thread's rows
    const long long s0 = a.seq.start(b - 1), e0 = a.seq.end(b - 1);
    long long r = s0 + K - 1 > r0 ? s0 + K - 1 : r0;
    const long long end = e0 < r1 ? e0 : r1;
    if (s0 < r0 && r < end) {
#pragma unroll
      for (int j = 0; j + 1 < K; ++j) {
        Vec4<T> t;
        t.load(x + (r - (K - 1) + j) * a.x_stride);
        t.get2(lane.win[j]);
      }
      walk(r, end);
    }
  }
  for (; b < a.seq.B; ++b) {
    const long long s0 = a.seq.start(b), e0 = a.seq.end(b);
    if (s0 >= r1 && !last_tile) break;
    Vec4<T> win[K - 1];
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) {
      if (a.from_zero)
        win[j].zero();
      else
        win[j].load(state + ((size_t)b * (K - 1) + j) * a.C);
    }
    if (state) {  // the sequence's last K - 1 inputs, older ones from the kept state
#pragma unroll
      for (int j = 0; j + 1 < K; ++j) {
        const long long r = e0 - (K - 1) + j;
        Vec4<T> t;
        if (r >= s0) {
          t.load(x + r * a.x_stride);
        } else {
          const long long o = r - s0 + (K - 1);  // index among the kept inputs, 0..K-2
          t = win[0];
#pragma unroll
          for (int i = 1; i + 1 < K; ++i)
            if (o == i) t = win[i];
        }
        t.store(state + ((size_t)b * (K - 1) + j) * a.C);
      }
    }
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) win[j].get2(lane.win[j]);
    long long end = s0 + K - 1 > r1 ? s0 + K - 1 : r1;
    if (e0 < end) end = e0;
    walk(s0, end);
  }
}

// One token: the state's K - 1 inputs and the new one give the output, and the state moves up
// by one.  A thread per four channels of a sequence.
template <typename T, int K>
__global__ void __launch_bounds__(128) conv_step_kernel(ConvArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long b = idx / a.cv;
  if (b >= a.seq.B) return;
  const int c0 = (int)(idx - b * a.cv) * 4;
  T* state = static_cast<T*>(a.state) + (size_t)b * (K - 1) * a.C + c0;
  Vec4<T> win[K];
#pragma unroll
  for (int j = 0; j + 1 < K; ++j) win[j].load(state + (size_t)j * a.C);
  win[K - 1].load(static_cast<const T*>(a.x) + b * a.x_stride + c0);
  ConvLane<T, K> lane;
  lane.load_weights(a.w, a.bias, c0);
#pragma unroll
  for (int j = 0; j + 1 < K; ++j) {
    win[j].get2(lane.win[j]);
    win[j + 1].store(state + (size_t)j * a.C);
  }
  lane.row(win[K - 1], a.act, static_cast<T*>(a.y) + (size_t)b * a.C + c0);
}

}  // namespace sdm
