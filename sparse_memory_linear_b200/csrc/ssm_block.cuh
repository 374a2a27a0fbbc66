// ssm_block.cuh -- block-wise state-space scan on the tensor cores (bf16 inputs, N <= 128).
//
// Blocks of L = 128 tokens.  With c_t the summed log-decay d A of a block's tokens up to t and M
// the state before the block,
//   y_t = exp(c_t) q_t M + sum_{s<=t} exp(c_t - c_s) d_s (q_t . k_s) v_s
//   M'  = exp(c_L) M + sum_s exp(c_L - c_s) d_s k_s (x) v_s
// so a block is four matrix products, all on tcgen05 with fp32 sums in tensor memory:
//   S  = q k^T                      128 x 128 x N
//   Y2 = q M                        128 x (2 x 64) x N, M as two bf16 parts (16 bits of it)
//   Y1 = (S o weights) v            128 x 64 x 128, weights rounded to bf16
//   dM = k^T (w o v)                N x (3 x 64) x 128, w o v as three bf16 parts (24 bits)
// The parts lie side by side as columns of one product, so that q and k are read from shared
// memory once for all of them: its bandwidth is what the matrix unit waits for at these sizes.
// The state is kept in fp32 registers and never rounded to less: dM has to be exact to fp32,
// hence the three parts.  What enters y may be rounded to the type of y once: each token's
// weight in another's read (half a step of bf16); two parts of M keep the second term below
// that.
//
// One CTA walks the blocks of (sequence segment, head, 64 value columns) in order:
//   warps 0-3    a thread per token row: weighs S into P (tensor memory), then joins
//                y = exp(c_t) Y2 + Y1 + D v, gates and stores it
//   warps 4-7    a thread per state row: adds dM to the decayed state, publishes its two parts
//   warps 8-11   a thread per quarter row of v: w o v in parts
//   warp 12      issues S, Y1            warp 13  issues dM
//   warp 14      TMA loads of q, k, v    warp 15  step sizes and decay sums, two blocks ahead;
//                                                 issues Y2
// joined by mbarriers.
//
// Decays are summed within runs of 32 tokens (a warp's rows) and the runs' totals added, never as
// differences of long sums: exp(c_t - c_s) is one exponential inside a run, and the product of
// exp(sum from t's run start) and exp(sum to s's run end) across runs; for A <= 0 no factor
// exceeds 1.
#pragma once

#include "ssm.cuh"
#include "tc.cuh"

namespace sdm {

constexpr int SB_L = 128;      // tokens of a block
constexpr int SB_P = 64;       // value columns of a CTA
constexpr int SB_THREADS = 512;

// Shared memory, from a 1024-byte boundary.
constexpr uint32_t SB_PANEL = 16384;                       // 128 rows of 128 bytes
constexpr uint32_t SB_Q = 0;                               // 2 stages x 2 panels
constexpr uint32_t SB_K = SB_Q + 4 * SB_PANEL;             // 2 stages x 2 panels
constexpr uint32_t SB_V = SB_K + 4 * SB_PANEL;             // 2 stages
constexpr uint32_t SB_H = SB_V + 2 * SB_PANEL;             // two parts of the state
constexpr uint32_t SB_W = SB_H + 2 * SB_PANEL;             // 2 quarters x 3 parts x 32 rows
constexpr uint32_t SB_WPART = 4096;
constexpr uint32_t SB_PREP = SB_W + 6 * SB_WPART;          // 2 x SsmPrep
struct SsmPrep {
  float d[SB_L];      // step size
  float in[SB_L];     // log2 decay from the run's start up to and with the token
  float out[SB_L];    // d * 2^(log2 decay after the token to the run's end)
  float w[SB_L];      // d * 2^(log2 decay after the token to the block's end)
  float run[4];       // log2 decay of each run
  float pad[28];
};
constexpr uint32_t SB_BARS = SB_PREP + 2 * sizeof(SsmPrep);
enum {
  BAR_QFULL = 0, BAR_QFREE = 2, BAR_KFULL = 4, BAR_KFREE = 6, BAR_VFULL = 8, BAR_VFREE = 10,
  BAR_PREP = 12, BAR_PREPFREE = 14, BAR_WREADY = 16, BAR_WFREE = 18, BAR_CLEAN = 20,
  BAR_S = 22, BAR_P, BAR_Y, BAR_Y2, BAR_Y2FREE, BAR_DM, BAR_DMFREE, BAR_HREADY, BAR_HFREE,
  BAR_DRAIN, BAR_COUNT = BAR_DRAIN + 3
};
constexpr uint32_t SB_TMEM_PTR = SB_BARS + 40 * 8;
static_assert(BAR_COUNT <= 40, "barriers");
constexpr uint32_t SB_SMEM = SB_TMEM_PTR + 32 + 1024;      // and room to align
static_assert(SB_SMEM <= 232448 - 64, "shared memory of a block");

// Tensor memory columns; P takes the first half of S's.
constexpr uint32_t TM_S = 0, TM_Y1 = 128, TM_Y2 = 192, TM_DM = 320;

constexpr float SB_LOG2E = 1.4426950408889634f;

struct SsmBlockArgs {
  SsmArgs a;
  CUtensorMap mq, mk, mv, my;
  int seg_blocks;   // blocks of a segment
  int ptiles;       // 64-column tiles of d_v
};

// The (sequence, segment) of work item `item`: a sequence of n rows has max(1, ceil(n / seg))
// segments.  Called by one warp; false past the last.
__device__ __forceinline__ bool ssm_find_item(const SeqBounds& seq, long long item, long long seg,
                                              int* b_out, long long* s_out) {
  if (!seq.cu) {
    const long long per = seq.T > 0 ? (seq.T + seg - 1) / seg : 1;
    *b_out = (int)(item / per);
    *s_out = item % per;
    return *b_out < seq.B;
  }
  const int lane = threadIdx.x & 31;
  for (int b0 = 0; b0 < seq.B; b0 += 32) {
    const int b = b0 + lane;
    long long n = 0;
    if (b < seq.B) {
      const long long len = seq.end(b) - seq.start(b);
      n = len > 0 ? (len + seg - 1) / seg : 1;
    }
    long long upto = n;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const long long o = __shfl_up_sync(FULL_MASK, upto, s);
      if (lane >= s) upto += o;
    }
    const unsigned hit = __ballot_sync(FULL_MASK, upto > item);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *b_out = b0 + l;
      *s_out = item - __shfl_sync(FULL_MASK, upto - n, l);
      return true;
    }
    item -= __shfl_sync(FULL_MASK, upto, 31);
  }
  return false;
}

__global__ void __launch_bounds__(SB_THREADS, 1)
    ssm_block_kernel(const __grid_constant__ SsmBlockArgs ba) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_abort;
  __shared__ int s_item_ok, s_b;
  __shared__ long long s_seg;
  const SsmArgs& a = ba.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - smem_addr(smem_raw));
  const uint32_t bars = base + SB_BARS;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };

  if (blockIdx.x == 0) a.seq.check();
  const int per_item = a.H * ba.ptiles;
  const long long item = blockIdx.x / per_item;
  const int hp = blockIdx.x % per_item, h = hp / ba.ptiles, p0 = hp % ba.ptiles * SB_P;
  const int g = h / (a.H / a.G);
  const long long seg_rows = (long long)ba.seg_blocks * SB_L;
  if (warp == 0) {
    int b = 0;
    long long s = 0;
    const bool ok = ssm_find_item(a.seq, item, seg_rows, &b, &s);
    if (lane == 0) {
      s_item_ok = ok;
      s_b = b;
      s_seg = s;
      s_abort = 0;
    }
  }
  __syncthreads();
  if (!s_item_ok) return;
  const int b = s_b;
  const long long seq0 = a.seq.start(b), seq1 = a.seq.end(b);
  const long long row0 = seq0 + s_seg * seg_rows;
  const long long row1 = row0 + seg_rows < seq1 ? row0 + seg_rows : seq1;
  const int nb = (int)((row1 - row0 + SB_L - 1) / SB_L);
  float* const Mp = a.M + ((size_t)b * a.H + h) * a.N * a.P;
  if (nb == 0) {  // an empty sequence
    if (a.from_zero)
      for (int i = tid; i < a.N * SB_P; i += SB_THREADS) {
        const int p = p0 + i % SB_P;
        if (p < a.P) Mp[(size_t)(i / SB_P) * a.P + p] = 0.0f;
      }
    return;
  }
  const int npanels = a.N > 64 ? 2 : 1, nk = (a.N + 15) / 16;

  if (warp == 0) tmem_alloc(base + SB_TMEM_PTR, 512);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_QFULL + i), 1);
      mbar_init(bar(BAR_QFREE + i), 2);
      mbar_init(bar(BAR_KFULL + i), 1);
      mbar_init(bar(BAR_KFREE + i), 2);
      mbar_init(bar(BAR_VFULL + i), 1);
      mbar_init(bar(BAR_VFREE + i), 4);
      mbar_init(bar(BAR_PREP + i), 1);
      mbar_init(bar(BAR_PREPFREE + i), 12);
      mbar_init(bar(BAR_WREADY + i), 4);
      mbar_init(bar(BAR_WFREE + i), 1);
      mbar_init(bar(BAR_CLEAN + i), 4);
    }
    mbar_init(bar(BAR_S), 1);
    mbar_init(bar(BAR_P), 4);
    mbar_init(bar(BAR_Y), 1);
    mbar_init(bar(BAR_Y2), 1);
    mbar_init(bar(BAR_Y2FREE), 4);
    mbar_init(bar(BAR_DM), 1);
    mbar_init(bar(BAR_DMFREE), 4);
    mbar_init(bar(BAR_HREADY), 4);
    mbar_init(bar(BAR_HFREE), 1);
    for (int i = 0; i < 3; ++i) mbar_init(bar(BAR_DRAIN + i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (npanels == 1) {  // state rows 64 and up: k is 0 there
    uint4* z = reinterpret_cast<uint4*>(sm + SB_K);
    for (int i = tid; i < 2 * (int)SB_PANEL / 16; i += SB_THREADS) {
      const int stage = i / (SB_PANEL / 16), j = i % (SB_PANEL / 16);
      z[(2 * stage + 1) * (SB_PANEL / 16) + j] = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + SB_TMEM_PTR);
  volatile int* const abort = &s_abort;
  // phase of the c-th use of a barrier that completes once per block, or per two of them
  auto wait = [&](int i, int use) { return mbar_wait(bar(i), (uint32_t)use & 1u, abort); };
  auto prep = [&](int c) {
    return reinterpret_cast<SsmPrep*>(sm + SB_PREP + (c & 1) * sizeof(SsmPrep));
  };

  if (warp < 4) {
    // ------------------------------------------------ rows of y: t = tid
    const int t = tid;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const float D = a.D ? a.D[h] : 0.0f;
    const float2 D2 = make_float2(D, D);
    const int pn = a.P - p0 < SB_P ? a.P - p0 : SB_P;  // columns that exist
    __nv_bfloat16* const yp = static_cast<__nv_bfloat16*>(a.y) + (size_t)h * a.P + p0;
    const __nv_bfloat16* const zp =
        a.gate ? static_cast<const __nv_bfloat16*>(a.gate) + (size_t)h * a.P + p0 : nullptr;
    for (int c = 0; c < nb; ++c) {
      if (!wait(BAR_PREP + (c & 1), c >> 1) || !wait(BAR_S, c)) break;
      tc_fence_after();
      float decay;  // from the block's start up to t
      const SsmPrep& pr = *prep(c);
      const float in_t = pr.in[t];
      // decay from the end of each earlier run up to t
      float to[4];
      {
        float e = in_t;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          to[j] = 0.0f;
          if (j < warp) {
            to[j] = fast_exp2(e);
            e += pr.run[j];
          }
        }
        decay = fast_exp2(e);
      }
      const uint32_t sbuf = tm + TM_S + lanes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t pk[16];
        if (j > warp) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        } else {
          float s[32];
          tmem_ld32(sbuf + 32 * j, s);
          tmem_wait_ld();
          if (j < warp) {
            const float2 f2 = make_float2(to[j], to[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 o = *reinterpret_cast<const float4*>(&pr.out[32 * j + 4 * i]);
              const float2 u = mul2(mul2(make_float2(o.x, o.y), f2),
                                    make_float2(s[4 * i], s[4 * i + 1]));
              const float2 v = mul2(mul2(make_float2(o.z, o.w), f2),
                                    make_float2(s[4 * i + 2], s[4 * i + 3]));
              pk[2 * i] = pack_bf16(u.x, u.y);
              pk[2 * i + 1] = pack_bf16(v.x, v.y);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 in = *reinterpret_cast<const float4*>(&pr.in[32 * j + 4 * i]);
              const float4 d = *reinterpret_cast<const float4*>(&pr.d[32 * j + 4 * i]);
              float w[4] = {s[4 * i] * d.x * fast_exp2(in_t - in.x),
                            s[4 * i + 1] * d.y * fast_exp2(in_t - in.y),
                            s[4 * i + 2] * d.z * fast_exp2(in_t - in.z),
                            s[4 * i + 3] * d.w * fast_exp2(in_t - in.w)};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (4 * i + e > lane) w[e] = 0.0f;
              pk[2 * i] = pack_bf16(w[0], w[1]);
              pk[2 * i + 1] = pack_bf16(w[2], w[3]);
            }
          }
        }
        // P's columns 16 j .. lie in columns of S that are already read
        tmem_st16(sbuf + 16 * j, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(BAR_P));
        mbar_arrive(bar(BAR_PREPFREE + (c & 1)));
      }
      const long long first = row0 + (long long)c * SB_L, row = first + t;
      const bool live = row < row1, whole = first + SB_L <= row1;
      uint4 zz[8];
      if (zp) {  // on its way while the products finish
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (live && 8 * i < pn)
            zz[i] = *reinterpret_cast<const uint4*>(zp + row * a.gate_stride + 8 * i);
      }
      if (!wait(BAR_Y2, c) || !wait(BAR_Y, c)) break;
      tc_fence_after();
      uint8_t* vtile = sm + SB_V + (c & 1) * SB_PANEL;
      const float2 f2 = make_float2(decay, decay);
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float y1[16], y2[16], y3[16];
        tmem_ld16(tm + TM_Y1 + 16 * part + lanes, y1);
        tmem_ld16(tm + TM_Y2 + 16 * part + lanes, y2);
        tmem_ld16(tm + TM_Y2 + 64 + 16 * part + lanes, y3);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int ch = 2 * part + i;
          uint4* place = reinterpret_cast<uint4*>(vtile + tile_offset(t, ch));
          const uint4 vv = *place;
          const uint32_t vw[4] = {vv.x, vv.y, vv.z, vv.w};
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = 8 * i + 2 * j;
            const float2 r = fma2(f2, make_float2(y3[e], y3[e + 1]),
                                  fma2(f2, make_float2(y2[e], y2[e + 1]),
                                       make_float2(y1[e], y1[e + 1])));
            o[j] = fma2(D2, unpack_bf16(vw[j]), r);
          }
          if (zp) {
            const uint32_t zw[4] = {zz[ch].x, zz[ch].y, zz[ch].z, zz[ch].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 z = unpack_bf16(zw[j]);
              o[j] = mul2(o[j], make_float2(fast_gate_act(z.x, a.act), fast_gate_act(z.y, a.act)));
            }
          }
          const uint4 out = make_uint4(pack_bf16(o[0].x, o[0].y), pack_bf16(o[1].x, o[1].y),
                                       pack_bf16(o[2].x, o[2].y), pack_bf16(o[3].x, o[3].y));
          if (whole)
            *place = out;  // v's last reader leaves y in its place
          else if (live && 8 * ch < pn)
            *reinterpret_cast<uint4*>(yp + (size_t)row * a.H * a.P + 8 * ch) = out;
        }
      }
      if (whole) fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(BAR_Y2FREE));
        if (whole) {
          tma_store_3d(&ba.my, p0, h, (int)first + 32 * warp,
                       base + SB_V + (c & 1) * SB_PANEL + warp * 4096);
          tma_store_commit();
          tma_store_wait_read();
        }
        mbar_arrive(bar(BAR_VFREE + (c & 1)));
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------ the state: row n = tid - 128
    const int n = tid - 128;
    const uint32_t lanes = (uint32_t)((warp - 4) * 32) << 16;
    const int pn = a.P - p0 < SB_P ? a.P - p0 : SB_P;
    float* const mrow = Mp + (size_t)n * a.P + p0;
    float st[SB_P];
#pragma unroll
    for (int i = 0; i < SB_P; i += 4) {
      float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!a.from_zero && n < a.N && i < pn) m = *reinterpret_cast<const float4*>(mrow + i);
      st[i] = m.x;
      st[i + 1] = m.y;
      st[i + 2] = m.z;
      st[i + 3] = m.w;
    }
    // two bf16 parts of the state row, as rows of the B operand of Y2
    auto publish = [&]() {
      uint8_t* hi = sm + SB_H;
      uint8_t* lo = sm + SB_H + SB_PANEL;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        uint32_t u[4], v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float x0 = st[8 * ch + 2 * j], x1 = st[8 * ch + 2 * j + 1];
          u[j] = pack_bf16(x0, x1);
          const float2 r = unpack_bf16(u[j]);
          v[j] = pack_bf16(x0 - r.x, x1 - r.y);
        }
        const uint32_t o = tile_offset(n, ch);
        *reinterpret_cast<uint4*>(hi + o) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(lo + o) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_HREADY));
    };
    publish();
    bool ok = true;
    for (int c = 0; c < nb; ++c) {
      ok = wait(BAR_PREP + (c & 1), c >> 1);
      if (!ok) break;
      const SsmPrep& pr = *prep(c);
      const float keep = exp2f((pr.run[0] + pr.run[1]) + (pr.run[2] + pr.run[3]));
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_PREPFREE + (c & 1)));
      ok = wait(BAR_DM, c);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int part = 0; part < 4; ++part) {
        float r1[16], r2[16], r3[16];
        tmem_ld16(tm + TM_DM + 16 * part + lanes, r1);
        tmem_ld16(tm + TM_DM + 64 + 16 * part + lanes, r2);
        tmem_ld16(tm + TM_DM + 128 + 16 * part + lanes, r3);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          st[16 * part + i] = fmaf(st[16 * part + i], keep, r1[i] + (r2[i] + r3[i]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_DMFREE));
      if (c + 1 < nb) {
        ok = wait(BAR_HFREE, c);
        if (!ok) break;
        publish();
      }
    }
    if (ok && row1 == seq1 && n < a.N) {
#pragma unroll
      for (int i = 0; i < SB_P; i += 4)
        if (i < pn)
          *reinterpret_cast<float4*>(mrow + i) =
              make_float4(st[i], st[i + 1], st[i + 2], st[i + 3]);
    }
  } else if (warp < 12) {
    // ------------------------------------------------ w o v in three bf16 parts
    const int i0 = tid - 256, rq = i0 >> 2;  // row in the quarter, and 16 of its values
    for (int c = 0; c < nb; ++c) {
      const int stage = c & 1;
      if (!wait(BAR_PREP + stage, c >> 1) || !wait(BAR_VFULL + stage, c >> 1)) break;
      uint8_t* vtile = sm + SB_V + stage * SB_PANEL;
      const long long left = row1 - (row0 + (long long)c * SB_L);
      uint4 vv[8];
      float w[4];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        vv[i] = *reinterpret_cast<const uint4*>(
            vtile + tile_offset(32 * (i >> 1) + rq, 2 * (i0 & 3) + (i & 1)));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = prep(c)->w[32 * i + rq];
      if (left < SB_L) {
        // rows behind the segment's end, whatever they hold, become zeros
        if (!wait(BAR_KFULL + stage, c >> 1)) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int t = 32 * (i >> 1) + rq;
          if (t < left) continue;
          const uint32_t o = tile_offset(t, 2 * (i0 & 3) + (i & 1));
          vv[i] = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(vtile + o) = vv[i];
          for (int pl = 0; pl < npanels; ++pl)
            *reinterpret_cast<uint4*>(sm + SB_K + (2 * stage + pl) * SB_PANEL + o) = vv[i];
        }
      }
      bool ok = true;
#pragma unroll
      for (int qd = 0; qd < 4; ++qd) {
        const int use = 4 * c + qd, buf = qd & 1;
        uint32_t p[3][8];
        const float2 w2 = make_float2(w[qd], w[qd]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint4 u = vv[2 * qd + (j >> 2)];
          const uint32_t word = (j & 3) == 0 ? u.x : (j & 3) == 1 ? u.y : (j & 3) == 2 ? u.z : u.w;
          float2 x = mul2(unpack_bf16(word), w2);
          p[0][j] = pack_bf16(x.x, x.y);
          x = sub2(x, unpack_bf16(p[0][j]));
          p[1][j] = pack_bf16(x.x, x.y);
          x = sub2(x, unpack_bf16(p[1][j]));
          p[2][j] = pack_bf16(x.x, x.y);
        }
        ok = ok && (use < 2 || wait(BAR_WFREE + buf, (use >> 1) - 1));
        uint8_t* wt = sm + SB_W + buf * 3 * SB_WPART;
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(wt + part * SB_WPART + tile_offset(rq, 2 * (i0 & 3) + i)) =
                make_uint4(p[part][4 * i], p[part][4 * i + 1], p[part][4 * i + 2],
                           p[part][4 * i + 3]);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_WREADY + buf));
      }
      if (lane == 0) {
        mbar_arrive(bar(BAR_CLEAN + stage));
        mbar_arrive(bar(BAR_PREPFREE + stage));
      }
      if (!ok) break;
    }
  } else if (warp == 12) {
    // ------------------------------------------------ products S and Y1
    constexpr uint32_t dS = mma_desc(128, 128, 0, 0), dY1 = mma_desc(128, 64, 0, 1);
    const uint32_t q0 = tile_desc(base + SB_Q), k0 = tile_desc(base + SB_K),
                   v0 = tile_desc(base + SB_V);
    for (int c = 0; c <= nb; ++c) {
      if (c > 0) {
        const int e = c - 1;
        const uint32_t stage = e & 1;
        if (!wait(BAR_CLEAN + stage, e >> 1) || !wait(BAR_VFULL + stage, e >> 1) ||
            !wait(BAR_P, e))
          break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t v = v0 + stage * (SB_PANEL >> 4);
#pragma unroll
          for (int i = 0; i < SB_L / 16; ++i)
            mma_ts(tm + TM_Y1, tm + TM_S + 8 * i, v + i * (2048 >> 4), dY1, i > 0);
          mma_commit(bar(BAR_Y));
        }
        __syncwarp();
      }
      if (c < nb) {
        const uint32_t stage = c & 1;
        if (!wait(BAR_QFULL + stage, c >> 1) || !wait(BAR_KFULL + stage, c >> 1)) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t q = q0 + stage * (2 * SB_PANEL >> 4), k = k0 + stage * (2 * SB_PANEL >> 4);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t o = ((i >> 2) * SB_PANEL + (i & 3) * 32) >> 4;
            if (i < nk) mma_ss(tm + TM_S, q + o, k + o, dS, i > 0);
          }
          mma_commit(bar(BAR_S));
          mma_commit(bar(BAR_KFREE + stage));
          mma_commit(bar(BAR_QFREE + stage));
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(bar(BAR_DRAIN));
    __syncwarp();
    mbar_wait(bar(BAR_DRAIN), 0, abort);
  } else if (warp == 13) {
    // ------------------------------------------------ product dM
    constexpr uint32_t dM = mma_desc(128, 192, 1, 1);
    const uint32_t k0 = tile_desc(base + SB_K, SB_PANEL), w0 = tile_desc(base + SB_W, SB_WPART);
    bool ok = true;
    for (int c = 0; c < nb && ok; ++c) {
      const uint32_t stage = c & 1, k = k0 + stage * (2 * SB_PANEL >> 4);
      ok = wait(BAR_KFULL + stage, c >> 1) && (c == 0 || wait(BAR_DMFREE, c - 1));
      for (int qd = 0; qd < 4 && ok; ++qd) {
        const uint32_t use = 4 * c + qd, buf = use & 1;
        ok = wait(BAR_WREADY + buf, use >> 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t kq = k + qd * (4096 >> 4), w = w0 + buf * (3 * SB_WPART >> 4);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mma_ss(tm + TM_DM, kq + i * (2048 >> 4), w + i * (2048 >> 4), dM, qd + i > 0);
          mma_commit(bar(BAR_WFREE + buf));
          if (qd == 3) {
            mma_commit(bar(BAR_DM));
            mma_commit(bar(BAR_KFREE + stage));
          }
        }
        __syncwarp();
      }
    }
    if (elect_one()) mma_commit(bar(BAR_DRAIN + 1));
    __syncwarp();
    mbar_wait(bar(BAR_DRAIN + 1), 0, abort);
  } else if (warp == 14) {
    // ------------------------------------------------ loads: each tile as soon as its place is free
    if (lane == 0) {
      int kc = 0, vc = 0, qc = 0;  // blocks whose load is issued
      const int r0 = (int)row0;
      unsigned long long since = 0;
      while (kc < nb || vc < nb || qc < nb) {
        bool moved = false;
        auto may = [&](int c, int free_bar) {
          return c < nb &&
                 (c < 2 || mbar_test(bar(free_bar + (c & 1)), (uint32_t)((c >> 1) - 1) & 1u));
        };
        if (may(qc, BAR_QFREE)) {
          const uint32_t stage = qc & 1;
          mbar_expect(bar(BAR_QFULL + stage), npanels * SB_PANEL);
          for (int pl = 0; pl < npanels; ++pl)
            tma_load_3d(base + SB_Q + (2 * stage + pl) * SB_PANEL, &ba.mq, 64 * pl, g,
                        r0 + qc * SB_L, bar(BAR_QFULL + stage));
          ++qc;
          moved = true;
        }
        if (may(kc, BAR_KFREE)) {
          const uint32_t stage = kc & 1;
          mbar_expect(bar(BAR_KFULL + stage), npanels * SB_PANEL);
          for (int pl = 0; pl < npanels; ++pl)
            tma_load_3d(base + SB_K + (2 * stage + pl) * SB_PANEL, &ba.mk, 64 * pl, g,
                        r0 + kc * SB_L, bar(BAR_KFULL + stage));
          ++kc;
          moved = true;
        }
        if (may(vc, BAR_VFREE)) {
          const uint32_t stage = vc & 1;
          mbar_expect(bar(BAR_VFULL + stage), SB_PANEL);
          tma_load_3d(base + SB_V + stage * SB_PANEL, &ba.mv, p0, h, r0 + vc * SB_L,
                      bar(BAR_VFULL + stage));
          ++vc;
          moved = true;
        }
        if (moved) {
          since = 0;
          continue;
        }
        if (*abort) break;
        const unsigned long long now = wall_ns();
        if (since == 0) since = now;
        if (now - since > MBAR_LIMIT_NS) {
          *abort = 1;
          record_status(STATUS_TIMEOUT);
          break;
        }
        __nanosleep(40);
      }
      if (*abort) {
        // loads in flight land before the block's memory is given up (each wait limited)
        int none = 0;
        const int n[3] = {qc, kc, vc}, full[3] = {BAR_QFULL, BAR_KFULL, BAR_VFULL};
        for (int i = 0; i < 3; ++i)
          for (int c = n[i] > 2 ? n[i] - 2 : 0; c < n[i]; ++c)
            mbar_wait(bar(full[i] + (c & 1)), (uint32_t)(c >> 1) & 1u, &none);
      }
    }
  } else {
    // ------------------------------------------------ step sizes and decay sums
    const __nv_bfloat16* dp = static_cast<const __nv_bfloat16*>(a.dt) + h;
    const float A2 = a.A[h] * SB_LOG2E, bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
    float raw[4];
    auto fetch = [&](int c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long r = row0 + (long long)c * SB_L + 4 * lane + i;
        raw[i] = r < row1 ? __bfloat162float(dp[r * a.dt_stride]) : 0.0f;
      }
    };
    fetch(0);
    auto prepare = [&](int c) -> bool {
      float d[4], la[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long r = row0 + (long long)c * SB_L + 4 * lane + i;
        d[i] = r < row1 ? ssm_step_size(raw[i] + bias, a.softplus) : 0.0f;
        // 2^-160 is 0 in fp32: a stronger decay changes nothing and would cost the sums their
        // low bits
        la[i] = fmaxf(d[i] * A2, -160.0f);
      }
      if (c + 1 < nb) fetch(c + 1);
      // sums over the run's 8 lanes, from its start and from its end
      const float own = (la[0] + la[1]) + (la[2] + la[3]);
      float up = own, down = own;
#pragma unroll
      for (int s = 1; s < 8; s <<= 1) {
        const float o = __shfl_up_sync(FULL_MASK, up, s, 8);
        const float u = __shfl_down_sync(FULL_MASK, down, s, 8);
        if ((lane & 7) >= s) up += o;
        if ((lane & 7) + s < 8) down += u;
      }
      float before = __shfl_up_sync(FULL_MASK, up, 1, 8),
            after = __shfl_down_sync(FULL_MASK, down, 1, 8);
      if ((lane & 7) == 0) before = 0.0f;
      if ((lane & 7) == 7) after = 0.0f;
      float run[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) run[j] = __shfl_sync(FULL_MASK, up, 8 * j + 7);
      float later = 0.0f;  // runs behind this lane's
#pragma unroll
      for (int j = 3; j >= 1; --j)
        if (j > (lane >> 3)) later += run[j];
      float in[4], out[4], w[4];
      in[0] = before + la[0];
      in[1] = before + (la[0] + la[1]);
      in[2] = before + (la[0] + la[1] + la[2]);
      in[3] = before + own;
      const float tail[4] = {after + (la[1] + la[2] + la[3]), after + (la[2] + la[3]),
                             after + la[3], after};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        out[i] = d[i] * exp2f(tail[i]);
        w[i] = d[i] * exp2f(tail[i] + later);
      }
      if (c >= 2 && !wait(BAR_PREPFREE + (c & 1), (c >> 1) - 1)) return false;
      SsmPrep* pr = prep(c);
      reinterpret_cast<float4*>(pr->d)[lane] = make_float4(d[0], d[1], d[2], d[3]);
      reinterpret_cast<float4*>(pr->in)[lane] = make_float4(in[0], in[1], in[2], in[3]);
      reinterpret_cast<float4*>(pr->out)[lane] = make_float4(out[0], out[1], out[2], out[3]);
      reinterpret_cast<float4*>(pr->w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
      if (lane < 4) pr->run[lane] = lane == 0 ? run[0] : lane == 1 ? run[1] : lane == 2 ? run[2] : run[3];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_PREP + (c & 1)));
      return true;
    };
    constexpr uint32_t dY2 = mma_desc(128, 128, 0, 1);
    const uint32_t q0 = tile_desc(base + SB_Q), h0 = tile_desc(base + SB_H, SB_PANEL);
    bool ok = prepare(0) && (nb < 2 || prepare(1));
    for (int c = 0; c < nb && ok; ++c) {
      const uint32_t stage = c & 1;
      ok = wait(BAR_HREADY, c) && wait(BAR_QFULL + stage, c >> 1) &&
           (c == 0 || wait(BAR_Y2FREE, c - 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        const uint32_t q = q0 + stage * (2 * SB_PANEL >> 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t o = ((i >> 2) * SB_PANEL + (i & 3) * 32) >> 4;
          if (i < nk) mma_ss(tm + TM_Y2, q + o, h0 + i * (2048 >> 4), dY2, i > 0);
        }
        mma_commit(bar(BAR_Y2));
        mma_commit(bar(BAR_HFREE));
        mma_commit(bar(BAR_QFREE + stage));
      }
      __syncwarp();
      if (c + 2 < nb) ok = prepare(c + 2);
    }
    if (elect_one()) mma_commit(bar(BAR_DRAIN + 2));
    __syncwarp();
    mbar_wait(bar(BAR_DRAIN + 2), 0, abort);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tm, 512);
}

}  // namespace sdm
