// ssm_block.cuh -- block-wise state-space scan on the tensor cores (bf16 inputs, N <= 128).
//
// Blocks of L = 128 tokens.  With c_t the summed log-decay d A of a block's tokens up to t and M
// the state before the block,
//   y_t = exp(c_t) q_t M + sum_{s<=t} exp(c_t - c_s) d_s (q_t . k_s) v_s
//   M'  = exp(c_L) M + sum_s exp(c_L - c_s) d_s k_s (x) v_s
// so a block is four matrix products, all on tcgen05 with fp32 sums in tensor memory:
//   S  = q k^T                      128 x 128 x N
//   Y2 = q M                        2 products 128 x 64 x N, M as two bf16 parts (16 bits of it)
//   Y1 = (S o weights) v            2 products 128 x 64 x 128, weights as two bf16 parts
//   dM = k^T (w o v)                3 products N x 64 x 128, w o v as three bf16 parts (24 bits)
// The state is kept in fp32 registers and never rounded to less: dM has to be exact to fp32,
// hence the three parts.  y is rounded to bf16 once, half a step of 2^-8; what it reads, each token's
// weight in another's read and the state before the block, is held to 2^-16, so that y's error
// is its own rounding.  (With the weights in one part the error against 64 bits was up to 1.5
// times that of a scan in fp32, rounded once.)
//
// One CTA walks the blocks of its (sequence segment, head, 64 value columns) pieces in order, four
// groups of four warps each at its own block:
//   P   a thread per token row: weighs S into P (tensor memory, in place)
//   Y   a thread per token row: y = exp(c_t) Y2 + Y1 + D v, gated and stored
//   H   a thread per state row: adds dM to the decayed state, publishes the state's two parts
//   W   a thread per quarter row of v: w o v in parts, 32 tokens at a time
//   and four single warps: dM and Y1; Y2 and S; loads of q and k; loads of v and of the blocks'
//   sums
// joined by mbarriers.  A block's work is a chain of short dependent steps; with the steps on
// warps of their own the chains of successive blocks overlap.  One group for everything took 11
// us a block, two groups 3.5, these 3.0 (3.8 with a gate; 128 tokens, N = 128, all
// multiprocessors busy).  No unit is full at that: 46 % of the issue slots are used (10300 warp
// instructions a block), the matrix unit 42 % of the time, memory less, and a group alone needs
// about half of a block's 5850 cycles.  What bounds it is the loop of waits from one group to the
// next; which of them sets the period is not established (q, with its one stage, is one: the
// load of block c + 1 waits for Y2 of block c, and S of block c + 1 for the load).
//
// Decays are summed within runs of 32 tokens (a warp's rows) and the runs' totals added, never as
// differences of long sums: exp(c_t - c_s) is one exponential inside a run, and the product of
// exp(sum from t's run start) and exp(sum to s's run end) across runs; for A <= 0 no factor
// exceeds 1.
#pragma once

#include <cfloat>

#include "ssm.cuh"
#include "tc.cuh"

namespace sdm {

constexpr int SB_L = 128;      // tokens of a block
constexpr int SB_P = 64;       // value columns of a CTA
constexpr int SB_THREADS = 640;

// Shared memory, from a 1024-byte boundary.
constexpr uint32_t SB_PANEL = 16384;                       // 128 rows of 128 bytes
constexpr uint32_t SB_Q = 0;                               // 2 panels
constexpr uint32_t SB_K = SB_Q + 2 * SB_PANEL;             // 2 stages x 2 panels
constexpr uint32_t SB_V = SB_K + 4 * SB_PANEL;             // 4 stages
constexpr uint32_t SB_H = SB_V + 4 * SB_PANEL;             // two parts of the state
constexpr uint32_t SB_W = SB_H + 2 * SB_PANEL;             // 2 quarters x 3 parts x 32 rows
constexpr uint32_t SB_WPART = 4096;
constexpr uint32_t SB_PREP = SB_W + 6 * SB_WPART;          // 4 x SsmPrep

// What the kernels need of a block's step sizes (ssm_prep_kernel).
struct SsmPrep {
  float d[SB_L];      // step size
  float in[SB_L];     // log2 decay from the run's start up to and with the token
  float out[SB_L];    // d * 2^(log2 decay after the token to the run's end)
  float w[SB_L];      // d * 2^(log2 decay after the token to the block's end)
  float run[4];       // log2 decay of each run
  float pad[28];      // a multiple of 128 bytes
};
static_assert(sizeof(SsmPrep) == 2176, "a block's sums");
constexpr uint32_t SB_BARS = SB_PREP + 4 * sizeof(SsmPrep);
enum {
  BAR_QFULL = 0, BAR_QFREE, BAR_KFULL = 2, BAR_KFREE = 4, BAR_VFULL = 6, BAR_VFREE = 10,
  BAR_PREP = 14, BAR_PREPFREE = 18, BAR_WREADY = 22, BAR_WFREE = 24, BAR_YFREE = 26,
  BAR_S = 28, BAR_P = 30, BAR_Y = 32, BAR_DM = 34, BAR_DMFREE, BAR_Y2 = 38,
  BAR_HREADY = 40, BAR_HFREE, BAR_DRAIN, BAR_COUNT = BAR_DRAIN + 2
};
constexpr uint32_t SB_TMEM_PTR = SB_BARS + 44 * 8;
static_assert(BAR_COUNT <= 44, "barriers");
constexpr uint32_t SB_SMEM = SB_TMEM_PTR + 32 + 1024;      // and room to align
static_assert(SB_SMEM <= 232448 - 64, "shared memory of a block");

// Tensor memory columns: two buffers of S, which becomes P in place (16 columns of S, 8 of each
// part); one of Y1; one of dM; two of Y2.
constexpr uint32_t TM_S = 0, TM_Y1 = 256, TM_DM = 320, TM_Y2 = 384;

constexpr float SB_LOG2E = 1.4426950408889634f;

struct SsmBlockArgs {
  SsmArgs a;
  CUtensorMap mq, mk, mv, mz;  // mz: the gate, where there is one
  SsmSplit sp;      // segments of whole blocks
  SsmPrep* prep;    // [blocks, H]
  int4* items;      // [items] (sequence, its first and past-last row, the segment's first row),
                    // longest first, then [items] ints: the place of each one's state (SsmSplit)
  int ptiles;       // 64-column tiles of d_v
  int step_items, step_parts;  // gridDim.x = step_items x (H x ptiles) + step_parts
};

// The place of a sequence's first block among all blocks' sums: sequences of T rows one after
// another, or for packed ones start / L + b, which leaves each room for ceil(length / L).
__device__ __forceinline__ long long ssm_first_block(const SeqBounds& seq, int b) {
  return seq.cu ? seq.start(b) / SB_L + b : (long long)b * ((seq.T + SB_L - 1) / SB_L);
}

// A block's step sizes and decay sums, by one warp: lane l holds tokens 4 l .. 4 l + 3.
struct SsmSums {
  float d[4], in[4], tail[4];  // step size; log2 decays from the run's start, to the run's end
  float run[4], later;         // log2 decay of each run, and of the runs behind this lane's
};
__device__ __forceinline__ void ssm_sums(const float raw[4], const bool live[4], float bias,
                                         float A2, int softplus, SsmSums& o) {
  const int lane = threadIdx.x & 31;
  float la[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.d[i] = live[i] ? ssm_step_size(raw[i] + bias, softplus) : 0.0f;
    // 2^-160 is 0 in fp32: a stronger decay changes nothing and would cost the sums their low
    // bits
    la[i] = fmaxf(o.d[i] * A2, -160.0f);
  }
  const float own = (la[0] + la[1]) + (la[2] + la[3]);
  float up = own, down = own;  // sums over the run's 8 lanes, from its start and from its end
#pragma unroll
  for (int s = 1; s < 8; s <<= 1) {
    const float p = __shfl_up_sync(FULL_MASK, up, s, 8);
    const float n = __shfl_down_sync(FULL_MASK, down, s, 8);
    if ((lane & 7) >= s) up += p;
    if ((lane & 7) + s < 8) down += n;
  }
  float before = __shfl_up_sync(FULL_MASK, up, 1, 8),
        after = __shfl_down_sync(FULL_MASK, down, 1, 8);
  if ((lane & 7) == 0) before = 0.0f;
  if ((lane & 7) == 7) after = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.run[j] = __shfl_sync(FULL_MASK, up, 8 * j + 7);
  o.later = 0.0f;
#pragma unroll
  for (int j = 3; j >= 1; --j)
    if (j > (lane >> 3)) o.later += o.run[j];
  o.in[0] = before + la[0];
  o.in[1] = before + (la[0] + la[1]);
  o.in[2] = before + (la[0] + la[1] + la[2]);
  o.in[3] = before + own;
  o.tail[0] = after + (la[1] + la[2] + la[3]);
  o.tail[1] = after + (la[2] + la[3]);
  o.tail[2] = after + la[3];
  o.tail[3] = after;
}

// Step sizes and decay sums of every block and head, once for all tiles and passes, and the table
// of work items (a packed batch's lengths are known only here): a warp per
// (block, head), a CTA's eight warps on neighbouring heads, whose dt share sectors.  Made inside
// the scan by one warp a block this was a chain of 3000 cycles, most of a block's time.
__global__ void __launch_bounds__(256) ssm_prep_kernel(SsmArgs a, SsmSplit sp, SsmPrep* prep,
                                                        int blocks, int4* items, int n_items) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y * 8 + warp;
  if ((int)blockIdx.x >= blocks) {  // work items, a warp each
    const int item = ((int)blockIdx.x - blocks) * 8 + warp;
    if (blockIdx.y != 0 || item >= n_items) return;
    int b = 0;
    long long seg = 0, slot = 0;
    const bool ok = ssm_find_item(a.seq, item, sp.seg_rows, &b, &seg, &slot);
    // Longest first: CTAs that walk every gridDim.x-th piece then end at about the same time.  The
    // place is the number of longer items and of equal ones before (bad offsets can make up
    // more items than there are places: their order is left alone).
    int place = item;
    if (ok && a.seq.cu) {
      const int whole = (int)(sp.seg_rows / SB_L);
      auto blocks_of = [&](long long rows) { return (int)((rows + SB_L - 1) / SB_L); };
      const long long own = a.seq.end(b) - a.seq.start(b) - seg * sp.seg_rows;
      const int nb = blocks_of(own < sp.seg_rows ? own : sp.seg_rows);
      int total = 0, before = 0;
      for (int e = lane; e < a.seq.B; e += 32) {
        const long long len = a.seq.end(e) - a.seq.start(e), full = len / sp.seg_rows;
        const long long left = len - full * sp.seg_rows;
        const int tail = left > 0 || len == 0, tail_nb = blocks_of(left);
        total += (int)full + tail;
        before += (whole > nb ? (int)full : 0) + (tail && tail_nb > nb);
        if (e < b) before += (whole == nb ? (int)full : 0) + (tail && tail_nb == nb);
        if (e == b && whole == nb) before += (int)(seg < full ? seg : full);
      }
      total = __reduce_add_sync(FULL_MASK, total);
      before = __reduce_add_sync(FULL_MASK, before);
      if (total <= n_items) place = before;
    }
    if (lane == 0) {
      items[place] = ok ? make_int4(b, (int)a.seq.start(b), (int)a.seq.end(b),
                                    (int)(a.seq.start(b) + seg * sp.seg_rows))
                        : make_int4(-1, 0, 0, 0);
      reinterpret_cast<int*>(items + n_items)[place] = (int)sp.place(slot);
    }
    return;
  }
  if (h >= a.H) return;
  // the last sequence whose first block is at or before this one
  int b = 0;
  if (!a.seq.cu) {
    b = (int)(blockIdx.x / (unsigned)((a.seq.T + SB_L - 1) / SB_L));
  } else {
    int hi = a.seq.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (ssm_first_block(a.seq, mid) <= (long long)blockIdx.x) b = mid; else hi = mid;
    }
  }
  const long long seq0 = a.seq.start(b), seq1 = a.seq.end(b);
  const long long row0 = seq0 + ((long long)blockIdx.x - ssm_first_block(a.seq, b)) * SB_L;
  if (row0 < seq0 || row0 >= seq1) return;
  const __nv_bfloat16* dp = static_cast<const __nv_bfloat16*>(a.dt) + h;
  // finite where A is: a step of size 0 times infinity would be NaN
  const float A2 = fmaxf(a.A[h] * SB_LOG2E, -FLT_MAX), bias = a.dt_bias ? a.dt_bias[h] : 0.0f;
  float raw[4];
  bool live[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long r = row0 + 4 * lane + i;
    live[i] = r < seq1;
    raw[i] = live[i] ? __bfloat162float(dp[r * a.dt_stride]) : 0.0f;
  }
  SsmSums o;
  ssm_sums(raw, live, bias, A2, a.softplus, o);
  float out[4], w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out[i] = o.d[i] * exp2f(o.tail[i]);
    w[i] = o.d[i] * exp2f(o.tail[i] + o.later);
  }
  SsmPrep* pr = prep + (size_t)blockIdx.x * a.H + h;
  reinterpret_cast<float4*>(pr->d)[lane] = make_float4(o.d[0], o.d[1], o.d[2], o.d[3]);
  reinterpret_cast<float4*>(pr->in)[lane] = make_float4(o.in[0], o.in[1], o.in[2], o.in[3]);
  reinterpret_cast<float4*>(pr->out)[lane] = make_float4(out[0], out[1], out[2], out[3]);
  reinterpret_cast<float4*>(pr->w)[lane] = make_float4(w[0], w[1], w[2], w[3]);
  if (lane < 4)
    pr->run[lane] = lane == 0 ? o.run[0] : lane == 1 ? o.run[1] : lane == 2 ? o.run[2] : o.run[3];
}

// Eight pairs of values times w, in three bf16 parts that add up to the fp32 products exactly:
// each part is the next eight bits of what is left (cut, not rounded: the upper half of the word
// as it stands, two fewer instructions a pair than a conversion and its way back).
__device__ __forceinline__ void ssm_parts(const uint4& va, const uint4& vb, float w,
                                          uint32_t p[3][8]) {
  const float2 w2 = make_float2(w, w);
  const uint32_t vw[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
  auto upper = [](float2 x) {  // the upper halves of both words
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
  };
  auto rest = [](float2 x) {
    return sub2(x, make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                               __uint_as_float(__float_as_uint(x.y) & 0xffff0000u)));
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float2 x = mul2(unpack_bf16(vw[j]), w2);
    p[0][j] = upper(x);
    x = rest(x);
    p[1][j] = upper(x);
    x = rest(x);
    p[2][j] = upper(x);
  }
}
__device__ __forceinline__ void ssm_store_parts(uint8_t* place, uint32_t o0, uint32_t o1,
                                                const uint32_t p[3][8]) {
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    *reinterpret_cast<uint4*>(place + part * SB_WPART + o0) =
        make_uint4(p[part][0], p[part][1], p[part][2], p[part][3]);
    *reinterpret_cast<uint4*>(place + part * SB_WPART + o1) =
        make_uint4(p[part][4], p[part][5], p[part][6], p[part][7]);
  }
}

// One piece of the scan's work: a segment of a sequence, a head and 64 of its columns.  A CTA
// walks every gridDim.x-th piece.
struct SsmPiece {
  int place, part;  // place in the list of work items, and part: head + H x tile
  int slot, b, seq0, seq1, row0, row1, h, p0, nb;  // slot: of its state; nb blocks
  __device__ __forceinline__ void begin(const SsmBlockArgs& ba) {
    const int parts = ba.a.H * ba.ptiles;
    place = (int)blockIdx.x / parts;
    part = (int)blockIdx.x - place * parts;
  }
  // The piece at hand; false past the last.
  __device__ __forceinline__ bool get(const SsmBlockArgs& ba) {
    if (place >= ba.sp.items) return false;
    const int4 at = __ldg(ba.items + place);
    const int H = ba.a.H;
    h = part;
    p0 = 0;
    while (h >= H) {  // at most three times: d_v <= 256
      h -= H;
      p0 += SB_P;
    }
    slot = __ldg(reinterpret_cast<const int*>(ba.items + ba.sp.items) + place);
    b = at.x;
    seq0 = at.y;
    seq1 = at.z;
    row0 = at.w;
    const int left = seq1 - row0, most = (int)ba.sp.seg_rows;
    row1 = row0 + (left < most ? left : most);
    nb = (row1 - row0 + SB_L - 1) / SB_L;
    return b >= 0;
  }
  __device__ __forceinline__ void advance(const SsmBlockArgs& ba) {
    place += ba.step_items;
    part += ba.step_parts;
    const int parts = ba.a.H * ba.ptiles;
    if (part >= parts) {
      part -= parts;
      ++place;
    }
  }
};

__global__ void __launch_bounds__(SB_THREADS, 1)
    ssm_block_kernel(const __grid_constant__ SsmBlockArgs ba) {
  extern __shared__ uint8_t smem_raw[];
  const SsmArgs& a = ba.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - smem_addr(smem_raw));
  const uint32_t bars = base + SB_BARS;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  if (blockIdx.x == 0) a.seq.check();
  const int npanels = a.N > 64 ? 2 : 1, nk = (a.N + 15) / 16;

  if (warp == 0) tmem_alloc(base + SB_TMEM_PTR, 512);
  if (tid == 32) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_KFULL + i), 1);
      mbar_init(bar(BAR_KFREE + i), 2);
      mbar_init(bar(BAR_WREADY + i), 4);
      mbar_init(bar(BAR_WFREE + i), 1);
      mbar_init(bar(BAR_S + i), 1);
      mbar_init(bar(BAR_P + i), 4);
      mbar_init(bar(BAR_Y + i), 1);
      mbar_init(bar(BAR_Y2 + i), 1);
      mbar_init(bar(BAR_YFREE + i), 4);
    }
    mbar_init(bar(BAR_DM), 1);
    mbar_init(bar(BAR_DMFREE), 4);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(BAR_PREP + i), 1);
      mbar_init(bar(BAR_PREPFREE + i), 16);
      mbar_init(bar(BAR_VFULL + i), 1);
      mbar_init(bar(BAR_VFREE + i), 4);
    }
    mbar_init(bar(BAR_QFULL), 1);
    mbar_init(bar(BAR_QFREE), 1);
    mbar_init(bar(BAR_HREADY), 4);
    mbar_init(bar(BAR_HFREE), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(BAR_DRAIN + i), 1);
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
  // use: how many times the barrier completed before; by a whole warp, or by a lane of its own
  auto wait = [&](int i, int use) { return mbar_wait_warp(bar(i), (uint32_t)use & 1u); };
  auto wait_lane = [&](int i, int use) { return mbar_wait(bar(i), (uint32_t)use & 1u); };
  auto prep = [&](int c) {
    return reinterpret_cast<SsmPrep*>(sm + SB_PREP + (c & 3) * sizeof(SsmPrep));
  };

  // The CTA's work: every gridDim.x-th of the (sequence, segment, head, tile) pieces.  Each group
  // walks them on its own; u0 counts the blocks of the pieces before, for the barriers' phases.
  // With a CTA per piece a short piece cost more in filling the pipeline than in its blocks.
  SsmPiece w;
  bool ok = true;
  int u0 = 0;
  w.begin(ba);

  if (warp < 4) {
    // ------------------------------------------------ P: row t = tid
    const int t = tid;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba))
      for (int c = u0; c < u0 + w.nb; ++c) {
        const uint32_t stage = c & 1;
        ok = wait(BAR_PREP + (c & 3), c >> 2) && wait(BAR_S + stage, c >> 1);
        if (!ok) break;
        tc_fence_after();
        const SsmPrep& pr = *prep(c);
        const uint32_t sbuf = tm + TM_S + stage * 128 + lanes;
        const float in_t = pr.in[t];
        float e = in_t;  // log2 decay from the end of run j up to t, j from warp - 1 down
        float to[3];
#pragma unroll
        for (int j = 2; j >= 0; --j) {
          to[j] = 0.0f;
          if (j < warp) {
            to[j] = fast_exp2(e);
            e += pr.run[j];
          }
        }
        // 16 columns at a time, the next 16 on their way from tensor memory; the row's warp needs
        // the runs up to its own
        const int groups = 2 * warp + 2;
        float next[16];
        tmem_ld16(sbuf, next);
#pragma unroll 1
        for (int grp = 0; grp < groups; ++grp) {
          float s[16];
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = next[i];
          if (grp + 1 < groups) tmem_ld16(sbuf + 16 * (grp + 1), next);
          float2 pw[8];
          if (grp < 2 * warp) {
            const float f = grp < 2 ? to[0] : grp < 4 ? to[1] : to[2];
            const float2 f2 = make_float2(f, f);
            const float4* o4 = reinterpret_cast<const float4*>(&pr.out[16 * grp]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 o = o4[i];
              pw[2 * i] = mul2(mul2(make_float2(o.x, o.y), f2),
                               make_float2(s[4 * i], s[4 * i + 1]));
              pw[2 * i + 1] = mul2(mul2(make_float2(o.z, o.w), f2),
                                   make_float2(s[4 * i + 2], s[4 * i + 3]));
            }
          } else {
            const float4* in4 = reinterpret_cast<const float4*>(&pr.in[16 * grp]);
            const float4* d4 = reinterpret_cast<const float4*>(&pr.d[16 * grp]);
            const float2 t2 = make_float2(in_t, in_t);
            const int own = t - 16 * grp;  // the row's own column among these
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 in = in4[i], d = d4[i];
              const float2 e0 = sub2(t2, make_float2(in.x, in.y)),
                           e1 = sub2(t2, make_float2(in.z, in.w));
              float2 u = mul2(mul2(make_float2(s[4 * i], s[4 * i + 1]), make_float2(d.x, d.y)),
                              make_float2(fast_exp2(e0.x), fast_exp2(e0.y)));
              float2 v = mul2(mul2(make_float2(s[4 * i + 2], s[4 * i + 3]), make_float2(d.z, d.w)),
                              make_float2(fast_exp2(e1.x), fast_exp2(e1.y)));
              if (4 * i > own) u.x = 0.0f;
              if (4 * i + 1 > own) u.y = 0.0f;
              if (4 * i + 2 > own) v.x = 0.0f;
              if (4 * i + 3 > own) v.y = 0.0f;
              pw[2 * i] = u;
              pw[2 * i + 1] = v;
            }
          }
          // both parts in the place of the columns of S that they come from
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            pk[i] = pack_bf16(pw[i].x, pw[i].y);
            const float2 rest = sub2(pw[i], unpack_bf16(pk[i]));
            pk[8 + i] = pack_bf16(rest.x, rest.y);
          }
          tmem_st16(sbuf + 16 * grp, pk);
        }
        {
          const uint32_t none[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          for (int grp = groups; grp < 8; ++grp) tmem_st16(sbuf + 16 * grp, none);
        }
        tmem_wait_st();
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(BAR_P + stage));
          mbar_arrive(bar(BAR_PREPFREE + (c & 3)));
        }
      }
  } else if (warp < 8) {
    // ------------------------------------------------ Y: row t = tid - 128
    const int t = tid - 128, quad = warp - 4;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba)) {
      const float D = a.D ? a.D[w.h] : 0.0f;
      const float2 D2 = make_float2(D, D);
      const int pn = a.P - w.p0 < SB_P ? a.P - w.p0 : SB_P;  // columns that exist
      __nv_bfloat16* const yp = static_cast<__nv_bfloat16*>(a.y) + (size_t)w.h * a.P + w.p0;
      const __nv_bfloat16* const zp =
          a.gate ? static_cast<const __nv_bfloat16*>(a.gate) + (size_t)w.h * a.P + w.p0 : nullptr;
      // whole sectors where rows start on them and hold a multiple of 16 values
      const uintptr_t bases = reinterpret_cast<uintptr_t>(yp) | reinterpret_cast<uintptr_t>(zp);
      const bool sectors = a.P % 16 == 0 && a.gate_stride % 16 == 0 && (bases & 31) == 0;
      for (int c = u0; c < u0 + w.nb; ++c) {
        const uint32_t stage = c & 1;
        const int row = w.row0 + (c - u0) * SB_L + t;
        const bool live = row < w.row1;
        const __nv_bfloat16* const zrow = zp + (long long)row * a.gate_stride;
        __nv_bfloat16* const yrow = yp + (size_t)row * a.H * a.P;
        ok = wait(BAR_PREP + (c & 3), c >> 2) && wait(BAR_VFULL + (c & 3), c >> 2);
        if (!ok) break;
        float decay;  // from the block's start up to t
        {
          // used behind the release below: volatile, so that no read is put off or made again
          const volatile SsmPrep& pr = *prep(c);
          float e = pr.in[t];
#pragma unroll
          for (int j = 0; j < 3; ++j)
            if (j < quad) e += pr.run[j];
          decay = fast_exp2(e);
        }
        const float2 f2 = make_float2(decay, decay);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PREPFREE + (c & 3)));
        uint32_t z[8];
        auto load_z = [&](int part) {
          if (!zp || !live || 16 * part >= pn) return;
          if (sectors) {
            load_sector(zrow + 16 * part, z);
          } else {
            *reinterpret_cast<uint4*>(z) = *reinterpret_cast<const uint4*>(zrow + 16 * part);
            if (16 * part + 8 < pn)
              *reinterpret_cast<uint4*>(z + 4) =
                  *reinterpret_cast<const uint4*>(zrow + 16 * part + 8);
          }
        };
        load_z(0);  // on its way while the products finish
        ok = wait(BAR_Y2 + stage, c >> 1) && wait(BAR_Y + stage, c >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint8_t* vtile = sm + SB_V + (c & 3) * SB_PANEL;
        const uint32_t ybuf = tm + TM_Y1 + lanes, y2buf = tm + TM_Y2 + stage * 64 + lanes;
#pragma unroll 1
        for (int part = 0; part < 4; ++part) {
          float y1[16], y2[16];
          tmem_ld16(ybuf + 16 * part, y1);
          tmem_ld16(y2buf + 16 * part, y2);
          const uint4 va = *reinterpret_cast<const uint4*>(vtile + tile_offset(t, 2 * part)),
                      vb = *reinterpret_cast<const uint4*>(vtile + tile_offset(t, 2 * part + 1));
          const uint32_t vw[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
          float2 o[8];
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[j] = fma2(D2, unpack_bf16(vw[j]),
                        fma2(f2, make_float2(y2[2 * j], y2[2 * j + 1]),
                             make_float2(y1[2 * j], y1[2 * j + 1])));
          }
          if (zp) {
            float2 g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = unpack_bf16(z[j]);
            pair_act<__nv_bfloat16, 8>(g, a.act);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = mul2(o[j], g[j]);
            if (part < 3) load_z(part + 1);
          }
          uint32_t out[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) out[j] = pack_bf16(o[j].x, o[j].y);
          if (live && 16 * part < pn) {
            if (sectors) {
              store_sector(yrow + 16 * part, out);
            } else {
              *reinterpret_cast<uint4*>(yrow + 16 * part) =
                  make_uint4(out[0], out[1], out[2], out[3]);
              if (16 * part + 8 < pn)
                *reinterpret_cast<uint4*>(yrow + 16 * part + 8) =
                    make_uint4(out[4], out[5], out[6], out[7]);
            }
          }
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(BAR_YFREE + stage));
          mbar_arrive(bar(BAR_VFREE + (c & 3)));
        }
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------ H: row n = tid - 256
    const int n = tid - 256;
    const uint32_t lanes = (uint32_t)((warp - 8) * 32) << 16;
    float2 st[SB_P / 2];
    // two bf16 parts of eight of the row's values, as a chunk of the B operand of Y2
    auto publish = [&](int ch) {
      uint32_t u[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 x = st[4 * ch + j];
        u[j] = pack_bf16(x.x, x.y);
        const float2 r = sub2(x, unpack_bf16(u[j]));
        v[j] = pack_bf16(r.x, r.y);
      }
      uint8_t* place = sm + SB_H + tile_offset(n, ch);
      *reinterpret_cast<uint4*>(place) = make_uint4(u[0], u[1], u[2], u[3]);
      *reinterpret_cast<uint4*>(place + SB_PANEL) = make_uint4(v[0], v[1], v[2], v[3]);
    };
    auto published = [&]() {
      fence_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_HREADY));
    };
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba)) {
      const int pn = a.P - w.p0 < SB_P ? a.P - w.p0 : SB_P;
      float* const mrow = a.M + (((size_t)w.b * a.H + w.h) * a.N + n) * a.P + w.p0;
      const bool split = w.seq1 - w.seq0 > ba.sp.seg_rows;
      const float* const from =
          split ? ba.sp.starts + (((size_t)w.slot * a.H + w.h) * a.N + n) * a.P + w.p0 : mrow;
#pragma unroll
      for (int i = 0; i < SB_P; i += 4) {
        float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
        if ((split || !a.from_zero) && n < a.N && i < pn)
          m = *reinterpret_cast<const float4*>(from + i);
        st[i / 2] = make_float2(m.x, m.y);
        st[i / 2 + 1] = make_float2(m.z, m.w);
      }
      if (w.nb > 0) {  // the state before the piece; the last block before has read its own
        ok = u0 == 0 || wait(BAR_HFREE, u0 - 1);
        if (!ok) break;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) publish(ch);
        published();
      }
      for (int c = u0; c < u0 + w.nb; ++c) {
        ok = wait(BAR_PREP + (c & 3), c >> 2);
        if (!ok) break;
        const volatile SsmPrep& pr = *prep(c);  // as in group Y
        const float keep = exp2f((pr.run[0] + pr.run[1]) + (pr.run[2] + pr.run[3]));
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_PREPFREE + (c & 3)));
        ok = wait(BAR_DM, c);
        if (!ok) break;
        tc_fence_after();
        const uint32_t dm = tm + TM_DM + lanes;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          float r[16];
          tmem_ld16(dm + 16 * part, r);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            // one by one: as pairs the state would be held twice, and spilled
            st[8 * part + i] = make_float2(fmaf(st[8 * part + i].x, keep, r[2 * i]),
                                           fmaf(st[8 * part + i].y, keep, r[2 * i + 1]));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_DMFREE));
        if (c + 1 < u0 + w.nb) {
          ok = wait(BAR_HFREE, c);
          if (!ok) break;
#pragma unroll
          for (int ch = 0; ch < 8; ++ch) publish(ch);
          published();
        }
      }
      if (ok && w.row1 == w.seq1 && n < a.N) {
#pragma unroll
        for (int i = 0; i < SB_P; i += 4)
          if (i < pn)
            *reinterpret_cast<float4*>(mrow + i) =
                make_float4(st[i / 2].x, st[i / 2].y, st[i / 2 + 1].x, st[i / 2 + 1].y);
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------ W: three bf16 parts of w o v
    const int i0 = tid - 384, rq = i0 >> 2;  // row in the quarter, and 16 of its values
    const uint32_t o0 = tile_offset(rq, 2 * (i0 & 3)), o1 = tile_offset(rq, 2 * (i0 & 3) + 1);
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba))
      for (int c = u0; c < u0 + w.nb; ++c) {
        const int stage = c & 1;
        ok = wait(BAR_PREP + (c & 3), c >> 2) && wait(BAR_VFULL + (c & 3), c >> 2);
        if (!ok) break;
        uint8_t* vtile = sm + SB_V + (c & 3) * SB_PANEL;
        const float* weights = prep(c)->w;
        const int left = w.row1 - (w.row0 + (c - u0) * SB_L);
        if (left < SB_L) {
          // rows behind the segment's end, whatever they hold, become zeros
          ok = wait(BAR_KFULL + stage, c >> 1);
          if (!ok) break;
          for (int t = rq; t < SB_L; t += 32) {
            if (t < left) continue;
            for (int i = 0; i < 2; ++i) {
              const uint32_t o = (i ? o1 : o0) + (t - rq) * 128;
              *reinterpret_cast<uint4*>(vtile + o) = make_uint4(0, 0, 0, 0);
              for (int pl = 0; pl < npanels; ++pl)
                *reinterpret_cast<uint4*>(sm + SB_K + (2 * stage + pl) * SB_PANEL + o) =
                    make_uint4(0, 0, 0, 0);
            }
          }
        }
        uint4 na = *reinterpret_cast<const uint4*>(vtile + o0),
              nb4 = *reinterpret_cast<const uint4*>(vtile + o1);
        float nw = weights[rq];
#pragma unroll 1
        for (int qd = 0; qd < 4; ++qd) {
          const int use = 4 * c + qd, buf = qd & 1;
          uint32_t p[3][8];
          ssm_parts(na, nb4, nw, p);
          if (qd < 3) {
            na = *reinterpret_cast<const uint4*>(vtile + 4096 * (qd + 1) + o0);
            nb4 = *reinterpret_cast<const uint4*>(vtile + 4096 * (qd + 1) + o1);
            nw = weights[32 * (qd + 1) + rq];
          }
          ok = use < 2 || wait(BAR_WFREE + buf, (use >> 1) - 1);
          if (!ok) break;
          ssm_store_parts(sm + SB_W + buf * 3 * SB_WPART, o0, o1, p);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_WREADY + buf));
        }
        if (!ok) break;
        if (lane == 0) mbar_arrive(bar(BAR_PREPFREE + (c & 3)));
      }
  } else if (warp == 18) {
    // ------------------------------------------------ products Y2 of a block and S of the next
    constexpr uint32_t dS = mma_desc(128, 128, 0, 0), dY2 = mma_desc(128, 64, 0, 1);
    const uint32_t q0 = tile_desc(base + SB_Q), k0 = tile_desc(base + SB_K),
                   h0 = tile_desc(base + SB_H);
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba))
      for (int c = u0 - 1; c < u0 + w.nb; ++c) {
        if (c >= u0) {
          const uint32_t stage = c & 1;
          // the block's buffer of Y2 is free since its S was issued: group Y reads both
          ok = wait(BAR_HREADY, c);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t o = ((i >> 2 & 1) * SB_PANEL + (i & 3) * 32) >> 4;
              if ((i & 7) < nk)
                mma_ss(tm + TM_Y2 + stage * 64, q0 + o,
                       h0 + (((i >> 3) * SB_PANEL + (i & 7) * 2048) >> 4), dY2, i > 0);
            }
            mma_commit(bar(BAR_Y2 + stage));
            mma_commit(bar(BAR_HFREE));
            mma_commit(bar(BAR_QFREE));
          }
          __syncwarp();
        }
        const int e = c + 1;
        if (e < u0 + w.nb) {
          const uint32_t stage = e & 1;
          ok = wait(BAR_QFULL, e) && wait(BAR_KFULL + stage, e >> 1) &&
               (e < 2 || wait(BAR_YFREE + stage, (e >> 1) - 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t k = k0 + stage * (2 * SB_PANEL >> 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t o = ((i >> 2) * SB_PANEL + (i & 3) * 32) >> 4;
              if (i < nk) mma_ss(tm + TM_S + stage * 128, q0 + o, k + o, dS, i > 0);
            }
            mma_commit(bar(BAR_S + stage));
            mma_commit(bar(BAR_KFREE + stage));
          }
          __syncwarp();
        }
      }
    if (elect_one()) mma_commit(bar(BAR_DRAIN));
    __syncwarp();
    ok = mbar_wait_warp(bar(BAR_DRAIN), 0) && ok;
  } else if (warp == 17) {
    // ------------------------------------------------ products dM, part onto part, and Y1
    constexpr uint32_t dM = mma_desc(128, 64, 1, 1), dY1 = mma_desc(128, 64, 0, 1);
    const uint32_t k0 = tile_desc(base + SB_K, SB_PANEL), w0 = tile_desc(base + SB_W),
                   v0 = tile_desc(base + SB_V);
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba))
      for (int c = u0; c < u0 + w.nb && ok; ++c) {
        const uint32_t stage = c & 1, k = k0 + stage * (2 * SB_PANEL >> 4);
        ok = wait(BAR_KFULL + stage, c >> 1) && (c < 1 || wait(BAR_DMFREE, c - 1));
        for (int qd = 0; qd < 4 && ok; ++qd) {
          const uint32_t use = 4 * c + qd, buf = use & 1;
          ok = wait(BAR_WREADY + buf, use >> 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t kq = k + qd * (4096 >> 4), wb = w0 + buf * (3 * SB_WPART >> 4);
#pragma unroll
            for (int i = 0; i < 6; ++i)
              mma_ss(tm + TM_DM, kq + (i & 1) * (2048 >> 4),
                     wb + (((i >> 1) * SB_WPART + (i & 1) * 2048) >> 4), dM, qd + i > 0);
            mma_commit(bar(BAR_WFREE + buf));
            if (qd == 3) {
              mma_commit(bar(BAR_DM));
              mma_commit(bar(BAR_KFREE + stage));
            }
          }
          __syncwarp();
        }
        // the last quarter is also the sign that v's rows behind the end are zeros
        ok = ok && wait(BAR_VFULL + (c & 3), c >> 2) && wait(BAR_P + stage, c >> 1) &&
             (c < 1 || wait(BAR_YFREE + (stage ^ 1), (c - 1) >> 1));  // Y1 of c - 1 is read
        if (!ok) break;
        tc_fence_after();
        const uint32_t slot = c & 3;
        if (elect_one()) {
          const uint32_t v = v0 + slot * (SB_PANEL >> 4), s = tm + TM_S + stage * 128;
#pragma unroll
          for (int i = 0; i < SB_L / 8; ++i)
            mma_ts(tm + TM_Y1, s + 8 * i, v + (i >> 1) * (2048 >> 4), dY1, i > 0);
          mma_commit(bar(BAR_Y + stage));
        }
        __syncwarp();
      }
    if (elect_one()) mma_commit(bar(BAR_DRAIN + 1));
    __syncwarp();
    ok = mbar_wait_warp(bar(BAR_DRAIN + 1), 0) && ok;
  } else if (warp == 19) {
    // ------------------------------------------------ loads of k and q
    int kc = 0, qc = 0;  // blocks whose load is issued
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba)) {
      if (lane == 0) {
        const int g = w.h / (a.H / a.G);
        for (int c = u0; c < u0 + w.nb; ++c) {
          const uint32_t stage = c & 1;
          const int r = w.row0 + (c - u0) * SB_L;
          ok = c < 2 || wait_lane(BAR_KFREE + stage, (c >> 1) - 1);
          if (!ok) break;
          mbar_expect(bar(BAR_KFULL + stage), npanels * SB_PANEL);
          for (int pl = 0; pl < npanels; ++pl)
            tma_load_3d(base + SB_K + (2 * stage + pl) * SB_PANEL, &ba.mk, 64 * pl, g, r,
                        bar(BAR_KFULL + stage));
          kc = c + 1;
          ok = c < 1 || wait_lane(BAR_QFREE, c - 1);
          if (!ok) break;
          mbar_expect(bar(BAR_QFULL), npanels * SB_PANEL);
          for (int pl = 0; pl < npanels; ++pl)
            tma_load_3d(base + SB_Q + pl * SB_PANEL, &ba.mq, 64 * pl, g, r, bar(BAR_QFULL));
          qc = c + 1;
        }
      }
      ok = __shfl_sync(FULL_MASK, (int)ok, 0);
    }
    if (!ok && lane == 0) {
      // loads in flight land before the block's memory is given up (each wait limited)
      if (qc) mbar_wait(bar(BAR_QFULL), (uint32_t)(qc - 1) & 1u);
      for (int c = kc > 2 ? kc - 2 : 0; c < kc; ++c)
        mbar_wait(bar(BAR_KFULL + (c & 1)), (uint32_t)(c >> 1) & 1u);
    }
  } else {
    // ------------------------------------------------ loads of v and the blocks' sums
    int pc = 0, vc = 0;  // blocks whose load is issued
    for (; ok && w.get(ba); u0 += w.nb, w.advance(ba)) {
      // what groups H and Y read on their own comes into the L2 ahead of them: the state before
      // the piece, and block by block the gate
      const bool split = w.seq1 - w.seq0 > ba.sp.seg_rows;
      if (w.nb > 0 && (split || !a.from_zero)) {
        const float* m = (split ? ba.sp.starts + ((size_t)w.slot * a.H + w.h) * a.N * a.P
                                : a.M + ((size_t)w.b * a.H + w.h) * a.N * a.P) + w.p0;
        const int bytes = 4 * (a.P - w.p0 < SB_P ? a.P - w.p0 : SB_P);
        for (int n = lane; n < a.N; n += 32)
          for (int o = 0; o < bytes; o += 128)
            prefetch_l2(reinterpret_cast<const char*>(m + (size_t)n * a.P) + o);
      }
      if (lane == 0) {
        const SsmPrep* from =
            ba.prep + (ssm_first_block(a.seq, w.b) + (w.row0 - w.seq0) / SB_L) * a.H + w.h;
        for (int c = u0; c < u0 + w.nb; ++c) {
          const uint32_t slot = c & 3;
          const int r = w.row0 + (c - u0) * SB_L;
          ok = c < 4 || wait_lane(BAR_PREPFREE + slot, (c >> 2) - 1);
          if (!ok) break;
          mbar_expect(bar(BAR_PREP + slot), sizeof(SsmPrep));
          bulk_load(base + SB_PREP + slot * sizeof(SsmPrep), from + (size_t)(c - u0) * a.H,
                    sizeof(SsmPrep), bar(BAR_PREP + slot));
          pc = c + 1;
          ok = c < 4 || wait_lane(BAR_VFREE + slot, (c >> 2) - 1);
          if (!ok) break;
          mbar_expect(bar(BAR_VFULL + slot), SB_PANEL);
          tma_load_3d(base + SB_V + slot * SB_PANEL, &ba.mv, w.p0, w.h, r, bar(BAR_VFULL + slot));
          if (a.gate) tma_prefetch_3d(&ba.mz, w.p0, w.h, r);
          vc = c + 1;
        }
      }
      ok = __shfl_sync(FULL_MASK, (int)ok, 0);
    }
    if (!ok && lane == 0) {
      for (int c = pc > 4 ? pc - 4 : 0; c < pc; ++c)
        mbar_wait(bar(BAR_PREP + (c & 3)), (uint32_t)(c >> 2) & 1u);
      for (int c = vc > 4 ? vc - 4 : 0; c < vc; ++c)
        mbar_wait(bar(BAR_VFULL + (c & 3)), (uint32_t)(c >> 2) & 1u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tm, 512);
  if (!ok) record_status(STATUS_TIMEOUT);
}

// ------------------------------------------------------------------------ split sequences
// The first pass of a split (SsmSplit): each segment's own contribution, dM over all its tokens
// at once; one product, no state to carry.
//
// A segment's contribution is summed from its last block to its first, so that every token's
// weight, its decay up to the segment's end, is known when its block is read, and all blocks
// accumulate in the same tensor memory.
//   warps 0-7  w o v in parts, two groups at alternate quarters
//   warp 8 products, warp 9 loads
constexpr int SG_THREADS = 320;
constexpr int SG_STAGES = 3;
constexpr uint32_t SG_K = 0;                                // stages x 2 panels
constexpr uint32_t SG_V = SG_K + SG_STAGES * 2 * SB_PANEL;  // stages
constexpr uint32_t SG_W = SG_V + SG_STAGES * SB_PANEL;      // 4 quarters x 3 parts
constexpr uint32_t SG_PREP = SG_W + 12 * SB_WPART;          // stages x SsmPrep
constexpr uint32_t SG_BARS = SG_PREP + SG_STAGES * sizeof(SsmPrep);
enum { GB_FULL = 0, GB_FREE = 3, GB_WREADY = 6, GB_WFREE = 10, GB_DONE = 14, GB_READ, GB_DRAIN,
       GB_COUNT };
constexpr uint32_t SG_TMEM_PTR = SG_BARS + 20 * 8;
constexpr uint32_t SG_SMEM = SG_TMEM_PTR + 32 + 1024;

__global__ void __launch_bounds__(SG_THREADS, 1)
    ssm_segment_kernel(const __grid_constant__ SsmBlockArgs ba) {
  extern __shared__ uint8_t smem_raw[];
  const SsmArgs& a = ba.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const sm = smem_raw + (base - smem_addr(smem_raw));
  const uint32_t bars = base + SG_BARS;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  const int nb = (int)(ba.sp.seg_rows / SB_L);  // blocks of a segment that another follows
  const int npanels = a.N > 64 ? 2 : 1;

  if (warp == 0) tmem_alloc(base + SG_TMEM_PTR, 128);
  if (tid == 32) {
    for (int i = 0; i < SG_STAGES; ++i) {
      mbar_init(bar(GB_FULL + i), 1);
      mbar_init(bar(GB_FREE + i), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(GB_WREADY + i), 4);
      mbar_init(bar(GB_WFREE + i), 1);
    }
    mbar_init(bar(GB_DONE), 1);
    mbar_init(bar(GB_READ), 4);
    mbar_init(bar(GB_DRAIN), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (npanels == 1) {
    uint4* z = reinterpret_cast<uint4*>(sm + SG_K);
    for (int i = tid; i < SG_STAGES * (int)SB_PANEL / 16; i += SG_THREADS) {
      const int stage = i / (SB_PANEL / 16), j = i % (SB_PANEL / 16);
      z[(2 * stage + 1) * (SB_PANEL / 16) + j] = make_uint4(0, 0, 0, 0);
    }
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *reinterpret_cast<volatile uint32_t*>(sm + SG_TMEM_PTR);
  auto wait = [&](int i, int use) { return mbar_wait_warp(bar(i), (uint32_t)use & 1u); };
  auto wait_lane = [&](int i, int use) { return mbar_wait(bar(i), (uint32_t)use & 1u); };
  auto prep = [&](int stage) {
    return reinterpret_cast<const SsmPrep*>(sm + SG_PREP + stage * sizeof(SsmPrep));
  };

  // The pieces of this CTA that a segment follows: each group walks them on its own, `turn` of
  // them before; their blocks are counted on for the barriers' phases.
  SsmPiece w;
  bool ok = true;
  int turn = -1;
  w.begin(ba);
  auto next_piece = [&]() {
    if (turn >= 0) w.advance(ba);
    ++turn;
    for (; ok && w.get(ba); w.advance(ba))
      if (w.row1 < w.seq1 && w.slot + 1 < ba.sp.slots) return true;
    return false;
  };

  if (warp < 8) {
    const int grp = warp >> 2, i0 = tid & 127, rq = i0 >> 2;
    const uint32_t o0 = tile_offset(rq, 2 * (i0 & 3)), o1 = tile_offset(rq, 2 * (i0 & 3) + 1);
    int stage = 0, round = 0;
    while (next_piece()) {
      const int u0 = turn * nb;
      float carry = 0.0f;  // log2 decay of the blocks behind
      for (int c = 0; c < nb && ok; ++c) {
        ok = wait(GB_FULL + stage, round);
        if (!ok) break;
        const uint8_t* vtile = sm + SG_V + stage * SB_PANEL;
        const SsmPrep& pr = *prep(stage);
        const float f = exp2f(carry);
        const volatile float* run = pr.run;  // used behind the stage's release, too
        carry += (run[0] + run[1]) + (run[2] + run[3]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int qd = 2 * i + grp;  // the group's buffers: qd
          uint32_t p[3][8];
          ssm_parts(*reinterpret_cast<const uint4*>(vtile + 4096 * qd + o0),
                    *reinterpret_cast<const uint4*>(vtile + 4096 * qd + o1),
                    pr.w[32 * qd + rq] * f, p);
          ok = ok && (u0 + c == 0 || wait(GB_WFREE + qd, u0 + c - 1));
          ssm_store_parts(sm + SG_W + qd * 3 * SB_WPART, o0, o1, p);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(GB_WREADY + qd));
        }
        if (++stage == SG_STAGES) {
          stage = 0;
          ++round;
        }
      }
      if (tid == 0 && w.p0 == 0) ba.sp.decays[(size_t)w.slot * a.H + w.h] = exp2f(carry);
      if (warp < 4 && ok) {
        ok = wait(GB_DONE, turn);
        if (!ok) break;
        tc_fence_after();
        const int n = tid, pn = a.P - w.p0 < SB_P ? a.P - w.p0 : SB_P;
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        // the state before the next segment gets this one's contribution
        float* to = ba.sp.starts + (((size_t)(w.slot + 1) * a.H + w.h) * a.N + n) * a.P + w.p0;
#pragma unroll
        for (int part = 0; part < 4; ++part) {
          float r1[16], r2[16];
          tmem_ld16(tm + 16 * part + lanes, r1);
          tmem_ld16(tm + 64 + 16 * part + lanes, r2);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            if (n < a.N && 16 * part + i < pn)
              *reinterpret_cast<float4*>(to + 16 * part + i) =
                  make_float4(r1[i] + r2[i], r1[i + 1] + r2[i + 1], r1[i + 2] + r2[i + 2],
                              r1[i + 3] + r2[i + 3]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(GB_READ));
      }
    }
  } else if (warp == 8) {
    constexpr uint32_t dM = mma_desc(128, 128, 1, 1), dM2 = mma_desc(128, 64, 1, 1);
    const uint32_t k0 = tile_desc(base + SG_K, SB_PANEL), w0 = tile_desc(base + SG_W, SB_WPART);
    int stage = 0;
    while (next_piece()) {
      ok = turn == 0 || wait(GB_READ, turn - 1);  // the sums of the piece before are read
      for (int c = 0; c < nb && ok; ++c) {
        const uint32_t k = k0 + stage * (2 * SB_PANEL >> 4);
        for (int qd = 0; qd < 4 && ok; ++qd) {
          // the block's tiles are there: its weights were made
          ok = wait(GB_WREADY + qd, turn * nb + c);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t kq = k + qd * (4096 >> 4), wq = w0 + qd * (3 * SB_WPART >> 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              mma_ss(tm, kq + i * (2048 >> 4), wq + i * (2048 >> 4), dM, c + qd + i > 0);
              mma_ss(tm, kq + i * (2048 >> 4), wq + ((2 * SB_WPART + i * 2048) >> 4), dM2, true);
            }
            mma_commit(bar(GB_WFREE + qd));
            if (qd == 3) mma_commit(bar(GB_FREE + stage));
          }
          __syncwarp();
        }
        if (++stage == SG_STAGES) stage = 0;
      }
      if (ok && elect_one()) mma_commit(bar(GB_DONE));
      __syncwarp();
    }
    if (elect_one()) mma_commit(bar(GB_DRAIN));
    __syncwarp();
    ok = mbar_wait_warp(bar(GB_DRAIN), 0) && ok;
  } else {
    int stage = 0, round = 0, n = 0;
    while (next_piece()) {
      if (lane == 0) {
        const SsmPrep* from =
            ba.prep + (ssm_first_block(a.seq, w.b) + (w.row0 - w.seq0) / SB_L) * a.H + w.h;
        const int g = w.h / (a.H / a.G);
        for (int c = 0; c < nb; ++c) {
          const int at = nb - 1 - c, r = w.row0 + at * SB_L;
          ok = n < SG_STAGES || wait_lane(GB_FREE + stage, round - 1);
          if (!ok) break;
          mbar_expect(bar(GB_FULL + stage), (npanels + 1) * SB_PANEL + sizeof(SsmPrep));
          bulk_load(base + SG_PREP + stage * sizeof(SsmPrep), from + (size_t)at * a.H,
                    sizeof(SsmPrep), bar(GB_FULL + stage));
          tma_load_3d(base + SG_V + stage * SB_PANEL, &ba.mv, w.p0, w.h, r, bar(GB_FULL + stage));
          for (int pl = 0; pl < npanels; ++pl)
            tma_load_3d(base + SG_K + (2 * stage + pl) * SB_PANEL, &ba.mk, 64 * pl, g, r,
                        bar(GB_FULL + stage));
          ++n;
          if (++stage == SG_STAGES) {
            stage = 0;
            ++round;
          }
        }
      }
      ok = __shfl_sync(FULL_MASK, (int)ok, 0);
    }
    if (!ok && lane == 0)  // loads in flight land before the memory is given up
      for (int c = n > SG_STAGES ? n - SG_STAGES : 0; c < n; ++c)
        mbar_wait(bar(GB_FULL + c % SG_STAGES), (uint32_t)(c / SG_STAGES) & 1u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_free(tm, 128);
  if (!ok) record_status(STATUS_TIMEOUT);
}

}  // namespace sdm
