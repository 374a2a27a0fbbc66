// dense_api.cuh -- the C ABI of the dense-state layer's operators (declared in include/sdm.h):
// host-side validation and launches.  Part of sdm.cu, whose helpers it uses.
#pragma once

namespace {

// Whether [p, p + n) and [q, q + m) share a byte; null overlaps nothing.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && n && m && a < b + m && b < a + n;
}

struct Span {
  const void* p;
  size_t n;
};

// Whether `out` overlaps any of the spans.
bool overlaps_any(Span out, std::initializer_list<Span> in) {
  for (const Span& s : in)
    if (overlap(out.p, out.n, s.p, s.n)) return true;
  return false;
}

bool dtype_ok(int t) { return t == SDM_F32 || t == SDM_BF16; }
size_t dtype_size(int t) { return t == SDM_BF16 ? 2 : 4; }

// The pitch of rows of `width` values: 0 stands for contiguous; -1 for one that is not accepted.
long long pitch_of(int64_t stride, long long width, int dtype) {
  if (stride == 0) return width;
  const int mul = dtype == SDM_BF16 ? 8 : 4;
  return stride >= width && stride % mul == 0 && stride < (1LL << 40) ? stride : -1;
}

// Bytes spanned by `rows` rows of `width` values.
size_t span_bytes(long long rows, long long pitch, long long width, int dtype) {
  return rows > 0 ? ((size_t)(rows - 1) * pitch + width) * dtype_size(dtype) : 0;
}

bool conv_shape_ok(const sdm_conv_shape& s, bool step) {
  return s.B >= 1 && (step || s.T >= 0) && s.C >= 8 && s.C % 8 == 0 && s.C <= (1 << 24) &&
         dtype_ok(s.in_dtype) && pitch_of(s.x_stride, s.C, s.in_dtype) > 0;
}

template <typename T>
cudaError_t launch_conv(bool step, int K, unsigned blocks, cudaStream_t st, const ConvArgs& a) {
  const dim3 grid(blocks), block(128);
  if (step) {
    if (K == 2) return launch_pdl<true>(conv_step_kernel<T, 2>, grid, block, 0, st, a);
    if (K == 3) return launch_pdl<true>(conv_step_kernel<T, 3>, grid, block, 0, st, a);
    return launch_pdl<true>(conv_step_kernel<T, 4>, grid, block, 0, st, a);
  }
  if (K == 2) return launch_pdl<true>(conv_forward_kernel<T, 2>, grid, block, 0, st, a);
  if (K == 3) return launch_pdl<true>(conv_forward_kernel<T, 3>, grid, block, 0, st, a);
  return launch_pdl<true>(conv_forward_kernel<T, 4>, grid, block, 0, st, a);
}

sdm_status conv_run(const void* x, const float* w, const float* bias, void* state, int32_t init,
                    int32_t act, const int32_t* cu, void* y, const sdm_conv_shape& s,
                    void* stream, bool step) {
  if (!conv_shape_ok(s, step)) return SDM_ERR_INVALID_ARG;
  if (init != SDM_INIT_ZERO && init != SDM_CONTINUE) return SDM_ERR_INVALID_ARG;
  if (!act_ok(act) || !w || (init == SDM_CONTINUE && !state)) return SDM_ERR_INVALID_ARG;
  const long long R = step || cu ? (step ? s.B : s.T) : (long long)s.B * s.T;
  if (R > 0 && (!x || !y)) return SDM_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(bias) || !aligned16(state) || !aligned16(y) ||
      (reinterpret_cast<uintptr_t>(cu) & 3u))
    return SDM_ERR_INVALID_ARG;
  if (s.K < 2 || s.K > 4) return SDM_ERR_UNSUPPORTED;
  const long long pitch = pitch_of(s.x_stride, s.C, s.in_dtype);
  const size_t e = dtype_size(s.in_dtype);
  const Span sx{x, span_bytes(R, pitch, s.C, s.in_dtype)}, sw{w, (size_t)s.C * s.K * 4},
      sb{bias, (size_t)s.C * 4}, ss{state, (size_t)s.B * (s.K - 1) * s.C * e},
      sy{y, (size_t)R * s.C * e}, sc{cu, ((size_t)s.B + 1) * 4};
  if (overlaps_any(sy, {sx, sw, sb, ss, sc}) || overlaps_any(ss, {sx, sw, sb, sc}))
    return SDM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (R == 0) {  // every sequence is empty
    if (state && init == SDM_INIT_ZERO) SDM_CUDA_TRY(cudaMemsetAsync(state, 0, ss.n, st));
    return SDM_OK;
  }
  DeviceInfo* di;
  const sdm_status rc = device_info(&di);
  if (rc != SDM_OK) return rc;
  ConvArgs a = {};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.state = state;
  a.y = y;
  a.seq = SeqBounds{cu, s.B, step ? 1 : s.T, R};
  a.C = s.C;
  a.cv = s.C / 4;
  a.from_zero = init == SDM_INIT_ZERO;
  a.act = act;
  a.x_stride = pitch;
  // rows of a thread: enough threads for two waves of a full device, at least eight rows (a
  // thread's weights and the K - 1 rows before its own are read once for all of them), at most 32
  const long long threads = (long long)di->sms * 896 * 2;
  a.rows_per_thread = 8;
  while (a.rows_per_thread < 32 && R * a.cv > threads * a.rows_per_thread * 3 / 2)
    a.rows_per_thread *= 2;
  a.tiles = step ? s.B : (R + a.rows_per_thread - 1) / a.rows_per_thread;
  const long long blocks = (a.tiles * a.cv + 127) / 128;
  if (blocks > 2147483647LL) return SDM_ERR_UNSUPPORTED;
  ProfScope ps(SDM_KERNEL_CONV, st);
  if (s.in_dtype == SDM_BF16)
    SDM_CUDA_TRY(launch_conv<__nv_bfloat16>(step, s.K, (unsigned)blocks, st, a));
  else
    SDM_CUDA_TRY(launch_conv<float>(step, s.K, (unsigned)blocks, st, a));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SDM_OK;
}

// Fills everything but the pointers; false for a shape that is not accepted.
bool ssm_args(const sdm_ssm_shape& s, bool step, SsmArgs* a) {
  if (s.B < 1 || (!step && s.T < 0) || s.H < 1 || s.H > 65535 || s.G < 1 || s.H % s.G != 0)
    return false;
  if (s.N < 8 || s.N > 256 || s.N % 8 || s.d_v < 8 || s.d_v > 256 || s.d_v % 8) return false;
  if (!dtype_ok(s.in_dtype)) return false;
  *a = SsmArgs{};
  a->H = s.H;
  a->G = s.G;
  a->N = s.N;
  a->P = s.d_v;
  a->softplus = s.softplus != 0;
  a->k_stride = pitch_of(s.k_stride, (long long)s.G * s.N, s.in_dtype);
  a->q_stride = pitch_of(s.q_stride, (long long)s.G * s.N, s.in_dtype);
  a->v_stride = pitch_of(s.v_stride, (long long)s.H * s.d_v, s.in_dtype);
  a->gate_stride = pitch_of(s.gate_stride, (long long)s.H * s.d_v, s.in_dtype);
  a->dt_stride = s.dt_stride == 0 ? s.H : s.dt_stride;
  return a->k_stride > 0 && a->q_stride > 0 && a->v_stride > 0 && a->gate_stride > 0 &&
         a->dt_stride >= s.H && a->dt_stride < (1LL << 40);
}

// Checks the pointers of a call over R rows and puts them into `a`.
bool ssm_pointers(const sdm_ssm_shape& s, long long R, const void* k, const void* q,
                  const void* v, const void* dt, const float* A, const float* dt_bias,
                  const float* D, float* M, const void* gate, int act, const int32_t* cu, void* y,
                  SsmArgs* a) {
  if (!A || !M || !act_ok(act)) return false;
  if (R > 0 && (!k || !q || !v || !dt || !y)) return false;
  if (!aligned16(k) || !aligned16(q) || !aligned16(v) || !aligned16(gate) || !aligned16(y) ||
      !aligned16(M) || !aligned16(A) || !aligned16(dt_bias) || !aligned16(D) ||
      (reinterpret_cast<uintptr_t>(cu) & 3u) ||
      reinterpret_cast<uintptr_t>(dt) % dtype_size(s.in_dtype))
    return false;
  const long long gn = (long long)s.G * s.N, hp = (long long)s.H * s.d_v;
  const Span sk{k, span_bytes(R, a->k_stride, gn, s.in_dtype)},
      sq{q, span_bytes(R, a->q_stride, gn, s.in_dtype)},
      sv{v, span_bytes(R, a->v_stride, hp, s.in_dtype)},
      sg{gate, span_bytes(R, a->gate_stride, hp, s.in_dtype)},
      sdt{dt, span_bytes(R, a->dt_stride, s.H, s.in_dtype)}, sA{A, (size_t)s.H * 4},
      sb{dt_bias, (size_t)s.H * 4}, sD{D, (size_t)s.H * 4}, sc{cu, ((size_t)s.B + 1) * 4},
      sM{M, (size_t)s.B * hp * s.N * 4}, sy{y, (size_t)R * hp * dtype_size(s.in_dtype)};
  if (overlaps_any(sy, {sk, sq, sv, sg, sdt, sA, sb, sD, sc, sM}) ||
      overlaps_any(sM, {sk, sq, sv, sg, sdt, sA, sb, sD, sc}))
    return false;
  a->k = k;
  a->q = q;
  a->v = v;
  a->dt = dt;
  a->A = A;
  a->dt_bias = dt_bias;
  a->D = D;
  a->M = M;
  a->gate = gate;
  a->act = act;
  a->y = y;
  return true;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor map encoder, looked up once per process.
EncodeTiledFn tensor_map_encoder() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Rows of `heads` x `width` bf16 values at a pitch, read in tiles of 128 rows x 64 values of one
// head, with zeros where the head or the rows end.
bool tile_map(CUtensorMap* map, const void* p, int width, int heads, long long rows,
              long long pitch) {
  const EncodeTiledFn encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)pitch * 2};
  const cuuint32_t box[3] = {64, 1, SB_L}, steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p), dims, strides, box,
                steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which prompts the block-wise scan takes: bf16, at most 128 state rows, and sequences of 24
// tokens or more (on average, when packed: their own lengths are on the device).  A block costs
// the same for one token as for 128, the token-by-token scan goes by tiles of 16 tokens.  Measured
// (us, N = 128, calls replayed from a graph): 8 x 32 heads of 64, 16 tokens 14.4 token by token, 23
// tokens 19.9, 24 to 32 tokens 16.5 in blocks; 8 heads of 64, where neither fills the device, 5.0,
// 6.6 and 10.2.
// Its row numbers are 32 bits wide and, in the last block, reach SB_L - 1 rows behind the batch.
bool ssm_block_fits(const sdm_ssm_shape& s, bool packed) {
  const long long rows = packed ? s.T : (long long)s.B * s.T, length = packed ? s.T / s.B : s.T;
  return s.in_dtype == SDM_BF16 && s.N <= 128 && length >= 24 && rows <= 2147483647LL - SB_L;
}

// How a scan cuts sequences into segments.  A CTA walks a segment `unit` rows at a time in about
// walk_us each and walk_piece_us for all, `slots` CTAs at once; the pass that makes the segments'
// own contributions costs pre_us a unit and pre_piece_us a segment, and with the chain over
// segments split_us at least.  The number of segments is the one
// with the least estimated time; packed batches, whose lengths only the device knows, are cut
// as one sequence of all rows would be.
struct SsmCost {
  int unit, slots;
  double walk_us, walk_piece_us, pre_us, pre_piece_us, split_us;
};

struct SsmPlan {
  // rows of a segment; (sequence, segment) pairs, and segments of split sequences, at most
  long long seg_rows, items, slots;
  bool split;
  size_t off_decays, off_prep, off_items, bytes;
};

SsmPlan ssm_plan(const sdm_ssm_shape& s, bool packed, long long ctas_per_item, const SsmCost& c) {
  const long long L = ((long long)s.T + c.unit - 1) / c.unit, seqs = packed ? 1 : s.B;
  auto waves = [&](long long items) {
    return (double)((items * ctas_per_item + c.slots - 1) / c.slots);
  };
  long long best = 1;
  double least = waves(seqs) * (L * c.walk_us + c.walk_piece_us);
  const long long most = 6LL * c.slots / (seqs * ctas_per_item) + 1;  // more waves gain nothing
  for (long long n = 2; n <= L && n <= most; n += n < 16 ? 1 : n / 16) {
    const long long len = (L + n - 1) / n;
    if ((L + len - 1) / len != n) continue;
    const double t = waves(seqs * n) * (len * c.walk_us + c.walk_piece_us) +
                     waves(seqs * (n - 1)) * (len * c.pre_us + c.pre_piece_us) + c.split_us;
    if (t < least) {
      least = t;
      best = n;
    }
  }
  SsmPlan p = {};
  p.split = best > 1;
  p.seg_rows = (L > 0 ? (L + best - 1) / best : 1) * c.unit;
  p.items = packed ? s.T / p.seg_rows + s.B
                   : s.B * (s.T > 0 ? (s.T + p.seg_rows - 1) / p.seg_rows : 1);
  if (p.split) {
    // a packed sequence of n > seg_rows rows has at most 2 n / seg_rows segments
    p.slots = p.items;
    if (packed && 2LL * s.T / p.seg_rows < p.slots) p.slots = 2LL * s.T / p.seg_rows;
    p.off_decays = round_up((size_t)p.slots * s.H * s.N * s.d_v * 4, WS_ALIGN);
    p.bytes = p.off_decays + round_up((size_t)p.slots * s.H * 4, WS_ALIGN);
  }
  return p;
}

// Places for blocks' sums (ssm_first_block).
long long ssm_prep_blocks(const sdm_ssm_shape& s, bool packed) {
  return packed ? (long long)s.T / SB_L + s.B + 1 : s.B * (((long long)s.T + SB_L - 1) / SB_L);
}

SsmPlan ssm_plan(const sdm_ssm_shape& s, bool packed, int sms, bool block) {
  if (!block)
    return ssm_plan(s, packed, (long long)s.H * ((s.d_v + SSM_COLS - 1) / SSM_COLS),
                    SsmCost{16, 5 * sms, 1.6, 2.0, 1.2, 2.0, 8.0});
  SsmPlan p = ssm_plan(s, packed, (long long)s.H * ((s.d_v + SB_P - 1) / SB_P),
                       SsmCost{SB_L, sms, 3.1, 1.0, 1.2, 4.0, 8.0});
  // every block's sums, where ssm_first_block puts them
  const long long blocks = ssm_prep_blocks(s, packed);
  p.off_prep = p.bytes;
  p.off_items = p.bytes + round_up((size_t)blocks * s.H * sizeof(SsmPrep), WS_ALIGN);
  p.bytes = p.off_items + round_up((size_t)p.items * (sizeof(int4) + sizeof(int)), WS_ALIGN);
  return p;
}

SsmSplit ssm_split(const SsmPlan& plan, void* ws) {
  return SsmSplit{plan.seg_rows, plan.items, plan.slots, static_cast<float*>(ws),
                  reinterpret_cast<float*>(static_cast<char*>(ws) + plan.off_decays)};
}

cudaError_t launch_ssm_chain(const sdm_ssm_shape& s, const SsmArgs& a, const SsmSplit& sp,
                             const DeviceInfo* di, cudaStream_t st) {
  const long long units = (long long)s.H * ((s.N * s.d_v / 4 + 255) / 256);
  const long long seqs = a.seq.cu ? 1 : s.B;  // uniform batches: every sequence is split
  const long long most = 8LL * di->sms, blocks = units * seqs < most ? units : most;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return launch_pdl<true>(ssm_chain_kernel, dim3((unsigned)blocks), dim3(256), 0, st, a, sp);
}

template <typename T, bool CONTRIB>
cudaError_t launch_ssm_scan(const SsmArgs& a, const SsmSplit& sp, dim3 grid, cudaStream_t st) {
  const dim3 block(128);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (a.N <= 32)
    return launch_pdl<true>(ssm_scan_kernel<T, 1, CONTRIB>, grid, block, 0, st, a, sp);
  if (a.N <= 64)
    return launch_pdl<true>(ssm_scan_kernel<T, 2, CONTRIB>, grid, block, 0, st, a, sp);
  if (a.N <= 128)
    return launch_pdl<true>(ssm_scan_kernel<T, 4, CONTRIB>, grid, block, 0, st, a, sp);
  return launch_pdl<true>(ssm_scan_kernel<T, 8, CONTRIB>, grid, block, 0, st, a, sp);
}

template <typename T>
sdm_status ssm_scan_run(const sdm_ssm_shape& s, const SsmArgs& a, const DeviceInfo* di, void* ws,
                        cudaStream_t st) {
  const SsmPlan plan = ssm_plan(s, a.seq.cu != nullptr, di->sms, false);
  if (plan.items > 2147483647LL) return SDM_ERR_UNSUPPORTED;
  const SsmSplit sp = ssm_split(plan, ws);
  const dim3 grid((unsigned)plan.items, (unsigned)s.H,
                  (unsigned)((s.d_v + SSM_COLS - 1) / SSM_COLS));
  if (plan.split) {
    SDM_CUDA_TRY((launch_ssm_scan<T, true>(a, sp, grid, st)));
    SDM_CUDA_TRY(launch_ssm_chain(s, a, sp, di, st));
  }
  SDM_CUDA_TRY((launch_ssm_scan<T, false>(a, sp, grid, st)));
  return SDM_OK;
}

template <typename T>
sdm_status ssm_step_run(const sdm_ssm_shape& s, const SsmArgs& a, cudaStream_t st) {
  if ((long long)s.B * s.H > 2147483647LL) return SDM_ERR_UNSUPPORTED;
  SDM_CUDA_TRY(launch_pdl<true>(ssm_step_kernel<T>, dim3((unsigned)(s.B * s.H)), dim3(256), 0, st,
                                a));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SDM_OK;
}

sdm_status ssm_block_run(const sdm_ssm_shape& s, const SsmArgs& a, const DeviceInfo* di, void* ws,
                         cudaStream_t st) {
  const SsmPlan plan = ssm_plan(s, a.seq.cu != nullptr, di->sms, true);
  SsmBlockArgs ba;
  ba.a = a;
  ba.sp = ssm_split(plan, ws);
  ba.prep = reinterpret_cast<SsmPrep*>(static_cast<char*>(ws) + plan.off_prep);
  ba.items = reinterpret_cast<int4*>(static_cast<char*>(ws) + plan.off_items);
  ba.ptiles = (s.d_v + SB_P - 1) / SB_P;
  if (!tile_map(&ba.mq, a.q, s.N, s.G, a.seq.R, a.q_stride) ||
      !tile_map(&ba.mk, a.k, s.N, s.G, a.seq.R, a.k_stride) ||
      !tile_map(&ba.mv, a.v, s.d_v, s.H, a.seq.R, a.v_stride) ||
      (a.gate && !tile_map(&ba.mz, a.gate, s.d_v, s.H, a.seq.R, a.gate_stride)))
    return SDM_ERR_CUDA;
  const long long blocks = plan.items * s.H * ba.ptiles;
  if (blocks > 2147483647LL) return SDM_ERR_UNSUPPORTED;
  const unsigned ctas = (unsigned)(blocks < di->sms ? blocks : di->sms);
  ba.step_items = (int)ctas / (s.H * ba.ptiles);
  ba.step_parts = (int)ctas % (s.H * ba.ptiles);
  const long long preps = ssm_prep_blocks(s, a.seq.cu != nullptr);
  SDM_CUDA_TRY(launch_pdl<true>(ssm_prep_kernel,
                                dim3((unsigned)(preps + (plan.items + 7) / 8),
                                     (unsigned)(s.H + 7) / 8),
                                dim3(256), 0, st, a, ba.sp, ba.prep, (int)preps, ba.items,
                                (int)plan.items));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (plan.split) {
    SDM_CUDA_TRY(launch_pdl(ssm_segment_kernel, dim3(ctas), dim3(SG_THREADS),
                            (size_t)SG_SMEM, st, ba));
    g_launches.fetch_add(1, std::memory_order_relaxed);
    SDM_CUDA_TRY(launch_ssm_chain(s, a, ba.sp, di, st));
  }
  SDM_CUDA_TRY(launch_pdl(ssm_block_kernel, dim3(ctas), dim3(SB_THREADS),
                          (size_t)SB_SMEM, st, ba));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SDM_OK;
}

template <typename T, typename TR>
cudaError_t launch_block_norm(const BlockNormArgs& a, const DeviceInfo* di, cudaStream_t st) {
  const int nvec = a.D / 8;
  auto go = [&](auto kernel, int tpr) {
    const int threads = tpr > 256 ? tpr : 256, rpb = threads / tpr;
    long long blocks = (a.rows + rpb - 1) / rpb;
    const long long most = (long long)di->sms * (threads > 256 ? 1 : 2);  // all resident
    if (blocks > most) blocks = most;
    return launch_pdl<true>(kernel, dim3((unsigned)blocks), dim3(threads), 0, st, a);
  };
  if (nvec <= 32) return go(block_norm_kernel<T, TR, 32, 1>, 32);
  if (nvec <= 64) return go(block_norm_kernel<T, TR, 64, 1>, 64);
  if (nvec <= 128) return go(block_norm_kernel<T, TR, 128, 1>, 128);
  if (nvec <= 256) return go(block_norm_kernel<T, TR, 256, 1>, 256);
  if (nvec <= 512) return go(block_norm_kernel<T, TR, 512, 1>, 512);
  if (nvec <= 1024) return go(block_norm_kernel<T, TR, 512, 2>, 512);
  return go(block_norm_kernel<T, TR, 512, 4>, 512);
}

}  // namespace

extern "C" {

sdm_status sdm_conv_forward(const void* x, const float* w, const float* bias, void* state,
                            int32_t init, int32_t act, const int32_t* cu, void* y,
                            sdm_conv_shape shape, void* stream) {
  NvtxRange nvtx_range("sdm_conv_forward");
  return conv_run(x, w, bias, state, init, act, cu, y, shape, stream, false);
}

sdm_status sdm_conv_step(const void* x, const float* w, const float* bias, void* state,
                         int32_t act, void* y, sdm_conv_shape shape, void* stream) {
  NvtxRange nvtx_range("sdm_conv_step");
  return conv_run(x, w, bias, state, SDM_CONTINUE, act, nullptr, y, shape, stream, true);
}

size_t sdm_ssm_workspace_size(sdm_ssm_shape shape) {
  SsmArgs a;
  DeviceInfo* di;
  if (!ssm_args(shape, false, &a)) return 0;
  size_t need = 0;
  // without a device (sizes asked for ahead of time) a B200's number of multiprocessors
  const int sms = device_info(&di) == SDM_OK ? di->sms : 148;
  for (const bool packed : {false, true}) {
    const size_t n = ssm_plan(shape, packed, sms, ssm_block_fits(shape, packed)).bytes;
    if (n > need) need = n;
  }
  return need;
}

sdm_status sdm_ssm_forward(const void* k, const void* q, const void* v, const void* dt,
                           const float* A, const float* dt_bias, const float* D, float* M,
                           int32_t init, const void* gate, int32_t act, const int32_t* cu,
                           void* y, void* ws, size_t ws_bytes, sdm_ssm_shape shape,
                           void* stream) {
  NvtxRange nvtx_range("sdm_ssm_forward");
  const sdm_ssm_shape& s = shape;
  SsmArgs a;
  if (!ssm_args(s, false, &a)) return SDM_ERR_INVALID_ARG;
  if (init != SDM_INIT_ZERO && init != SDM_CONTINUE) return SDM_ERR_INVALID_ARG;
  const long long R = cu ? s.T : (long long)s.B * s.T;
  if (!ssm_pointers(s, R, k, q, v, dt, A, dt_bias, D, M, gate, act, cu, y, &a))
    return SDM_ERR_INVALID_ARG;
  const size_t need = sdm_ssm_workspace_size(s);
  if (need && (!ws || ws_bytes < need || reinterpret_cast<uintptr_t>(ws) % WS_ALIGN != 0))
    return SDM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (R == 0) {
    if (init == SDM_INIT_ZERO)
      SDM_CUDA_TRY(cudaMemsetAsync(M, 0, (size_t)s.B * s.H * s.N * s.d_v * 4, st));
    return SDM_OK;
  }
  DeviceInfo* di;
  const sdm_status rc = device_info(&di);
  if (rc != SDM_OK) return rc;
  a.seq = SeqBounds{cu, s.B, s.T, R};
  a.from_zero = init == SDM_INIT_ZERO;
  ProfScope ps(SDM_KERNEL_SSM, st);
  if (ssm_block_fits(s, cu != nullptr)) return ssm_block_run(s, a, di, ws, st);
  const bool bf16 = s.in_dtype == SDM_BF16;
  if (!cu && s.T == 1)  // one token: the step's kernel moves the state in whole rows
    return bf16 ? ssm_step_run<__nv_bfloat16>(s, a, st) : ssm_step_run<float>(s, a, st);
  return bf16 ? ssm_scan_run<__nv_bfloat16>(s, a, di, ws, st)
              : ssm_scan_run<float>(s, a, di, ws, st);
}

sdm_status sdm_ssm_step(const void* k, const void* q, const void* v, const void* dt,
                        const float* A, const float* dt_bias, const float* D, float* M,
                        const void* gate, int32_t act, void* y, sdm_ssm_shape shape,
                        void* stream) {
  NvtxRange nvtx_range("sdm_ssm_step");
  const sdm_ssm_shape& s = shape;
  SsmArgs a;
  if (!ssm_args(s, true, &a)) return SDM_ERR_INVALID_ARG;
  if (!ssm_pointers(s, s.B, k, q, v, dt, A, dt_bias, D, M, gate, act, nullptr, y, &a))
    return SDM_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(SDM_KERNEL_SSM, st);
  return s.in_dtype == SDM_BF16 ? ssm_step_run<__nv_bfloat16>(s, a, st)
                                : ssm_step_run<float>(s, a, st);
}

sdm_status sdm_block_norm(const void* u, const void* gate, int32_t act, int32_t post_norm,
                          const float* post_gamma, const float* scale, const void* r,
                          int32_t r_dtype, const float* pre_gamma, float eps, void* r_out,
                          void* n, int64_t rows, int32_t D, int32_t in_dtype, void* stream) {
  NvtxRange nvtx_range("sdm_block_norm");
  if (rows < 0 || rows > (1LL << 40) || D < 8 || D > 16384 || D % 8 || !dtype_ok(in_dtype) ||
      !dtype_ok(r_dtype) || !act_ok(act) || !(eps >= 0.0f))
    return SDM_ERR_INVALID_ARG;
  if (rows > 0 && (!u || !r || !r_out)) return SDM_ERR_INVALID_ARG;
  for (const void* p : {u, gate, r, (const void*)r_out, (const void*)n,
                        (const void*)post_gamma, (const void*)scale, (const void*)pre_gamma})
    if (!aligned16(p)) return SDM_ERR_INVALID_ARG;
  const size_t in = (size_t)rows * D * dtype_size(in_dtype),
               res = (size_t)rows * D * dtype_size(r_dtype), par = (size_t)D * 4;
  const Span su{u, in}, sg{gate, in}, sr{r, res}, so{r_out, res}, sn{n, in},
      p1{post_gamma, par}, p2{scale, par}, p3{pre_gamma, par};
  if (overlaps_any(so, {su, sg, sn, p1, p2, p3}) || (r_out != r && overlap(so.p, so.n, sr.p, sr.n)))
    return SDM_ERR_INVALID_ARG;
  if (overlaps_any(sn, {sr, p1, p2, p3}) || (n != u && overlap(sn.p, sn.n, su.p, su.n)) ||
      (n != gate && overlap(sn.p, sn.n, sg.p, sg.n)))
    return SDM_ERR_INVALID_ARG;
  if (rows == 0) return SDM_OK;
  DeviceInfo* di;
  const sdm_status rc = device_info(&di);
  if (rc != SDM_OK) return rc;
  BlockNormArgs a = {};
  a.u = u;
  a.gate = gate;
  a.r = r;
  a.r_out = r_out;
  a.n = n;
  a.post_gamma = post_gamma;
  a.pre_gamma = pre_gamma;
  a.scale = scale;
  a.rows = rows;
  a.D = D;
  a.act = act;
  a.post = post_norm != 0;
  a.eps = eps;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(SDM_KERNEL_BLOCK_NORM, st);
  if (in_dtype == SDM_BF16 && r_dtype == SDM_BF16)
    SDM_CUDA_TRY((launch_block_norm<__nv_bfloat16, __nv_bfloat16>(a, di, st)));
  else if (in_dtype == SDM_BF16)
    SDM_CUDA_TRY((launch_block_norm<__nv_bfloat16, float>(a, di, st)));
  else if (r_dtype == SDM_BF16)
    SDM_CUDA_TRY((launch_block_norm<float, __nv_bfloat16>(a, di, st)));
  else
    SDM_CUDA_TRY((launch_block_norm<float, float>(a, di, st)));
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return SDM_OK;
}

}  // extern "C"
