// api_serve.cuh — the entries around the head: the RMS norm that makes H, the e4m3 quantisation,
// the 8-bit logits and the sampling. Part of the one translation unit lmh_api.cu.
#pragma once

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Shared memory above the default has to be asked for once per kernel and device.
template <class K>
lmh_status allow_smem(K kernel, int bytes, int dev, std::atomic<uint64_t>* done) {
  const uint64_t bit = 1ull << dev;
  if (done->load() & bit) return LMH_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return LMH_ERR_CUDA;
  done->fetch_or(bit);
  return LMH_OK;
}

// Blocks of the forward: as many as can be resident (threads, shared memory), or a row each.
template <int VPT>
lmh_status launch_norm(const NormParams& p, int threads, int dev, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const int smem = norm_stages(VPT) * 2 * threads * VPT * 16;
  LMH_TRY(allow_smem(rms_norm_kernel<VPT>, norm_stages(VPT) * 2 * 512 * VPT * 16, dev, &done));
  const int by_smem = 220 * 1024 / (smem + 1024), by_threads = 1536 / threads;
  const int64_t most = static_cast<int64_t>(sms) * (by_smem < by_threads ? by_smem : by_threads);
  ProfScope ps(KID_RMS_NORM, st);
  rms_norm_kernel<VPT><<<static_cast<unsigned>(p.N < most ? p.N : most), threads, smem, st>>>(p);
  return last_launch();
}

template <int VPT>
lmh_status launch_norm_bwd(const NormBwdParams& p, int threads, int dev, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  LMH_TRY(allow_smem(rms_norm_bwd_kernel<VPT>, norm_bwd_stages(VPT) * 3 * 512 * VPT * 16, dev, &done));
  ProfScope ps(KID_RMS_NORM_BWD, st);
  rms_norm_bwd_kernel<VPT><<<static_cast<unsigned>(p.slices), threads,
                              norm_bwd_stages(VPT) * 3 * threads * VPT * 16, st>>>(p);
  return last_launch();
}

}  // namespace

extern "C" lmh_status lmh_rms_norm(int64_t N, int64_t d, const lmh_bf16* x,
                                   const lmh_bf16* residual, const lmh_bf16* weight, float eps,
                                   lmh_bf16* sum, lmh_bf16* y, uint8_t* q, float* scale,
                                   float* rstd, void* stream) {
  if (!norm_shape_ok(N, d) || !(eps >= 0.f && eps < 3.0e38f)) return LMH_ERR_INVALID_ARG;
  if (N > 0 && ((!y && !q) || (q == nullptr) != (scale == nullptr) || !x || !weight))
    return LMH_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(sum) ||
      !aligned16(y) || !aligned16(q) || !aligned4(scale) || !aligned4(rstd))
    return LMH_ERR_ALIGNMENT;
  int dev, sms;
  LMH_TRY(current_device(&dev, &sms));
  if (N == 0) return LMH_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NormParams p;
  p.N = N;
  p.d = static_cast<int>(d);
  p.eps = eps;
  p.inv_d = 1.f / static_cast<float>(d);
  p.x = reinterpret_cast<const uint4*>(x);
  p.residual = reinterpret_cast<const uint4*>(residual);
  p.weight = reinterpret_cast<const uint4*>(weight);
  p.sum = reinterpret_cast<uint4*>(sum);
  p.y = reinterpret_cast<uint4*>(y);
  p.q = reinterpret_cast<uint2*>(q);
  p.scale = scale;
  p.rstd = rstd;
  int vpt, threads;
  norm_threads(d, &vpt, &threads);
  if (vpt == 1) return launch_norm<1>(p, threads, dev, sms, st);
  if (vpt == 2) return launch_norm<2>(p, threads, dev, sms, st);
  return launch_norm<4>(p, threads, dev, sms, st);
}

extern "C" lmh_status lmh_rms_norm_bwd(int64_t N, int64_t d, const lmh_bf16* sum,
                                       const lmh_bf16* weight, const float* rstd,
                                       const lmh_bf16* dy, const lmh_bf16* dsum, lmh_bf16* dx,
                                       lmh_bf16* dweight, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!norm_shape_ok(N, d) || !workspace) return LMH_ERR_INVALID_ARG;
  if (N > 0 && (!sum || !weight || !rstd || !dy || (!dx && !dweight))) return LMH_ERR_INVALID_ARG;
  if (!aligned16(sum) || !aligned16(weight) || !aligned16(dy) || !aligned16(dsum) ||
      !aligned16(dx) || !aligned16(dweight) || !aligned4(rstd) ||
      (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return LMH_ERR_ALIGNMENT;
  const int slices = norm_slices(N, d);
  if (workspace_bytes < norm_bwd_bytes(N, d))
    return LMH_ERR_WORKSPACE_TOO_SMALL;
  int dev, sms;
  LMH_TRY(current_device(&dev, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws ws{static_cast<uint8_t*>(workspace), static_cast<WsHeader*>(workspace)};
  if (N == 0) {
    if (dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(d) * 2, st) != cudaSuccess)
      return LMH_ERR_CUDA;
    return clear_header(ws, st);
  }
  NormBwdParams p;
  p.N = N;
  p.d = static_cast<int>(d);
  p.slices = slices;
  p.sum = reinterpret_cast<const uint4*>(sum);
  p.weight = reinterpret_cast<const uint4*>(weight);
  p.rstd = rstd;
  p.inv_d = 1.f / static_cast<float>(d);
  p.dy = reinterpret_cast<const uint4*>(dy);
  p.dsum = reinterpret_cast<const uint4*>(dsum);
  p.dx = reinterpret_cast<uint4*>(dx);
  p.part = dweight ? ws.at<float>(sizeof(WsHeader)) : nullptr;
  p.h = ws.h;
  int vpt, threads;
  norm_threads(d, &vpt, &threads);
  if (vpt == 1) LMH_TRY(launch_norm_bwd<1>(p, threads, dev, st));
  else if (vpt == 2) LMH_TRY(launch_norm_bwd<2>(p, threads, dev, st));
  else LMH_TRY(launch_norm_bwd<4>(p, threads, dev, st));
  if (!dweight) return LMH_OK;
  ProfScope ps(KID_NORM_DWEIGHT, st);
  norm_dweight_kernel<<<static_cast<unsigned>(d / 32), dim3(32, 16), 0, st>>>(
      slices, static_cast<int>(d), p.part, reinterpret_cast<__nv_bfloat16*>(dweight));
  return last_launch();
}

extern "C" lmh_status lmh_quantize_fp8(int64_t rows, int64_t d, int32_t block_rows,
                                       const lmh_bf16* x, uint8_t* q, float* scale,
                                       void* stream) {
  if (rows < 0 || rows > 0x7fffffffLL || d <= 0 || d % 64 != 0 || d > (1LL << 24) ||
      (block_rows != 1 && block_rows != kQBlock))
    return LMH_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !q || !scale)) return LMH_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(q) || !aligned4(scale)) return LMH_ERR_ALIGNMENT;
  const int64_t nb = cdiv(d, kQBlock);
  // A warp a row where the rows fill the GPU, a block of threads a row where they do not: d = 4096,
  // 600 rows 10.9 us by warps, 8.9 by blocks; 4096 rows 16.8 and 19.6 (from cold caches; 4096 rows by
  // warps take 9.9 in a loop over 34 MB, which L2 holds).
  const int per = rows < 8 * 148 ? 256 : 32;
  const int64_t grid = block_rows == 1 ? cdiv(rows, 256 / per) : cdiv(rows, kQBlock) * nb;
  if (cdiv(rows, block_rows) * nb > 0x7fffffffLL) return LMH_ERR_INVALID_ARG;
  int dev, sms;
  LMH_TRY(current_device(&dev, &sms));
  if (rows == 0) return LMH_OK;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  ProfScope ps(KID_QUANTIZE, st);
  if (block_rows == 1)
    quantize_rows_kernel<<<static_cast<unsigned>(grid), 256, 0, st>>>(
        rows, static_cast<int>(d), per, reinterpret_cast<const uint4*>(x), reinterpret_cast<uint2*>(q), scale);
  else
    quantize_blocks_kernel<<<static_cast<unsigned>(grid), 256, 0, st>>>(
        rows, static_cast<int>(d), reinterpret_cast<const uint4*>(x), reinterpret_cast<uint2*>(q), scale);
  return last_launch();
}

namespace {

// 8-bit [outer, inner] matrix; box {128, box_outer}, 128-byte swizzle, zero fill out of bounds.
bool tmap_8bit(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_outer) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner};
  cuuint32_t box[2] = {kFpK, box_outer};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int TN, class Out>
lmh_status launch_few(FpParams p, const uint8_t* H8, const uint8_t* W8, int64_t d, int dev, int sms,
                      cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  LMH_TRY(allow_smem(fp8_few_kernel<TN, Out>, FpFew<TN>::SMEM, dev, &done));
  CUtensorMap tw, th;
  if (!tmap_8bit(&tw, W8, d, p.V, kFpM) || !tmap_8bit(&th, H8, d, p.N, TN)) return LMH_ERR_CUDA;
  p.vtiles = static_cast<int>(cdiv(p.V, kFpM));
  p.ntiles = 1;
  const int64_t tiles = p.vtiles;
  ProfScope ps(KID_FP8_LOGITS, st);
  fp8_few_kernel<TN, Out><<<static_cast<unsigned>(tiles < sms ? tiles : sms), FpFew<TN>::THREADS,
                            FpFew<TN>::SMEM, st>>>(tw, th, p);
  return last_launch();
}

// Logits [N, V] for stores of 32 rows x 64 bytes.
bool tmap_logits(CUtensorMap* m, void* base, uint64_t V, uint64_t N, bool f32) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const uint64_t es = f32 ? 4 : 2;
  cuuint64_t dims[2] = {V, N};
  cuuint64_t strides[1] = {V * es};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(64 / es), 32};
  cuuint32_t one[2] = {1, 1};
  return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
            box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Out, bool TMA>
lmh_status launch_many(FpParams p, const uint8_t* H8, const uint8_t* W8, int64_t d, int dev, int sms,
                       cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  LMH_TRY(allow_smem(fp8_many_kernel<Out, TMA>, FpMany::SMEM, dev, &done));
  CUtensorMap tw, th, to;
  if (!tmap_8bit(&tw, W8, d, p.V, FpMany::TV) || !tmap_8bit(&th, H8, d, p.N, kFpM))
    return LMH_ERR_CUDA;
  to = th;
  if (TMA && !tmap_logits(&to, p.out, p.V, p.N, sizeof(Out) == 4)) return LMH_ERR_CUDA;
  p.vtiles = static_cast<int>(cdiv(p.V, FpMany::TV));
  p.ntiles = static_cast<int>(cdiv(p.N, kFpM));
  const int64_t tiles = static_cast<int64_t>(p.vtiles) * p.ntiles;
  if (tiles > 0x7fff0000LL) return LMH_ERR_INVALID_ARG;
  ProfScope ps(KID_FP8_LOGITS, st);
  fp8_many_kernel<Out, TMA><<<static_cast<unsigned>(tiles < sms ? tiles : sms), FpMany::THREADS,
                              FpMany::SMEM, st>>>(tw, th, to, p);
  return last_launch();
}

// The kernel with few columns of tokens as far as it goes: 128256 x 4096 from cold caches, 1 / 32 / 64
// tokens 108 / 108 / 113 us, by the other kernel 120 / 115 / 118. (A weight that L2 holds may be faster by
// the other: 32000 x 2048 in a loop, 64 tokens 21.9 us, 65 by the other 16.4.) The narrowest that holds the
// tokens: with 64 columns 1 / 16 / 32 tokens took 113 / 107 / 110 us, with their own 108 / 106 / 108.
template <class Out>
lmh_status launch_fp8(const FpParams& p, const uint8_t* H8, const uint8_t* W8, int64_t d, int dev,
                      int sms, cudaStream_t st) {
  const bool few = p.nb <= kFewBlocks;
  if (few && p.N <= 16) return launch_few<16, Out>(p, H8, W8, d, dev, sms, st);
  if (few && p.N <= 32) return launch_few<32, Out>(p, H8, W8, d, dev, sms, st);
  if (few && p.N <= 64) return launch_few<64, Out>(p, H8, W8, d, dev, sms, st);
  const bool tma = aligned16(p.out) && p.V * sizeof(Out) % 16 == 0;
  return tma ? launch_many<Out, true>(p, H8, W8, d, dev, sms, st)
             : launch_many<Out, false>(p, H8, W8, d, dev, sms, st);
}

}  // namespace

extern "C" lmh_status lmh_fp8_logits(const lmh_shape* shape, const uint8_t* H8,
                                     const float* h_scale, const uint8_t* W8,
                                     const float* w_scale, void* logits, int32_t dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!shape_ok(shape) || shape->N > 0x7fffffffLL ||
      (dtype != LMH_DTYPE_F32 && dtype != LMH_DTYPE_BF16) || !workspace)
    return LMH_ERR_INVALID_ARG;
  if (shape->N > 0 && (!H8 || !h_scale || !W8 || !w_scale || !logits)) return LMH_ERR_INVALID_ARG;
  const uintptr_t esize = dtype == LMH_DTYPE_F32 ? 4 : 2;
  if (!aligned16(H8) || !aligned16(W8) || !aligned4(h_scale) || !aligned4(w_scale) ||
      (reinterpret_cast<uintptr_t>(logits) & (esize - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return LMH_ERR_ALIGNMENT;
  if (workspace_bytes < lmh_workspace_size(shape, LMH_ENTRY_FP8_LOGITS))
    return LMH_ERR_WORKSPACE_TOO_SMALL;
  int dev, sms;
  LMH_TRY(current_device(&dev, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws ws{static_cast<uint8_t*>(workspace), static_cast<WsHeader*>(workspace)};
  if (shape->N == 0) return clear_header(ws, st);  // else the kernel clears the error word
  FpParams p{};
  p.N = shape->N;
  p.V = shape->V;
  p.nb = static_cast<int>(cdiv(shape->d, kFpK));
  p.hs = h_scale;
  p.ws = w_scale;
  p.out = logits;
  p.err = &ws.h->err;
  return dtype == LMH_DTYPE_F32 ? launch_fp8<float>(p, H8, W8, shape->d, dev, sms, st)
                                : launch_fp8<__nv_bfloat16>(p, H8, W8, shape->d, dev, sms, st);
}

namespace {

// CTAs per row of the row kernel: 1, 2, 4 or 8, at least 4096 logits each. No result depends on
// it. How many rows are left to that kernel only the device knows; it is made for few: thirty rows of
// 151936 took 218 / 71 / 66 us with 1 / 4 / 8, some of 33 of 50001 68 / 44 / 40.
int sample_cluster(int64_t V) {
  int C = 1;
  while (C < kSampMaxC && V / (2 * C) >= 4096) C *= 2;
  return C;
}

// The kernels of one call, each waiting for the one before at its own start, so that its launch
// overlaps that one's end.
template <class K>
lmh_status launch_sample(K kernel, const SampParams& p, int64_t grid, int threads, size_t smem,
                         int cluster, bool follows, cudaStream_t st) {
  if (grid > 0x7fffffffLL) return LMH_ERR_INVALID_ARG;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  int n = 0;
  if (cluster > 0) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (follows) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = static_cast<unsigned>(n);
  if (cudaLaunchKernelEx(&cfg, kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return LMH_ERR_CUDA;
  }
  return last_launch();
}

// may_leave: a row may be left to the row kernel.
template <class T>
lmh_status run_sample(SampParams p, bool may_leave, int dev, cudaStream_t st) {
  {
    ProfScope ps(KID_SAMPLE_GROUPS, st);
    LMH_TRY(launch_sample(sample_groups_kernel<T>, p, p.N * cdiv(p.blocks, kGroupWarps * kGroupPer),
                          32 * kGroupWarps, 0, 0, false, st));
  }
  {
    ProfScope ps(KID_SAMPLE, st);
    LMH_TRY(launch_sample(sample_list_kernel<T>, p, p.N, kSampThreads, 0, 0, true, st));
  }
  if (!may_leave) return LMH_OK;
  static std::atomic<uint64_t> done{0};
  LMH_TRY(allow_smem(sample_row_kernel<T>, kMaxDynSmem, dev, &done));
  p.C = sample_cluster(p.V);
  p.L = static_cast<int>(cdiv(cdiv(p.V, p.C), 8) * 8);
  size_t smem = sizeof(RowShared) + static_cast<size_t>(p.L) * sizeof(T) + 16;  // 16: the row's alignment
  p.resident = smem <= kMaxDynSmem ? 1 : 0;
  if (!p.resident) smem = sizeof(RowShared);
  ProfScope ps(KID_SAMPLE_ROWS, st);
  return launch_sample(sample_row_kernel<T>, p, p.N * p.C, kSampThreads, smem, p.C, true, st);
}

}  // namespace

extern "C" lmh_status lmh_sample(const lmh_shape* shape, const lmh_sampling* opt,
                                 const void* logits, int32_t dtype, const float* u,
                                 int32_t* tokens, float* logprob, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (!shape_ok(shape) || !opt || shape->N > 0xfffffffLL ||
      (dtype != LMH_DTYPE_F32 && dtype != LMH_DTYPE_BF16) || !workspace)
    return LMH_ERR_INVALID_ARG;
  if (!opt->row_top_p && opt->top_p != opt->top_p) return LMH_ERR_INVALID_ARG;
  if (!opt->row_min_p && opt->min_p != opt->min_p) return LMH_ERR_INVALID_ARG;
  if (shape->N > 0 && (!logits || !u || !tokens)) return LMH_ERR_INVALID_ARG;
  const uintptr_t esize = dtype == LMH_DTYPE_F32 ? 4 : 2;
  if ((reinterpret_cast<uintptr_t>(logits) & (esize - 1)) != 0 || !aligned4(u) || !aligned4(tokens) ||
      !aligned4(logprob) || !aligned4(opt->row_top_k) || !aligned4(opt->row_top_p) ||
      !aligned4(opt->row_min_p) || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) != 0)
    return LMH_ERR_ALIGNMENT;
  if (workspace_bytes < lmh_workspace_size(shape, LMH_ENTRY_SAMPLE)) return LMH_ERR_WORKSPACE_TOO_SMALL;
  int dev, sms;
  LMH_TRY(current_device(&dev, &sms));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const Ws ws{static_cast<uint8_t*>(workspace), static_cast<WsHeader*>(workspace)};
  if (shape->N == 0) return clear_header(ws, st);  // else the first kernel clears the error word
  SampParams p{};
  p.N = shape->N;
  p.V = static_cast<int>(shape->V);
  p.blocks = static_cast<int>(cdiv(shape->V, kBlock));
  const SampSpace space = sample_space(shape->N, shape->V);
  p.gmax = ws.at<float>(space.gmax);
  p.gsum = ws.at<double>(space.gsum);
  p.rsum = ws.at<double>(space.rsum);
  int bits = 0;  // V <= 2^bits weights of up to 2^F stay below 2^62
  while ((1LL << bits) < shape->V) ++bits;
  p.F = 62 - bits < 50 ? 62 - bits : 50;
  p.logits = logits;
  p.u = u;
  p.tau = shape->temperature > 0.f ? shape->temperature : 1.f;
  p.row_tau = shape->row_temperature;
  p.top_k = opt->top_k;
  p.top_p = opt->top_p;
  p.min_p = opt->min_p;
  p.row_top_k = opt->row_top_k;
  p.row_top_p = opt->row_top_p;
  p.row_min_p = opt->row_min_p;
  p.tokens = tokens;
  p.logprob = logprob;
  p.err = &ws.h->err;
  // from the scalars alone the host sees when no row can be left to the row kernel
  const bool filtered = opt->row_top_k || opt->row_top_p || opt->row_min_p ||
                        (opt->top_k > 0 && opt->top_k < shape->V) || opt->top_p < 1.f || opt->min_p > 0.f;
  const bool may_leave = shape->V > kSampList && filtered;
  return dtype == LMH_DTYPE_F32 ? run_sample<float>(p, may_leave, dev, st)
                                : run_sample<__nv_bfloat16>(p, may_leave, dev, st);
}
