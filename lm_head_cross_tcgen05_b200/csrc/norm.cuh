// norm.cuh — the final RMS norm with the residual's addition (bf16 output, or e4m3 with one scale
// per row and 128 columns), its backward pass, and the e4m3 quantisation of matrices by blocks.
// All are HBM bound: each row is held in registers between its two uses, so every tensor crosses
// memory once. Sums are fp32 in a fixed order (a thread's elements in ascending order, then a
// butterfly over the warp, then one over the warps): no result depends on the device.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "rowops.cuh"

namespace lmh {

constexpr int kNormMaxD = 16384;   // 512 threads x 4 vectors of 8
constexpr int kQBlock = 128;       // columns per scale
constexpr float kE4m3Max = 448.f;
constexpr float kAmaxFloor = 7.888609052210118e-31f;  // 2^-100

// Larger of m and |x|, NaN if either is: a NaN reaches its block's scale.
__device__ __forceinline__ float max_abs(float m, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(x)));
  return r;
}

// Scale of a block with this largest magnitude: max(amax, 2^-100) / 448, as a product with 1 / 448
// (off by at most 2^-23 of itself). The floor keeps the scale and its reciprocal normal numbers,
// for a block of zeros too; NaN stays NaN.
__device__ __forceinline__ float block_scale(float amax) {
  return amax < kAmaxFloor ? kAmaxFloor / kE4m3Max : amax * (1.f / kE4m3Max);
}

// Eight values times 1 / scale, rounded to nearest even e4m3 (saturating; NaN stays NaN). The
// scale's, the reciprocal's and the product's roundings move a quotient by less than 2^-21 of
// itself, so a block's largest value still becomes 448; eight divisions instead bound the kernels
// (quantising 151936 x 5120 took 706 us with them, 430 without).
__device__ __forceinline__ uint2 to_e4m3x8(const float (&y)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __nv_fp8x2_storage_t a =
        __nv_cvt_float2_to_fp8x2(make_float2(y[4 * h] * inv, y[4 * h + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t b =
        __nv_cvt_float2_to_fp8x2(make_float2(y[4 * h + 2] * inv, y[4 * h + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[h] = static_cast<uint32_t>(a) | (static_cast<uint32_t>(b) << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack_bf16x2(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// bf16 sums, each rounded once (the unit adds in fp32).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s = __hadd2_rn(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
  return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

// Sum over the block's threads (whole warps, 16 at most): every thread gets it. The warps' sums
// are added by a butterfly too.
__device__ __forceinline__ float row_sum(float x, float* s) {
  x = warp_sum(x);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return x;
  const int lane = threadIdx.x & 31;
  if (lane == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = lane < warps ? s[lane] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return __shfl_sync(0xffffffffu, x, 0);
}

// Rows on their way from memory: every thread copies its own vectors of the next rows to its own
// places in shared memory and waits for its own copies alone, so a ring of rows needs no barrier.
// What bounds these kernels is the number of bytes under way; registers hold one row at most.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Rows of the ring, that under work included. Forward: 64 KB a block at most where a thread has one
// vector, 96 KB with two, 192 KB with four; backward: 96, 144 and 192 KB.
__host__ __device__ constexpr int norm_stages(int vpt) { return vpt == 1 ? 4 : 3; }
__host__ __device__ constexpr int norm_bwd_stages(int vpt) { return vpt == 1 ? 4 : (vpt == 2 ? 3 : 2); }

struct NormParams {
  long long N;
  int d;
  float eps, inv_d;
  const uint4* x;
  const uint4* residual;  // or null
  const uint4* weight;
  uint4* sum;      // or null; may be x or residual
  uint4* y;        // or null
  uint2* q;        // or null
  float* scale;    // [N, ceil(d / 128)], with q
  float* rstd;     // or null
};

// Row blockIdx.x + i * gridDim.x; VPT vectors of 8 per thread at v = threadIdx.x + j * blockDim.x.
// The sum is rounded to bf16 before the norm: the norm is that of the stream as it is stored,
// which is what the backward pass and a next layer read. A scale's 16 vectors lie in 16 adjacent
// lanes (blockDim.x is a multiple of 32), so the block's maximum is four shuffles. Rows come
// through a ring of asynchronous copies, which keeps loads under way while a row waits for its sum:
// 4096 x 5120 with a residual to e4m3 28 us (147 MB, 5.3 TB/s; 35 without the ring), 8192 x 4096
// to bf16 40 us (268 MB, 6.7 TB/s, part of the writes still in L2).
template <int VPT>
__global__ void __launch_bounds__(512) rms_norm_kernel(const NormParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sh[2][32];
  constexpr int S = norm_stages(VPT);
  const int nv = p.d >> 3, nb = (p.d + kQBlock - 1) / kQBlock;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t tensor = blockDim.x * VPT * 16, stage = 2 * tensor;
  auto fetch = [&](long long row, int at) {
    if (row < p.N)
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < nv) {
          const uint32_t dst = mine + at * stage + j * blockDim.x * 16;
          copy_async16(dst, p.x + row * nv + v);
          if (p.residual) copy_async16(dst + tensor, p.residual + row * nv + v);
        }
      }
    copy_commit();  // empty past the last row: the groups are counted
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(blockIdx.x + static_cast<long long>(i) * gridDim.x, i);
  float w[VPT][8];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    unpack8(v < nv ? __ldg(p.weight + v) : make_uint4(0, 0, 0, 0), w[j]);
  }
  int at = 0, flip = 0;
  for (long long row = blockIdx.x; row < p.N; row += gridDim.x, at = (at + 1) % S, flip ^= 1) {
    const long long base = row * nv;
    fetch(row + static_cast<long long>(S - 1) * gridDim.x, (at + S - 1) % S);
    copy_wait<S - 1>();
    uint4 s[VPT];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      const uint32_t src = mine + at * stage + j * blockDim.x * 16;
      s[j] = v < nv ? ld_shared_v4(src) : make_uint4(0, 0, 0, 0);
      if (p.residual && v < nv) s[j] = add8(s[j], ld_shared_v4(src + tensor));
      float a[8];
      unpack8(s[j], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], ss);
    }
    ss = row_sum(ss, sh[flip]);  // a barrier lies between the uses of either half
    const float rstd = rsqrtf(fmaf(ss, p.inv_d, p.eps));
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      const bool in = v < nv;
      float a[8];
      unpack8(s[j], a);
      if (in && p.sum) p.sum[base + v] = s[j];
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] = a[e] * rstd * w[j][e];  // 0 (or NaN, as the row) past the row's end
      if (in && p.y) p.y[base + v] = pack8(a);
      if (p.q) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_abs(m, a[e]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float sc = block_scale(m);
        if (in) {
          p.q[base + v] = to_e4m3x8(a, __fdividef(1.f, sc));
          if ((v & 15) == 0) p.scale[row * nb + (v >> 4)] = sc;
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- backward
// With n = r rstd and c = mean(w dy n):  dx = rstd (w dy - n c) + dsum,  dw = sum_rows dy n.
// Slice blockIdx.x of the rows, one row at a time; a thread keeps its columns' share of dw in
// registers over the slice and leaves it in part[slice]. The slices depend on N and d alone.

struct NormBwdParams {
  long long N;
  int d, slices;
  const uint4* sum;
  const uint4* weight;
  const float* rstd;
  float inv_d;
  const uint4* dy;
  const uint4* dsum;  // or null
  uint4* dx;          // or null; may be dy or dsum
  float* part;        // [slices, d], or null
  WsHeader* h;
};

// A slice of rows per block of threads, which holds dweight's share of its columns in registers.
// With n = r rstd: dx = rstd (w dy - n mean(w dy n)) + dsum. 8192 x 4096 with dsum: 49 us (268 MB,
// 5.5 TB/s) and 7 us for the sum over the slices.
template <int VPT>
__global__ void __launch_bounds__(512, VPT == 1 ? 2 : 1) rms_norm_bwd_kernel(const NormBwdParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float sh[2][32];
  constexpr int S = norm_bwd_stages(VPT);
  if (blockIdx.x == 0 && threadIdx.x == 0) p.h->err = 0;
  const int nv = p.d >> 3;
  const long long r0 = p.N * blockIdx.x / p.slices, r1 = p.N * (blockIdx.x + 1) / p.slices;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const uint32_t tensor = blockDim.x * VPT * 16, stage = 3 * tensor;
  auto fetch = [&](long long row, int at) {
    if (row < r1)
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        const int v = threadIdx.x + j * blockDim.x;
        if (v < nv) {
          const uint32_t dst = mine + at * stage + j * blockDim.x * 16;
          copy_async16(dst, p.sum + row * nv + v);
          copy_async16(dst + tensor, p.dy + row * nv + v);
          if (p.dsum) copy_async16(dst + 2 * tensor, p.dsum + row * nv + v);
        }
      }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) fetch(r0 + i, i);
  float acc[VPT][8] = {};
  uint4 w[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    w[j] = v < nv ? __ldg(p.weight + v) : make_uint4(0, 0, 0, 0);
  }
  int at = 0, flip = 0;
  for (long long row = r0; row < r1; ++row, at = (at + 1) % S, flip ^= 1) {
    const long long base = row * nv;
    const float rstd = p.rstd[row];
    fetch(row + S - 1, (at + S - 1) % S);
    copy_wait<S - 1>();
    uint4 s[VPT], g[VPT];
    float c = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      const uint32_t src = mine + at * stage + j * blockDim.x * 16;
      s[j] = v < nv ? ld_shared_v4(src) : make_uint4(0, 0, 0, 0);
      g[j] = v < nv ? ld_shared_v4(src + tensor) : make_uint4(0, 0, 0, 0);
      float r[8], dy[8], wf[8];
      unpack8(s[j], r);
      unpack8(g[j], dy);
      unpack8(w[j], wf);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dn = dy[e] * (r[e] * rstd);  // n is of order one, whatever the row's size
        c = fmaf(wf[e], dn, c);
        acc[j][e] += dn;
      }
    }
    if (!p.dx) continue;
    c = row_sum(c, sh[flip]) * p.inv_d;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = threadIdx.x + j * blockDim.x;
      if (v >= nv) continue;
      float r[8], dy[8], wf[8], ds[8];
      unpack8(s[j], r);
      unpack8(g[j], dy);
      unpack8(w[j], wf);
      unpack8(p.dsum ? ld_shared_v4(mine + at * stage + j * blockDim.x * 16 + 2 * tensor) : make_uint4(0, 0, 0, 0), ds);
#pragma unroll
      for (int e = 0; e < 8; ++e) ds[e] = fmaf(rstd, fmaf(-c, r[e] * rstd, wf[e] * dy[e]), ds[e]);
      p.dx[base + v] = pack8(ds);
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = threadIdx.x + j * blockDim.x;
    if (v >= nv) continue;
    float4* o = reinterpret_cast<float4*>(p.part + static_cast<long long>(blockIdx.x) * p.d + v * 8);
    o[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
    o[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
  }
}

// dweight = bf16(sum over the slices): 32 columns per block, threadIdx.y sums every 16th slice in
// ascending order, then the 16 sums are added in ascending order.
__global__ void __launch_bounds__(512) norm_dweight_kernel(int slices, int d,
                                                           const float* __restrict__ part,
                                                           __nv_bfloat16* __restrict__ dweight) {
  __shared__ float sh[16][32];
  const int c = blockIdx.x * 32 + threadIdx.x;  // d is a multiple of 64
  float a = 0.f;
#pragma unroll 8
  for (int s = threadIdx.y; s < slices; s += 16) a += part[static_cast<long long>(s) * d + c];
  sh[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y != 0) return;
  a = 0.f;
  for (int i = 0; i < 16; ++i) a += sh[i][threadIdx.x];
  dweight[c] = __float2bfloat16_rn(a);
}

// ---------------------------------------------------------------------------- quantisation
// One scale per row and 128 columns: 16 adjacent lanes hold a block. `per` threads (whole warps) a
// row, four vectors of each under way.
__global__ void __launch_bounds__(256) quantize_rows_kernel(long long rows, int d, int per,
                                                            const uint4* __restrict__ x,
                                                            uint2* __restrict__ q,
                                                            float* __restrict__ scale) {
  const int nb = (d + kQBlock - 1) / kQBlock, nv = d >> 3, l = threadIdx.x % per;
  const long long row = static_cast<long long>(blockIdx.x) * (256 / per) + threadIdx.x / per;
  if (row >= rows) return;  // whole warps
  for (int c = l - (l & 31); c < nv; c += 4 * per) {
    uint4 t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = c + j * per + (l & 31);
      t[j] = v < nv ? __ldcs(x + row * nv + v) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int v = c + j * per + (l & 31);
      float a[8], m = 0.f;
      unpack8(t[j], a);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_abs(m, a[e]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float sc = block_scale(m);
      if (v < nv) {
        q[row * nv + v] = to_e4m3x8(a, __fdividef(1.f, sc));
        if ((v & 15) == 0) scale[row * nb + (v >> 4)] = sc;
      }
    }
  }
}

// One scale per 128 x 128 block, one block of threads each: 16 lanes per row, 8 rows a thread, four
// blocks an SM (151936 x 5120: 345 us, 6.8 TB/s; 430 us with the three that 85 registers leave).
__global__ void __launch_bounds__(256, 4) quantize_blocks_kernel(long long rows, int d,
                                                              const uint4* __restrict__ x,
                                                              uint2* __restrict__ q,
                                                              float* __restrict__ scale) {
  __shared__ float sh[8];
  const int nb = (d + kQBlock - 1) / kQBlock, nv = d >> 3;
  const long long rb = blockIdx.x / nb;
  const int b = static_cast<int>(blockIdx.x - rb * nb);
  const int v = b * 16 + (threadIdx.x & 15);
  const long long r0 = rb * kQBlock + (threadIdx.x >> 4);
  uint4 t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long r = r0 + 16 * i;
    t[i] = (r < rows && v < nv) ? __ldcs(x + r * nv + v) : make_uint4(0, 0, 0, 0);
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a[8];
    unpack8(t[i], a);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_abs(m, a[e]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) m = max_abs(m, sh[w]);
  const float sc = block_scale(m);
  const float inv = __fdividef(1.f, sc);
  if (threadIdx.x == 0) scale[rb * nb + b] = sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const long long r = r0 + 16 * i;
    if (r < rows && v < nv) {
      float a[8];
      unpack8(t[i], a);
      q[r * nv + v] = to_e4m3x8(a, inv);
    }
  }
}

}  // namespace lmh
