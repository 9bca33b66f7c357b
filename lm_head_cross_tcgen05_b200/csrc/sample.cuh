// sample.cuh — one token per row of logits, by inversion of the filtered softmax at a given
// uniform number. A cluster of 1, 2, 4 or 8 CTAs takes one row: each holds a contiguous chunk of
// the vocabulary in shared memory (or, where it does not fit, reads it again from global memory),
// so the row crosses memory once.
//
// All sums are of whole numbers, so no order of addition can change a result: the weight of logit
// z is w(z) = round(2^F exp((z - zmax) / tau)), computed in fp64, with 2^F as large as V weights
// can be added in 63 bits (F = 44 for a vocabulary of 152 thousand, at most 50). A token whose
// probability is below 2^-F of the most likely one's counts as impossible.
//
// Candidates are ordered by logit, the largest first, equal ones by id. Every filter keeps a
// prefix of that order. Two ways to the token:
//  * The list. Where the kept prefix is short, everything that can be in it goes to the first CTA
//    (up to 1024 candidates), which sorts, filters and draws. What can be in a top-k prefix is
//    bounded by the maxima of groups of the row's elements: at least k elements lie at or above
//    the k-th largest group maximum. A top-p prefix without top-k needs the sum of all weights;
//    here that sum is formed in fp32 (fast_weight) with a bound on its error, and the row goes
//    the other way if the bound leaves the prefix's end open.
//  * The whole row. A prefix that reaches a count or a weight is found by a histogram over 2048
//    linear buckets of (zmax - z) / tau, whose threshold bucket's few members go to the first CTA
//    and are sorted there. A bucket with too many members (equal logits, mostly) is split again
//    by the bits of its keys until they fit or are all equal; equal ones are counted in
//    vocabulary order. What is kept is then (key, id) of the prefix's last candidate.
#pragma once

#include <cuda_bf16.h>

#include "rowops.cuh"

namespace lmh {

constexpr uint32_t kErrSampling = 0x10u;
constexpr int kSampThreads = 512, kSampWarps = kSampThreads / 32;
constexpr int kSampBuckets = 2048;
constexpr int kSampList = 1024;   // candidates that the first CTA sorts
constexpr int kSampListK = 512;   // largest top-k that takes the list
constexpr int kSampGroups = kSampThreads / 4;  // group maxima per CTA
constexpr int kSampMaxC = 8;
constexpr int kFastF = 40;        // fast weights are fractions of 2^40

struct SampParams {
  long long N;
  int V, L, C;          // row length, chunk per CTA, CTAs per row
  int F;                // weights are fractions of 2^F
  int resident;         // the chunk is copied to shared memory
  const void* logits;   // [N, V]
  const float* u;       // [N]
  float tau;            // scalar temperature (1: none)
  const float* row_tau; // or null
  int top_k;
  float top_p, min_p;
  const int32_t* row_top_k;  // each or null: used instead of the scalar
  const float* row_top_p;
  const float* row_min_p;
  int32_t* tokens;      // [N]
  float* logprob;       // [N] or null
  uint32_t* err;
};

typedef unsigned long long u64;

__device__ __forceinline__ void samp_sync() {
  __syncwarp();  // the cluster barrier wants whole warps
  cluster_sync();
}

// ---- distributed shared memory (the address is this CTA's own; rank picks the CTA)
__device__ __forceinline__ void dsm_st64(const void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_to_rank(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void dsm_st32f(const void* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(p), rank)), "f"(v) : "memory");
}
__device__ __forceinline__ u64 dsm_ld64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t dsm_ld32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t dsm_add32(const void* p, uint32_t rank, uint32_t x) {
  uint32_t v;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)), "r"(x) : "memory");
  return v;
}

// Order-preserving bits of a float (-0 as +0): larger key, larger value.
__device__ __forceinline__ uint32_t sort_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

struct SampShared {
  union {
    u64 whist[kSampBuckets];  // dead once merge() has brought its sums into registers
    struct {
      u64 list[kSampList];    // (key << 32 | ~id), on the cluster's first CTA
      u64 wlist[kSampList];   // their weights, once sorted
    };
  };
  uint32_t chist[kSampBuckets];
  float gmax[kSampMaxC * kSampGroups];     // every CTA's group maxima
  double table[64];                        // 2^(j / 64)
  u64 tot_c[kSampMaxC], tot_w[kSampMaxC];  // per CTA, written by each into all
  u64 tot_l[kSampMaxC], tot_f[kSampMaxC];  // the same, of locate() and of the fast weights
  u64 red[2][kSampWarps];
  u64 warp_sum[kSampWarps];
  u64 found[4];                            // bucket, its count, count before, weight before
  u64 cut[2];                              // (key << 32 | ~id) of the last kept, weight kept
  u64 verdict;
  uint32_t list_n;
  int pick[4];
};

// What a row's threads share about it.
struct SampRow {
  double zmaxd, c64;             // zmax; 64 log2(e) / tau
  float half_max, bucket_scale;  // zmax / 2, 2 * 2048 / F * log2(e) / tau
  float zmax, c32;               // 2 log2(e) / tau
  int F;
  const double* table;

  __device__ __forceinline__ int bucket(float z) const {
    // monotone in z, as each of the two roundings is; halved, no finite difference overflows
    const float x = fmaf(-0.5f, z, half_max) * bucket_scale;
    return x < static_cast<float>(kSampBuckets) ? static_cast<int>(x) : kSampBuckets;
  }
  // 64 log2 of the probability over the largest one's
  __device__ __forceinline__ double y64(float z) const { return (static_cast<double>(z) - zmaxd) * c64; }
  // 2^F 2^(y / 64): with n the whole number next to y and g = (y - n) ln2 / 64, the table's
  // 2^(n / 64) times the Taylor polynomial of e^g, |g| <= ln2 / 128, whose first left-out term
  // is below 4e-17. Whole numbers are taken from the low bits of sums with 2^52, which costs an
  // addition where a conversion of 64-bit types runs at a fraction of that rate.
  __device__ __forceinline__ u64 weight(float z) const {
    const double y = y64(z);
    if (y < -64.0 * (F + 1)) return 0;
    const double m = y + 6755399441055744.0;  // 1.5 * 2^52
    const int n = __double2loint(m);
    const double f = y - (m - 6755399441055744.0);
    constexpr double a = 0.6931471805599453 / 64;
    double e = fma(f, a * a * a * a * a / 120, a * a * a * a / 24);
    e = fma(f, e, a * a * a / 6);
    e = fma(f, e, a * a / 2);
    e = fma(f, e, a);
    e = fma(f, e, 1.0);
    const double tb = table[n & 63];
    const double sc = __hiloint2double(__double2hiint(tb) + ((F + (n >> 6)) << 20), __double2loint(tb));
    return static_cast<u64>(__double_as_longlong(fma(e, sc, 4503599627370496.0))) - 0x4330000000000000ull;
  }
  // 2^40 2^(y / 64) in fp32. Relative error: 2^-22 of ex2.approx, and y / 64 (of magnitude below
  // F <= 50) is off by three roundings, 50 * 3 * 2^-24 * ln2 < 2^-17; the sum of the two and of the
  // 2^-41 of the rounding is below kFastErr of a row's sum for V < 2^21.
  __device__ __forceinline__ u64 fast_weight(float z) const {
    return __float2ull_rn(fast_exp2(-fmaf(-0.5f, z, half_max) * c32) * 1099511627776.f);
  }
};
constexpr double kFastErr = 1.0 / 65536;
constexpr int kFastMaxV = 1 << 21;

__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ u64 warp_scan64(u64 x, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Exclusive prefix of two values over the block's threads, and their totals.
__device__ __forceinline__ void block_scan2(u64 a, u64 b, u64* pa, u64* pb, u64* ta, u64* tb, u64 (*red)[kSampWarps]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 ia = warp_scan64(a, lane), ib = warp_scan64(b, lane);
  __syncthreads();
  if (lane == 31) {
    red[0][warp] = ia;
    red[1][warp] = ib;
  }
  __syncthreads();
  u64 ba = 0, bb = 0, sa = 0, sb = 0;
  for (int w = 0; w < kSampWarps; ++w) {
    if (w == warp) {
      ba = sa;
      bb = sb;
    }
    sa += red[0][w];
    sb += red[1][w];
  }
  *pa = ba + ia - a;
  *pb = bb + ib - b;
  *ta = sa;
  *tb = sb;
}

// Sorts a[0 .. P) in descending order; P a power of two, at most 2 * kSampThreads. All threads.
__device__ __forceinline__ void bitonic_desc(u64* a, int P) {
  for (int size = 2; size <= P; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      const int t = threadIdx.x;
      if (t < P / 2) {
        const int i = 2 * t - (t & (stride - 1)), j = i + stride;
        const u64 x = a[i], y = a[j];
        if ((x < y) == ((i & size) == 0)) {
          a[i] = y;
          a[j] = x;
        }
      }
      if (P > 64) __syncthreads();  // up to 64 are warp 0's own
      else __syncwarp();
    }
  __syncthreads();
}

// f(z, i) over the chunk, 16 bytes a load where the row's alignment allows. `mis`: elements by
// which p lies past a 16-byte boundary.
template <class T, class Fn>
__device__ __forceinline__ void for_chunk(const T* p, int len, int mis, Fn f) {
  constexpr int E = 16 / sizeof(T);
  const int head = min(len, mis ? E - mis : 0);
  const int nv = (len - head) / E;
  if (static_cast<int>(threadIdx.x) < head) f(as_float(p[threadIdx.x]), static_cast<int>(threadIdx.x));
  const uint4* v = reinterpret_cast<const uint4*>(p + head);
#pragma unroll 2
  for (int j = threadIdx.x; j < nv; j += kSampThreads) {
    const uint4 w = v[j];
    const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int q = 0; q < E; ++q) f(as_float(e[q]), head + j * E + q);
  }
  const int i = head + nv * E + threadIdx.x;
  if (i < len) f(as_float(p[i]), i);
}

template <class T>
__global__ void __launch_bounds__(kSampThreads, 2) sample_kernel(const SampParams p) {
  constexpr int E = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t dyn[];
  SampShared& sh = *reinterpret_cast<SampShared*>(dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int C = p.C;
  const long long row = blockIdx.x / C;
  const int c0 = static_cast<int>(min(static_cast<long long>(rank) * p.L, static_cast<long long>(p.V)));
  const int len = min(p.L, p.V - c0);
  const T* gsrc = static_cast<const T*>(p.logits) + row * p.V + c0;
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(gsrc) & 15) / sizeof(T));
  T* chunk = reinterpret_cast<T*>(dyn + sizeof(SampShared)) + mis;  // aligned as the row is
  const T* src = p.resident ? chunk : gsrc;

  // before any CTA writes another's shared memory, all have started
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ---- the row, its largest logit, whether any is NaN, and the maxima of groups of 4 threads
  float tmax = -INFINITY;
  bool bad = false;
  {
    const int head = min(len, mis ? E - mis : 0);
    const int nv = (len - head) / E;
    auto one = [&](int i) {
      const T t = gsrc[i];
      if (p.resident) chunk[i] = t;
      const float z = as_float(t);
      bad |= z != z;
      tmax = fmaxf(tmax, z);
    };
    if (tid < head) one(tid);
    if (head + nv * E + tid < len) one(head + nv * E + tid);
    const uint4* gv = reinterpret_cast<const uint4*>(gsrc + head);
    uint4* sv = reinterpret_cast<uint4*>(chunk + head);
    for (int j0 = tid; j0 < nv; j0 += 4 * kSampThreads) {
      uint4 w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j0 + q * kSampThreads < nv) w[q] = p.resident ? __ldcs(gv + j0 + q * kSampThreads) : gv[j0 + q * kSampThreads];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j0 + q * kSampThreads < nv) {
          if (p.resident) sv[j0 + q * kSampThreads] = w[q];
          const T* e = reinterpret_cast<const T*>(&w[q]);
#pragma unroll
          for (int x = 0; x < E; ++x) {
            const float z = as_float(e[x]);
            bad |= z != z;
            tmax = fmaxf(tmax, z);
          }
        }
    }
  }
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  if (tid == 0) sh.list_n = 0;
  float gm = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, 1));
  gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, 2));
  const uint32_t kmax = __reduce_max_sync(0xffffffffu, sort_key(gm));
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) sh.red[0][warp] = (static_cast<u64>(bad) << 32) | kmax;
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if ((lane & 3) == 0)
    for (int r = 0; r < C; ++r) dsm_st32f(&sh.gmax[rank * kSampGroups + (tid >> 2)], r, gm);
  if (tid < C) {
    u64 m = 0;
    for (int w = 0; w < kSampWarps; ++w) m = max(m, sh.red[0][w]);  // a NaN above every key
    dsm_st64(&sh.tot_c[rank], tid, m);
  }
  for (int i = tid; i < kSampBuckets; i += kSampThreads) sh.chist[i] = 0;
  samp_sync();
  u64 m = 0;
  for (int r = 0; r < C; ++r) m = max(m, sh.tot_c[r]);
  SampRow R;
  R.zmax = key_value(static_cast<uint32_t>(m));
  if ((m >> 32) != 0 || !(fabsf(R.zmax) <= 3.402823466e38f)) {  // no finite log-sum-exp
    if (rank == 0 && tid == 0) {
      p.tokens[row] = -1;
      if (p.logprob) p.logprob[row] = 0.f;
      atomicOr(p.err, kErrNonFinite);
    }
    return;  // the same decision in every CTA; none reads another's memory any more
  }

  // ---- parameters
  uint32_t flag = 0;
  double tau = p.tau;
  if (p.row_tau) {
    const float t = p.row_tau[row];
    if (temperature_ok(t)) tau *= t;
    else flag |= kErrTemperature;
  }
  int k = p.row_top_k ? p.row_top_k[row] : p.top_k;
  if (k <= 0 || k >= p.V) k = 0;
  const float top_p = p.row_top_p ? p.row_top_p[row] : p.top_p;
  const float min_p = p.row_min_p ? p.row_min_p[row] : p.min_p;
  const float u = p.u[row];
  if (top_p != top_p || min_p != min_p || !(u >= 0.f && u < 1.f)) flag |= kErrSampling;
  const bool use_p = top_p < 1.f;  // NaN: off
  const bool use_m = min_p > 0.f;
  const double low64 = use_m ? 64.0 * log2(fmin(static_cast<double>(min_p), 1.0)) : -HUGE_VAL;
  const double ud = u >= 0.f ? static_cast<double>(u) : 0.0;  // NaN: 0
  if (flag && rank == 0 && tid == 0) atomicOr(p.err, flag);

  const double c = 1.4426950408889634 / tau;
  R.zmaxd = R.zmax;
  R.c64 = 64.0 * c;
  R.c32 = static_cast<float>(fmin(2.0 * c, 3e38));
  R.half_max = 0.5f * R.zmax;
  R.bucket_scale = static_cast<float>(fmin(c * (2.0 * kSampBuckets / p.F), 3e38));
  R.F = p.F;
  R.table = sh.table;

  auto log_prob = [&](float z, u64 total, int f) {  // total in units of 2^-f
    return static_cast<float>((R.y64(z) / 64.0 - (log2(static_cast<double>(total)) - f)) * 0.6931471805599453);
  };
  auto draw_at = [&](u64 all) -> u64 {
    const u64 r = static_cast<u64>(ud * static_cast<double>(all));
    return r < all ? r : all - 1;
  };
  auto p_target = [&](u64 all) -> u64 {
    const u64 t = top_p > 0.f ? __double2ull_ru(static_cast<double>(top_p) * static_cast<double>(all)) : 1;
    return t < 1 ? 1 : (t > all ? all : t);
  };

  // ---- the list
  const bool all_listed = p.V <= kSampList;
  const bool filtered = k > 0 || use_p || use_m;
  bool fast = false;  // tot_f holds the fast weights' sums
  if (all_listed || (k > 0 ? k <= kSampListK : (use_p ? p.V < kFastMaxV : use_m))) {
    // candidates lie in the buckets up to b0
    int b0 = kSampBuckets - 1;
    const int want = k > 0 ? k : kSampListK / 2;
    if (!all_listed && (k > 0 || use_p)) {
      for (int i = tid; i < C * kSampGroups; i += kSampThreads) {
        const int b = R.bucket(sh.gmax[i]);
        if (b < kSampBuckets) atomicAdd(&sh.chist[b], 1u);
      }
      if (tid == 0) sh.pick[0] = kSampBuckets - 1;
      __syncthreads();
      uint4 h = *reinterpret_cast<const uint4*>(&sh.chist[tid * 4]);
      u64 pc, px, tc, tx;
      block_scan2(h.x + h.y + h.z + h.w, 0, &pc, &px, &tc, &tx, sh.red);
      const uint32_t hv[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (pc < static_cast<u64>(want) && static_cast<u64>(want) <= pc + hv[j]) sh.pick[0] = tid * 4 + j;
        pc += hv[j];
      }
      __syncthreads();
      b0 = sh.pick[0];
    }
    if (use_m && !use_p) {
      const double bm = -low64 / 64.0 * (kSampBuckets / static_cast<double>(p.F)) + 1.0;
      if (bm < b0) b0 = static_cast<int>(bm);
    }
    u64 sum = 0;
    fast = true;
    for_chunk(src, len, mis, [&](float z, int i) {
      const int b = R.bucket(z);
      if (b <= b0) {
        const uint32_t at = dsm_add32(&sh.list_n, 0, 1);
        if (at < kSampList) dsm_st64(&sh.list[at], 0, (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~(c0 + i)));
      }
      if (b < kSampBuckets) sum += R.fast_weight(z);
    });
    sum = warp_sum64(sum);
    __syncthreads();
    if (lane == 0) sh.red[0][warp] = sum;
    __syncthreads();
    if (tid < C) {
      u64 t = 0;
      for (int w = 0; w < kSampWarps; ++w) t += sh.red[0][w];
      dsm_st64(&sh.tot_f[rank], tid, t);
    }
    samp_sync();
    if (rank == 0) {
      const int n = static_cast<int>(min(sh.list_n, static_cast<uint32_t>(kSampList)));
      bool ok = sh.list_n <= kSampList;
      u64 fsum = 0;
      for (int r = 0; r < C; ++r) fsum += sh.tot_f[r];
      if (ok) {  // uniform over the block
        int P = 2;
        while (P < n) P <<= 1;
        for (int i = n + tid; i < P; i += kSampThreads) sh.list[i] = 0;
        __syncthreads();
        bitonic_desc(sh.list, P);
        // this thread's two candidates, and the weight before them
        u64 w[2] = {0, 0}, pw, px, tw, tx;
        bool in_m[2] = {false, false};
        const int nk = k > 0 ? min(n, k) : n;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (tid * 2 + j < nk) {
            const float z = key_value(static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32));
            w[j] = R.weight(z);
            in_m[j] = R.y64(z) >= low64;
            sh.wlist[tid * 2 + j] = w[j];
          }
        block_scan2(w[0] + w[1], static_cast<u64>(in_m[0]) + in_m[1], &pw, &px, &tw, &tx, sh.red);
        // kept: nk by count, tx by min-p, and by top-p the first whose running weight reaches the
        // target; without top-k and with more candidates than the list's, the target is only
        // known to lie in [t0, t1]
        u64 t0 = tw, t1 = tw;
        if (use_p) {
          if (k > 0 || all_listed) {
            t0 = t1 = p_target(tw);
          } else {
            const double s = static_cast<double>(top_p > 0.f ? top_p : 0.f) * static_cast<double>(fsum) *
                             __hiloint2double((1023 + p.F - kFastF) << 20, 0);
            t0 = max(static_cast<u64>(s * (1.0 - kFastErr)), 1ull);
            t1 = static_cast<u64>(s * (1.0 + kFastErr)) + 2;
            if (top_p <= 0.f) t1 = 1;
          }
        }
        if (tid < 2) sh.pick[tid] = -1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (pw < t0 && t0 <= pw + w[j]) sh.pick[0] = tid * 2 + j;
          if (pw < t1 && t1 <= pw + w[j]) sh.pick[1] = tid * 2 + j;
          pw += w[j];
        }
        __syncthreads();
        int nkeep = min(nk, static_cast<int>(tx));
        if (use_p) {
          ok = sh.pick[0] >= 0 && sh.pick[0] == sh.pick[1];
          nkeep = min(nkeep, sh.pick[0] + 1);
        }
        if (ok) {
          // in the order of the ids
          u64 x[2] = {0, 0};
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (tid * 2 + j < nkeep) x[j] = (sh.list[tid * 2 + j] << 32) | static_cast<uint32_t>(tid * 2 + j);
          __syncthreads();
          P = 2;
          while (P < nkeep) P <<= 1;
          if (tid * 2 < P) {
            sh.list[tid * 2] = x[0];
            sh.list[tid * 2 + 1] = x[1];
          }
          __syncthreads();
          bitonic_desc(sh.list, P);
          w[0] = tid * 2 < nkeep ? sh.wlist[static_cast<uint32_t>(sh.list[tid * 2])] : 0;
          w[1] = tid * 2 + 1 < nkeep ? sh.wlist[static_cast<uint32_t>(sh.list[tid * 2 + 1])] : 0;
          block_scan2(w[0] + w[1], 0, &pw, &px, &tx, &px, sh.red);
          const u64 r = draw_at(tx);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (pw <= r && r < pw + w[j]) {
              const int id = static_cast<int>(~static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32));
              p.tokens[row] = id;
              if (p.logprob) {
                const float z = as_float(static_cast<const T*>(p.logits)[row * p.V + id]);
                p.logprob[row] = log_prob(z, fsum, kFastF);
              }
            }
            pw += w[j];
          }
        }
      }
      __syncthreads();
      if (tid == 0) sh.list_n = 0;
      if (tid < C) dsm_st64(&sh.verdict, tid, ok ? 1 : 0);
    }
    samp_sync();
    if (sh.verdict) return;  // in every CTA alike; none reads another's memory any more
  }

  // ---- the whole row
  for (int i = tid; i < kSampBuckets; i += kSampThreads) {
    sh.whist[i] = 0;
    sh.chist[i] = 0;
  }
  __syncthreads();

  // Merges the CTAs' histograms: this thread's buckets of this CTA's slice (up to 4), what lies
  // before them over the whole cluster, and the cluster's totals.
  const int slice = kSampBuckets / C;
  u64 hc[4], hw[4], before_c, before_w, all_c, all_w;
  auto merge = [&](u64* bc, u64* bw, u64* tc, u64* tw) {
    samp_sync();  // every CTA's histogram is complete
    u64 sc = 0, sw = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hc[j] = hw[j] = 0;
      const int per = (slice + kSampThreads - 1) / kSampThreads;
      const int b = tid * per + j;
      if (j < per && b < slice) {
        for (int r = 0; r < C; ++r) {
          hc[j] += dsm_ld32(&sh.chist[rank * slice + b], r);
          hw[j] += dsm_ld64(&sh.whist[rank * slice + b], r);
        }
        sc += hc[j];
        sw += hw[j];
      }
    }
    u64 xc, xw;
    block_scan2(sc, sw, bc, bw, &xc, &xw, sh.red);
    if (tid < C) {
      dsm_st64(&sh.tot_c[rank], tid, xc);
      dsm_st64(&sh.tot_w[rank], tid, xw);
    }
    samp_sync();
    *tc = *tw = 0;
    for (int r = 0; r < C; ++r) {
      if (r == static_cast<int>(rank)) {
        *bc += *tc;
        *bw += *tw;
      }
      *tc += sh.tot_c[r];
      *tw += sh.tot_w[r];
    }
  };
  // The bucket in which the running count (by_w false) or weight reaches `target` (which the
  // totals reach): sh.found = bucket, members, count before, weight before; in every CTA.
  auto search = [&](bool by_w, u64 target, const u64* c, const u64* w, u64 bc, u64 bw) {
    const int per = (slice + kSampThreads - 1) / kSampThreads;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 lo = by_w ? bw : bc, hi = lo + (by_w ? w[j] : c[j]);
      if (lo < target && target <= hi)
        for (int r = 0; r < C; ++r) {
          dsm_st64(&sh.found[0], r, static_cast<u64>(rank * slice + tid * per + j));
          dsm_st64(&sh.found[1], r, c[j]);
          dsm_st64(&sh.found[2], r, bc);
          dsm_st64(&sh.found[3], r, bw);
        }
      bc += c[j];
      bw += w[j];
    }
    samp_sync();
  };
  // The id at which the running sum, in vocabulary order, of f(z, id) passes r (which the sum
  // over the row does); -1 where another warp holds it. Each warp has a contiguous segment.
  const int seg = ((len + kSampThreads - 1) / kSampThreads) * 32;
  auto locate = [&](auto f, auto target) -> int {
    u64 s = 0;
    const int s0 = min(len, warp * seg), s1 = min(len, s0 + seg);
#pragma unroll 4
    for (int i = s0 + lane; i < s1; i += 32) s += f(as_float(src[i]), c0 + i);
    s = warp_sum64(s);
    if (lane == 0) sh.warp_sum[warp] = s;
    __syncthreads();
    u64 mine = 0;
    for (int w = 0; w < kSampWarps; ++w) mine += sh.warp_sum[w];
    if (tid < C) dsm_st64(&sh.tot_l[rank], tid, mine);
    samp_sync();
    u64 base = 0, all = 0;
    for (int r = 0; r < C; ++r) {
      if (r < static_cast<int>(rank)) base += sh.tot_l[r];
      all += sh.tot_l[r];
    }
    const u64 r = target(all);
    for (int w = 0; w < warp; ++w) base += sh.warp_sum[w];
    if (!(base <= r && r < base + s)) return -1;
    // the lane whose run of the segment holds it, then the place in that run
    const int run = (s1 - s0 + 31) / 32;
    const int r0 = min(s1, s0 + lane * run), r1 = min(s1, r0 + run);
    u64 x = 0;
    for (int i = r0; i < r1; ++i) x += f(as_float(src[i]), c0 + i);
    const u64 incl = warp_scan64(x, lane);
    const int owner = __ffs(__ballot_sync(0xffffffffu, r < base + incl)) - 1;
    base += __shfl_sync(0xffffffffu, incl - x, owner);
    const int e1 = __shfl_sync(0xffffffffu, r1, owner);
    for (int i0 = __shfl_sync(0xffffffffu, r0, owner); i0 < e1; i0 += 32) {
      const int i = i0 + lane;
      const u64 y = warp_scan64(i < e1 ? f(as_float(src[i]), c0 + i) : 0, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, r < base + y);
      if (hit) return c0 + i0 + __ffs(hit) - 1;
      base += __shfl_sync(0xffffffffu, y, 31);
    }
    return -1;
  };

  // Shortest prefix that reaches the target in the bucket sh.found: sh.cut in every CTA.
  auto finish = [&](bool by_w, u64 target) {
    const int bucket0 = static_cast<int>(sh.found[0]);
    u64 members = sh.found[1], bc = sh.found[2], bw = sh.found[3];
    uint32_t klo = 0, khi = 0xffffffffu;
    // 2048 ranges a level: after three levels a range is one key
    for (int level = 0; level < 4 && members > kSampList; ++level) {
      // the members' smallest and largest key
      uint32_t lo = 0xffffffffu, hi = 0;
      for (int i = tid; i < len; i += kSampThreads) {
        const float z = as_float(src[i]);
        const uint32_t key = sort_key(z);
        if (key >= klo && key <= khi && R.bucket(z) == bucket0) {
          lo = min(lo, key);
          hi = max(hi, key);
        }
      }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      __syncthreads();
      if (lane == 0) {
        sh.red[0][warp] = lo;
        sh.red[1][warp] = hi;
      }
      for (int i = tid; i < kSampBuckets; i += kSampThreads) {
        sh.whist[i] = 0;
        sh.chist[i] = 0;
      }
      __syncthreads();
      if (tid < C) {
        u64 a = 0xffffffffu, b = 0;
        for (int w = 0; w < kSampWarps; ++w) {
          a = min(a, sh.red[0][w]);
          b = max(b, sh.red[1][w]);
        }
        dsm_st64(&sh.tot_c[rank], tid, a);
        dsm_st64(&sh.tot_w[rank], tid, b);
      }
      samp_sync();
      klo = 0xffffffffu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, static_cast<uint32_t>(sh.tot_c[r]));
        khi = max(khi, static_cast<uint32_t>(sh.tot_w[r]));
      }
      if (klo == khi) {  // equal logits: the first ones in vocabulary order
        const u64 w = R.weight(key_value(klo));
        const u64 need = by_w ? (target - bw + w - 1) / w : target - bc;
        const int id = locate([&](float z, int) -> u64 { return sort_key(z) == klo; }, [&](u64) -> u64 { return need - 1; });
        if (id >= 0 && lane == 0)
          for (int r = 0; r < C; ++r) {
            dsm_st64(&sh.cut[0], r, (static_cast<u64>(klo) << 32) | static_cast<uint32_t>(~id));
            dsm_st64(&sh.cut[1], r, bw + need * w);
          }
        samp_sync();
        return;
      }
      const int shift = max(0, 32 - __clz(khi - klo) - 11);
      for (int i = tid; i < len; i += kSampThreads) {
        const float z = as_float(src[i]);
        const uint32_t key = sort_key(z);
        if (key >= klo && key <= khi && R.bucket(z) == bucket0) {
          atomicAdd(&sh.chist[(khi - key) >> shift], 1u);
          if (use_p) atomicAdd(&sh.whist[(khi - key) >> shift], R.weight(z));
        }
      }
      u64 c2[4], w2[4], b2c, b2w, t2c, t2w;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c2[j] = hc[j];
        w2[j] = hw[j];
      }
      merge(&b2c, &b2w, &t2c, &t2w);
      search(by_w, target, hc, hw, bc + b2c, bw + b2w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // the linear histogram's buckets stay the thread's own
        hc[j] = c2[j];
        hw[j] = w2[j];
      }
      members = sh.found[1];
      bc = sh.found[2];
      bw = sh.found[3];
      khi -= static_cast<uint32_t>(sh.found[0]) << shift;
      const uint32_t low = khi - ((1u << shift) - 1);
      klo = low > khi ? klo : max(klo, low);
      samp_sync();  // found is read before a next search writes it
    }
    // the members go to the first CTA and are sorted
    for (int i = tid; i < len; i += kSampThreads) {
      const float z = as_float(src[i]);
      const uint32_t key = sort_key(z);
      if (key >= klo && key <= khi && R.bucket(z) == bucket0) {
        const uint32_t at = dsm_add32(&sh.list_n, 0, 1);
        if (at < kSampList) dsm_st64(&sh.list[at], 0, (static_cast<u64>(key) << 32) | static_cast<uint32_t>(~(c0 + i)));
      }
    }
    samp_sync();
    if (rank == 0) {
      const int n = static_cast<int>(min(members, static_cast<u64>(kSampList)));
      int P = 2;
      while (P < n) P <<= 1;
      for (int i = n + tid; i < P; i += kSampThreads) sh.list[i] = 0;
      __syncthreads();
      bitonic_desc(sh.list, P);
      u64 w[2] = {0, 0}, c[2] = {0, 0}, pc, pw, tc, tw;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (tid * 2 + j < n) {
          w[j] = R.weight(key_value(static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32)));
          c[j] = 1;
        }
      block_scan2(c[0] + c[1], w[0] + w[1], &pc, &pw, &tc, &tw, sh.red);
      pc += bc;
      pw += bw;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const u64 lo = by_w ? pw : pc;
        pc += c[j];
        pw += w[j];
        const u64 hi = by_w ? pw : pc;
        if (lo < target && target <= hi)
          for (int r = 0; r < C; ++r) {
            dsm_st64(&sh.cut[0], r, sh.list[tid * 2 + j]);
            dsm_st64(&sh.cut[1], r, pw);
          }
      }
      if (tid == 0) sh.list_n = 0;
    }
    samp_sync();
  };

  u64 cut = 0;  // nothing is cut: every (key, id) is above
  if (k > 0 || use_p || (use_m && !fast)) {
    u64 sum = 0;
    for_chunk(src, len, mis, [&](float z, int) {
      const int b = R.bucket(z);
      if (b < kSampBuckets) {
        if (!fast) sum += R.fast_weight(z);
        if (k > 0 || use_p) atomicAdd(&sh.chist[b], 1u);
        if (use_p) atomicAdd(&sh.whist[b], R.weight(z));
      }
    });
    if (!fast) {
      sum = warp_sum64(sum);
      __syncthreads();
      if (lane == 0) sh.red[0][warp] = sum;
      __syncthreads();
      if (tid < C) {
        u64 t = 0;
        for (int w = 0; w < kSampWarps; ++w) t += sh.red[0][w];
        dsm_st64(&sh.tot_f[rank], tid, t);
      }
    }
  }
  if (k > 0 || use_p) {
    merge(&before_c, &before_w, &all_c, &all_w);
    u64 kept_w = all_w;
    if (k > 0 && all_c >= static_cast<u64>(k)) {
      search(false, k, hc, hw, before_c, before_w);
      finish(false, k);
      cut = sh.cut[0];
      kept_w = sh.cut[1];
      samp_sync();  // cut and found are read before they are written again
    }
    if (use_p) {
      const u64 target = p_target(kept_w);
      search(true, target, hc, hw, before_c, before_w);
      finish(true, target);
      cut = max(cut, sh.cut[0]);
    }
  }

  // ---- the token
  const int id = locate(
      [&](float z, int i) -> u64 {
        if (filtered) {
          const u64 x = (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~i);
          if (x < cut || R.y64(z) < low64) return 0;
        }
        return R.weight(z);
      },
      draw_at);
  if (id >= 0 && lane == 0) {
    u64 exact = 0, rough = 0;
    for (int r = 0; r < C; ++r) {
      exact += sh.tot_l[r];
      rough += sh.tot_f[r];
    }
    p.tokens[row] = id;
    if (p.logprob)
      p.logprob[row] = filtered ? log_prob(as_float(src[id - c0]), rough, kFastF) : log_prob(as_float(src[id - c0]), exact, R.F);
  }
}

}  // namespace lmh
