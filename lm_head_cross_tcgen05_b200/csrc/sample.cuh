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
// prefix of that order, so what is kept is (key, id): the last candidate of the shortest prefix.
// A prefix that reaches a count (top-k) or a weight (top-p) is found by a histogram over 2048
// linear buckets of (zmax - z) / tau, whose threshold bucket's few members go to the first CTA and
// are ranked there. A bucket with too many members (equal logits, mostly) is split again by the
// bits of its keys until they fit or are all equal; equal ones are counted in vocabulary order.
#pragma once

#include <cuda_bf16.h>

#include "rowops.cuh"

namespace lmh {

constexpr uint32_t kErrSampling = 0x10u;
constexpr int kSampThreads = 512, kSampWarps = kSampThreads / 32;
constexpr int kSampBuckets = 2048;
constexpr int kSampList = 1024;   // members of a threshold bucket that are ranked at once
constexpr int kSampMaxC = 8;

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
      u64 list[kSampList], sorted[kSampList];  // (key << 32 | ~id), on the cluster's first CTA
    };
  };
  uint32_t chist[kSampBuckets];
  double table[64];                        // 2^(j / 64)
  u64 tot_c[kSampMaxC], tot_w[kSampMaxC];  // per CTA, written by each into all
  u64 tot_l[kSampMaxC];                    // the same, of locate()
  u64 red[2][kSampWarps];
  u64 warp_sum[kSampWarps];
  u64 found[4];                            // bucket, its count, count before, weight before
  u64 cut[2];                              // (key << 32 | ~id) of the last kept, weight kept
  u64 idx;
  uint32_t list_n;
};

// What a row's threads share about it.
struct SampRow {
  float zmax;
  double zmaxd, inv_tau, inv_tau_log2;
  float half_max, bucket_scale;  // zmax / 2, 2 * 2048 / F * log2(e) / tau
  int F;
  const double* table;

  __device__ __forceinline__ int bucket(float z) const {
    // monotone in z, as each of the two roundings is; halved, no finite difference overflows
    const float x = fmaf(-0.5f, z, half_max) * bucket_scale;
    return x < static_cast<float>(kSampBuckets) ? static_cast<int>(x) : kSampBuckets;
  }
  __device__ __forceinline__ double scaled(float z) const { return (static_cast<double>(z) - zmaxd) * inv_tau; }
  // 2^F exp((z - zmax) / tau): 2^(n / 64) from the table times a Taylor polynomial of e^r with
  // |r| <= ln2 / 128, whose first left-out term is below 4e-17
  __device__ __forceinline__ u64 weight(float z) const {
    const double y = (static_cast<double>(z) - zmaxd) * inv_tau_log2;
    const int n = __double2int_rn(y * 64.0);
    const double r = fma(static_cast<double>(n), -1.0 / 64.0, y) * 0.6931471805599453;
    double e = fma(r, 1.0 / 120.0, 1.0 / 24.0);
    e = fma(r, e, 1.0 / 6.0);
    e = fma(r, e, 0.5);
    e = fma(r, e, 1.0);
    e = fma(r, e, 1.0);
    const int ex = F + (n >> 6);
    if (ex < -2) return 0;
    return __double2ull_rn(e * table[n & 63] * __hiloint2double((1023 + ex) << 20, 0));
  }
};

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

template <class T>
__global__ void __launch_bounds__(kSampThreads) sample_kernel(const SampParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  SampShared& sh = *reinterpret_cast<SampShared*>(dyn);
  T* chunk = reinterpret_cast<T*>(dyn + sizeof(SampShared));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int C = p.C;
  const long long row = blockIdx.x / C;
  const int c0 = static_cast<int>(min(static_cast<long long>(rank) * p.L, static_cast<long long>(p.V)));
  const int len = min(p.L, p.V - c0);
  const T* gsrc = static_cast<const T*>(p.logits) + row * p.V + c0;
  const T* src = p.resident ? chunk : gsrc;

  // before any CTA writes another's shared memory, all have started
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  // ---- the row's largest logit, and whether any is NaN
  uint32_t kmax = 0, bad = 0;
  for (int i = tid; i < len; i += kSampThreads) {
    const T t = gsrc[i];
    if (p.resident) chunk[i] = t;
    const float z = as_float(t);
    bad |= z != z;
    kmax = max(kmax, sort_key(z));
  }
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  for (int i = tid; i < kSampBuckets; i += kSampThreads) {
    sh.whist[i] = 0;
    sh.chist[i] = 0;
  }
  if (tid == 0) sh.list_n = 0;
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) sh.red[0][warp] = (static_cast<u64>(bad) << 32) | kmax;
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  __syncthreads();
  if (tid < C) {
    u64 m = 0;
    for (int w = 0; w < kSampWarps; ++w) m = max(m, sh.red[0][w]);  // a NaN above every key
    dsm_st64(&sh.tot_c[rank], tid, m);
  }
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
  long long k = p.row_top_k ? p.row_top_k[row] : p.top_k;
  if (k <= 0 || k >= p.V) k = 0;
  float top_p = p.row_top_p ? p.row_top_p[row] : p.top_p;
  float min_p = p.row_min_p ? p.row_min_p[row] : p.min_p;
  float u = p.u[row];
  if (top_p != top_p || min_p != min_p || !(u >= 0.f && u < 1.f)) flag |= kErrSampling;
  const bool use_p = top_p < 1.f;  // NaN: off
  const double log_min = min_p > 0.f ? log(fmin(static_cast<double>(min_p), 1.0)) : -HUGE_VAL;
  const double ud = u >= 0.f ? static_cast<double>(u) : 0.0;  // NaN: 0
  if (flag && rank == 0 && tid == 0) atomicOr(p.err, flag);

  R.zmaxd = R.zmax;
  R.inv_tau = 1.0 / tau;
  R.inv_tau_log2 = 1.4426950408889634 / tau;
  R.half_max = 0.5f * R.zmax;
  R.bucket_scale = static_cast<float>(fmin(R.inv_tau_log2 * (2.0 * kSampBuckets / p.F), 3e38));
  R.F = p.F;
  R.table = sh.table;

  // ---- histogram of counts and weights; all weights
  const bool cuts = k > 0 || use_p;
  u64 total = 0;
  for (int i = tid; i < len; i += kSampThreads) {
    const float z = as_float(src[i]);
    const int b = R.bucket(z);
    if (b < kSampBuckets) {
      const u64 w = R.weight(z);
      total += w;
      if (cuts) {
        atomicAdd(&sh.chist[b], 1u);
        atomicAdd(&sh.whist[b], w);
      }
    }
  }

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
  // over the row does); -1 where another CTA holds it. Each warp has a contiguous segment.
  const int seg = ((len + kSampThreads - 1) / kSampThreads) * 32;
  auto locate = [&](auto f, auto target) -> int {
    u64 s = 0;
    const int s0 = warp * seg, s1 = min(len, s0 + seg);
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
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int i = i0 + lane;
      const u64 x = warp_scan64(i < s1 ? f(as_float(src[i]), c0 + i) : 0, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, r < base + x);
      if (hit) return c0 + i0 + __ffs(hit) - 1;
      base += __shfl_sync(0xffffffffu, x, 31);
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
          atomicAdd(&sh.whist[(khi - key) >> shift], R.weight(z));
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
    // the members go to the first CTA and are ranked
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
      for (int i = tid; i < n; i += kSampThreads) {
        const u64 x = sh.list[i];
        int at = 0;
        for (int j = 0; j < n; ++j) at += sh.list[j] > x;
        sh.sorted[at] = x;
      }
      __syncthreads();
      u64 w[2] = {0, 0}, c[2] = {0, 0}, pc, pw, tc, tw;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (tid * 2 + j < n) {
          w[j] = R.weight(key_value(static_cast<uint32_t>(sh.sorted[tid * 2 + j] >> 32)));
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
            dsm_st64(&sh.cut[0], r, sh.sorted[tid * 2 + j]);
            dsm_st64(&sh.cut[1], r, pw);
          }
      }
      if (tid == 0) sh.list_n = 0;
    }
    samp_sync();
  };

  u64 cut = 0;  // nothing is cut: every (key, id) is above
  merge(&before_c, &before_w, &all_c, &all_w);
  if (cuts) {
    u64 kept_w = all_w;
    if (k > 0 && all_c >= static_cast<u64>(k)) {
      search(false, k, hc, hw, before_c, before_w);
      finish(false, k);
      cut = sh.cut[0];
      kept_w = sh.cut[1];
      samp_sync();  // cut and found are read before they are written again
    }
    if (use_p) {
      u64 target = top_p > 0.f ? __double2ull_ru(static_cast<double>(top_p) * static_cast<double>(kept_w)) : 1;
      target = target < 1 ? 1 : (target > kept_w ? kept_w : target);
      search(true, target, hc, hw, before_c, before_w);
      finish(true, target);
      cut = max(cut, sh.cut[0]);
      samp_sync();
    }
  }

  // ---- the token
  const int id = locate(
      [&](float z, int i) -> u64 {
        const u64 x = (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~i);
        if (x < cut || R.bucket(z) >= kSampBuckets || R.scaled(z) < log_min) return 0;
        return R.weight(z);
      },
      [&](u64 all) -> u64 {
        const u64 r = static_cast<u64>(ud * static_cast<double>(all));
        return r < all ? r : all - 1;
      });
  // all weights, for the log-prob
  total = warp_sum64(total);
  __syncthreads();
  if (lane == 0) sh.red[0][warp] = total;
  __syncthreads();
  if (tid < C) {
    u64 t = 0;
    for (int w = 0; w < kSampWarps; ++w) t += sh.red[0][w];
    dsm_st64(&sh.tot_w[rank], tid, t);
  }
  samp_sync();
  if (id >= 0 && lane == 0) {
    u64 t = 0;
    for (int r = 0; r < C; ++r) t += sh.tot_w[r];
    p.tokens[row] = id;
    if (p.logprob)
      p.logprob[row] = static_cast<float>(R.scaled(as_float(src[id - c0])) - (log(static_cast<double>(t)) - R.F * 0.6931471805599453));
  }
}

}  // namespace lmh
