// sample.cuh — one token per row of logits, by inversion of the filtered softmax at a given
// uniform number. Candidates are ordered by logit, the largest first, equal ones by id; every
// filter keeps a prefix of that order. Three kernels:
//
//  * sample_groups_kernel streams the logits once: the maximum of every 32 of a row, and the sum
//    of exponentials of every 256 relative to their own maximum. This is the pass that is bound
//    by memory; no thread waits for another beyond its warp.
//  * sample_list_kernel, one CTA per row, draws the token from those records and a few logits.
//    Unfiltered, the running sums of the groups lead to the one whose 256 logits decide. With a
//    short prefix, everything that can be in it is collected and sorted (up to 1024 candidates):
//    at least k logits lie at or above the k-th largest group maximum, so only groups whose
//    maximum lies there are read again, 128 bytes for most of k candidates. A top-p prefix
//    without top-k ends where the candidates' weight reaches a part of the whole sum, which is
//    known from fp32 exponentials within a bound; if that does not decide it, the row is left.
//  * sample_row_kernel takes the rows left over (long prefixes), a cluster of 1 to 8 CTAs each. A
//    prefix that reaches a count or a weight is found by a histogram over 2048 linear buckets of
//    (zmax - z) / tau, whose threshold bucket's few members go to the first CTA and are sorted
//    there. Adding every weight to its bucket in shared memory would cost more than the rest, so
//    counts of an eighth of the row first give a window of buckets; the pass over the row adds
//    what lies above the window in registers and only the window's weights to buckets, and is
//    repeated with all buckets if the prefix does not end in the window. A bucket with too many
//    members (equal logits, mostly) is split again by the bits of its keys until they fit or are
//    all equal; equal ones are counted in vocabulary order.
//
// Where a token depends on sums of weights, the weights are whole numbers, so that no order of
// addition can change it: w(z) = round(2^F exp((z - zmax) / tau)), computed in fp64, with 2^F as
// large as V weights can be added in 63 bits (F = 44 for a vocabulary of 152 thousand, at most
// 50). A token whose probability is below 2^-F of the most likely one's counts as impossible.
#pragma once

#include <cuda_bf16.h>

#include "rowops.cuh"

namespace lmh {

constexpr uint32_t kErrSampling = 0x10u;
constexpr int kSampThreads = 512, kSampWarps = kSampThreads / 32;
constexpr int kSampBuckets = 2048;
constexpr int kSampList = 1024;   // candidates that the first CTA sorts
constexpr int kSampListK = 512;   // largest top-k that takes the list
constexpr int kSampMaxC = 8;
constexpr int kGroup = 32;        // logits per maximum
constexpr int kSum = 256;         // logits per sum
constexpr int kBatch = 16;        // groups that a warp of the row kernel loads at once
constexpr int kParts = 64;        // partial sums per warp that locate() keeps
constexpr int kSampPending = -2;  // tokens[row] of a row that the list kernel leaves

struct SampParams {
  long long N;
  int V, C;             // row length; row kernel: CTAs per row
  int F;                // weights are fractions of 2^F
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
  int g32, g256;        // groups per row
  float* gmax;          // [N, g32] largest logit of each 32 (NaN if one is)
  double* gsum;         // [N, g256] sum of exp((z - max) / tau) over each 256, max their largest
  double* rsum;         // [N] sum of exp((z - zmax) / tau), of the rows left by the list kernel
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
__device__ __forceinline__ uint4 dsm_ld128(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(map_to_rank(smem_u32(p), rank)) : "memory");
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

struct ListShared {
  double table[64];
  u64 red[2][kSampWarps];
  double dred[kSampWarps];
  u64 list[kSampList];       // candidates, key << 32 | ~id
  u64 wlist[kSampList];      // their weights, once sorted
  uint32_t queue[kSampList]; // groups that hold candidates
  uint4 chist[kSampBuckets / 4];
  uint32_t list_n, queue_n;
  int pick[2];
  u64 base;
};
struct RowShared {
  double table[64];
  u64 red[2][kSampWarps];
  u64 whist[kSampBuckets];
  uint4 chist[kSampBuckets / 4];
  u64 list[kSampList];                       // members of a bucket, on the cluster's first CTA
  u64 part[kSampWarps][kParts];              // locate(): partial sums of each warp's segment
  u64 tot_a[kSampMaxC], tot_b[kSampMaxC];    // per CTA, written by each into all
  u64 tot_l[kSampMaxC];                      // the same, of locate()
  u64 found[4];                              // bin, its members, count before, weight before
  u64 cut;                                   // (key << 32 | ~id) of the last kept
  uint32_t list_n;
  int hit, window[2];
};

// 2^up 2^(y / 64) as e * sc: with n the whole number next to y and g = (y - n) ln2 / 64, the
// table's 2^(n / 64) times the Taylor polynomial of e^g, |g| <= ln2 / 128, whose first left-out
// term is below 4e-17. |y| < 2^31 and a normal result.
__device__ __forceinline__ void exp2_64(double y, int up, const double* table, double* e, double* sc) {
  const double m = y + 6755399441055744.0;  // 1.5 * 2^52: the low bits hold n
  const int n = __double2loint(m);
  const double f = y - (m - 6755399441055744.0);
  constexpr double a = 0.6931471805599453 / 64;
  double x = fma(f, a * a * a * a * a / 120, a * a * a * a / 24);
  x = fma(f, x, a * a * a / 6);
  x = fma(f, x, a * a / 2);
  x = fma(f, x, a);
  *e = fma(f, x, 1.0);
  const double tb = table[n & 63];
  *sc = __hiloint2double(__double2hiint(tb) + ((up + (n >> 6)) << 20), __double2loint(tb));
}

// What a row's threads share about it.
struct SampRow {
  double zmaxd, c64;             // zmax; 64 log2(e) / tau
  float half_max, bucket_scale;  // zmax / 2, 2 * 2048 / F * log2(e) / tau
  int F;
  const double* table;

  __device__ __forceinline__ int bucket(float z) const {
    // monotone in z, as each of the two roundings is; halved, no finite difference overflows
    const float x = fmaf(-0.5f, z, half_max) * bucket_scale;
    return x < static_cast<float>(kSampBuckets) ? static_cast<int>(x) : kSampBuckets;
  }
  // 64 log2 of the probability over the largest one's
  __device__ __forceinline__ double y64(float z) const { return (static_cast<double>(z) - zmaxd) * c64; }
  // 2^F 2^(y / 64) as a whole number, read from the low bits of a sum with 2^52: an addition
  // where a conversion of 64-bit types runs at a fraction of that rate
  __device__ __forceinline__ u64 weight(float z) const {
    const double y = y64(z);
    if (y < -64.0 * (F + 1)) return 0;
    double e, sc;
    exp2_64(y, F, table, &e, &sc);
    return static_cast<u64>(__double_as_longlong(fma(e, sc, 4503599627370496.0))) - 0x4330000000000000ull;
  }
};
// Bound on the relative error of a row's sum of fp32 exponentials 2^y: 2^-22 of ex2.approx, four
// roundings of y (|y| <= 50 where it matters), 50 * 4 * 2^-24 * ln2 < 2^-16.8, and 13 additions
// (2^-24 each).
constexpr double kFastErr = 1.0 / 65536;

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

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A row's parameters, off where they do nothing.
struct SampFilter {
  int k;            // 0: off
  float top_p;
  bool use_p, use_m;
  double tau, ud, low64;  // low64: 64 log2(min_p)
  uint32_t flag;
  __device__ __forceinline__ SampFilter(const SampParams& p, long long row) {
    flag = 0;
    tau = p.tau;
    if (p.row_tau) {
      const float t = p.row_tau[row];
      if (temperature_ok(t)) tau *= t;
      else flag |= kErrTemperature;
    }
    k = p.row_top_k ? p.row_top_k[row] : p.top_k;
    if (k <= 0 || k >= p.V) k = 0;
    top_p = p.row_top_p ? p.row_top_p[row] : p.top_p;
    const float min_p = p.row_min_p ? p.row_min_p[row] : p.min_p;
    const float u = p.u[row];
    if (top_p != top_p || min_p != min_p || !(u >= 0.f && u < 1.f)) flag |= kErrSampling;
    use_p = top_p < 1.f;  // NaN: off
    use_m = min_p > 0.f;
    low64 = use_m ? 64.0 * log2(fmin(static_cast<double>(min_p), 1.0)) : -HUGE_VAL;
    ud = u >= 0.f ? static_cast<double>(u) : 0.0;  // NaN: 0
  }
  __device__ __forceinline__ u64 draw_at(u64 all) const {
    const u64 r = static_cast<u64>(ud * static_cast<double>(all));
    return r < all ? r : all - 1;
  }
  __device__ __forceinline__ u64 p_target(u64 all) const {
    const u64 t = top_p > 0.f ? __double2ull_ru(static_cast<double>(top_p) * static_cast<double>(all)) : 1;
    return t < 1 ? 1 : (t > all ? all : t);
  }
  // Whether the list kernel may draw the row: nothing is filtered, or the prefix may be short.
  __device__ __forceinline__ bool listed(int V) const { return V <= kSampList || k <= kSampListK; }
  __device__ __forceinline__ bool exact() const { return k == 0 && !use_p && !use_m; }
};
// SampFilter::exact() of a row: its groups' sums alone decide the token, so they are fp64.
__device__ __forceinline__ bool samp_exact(const SampParams& p, long long row) {
  const int k = p.row_top_k ? p.row_top_k[row] : p.top_k;
  const float top_p = p.row_top_p ? p.row_top_p[row] : p.top_p;
  const float min_p = p.row_min_p ? p.row_min_p[row] : p.min_p;
  return (k <= 0 || k >= p.V) && !(top_p < 1.f) && !(min_p > 0.f);
}

__device__ __forceinline__ SampRow samp_row(const SampParams& p, float zmax, double tau, const double* table) {
  const double c = 1.4426950408889634 / tau;
  SampRow R;
  R.zmaxd = zmax;
  R.c64 = 64.0 * c;
  R.half_max = 0.5f * zmax;
  R.bucket_scale = static_cast<float>(fmin(c * (2.0 * kSampBuckets / p.F), 3e38));
  R.F = p.F;
  R.table = table;
  return R;
}
__device__ __forceinline__ bool no_sum(const SampParams& p, long long row, float zmax, bool writer) {
  if (fabsf(zmax) <= 3.402823466e38f) return false;
  if (writer) {  // no finite log-sum-exp
    p.tokens[row] = -1;
    if (p.logprob) p.logprob[row] = 0.f;
    atomicOr(p.err, kErrNonFinite);
  }
  return true;
}

// total: the sum of the row's weights, the largest one's being 1
__device__ __forceinline__ float samp_logprob(const SampRow& R, float z, double total) {
  return static_cast<float>((R.y64(z) / 64.0 - log2(total)) * 0.6931471805599453);
}

__device__ __forceinline__ float warp_max_nan(float x) {
  float r;
  asm("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// One warp per 256 logits of a row at a time, two such under way.
constexpr int kGroupWarps = 8, kGroupPer = 2;
template <class T>
__global__ void __launch_bounds__(32 * kGroupWarps) sample_groups_kernel(const SampParams p) {
  __shared__ double table[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = (p.g256 + kGroupWarps * kGroupPer - 1) / (kGroupWarps * kGroupPer);
  const long long row = blockIdx.x / per_row;
  const int g0 = (static_cast<int>(blockIdx.x - row * per_row) * kGroupWarps + warp) * kGroupPer;
  const T* src = static_cast<const T*>(p.logits) + row * p.V;
  float z[kGroupPer][8];
#pragma unroll
  for (int q = 0; q < kGroupPer; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long i = static_cast<long long>(g0 + q) * kSum + j * kGroup + lane;
      z[q][j] = i < p.V ? as_float(src[i]) : -INFINITY;
    }
  float tau = 1.f;
  if (p.row_tau) {
    tau = p.row_tau[row];
    if (!temperature_ok(tau)) tau = 1.f;
  }
  const bool exact = samp_exact(p, row);  // of the whole block
  if (exact) {
    if (threadIdx.x < 64) table[threadIdx.x] = exp2(threadIdx.x / 64.0);
    __syncthreads();
  }
  const double c64 = exact ? 64.0 * 1.4426950408889634 / (static_cast<double>(tau) * p.tau) : 0.0;
  const float c2 = fminf(2.8853900817779268f / p.tau / tau, 3e38f);  // 2 log2(e) / tau
#pragma unroll
  for (int q = 0; q < kGroupPer; ++q) {
    if (g0 + q >= p.g256) break;
    float mine = -INFINITY, m = -INFINITY;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = warp_max_nan(z[q][j]);
      if (lane == j) mine = x;
      m = max_nan(m, x);
    }
    const int g = (g0 + q) * 8 + lane;
    if (lane < 8 && g < p.g32) p.gmax[row * p.g32 + g] = mine;
    double s = 0.0;
    if (fabsf(m) <= 3.402823466e38f) {  // else no finite logit, or the row has no finite sum
      if (exact) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double y = (static_cast<double>(z[q][j]) - m) * c64;
          double e = 0.0, sc = 0.0;
          if (y > -64.0 * 100) exp2_64(y, 0, table, &e, &sc);  // less cannot be drawn
          s = fma(e, sc, s);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      } else {
        float e = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float x = fmaf(-0.5f, z[q][j], 0.5f * m);
          e += x < INFINITY ? fast_exp2(-x * c2) : 0.f;  // c2 may be 0
        }
        s = warp_sum(e);
      }
    }
    if (lane == 0) p.gsum[row * p.g256 + g0 + q] = s;
  }
}

template <class T>
__global__ void __launch_bounds__(kSampThreads) sample_list_kernel(const SampParams p) {
  __shared__ ListShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x;
  const SampFilter f(p, row);
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  if (tid < 2) sh.pick[tid] = kSampBuckets - 1;
  if (tid == 0) sh.list_n = sh.queue_n = 0;
  for (int i = tid; i < kSampBuckets / 4; i += kSampThreads) sh.chist[i] = make_uint4(0, 0, 0, 0);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the groups' records
  const T* src = static_cast<const T*>(p.logits) + row * p.V;
  const float* gmax = p.gmax + row * p.g32;
  const double* gsum = p.gsum + row * p.g256;

  float tmax = -INFINITY;
  for (int g = tid; g < p.g32; g += kSampThreads) tmax = max_nan(tmax, gmax[g]);
  tmax = warp_max_nan(tmax);
  if (lane == 0) sh.red[0][warp] = __float_as_uint(tmax);
  __syncthreads();
  float zmax = -INFINITY;
  for (int w = 0; w < kSampWarps; ++w) zmax = max_nan(zmax, __uint_as_float(static_cast<uint32_t>(sh.red[0][w])));
  if (no_sum(p, row, zmax, tid == 0)) return;
  if (f.flag && tid == 0) atomicOr(p.err, f.flag);
  const SampRow R = samp_row(p, zmax, f.tau, sh.table);
  // the largest logit of 256
  auto max256 = [&](int g) {
    float m = -INFINITY;
    for (int j = g * 8; j < min(g * 8 + 8, p.g32); ++j) m = fmaxf(m, gmax[j]);
    return m;
  };

  if (f.exact()) {
    // whole numbers of 2^-F again; each thread has a run of groups
    const double up = __hiloint2double((1023 + p.F) << 20, 0);
    const int run = (p.g256 + kSampThreads - 1) / kSampThreads;
    const int r0 = min(p.g256, tid * run), r1 = min(p.g256, r0 + run);
    auto group_weight = [&](int g) -> u64 {
      const double s = gsum[g];
      return s > 0.0 ? __double2ull_rn(s * exp2(R.y64(max256(g)) / 64.0) * up) : 0;
    };
    u64 s = 0, before, px, total, tx;
    for (int g = r0; g < r1; ++g) s += group_weight(g);
    block_scan2(s, 0, &before, &px, &total, &tx, sh.red);
    const u64 r = f.draw_at(total);
    if (before <= r && r < before + s) {
      int g = r0;
      for (; g < r1 - 1; ++g) {
        const u64 w = group_weight(g);
        if (r < before + w) break;
        before += w;
      }
      sh.pick[0] = g;
      sh.base = r - before;
    }
    __syncthreads();
    if (warp != 0) return;
    // within the group, 8 adjacent logits a lane; its weights' sum is its rounded sum up to their
    // own roundings, so a remainder past the last goes to the last that can be drawn
    const long long i0 = static_cast<long long>(sh.pick[0]) * kSum + lane * 8;
    const u64 rest = sh.base;
    u64 w[8], sum = 0;
    int last = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = i0 + j < p.V ? R.weight(as_float(src[i0 + j])) : 0;
      sum += w[j];
      if (w[j] > 0) last = j;
    }
    const u64 incl = warp_scan64(sum, lane);
    u64 at = incl - sum;
    int hit = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (hit < 0 && at <= rest && rest < at + w[j]) hit = j;
      at += w[j];
    }
    const uint32_t found = __ballot_sync(0xffffffffu, hit >= 0);
    const uint32_t can = __ballot_sync(0xffffffffu, last >= 0);
    const int owner = found ? __ffs(found) - 1 : (can ? 31 - __clz(can) : 0);
    if (lane == owner) {
      const long long id = i0 + (found ? hit : max(last, 0));
      p.tokens[row] = static_cast<int>(id);
      if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(src[id]), static_cast<double>(total) / up);
    }
    return;
  }

  // ---- the row's sum, in a fixed order
  double part = 0.0;
  for (int g = tid; g < p.g256; g += kSampThreads) {
    const double s = gsum[g];
    if (s > 0.0) part += s * exp2(R.y64(max256(g)) / 64.0);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) sh.dred[warp] = part;
  if (!f.listed(p.V)) {
    __syncthreads();
    if (tid == 0) {
      double total = 0.0;
      for (int w = 0; w < kSampWarps; ++w) total += sh.dred[w];
      p.rsum[row] = total;
      p.tokens[row] = kSampPending;
    }
    return;
  }

  // ---- candidates lie in the buckets up to b0
  const bool all_listed = p.V <= kSampList;
  int b0 = kSampBuckets - 1;
  if (!all_listed && (f.k > 0 || f.use_p)) {
    const u64 want = f.k > 0 ? f.k : kSampListK / 2;
    uint32_t* hist = reinterpret_cast<uint32_t*>(sh.chist);
    for (int g = tid; g < p.g32; g += kSampThreads) {
      const int b = R.bucket(gmax[g]);
      if (b < kSampBuckets) atomicAdd(&hist[b], 1u);
    }
    __syncthreads();
    const uint4 h = sh.chist[tid];
    const uint32_t hv[4] = {h.x, h.y, h.z, h.w};
    u64 pc, px, tc, tx;
    block_scan2(h.x + h.y + h.z + h.w, 0, &pc, &px, &tc, &tx, sh.red);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (pc < want && want <= pc + hv[j]) sh.pick[0] = tid * 4 + j;
      pc += hv[j];
    }
    __syncthreads();
    b0 = sh.pick[0];
  }
  if (f.use_m && !f.use_p) {
    const double bm = -f.low64 / 64.0 * (kSampBuckets / static_cast<double>(p.F)) + 1.0;
    if (bm < b0) b0 = static_cast<int>(bm);
  }
  for (int g = tid; g < p.g32; g += kSampThreads)
    if (R.bucket(gmax[g]) <= b0) {
      const uint32_t at = atomicAdd(&sh.queue_n, 1u);
      if (at < kSampList) sh.queue[at] = g;
    }
  __syncthreads();
  double total = 0.0;
  for (int w = 0; w < kSampWarps; ++w) total += sh.dred[w];
  // every queued group holds a candidate: more of them than the list holds leave the row
  const int groups = static_cast<int>(min(sh.queue_n, static_cast<uint32_t>(kSampList)));
  if (sh.queue_n <= kSampList) {
    for (int q0 = warp; q0 < groups; q0 += 4 * kSampWarps) {
      float z[4];
      int id[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int q = q0 + j * kSampWarps;
        id[j] = q < groups ? static_cast<int>(sh.queue[q]) * kGroup + lane : -1;
        const bool in = id[j] >= 0 && id[j] < p.V;
        z[j] = in ? as_float(src[id[j]]) : 0.f;
        if (!in) id[j] = -1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool hit = id[j] >= 0 && R.bucket(z[j]) <= b0;
        const uint32_t mask = __ballot_sync(0xffffffffu, hit);
        uint32_t at = 0;
        if (mask && lane == 0) at = atomicAdd(&sh.list_n, __popc(mask));
        at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1));
        if (hit && at < kSampList) sh.list[at] = (static_cast<u64>(sort_key(z[j])) << 32) | static_cast<uint32_t>(~id[j]);
      }
    }
  }
  __syncthreads();
  const int n = static_cast<int>(min(sh.list_n, static_cast<uint32_t>(kSampList)));
  bool ok = sh.queue_n <= kSampList && sh.list_n <= kSampList;  // alike in all threads, as every `ok` below
  if (ok) {
    int P = 2;
    while (P < n) P <<= 1;
    for (int i = n + tid; i < P; i += kSampThreads) sh.list[i] = 0;
    if (tid < 2) sh.pick[tid] = -1;
    __syncthreads();
    bitonic_desc(sh.list, P);
    // this thread's two candidates, and the weight before them
    u64 w[2] = {0, 0}, pw, px, tw, tx;
    bool in_m[2] = {false, false};
    const int nk = f.k > 0 ? min(n, f.k) : n;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (tid * 2 + j < nk) {
        const float z = key_value(static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32));
        w[j] = R.weight(z);
        in_m[j] = R.y64(z) >= f.low64;
        sh.wlist[tid * 2 + j] = w[j];
      }
    block_scan2(w[0] + w[1], static_cast<u64>(in_m[0]) + in_m[1], &pw, &px, &tw, &tx, sh.red);
    // kept: nk by count, tx by min-p, and by top-p up to the first whose running weight reaches
    // the target; without top-k and with candidates outside the list, the target is only known
    // to lie in [t0, t1]
    int nkeep = min(nk, static_cast<int>(tx));
    if (f.use_p) {
      u64 t0, t1;
      if (f.k > 0 || all_listed) {
        t0 = t1 = f.p_target(tw);
      } else if (!(f.top_p > 0.f)) {
        t0 = t1 = 1;
      } else {
        const double s = static_cast<double>(f.top_p) * total * __hiloint2double((1023 + p.F) << 20, 0);
        t0 = max(static_cast<u64>(s * (1.0 - kFastErr)), 1ull);
        t1 = static_cast<u64>(s * (1.0 + kFastErr)) + 2;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (pw < t0 && t0 <= pw + w[j]) sh.pick[0] = tid * 2 + j;
        if (pw < t1 && t1 <= pw + w[j]) sh.pick[1] = tid * 2 + j;
        pw += w[j];
      }
      __syncthreads();
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
#pragma unroll
      for (int j = 0; j < 2; ++j) w[j] = tid * 2 + j < nkeep ? sh.wlist[static_cast<uint32_t>(sh.list[tid * 2 + j])] : 0;
      block_scan2(w[0] + w[1], 0, &pw, &px, &tw, &tx, sh.red);
      const u64 r = f.draw_at(tw);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (pw <= r && r < pw + w[j]) {
          const int id = static_cast<int>(~static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32));
          p.tokens[row] = id;
          if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(src[id]), total);
        }
        pw += w[j];
      }
      return;
    }
  }
  if (tid == 0) {
    p.rsum[row] = total;
    p.tokens[row] = kSampPending;
  }
}

// One row per cluster; rows that are not pending cost an exit.
template <class T>
__global__ void __launch_bounds__(kSampThreads, 2) sample_row_kernel(const SampParams p) {
  __shared__ RowShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int C = p.C;
  const long long row = blockIdx.x / C;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list kernel's tokens
  if (p.tokens[row] != kSampPending) return;          // in every CTA alike
  cluster_arrive();  // before any CTA writes another's shared memory, all have started
  const SampFilter f(p, row);
  const T* src = static_cast<const T*>(p.logits) + row * p.V;
  const float* gmax = p.gmax + row * p.g32;
  uint32_t* chist = reinterpret_cast<uint32_t*>(sh.chist);
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  if (tid == 0) sh.list_n = 0;
  float zmax = -INFINITY;
  for (int g = tid; g < p.g32; g += kSampThreads) zmax = fmaxf(zmax, gmax[g]);  // finite: the list kernel saw it
  zmax = warp_max_nan(zmax);
  if (lane == 0) sh.red[0][warp] = __float_as_uint(zmax);
  __syncthreads();
  for (int w = 0; w < kSampWarps; ++w) zmax = fmaxf(zmax, __uint_as_float(static_cast<uint32_t>(sh.red[0][w])));
  const SampRow R = samp_row(p, zmax, f.tau, sh.table);
  cluster_wait();

  // groups [s0, s1) are this warp's: contiguous, in the order of the CTAs and their warps
  const int per_cta = (p.g32 + C - 1) / C;
  const int cta0 = min(p.g32, static_cast<int>(rank) * per_cta), cta1 = min(p.g32, cta0 + per_cta);
  const int per_warp = ((cta1 - cta0 + kSampWarps - 1) / kSampWarps + kBatch - 1) / kBatch * kBatch;
  const int s0 = min(cta1, cta0 + warp * per_warp), s1 = min(cta1, s0 + per_warp);
  // fn(z, id) for every logit of the batch's groups whose maximum passes `pred` (-inf past the
  // row's end)
  auto batch = [&](int b, auto pred, auto fn) {
    const bool mine = lane < kBatch && b + lane < s1;
    const uint32_t mask = __ballot_sync(0xffffffffu, mine && pred(mine ? gmax[b + lane] : 0.f));
    if (!mask) return;
    float z[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const long long i = static_cast<long long>(b + j) * kGroup + lane;
      z[j] = ((mask >> j) & 1) && i < p.V ? as_float(src[i]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if ((mask >> j) & 1) fn(z[j], (b + j) * kGroup + lane);
  };
  auto compose = [](float z, int id) { return (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~id); };
  // Sums over the row of two values per thread, in every thread of the cluster.
  auto sum2 = [&](u64 a, u64 b, u64* ta, u64* tb) {
    a = warp_sum64(a);
    b = warp_sum64(b);
    __syncthreads();
    if (lane == 0) {
      sh.red[0][warp] = a;
      sh.red[1][warp] = b;
    }
    __syncthreads();
    if (tid < C) {
      u64 x = 0, y = 0;
      for (int w = 0; w < kSampWarps; ++w) {
        x += sh.red[0][w];
        y += sh.red[1][w];
      }
      dsm_st64(&sh.tot_a[rank], tid, x);
      dsm_st64(&sh.tot_b[rank], tid, y);
    }
    samp_sync();
    *ta = *tb = 0;
    for (int r = 0; r < C; ++r) {
      *ta += sh.tot_a[r];
      *tb += sh.tot_b[r];
    }
  };
  auto zero = [&](bool w) {
    for (int i = tid; i < kSampBuckets / 4; i += kSampThreads) sh.chist[i] = make_uint4(0, 0, 0, 0);
    if (w)
      for (int i = tid; i < kSampBuckets; i += kSampThreads) sh.whist[i] = 0;
    __syncthreads();
  };
  // This thread's four bins of the cluster's histograms. The barrier before it has been passed.
  auto bins = [&](bool w, u64 (&hc)[4], u64 (&hw)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) hc[j] = hw[j] = 0;
    for (int r = 0; r < C; ++r) {
      const uint4 h = dsm_ld128(&sh.chist[tid], r);
      hc[0] += h.x;
      hc[1] += h.y;
      hc[2] += h.z;
      hc[3] += h.w;
      if (w)
#pragma unroll
        for (int j = 0; j < 4; ++j) hw[j] += dsm_ld64(&sh.whist[tid * 4 + j], r);
    }
  };
  // The bin in which the running count or weight, from (bc, bw), reaches the target: sh.found in
  // every CTA, which each works out for itself; false if none does.
  auto search = [&](bool by_w, u64 target, u64 bc, u64 bw) -> bool {
    u64 hc[4], hw[4], pc, pw, tc, tw;
    bins(by_w, hc, hw);
    if (tid == 0) sh.hit = 0;
    block_scan2(hc[0] + hc[1] + hc[2] + hc[3], hw[0] + hw[1] + hw[2] + hw[3], &pc, &pw, &tc, &tw, sh.red);
    pc += bc;
    pw += bw;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 lo = by_w ? pw : pc, hi = lo + (by_w ? hw[j] : hc[j]);
      if (lo < target && target <= hi) {
        sh.found[0] = tid * 4 + j;
        sh.found[1] = hc[j];
        sh.found[2] = pc;
        sh.found[3] = pw;
        sh.hit = 1;
      }
      pc += hc[j];
      pw += hw[j];
    }
    samp_sync();  // also: every CTA has read the histograms
    return sh.hit != 0;
  };
  // The id at which the running sum, in vocabulary order, of fn(z, id) passes r = target(sum over
  // the row), fn being 0 in groups whose maximum fails `pred`; -1 where another warp holds it.
  auto locate = [&](auto pred, auto fn, auto target) -> int {
    const int nb = (s1 - s0 + kBatch - 1) / kBatch, span = (nb + kParts - 1) / kParts;  // batches per part
    u64 mine = 0;
    for (int q = 0; q < kParts; ++q) {
      if (q * span >= nb) break;
      u64 s = 0;
      for (int b = q * span; b < min(nb, (q + 1) * span); ++b)
        batch(s0 + b * kBatch, pred, [&](float z, int id) { s += fn(z, id); });
      s = warp_sum64(s);
      if (lane == 0) sh.part[warp][q] = s;
      mine += s;
    }
    __syncthreads();
    if (lane == 0) sh.red[0][warp] = mine;
    __syncthreads();
    if (tid < C) {
      u64 x = 0;
      for (int w = 0; w < kSampWarps; ++w) x += sh.red[0][w];
      dsm_st64(&sh.tot_l[rank], tid, x);
    }
    samp_sync();
    u64 base = 0, all = 0;
    for (int r = 0; r < C; ++r) {
      if (r < static_cast<int>(rank)) base += sh.tot_l[r];
      all += sh.tot_l[r];
    }
    const u64 r = target(all);
    for (int w = 0; w < warp; ++w) base += sh.red[0][w];
    if (!(base <= r && r < base + mine)) return -1;
    int q = 0;
    for (; q < kParts - 1; ++q) {
      const u64 s = sh.part[warp][q];
      if (r < base + s) break;
      base += s;
    }
    int found = -1;
    for (int b = q * span; b < min(nb, (q + 1) * span) && found < 0; ++b)
      batch(s0 + b * kBatch, pred, [&](float z, int id) {
        const u64 x = warp_scan64(fn(z, id), lane);
        const uint32_t hit = __ballot_sync(0xffffffffu, r < base + x);
        if (found < 0 && hit) found = __shfl_sync(0xffffffffu, id, __ffs(hit) - 1);
        base += __shfl_sync(0xffffffffu, x, 31);
      });
    return found;
  };

  // The last candidate of the shortest prefix of those at or above `from` that reaches top-k's
  // count (by_w false) or top-p's weight; 0 if all of them do not reach it.
  auto prefix = [&](bool by_w, u64 from) -> u64 {
    const float from_z = from ? key_value(static_cast<uint32_t>(from >> 32)) : -INFINITY;
    auto in_range = [&](float m) { return m >= from_z && R.bucket(m) < kSampBuckets; };
    // a window of buckets from an eighth of the row; all buckets for a short one
    int lo = 0, hi = kSampBuckets - 1;
    if (p.g32 > 64 * kBatch) {
      zero(false);
      int seen = 0;
      for (int b = s0 + (warp & 7) * kBatch; b < s1; b += 8 * kBatch) {
        seen += min(s1 - b, kBatch);
        batch(b, in_range, [&](float z, int id) {
          const int k = R.bucket(z);
          if (k < kSampBuckets && compose(z, id) >= from) atomicAdd(&chist[k], 1u);
        });
      }
      u64 groups, none;
      sum2(lane == 0 ? seen : 0, 0, &groups, &none);
      u64 hc[4], hw[4], pc, px, tc, tx;
      bins(false, hc, hw);
      if (tid == 0) {
        sh.window[0] = 0;
        sh.window[1] = kSampBuckets - 1;
      }
      u64 own = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // counts, or counts times the weight of the bucket's middle
        hw[j] = by_w ? static_cast<u64>(static_cast<double>(hc[j]) * exp2(30.0 - (tid * 4 + j + 0.5) * p.F / kSampBuckets)) : hc[j];
        own += hw[j];
      }
      block_scan2(own, 0, &pc, &px, &tc, &tx, sh.red);
      const double t = by_w ? static_cast<double>(f.top_p) * static_cast<double>(tc)
                            : static_cast<double>(f.k) * static_cast<double>(groups) / p.g32;
      const double t0 = by_w ? 0.94 * t : 0.9 * t - 16.0, t1 = by_w ? t + 0.06 * static_cast<double>(tc) : 1.1 * t + 16.0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double a = static_cast<double>(pc), b = static_cast<double>(pc + hw[j]);
        if (a < t0 && t0 <= b) sh.window[0] = tid * 4 + j;
        if (a < t1 && t1 <= b) sh.window[1] = tid * 4 + j;
        pc += hw[j];
      }
      samp_sync();  // also: every CTA has read the histograms
      lo = sh.window[0];
      hi = sh.window[1];
    }
    u64 target = f.k;
    for (int pass = 0; pass < 2; ++pass) {  // the second with all buckets, one of which holds it
      zero(by_w);
      u64 above = 0, total = 0;
      for (int b = s0; b < s1; b += kBatch)
        batch(b, in_range, [&](float z, int id) {
          const int k = R.bucket(z);
          if (k >= kSampBuckets || compose(z, id) < from) return;
          const u64 w = by_w ? R.weight(z) : 1;
          total += w;
          if (k < lo) above += w;
          else if (k <= hi) {
            atomicAdd(&chist[k], 1u);
            if (by_w) atomicAdd(&sh.whist[k], w);
          }
        });
      u64 ta, tt;
      sum2(above, total, &ta, &tt);
      if (by_w) target = f.p_target(tt);
      else if (tt < target) {
        samp_sync();  // the sums are read before they are written again
        return 0;
      }
      if (search(by_w, target, ta, ta)) break;
      lo = 0;
      hi = kSampBuckets - 1;
    }
    const int bucket0 = static_cast<int>(sh.found[0]);
    u64 members = sh.found[1], bc = sh.found[2], bw = sh.found[3];
    uint32_t klo = 0, khi = 0xffffffffu;
    auto has = [&](float m) { return R.bucket(m) <= bucket0; };
    auto member = [&](float z, int id) {
      const uint32_t key = sort_key(z);
      return key >= klo && key <= khi && R.bucket(z) == bucket0 && compose(z, id) >= from;
    };
    // 2048 ranges a level: after three levels a range is one key
    for (int level = 0; level < 4 && members > kSampList; ++level) {
      uint32_t l = 0xffffffffu, h = 0;  // the members' smallest and largest key
      for (int b = s0; b < s1; b += kBatch)
        batch(b, has, [&](float z, int id) {
          if (member(z, id)) {
            l = min(l, sort_key(z));
            h = max(h, sort_key(z));
          }
        });
      l = __reduce_min_sync(0xffffffffu, l);
      h = __reduce_max_sync(0xffffffffu, h);
      zero(by_w);  // its barrier also parts the uses of red
      if (lane == 0) {
        sh.red[0][warp] = l;
        sh.red[1][warp] = h;
      }
      __syncthreads();
      if (tid < C) {
        u64 x = 0xffffffffu, y = 0;
        for (int w = 0; w < kSampWarps; ++w) {
          x = min(x, sh.red[0][w]);
          y = max(y, sh.red[1][w]);
        }
        dsm_st64(&sh.tot_a[rank], tid, x);
        dsm_st64(&sh.tot_b[rank], tid, y);
      }
      samp_sync();
      klo = 0xffffffffu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, static_cast<uint32_t>(sh.tot_a[r]));
        khi = max(khi, static_cast<uint32_t>(sh.tot_b[r]));
      }
      if (klo == khi) {  // equal logits: the first ones in vocabulary order
        u64 need = target - bc;
        if (by_w) {
          const u64 w = R.weight(key_value(klo));
          need = (target - bw + w - 1) / w;
        }
        const int id = locate(has, [&](float z, int i) -> u64 { return member(z, i); }, [&](u64) -> u64 { return need - 1; });
        if (id >= 0 && lane == 0)
          for (int r = 0; r < C; ++r) dsm_st64(&sh.cut, r, (static_cast<u64>(klo) << 32) | static_cast<uint32_t>(~id));
        samp_sync();
        return sh.cut;
      }
      const int shift = max(0, 32 - __clz(khi - klo) - 11);
      for (int b = s0; b < s1; b += kBatch)
        batch(b, has, [&](float z, int id) {
          if (member(z, id)) {
            const int k = (khi - sort_key(z)) >> shift;
            atomicAdd(&chist[k], 1u);
            if (by_w) atomicAdd(&sh.whist[k], R.weight(z));
          }
        });
      samp_sync();
      search(by_w, target, bc, bw);
      members = sh.found[1];
      bc = sh.found[2];
      bw = sh.found[3];
      khi -= static_cast<uint32_t>(sh.found[0]) << shift;
      const uint32_t low = khi - ((1u << shift) - 1);
      klo = low > khi ? klo : max(klo, low);
    }
    // the members go to the first CTA and are sorted
    for (int b = s0; b < s1; b += kBatch)
      batch(b, has, [&](float z, int id) {
        if (member(z, id)) {
          const uint32_t at = dsm_add32(&sh.list_n, 0, 1);
          if (at < kSampList) dsm_st64(&sh.list[at], 0, compose(z, id));
        }
      });
    samp_sync();
    if (rank == 0) {
      const int n = static_cast<int>(min(members, static_cast<u64>(kSampList)));
      int P = 2;
      while (P < n) P <<= 1;
      for (int i = n + tid; i < P; i += kSampThreads) sh.list[i] = 0;
      __syncthreads();
      bitonic_desc(sh.list, P);
      u64 x[2] = {0, 0}, px, pt, tx, tt;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (tid * 2 + j < n) x[j] = by_w ? R.weight(key_value(static_cast<uint32_t>(sh.list[tid * 2 + j] >> 32))) : 1;
      block_scan2(x[0] + x[1], 0, &px, &pt, &tx, &tt, sh.red);
      px += by_w ? bw : bc;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (px < target && target <= px + x[j])
          for (int r = 0; r < C; ++r) dsm_st64(&sh.cut, r, sh.list[tid * 2 + j]);
        px += x[j];
      }
      if (tid == 0) sh.list_n = 0;
    }
    samp_sync();
    return sh.cut;
  };

  u64 cut = 0;  // every (key, id) is above
  if (f.k > 0) cut = prefix(false, 0);
  if (f.use_p) {
    samp_sync();  // cut is read before it is written again
    cut = prefix(true, cut);
  }
  const float cut_z = cut ? key_value(static_cast<uint32_t>(cut >> 32)) : -INFINITY;
  const int id = locate([&](float m) { return m >= cut_z; },
                        [&](float z, int i) -> u64 { return compose(z, i) < cut || R.y64(z) < f.low64 ? 0 : R.weight(z); },
                        [&](u64 all) { return f.draw_at(all); });
  if (id >= 0 && lane == 0) {
    p.tokens[row] = id;
    if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(src[id]), p.rsum[row]);
  }
}

}  // namespace lmh
