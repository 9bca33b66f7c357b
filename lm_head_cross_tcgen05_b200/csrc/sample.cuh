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
//    there. A bucket with too many members (equal logits, mostly) is split again by the bits of
//    its keys until they fit or are all equal; equal ones are counted in vocabulary order.
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
constexpr int kFastF = 40;        // the row kernel's fast weights are fractions of 2^40
constexpr int kSampPending = -2;  // tokens[row] of a row that the list kernel leaves

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
  int g32, g256;        // groups per row
  float* gmax;          // [N, g32] largest logit of each 32 (NaN if one is)
  double* gsum;         // [N, g256] sum of exp((z - max) / tau) over each 256, max their largest
  int all_rows;         // row kernel: every row, not only those left by the list kernel
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

struct SampCommon {
  double table[64];                        // 2^(j / 64)
  u64 red[2][kSampWarps];
  u64 tot_m[kSampMaxC], tot_f[kSampMaxC];  // per CTA, written by each into all: maximum, fast sum
};
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
struct alignas(16) RowShared {
  SampCommon c;
  union {
    u64 whist[kSampBuckets];  // dead once merge() has brought its sums into registers
    u64 list[kSampList];      // as above
  };
  uint32_t chist[kSampBuckets];
  u64 tot_c[kSampMaxC], tot_w[kSampMaxC], tot_l[kSampMaxC];  // per CTA, written by each into all
  u64 warp_sum[kSampWarps];
  u64 found[4];                            // bucket, its count, count before, weight before
  u64 cut[2];                              // (key << 32 | ~id) of the last kept, weight kept
  uint32_t list_n;
};

static_assert(sizeof(RowShared) % 16 == 0, "the row's copy follows, in 16-byte vectors");

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
  // 2^40 2^(y / 64), from an fp32 exponential
  __device__ __forceinline__ u64 fast_weight(float z) const {
    return __float2ull_rn(fast_exp2(-fmaf(-0.5f, z, half_max) * c32) * 1099511627776.f);
  }
};
// Bound on the relative error of a row's sum of fp32 exponentials 2^y: 2^-22 of ex2.approx, three
// roundings of y (|y| <= 50 where it matters), 50 * 3 * 2^-24 * ln2 < 2^-17, and 13 additions.
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

// The place of this CTA's chunk of a row.
template <class T>
struct SampChunk {
  const T* gsrc;
  T* chunk;       // its copy in shared memory, aligned as the row is
  const T* src;   // the copy, or the row itself where it does not fit
  int c0, len, mis;
  __device__ __forceinline__ SampChunk(const SampParams& p, long long row, uint32_t rank, uint8_t* room) {
    c0 = static_cast<int>(min(static_cast<long long>(rank) * p.L, static_cast<long long>(p.V)));
    len = min(p.L, p.V - c0);
    gsrc = static_cast<const T*>(p.logits) + row * p.V + c0;
    mis = static_cast<int>((reinterpret_cast<uintptr_t>(gsrc) & 15) / sizeof(T));
    chunk = reinterpret_cast<T*>(room) + mis;
    src = p.resident ? chunk : gsrc;
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Copies the chunk to shared memory (where it fits) and returns this thread's largest logit, NaN
// if it saw one.
template <class T>
__device__ __forceinline__ float load_chunk(const SampParams& p, const SampChunk<T>& k) {
  constexpr int E = 16 / sizeof(T);
  const int tid = threadIdx.x;
  float tmax = -INFINITY;
  const int head = min(k.len, k.mis ? E - k.mis : 0);
  const int nv = (k.len - head) / E;
  auto one = [&](int i) {
    const T t = k.gsrc[i];
    if (p.resident) k.chunk[i] = t;
    tmax = max_nan(tmax, as_float(t));
  };
  if (tid < head) one(tid);
  if (head + nv * E + tid < k.len) one(head + nv * E + tid);
  const uint4* gv = reinterpret_cast<const uint4*>(k.gsrc + head);
  uint4* sv = reinterpret_cast<uint4*>(k.chunk + head);
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
        for (int x = 0; x < E; ++x) tmax = max_nan(tmax, as_float(e[x]));
      }
  }
  return tmax;
}

// The row's maximum from the threads' (NaN: one is NaN), in every thread of the cluster. Contains
// the cluster barrier before which every CTA has started.
__device__ __forceinline__ float row_max(float tmax, SampCommon& sh, uint32_t rank, int C) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool bad = __any_sync(0xffffffffu, tmax != tmax);
  const uint32_t kmax = __reduce_max_sync(0xffffffffu, bad ? 0u : sort_key(tmax));
  __syncthreads();
  if (lane == 0) sh.red[0][warp] = (static_cast<u64>(bad) << 32) | kmax;
  __syncthreads();
  if (tid < C) {
    u64 m = 0;
    for (int w = 0; w < kSampWarps; ++w) m = max(m, sh.red[0][w]);  // a NaN above every key
    dsm_st64(&sh.tot_m[rank], tid, m);
  }
  samp_sync();
  u64 m = 0;
  for (int r = 0; r < C; ++r) m = max(m, sh.tot_m[r]);
  return (m >> 32) != 0 ? NAN : key_value(static_cast<uint32_t>(m));
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
  // Whether the row goes by its groups, and whether their sums have to be exact: nothing but the
  // sums then decides the token.
  __device__ __forceinline__ bool grouped(int V) const { return V <= kSampList || k <= kSampListK; }
  __device__ __forceinline__ bool exact() const { return k == 0 && !use_p && !use_m; }
};

__device__ __forceinline__ SampRow samp_row(const SampParams& p, float zmax, double tau, const double* table) {
  const double c = 1.4426950408889634 / tau;
  SampRow R;
  R.zmaxd = zmax;
  R.c64 = 64.0 * c;
  R.c32 = static_cast<float>(fmin(2.0 * c, 3e38));
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

// One warp per 256 logits of a row, two such per warp so that 16 loads are under way.
constexpr int kGroupWarps = 8, kGroupPer = 2;
template <class T>
__global__ void __launch_bounds__(32 * kGroupWarps) sample_groups_kernel(const SampParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_row = (p.g256 + kGroupWarps * kGroupPer - 1) / (kGroupWarps * kGroupPer);
  const long long row = blockIdx.x / per_row;
  const int g0 = (static_cast<int>(blockIdx.x - row * per_row) * kGroupWarps + warp) * kGroupPer;
  if (g0 >= p.g256) return;
  const SampFilter f(p, row);
  if (!f.grouped(p.V)) return;
  const T* src = static_cast<const T*>(p.logits) + row * p.V;
  float z[kGroupPer][8];
#pragma unroll
  for (int q = 0; q < kGroupPer; ++q)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const long long i = static_cast<long long>(g0 + q) * kSum + j * kGroup + lane;
      z[q][j] = i < p.V ? as_float(src[i]) : -INFINITY;
    }
  const double c = 1.4426950408889634 / f.tau;
  const float c2 = static_cast<float>(fmin(2.0 * c, 3e38));
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
      if (f.exact()) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s += exp2((static_cast<double>(z[q][j]) - m) * c);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      } else {
        float e = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) e += fast_exp2(-fmaf(-0.5f, z[q][j], 0.5f * m) * c2);
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
  if (!f.grouped(p.V)) {
    if (tid == 0) p.tokens[row] = kSampPending;
    return;
  }
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
  if (tid == 0) p.tokens[row] = kSampPending;
}

// One row per cluster; it needs no other row's turn, so rows that are not pending cost an exit.
template <class T>
__global__ void __launch_bounds__(kSampThreads, 1) sample_row_kernel(const SampParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  RowShared& sh = *reinterpret_cast<RowShared*>(dyn);
  const uint32_t rank = cluster_ctarank();
  const long long row = blockIdx.x / p.C;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list kernel's tokens
  if (!p.all_rows && p.tokens[row] != kSampPending) return;  // in every CTA alike
  if (threadIdx.x < 64) sh.c.table[threadIdx.x] = exp2(threadIdx.x / 64.0);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.C;
  const SampFilter f(p, row);
  cluster_arrive();
  const SampChunk<T> ch(p, row, rank, dyn + sizeof(RowShared));
  const int len = ch.len;
  const float tmax = load_chunk(p, ch);
  if (tid == 0) sh.list_n = 0;
  cluster_wait();
  const float zmax = row_max(tmax, sh.c, rank, C);
  if (no_sum(p, row, zmax, rank == 0 && tid == 0)) return;
  if (f.flag && rank == 0 && tid == 0) atomicOr(p.err, f.flag);
  const SampRow R = samp_row(p, zmax, f.tau, sh.c.table);
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
    block_scan2(sc, sw, bc, bw, &xc, &xw, sh.c.red);
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
  // The id at which the running sum, in vocabulary order, of fn(z, id) passes r (which the sum
  // over the row does); -1 where another warp holds it. Each warp has a contiguous segment.
  const int seg = ((len + kSampThreads - 1) / kSampThreads) * 32;
  auto locate = [&](auto fn, auto target) -> int {
    u64 s = 0;
    const int s0 = min(len, warp * seg), s1 = min(len, s0 + seg);
#pragma unroll 4
    for (int i = s0 + lane; i < s1; i += 32) s += fn(as_float(ch.src[i]), ch.c0 + i);
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
    for (int i = r0; i < r1; ++i) x += fn(as_float(ch.src[i]), ch.c0 + i);
    const u64 incl = warp_scan64(x, lane);
    const int owner = __ffs(__ballot_sync(0xffffffffu, r < base + incl)) - 1;
    base += __shfl_sync(0xffffffffu, incl - x, owner);
    const int e1 = __shfl_sync(0xffffffffu, r1, owner);
    for (int i0 = __shfl_sync(0xffffffffu, r0, owner); i0 < e1; i0 += 32) {
      const int i = i0 + lane;
      const u64 y = warp_scan64(i < e1 ? fn(as_float(ch.src[i]), ch.c0 + i) : 0, lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, r < base + y);
      if (hit) return ch.c0 + i0 + __ffs(hit) - 1;
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
        const float z = as_float(ch.src[i]);
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
        sh.c.red[0][warp] = lo;
        sh.c.red[1][warp] = hi;
      }
      for (int i = tid; i < kSampBuckets; i += kSampThreads) {
        sh.whist[i] = 0;
        sh.chist[i] = 0;
      }
      __syncthreads();
      if (tid < C) {
        u64 a = 0xffffffffu, b = 0;
        for (int w = 0; w < kSampWarps; ++w) {
          a = min(a, sh.c.red[0][w]);
          b = max(b, sh.c.red[1][w]);
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
        const float z = as_float(ch.src[i]);
        const uint32_t key = sort_key(z);
        if (key >= klo && key <= khi && R.bucket(z) == bucket0) {
          atomicAdd(&sh.chist[(khi - key) >> shift], 1u);
          if (f.use_p) atomicAdd(&sh.whist[(khi - key) >> shift], R.weight(z));
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
      const float z = as_float(ch.src[i]);
      const uint32_t key = sort_key(z);
      if (key >= klo && key <= khi && R.bucket(z) == bucket0) {
        const uint32_t at = dsm_add32(&sh.list_n, 0, 1);
        if (at < kSampList) dsm_st64(&sh.list[at], 0, (static_cast<u64>(key) << 32) | static_cast<uint32_t>(~(ch.c0 + i)));
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
      block_scan2(c[0] + c[1], w[0] + w[1], &pc, &pw, &tc, &tw, sh.c.red);
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
  {
    u64 sum = 0;
    for_chunk(ch.src, len, ch.mis, [&](float z, int) {
      const int b = R.bucket(z);
      if (b < kSampBuckets) {
        sum += R.fast_weight(z);
        if (f.k > 0 || f.use_p) atomicAdd(&sh.chist[b], 1u);
        if (f.use_p) atomicAdd(&sh.whist[b], R.weight(z));
      }
    });
    sum = warp_sum64(sum);
    __syncthreads();
    if (lane == 0) sh.c.red[0][warp] = sum;
    __syncthreads();
    if (tid < C) {
      u64 t = 0;
      for (int w = 0; w < kSampWarps; ++w) t += sh.c.red[0][w];
      dsm_st64(&sh.c.tot_f[rank], tid, t);
    }
  }
  if (f.k > 0 || f.use_p) {
    merge(&before_c, &before_w, &all_c, &all_w);
    u64 kept_w = all_w;
    if (f.k > 0 && all_c >= static_cast<u64>(f.k)) {
      search(false, f.k, hc, hw, before_c, before_w);
      finish(false, f.k);
      cut = sh.cut[0];
      kept_w = sh.cut[1];
      samp_sync();  // cut and found are read before they are written again
    }
    if (f.use_p) {
      const u64 target = f.p_target(kept_w);
      search(true, target, hc, hw, before_c, before_w);
      finish(true, target);
      cut = max(cut, sh.cut[0]);
    }
  }

  // ---- the token
  const int id = locate(
      [&](float z, int i) -> u64 {
        const u64 x = (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~i);
        return x < cut || R.y64(z) < f.low64 ? 0 : R.weight(z);
      },
      [&](u64 all) { return f.draw_at(all); });
  if (id >= 0 && lane == 0) {
    u64 rough = 0;
    for (int r = 0; r < C; ++r) rough += sh.c.tot_f[r];
    p.tokens[row] = id;
    if (p.logprob)
      p.logprob[row] = samp_logprob(R, as_float(ch.src[id - ch.c0]), static_cast<double>(rough) / __hiloint2double((1023 + kFastF) << 20, 0));
  }
}

}  // namespace lmh
