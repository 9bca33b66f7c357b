// sample.cuh — one token per row of logits, by inversion of the filtered softmax at a given
// uniform number. Candidates are ordered by logit, the largest first, equal ones by id; every
// filter keeps a prefix of that order. Three kernels:
//
//  * sample_groups_kernel streams the logits once: of every 256 of a row (a block), eight maxima
//    of 32 each and the sum of exponentials relative to the largest of them. No thread waits for
//    another beyond its warp. Memory bounds it (256 x 151936 fp32: 41 us, 3.8 TB/s) where fp32
//    exponentials do; rows whose token depends on the whole sum take fp64 ones, which bound it
//    then (85 us if all rows do).
//  * sample_list_kernel, one CTA per row, draws the token from those records and a few logits.
//    Unfiltered, the running sums of the blocks lead to the one whose 256 logits decide. With a
//    short prefix, everything that can be in it is collected and sorted (up to 2048 candidates):
//    at least k logits lie at or above the k-th largest group maximum, so only groups whose
//    maximum lies there are read again, 128 bytes for most of k candidates. A top-p prefix
//    without top-k ends where the candidates' weight reaches a part of the whole sum; the weight of
//    those maxima leads there (a lower bound), so one list is tried at most. A chain of short steps, each
//    waiting for the one before: 256 rows take 13 us unfiltered, 20 with k = 50 and 46 with
//    k = 1000, hardly more than one row does.
//  * sample_row_kernel takes the rows left over (long prefixes), a cluster of 1 to 8 CTAs each,
//    which hold the row in shared memory (where it fits; else they read it again). A prefix that
//    reaches a count or a weight is found by a histogram over 2048 linear buckets of
//    (zmax - z) / tau, whose threshold bucket's few members go to the first CTA and are sorted
//    there. Adding every weight to its bucket in shared memory would cost more than the rest, so
//    counts of an eighth of the row first give a window of buckets; the pass over the row adds
//    what lies above the window in registers and only the window's weights to buckets, and is
//    repeated with all buckets if the prefix does not end in the window. The draw then starts
//    from the sums above the window. A bucket with too many members (equal logits, mostly) is
//    split again by the bits of its keys until they fit or are all equal; equal ones are counted
//    in vocabulary order. A call of one such row of 151936 takes 50 to 58 us, of 30 rows 70 to 84,
//    of 256 480 to 575 (top-p 0.9, logits of standard deviation 2.5 to 0.5): of a pass's 20 thousand
//    cycles with 40 percent kept, 8 go to finding the kept, 4 to their fp64 weights, 4 to the
//    window's atomics.
//
// Where a token depends on sums of weights, the weights are whole numbers, so that no order of
// addition can change it: w(z) = round(2^F exp((z - zmax) / tau)), computed in fp64, with 2^F as
// large as V weights can be added in 63 bits (F = 44 for a vocabulary of 152 thousand, at most
// 50). A token whose probability is below 2^-F of the most likely one's has none.
#pragma once

#include <cuda_bf16.h>

#include "rowops.cuh"

namespace lmh {

constexpr uint32_t kErrSampling = 0x10u;
constexpr int kSampThreads = 512, kSampWarps = kSampThreads / 32;
constexpr int kSampBuckets = 2048;
constexpr int kSampList = 2048;   // candidates that one CTA sorts
constexpr int kSampListK = 1024;  // largest top-k that takes the list (256 x 151936: k = 600 or 1000
                                  // 38 or 46 us from the list, 300 from the row kernel); not more,
                                  // since the last candidates' groups bring others along
constexpr int kSampMaxC = 8;
constexpr int kBlock = 256;       // logits per sum of exponentials
constexpr int kGroups = 8;        // maxima per block: group g has the logits 32 j + 4 g + i of the
                                  // block, j < 8 and i < 4 (what four lanes load)
constexpr int kSampBatch = 96;  // logits that a warp of the row kernel gathers before it works on them
constexpr int kParts = 4;         // partial sums per warp that locate() keeps
constexpr int kSampPending = -2;  // tokens[row] of a row that the list kernel leaves

struct SampParams {
  long long N;
  int V;                // row length
  int C, L, resident;   // row kernel: CTAs per row, logits per CTA, whether these are copied
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
  int blocks;           // blocks per row
  float* gmax;          // [N, blocks, 8] largest logit of each group (NaN if one is NaN)
  double* gsum;         // [N, blocks] sum of exp((z - max) / tau), max the block's largest
  double* rsum;         // [N, 2] of the rows left by the list kernel: sum of exp((z - zmax) / tau), zmax
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
  u64 list[kSampList];           // candidates, key << 32 | ~id
  union {
    u64 wlist[kSampList];        // their weights, once sorted
    uint32_t queue[kSampList];   // groups that hold candidates
  };
  uint4 chist[kSampBuckets / 4];
  uint32_t list_n, queue_n;
  int pick, reach;
  u64 base;
};
struct alignas(16) RowShared {
  double table[64];
  u64 red[2][kSampWarps];
  union {                                    // one at a time
    struct {
      uint32_t lo[kSampBuckets], hi[kSampBuckets];
    } whist;                                 // halves of the bins' weights
    u64 list[kSampList];                     // members of a bucket, on the cluster's first CTA
  };
  int keep[kSampWarps][kSampBatch + 64];     // gather(): places in the chunk
  uint4 chist[kSampBuckets / 4];
  u64 part[kSampWarps][kParts];              // locate(): partial sums of each warp's segment
  u64 top[kSampWarps][kParts];               // prefix(): those of the weights above its window
  u64 tot_a[kSampMaxC], tot_l[kSampMaxC];    // per CTA, written by each into all: sum_row(), locate()
  u64 tot_b[kSampMaxC];
  u64 found[4];                              // bin, its members, count before, weight before
  u64 cut;                                   // (key << 32 | ~id) of the last kept
  uint32_t list_n;
  int hit, window[2];
};
static_assert(sizeof(RowShared) % 16 == 0, "the row's copy follows, in 16-byte vectors");

// A float as a double by its bits: a conversion runs at a quarter of this rate. Infinities come out
// as +-2^128. Not for zeros and subnormal numbers, whose bits mean something else.
__device__ __forceinline__ double widen_normal(float x) {
  const uint32_t b = __float_as_uint(x);
  return __hiloint2double(static_cast<int>((b & 0x80000000u) | (((b & 0x7fffffffu) >> 3) + 0x38000000u)), static_cast<int>(b << 29));
}
constexpr float kLeastNormal = 1.17549435e-38f;  // 2^-126
__device__ __forceinline__ double widen(float x) {
  return fabsf(x) < kLeastNormal ? static_cast<double>(x) : widen_normal(x);
}

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

  // monotone in z, as each of the two roundings is; halved, no finite difference overflows
  __device__ __forceinline__ float place(float z) const { return fmaf(-0.5f, z, half_max) * bucket_scale; }
  __device__ __forceinline__ int bucket(float z) const {
    const float x = place(z);
    return x < static_cast<float>(kSampBuckets) ? static_cast<int>(x) : kSampBuckets;
  }
  // 64 log2 of the probability over the largest one's
  __device__ __forceinline__ double y64(float z) const { return (widen(z) - zmaxd) * c64; }
  // whether a token with this y64() may be drawn: its probability is at least 2^-F of the largest
  __device__ __forceinline__ bool may_draw(double y) const { return y >= -64.0 * F; }
  // 2^F 2^(y / 64) as a whole number (1 at least where the token may be drawn, else 0), read from
  // the low bits of a sum with 2^52: an addition where a conversion of 64-bit types runs at a
  // fraction of that rate
  __device__ __forceinline__ u64 weight(float z) const {
    const double y = y64(z);
    if (!may_draw(y) || !(z > -INFINITY)) return 0;
    double e, sc;
    exp2_64(y, F, table, &e, &sc);
    return static_cast<u64>(__double_as_longlong(fma(e, sc, 4503599627370496.0))) - 0x4330000000000000ull;
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

// Exclusive prefix of a value over the block's threads, and its total.
__device__ __forceinline__ void block_scan(u64 a, u64* pa, u64* ta, u64* red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const u64 ia = warp_scan64(a, lane);
  __syncthreads();
  if (lane == 31) red[warp] = ia;
  __syncthreads();
  const u64 s = warp_scan64(lane < kSampWarps ? red[lane] : 0, lane);
  const u64 before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
  *pa = (warp ? before : 0) + ia - a;
  *ta = __shfl_sync(0xffffffffu, s, kSampWarps - 1);
}

// Sorts a[0 .. n) in descending order, all values different and not 0; a (16-byte aligned) has room
// for the next power of two. By counting the larger ones up to 512 values (no barriers between its
// steps: 1100 cycles for 64, where the network took 3900), by a bitonic network above. All
// threads; a barrier before and after.
__device__ __forceinline__ void sort_desc(u64* a, int n) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (n <= kSampThreads) {
    if (tid == 0 && (n & 1)) a[n] = 0;
    const u64 x = tid < n ? a[tid] : 0;
    __syncthreads();
    int at = 0;
    if (tid < n) {
      const ulonglong2* v = reinterpret_cast<const ulonglong2*>(a);
#pragma unroll 8
      for (int j = 0; j < (n + 1) / 2; ++j) {
        const ulonglong2 y = v[j];
        at += (y.x > x) + (y.y > x);
      }
    }
    __syncthreads();
    if (tid < n) a[at] = x;
    __syncthreads();
    return;
  }
  int P = 2 * kSampThreads;
  while (P < n) P <<= 1;
  for (int i = n + tid; i < P; i += kSampThreads) a[i] = 0;
  __syncthreads();
  for (int size = 2; size <= P; size <<= 1)
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int t = tid; t < P / 2; t += kSampThreads) {
        const int i = 2 * t - (t & (stride - 1)), j = i + stride;
        const u64 x = a[i], y = a[j];
        if ((x < y) == ((i & size) == 0)) {
          a[i] = y;
          a[j] = x;
        }
      }
      // a warp's pairs at strides up to 32 lie in its own 64 values
      if (stride > 32 || (stride == 1 && size >= 64)) __syncthreads();
      else __syncwarp();
    }
}

// The same for up to 2048 values, bucket(x) from 0 to 2047 never falling as x does: by a histogram of
// the buckets, then within each, unless one has more than 64. 330 values take 3000 cycles and 1400 values 5000,
// where counting took 5500 and the network 29000. Up to 128 counting is as fast or faster (256 rows
// of 151936, top-k 50 / 100 / 200: 47.4 / 49.3 / 53.3 us; with 32 for the 128 49.4 / 50.4 / 53.2, with 64
// 47.4 / 50.4 / 53.3, with 256 47.4 / 49.3 / 55.3).
template <class B>
__device__ __forceinline__ void sort_buckets(u64* a, int n, uint4* chist, u64* red, B bucket) {
  const int tid = threadIdx.x;
  if (n <= 128) return sort_desc(a, n);
  constexpr int PER = kSampList / kSampThreads;
  uint32_t* hist = reinterpret_cast<uint32_t*>(chist);
  static_assert(kSampBuckets == 4 * kSampThreads, "four buckets a thread");
  chist[tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  u64 x[PER];
  int b[PER], at[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    x[j] = tid + j * kSampThreads < n ? a[tid + j * kSampThreads] : 0;
    if (x[j]) {
      b[j] = bucket(x[j]);
      at[j] = static_cast<int>(atomicAdd(&hist[b[j]], 1u));
    }
  }
  __syncthreads();
  const uint4 h = chist[tid];
  if (__syncthreads_or(max(max(h.x, h.y), max(h.z, h.w)) > 64u)) return sort_desc(a, n);
  u64 before, all;
  block_scan(h.x + h.y + h.z + h.w, &before, &all, red);
  const uint32_t c = static_cast<uint32_t>(before);
  chist[tid] = make_uint4(c, c + h.x, c + h.x + h.y, c + h.x + h.y + h.z);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (x[j]) a[hist[b[j]] + at[j]] = x[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    if (!x[j]) continue;
    const int from = hist[b[j]], to = b[j] + 1 < kSampBuckets ? static_cast<int>(hist[b[j] + 1]) : n;
    at[j] = from;
    for (int i = from; i < to; ++i) at[j] += a[i] > x[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (x[j]) a[at[j]] = x[j];
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
  // A sum of weights, the largest being 1, in units of 2^-F.
  __device__ __forceinline__ static u64 whole(double total, int F) {
    return __double2ull_rn(total * __hiloint2double((1023 + F) << 20, 0));
  }
  // Whether the list kernel may draw the row: nothing is filtered, or the prefix may be short.
  __device__ __forceinline__ bool listed(int V) const { return V <= kSampList || k <= kSampListK; }
  __device__ __forceinline__ bool off() const { return k == 0 && !use_p && !use_m; }
};
// Whether the sum of the whole row decides the token: nothing is filtered, or top-p is a part of
// all. The blocks' sums are fp64 then; for the log-prob alone fp32 exponentials do.
__device__ __forceinline__ bool samp_exact(const SampParams& p, long long row) {
  const int k = p.row_top_k ? p.row_top_k[row] : p.top_k;
  const float top_p = p.row_top_p ? p.row_top_p[row] : p.top_p;
  const float min_p = p.row_min_p ? p.row_min_p[row] : p.min_p;
  return (k <= 0 || k >= p.V) && (top_p < 1.f || !(min_p > 0.f));
}

__device__ __forceinline__ SampRow samp_row(const SampParams& p, float zmax, double tau, const double* table) {
  const double c = 1.4426950408889634 / tau;
  SampRow R;
  R.zmaxd = widen(zmax);
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

// One warp per block at a time, two under way.
constexpr int kGroupWarps = 8, kGroupPer = 2;
template <class T>
__global__ void __launch_bounds__(32 * kGroupWarps) sample_groups_kernel(const SampParams p) {
  __shared__ double table[64];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;  // the kernels that follow set its bits
  const int per_row = (p.blocks + kGroupWarps * kGroupPer - 1) / (kGroupWarps * kGroupPer);
  const long long row = blockIdx.x / per_row;
  const int b0 = (static_cast<int>(blockIdx.x - row * per_row) * kGroupWarps + warp) * kGroupPer;
  const T* src = static_cast<const T*>(p.logits) + row * p.V + static_cast<long long>(b0) * kBlock + lane;
  const long long left = p.V - static_cast<long long>(b0) * kBlock - lane;  // logits from src on
  float z[kGroupPer][8];
  if (left >= kGroupPer * kBlock) {
#pragma unroll
    for (int q = 0; q < kGroupPer; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[q][j] = as_float(src[q * kBlock + j * 32]);
  } else {
#pragma unroll
    for (int q = 0; q < kGroupPer; ++q)
#pragma unroll
      for (int j = 0; j < 8; ++j) z[q][j] = q * kBlock + j * 32 < left ? as_float(src[q * kBlock + j * 32]) : -INFINITY;
  }
  float tau = 1.f;
  if (p.row_tau) {
    tau = p.row_tau[row];
    if (!temperature_ok(tau)) tau = 1.f;
  }
  // Of the product, since one factor alone may leave the range that 2 log2(e) / tau is in. Where that
  // is no normal number, the sums are in fp64.
  const float product = p.tau * tau;
  // the same for the whole block of threads
  const bool exact = samp_exact(p, row) || !(product > 1e-38f && product < 2e38f);
  if (exact) {
    if (threadIdx.x < 64) table[threadIdx.x] = exp2(threadIdx.x / 64.0);
    __syncthreads();
  }
  const double c64 = exact ? 64.0 * 1.4426950408889634 / (static_cast<double>(tau) * p.tau) : 0.0;
  const float c2 = 2.8853900817779268f / product;
#pragma unroll
  for (int q = 0; q < kGroupPer; ++q) {
    if (b0 + q >= p.blocks) break;
    float m = z[q][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = max_nan(m, z[q][j]);
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
    if ((lane & 3) == 0) p.gmax[(row * p.blocks + b0 + q) * kGroups + (lane >> 2)] = m;
    m = warp_max_nan(m);
    double s = 0.0;
    if (fabsf(m) <= 3.402823466e38f) {  // else no finite logit, or the row has no finite sum
      if (exact) {
        const double md = widen(m);
        auto add = [&](auto wide) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const double y = (wide(z[q][j]) - md) * c64;
            double e = 0.0, sc = 0.0;
            if (y > -64.0 * 100 && z[q][j] > -INFINITY) exp2_64(y, 0, table, &e, &sc);  // less cannot be drawn
            s = fma(e, sc, s);
          }
        };
        // one look at eight logits (256 x 151936: 83.4 us, as without; 86 with one at each)
        float least = fabsf(z[q][0]);
#pragma unroll
        for (int j = 1; j < 8; ++j) least = fminf(least, fabsf(z[q][j]));
        if (least >= kLeastNormal) add([](float x) { return widen_normal(x); });
        else add([](float x) { return widen(x); });
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      } else {
        const float hm = 0.5f * m;
        float e = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) e += fast_exp2(-fmaf(-0.5f, z[q][j], hm) * c2);
        s = warp_sum(e);
      }
    }
    if (lane == 0) p.gsum[row * p.blocks + b0 + q] = s;
  }
}

template <class T>
__global__ void __launch_bounds__(kSampThreads, 2) sample_list_kernel(const SampParams p) {
  __shared__ ListShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x;
  const SampFilter f(p, row);
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the groups' records
  const T* src = static_cast<const T*>(p.logits) + row * p.V;
  const float* gmax = p.gmax + row * p.blocks * kGroups;
  const double* gsum = p.gsum + row * p.blocks;
  const int groups = p.blocks * kGroups;
  // fn(maximum, group) over the groups (-inf past the last), whole warps, four loads under way
  auto each_group = [&](auto fn) {
#pragma unroll 1
    for (int g0 = tid; g0 - tid < groups; g0 += 4 * kSampThreads) {
      float m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = g0 + j * kSampThreads < groups ? gmax[g0 + j * kSampThreads] : -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) fn(m[j], g0 + j * kSampThreads);
    }
  };

  float tmax = -INFINITY;
  each_group([&](float m, int) { tmax = max_nan(tmax, m); });
  tmax = warp_max_nan(tmax);
  if (lane == 0) sh.red[0][warp] = __float_as_uint(tmax);
  __syncthreads();
  const float zmax = warp_max_nan(__uint_as_float(static_cast<uint32_t>(sh.red[0][lane & (kSampWarps - 1)])));
  if (f.flag && tid == 0) atomicOr(p.err, f.flag);
  if (no_sum(p, row, zmax, tid == 0)) return;
  const SampRow R = samp_row(p, zmax, f.tau, sh.table);
  auto block_max = [&](int b) -> float {
    const float4 u = reinterpret_cast<const float4*>(gmax)[b * 2], v = reinterpret_cast<const float4*>(gmax)[b * 2 + 1];
    return fmaxf(fmaxf(fmaxf(u.x, u.y), fmaxf(u.z, u.w)), fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)));
  };
  // block b's sum of exponentials relative to the row's maximum
  auto block_sum = [&](int b) -> double {
    const double s = gsum[b];
    const double y = R.y64(block_max(b));
    if (!(s > 0.0) || y < -64.0 * 100) return 0.0;  // less than 2^-100 of the largest weight
    double e, sc;
    exp2_64(y, 0, sh.table, &e, &sc);
    return s * (e * sc);
  };

  if (f.off()) {
    // whole numbers of 2^-F again; each thread has a run of blocks. A block whose largest logit may
    // not be drawn is passed over, whatever they weigh together. For the log-prob it counts.
    const double up = __hiloint2double((1023 + p.F) << 20, 0);
    const int run = (p.blocks + kSampThreads - 1) / kSampThreads;
    const int r0 = min(p.blocks, tid * run), r1 = min(p.blocks, r0 + run);
    auto block_weight = [&](int b, double sum) -> u64 {
      return R.may_draw(R.y64(block_max(b))) ? __double2ull_rn(sum * up) : 0;
    };
    u64 s = 0, before, total;
    double all = 0.0;
    for (int b = r0; b < r1; ++b) {
      const double x = block_sum(b);
      s += block_weight(b, x);
      all += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (lane == 0) sh.dred[warp] = all;
    block_scan(s, &before, &total, sh.red[1]);
    const u64 r = f.draw_at(total);
    if (before <= r && r < before + s) {
      int b = r0;
      for (; b < r1 - 1; ++b) {
        const u64 w = block_weight(b, block_sum(b));
        if (r < before + w) break;
        before += w;
      }
      sh.pick = b;
      sh.base = r - before;
    }
    __syncthreads();
    if (warp != 0) return;
    all = sh.dred[lane & (kSampWarps - 1)];
#pragma unroll
    for (int o = kSampWarps / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    // within the block, 8 adjacent logits a lane; its weights' sum is its rounded sum up to their
    // own roundings, so a remainder past the last goes to the last that can be drawn
    const long long i0 = static_cast<long long>(sh.pick) * kBlock + lane * 8;
    const u64 rest = sh.base;
    u64 w[8], sum = 0;
    int last = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = i0 + j < p.V ? R.weight(as_float(src[i0 + j])) : 0;
      sum += w[j];
      if (w[j] > 0) last = j;
    }
    u64 at = warp_scan64(sum, lane) - sum;
    int hit = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (hit < 0 && at <= rest && rest < at + w[j]) hit = j;
      at += w[j];
    }
    const uint32_t found = __ballot_sync(0xffffffffu, hit >= 0);
    const uint32_t can = __ballot_sync(0xffffffffu, last >= 0);
    const int owner = found ? __ffs(found) - 1 : 31 - __clz(can);  // the block's largest can
    if (lane == owner) {
      const long long id = i0 + (found ? hit : last);
      p.tokens[row] = static_cast<int>(id);
      if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(src[id]), all);
    }
    return;
  }

  // ---- the row's sum, in a fixed order
  double total = 0.0;
  for (int b = tid; b < p.blocks; b += kSampThreads) total += block_sum(b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sh.dred[warp] = total;
  __syncthreads();
  total = sh.dred[lane & (kSampWarps - 1)];
#pragma unroll
  for (int o = kSampWarps / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);

  const bool all_listed = p.V <= kSampList;
  while (f.listed(p.V)) {  // once; break: the row is left
    // ---- candidates lie in the buckets up to b0
    int b0 = kSampBuckets - 1;
    if (tid == 0) {
      sh.pick = kSampBuckets - 1;
      sh.reach = kSampBuckets;
      sh.list_n = sh.queue_n = 0;
    }
    if (!all_listed && (f.k > 0 || f.use_p)) {
      for (int i = tid; i < kSampBuckets / 4; i += kSampThreads) sh.chist[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      uint32_t* hist = reinterpret_cast<uint32_t*>(sh.chist);
      each_group([&](float m, int) {
        const int b = R.bucket(m);
        if (b < kSampBuckets) atomicAdd(&hist[b], 1u);
      });
      __syncthreads();
      const uint4 h = sh.chist[tid];
      const uint32_t hv[4] = {h.x, h.y, h.z, h.w};
      u64 pc, tc;
      block_scan(h.x + h.y + h.z + h.w, &pc, &tc, sh.red[0]);
      if (f.k > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (pc < static_cast<u64>(f.k) && static_cast<u64>(f.k) <= pc + hv[j]) sh.pick = tid * 4 + j;
          pc += hv[j];
        }
      } else {
        // Top-p alone. The maxima themselves weigh at least so much, in 2^-30 of the largest; where
        // they reach the target, or a list of the largest size may, the list has a chance. With c
        // of G groups reaching a bucket, logits in any order, G log(G / (G - c)) logits do. What
        // is misjudged here costs time: the token is the same from either kernel. 256 rows of
        // 50001 / 151936, standard deviations 2 to 8, p = 0.5: 65.5 / 184 us; 103 / 182 if the list
        // is taken only where the maxima reach the target. Of the constants, 0 or 200 for the 48
        // and 0.8 or 1.05 for the 0.95 make 2 percent at most; 150 for the 348 66 / 165, but 75 / 116
        // in 64 rows of bf16 with p = 0.9 that take 73 / 114; 700 62 / 181 and 72 / 123.
        u64 hw[4], pw, tw;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          double e, sc;
          exp2_64(-64.0 * p.F / kSampBuckets * (tid * 4 + j + 1), 30, sh.table, &e, &sc);
          hw[j] = hv[j] ? static_cast<u64>(hv[j] * (e * sc)) : 0;
        }
        block_scan(hw[0] + hw[1] + hw[2] + hw[3], &pw, &tw, sh.red[1]);
        const float goal = fmaxf(f.top_p * static_cast<float>(total) * 1073741824.f, 1.f), G = static_cast<float>(groups);
        auto members = [&](u64 c) { return G * -log1pf(-fminf(static_cast<float>(c) / G, 0.9999f)); };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u64 c = pc + hv[j], w = pw + hw[j];
          if (hv[j]) {
            const float n = members(c);
            if (static_cast<float>(pw) < goal && goal <= static_cast<float>(w) && n <= kSampList - 48) sh.reach = tid * 4 + j;
            if (n > kSampList - 348 && (pc == 0 || members(pc) <= kSampList - 348))
              sh.pick = n <= kSampList && static_cast<float>(w) * (n / c) >= 0.95f * goal ? tid * 4 + j : -1;
          }
          pc = c;
          pw = w;
        }
      }
      __syncthreads();
      b0 = sh.reach < kSampBuckets ? sh.reach : sh.pick;
      if (b0 < 0) break;
    }
    if (f.use_m && !f.use_p) {
      const double bm = -f.low64 / 64.0 * (kSampBuckets / static_cast<double>(p.F)) + 1.0;
      if (bm < b0) b0 = static_cast<int>(bm);
    }
    __syncthreads();
    // up_to(z): bucket(z) <= b0, z not -inf
    const float last_x = static_cast<float>(b0 + 1);
    auto up_to = [&](float z) { return R.place(z) < last_x; };
#pragma unroll 1
    for (int g0 = tid; g0 - tid < groups; g0 += 4 * kSampThreads) {
      float m[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) m[j] = g0 + j * kSampThreads < groups ? gmax[g0 + j * kSampThreads] : -INFINITY;
      uint32_t mask[4], count = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mask[j] = __ballot_sync(0xffffffffu, up_to(m[j]));
        count += __popc(mask[j]);
      }
      if (!count) continue;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&sh.queue_n, count);
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t to = at + __popc(mask[j] & ((1u << lane) - 1));
        if (((mask[j] >> lane) & 1) && to < kSampList) sh.queue[to] = g0 + j * kSampThreads;
        at += __popc(mask[j]);
      }
    }
    __syncthreads();
    // every queued group holds a candidate: more of them than the list holds leave the row
    if (sh.queue_n > kSampList) break;
    const int queued = static_cast<int>(sh.queue_n);
    // eight groups at a time, their candidates counted in one step (the counter is one address),
    // while the next eight are loaded
    float z[8];
    const uint32_t lane_at = (lane >> 2) * 32 + (lane & 3);
    auto place = [&](int q) -> uint32_t {
      const uint32_t g = sh.queue[q];
      return g / kGroups * kBlock + g % kGroups * 4 + lane_at;
    };
    auto load = [&](int q0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = q0 + j * kSampWarps;
        const uint32_t id = q < queued ? place(q) : p.V;
        z[j] = id < static_cast<uint32_t>(p.V) ? as_float(src[id]) : -INFINITY;  // no candidate
      }
    };
    if (warp < queued) load(warp);
#pragma unroll 1
    for (int q0 = warp; q0 < queued; q0 += 8 * kSampWarps) {
      float y[8];
      uint32_t mask[8], count = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = z[j];
        mask[j] = __ballot_sync(0xffffffffu, up_to(y[j]));
        count += __popc(mask[j]);
      }
      if (q0 + 8 * kSampWarps < queued) load(q0 + 8 * kSampWarps);
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&sh.list_n, count);
      at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if ((mask[j] >> lane) & 1) {
          const uint32_t slot = at + __popc(mask[j] & ((1u << lane) - 1));
          if (slot < kSampList) sh.list[slot] = (static_cast<u64>(sort_key(y[j])) << 32) | ~place(q0 + j * kSampWarps);
        }
        at += __popc(mask[j]);
      }
    }
    __syncthreads();
    if (sh.list_n > kSampList) break;
    const int n = static_cast<int>(sh.list_n);
    // as bucket(), but those up to b0 fill all of them
    const float finer = R.bucket_scale * (static_cast<float>(kSampBuckets) / (b0 + 1));
    sort_buckets(sh.list, n, sh.chist, sh.red[0], [&](u64 x) {
      const float z = key_value(static_cast<uint32_t>(x >> 32));
      return static_cast<int>(fminf(fmaf(-0.5f, z, R.half_max) * finer, kSampBuckets - 1.f));
    });

    // ---- kept: nk by count, the first by min-p, and by top-p up to the first whose running
    // weight reaches its part of what top-k kept, or of the row
    const int nk = f.k > 0 ? min(n, f.k) : n;
    u64 before = 0, sum = 0, weight = 0, by_m = 0;
    for (int c = 0; c < nk; c += kSampThreads) {
      const int i = c + tid;
      u64 w = 0, in = 0;
      if (i < nk) {
        const float z = key_value(static_cast<uint32_t>(sh.list[i] >> 32));
        w = R.weight(z);
        in = !f.use_m || R.y64(z) >= f.low64;
        sh.wlist[i] = w;
      }
      block_scan(w, &before, &sum, sh.red[0]);
      weight += sum;
      block_scan(in, &before, &sum, sh.red[1]);
      by_m += sum;
    }
    int keep = min(nk, static_cast<int>(by_m));
    if (f.use_p) {
      const u64 target = f.p_target(f.k > 0 ? weight : f.whole(total, p.F));
      if (tid == 0) sh.pick = -1;
      u64 run = 0;
      for (int c = 0; c < nk; c += kSampThreads) {
        const int i = c + tid;
        const u64 w = i < nk ? sh.wlist[i] : 0;
        block_scan(w, &before, &sum, sh.red[0]);
        before += run;
        if (before < target && target <= before + w) sh.pick = i;
        run += sum;
      }
      __syncthreads();
      const int at = sh.pick;
      __syncthreads();
      if (at >= 0) {
        keep = min(keep, at + 1);
      } else if (!all_listed) {  // else all are listed, and the target past them by a rounding
        break;
      }
    }

    // ---- the kept in the order of their ids, their weights found by their old places
    for (int c = 0; c < keep; c += kSampThreads) {
      const u64 x = c + tid < keep ? (sh.list[c + tid] << 32) | static_cast<uint32_t>(c + tid) : 0;
      if (c + tid < keep) sh.list[c + tid] = x;
    }
    const float per_id = static_cast<float>(kSampBuckets) / p.V;
    sort_buckets(sh.list, keep, sh.chist, sh.red[0], [&](u64 x) {
      return static_cast<int>(fminf(static_cast<float>(~static_cast<uint32_t>(x >> 32)) * per_id, kSampBuckets - 1.f));
    });
    u64 all = 0;
    for (int c = 0; c < keep; c += kSampThreads) {
      const int i = c + tid;
      block_scan(i < keep ? sh.wlist[static_cast<uint32_t>(sh.list[i])] : 0, &before, &sum, sh.red[0]);
      all += sum;
    }
    const u64 r = f.draw_at(all);
    u64 run = 0;
    for (int c = 0; c < keep; c += kSampThreads) {
      const int i = c + tid;
      const u64 w = i < keep ? sh.wlist[static_cast<uint32_t>(sh.list[i])] : 0;
      if (keep > kSampThreads) block_scan(w, &before, &sum, sh.red[0]);  // else it is that of above
      before += run;
      run += sum;
      if (before <= r && r < before + w) {
        const int id = static_cast<int>(~static_cast<uint32_t>(sh.list[i] >> 32));
        p.tokens[row] = id;
        if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(src[id]), total);
      }
    }
    return;
  }
  if (tid == 0) {
    p.rsum[2 * row] = total;
    p.rsum[2 * row + 1] = zmax;
    p.tokens[row] = kSampPending;
  }
}

// One row per cluster; rows that are not pending cost an exit.
template <class T>
__global__ void __launch_bounds__(kSampThreads, 2) sample_row_kernel(const SampParams p) {
  extern __shared__ __align__(16) uint8_t dyn[];
  RowShared& sh = *reinterpret_cast<RowShared*>(dyn);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int C = p.C;
  const long long row = blockIdx.x / C;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the list kernel's tokens
  if (p.tokens[row] != kSampPending) return;          // in every CTA alike
  cluster_arrive();  // before any CTA writes another's shared memory, all have started

  // ---- this CTA's chunk of the row, in shared memory at the row's own alignment
  const int c0 = static_cast<int>(min(static_cast<long long>(rank) * p.L, static_cast<long long>(p.V)));
  const int len = min(p.L, p.V - c0);
  const T* src = static_cast<const T*>(p.logits) + row * p.V + c0;
  if (p.resident) {
    constexpr int E = 16 / sizeof(T);
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(T));
    T* chunk = reinterpret_cast<T*>(dyn + sizeof(RowShared)) + mis;
    const int head = min(len, mis ? E - mis : 0), nv = (len - head) / E, tail = head + nv * E;
    if (tid < head) chunk[tid] = src[tid];
    if (tail + tid < len) chunk[tail + tid] = src[tail + tid];
    const uint4* from = reinterpret_cast<const uint4*>(src + head);
    uint4* to = reinterpret_cast<uint4*>(chunk + head);
    for (int j0 = tid; j0 < nv; j0 += 4 * kSampThreads) {
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j * kSampThreads < nv) v[j] = from[j0 + j * kSampThreads];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j0 + j * kSampThreads < nv) to[j0 + j * kSampThreads] = v[j];
    }
    src = chunk;
  }
  const SampFilter f(p, row);
  uint32_t* chist = reinterpret_cast<uint32_t*>(sh.chist);
  if (tid < 64) sh.table[tid] = exp2(tid / 64.0);
  if (tid == 0) sh.list_n = 0;
  const double total = p.rsum[2 * row];
  const SampRow R = samp_row(p, static_cast<float>(p.rsum[2 * row + 1]), f.tau, sh.table);
  cluster_wait();
  __syncthreads();

  // [s0, s1) of the chunk are this warp's: contiguous, in the order of the CTAs and their warps
  const int per_warp = ((len + kSampWarps - 1) / kSampWarps + 31) / 32 * 32;
  const int s0 = min(len, warp * per_warp), s1 = min(len, s0 + per_warp);
  // fn(z, id) for 32 logits at a time of the warp's [b0, b1), every `step` th 32 (-inf past the
  // end), four at a time: the arithmetic of one is a long chain, and the SM has few warps
  auto sweep = [&](int b0, int b1, int step, auto fn) {
#pragma unroll 1
    for (int i = b0 + lane; i - lane < b1; i += 128 * step) {
      float z[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = i + 32 * step * j < b1 ? as_float(src[i + 32 * step * j]) : -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) fn(z[j], c0 + i + 32 * step * j);
    }
  };
  auto compose = [](float z, int id) { return (static_cast<u64>(sort_key(z)) << 32) | static_cast<uint32_t>(~id); };
  // Sum over the row of a value per thread, in every thread of the cluster.
  auto sum_row = [&](u64 a) -> u64 {
    a = warp_sum64(a);
    __syncthreads();
    if (lane == 0) sh.red[0][warp] = a;
    __syncthreads();
    if (tid < C) {
      u64 x = 0;
      for (int w = 0; w < kSampWarps; ++w) x += sh.red[0][w];
      dsm_st64(&sh.tot_a[rank], tid, x);
    }
    samp_sync();
    u64 t = 0;
    for (int r = 0; r < C; ++r) t += sh.tot_a[r];
    samp_sync();  // read before they are written again
    return t;
  };
  auto zero = [&](bool w) {
    for (int i = tid; i < kSampBuckets / 4; i += kSampThreads) sh.chist[i] = make_uint4(0, 0, 0, 0);
    if (w)
      for (int i = tid; i < kSampBuckets / 2; i += kSampThreads) reinterpret_cast<uint4*>(&sh.whist)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  };
  // 64-bit additions in shared memory are loops of compare-and-swap; two of 32 bits with a carry
  // are not, and their sum does not depend on their order either.
  auto add_weight = [&](int k, u64 w) {
    const uint32_t lo = static_cast<uint32_t>(w), old = atomicAdd(&sh.whist.lo[k], lo);
    atomicAdd(&sh.whist.hi[k], static_cast<uint32_t>(w >> 32) + (old + lo < old ? 1u : 0u));
  };
  // This thread's four bins of the cluster's histograms. The barrier before it has been passed.
  // Bins outside [b0, b1] are not read: a cluster reading all of all its histograms takes longer
  // than the pass that fills them.
  auto bins = [&](bool w, int b0, int b1, u64 (&hc)[4], u64 (&hw)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) hc[j] = hw[j] = 0;
    if (tid * 4 + 3 < b0 || tid * 4 > b1) return;
#pragma unroll 2
    for (int r = 0; r < C; ++r) {
      const uint4 h = dsm_ld128(&sh.chist[tid], r);
      hc[0] += h.x;
      hc[1] += h.y;
      hc[2] += h.z;
      hc[3] += h.w;
      if (w) {
        const uint4 l = dsm_ld128(&sh.whist.lo[tid * 4], r), g = dsm_ld128(&sh.whist.hi[tid * 4], r);
        hw[0] += (static_cast<u64>(g.x) << 32) + l.x;
        hw[1] += (static_cast<u64>(g.y) << 32) + l.y;
        hw[2] += (static_cast<u64>(g.z) << 32) + l.z;
        hw[3] += (static_cast<u64>(g.w) << 32) + l.w;
      }
    }
  };
  // The bin in which the running count or weight, from `base`, reaches the target: sh.found in
  // every CTA, which each works out for itself; false if none does.
  auto search = [&](bool by_w, u64 target, u64 base, int b0, int b1) -> bool {
    u64 hc[4], hw[4], at, all;
    bins(by_w, b0, b1, hc, hw);
    if (tid == 0) sh.hit = 0;
    block_scan(by_w ? hw[0] + hw[1] + hw[2] + hw[3] : hc[0] + hc[1] + hc[2] + hc[3], &at, &all, sh.red[0]);
    at += base;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u64 end = at + (by_w ? hw[j] : hc[j]);
      if (at < target && target <= end) {
        sh.found[0] = tid * 4 + j;
        sh.found[1] = hc[j];
        sh.found[2] = at;
        sh.hit = 1;
      }
      at = end;
    }
    samp_sync();  // also: every CTA has read the histograms
    return sh.hit != 0;
  };
  // work(n) for the logits of the warp's [b0, b1) that `has` keeps, up to 96 of them at a time:
  // their places in the chunk are keep[0 .. n). What a kept one costs is paid for full warps; done
  // where they lie, with one lane in ten, a pass took three times as long.
  int* keep = sh.keep[warp];
  auto gather = [&](int b0, int b1, auto has, auto work) {
    int n = 0;
    float z[2], next[2];
    auto load = [&](int i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) next[j] = i + 32 * j < b1 ? as_float(src[i + 32 * j]) : -INFINITY;
    };
    load(b0 + lane);
#pragma unroll 1
    for (int i = b0 + lane; i - lane < b1; i += 64) {
      uint32_t mask[2];
      bool mine[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) z[j] = next[j];
      load(i + 64);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mine[j] = has(z[j], c0 + i + 32 * j);
        mask[j] = __ballot_sync(0xffffffffu, mine[j]);
      }
      if (!(mask[0] | mask[1])) continue;
      const uint32_t below = (1u << lane) - 1;
      if (mine[0]) keep[n + __popc(mask[0] & below)] = i;
      n += __popc(mask[0]);
      if (mine[1]) keep[n + __popc(mask[1] & below)] = i + 32;
      n += __popc(mask[1]);
      if (n >= kSampBatch) {
        __syncwarp();
        work(kSampBatch);
        __syncwarp();
        n -= kSampBatch;  // below 64; the rest moves down
        const int x = lane < n ? keep[kSampBatch + lane] : 0, y = lane + 32 < n ? keep[kSampBatch + lane + 32] : 0;
        if (lane < n) keep[lane] = x;
        if (lane + 32 < n) keep[lane + 32] = y;
      }
    }
    __syncwarp();
    if (n) work(n);
    __syncwarp();
  };
  // This lane's part of the sum of the weights in the warp's [b0, b1) that `has` keeps.
  auto weigh = [&](int b0, int b1, auto has) -> u64 {
    u64 s = 0;
    gather(b0, b1, has, [&](int n) {
#pragma unroll
      for (int j = 0; j < kSampBatch / 32; ++j) s += lane + 32 * j < n ? R.weight(as_float(src[keep[lane + 32 * j]])) : 0;
    });
    return s;
  };
  // The id at which the running sum, in vocabulary order, of fn(z, id) passes r = target(sum over
  // the row); -1 where another warp holds it. part(q, b0, b1) is this lane's part of the sum of fn
  // over part q of the warp's logits.
  const int span = ((s1 - s0 + kParts - 1) / kParts + 31) / 32 * 32;  // logits per part
  auto locate = [&](auto fn, auto part, auto target) -> int {
    u64 mine = 0;
#pragma unroll 1
    for (int q = 0; q < kParts; ++q) {
      if (s0 + q * span >= s1) break;
      const u64 s = warp_sum64(part(q, s0 + q * span, min(s1, s0 + (q + 1) * span)));
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
    sweep(s0 + q * span, min(s1, s0 + (q + 1) * span), 1, [&](float z, int id) {
      const u64 x = warp_scan64(fn(z, id), lane);
      const uint32_t hit = __ballot_sync(0xffffffffu, r < base + x);
      if (found < 0 && hit) found = __shfl_sync(0xffffffffu, id, __ffs(hit) - 1);
      base += __shfl_sync(0xffffffffu, x, 31);
    });
    return found;
  };

  // The last candidate of the shortest prefix of those at or above `from` whose count (by_w false)
  // or weight reaches the target; 0 if all of them do not reach it. whole: the weight of all of them.
  int top_lo = 0;  // sh.top has the weights of the buckets below it
  auto prefix = [&](bool by_w, u64 from, u64 target, u64 whole) -> u64 {
    // a window of buckets from an eighth of the row; all buckets for a short one (32 rows, top-p 0.9
    // / top-k 3000, without and with: 20000 logits 36.3 / 25.4 and 36.7 / 27.3 us, 30000 40.3 / 27.0
    // and 39.4 / 28.4, 40000 64.4 / 35.3 and 50.9 / 37.0, 60000 69 / 37.3 and 54.8 / 39.4)
    int lo = 0, hi = kSampBuckets - 1;
    if (p.V > 32768) {
      zero(false);
      u64 sampled = 0;
      sweep(s0 + (warp & 7) * 32, s1, 8, [&](float z, int id) {
        const int k = R.bucket(z);
        sampled += id < c0 + s1;
        if (k < kSampBuckets && (from == 0 || compose(z, id) >= from)) atomicAdd(&chist[k], 1u);
      });
      sampled = sum_row(sampled);
      u64 hc[4], hw[4], at, all;
      bins(false, 0, kSampBuckets - 1, hc, hw);
      if (tid == 0) {
        sh.window[0] = 0;
        sh.window[1] = kSampBuckets - 1;
      }
      u64 own = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {  // counts, or counts times the weight of the bucket's middle
        hw[j] = hc[j];
        if (by_w && hc[j]) {
          double e, sc;
          exp2_64(-64.0 * p.F / kSampBuckets * (tid * 4 + j + 0.5), 30, sh.table, &e, &sc);
          hw[j] = static_cast<u64>(static_cast<double>(hc[j]) * (e * sc));
        }
        own += hw[j];
      }
      block_scan(own, &at, &all, sh.red[0]);
      // the weight from the target on, as a part of the eighth's: of many small weights, where
      // those before may be of a few large ones, which an eighth may miss
      const double rest = static_cast<double>(whole - target) * __hiloint2double((1023 + 30 - p.F) << 20, 0) *
                          static_cast<double>(sampled) / p.V;
      const double t = by_w ? static_cast<double>(all) - rest
                            : static_cast<double>(target) * static_cast<double>(sampled) / p.V;
      // Margins, 64 rows of 151936. Weights: 0.5, 1, 2 and 5 percent take 142, 144, 145 and 149 us
      // for p = 0.9 and logits of standard deviation 1.5; with 0.5 percent p = 0.5 misses and takes
      // 155 where the others take 125 to 129. Counts: without the 16 k = 1100 misses (104 us for 91),
      // with half the 10 percent k = 5000 does (108 for 98); twice either costs nothing.
      const double t0 = by_w ? t - 0.02 * static_cast<double>(all) : 0.9 * t - 16.0;
      const double t1 = by_w ? t + 0.02 * static_cast<double>(all) : 1.1 * t + 16.0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double a = static_cast<double>(at), b = static_cast<double>(at + hw[j]);
        if (a < t0 && t0 <= b) sh.window[0] = tid * 4 + j;
        if (a < t1 && t1 <= b) sh.window[1] = tid * 4 + j;
        at += hw[j];
      }
      samp_sync();  // also: every CTA has read the histograms
      lo = sh.window[0];
      hi = sh.window[1];
    }
    for (int pass = 0;; ++pass) {  // the second with all buckets
      u64 above = 0;
      zero(by_w);
      // up to the window's end; those before it are counted or weighed, those in it join its buckets
      const float hi_x = static_cast<float>(hi + 1);
      auto up_to = [&](float z, int id) {
        const bool in = R.place(z) < hi_x;
        return from == 0 ? in : in && compose(z, id) >= from;
      };
      top_lo = by_w ? lo : 0;
#pragma unroll 1
      for (int q = 0; q < kParts; ++q) {
        if (s0 + q * span >= s1) break;
        u64 s = 0;
        gather(s0 + q * span, min(s1, s0 + (q + 1) * span), up_to, [&](int n) {
          float z[kSampBatch / 32];
          u64 w[kSampBatch / 32];
#pragma unroll
          for (int j = 0; j < kSampBatch / 32; ++j) {
            z[j] = lane + 32 * j < n ? as_float(src[keep[lane + 32 * j]]) : -INFINITY;
            w[j] = by_w ? R.weight(z[j]) : 1;
          }
#pragma unroll
          for (int j = 0; j < kSampBatch / 32; ++j) {
            if (lane + 32 * j >= n) continue;
            const int k = R.bucket(z[j]);
            if (k < lo) {
              s += w[j];
            } else {
              atomicAdd(&chist[k], 1u);
              if (by_w) add_weight(k, w[j]);
            }
          }
        });
        above += s;
        if (top_lo > 0) {
          const u64 of_warp = warp_sum64(s);
          if (lane == 0) sh.top[warp][q] = of_warp;
        }
      }
      if (search(by_w, target, sum_row(above), lo, hi)) break;
      if (pass == 1 || (lo == 0 && hi == kSampBuckets - 1)) return 0;
      lo = 0;
      hi = kSampBuckets - 1;
    }
    const int bucket0 = static_cast<int>(sh.found[0]);
    u64 members = sh.found[1], before = sh.found[2];
    const float bucket_from = static_cast<float>(bucket0), bucket_end = static_cast<float>(bucket0 + 1);
    uint32_t klo = 0, khi = 0xffffffffu;
    bool all_keys = true;
    auto member = [&](float z, int id) {
      const float x = R.place(z);
      const bool in = (x >= bucket_from) & (x < bucket_end);
      if (from == 0 && all_keys) return in;
      const uint32_t key = sort_key(z);
      return in && key >= klo && key <= khi && compose(z, id) >= from;
    };
    // 2048 ranges a level: after three levels a range is one key
    int levels = 0;
    for (; levels < 4 && members > kSampList; ++levels) {
      uint32_t l = 0xffffffffu, h = 0;  // the members' smallest and largest key
      sweep(s0, s1, 1, [&](float z, int id) {
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
      all_keys = false;
      klo = 0xffffffffu;
      khi = 0;
      for (int r = 0; r < C; ++r) {
        klo = min(klo, static_cast<uint32_t>(sh.tot_a[r]));
        khi = max(khi, static_cast<uint32_t>(sh.tot_b[r]));
      }
      if (klo == khi) {  // equal logits: the first ones in vocabulary order
        u64 need = target - before;
        if (by_w) {
          const u64 w = R.weight(key_value(klo));
          need = (need + w - 1) / w;
        }
        auto one = [&](float z, int i) -> u64 { return member(z, i); };
        const int id = locate(one, [&](int, int b0, int b1) {
          u64 s = 0;
          sweep(b0, b1, 1, [&](float z, int i) { s += one(z, i); });
          return s;
        }, [&](u64) -> u64 { return need - 1; });
        if (id >= 0 && lane == 0)
          for (int r = 0; r < C; ++r) dsm_st64(&sh.cut, r, (static_cast<u64>(klo) << 32) | static_cast<uint32_t>(~id));
        samp_sync();
        return sh.cut;
      }
      const int shift = max(0, 32 - __clz(khi - klo) - 11);
      sweep(s0, s1, 1, [&](float z, int id) {
        if (member(z, id)) {
          const int k = (khi - sort_key(z)) >> shift;
          atomicAdd(&chist[k], 1u);
          if (by_w) add_weight(k, R.weight(z));
        }
      });
      samp_sync();
      search(by_w, target, before, 0, kSampBuckets - 1);
      members = sh.found[1];
      before = sh.found[2];
      khi -= static_cast<uint32_t>(sh.found[0]) << shift;
      const uint32_t low = khi - ((1u << shift) - 1);
      klo = low > khi ? klo : max(klo, low);
    }
    // the members go to the first CTA and are sorted
    gather(s0, s1, member, [&](int n) {
      uint32_t at = 0;
      if (lane == 0) at = dsm_add32(&sh.list_n, 0, n);
      at = __shfl_sync(0xffffffffu, at, 0) + lane;
#pragma unroll
      for (int j = 0; j < kSampBatch / 32; ++j) {
        if (lane + 32 * j >= n || at + 32 * j >= kSampList) continue;
        const int i = keep[lane + 32 * j];
        dsm_st64(&sh.list[at + 32 * j], 0, compose(as_float(src[i]), c0 + i));
      }
    });
    samp_sync();
    if (rank == 0) {
      const int n = static_cast<int>(min(members, static_cast<u64>(kSampList)));
      // by the place within the bucket, or within what is left of its keys
      const int shift = max(0, 32 - __clz(khi - klo) - 11);
      sort_buckets(sh.list, n, sh.chist, sh.red[0], [&](u64 x) {
        const uint32_t key = static_cast<uint32_t>(x >> 32);
        if (levels > 0) return static_cast<int>(min((khi - key) >> shift, kSampBuckets - 1u));
        const float at = R.place(key_value(key)) - static_cast<float>(bucket0);
        return static_cast<int>(fminf(fmaxf(at, 0.f) * static_cast<float>(kSampBuckets), kSampBuckets - 1.f));
      });
      for (int c = 0; c < n; c += kSampThreads) {
        const int i = c + tid;
        const u64 x = i >= n ? 0 : (by_w ? R.weight(key_value(static_cast<uint32_t>(sh.list[i] >> 32))) : 1);
        u64 at, sum;
        block_scan(x, &at, &sum, sh.red[0]);
        at += before;
        before += sum;
        if (at < target && target <= at + x)
          for (int r = 0; r < C; ++r) dsm_st64(&sh.cut, r, sh.list[i]);
      }
      if (tid == 0) sh.list_n = 0;
    }
    samp_sync();
    return sh.cut;
  };

  u64 cut = 0;  // every (key, id) is above
  if (f.k > 0) {
    cut = prefix(false, 0, f.k, 0);
    samp_sync();  // cut is read before it is written again
  }
  if (f.use_p) {
    u64 all = f.whole(total, p.F);
    if (f.k > 0) all = sum_row(weigh(s0, s1, [&](float z, int id) { return R.bucket(z) < kSampBuckets && compose(z, id) >= cut; }));
    cut = max(cut, prefix(true, cut, f.p_target(all), all));  // 0 if the target is past all by a rounding
  }
  // min-p as a bucket, to pass over most of the row; a logit's own test is in fp64
  const double bm = f.use_m ? -f.low64 / 64.0 * (kSampBuckets / static_cast<double>(p.F)) + 1.0 : kSampBuckets;
  const int last = static_cast<int>(fmin(bm, kSampBuckets - 1.0));
  // the bucket of the cut; those before it lie above, whatever their ids
  const int cut_bucket = cut ? R.bucket(key_value(static_cast<uint32_t>(cut >> 32))) : kSampBuckets;
  const float end_x = static_cast<float>(min(last, cut_bucket) + 1), cut_x = static_cast<float>(cut_bucket);
  auto kept = [&](float z, int id) {
    const float x = R.place(z);
    if (!(x < end_x)) return false;
    if (x >= cut_x && compose(z, id) < cut) return false;
    return !f.use_m || R.y64(z) >= f.low64;
  };
  // What prefix() weighed is kept whole where the cut lies below it and min-p does not cut: the
  // rest of the row has few that are kept.
  if (f.use_m || cut_bucket < top_lo) top_lo = 0;
  const float top_x = static_cast<float>(top_lo);
  const int id = locate([&](float z, int i) -> u64 { return kept(z, i) ? R.weight(z) : 0; },
                        [&](int q, int b0, int b1) {
                          const u64 s = weigh(b0, b1, [&](float z, int i) { return R.place(z) >= top_x && kept(z, i); });
                          return s + (top_lo > 0 && lane == 0 ? sh.top[warp][q] : 0);
                        },
                        [&](u64 all) { return f.draw_at(all); });
  if (id >= 0 && lane == 0) {
    p.tokens[row] = id;
    if (p.logprob) p.logprob[row] = samp_logprob(R, as_float(static_cast<const T*>(p.logits)[row * p.V + id]), total);
  }
}

}  // namespace lmh
