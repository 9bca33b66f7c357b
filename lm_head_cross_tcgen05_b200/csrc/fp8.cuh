// fp8.cuh — the 8-bit logits product on the tensor cores:
//   z[n, v] = sum_b hs[n, b] ws[v / 128, b] sum_{k in block b} H8[n, k] W8[v, k]
// with b over blocks of 128 columns. The scales are general fp32 numbers, so they cannot ride on
// the MMA: each block of 128 columns (four tcgen05.mma kind::f8f6f4 steps of K = 32) goes into a
// fresh TMEM accumulator, which the epilogue warps read and add, times its scale, into fp32
// registers while the next block's MMAs fill another one. That also bounds what the tensor core
// itself accumulates to 128 terms.
//
// Two kernels, by which operand takes the accumulator's 128 lanes:
//  * few tokens (decode): W8 is the A operand (128 vocabulary rows, one scale of ws each) and H8
//    the B operand (TN = 16, 32 or 64 tokens), so the tensor core wastes no rows on a few tokens,
//    and an epilogue warp writes 32 adjacent logits of one token with each store.
//  * many tokens: H8 is A (128 tokens) and W8 is B (256 vocabulary rows), so a thread's scales
//    are one hs and two ws per block, held in registers, and its accumulator row is one token's.
//
// Roles (per CTA): warp 0 lane 0 loads the operands with TMA; warp 1 lane 0 issues the MMAs; the
// other warps scale and add. Every wait is bounded; no warp waits for another except on those
// mbarriers and at the end.
#pragma once

#include <cuda_bf16.h>

#include "sm100.cuh"

namespace lmh {

constexpr int kFpK = 128;  // columns per scale block
constexpr int kFpM = 128;  // accumulator lanes

// Scale blocks per row (d up to 8192) whose token scales the few-token kernel keeps.
constexpr int kFewBlocks = 64;

template <int TN>
struct FpFew {
  static constexpr int THREADS = 192;
  static constexpr int NBUF = 8;  // TMEM accumulators (128256 x 4096, 64 tokens: 103 us with 4, 98 with 8)
  static constexpr int TMEM = TN * NBUF;
  // A stage is KB blocks: the MMA thread's wait and commit per stage hold up the next loads.
  // 128256 x 4096, 1 / 64 tokens: one block a stage 100.6 / 116 us, two 87.3 / 104.5, four (two
  // stages) 87.1 / 102.5 (with four accumulators).
  static constexpr int KB = 2, A_BYTES = kFpM * kFpK, B_BYTES = TN * kFpK, STAGE = KB * (A_BYTES + B_BYTES);
  static constexpr int STAGES = TN == 64 ? 4 : 5;
  static constexpr int HS = kFewBlocks * TN * 4;  // the tokens' scales
  static constexpr int SMEM = STAGES * STAGE + HS + 1024;
};

// kind::f8f6f4: e4m3 A and B (format 0), K-major both, fp32 accumulator.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

struct FpParams {
  long long N, V;
  int nb;              // scale blocks per row
  int vtiles, ntiles;  // tiles over the vocabulary and the tokens (few tokens: one)
  const float* hs;     // [N, nb]
  const float* ws;     // [ceil(V / 128), nb]
  void* out;           // [N, V] fp32 or bf16
  uint32_t* err;       // cleared by the first block: a wait that sets it gives up seconds later
};

__device__ __forceinline__ void put_logit(float* out, long long i, float x) { out[i] = x; }
__device__ __forceinline__ void put_logit(__nv_bfloat16* out, long long i, float x) {
  out[i] = __float2bfloat16_rn(x);
}

// The producer's last act: the loads still in flight land before the CTA may exit. `issued`
// stages were filled in ring order.
template <int STAGES>
__device__ __forceinline__ void wait_loads(const uint64_t* full_bar, uint32_t issued, uint32_t* err) {
  const uint32_t first = issued > STAGES ? issued - STAGES : 0;
  for (uint32_t i = first; i < issued; ++i)
    mbar_wait(smem_u32(&full_bar[i % STAGES]), (i / STAGES) & 1u, err);
}

// acc += (a, b) * (h * w) in both halves; the product of the scales is rounded once.
__device__ __forceinline__ void add_scaled(uint64_t& acc, float a, float b, uint64_t h, uint64_t w) {
  asm("{\n\t.reg .b64 v, s;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 s, %3, %4;\n\tfma.rn.f32x2 %0, v, s, %0;\n\t}"
      : "+l"(acc) : "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "l"(h), "l"(w));
}

// Bound by the stream of W8: 128256 x 4096 takes 87 us for one token (6.0 TB/s of the 6.5 that a
// copy reaches) and 98 for 64 (with 33 MB of logits, 5.7 TB/s). 32000 x 2048 takes 18.5 us: the launch,
// the first loads' way and two tiles for most SMs where 1.7 would do. The token scales are read
// from shared memory, since they are the same for every tile; a tile's 128 x nb vocabulary scales
// are one per block, broadcast by a shuffle.
template <int TN, class Out>
__global__ void __launch_bounds__(FpFew<TN>::THREADS, 1)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH,
                   const FpParams p) {
  using C = FpFew<TN>;
  constexpr int STAGES = C::STAGES, NBUF = C::NBUF;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], empty_bar[STAGES], tfull_bar[NBUF],
      tempty_bar[NBUF], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const uint32_t smem_base = (smem_u32(dsmem) + 1023u) & ~1023u;
  float* hs = reinterpret_cast<float*>(dsmem + (smem_base - smem_u32(dsmem)) + STAGES * C::STAGE);  // [nb][TN]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = p.vtiles;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 1);
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(smem_u32(&tfull_bar[b]), 1);
      mbar_init(smem_u32(&tempty_bar[b]), 4);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmH);
      uint32_t it = 0;
      for (int t = blockIdx.x; t < tiles && !abort_flag; t += gridDim.x) {
        const int v0 = t * kFpM;
        for (int kb = 0; kb < p.nb; kb += C::KB, ++it) {
          const uint32_t s = it % STAGES;
          if (!mbar_wait(smem_u32(&empty_bar[s]), ((it / STAGES) & 1u) ^ 1u, p.err)) {
            abort_flag = 1;
            break;
          }
          const uint32_t bar = smem_u32(&full_bar[s]), dst = smem_base + s * C::STAGE;
          mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
          for (int j = 0; j < C::KB; ++j) {  // past the last block: zeros
            tma_load_2d(dst + j * C::A_BYTES, &tmW, bar, (kb + j) * kFpK, v0);
            tma_load_2d(dst + C::KB * C::A_BYTES + j * C::B_BYTES, &tmH, bar, (kb + j) * kFpK, 0);
          }
        }
      }
      wait_loads<STAGES>(full_bar, it, p.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(kFpM, TN);
      uint32_t kbg = 0, it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        for (int kb = 0; kb < p.nb && ok; kb += C::KB, ++it) {
          const uint32_t s = it % STAGES;
          ok = !abort_flag && mbar_wait(smem_u32(&full_bar[s]), (it / STAGES) & 1u, p.err);
#pragma unroll
          for (int j = 0; j < C::KB; ++j) {
            if (!ok || kb + j >= p.nb) break;
            const uint32_t b = kbg % NBUF;
            ok = mbar_wait(smem_u32(&tempty_bar[b]), ((kbg / NBUF) & 1u) ^ 1u, p.err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = smem_base + s * C::STAGE + j * C::A_BYTES;
            const uint32_t h = smem_base + s * C::STAGE + C::KB * C::A_BYTES + j * C::B_BYTES;
#pragma unroll
            for (int k = 0; k < kFpK / 32; ++k)
              mma_e4m3(tmem_base + b * TN, make_sw128_desc(a + k * 32, 16, 1024),
                       make_sw128_desc(h + k * 32, 16, 1024), idesc, k != 0);
            mma_commit(smem_u32(&tfull_bar[b]));
            ++kbg;
          }
          if (ok) mma_commit(smem_u32(&empty_bar[s]));
        }
      }
      if (!ok) abort_flag = 1;
      // No MMA may still be writing TMEM when the columns are released.
      mma_commit(smem_u32(&drain_bar));
      mbar_wait(smem_u32(&drain_bar), 0, p.err);
    }
  } else {
    constexpr int G = TN >= 32 ? 32 : 16;
    const int q = warp & 3;  // TMEM lanes 32 q .. 32 q + 31
    // every tile has the same tokens: their scales stay in shared memory, block by block
    for (int i = threadIdx.x - 64; i < p.nb * TN; i += 128) {
      const int n = i % TN;
      hs[i] = n < p.N ? __ldg(p.hs + n * p.nb + i / TN) : 0.f;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // the four epilogue warps, which all come here
    // a tile's scales of W8, 32 blocks in a warp's lanes, the next 32 (of the next tile, at the end)
    // on their way
    auto w32 = [&](int t, int kb0) {
      return t < tiles && kb0 + lane < p.nb ? __ldg(p.ws + static_cast<long long>(t) * p.nb + kb0 + lane) : 0.f;
    };
    uint32_t kbg = 0;
    float wnext = w32(blockIdx.x, 0);
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      uint64_t acc[TN / 2];
#pragma unroll
      for (int i = 0; i < TN / 2; ++i) acc[i] = 0;
      float wnow = 0.f;
      bool ok = true;
      for (int kb = 0; kb < p.nb; ++kb, ++kbg) {
        if ((kb & 31) == 0) {
          wnow = wnext;
          wnext = kb + 32 < p.nb ? w32(t, kb + 32) : w32(t + gridDim.x, 0);
        }
        const float w = __shfl_sync(0xffffffffu, wnow, kb & 31);
        uint64_t w2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(w2) : "r"(__float_as_uint(w)));
        const uint32_t b = kbg % NBUF;
        ok = !abort_flag && mbar_wait(smem_u32(&tfull_bar[b]), (kbg / NBUF) & 1u, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * TN;
        const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(hs + kb * TN);  // two pairs each
#pragma unroll
        for (int g = 0; g < TN; g += G) {
          float v[G];
          if constexpr (G == 32) tmem_ld32(taddr + g, v);
          else tmem_ld16(taddr + g, v);
#pragma unroll
          for (int i = 0; i < G; i += 4) {
            const ulonglong2 f = s2[(g + i) / 4];
            add_scaled(acc[(g + i) / 2], v[i], v[i + 1], f.x, w2);
            add_scaled(acc[(g + i) / 2 + 1], v[i + 2], v[i + 3], f.y, w2);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&tempty_bar[b]));
      }
      if (!ok) {
        abort_flag = 1;
        break;
      }
      const long long v = static_cast<long long>(t) * kFpM + q * 32 + lane;
      if (v < p.V) {
        Out* out = static_cast<Out*>(p.out);
#pragma unroll
        for (int i = 0; i < TN; ++i)
          if (i < p.N)
            put_logit(out, i * p.V + v, __uint_as_float(static_cast<uint32_t>(i & 1 ? acc[i / 2] >> 32 : acc[i / 2])));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::TMEM);
}

// ---------------------------------------------------------------------------- many tokens
// 32 TMEM columns of a warp's lanes, not waited for; tmem_landed() is what the values pass through.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_landed(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]),
                 "+r"(r[31])
               :
               : "memory");
}
// acc += (a, b) * f in both halves, one instruction for the two.
__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t a, uint32_t b, uint64_t f) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
      : "+l"(acc) : "r"(a), "r"(b), "l"(f));
}

struct FpMany {
  static constexpr int TV = 256;          // vocabulary rows per tile
  static constexpr int EPI = 16;          // epilogue warps: 64 columns each of a lane quarter
  static constexpr int COLS = TV / (EPI / 4);
  static constexpr int THREADS = 128 + 32 * EPI;
  static constexpr int NBUF = 2, TMEM = 512;
  static constexpr int A_BYTES = kFpM * kFpK, B_BYTES = TV * kFpK, STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = 3;
  // Barriers for "the MMAs of this block are done". A block that comes DONE later cannot be done
  // before either waiter has seen this one: it is loaded, and its columns are freed, after that.
  static constexpr int DONE = 8;
  static_assert(DONE >= STAGES + NBUF, "a waiter is at most so many blocks behind");
  static constexpr int GROUPS = 4;        // of four blocks, whose scales are in shared memory
  static constexpr int BOX = 2048;        // per epilogue warp: 32 tokens x 64 bytes (512-byte aligned)
  static constexpr int SC = 520;          // floats per group: 128 tokens' and 2 vocabulary blocks', by fours
  static constexpr int SMEM = STAGES * STAGE + EPI * BOX + GROUPS * SC * 4 + 1024;
  // registers a thread: 640 x 96 at the launch, then 128 x 32 + 512 x 112, which is the same sum
  static constexpr int REG_LOAD = 32, REG_EPI = 112;
};

// An accumulator is held from its MMAs (512 cycles) until its last column is read, and two of them
// are all that TMEM holds, so the way round counts: commit, wake, read, arrive, wake, MMAs. It is
// not what bounds this kernel, though: bare, it takes 173 us of 301 in the case below, 6 percent
// over the MMAs' own time. What lies on top does: the readers' waits, scales, additions and the
// tile's output, with the tensor pipe active 41 percent of the time. 16 warps read at once, 64
// columns each with the sums in registers, which the loading warps give up theirs for; the
// additions take two values an instruction; one commit a block both frees its stage and hands over
// its columns; and a spare warp brings the scales to shared memory four blocks at a time, up to 16
// ahead, since loads of their own would make the reading warps wait. 4096 x 32000 x 2048 to bf16:
// 349 us with eight warps of 128 columns, 311 with 16, 301 with the scales by fours (1780 TFLOP/s,
// 54 percent of twice the measured bf16 rate). In copies for timing, without the operands' loads it
// took 300 where this took 312, without the scales 285, without TMEM reads 273, without output 287,
// and with none of these, one MMA a block and no additions 173. Accumulators of 128 columns, whose
// way round would be shorter, took 367, and pairs of CTAs that share a 256 x 256 tile 660.
// TMA: the output goes out by TMA from staged boxes of 32 tokens x 64 bytes, where its rows are
// 16-byte aligned; otherwise by transposes of 32 x 16 through shared memory.
template <class Out, bool TMA>
__global__ void __launch_bounds__(FpMany::THREADS, 1)
    fp8_many_kernel(const __grid_constant__ CUtensorMap tmW,
                    const __grid_constant__ CUtensorMap tmH,
                    const __grid_constant__ CUtensorMap tmOut, const FpParams p) {
  using C = FpMany;
  constexpr int STAGES = C::STAGES, NBUF = C::NBUF, TV = C::TV, DONE = C::DONE;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[STAGES], done_bar[DONE], tempty_bar[NBUF], drain_bar;
  __shared__ __align__(8) uint64_t sfull_bar[C::GROUPS], sfree_bar[C::GROUPS];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  const uint32_t smem_base = (smem_u32(dsmem) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles = p.vtiles * p.ntiles;  // tokens fastest: a wave shares few tiles of W8
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.err = 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&full_bar[s]), 1);
    for (int i = 0; i < DONE; ++i) mbar_init(smem_u32(&done_bar[i]), 1);
    for (int b = 0; b < NBUF; ++b) mbar_init(smem_u32(&tempty_bar[b]), C::EPI);
    for (int i = 0; i < C::GROUPS; ++i) {
      mbar_init(smem_u32(&sfull_bar[i]), 32);
      mbar_init(smem_u32(&sfree_bar[i]), C::EPI);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::TMEM);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_LOAD));
    if (warp == 0 && lane == 0) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmH);
      uint32_t kbg = 0;
      for (int t = blockIdx.x; t < tiles && !abort_flag; t += gridDim.x) {
        const int v0 = (t / p.ntiles) * TV, n0 = (t % p.ntiles) * kFpM;
        for (int kb = 0; kb < p.nb; ++kb, ++kbg) {
          const uint32_t s = kbg % STAGES;
          if (kbg >= STAGES && !mbar_wait(smem_u32(&done_bar[(kbg - STAGES) % DONE]), ((kbg - STAGES) / DONE) & 1u, p.err)) {
            abort_flag = 1;
            break;
          }
          const uint32_t bar = smem_u32(&full_bar[s]), dst = smem_base + s * C::STAGE;
          mbar_arrive_expect_tx(bar, C::STAGE);
          tma_load_2d(dst, &tmH, bar, kb * kFpK, n0);
          tma_load_2d(dst + C::A_BYTES, &tmW, bar, kb * kFpK, v0);
        }
      }
      wait_loads<STAGES>(full_bar, kbg, p.err);
    } else if (warp == 1 && lane == 0) {
      constexpr uint32_t idesc = make_idesc_e4m3(kFpM, TV);
      uint32_t kbg = 0;
      for (int t = blockIdx.x; t < tiles && !abort_flag; t += gridDim.x) {
        for (int kb = 0; kb < p.nb; ++kb, ++kbg) {
          const uint32_t s = kbg % STAGES, b = kbg % NBUF;
          if (!mbar_wait(smem_u32(&tempty_bar[b]), ((kbg / NBUF) & 1u) ^ 1u, p.err) ||
              !mbar_wait(smem_u32(&full_bar[s]), (kbg / STAGES) & 1u, p.err)) {
            abort_flag = 1;
            break;
          }
          tc_fence_after();
          const uint32_t h = smem_base + s * C::STAGE, w = h + C::A_BYTES;
#pragma unroll
          for (int k = 0; k < kFpK / 32; ++k)
            mma_e4m3(tmem_base + b * TV, make_sw128_desc(h + k * 32, 16, 1024),
                     make_sw128_desc(w + k * 32, 16, 1024), idesc, k != 0);
          mma_commit(smem_u32(&done_bar[kbg % DONE]));
        }
      }
      mma_commit(smem_u32(&drain_bar));
      mbar_wait(smem_u32(&drain_bar), 0, p.err);
    } else if (warp == 2) {
      // the scales of four blocks at a time, up to GROUPS * 4 blocks ahead of the epilogue
      const bool wide = (p.nb & 3) == 0 && (reinterpret_cast<uintptr_t>(p.hs) & 15) == 0;
      uint32_t gi = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
        const int v = (t / p.ntiles) * (TV / kFpK) + (lane >> 2), n0 = (t % p.ntiles) * kFpM;
        const float* ws = p.ws + static_cast<long long>(v) * p.nb + (lane & 3);
        const bool wv = lane < 4 * (TV / kFpK) && static_cast<long long>(v) * kFpK < p.V;
        for (int kb = 0; kb < p.nb && ok; kb += 4, ++gi) {
          const uint32_t slot = gi % C::GROUPS;
          ok = !abort_flag && mbar_wait(smem_u32(&sfree_bar[slot]), ((gi / C::GROUPS) & 1u) ^ 1u, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t dst = smem_base + STAGES * C::STAGE + C::EPI * C::BOX + slot * C::SC * 4;
#pragma unroll
          for (int j = 0; j < kFpM / 32; ++j) {
            const int n = n0 + lane + 32 * j;
            const float* hs = p.hs + (n < p.N ? static_cast<long long>(n) * p.nb + kb : 0ll);
            const uint32_t to = dst + (lane + 32 * j) * 16;
            if (wide) {
              asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(hs), "r"(n < p.N ? 16 : 0) : "memory");
            } else {
              for (int i = 0; i < 4 && kb + i < p.nb; ++i)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * i), "l"(n < p.N ? hs + i : hs), "r"(n < p.N ? 4 : 0) : "memory");
            }
          }
          if (wv && kb + (lane & 3) < p.nb)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + (kFpM * 4 + lane) * 4), "l"(ws + kb) : "memory");
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sfull_bar[slot])) : "memory");
        }
      }
      if (!ok) abort_flag = 1;
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_EPI));
    constexpr int COLS = C::COLS;
    const int q = warp & 3, c0 = ((warp - 4) >> 2) * COLS;  // TMEM lanes 32 q .., columns c0 ..
    const uint32_t box = smem_base + STAGES * C::STAGE + (warp - 4) * C::BOX;
    const float* sc = reinterpret_cast<const float*>(dsmem + (smem_base - smem_u32(dsmem)) + STAGES * C::STAGE + C::EPI * C::BOX);
    Out* out = static_cast<Out*>(p.out);
    uint32_t kbg = 0, gi = 0;
    for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
      const long long v0 = static_cast<long long>(t / p.ntiles) * TV + c0;
      const long long r0 = static_cast<long long>(t % p.ntiles) * kFpM + q * 32;  // warp's tokens
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int i = 0; i < COLS / 2; ++i) acc[i] = 0;
      bool ok = true;
      for (int kb = 0; kb < p.nb; kb += 4, ++gi) {
        const uint32_t slot = gi % C::GROUPS;
        ok = !abort_flag && mbar_wait(smem_u32(&sfull_bar[slot]), (gi / C::GROUPS) & 1u, p.err);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float4 h4 = *reinterpret_cast<const float4*>(sc + slot * C::SC + (q * 32 + lane) * 4);
        const float4 w4 = *reinterpret_cast<const float4*>(sc + slot * C::SC + (kFpM + c0 / kFpK) * 4);
        const float s[4] = {h4.x * w4.x, h4.y * w4.y, h4.z * w4.z, h4.w * w4.w};
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sfree_bar[slot]));
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4, ++kbg) {
          if (kb + i4 >= p.nb) break;
          const uint32_t b = kbg % NBUF;
          ok = mbar_wait(smem_u32(&done_bar[kbg % DONE]), (kbg / DONE) & 1u, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          uint64_t f;
          asm("mov.b64 %0, {%1, %1};" : "=l"(f) : "r"(__float_as_uint(s[i4])));
          const uint32_t taddr = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * TV + c0;
#pragma unroll
          for (int g = 0; g < COLS / 32; ++g) {
            uint32_t v[32];
            tmem_ld32_start(taddr + 32 * g, v);
            tmem_landed(v);
            if (g == COLS / 32 - 1) {  // all columns are read: the block after next may go here
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&tempty_bar[b]));
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) fma2(acc[g * 16 + i], v[2 * i], v[2 * i + 1], f);
          }
        }
        if (!ok) break;
      }
      if (!ok) {
        abort_flag = 1;
        break;
      }
      if (TMA) {
        constexpr int PER = 64 / sizeof(Out);  // columns per box
#pragma unroll
        for (int g = 0; g < COLS / PER; ++g) {
          if (v0 + g * PER >= p.V || r0 >= p.N) continue;  // of the whole warp
          if (lane == 0) bulk_wait_read_all();  // the box before has been read
          __syncwarp();
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (sizeof(Out) == 4) {
              w[i] = (i & 1) ? static_cast<uint32_t>(acc[g * 8 + i / 2] >> 32) : static_cast<uint32_t>(acc[g * 8 + i / 2]);
            } else {
              const uint64_t a = acc[g * 16 + i];
              w[i] = pack_bf16x2(__uint_as_float(static_cast<uint32_t>(a)), __uint_as_float(static_cast<uint32_t>(a >> 32)));
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)  // 64-byte rows, 16-byte chunks permuted by the row as TMA reads them
            st_shared_v4(box + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4),
                         make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tmOut, box, static_cast<int>(v0 + g * PER), static_cast<int>(r0));
            bulk_commit();
          }
        }
      } else {
        // a lane holds one token's columns: turn 32 x 16 blocks so that half a warp stores adjacent
        // columns of one token, whatever V's alignment; column c of row r lies at c ^ (r & 15)
        float* tr = reinterpret_cast<float*>(dsmem + (box - smem_u32(dsmem)));
        const int c = lane & 15;
#pragma unroll
        for (int g = 0; g < COLS / 16; ++g) {
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            tr[lane * 16 + ((2 * i) ^ (lane & 15))] = __uint_as_float(static_cast<uint32_t>(acc[g * 8 + i]));
            tr[lane * 16 + ((2 * i + 1) ^ (lane & 15))] = __uint_as_float(static_cast<uint32_t>(acc[g * 8 + i] >> 32));
          }
          __syncwarp();
          const long long v = v0 + g * 16 + c;
          if (v < p.V) {
#pragma unroll 8
            for (int i = lane >> 4; i < 32; i += 2)
              if (r0 + i < p.N) put_logit(out, (r0 + i) * p.V + v, tr[i * 16 + (c ^ (i & 15))]);
          }
        }
      }
    }
    if (TMA && lane == 0) bulk_wait_all();  // every box has reached global memory
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::TMEM);
}

}  // namespace lmh
