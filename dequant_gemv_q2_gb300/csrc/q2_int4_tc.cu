// y = W x for 4-bit weights with group scales at many tokens, on the
// 5th-generation tensor cores (tcgen05); the formula, the weights' layout and
// the exact operands q - z are those of q2_int4.cuh.
//
// A CTA owns 128 rows (the instruction's M) and a range of 128-column blocks,
// and runs them through rings of stages with four roles:
//   - 8 decoder warps, two per TMEM lane quarter, copy their weights to
//     shared memory RAW blocks ahead, unpack them to q - z in fp16 and store
//     them to tensor memory.  The packed order is that of a 16 x 16 operand
//     fragment, which is what tcgen05.st's 16x128b shape stores: no exchange;
//   - 4 staging warps bring x of all tokens to shared memory in the 128-byte
//     swizzle, columns in the packed order (a thread's 32 columns are four
//     16-byte pieces transposed in registers) and 8-bit x turned to fp16;
//   - 2 issuing warps take blocks in turn: lane 0 issues the block's eight
//     M = 128, K = 16 products and commits them.  An issuing thread that
//     touches memory waits for its own queue of products, so with two of them
//     one waits while the other's products run;
//   - 4 summing warps, one per lane quarter, a row per lane, read each scale
//     group's product from one of kAccs accumulators, multiply it by the
//     group's scale and add it to the row's fp32 sums in registers: group
//     scales cost no rounding, and the accumulator is free for another group.
// An instruction costs the same for 16 to 64 tokens, so nothing depends on
// the token count but the bytes of x.  The column range is split over a
// cluster's CTAs where there are few row tiles, whose sums meet in rank order
// in distributed shared memory.
//
// Every wait is bounded: one that runs out sets the error word
// (q2_device_errors) and a flag on which the other roles give up; the
// products issued are waited for before tensor memory is released, and the
// CTA's rows come out NaN.
#include <cooperative_groups.h>

#include <algorithm>

#include "q2_int4.cuh"
#include "q2_tcgen.cuh"

namespace cg = cooperative_groups;

__device__ unsigned int q2_int4_error = 0;
__device__ long long q2_int4_stage_wait_limit = 0;           // 0: the normal bound (q2_debug_wait_limit)

namespace q2 {
namespace {

constexpr int kRows = 128, kDec = 8, kStage = 4, kIssue = 2, kSum = 4;   // rows; warps of each role
constexpr int kThreads = (kDec + kStage + kIssue + kSum) * 32;
constexpr int kRing = 4;                      // blocks in flight: A in tensor memory, x in shared memory
constexpr int kAccs = 4;                      // accumulators of 64 columns
constexpr int kRaw = 4;                       // blocks of packed weights in shared memory per decoder warp
constexpr int kRawBytes = 2 * (512 + 64);     // two row tiles: half a block and the zero points
constexpr uint32_t kTmem = 512, kAcol = 64 * kAccs;
constexpr int kOutLd = kRows + 4, kMaxSplit = 8;
#ifndef TCB
#define TCB (1ll << 22)
#endif
constexpr long long kBound = TCB;
constexpr int kOneCta = 116 * 1024;           // at most one CTA of this or the other tcgen05 kernels per SM (each holds all of TMEM)

struct TcArgs {
  Int4Args a;
  int N, nsplit;                              // tokens rounded up to 16; CTAs of a row tile
};

// 16 rows x 64 columns of operand fragments (four 16-column steps).
__device__ __forceinline__ void tmem_st_frag(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

struct Bars {
  uint64_t full[kRing];       // A and x of a block are there (decoder and staging warps)
  uint64_t done[kRing];       // its products are done: the stage is free (commit)
  uint64_t ready[kAccs];      // an accumulator holds a group's product (commit)
  uint64_t taken[kAccs];      // it has been read (summing warps)
  uint64_t drain[kIssue];     // everything an issuing warp has issued is done
  uint32_t tmem;
  int abort;
};

template <int GPB, bool X8>
__global__ void __launch_bounds__(kThreads, 1) k_int4_tc(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char q2_int4tc_smem[];
  const Int4Args& a = ta.a;
  constexpr int STEPS = 8 / GPB, esz = X8 ? 1 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = ta.N, nsplit = ta.nsplit, atom = N * 128, bbytes = 2 * atom;
  const int rank = (int)blockIdx.x % nsplit, tile0 = (int)blockIdx.x / nsplit * (kRows / 16);
  const int b0 = (int)((long long)a.nblk * rank / nsplit), n = (int)((long long)a.nblk * (rank + 1) / nsplit) - b0;
  const uint32_t sB = (saddr(q2_int4tc_smem) + 1023u) & ~1023u;
  unsigned char* B = q2_int4tc_smem + (sB - saddr(q2_int4tc_smem));
  const uint32_t sraw = sB + kRing * bbytes;
  Bars* bar = reinterpret_cast<Bars*>(B + std::max(kRing * bbytes + kDec * kRaw * kRawBytes, N * kOutLd * 4));
  volatile int* give_up = &bar->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(saddr(&bar->full[i]), kDec + kStage);
      mbar_init(saddr(&bar->done[i]), 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(saddr(&bar->ready[i]), 1);
      mbar_init(saddr(&bar->taken[i]), kSum);
    }
    for (int i = 0; i < kIssue; ++i) mbar_init(saddr(&bar->drain[i]), 1);
    bar->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(&bar->tmem)), "r"(kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  pdl_trigger();
  bool ok = true;
  auto failed = [&](unsigned int code) {
    if (lane == 0) {
      atomicExch(&q2_int4_error, code);
      *give_up = 1;
    }
    return false;
  };
  auto wait = [&](uint64_t& b, int phase, unsigned int code, long long limit = kBound) {
    return __all_sync(~0u, mbar_wait(saddr(&b), (uint32_t)phase & 1u, limit, give_up)) ? true : failed(code);
  };
  float acc[64];

  if (warp < kDec) {
    // ---- decoders: half `hf` of the blocks of row tiles 2 * quarter, + 1
    const int quarter = warp & 3, hf = warp >> 2, g = lane >> 2;
    const uint32_t raw = sraw + warp * (kRaw * kRawBytes);
    const unsigned char* src[2];
    for (int m = 0; m < 2; ++m)                     // a missing row tile: the last one; its rows are not stored
      src[m] = a.w + ((size_t)min(tile0 + 2 * quarter + m, a.ntile - 1) * a.nblk + b0) * a.item;
    auto copy = [&](int i) {
      if (i < n) {
        const uint32_t d = raw + (i % kRaw) * kRawBytes;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          cp16(d + m * 576 + lane * 16, src[m] + hf * 512 + lane * 16);
          if (a.zeros && lane < GPB) cp16(d + m * 576 + 512 + lane * 16, src[m] + 1024 + GPB * 32 + lane * 16);
          src[m] += a.item;
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < kRaw - 1; ++i) copy(i);
    for (int i = 0; i < n && ok; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRaw - 2) : "memory");
      __syncwarp();
      copy(i + kRaw - 1);
      const int st = i % kRing;
      uint32_t A[2][16];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t at = raw + (i % kRaw) * kRawBytes + m * 576;
        const uint4 w = lds128(at + lane * 16);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int q = GPB == 1 ? 0 : GPB == 2 ? hf : 2 * hf + (t >> 1);          // the step's scale group
          const uint32_t zz = a.zeros ? lds16(at + 512 + (g * GPB + q) * 2) : 0x0808u;
          unpack_step(word(w, t), zz, A[m][4 * t], A[m][4 * t + 1], A[m][4 * t + 2], A[m][4 * t + 3]);
        }
      }
      if (i == kRing) pdl_wait();                   // no bounded wait may have to wait for the previous kernel
      if (i >= kRing) ok = wait(bar->done[st], i / kRing - 1, 1u);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int m = 0; m < 2; ++m)
        tmem_st_frag(tmem + ((uint32_t)(quarter * 32 + m * 16) << 16) + kAcol + st * 64 + hf * 32, A[m]);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&bar->full[st]));
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  } else if (warp < kDec + kStage) {
    // ---- x: task (token t, run q of 32 columns): 64 (32) bytes in, four 16-byte pieces out
    const int tid = threadIdx.x - kDec * 32, ntask = N * 4;
    uint4 v[2][4];
    auto load = [&](int i) {
      if (i < n) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = tid + k * (kStage * 32), t = e % N, q = e / N, c = (b0 + i) * 128 + q * 32;
          const bool live = e < ntask && t < a.ntok && c < a.C;
          const uint4* from =
              reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.x) + ((size_t)t * a.C + c) * esz);
#pragma unroll
          for (int p = 0; p < (X8 ? 2 : 4); ++p) v[k][p] = live ? from[p] : make_uint4(0, 0, 0, 0);
        }
      }
    };
    pdl_wait();                                     // x may come from the previous kernel
    load(0);
    for (int i = 0; i < n && ok; ++i) {
      const int st = i % kRing;
      if (i >= kRing) ok = wait(bar->done[st], i / kRing - 1, 2u);
      if (!ok) break;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int e = tid + k * (kStage * 32), t = e % N, q = e / N;
        if (e < ntask) {
          uint32_t in[4][4];                        // run j of 8 columns, pair p
          if constexpr (X8) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              int8x4(word(v[k][j >> 1], 2 * (j & 1)), in[j][0], in[j][1]);
              int8x4(word(v[k][j >> 1], 2 * (j & 1) + 1), in[j][2], in[j][3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int p = 0; p < 4; ++p) in[j][p] = word(v[k][j], p);
          }
          unsigned char* d = B + st * bbytes + (q >> 1) * atom + t * 128;
#pragma unroll
          for (int p = 0; p < 4; ++p)
            *reinterpret_cast<uint4*>(d + (((4 * (q & 1) + p) ^ (t & 7)) << 4)) =
                make_uint4(in[0][p], in[1][p], in[2][p], in[3][p]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&bar->full[st]));
      load(i + 1);
    }
  } else if (warp < kDec + kStage + kIssue) {
    // ---- products of every kIssue-th block
    pdl_wait();
    const int me = warp - kDec - kStage;
    const uint32_t idesc = idesc_f16(kRows, N);
    const long long limit = q2_int4_stage_wait_limit > 0 ? q2_int4_stage_wait_limit : kBound;
    for (int i = me; i < n && ok; i += kIssue) {
      const int st = i % kRing;
      ok = wait(bar->full[st], i / kRing, 3u, limit);
      for (int q = 0; q < GPB && ok; ++q) {
        const int gi = i * GPB + q, d = gi % kAccs;
        if (gi >= kAccs) ok = wait(bar->taken[d], gi / kAccs - 1, 4u);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t bs = sB + st * bbytes, at = tmem + kAcol + st * 64;
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int k = q * STEPS + s;
            mma_f16_ta(tmem + d * 64, at + k * 8, sdesc_sw128(bs + (k >> 2) * atom + (k & 3) * 32), idesc, s > 0 ? 1u : 0u);
          }
          mma_commit(saddr(&bar->ready[d]));
          if (q + 1 == GPB) mma_commit(saddr(&bar->done[st]));
        }
        __syncwarp();
      }
    }
    // whatever was issued is waited for, with the full bound, on every path
    if (lane == 0) mma_commit(saddr(&bar->drain[me]));
    __syncwarp();
    if (!__all_sync(~0u, mbar_wait(saddr(&bar->drain[me]), 0u, kBound))) ok = failed(5u);
  } else {
    // ---- sums: lane = row `row` of the tile
    const int quarter = warp & 3, row = quarter * 32 + lane, g = row & 7, half = (row >> 3) & 1;
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
    const unsigned char* side = a.w + ((size_t)min(tile0 + (row >> 4), a.ntile - 1) * a.nblk + b0) * a.item + 1024;
    auto scales = [&](__half(&s)[GPB], int i) {
      if (i < n) {
        const __half* p = reinterpret_cast<const __half*>(side + (size_t)i * a.item) + g * (2 * GPB) + half;
#pragma unroll
        for (int q = 0; q < GPB; ++q) s[q] = p[2 * q];
      }
    };
#pragma unroll
    for (int t = 0; t < 64; ++t) acc[t] = 0.f;
    pdl_wait();
    __half s0[GPB], s1[GPB], s2[GPB];
    scales(s0, 0);
    scales(s1, 1);
    for (int i = 0; i < n && ok; ++i) {
      scales(s2, i + 2);
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        const int gi = i * GPB + q, d = gi % kAccs;
        if (ok) ok = wait(bar->ready[d], gi / kAccs, 6u);
        if (!ok) break;
        tc_fence_after();
        const float s = __half2float(s0[q]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c * 16 < N) {
            float v[16];
            tmem_ld16(tl + d * 64 + c * 16, v);
#pragma unroll
            for (int t = 0; t < 16; ++t) acc[c * 16 + t] = fmaf(s, v[t], acc[c * 16 + t]);
          }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(saddr(&bar->taken[d]));
      }
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        s0[q] = s1[q];
        s1[q] = s2[q];
      }
    }
  }
  pdl_wait();                                       // before anything writes y (returns at once if done)
  ok = __syncthreads_and(ok);
  // ---- the sums, or NaN where a wait ran out, over the rings (all copies and products are done)
  float* out = reinterpret_cast<float*>(B);
  if (warp >= kDec + kStage + kIssue) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll
    for (int t = 0; t < 64; ++t)
      if (t < N) out[t * kOutLd + row] = ok ? acc[t] : __int_as_float(0x7fc00000);
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (nsplit > 1) cluster.sync();
  else __syncthreads();
  const int row0 = tile0 * 16, all = a.ntok * kRows;
  const int e0 = (int)((long long)all * rank / nsplit), e1 = (int)((long long)all * (rank + 1) / nsplit);
  for (int e = e0 + threadIdx.x; e < e1; e += kThreads) {
    const int t = e / kRows, r = e % kRows;
    float v;
    if (nsplit == 1) {
      v = out[t * kOutLd + r];
    } else {
      float p[kMaxSplit];
#pragma unroll
      for (int k = 0; k < kMaxSplit; ++k) p[k] = k < nsplit ? cluster.map_shared_rank(out, k)[t * kOutLd + r] : 0.f;
      v = p[0];
#pragma unroll
      for (int k = 1; k < kMaxSplit; ++k) v += p[k];
    }
    if (X8) v *= a.xs[t];
    if (row0 + r < a.R) a.y[(size_t)t * a.R + row0 + r] = __float2half_rn(v);
  }
  if (nsplit > 1) cluster.sync();                   // every CTA's sums stay readable until all are done
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

template <int GPB, bool X8>
int launch_tc(const Int4Args& a, void* stream) {
  TcArgs ta = {};
  ta.a = a;
  ta.N = (a.ntok + 15) / 16 * 16;
  const int work = std::max(kRing * ta.N * 256 + kDec * kRaw * kRawBytes, ta.N * kOutLd * 4);
  const int smem = std::max(kOneCta, 1024 + work + (int)sizeof(Bars));
  if (set_smem(reinterpret_cast<const void*>(k_int4_tc<GPB, X8>), smem)) return Q2_ECUDA;
  const int tiles = (a.ntile + kRows / 16 - 1) / (kRows / 16), sms = dev_info().sms;
  // Waves of CTAs (one per SM) times their blocks plus a fixed cost of about ten.
  ta.nsplit = 1;
  long long best = 0;
  for (int s = 1; s <= kMaxSplit && 2 * s <= a.nblk; ++s) {
    const long long cost = (long long)((tiles * s + sms - 1) / sms) * ((a.nblk + s - 1) / s + 10);
    if (s == 1 || cost < best) {
      best = cost;
      ta.nsplit = s;
    }
  }
  return launch_clusters(k_int4_tc<GPB, X8>, tiles, ta.nsplit, kThreads, smem, stream, ta);
}

}  // namespace
}  // namespace q2

int q2_int4_tc(const q2::Int4Args& a, int group, bool x8, void* stream) {
  using namespace q2;
  switch (Q2_INT4_COLS / group) {
    case 1: return x8 ? launch_tc<1, true>(a, stream) : launch_tc<1, false>(a, stream);
    case 2: return x8 ? launch_tc<2, true>(a, stream) : launch_tc<2, false>(a, stream);
    default: return x8 ? launch_tc<4, true>(a, stream) : launch_tc<4, false>(a, stream);
  }
}

extern "C" int q2_int4_wait_limit(long long polls) {
  return cudaMemcpyToSymbol(q2_int4_stage_wait_limit, &polls, sizeof(polls)) == cudaSuccess ? Q2_OK : Q2_ECUDA;
}

// The error word of these kernels, then cleared (q2_device_errors).
extern "C" int q2_int4_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_int4_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_int4_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
