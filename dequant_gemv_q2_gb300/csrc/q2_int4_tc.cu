// y = W x for 4-bit weights with group scales at many tokens, on the
// 5th-generation tensor cores (tcgen05); the formula, the weights' layout and
// the exact operands q - z are those of q2_int4.cuh.
//
// Tiles of 128 rows (the instruction's M) are shared out over clusters of
// CTAs, and the 128-column blocks of a cluster's tiles evenly over its CTAs,
// one per SM: a CTA runs its run of blocks, across the ends of tiles, through
// rings of stages with four roles:
//   - 8 decoder warps, two per TMEM lane quarter taking blocks in turn, bring
//     their weights to shared memory kRaw - 1 of their blocks ahead (one bulk
//     copy per row tile, scales and zero points with it), unpack them to q - z
//     in fp16 and store them to tensor memory.  The packed order is that of a
//     16 x 16 operand fragment, which is what tcgen05.st's 16x128b shape
//     stores: no exchange.  The scales go to a ring for the summing warps;
//   - x of all tokens comes to shared memory in the 128-byte swizzle: fp16 by
//     TMA, which one warp asks for; 8-bit x through the registers of 8 staging
//     warps, which turn it to fp16;
//   - 2 warps issue the products: one waits for a block and a free accumulator
//     and grants the group at a named barrier, lane 0 of the other issues its
//     M = 128, K = 16 products and commits them.  An issuing thread that
//     touches memory waits for its own queue of products; this one does not;
//   - 8 summing warps, two per lane quarter (half of the tokens each), a row
//     per lane, read each scale group's product from one of kAccs
//     accumulators, multiply it by the group's scale and add it to the row's
//     fp32 sums in registers: group scales cost no rounding, and the
//     accumulator is free for another group.
// A tile that begins and ends inside a CTA's run is written from those
// registers while the next one's products run.  The others' sums meet at the
// end in distributed shared memory, after one barrier of the cluster, and are
// added in column order.
//
// 34816 x 5120 at 64 tokens, groups of 128 with zero points: 36.9 us on the
// device, 2.6 TB/s, 0.61 PFLOP/s (a block of 128 x 128 every 900 cycles of an
// SM).  What bounds it is not one unit: the decoders (about 800 cycles per
// block, their 9 instructions per 8 weights being half of the issue slots
// used), the way of x from L2 (1400 to 1900 cycles from the request to the
// stage, 16 KB of x per 8.8 KB of weights) and the chain block - grant -
// products - free stage (1000, four blocks in it) come to about the same: in
// trials without the unpacking it took 14% less, without the products 10%,
// without x 2%; 12 or 16 decoder warps and deeper rings of weights or x gain
// nothing.  What waits cost shows in the steps: a barrier's address that the
// compiler cannot show to be uniform costs 200 cycles and more at each wait
// (58 -> 42 us at 24576 x 4096 in groups of 32, 39.0 now).  Matrices of few rows
// and many columns also pay for whole tiles: a cluster gets whole tiles and has
// 1, 2, 4 or 8 CTAs, so the longest run of 5120 x 17408 is 51 blocks where an
// even share of its 40 tiles of 136 is 36 (32 tokens 26.5 us, 64 29.3), and that
// of 34816 x 5120 80 of 72.  8-bit x is turned to fp16 by every CTA for every
// tile: 5120 x 17408 in groups of 64 at 32 tokens 36.5 us, at 64 43.2; 34816 x
// 5120 49.5 and 58.3.  That variant with groups of 32 spills 20 bytes.
//
// Every wait is bounded: one that runs out sets the error word
// (q2_device_errors) and a flag on which the other roles give up (the issuing
// warp, which reads no memory, is led to its end by the granting one: its
// products then work on whatever is there).  The products issued are waited
// for before tensor memory is released, and the CTA's rows come out NaN.
#include <cooperative_groups.h>
#include <cuda.h>

#include <algorithm>

#include "q2_int4.cuh"
#include "q2_tcgen.cuh"

namespace cg = cooperative_groups;

__device__ unsigned int q2_int4_error = 0;
__device__ long long q2_int4_stage_wait_limit = 0;           // 0: the normal bound (q2_debug_wait_limit)

namespace q2 {
namespace {

constexpr int kRows = 128, kDec = 8, kIssue = 2, kSum = 8;   // rows; warps of the roles but staging
template <bool X8>
__host__ __device__ constexpr int stage_warps() { return X8 ? 8 : 2; }
template <bool X8>
__host__ __device__ constexpr int tc_threads() { return (kDec + stage_warps<X8>() + kIssue + kSum) * 32; }
constexpr int kTurn = 2;                      // decoder warps of a lane quarter, blocks in turn
constexpr int kRing = 4;                      // blocks in flight: A in tensor memory, x in shared memory
constexpr int kAccs = 4;                      // accumulators of 64 columns
static_assert(kAccs == kRing, "with one group to a block its accumulator's barrier tells of its stage too");
constexpr int kGrants = 8;                    // named barriers of the granting and the issuing warp, more than kAccs
constexpr int kRaw = 3;                       // its blocks of packed weights in shared memory per decoder warp
template <int GPB>
__host__ __device__ constexpr int raw_tile() { return Q2_INT4_BLOCK_BYTES + GPB * 48; }   // a row tile's block with its sides
constexpr uint32_t kTmem = 512, kAcol = 64 * kAccs;
constexpr int kScales = kRing + kAccs;        // blocks of scales in shared memory: a block's products done means that the
                                              // scales kAccs blocks before have been used
constexpr int kStageWarps = 4;                // staging warps of a group (8-bit x)
constexpr int kOutLd = kRows + 4, kMaxCluster = 8;
constexpr int kOneCta = 116 * 1024;           // at most one CTA of this or the other tcgen05 kernels per SM (each holds all of TMEM)

// One product, issued by lane 0 of a converged warp: outside a divergent
// branch the operands stay in uniform registers (inside one each of them was
// moved there again, about 115 cycles per product).
__device__ __forceinline__ void mma_lane0(int lane, uint32_t d, uint32_t at, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "setp.eq.u32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(at), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lane)
      : "memory");
}
__device__ __forceinline__ void commit_lane0(int lane, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.eq.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lane)
      : "memory");
}

// Whether the phase of the given parity is complete (after a short sleep at most).
__device__ __forceinline__ uint32_t try_phase(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done;
}

// `bytes` of global memory to shared memory, reported to the mbarrier.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

struct TcArgs {
  CUtensorMap xmap;                           // fp16 x: box of 64 columns x N tokens, 128-byte swizzle, zeros outside
  Int4Args a;
  int N, cs, ntiles;                          // tokens rounded up to 16; CTAs of a cluster; tiles of 128 rows
};

// 16 rows x 128 columns of operand fragments (eight 16-column steps).
__device__ __forceinline__ void tmem_st_frag(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

struct Bars {
  uint64_t raw[kDec][kRaw];   // a decoder warp's packed weights are there
  uint64_t full[kRing];       // A and x of a block are there (decoder and staging warps)
  uint64_t done[kRing];       // its products are done: the stage is free (commit)
  uint64_t ready[kAccs];      // an accumulator holds a group's product (commit)
  uint64_t taken[kAccs];      // it has been read (summing warps)
  uint64_t drain;             // everything issued is done
  uint32_t tmem;
  int abort, copied;          // a wait ran out; blocks of x requested by TMA
};

template <int GPB, bool X8>
__global__ void __launch_bounds__(tc_threads<X8>(), 1) k_int4_tc(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char q2_int4tc_smem[];
  const Int4Args& a = ta.a;
  constexpr int STEPS = 8 / GPB, kStage = stage_warps<X8>(), TILE = raw_tile<GPB>();
    const int warp = __shfl_sync(~0u, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;   // uniform, and so are the barriers' addresses
  const int N = ta.N, cs = ta.cs, atom = N * 128, bbytes = 2 * atom;
  // this CTA's run: blocks u0 .. u0 + n - 1 of the cluster's T, tile by tile
  const int rank = (int)blockIdx.x % cs, cl = (int)blockIdx.x / cs, ncl = (int)gridDim.x / cs;
  const int t0 = (int)((long long)ta.ntiles * cl / ncl), t1 = (int)((long long)ta.ntiles * (cl + 1) / ncl);
  const int T = (t1 - t0) * a.nblk;
  auto first_of = [&](int r) { return (int)((long long)T * r / cs); };
  const int u0 = first_of(rank), n = first_of(rank + 1) - u0;
  struct Place {
    int tile, blk;
  };
  auto place_of = [&](int u) { return Place{t0 + u / a.nblk, u % a.nblk}; };
  auto move = [&](Place& p, int by) {               // by <= 2 <= nblk; whether it is another tile
    p.blk += by;
    if (p.blk < a.nblk) return false;
    p.blk -= a.nblk;
    ++p.tile;
    return true;
  };
  const uint32_t sB = (saddr(q2_int4tc_smem) + 1023u) & ~1023u;
  unsigned char* B = q2_int4tc_smem + (sB - saddr(q2_int4tc_smem));
  const uint32_t sraw = sB + kRing * bbytes, ssc = sraw + kDec * kRaw * 2 * TILE;
  // the sums of a tile begun before this run, and of one not finished in it
  float* part = reinterpret_cast<float*>(B + kRing * bbytes + kDec * kRaw * 2 * TILE + kScales * kRows * 2 * GPB);   // [2][N][kOutLd]
  Bars* bar = reinterpret_cast<Bars*>(part + 2 * N * kOutLd);
  volatile int* give_up = &bar->abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(saddr(&bar->full[i]), kDec / kTurn + (!X8 ? 1 : N < 8 * kStageWarps ? N / 8 : kStageWarps));
      mbar_init(saddr(&bar->done[i]), 1);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(saddr(&bar->ready[i]), 1);
      mbar_init(saddr(&bar->taken[i]), N > 32 ? kSum : kSum / 2);
    }
    mbar_init(saddr(&bar->drain), 1);
    for (int i = 0; i < kDec * kRaw; ++i) mbar_init(saddr(&bar->raw[0][i]), 1);
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
  int undone = n;                                   // a decoder's next block when it gave up
  auto failed = [&](unsigned int code) {
    if (lane == 0) {
      atomicExch(&q2_int4_error, code);
      *give_up = 1;
    }
    return false;
  };
  // A block's products are done when its last group's are (with several groups
  // to a block an accumulator's barrier may be phases ahead of a stage's).
  auto done = [&](unsigned st) -> uint64_t& { return GPB == 1 ? bar->ready[st] : bar->done[st]; };
  // All lanes poll and leave together: the loop and what it reads stay uniform.
  auto wait = [&](uint64_t& b, unsigned phase, unsigned int code) {
    const uint32_t at = saddr(&b), parity = phase & 1u;
    for (int k = 0; k < (int)kSpinLimit; ++k) {
      if (__all_sync(~0u, try_phase(at, parity))) return true;
      if ((k & 31) == 31 && __any_sync(~0u, *give_up)) break;
    }
    return failed(code);
  };
  float2 acc[16];                                   // 32 tokens

  if (warp < kDec) {
    // ---- decoders: row tiles 2 * quarter, + 1 of every kTurn-th block
    const int quarter = warp & 3, turn = warp >> 2, g = lane >> 2;
    const uint32_t raw = sraw + warp * (kRaw * 2 * TILE);
    Place at = place_of(u0 + turn);                 // of the next block to copy
    const unsigned char* src[2];
    auto point = [&]() {
#pragma unroll
      for (int m = 0; m < 2; ++m)                   // a missing row tile: the last one; its rows are not stored
        src[m] = a.w + ((size_t)min(at.tile * (kRows / 16) + 2 * quarter + m, a.ntile - 1) * a.nblk + at.blk) * a.item;
    };
    point();
    auto copy = [&](int i, int k) {                 // block i to slot k
      if (i < n) {
        if (lane == 0) {
          const uint32_t b = saddr(&bar->raw[warp][k]), d = raw + k * (2 * TILE);
          mbar_expect_tx(b, 2u * a.item);
          bulk_load(d, src[0], a.item, b);
          bulk_load(d + TILE, src[1], a.item, b);
        }
        src[0] += kTurn * a.item;
        src[1] += kTurn * a.item;
        if (move(at, kTurn)) point();
      }
    };
    for (int k = 0; k < kRaw - 1; ++k) copy(turn + k * kTurn, k);
    int k = 0, free = kRaw - 1;                     // slot in use, slot before it
    unsigned turned = 0;                            // phase of the slot in use
    for (unsigned i = turn; i < (unsigned)n; i += kTurn) {
      const unsigned st = i % kRing;
      if (i >= kRing && i < kRing + kTurn) pdl_wait();       // no bounded wait may have to wait for the previous kernel
      ok = wait(bar->raw[warp][k], turned, 7u);
      const uint32_t slot = raw + k * (2 * TILE);
      uint4 w[2][2];
      uint32_t zz[2][GPB];
      auto read = [&](int m) {
        const uint32_t from = slot + m * TILE;
        w[m][0] = lds128(from + lane * 16);
        w[m][1] = lds128(from + 512 + lane * 16);
#pragma unroll
        for (int q = 0; q < GPB; ++q)
          zz[m][q] = a.zeros ? lds16(from + Q2_INT4_BLOCK_BYTES + GPB * 32 + (g * GPB + q) * 2) : 0x0808u;
      };
      read(0);
      if constexpr (!X8) read(1);                   // both at once where registers allow (37.2 -> 34.5 us at 19456 x 10240)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        if (X8 && m == 1) read(1);
        uint32_t A[32];
#pragma unroll
        for (int q = 0; q < GPB; ++q) {
          const Zeros z = zeros_of(zz[m][q]);
#pragma unroll
          for (int t = q * STEPS; t < (q + 1) * STEPS; ++t)
            unpack_step(word(w[m][t >> 2], t & 3), z, A[4 * t], A[4 * t + 1], A[4 * t + 2], A[4 * t + 3]);
        }
        if (m == 0) {
          if (ok && i >= kRing) ok = wait(done(st), i / kRing - 1, 1u);
          if (!ok) break;
          tc_fence_after();
          // the scales of both row tiles, as they are, for the summing warps
          if (lane < 4 * GPB) {
            const int e = lane % (2 * GPB), mm = lane / (2 * GPB);
            const uint4 v = lds128(slot + mm * TILE + Q2_INT4_BLOCK_BYTES + e * 16);
            sts128(ssc + (i % kScales) * (kRows * 2 * GPB) + (2 * quarter + mm) * (32 * GPB) + e * 16, v);
          }
        }
        tmem_st_frag(tmem + ((uint32_t)(quarter * 32 + m * 16) << 16) + kAcol + st * 64, A);
      }
      if (!ok) {
        undone = i;
        break;
      }
      copy(i + (kRaw - 1) * kTurn, free);           // while the stores are on their way
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(saddr(&bar->full[st]));
      free = k;
      k = k + 1 == kRaw ? 0 : k + 1;
      turned ^= k == 0;
    }
    // no copy may land after the CTA has gone: those asked for when this warp gave up
    if (!ok)
      for (int i = undone, e = 0; e < kRaw - 1 && i < n; i += kTurn, ++e) {
        (void)mbar_wait(saddr(&bar->raw[warp][k]), turned);
        k = k + 1 == kRaw ? 0 : k + 1;
        turned ^= k == 0;
      }
  } else if (warp < kDec + kStage) {
    // ---- x of all tokens: copied as it is by TMA (fp16), or turned to fp16 on the way
    pdl_wait();                                     // x may come from the previous kernel
    if constexpr (!X8) {
      if (warp == kDec) {
        Place at = place_of(u0);
        int copied = 0;
        for (unsigned i = 0; i < (unsigned)n; ++i) {
          const unsigned st = i % kRing;
          if (i >= kRing) ok = wait(done(st), i / kRing - 1, 2u) && !__any_sync(~0u, *give_up);   // (done is also told of products given up)
          if (!ok) break;
          if (lane == 0) {
            const uint32_t full = saddr(&bar->full[st]), d = sB + st * bbytes;
            mbar_expect_tx(full, (uint32_t)bbytes);
            tma_load_2d(d, &ta.xmap, at.blk * 128, 0, full);
            tma_load_2d(d + atom, &ta.xmap, at.blk * 128 + 64, 0, full);
          }
          __syncwarp();
          copied = i + 1;
          move(at, 1);
        }
        if (lane == 0) bar->copied = copied;
      }
    } else {
      // two groups of warps, blocks in turn; task (token t, run q of 32
      // columns): 32 bytes in, four 16-byte pieces out
      const int group = (warp - kDec) / kStageWarps, tid = threadIdx.x - (kDec + group * kStageWarps) * 32;
      constexpr int TASKS = 256 / (kStageWarps * 32);
      if (tid / 32 < N / 8) {                       // a warp for 32 of the 4 * N tasks
        const unsigned char* row[TASKS];
        unsigned char* to[TASKS];
        int key[TASKS], last[TASKS];                // blocks in which the token has this run
#pragma unroll
        for (int k = 0; k < TASKS; ++k) {
          const int e = tid + k * (kStageWarps * 32), t = e % N, q = e / N;
          const bool live = q < 4 && t < a.ntok;
          row[k] = static_cast<const unsigned char*>(a.x) + (size_t)(live ? t : 0) * a.C + q * 32;
          to[k] = B + (q >> 1) * atom + t * 128;
          key[k] = (4 * (q & 1)) ^ (t & 7);
          last[k] = live ? (a.C - q * 32 + 127) / 128 : 0;
        }
        const bool second = TASKS > 1 && tid + kStageWarps * 32 < 4 * N;
        uint4 v[TASKS][2];
        Place at = place_of(u0 + group);            // of the next block to load
        auto load = [&](int i) {
          if (i < n) {
#pragma unroll
            for (int k = 0; k < TASKS; ++k) {
              const uint4* from = reinterpret_cast<const uint4*>(row[k] + at.blk * 128);
#pragma unroll
              for (int p = 0; p < 2; ++p) v[k][p] = at.blk < last[k] ? from[p] : make_uint4(0, 0, 0, 0);
            }
            move(at, 2);
          }
        };
        load(group);
        for (unsigned i = group; i < (unsigned)n; i += 2) {
          const unsigned st = i % kRing;
          if (i >= kRing) ok = wait(done(st), i / kRing - 1, 2u);
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < TASKS; ++k) {
            if (k == 0 || second) {
              unsigned char* d = to[k] + st * bbytes;
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                uint4 o;
                int8x4(word(v[k][p >> 1], 2 * (p & 1)), o.x, o.y);
                int8x4(word(v[k][p >> 1], 2 * (p & 1) + 1), o.z, o.w);
                *reinterpret_cast<uint4*>(d + ((key[k] ^ p) << 4)) = o;
              }
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(saddr(&bar->full[st]));
          load(i + 2);
        }
      }
    }
  } else if (warp < kDec + kStage + kIssue) {
    // ---- products: a granting and an issuing warp, which meet at named barriers
    pdl_wait();
    if (warp == kDec + kStage) {
      const long long limit = q2_int4_stage_wait_limit;       // in plain polls, which do not sleep
      for (unsigned i = 0; i < (unsigned)n; ++i) {
        const unsigned st = i % kRing;
        if (ok && limit > 0 && !__all_sync(~0u, mbar_wait(saddr(&bar->full[st]), (uint32_t)(i / kRing) & 1u, limit)))
          ok = failed(3u);
        if (ok) ok = wait(bar->full[st], i / kRing, 3u);
#pragma unroll
        for (int q = 0; q < GPB; ++q) {
          const unsigned gi = i * GPB + q, d = gi % kAccs;
          if (ok && gi >= kAccs) ok = wait(bar->taken[d], gi / kAccs - 1, 4u);
          tc_fence_after();
          tc_fence_before();
          if (ok) asm volatile("bar.arrive %0, 64;" ::"r"(1 + gi % kGrants) : "memory");
          else asm volatile("bar.sync %0, 64;" ::"r"(1 + gi % kGrants) : "memory");
        }
      }
    } else {
      const uint32_t idesc = idesc_f16(kRows, N);
      for (unsigned i = 0; i < (unsigned)n; ++i) {
        const unsigned st = i % kRing;
        const uint64_t lo = sdesc_sw128(sB + st * bbytes), hi = sdesc_sw128(sB + st * bbytes + atom);
#pragma unroll
        for (int q = 0; q < GPB; ++q) {
          const unsigned gi = i * GPB + q, d = gi % kAccs;
          asm volatile("bar.sync %0, 64;" ::"r"(1 + gi % kGrants) : "memory");
          tc_fence_after();
          const uint32_t at = tmem + kAcol + st * 64 + q * (STEPS * 8), acc0 = tmem + d * 64;
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int k = q * STEPS + s;
            mma_lane0(lane, acc0, at + s * 8, (k < 4 ? lo : hi) + (k & 3) * 2, idesc, s > 0 ? 1u : 0u);
          }
          commit_lane0(lane, saddr(&bar->ready[d]));
          if (GPB > 1 && q + 1 == GPB) commit_lane0(lane, saddr(&bar->done[st]));
        }
      }
      // whatever was issued is waited for, on every path
      if (lane == 0) mma_commit(saddr(&bar->drain));
      __syncwarp();
      if (!__all_sync(~0u, mbar_wait(saddr(&bar->drain), 0u))) ok = failed(5u);
    }
  } else {
    // ---- sums: lane = row `row` of the tile, tokens c0 .. c0 + 31
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const int c0 = (warp - kDec - kStage - kIssue) / 4 * 32;
    if (c0 < N) {
    const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16) + c0;
    const uint32_t sc = ssc + (row >> 4) * (32 * GPB) + (row & 7) * (GPB * 4) + ((row >> 3) & 1) * 2;   // this row's scales
    Place now = place_of(u0);
#pragma unroll
    for (int t = 0; t < 16; ++t) acc[t] = make_float2(0.f, 0.f);
    pdl_wait();
    bool begun = now.blk == 0;                      // the tile in use began in this run
    for (unsigned i = 0; i < (unsigned)n; ++i) {
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        const unsigned gi = i * GPB + q, d = gi % kAccs;
        if (ok) ok = wait(bar->ready[d], gi / kAccs, 6u);
        if (ok) {
          tc_fence_after();
          const float s1 = __half2float(__ushort_as_half((unsigned short)lds16(sc + (i % kScales) * (kRows * 2 * GPB) + q * 4)));
          const float2 s2 = make_float2(s1, s1);
#pragma unroll
          for (int h = 0; h < 2; ++h) {             // (past N: whatever is there)
            float v[16];
            tmem_ld16(tl + d * 64 + 16 * h, v);
#pragma unroll
            for (int t = 0; t < 8; ++t) fma2(acc[8 * h + t], s2, make_float2(v[2 * t], v[2 * t + 1]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(saddr(&bar->taken[d]));
        }
      }
      const bool ends = now.blk + 1 == a.nblk;
      if (ends || i + 1 == (unsigned)n) {                     // a tile's end, or the run's; NaN where a wait ran out
        if (__any_sync(~0u, *give_up)) ok = false;
        const int r = now.tile * kRows + row;
        float* o = part + (begun ? N * kOutLd : 0) + c0 * kOutLd + row;
#pragma unroll
        for (int t = 0; t < 32; ++t) {
          const float v = ok ? (t & 1 ? acc[t >> 1].y : acc[t >> 1].x) : __int_as_float(0x7fc00000);
          if (!(ends && begun)) {
            if (c0 + t < N) o[t * kOutLd] = v;
          } else if (r < a.R && c0 + t < a.ntok) {
            a.y[(size_t)(c0 + t) * a.R + r] = __float2half_rn(X8 ? v * a.xs[c0 + t] : v);
          }
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) acc[t] = make_float2(0.f, 0.f);
        begun = true;
      }
      move(now, 1);
    }
    }
  }
  // no copy may land after the CTA has gone: on an error the decoders make up
  // for the arrivals that they left out, and the copies under way are waited for
  if (__syncthreads_or(!ok) && !X8 && warp <= kDec) {
    const int copied = bar->copied;
    if (warp < kDec) {
      if (lane == 0)
        for (int i = undone; i < copied; i += kTurn) mbar_arrive(saddr(&bar->full[i % kRing]));
    } else {
      for (int i = copied - kRing > 0 ? copied - kRing : 0; i < copied; ++i)
        (void)mbar_wait(saddr(&bar->full[i % kRing]), (uint32_t)(i / kRing) & 1u);
    }
  }
  pdl_wait();                                       // before anything writes y (returns at once if done)
  cg::cluster_group cluster = cg::this_cluster();
  if (cs > 1) {
    cluster_meet();
    // The tile that this run begins in the middle of, and the one it leaves
    // unfinished: this CTA's share of the rows of each.  The sums of all CTAs
    // are added up in the ring, which is free now, and stored when this CTA
    // has said that it has read them.
    const int head = u0 / a.nblk, tail = (u0 + n - 1) / a.nblk;
    auto each = [&](auto use) {
#pragma unroll 1
      for (int k = 0; k < 2; ++k) {
        const int tile = k ? tail : head, s = tile * a.nblk, e = s + a.nblk;
        const bool open = k ? tail != head && e > u0 + n : s < u0 || e > u0 + n;
        if (!open) continue;
        auto rank_of = [&](int u) { return (int)((((long long)u + 1) * cs - 1) / T); };
        const int r0 = rank_of(s), cnt = rank_of(e - 1) - r0 + 1, all = a.ntok * kRows;   // cnt >= 2
        const int e0 = all * (rank - r0) / cnt, e1 = all * (rank - r0 + 1) / cnt;
        float* sum = reinterpret_cast<float*>(B) + k * (N * kRows / 2);
        for (int x = e0 + threadIdx.x; x < e1; x += blockDim.x)
          use(sum[x - e0], r0, cnt, x / kRows, x % kRows, (t0 + tile) * kRows + x % kRows);
      }
    };
    each([&](float& sum, int r0, int cnt, int t, int r, int) {
      float p[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c)         // the first CTA has the tile as its last, the others as their first
        p[c] = c < cnt ? cluster.map_shared_rank(part, r0 + c)[(c ? 0 : N * kOutLd) + t * kOutLd + r] : 0.f;
      float v = p[0];
#pragma unroll
      for (int c = 1; c < kMaxCluster; ++c) v += p[c];
      sum = v;
    });
    cluster_arrive();                               // this CTA has read the others' sums
    each([&](float& sum, int, int, int t, int, int row) {
      if (row < a.R) a.y[(size_t)t * a.R + row] = __float2half_rn(X8 ? sum * a.xs[t] : sum);
    });
    cluster_wait();                                 // and they this one's
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmem) : "memory");
}

template <int GPB, bool X8>
int launch_tc(const Int4Args& a, void* stream) {
  static ClusterCounts counts;
  auto kernel = k_int4_tc<GPB, X8>;
  const void* fn = reinterpret_cast<const void*>(kernel);
  TcArgs ta = {};
  ta.a = a;
  ta.N = (a.ntok + 15) / 16 * 16;
  ta.ntiles = (a.ntile + kRows / 16 - 1) / (kRows / 16);
  const int work = kRing * ta.N * 256 + kDec * kRaw * 2 * raw_tile<GPB>() + kScales * kRows * 2 * GPB + 2 * ta.N * kOutLd * 4;
  const int smem = std::max(kOneCta, 1024 + work + (int)sizeof(Bars));
  if (set_smem(fn, smem)) return Q2_ECUDA;
  // The cluster size with the shortest run of blocks, each doubling of it
  // counted as three blocks (its barriers and the meeting of its sums).
  int clusters = 1;
  double best = 0;
  for (int cs = 1, lg = 0; cs <= kMaxCluster && cs <= a.nblk; cs *= 2, ++lg) {
    const int n = std::min(ta.ntiles, cs == 1 ? dev_info().sms : counts.get(fn, cs, tc_threads<X8>(), smem));
    const double cost = (double)((ta.ntiles + n - 1) / n) * a.nblk / cs + 3 * lg;
    if (cs == 1 || cost < best) {
      best = cost;
      ta.cs = cs;
      clusters = n;
    }
  }
  if (!X8 && !encode_x_map(&ta.xmap, a.x, a.C, a.ntok, ta.N)) return Q2_ECUDA;
  return launch_clusters(kernel, clusters, ta.cs, tc_threads<X8>(), smem, stream, ta);
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
