// y = W x for 4-bit weights with group scales, 1..64 tokens,
//
//   y[t][r] = sum_g s[r][g] * sum_{c in g} (q[r][c] - z[r][g]) * x[t][c],
//
// for x in fp16, or in 8 bits with one fp32 scale per token.
//
// The inner sums run on the tensor cores, 16 rows x 16 columns of weights
// against 8 tokens per instruction, fp32 accumulators.  q - z is a small
// integer and exact in fp16: four bits OR-ed into the mantissa of 1024 (or,
// shifted left by four, of 64 after a multiplication by 1/16) give 1024 + q
// (64 + q) without a conversion, and one subtraction (one fused
// multiply-add) takes 1024 + z (64 + z) off again, so 8 weights cost 9
// instructions.  The group's fp32 sum is multiplied by the scale and added to
// the row's fp32 sum: nothing but y itself is rounded to fp16.  For 8-bit x
// the group sums are sums of at most 128 products of magnitude at most
// 15 * 128 each and thus exact.
//
// Weights are stored in the order in which lanes use them: the unit is a
// block of 16 rows x 128 columns, 1 KB, as two 16-byte loads per lane.  The
// columns that a lane holds are its own choice of the contraction's order
// (any bijection is right as long as x uses it too, and as long as a step
// stays inside a scale group); it is the one that makes a lane's share of x in
// 32 columns of a token, 8 consecutive ones, contiguous.
//
// Weights are never staged through shared memory: every weight is used by one
// warp only.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <mutex>
#include <utility>
#include <vector>

#include "q2_common.cuh"

namespace cg = cooperative_groups;

namespace q2 {
namespace {

struct Int4Args {
  const unsigned char* w;     // [ntile][nblk][2][32 lanes][16 bytes]
  const unsigned char* s;     // [ntile][nblk][8][groups per block][2] fp16: rows g and g + 8
  const unsigned char* z;     // the same order, one byte each; null: 8 everywhere
  const void* x;              // [ntok][C] fp16 or int8
  const float* xs;            // [ntok], 8-bit x only
  __half* y;                  // [ntok][R]
  int R, C, nblk, ntile, ntok;
};

// One block (16 rows x 128 columns) as a lane holds it before use.
template <int GPB>            // groups per block: 1, 2 or 4
struct Block {
  uint4 w[2];
  uint32_t s[GPB];
  uint32_t z[(GPB + 1) / 2];
};

template <int GPB>
__device__ __forceinline__ void load_block(Block<GPB>& k, const Int4Args& a, size_t blk, int lane) {
  const unsigned char* w = a.w + blk * Q2_INT4_BLOCK_BYTES + lane * 16;
  k.w[0] = ldg_stream(w);
  k.w[1] = ldg_stream(w + 512);
  const unsigned char* s = a.s + (blk * 8 + (lane >> 2)) * (GPB * 4);
  const unsigned char* z = a.z + (blk * 8 + (lane >> 2)) * (GPB * 2);
  if (GPB == 1) {
    k.s[0] = __ldg(reinterpret_cast<const unsigned int*>(s));
    k.z[0] = a.z ? __ldg(reinterpret_cast<const unsigned short*>(z)) : 0x0808u;
  } else if (GPB == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
    k.s[0] = v.x;
    k.s[GPB - 1] = v.y;
    k.z[0] = a.z ? __ldg(reinterpret_cast<const unsigned int*>(z)) : 0x08080808u;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
    k.s[0] = v.x;
    k.s[1 % GPB] = v.y;
    k.s[2 % GPB] = v.z;
    k.s[3 % GPB] = v.w;
    const uint2 u = a.z ? __ldg(reinterpret_cast<const uint2*>(z)) : make_uint2(0x08080808u, 0x08080808u);
    k.z[0] = u.x;
    k.z[(GPB + 1) / 2 - 1] = u.y;
  }
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) { return (v & mask) | bits; }

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// The block's q - z as the A operands of its eight 16-column steps: rows g
// (a0, a2) and g + 8 (a1, a3) of lane group g = lane / 4.  A word holds, from
// its lowest four bits up, columns 0, 0, 2, 2, 1, 1, 3, 3 of the step's four,
// rows g and g + 8 in turn.
template <int GPB>
__device__ __forceinline__ void unpack(const Block<GPB>& k, uint32_t (&A)[8][4]) {
#pragma unroll
  for (int q = 0; q < GPB; ++q) {
    const uint32_t zz = k.z[q >> 1] >> (16 * (q & 1));
    const uint32_t z0 = and_or(zz, 0xffu, 0x6400u) * 0x10001u;                  // 1024 + z of row g
    const uint32_t z1 = and_or(zz >> 4, 0xff0u, 0xd400u) * 0x10001u;            // -(64 + z) of row g + 8
#pragma unroll
    for (int t = 0; t < 8 / GPB; ++t) {
      const int st = q * (8 / GPB) + t;
      const uint32_t v = word(k.w[st >> 2], st & 3), v8 = v >> 8;
      A[st][0] = hsub2(and_or(v, 0x000f000fu, 0x64006400u), z0);
      A[st][1] = hfma2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z1);
      A[st][2] = hsub2(and_or(v8, 0x000f000fu, 0x64006400u), z0);
      A[st][3] = hfma2(and_or(v8, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z1);
    }
  }
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// acc += s_g * (the group's products), over the block's groups.
template <int GPB>
__device__ __forceinline__ void products(const uint32_t (&A)[8][4], const uint32_t (&s)[GPB], const uint32_t (&b)[16],
                                         float (&acc)[4]) {
#pragma unroll
  for (int q = 0; q < GPB; ++q) {
    float g[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int t = 0; t < 8 / GPB; ++t) {
      const int st = q * (8 / GPB) + t;
      mma(g, A[st], b[2 * st], b[2 * st + 1]);
    }
    const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&s[q]));
    acc[0] = fmaf(sc.x, g[0], acc[0]);
    acc[1] = fmaf(sc.x, g[1], acc[1]);
    acc[2] = fmaf(sc.y, g[2], acc[2]);
    acc[3] = fmaf(sc.y, g[3], acc[3]);
  }
}

// Four 8-bit integers as two pairs of fp16: the byte plus 128 in the mantissa
// of 1024, minus 1152.
__device__ __forceinline__ void int8x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  v ^= 0x80808080u;
  lo = hsub2(__byte_perm(v, 0x64646464u, 0x4140), 0x64806480u);
  hi = hsub2(__byte_perm(v, 0x64646464u, 0x4342), 0x64806480u);
}

// The B operands of one block for one token: 8 consecutive columns in each of
// the block's four runs of 32, 16 bytes of fp16 or 8 bytes of 8-bit integers.
template <bool X8, typename L>
__device__ __forceinline__ void load_b(uint32_t (&b)[16], L&& load) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto v = load(k);
    if constexpr (X8) {
      int8x4(v.x, b[4 * k], b[4 * k + 1]);
      int8x4(v.y, b[4 * k + 2], b[4 * k + 3]);
    } else {
      b[4 * k] = v.x;
      b[4 * k + 1] = v.y;
      b[4 * k + 2] = v.z;
      b[4 * k + 3] = v.w;
    }
  }
}

template <bool X8>
struct XVec {
  using T = uint4;
};
template <>
struct XVec<true> {
  using T = uint2;
};

// ------------------------------------------------------- up to 8 tokens
// A CTA's warps split the columns of MT row tiles (16 rows each) and keep
// their column range over all row tiles that the CTA takes (every gridDim.x-th), so
// the weight stream of a warp never stops: DEPTH blocks are in flight across
// the ends of row tiles, the first of them requested before the wait on the
// previous kernel.  x goes straight from L1 to registers.  At a row tile's
// end the warps leave their sums in one of two shared-memory buffers and the
// first threads add them in warp order: one barrier per row tile, no atomics.
constexpr int kFewWarps = 8;

template <int MT, int GPB, int DEPTH, bool X8>
__global__ void __launch_bounds__(kFewWarps * 32, 2) k_int4_few(const __grid_constant__ Int4Args a) {
  constexpr int LD = 16 * MT + 4;                           // floats per token in a buffer: conflict-free writes
  __shared__ float red[2][kFewWarps][8 * LD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int b0 = a.nblk * warp / nwarp, nb = a.nblk * (warp + 1) / nwarp - b0;   // nwarp <= nblk: nb >= 1
  const int nunit = (a.ntile + MT - 1) / MT;                // row tiles in bundles of MT
  const int mine = (nunit - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const int n = mine * nb;                                  // blocks of this warp's stream

  Block<GPB> ring[DEPTH][MT];
  // the next block to load: bundle lu (0..mine-1), column block lb
  int lu = 0, lb = 0;
  auto fetch = [&](Block<GPB>(&k)[MT]) {
    if (lu < mine) {
      const int unit = (int)blockIdx.x + lu * (int)gridDim.x;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int tile = min(unit * MT + m, a.ntile - 1);   // a missing tile repeats the last; its rows are not stored
        load_block(k[m], a, (size_t)tile * a.nblk + b0 + lb, lane);
      }
      if (++lb == nb) {
        lb = 0;
        ++lu;
      }
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(ring[d]);

  pdl_wait();                                               // x may come from the previous kernel
  pdl_trigger();
  const int esz = X8 ? 1 : 2;
  const bool live = g < a.ntok;
  const unsigned char* xt = static_cast<const unsigned char*>(a.x) + (size_t)(live ? g : 0) * a.C * esz;
  const int col0 = b0 * 128 + j * 8;                        // this lane's columns: +0..7 of each run of 32
  const float xsc0 = X8 && 2 * j < a.ntok ? a.xs[2 * j] : 1.f, xsc1 = X8 && 2 * j + 1 < a.ntok ? a.xs[2 * j + 1] : 1.f;

  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
  int cb = 0, cu = 0;                                       // block and bundle being used
  for (int i = 0; i < n; i += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (i + d < n) {
        uint32_t b[16];
        const int c = col0 + cb * 128;
        load_b<X8>(b, [&](int k) {
          using V = typename XVec<X8>::T;
          const int cc = c + k * 32;
          return live && cc < a.C ? *reinterpret_cast<const V*>(xt + (size_t)cc * esz) : V{};
        });
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t A[8][4];
          unpack(ring[d][m], A);
          products(A, ring[d][m].s, b, acc[m]);
        }
        fetch(ring[d]);
        if (++cb == nb) {                                   // the bundle's end
          float* r = red[cu & 1][warp];
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            r[(2 * j) * LD + 16 * m + g] = acc[m][0] * xsc0;
            r[(2 * j + 1) * LD + 16 * m + g] = acc[m][1] * xsc1;
            r[(2 * j) * LD + 16 * m + g + 8] = acc[m][2] * xsc0;
            r[(2 * j + 1) * LD + 16 * m + g + 8] = acc[m][3] * xsc1;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[m][q] = 0.f;
          }
          __syncthreads();
          const int row0 = ((int)blockIdx.x + cu * (int)gridDim.x) * MT * 16;
          for (int e = threadIdx.x; e < a.ntok * MT * 16; e += blockDim.x) {
            const int t = e / (MT * 16), rr = e % (MT * 16);
            float v = 0.f;
            for (int w = 0; w < nwarp; ++w) v += red[cu & 1][w][t * LD + rr];
            if (row0 + rr < a.R) a.y[(size_t)t * a.R + row0 + rr] = __float2half_rn(v);
          }
          cb = 0;
          ++cu;
        }
      }
    }
  }
}

// ------------------------------------------------------- 9..64 tokens
// A CTA takes 128 rows and a range of 256-column stages.  Its eight warps are
// four pairs of row tiles times the two 128-column blocks of a stage.  x of
// all tokens comes through a ring of shared-memory stages by asynchronous
// 16-byte copies (a token's row is padded so that the lanes that load
// together fall on different banks); weights go from memory to registers,
// DEPTH blocks ahead.  A block's A operands are unpacked once and used for
// all tokens.  When the column range is split over CTAs, they form a cluster
// and add their fp32 sums through distributed shared memory in rank order.
constexpr int kManyWarps = 8, kManyRows = 128, kManyStages = 3;

template <bool X8>
__host__ __device__ constexpr int x_row_bytes() { return X8 ? 256 + 32 : 512 + 64; }

constexpr int kOutLd = kManyRows + 4;

template <int NT, bool X8>
constexpr int many_smem() {
  const int ring = kManyStages * NT * 8 * x_row_bytes<X8>(), out = NT * 8 * kOutLd * 4;
  return ring > out ? ring : out;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

template <int NT, int GPB, bool X8>
__global__ void __launch_bounds__(kManyWarps * 32, 1) k_int4_many(const __grid_constant__ Int4Args a,
                                                                              const int nsplit) {
  constexpr int DEPTH = NT <= 4 ? 3 : 2, MT = 2, NTOK = NT * 8, ROWB = x_row_bytes<X8>();
  constexpr int esz = X8 ? 1 : 2, PIECES = 256 * esz / 16;
  extern __shared__ __align__(16) unsigned char q2_int4_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3, wm = warp & 3, wk = warp >> 2;
  const int rank = (int)blockIdx.x % nsplit, tile0 = (int)blockIdx.x / nsplit * (kManyRows / 16) + wm * MT;
  const int nstage = (a.nblk + 1) / 2;
  const int s0 = nstage * rank / nsplit, n = nstage * (rank + 1) / nsplit - s0;   // stages of this CTA

  Block<GPB> ring[DEPTH][MT];
  auto fetch = [&](Block<GPB>(&k)[MT], int i) {
    const int blk = min(2 * (s0 + i) + wk, a.nblk - 1);     // past the last block: any block, its x is zero
    if (i < n) {
#pragma unroll
      for (int m = 0; m < MT; ++m) load_block(k[m], a, (size_t)min(tile0 + m, a.ntile - 1) * a.nblk + blk, lane);
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(ring[d], d);

  pdl_wait();
  pdl_trigger();
  const uint32_t sx = saddr(q2_int4_smem);
  auto stage = [&](int i) {
    if (i < n) {
      const uint32_t base = sx + (i % kManyStages) * (NTOK * ROWB);
      for (int e = threadIdx.x; e < NTOK * PIECES; e += kManyWarps * 32) {
        const int t = e / PIECES, p = e % PIECES;
        const int c = (s0 + i) * 256 + p * (16 / esz);
        const bool live = t < a.ntok && c < a.C;
        cp16(base + t * ROWB + p * 16,
             static_cast<const unsigned char*>(a.x) + (live ? ((size_t)t * a.C + c) * esz : 0), live);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < kManyStages - 1; ++d) stage(d);

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.f;

  for (int i0 = 0; i0 < n; i0 += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int i = i0 + d;
      if (i < n) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kManyStages - 2) : "memory");
        __syncthreads();                                    // stage i has arrived for all, stage i - 1 is free
        stage(i + kManyStages - 1);
        uint32_t A[MT][8][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) unpack(ring[d][m], A[m]);
        const uint32_t xb = sx + (i % kManyStages) * (NTOK * ROWB) + g * ROWB + wk * (128 * esz) + j * (8 * esz);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t b[16];
          load_b<X8>(b, [&](int k) {
            const uint32_t at = xb + t * 8 * ROWB + k * (32 * esz);
            typename XVec<X8>::T v;
            if constexpr (X8)
              asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
            else
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
            return v;
          });
#pragma unroll
          for (int m = 0; m < MT; ++m) products(A[m], ring[d][m].s, b, acc[m][t]);
        }
        fetch(ring[d], i + DEPTH);
      }
    }
  }
  // the second block's warps add to the first block's, in shared memory
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* out = reinterpret_cast<float*>(q2_int4_smem);
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (wk == half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float* o = out + (t * 8 + 2 * j + (q & 1)) * kOutLd + wm * 32 + m * 16 + g + (q >> 1) * 8;
            *o = half ? acc[m][t][q] : *o + acc[m][t][q];
          }
    }
    __syncthreads();
  }
  cg::cluster_group cluster = cg::this_cluster();
  if (nsplit > 1) cluster.sync();
  const int row0 = (int)blockIdx.x / nsplit * kManyRows;
  const int all = a.ntok * kManyRows, e0 = all * rank / nsplit, e1 = all * (rank + 1) / nsplit;
  const float* peer[8];
  for (int k = 0; k < 8; ++k) peer[k] = k < nsplit && nsplit > 1 ? cluster.map_shared_rank(out, k) : out;
  for (int e = e0 + threadIdx.x; e < e1; e += kManyWarps * 32) {
    const int t = e / kManyRows, r = e % kManyRows;
    float p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = k < nsplit ? peer[k][t * kOutLd + r] : 0.f;
    float v = p[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += p[k];
    if (X8) v *= a.xs[t];
    if (row0 + r < a.R) a.y[(size_t)t * a.R + row0 + r] = __float2half_rn(v);
  }
  if (nsplit > 1) cluster.sync();                           // every CTA's sums stay readable until all are done
}

// ------------------------------------------------------- launch
template <int MT, int GPB, bool X8>
int launch_few(const Int4Args& a, void* stream) {
  constexpr int DEPTH = 4 / MT;
  const int nwarp = a.nblk < kFewWarps ? a.nblk : kFewWarps;
  const int nunit = (a.ntile + MT - 1) / MT, most = 2 * dev_info().sms;
  return launch_pdl(k_int4_few<MT, GPB, DEPTH, X8>, a, nunit < most ? nunit : most, nwarp * 32, 0, stream);
}

template <int NT, int GPB, bool X8>
int launch_many(const Int4Args& a, void* stream) {
  auto kernel = k_int4_many<NT, GPB, X8>;
  constexpr int smem = many_smem<NT, X8>();
  if (set_smem(reinterpret_cast<const void*>(kernel), smem)) return Q2_ECUDA;
  const int tiles = (a.ntile + kManyRows / 16 - 1) / (kManyRows / 16), nstage = (a.nblk + 1) / 2;
  const int slots = dev_info().sms;
  // Waves of CTAs times their stages plus a fixed cost of about six stages.
  int nsplit = 1;
  double best = 0;
  for (int s = 1; s <= 8 && s <= nstage; s *= 2) {
    const double cost = (double)((tiles * s + slots - 1) / slots) * ((nstage + s - 1) / s + 6);
    if (s == 1 || cost < best) {
      best = cost;
      nsplit = s;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * nsplit);
  cfg.blockDim = dim3(kManyWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nsplit;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, a, nsplit) != cudaSuccess) {
    (void)cudaGetLastError();
    return Q2_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? Q2_OK : Q2_ECUDA;
}

template <int GPB, bool X8>
int launch_tokens(const Int4Args& a, void* stream) {
  if (a.ntok <= 2) return launch_few<1, GPB, X8>(a, stream);
  if (a.ntok <= 8) return launch_few<2, GPB, X8>(a, stream);
  if (a.ntok <= 16) return launch_many<2, GPB, X8>(a, stream);
  if (a.ntok <= 32) return launch_many<4, GPB, X8>(a, stream);
  return launch_many<8, GPB, X8>(a, stream);
}

template <bool X8>
int launch_int4(const q2_handle* h, const void* x, const float* xs, void* y, int ntok, void* stream) {
  const q2_blob_header& d = h->hdr;
  Int4Args a = {};
  a.w = h->dev + d.off[SEC_INT4_W];
  a.s = h->dev + d.off[SEC_INT4_SCALE];
  a.z = d.len[SEC_INT4_ZERO] ? h->dev + d.off[SEC_INT4_ZERO] : nullptr;
  a.x = x;
  a.xs = xs;
  a.y = static_cast<__half*>(y);
  a.R = d.R;
  a.C = d.C;
  a.nblk = d.nblock;
  a.ntile = (d.R + 15) / 16;
  a.ntok = ntok;
  switch (Q2_INT4_COLS / d.reserved) {
    case 1: return launch_tokens<1, X8>(a, stream);
    case 2: return launch_tokens<2, X8>(a, stream);
    default: return launch_tokens<4, X8>(a, stream);
  }
}

}  // namespace
}  // namespace q2

// Later products' weights are not fetched into L2 from here (q2_gemv_chain's
// lookahead): pf is not used.
extern "C" int q2_launch_int4(const q2_handle* h, const void* x, void* y, int ntok, void* stream, const q2_pf*) {
  return q2::launch_int4<false>(h, x, nullptr, y, ntok, stream);
}

extern "C" int q2_launch_int4_x8(const q2_handle* h, const void* x8, const float* xscale, void* y, int ntok,
                                 void* stream) {
  return q2::launch_int4<true>(h, x8, xscale, y, ntok, stream);
}
