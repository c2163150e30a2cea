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
// block of 16 rows x 128 columns, 1 KB as two 16-byte loads per lane, with
// its scales and zero points behind it, so that a warp reads one stream.  The
// columns that a lane holds are its own choice of the contraction's order
// (any bijection is right as long as x uses it too, and as long as a step
// stays inside a scale group); it is the one that makes a lane's share of x in
// 32 columns of a token, 8 consecutive ones, contiguous.
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
  const unsigned char* w;     // [ntile][nblk] blocks of `item` bytes: weights, scales, zero points
  const void* x;              // [ntok][C] fp16 or int8
  const float* xs;            // [ntok], 8-bit x only
  __half* y;                  // [ntok][R]
  int R, C, nblk, ntile, ntok, item;
  int zeros;                  // blocks hold zero points; else 8 everywhere
};

// The scales (rows g and g + 8) and zero points of a lane's rows in one block.
template <int GPB>            // groups per block: 1, 2 or 4
struct Sides {
  uint32_t s[GPB];
  uint32_t z[(GPB + 1) / 2];
};

// Blocks go to shared memory by asynchronous 16-byte copies (a register ring
// was bound by the six scoreboards a warp has: waiting for x meant waiting
// for weights requested after it; 19.1 us instead of 10.3 at 24576 x 4096).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void copy_block(uint32_t dst, const unsigned char* src, int item, int lane) {
  cp16(dst + lane * 16, src + lane * 16);
  cp16(dst + 512 + lane * 16, src + 512 + lane * 16);
  if (lane * 16 < item - 1024) cp16(dst + 1024 + lane * 16, src + 1024 + lane * 16);
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}

template <int GPB>
__device__ __forceinline__ void load_sides(Sides<GPB>& k, uint32_t blk, int zeros, int g) {
  const uint32_t s = blk + 1024 + g * (GPB * 4), z = blk + 1024 + GPB * 32 + g * (GPB * 2);
  if constexpr (GPB == 1) {
    k.s[0] = lds32(s);
    k.z[0] = zeros ? lds16(z) : 0x0808u;
  } else if constexpr (GPB == 2) {
    const uint2 v = lds64(s);
    k.s[0] = v.x;
    k.s[1] = v.y;
    k.z[0] = zeros ? lds32(z) : 0x08080808u;
  } else {
    const uint4 v = lds128(s);
    k.s[0] = v.x;
    k.s[1] = v.y;
    k.s[2] = v.z;
    k.s[3] = v.w;
    const uint2 u = zeros ? lds64(z) : make_uint2(0x08080808u, 0x08080808u);
    k.z[0] = u.x;
    k.z[1] = u.y;
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
__device__ __forceinline__ void unpack(const uint4 (&w)[2], const Sides<GPB>& k, uint32_t (&A)[8][4]) {
#pragma unroll
  for (int q = 0; q < GPB; ++q) {
    const uint32_t zz = k.z[q >> 1] >> (16 * (q & 1));
    const uint32_t z0 = and_or(zz, 0xffu, 0x6400u) * 0x10001u;                  // 1024 + z of row g
    const uint32_t z1 = and_or(zz >> 4, 0xff0u, 0xd400u) * 0x10001u;            // -(64 + z) of row g + 8
#pragma unroll
    for (int t = 0; t < 8 / GPB; ++t) {
      const int st = q * (8 / GPB) + t;
      const uint32_t v = word(w[st >> 2], st & 3), v8 = v >> 8;
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
// At one token a block's 2048 weights have to pass in about 50 cycles per SM,
// so instructions are what is scarce.  Here the four bits are used as they
// are: in the lowest bits of an fp16 number they are the subnormal q * 2^-24
// (shifted left by four: q * 2^-20), which the tensor cores multiply exactly,
// so 8 weights cost 5 instructions.  The powers of two go into the scales,
// and the zero point is taken off the group's sum,
//   sum (q - z) x = 2^24 sum (q 2^-24) x - z sum x,
// with the sums of x over each group computed once per CTA (as a product with
// ones).  Both terms are of the size of the result, so nothing is lost.
//
// A CTA's warps split the columns of MT row tiles (16 rows each) and keep
// their column range over all row tiles that the CTA takes (every
// gridDim.x-th), so the weight stream of a warp never stops: its ring of
// STAGES blocks is filled across the ends of row tiles, the first of them
// before the wait on the previous kernel.  x goes straight from L1 to
// registers.  At a row tile's end the warps leave their sums in one of two
// shared-memory buffers and the first threads add them in warp order: one
// barrier per row tile, no atomics.
constexpr int kFewWarps = 8;

// A lane's share of x in one block: its columns of one token (any token where
// there are fewer: a column of the product that is not stored).
template <bool X8>
__device__ __forceinline__ void few_b(uint32_t (&b)[16], const unsigned char* p, int runs) {
  using V = typename XVec<X8>::T;
  if (runs >= 4) {
    load_b<X8>(b, [&](int k) { return *reinterpret_cast<const V*>(p + k * (X8 ? 32 : 64)); });
  } else {                                          // the last block of a C that 128 does not divide
    load_b<X8>(b, [&](int k) { return k < runs ? *reinterpret_cast<const V*>(p + k * (X8 ? 32 : 64)) : V{}; });
  }
}

template <int MT, int GPB>
__host__ __device__ constexpr int few_stages() { return 8 / MT; }
template <int MT>
__host__ __device__ constexpr int few_ld() { return 16 * MT + 4; }   // floats per token in a buffer: conflict-free writes
template <int MT>
__host__ __device__ constexpr int few_red_bytes() { return 2 * kFewWarps * 8 * few_ld<MT>() * 4; }

// red, then a ring of blocks per warp, then the sums of x
template <int MT, int GPB>
int few_smem(const Int4Args& a, int nwarp) {
  return few_red_bytes<MT>() + nwarp * few_stages<MT, GPB>() * MT * a.item + a.nblk * GPB * 32;
}

template <int MT, int GPB, bool X8>
__global__ void __launch_bounds__(kFewWarps * 32, 2) k_int4_few(const __grid_constant__ Int4Args a) {
  constexpr int LD = few_ld<MT>(), RED = few_red_bytes<MT>();
  constexpr int esz = X8 ? 1 : 2, STEPS = 8 / GPB, STAGES = few_stages<MT, GPB>();
  extern __shared__ __align__(16) unsigned char q2_int4_smem[];
  float* red = reinterpret_cast<float*>(q2_int4_smem);      // [2][kFewWarps][8 * LD]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int b0 = a.nblk * warp / nwarp, nb = a.nblk * (warp + 1) / nwarp - b0;   // nwarp <= nblk: nb >= 1
  const int nunit = (a.ntile + MT - 1) / MT;                // row tiles in bundles of MT
  const int mine = (nunit - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  const int n = mine * nb;                                  // blocks (times MT) of this warp's stream
  const uint32_t ring = saddr(q2_int4_smem) + RED + warp * (STAGES * MT * a.item);
  float* sums = reinterpret_cast<float*>(q2_int4_smem + RED + nwarp * (STAGES * MT * a.item));   // [nblk][GPB][8 tokens]

  // the stream: block fb of the warp's range in bundle `unit`
  int left = n, fb = 0, unit = blockIdx.x;
  uint32_t fslot = ring;
  const unsigned char* src = a.w + ((size_t)unit * MT * a.nblk + b0) * a.item;
  auto fetch = [&]() {
    if (left > 0) {
      --left;
#pragma unroll
      for (int m = 0; m < MT; ++m)                          // a missing row tile repeats the one before; its rows are not stored
        copy_block(fslot + m * a.item, src + (m && unit * MT + m < a.ntile ? (size_t)m * a.nblk * a.item : 0), a.item, lane);
      src += a.item;
      fslot += MT * a.item;
      if (fslot == ring + STAGES * MT * a.item) fslot = ring;
      if (++fb == nb) {
        fb = 0;
        unit += gridDim.x;
        src = a.w + ((size_t)unit * MT * a.nblk + b0) * a.item;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int d = 0; d < STAGES - 1; ++d) fetch();

  pdl_wait();                                               // x may come from the previous kernel
  pdl_trigger();
  const unsigned char* xp = static_cast<const unsigned char*>(a.x) + ((size_t)min(g, a.ntok - 1) * a.C + b0 * 128 + j * 8) * esz;
  for (int k = 0; k < nb; ++k) {
    uint32_t b[16];
    few_b<X8>(b, xp + k * (128 * esz), (a.C - (b0 + k) * 128) / 32);
    const uint32_t one[4] = {0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u};
#pragma unroll
    for (int q = 0; q < GPB; ++q) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int t = 0; t < STEPS; ++t) mma(c, one, b[2 * (q * STEPS + t)], b[2 * (q * STEPS + t) + 1]);
      if (g == 0) *reinterpret_cast<float2*>(sums + ((b0 + k) * GPB + q) * 8 + 2 * j) = make_float2(c[0], c[1]);
    }
  }
  __syncwarp();
  const float xsc0 = X8 && 2 * j < a.ntok ? a.xs[2 * j] : 1.f, xsc1 = X8 && 2 * j + 1 < a.ntok ? a.xs[2 * j + 1] : 1.f;

  float acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
  int cb = 0, cu = 0;                                       // block and bundle in use
  uint32_t slot = ring;
  for (int i = 0; i < n; ++i) {
    uint32_t b[16];
    few_b<X8>(b, xp + cb * (128 * esz), (a.C - (b0 + cb) * 128) / 32);
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    __syncwarp();                                           // block i has arrived for all lanes, block i - 1 is done with
    fetch();
    uint4 w[MT][2];
    Sides<GPB> sd[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      w[m][0] = lds128(slot + m * a.item + lane * 16);
      w[m][1] = lds128(slot + m * a.item + 512 + lane * 16);
      load_sides(sd[m], slot + m * a.item, a.zeros, g);
    }
    slot += MT * a.item;
    if (slot == ring + STAGES * MT * a.item) slot = ring;
#pragma unroll
    for (int q = 0; q < GPB; ++q) {
      float c[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m) c[m][0] = c[m][1] = c[m][2] = c[m][3] = 0.f;
#pragma unroll
      for (int t = 0; t < STEPS; ++t) {
        const int st = q * STEPS + t;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t v = word(w[m][st >> 2], st & 3), v8 = v >> 8;
          const uint32_t A[4] = {v & 0x000f000fu, v & 0x00f000f0u, v8 & 0x000f000fu, v8 & 0x00f000f0u};
          mma(c[m], A, b[2 * st], b[2 * st + 1]);
        }
      }
      const float2 X = *reinterpret_cast<const float2*>(sums + ((b0 + cb) * GPB + q) * 8 + 2 * j);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&sd[m].s[q]));
        const uint32_t zz = sd[m].z[q >> 1] >> (16 * (q & 1));
        const float z0 = (float)(zz & 0xffu), z1 = (float)((zz >> 8) & 0xffu);
        acc[m][0] = fmaf(sc.x, fmaf(c[m][0], 16777216.f, -z0 * X.x), acc[m][0]);
        acc[m][1] = fmaf(sc.x, fmaf(c[m][1], 16777216.f, -z0 * X.y), acc[m][1]);
        acc[m][2] = fmaf(sc.y, fmaf(c[m][2], 1048576.f, -z1 * X.x), acc[m][2]);
        acc[m][3] = fmaf(sc.y, fmaf(c[m][3], 1048576.f, -z1 * X.y), acc[m][3]);
      }
    }
    if (++cb == nb) {                                       // the bundle's end
      float* r = red + ((cu & 1) * kFewWarps + warp) * (8 * LD);
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
        for (int k = 0; k < nwarp; ++k) v += red[((cu & 1) * kFewWarps + k) * (8 * LD) + t * LD + rr];
        if (row0 + rr < a.R) a.y[(size_t)t * a.R + row0 + rr] = __float2half_rn(v);
      }
      cb = 0;
      ++cu;
    }
  }
}

// ------------------------------------------------------- 9..64 tokens
// A CTA takes 128 rows and a range of 256-column stages.  Its eight warps are
// four pairs of row tiles times the two 128-column blocks of a stage.  x of
// all tokens (a token's row is padded so that the lanes that load together
// fall on different banks) and each warp's own weights come through a ring of
// shared-memory stages by asynchronous 16-byte copies.  A block's A operands
// (here q - z itself: the tensor cores, not the instructions, are what is
// scarce) are unpacked once and used for all tokens, two tiles of 8 tokens
// and two row tiles at a time, so that four chains of dependent products are
// in flight.  When the column range is split over CTAs, they form a cluster
// and add their fp32 sums through distributed shared memory in rank order.
constexpr int kManyWarps = 8, kManyRows = 128, kManyStages = 3;

template <bool X8>
__host__ __device__ constexpr int x_row_bytes() { return X8 ? 256 + 32 : 512 + 64; }

constexpr int kOutLd = kManyRows + 4;

template <int NT, bool X8>
int many_smem(const Int4Args& a) {
  const int ring = kManyStages * (NT * 8 * x_row_bytes<X8>() + kManyWarps * 2 * a.item), out = NT * 8 * kOutLd * 4;
  return ring > out ? ring : out;
}

template <int NT, int GPB, bool X8>
__global__ void __launch_bounds__(kManyWarps * 32, 1) k_int4_many(const __grid_constant__ Int4Args a, const int nsplit) {
  constexpr int MT = 2, NTOK = NT * 8, ROWB = x_row_bytes<X8>(), STEPS = 8 / GPB;
  constexpr int esz = X8 ? 1 : 2, PIECES = 256 * esz / 16;
  extern __shared__ __align__(16) unsigned char q2_int4_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3, wm = warp & 3, wk = warp >> 2;
  const int rank = (int)blockIdx.x % nsplit, tile0 = (int)blockIdx.x / nsplit * (kManyRows / 16) + wm * MT;
  const int nstage = (a.nblk + 1) / 2;
  const int s0 = nstage * rank / nsplit, n = nstage * (rank + 1) / nsplit - s0;   // stages of this CTA
  const uint32_t sx = saddr(q2_int4_smem), sw = sx + kManyStages * (NTOK * ROWB) + warp * (MT * a.item);
  const int wstage = kManyWarps * MT * a.item;

  auto weights = [&](int i) {
    if (i < n) {
      const int blk = min(2 * (s0 + i) + wk, a.nblk - 1);   // past the last block: any block, its x is zero
#pragma unroll
      for (int m = 0; m < MT; ++m)                          // a missing row tile: any; its rows are not stored
        copy_block(sw + (i % kManyStages) * wstage + m * a.item,
                   a.w + ((size_t)min(tile0 + m, a.ntile - 1) * a.nblk + blk) * a.item, a.item, lane);
    }
  };
  auto xstage = [&](int i) {
    if (i < n) {
      const uint32_t base = sx + (i % kManyStages) * (NTOK * ROWB);
      for (int e = threadIdx.x; e < NTOK * PIECES; e += kManyWarps * 32) {
        const int t = e / PIECES, p = e % PIECES;
        const int c = (s0 + i) * 256 + p * (16 / esz);
        const bool live = t < a.ntok && c < a.C;
        const unsigned char* from = static_cast<const unsigned char*>(a.x) + (live ? ((size_t)t * a.C + c) * esz : 0);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(base + t * ROWB + p * 16), "l"(from),
                     "r"(live ? 16 : 0)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < kManyStages - 1; ++d) weights(d);
  pdl_wait();                                               // x may come from the previous kernel
  pdl_trigger();
#pragma unroll
  for (int d = 0; d < kManyStages - 1; ++d) xstage(d);

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[m][t][q] = 0.f;

  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kManyStages - 2) : "memory");
    __syncthreads();                                        // stage i has arrived for all, stage i - 1 is free
    weights(i + kManyStages - 1);
    xstage(i + kManyStages - 1);
    uint32_t A[MT][8][4];
    Sides<GPB> sd[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t at = sw + (i % kManyStages) * wstage + m * a.item;
      const uint4 w[2] = {lds128(at + lane * 16), lds128(at + 512 + lane * 16)};
      load_sides(sd[m], at, a.zeros, g);
      unpack(w, sd[m], A[m]);
    }
    const uint32_t xb = sx + (i % kManyStages) * (NTOK * ROWB) + g * ROWB + wk * (128 * esz) + j * (8 * esz);
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      uint32_t b[2][16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        load_b<X8>(b[h], [&](int k) {
          const uint32_t at = xb + (t + h) * 8 * ROWB + k * (32 * esz);
          if constexpr (X8) return lds64(at);
          else return lds128(at);
        });
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        float c[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) c[m][h][0] = c[m][h][1] = c[m][h][2] = c[m][h][3] = 0.f;
#pragma unroll
        for (int st = q * STEPS; st < (q + 1) * STEPS; ++st)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) mma(c[m][h], A[m][st], b[h][2 * st], b[h][2 * st + 1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&sd[m].s[q]));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            acc[m][t + h][0] = fmaf(sc.x, c[m][h][0], acc[m][t + h][0]);
            acc[m][t + h][1] = fmaf(sc.x, c[m][h][1], acc[m][t + h][1]);
            acc[m][t + h][2] = fmaf(sc.y, c[m][h][2], acc[m][t + h][2]);
            acc[m][t + h][3] = fmaf(sc.y, c[m][h][3], acc[m][t + h][3]);
          }
        }
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
  const int nwarp = a.nblk < kFewWarps ? a.nblk : kFewWarps;
  const int nunit = (a.ntile + MT - 1) / MT, most = 2 * dev_info().sms;
  return launch_pdl(k_int4_few<MT, GPB, X8>, a, nunit < most ? nunit : most, nwarp * 32, few_smem<MT, GPB>(a, nwarp), stream);
}

template <int NT, int GPB, bool X8>
int launch_many(const Int4Args& a, void* stream) {
  auto kernel = k_int4_many<NT, GPB, X8>;
  const int smem = many_smem<NT, X8>(a);
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
  a.item = q2_int4_item(d.reserved, d.layout);
  a.zeros = d.layout;
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
