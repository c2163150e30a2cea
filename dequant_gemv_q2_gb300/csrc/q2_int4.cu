// y = W x for 4-bit weights with group scales, 1..64 tokens (up to 16 here),
//
//   y[t][r] = sum_g s[r][g] * sum_{c in g} (q[r][c] - z[r][g]) * x[t][c],
//
// for x in fp16, or in 8 bits with one fp32 scale per token.
//
// The inner sums run on the tensor cores, 16 rows x 16 columns of weights
// against 8 tokens per instruction, fp32 accumulators.  The operands are q - z,
// exact in fp16 (9 instructions per 8 weights, unpack_step), so a group's sum
// is an fp32 sum of its exact products, for 8-bit x exact itself (integers
// below 2^18); group sums are scaled and added in fp32, and nothing but y is
// rounded to fp16.  The four bits as they are, as the fp16 subnormals q 2^-24,
// with the zero point taken off through the sums of x, cost 5 instructions but
// lost up to ten bits of the smaller terms beside a large one (the tensor cores
// line products up without normalising a subnormal): an activation of 6e4 over
// a zero weight put outputs off by their own size.
//
// Weights are stored in the order in which lanes use them: the unit is a
// block of 16 rows x 128 columns, 1 KB as two 16-byte loads per lane, with
// its scales and zero points behind it, so that a warp reads one stream.
//
// Up to 2 tokens: k_int4_few.  3 to 16: k_int4_many.  More: q2_int4_tc.cu.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "q2_int4.cuh"

namespace cg = cooperative_groups;

namespace q2 {
namespace {

// ------------------------------------------------------- 1 and 2 tokens
// At one token a block's 2048 weights have to pass in about 50 cycles per SM,
// so instructions are what is scarce.
//
// A CTA's warps split the columns of a row tile (16 rows) and keep their
// column range over all row tiles that the CTA takes (every gridDim.x-th): a
// warp's share of x stays in shared memory, and its weight stream never
// stops: its ring of pairs of blocks is filled across the ends of row tiles,
// the first of them before the wait on the previous kernel.  At a row tile's
// end the warps leave their sums in one of two shared-memory buffers and the
// first threads add them in warp order: one barrier per row tile, no atomics.
//
// 24576 x 4096 at one token, groups of 128 with zero points: 11.3 us on the
// device, 4.6 TB/s (without zero points 10.9); two tokens 11.9; from 8-bit x,
// which becomes fp16 on its way into shared memory, 11.2 (groups of 64).  4096 x
// 4096: 3.1 us, of which 2 are the launch and the first bytes' way.  What remains
// is instructions (2.2 of 4 issue slots per cycle under the profiler) and the
// ends: the first loads, x before them, the last row tiles.
constexpr int kFewWarps = 8, kFewTok = 2, kFewStages = 3, kFewCtas = 2;
constexpr int kFewRed = 2 * kFewWarps * kFewTok * 16 * 4;

// The buffers, then a ring of pairs of blocks per warp, x in fp16 by blocks and
// tokens (whole blocks, zeros past C).
int few_smem(const Int4Args& a, int nwarp) {
  return kFewRed + nwarp * kFewStages * 2 * a.item + a.nblk * a.ntok * 256;
}

template <int GPB, bool Z, bool X8>
__global__ void __launch_bounds__(kFewWarps * 32, kFewCtas) k_int4_few(const __grid_constant__ Int4Args a) {
  constexpr int STEPS = 8 / GPB, XB = 256;                              // bytes of a token's x in a block
  constexpr int ITEM = Q2_INT4_BLOCK_BYTES + GPB * (Z ? 48 : 32), STAGE = 2 * ITEM;
  extern __shared__ __align__(16) unsigned char q2_int4_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarp = blockDim.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int b0 = a.nblk * warp / nwarp, nb = a.nblk * (warp + 1) / nwarp - b0;   // nwarp <= nblk: nb >= 1
  const int mine = (a.ntile - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  float* red = reinterpret_cast<float*>(q2_int4_smem);      // [2][kFewWarps][kFewTok][16]
  const uint32_t ring = saddr(q2_int4_smem) + kFewRed + warp * (kFewStages * STAGE);
  unsigned char* xs = q2_int4_smem + kFewRed + nwarp * (kFewStages * STAGE) + b0 * (a.ntok * XB);   // this warp's x

  // the stream: pairs of blocks (the last of a row tile may be one block)
  int left = mine, fb = 0;                                  // row tiles to load; block of the row tile at `src`
  uint32_t fslot = ring + lane * 16;
  const size_t jump = ((size_t)gridDim.x * a.nblk - nb) * ITEM;
  const unsigned char* src = a.w + ((size_t)blockIdx.x * a.nblk + b0) * ITEM + lane * 16;
  auto fetch = [&]() {
    if (left > 0) {
      const int bytes = fb + 1 < nb ? STAGE : ITEM;
#pragma unroll
      for (int k = 0; k < STAGE; k += 512)
        if (lane * 16 + k < bytes) cp16(fslot + k, src + k);
      src += bytes;
      fslot = fslot == ring + (kFewStages - 1) * STAGE + lane * 16 ? ring + lane * 16 : fslot + STAGE;
      fb += 2;
      if (fb >= nb) {
        fb = 0;
        src += jump;
        --left;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int d = 0; d < kFewStages - 1; ++d) fetch();

  pdl_wait();                                               // x may come from the previous kernel
  pdl_trigger();
  // x in the order of the products' operands: a lane's words of two steps are
  // consecutive.  8-bit x becomes fp16 here, once (in the loop below it would
  // be as many instructions again as half of the weights').
  constexpr int PIECES = X8 ? 8 : 16, COLS = 128 / PIECES;  // 16-byte loads of a block, columns of each
  for (int e = lane; e < nb * a.ntok * PIECES; e += 32) {
    const int p = e % PIECES, kt = e / PIECES, k = a.ntok == 2 ? kt >> 1 : kt, t = kt - k * a.ntok;
    const int c = (b0 + k) * 128 + p * COLS;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(a.x) + ((size_t)t * a.C + c) * (16 / COLS));
    const uint4 v = c < a.C ? *from : make_uint4(0, 0, 0, 0);
    auto put = [&](int half, const uint4& u) {              // columns 8 half ..: half % 2 of step half / 2
      uint32_t* to = reinterpret_cast<uint32_t*>(xs + kt * XB) + (half >> 2) * 16 + (half & 3);
      to[0] = u.x;
      to[4] = u.y;
      to[8] = u.z;
      to[12] = u.w;
    };
    if constexpr (X8) {
      uint4 u;
      int8x4(v.x, u.x, u.y);
      int8x4(v.y, u.z, u.w);
      put(2 * p, u);
      int8x4(v.z, u.x, u.y);
      int8x4(v.w, u.z, u.w);
      put(2 * p + 1, u);
    } else {
      put(p, v);
    }
  }
  __syncwarp();
  // A lane's columns of one token (token g, of two: the other columns of the
  // products repeat them and are not stored).
  const uint32_t xl = saddr(xs) + (g & (a.ntok - 1)) * XB + j * 16;
  const int xblk = a.ntok * XB;
  auto xload = [&](uint32_t(&b)[16], uint32_t from) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint4 v = lds128(from + r * 64);
      b[4 * r] = v.x;
      b[4 * r + 1] = v.y;
      b[4 * r + 2] = v.z;
      b[4 * r + 3] = v.w;
    }
  };
  const float xsc0 = X8 ? a.xs[0] : 1.f, xsc1 = X8 && a.ntok > 1 ? a.xs[1] : 1.f;

  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};   // rows g and g + 8, tokens 0 and 1
  // K blocks at `from`, columns from block b on: K independent chains of products
  auto use = [&](auto kc, uint32_t from, int blk) {
    constexpr int K = decltype(kc)::value;
    const uint32_t xat = xl + blk * xblk;
    uint32_t b[K][16];
    uint4 w[K][2];
    Sides<GPB> sd[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      w[k][0] = lds128(from + k * ITEM + lane * 16);
      w[k][1] = lds128(from + k * ITEM + 512 + lane * 16);
      load_sides(sd[k], from + k * ITEM, Z, g);
      xload(b[k], xat + k * xblk);
    }
#pragma unroll
    for (int q = 0; q < GPB; ++q) {
      float c[K][4];
      Zeros z[K];
#pragma unroll
      for (int k = 0; k < K; ++k) z[k] = zeros_of(Z ? sd[k].z[q >> 1] >> (16 * (q & 1)) : 0x0808u);
#pragma unroll
      for (int t = 0; t < STEPS; ++t) {
        const int st = q * STEPS + t;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          uint32_t A[4];
          unpack_step(word(w[k][st >> 2], st & 3), z[k], A[0], A[1], A[2], A[3]);
          if (t == 0) mma_first(c[k], A, b[k][2 * st], b[k][2 * st + 1]);
          else mma(c[k], A, b[k][2 * st], b[k][2 * st + 1]);
        }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&sd[k].s[q]));
        fma2(acc[0], make_float2(sc.x, sc.x), make_float2(c[k][0], c[k][1]));
        fma2(acc[1], make_float2(sc.y, sc.y), make_float2(c[k][2], c[k][3]));
      }
    }
  };
  uint32_t slot = ring;
  for (int u = 0; u < mine; ++u) {
    for (int cb = 0; cb < nb; cb += 2) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kFewStages - 2) : "memory");
      __syncwarp();                                         // the pair has arrived for all lanes, the one before is done with
      fetch();
      if (cb + 1 < nb) use(std::integral_constant<int, 2>(), slot, cb);
      else use(std::integral_constant<int, 1>(), slot, cb);
      slot = slot == ring + (kFewStages - 1) * STAGE ? ring : slot + STAGE;
    }
    float* r = red + ((u & 1) * kFewWarps + warp) * (kFewTok * 16);
    if (j == 0) {                                           // tokens 0 and 1
      r[g] = acc[0].x * xsc0;
      r[16 + g] = acc[0].y * xsc1;
      r[g + 8] = acc[1].x * xsc0;
      r[16 + g + 8] = acc[1].y * xsc1;
    }
    acc[0] = acc[1] = make_float2(0.f, 0.f);
    __syncthreads();
    const int row = ((int)blockIdx.x + u * (int)gridDim.x) * 16 + (threadIdx.x & 15), t = threadIdx.x >> 4;
    if (t < a.ntok && row < a.R) {
      float v = 0.f;
      for (int k = 0; k < nwarp; ++k) v += red[((u & 1) * kFewWarps + k) * (kFewTok * 16) + threadIdx.x];
      a.y[(size_t)t * a.R + row] = __float2half_rn(v);
    }
  }
}

// ------------------------------------------------------- 3..16 tokens
// A CTA takes 128 rows and a range of 128-column blocks.  Its eight warps are
// two groups of four, which take alternate blocks and run on their own (the
// two warps of a scheduler belong to different groups, so one waits or unpacks
// while the other multiplies); each warp of a group has two row tiles.  A
// group's x of all tokens (a token's row is padded so that the lanes that load
// together fall on different banks) and each warp's own weights come through a
// ring of shared-memory stages by asynchronous 16-byte copies.  A block's
// operands are unpacked once and used for all tokens.
// When the column range is split over CTAs, they form a cluster and add their
// fp32 sums through distributed shared memory in rank order.
//
// What bounds it at 8 tokens is instructions and uneven SMs (240 CTAs, two on
// some and one on others: an even spread would save 20%), 3.2 TB/s at
// 5120 x 17408 (8-bit x, groups of 64: 14.9 us) and 3.7 at 24576 x 4096 (14.3
// us); at 16 tokens (20.7 us at 24576 x 4096) the products and, with two CTAs
// per SM, the latencies between them.  More than 16 tokens would cost 32
// accumulators more per thread: they go to the kernel in q2_int4_tc.cu
// (24576 x 4096 at 32 tokens 25.7 us, twice the 16-token time here 42).  In
// groups of 32 the variants of three stages spill 4 to 16 bytes.
constexpr int kManyWarps = 8, kManyRows = 128, kManyMax = 8;

template <bool X8>
__host__ __device__ constexpr int x_row_bytes() { return X8 ? 128 + 16 : 256 + 16; }
// Stages of a group's ring with so many CTAs per SM.  At up to 8 tokens one or
// two take four, and 128 registers a thread instead of 80 (34816 x 5120 from
// 8-bit x at 7 tokens 22.4 us, 23.5 with what three CTAs per SM leave room for).
template <int NT>
__host__ __device__ constexpr int many_stages(int share) { return NT == 1 && share <= 2 ? 4 : 3; }
template <int NT>
__host__ __device__ constexpr int many_ctas() { return NT == 1 ? 3 : 2; }   // per SM, at most

constexpr int kOutLd = kManyRows + 4;

template <int NT, bool X8>
int many_smem(const Int4Args& a, int stages) {
  const int ring = 2 * stages * (NT * 8 * x_row_bytes<X8>() + 8 * a.item), out = NT * 8 * kOutLd * 4;
  return ring > out ? ring : out;
}

template <int NT, int GPB, bool X8, int STAGES>
__global__ void __launch_bounds__(kManyWarps * 32, STAGES == 4 ? 2 : many_ctas<NT>())
    k_int4_many(const __grid_constant__ Int4Args a, const int nsplit) {
  constexpr int MT = 2, NTOK = NT * 8, ROWB = x_row_bytes<X8>(), STEPS = 8 / GPB;
  constexpr int esz = X8 ? 1 : 2, PIECES = 128 * esz / 16, PASS = 128 / PIECES;   // pieces of a row; tokens of a pass
  extern __shared__ __align__(16) unsigned char q2_int4_smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3, wm = warp & 3, wk = warp >> 2;
  const int rank = (int)blockIdx.x % nsplit, tile0 = (int)blockIdx.x / nsplit * (kManyRows / 16) + wm * MT;
  const int b0 = a.nblk * rank / nsplit + wk, n = (a.nblk * (rank + 1) / nsplit - b0 + 1) / 2;   // this group: b0, b0 + 2, ..
  const int stage = NTOK * ROWB + 8 * a.item;
  const uint32_t ring = saddr(q2_int4_smem) + wk * (STAGES * stage);

  const unsigned char* wsrc[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m)                              // a missing row tile: the last one; its rows are not stored
    wsrc[m] = a.w + ((size_t)min(tile0 + m, a.ntile - 1) * a.nblk + b0) * a.item + lane * 16;
  const bool sides = lane * 16 < a.item - 1024;
  const uint32_t wdst = ring + NTOK * ROWB + wm * MT * a.item + lane * 16;
  auto weights = [&](int i, int st) {
    if (i < n) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t d = wdst + st * stage + m * a.item;
        cp16(d, wsrc[m]);
        cp16(d + 512, wsrc[m] + 512);
        if (sides) cp16(d + 1024, wsrc[m] + 1024);
        wsrc[m] += 2 * a.item;
      }
    }
  };
  const int xp = (threadIdx.x & 127) % PIECES, xt = (threadIdx.x & 127) / PIECES;   // this thread's piece and first token
  const unsigned char* xsrc = static_cast<const unsigned char*>(a.x) + ((size_t)xt * a.C + b0 * 128) * esz + xp * 16;
  const size_t xpass = (size_t)PASS * a.C * esz;
  const uint32_t xdst = ring + xt * ROWB + xp * 16;
  int xleft = a.C - b0 * 128 - xp * (16 / esz);             // columns from this piece to the end of the row
  auto xstage = [&](int i, int st) {
    if (i < n) {
      const unsigned char* from = xsrc;
#pragma unroll
      for (int t = 0; t < NTOK; t += PASS) {
        const bool live = xt + t < a.ntok && xleft > 0;
        if (PASS <= NTOK || xt + t < NTOK)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(xdst + st * stage + t * ROWB),
                       "l"(live ? from : static_cast<const unsigned char*>(a.x)), "r"(live ? 16 : 0)
                       : "memory");
        from += xpass;
      }
      xsrc += 256 * esz;
      xleft -= 256;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < STAGES - 1; ++d) weights(d, d);
  pdl_wait();                                               // x may come from the previous kernel
  pdl_trigger();
#pragma unroll
  for (int d = 0; d < STAGES - 1; ++d) xstage(d, d);

  float2 acc[MT][NT][2];                                    // rows g and g + 8, tokens 2j and 2j + 1
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int q = 0; q < 2; ++q) acc[m][t][q] = make_float2(0.f, 0.f);

  int st = 0, last = STAGES - 1;                            // stage in use, stage before it (free)
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
    asm volatile("bar.sync %0, 128;" ::"r"(1 + wk) : "memory");   // block i has arrived for the group, block i - 1 is done with
    weights(i + STAGES - 1, last);
    xstage(i + STAGES - 1, last);
    Sides<GPB> sd[MT];
    const uint32_t base = ring + st * stage;
    // 8-bit x: this lane's pairs of token g; fp16: the row and piece whose address this lane gives a matrix load
    const uint32_t xb = base + (X8 ? g * ROWB + 2 * j : (lane & 7) * ROWB + (lane >> 3) * 16);
    auto xload = [&](uint32_t(&b)[16], int t) {
      if constexpr (X8) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t at = xb + t * 8 * ROWB + k * 16;
          int8x4(lds16(at) | lds16(at + 8) << 16, b[2 * k], b[2 * k + 1]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(b[4 * k]), "=r"(b[4 * k + 1]), "=r"(b[4 * k + 2]), "=r"(b[4 * k + 3])
                       : "r"(xb + t * 8 * ROWB + k * 64));
      }
    };
    uint4 w[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t at = base + NTOK * ROWB + (wm * MT + m) * a.item;
      w[m][0] = lds128(at + lane * 16);
      w[m][1] = lds128(at + 512 + lane * 16);
      load_sides(sd[m], at, a.zeros, g);
    }
    uint32_t b[NT][16];
#pragma unroll
    for (int t = 0; t < NT; ++t) xload(b[t], t);
#pragma unroll
    for (int q = 0; q < GPB; ++q) {
      float c[MT][NT][4];
      Zeros z[MT];
#pragma unroll
      for (int m = 0; m < MT; ++m) z[m] = zeros_of(sd[m].z[q >> 1] >> (16 * (q & 1)));
#pragma unroll
      for (int k = q * STEPS; k < (q + 1) * STEPS; ++k) {
        uint32_t A[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) unpack_step(word(w[m][k >> 2], k & 3), z[m], A[m][0], A[m][1], A[m][2], A[m][3]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (k == q * STEPS) mma_first(c[m][t], A[m], b[t][2 * k], b[t][2 * k + 1]);
            else mma(c[m][t], A[m], b[t][2 * k], b[t][2 * k + 1]);
          }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const float2 sc = __half22float2(*reinterpret_cast<const __half2*>(&sd[m].s[q]));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          fma2(acc[m][t][0], make_float2(sc.x, sc.x), make_float2(c[m][t][0], c[m][t][1]));
          fma2(acc[m][t][1], make_float2(sc.y, sc.y), make_float2(c[m][t][2], c[m][t][3]));
        }
      }
    }
    last = st;
    st = st + 1 == STAGES ? 0 : st + 1;
  }
  // the second group's warps add to the first group's, in shared memory
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
            const float v = q & 1 ? acc[m][t][q >> 1].y : acc[m][t][q >> 1].x;
            *o = half ? v : *o + v;
          }
    }
    __syncthreads();
  }
  const int row0 = (int)blockIdx.x / nsplit * kManyRows;
  auto store = [&](int e, float v) {
    const int t = e / kManyRows, r = e % kManyRows;
    if (row0 + r < a.R) a.y[(size_t)t * a.R + row0 + r] = __float2half_rn(X8 ? v * a.xs[t] : v);
  };
  const int all = a.ntok * kManyRows;
  if (nsplit == 1) {
    for (int e = threadIdx.x; e < all; e += kManyWarps * 32) store(e, out[e / kManyRows * kOutLd + e % kManyRows]);
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster_meet();
  constexpr int PER = NTOK * kManyRows / 2 / (kManyWarps * 32);   // elements of a thread: two CTAs at least share them
  const int e0 = all * rank / nsplit + threadIdx.x, e1 = all * (rank + 1) / nsplit;
  const float* peer[kManyMax];
#pragma unroll
  for (int k = 0; k < kManyMax; ++k) peer[k] = k < nsplit ? cluster.map_shared_rank(out, k) : out;
  float v[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = e0 + i * (kManyWarps * 32), at = e / kManyRows * kOutLd + e % kManyRows;
    float p[kManyMax];
#pragma unroll
    for (int k = 0; k < kManyMax; ++k) p[k] = k < nsplit && e < e1 ? peer[k][at] : 0.f;
    v[i] = p[0];
#pragma unroll
    for (int k = 1; k < kManyMax; ++k) v[i] += p[k];
  }
  cluster_arrive();                                         // this CTA has read the others' sums
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (e0 + i * (kManyWarps * 32) < e1) store(e0 + i * (kManyWarps * 32), v[i]);
  cluster_wait();                                           // and they this one's
}

// ------------------------------------------------------- launch
template <int GPB, bool X8>
int launch_few(const Int4Args& a, int slots, void* stream) {
  const int nwarp = a.nblk < kFewWarps ? a.nblk : kFewWarps, smem = few_smem(a, nwarp);
  const int grid = a.ntile < slots ? a.ntile : slots;
  return a.zeros ? launch_pdl(k_int4_few<GPB, true, X8>, a, grid, nwarp * 32, smem, stream)
                 : launch_pdl(k_int4_few<GPB, false, X8>, a, grid, nwarp * 32, smem, stream);
}

// The split of the columns over a cluster, from the time of a CTA: its blocks
// (about 0.22 us each for a CTA alone on its SM, 0.2 + 0.8 n of that with n of
// them on it), three blocks for the cluster's barriers, and waves where the
// clusters do not all run at once.  Against all sizes and spreads timed (8
// shapes of the 8B and 14B stacks, 1 to 16 tokens) the choice is within 10%.
template <int NT, int GPB, bool X8>
int launch_many(const Int4Args& a, void* stream) {
  static ClusterCounts counts;
  auto kernel_of = [](int share) {
    return many_stages<NT>(share) == 4 ? k_int4_many<NT, GPB, X8, many_stages<NT>(1)> : k_int4_many<NT, GPB, X8, 3>;
  };
  auto fn_of = [&](int share) { return reinterpret_cast<const void*>(kernel_of(share)); };
  const int tiles = (a.ntile + kManyRows / 16 - 1) / (kManyRows / 16), sms = dev_info().sms;
  if (set_smem(fn_of(1), kSmemPerSm - 1024) || set_smem(fn_of(3), kSmemPerSm - 1024)) return Q2_ECUDA;
  // No more CTAs on an SM than an even spread needs (the next one's shared
  // memory is taken): left alone they fill some SMs and leave others idle
  // (256 CTAs of 4096 x 4096: 5.6 us instead of 4.4).
  auto smem_of = [&](int share) {
    const int smem = many_smem<NT, X8>(a, many_stages<NT>(share));
    return share < many_ctas<NT>() ? std::max(smem, kSmemPerSm / (share + 1)) : smem;
  };
  int nsplit = 1, with = 1;
  long long best = 0;
  for (int s = 1; s <= kManyMax && 2 * s <= a.nblk; ++s) {
    int share = std::min((tiles * s + sms - 1) / sms, many_ctas<NT>()), fit = 0;
    for (; share <= many_ctas<NT>(); ++share) {               // the clusters that run at once with so many CTAs per SM
      fit = counts.get(fn_of(share), s, kManyWarps * 32, smem_of(share));
      if (fit >= tiles) break;
    }
    share = std::min(share, many_ctas<NT>());
    const long long waves = (tiles + fit - 1) / fit, cost = (a.nblk + s - 1) / s * (1 + 4 * share) * waves + (s > 1 ? 15 : 0);
    if (s == 1 || cost < best) {
      best = cost;
      nsplit = s;
      with = share;
    }
  }
  return launch_clusters(kernel_of(with), tiles, nsplit, kManyWarps * 32, smem_of(with), stream, a, nsplit);
}

template <int GPB, bool X8>
int launch_tokens(const Int4Args& a, void* stream) {
  if (a.ntok <= kFewTok) {
    // k_int4_few keeps x in shared memory and hands out whole row tiles: it is
    // taken where two CTAs fit an SM with it (5120 x 17408 at two tokens, one
    // CTA: 16.0 us, 12.6 with k_int4_many), unless the last of several rounds is
    // mostly empty (5120 x 17408 at one token, 1.05 rounds: 13.1 us, 12.4 with
    // k_int4_many; 6144 x 4096, 1.26 rounds: 4.7 and 5.4; 24576 x 4096, 5.05: 11.0
    // and 13.5).
    const int slots = kFewCtas * dev_info().sms, rounds = (a.ntile + slots - 1) / slots;
    const bool fits = kFewCtas * (few_smem(a, kFewWarps) + 1024) <= kSmemPerSm;
    if (fits && (rounds == 1 || 5ll * a.ntile >= 3ll * rounds * slots)) return launch_few<GPB, X8>(a, slots, stream);
  }
  if (a.ntok <= 8) return launch_many<1, GPB, X8>(a, stream);
  if (a.ntok <= 16) return launch_many<2, GPB, X8>(a, stream);
  if (a.nblk > 1) return q2_int4_tc(a, Q2_INT4_COLS / GPB, X8, stream);
  // One block per row tile (up to 128 columns): q2_int4_tc takes two in turn.
  for (int t = 0; t < a.ntok; t += 16) {
    Int4Args b = a;
    b.x = static_cast<const unsigned char*>(a.x) + (size_t)t * a.C * (X8 ? 1 : 2);
    b.xs = X8 ? a.xs + t : nullptr;
    b.y = a.y + (size_t)t * a.R;
    b.ntok = std::min(16, a.ntok - t);
    if (const int e = launch_many<2, GPB, X8>(b, stream)) return e;
  }
  return Q2_OK;
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
