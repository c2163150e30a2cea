// Root-mean-square norm of rows, with the residual's addition in front and an
// fp16 and/or an 8-bit output behind it: what runs ahead of each projection
// of a decode step.  Per row of C values,
//
//   h = x + r,   y = h * w / sqrt(mean(h^2) + eps),
//   r' = fp16(h),  y16 = fp16(y),  s = max|y| / 127,  y8 = rint(y / s),
//
// all in fp32 from the fp16 inputs; h, y and s are each rounded once.  The sum
// of squares is a tree over the row's threads in a fixed order, so a row's
// result does not depend on the batch.
//
// A row is read once and stays in registers between the sum, the maximum and
// the stores, so the bytes of the inputs and outputs are all that moves.  Rows
// of up to 512 columns take 16 or 32 threads each (a reduction is five
// shuffles, no barrier); longer ones a block each.
#include <cuda_fp16.h>

#include "q2_common.cuh"

namespace q2 {
namespace {

struct NormArgs {
  const __half* x;            // row (t, h) at x + t * ldx + h * C
  const __half* res;          // [rows][C] or null
  __half* res_out;            // [rows][C] or null
  const __half* w;            // [C]
  __half* y;                  // row (t, h) at y + t * ldy + h * C, or null
  int8_t* y8;                 // [rows][C] or null
  float* s8;                  // [rows]
  long long ldx, ldy, rows;
  int heads, C;
  float eps;
};

// Sum (or maximum of the bit patterns of magnitudes, which puts NaN above
// infinity above every finite value) over the threads of a row: TPR lanes of
// a warp, or the whole block when TPR is 0.
template <int TPR, bool MAX, typename T>
__device__ __forceinline__ T row_reduce(T v, T* part) {
#pragma unroll
  for (int o = (TPR ? TPR : 32) / 2; o > 0; o >>= 1) {
    const T u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max(v, u) : v + u;
  }
  if (TPR) return v;
  const int nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < nw ? part[threadIdx.x & 31] : T(0);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const T u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max(v, u) : v + u;
  }
  return v;
}

// TPR: threads per row (16 or 32, several rows per block; 0: one row per
// block).  CH: pieces of 8 columns a thread holds.  VEC: pieces are 16-byte
// loads; otherwise a thread's columns are strided by the row's threads.
template <int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(TPR ? 256 : 1024) k_rmsnorm(const __grid_constant__ NormArgs a) {
  __shared__ float psum[32];
  __shared__ uint32_t pmax[32];
  const int nt = TPR ? TPR : blockDim.x;
  const int tid = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  const long long row = TPR ? (long long)blockIdx.x * (256 / (TPR ? TPR : 1)) + threadIdx.x / (TPR ? TPR : 1)
                            : (long long)blockIdx.x;
  const bool live = !TPR || row < a.rows;
  const long long t = row / a.heads;
  const int C = a.C;
  const __half* x = a.x + t * a.ldx + (row - t * a.heads) * C;
  const size_t flat = (size_t)row * C;
  auto col = [&](int c, int i) { return VEC ? (c * nt + tid) * 8 + i : (c * 8 + i) * nt + tid; };
  auto load8 = [&](const __half* p, int c, float* v) {
    if (VEC) {
      if (live && col(c, 0) < C) {
        const uint4 raw = *reinterpret_cast<const uint4*>(p + col(c, 0));
        const __half2* h2 = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = __half22float2(h2[i]);
          v[2 * i] = f.x;
          v[2 * i + 1] = f.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = live && col(c, i) < C ? __half2float(p[col(c, i)]) : 0.f;
    }
  };
  auto store8 = [&](__half* p, int c, const float* v) {
    if (!live) return;
    if (VEC) {
      if (col(c, 0) >= C) return;
      uint4 raw;
      __half2* h2 = reinterpret_cast<__half2*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) h2[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      *reinterpret_cast<uint4*>(p + col(c, 0)) = raw;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col(c, i) < C) p[col(c, i)] = __float2half_rn(v[i]);
    }
  };

  pdl_wait();                                   // x and the residual may come from the previous kernel
  pdl_trigger();
  float h[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) load8(x, c, h[c]);
  if (a.res) {
    float r[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) load8(a.res + flat, c, r[c]);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] += r[c][i];
  }
  float w[CH][8];
  if (CH < 4) {                                 // in flight with the row; wider rows have no registers for it
#pragma unroll
    for (int c = 0; c < CH; ++c) load8(a.w, c, w[c]);
  }
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
  ss = row_reduce<TPR, false>(ss, psum);
  if (a.res_out) {
#pragma unroll
    for (int c = 0; c < CH; ++c) store8(a.res_out + flat, c, h[c]);
  }
  const float k = rsqrtf(ss / (float)C + a.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (CH >= 4) load8(a.w, c, w[c]);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * k * w[c][i];
  }
  if (a.y) {
    __half* y = a.y + t * a.ldy + (row - t * a.heads) * C;
#pragma unroll
    for (int c = 0; c < CH; ++c) store8(y, c, h[c]);
  }
  if (a.y8) {
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(h[c][i]) & 0x7fffffffu);
    m = row_reduce<TPR, true>(m, pmax);
    const float top = __uint_as_float(m);
    // A zero row has scale 0 and zeros; a row with a NaN (or an infinity) has
    // a scale that is NaN (or infinite), which its consumer multiplies by.
    const float inv = top > 0.f ? 127.f / top : 0.f;
    if (live && tid == 0) a.s8[row] = top / 127.f;
    if (live) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (VEC) {
          if (col(c, 0) < C) {
            uint32_t lo = 0, hi = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo |= (uint32_t)(__float2int_rn(h[c][i] * inv) & 0xff) << (8 * i);
              hi |= (uint32_t)(__float2int_rn(h[c][i + 4] * inv) & 0xff) << (8 * i);
            }
            *reinterpret_cast<uint2*>(a.y8 + flat + col(c, 0)) = make_uint2(lo, hi);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col(c, i) < C) a.y8[flat + col(c, i)] = (int8_t)__float2int_rn(h[c][i] * inv);
        }
      }
    }
  }
}

template <bool VEC>
int launch_norm(const NormArgs& a, void* stream) {
  const int pieces = (a.C + 7) / 8;
  auto blocks = [&](int per) { return (int)((a.rows + per - 1) / per); };
  if (pieces <= 16) return launch_pdl(k_rmsnorm<16, 1, VEC>, a, blocks(16), 256, 0, stream);
  if (pieces <= 32) return launch_pdl(k_rmsnorm<32, 1, VEC>, a, blocks(8), 256, 0, stream);
  if (pieces <= 64) return launch_pdl(k_rmsnorm<32, 2, VEC>, a, blocks(8), 256, 0, stream);
  auto threads = [&](int ch) { return ((pieces + ch - 1) / ch + 31) / 32 * 32; };
  if (pieces <= 512) return launch_pdl(k_rmsnorm<0, 1, VEC>, a, blocks(1), threads(1), 0, stream);
  if (pieces <= 1024) return launch_pdl(k_rmsnorm<0, 2, VEC>, a, blocks(1), threads(2), 0, stream);
  return launch_pdl(k_rmsnorm<0, 4, VEC>, a, blocks(1), threads(4), 0, stream);
}

}  // namespace
}  // namespace q2

extern "C" int q2_rmsnorm(const void* x, long long ldx, int ntok, int heads, int C, const void* residual,
                          void* residual_out, const void* weight, float eps, void* y, long long ldy, void* y8,
                          float* scale8, q2_stream stream) {
  using namespace q2;
  if (ntok < 0 || !(eps >= 0.f)) return Q2_EINVAL;
  if (heads < 1 || C < 1 || C > Q2_NORM_MAX_C || (long long)ntok * heads > 0x7fffffffll) return Q2_ESHAPE;
  const long long width = (long long)heads * C;
  if ((ntok > 1 && ldx < width) || (y && ntok > 1 && ldy < width)) return Q2_ESHAPE;
  if (ntok == 0) return Q2_OK;                  // an empty tensor's pointers may be null
  if (!x || !weight || (!y && !y8) || (y8 && !scale8) || (!residual) != (!residual_out)) return Q2_EINVAL;
  NormArgs a = {};
  a.x = static_cast<const __half*>(x);
  a.res = static_cast<const __half*>(residual);
  a.res_out = static_cast<__half*>(residual_out);
  a.w = static_cast<const __half*>(weight);
  a.y = static_cast<__half*>(y);
  a.y8 = static_cast<int8_t*>(y8);
  a.s8 = scale8;
  a.ldx = ldx;
  a.ldy = ldy;
  a.rows = (long long)ntok * heads;
  a.heads = heads;
  a.C = C;
  a.eps = eps;
  auto on = [](const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  // 2-byte (and, for the scales, 4-byte) elements have to be on their own boundary
  if (!on(x, 2) || !on(residual, 2) || !on(residual_out, 2) || !on(weight, 2) || !on(y, 2) || !on(scale8, 4))
    return Q2_EALIGN;
  const bool vec = C % 8 == 0 && (ntok == 1 || (ldx % 8 == 0 && (!y || ldy % 8 == 0))) && on(x, 16) &&
                   on(residual, 16) && on(residual_out, 16) && on(weight, 16) && on(y, 16) && on(y8, 8);
  return vec ? launch_norm<true>(a, stream) : launch_norm<false>(a, stream);
}
