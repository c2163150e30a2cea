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
// shuffles, no barrier); longer ones a block, which goes on to further rows
// with the next row's loads in flight during the reductions of the one before.
#include <cuda_fp16.h>

#include <algorithm>

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

// One thread's share of a row: CH pieces of 8 columns.  VEC: a piece is one
// 16-byte access; otherwise its columns are strided by the row's nt threads.
template <int CH, bool VEC>
struct Row {
  int tid, nt, C;
  bool live;
  __device__ __forceinline__ int col(int c, int i) const { return VEC ? (c * nt + tid) * 8 + i : (c * 8 + i) * nt + tid; }

  __device__ __forceinline__ void load(const __half* p, uint4 (&r)[CH]) const {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (VEC) {
        r[c] = live && col(c, 0) < C ? *reinterpret_cast<const uint4*>(p + col(c, 0)) : make_uint4(0, 0, 0, 0);
      } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(&r[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          h[i] = live && col(c, i) < C ? reinterpret_cast<const uint16_t*>(p)[col(c, i)] : (uint16_t)0;
      }
    }
  }
  __device__ __forceinline__ static void floats(const uint4& r, float (&v)[8]) {
    const __half2* h2 = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(h2[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void store(__half* p, const float (&v)[CH][8]) const {
    if (!live) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (VEC) {
        uint4 raw;
        __half2* h2 = reinterpret_cast<__half2*>(&raw);
#pragma unroll
        for (int i = 0; i < 4; ++i) h2[i] = __floats2half2_rn(v[c][2 * i], v[c][2 * i + 1]);
        if (col(c, 0) < C) *reinterpret_cast<uint4*>(p + col(c, 0)) = raw;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col(c, i) < C) p[col(c, i)] = __float2half_rn(v[c][i]);
      }
    }
  }
  __device__ __forceinline__ void store8(int8_t* p, const float (&v)[CH][8], float inv) const {
    if (!live) return;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (VEC) {
        uint32_t lo = 0, hi = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo |= (uint32_t)(__float2int_rn(v[c][i] * inv) & 0xff) << (8 * i);
          hi |= (uint32_t)(__float2int_rn(v[c][i + 4] * inv) & 0xff) << (8 * i);
        }
        if (col(c, 0) < C) *reinterpret_cast<uint2*>(p + col(c, 0)) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col(c, i) < C) p[col(c, i)] = (int8_t)__float2int_rn(v[c][i] * inv);
      }
    }
  }
};

// TPR: threads per row (16 or 32, several rows per block; 0: a block per row,
// then every gridDim.x-th).  NT: threads of a block at most.
template <int TPR, int CH, bool VEC, int NT>
__global__ void __launch_bounds__(NT) k_rmsnorm(const __grid_constant__ NormArgs a) {
  // Rows ahead: where the registers hold them (wider rows wait for theirs).
  constexpr bool AHEAD = TPR == 0 && CH <= 2;
  __shared__ float psum[2][32];
  __shared__ uint32_t pmax[2][32];
  Row<CH, VEC> me;
  me.nt = TPR ? TPR : blockDim.x;
  me.tid = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  me.C = a.C;
  long long row = TPR ? (long long)blockIdx.x * (256 / (TPR ? TPR : 1)) + threadIdx.x / (TPR ? TPR : 1)
                      : (long long)blockIdx.x;
  me.live = !TPR || row < a.rows;
  auto place = [&](long long r, long long ld) {                  // element offset of row r = (token, head)
    const long long t = a.heads == 1 ? r : r / a.heads;
    return t * ld + (r - t * a.heads) * a.C;
  };
  uint4 xr[CH], rr[CH], wr[CH];
  pdl_wait();                                   // x and the residual may come from the previous kernel
  pdl_trigger();
  me.load(a.x + place(row, a.ldx), xr);
  if (a.res) me.load(a.res + (size_t)row * a.C, rr);
  if (CH <= 2) me.load(a.w, wr);
  for (int turn = 0;; turn ^= 1) {
    float h[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      me.floats(xr[c], h[c]);
      if (a.res) {
        float r[8];
        me.floats(rr[c], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c][i] += r[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[c][i], h[c][i], ss);
    }
    const long long next = row + gridDim.x;
    if (AHEAD && next < a.rows) {
      me.load(a.x + place(next, a.ldx), xr);
      if (a.res) me.load(a.res + (size_t)next * a.C, rr);
    }
    if (CH > 2) me.load(a.w, wr);
    ss = row_reduce<TPR, false>(ss, psum[turn]);
    if (a.res_out) me.store(a.res_out + (size_t)row * a.C, h);
    const float k = rsqrtf(ss / (float)a.C + a.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      me.floats(wr[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * k * w[i];
    }
    if (a.y) me.store(a.y + place(row, a.ldy), h);
    if (a.y8) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(h[c][i]) & 0x7fffffffu);
      m = row_reduce<TPR, true>(m, pmax[turn]);
      const float top = __uint_as_float(m);
      // A zero row has scale 0 and zeros; a row with a NaN (or an infinity) has
      // a scale that is NaN (or infinite), which its consumer multiplies by.
      if (me.live && me.tid == 0) a.s8[row] = top / 127.f;
      me.store8(a.y8 + (size_t)row * a.C, h, top > 0.f ? 127.f / top : 0.f);
    }
    if (TPR || next >= a.rows) return;
    row = next;
    if (!AHEAD) {
      me.load(a.x + place(row, a.ldx), xr);
      if (a.res) me.load(a.res + (size_t)row * a.C, rr);
    }
  }
}

template <bool VEC>
int launch_norm(const NormArgs& a, void* stream) {
  const int pieces = (a.C + 7) / 8;
  auto blocks = [&](int per) { return (int)((a.rows + per - 1) / per); };
  if (pieces <= 16) return launch_pdl(k_rmsnorm<16, 1, VEC, 256>, a, blocks(16), 256, 0, stream);
  if (pieces <= 32) return launch_pdl(k_rmsnorm<32, 1, VEC, 256>, a, blocks(8), 256, 0, stream);
  if (pieces <= 64) return launch_pdl(k_rmsnorm<32, 2, VEC, 256>, a, blocks(8), 256, 0, stream);
  // A block per row, up to as many blocks as fit 1024 threads on every SM.
  auto threads = [&](int ch) { return ((pieces + ch - 1) / ch + 31) / 32 * 32; };
  auto grid = [&](int nt) {
    const long long most = (long long)dev_info().sms * std::max(1, 1024 / nt);
    return (int)std::min(a.rows, most);
  };
  // Few rows: more threads, for the latency; many: two pieces in flight each.
  const bool few = a.rows <= 2 * dev_info().sms;
  if (few && pieces <= 512) return launch_pdl(k_rmsnorm<0, 1, VEC, 512>, a, (int)a.rows, threads(1), 0, stream);
  if (pieces <= 512) return launch_pdl(k_rmsnorm<0, 2, VEC, 256>, a, grid(threads(2)), threads(2), 0, stream);
  if (pieces <= 1024) return launch_pdl(k_rmsnorm<0, 2, VEC, 512>, a, grid(threads(2)), threads(2), 0, stream);
  return launch_pdl(k_rmsnorm<0, 4, VEC, 1024>, a, grid(threads(4)), threads(4), 0, stream);
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
