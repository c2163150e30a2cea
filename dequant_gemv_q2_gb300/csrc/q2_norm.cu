// Root-mean-square norm of rows, with the residual's addition in front and an
// fp16 and/or an 8-bit output behind it: what runs ahead of each projection
// of a decode step.  Per row of C values,
//
//   h = x + r,   y = h * w / sqrt(mean(h^2) + eps),
//   r' = fp16(h),  y16 = fp16(y),  s = max|y| / 127,  y8 = rint(y / s),
//
// all in fp32 from the fp16 inputs; h, y and s are each rounded once.  The sum
// of squares is a tree over the row's threads in an order that follows from the
// width, from whether all rows lie on 16-byte boundaries, and there, up to 4096
// columns, from whether there are more rows than SMs; nothing else changes it.
//
// A row is read once and stays in registers between the sum, the maximum and
// the stores, so the bytes of the inputs and outputs are all that moves.  Rows
// of up to 512 columns take 16 or 32 threads each (a reduction is five
// shuffles, no barrier); longer ones a block, which goes on to further rows
// with the next row's loads in flight during the reductions of the one before.
//
// 16384 rows of 4096 with residual and both outputs: 107 us on the device, 5.6
// of the 6.8 TB/s that a copy reaches (one row per block and no row ahead:
// 164).  One row of 4096: 1.6 us, which is a launch, one trip to memory and
// one block reduction; 64 rows of 5120 to 8 bits 2.3.
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

// 16 bytes that begin m bytes (even) into the 32 of a and b.
__device__ __forceinline__ uint4 cut16(const uint4& a, const uint4& b, uint32_t m) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t t[6], u[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) t[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) u[i] = m & 4 ? t[i + 1] : t[i];
  const uint32_t s = (m & 2) * 8;
  return make_uint4(__funnelshift_r(u[0], u[1], s), __funnelshift_r(u[1], u[2], s), __funnelshift_r(u[2], u[3], s),
                    __funnelshift_r(u[3], u[4], s));
}
// 8 bytes that begin m bytes into the 16 of a and b.
__device__ __forceinline__ uint2 cut8(const uint2& a, const uint2& b, uint32_t m) {
  const uint32_t w0 = m & 4 ? a.y : a.x, w1 = m & 4 ? b.x : a.y, w2 = m & 4 ? b.y : b.x, s = (m & 3) * 8;
  return make_uint2(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s));
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t pack4(const float* r) {
  auto w = [&](int i) { return __float_as_uint(r[i]); };
  return __byte_perm(__byte_perm(w(0), w(1), 0x0040), __byte_perm(w(2), w(3), 0x0040), 0x5410);
}

// One thread's share of a row: CH pieces of 8 columns, in turn with the row's
// other nt - 1 threads.  VEC: a piece is one 16-byte access.  Otherwise rows
// may begin anywhere: a piece is cut out of two 16-byte loads, and written
// through shared memory in pieces of 16 bytes as they lie in global memory;
// the ends of a row go element by element (4096 rows of 5125 columns with
// residual 50 us, with both outputs 69.5; 91 to fp16 with every element by
// itself; 16 rows of 3001, where only the latency counts, 3.6 and 2.7).  A
// thread's columns, and with them the order of the sums, do not depend on where
// such a row begins.  A block's threads spill 64 bytes at their 32 registers,
// beyond 8192 columns 204 at 64; on 16-byte boundaries 144 there (2048 rows of
// 17408 with residual 72 us, 4.0 TB/s), nothing up to 8192.
template <int TPR, int CH, bool VEC>
struct Row {
  int tid, nt, C;
  bool live;
  __device__ __forceinline__ int col(int c) const { return (c * nt + tid) * 8; }
  __device__ __forceinline__ static void sync() {
    if (TPR) __syncwarp();
    else __syncthreads();
  }

  __device__ __forceinline__ void load(const __half* p, uint4 (&r)[CH]) const {
    const uint32_t m = VEC ? 0 : (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = col(c);
      r[c] = make_uint4(0, 0, 0, 0);
      if (!live || k >= C) continue;
      if (VEC || (m == 0 && k + 8 <= C)) {
        r[c] = *reinterpret_cast<const uint4*>(p + k);
      } else if (m && k > 0 && k + 16 <= C) {          // both loads lie inside the row
        const uint4* from = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p + k) - m);
        r[c] = cut16(from[0], from[1], m);
      } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(&r[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i < C) h[i] = reinterpret_cast<const uint16_t*>(p)[k + i];
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
  // buf: the row's place in shared memory (not VEC), 8 columns to an element
  __device__ __forceinline__ void store(__half* p, const float (&v)[CH][8], uint4* buf) const {
    const uint32_t m = VEC ? 0 : (uint32_t)reinterpret_cast<uintptr_t>(p) & 15u;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = col(c);
      uint4 raw;
      __half2* h2 = reinterpret_cast<__half2*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) h2[i] = __floats2half2_rn(v[c][2 * i], v[c][2 * i + 1]);
      if (!live || k >= C) continue;
      if (VEC || (m == 0 && k + 8 <= C)) *reinterpret_cast<uint4*>(p + k) = raw;
      else buf[k / 8] = raw;
    }
    if (VEC) return;
    sync();
    if (!live) return;
    for (int g = m ? tid : C / 8; g * 8 < C + (int)m / 2; g += m ? nt : C) {   // columns k .. k + 7 (m == 0: the last ones)
      const int k = g * 8 - (int)m / 2;
      if (m && k >= 0 && k + 8 <= C) {
        *reinterpret_cast<uint4*>(p + k) = cut16(buf[g - 1], buf[g], 16 - m);
      } else if (m || tid == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i >= 0 && k + i < C) p[k + i] = reinterpret_cast<const __half*>(buf)[k + i];
      }
    }
  }
  // rint(v / s), to the last step.  t = v * inv, inv = 127 / max, is within
  // 2^-15 of v / s (three roundings of numbers up to 127), so it only leaves
  // open what is within kNear of a tie T = n + 1/2; there the sign of v - T s,
  // which one fma gives exactly, decides.  (64 rows of 5120 2.31 us; with a
  // division there 2.56.)  The other integers are the low bits of t + 1.5 2^23.
  // Rows that are not finite (inv 0) give 0 where v is not.
  __device__ __forceinline__ void store8(int8_t* p, const float (&v)[CH][8], float s, float inv, uint2* buf) const {
    constexpr float kRint = 12582912.f, kNear = 1.f / 32768.f;
    constexpr int kGroup = VEC ? 8 : 2;            // values to a test: two where registers are short
    const uint32_t m = VEC ? 0 : (uint32_t)reinterpret_cast<uintptr_t>(p) & 7u;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int k = col(c);
      float r[8];
#pragma unroll
      for (int g = 0; g < 8; g += kGroup) {
        float far = 0.f;                           // largest distance from an integer
#pragma unroll
        for (int i = g; i < g + kGroup; ++i) {
          const float t = v[c][i] * inv;
          r[i] = t + kRint;
          far = fmaxf(far, fabsf(t - (r[i] - kRint)));
        }
        if (far > 0.5f - kNear || inv == 0.f) {
#pragma unroll
          for (int i = g; i < g + kGroup; ++i) {
            const float x = v[c][i], t = x * inv, q = r[i] - kRint, d = t - q, T = q + copysignf(0.5f, d);
            const float e = fmaf(-T, s, x);
            r[i] = __int_as_float(__float2int_rn(fabsf(d) > 0.5f - kNear ? T + (e == 0.f ? 0.f : copysignf(0.5f, e)) : t));
          }
        }
      }
      const uint32_t lo = pack4(r), hi = pack4(r + 4);
      if (!live || k >= C) continue;
      if (VEC || (m == 0 && k + 8 <= C)) *reinterpret_cast<uint2*>(p + k) = make_uint2(lo, hi);
      else buf[k / 8] = make_uint2(lo, hi);
    }
    if (VEC) return;
    sync();
    if (!live) return;
    for (int g = m ? tid : C / 8; g * 8 < C + (int)m; g += m ? nt : C) {
      const int k = g * 8 - (int)m;
      if (m && k >= 0 && k + 8 <= C) {
        *reinterpret_cast<uint2*>(p + k) = cut8(buf[g - 1], buf[g], 8 - m);
      } else if (m || tid == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (k + i >= 0 && k + i < C) p[k + i] = reinterpret_cast<const int8_t*>(buf)[k + i];
      }
    }
  }
};

// Shared memory of a block of `rows` rows: the outputs' images (not VEC).
template <bool VEC>
int norm_smem(const NormArgs& a, int rows) {
  if (VEC) return 0;
  const int pieces = (a.C + 7) / 8;
  return rows * pieces * ((a.res_out ? 16 : 0) + (a.y ? 16 : 0) + (a.y8 ? 8 : 0));
}

// Blocks that have to fit an SM: the grid counts on them where a block takes
// every gridDim.x-th row.
template <int TPR, int CH, bool VEC, int NT>
constexpr int norm_ctas() { return TPR ? 0 : VEC ? (CH == 2 ? 1024 / NT : 0) : (CH > 1 ? 0 : 2048 / NT); }

// TPR: threads per row (16 or 32, several rows per block; 0: a block per row,
// then every gridDim.x-th).  NT: threads of a block at most.
template <int TPR, int CH, bool VEC, int NT>
__global__ void __launch_bounds__(NT, norm_ctas<TPR, CH, VEC, NT>()) k_rmsnorm(const __grid_constant__ NormArgs a) {
  // Rows ahead: where the registers hold them (wider rows wait for theirs, rows
  // that may begin anywhere leave it to the other blocks of their SM).
  constexpr bool AHEAD = VEC && TPR == 0 && CH <= 2;
  __shared__ float psum[2][32];
  __shared__ uint32_t pmax[2][32];
  extern __shared__ __align__(16) unsigned char q2_norm_smem[];
  Row<TPR, CH, VEC> me;
  me.nt = TPR ? TPR : blockDim.x;
  me.tid = TPR ? threadIdx.x % (TPR ? TPR : 1) : threadIdx.x;
  me.C = a.C;
  long long row = TPR ? (long long)blockIdx.x * (256 / (TPR ? TPR : 1)) + threadIdx.x / (TPR ? TPR : 1)
                      : (long long)blockIdx.x;
  me.live = !TPR || row < a.rows;
  // the images of this row's outputs: all rows' sums, then y, then y8
  const int pieces = (a.C + 7) / 8, rows = TPR ? 256 / (TPR ? TPR : 1) : 1, at = TPR ? threadIdx.x / (TPR ? TPR : 1) : 0;
  uint4* hbuf = reinterpret_cast<uint4*>(q2_norm_smem) + at * pieces;
  uint4* ybuf = hbuf + (a.res_out ? rows * pieces : 0);
  uint2* qbuf = reinterpret_cast<uint2*>(q2_norm_smem) + ((a.res_out ? 2 : 0) + (a.y ? 2 : 0)) * rows * pieces + at * pieces;
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
    if (a.res_out) me.store(a.res_out + (size_t)row * a.C, h, hbuf);
    const float d = ss / (float)a.C + a.eps, k = d == 0.f ? 0.f : rsqrtf(d);   // eps = 0: zeros for a row of zeros
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      me.floats(wr[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = h[c][i] * k * w[i];
    }
    if (a.y) me.store(a.y + place(row, a.ldy), h, ybuf);
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
      const float scale = top / 127.f;
      if (me.live && me.tid == 0) a.s8[row] = scale;
      me.store8(a.y8 + (size_t)row * a.C, h, scale, top > 0.f ? 127.f / top : 0.f, qbuf);
    }
    if (TPR || next >= a.rows) return;
    row = next;
    if (!AHEAD) {
      me.load(a.x + place(row, a.ldx), xr);
      if (a.res) me.load(a.res + (size_t)row * a.C, rr);
    }
  }
}

template <int TPR, int CH, bool VEC, int NT>
int launch_rows(const NormArgs& a, int grid, int threads, void* stream) {
  return launch_pdl(k_rmsnorm<TPR, CH, VEC, NT>, a, grid, threads, norm_smem<VEC>(a, TPR ? 256 / (TPR ? TPR : 1) : 1), stream);
}

template <bool VEC>
int launch_norm(const NormArgs& a, void* stream) {
  const int pieces = (a.C + 7) / 8;
  auto blocks = [&](int per) { return (int)((a.rows + per - 1) / per); };
  // Short rows by half warps and warps (64 x 40 rows of 128: 1.6 us, 2.9 with
  // a block per row; 4096 rows of 512 with residual: 3.0 and 4.5; a few rows
  // of 512 1.9 and 1.8).
  if (pieces <= 16) return launch_rows<16, 1, VEC, 256>(a, blocks(16), 256, stream);
  if (pieces <= 32) return launch_rows<32, 1, VEC, 256>(a, blocks(8), 256, stream);
  if (pieces <= 64) return launch_rows<32, 2, VEC, 256>(a, blocks(8), 256, stream);
  // A block per row, up to as many blocks as fit 1024 threads on every SM; rows
  // that may begin anywhere, which have more barriers, 2048 threads of 32
  // registers (4096 rows of 5125: 50 us, 72 with 1024 threads).
  auto threads = [&](int ch) { return ((pieces + ch - 1) / ch + 31) / 32 * 32; };
  auto grid = [&](int nt) {
    const long long most = (long long)dev_info().sms * std::max(1, (VEC ? 1024 : 2048) / nt);
    return (int)std::min(a.rows, most);
  };
  if (!VEC && pieces <= 256) return launch_rows<0, 1, false, 256>(a, grid(threads(1)), threads(1), stream);
  if (!VEC && pieces <= 512) return launch_rows<0, 1, false, 512>(a, grid(threads(1)), threads(1), stream);
  if (!VEC && pieces <= 1024) return launch_rows<0, 1, false, 1024>(a, grid(threads(1)), threads(1), stream);
  if (!VEC) return launch_rows<0, 4, false, 1024>(a, grid(threads(4)), threads(4), stream);
  // Few rows: more threads, for the latency (1 or 64 rows of 4096: 1.71 us,
  // 1.78 with two pieces per thread); many: two pieces in flight each (600
  // rows with residual 3.2 us, 3.9 with one).
  const bool few = a.rows <= dev_info().sms;
  if (few && pieces <= 512) return launch_rows<0, 1, true, 512>(a, (int)a.rows, threads(1), stream);
  if (pieces <= 512) return launch_rows<0, 2, true, 256>(a, grid(threads(2)), threads(2), stream);
  if (pieces <= 1024) return launch_rows<0, 2, true, 512>(a, grid(threads(2)), threads(2), stream);
  return launch_rows<0, 4, true, 1024>(a, grid(threads(4)), threads(4), stream);
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
