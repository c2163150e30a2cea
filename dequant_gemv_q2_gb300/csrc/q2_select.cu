// The blocks of 64 tokens that promise the most to a token's queries: with the
// least and greatest key of a block, lo and hi, no key in it can give query q
// more than
//
//   U = sum_d max(q_d lo_d, q_d hi_d)
//
// and of the blocks of a (sequence, key-value head) the nsel with the largest U
// of any of the head's queries are selected.  Reads 4 D bytes per block and
// head, a 32nd of the block's own in fp16, and multiplies each (query head,
// block, column) once.
//
// One cluster per (sequence, key-value head).  Its CTAs share out the blocks,
// score them and leave the scores in the shared memory of the first, which
// finds the nsel-th largest by its digits (three histograms) and writes the
// selection in order.
//
// Which of two blocks is selected must not depend on the order of a sum, so U
// is summed exactly enough to be the exact value's rounding to fp32.  Products
// of fp16 numbers are exact in fp32.  A lane adds its columns to a number M
// above 2^log2(columns) times any of them, so that every sum s = fl(s' + p) has
// the same exponent: s - s' and p - (s - s') are exact, the first parts add up
// without error in s, the second in a sum of their own.  Lanes join pairs of
// sums with the error of the larger added to the smaller (Knuth, "The Art of
// Computer Programming" 2, 4.2.2, theorem B).
#include <cooperative_groups.h>

#include "q2_page.cuh"

namespace cg = cooperative_groups;

namespace q2 {
namespace {

__device__ unsigned int q2_select_error;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kAtOnce = 4;                          // blocks of a warp's step
constexpr int kBins = 2048;                         // of a histogram: 11, 11 and 10 bits of a key

struct SelectArgs {
  const int* table;
  long long table_stride;
  int npages, page, sub;
  uint32_t page_mul, page_sh;
  const __half* bounds;
  const __half* q;
  long long ldq;
  const int* lens;
  int cap, kv_heads, group, nsel, first, last, cs;
  int* sel;
};

// (h, e) + (h2, e2), h and e the sum's fp32 value and what it lacks
__device__ __forceinline__ void join(float& h, float& e, float h2, float e2) {
  const float t = h + h2, z = t - h;
  e = (e + e2) + ((h - (t - z)) + (h2 - z));
  h = t;
}

template <int N>
__device__ __forceinline__ void halves(const __half* p, float (&x)[N]) {
  if constexpr (N == 2) {
    const __half2 r = *reinterpret_cast<const __half2*>(p);
    const float2 f = __half22float2(r);
    x[0] = f.x;
    x[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint2 r = *reinterpret_cast<const uint2*>(p + i);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.x)), g = __half22float2(*reinterpret_cast<const __half2*>(&r.y));
      x[i] = f.x;
      x[i + 1] = f.y;
      x[i + 2] = g.x;
      x[i + 3] = g.y;
    }
  }
}

// The exponent field of a bound above every |x| (of 2^-25 at least, 2^16 at most)
template <int N>
__device__ __forceinline__ uint32_t exponent(const float (&x)[N], uint32_t least) {
#pragma unroll
  for (int i = 0; i < N; ++i) least = max(least, __float_as_uint(x[i]) >> 23 & 255u);
  return min(least, 143u);
}

// Larger keys for larger scores; what is not a finite number above them all.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(fabsf(x) <= 3.4028235e38f)) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(x + 0.f);      // (-0 as 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

template <int D>
__global__ void __launch_bounds__(kThreads) k_select(const __grid_constant__ SelectArgs a) {
  constexpr int CPL = D / 32;                       // columns of a lane
  constexpr uint32_t kBits = CPL == 2 ? 1 : CPL == 4 ? 2 : 3;
  extern __shared__ __align__(16) unsigned char q2_sel_smem[];
  float* qs = reinterpret_cast<float*>(q2_sel_smem);                        // [group][32][CPL]
  uint32_t* qe = reinterpret_cast<uint32_t*>(qs + a.group * D);             // [group][32] exponents
  uint32_t* hist = qe + a.group * 32;                                       // [kBins]
  uint32_t* keys = hist + kBins;                                            // [blocks] of the first CTA
  __shared__ uint32_t wsum[2][kWarps];
  __shared__ uint32_t found[2];                     // digits so far, how many more are above
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = a.cs == 1 ? 0 : (int)cluster.block_rank();
  const int id = blockIdx.x / a.cs, b = id / a.kv_heads, kvh = id - b * a.kv_heads;

  pdl_wait();
  pdl_trigger();
  int len = a.lens[b];
  if (len < 0 || len > a.cap) {
    if (rank == 0 && kvh == 0 && threadIdx.x == 0) atomicOr(&q2_select_error, Q2_ERR_LENGTH);
    len = 0;
  }
  const int n = (len + Q2_BLOCK - 1) / Q2_BLOCK;
  int* sel = a.sel + (long long)id * a.nsel;
  if (n <= a.nsel) {                                // all there are
    if (rank == 0)
      for (int i = threadIdx.x; i < a.nsel; i += kThreads) sel[i] = i < n ? i : -1;
    return;
  }
  if (a.cs > 1) cluster_arrive();
  for (int i = threadIdx.x; i < a.group * 32; i += kThreads) {
    float x[CPL];
    halves<CPL>(a.q + b * a.ldq + (long long)kvh * a.group * D + i * CPL, x);
#pragma unroll
    for (int k = 0; k < CPL; ++k) qs[i * CPL + k] = x[k];
    qe[i] = exponent<CPL>(x, 102u);
  }
  __syncthreads();
  if (a.cs > 1) cluster_wait();                     // the first CTA is there
  uint32_t* to = a.cs > 1 ? cluster.map_shared_rank(keys, 0) : keys;

  const int* trow = a.table + b * a.table_stride;
  const int step = a.cs * kWarps * kAtOnce;
  for (int n0 = (rank * kWarps + warp) * kAtOnce; n0 < n; n0 += step) {
    // lanes 0..3: the places of the blocks' bounds
    int place = -1;
    if (lane < kAtOnce && n0 + lane < n) {
      const int t = (n0 + lane) * Q2_BLOCK, pi = page_of(a, t), page = trow[pi];
      if ((unsigned)page < (unsigned)a.npages) place = page * a.sub + (t - pi * a.page) / Q2_BLOCK;
      else atomicOr(&q2_select_error, Q2_ERR_PAGE);
    }
    float lo[kAtOnce][CPL], hi[kAtOnce][CPL];
    uint32_t be[kAtOnce];
    bool there[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int at = __shfl_sync(0xffffffffu, place, u);
      there[u] = at >= 0;
      const __half* p = a.bounds + ((long long)max(at, 0) * a.kv_heads + kvh) * (2 * D) + lane * CPL;
      if (there[u]) {
        halves<CPL>(p, lo[u]);
        halves<CPL>(p + D, hi[u]);
      } else {
#pragma unroll
        for (int k = 0; k < CPL; ++k) lo[u][k] = hi[u][k] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) be[u] = exponent<CPL>(lo[u], exponent<CPL>(hi[u], 102u));

    float best = -INFINITY;
    bool odd = false;                               // a score that is not a finite number
    for (int h = 0; h < a.group; ++h) {
      float q[CPL];
      const float* qp = qs + (h * 32 + lane) * CPL;
      if constexpr (CPL == 2) {
        const float2 f = *reinterpret_cast<const float2*>(qp);
        q[0] = f.x;
        q[1] = f.y;
      } else {
#pragma unroll
        for (int k = 0; k < CPL; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(qp + k);
          q[k] = f.x;
          q[k + 1] = f.y;
          q[k + 2] = f.z;
          q[k + 3] = f.w;
        }
      }
      const uint32_t me = qe[h * 32 + lane];
      float s[kAtOnce], e[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const float M = __uint_as_float((me + be[u] - 124u + kBits) << 23 | 0x400000u);
        float acc = M;
        e[u] = 0.f;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
          const float y = q[k] >= 0.f ? hi[u][k] : lo[u][k];
          const float t = fmaf(q[k], y, acc), z = t - acc;
          e[u] += fmaf(q[k], y, -z);
          acc = t;
        }
        s[u] = acc - M;
      }
      // lanes' sums joined, four blocks at a time: two exchanges leave a lane one block, three more its sum
#pragma unroll
      for (int o = 16, w = kAtOnce / 2; w > 0; o >>= 1, w >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int u = 0; u < w; ++u) {
          const float hs = __shfl_xor_sync(0xffffffffu, up ? s[u] : s[u + w], o);
          const float es = __shfl_xor_sync(0xffffffffu, up ? e[u] : e[u + w], o);
          if (up) {
            s[u] = s[u + w];
            e[u] = e[u + w];
          }
          join(s[u], e[u], hs, es);
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const float hs = __shfl_xor_sync(0xffffffffu, s[0], o), es = __shfl_xor_sync(0xffffffffu, e[0], o);
        join(s[0], e[0], hs, es);
      }
      const float v = s[0] + e[0];
      odd = odd || !(fabsf(v) <= 3.4028235e38f);
      best = fmaxf(best, v);
    }
    // lane 8 u holds block u in the order of the exchanges: bit 4 took the upper two, bit 3 the upper one
    const int u = lane >> 3, i = n0 + u;
    if ((lane & 7) == 0 && i < n) {
      bool mine = false;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) mine = k == u ? there[k] : mine;
      to[i] = i < a.first || i >= n - a.last ? 0xffffffffu : odd || !mine ? 0xfffffffeu : key_of(best);
    }
  }
  if (a.cs > 1) {
    cluster_meet();
    if (rank) return;
  } else {
    __syncthreads();
  }

  // the nsel-th largest key, digit by digit
  uint32_t prefix = 0, need = a.nsel;               // keys with the digits so far: how many of them are to be taken
  for (int shift = 21; ; shift = shift == 21 ? 10 : 0) {
    const int bits = shift == 0 ? 10 : 11, bins = 1 << bits;
    for (int i = threadIdx.x; i < bins; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint32_t k = keys[i];
      if (shift == 21 || (k >> (shift + bits)) == (prefix >> (shift + bits))) atomicAdd(&hist[k >> shift & (bins - 1)], 1u);
    }
    __syncthreads();
    // counts from the highest bin down: thread t has bins [t * each, (t + 1) * each) of that order
    const int each = bins / kThreads;
    uint32_t sum = 0;
    for (int k = 0; k < each; ++k) sum += hist[bins - 1 - (threadIdx.x * each + k)];
    uint32_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += x;
    }
    if (lane == 31) wsum[0][warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run += wsum[0][w];
    uint32_t before = run - sum;
    if (before < need && run >= need) {             // in one thread
      for (int k = 0; k < each; ++k) {
        const uint32_t d = bins - 1 - (threadIdx.x * each + k), c = hist[d];
        if (before + c >= need) {
          found[0] = prefix | d << shift;
          found[1] = need - before;
          break;
        }
        before += c;
      }
    }
    __syncthreads();
    prefix = found[0];
    need = found[1];
    if (shift == 0) break;
  }

  // in order: all above the key, and the first `need` of those that have it
  const int each = (n + kThreads - 1) / kThreads, i0 = min(n, (int)threadIdx.x * each), i1 = min(n, i0 + each);
  uint32_t above = 0, equal = 0;
  for (int i = i0; i < i1; ++i) {
    above += keys[i] > prefix;
    equal += keys[i] == prefix;
  }
  uint32_t ra = above, re = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, ra, o), y = __shfl_up_sync(0xffffffffu, re, o);
    if (lane >= o) {
      ra += x;
      re += y;
    }
  }
  if (lane == 31) {
    wsum[0][warp] = ra;
    wsum[1][warp] = re;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    ra += wsum[0][w];
    re += wsum[1][w];
  }
  ra -= above;
  re -= equal;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = keys[i];
    if (k > prefix || (k == prefix && re < need)) sel[ra + min(re, need)] = i;
    ra += k > prefix;
    re += k == prefix;
  }
}

int select(const Pages& pg, const CacheShape& c, const void* bounds, const void* q, long long ldq, const int* lens,
           int batch, int q_heads, int nsel, int first, int last, int* sel, void* stream) {
  if (batch < 0 || batch > Q2_ATT_MAX_BATCH || q_heads < 1 || q_heads % c.kv_heads || q_heads / c.kv_heads > Q2_ATT_MAX_GROUP)
    return Q2_ESHAPE;
  if (nsel < 1 || nsel > Q2_MAX_BLOCKS || first < 0 || last < 0 || (long long)first + last > nsel) return Q2_ESHAPE;
  if (c.page % Q2_BLOCK && Q2_BLOCK % c.page) return Q2_ESHAPE;
  if (c.cap > (long long)Q2_MAX_BLOCKS * Q2_BLOCK) return Q2_ESHAPE;
  if (batch == 0) return Q2_OK;
  if (!bounds || !q || !lens || !sel) return Q2_EINVAL;
  if (batch > 1 && ldq < (long long)q_heads * c.D) return Q2_ESHAPE;
  if (misaligned(bounds, 16) || misaligned(q, 16) || misaligned(lens, 4) || misaligned(sel, 4) || (batch > 1 && ldq % 8))
    return Q2_EALIGN;
  SelectArgs a = {};
  a.table = pg.table;
  a.table_stride = pg.table_stride;
  a.npages = pg.npages;
  a.page = pg.page;
  a.sub = (pg.page + Q2_BLOCK - 1) / Q2_BLOCK;
  a.page_mul = pg.page_mul;
  a.page_sh = pg.page_sh;
  a.bounds = static_cast<const __half*>(bounds);
  a.q = static_cast<const __half*>(q);
  a.ldq = ldq;
  a.lens = lens;
  a.cap = (int)c.cap;
  a.kv_heads = c.kv_heads;
  a.group = q_heads / c.kv_heads;
  a.nsel = nsel;
  a.first = first;
  a.last = last;
  a.sel = sel;
  // CTAs of a cluster: two per SM in all, while each has a step for its warps
  const int blocks = (int)((c.cap + Q2_BLOCK - 1) / Q2_BLOCK), clusters = batch * c.kv_heads;
  a.cs = 1;
  while (a.cs < 8 && (long long)clusters * a.cs * 2 <= 2 * dev_info().sms && blocks >= 2 * a.cs * kWarps * kAtOnce) a.cs *= 2;
  const int smem = a.group * (c.D + 32) * 4 + (kBins + blocks) * 4;
  auto launch = [&](auto kernel) {
    if (set_smem(reinterpret_cast<const void*>(kernel), smem)) return (int)Q2_ECUDA;
    return launch_clusters(kernel, clusters, a.cs, kThreads, smem, stream, a);
  };
  return c.D == 64 ? launch(k_select<64>) : c.D == 128 ? launch(k_select<128>) : launch(k_select<256>);
}

}  // namespace
}  // namespace q2

using namespace q2;

extern "C" int q2_select(const q2_kv* kv, const void* bounds, const void* q, long long ldq, const int* lens, int batch,
                         int q_heads, int nsel, int first, int last, int* sel, q2_stream stream) {
  Pages pg;
  CacheShape c;
  const int st = check_cache(kv, batch, pg, c);
  return st ? st : select(pg, c, bounds, q, ldq, lens, batch, q_heads, nsel, first, last, sel, stream);
}

extern "C" int q2_select4(const q2_kv4* kv, const void* bounds, const void* q, long long ldq, const int* lens, int batch,
                          int q_heads, int nsel, int first, int last, int* sel, q2_stream stream) {
  Pages pg, sp;
  CacheShape c;
  const int st = check_cache4(kv, batch, pg, sp, c);
  return st ? st : select(pg, c, bounds, q, ldq, lens, batch, q_heads, nsel, first, last, sel, stream);
}

// The error word of this kernel, then cleared (q2_device_errors).
extern "C" int q2_select_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_select_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_select_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
