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
// finds the nsel-th largest and writes the selection in order.
//
// The scores are first taken on the tensor cores, with q+ = max(q, 0) on hi and
// q- = min(q, 0) on lo as one product of 2 D columns: eight blocks and eight
// heads to an instruction, every lane on the bounds that it has copied itself,
// a few steps ahead.
//
// Which of two blocks is selected must not depend on the order of a sum.  An
// instruction of 16 products and the sum so far drops at most 17 2^-23 of the sum
// of the terms' magnitudes M, D / 16 of them for either of q+ hi and q- lo, and
// one addition 2^-24 of it: less than e = 17 D 2^-26 M.  M is taken once per warp,
// of the queries on the largest magnitudes of its blocks' bounds: one instruction
// for two packed numbers in place of a second product for each block (22.4 ->
// 21.1 us for the second case below; 0.2 us more where a warp has one step).
// Blocks that are further than 2 e from the nsel-th largest sum are in or out; the
// others, mostly the nsel-th itself and a few more or none, are decided by sums that
// are exact enough to be the exact value's rounding to fp32: products of fp16
// numbers are exact in fp32, and their sums keep each addition's error (Knuth, "The
// Art of Computer Programming" 2, 4.2.2, theorem B).
//
// Measured (GB300, 8 key-value heads of 128): one sequence of 131072 tokens, 64 of
// 2048 blocks per head, 12.2 us, of them 7.6 scoring 8.4 MB, 1.5 the threshold and
// 3 the exact sums and the writing; 32 sequences of up to 32768 tokens, 64 blocks,
// 21.1 us, of them 17.4 scoring 33.6 MB (14.7 without the products, 9.7 without
// the loads, 5.2 with neither).  Latency bounds the first (one CTA of
// each cluster works behind the scores), the clusters of the longest sequences
// the second.  Larger clusters were slower in both; the table looked up four steps
// at a time gained nothing.
#include <cooperative_groups.h>

#include "q2_attend.cuh"

namespace cg = cooperative_groups;

namespace q2 {
namespace {

__device__ unsigned int q2_select_error;

constexpr int kAtOnce = 8;                          // blocks of a warp's step
constexpr int kBins = 2048;
constexpr int kFew = 64;                            // keys that are ranked by comparing all (some 35 cycles each; a histogram is a microsecond)
constexpr int kMostSmem = 226 * 1024;
constexpr uint32_t kAlways = 0xffffffffu, kOdd = 0xfffffffeu;    // keys of first and last blocks, of scores that are not finite

struct SelectArgs {
  const int* table;
  long long table_stride;
  int npages, page, sub;
  uint32_t page_mul, page_sh;
  const __half* bounds;
  const __half* q;
  long long ldq;
  const int* lens;
  int cap, kv_heads, group, nsel, first, last, cs, stages;
  int* sel;
};

// Shared memory behind the queries' fragments, of a CTA of T threads.
template <int T>
struct SelectShared {
  static constexpr int kWarps = T / 32;
  uint32_t hist[kBins];
  uint32_t wsum[2][kWarps];
  float4 warps[8 * kWarps];                         // of each warp of the cluster: largest sum of magnitudes; least and greatest key, keys kOdd
  uint32_t found[4];
  uint32_t list[T];
};

// (h, e) + (h2, e2), h and e the sum's fp32 value and what it lacks.  (Plain
// operations: h2 may be a product that the compiler fuses into a sum, but only one of
// fp16 numbers, which is exact.)
__device__ __forceinline__ void join(float& h, float& e, float h2, float e2) {
  const float t = h + h2, z = t - h;
  e = (e + e2) + ((h - (t - z)) + (h2 - z));
  h = t;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028235e38f; }

// Larger keys for larger scores; what is not a finite number above them all.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!finite(x)) return kOdd;
  const uint32_t b = __float_as_uint(x + 0.f);      // (-0 as 0)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// An exclusive sum over the CTA's threads of a and b; `total` of them (all threads get them).
template <int T>
__device__ __forceinline__ uint2 scan(SelectShared<T>& s, uint32_t a, uint32_t b, uint2& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  __syncthreads();
  if (lane == 31) {
    s.wsum[0][warp] = x;
    s.wsum[1][warp] = y;
  }
  __syncthreads();
  const uint32_t u = lane < (T / 32) ? s.wsum[0][lane] : 0u, v = lane < (T / 32) ? s.wsum[1][lane] : 0u;
  total.x = __reduce_add_sync(0xffffffffu, u);
  total.y = __reduce_add_sync(0xffffffffu, v);
  const uint32_t p = __reduce_add_sync(0xffffffffu, lane < warp ? u : 0u), q = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
  return make_uint2(x - a + p, y - b + q);
}

// The need-th largest of n keys, `always` of them kAlways, `odds` kOdd and the
// others from lo to hi; `need` becomes how many of those equal to it count among
// the largest (1 <= need <= n).
template <int T>
__device__ uint32_t largest(SelectShared<T>& s, const uint32_t* keys, int n, uint32_t always, uint32_t odds, uint32_t lo,
                            uint32_t hi, uint32_t& need) {
  if (need <= always) return kAlways;
  need -= always;
  if (need <= odds) return kOdd;
  need -= odds;
  // Histograms of even steps over a range that holds the key sought, until few
  // are left in its bin.
  uint32_t left = n - always - odds;                // keys in lo .. hi
  while (left > kFew && lo < hi) {
    const uint32_t span = hi - lo;
    const int shift = max(0, 32 - __clz(span) - 11);                          // (span >> shift) < kBins
    for (int i = threadIdx.x; i < kBins; i += T) s.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += T) {
      const uint32_t k = keys[i];
      if (k >= lo && k <= hi) atomicAdd(&s.hist[(k - lo) >> shift], 1u);
    }
    __syncthreads();
    // from the highest bin down, kBins / T to a thread
    constexpr int each = kBins / T;
    uint32_t c[each], sum = 0;
#pragma unroll
    for (int k = 0; k < each; ++k) sum += c[k] = s.hist[kBins - 1 - (threadIdx.x * each + k)];
    uint2 total;
    uint32_t before = scan(s, sum, 0u, total).x;
    if (before < need && before + sum >= need) {    // in one thread
#pragma unroll
      for (int k = 0; k < each; ++k) {
        if (before < need && before + c[k] >= need) {
          s.found[0] = kBins - 1 - (threadIdx.x * each + k);
          s.found[1] = need - before;
          s.found[2] = c[k];
        }
        before += c[k];
      }
    }
    __syncthreads();
    const uint32_t bin = s.found[0];
    need = s.found[1];
    left = s.found[2];
    lo += bin << shift;
    hi = min(hi, lo + ((1u << shift) - 1u));
    __syncthreads();
  }
  if (lo == hi) return lo;
  // few are left: each counts those above it
  if (threadIdx.x == 0) s.found[3] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += T) {
    const uint32_t k = keys[i];
    if (k >= lo && k <= hi) s.list[atomicAdd(&s.found[3], 1u)] = k;
  }
  __syncthreads();
  if (threadIdx.x < left) {
    const uint32_t k = s.list[threadIdx.x];
    uint32_t above = 0, equal = 0;
    for (uint32_t i = 0; i < left; ++i) {
      above += s.list[i] > k;
      equal += s.list[i] == k;
    }
    if (above < need && need <= above + equal) {    // (all that are equal write the same)
      s.found[0] = k;
      s.found[1] = need - above;
    }
  }
  __syncthreads();
  need = s.found[1];
  const uint32_t k = s.found[0];
  __syncthreads();
  return k;
}

// The exact score of a block, to the rounding to fp32.  By a warp.
template <int D>
__device__ __forceinline__ uint32_t exact_key(const SelectArgs& a, const __half* p, const __half* q) {
  constexpr int CPL = D / 32;
  const int lane = threadIdx.x & 31;
  float lo[CPL], hi[CPL], best = -INFINITY;
#pragma unroll
  for (int k = 0; k < CPL; ++k) {
    lo[k] = __half2float(p[lane + 32 * k]);
    hi[k] = __half2float(p[D + lane + 32 * k]);
  }
#pragma unroll 4
  for (int h = 0; h < a.group; ++h) {
    float x = 0.f, e = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
      const float y = __half2float(q[h * D + lane + 32 * k]);
      join(x, e, y * (y >= 0.f ? hi[k] : lo[k]), 0.f);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) join(x, e, __shfl_xor_sync(0xffffffffu, x, o), __shfl_xor_sync(0xffffffffu, e, o));
    best = fmaxf(best, x + e);
  }
  return key_of(best);
}

// STAGED: bounds by way of shared memory, a.stages - 1 steps ahead
template <int D, int T, bool STAGED>
__global__ void __launch_bounds__(T, 512 / T) k_select(const __grid_constant__ SelectArgs a) {
  constexpr int NB = D / 32, W = T / 32;            // 32 columns each
  constexpr int kStage = kAtOnce * 4 * D;           // bytes of a warp's step
  extern __shared__ __align__(16) unsigned char q2_sel_smem[];
  // q+ and q- in 16-byte pieces: [head tile][32 columns][q+, q-][lane]
  uint4* frag = reinterpret_cast<uint4*>(q2_sel_smem);
  const int tiles = (a.group + 7) / 8;
  SelectShared<T>& s = *reinterpret_cast<SelectShared<T>*>(frag + tiles * NB * 64);
  unsigned char* ring = reinterpret_cast<unsigned char*>(&s + 1);           // [warp][stage][32 columns][lo, hi][lane] of 16 bytes
  uint32_t* keys = reinterpret_cast<uint32_t*>(ring + (STAGED ? W * a.stages * kStage : 0));   // [blocks]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
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
      for (int i = threadIdx.x; i < a.nsel; i += T) sel[i] = i < n ? i : -1;
    return;
  }
  if (a.cs > 1) cluster_arrive();
  const int* trow = a.table + b * a.table_stride;
  const __half* qrows = a.q + b * a.ldq + (long long)kvh * a.group * D;
  auto page_at = [&](int i) {                       // the page of a block's first token; -1 behind the last block
    return i < n ? trow[page_of(a, i * Q2_BLOCK)] : -1;
  };
  auto bounds_of = [&](int i, int page) {
    const int t = i * Q2_BLOCK;
    return a.bounds + (((long long)page * a.sub + (t - page_of(a, t) * a.page) / Q2_BLOCK) * a.kv_heads + kvh) * (2 * D);
  };
  const int stride = a.cs * W * kAtOnce;
  const int first = (rank * W + warp) * kAtOnce;
  // Each lane copies the pieces that it will use: columns 32 c + 8 j .. of block g.
  const uint32_t mine = saddr(ring) + warp * (a.stages * kStage) + lane * 16;
  int m0 = first, mslot = 0, page = page_at(first + g);             // the step to be copied
  uint32_t odds = 0;                                // bit `stage`: block g of it has no page
  auto copy = [&]() {
    if (m0 < n) {
      const bool there = (unsigned)page < (unsigned)a.npages;
      if (m0 + g < n && !there && j == 0) atomicOr(&q2_select_error, Q2_ERR_PAGE);
      odds = (odds & ~(1u << mslot)) | (there ? 0u : 1u << mslot);
      const __half* p = there ? bounds_of(m0 + g, page) + 8 * j : a.bounds;
      const uint32_t d = mine + mslot * kStage;
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        cp16(d + c * 1024, p + 32 * c, there);
        cp16(d + c * 1024 + 512, p + D + 32 * c, there);
      }
      m0 += stride;
      page = page_at(m0 + g);
      mslot = mslot + 1 == a.stages ? 0 : mslot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (STAGED)
    for (int k = 1; k < a.stages; ++k) copy();
  for (int i = threadIdx.x; i < tiles * NB * 32; i += T) {
    const int l = i & 31, head = i / (NB * 32) * 8 + (l >> 2), c = i / 32 % NB;
    uint4 r = make_uint4(0u, 0u, 0u, 0u), up, dn;
    if (head < a.group) r = *reinterpret_cast<const uint4*>(qrows + (long long)head * D + 32 * c + 8 * (l & 3));
    const __half2 zero = __float2half2_rn(0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __half2 x = reinterpret_cast<const __half2*>(&r)[k];
      reinterpret_cast<__half2*>(&up)[k] = __hmax2_nan(x, zero);
      reinterpret_cast<__half2*>(&dn)[k] = __hmin2_nan(x, zero);
    }
    frag[i / 32 * 64 + l] = up;
    frag[i / 32 * 64 + 32 + l] = dn;
  }
  __syncthreads();
  if (a.cs > 1) cluster_wait();                     // the first CTA is there
  uint32_t* to = a.cs > 1 ? cluster.map_shared_rank(keys, 0) : keys;
  float4* warps_to = a.cs > 1 ? cluster.map_shared_rank(s.warps, 0) : s.warps;

  __half2 size[4];                                  // the largest magnitudes of the blocks n0 + g: of columns 8 j .. of any 32
#pragma unroll
  for (int k = 0; k < 4; ++k) size[k] = __float2half2_rn(0.f);
  uint32_t kmin = 0xffffffffu, kmax = 0, kodd = 0;  // keys of this lane's blocks
  int slot = 0;
  for (int n0 = first; n0 < n; n0 += stride) {
    const uint4* held = nullptr;
    const __half* p = nullptr;
    bool there = true;
    if (STAGED) {
      copy();
      if (a.stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
      else if (a.stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 0;" ::: "memory");
      held = reinterpret_cast<const uint4*>(ring + (warp * a.stages + slot) * kStage) + lane;
      there = !(odds >> slot & 1u);
    } else {
      there = (unsigned)page < (unsigned)a.npages;
      if (n0 + g < n && !there && j == 0) atomicOr(&q2_select_error, Q2_ERR_PAGE);
      p = there ? bounds_of(n0 + g, page) + 8 * j : nullptr;
      page = page_at(n0 + stride + g);
    }
    auto piece = [&](int c, int w) {
      return STAGED ? held[c * 64 + w * 32]
             : p    ? *reinterpret_cast<const uint4*>(p + w * D + 32 * c)
                    : make_uint4(0u, 0u, 0u, 0u);
    };
    const uint32_t odd = __ballot_sync(0xffffffffu, !there);       // (lane 4 g + j: block n0 + g)
    float best[2] = {-INFINITY, -INFINITY};         // of blocks n0 + 2j, + 1
    for (int ht = 0; ht < tiles; ++ht) {
      float u[4] = {0.f, 0.f, 0.f, 0.f}, w[4] = {0.f, 0.f, 0.f, 0.f};          // on greatest keys, on least
#pragma unroll (NB < 8 ? NB : 2)
      for (int c = 0; c < NB; ++c) {
        const uint4* f = frag + (ht * NB + c) * 64 + lane;
        const uint4 up = f[0], dn = f[32], y = piece(c, 0), x = piece(c, 1);
        mma(u, up.x, 0u, up.y, 0u, x.x, x.y);
        mma(w, dn.x, 0u, dn.y, 0u, y.x, y.y);
        mma(u, up.z, 0u, up.w, 0u, x.z, x.w);
        mma(w, dn.z, 0u, dn.w, 0u, y.z, y.w);
        if (ht == 0) {
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            size[k] = __hmax2(size[k], __habs2(*reinterpret_cast<const __half2*>(&xs[k])));
            size[k] = __hmax2(size[k], __habs2(*reinterpret_cast<const __half2*>(&ys[k])));
          }
        }
      }
      if (ht * 8 + g < a.group) {                   // rows are heads
#pragma unroll
        for (int e = 0; e < 2; ++e) best[e] = fmaxf(best[e], finite(u[e] + w[e]) ? u[e] + w[e] : INFINITY);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) best[e] = fmaxf(best[e], __shfl_xor_sync(0xffffffffu, best[e], o));
      const int k = n0 + 2 * j + e;
      if (g == 0 && k < n) {
        const uint32_t key = odd >> (8 * j + 4 * e) & 1u ? kOdd : key_of(best[e]);
        const bool always = k < a.first || k >= n - a.last;
        to[k] = always ? kAlways : key;
        kodd += !always && key == kOdd;
        if (!always && key != kOdd) {
          kmin = min(kmin, key);
          kmax = max(kmax, key);
        }
      }
    }
    slot = slot + 1 == a.stages ? 0 : slot + 1;
  }
  // What no sum of magnitudes is above: that of the queries' on the largest ones of
  // these blocks (finite ones: a block with others is not decided by its sum), none
  // of the magnitudes below 2^-14.
  const __half2 least = __float2half2_rn(0x1p-14f);
  uint32_t big[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 z = __hmin2(__hmax2(size[k], least), __float2half2_rn(65504.f));
    big[k] = *reinterpret_cast<const uint32_t*>(&z);
  }
  float most = 0.f;
  for (int ht = 0; ht < tiles; ++ht) {
    float w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NB; ++c) {
      const uint4* f = frag + (ht * NB + c) * 64 + lane;
      const uint4 up = f[0], dn = f[32];            // (one of the two is zero, or both are NaN)
      auto size_of = [&](uint32_t x, uint32_t y) {
        const uint32_t z = (x | y) & 0x7fff7fffu;
        const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&z), least);
        return *reinterpret_cast<const uint32_t*>(&m);
      };
      mma(w, size_of(up.x, dn.x), 0u, size_of(up.y, dn.y), 0u, big[0], big[1]);
      mma(w, size_of(up.z, dn.z), 0u, size_of(up.w, dn.w), 0u, big[2], big[3]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (finite(w[e])) most = fmaxf(most, w[e]);   // (else no block is decided by its sum)
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kodd = __reduce_add_sync(0xffffffffu, kodd);
  if (lane == 0)
    warps_to[rank * W + warp] = make_float4(most, __uint_as_float(kmin), __uint_as_float(kmax), __uint_as_float(kodd));
  if (a.cs > 1) {
    cluster_meet();
    if (rank) return;
  } else {
    __syncthreads();
  }

  // of all warps
  most = 0.f;
  kmin = 0xffffffffu;
  kmax = kodd = 0;
  for (int i = lane; i < a.cs * W; i += 32) {
    const float4 f = s.warps[i];
    most = fmaxf(most, f.x);
    kmin = min(kmin, __float_as_uint(f.y));
    kmax = max(kmax, __float_as_uint(f.z));
    kodd += __float_as_uint(f.w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  kmin = __reduce_min_sync(0xffffffffu, kmin);
  kmax = __reduce_max_sync(0xffffffffu, kmax);
  kodd = __reduce_add_sync(0xffffffffu, kodd);

  // threads have consecutive blocks from here on; of many an odd number, for the
  // banks (2^20 tokens 82 -> 49 us; with 4 of 2048 it cost 0.4)
  const int some = (n + T - 1) / T, each = some > 8 ? some | 1 : some, i0 = min(n, (int)threadIdx.x * each), i1 = min(n, i0 + each);
  uint32_t need = a.nsel, key = largest(s, keys, n, a.first + a.last, kodd, kmin, kmax, need);
  if (key < kOdd) {
    // blocks whose sums lie within the error of the nsel-th
    const float err = 2.f * (17.f * D / 67108864.f) * 1.01f * most, t = score_of(key), top = t + err, bottom = t - err;
    auto near = [&](uint32_t k) { return k < kOdd && score_of(k) <= top && score_of(k) >= bottom; };
    uint32_t in = 0, open = 0;
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = keys[i];
      const bool is = near(k);
      open += is;
      in += !is && k > key;
    }
    uint2 total;
    uint32_t at = scan(s, in, open, total).y;
    need = a.nsel - total.x;                        // of the open ones
    const bool all = total.y == need, few = total.y <= T;
    for (int i = i0; i < i1; ++i) {
      const uint32_t k = keys[i];
      const bool is = near(k);
      if (is && !all && few) s.list[at++] = i;
      keys[i] = is ? 1u : k > key ? kAlways : 0u;
    }
    __syncthreads();
    key = 1;
    if (!all && few) {
      for (uint32_t k = warp; k < total.y; k += W) {
        const int i = s.list[k];
        const uint32_t x = exact_key<D>(a, bounds_of(i, page_at(i)), qrows);
        if (lane == 0) s.hist[k] = x;
      }
      __syncthreads();
      if (threadIdx.x < total.y) {                  // (the list is in the order of the blocks)
        const uint32_t k = s.hist[threadIdx.x];
        uint32_t before = 0;
        for (uint32_t i = 0; i < total.y; ++i) before += s.hist[i] > k || (s.hist[i] == k && i < threadIdx.x);
        keys[s.list[threadIdx.x]] = before < need ? kAlways : 0u;
      }
      __syncthreads();
    } else if (!all) {
      uint32_t greatest = 0;
      for (int k = warp * 32; k < n; k += T) {
        uint32_t todo = __ballot_sync(0xffffffffu, k + lane < n && keys[k + lane] == 1u);
        while (todo) {
          const int i = k + __ffs(todo) - 1;
          todo &= todo - 1;
          const uint32_t x = exact_key<D>(a, bounds_of(i, page_at(i)), qrows);
          greatest = max(greatest, x);
          __syncwarp();
          if (lane == 0) keys[i] = x;               // (above 1)
        }
      }
      if (lane == 0) s.wsum[1][warp] = greatest;
      __syncthreads();
      greatest = __reduce_max_sync(0xffffffffu, lane < W ? s.wsum[1][lane] : 0u);
      __syncthreads();
      need = a.nsel;
      key = largest(s, keys, n, total.x, 0u, 0u, greatest, need);
    }
  }

  // in order: all above the key, and the first `need` of those that have it
  uint32_t above = 0, equal = 0;
  for (int i = i0; i < i1; ++i) {
    above += keys[i] > key;
    equal += keys[i] == key;
  }
  uint2 total;
  uint2 run = scan(s, above, equal, total);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = keys[i];
    if (k > key || (k == key && run.y < need)) sel[run.x + min(run.y, need)] = i;
    run.x += k > key;
    run.y += k == key;
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
  // Up to eight CTAs to a cluster where the clusters leave SMs idle and there are
  // steps for their warps.  With few clusters and some blocks CTAs of 512 threads,
  // one per SM (4 sequences of 65536 tokens and 8 heads: 12.3 us, 15.2 of 256
  // threads; 8 of 32768: 11.9 and 11.5; one of 4096: 6.6 and 6.0).  Eight to a
  // cluster only where they leave half of the SMs: all may not find room at once
  // (2 sequences of 131072: 18.2 us, 16.7 with four).
  const int blocks = (int)((c.cap + Q2_BLOCK - 1) / Q2_BLOCK), clusters = batch * c.kv_heads;
  auto launch = [&](auto kernel, int T, int D, int shared, bool staged) {
    a.cs = 1;
    while (a.cs < 8 && (long long)clusters * a.cs * 2 * T <= (a.cs == 4 ? 256ll : 512ll) * dev_info().sms &&
           blocks >= 2 * a.cs * (T / 32) * kAtOnce)
      a.cs *= 2;
    const int smem = (a.group + 7) / 8 * (D / 32) * 1024 + shared + blocks * 4;
    const int stage = T / 32 * kAtOnce * 4 * D, room = (T == 512 ? kMostSmem : kMostSmem / 2) - smem;
    a.stages = staged ? std::max(1, std::min(3, room / stage)) : 0;
    const int bytes = smem + a.stages * stage;
    if (staged && bytes > kMostSmem) return (int)Q2_ESIZE;         // (for the form that holds no stages)
    if (set_smem(reinterpret_cast<const void*>(kernel), bytes)) return (int)Q2_ECUDA;
    return launch_clusters(kernel, clusters, a.cs, T, bytes, stream, a);
  };
  auto with = [&](auto Dc) {
    constexpr int D = Dc();
    int st = Q2_ESIZE;
    if constexpr (D <= 128)
      if (clusters * 4 <= dev_info().sms && blocks > 256) st = launch(k_select<D, 512, true>, 512, D, sizeof(SelectShared<512>), true);
    if (st == Q2_ESIZE) st = launch(k_select<D, 256, true>, 256, D, sizeof(SelectShared<256>), true);
    return st == Q2_ESIZE ? launch(k_select<D, 256, false>, 256, D, sizeof(SelectShared<256>), false) : st;
  };
  return c.D == 64    ? with(std::integral_constant<int, 64>())
         : c.D == 128 ? with(std::integral_constant<int, 128>())
                      : with(std::integral_constant<int, 256>());
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
