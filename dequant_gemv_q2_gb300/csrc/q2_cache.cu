// The paged key-value cache's rows: new tokens in (q2_append, q2_append4), with
// the position rotation on the way, and tokens out (q2_read, q2_read4).
//
// A token's pairs of columns are turned by its position's angles,
//
//   (a, b) -> (a cos - b sin, b cos + a sin),
//
// and keys go to the cache in fp16, or in 4 bits (offset and step per group of
// 32 or 64 columns: least value m, range / 15 = s, code rint((x - m) / s)).
// Every row is read and written once: a row's head is 16 bytes per lane, 8, 16 or
// 32 lanes (a slot); the partner of a column is in another lane of the same row (a
// shuffle) or in the next register.
//
// Work is cut into tiles: the new tokens of one block of 64 positions (of 8 at
// least where no bounds are kept) of one sequence, times a few heads of one kind
// (queries, keys or values).  The slots of a CTA take tokens side by side as far as
// there are any, and heads with the rest; where bounds are kept, all heads first,
// so that a slot's keys are of one head.
// Tiles are cut at blocks so that a block's bounds (least and greatest key per
// column) are one CTA's: no atomics, and what a block held before is read only
// where it goes on.
//
// Measured (GB300, 32 or 40 query heads, 8 key-value heads of 128):
//   - one token, fp16: 2.2 us, a launch and one trip to memory.
//   - 64 sequences' token each into 4 bits and out again: 5.6 us, two of those.
//   - four prompts, 16384 tokens in all, fp16, with bounds: 78.6 us, 5.2 TB/s of
//     the 6.8 of a copy.  2.7 instructions per cycle: the exact products of the
//     keys, the bounds; three CTAs of 80 registers per SM.
//   - the same into 4 bits in groups of 64: 104 us, 3.5 TB/s (100 without bounds):
//     instructions, the exact products and some 6 per code.  Out again 37.5 us, 2.3
//     TB/s: every thread finds sequence, length and page of its 16 bytes anew.  16384
//     tokens out of fp16 30 us, 4.4 TB/s.
//
// The bounds and the codes decide by comparison what later calls read, so keys
// are turned to the last bit of fp32: a key next to the border of two codes
// falls on the side that the exact value is on (but for one in 2^20 of those).
#include <cuda_fp16.h>

#include <algorithm>

#include "q2_page.cuh"

namespace q2 {
namespace {

__device__ unsigned int q2_cache_error;

constexpr int kThreads = 256;

// Which rows belong to which sequence.
struct RowArgs {
  const int* starts;            // [batch + 1], or null: one token each
  const int* lens;
  int batch, ntok, cap;         // cap: tokens that a table row, and the angles, reach
};

struct Seq {
  int row0, n, len;             // rows row0 .. row0 + n - 1 are its last tokens
  bool ok;                      // the length is one
};

__device__ __forceinline__ Seq seq_of(const RowArgs& a, int b) {
  Seq s{b, 1, a.lens[b], true};
  if (a.starts) {
    const int s0 = a.starts[b], s1 = a.starts[b + 1];
    s.row0 = s0;
    s.n = s1 - s0;
    if (s0 < 0 || s1 < s0 || s1 > a.ntok) {
      s.n = 0;
      s.ok = false;
    }
  }
  if (s.len < 0 || s.len > a.cap || (s.len && s.len < s.n)) s.ok = false;
  if (s.len == 0) s.n = 0;
  return s;
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(h[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint4 r;
  __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  return r;
}

// x c + y s to the last bit (but where the exact sum is within 2^-20 of a step
// of the middle of two): the products' and the sum's rounding errors (Knuth,
// "The Art of Computer Programming" 2, 4.2.2, theorem B) added at the end.  In
// explicitly rounded operations: of plain ones the compiler may fuse a product
// into the sum behind it, whose error is then another.
__device__ __forceinline__ float turn_exact(float x, float c, float y, float s) {
  const float p = __fmul_rn(x, c), q = __fmul_rn(y, s), pe = fmaf(x, c, -p), qe = fmaf(y, s, -q);
  const float t = __fadd_rn(p, q), z = __fsub_rn(t, p), e = __fadd_rn(__fsub_rn(p, __fsub_rn(t, z)), __fsub_rn(q, z));
  const float r = __fadd_rn(t, __fadd_rn(e, __fadd_rn(pe, qe)));
  return fabsf(t) <= 3.4028235e38f ? r : t;         // (an infinite t has no error term)
}

struct AppendArgs {
  RowArgs rows;
  Pages pg;                     // codes or fp16 rows, in bytes
  Pages sp;                     // (step, offset) pairs, in bytes
  const __half* q;
  __half* qo;
  const __half* k;
  const __half* v;
  long long ldq, ldqo, ldk, ldv;
  __half* bounds;
  const float* angles;
  int q_heads, kv_heads, chunk, cq, ck; // chunk: heads of a CTA; cq, ck: CTAs of a tile's queries, keys
  int rot, interleaved, sub;            // sub: bounds of a page
  int tile;                             // 2^tile positions to a tile
};

__device__ __forceinline__ uint4 hmin8(const uint4& a, const uint4& b) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__half2*>(&r)[i] =
        __hmin2_nan(reinterpret_cast<const __half2*>(&a)[i], reinterpret_cast<const __half2*>(&b)[i]);
  return r;
}

__device__ __forceinline__ uint4 hmax8(const uint4& a, const uint4& b) {
  uint4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<__half2*>(&r)[i] =
        __hmax2_nan(reinterpret_cast<const __half2*>(&a)[i], reinterpret_cast<const __half2*>(&b)[i]);
  return r;
}

// Codes of this lane's 8 columns, and the (step, offset) of its group, whose
// GRP / 8 lanes are neighbours.  All lanes of the warp call it.
template <int GRP>
__device__ __forceinline__ uint32_t quantise(const float (&y)[8], __half2& pair) {
  float lo = y[0], hi = y[0];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = fminf(lo, y[e]);
    hi = fmaxf(hi, y[e]);
    bad = bad || !(fabsf(y[e]) <= 3.4028235e38f);
  }
#pragma unroll
  for (int o = 1; o < GRP / 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  const uint32_t all = __ballot_sync(0xffffffffu, bad);
  const int lane = threadIdx.x & 31;
  bad = (all >> (lane & ~(GRP / 8 - 1))) & ((1u << (GRP / 8)) - 1u);
  const __half mh = __float2half_rn(lo), sh = __float2half_rn(__fdiv_rn(hi - lo, 15.f));
  const float m = __half2float(mh), s = __half2float(sh);
  if (bad || __hisinf(mh)) {
    pair = __halves2half2(__ushort_as_half(0), __ushort_as_half(0x7e00));
    return 0;
  }
  pair = __halves2half2(sh, mh);
  if (s == 0.f) return 0;
  // (y - m) / s rounded to nearest: from the rounded reciprocal one correction by
  // the remainder gives it (Markstein, "Computation of elementary functions on
  // the IBM RISC System/6000 processor", 1990, theorem 4.1)
  const float r = __frcp_rn(s);
  // Added to 1.5 2^23 a number of 0..15 is rounded to a whole one, ties to even,
  // in the sum's last bits; the codes are the sums' bits, 4 e up, less what
  // 1.5 2^23 adds to that.
  constexpr float kWhole = 12582912.f;
  constexpr uint32_t kBits = 0x4b400000u, kAll = kBits * 0x11111111u;
  uint32_t c = 0u - kAll;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = y[e] - m, q = d * r, f = fminf(fmaxf(fmaf(fmaf(-q, s, d), r, q), 0.f), 15.f);
    c += __float_as_uint(f + kWhole) << (4 * e);
  }
  return c;
}

// GRP: columns of a group of the 4-bit cache, 0 for an fp16 cache.  ONE: one
// token per sequence (no starts): every lane reads its angles and the page, and
// nothing is waited for (64 sequences into 4 bits 0.6 us less; as a branch of the
// general kernel it gained nothing).
template <int D, int GRP, bool ONE>
__global__ void __launch_bounds__(kThreads, 3) k_append(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 8, SLOTS = kThreads / LPR;
  constexpr int kBatch = ONE ? 1 : GRP ? 2 : 3;     // rows of a slot whose loads are in flight together (long code costs fetches)
  extern __shared__ __align__(16) float4 q2_append_smem[];                   // angles of the tile's tokens, [token][rot / 4]
  __shared__ long long places[2][ONE ? 1 : Q2_BLOCK];         // of its tokens in the pools, and in those of the pairs; -1: none
  __shared__ uint4 red[SLOTS][2][LPR];
  __shared__ int pre[ONE ? 1 : Q2_ATT_MAX_BATCH + 1];         // tiles before each sequence
  __shared__ int wsum[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = threadIdx.x / LPR, piece = threadIdx.x % LPR;

  pdl_wait();
  pdl_trigger();
  const RowArgs& rw = a.rows;
  int total = rw.batch;
  if constexpr (!ONE) {                             // four sequences per thread, then a scan of the threads' sums
    constexpr int EACH = Q2_ATT_MAX_BATCH / kThreads;
    int n[EACH], sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = threadIdx.x * EACH + i;
      n[i] = 0;
      if (b < rw.batch) {
        const Seq s = seq_of(rw, b);
        bad = bad || !s.ok;
        if (s.n) n[i] = s.ok ? ((s.len - 1) >> a.tile) - ((s.len - s.n) >> a.tile) + 1 : ((s.n - 1) >> a.tile) + 1;
      }
      sum += n[i];
    }
    if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(&q2_cache_error, Q2_ERR_LENGTH);
    int run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) wsum[warp] = run;
    __syncthreads();
    run -= sum;
    for (int w = 0; w < warp; ++w) run += wsum[w];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int b = threadIdx.x * EACH + i;
      if (b <= rw.batch) pre[b] = run;              // (batch < 1024: the last entry too; else below)
      run += n[i];
    }
    if (threadIdx.x == kThreads - 1 && rw.batch == Q2_ATT_MAX_BATCH) pre[rw.batch] = run;
    __syncthreads();
    total = pre[rw.batch];
  }

  // This CTA's heads, all of one kind.
  enum { QUERY, KEY, VALUE };
  const int y = blockIdx.y, kind = y < a.cq ? QUERY : y < a.cq + a.ck ? KEY : VALUE;
  const int h0 = (kind == QUERY ? y : kind == KEY ? y - a.cq : y - a.cq - a.ck) * a.chunk;
  const int nh = min(a.chunk, (kind == QUERY ? a.q_heads : a.kv_heads) - h0);
  const __half* src = kind == QUERY ? a.q : kind == KEY ? a.k : a.v;
  const long long ld = kind == QUERY ? a.ldq : kind == KEY ? a.ldk : a.ldv;
  src += (long long)h0 * D + piece * 8;
  const bool turns = a.angles && kind != VALUE, bounded = a.bounds && kind == KEY;
  const int RP = a.rot / 8;                         // pieces of a head that are turned
  const bool turned = turns && piece < RP, first_half = piece < RP / 2;
  // this lane's first four angles of a token, in 16-byte pieces
  const int apiece = a.interleaved ? piece * 2 : (first_half ? piece : piece - RP / 2) * 4;
  const int partner = lane - piece + (!turned ? piece : first_half ? piece + RP / 2 : piece - RP / 2);

  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int b = tile, j = 0;
    if constexpr (!ONE) {                           // the sequence with pre[b] <= tile < pre[b + 1]
      int lo = 0, hi = rw.batch - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid + 1] <= tile) lo = mid + 1;
        else hi = mid;
      }
      b = lo;
      j = tile - pre[lo];
    }
    const Seq s = seq_of(rw, b);
    if (ONE) {
      if (!s.ok && y == 0 && threadIdx.x == 0) atomicOr(&q2_cache_error, Q2_ERR_LENGTH);
      if (!s.n) continue;
    }
    const int past = s.len - s.n, block = ONE ? past / Q2_BLOCK : (past >> a.tile) + j;
    const int p0 = !s.ok ? 0 : ONE ? past : max(past, block << a.tile);
    const int n = ONE ? 1 : s.ok ? min(s.len, (block + 1) << a.tile) - p0 : min(1 << a.tile, s.n - (j << a.tile));
    const int row0 = s.row0 + (s.ok ? p0 - past : j << a.tile);
    const int* trow = a.pg.table + b * a.pg.table_stride;

    // The slots take T tokens side by side and SLOTS / T heads; keys with bounds
    // all heads, so that a slot's rows are of one head.
    int T = ONE ? 1 : SLOTS;
    if (!ONE && bounded)
      while (T > 1 && SLOTS / T < nh) T >>= 1;
    while (T > 1 && T / 2 >= n) T >>= 1;
    const int tk = slot & (T - 1), part = slot / T, HS = SLOTS / T;
    const int steps = (nh + HS - 1) / HS, items = (n + T - 1) / T * steps;   // a slot's rows: tokens in turn, and the heads of each

    // what is to be read from memory goes out first: the first rows, the angles, the pages
    auto load = [&](int t, int e) {
      return t < n && e < nh ? *reinterpret_cast<const uint4*>(src + (row0 + t) * ld + (long long)e * D) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 raw[kBatch];
    int lt = tk, le = part;                         // the row to be loaded: token, head
    auto fetch = [&]() {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        raw[u] = load(lt, le);
        le += HS;
        if (le - part >= steps * HS) {
          le = part;
          lt += T;
        }
      }
    };
    fetch();
    long long place = -1, pair_place = -1;          // of the token in the pools, and in those of the pairs
    auto place_of = [&](int pos) {
      const int pi = s.ok ? page_of(a.pg, pos) : 0, page = s.ok ? trow[pi] : -1;
      const bool there = (unsigned)page < (unsigned)a.pg.npages;
      if (s.ok && !there) atomicOr(&q2_cache_error, Q2_ERR_PAGE);
      const int at = pos - pi * a.pg.page;
      place = there ? page * a.pg.page_stride + at * a.pg.token_stride : -1;
      if (GRP) pair_place = there ? page * a.sp.page_stride + at * a.sp.token_stride : -1;
    };
    if (!ONE && turns && s.ok) {
      const float4* from = reinterpret_cast<const float4*>(a.angles + (long long)p0 * a.rot);
      for (int i = threadIdx.x; i < n * (a.rot / 4); i += kThreads)          // (exchanged by the lane that reads them, for the banks)
        cp16(saddr(q2_append_smem + (i ^ (i >> 2 & 3))), from + i, true);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (kind != QUERY && (ONE || threadIdx.x < n)) {
      place_of(p0 + (ONE ? 0 : threadIdx.x));
      if (!ONE) {
        places[0][threadIdx.x] = place;
        places[1][threadIdx.x] = pair_place;
      }
    }
    if (!ONE) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }

    uint4 lo = make_uint4(0x7c007c00u, 0x7c007c00u, 0x7c007c00u, 0x7c007c00u);       // bounds of a slot's keys
    uint4 hi = make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
    float cs[8], sn[8];                             // this lane's angles; of a first half's columns the sine is negated
    int t = tk, e = part;
    for (int k0 = 0; k0 < items; k0 += kBatch) {
      uint4 now[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) now[u] = raw[u];
      if (k0 + kBatch < items) fetch();
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (k0 + u < items) {                       // (the same for all)
          const bool live = t < n && e < nh;
          uint4 h8 = now[u];
          float x[8];
          if (turns || GRP) unpack8(h8, x);
          if (turns) {
            if (turned && e == part) {              // another token
              const int f = min(t, n - 1) * (a.rot / 4) + apiece;
              const float4* one = reinterpret_cast<const float4*>(a.angles + (long long)p0 * a.rot) + apiece;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i < 2 || !a.interleaved) {
                  const float4 v = !ONE ? q2_append_smem[(f + i) ^ ((f + i) >> 2 & 3)] : s.ok ? __ldg(one + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                  const float sign = a.interleaved || !first_half ? 1.f : -1.f;
                  cs[2 * i] = v.x;
                  sn[2 * i] = v.y * sign;
                  cs[2 * i + 1] = v.z;
                  sn[2 * i + 1] = v.w * sign;
                }
              }
            }
            if (a.interleaved) {
              if (turned) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float v = x[2 * i], w = x[2 * i + 1];
                  x[2 * i] = kind == KEY ? turn_exact(v, cs[i], w, -sn[i]) : fmaf(v, cs[i], -w * sn[i]);
                  x[2 * i + 1] = kind == KEY ? turn_exact(w, cs[i], v, sn[i]) : fmaf(w, cs[i], v * sn[i]);
                }
              }
            } else {
              uint4 other;                          // the other half's columns
              other.x = __shfl_sync(0xffffffffu, h8.x, partner);
              other.y = __shfl_sync(0xffffffffu, h8.y, partner);
              other.z = __shfl_sync(0xffffffffu, h8.z, partner);
              other.w = __shfl_sync(0xffffffffu, h8.w, partner);
              if (turned) {
                float o[8];
                unpack8(other, o);
                if (kind == KEY) {
#pragma unroll
                  for (int i = 0; i < 8; ++i) x[i] = turn_exact(x[i], cs[i], o[i], sn[i]);
                } else {
#pragma unroll
                  for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], cs[i], o[i] * sn[i]);
                }
              }
            }
            h8 = pack8(x);
          }
          if (kind == QUERY) {
            if (!s.ok) h8 = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
            if (live) *reinterpret_cast<uint4*>(a.qo + (row0 + t) * a.ldqo + (long long)(h0 + e) * D + piece * 8) = h8;
          } else {
            const long long at = !live ? -1 : ONE ? place : places[0][t];
            unsigned char* to = (kind == VALUE ? a.pg.v : a.pg.k) + at + (h0 + e) * a.pg.head_stride;
            if constexpr (GRP == 0) {
              if (at >= 0) *reinterpret_cast<uint4*>(to + piece * 16) = h8;
            } else {
              __half2 pair;
              const uint32_t code = quantise<GRP>(x, pair);
              if (at >= 0) {
                *reinterpret_cast<uint32_t*>(to + piece * 4) = code;
                if (piece % (GRP / 8) == 0)
                  *reinterpret_cast<__half2*>((kind == VALUE ? a.sp.v : a.sp.k) + (ONE ? pair_place : places[1][t]) + (h0 + e) * a.sp.head_stride +
                                              piece / (GRP / 8) * 4) = pair;
              }
            }
            if (bounded && live) {
              lo = hmin8(lo, h8);
              hi = hmax8(hi, h8);
            }
          }
          e += HS;
          if (e - part >= steps * HS) {
            e = part;
            t += T;
          }
        }
      }
    }
    if (bounded) {                                  // (a slot's keys are of head `part`; a tile is a block)
      const int begin = s.ok ? block * Q2_BLOCK : 0, pi = page_of(a.pg, begin);
      const int page = s.ok ? trow[pi] : -1;
      const bool kept = (unsigned)page < (unsigned)a.pg.npages;
      red[slot][0][piece] = lo;
      red[slot][1][piece] = hi;
      __syncthreads();
      for (int i = threadIdx.x; i < nh * 2 * LPR; i += kThreads) {
        const int h = i / (2 * LPR), w = i / LPR % 2, pc = i % LPR;
        if (kept) {
          uint4 x = red[h * T][w][pc];
          for (int k = 1; k < T; ++k) x = w ? hmax8(x, red[h * T + k][w][pc]) : hmin8(x, red[h * T + k][w][pc]);
          uint4* to = reinterpret_cast<uint4*>(
              a.bounds +
              ((((long long)page * a.sub + (begin - pi * a.pg.page) / Q2_BLOCK) * a.kv_heads + h0 + h) * 2 + w) * D + pc * 8);
          if (p0 > begin) x = w ? hmax8(x, *to) : hmin8(x, *to);              // the block goes on
          *to = x;
        } else if (s.ok && i == 0) {                // (may be another page than the tokens')
          atomicOr(&q2_cache_error, Q2_ERR_PAGE);
        }
      }
    }
    if (!ONE || bounded) __syncthreads();           // angles, places and bounds are another tile's from here on
  }
}

struct ReadArgs {
  RowArgs rows;
  Pages pg, sp;
  __half* out[2];               // keys and values; where there is one, `both` is 0 and it comes first
  const unsigned char* pool[2];
  const unsigned char* pairs[2];
  long long ld[2];
  int kv_heads, both;
  uint32_t each_mul, each_sh;   // of a division by the pieces of a row
};

// Tokens out: a thread per piece of 8 columns of a row, or four pieces (kReads)
// whose loads are in flight together where that still leaves four CTAs per SM.
template <int D, int GRP, int kReads>
__global__ void __launch_bounds__(kThreads) k_read(const __grid_constant__ ReadArgs a) {
  constexpr int LPR = D / 8;
  __shared__ int starts[Q2_ATT_MAX_BATCH + 1];
  pdl_wait();
  pdl_trigger();
  const RowArgs& rw = a.rows;
  if (rw.starts) {
    for (int i = threadIdx.x; i <= rw.batch; i += kThreads) starts[i] = rw.starts[i];
    __syncthreads();
  }
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < rw.batch; b += kThreads)
      if (!seq_of(rw, b).ok) atomicOr(&q2_cache_error, Q2_ERR_LENGTH);
  const uint32_t per = a.kv_heads * LPR, each = per << a.both;               // pieces of a row's keys or values; of a row
  const long long first = (long long)blockIdx.x * (kThreads * kReads);
  const int row0 = (int)(first / each);
  const uint32_t skip = (uint32_t)(first - (long long)row0 * each) + threadIdx.x;
  __half* to[kReads];
  const unsigned char* from[kReads];
  const unsigned char* pair[kReads];
#pragma unroll
  for (int u = 0; u < kReads; ++u) {
    const uint32_t i = skip + u * kThreads, rows = (__umulhi(i, a.each_mul) + i) >> a.each_sh;      // (below 2^31: page_of()'s division)
    const int row = row0 + (int)rows;
    to[u] = nullptr;
    from[u] = pair[u] = nullptr;
    if (row >= rw.ntok) continue;
    const uint32_t r = i - rows * each, w = r >= per, h = (r - w * per) / LPR, piece = r % LPR;
    int b = row;
    if (rw.starts) {                                // the last sequence that begins at or before the row
      int lo = 0, hi = rw.batch;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= row) lo = mid + 1;
        else hi = mid;
      }
      b = lo - 1;
      if (b < 0 || b >= rw.batch) continue;
    }
    const Seq s = seq_of(rw, b);
    if (s.n == 0 || row < s.row0 || row >= s.row0 + s.n) continue;
    to[u] = a.out[w] + row * a.ld[w] + (long long)h * D + piece * 8;
    if (!s.ok) continue;
    const int pos = s.len - s.n + (row - s.row0), pi = page_of(a.pg, pos), page = a.pg.table[b * a.pg.table_stride + pi];
    if ((unsigned)page >= (unsigned)a.pg.npages) {
      if (r == 0) atomicOr(&q2_cache_error, Q2_ERR_PAGE);
      continue;
    }
    const int at = pos - pi * a.pg.page;
    from[u] = a.pool[w] + page * a.pg.page_stride + at * a.pg.token_stride + h * a.pg.head_stride + piece * (GRP ? 4 : 16);
    if (GRP)
      pair[u] = a.pairs[w] + page * a.sp.page_stride + at * a.sp.token_stride + h * a.sp.head_stride + piece / (GRP ? GRP / 8 : 1) * 4;
  }
  uint4 raw[kReads];
  __half2 sm[kReads];
#pragma unroll
  for (int u = 0; u < kReads; ++u) {
    raw[u] = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
    if (from[u]) {
      if constexpr (GRP == 0) {
        raw[u] = *reinterpret_cast<const uint4*>(from[u]);
      } else {
        raw[u].x = *reinterpret_cast<const uint32_t*>(from[u]);
        sm[u] = *reinterpret_cast<const __half2*>(pair[u]);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kReads; ++u) {
    if (GRP && from[u]) {
      const float2 f = __half22float2(sm[u]);
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)                   // (2^23 + the code, less 2^23)
        x[k] = fmaf(__uint_as_float(0x4b000000u | (raw[u].x >> (4 * k) & 15u)) - 8388608.f, f.x, f.y);
      raw[u] = pack8(x);
    }
    if (to[u]) *reinterpret_cast<uint4*>(to[u]) = raw[u];
  }
}

int check_rows(RowArgs& r, const int* starts, const int* lens, int batch, int ntok, long long cap) {
  if (batch < 0 || batch > Q2_ATT_MAX_BATCH || ntok < 0) return Q2_ESHAPE;
  if (batch && ntok && !lens) return Q2_EINVAL;
  if (!starts && ntok != batch) return Q2_ESHAPE;
  if (misaligned(starts, 4) || misaligned(lens, 4)) return Q2_EALIGN;
  r = {starts, lens, batch, ntok, (int)cap};
  return Q2_OK;
}

int check_ld(const void* p, long long ld, long long width, int ntok) {
  if (misaligned(p, 16) || (ntok > 1 && ld % 8)) return Q2_EALIGN;
  return ntok > 1 && ld < width ? Q2_ESHAPE : Q2_OK;
}

int append(const Pages& pg, const Pages& sp, const CacheShape& c, void* bounds, const void* q, long long ldq, void* q_out,
           long long ldqo, int q_heads, const void* k, long long ldk, const void* v, long long ldv, const int* starts,
           const int* lens, int batch, int ntok, const q2_rope* rope, void* stream) {
  if ((!q) != (!q_out)) return Q2_EINVAL;
  if (!q) q_heads = 0;
  if (q && (q_heads < 1 || q_heads > 65536)) return Q2_ESHAPE;
  AppendArgs a = {};
  long long cap = c.cap;
  if (rope) {
    if (rope->positions < 0 || rope->rot < 16 || rope->rot % 16 || rope->rot > c.D) return Q2_ESHAPE;
    if (!rope->table) return Q2_EINVAL;
    if (misaligned(rope->table, 16)) return Q2_EALIGN;
    a.angles = rope->table;
    a.rot = rope->rot;
    a.interleaved = rope->interleaved != 0;
    cap = std::min(cap, (long long)rope->positions);
  }
  int st = check_rows(a.rows, starts, lens, batch, ntok, cap);
  if (st) return st;
  if (bounds) {
    if (c.page % Q2_BLOCK && Q2_BLOCK % c.page) return Q2_ESHAPE;
    if (misaligned(bounds, 16)) return Q2_EALIGN;
  }
  if (batch == 0 || ntok == 0) return Q2_OK;
  if (!k || !v) return Q2_EINVAL;
  const long long kw = (long long)c.kv_heads * c.D, qw = (long long)q_heads * c.D;
  if ((st = check_ld(k, ldk, kw, ntok)) || (st = check_ld(v, ldv, kw, ntok))) return st;
  if (q && ((st = check_ld(q, ldq, qw, ntok)) || (st = check_ld(q_out, ldqo, qw, ntok)))) return st;
  a.pg = pg;
  a.sp = sp;
  a.q = static_cast<const __half*>(q);
  a.qo = static_cast<__half*>(q_out);
  a.k = static_cast<const __half*>(k);
  a.v = static_cast<const __half*>(v);
  a.ldq = ldq;
  a.ldqo = ldqo;
  a.ldk = ldk;
  a.ldv = ldv;
  a.bounds = static_cast<__half*>(bounds);
  a.q_heads = q_heads;
  a.kv_heads = c.kv_heads;
  a.sub = (c.page + Q2_BLOCK - 1) / Q2_BLOCK;
  // Heads per CTA: as many as its row slots take side by side at the usual
  // number of tokens, more where there would be more CTAs than run at once; keys
  // whose bounds are kept no more than the slots.
  const int slots = kThreads * 8 / c.D;
  // Blocks of 64 positions are tiles where bounds are kept; else, with few tokens
  // to a sequence, fewer: a prompt among them were the end of all (238 tokens of
  // 126 sequences, 32 heads of 256: 36.2 -> 9.8 us).
  const int usual = std::min(Q2_BLOCK, (ntok + batch - 1) / batch);
  a.tile = 6;
  while (!bounds && a.tile > 3 && (1 << (a.tile - 1)) >= 2 * usual) --a.tile;
  const long long tiles = starts ? ((long long)ntok >> a.tile) + 2ll * std::min(batch, ntok) : batch;
  int side = slots;
  for (int t = 1; t < usual && side > 1; t <<= 1) side >>= 1;
  const long long heads = q_heads + 2ll * c.kv_heads;
  const long long at_once = 3ll * dev_info().sms;
  a.chunk = std::max(side, (int)std::min((long long)std::min(16, slots), (heads * tiles + at_once - 1) / at_once));
  auto ctas = [&](int h) { return (h + a.chunk - 1) / a.chunk; };
  while (ctas(q_heads) + 2 * ctas(c.kv_heads) > 65535) a.chunk *= 2;
  if (bounds) a.chunk = std::min(a.chunk, slots);
  a.cq = ctas(q_heads);
  a.ck = ctas(c.kv_heads);
  const dim3 grid((unsigned)std::min(tiles, 65535ll), a.cq + 2 * a.ck);
  const int smem = rope && starts ? a.rot * 4 << a.tile : 0;
  return by_shape(c, [&](auto D, auto G) {
    return starts ? launch_pdl(k_append<D(), G(), false>, a, grid, kThreads, smem, stream)
                  : launch_pdl(k_append<D(), G(), true>, a, grid, kThreads, 0, stream);
  });
}

int read(const Pages& pg, const Pages& sp, const CacheShape& c, void* k, long long ldk, void* v, long long ldv,
         const int* starts, const int* lens, int batch, int ntok, void* stream) {
  ReadArgs a = {};
  int st = check_rows(a.rows, starts, lens, batch, ntok, c.cap);
  if (st) return st;
  if (batch == 0 || ntok == 0 || (!k && !v)) return Q2_OK;
  const long long kw = (long long)c.kv_heads * c.D;
  if ((k && (st = check_ld(k, ldk, kw, ntok))) || (v && (st = check_ld(v, ldv, kw, ntok)))) return st;
  a.pg = pg;
  a.sp = sp;
  a.both = k && v;
  int w = 0;
  auto add = [&](void* out, long long ld, const unsigned char* pool, const unsigned char* pairs) {
    if (!out) return;
    a.out[w] = static_cast<__half*>(out);
    a.ld[w] = ld;
    a.pool[w] = pool;
    a.pairs[w++] = pairs;
  };
  add(k, ldk, pg.k, sp.k);
  add(v, ldv, pg.v, sp.v);
  a.kv_heads = c.kv_heads;
  const long long each = (long long)c.kv_heads * (c.D / 8) << a.both, items = each * ntok;
  if (each > 0x3fffffffll) return Q2_ESHAPE;
  set_page((int)each, a.each_mul, a.each_sh);
  // four pieces to a thread where that leaves four CTAs per SM
  const int reads = items >= 4ll * kThreads * 4 * dev_info().sms ? 4 : 1;
  const long long ctas = (items + kThreads * reads - 1) / (kThreads * reads);
  if (ctas > 0x7fffffffll) return Q2_ESHAPE;
  return by_shape(c, [&](auto D, auto G) {
    return reads == 4 ? launch_pdl(k_read<D(), G(), 4>, a, (int)ctas, kThreads, 0, stream)
                      : launch_pdl(k_read<D(), G(), 1>, a, (int)ctas, kThreads, 0, stream);
  });
}

}  // namespace
}  // namespace q2

using namespace q2;

extern "C" int q2_append(const q2_kv* kv, void* bounds, const void* q, long long ldq, void* q_out, long long ldqo,
                         int q_heads, const void* k, long long ldk, const void* v, long long ldv, const int* starts,
                         const int* lens, int batch, int ntok, const q2_rope* rope, q2_stream stream) {
  Pages pg, sp = {};
  CacheShape c;
  const int st = check_cache(kv, batch, pg, c);
  return st ? st : append(pg, sp, c, bounds, q, ldq, q_out, ldqo, q_heads, k, ldk, v, ldv, starts, lens, batch, ntok, rope, stream);
}

extern "C" int q2_append4(const q2_kv4* kv, void* bounds, const void* q, long long ldq, void* q_out, long long ldqo,
                          int q_heads, const void* k, long long ldk, const void* v, long long ldv, const int* starts,
                          const int* lens, int batch, int ntok, const q2_rope* rope, q2_stream stream) {
  Pages pg, sp;
  CacheShape c;
  const int st = check_cache4(kv, batch, pg, sp, c);
  return st ? st : append(pg, sp, c, bounds, q, ldq, q_out, ldqo, q_heads, k, ldk, v, ldv, starts, lens, batch, ntok, rope, stream);
}

extern "C" int q2_read(const q2_kv* kv, void* k, long long ldk, void* v, long long ldv, const int* starts, const int* lens,
                       int batch, int ntok, q2_stream stream) {
  Pages pg, sp = {};
  CacheShape c;
  const int st = check_cache(kv, batch, pg, c);
  return st ? st : read(pg, sp, c, k, ldk, v, ldv, starts, lens, batch, ntok, stream);
}

extern "C" int q2_read4(const q2_kv4* kv, void* k, long long ldk, void* v, long long ldv, const int* starts,
                        const int* lens, int batch, int ntok, q2_stream stream) {
  Pages pg, sp;
  CacheShape c;
  const int st = check_cache4(kv, batch, pg, sp, c);
  return st ? st : read(pg, sp, c, k, ldk, v, ldv, starts, lens, batch, ntok, stream);
}

// The error word of these kernels, then cleared (q2_device_errors).
extern "C" int q2_cache_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_cache_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_cache_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
