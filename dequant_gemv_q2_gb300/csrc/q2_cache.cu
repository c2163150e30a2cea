// The paged key-value cache's rows: new tokens in (q2_append, q2_append4), with
// the position rotation on the way, and tokens out (q2_read, q2_read4).
//
// A token's pairs of columns are turned by its position's angles,
//
//   (a, b) -> (a cos - b sin, b cos + a sin),
//
// and keys go to the cache in fp16, or in 4 bits (offset and step per group of
// 32 or 64 columns: least value m, range / 15 = s, code rint((x - m) / s)).
// Every row is read and written once, so memory bounds it: a row's head is 16
// bytes per lane, 8, 16 or 32 lanes; the partner of a column is in another lane
// of the same row (a shuffle) or in the next register.
//
// Work is cut into tiles: the new tokens of one block of 64 positions of one
// sequence, times a few heads.  With few tokens in a tile (one, when decoding)
// the row slots of a CTA take its heads side by side, with many its tokens.
// Tiles are cut at blocks so that a block's bounds (least and greatest key per
// column) are one CTA's: no atomics, and what a block held before is read only
// where it goes on.
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
// "The Art of Computer Programming" 2, 4.2.2, theorem B) added at the end.
__device__ __forceinline__ float turn_exact(float x, float c, float y, float s) {
  const float p = x * c, q = y * s, pe = fmaf(x, c, -p), qe = fmaf(y, s, -q);
  const float t = p + q, z = t - p, e = (p - (t - z)) + (q - z);
  const float r = t + (e + (pe + qe));
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
  int q_heads, kv_heads, chunk;         // chunk: heads of a CTA
  int rot, interleaved, sub;            // sub: bounds of a page
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
  uint32_t c = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    c |= (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(y[e] - m, s)), 0.f), 15.f) << (4 * e);
  return c;
}

// GRP: columns of a group of the 4-bit cache, 0 for an fp16 cache
template <int D, int GRP>
__global__ void __launch_bounds__(kThreads) k_append(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 8, SLOTS = kThreads / LPR;
  __shared__ uint4 red[SLOTS][2][LPR];
  __shared__ int pre[Q2_ATT_MAX_BATCH + 1];         // tiles before each sequence
  __shared__ int wsum[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slot = threadIdx.x / LPR, piece = threadIdx.x % LPR;

  pdl_wait();
  pdl_trigger();
  const RowArgs& rw = a.rows;
  int total = rw.batch;
  if (rw.starts) {                                  // four sequences per thread, then a scan of the threads' sums
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
        if (s.n) n[i] = s.ok ? (s.len - 1) / Q2_BLOCK - (s.len - s.n) / Q2_BLOCK + 1 : (s.n + Q2_BLOCK - 1) / Q2_BLOCK;
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

  const int qk = a.q_heads + a.kv_heads, heads = qk + a.kv_heads;
  const int h0 = blockIdx.y * a.chunk, h1 = min(h0 + a.chunk, heads);
  const int RP = a.rot / 8;                         // pieces of a head that are turned
  const bool turned = a.angles && piece < RP;

  for (int tile = blockIdx.x; tile < total; tile += gridDim.x) {
    int b = tile, j = 0;
    if (rw.starts) {                                // the sequence with pre[b] <= tile < pre[b + 1]
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
    if (!rw.starts) {
      if (!s.ok && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(&q2_cache_error, Q2_ERR_LENGTH);
      if (!s.n) continue;
    }
    const int past = s.len - s.n, block = past / Q2_BLOCK + j;
    const int p0 = s.ok ? max(past, block * Q2_BLOCK) : 0;
    const int n = s.ok ? min(s.len, (block + 1) * Q2_BLOCK) - p0 : min(Q2_BLOCK, s.n - j * Q2_BLOCK);
    const int row0 = s.row0 + (s.ok ? p0 - past : j * Q2_BLOCK);
    int T = 1;                                      // tokens side by side
    while (T < n && T < SLOTS) T <<= 1;
    const int tk = slot & (T - 1), part = slot / T, HS = SLOTS / T;
    const int* trow = a.pg.table + b * a.pg.table_stride;

    float cs[8], sn[8];                             // this lane's angles; of a first half's columns the sine is negated
    // row t of the tile: where it goes
    bool live = false, there = false;
    int row = 0;
    long long at = 0, sat = 0;                      // the token's place in the pools, and in those of the pairs
    auto token = [&](int t) {
      live = t < n;
      row = row0 + t;
      const int pos = p0 + t;
      there = false;
      if (live && s.ok) {
        if (h1 > a.q_heads) {
          const int pi = page_of(a.pg, pos), page = trow[pi];
          there = (unsigned)page < (unsigned)a.pg.npages;
          if (!there && piece == 0) atomicOr(&q2_cache_error, Q2_ERR_PAGE);
          if (there) {
            at = page * a.pg.page_stride + (pos - pi * a.pg.page) * a.pg.token_stride;
            if constexpr (GRP > 0) sat = page * a.sp.page_stride + (pos - pi * a.pg.page) * a.sp.token_stride;
          }
        }
        if (turned && h0 < qk) {
          const float* base = a.angles + (long long)pos * a.rot;
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float4 f = __ldg(reinterpret_cast<const float4*>(base + piece * 8) + i);
              cs[2 * i] = f.x;
              sn[2 * i] = f.y;
              cs[2 * i + 1] = f.z;
              sn[2 * i + 1] = f.w;
            }
          } else {
            const bool first = piece < RP / 2;
            const float4* at4 = reinterpret_cast<const float4*>(base + (first ? piece : piece - RP / 2) * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = __ldg(at4 + i);
              cs[2 * i] = f.x;
              sn[2 * i] = first ? -f.y : f.y;
              cs[2 * i + 1] = f.z;
              sn[2 * i + 1] = first ? -f.w : f.w;
            }
          }
        }
      }
    };
    auto load = [&](int h) {
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (live && h < h1) {
        const __half* src = h < a.q_heads ? a.q + row * a.ldq + (long long)h * D
                            : h < qk      ? a.k + row * a.ldk + (long long)(h - a.q_heads) * D
                                          : a.v + row * a.ldv + (long long)(h - qk) * D;
        r = *reinterpret_cast<const uint4*>(src + piece * 8);
      }
      return r;
    };
    // turns and stores the row's head h; returns it in fp16.  All lanes of the warp call it.
    auto put = [&](int h, const uint4& raw) {
      float x[8], y[8];
      unpack8(raw, x);
      const bool key = h >= a.q_heads;              // keys (and values, which are not turned)
      if (a.angles && h0 < qk) {
        uint4 other = raw;
        if (!a.interleaved) {                       // the other half's columns
          const int from = lane - piece + (piece < RP / 2 ? piece + RP / 2 : piece < RP ? piece - RP / 2 : piece);
          other.x = __shfl_sync(0xffffffffu, raw.x, from);
          other.y = __shfl_sync(0xffffffffu, raw.y, from);
          other.z = __shfl_sync(0xffffffffu, raw.z, from);
          other.w = __shfl_sync(0xffffffffu, raw.w, from);
        }
        if (turned && h < qk) {
          float o[8];
          unpack8(other, o);
          if (a.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float u = x[2 * i], w = x[2 * i + 1];
              y[2 * i] = key ? turn_exact(u, cs[i], w, -sn[i]) : fmaf(u, cs[i], -w * sn[i]);
              y[2 * i + 1] = key ? turn_exact(w, cs[i], u, sn[i]) : fmaf(w, cs[i], u * sn[i]);
            }
          } else if (key) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = turn_exact(x[i], cs[i], o[i], sn[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fmaf(x[i], cs[i], o[i] * sn[i]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = y[i];
        }
      }
      uint4 h8 = pack8(x);
      const bool mine = live && h < h1;
      if (!key) {
        if (!s.ok) h8 = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
        if (mine) *reinterpret_cast<uint4*>(a.qo + row * a.ldqo + (long long)h * D + piece * 8) = h8;
      }
      const bool val = h >= qk;
      const int hk = h - (val ? qk : a.q_heads);
      unsigned char* to = (val ? a.pg.v : a.pg.k) + at + hk * a.pg.head_stride;
      if constexpr (GRP == 0) {
        if (key && mine && there) *reinterpret_cast<uint4*>(to + piece * 16) = h8;
      } else {
        if (__any_sync(0xffffffffu, key)) {
          __half2 pair;
          const uint32_t code = quantise<GRP>(x, pair);
          if (key && mine && there) {
            *reinterpret_cast<uint32_t*>(to + piece * 4) = code;
            if (piece % (GRP / 8) == 0)
              *reinterpret_cast<__half2*>((val ? a.sp.v : a.sp.k) + sat + hk * a.sp.head_stride + piece / (GRP / 8) * 4) = pair;
          }
        }
      }
      return h8;
    };

    // keys whose bounds are kept are taken below, head by head
    const int k0 = a.bounds ? max(h0, a.q_heads) : h1, k1 = a.bounds ? min(h1, qk) : h1;
    if (k0 > h0 || k1 < h1 || !a.bounds) {
      for (int t0 = 0; t0 < n; t0 += T) {
        token(t0 + tk);
        for (int e0 = h0; e0 < h1; e0 += HS) {
          if (a.bounds && e0 >= k0 && e0 + HS <= k1) continue;
          const int h = e0 + part;
          const bool skip = a.bounds && h >= k0 && h < k1;
          const uint4 raw = skip ? make_uint4(0u, 0u, 0u, 0u) : load(h);
          put(skip ? h1 : h, raw);
        }
      }
    }
    if (a.bounds && k0 < k1) {
      const int first = s.ok ? block * Q2_BLOCK : 0, pi = page_of(a.pg, first);
      const int page = s.ok ? trow[pi] : -1;
      const bool kept = (unsigned)page < (unsigned)a.pg.npages;
      const int place = (first - pi * a.pg.page) / Q2_BLOCK;
      for (int e0 = k0; e0 < k1; e0 += HS) {
        const int h = e0 + part;
        uint4 lo = make_uint4(0x7c007c00u, 0x7c007c00u, 0x7c007c00u, 0x7c007c00u);
        uint4 hi = make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
        for (int t0 = 0; t0 < n; t0 += T) {
          token(t0 + tk);
          const bool mine = h < k1;
          const uint4 y = put(mine ? h : h1, mine ? load(h) : make_uint4(0u, 0u, 0u, 0u));
          if (live && mine) {
            lo = hmin8(lo, y);
            hi = hmax8(hi, y);
          }
        }
        red[slot][0][piece] = lo;
        red[slot][1][piece] = hi;
        __syncthreads();
        for (int i = threadIdx.x; i < HS * 2 * LPR; i += kThreads) {
          const int hh = i / (2 * LPR), w = i / LPR % 2, pc = i % LPR;
          if (kept && e0 + hh < k1) {
            uint4 x = red[hh * T][w][pc];
            for (int t = 1; t < T; ++t) x = w ? hmax8(x, red[hh * T + t][w][pc]) : hmin8(x, red[hh * T + t][w][pc]);
            uint4* to = reinterpret_cast<uint4*>(
                a.bounds + ((((long long)page * a.sub + place) * a.kv_heads + (e0 + hh - a.q_heads)) * 2 + w) * D + pc * 8);
            if (p0 > first) x = w ? hmax8(x, *to) : hmin8(x, *to);      // the block goes on
            *to = x;
          }
        }
        __syncthreads();
      }
    }
  }
}

struct ReadArgs {
  RowArgs rows;
  Pages pg, sp;
  __half* k;
  __half* v;
  long long ldk, ldv;
  int kv_heads;
};

// One row (all heads, keys then values) per step of a CTA; 8 columns per thread
// and step.
template <int D, int GRP>
__global__ void __launch_bounds__(kThreads) k_read(const __grid_constant__ ReadArgs a) {
  constexpr int LPR = D / 8;
  __shared__ int starts[Q2_ATT_MAX_BATCH + 1];
  pdl_wait();
  pdl_trigger();
  const RowArgs& rw = a.rows;
  if (rw.starts)
    for (int i = threadIdx.x; i <= rw.batch; i += kThreads) starts[i] = rw.starts[i];
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < rw.batch; b += kThreads)
      if (!seq_of(rw, b).ok) atomicOr(&q2_cache_error, Q2_ERR_LENGTH);
  __syncthreads();
  for (int row = blockIdx.x; row < rw.ntok; row += gridDim.x) {
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
    const int pos = s.len - s.n + (row - s.row0);
    const int pi = s.ok ? page_of(a.pg, pos) : 0, page = s.ok ? a.pg.table[b * a.pg.table_stride + pi] : -1;
    const bool there = (unsigned)page < (unsigned)a.pg.npages;
    if (s.ok && !there && threadIdx.x == 0) atomicOr(&q2_cache_error, Q2_ERR_PAGE);
    const long long e = there ? page * a.pg.page_stride + (pos - pi * a.pg.page) * a.pg.token_stride : 0;
    const long long f = there && GRP ? page * a.sp.page_stride + (pos - pi * a.pg.page) * a.sp.token_stride : 0;
    for (int i = threadIdx.x; i < 2 * a.kv_heads * LPR; i += kThreads) {
      const int w = i >= a.kv_heads * LPR, h = (i - w * a.kv_heads * LPR) / LPR, piece = i % LPR;
      __half* to = w ? a.v : a.k;
      if (!to) continue;
      uint4 r = make_uint4(0x7e007e00u, 0x7e007e00u, 0x7e007e00u, 0x7e007e00u);
      if (there) {
        const unsigned char* src = (w ? a.pg.v : a.pg.k) + e + h * a.pg.head_stride;
        if constexpr (GRP == 0) {
          r = *reinterpret_cast<const uint4*>(src + piece * 16);
        } else {
          const uint32_t c = *reinterpret_cast<const uint32_t*>(src + piece * 4);
          const float2 sm = __half22float2(*reinterpret_cast<const __half2*>((w ? a.sp.v : a.sp.k) + f + h * a.sp.head_stride +
                                                                             piece / (GRP / 8) * 4));
          float x[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = fmaf((float)((c >> (4 * k)) & 15u), sm.x, sm.y);
          r = pack8(x);
        }
      }
      *reinterpret_cast<uint4*>(to + row * (w ? a.ldv : a.ldk) + (long long)h * D + piece * 8) = r;
    }
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
  // number of tokens, more where the tiles alone fill the SMs six times over.
  const int heads = q_heads + 2 * c.kv_heads, slots = kThreads * 8 / c.D;
  const long long tiles = starts ? (long long)ntok / Q2_BLOCK + 2ll * std::min(batch, ntok) : batch;
  const int usual = std::min(Q2_BLOCK, (ntok + batch - 1) / batch);
  int side = slots;
  for (int t = 1; t < usual && side > 1; t <<= 1) side >>= 1;
  const long long fill = (heads * tiles + 6 * dev_info().sms - 1) / (6 * dev_info().sms);
  a.chunk = std::max(side, (int)std::min(16ll, fill));
  dim3 grid((unsigned)std::min(tiles, 65535ll), (heads + a.chunk - 1) / a.chunk);
  while (grid.y > 65535u) {
    a.chunk *= 2;
    grid.y = (heads + a.chunk - 1) / a.chunk;
  }
  return by_shape(c, [&](auto D, auto G) { return launch_pdl(k_append<D(), G()>, a, grid, kThreads, 0, stream); });
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
  a.k = static_cast<__half*>(k);
  a.v = static_cast<__half*>(v);
  a.ldk = ldk;
  a.ldv = ldv;
  a.kv_heads = c.kv_heads;
  const int grid = std::min(ntok, dev_info().sms * 8);
  return by_shape(c, [&](auto D, auto G) { return launch_pdl(k_read<D(), G()>, a, grid, kThreads, 0, stream); });
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
