// What the attention kernels share: how the tokens of a batch are shared out
// over the CTAs, how the warps' and the CTAs' sums are joined, and the tensor
// instructions.  (How it all works is told at the head of q2_attend.cu.)
#pragma once
#include <cuda_fp16.h>

#include <algorithm>

#include "q2_page.cuh"

namespace q2 {

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16, kUnit = kTile * kWarps;   // tokens of a warp's tile, of the fp16 cache's units
constexpr int kMostHeads = 16;                      // query heads of a unit at most

// The part of a call's arguments that does not depend on how the cache is held.
struct UnitArgs {
  const int* lens;
  const __half* q;
  __half* o;
  long long ldq, ldo;
  unsigned int* count;        // [batch][units' heads] arrivals, zero between calls
  float* part;                // [2 * CTAs][H][D] numerators, H the query heads of a unit
  float2* ml;                 // [2 * CTAs][H] maximum, denominator
  const int* sel;             // [batch][key-value heads][nsel] blocks to attend (the SP kernels)
  int nsel;
  int batch, cap;             // cap: tokens that a table row can hold
  int hu, nht, group;         // heads of units = kv_heads * nht; query heads of a key-value head
  float sc2;                  // scale * log2(e)
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at));
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A place in the order of units.
struct Walk {
  int b, h, chunk, nch, len;
};

// What the end of a (sequence, head) costs a CTA, in units: the shares are cut
// by units plus this, so that a CTA with many short sequences gets fewer units
// (16 sequences of 1 to 4096 tokens, 40 query heads of 128: 31.6 us; 34.2 with
// 0, 31.9 with 4).
constexpr int kEnd = 2;

// Counts a part in; before it what this CTA wrote becomes visible, and behind
// it what the parts counted before wrote.
__device__ __forceinline__ unsigned count_part(unsigned* count) {
  unsigned before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  return before;
}

// Units of UNIT tokens of a sequence, per head.  SP: only selected blocks are
// attended, UNIT / 64 list entries to a unit.
template <bool SP, int UNIT>
__device__ __forceinline__ int units_of(const UnitArgs& a, int len) {
  static_assert(UNIT % Q2_BLOCK == 0, "a unit is made of blocks that q2_select selects");
  if (!SP) return (len + UNIT - 1) / UNIT;
  return (min((len + Q2_BLOCK - 1) / Q2_BLOCK, a.nsel) + UNIT / Q2_BLOCK - 1) / (UNIT / Q2_BLOCK);
}

// The order of units: each (sequence, head) has its units and kEnd places
// without one.  A CTA takes the units at places u0 .. u1 - 1.
struct Share {
  int total, ncta, u0, u1;
  __device__ int cta_of(int v) const { return (int)((((long long)v + 1) * ncta - 1) / total); }
};

// Shared memory behind a kernel's own: `nowed` (4 ints, at first how many CTAs
// have work), pre [batch + 1] places before each sequence, lens [batch].  Writes
// the outputs of sequences without a token, and of lengths that cannot be.
template <int D, bool SP, int UNIT>
__device__ __forceinline__ Share share_out(const UnitArgs& a, int* nowed, int* pre, int* lens, unsigned* error) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp == 0) {                                  // the units before each sequence
    int carry = 0, longest = 0, used = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + lane;
      int len = b < a.batch ? a.lens[b] : 0;
      if (len < 0 || len > a.cap) len = 0;
      if (b < a.batch) lens[b] = len;
      const int n = units_of<SP, UNIT>(a, len);
      longest = max(longest, n);
      used += __popc(__ballot_sync(0xffffffffu, len > 0));
      int v = len ? (n + kEnd) * a.hu : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (b < a.batch) pre[b + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      pre[0] = 0;
      // How many CTAs.  Each part of a (sequence, head) costs its join about a
      // quarter of what a unit costs its CTA, so n units are best cut into
      // about 2 sqrt(n) parts; with few (sequence, head)s, a multiple of their
      // number, so that sequences of one length are cut at their heads.  (Units
      // of the 4-bit cache and of selected blocks wait longer for their first
      // rows than they take: twice and one and a half times as many parts.  One
      // sequence of 777 tokens in 4 bits 8.0 -> 7.1 us.)
      constexpr float kParts = UNIT > kUnit ? 4.f : SP ? 3.f : 2.f;
      const int heads = used * a.hu, parts = max(1, (int)(kParts * sqrtf((float)longest)));
      *nowed = heads * 4 > (int)gridDim.x ? (int)gridDim.x : heads * min(parts, (int)gridDim.x / max(heads, 1));
    }
  }
  // sequences without a token give zeros, lengths that the table cannot hold NaN
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int len = a.lens[b];
    if (len > 0 && len <= a.cap) continue;
    if (len != 0 && threadIdx.x == 0) atomicOr(error, Q2_ERR_LENGTH);
    const int n = a.hu / a.nht * a.group * D;
    for (int e = threadIdx.x; e < n; e += kThreads)
      a.o[b * a.ldo + e] = len ? __ushort_as_half(0x7e00) : __ushort_as_half(0);
  }
  __syncthreads();
  Share s;
  s.total = pre[a.batch];
  s.ncta = min(*nowed, s.total);
  s.u0 = s.u1 = 0;
  if ((int)blockIdx.x < s.ncta) {
    const int each = s.total / s.ncta, over = s.total - each * s.ncta;
    auto first_of = [&](int cta) { return each * cta + over * cta / s.ncta; };   // total * cta / ncta in 32 bits
    s.u0 = first_of(blockIdx.x);
    s.u1 = first_of(blockIdx.x + 1);
  }
  return s;
}

// To the next unit; how many places further it is.
template <bool SP, int UNIT>
__device__ __forceinline__ int advance(const UnitArgs& a, const int* pre, const int* lens, Walk& w) {
  if (++w.chunk < w.nch) return 1;
  const int skipped = w.nch + kEnd - w.chunk;
  w.chunk = 0;
  if (++w.h == a.hu) {
    w.h = 0;
    do ++w.b;
    while (w.b < a.batch && pre[w.b + 1] == pre[w.b]);
    if (w.b < a.batch) {
      w.len = lens[w.b];
      w.nch = units_of<SP, UNIT>(a, w.len);
    }
  }
  return 1 + skipped;
}

// The unit at place u0, or the next one behind it (then u0 moves too).
template <bool SP, int UNIT>
__device__ __forceinline__ Walk walk_from(const UnitArgs& a, const int* pre, const int* lens, int& u0) {
  Walk c;
  int lo = 0, hi = a.batch - 1;                     // the sequence b with pre[b] <= u0 < pre[b + 1]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] <= u0) lo = mid + 1;
    else hi = mid;
  }
  c.b = lo;
  c.len = lens[lo];
  c.nch = units_of<SP, UNIT>(a, c.len);
  const int r = u0 - pre[lo];
  c.h = r / (c.nch + kEnd);
  c.chunk = r - c.h * (c.nch + kEnd);
  if (c.chunk >= c.nch) {                           // behind the last unit of a (sequence, head)
    --c.chunk;
    u0 += advance<SP, UNIT>(a, pre, lens, c) - 1;
  }
  return c;
}

// A denominator's reciprocal, of numerators that are `up` times too large; with
// SP nothing may have been selected, and nothing gives zeros.
template <bool SP>
__device__ __forceinline__ float part_of(float up, float l) {
  return SP && l == 0.f ? 0.f : 1.f / (up * l);
}

// The warps' sums of a (sequence, head), or of this CTA's share of it, joined:
// wml [kWarps][H] maximum and denominator, numerators of warp k at sums + k *
// wstride, row r of D floats in 16-byte pieces exchanged by r's low three bits.
// Writes the output (whole) or the part.  All threads, between two barriers.
template <int D, int H, bool SP>
__device__ __forceinline__ void join_warps(const UnitArgs& a, const unsigned char* sums, int wstride, const float2* wml,
                                           bool whole, int part, int rows, int b, int qh, float up) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;
  constexpr int PPL = D / kWarps / 16;              // 16-byte pieces of a lane: row lane / 4, a quarter of the warp's columns
#pragma unroll
  for (int row = g; row < H; row += 8) {
    float wt[kWarps], mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, wml[k * H + row].x);
    const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 v = wml[k * H + row];
      wt[k] = exp2f(v.x - ref);
      ll += wt[k] * v.y;
    }
    if (row < rows) {
      const float inv = part_of<SP>(up, ll);
#pragma unroll
      for (int q = 0; q < PPL; ++q) {
        const int piece4 = (warp * 4 + j) * PPL + q;          // columns 4 * piece4 ..
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(sums + k * wstride + row * (D * 4) + ((piece4 ^ g) << 4));
          x.x += v.x * wt[k];
          x.y += v.y * wt[k];
          x.z += v.z * wt[k];
          x.w += v.w * wt[k];
        }
        if (whole) {
          __half2 h[2] = {__floats2half2_rn(x.x * inv, x.y * inv), __floats2half2_rn(x.z * inv, x.w * inv)};
          *reinterpret_cast<uint2*>(a.o + b * a.ldo + (long long)(qh + row) * D + piece4 * 4) = *reinterpret_cast<uint2*>(h);
        } else {
          *reinterpret_cast<float4*>(a.part + ((size_t)part * H + row) * D + piece4 * 4) = x;
        }
      }
      if (!whole && warp == 0 && j == 0) a.ml[(size_t)part * H + row] = make_float2(mm, ll);
    }
  }
}

// Thread 0 counts this CTA's part of w's (sequence, head) in; the part that
// completes it owes its join.  A CTA has two parts at most (the one it begins
// with and the one it ends with) and joins at its end, so that nothing waits
// for the counter here.
__device__ __forceinline__ void owe_part(const UnitArgs& a, const Share& sh, const int* pre, const Walk& w, int4* owe,
                                         int& owed) {
  const unsigned before = count_part(a.count + (size_t)w.b * a.hu + w.h);
  // the CTAs that hold parts of this (sequence, head): c0 (from its first unit) .. c1
  const int s = pre[w.b] + w.h * (w.nch + kEnd);
  const int c0 = sh.cta_of(s), c1 = sh.cta_of(s + w.nch - 1);
  if (before == (unsigned)(c1 - c0)) owe[owed++] = make_int4(w.b, w.h, c0, c1);
}

// The joins that this CTA owes.  JOIN: parts whose loads are in flight together
// (a trip to memory per JOIN parts: one sequence of 131072 tokens in 4 bits, 38
// parts per head, 43.2 us with 8, 42.6 with 12, 41.1 with 20; but one of 777
// tokens, 7 parts, 7.3, 7.3 and 7.6: longer code).
template <int D, int H, bool SP, int JOIN>
__device__ __forceinline__ void join_parts(const UnitArgs& a, const int4* owe, int owed, float up) {
  for (int q = 0; q < owed; ++q) {
    const int4 w = owe[q];
    const int kvh = a.nht == 1 ? w.y : w.y / a.nht, ht = w.y - kvh * a.nht, rows = min(H, a.group - ht * H);
    const int parts = w.w - w.z + 1;
    if (threadIdx.x == 0) a.count[(size_t)w.x * a.hu + w.y] = 0;
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d4 = e % (D / 4);
      float mj = -INFINITY, lj = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int k0 = 0; k0 < parts; k0 += JOIN) {       // JOIN parts' loads at a time
        float2 v[JOIN];
        float4 f[JOIN];
#pragma unroll
        for (int k = 0; k < JOIN; ++k) {
          // the first CTA's second part, the others' first
          const size_t at = (size_t)(2 * (w.z + min(k0 + k, parts - 1)) + (k0 + k == 0)) * H + r;
          v[k] = __ldcg(&a.ml[at]);
          f[k] = __ldcg(reinterpret_cast<const float4*>(a.part + at * D) + d4);
          if (k0 + k >= parts) v[k].x = -INFINITY;
        }
        float mn = mj;
#pragma unroll
        for (int k = 0; k < JOIN; ++k) mn = fmaxf(mn, v[k].x);
        const float ref = mn == -INFINITY ? 0.f : mn, old = exp2f(mj - ref);
        mj = mn;
        lj *= old;
        x.x *= old;
        x.y *= old;
        x.z *= old;
        x.w *= old;
#pragma unroll
        for (int k = 0; k < JOIN; ++k) {
          if (k0 + k < parts) {
            const float wk = exp2f(v[k].x - ref);
            lj += wk * v[k].y;
            x.x += wk * f[k].x;
            x.y += wk * f[k].y;
            x.z += wk * f[k].z;
            x.w += wk * f[k].w;
          }
        }
      }
      const float inv = part_of<SP>(up, lj);
      __half2 h[2] = {__floats2half2_rn(x.x * inv, x.y * inv), __floats2half2_rn(x.z * inv, x.w * inv)};
      *reinterpret_cast<uint2*>(a.o + w.x * a.ldo + (long long)(kvh * a.group + ht * H + r) * D + d4 * 4) =
          *reinterpret_cast<uint2*>(h);
    }
  }
}

// The first token of the TW that a warp has of a unit; SP: behind the sequence's
// last where the list names no block.
template <bool SP, int UNIT, int TW>
__device__ __forceinline__ int first_token(const UnitArgs& a, const Walk& w, int warp, bool there) {
  if (!SP) return w.chunk * UNIT + warp * TW;
  const int kvh = a.nht == 1 ? w.h : w.h / a.nht, n = (w.len + Q2_BLOCK - 1) / Q2_BLOCK;
  const int i = w.chunk * (UNIT / Q2_BLOCK) + warp * TW / Q2_BLOCK;
  int block = n;
  if (there && i < min(n, a.nsel)) block = a.sel[((long long)w.b * (a.hu / a.nht) + kvh) * a.nsel + i];
  return ((unsigned)block < (unsigned)n ? block : n) * Q2_BLOCK + warp * TW % Q2_BLOCK;
}

// ---------------------------------------------------------------- host side

// The most CTAs per SM, and query heads of a unit, that any of the kernels has.
constexpr int most_ctas(int D) { return D == 64 ? 3 : 2; }
constexpr int most_heads(int D) { return D == 256 ? 8 : kMostHeads; }

// Parts of a call at most, two to a CTA, times their heads.
inline size_t part_rows(int D, int sms) { return (size_t)2 * most_ctas(D) * sms * most_heads(D); }

// The workspace: the parts' sums, in a region that fits every head_dim and both
// kinds of cache (so the counters behind it have one place for all calls), then
// counters.
inline size_t part_bytes(int sms) {
  size_t n = 0;
  for (int D : {64, 128, 256}) n = std::max(n, part_rows(D, sms) * (D * 4 + 8));
  return (n + 255) / 256 * 256;
}

// Query heads of a unit.  Sixteen where a key-value head has more than eight
// and the registers hold them, so that its tokens are read once for sixteen:
// there lo has its own products (52 to 56 us by the pages' order, instead of
// 89, for 8 sequences of 8192 tokens, 128 query and 8 key-value heads of 128).
inline int unit_heads(int group, int D) { return group > 8 && D <= 128 ? 16 : 8; }

// Shared checks of the head counts; hu: heads of units.
inline int check_heads(int batch, int q_heads, int kv_heads, int D, int* hu, int* nht) {
  if (batch < 0 || batch > Q2_ATT_MAX_BATCH || kv_heads < 1 || kv_heads > 65536 || q_heads < 1 || q_heads % kv_heads)
    return Q2_ESHAPE;
  if (q_heads / kv_heads > Q2_ATT_MAX_GROUP || (D != 64 && D != 128 && D != 256)) return Q2_ESHAPE;
  const int H = unit_heads(q_heads / kv_heads, D);
  *nht = (q_heads / kv_heads + H - 1) / H;
  *hu = kv_heads * *nht;
  return Q2_OK;
}

// The arguments that calls on both kinds of cache share.
struct UnitCall {
  const void* q;
  long long ldq;
  const int* lens;
  int batch, q_heads;
  const int* sel;
  int nsel;
  float scale;
  void* out;
  long long ldo;
  void* ws;
  size_t ws_bytes;
  long long units = 0;          // at most; set by fill()

  // What is refused even for a batch of none.
  template <class KV>
  int check(const KV* kv) const {
    int hu, nht;
    const int st = check_heads(batch, q_heads, kv->kv_heads, kv->head_dim, &hu, &nht);
    if (st) return st;
    if (kv->page_size < 1 || kv->npages < 0 || kv->max_pages < 0) return Q2_ESHAPE;
    return !(scale == scale) || scale - scale != 0.f ? Q2_EINVAL : Q2_OK;
  }

  int fill(const CacheShape& c, bool sp, UnitArgs& a) {
    int hu, nht;
    check_heads(batch, q_heads, c.kv_heads, c.D, &hu, &nht);
    if (!q || !lens || !out || (sp && !sel)) return Q2_EINVAL;
    const long long qw = (long long)q_heads * c.D;
    if (batch > 1 && (ldq < qw || ldo < qw)) return Q2_ESHAPE;
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(lens, 4) || misaligned(sel, 4) ||
        (batch > 1 && (ldq % 8 || ldo % 8)))
      return Q2_EALIGN;
    const size_t parts = part_bytes(dev_info().sms), need = parts + (size_t)batch * hu * 4;
    if (!ws || ws_bytes < need) return Q2_EWORKSPACE;
    if (misaligned(ws, 256)) return Q2_EALIGN;
    // units of all sequences are counted in 32 bits on the device
    units = c.cap / kUnit + 1;
    if (sp) units = std::min(units, (long long)nsel);
    units = (units + kEnd) * hu * batch;
    if (units > 0x7fffffffll) return Q2_ESHAPE;
    a.lens = lens;
    a.q = static_cast<const __half*>(q);
    a.o = static_cast<__half*>(out);
    a.ldq = ldq;
    a.ldo = ldo;
    a.part = static_cast<float*>(ws);
    a.count = reinterpret_cast<unsigned int*>(static_cast<char*>(ws) + parts);
    a.ml = reinterpret_cast<float2*>(a.part + part_rows(c.D, dev_info().sms) * c.D);
    a.sel = sel;
    a.nsel = nsel;
    a.batch = batch;
    a.cap = (int)c.cap;
    a.hu = hu;
    a.nht = nht;
    a.group = q_heads / c.kv_heads;
    a.sc2 = (float)((double)scale * 1.4426950408889634);
    return Q2_OK;
  }
};

}  // namespace q2
