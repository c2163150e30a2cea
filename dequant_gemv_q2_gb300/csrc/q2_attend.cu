// Attention of one new token per sequence over a paged key-value cache,
//
//   o[b][h] = sum_l p_l v_l / sum_l p_l,   p_l = exp(scale * q[b][h] . k_l),
//
// l over the sequence's lens[b] tokens, k and v of head h / (q_heads /
// kv_heads) (grouped heads).  Each token's key and value are read once for
// all query heads of the group and take part in 4 D operations per head, so
// the cache's bytes bound it.
//
// Work is cut into units of 64 tokens of one (sequence, key-value head), in
// the order (sequence, head, token), and every CTA takes an equal contiguous
// share of them, worked out on the device from lens: sequences of any mix of
// lengths load the SMs alike, and one long sequence spreads over all of them.
// Where a (sequence, head)'s units lie in several CTAs each leaves its sums
// (maximum, denominator, fp32 numerators) in the workspace, and the CTA that
// finishes last, by a counter, joins them in CTA order: one launch, and a
// result that does not depend on which was last.
//
// Inside a CTA the four warps take 16 tokens of a unit each, on their own:
// every warp has a ring of shared-memory stages that it fills with
// asynchronous 16-byte copies STAGES - 1 units ahead (across the ends of
// sequences and heads), its own running maximum, denominator and numerators,
// and meets the others only at the end of a (sequence, head).  Rows past a
// sequence's end are filled with zeros by the copy and masked, so what an
// unused part of a page holds (infinities, NaN) has no effect.  The 16-byte
// pieces of a row are exchanged by the row's low three bits, so that eight
// rows of one piece (what one matrix load takes) lie in different banks.
//
// Both products run on the tensor cores (16 x 8 x 16, fp32 accumulators) with
// the group's query heads as rows 0..7.  The probabilities, at most 1, are
// split into two fp16 numbers, 2^15 p = hi + lo, and lo takes rows 8..15 of the
// same instructions: an error of 2^-20 instead of 2^-11 per term at no cost
// (with more than eight heads lo has its own instructions).  The factor keeps
// small ones apart from fp16's smallest numbers: without it a p below 2^-14
// lost bits and one below 2^-25 was zero, and behind a token that takes nearly
// all of the weight and has a value near zero the output is made of those (8192
// tokens behind one with a score 18 above theirs: 1 % off, behind four 4 %).  More than 16
// query heads to a key-value head (eight of 256 columns) are taken 16 (eight)
// at a time, each reading the tokens again.
//
// 64 sequences of 8192 tokens, 32 query and 8 key-value heads of 128: 318 us
// on the device, 6.8 TB/s, the rate of a copy; one of 131072: 89 us, 6.0; 16
// of 1 to 4096 with 40 query heads 30 us, 4.5 (each CTA's start, its ends of
// sequences and the joins are 9 of them); one of 777 tokens 7.0 us: the
// lengths, the first pages' numbers, the first rows and the join behind one
// another.  Heads of 256 have one CTA per SM, whose threads spill 164 bytes at
// 255 registers: 64 of 4096 tokens 336 us, 6.4 TB/s, 16 of 2048 53, 5.0.
#include <cuda_fp16.h>

#include <algorithm>

#include "q2_common.cuh"

namespace q2 {
namespace {

__device__ unsigned int q2_attend_error;

constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16, kUnit = kTile * kWarps;   // tokens of a warp's tile, of a unit
constexpr int kMostHeads = 16;                      // query heads of a unit at most

struct AttendArgs {
  __half* k;
  __half* v;
  long long page_stride, token_stride, head_stride;
  const int* table;
  long long table_stride;
  const int* lens;
  const __half* q;
  const __half* nk;           // new keys and values, or null
  const __half* nv;
  __half* o;
  long long ldq, ldn, ldo;
  unsigned int* count;        // [batch][units' heads] arrivals, zero between calls
  float* part;                // [2 * CTAs][H][D] numerators, H the query heads of a unit
  float2* ml;                 // [2 * CTAs][H] maximum, denominator
  int batch, npages, page, cap;   // cap: tokens that a table row can hold
  int hu, nht, group;         // heads of units = kv_heads * nht; query heads of a key-value head
  uint32_t page_mul, page_sh; // t / page = (high half of t * page_mul, + t) >> page_sh, t < 2^31
  int aligned;                // page % 16 == 0: a tile lies in one page
  float sc2;                  // scale * log2(e)
};

// Division by an invariant with a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994).
__device__ __forceinline__ int page_of(const AttendArgs& a, int t) {
  return (int)((__umulhi((uint32_t)t, a.page_mul) + (uint32_t)t) >> a.page_sh);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

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

// 2^15 p0 and 2^15 p1 (0 <= p <= 1) as pairs of fp16 numbers whose sums they
// are, to 2^-20 of each or half of fp16's smallest, 2^-40 of the largest p.
// hi is cut off a little below 2^15 p and lo is the rest, so both are above
// zero where p is at least 2^-37: an infinite value times either has its sign
// (0 * inf and inf - inf would make NaN of it).
constexpr float kUp = 32768.f;
__device__ __forceinline__ void split2(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  constexpr float kCut = kUp * (1.f - 1.f / 4096.f), kLeast = 1.f / 16777216.f;
  asm("cvt.rz.relu.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(fmaf(p1, kCut, -kLeast)), "f"(fmaf(p0, kCut, -kLeast)));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  const __half2 l = __floats2half2_rn(fmaf(p0, kUp, -f.x), fmaf(p1, kUp, -f.y));
  lo = *reinterpret_cast<const uint32_t*>(&l);
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

// CTAs per SM: what registers and the rings of three stages leave room for, but
// no more than three (64 sequences of 8192 tokens, heads of 64, pages of 64
// stored head by head: 161 us; with two CTAs of six stages 199, with four of
// three 169; stored token by token 182).
template <int D>
__host__ __device__ constexpr int att_ctas() { return D == 64 ? 3 : D == 128 ? 2 : 1; }

template <int D, int H>
struct Shape {
  static constexpr int STAGES = 3;
  static constexpr int kTileBytes = kTile * D * 2;                     // keys or values of a tile
  static constexpr int kRing = kWarps * STAGES * 2 * kTileBytes;
  static constexpr int kMl = kWarps * H * 8;
  static constexpr int fixed = kRing + kMl + 48;
  static_assert(H * D * 4 <= 2 * kTileBytes, "a warp's numerators take the place of a tile's keys and values");
  static int smem(int batch) { return fixed + 4 * (2 * batch + 1); }
};

constexpr int kJoin = 8;                            // parts whose loads are in flight together in a join

// Counts a part in; before it what this CTA wrote becomes visible, and behind
// it what the parts counted before wrote.
__device__ __forceinline__ unsigned count_part(unsigned* count) {
  unsigned before;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(before) : "l"(count) : "memory");
  return before;
}

// H: query heads of a unit, 8 or 16 (rows of the products)
template <int D, int H>
__global__ void __launch_bounds__(kThreads, att_ctas<D>()) k_attend(const __grid_constant__ AttendArgs a) {
  using S = Shape<D, H>;
  constexpr int RH = H / 8;                         // rows g, g + 8 of a lane that are heads
  constexpr int STAGES = S::STAGES, CPR = D / 8, RPI = 32 / CPR, NT = D / 8;
  extern __shared__ __align__(128) unsigned char q2_att_smem[];
  float2* wml = reinterpret_cast<float2*>(q2_att_smem + S::kRing);     // [kWarps][H] maximum, denominator
  int4* owe = reinterpret_cast<int4*>(q2_att_smem + S::kRing + S::kMl);   // joins that are this CTA's: sequence, head, CTAs
  int* nowed = reinterpret_cast<int*>(owe + 2);                           // at first: how many CTAs have work
  int* pre = nowed + 4;                                                // [batch + 1] units before each sequence
  int* lens = pre + a.batch + 1;                                       // [batch] lengths; what cannot be is 0
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;

  pdl_wait();                                       // everything may come from the previous kernel
  pdl_trigger();
  if (warp == 0) {                                  // the units before each sequence
    int carry = 0, longest = 0, used = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
      const int b = b0 + lane;
      int len = b < a.batch ? a.lens[b] : 0;
      if (len < 0 || len > a.cap) len = 0;
      if (b < a.batch) lens[b] = len;
      longest = max(longest, (len + kUnit - 1) / kUnit);
      used += __popc(__ballot_sync(0xffffffffu, len > 0));
      int v = len ? ((len + kUnit - 1) / kUnit + kEnd) * a.hu : 0;
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
      // number, so that sequences of one length are cut at their heads.
      const int heads = used * a.hu, parts = max(1, (int)(2.f * sqrtf((float)longest)));
      *nowed = heads * 4 > (int)gridDim.x ? (int)gridDim.x : heads * min(parts, (int)gridDim.x / max(heads, 1));
    }
  }
  // sequences without a token give zeros, lengths that the table cannot hold NaN
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int len = a.lens[b];
    if (len > 0 && len <= a.cap) continue;
    if (len != 0 && threadIdx.x == 0) atomicOr(&q2_attend_error, Q2_ERR_LENGTH);
    const int n = a.hu / a.nht * a.group * D;
    for (int e = threadIdx.x; e < n; e += kThreads)
      a.o[b * a.ldo + e] = len ? __ushort_as_half(0x7e00) : __ushort_as_half(0);
  }
  __syncthreads();
    // The order of units: each (sequence, head) has its units and kEnd places
  // without one.  This CTA takes the units at places u0 .. u1 - 1.
  const int total = pre[a.batch], ncta = min(*nowed, total);
  if ((int)blockIdx.x >= ncta) return;
  const int each = total / ncta, over = total - each * ncta;
  auto first_of = [&](int cta) { return each * cta + over * cta / ncta; };   // total * cta / ncta in 32 bits
  int u0 = first_of(blockIdx.x);
  const int u1 = first_of(blockIdx.x + 1);

  Walk c;                                           // the unit in use
  {
    int lo = 0, hi = a.batch - 1;                   // the sequence b with pre[b] <= u0 < pre[b + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid + 1] <= u0) lo = mid + 1;
      else hi = mid;
    }
    c.b = lo;
    c.len = lens[lo];
    c.nch = (c.len + kUnit - 1) / kUnit;
    const int r = u0 - pre[lo];
    c.h = r / (c.nch + kEnd);
    c.chunk = r - c.h * (c.nch + kEnd);
  }
  // to the next unit; how many places further it is
  auto advance = [&](Walk& w) {
    if (++w.chunk < w.nch) return 1;
    const int skipped = w.nch + kEnd - w.chunk;
    w.chunk = 0;
    if (++w.h == a.hu) {
      w.h = 0;
      do ++w.b;
      while (w.b < a.batch && pre[w.b + 1] == pre[w.b]);
      if (w.b < a.batch) {
        w.len = lens[w.b];
        w.nch = (w.len + kUnit - 1) / kUnit;
      }
    }
    return 1 + skipped;
  };
  if (c.chunk >= c.nch) {                           // the share begins behind the last unit of a (sequence, head)
    --c.chunk;
    u0 += advance(c) - 1;
  }
  if (u0 >= u1) return;

  // ---- the warp's loads, STAGES - 1 units ahead of their use
  const uint32_t ring = saddr(q2_att_smem) + warp * (STAGES * 2 * S::kTileBytes);
  Walk p = c;
  int pu = u0, pslot = 0, ppage = -1;               // place of the unit to load, its stage, the page of this lane's row
  uint32_t badslots = 0;                            // stages with a row whose page does not exist
  const int piece = lane % CPR, row0 = lane / CPR;
  const long long lrow = row0 * a.token_stride + piece * 8;            // this lane's place in a tile that lies in one page
  const uint32_t ldst = ring + row0 * (D * 2), lpiece = (uint32_t)((piece ^ row0) << 4);   // row0 < 8; ring and rows on 128 bytes
  auto lookup = [&]() {                             // a tile in one page: its page; else lanes l and l + 16: that of row l
    const int t = p.chunk * kUnit + warp * kTile + (a.aligned ? 0 : lane & 15);
    ppage = pu < u1 && t < p.len ? a.table[p.b * a.table_stride + page_of(a, t)] : -1;
  };
  lookup();
  auto issue = [&]() {
    if (pu < u1) {
      const int t0 = p.chunk * kUnit + warp * kTile;
      if (t0 < p.len) {
        const int have = p.len - t0 - (a.nk ? 1 : 0);                  // rows to copy: the new token does not come from the cache
        const int kvh = a.nht == 1 ? p.h : p.h / a.nht;
        const uint32_t dst = ldst + pslot * (2 * S::kTileBytes);
        bool bad;
        if (a.aligned) {
          bad = (unsigned)ppage >= (unsigned)a.npages;
          const long long off = bad ? 0 : ppage * a.page_stride + (t0 - page_of(a, t0) * a.page) * a.token_stride +
                                              kvh * a.head_stride + lrow;
          const __half* k = a.k + off;
          const __half* v = a.v + off;
          const long long step = RPI * a.token_stride;
          const int rows = bad ? 0 : have - row0;                      // live rows from this lane's first on
#pragma unroll
          for (int i = 0; i < kTile / RPI; ++i) {
            const uint32_t d = ((dst + lpiece) ^ (((i * RPI) & 7) << 4)) + i * (RPI * D * 2);
            const bool live = i * RPI < rows;       // else nothing is read: a row of the page all the same
            cp16(d, k, live);
            cp16(d + S::kTileBytes, v, live);
            k += step;
            v += step;
          }
        } else {
          const int t = t0 + (lane & 15);
          const bool there = (unsigned)ppage < (unsigned)a.npages;
          bad = __any_sync(0xffffffffu, t < p.len && !there);
          const long long off = (lane & 15) < have && there
                                    ? ppage * a.page_stride + (t - page_of(a, t) * a.page) * a.token_stride + kvh * a.head_stride
                                    : -1;
#pragma unroll 2
          for (int i = 0; i < kTile / RPI; ++i) {
            const int row = i * RPI + row0;
            const long long o = __shfl_sync(0xffffffffu, off, row);
            const long long e = (o < 0 ? 0 : o) + piece * 8;
            const uint32_t d = dst + i * (RPI * D * 2) + ((piece ^ (row & 7)) << 4);
            cp16(d, a.k + e, o >= 0);
            cp16(d + S::kTileBytes, a.v + e, o >= 0);
          }
        }
        if (bad && lane == 0) atomicOr(&q2_attend_error, Q2_ERR_PAGE);
        badslots = (badslots & ~(1u << pslot)) | (bad ? 1u << pslot : 0u);
      }
      pu += advance(p);
      lookup();
      pslot = pslot + 1 == STAGES ? 0 : pslot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // ---- sums of the current (sequence, head)
  uint32_t qa[D / 16][2 * RH];                      // the queries: rows g (+ 8), columns 2j.. and 2j + 8.. of each 16
  uint4 newk, newv;                                 // lane l < CPR: piece l of the new token's key and value
  float o[NT][4], m[RH], l[RH];
  bool fresh = true;
  int seg = c.chunk, slot = 0;                      // first unit of this part of the (sequence, head)
  int ahead = STAGES - 1;                           // units still to be requested before the first is used
  int owed = 0;                                     // parts of this CTA that were the last of their (sequence, head)
  for (int u = u0; u < u1;) {
    const int kvh = a.nht == 1 ? c.h : c.h / a.nht, ht = c.h - kvh * a.nht, rows = min(H, a.group - ht * H);
    const int qh = kvh * a.group + ht * H;
    const int t0 = c.chunk * kUnit + warp * kTile;
    if (fresh) {
      fresh = false;
      const __half* q = a.q + c.b * a.ldq + (long long)(qh + g) * D + 2 * j;
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int y = 0; y < RH; ++y) {
          const bool is = g + 8 * y < rows;
          qa[s][2 * y] = is ? *reinterpret_cast<const uint32_t*>(q + 8 * y * D + 16 * s) : 0u;
          qa[s][2 * y + 1] = is ? *reinterpret_cast<const uint32_t*>(q + 8 * y * D + 16 * s + 8) : 0u;
        }
      if (a.nk && lane < CPR) {
        const long long e = c.b * a.ldn + kvh * D + lane * 8;
        newk = *reinterpret_cast<const uint4*>(a.nk + e);
        newv = *reinterpret_cast<const uint4*>(a.nv + e);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][x] = 0.f;
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        m[y] = -INFINITY;
        l[y] = 0.f;
      }
    }
    if (!ahead) {                                   // this unit has arrived for all lanes, the one before is done with
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncwarp();
    }
    issue();                                        // (in one place: a short call's time is a good part instruction fetch)
    if (ahead) {
      --ahead;
      continue;
    }
    if (t0 < c.len) {
      const uint32_t kt = ring + slot * (2 * S::kTileBytes), vt = kt + S::kTileBytes;
      const int fin = c.len - 1 - t0;               // row of the last token, if below kTile
      if (a.nk && fin < kTile) {                    // the new token's row, and its place in the cache
        if (lane < CPR) {
          const uint32_t d = fin * (D * 2) + ((lane ^ (fin & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(kt + d), "r"(newk.x), "r"(newk.y), "r"(newk.z),
                       "r"(newk.w)
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(vt + d), "r"(newv.x), "r"(newv.y), "r"(newv.z),
                       "r"(newv.w)
                       : "memory");
          const int at = page_of(a, c.len - 1), page = a.table[c.b * a.table_stride + at];
          if (ht == 0 && (unsigned)page < (unsigned)a.npages) {
            const long long e = page * a.page_stride + (c.len - 1 - at * a.page) * a.token_stride + kvh * a.head_stride +
                                lane * 8;
            *reinterpret_cast<uint4*>(a.k + e) = newk;
            *reinterpret_cast<uint4*>(a.v + e) = newv;
          }
        }
        __syncwarp();
      }
      // scores of 16 tokens: columns 2j, 2j + 1 of tokens 0..7 (s0) and 8..15 (s1)
      float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
      const int krow = (lane & 7) + ((lane >> 4) << 3), kpiece = (lane >> 3) & 1;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        uint32_t b[4];
        ldsm4(b, kt + krow * (D * 2) + (((2 * s + kpiece) ^ (krow & 7)) << 4));
        const uint32_t a1 = RH == 2 ? qa[s][2 * RH - 2] : 0u, a3 = RH == 2 ? qa[s][2 * RH - 1] : 0u;
        mma(s0, qa[s][0], a1, qa[s][1], a3, b[0], b[1]);
        mma(s1, qa[s][0], a1, qa[s][1], a3, b[2], b[3]);
      }
      float x[RH][4], al[RH];
      bool rise = false;
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        x[y][0] = s0[2 * y] * a.sc2;
        x[y][1] = s0[2 * y + 1] * a.sc2;
        x[y][2] = s1[2 * y] * a.sc2;
        x[y][3] = s1[2 * y + 1] * a.sc2;
        if (fin < kTile - 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (2 * j + (e & 1) + (e >> 1) * 8 > fin) x[y][e] = -INFINITY;
        }
        float top = fmaxf(fmaxf(x[y][0], x[y][1]), fmaxf(x[y][2], x[y][3]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float mn = fmaxf(m[y], top), ref = mn == -INFINITY ? 0.f : mn;
        rise = rise || mn > m[y];
        al[y] = exp2f(m[y] - ref);
        m[y] = mn;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[y][e] = exp2f(x[y][e] - ref);
      }
      if (__any_sync(0xffffffffu, rise)) {          // a new maximum somewhere: scale what there is
#pragma unroll
        for (int y = 0; y < RH; ++y) l[y] *= al[y];
#pragma unroll
        for (int t = 0; t < NT; ++t) {              // of 8 heads rows 0..7 and 8..15 are halves of the same head
          o[t][0] *= al[0];
          o[t][1] *= al[0];
          o[t][2] *= al[RH - 1];
          o[t][3] *= al[RH - 1];
        }
      }
      uint32_t hi[RH][2], lo[RH][2];
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        l[y] += (x[y][0] + x[y][1]) + (x[y][2] + x[y][3]);
        if ((badslots >> slot) & 1u) l[y] = __int_as_float(0x7fc00000);
        split2(x[y][0], x[y][1], hi[y][0], lo[y][0]);
        split2(x[y][2], x[y][3], hi[y][1], lo[y][1]);
      }
      const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vpiece = lane >> 4;
#pragma unroll
      for (int t = 0; t < NT; t += 2) {
        uint32_t b[4];
        ldsm4t(b, vt + vrow * (D * 2) + (((t + vpiece) ^ (vrow & 7)) << 4));
        if constexpr (RH == 1) {                    // hi in rows 0..7, lo in rows 8..15
          mma(o[t], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[0], b[1]);
          mma(o[t + 1], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[2], b[3]);
        } else {
          mma(o[t], hi[0][0], hi[1][0], hi[0][1], hi[1][1], b[0], b[1]);
          mma(o[t + 1], hi[0][0], hi[1][0], hi[0][1], hi[1][1], b[2], b[3]);
          mma(o[t], lo[0][0], lo[1][0], lo[0][1], lo[1][1], b[0], b[1]);
          mma(o[t + 1], lo[0][0], lo[1][0], lo[0][1], lo[1][1], b[2], b[3]);
        }
      }
    }
    const uint32_t mine = slot * (2 * S::kTileBytes);       // this unit's stage, free until the next issue()
    slot = slot + 1 == STAGES ? 0 : slot + 1;

    const Walk w = c;
    u += advance(c);
    const bool ends = w.chunk + 1 == w.nch, all = u >= u1;
    if (ends || all) {                              // the end of this (sequence, head), or of this CTA's share of it
      // Every warp leaves its sums (the numerators in place of the keys it has
      // just used, 16-byte pieces exchanged by the row as the keys were), then
      // joins a quarter of the columns of all warps.
      unsigned char* sums = q2_att_smem + warp * (STAGES * 2 * S::kTileBytes) + mine;
      __syncwarp();
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
        if (j == 0) wml[warp * H + g + 8 * y] = make_float2(m[y], l[y]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          *reinterpret_cast<float2*>(sums + (g + 8 * y) * (D * 4) + (((2 * t + (j >> 1)) ^ g) << 4) + (j & 1) * 8) =
              RH == 1 ? make_float2(o[t][0] + o[t][2], o[t][1] + o[t][3]) : make_float2(o[t][2 * y], o[t][2 * y + 1]);
      }
      __syncthreads();
      const bool whole = ends && seg == 0;
      const int part = 2 * (int)blockIdx.x + (seg == 0 ? 1 : 0);
      constexpr int PPL = D / kWarps / 16;          // 16-byte pieces of a lane: row lane / 4, a quarter of the warp's columns
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
          const float inv = 1.f / (kUp * ll);      // (the numerators are 2^15 too large)
#pragma unroll
          for (int q = 0; q < PPL; ++q) {
            const int piece4 = (warp * 4 + j) * PPL + q;      // columns 4 * piece4 ..
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
              const float4 v = *reinterpret_cast<const float4*>(q2_att_smem + k * (STAGES * 2 * S::kTileBytes) + mine +
                                                                row * (D * 4) + ((piece4 ^ g) << 4));
              x.x += v.x * wt[k];
              x.y += v.y * wt[k];
              x.z += v.z * wt[k];
              x.w += v.w * wt[k];
            }
            if (whole) {
              __half2 h[2] = {__floats2half2_rn(x.x * inv, x.y * inv), __floats2half2_rn(x.z * inv, x.w * inv)};
              *reinterpret_cast<uint2*>(a.o + w.b * a.ldo + (long long)(qh + row) * D + piece4 * 4) = *reinterpret_cast<uint2*>(h);
            } else {
              *reinterpret_cast<float4*>(a.part + ((size_t)part * H + row) * D + piece4 * 4) = x;
            }
          }
          if (!whole && warp == 0 && j == 0) a.ml[(size_t)part * H + row] = make_float2(mm, ll);
        }
      }
      __syncthreads();                              // the stages may be filled again; the part is written
      if (!whole) {
        // The part that completes a (sequence, head) owes its join; a CTA has
        // two parts at most (the one it begins with and the one it ends with)
        // and joins at its end, so that nothing waits for the counter here.
        if (threadIdx.x == 0) {
          const unsigned before = count_part(a.count + (size_t)w.b * a.hu + w.h);
          // the CTAs that hold parts of this (sequence, head): c0 (from its first unit) .. c1
          const int s = pre[w.b] + w.h * (w.nch + kEnd);
          auto cta_of = [&](int v) { return (int)((((long long)v + 1) * ncta - 1) / total); };
          const int c0 = cta_of(s), c1 = cta_of(s + w.nch - 1);
          if (before == (unsigned)(c1 - c0)) owe[owed++] = make_int4(w.b, w.h, c0, c1);
        }
      }
      fresh = true;
      seg = 0;
    }
  }

  if (threadIdx.x == 0) *nowed = owed;
  __syncthreads();
  for (int q = 0; q < *nowed; ++q) {
    const int4 w = owe[q];
    const int kvh = a.nht == 1 ? w.y : w.y / a.nht, ht = w.y - kvh * a.nht, rows = min(H, a.group - ht * H);
    const int parts = w.w - w.z + 1;
    if (threadIdx.x == 0) a.count[(size_t)w.x * a.hu + w.y] = 0;
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
      const int r = e / (D / 4), d4 = e % (D / 4);
      float mj = -INFINITY, lj = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int k0 = 0; k0 < parts; k0 += kJoin) {       // kJoin parts' loads at a time
        float2 v[kJoin];
        float4 f[kJoin];
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
          // the first CTA's second part, the others' first
          const size_t at = (size_t)(2 * (w.z + min(k0 + k, parts - 1)) + (k0 + k == 0)) * H + r;
          v[k] = __ldcg(&a.ml[at]);
          f[k] = __ldcg(reinterpret_cast<const float4*>(a.part + at * D) + d4);
          if (k0 + k >= parts) v[k].x = -INFINITY;
        }
        float mn = mj;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) mn = fmaxf(mn, v[k].x);
        const float ref = mn == -INFINITY ? 0.f : mn, old = exp2f(mj - ref);
        mj = mn;
        lj *= old;
        x.x *= old;
        x.y *= old;
        x.z *= old;
        x.w *= old;
#pragma unroll
        for (int k = 0; k < kJoin; ++k) {
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
      const float inv = 1.f / (kUp * lj);
      __half2 h[2] = {__floats2half2_rn(x.x * inv, x.y * inv), __floats2half2_rn(x.z * inv, x.w * inv)};
      *reinterpret_cast<uint2*>(a.o + w.x * a.ldo + (long long)(kvh * a.group + ht * H + r) * D + d4 * 4) =
          *reinterpret_cast<uint2*>(h);
    }
  }
}

int most_ctas(int D, int sms) { return sms * (D == 64 ? att_ctas<64>() : D == 128 ? att_ctas<128>() : att_ctas<256>()); }

// The workspace: the parts' sums, in a region that fits every head_dim (so the
// counters behind it have one place for calls of all shapes), then counters.
size_t part_bytes(int sms) {
  size_t n = 0;
  for (int D : {64, 128, 256}) n = std::max(n, (size_t)2 * most_ctas(D, sms) * kMostHeads * (D * 4 + 8));
  return (n + 255) / 256 * 256;
}

// Query heads of a unit.  Sixteen where a key-value head has more than eight
// and the registers hold them, so that its tokens are read once for sixteen:
// there lo has its own products (52 to 56 us by the pages' order, instead of
// 89, for 8 sequences of 8192 tokens, 128 query and 8 key-value heads of 128).
int unit_heads(int group, int D) { return group > 8 && D <= 128 ? 16 : 8; }

// Shared checks of the head counts; hu: heads of units.
int check_heads(int batch, int q_heads, int kv_heads, int D, int* hu, int* nht) {
  if (batch < 0 || batch > Q2_ATT_MAX_BATCH || kv_heads < 1 || kv_heads > 65536 || q_heads < 1 || q_heads % kv_heads)
    return Q2_ESHAPE;
  if (q_heads / kv_heads > Q2_ATT_MAX_GROUP || (D != 64 && D != 128 && D != 256)) return Q2_ESHAPE;
  const int H = unit_heads(q_heads / kv_heads, D);
  *nht = (q_heads / kv_heads + H - 1) / H;
  *hu = kv_heads * *nht;
  return Q2_OK;
}

}  // namespace
}  // namespace q2

using namespace q2;

extern "C" int q2_attend_workspace_bytes(int batch, int q_heads, int kv_heads, int head_dim, size_t* bytes) {
  if (!bytes) return Q2_EINVAL;
  int hu, nht;
  const int st = check_heads(batch, q_heads, kv_heads, head_dim, &hu, &nht);
  if (st) return st;
  *bytes = part_bytes(dev_info().sms) + (size_t)batch * hu * 4;
  return Q2_OK;
}

extern "C" int q2_attend(const q2_kv* kv, const void* q, long long ldq, const void* new_k, const void* new_v,
                         long long ldn, const int* lens, int batch, int q_heads, float scale, void* out, long long ldo,
                         void* ws, size_t ws_bytes, q2_stream stream) {
  if (!kv || (!new_k) != (!new_v)) return Q2_EINVAL;
  const int D = kv->head_dim;
  int hu, nht;
  int st = check_heads(batch, q_heads, kv->kv_heads, D, &hu, &nht);
  if (st) return st;
  if (kv->page_size < 1 || kv->npages < 0 || kv->max_pages < 0) return Q2_ESHAPE;
  if (!(scale == scale) || scale - scale != 0.f) return Q2_EINVAL;
  if (batch == 0) return Q2_OK;
  if (!q || !lens || !out || !kv->k || !kv->v || !kv->table) return Q2_EINVAL;
  const long long qw = (long long)q_heads * D, kw = (long long)kv->kv_heads * D;
  if (batch > 1 && (ldq < qw || ldo < qw || (new_k && ldn < kw) || kv->table_stride < kv->max_pages)) return Q2_ESHAPE;
  if (kv->page_stride < 0 || kv->token_stride < 0 || kv->head_stride < 0) return Q2_ESHAPE;
  auto off = [](const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
  if (off(q, 16) || off(out, 16) || off(new_k, 16) || off(new_v, 16) || off(kv->k, 16) || off(kv->v, 16) ||
      off(kv->table, 4) || off(lens, 4) || kv->page_stride % 8 || kv->token_stride % 8 || kv->head_stride % 8 ||
      (batch > 1 && (ldq % 8 || ldo % 8 || (new_k && ldn % 8))))
    return Q2_EALIGN;
  const int sms = dev_info().sms;
  const size_t parts = part_bytes(sms), need = parts + (size_t)batch * hu * 4;
  if (!ws || ws_bytes < need) return Q2_EWORKSPACE;
  if (off(ws, 256)) return Q2_EALIGN;
  // tokens of a table row, and of all units: both are counted in 32 bits on the device
  const long long cap = (long long)kv->max_pages * kv->page_size;
  const long long units = (cap / kUnit + 1 + kEnd) * hu * batch;
  if (cap > 0x7fffff00ll || units > 0x7fffffffll) return Q2_ESHAPE;
  AttendArgs a = {};
  a.k = static_cast<__half*>(kv->k);
  a.v = static_cast<__half*>(kv->v);
  a.page_stride = kv->page_stride;
  a.token_stride = kv->token_stride;
  a.head_stride = kv->head_stride;
  a.table = kv->table;
  a.table_stride = kv->table_stride;
  a.lens = lens;
  a.q = static_cast<const __half*>(q);
  a.nk = static_cast<const __half*>(new_k);
  a.nv = static_cast<const __half*>(new_v);
  a.o = static_cast<__half*>(out);
  a.ldq = ldq;
  a.ldn = ldn;
  a.ldo = ldo;
  const int most = most_ctas(D, sms);
  a.part = static_cast<float*>(ws);
  a.count = reinterpret_cast<unsigned int*>(static_cast<char*>(ws) + parts);
  a.ml = reinterpret_cast<float2*>(a.part + (size_t)2 * most * unit_heads(q_heads / kv->kv_heads, D) * D);
  a.batch = batch;
  a.npages = kv->npages;
  a.page = kv->page_size;
  a.aligned = kv->page_size % kTile == 0;
  while ((1ll << a.page_sh) < a.page) ++a.page_sh;
  a.page_mul = (uint32_t)(((1ull << 32) * ((1ull << a.page_sh) - a.page)) / a.page + 1);
  a.cap = (int)cap;
  a.hu = hu;
  a.nht = nht;
  a.group = q_heads / kv->kv_heads;
  a.sc2 = (float)((double)scale * 1.4426950408889634);
  const int grid = units < most ? (int)units : most;
  auto launch = [&](auto kernel, int smem) { return launch_pdl(kernel, a, grid, kThreads, smem, stream); };
  const bool wide = unit_heads(a.group, D) == 16;
  if (D == 64) return wide ? launch(k_attend<64, 16>, Shape<64, 16>::smem(batch)) : launch(k_attend<64, 8>, Shape<64, 8>::smem(batch));
  if (D == 128)
    return wide ? launch(k_attend<128, 16>, Shape<128, 16>::smem(batch)) : launch(k_attend<128, 8>, Shape<128, 8>::smem(batch));
  return launch(k_attend<256, 8>, Shape<256, 8>::smem(batch));
}

// The error word of the attention kernels, then cleared (q2_device_errors).
extern "C" int q2_attend_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_attend_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_attend_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
