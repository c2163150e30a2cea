// Attention of one new token per sequence over a paged key-value cache in 4
// bits,
//
//   o[b][h] = sum_l p_l v_l / sum_l p_l,   p_l = exp(scale * q[b][h] . k_l),
//
// where column d of k_l is m + s c: a code c of 0..15, and the (s, m) of the
// column's group of 32 or 64.  With both products taken apart by groups,
//
//   q . k_l          = sum_g  s_lg (sum_d q_d c_ld) + m_lg (sum_d q_d)
//   sum_l p_l v_ld   = sum_l (p_l s_lg) (c_ld - 8) + sum_l p_l (m_lg + 8 s_lg),
//
// the codes go to the tensor cores as small numbers and no value is ever
// expanded: what depends on s and m is done per (token, group), not per column.
//
// Units, shares, joins, rings and the softmax are those of the fp16 cache (see
// q2_attend.cu).  What differs:
//
// A 16-bit word holds four columns of a row; loaded by ldmatrix, a register
// holds two words, of neighbouring columns of one token (keys) or of one place
// in neighbouring tokens (values, transposed), so one masked register is an
// operand of the tensor instruction.  The columns' order inside the sums is that
// of the words; the queries, and the places of the outputs, follow it.
//
// Keys: four bits masked out of an fp16 number are one below the normal ones, c
// 2^-22 in bits 2..5 and c 2^-18 in bits 6..9: three instructions for two
// registers of operands.  (The tensor cores align such products as if they were
// 2^-14 and cut them off: an error of 2^-16 of a step times the largest q column
// there.  Bits 0..3 and 4..7 would save one shift in six and lose two bits more.)
//
// Values: c - 8, by 1024 + c and a subtraction, two instructions for a register.
// With c itself both terms of the numerator are some eight steps times the
// denominator and nearly cancel, and the fp32 sums' roundings showed in a long
// sequence's output (one of 131072 tokens: 4.1e-4 off, 2.1e-4 of it fp16's own).
//
// p s is split into two fp16 numbers, in the two halves of the rows as p is for
// the fp16 cache.  It is scaled by a power of two above the largest s so far
// (of the warp's tiles), which changes as rarely as the maximum does.
#include "q2_attend.cuh"

namespace q2 {
namespace {

__device__ unsigned int q2_attend4_error;

struct Attend4Args : UnitArgs {
  Pages pg;                     // codes
  Pages sp;                     // steps and offsets
  int aligned;                  // page % 16 == 0: a tile lies in one page
};

template <int D>
__host__ __device__ constexpr int ctas_of() { return D == 256 ? 1 : D == 128 ? 2 : 3; }

template <int D, int G, int H>
struct Shape {
  static constexpr int STAGES = 4;
  static constexpr int kCodes = kTile * D / 2, kPairs = kTile * G * 4;   // bytes of a tile, keys or values
  static constexpr int kStage = 2 * (kCodes + kPairs);
  static constexpr int kRing = kWarps * STAGES * kStage;
  static constexpr int kSums = H * D * 4;                                // a warp's numerators
  static constexpr int kMl = kWarps * H * 8;
  static constexpr int fixed = kRing + kWarps * kSums + kMl + 48;
  static_assert(kStage % 128 == 0, "stages begin on 128 bytes");
  static int smem(int batch) { return fixed + 4 * (2 * batch + 1); }
};

template <int N>
__device__ __forceinline__ void cp_pairs(uint32_t dst, const void* src, bool live) {
  if constexpr (N == 32) {
    cp16(dst, src, live);
    cp16(dst + 16, static_cast<const char*>(src) + 16, live);
  } else if constexpr (N == 16) {
    cp16(dst, src, live);
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0) : "memory");
  }
}

// The (step, offset) of group g of tokens t and t + 1 of a tile.
template <int G>
__device__ __forceinline__ void pairs_of(const unsigned char* tile, int t, int g, float2& a, float2& b) {
  const __half2* h = reinterpret_cast<const __half2*>(tile) + t * G + g;
  a = __half22float2(h[0]);
  b = __half22float2(h[G]);
}

// w0, w1 >= 0 as pairs of fp16 numbers whose sums they are, to 2^-22.
__device__ __forceinline__ void split2(float w0, float w1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(w0, w1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(w0 - f.x, w1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

// Codes in bits 0..3 (high: 4..7) of both halves as c - 8 in fp16: 1024 + c (1024 + 16 c), then what is too much.
__device__ __forceinline__ uint32_t centred(uint32_t w, bool high) {
  const uint32_t x = (w & (high ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
  const __half2 h = *reinterpret_cast<const __half2*>(&x);
  const __half2 y = high ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.f)) : __hsub2(h, __float2half2_rn(1032.f));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// H: query heads of a unit, 8 or 16 (rows of the products); G: groups of a row
template <int D, int G, int H, bool SP>
__global__ void __launch_bounds__(kThreads, ctas_of<D>()) k_attend4(const __grid_constant__ Attend4Args a) {
  using S = Shape<D, G, H>;
  constexpr int RH = H / 8, STAGES = S::STAGES, NB = D / 32;   // NB: 16-byte pieces of a row, 32 columns each
  constexpr int RPI = 32 / NB, NT = D / 8, BPG = NB / G;       // BPG: pieces of a group
  extern __shared__ __align__(128) unsigned char q2_att4_smem[];
  unsigned char* sums = q2_att4_smem + S::kRing;
  float2* wml = reinterpret_cast<float2*>(sums + kWarps * S::kSums);     // [kWarps][H] maximum, denominator
  int4* owe = reinterpret_cast<int4*>(wml + kWarps * H);
  int* nowed = reinterpret_cast<int*>(owe + 2);
  int* pre = nowed + 4;
  int* lens = pre + a.batch + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, j = lane & 3;

  pdl_wait();
  pdl_trigger();
  const Share sh = share_out<D, SP>(a, nowed, pre, lens, &q2_attend4_error);
  int u0 = sh.u0;
  const int u1 = sh.u1;
  if (u0 >= u1) return;
  Walk c = walk_from<SP>(a, pre, lens, u0);         // the unit in use
  if (u0 >= u1) return;

  // ---- the warp's loads, STAGES - 1 units ahead of their use
  unsigned char* const myring = q2_att4_smem + warp * (STAGES * S::kStage);
  const uint32_t ring = saddr(myring);
  Walk p = c;
  int pu = u0, pslot = 0, ppage = -1, pt0 = 0;      // place of the unit to load, its stage, page of this lane's row, first token
  uint32_t badslots = 0, haves = 0;                 // stages with a row whose page does not exist; a stage's tokens, 5 bits each
  const int piece = lane % NB, row0 = lane / NB;
  // the pieces of a row are exchanged so that eight rows of one piece lie in different banks
  auto place = [&](int row, int pc) { return row * (D / 2) + ((pc ^ (row / (8 / NB) & (NB - 1))) << 4); };
  auto lookup = [&]() {                             // a tile in one page: its page; else lanes l and l + 16: that of row l
    pt0 = (SP ? block_of(a, p, pu < u1) : p.chunk) * kUnit + warp * kTile;
    const int t = pt0 + (a.aligned ? 0 : lane & 15);
    ppage = pu < u1 && t < p.len ? a.pg.table[p.b * a.pg.table_stride + page_of(a.pg, t)] : -1;
  };
  lookup();
  auto issue = [&]() {
    if (pu < u1) {
      const int have = min(max(p.len - pt0, 0), kTile);
      haves = (haves & ~(31u << (5 * pslot))) | (uint32_t)have << (5 * pslot);
      if (have) {
        const int kvh = a.nht == 1 ? p.h : p.h / a.nht;
        const uint32_t dst = ring + pslot * S::kStage;
        // codes: this lane's piece of rows row0, row0 + RPI, ..; pairs: row lane % 16 of the keys, above lane 16 of the values
        const int t = pt0 + (a.aligned ? 0 : lane & 15), pi = page_of(a.pg, t);
        const bool there = (unsigned)ppage < (unsigned)a.pg.npages;
        const bool bad = __any_sync(0xffffffffu, t < p.len && !there);
        const int at = t - pi * a.pg.page;          // the place in the page of the tile's first token, or of this lane's row
        const int prow = lane & 15;
        const unsigned char* ps = (lane < 16 ? a.sp.k : a.sp.v);
        if (there)
          ps += ppage * a.sp.page_stride + (at + (a.aligned ? prow : 0)) * a.sp.token_stride + kvh * a.sp.head_stride;
        cp_pairs<4 * G>(dst + 2 * S::kCodes + (lane < 16 ? 0 : S::kPairs) + prow * (4 * G), ps, there && prow < have);
        if (a.aligned) {
          const long long off = there ? ppage * a.pg.page_stride + (at + row0) * a.pg.token_stride + kvh * a.pg.head_stride : 0;
          const unsigned char* k = a.pg.k + off + piece * 16;
          const unsigned char* v = a.pg.v + off + piece * 16;
#pragma unroll
          for (int i = 0; i < kTile / RPI; ++i) {
            const bool live = there && row0 + i * RPI < have;
            const uint32_t d = dst + place(row0 + i * RPI, piece);
            const long long step = live ? i * RPI * a.pg.token_stride : 0;
            cp16(d, k + step, live);
            cp16(d + S::kCodes, v + step, live);
          }
        } else {
          const long long off =
              there ? ppage * a.pg.page_stride + at * a.pg.token_stride + kvh * a.pg.head_stride : -1;
#pragma unroll
          for (int i = 0; i < kTile / RPI; ++i) {
            const int row = row0 + i * RPI;
            const long long o = __shfl_sync(0xffffffffu, off, row);
            const bool live = o >= 0 && row < have;
            const long long e = (live ? o : 0) + piece * 16;
            const uint32_t d = dst + place(row, piece);
            cp16(d, a.pg.k + e, live);
            cp16(d + S::kCodes, a.pg.v + e, live);
          }
        }
        if (bad && lane == 0) atomicOr(&q2_attend4_error, Q2_ERR_PAGE);
        badslots = (badslots & ~(1u << pslot)) | (bad ? 1u << pslot : 0u);
      }
      pu += advance<SP>(a, pre, lens, p);
      lookup();
      pslot = pslot + 1 == STAGES ? 0 : pslot + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // ---- sums of the current (sequence, head)
  uint32_t qa[NB][RH][4];                           // the queries of 32 columns: codes 0 and 2, then 1 and 3 of the words 2j, 2j + 1
  float qs[RH][G];                                  // their sums over the groups
  float o[NT][4], om[RH][G], m[RH], l[RH];          // numerators of codes and of offsets, maximum, denominator
  uint32_t top_s = 1;                               // exponent field of the largest step so far, 1 at least
  bool fresh = true;
  int seg = c.chunk, slot = 0;
  int ahead = STAGES - 1;
  int owed = 0;
  for (int u = u0; u < u1;) {
    const int kvh = a.nht == 1 ? c.h : c.h / a.nht, ht = c.h - kvh * a.nht, rows = min(H, a.group - ht * H);
    const int qh = kvh * a.group + ht * H;
    if (fresh) {
      fresh = false;
      top_s = 1;
      const __half* q = a.q + c.b * a.ldq + (long long)(qh + g) * D + 8 * j;
#pragma unroll
      for (int y = 0; y < RH; ++y) {
#pragma unroll
        for (int i = 0; i < G; ++i) qs[y][i] = om[y][i] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 r = g + 8 * y < rows ? *reinterpret_cast<const uint4*>(q + 8 * y * D + 32 * b) : make_uint4(0u, 0u, 0u, 0u);
          // columns 8j .. 8j + 7 are r.x = (0, 1), r.y = (2, 3), r.z = (4, 5), r.w = (6, 7); words 2j and 2j + 1 are 0..3 and 4..7
          qa[b][y][0] = __byte_perm(r.x, r.z, 0x5410);          // (0, 4): code 0
          qa[b][y][1] = __byte_perm(r.y, r.w, 0x5410);          // (2, 6): code 2
          qa[b][y][2] = __byte_perm(r.x, r.z, 0x7632);          // (1, 5): code 1
          qa[b][y][3] = __byte_perm(r.y, r.w, 0x7632);          // (3, 7): code 3
          const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            qs[y][b / BPG] += f.x + f.y;
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          qs[y][i] += __shfl_xor_sync(0xffffffffu, qs[y][i], 1);
          qs[y][i] += __shfl_xor_sync(0xffffffffu, qs[y][i], 2);
        }
        m[y] = -INFINITY;
        l[y] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][x] = 0.f;
    }
    if (!ahead) {                                   // this unit has arrived for all lanes, the one before is done with
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
      __syncwarp();
    }
    issue();
    if (ahead) {
      --ahead;
      continue;
    }
    const int fin = (int)(haves >> (5 * slot) & 31u) - 1;      // row of the last token; negative: none
    if (fin >= 0) {
      const unsigned char* stage = myring + slot * S::kStage;
      const uint32_t kt = ring + slot * S::kStage, vt = kt + S::kCodes;
      const unsigned char* ks = stage + 2 * S::kCodes;
      const unsigned char* vs = ks + S::kPairs;
      // ---- scores of 16 tokens: x[y] of row g + 8 y, tokens 2j, 2j + 1, 2j + 8, 2j + 9
      float x[RH][4], al[RH];
#pragma unroll
      for (int y = 0; y < RH; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[y][e] = 0.f;
      const int krow = (lane & 7) + ((lane >> 4) << 3), kpiece = (lane >> 3) & 1;
      float lowc[2][4], highc[2][4];                // sums of codes 0 and 2, of codes 1 and 3, per 8 tokens
#pragma unroll
      for (int b = 0; b < NB; b += 2) {
        uint32_t r[4];                              // pieces b, b + 1 of tokens 0..7, then of 8..15
        ldsm4(r, kt + place(krow, b + kpiece));
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          if ((b + bb) % BPG == 0) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) lowc[n][e] = highc[n][e] = 0.f;
          }
          const auto& q = qa[b + bb];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const uint32_t w = r[2 * n + bb], up = w << 2, dn = w >> 6;      // codes 0, 1 and 2, 3 in bits 2..5, 6..9
            mma(lowc[n], q[0][0], RH == 2 ? q[RH - 1][0] : 0u, q[0][1], RH == 2 ? q[RH - 1][1] : 0u, up & 0x003c003cu,
                dn & 0x003c003cu);
            mma(highc[n], q[0][2], RH == 2 ? q[RH - 1][2] : 0u, q[0][3], RH == 2 ? q[RH - 1][3] : 0u, up & 0x03c003c0u,
                dn & 0x03c003c0u);
          }
          if ((b + bb) % BPG == BPG - 1) {
            constexpr float kLow = 4194304.f, kHigh = 262144.f;            // 2^22, 2^18
            const int gi = (b + bb) / BPG;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float2 s0, s1;
              pairs_of<G>(ks, 8 * n + 2 * j, gi, s0, s1);
#pragma unroll
              for (int y = 0; y < RH; ++y) {
                const float t0 = fmaf(highc[n][2 * y], kHigh, lowc[n][2 * y] * kLow);
                const float t1 = fmaf(highc[n][2 * y + 1], kHigh, lowc[n][2 * y + 1] * kLow);
                x[y][2 * n] = fmaf(s0.x, t0, fmaf(s0.y, qs[y][gi], x[y][2 * n]));
                x[y][2 * n + 1] = fmaf(s1.x, t1, fmaf(s1.y, qs[y][gi], x[y][2 * n + 1]));
              }
            }
          }
        }
      }
      // ---- probabilities
      uint32_t most = 0;                            // the largest step of the tile's values
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          most = max(most, (uint32_t)reinterpret_cast<const unsigned short*>(vs)[2 * ((2 * j + (e & 1) + (e >> 1) * 8) * G + i)]);
      most = __reduce_max_sync(0xffffffffu, most & 0x7fffu) >> 10;
      bool rise = most > top_s;
      const uint32_t before_s = top_s;
      top_s = max(top_s, most);
#pragma unroll
      for (int y = 0; y < RH; ++y) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[y][e] *= a.sc2;
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
      if (__any_sync(0xffffffffu, rise)) {          // a new maximum somewhere, or a new scale: scale what there is
        const float fall = __uint_as_float((127u - (top_s - before_s)) << 23);
#pragma unroll
        for (int y = 0; y < RH; ++y) {
          l[y] *= al[y];
#pragma unroll
          for (int i = 0; i < G; ++i) om[y][i] *= al[y];
          al[y] *= fall;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {              // of 8 heads rows 0..7 and 8..15 are halves of the same head
          o[t][0] *= al[0];
          o[t][1] *= al[0];
          o[t][2] *= al[RH - 1];
          o[t][3] *= al[RH - 1];
        }
      }
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        l[y] += (x[y][0] + x[y][1]) + (x[y][2] + x[y][3]);
        if ((badslots >> slot) & 1u) l[y] = __int_as_float(0x7fc00000);
      }
      // ---- numerators: p s scaled so that it stays below 2^15
      const float scale = __uint_as_float((127u + 29u - top_s) << 23);
      uint32_t hi[RH][2], lo[RH][2];
      const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vpiece = lane >> 4;
#pragma unroll
      for (int b = 0; b < NB; b += 2) {
        uint32_t r[4];                              // tokens 0..7 and 8..15 of piece b, then of b + 1
        ldsm4t(r, vt + place(vrow, b + vpiece));
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          if ((b + bb) % BPG == 0) {
            const int gi = (b + bb) / BPG;
            float2 s[4];
            pairs_of<G>(vs, 2 * j, gi, s[0], s[1]);
            pairs_of<G>(vs, 2 * j + 8, gi, s[2], s[3]);
#pragma unroll
            for (int y = 0; y < RH; ++y) {
#pragma unroll
              for (int e = 0; e < 4; ++e) om[y][gi] = fmaf(x[y][e], fmaf(8.f, s[e].x, s[e].y), om[y][gi]);
              split2(x[y][0] * (s[0].x * scale), x[y][1] * (s[1].x * scale), hi[y][0], lo[y][0]);
              split2(x[y][2] * (s[2].x * scale), x[y][3] * (s[3].x * scale), hi[y][1], lo[y][1]);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {             // code i of the words: columns 32 (b + bb) + 4 word + i
            const uint32_t b0 = centred(i < 2 ? r[2 * bb] : r[2 * bb] >> 8, i % 2);
            const uint32_t b1 = centred(i < 2 ? r[2 * bb + 1] : r[2 * bb + 1] >> 8, i % 2);
            float(&t)[4] = o[4 * (b + bb) + i];
            if constexpr (RH == 1) {                // hi in rows 0..7, lo in rows 8..15
              mma(t, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
            } else {
              mma(t, hi[0][0], hi[RH - 1][0], hi[0][1], hi[RH - 1][1], b0, b1);
              mma(t, lo[0][0], lo[RH - 1][0], lo[0][1], lo[RH - 1][1], b0, b1);
            }
          }
        }
      }
    }
    slot = slot + 1 == STAGES ? 0 : slot + 1;

    const Walk w = c;
    u += advance<SP>(a, pre, lens, c);
    const bool ends = w.chunk + 1 == w.nch, all = u >= u1;
    if (ends || all) {                              // the end of this (sequence, head), or of this CTA's share of it
      // Every warp leaves its sums, then joins a quarter of the columns of all
      // warps.  (p s was scaled by 2^(29 - top_s).)
      const float unit = __uint_as_float((127u - 29u + top_s) << 23);
#pragma unroll
      for (int y = 0; y < RH; ++y) {
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
        l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
        if (j == 0) wml[warp * H + g + 8 * y] = make_float2(m[y], l[y]);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          om[y][i] += __shfl_xor_sync(0xffffffffu, om[y][i], 1);
          om[y][i] += __shfl_xor_sync(0xffffffffu, om[y][i], 2);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int half = 0; half < 2; ++half) {    // words 2j and 2j + 1
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float(&t)[4] = o[4 * b + i];
              const float v = RH == 1 ? t[half] + t[2 + half] : t[2 * y + half];
              f[i] = fmaf(v, unit, om[y][b / BPG]);
            }
            *reinterpret_cast<float4*>(sums + warp * S::kSums + (g + 8 * y) * (D * 4) + (((8 * b + 2 * j + half) ^ g) << 4)) =
                make_float4(f[0], f[1], f[2], f[3]);
          }
      }
      __syncthreads();
      const bool whole = ends && seg == 0;
      join_warps<D, H, SP>(a, sums, S::kSums, wml, whole, 2 * (int)blockIdx.x + (seg == 0 ? 1 : 0), rows, w.b, qh, 1.f);
      __syncthreads();                              // the sums may be written again; the part is written
      if (!whole && threadIdx.x == 0) owe_part(a, sh, pre, w, owe, owed);
      fresh = true;
      seg = 0;
    }
  }

  if (threadIdx.x == 0) *nowed = owed;
  __syncthreads();
  join_parts<D, H, SP>(a, owe, *nowed, 1.f);
}

template <bool SP>
int attend4(const q2_kv4* kv, const Attend4Args& a, const CacheShape& c, long long units, void* stream) {
  return by_shape(c, [&](auto Dc, auto Gc) {
    constexpr int D = Dc(), group = Gc();
    if constexpr (group == 0) {
      return (int)Q2_ESHAPE;                        // (an fp16 cache, which check_cache4 does not give)
    } else {
      constexpr int G = D / group;
      const int most = (int)std::min(units, (long long)ctas_of<D>() * dev_info().sms);
      if constexpr (D <= 128)
        if (unit_heads(a.group, D) == 16)
          return launch_pdl(k_attend4<D, G, 16, SP>, a, most, kThreads, Shape<D, G, 16>::smem(a.batch), stream);
      return launch_pdl(k_attend4<D, G, 8, SP>, a, most, kThreads, Shape<D, G, 8>::smem(a.batch), stream);
    }
  });
}

}  // namespace
}  // namespace q2

using namespace q2;

extern "C" int q2_attend4(const q2_kv4* kv, const void* q, long long ldq, const int* lens, int batch, int q_heads,
                          const int* sel, int nsel, float scale, void* out, long long ldo, void* ws, size_t ws_bytes,
                          q2_stream stream) {
  if (!kv) return Q2_EINVAL;
  if (sel ? nsel < 1 : nsel != 0) return Q2_ESHAPE;
  Attend4Args a = {};
  CacheShape c;
  UnitCall u = {q, ldq, lens, batch, q_heads, sel, nsel, scale, out, ldo, ws, ws_bytes};
  int st = u.check(kv);
  if (st) return st;
  if (batch == 0) return Q2_OK;
  if ((st = check_cache4(kv, batch, a.pg, a.sp, c)) || (st = u.fill(c, sel != nullptr, a))) return st;
  a.aligned = kv->page_size % kTile == 0;
  return sel ? attend4<true>(kv, a, c, u.units, stream) : attend4<false>(kv, a, c, u.units, stream);
}

// The error word of these kernels, then cleared (q2_device_errors).
extern "C" int q2_attend4_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_attend4_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_attend4_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
