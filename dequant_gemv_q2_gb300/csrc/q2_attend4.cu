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
// Keys: four bits masked out of the lower ten of an fp16 number are one below the
// normal ones, c 2^-24 times the place of the bits: a word in place has two codes
// there, shifted down by six the other two, so five instructions make four
// registers of operands.  (The tensor cores align such products as if they were
// 2^-14 and cut them off, an error of 2^-13 of a step times the largest q column
// at most, of 2^-17 for two codes of four.)
//
// Values: c - 8, by 1024 + c and a subtraction, two instructions for a register.
// With c itself both terms of the numerator are some eight steps times the
// denominator and nearly cancel, and the fp32 sums' roundings showed in a long
// sequence's output (one of 131072 tokens: 4.1e-4 off, 2.1e-4 of it fp16's own).
//
// A warp's step of 32 tokens is some 700 instructions, two warps to a scheduler: of
// 135 us for 64 sequences of 8192 tokens (8 key-value heads of 128, groups of 64,
// four query heads each; 605 MB, 4.5 TB/s of the 6.8 of a copy) the loads alone
// take 97, the instructions alone 117, 2.2 of them per cycle and SM.
//
// p s is split into two fp16 numbers, in the two halves of the rows as p is for
// the fp16 cache.  It is scaled by a power of two above the largest s so far
// (of the warp's tiles), which changes as rarely as the maximum does.
#include "q2_attend.cuh"

namespace q2 {
namespace {

__device__ unsigned int q2_attend4_error;

struct Attend4Args : UnitArgs {
  const unsigned char* k;       // codes; strides in 16 bytes
  const unsigned char* ks;      // pairs; strides in pairs
  long long v, vs;              // the values' pools, in bytes behind the keys'
  uint32_t page_stride, token_stride, head_stride;
  uint32_t s_page_stride, s_token_stride, s_head_stride;
  const int* table;
  long long table_stride;
  int npages, page;
  uint32_t page_mul, page_sh;   // of page_of()
  int aligned;                  // a step's tokens of a warp lie in one page
};

// Tokens of a warp's step: two tiles where registers allow it, which share the
// copies' addresses, the maximum and the rescaling.
template <int D>
__host__ __device__ constexpr int step_of() { return D == 256 ? 16 : 32; }

template <int D>
__host__ __device__ constexpr int ctas_of() { return D == 64 ? 3 : 2; }

template <int D, int G, int H>
struct Shape {
  static constexpr int STAGES = 3, TW = step_of<D>();
  static constexpr int kCodes = TW * D / 2, kPairs = TW * G * 4;         // bytes of a step, keys or values
  static constexpr int kStage = 2 * (kCodes + kPairs);
  static constexpr int kRing = kWarps * STAGES * kStage;
  static constexpr int kSums = H * D * 4;                                // a warp's numerators
  static constexpr int kMl = kWarps * H * 8;
  static constexpr int fixed = kRing + kWarps * kSums + kMl + 48;
  static_assert(kStage % 128 == 0, "stages begin on 128 bytes");
  static int smem(int batch) { return fixed + 4 * (2 * batch + 1); }
};

// N bytes, or zeros
template <int N>
__device__ __forceinline__ void cp_pairs(uint32_t dst, const unsigned char* src, bool live) {
  if constexpr (N >= 16) {
#pragma unroll
    for (int i = 0; i < N; i += 16) cp16(dst + i, src + i, live);
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(live ? N : 0) : "memory");
  }
}

__device__ __forceinline__ void cp16_all(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ float2 halves(uint32_t r) { return __half22float2(*reinterpret_cast<const __half2*>(&r)); }

// The pairs (step, offset) of a token, all groups.
template <int G>
__device__ __forceinline__ void load_pairs(const unsigned char* at, uint32_t (&r)[G]) {
  if constexpr (G == 1) {
    r[0] = *reinterpret_cast<const uint32_t*>(at);
  } else if constexpr (G == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(at);
    r[0] = x.x;
    r[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < G; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(at + 4 * i);
      r[i] = x.x;
      r[i + 1] = x.y;
      r[i + 2] = x.z;
      r[i + 3] = x.w;
    }
  }
}

// How far, in powers of two, a score may rise above the maximum before all is
// scaled anew: p is at most 2^kSlack.  (With 0 a third of the steps of 2048 tokens
// scaled: 45.0 us for 64 sequences, 43.4 with 4.  p s is held to 2^-20 of itself or,
// half of fp16's smallest number, 2^-35 of the largest; without the slack 2^-39.)
constexpr uint32_t kSlack = 4;

// 2^x to 2 units in the last place; what is below the normal numbers is zero
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Codes in bits 0..3 (high: 4..7) of both halves as c - 8 in fp16: 1024 + c (1024 + 16 c), then what is too much.
__device__ __forceinline__ uint32_t centred(uint32_t w, bool high) {
  const uint32_t x = (w & (high ? 0x00f000f0u : 0x000f000fu)) | 0x64006400u;
  const __half2 h = *reinterpret_cast<const __half2*>(&x);
  const __half2 y = high ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.f)) : __hsub2(h, __float2half2_rn(1032.f));
  return *reinterpret_cast<const uint32_t*>(&y);
}

// 8 x 8 numbers of 16 bits, transposed
__device__ __forceinline__ uint32_t transpose(uint32_t r) {
  uint32_t t;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(r));
  return t;
}

// mma(), or the product alone
__device__ __forceinline__ void mma_from(bool zero, float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (!zero) {
    mma(c, a0, a1, a2, a3, b0, b1);
    return;
  }
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// H: query heads of a unit, 8 or 16 (columns of the products); FOLD: four at
// most; G: groups of a row
template <int D, int G, int H, bool FOLD, bool SP>
__global__ void __launch_bounds__(kThreads, ctas_of<D>()) k_attend4(const __grid_constant__ Attend4Args a) {
  using S = Shape<D, G, H>;
  static_assert(ctas_of<D>() <= most_ctas(D) && H <= most_heads(D), "the workspace has room for all parts");
  constexpr int NH = H / 8, STAGES = S::STAGES, NB = D / 32;   // NB: 16-byte pieces of a row, 32 columns each
  constexpr int TW = S::TW, NTL = TW / kTile, UNIT = kWarps * TW;
  constexpr int RPI = 32 / NB, BPG = NB / G;                   // rows of a copy instruction; pieces of a group
  static_assert(!FOLD || H == 8, "");
  extern __shared__ __align__(128) unsigned char q2_att4_smem[];
  unsigned char* sums = q2_att4_smem + S::kRing;
  float2* wml = reinterpret_cast<float2*>(sums + kWarps * S::kSums);     // [kWarps][H] maximum, denominator
  int4* owe = reinterpret_cast<int4*>(wml + kWarps * H);
  int* nowed = reinterpret_cast<int*>(owe + 2);
  int* pre = nowed + 4;
  int* lens = pre + a.batch + 1;
  const int lane = threadIdx.x & 31, g = lane >> 2, j = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);      // (known to be the warp's)

  pdl_wait();
  pdl_trigger();
  const Share sh = share_out<D, SP, UNIT>(a, nowed, pre, lens, &q2_attend4_error);
  int u = sh.u0;
  const int u1 = sh.u1;
  if (u >= u1) return;
  Walk c = walk_from<SP, UNIT>(a, pre, lens, u);    // the unit in use, at place u
  if (u >= u1) return;
  // units of w's (sequence, head) from w on that are this CTA's, w at place v
  auto run_of = [&](const Walk& w, int v) { return min(w.nch - w.chunk, u1 - v); };

  // ---- the warp's loads, STAGES - 1 units ahead of their use
  unsigned char* const myring = q2_att4_smem + warp * (STAGES * S::kStage);
  const uint32_t ring = saddr(myring);
  Walk p = c;                                       // the unit to load, at place pu
  int pu = u, prun = run_of(p, u), pleft = prun, pslot = 0;    // units of its (sequence, head) in all and still to be loaded, its stage
  int pt0 = 0, ppage = -1;                          // its first token, its page (of this lane's row where not aligned)
  int pstep = 0, nt0 = 0, npage = -1;               // SP: its number of them; first token and page of the next
  uint32_t badslots = 0, haves = 0;                 // stages with a row whose page does not exist; SP: a stage's tokens, 8 bits each
  const int piece = lane % NB, row0 = lane / NB, prow = lane % TW;
  // the pieces of a row are exchanged so that eight rows of one piece lie in different banks
  auto place = [](int row, int pc) { return row * (D / 2) + ((pc ^ (row / (8 / NB) & (NB - 1))) << 4); };
  const uint32_t cdst = ring + place(row0, piece);  // (rows RPI apart have their pieces alike, of eight pieces the fifth for the first)
  const uint32_t pdst = ring + 2 * S::kCodes + prow * (4 * G);
  const uint32_t lrow = (uint32_t)row0 * a.token_stride + piece, step = a.token_stride * 16;
  const int* trow = nullptr;                        // of p's (sequence, head): the table's row, the head's place
  uint32_t phead = 0, pshead = 0;
  // SP: where a list says which blocks, two looks are behind one another, into the
  // list and into the table: 32 units' at a time, and those a unit further ahead
  // (32 sequences of up to 32768 tokens, 64 blocks of each: 50.4 -> 48.4 us).
  int found = 0, fpage = -1;                        // first token and page of unit 32 n + lane
  auto find = [&](int i, int& t0, int& pg) {        // unit i of p's: first token; page, if all its tokens are in one, or of this lane's row
    if (i % 32 == 0) {
      Walk w = p;
      w.chunk += i + lane;
      found = i + lane < prun ? first_token<SP, UNIT, TW>(a, w, warp, true) : p.len;
      if (a.aligned) fpage = found < p.len ? trow[page_of(a, found)] : -1;
    }
    t0 = __shfl_sync(0xffffffffu, found, i % 32);
    if (a.aligned) pg = __shfl_sync(0xffffffffu, fpage, i % 32);
    else pg = t0 + prow < p.len ? trow[page_of(a, t0 + prow)] : -1;
  };
  auto enter = [&]() {
    const uint32_t kvh = a.nht == 1 ? p.h : p.h / a.nht;
    trow = a.table + p.b * a.table_stride;
    phead = kvh * a.head_stride;
    pshead = kvh * a.s_head_stride;
    if (SP) {
      find(0, pt0, ppage);
      find(1, nt0, npage);
    } else {
      pt0 = p.chunk * UNIT + warp * TW;
    }
  };
  auto lookup = [&]() {
    const int t = pt0 + (a.aligned ? 0 : prow);
    ppage = pleft > 0 && t < p.len ? trow[page_of(a, t)] : -1;
  };
  enter();
  if (!SP) lookup();
  auto issue = [&]() {
    if (pleft > 0) {
      const int have = SP ? min(max(p.len - pt0, 0), TW) : p.len - pt0;       // tokens; negative: none
      if (SP) haves = (haves & ~(255u << (8 * pslot))) | (uint32_t)have << (8 * pslot);
      if (have > 0) {
        const bool there = (unsigned)ppage < (unsigned)a.npages;
        const bool bad = __any_sync(0xffffffffu, (a.aligned || prow < have) && !there);
        const uint32_t page = there ? ppage : 0;
        const int t = pt0 + (a.aligned ? 0 : prow);
        const uint32_t pat = t - page_of(a, t) * a.page;       // place in the page
        const unsigned long long off = (unsigned long long)page * a.page_stride + (pat * a.token_stride + phead);
        const unsigned long long soff = (unsigned long long)page * a.s_page_stride +
                                        ((pat + (a.aligned ? prow : 0)) * a.s_token_stride + pshead);
        const uint32_t cd = cdst + pslot * S::kStage, pd = pdst + pslot * S::kStage;
        const unsigned char* ps = a.ks + soff * 4;
        if (a.aligned && have >= TW && !bad) {      // the usual step: all rows, one behind another
          if constexpr (TW == 32) {
            cp_pairs<4 * G>(pd, ps, true);
            cp_pairs<4 * G>(pd + S::kPairs, ps + a.vs, true);
          } else {
            cp_pairs<4 * G>(pd + (lane < 16 ? 0 : S::kPairs), ps + (lane < 16 ? 0 : a.vs), true);
          }
          const unsigned char* k = a.k + (off + lrow) * 16;
          const unsigned char* v = k + a.v;
#pragma unroll
          for (int i = 0; i < TW / RPI; ++i) {
            const uint32_t d = (NB == 8 && i % 2 ? cd ^ 64u : cd) + i * (RPI * D / 2);
            const unsigned long long at = (unsigned long long)(i * RPI) * step;
            cp16_all(d, k + at);
            cp16_all(d + S::kCodes, v + at);
          }
        } else {
          const bool plive = there && prow < have;
          if (!plive) ps = a.ks;
          if constexpr (TW == 32) {
            cp_pairs<4 * G>(pd, ps, plive);
            cp_pairs<4 * G>(pd + S::kPairs, ps + a.vs, plive);
          } else {
            cp_pairs<4 * G>(pd + (lane < 16 ? 0 : S::kPairs), ps + (lane < 16 ? 0 : a.vs), plive);
          }
          const unsigned long long mine = there ? off : ~0ull;
#pragma unroll 2
          for (int i = 0; i < TW / RPI; ++i) {
            const int row = row0 + i * RPI;
            unsigned long long o = a.aligned ? mine : __shfl_sync(0xffffffffu, mine, row);
            const bool live = o != ~0ull && row < have;
            if (a.aligned) o += (uint32_t)row * a.token_stride;
            const unsigned char* k = a.k + (live ? o + piece : 0) * 16;
            const uint32_t d = (NB == 8 && i % 2 ? cd ^ 64u : cd) + i * (RPI * D / 2);
            cp16(d, k, live);
            cp16(d + S::kCodes, k + a.v, live);
          }
        }
        if (bad) {
          if (lane == 0) atomicOr(&q2_attend4_error, Q2_ERR_PAGE);
          badslots |= 1u << pslot;
        }
      }
      pslot = pslot + 1 == STAGES ? 0 : pslot + 1;
      pt0 += UNIT;
      if (--pleft == 0) {                           // on to the next (sequence, head)
        p.chunk += prun - 1;
        pu += prun - 1 + advance<SP, UNIT>(a, pre, lens, p);
        if (pu < u1) {
          pleft = prun = run_of(p, pu);
          pstep = 0;
          enter();
        }
      } else if (SP) {
        pt0 = nt0;
        ppage = npage;
        find(++pstep + 1, nt0, npage);
      }
      if (!SP) lookup();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  // ---- sums of the current (sequence, head)
  // The queries of 32 columns of head g (+ 8), for codes 0 and 2, then 1 and 3 of
  // the words 2j, 2j + 1: times a power of two that brings a head's largest to
  // 2^10 .. 2^11, and over the 16, 4 and 64 that codes 1, 2 and 3 come too large.
  // The rest is of the heads 2j, 2j + 1 (+ 8).
  uint32_t qa[NB][NH][4];
  float qs[NH][2][G], qf[NH][2];                    // sums over the groups, in the units of the products; what a score is to be multiplied by
  float o[NB][NH][2][4];                            // numerators: columns 32 b + 4 g + 2 k, + 1, each of two heads
  float om[NH][2][G], m[NH][2], ref[NH][2], l[NH][2];   // of the offsets; largest sum, its score (0 for none); denominator (this and om over the lane's tokens)
  float bar[NH][2];                                 // the sum above which the maximum is taken anew
  const unsigned short less = !FOLD || j >= 2 ? 0xbc00 : 0;     // -1 or 0
  uint32_t top_s;                                   // exponent field of the largest step so far, 1 at least
  int slot = 0;
  int ahead = STAGES - 1;                           // units still to be requested before the first is used
  int owed = 0;                                     // parts of this CTA that were the last of their (sequence, head)
  while (u < u1) {                                  // a (sequence, head), or what is this CTA's of it
    const int run = run_of(c, u), seg = c.chunk;
    const int kvh = a.nht == 1 ? c.h : c.h / a.nht, ht = c.h - kvh * a.nht, rows = min(H, a.group - ht * H);
    {
      const int row = FOLD ? g & 3 : g;
      const __half* q = a.q + c.b * a.ldq + (long long)(kvh * a.group + ht * H + row) * D + 8 * j;
#pragma unroll
      for (int y = 0; y < NH; ++y) {
        uint4 r[NB];
        uint32_t top = 0;                           // the largest exponent field
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          r[b] = row + 8 * y < rows ? *reinterpret_cast<const uint4*>(q + 8 * y * D + 32 * b) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {r[b].x, r[b].y, r[b].z, r[b].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = halves(w[i]);
            top = max(top, max(__float_as_uint(f.x) >> 23 & 255u, __float_as_uint(f.y) >> 23 & 255u));
          }
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = min(max(top, 90u), 142u);             // (a head of zeros; an infinite or NaN column, which stays one)
        // 2^10 over the largest's power of two, of the scale's sign: the largest score is the largest sum
        const float up = copysignf(__uint_as_float((127u + 10u + 127u - top) << 23), a.sc2);
        // (a code is c 2^-24; never zero, with which a masked sum of minus infinity were NaN: 2^-100 of a sum is none)
        const float down = fmaxf(fabsf(a.sc2) * __uint_as_float((127u + 24u - 10u - 127u + top) << 23), 0x1p-100f);
        float sum[G];
#pragma unroll
        for (int i = 0; i < G; ++i) sum[i] = 0.f;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint32_t w[4] = {r[b].x, r[b].y, r[b].z, r[b].w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 x = halves(w[i]);
            f[2 * i] = x.x * up;
            f[2 * i + 1] = x.y * up;
            sum[b / BPG] += f[2 * i] + f[2 * i + 1];
          }
          // words 2j and 2j + 1 are columns 0..3 and 4..7 of these eight
          qa[b][y][0] = pack2(f[0], f[4]);
          qa[b][y][1] = pack2(f[2] * 0.25f, f[6] * 0.25f);
          qa[b][y][2] = pack2(f[1] * 0.0625f, f[5] * 0.0625f);
          qa[b][y][3] = pack2(f[3] * 0.015625f, f[7] * 0.015625f);
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
          sum[i] *= 1.f / 16777216.f;               // 2^-24
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {               // from head g's lanes to those that have its scores
          qf[y][e] = __shfl_sync(0xffffffffu, down, (2 * j + e) * 4);
#pragma unroll
          for (int i = 0; i < G; ++i) {
            qs[y][e][i] = __shfl_sync(0xffffffffu, sum[i], (2 * j + e) * 4);
            om[y][e][i] = 0.f;
          }
          m[y][e] = bar[y][e] = -INFINITY;
          ref[y][e] = l[y][e] = 0.f;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[b][y][k][e] = 0.f;
      }
    }
    top_s = 1;
    int t0 = seg * UNIT + warp * TW;
#pragma unroll 1
    for (int left = run; left;) {
      if (!ahead) {                                   // this unit has arrived for all lanes, the one before is done with
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncwarp();
      }
      issue();
      if (ahead) {
        --ahead;
        continue;
      }
      // row of the last token, if below TW; negative: none
      const int fin = SP ? (int)(haves >> (8 * slot) & 255u) - 1 : c.len - 1 - t0;
      if (fin >= 0) {
        const unsigned char* ks = myring + slot * S::kStage + 2 * S::kCodes + g * (4 * G);   // the pairs of token g
        const unsigned char* vs = ks + S::kPairs;
        const uint32_t kt = ring + slot * S::kStage, vt = kt + S::kCodes;
        // ---- scores: x[n][y][e] of token 8 n + g, head 8 y + 2j + e, still to be multiplied by qf
        float x[2 * NTL][NH][2];
        const int krow = (lane & 7) + ((lane >> 4) << 3), kpiece = (lane >> 3) & 1;
        uint32_t sm[2 * NTL][G];
#pragma unroll
        for (int n = 0; n < 2 * NTL; ++n) load_pairs<G>(ks + 8 * n * (4 * G), sm[n]);
        float acc[NTL][NH][4];
#pragma unroll
        for (int b = 0; b < NB; b += 2) {
          uint32_t r[NTL][4];                         // pieces b, b + 1 of tokens 0..7, then of 8..15
#pragma unroll
          for (int i = 0; i < NTL; ++i) ldsm4(r[i], kt + i * (kTile * D / 2) + place(krow, b + kpiece));
#pragma unroll
          for (int bb = 0; bb < 2; ++bb) {
#pragma unroll
            for (int i = 0; i < NTL; ++i) {
              // codes 0, 1 in bits 0..3, 4..7 of w0 and w1, codes 2, 3 in bits 2..5, 6..9 of h0 and h1
              const uint32_t w0 = r[i][bb], w1 = r[i][2 + bb], h0 = w0 >> 6, h1 = w1 >> 6;
#pragma unroll
              for (int y = 0; y < NH; ++y) {
                const bool first = (b + bb) % BPG == 0;
                const auto& q = qa[b + bb][y];
                mma_from(first, acc[i][y], w0 & 0x000f000fu, w1 & 0x000f000fu, h0 & 0x003c003cu, h1 & 0x003c003cu, q[0], q[1]);
                mma(acc[i][y], w0 & 0x00f000f0u, w1 & 0x00f000f0u, h0 & 0x03c003c0u, h1 & 0x03c003c0u, q[2], q[3]);
              }
            }
            if ((b + bb) % BPG == BPG - 1) {
              const int gi = (b + bb) / BPG;
#pragma unroll
              for (int n = 0; n < 2 * NTL; ++n) {
                const float2 s = halves(sm[n][gi]);
#pragma unroll
                for (int y = 0; y < NH; ++y)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    float& z = x[n][y][e];
                    const auto& t = acc[n / 2][y];
                    z = fmaf(s.x, t[2 * (n % 2) + e], gi ? fmaf(s.y, qs[y][e][gi], z) : s.y * qs[y][e][0]);
                  }
              }
            }
          }
        }
        // ---- probabilities
        uint32_t vp[2 * NTL][G];                      // the pairs of the values of token 8 n + g
        __half2 most = __float2half2_rn(0.f);
#pragma unroll
        for (int n = 0; n < 2 * NTL; ++n) {
          load_pairs<G>(vs + 8 * n * (4 * G), vp[n]);
#pragma unroll
          for (int i = 0; i < G; ++i) most = __hmax2(most, *reinterpret_cast<const __half2*>(&vp[n][i]));
        }
        const uint32_t most_s = (uint32_t)__half_as_ushort(__low2half(most)) >> 10;
        bool rise = most_s > top_s || fin < TW - 1 || badslots;
#pragma unroll
        for (int y = 0; y < NH; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = x[0][y][e];
#pragma unroll
            for (int n = 1; n < 2 * NTL; ++n) top = fmaxf(top, x[n][y][e]);
            rise = rise || top > bar[y][e];
          }
        // A maximum far enough above the last, or a larger step: scale what there
        // is.  (Also a step that is not whole, or has a page that does not exist.)
        if (__any_sync(0xffffffffu, rise)) {
          const uint32_t now_s = max(top_s, __reduce_max_sync(0xffffffffu, most_s));
          const float fall = __uint_as_float((127u - (now_s - top_s)) << 23);
          const bool bad = (badslots >> slot) & 1u;
          badslots &= ~(1u << slot);
          top_s = now_s;
#pragma unroll
          for (int y = 0; y < NH; ++y)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float top = m[y][e];
#pragma unroll
              for (int n = 0; n < 2 * NTL; ++n) {
                if (8 * n + g > fin) x[n][y][e] = -INFINITY;
                top = fmaxf(top, x[n][y][e]);
              }
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
              ref[y][e] = top == -INFINITY ? 0.f : top * qf[y][e];
              const float al = m[y][e] == -INFINITY ? 0.f : ex2(fmaf(m[y][e], qf[y][e], -ref[y][e])), alf = al * fall;
              m[y][e] = top;
              bar[y][e] = top + (float)kSlack / qf[y][e];
              l[y][e] = bad ? __int_as_float(0x7fc00000) : l[y][e] * al;
#pragma unroll
              for (int i = 0; i < G; ++i) om[y][e][i] *= al;
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  o[b][y][k][e] *= alf;
                  o[b][y][k][2 + e] *= alf;
                }
            }
        }
#pragma unroll
        for (int y = 0; y < NH; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2 * NTL; ++n) {
              x[n][y][e] = ex2(fmaf(x[n][y][e], qf[y][e], -ref[y][e]));
              l[y][e] += x[n][y][e];
            }
        // ---- numerators: p s scaled so that it stays below 2^15
        const float scale = __uint_as_float((127u + 29u - kSlack - top_s) << 23);
        const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vpiece = lane >> 4;
#pragma unroll
        for (int i = 0; i < NTL; ++i) {
          uint32_t hi[NH][2], lo[NH][2];              // p s of 8 tokens each: tokens 2j, 2j + 1, head g
#pragma unroll
          for (int b = 0; b < NB; b += 2) {
            uint32_t r[4];                            // tokens 0..7 and 8..15 of piece b, then of b + 1
            ldsm4t(r, vt + i * (kTile * D / 2) + place(vrow, b + vpiece));
#pragma unroll
            for (int bb = 0; bb < 2; ++bb) {
              if ((b + bb) % BPG == 0) {
                const int gi = (b + bb) / BPG;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  float2 s = halves(vp[2 * i + n][gi]);
                  s.y = fmaf(8.f, s.x, s.y);
                  s.x *= scale;
#pragma unroll
                  for (int y = 0; y < NH; ++y) {
                    const float(&w)[2] = x[2 * i + n][y];
#pragma unroll
                    for (int e = 0; e < 2; ++e) om[y][e][gi] = fmaf(w[e], s.y, om[y][e][gi]);
                    const float w0 = w[0] * s.x, w1 = w[1] * s.x;
                    const uint32_t h = pack2(w0, w1);
                    // FOLD: lanes of columns 4..7 have heads 0..3 again, theirs is the lower part
                    const uint32_t t = pack2(fma_h(lo16(h), less, w0), fma_h(hi16(h), less, w1));
                    hi[y][n] = transpose(FOLD ? t : h);
                    if (!FOLD) lo[y][n] = transpose(t);
                  }
                }
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {           // codes 2k, 2k + 1 of the words: columns 32 (b + bb) + 4 word + 2k, + 1
                const uint32_t w0 = k ? r[2 * bb] >> 8 : r[2 * bb], w1 = k ? r[2 * bb + 1] >> 8 : r[2 * bb + 1];
                const uint32_t a0 = centred(w0, false), a1 = centred(w0, true), a2 = centred(w1, false), a3 = centred(w1, true);
#pragma unroll
                for (int y = 0; y < NH; ++y) {
                  mma(o[b + bb][y][k], a0, a1, a2, a3, hi[y][0], hi[y][1]);
                  if (!FOLD) mma(o[b + bb][y][k], a0, a1, a2, a3, lo[y][0], lo[y][1]);
                }
              }
            }
          }
        }
      }
      slot = slot + 1 == STAGES ? 0 : slot + 1;
      t0 += UNIT;
      --left;
    }

    {
      // Every warp leaves its sums, then joins a quarter of the columns of all
      // warps.  (p s was scaled by 2^(29 - kSlack - top_s).)
      const float unit = __uint_as_float((127u - 29u + kSlack + top_s) << 23);
#pragma unroll
      for (int y = 0; y < NH; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) {
            l[y][e] += __shfl_xor_sync(0xffffffffu, l[y][e], s);
#pragma unroll
            for (int i = 0; i < G; ++i) om[y][e][i] += __shfl_xor_sync(0xffffffffu, om[y][e][i], s);
          }
          const int head = 8 * y + 2 * j + e;
          if (g == 0) wml[warp * H + head] = make_float2(m[y][e] == -INFINITY ? -INFINITY : ref[y][e], l[y][e]);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float f[4] = {o[b][y][0][e], o[b][y][0][2 + e], o[b][y][1][e], o[b][y][1][2 + e]};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (FOLD) f[k] += __shfl_xor_sync(0xffffffffu, f[k], 2);
              f[k] = fmaf(f[k], unit, om[y][e][b / BPG]);
            }
            *reinterpret_cast<float4*>(sums + warp * S::kSums + head * (D * 4) + (((8 * b + g) ^ (head & 7)) << 4)) =
                make_float4(f[0], f[1], f[2], f[3]);
          }
        }
      __syncthreads();
      const bool whole = seg == 0 && run == c.nch;
      join_warps<D, H, SP>(a, sums, S::kSums, wml, whole, 2 * (int)blockIdx.x + (seg == 0 ? 1 : 0), rows, c.b,
                           kvh * a.group + ht * H, 1.f);
      __syncthreads();                              // the sums may be written again; the part is written
      if (!whole && threadIdx.x == 0) owe_part(a, sh, pre, c, owe, owed);
    }
    c.chunk += run - 1;
    u += run - 1 + advance<SP, UNIT>(a, pre, lens, c);
  }

  if (threadIdx.x == 0) *nowed = owed;
  __syncthreads();
  join_parts<D, H, SP, 12>(a, owe, *nowed, 1.f);
}

template <bool SP>
int attend4(const q2_kv4* kv, const Attend4Args& a, const CacheShape& c, long long units, void* stream) {
  return by_shape(c, [&](auto Dc, auto Gc) {
    constexpr int D = Dc(), group = Gc();
    if constexpr (group == 0) {
      return (int)Q2_ESHAPE;                        // (an fp16 cache, which check_cache4 does not give)
    } else {
      constexpr int G = D / group;
      auto launch = [&](auto kernel, int smem) {
        return launch_pdl(kernel, a, (int)std::min(units, (long long)ctas_of<D>() * dev_info().sms), kThreads, smem, stream);
      };
      if constexpr (D <= 128)
        if (unit_heads(a.group, D) == 16)
          return launch(k_attend4<D, G, 16, false, SP>, Shape<D, G, 16>::smem(a.batch));
      const int smem = Shape<D, G, 8>::smem(a.batch);
      return a.group <= 4 ? launch(k_attend4<D, G, 8, true, SP>, smem) : launch(k_attend4<D, G, 8, false, SP>, smem);
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
  Pages pg, sp;
  CacheShape c;
  UnitCall u = {q, ldq, lens, batch, q_heads, sel, nsel, scale, out, ldo, ws, ws_bytes};
  int st = u.check(kv);
  if (st) return st;
  if (batch == 0) return Q2_OK;
  if ((st = check_cache4(kv, batch, pg, sp, c)) || (st = u.fill(c, sel != nullptr, a))) return st;
  // strides, and places within a page, are counted in 32 bits (of 16 bytes, of pairs)
  auto within = [&](long long page, long long token, long long head) {
    return page <= 0xffffffffll && token * (c.page - 1) + head * (c.kv_heads - 1) <= 0xffffffffll && token <= 0xffffffffll &&
           head <= 0xffffffffll;
  };
  if (kv->token_stride > 0xffffffffll) return Q2_ESHAPE;
  if (!within(kv->page_stride / 16, kv->token_stride / 16, kv->head_stride / 16) ||
      !within(kv->s_page_stride, kv->s_token_stride, kv->s_head_stride))
    return Q2_ESHAPE;
  a.k = pg.k;
  a.ks = sp.k;
  a.v = pg.v - pg.k;
  a.vs = sp.v - sp.k;
  a.page_stride = (uint32_t)(kv->page_stride / 16);
  a.token_stride = (uint32_t)(kv->token_stride / 16);
  a.head_stride = (uint32_t)(kv->head_stride / 16);
  a.s_page_stride = (uint32_t)kv->s_page_stride;
  a.s_token_stride = (uint32_t)kv->s_token_stride;
  a.s_head_stride = (uint32_t)kv->s_head_stride;
  a.table = kv->table;
  a.table_stride = kv->table_stride;
  a.npages = kv->npages;
  a.page = kv->page_size;
  a.page_mul = pg.page_mul;
  a.page_sh = pg.page_sh;
  a.aligned = kv->page_size % (c.D == 256 ? step_of<256>() : step_of<128>()) == 0;
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
