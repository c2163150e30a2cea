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
// 64 sequences of 8192 tokens, 32 query and 8 key-value heads of 128: 318 to 327 us
// by the machine, 6.6 to 6.8 TB/s, the rate of a copy; one of 131072: 90 us, 5.9; 16
// of 1 to 4096 with 40 query heads 30 us, 4.5 (each CTA's start, its ends of
// sequences and the joins are 9 of them); one of 777 tokens 7.0 us: the
// lengths, the first pages' numbers, the first rows and the join behind one
// another.  Heads of 256 have one CTA per SM, whose threads spill 164 bytes at
// 255 registers: 64 of 4096 tokens 336 us, 6.4 TB/s, 16 of 2048 53, 5.0.
#include "q2_attend.cuh"

namespace q2 {
namespace {

__device__ unsigned int q2_attend_error;

struct AttendArgs : UnitArgs {
  __half* k;
  __half* v;
  long long page_stride, token_stride, head_stride;
  const int* table;
  long long table_stride;
  const __half* nk;           // new keys and values, or null
  const __half* nv;
  long long ldn;
  int npages, page;
  uint32_t page_mul, page_sh; // of page_of()
  int aligned;                // page % 16 == 0: a tile lies in one page
};

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

// CTAs per SM: what registers and the rings of three stages leave room for, but
// no more than three (64 sequences of 8192 tokens, heads of 64, pages of 64
// stored head by head: 161 us; with two CTAs of six stages 199, with four of
// three 169; stored token by token 182).
template <int D>
__host__ __device__ constexpr int ctas_of() { return D == 64 ? 3 : D == 128 ? 2 : 1; }

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

// H: query heads of a unit, 8 or 16 (rows of the products); SP: of selected blocks, see q2_attend_blocks
template <int D, int H, bool SP>
__global__ void __launch_bounds__(kThreads, ctas_of<D>()) k_attend(const __grid_constant__ AttendArgs a) {
  using S = Shape<D, H>;
  static_assert(ctas_of<D>() <= most_ctas(D) && H <= most_heads(D), "the workspace has room for all parts");
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
  const Share sh = share_out<D, SP, kUnit>(a, nowed, pre, lens, &q2_attend_error);
  int u0 = sh.u0;
  const int u1 = sh.u1;
  if (u0 >= u1) return;                             // no share
  Walk c = walk_from<SP, kUnit>(a, pre, lens, u0);         // the unit in use
  if (u0 >= u1) return;

  // ---- the warp's loads, STAGES - 1 units ahead of their use
  const uint32_t ring = saddr(q2_att_smem) + warp * (STAGES * 2 * S::kTileBytes);
  Walk p = c;
  int pu = u0, pslot = 0, ppage = -1;               // place of the unit to load, its stage, the page of this lane's row
  uint32_t badslots = 0;                            // stages with a row whose page does not exist
  const int piece = lane % CPR, row0 = lane / CPR;
  const long long lrow = row0 * a.token_stride + piece * 8;            // this lane's place in a tile that lies in one page
  const uint32_t ldst = ring + row0 * (D * 2), lpiece = (uint32_t)((piece ^ row0) << 4);   // row0 < 8; ring and rows on 128 bytes
  int pt0 = 0;                                      // SP: the warp's first token in the unit to load
  uint32_t haves = 0;                               // SP: a stage's tokens, a byte each
  auto lookup = [&]() {                             // a tile in one page: its page; else lanes l and l + 16: that of row l
    if (SP) pt0 = first_token<SP, kUnit, kTile>(a, p, warp, pu < u1);
    const int t = (SP ? pt0 : p.chunk * kUnit + warp * kTile) + (a.aligned ? 0 : lane & 15);
    ppage = pu < u1 && t < p.len ? a.table[p.b * a.table_stride + page_of(a, t)] : -1;
  };
  lookup();
  auto issue = [&]() {
    if (pu < u1) {
      const int t0 = SP ? pt0 : p.chunk * kUnit + warp * kTile;
      if (SP) haves = (haves & ~(255u << (8 * pslot))) | (uint32_t)min(max(p.len - t0, 0), kTile) << (8 * pslot);
      if (t0 < p.len) {
        const int have = p.len - t0 - (!SP && a.nk ? 1 : 0);                  // rows to copy: the new token does not come from the cache
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
      pu += advance<SP, kUnit>(a, pre, lens, p);
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
      if (!SP && a.nk && lane < CPR) {
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
    // row of the last token, if below kTile; negative: none
    const int fin = SP ? (int)(haves >> (8 * slot) & 255u) - 1 : c.len - 1 - (c.chunk * kUnit + warp * kTile);
    if (fin >= 0) {
      const uint32_t kt = ring + slot * (2 * S::kTileBytes), vt = kt + S::kTileBytes;
      if (!SP && a.nk && fin < kTile) {                    // the new token's row, and its place in the cache
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
    u += advance<SP, kUnit>(a, pre, lens, c);
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
      join_warps<D, H, SP>(a, q2_att_smem + mine, STAGES * 2 * S::kTileBytes, wml, whole,
                           2 * (int)blockIdx.x + (seg == 0 ? 1 : 0), rows, w.b, qh, kUp);
      __syncthreads();                              // the stages may be filled again; the part is written
      if (!whole && threadIdx.x == 0) owe_part(a, sh, pre, w, owe, owed);
      fresh = true;
      seg = 0;
    }
  }

  if (threadIdx.x == 0) *nowed = owed;
  __syncthreads();
  join_parts<D, H, SP, 8>(a, owe, *nowed, kUp);
}

template <bool SP>
int attend(const q2_kv* kv, const void* q, long long ldq, const void* new_k, const void* new_v, long long ldn,
           const int* lens, int batch, int q_heads, const int* sel, int nsel, float scale, void* out, long long ldo, void* ws,
           size_t ws_bytes, void* stream) {
  if (!kv || (!new_k) != (!new_v)) return Q2_EINVAL;
  AttendArgs a = {};
  Pages pg;
  CacheShape c;
  UnitCall u = {q, ldq, lens, batch, q_heads, sel, nsel, scale, out, ldo, ws, ws_bytes};
  int st = u.check(kv);
  if (st) return st;
  if (batch == 0) return Q2_OK;
  if ((st = check_cache(kv, batch, pg, c)) || (st = u.fill(c, SP, a))) return st;
  if (batch > 1 && new_k && ldn < (long long)kv->kv_heads * c.D) return Q2_ESHAPE;
  if (misaligned(new_k, 16) || misaligned(new_v, 16) || (batch > 1 && new_k && ldn % 8)) return Q2_EALIGN;
  a.k = static_cast<__half*>(kv->k);
  a.v = static_cast<__half*>(kv->v);
  a.page_stride = kv->page_stride;
  a.token_stride = kv->token_stride;
  a.head_stride = kv->head_stride;
  a.table = kv->table;
  a.table_stride = kv->table_stride;
  a.nk = static_cast<const __half*>(new_k);
  a.nv = static_cast<const __half*>(new_v);
  a.ldn = ldn;
  a.npages = kv->npages;
  a.page = kv->page_size;
  a.aligned = kv->page_size % kTile == 0;
  a.page_mul = pg.page_mul;
  a.page_sh = pg.page_sh;
  const bool wide = unit_heads(a.group, c.D) == 16;
  auto launch = [&](auto kernel, int ctas, int smem) {
    return launch_pdl(kernel, a, (int)std::min(u.units, (long long)ctas * dev_info().sms), kThreads, smem, stream);
  };
  if (c.D == 64)
    return wide ? launch(k_attend<64, 16, SP>, ctas_of<64>(), Shape<64, 16>::smem(batch))
                : launch(k_attend<64, 8, SP>, ctas_of<64>(), Shape<64, 8>::smem(batch));
  if (c.D == 128)
    return wide ? launch(k_attend<128, 16, SP>, ctas_of<128>(), Shape<128, 16>::smem(batch))
                : launch(k_attend<128, 8, SP>, ctas_of<128>(), Shape<128, 8>::smem(batch));
  return launch(k_attend<256, 8, SP>, ctas_of<256>(), Shape<256, 8>::smem(batch));
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
  return attend<false>(kv, q, ldq, new_k, new_v, ldn, lens, batch, q_heads, nullptr, 0, scale, out, ldo, ws, ws_bytes, stream);
}

extern "C" int q2_attend_blocks(const q2_kv* kv, const void* q, long long ldq, const int* lens, int batch, int q_heads,
                                const int* sel, int nsel, float scale, void* out, long long ldo, void* ws, size_t ws_bytes,
                                q2_stream stream) {
  if (nsel < 1) return Q2_ESHAPE;
  return attend<true>(kv, q, ldq, nullptr, nullptr, 0, lens, batch, q_heads, sel, nsel, scale, out, ldo, ws, ws_bytes, stream);
}

// The error word of the attention kernels, then cleared (q2_device_errors).
extern "C" int q2_attend_errors(unsigned int* out) {
  unsigned int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, q2_attend_error, sizeof(v)) != cudaSuccess) return Q2_ECUDA;
  if (v && cudaMemcpyToSymbol(q2_attend_error, &z, sizeof(z)) != cudaSuccess) return Q2_ECUDA;
  *out = v;
  return Q2_OK;
}
