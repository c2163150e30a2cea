// Paged key-value caches as the kernels see them: places of tokens, and the
// checks of what a caller describes.
#pragma once
#include <type_traits>

#include "q2_common.cuh"

namespace q2 {

// Pools of keys and values (or of their steps and offsets); strides in bytes.
struct Pages {
  unsigned char* k;
  unsigned char* v;
  long long page_stride, token_stride, head_stride;
  const int* table;
  long long table_stride;
  int npages, page;
  uint32_t page_mul, page_sh;   // t / page = (high half of t * page_mul, + t) >> page_sh, t < 2^31
};

// Division by an invariant with a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994).
inline void set_page(int page, uint32_t& mul, uint32_t& sh) {
  sh = 0;
  while ((1ll << sh) < page) ++sh;
  mul = (uint32_t)(((1ull << 32) * ((1ull << sh) - page)) / page + 1);
}

template <class A>
__device__ __forceinline__ int page_of(const A& a, int t) {
  return (int)((__umulhi((uint32_t)t, a.page_mul) + (uint32_t)t) >> a.page_sh);
}

// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

struct CacheShape {
  int D, group, kv_heads, page;   // group: columns of a group in 4 bits, 0 in fp16
  long long cap;                  // tokens that a table row can hold
};

inline bool misaligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

template <class KV>
int check_pages(const KV* kv, int batch, Pages& pg, CacheShape& c) {
  if (!kv) return Q2_EINVAL;
  c.D = kv->head_dim;
  c.kv_heads = kv->kv_heads;
  c.page = kv->page_size;
  c.cap = (long long)kv->max_pages * kv->page_size;
  if (c.D != 64 && c.D != 128 && c.D != 256) return Q2_ESHAPE;
  if (kv->kv_heads < 1 || kv->kv_heads > 65536 || kv->page_size < 1 || kv->npages < 0 || kv->max_pages < 0) return Q2_ESHAPE;
  if (kv->page_stride < 0 || kv->token_stride < 0 || kv->head_stride < 0) return Q2_ESHAPE;
  if (batch > 1 && kv->table_stride < kv->max_pages) return Q2_ESHAPE;
  if (c.cap > 0x7fffff00ll) return Q2_ESHAPE;     // tokens are counted in 32 bits on the device
  if (misaligned(kv->k, 16) || misaligned(kv->v, 16) || misaligned(kv->table, 4)) return Q2_EALIGN;
  pg = {};
  pg.k = static_cast<unsigned char*>(kv->k);
  pg.v = static_cast<unsigned char*>(kv->v);
  pg.table = kv->table;
  pg.table_stride = kv->table_stride;
  pg.npages = kv->npages;
  pg.page = kv->page_size;
  set_page(pg.page, pg.page_mul, pg.page_sh);
  return batch > 0 && (!kv->k || !kv->v || !kv->table) ? Q2_EINVAL : Q2_OK;
}

inline int check_cache(const q2_kv* kv, int batch, Pages& pg, CacheShape& c) {
  const int st = check_pages(kv, batch, pg, c);
  if (st) return st;
  if (kv->page_stride % 8 || kv->token_stride % 8 || kv->head_stride % 8) return Q2_EALIGN;
  pg.page_stride = kv->page_stride * 2;
  pg.token_stride = kv->token_stride * 2;
  pg.head_stride = kv->head_stride * 2;
  c.group = 0;
  return Q2_OK;
}

inline int check_cache4(const q2_kv4* kv, int batch, Pages& pg, Pages& sp, CacheShape& c) {
  const int st = check_pages(kv, batch, pg, c);
  if (st) return st;
  if (kv->group != 32 && kv->group != 64) return Q2_ESHAPE;
  if (kv->s_page_stride < 0 || kv->s_token_stride < 0 || kv->s_head_stride < 0) return Q2_ESHAPE;
  if (batch > 0 && (!kv->ks || !kv->vs)) return Q2_EINVAL;
  const int unit = std::min(4, c.D / kv->group);    // pairs that are copied as one
  if (kv->page_stride % 16 || kv->token_stride % 16 || kv->head_stride % 16 || misaligned(kv->ks, 16) ||
      misaligned(kv->vs, 16) || kv->s_page_stride % unit || kv->s_token_stride % unit || kv->s_head_stride % unit)
    return Q2_EALIGN;
  c.group = kv->group;
  pg.page_stride = kv->page_stride;
  pg.token_stride = kv->token_stride;
  pg.head_stride = kv->head_stride;
  sp = pg;
  sp.k = static_cast<unsigned char*>(kv->ks);
  sp.v = static_cast<unsigned char*>(kv->vs);
  sp.page_stride = kv->s_page_stride * 4;
  sp.token_stride = kv->s_token_stride * 4;
  sp.head_stride = kv->s_head_stride * 4;
  return Q2_OK;
}

// Calls f with the head's columns and the columns of a group as constants.
template <class F>
int by_shape(const CacheShape& c, F f) {
  auto with = [&](auto D) {
    return c.group == 0    ? f(D, std::integral_constant<int, 0>())
           : c.group == 32 ? f(D, std::integral_constant<int, 32>())
                           : f(D, std::integral_constant<int, 64>());
  };
  return c.D == 64    ? with(std::integral_constant<int, 64>())
         : c.D == 128 ? with(std::integral_constant<int, 128>())
                      : with(std::integral_constant<int, 256>());
}

}  // namespace q2
