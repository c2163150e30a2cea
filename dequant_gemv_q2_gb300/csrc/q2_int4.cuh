// What the kernels for 4-bit weights share (q2_int4.cu, q2_int4_tc.cu).
#pragma once
#include <cuda_fp16.h>

#include <mutex>
#include <vector>

#include "q2_common.cuh"

namespace q2 {

struct Int4Args {
  const unsigned char* w;     // [ntile][nblk] blocks of `item` bytes: weights, scales, zero points
  const void* x;              // [ntok][C] fp16 or int8
  const float* xs;            // [ntok], 8-bit x only
  __half* y;                  // [ntok][R]
  int R, C, nblk, ntile, ntok, item;
  int zeros;                  // blocks hold zero points; else 8 everywhere
};

// The scales (rows g and g + 8) and zero points of a lane's rows in one block.
template <int GPB>            // groups per block: 1, 2 or 4
struct Sides {
  uint32_t s[GPB];
  uint32_t z[(GPB + 1) / 2];
};

// Blocks go to shared memory by asynchronous 16-byte copies (a register ring
// was bound by the six scoreboards a warp has: waiting for x meant waiting
// for weights requested after it; 19.1 us instead of 14.3 at 24576 x 4096).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

__device__ __forceinline__ uint32_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}

template <int GPB>
__device__ __forceinline__ void load_sides(Sides<GPB>& k, uint32_t blk, int zeros, int g) {
  const uint32_t s = blk + 1024 + g * (GPB * 4), z = blk + 1024 + GPB * 32 + g * (GPB * 2);
  if constexpr (GPB == 1) {
    k.s[0] = lds32(s);
    k.z[0] = zeros ? lds16(z) : 0x0808u;
  } else if constexpr (GPB == 2) {
    const uint2 v = lds64(s);
    k.s[0] = v.x;
    k.s[1] = v.y;
    k.z[0] = zeros ? lds32(z) : 0x08080808u;
  } else {
    const uint4 v = lds128(s);
    k.s[0] = v.x;
    k.s[1] = v.y;
    k.s[2] = v.z;
    k.s[3] = v.w;
    const uint2 u = zeros ? lds64(z) : make_uint2(0x08080808u, 0x08080808u);
    k.z[0] = u.x;
    k.z[1] = u.y;
  }
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// (v & mask) | bits as one instruction (from two constants the compiler makes two)
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
  return d;
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// What unpack_step takes off: 1024 + z of row g and -(64 + z) of row g + 8, as
// pairs, from the rows' zero points as two bytes.
struct Zeros {
  uint32_t z0, z1;
};
__device__ __forceinline__ Zeros zeros_of(uint32_t zz) {
  return Zeros{and_or(zz, 0xffu, 0x6400u) * 0x10001u, and_or(zz >> 4, 0xff0u, 0xd400u) * 0x10001u};
}

// One step's q - z (four columns of rows g and g + 8) as an operand fragment:
// a0 and a2 of row g, a1 and a3 of row g + 8.  The word holds, from its lowest
// four bits up, columns 0, 0, 2, 2, 1, 1, 3, 3, rows g and g + 8 in turn.
// (Integers in the mantissa of 1024: Kim, Henry, Fahim and Awadalla, "Who Says
// Elephants Can't Run", 2022.)
__device__ __forceinline__ void unpack_step(uint32_t v, const Zeros& z, uint32_t& a0, uint32_t& a1, uint32_t& a2,
                                            uint32_t& a3) {
  const uint32_t v8 = v >> 8;
  a0 = hsub2(and_or(v, 0x000f000fu, 0x64006400u), z.z0);
  a1 = hfma2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z.z1);
  a2 = hsub2(and_or(v8, 0x000f000fu, 0x64006400u), z.z0);
  a3 = hfma2(and_or(v8, 0x00f000f0u, 0x64006400u), 0x2c002c00u, z.z1);
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Four 8-bit integers as two pairs of fp16: the byte plus 128 in the mantissa
// of 1024, minus 1152.
__device__ __forceinline__ void int8x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  v ^= 0x80808080u;
  lo = hsub2(__byte_perm(v, 0x64646464u, 0x4140), 0x64806480u);
  hi = hsub2(__byte_perm(v, 0x64646464u, 0x4342), 0x64806480u);
}

// c += a * b, a pair at a time
__device__ __forceinline__ void fma2(float2& c, float2 a, float2 b) {
  uint64_t& cc = reinterpret_cast<uint64_t&>(c);
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(cc) : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
}

// The cluster's barriers, by converged warps.  The first: what each CTA has left
// in its shared memory is there for the others.  The second, behind the last
// reads of other CTAs' shared memory, in two halves: the arrival orders those
// reads before it (a releasing one does, a relaxed one would not), and the
// stores of what was read come behind it, so that it does not wait for them.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_meet() {
  cluster_arrive();
  cluster_wait();
}

constexpr int kSmemPerSm = 228 * 1024;              // a CTA takes 1 KB beside its own

// How many clusters of cs CTAs of a kernel the device runs at once (a cluster
// lives in one GPC, so this is not SMs / cs), each asked for once: kernels that
// share a table differ in their registers.
class ClusterCounts {
  struct Known {
    const void* fn;
    int dev, cs, smem, n;
  };
  std::mutex mu;
  std::vector<Known> known;

 public:
  int get(const void* fn, int cs, int threads, int smem) {
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lk(mu);
    for (const Known& k : known)
      if (k.fn == fn && k.dev == dev && k.cs == cs && k.smem == smem) return k.n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cs);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return 1;
    }
    try {
      known.push_back({fn, dev, cs, smem, n});
    } catch (...) {}                                // no memory: asked for again
    return n;
  }
};

// Launch in clusters of cs CTAs, programmatic stream serialization allowed.
template <typename... A, typename... B>
int launch_clusters(void (*kernel)(A...), int clusters, int cs, int threads, int smem, void* stream, const B&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * cs);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    (void)cudaGetLastError();
    return Q2_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? Q2_OK : Q2_ECUDA;
}

}  // namespace q2

// 17..64 tokens on the 5th-generation tensor cores (q2_int4_tc.cu).
int q2_int4_tc(const q2::Int4Args& a, int group, bool x8, void* stream);
