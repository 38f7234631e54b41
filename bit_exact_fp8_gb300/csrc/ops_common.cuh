// ops_common.cuh -- what the operators around the 8-bit product share: element types,
// 16-byte loads, warp reductions, and the host side's errors and checks.  (The GEMM's own
// header holds kernels that belong to one translation unit, so nothing is taken from it.)
#pragma once

#include "emu_fp8.h"

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <initializer_list>

// host side (ops_norm.cu): records the message emu_ops_last_error returns; gives `code`
int emu_ops_fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void emu_ops_begin();                          // clears the message and a stale launch error
int emu_ops_launched(const char* what);        // EMU_OK, or EMU_ECUDA with the launch's error
int emu_ops_sm_count();                        // SMs of the current device
int emu_ops_int8_status(int* status, bool reset);          // ops_int8.cu's device status word
// the dynamic shared memory a kernel may take, set once a device (`done`: one flag a device)
bool emu_ops_allow_smem(const void* kernel, int bytes, std::atomic<bool>* done);

namespace emu_ops {

inline bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
inline size_t elem_bytes(emu_out_t t) { return t == EMU_OUT_F32 ? 4 : 2; }
inline bool is_float_type(emu_out_t t) { return t == EMU_OUT_F32 || t == EMU_OUT_BF16 || t == EMU_OUT_F16; }

// rows x cols elements of `esz` bytes, rows `ld` elements apart: the bytes they span
struct Span {
  uintptr_t lo, hi;
  Span(const void* p, int64_t rows, int64_t ld, int64_t cols, size_t esz)
      : lo(reinterpret_cast<uintptr_t>(p)), hi(lo) {
    if (p && rows > 0 && cols > 0) hi = lo + ((size_t)(rows - 1) * (size_t)ld + (size_t)cols) * esz;
  }
  bool meets(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};
// do all of `outs` lie apart, from each other and from all of `ins`
inline bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* p = o + 1; p != outs.end(); ++p)
      if (o->meets(*p)) return false;
    for (const Span& i : ins)
      if (o->meets(i)) return false;
  }
  return true;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// VEC elements loaded or stored at once (VEC * sizeof(T) = 16 bytes, or one element)
template <class T, int VEC> struct alignas(sizeof(T) * VEC) Pack {
  T v[VEC];
};
template <class T, int VEC> __device__ __forceinline__ void load_f(const T* p, float (&f)[VEC]) {
  const Pack<T, VEC> q = *reinterpret_cast<const Pack<T, VEC>*>(p);
#pragma unroll
  for (int i = 0; i < VEC; ++i) f[i] = to_f(q.v[i]);
}
constexpr int kMaxSmem = 227 * 1024;              // dynamic shared memory of a CTA at most

template <class T, int VEC> __device__ __forceinline__ void store_f(T* p, const float (&f)[VEC]) {
  Pack<T, VEC> q;
#pragma unroll
  for (int i = 0; i < VEC; ++i) q.v[i] = from_f<T>(f[i]);
  *reinterpret_cast<Pack<T, VEC>*>(p) = q;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// mbarriers and bulk copies (inline PTX)
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_init_fence() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred P;\n mbarrier.try_wait.parity.shared::cta.b64 P, [%1], %2;\n selp.u32 %0, 1, 0, P;\n}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0u;
}
// polls before a wait gives up; each suspends the thread for a short time set by the hardware, so a wait
// ends well within seconds
constexpr uint32_t kPolls = 1u << 20;
// Waits for the phase of this parity to complete; false once the limit is reached.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < kPolls; ++i)
    if (bar_try(bar, parity)) return true;
  return false;
}
// `bytes` (a multiple of 16) from 16-byte aligned memory to 16-byte aligned shared memory
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// every thread of every CTA of the cluster arrives; what it wrote before is seen after the others' waits
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// the address of `p`, of this CTA's shared memory, in that of the cluster's CTA `rank`
__device__ __forceinline__ uint32_t in_cluster(const void* p, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}

// fp32 pairs: one instruction for two values
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void halves(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// the larger of two, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

}  // namespace emu_ops
