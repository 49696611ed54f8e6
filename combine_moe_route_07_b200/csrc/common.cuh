// common.cuh -- device helpers shared by the route / layout / dispatch /
// combine kernels (sm_100a).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_route07.h"

namespace moe {

constexpr unsigned kFull = 0xffffffffu;

// Workspace header (first 256 bytes of every workspace).
struct WsHeader {
  int32_t err;             // first device-side error code (moe_status_t), 0 = none
  int32_t detail;          // index that caused it
  uint32_t reserved[2];
  uint32_t epoch;          // layout: which of the two tile tables the next call fills
  uint32_t done;           // layout: place CTAs finished (the last one bumps epoch)
  uint32_t words_used[2];  // layout: words of each table filled since it was last cleared
  uint32_t pad[56];        // (epoch..words_used form one 16-byte word at offset 16)
};
static_assert(sizeof(WsHeader) == 256, "workspace header is 256 bytes");

// Record the first device-side problem; later ones are dropped.
__device__ __forceinline__ void report(WsHeader* h, int code, int detail) {
  if (atomicCAS(&h->err, 0, code) == 0) atomicExch(&h->detail, detail);
}

// Relaxed, GPU-scope 32-bit load/store (one word carries flag and value, so
// no extra ordering is needed between them).
__device__ __forceinline__ uint32_t ld_relaxed(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_relaxed(uint32_t* p, uint32_t v) {
  asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// L2-coherent 32-bit load (bypasses L1), for data another CTA published.
__device__ __forceinline__ int32_t ld_cg(const int32_t* p) { return __ldcg(p); }

// Programmatic dependent launch.  pdl_wait(): block until the kernel this one
// was launched behind has finished and its writes are visible (returns at once
// when launched without the attribute).  pdl_trigger(): allow the kernel
// launched behind this one to start placing its CTAs.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ unsigned lanemask_lt() {
  unsigned m;
  asm("mov.u32 %0, %%lanemask_lt;" : "=r"(m));
  return m;
}

// 16-byte global accesses.
__device__ __forceinline__ uint4 ldg16(const void* p) {
  return __ldg(reinterpret_cast<const uint4*>(p));
}
// Streaming load: data read once, keep it out of L1.
__device__ __forceinline__ uint4 ld16_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void st16(void* p, const uint4& v) {
  *reinterpret_cast<uint4*>(p) = v;
}

// 2^x within 2^-22 of itself and 1/x within 2^-23, subnormals flushed; the logistic
// function from them, within (7 + 1.23 |x|) 2^-24 of itself (x log2(e) is rounded and
// log2(e) is, which the exponential turns into 1.23 |x| steps of 2^-24; 4 for 2^x, 1 for
// the addition, 2 for the reciprocal): 2^-19.9 at |x| = 8, 2^-17.5 at 64.  Below -87.3
// it is 0.  The library's fast forms handle subnormals too, at about three times the
// instructions.
__device__ __forceinline__ float ex2_f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_f(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.44269504f;
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_f(1.0f + ex2_f(x * -kLog2e)); }

// Phi(-|z|), the normal distribution's tail, and *e = exp(-z^2 / 2), which it shares:
// Phi(-x) exp(x^2 / 2) = t P(t), t = 1 / (1 + 0.3 x), P of degree 7 the polynomial with the
// smallest largest relative error over 0 <= x <= 13.5 (1.2e-7, by linear programming on 1500
// Chebyshev nodes; 2^-20.7 with its roundings in fp32).  Relative to the tail itself, so
// that z Phi(z) keeps its digits at far negative z: within (17 + 1.12 z^2) 2^-24 (2^x takes
// 4, three products 3, and the exponent's roundings 1.12 z^2); below z = -13.2 it is 0.
__device__ __forceinline__ float normal_tail(float z, float* e) {
  const float t = rcp_f(fmaf(0.3f, fabsf(z), 1.0f));
  float q = fmaf(3.591387346e-02f, t, -1.581697464e-01f);
  q = fmaf(q, t, 2.079638243e-01f);
  q = fmaf(q, t, -5.511194840e-02f);
  q = fmaf(q, t, 1.292886287e-01f);
  q = fmaf(q, t, 9.970111400e-02f);
  q = fmaf(q, t, 1.207870170e-01f);
  q = fmaf(q, t, 1.196271777e-01f);
  *e = ex2_f(z * z * (-0.5f * kLog2e));
  return q * t * *e;
}

// bf16 pair <-> fp32 (exact widening; nearest-even narrowing).
__device__ __forceinline__ float bf16lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace moe
