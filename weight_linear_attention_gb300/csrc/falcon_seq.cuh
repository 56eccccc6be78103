// Device helpers of the strided [B,H,T,d] operators: packed loads and stores in the tensors' type, the
// logistic function with its complement, and the cluster primitives of the recurrence.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace falcon {
namespace seq {

using bf16 = __nv_bfloat16;

// VW consecutive elements as they lie in memory.
template <typename E, int VW>
struct Pack;
template <>
struct Pack<float, 1> {
    float w;
};
template <>
struct __align__(16) Pack<float, 4> {
    float w[4];
};
template <>
struct Pack<bf16, 1> {
    uint16_t w;
};
template <>
struct __align__(8) Pack<bf16, 4> {
    uint32_t w[2];
};
template <>
struct __align__(16) Pack<bf16, 8> {
    uint32_t w[4];
};

__device__ __forceinline__ float elem(const Pack<float, 1>& p, int) { return p.w; }
__device__ __forceinline__ float elem(const Pack<float, 4>& p, int i) { return p.w[i]; }
__device__ __forceinline__ float elem(const Pack<bf16, 1>& p, int) { return __uint_as_float((uint32_t)p.w << 16); }
template <int VW>
__device__ __forceinline__ float elem(const Pack<bf16, VW>& p, int i) {
    const uint32_t u = p.w[i >> 1];
    return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
}

// The element type's nearest values, ties to even.
__device__ __forceinline__ void pack(Pack<float, 1>& p, const float* v) { p.w = v[0]; }
__device__ __forceinline__ void pack(Pack<float, 4>& p, const float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.w[i] = v[i];
}
__device__ __forceinline__ void pack(Pack<bf16, 1>& p, const float* v) { p.w = __bfloat16_as_ushort(__float2bfloat16_rn(v[0])); }
template <int VW>
__device__ __forceinline__ void pack(Pack<bf16, VW>& p, const float* v) {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        p.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <typename E, int VW>
__device__ __forceinline__ void zero(Pack<E, VW>& p) {
    float z[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) z[i] = 0.f;
    pack(p, z);
}
template <typename E, int VW>
__device__ __forceinline__ Pack<E, VW> load(const void* base, long long off) {
    return *reinterpret_cast<const Pack<E, VW>*>(static_cast<const E*>(base) + off);
}
template <typename E, int VW>
__device__ __forceinline__ void store(void* base, long long off, const Pack<E, VW>& p) {
    *reinterpret_cast<Pack<E, VW>*>(static_cast<E*>(base) + off) = p;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// s = 1 / (1 + e^-v) and c = 1 - s, both to a few units of the last place of fp32: with e = e^-v the
// smaller of the two is computed as a quotient and the larger as one minus it, so that an s close to 1
// (a long memory) carries the rounding of one subtraction and no bias of the reciprocal's.
// v = -inf: e = inf, s = 0, c = 1. v = +inf: e = 0, s = 1, c = 0. NaN stays NaN.
__device__ __forceinline__ void logistic(float v, float& s, float& c) {
    const float e = ex2(-kLog2e * v);
    const float r = rcp(1.f + e);
    const bool low = e < 1.f;
    const float small = low ? e * r : r;
    const float large = 1.f - small;
    s = low ? large : small;
    c = low ? small : large;
}

// e^v. Close to 0 (a log decay of a long memory) the hardware's base-2 exponential is off by up to two
// units, always on one side for a given argument, which a memory of n tokens multiplies by n: there the
// Taylor series to the sixth degree (remainder below 0.25^7 / 7! = 1.3e-8), whose one large rounding is
// that of the last sum.
__device__ __forceinline__ float decay_exp(float v) {
    float p = fmaf(v, 1.f / 720, 1.f / 120);
    p = fmaf(p, v, 1.f / 24);
    p = fmaf(p, v, 1.f / 6);
    p = fmaf(p, v, 0.5f);
    p = fmaf(p, v, 1.f);
    p = fmaf(p, v, 1.f);
    return fabsf(v) < 0.25f ? p : ex2(kLog2e * v);
}

// ---- thread-block clusters
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of `saddr` (shared memory of this CTA) in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_peer(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_peer4(uint32_t addr, const float* v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

}  // namespace seq
}  // namespace falcon
