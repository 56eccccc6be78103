// Device helpers of the strided [B,H,T,d] operators: packed loads and stores in the tensors' type, the
// logistic function with its complement, and the cluster primitives of the recurrence.
#pragma once

#include <cuda.h>
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
// units, the same for the same argument, which a memory of n tokens multiplies by n: there the Taylor
// series to the fourth degree (remainder below 16^-5 / 5! = 8e-9), whose one large rounding is that of the
// last sum.
__device__ __forceinline__ float decay_exp(float v) {
    float p = fmaf(v, 1.f / 24, 1.f / 6);
    p = fmaf(p, v, 0.5f);
    p = fmaf(p, v, 1.f);
    p = fmaf(p, v, 1.f);
    return fabsf(v) < 0.0625f ? p : ex2(kLog2e * v);
}

// ---- pairs of channels: the same functions on two values, packed where the hardware can
__device__ __forceinline__ float2 pair(float a, float b) { return make_float2(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }  // a b + c

// s = 1 / (1 + e^-v), c = 1 - s. With e = e^-|v| <= 1 the smaller of the two is e / (1 + e).
__device__ __forceinline__ void logistic2(float2 v, float2& s, float2& c) {
    const float2 e = pair(ex2(-kLog2e * fabsf(v.x)), ex2(-kLog2e * fabsf(v.y)));
    const float2 d = add2(e, pair(1.f, 1.f));
    const float2 small = mul2(e, pair(rcp(d.x), rcp(d.y)));
    const float2 large = fma2(small, pair(-1.f, -1.f), pair(1.f, 1.f));
    const bool px = v.x > 0.f, py = v.y > 0.f;
    s = pair(px ? large.x : small.x, py ? large.y : small.y);
    c = pair(px ? small.x : large.x, py ? small.y : large.y);
}
__device__ __forceinline__ float2 decay_exp2(float2 v) {
    float2 p = fma2(v, pair(1.f / 24, 1.f / 24), pair(1.f / 6, 1.f / 6));
    p = fma2(p, v, pair(0.5f, 0.5f));
    p = fma2(p, v, pair(1.f, 1.f));
    p = fma2(p, v, pair(1.f, 1.f));
    const float2 k = mul2(v, pair(kLog2e, kLog2e));
    return pair(fabsf(v.x) < 0.0625f ? p.x : ex2(k.x), fabsf(v.y) < 0.0625f ? p.y : ex2(k.y));
}

// ---- asynchronous copies of CB bytes, global to shared; `in` false writes zeros and reads nothing
template <int CB>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(CB), "r"(in ? CB : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- thread-block clusters
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The address of `saddr` (shared memory of this CTA) in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t peer(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
// Four floats into a peer's shared memory, counted as 16 bytes by the mbarrier `bar` of that peer.
__device__ __forceinline__ void st_async4(uint32_t addr, const float* v, uint32_t bar) {
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
        ::"r"(addr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
        "r"(__float_as_uint(v[3])), "r"(bar) : "memory");
}

// ---- TMA boxes of a [B,H,T,d] tensor (coordinates: channel, token, head, sequence)
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int c, int t, int h, int b,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(tm), "r"(c), "r"(t), "r"(h), "r"(b), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* tm, uint32_t src, int c, int t, int h, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
                 ::"l"(tm), "r"(src), "r"(c), "r"(t), "r"(h), "r"(b) : "memory");
}

}  // namespace seq
}  // namespace falcon
