// Group norm of a token's head with an activation and a gate: what the forward and the backward kernels
// share. A row is one (batch, head, token): d channels, held in registers by LPR neighbouring lanes, lane l
// with elements (l + LPR k) VW .. + VW - 1 for k < NCH.
#pragma once

#include "falcon_seq.cuh"
#include "falcon_seq.h"

namespace falcon {
namespace gn {

using namespace seq;

// ---- activations: v -> f(v), and its derivative
template <int ACT>
__device__ __forceinline__ float act(float v) {
    if (ACT == kActNone) return v;
    if (ACT == kActGelu) return 0.5f * v * erfcf(-0.70710678118654752f * v);
    float s, c;
    logistic(v, s, c);
    return ACT == kActSilu ? v * s : s;
}
template <int ACT>
__device__ __forceinline__ void act_slope(float v, float& f, float& df) {
    if (ACT == kActNone) {
        f = v;
        df = 1.f;
    } else if (ACT == kActGelu) {
        const float phi = 0.5f * erfcf(-0.70710678118654752f * v);
        f = v * phi;
        df = fmaf(v * 0.39894228040143268f, expf(-0.5f * v * v), phi);
    } else {
        float s, c;
        logistic(v, s, c);
        f = ACT == kActSilu ? v * s : s;
        df = ACT == kActSilu ? fmaf(v * s, c, s) : s * c;
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// x -> (x - mean) rstd in place, rows of d channels; elements behind d hold 0 on entry and return.
// Two passes over the registers: the variance is that of the centred values.
template <int LPR, int N>
__device__ __forceinline__ float normalise(float (&x)[N], const bool (&live)[N], int d, float inv_d, float eps) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) s += x[i];
    const float mean = row_sum<LPR>(s) * inv_d;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = live[i] ? x[i] - mean : 0.f;
        s = fmaf(x[i], x[i], s);
    }
    const float rstd = rsqrtf(row_sum<LPR>(s) * inv_d + eps);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= rstd;
    return rstd;
}

// n / d for 0 <= n < 2^31 by a multiplication: q = (n mul) >> 32 >> shift, with mul = ceil(2^(32+shift)/d)
// and 2^shift >= d / 2 (the error n (mul d - 2^(32+shift)) / (d 2^(32+shift)) stays below 1 / d).
struct FastDiv {
    uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f = {d, 0, 0};
    if (d == 1) return f;  // mul 0 marks it
    while ((1u << (f.shift + 1)) < d) ++f.shift;
    f.mul = (uint32_t)((((unsigned long long)1 << (32 + f.shift)) + d - 1) / d);
    return f;
}
__device__ __forceinline__ uint32_t div(uint32_t n, const FastDiv& f) {
    return f.mul ? __umulhi(n, f.mul) >> f.shift : n;
}

}  // namespace gn
}  // namespace falcon
