// Group norm of a token's head with an activation and a gate: what the forward and the backward kernels
// share. A row is one (batch, head, token): d channels, held in registers by LPR neighbouring lanes, lane l
// with elements (l + LPR k) VW .. + VW - 1 for k < NCH.
#pragma once

#include <atomic>
#include <type_traits>

#include "falcon_seq.cuh"
#include "falcon_seq.h"
#include "sm103_ptx.cuh"

namespace falcon {
namespace gn {

using namespace seq;

// ---- activations, of s = 1 / (1 + e) with e = e^-v. Where e overflows s is 0 (a logistic below 2^-126 is flushed to
// it), so that v s is 0 for every finite v down to the type's lowest, off by at most |v| 2^-126 where the exact value
// is not yet below that. NaN stays NaN.
__device__ __forceinline__ float2 exp_neg(float2 v) {
    const float2 k = mul2(v, pair(-kLog2e, -kLog2e));
    return pair(ex2(k.x), ex2(k.y));
}
// 1 - s as e s, exact to a few units. The cut at 2^126 keeps infinity times 0 out of it: s is 0 there, and the slopes
// multiply 1 - s by s or by v s.
__device__ __forceinline__ float2 one_minus(float2 e, float2 s) {
    float2 c;
    asm("min.NaN.f32 %0, %1, 0f7E800000;" : "=f"(c.x) : "f"(e.x));
    asm("min.NaN.f32 %0, %1, 0f7E800000;" : "=f"(c.y) : "f"(e.y));
    return mul2(c, s);
}
__device__ __forceinline__ float2 rcp2(float2 v) { return pair(rcp(v.x), rcp(v.y)); }

// The normal distribution function and e = exp(-v^2 / 2). With x = |v| / sqrt 2 and t = 1 / (1 + 0.45 x),
// exp(x^2) erfc(x) = t P(t); P is a least-squares fit of degree 9 over t in (0, 1], its weights moved to level the
// relative error. With the constants rounded to fp32 as below it is at most 1.2e-7 up to |v| = 5, 1.4e-7 up to 14 and
// 1.5e-7 everywhere (two and a half units). The lower tail keeps its relative accuracy; the upper is one minus it.
__device__ __forceinline__ void normal2(float2 v, float2& phi, float2& e) {
    constexpr float kT = 0.45f * 0.70710678118654752f, kE = -0.5f * kLog2e;
    const float2 t = pair(rcp(fmaf(kT, fabsf(v.x), 1.f)), rcp(fmaf(kT, fabsf(v.y), 1.f)));
    constexpr float c[10] = {0.25388533f, 0.25388315f, 0.22827165f, 0.17525212f, 0.11995047f,
                             -0.02235809f, 0.14240131f, -0.30058289f, 0.19068813f, -0.04139117f};
    float2 p = pair(c[9], c[9]);
#pragma unroll
    for (int k = 8; k >= 0; --k) p = fma2(p, t, pair(c[k], c[k]));
    const float2 s = mul2(mul2(v, v), pair(kE, kE));
    e = pair(ex2(s.x), ex2(s.y));
    const float2 low = mul2(mul2(t, pair(0.5f, 0.5f)), mul2(p, e));
    const float2 high = fma2(low, pair(-1.f, -1.f), pair(1.f, 1.f));
    phi = pair(v.x > 0.f ? high.x : low.x, v.y > 0.f ? high.y : low.y);
}

template <int ACT>
__device__ __forceinline__ float2 act(float2 v) {
    if (ACT == kActNone) return v;
    if (ACT == kActGelu) {
        float2 phi, e;
        normal2(v, phi, e);
        return mul2(v, phi);
    }
    const float2 s = rcp2(add2(exp_neg(v), pair(1.f, 1.f)));
    return ACT == kActSilu ? mul2(v, s) : s;
}
// f(v) and f'(v)
template <int ACT>
__device__ __forceinline__ void act_slope(float2 v, float2& f, float2& df) {
    if (ACT == kActNone) {
        f = v;
        df = pair(1.f, 1.f);
    } else if (ACT == kActGelu) {
        constexpr float q = 0.39894228040143268f;  // 1 / sqrt(2 pi)
        float2 phi, e;
        normal2(v, phi, e);
        f = mul2(v, phi);
        df = fma2(mul2(v, pair(q, q)), e, phi);
    } else {
        const float2 e = exp_neg(v), s = rcp2(add2(e, pair(1.f, 1.f))), c = one_minus(e, s);
        f = ACT == kActSilu ? mul2(v, s) : s;
        df = ACT == kActSilu ? fma2(f, c, s) : mul2(s, c);
    }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float2 p) {
    float v = p.x + p.y;
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A thread's share of a row: NCH chunks of VW channels as P pairs. FULL: every lane's channels exist.
template <int VW, int LPR, int NCH, bool FULL>
struct Row {
    static constexpr int P = NCH * VW / 2;
    static_assert(NCH * VW % 2 == 0, "pairs");
    int l;     // the lane of the row
    int d;
    __device__ __forceinline__ int chan(int k) const { return (l + LPR * k) * VW; }  // first of chunk k
    __device__ __forceinline__ bool live(int k) const { return FULL || chan(k) < d; }
    // the value of element e in pairs, 0 where it does not exist
    __device__ __forceinline__ float2 keep(int i, float2 v) const {
        return FULL ? v : pair(live(2 * i / VW) ? v.x : 0.f, live((2 * i + 1) / VW) ? v.y : 0.f);
    }
    template <typename E>
    __device__ __forceinline__ void get(const Pack<E, VW> (&p)[NCH], float2 (&v)[P]) const {
#pragma unroll
        for (int i = 0; i < P; ++i)
            v[i] = pair(elem(p[2 * i / VW], 2 * i % VW), elem(p[(2 * i + 1) / VW], (2 * i + 1) % VW));
    }
    // chunk k of pairs, in memory's form
    template <typename E>
    __device__ __forceinline__ Pack<E, VW> put(const float2 (&v)[P], int k) const {
        float w[VW];
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            const int e = k * VW + j;
            w[j] = e % 2 ? v[e / 2].y : v[e / 2].x;
        }
        Pack<E, VW> p;
        pack(p, w);
        return p;
    }
    // fp32 values per channel, `none` where there are none
    template <int FW>
    __device__ __forceinline__ void params(const float* s, float none, float2 (&v)[P]) const {
        float w[NCH * VW];
#pragma unroll
        for (int k = 0; k < NCH; ++k)
#pragma unroll
            for (int j = 0; j < VW; j += FW) {
                Pack<float, FW> q;
                zero(q);
                if (s && live(k)) q = load<float, FW>(s, chan(k) + j);
#pragma unroll
                for (int m = 0; m < FW; ++m) w[k * VW + j + m] = s ? elem(q, m) : live(k) ? none : 0.f;
            }
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = pair(w[2 * i], w[2 * i + 1]);
    }
    // x -> (x - mean) rstd in place; elements that do not exist hold 0 on entry and return. Two passes over the
    // registers: the variance is that of the centred values.
    __device__ __forceinline__ float normalise(float2 (&x)[P], float inv_d, float eps) const {
        float2 s = x[0];
#pragma unroll
        for (int i = 1; i < P; ++i) s = add2(s, x[i]);
        const float mean = row_sum<LPR>(s) * inv_d;
        s = pair(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            x[i] = keep(i, add2(x[i], pair(-mean, -mean)));
            s = fma2(x[i], x[i], s);
        }
        const float rstd = rsqrtf(row_sum<LPR>(s) * inv_d + eps);
#pragma unroll
        for (int i = 0; i < P; ++i) x[i] = mul2(x[i], pair(rstd, rstd));
        return rstd;
    }
};

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

// Where a group of lanes is: token t of sequence b, and its place in K tensors. A grid of groups steps `by` rows
// (of B T) at a time: qb sequences and qt tokens, inc = qb sb + qt st bytes, and where that leaves the sequence
// one sequence more, wrap = sb - T st bytes.
template <int K>
struct Tensors {
    char* base[K];
    long long sb[K], sh[K], st[K], inc[K], wrap[K];  // bytes
    FastDiv tokens;                                  // T
    uint32_t B, by, qb, qt;
};
template <int K>
inline void set_step(Tensors<K>& s, uint32_t by) {
    const uint32_t T = s.tokens.d;
    s.by = by, s.qb = by / T, s.qt = by % T;
    for (int k = 0; k < K; ++k) {
        s.inc[k] = (long long)s.qb * s.sb[k] + (long long)s.qt * s.st[k];
        s.wrap[k] = s.sb[k] - (long long)T * s.st[k];
    }
}
// A place in the N tensors from number FIRST on.
template <int FIRST, int N>
struct Walk {
    uint32_t b, t;
    char* at[N];
    // row r of head h, byte `c` of it
    template <int K>
    __device__ __forceinline__ void start(const Tensors<K>& s, uint32_t r, uint32_t h, int c) {
        b = div(r, s.tokens);
        t = r - b * s.tokens.d;
#pragma unroll
        for (int k = 0; k < N; ++k)
            at[k] = s.base[FIRST + k] + (b * s.sb[FIRST + k] + h * s.sh[FIRST + k] + t * s.st[FIRST + k] + c);
    }
    template <int K>
    __device__ __forceinline__ void step(const Tensors<K>& s) {
        b += s.qb;
        t += s.qt;
#pragma unroll
        for (int k = 0; k < N; ++k) at[k] += s.inc[FIRST + k];
        if (t >= s.tokens.d) {
            ++b;
            t -= s.tokens.d;
#pragma unroll
            for (int k = 0; k < N; ++k) at[k] += s.wrap[FIRST + k];
        }
    }
    template <int K>
    __device__ __forceinline__ bool exists(const Tensors<K>& s) const { return b < s.B; }
    // the row lies inside its sequence
    template <int K>
    __device__ __forceinline__ bool in(const Tensors<K>& s, const int32_t* lengths) const {
        return exists(s) && (!lengths || (int)t < lengths[b]);
    }
};

// A group's rows: the first NT of K tensors (all where GATED, else without number 1) are read ahead of their use, into
// a ring of D rows a thread in shared memory, each thread's bytes its own, or (D = 0) into registers, one row ahead where
// AHEAD; the others are written. Rows outside their sequence are not read, their place holds what was there before.
// Channels that do not exist are zero.
template <typename E, int VW, int LPR, int NCH, bool FULL, bool GATED, int NT, int K, int THREADS, int D, bool AHEAD>
struct Rows {
    using V = Pack<E, VW>;
    using Q = Row<VW, LPR, NCH, FULL>;
    using Held = std::conditional_t<sizeof(V) == 2, uint32_t, V>;  // halves of registers would wait for their loads
    static constexpr int CB = LPR * VW * sizeof(E);                // from one chunk of a lane to its next
    static constexpr int kRow = (GATED ? NT : NT - 1) * NCH * THREADS;  // packs of a row of the ring
    Walk<0, D ? NT : K> at;
    Walk<NT, K - NT> dst;  // with a ring: the row at hand
    Held reg[D ? 1 : NT][D ? 1 : NCH];
    V* ring;
    uint32_t to;
    int head;           // the ring's row at hand
    bool ahead_in;      // the row fetched last lies inside its sequence
    bool mine, in;      // the row at hand exists, and lies inside its sequence
    char* out[K - NT];  // where it is written

    static __device__ __forceinline__ constexpr bool has(int k) { return GATED || k != 1; }
    static __device__ __forceinline__ constexpr int slot(int k, int j) {
        return ((GATED || k == 0 ? k : k - 1) * NCH + j) * THREADS;
    }
    __device__ __forceinline__ void fetch(const Q& q, const Tensors<K>& s, const int32_t* lengths, int row) {
        ahead_in = at.in(s, lengths);
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if (ahead_in && q.live(j)) {
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    if (!has(k)) continue;
                    const char* from = at.at[k] + j * CB;
                    if constexpr (D > 0) copy_async<sizeof(V)>(to + (row * kRow + slot(k, j)) * (int)sizeof(V), from, true);
                    else if constexpr (sizeof(V) == 2) reg[k][j] = *reinterpret_cast<const uint16_t*>(from);
                    else reg[k][j] = *reinterpret_cast<const V*>(from);
                }
            }
        }
        if constexpr (D > 0) {
            at.step(s);
            copy_commit();
        }
    }
    __device__ __forceinline__ void start(const Q& q, const Tensors<K>& s, const int32_t* lengths, uint32_t r, uint32_t h,
                                          void* shared) {
        const int c0 = q.chan(0) * (int)sizeof(E);
        at.start(s, r, h, c0);
        if constexpr (D > 0) {
            dst.start(s, r, h, c0);
            ring = static_cast<V*>(shared) + threadIdx.x;
            to = ptx::smem_u32(ring);
            if (!FULL) {
                V none;
                zero(none);
#pragma unroll 1
                for (int i = 0; i < D * kRow / THREADS; ++i) ring[i * THREADS] = none;
            }
            head = 0;
#pragma unroll
            for (int i = 0; i < D - 1; ++i) fetch(q, s, lengths, i);
        } else {
#pragma unroll
            for (int k = 0; k < NT; ++k)
#pragma unroll
                for (int j = 0; j < NCH; ++j) reg[k][j] = Held{};
            if (AHEAD) fetch(q, s, lengths, 0);
        }
    }
    // Waits for the row at hand.
    __device__ __forceinline__ void wait(const Q& q, const Tensors<K>& s, const int32_t* lengths) {
        if constexpr (D > 0) {
            copy_wait<D - 2>();
            mine = dst.exists(s);
            in = dst.in(s, lengths);
#pragma unroll
            for (int k = 0; k < K - NT; ++k) out[k] = dst.at[k];
        } else {
            if (!AHEAD) fetch(q, s, lengths, 0);
            mine = at.exists(s);
            in = ahead_in;
#pragma unroll
            for (int k = 0; k < K - NT; ++k) out[k] = at.at[NT + k];
        }
    }
    template <int P>
    __device__ __forceinline__ void get(const Q& q, int k, float2 (&v)[P]) const {
        V w[NCH];
#pragma unroll
        for (int j = 0; j < NCH; ++j) {
            if constexpr (D > 0) w[j] = ring[head * kRow + slot(k, j)];
            else if constexpr (sizeof(V) == 2) w[j].w = (uint16_t)reg[k][j];
            else w[j] = reg[k][j];
        }
        q.get(w, v);
    }
    // Behind the row's `get`s: on to the next, or the one that its place in the ring is for.
    __device__ __forceinline__ void next(const Q& q, const Tensors<K>& s, const int32_t* lengths) {
        if constexpr (D > 0) {
            fetch(q, s, lengths, head == 0 ? D - 1 : head - 1);
            head = head == D - 1 ? 0 : head + 1;
            dst.step(s);
        } else {
            at.step(s);
            if (AHEAD) fetch(q, s, lengths, 0);
        }
    }
};

constexpr int kSms = 152;

constexpr int kMaxDevices = 64;
constexpr int kSmem = 220 * 1024;  // of an SM, for the CTAs that it is given

// The rows a ring has: three (more gain nothing: 60.5 us either way for [16,16,4096,64] bf16 forward), or two where
// that is too much for the shared memory of `ctas` CTAs with `other` bytes besides.
constexpr int depth(int row, int ctas, int other) {
    return ctas * (3 * row + other) <= kSmem ? 3 : ctas * (2 * row + other) <= kSmem ? 2 : 0;
}

// Launches kernel FN with programmatic stream serialisation: the launch overlaps the end of the kernel before it, so
// it waits (pdl_wait) before it reads or writes.
template <auto FN, typename... Args>
inline int launch_ahead(dim3 grid, int threads, int bytes, cudaStream_t s, Args... args) {
    if (bytes > 0) {
        static std::atomic<bool> ready[kMaxDevices];  // the kernel may have `bytes` of shared memory there
        int dev;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 4;
        if (!ready[dev].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return 4;
            ready[dev].store(true, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, FN, args...) == cudaSuccess ? 0 : 4;
}

}  // namespace gn
}  // namespace falcon
