// Root-mean-square norm of a token's d channels with the residual's addition, forward and backward.
//   h = x + residual (rounded to their type, as it is stored),  r = 1 / sqrt(mean h^2 + eps),  y = weight h r,
//   y in their type or, with s = max |y| / 448, as e4m3 values y / s;
//   p = weight dy,  dx = r (p - h r^2 mean(p h)) + dh,  dweight = sum over tokens of dy h r.
// A token's channels stay in registers from their one read to their one write, in the lanes of one warp (up to 1024
// of bf16) or of all warps of a CTA; the next token's are on their way meanwhile. Bound by the bytes.

#include <cuda_fp8.h>

#include "falcon.h"
#include "falcon_launch.h"
#include "falcon_rms.h"
#include "falcon_seq.cuh"
#include "sm103_ptx.cuh"

namespace falcon {
namespace rms {
namespace {

using namespace seq;

constexpr int kWarps = 4;       // of a CTA whose warps have a token each
constexpr int kMost = 512;      // threads of a CTA that has one token
constexpr int kSms = 152;
constexpr int kSums = kWarps * 4096;  // bytes: a warp's sums of a token's channels, 1024 at most

struct Args {
    RmsArgs a;
    long long rows;
    bool weight16;  // the weights start on 16 bytes
};

// The place of a token, and whether it lies inside its sequence.
struct Row {
    long long b;
    int t;
    bool live;
};
__device__ __forceinline__ Row row_of(const RmsArgs& a, long long row) {
    Row r;
    const unsigned q = (unsigned)row / (unsigned)a.T;
    r.b = q;
    r.t = (int)((unsigned)row - q * (unsigned)a.T);
    r.live = !a.lengths || r.t < a.lengths[q];
    return r;
}
__device__ __forceinline__ long long offset(const RowView& v, const Row& r) { return r.b * v.sb + r.t * v.st; }

// NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sums (or, with MAX, maxima) over the lanes that hold a token: every one gets the same bits. `slot` of shared memory
// is left alone until the next call but one.
template <bool MULTI, bool MAX, int N>
__device__ __forceinline__ void reduce(float (&v)[N], float* slot) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float o = __shfl_xor_sync(0xffffffffu, v[i], m);
            v[i] = MAX ? max_nan(v[i], o) : v[i] + o;
        }
    if (!MULTI) return;
    const int w = threadIdx.x >> 5, n = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) slot[i * 32 + w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = slot[i * 32];
        for (int k = 1; k < n; ++k) s = MAX ? max_nan(s, slot[i * 32 + k]) : s + slot[i * 32 + k];
        v[i] = s;
    }
}

template <typename E, int W, int N>
struct Line {
    Pack<E, W> v[N];
    // Vectors first, first + step, ... of the d / W of a token at p; nothing is read of one that is not live.
    __device__ __forceinline__ void fetch(const void* p, long long off, int first, int step, int count, bool live) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (live && first + i * step < count) v[i] = load<E, W>(p, off + (long long)(first + i * step) * W);
            else zero(v[i]);
        }
    }
};

template <int W>
__device__ __forceinline__ void store8(uint8_t* p, const float* v) {
    if (W == 1) {
        *p = __nv_cvt_float_to_fp8(v[0], __NV_SATFINITE, __NV_E4M3);
    } else {
        uint32_t u[W / 4 > 0 ? W / 4 : 1];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
            u[i] = lo | hi << 16;
        }
        if (W == 8) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[W / 4 - 1]);
        else *reinterpret_cast<uint32_t*>(p) = u[0];
    }
}

template <typename E, int W, int N, bool MULTI, bool EIGHT>
__global__ void __launch_bounds__(MULTI ? kMost : 32 * kWarps) rms_fwd(const Args g) {
    __shared__ float slots[2][2][32];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const RmsArgs& a = g.a;
    const int step = MULTI ? blockDim.x : 32, first = MULTI ? threadIdx.x : threadIdx.x & 31;
    const int count = a.d / W;
    const long long stride = MULTI ? gridDim.x : (long long)gridDim.x * kWarps;
    long long row = MULTI ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= g.rows) return;
    float wt[N * W];
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const int c = (first + i * step) * W + e;
            wt[i * W + e] = a.weight && c < a.d ? a.weight[c] : 1.f;
        }
    Line<E, W, N> x, r;
    Row at = row_of(a, row);
    x.fetch(a.x.p, offset(a.x, at), first, step, count, at.live);
    if (a.residual.p) r.fetch(a.residual.p, offset(a.residual, at), first, step, count, at.live);
    const float inv_d = 1.f / a.d;
    for (int turn = 0;; turn ^= 1) {
        float h[N * W], s[1] = {0.f};
        if (a.residual.p) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
#pragma unroll
                for (int e = 0; e < W; ++e) h[i * W + e] = elem(x.v[i], e) + elem(r.v[i], e);
                pack(x.v[i], h + i * W);  // as it is stored is how it is normalised
                if (a.h.p && first + i * step < count)
                    store<E, W>(a.h.p, offset(a.h, at) + (long long)(first + i * step) * W, x.v[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                h[i * W + e] = elem(x.v[i], e);
                s[0] = fmaf(h[i * W + e], h[i * W + e], s[0]);
            }
        const Row now = at;
        const long long here = row;
        row += stride;
        if (row < g.rows) {
            at = row_of(a, row);
            x.fetch(a.x.p, offset(a.x, at), first, step, count, at.live);
            if (a.residual.p) r.fetch(a.residual.p, offset(a.residual, at), first, step, count, at.live);
        }
        reduce<MULTI, false>(s, slots[turn][0]);
        const float rstd = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps));
        float top[1] = {0.f};
#pragma unroll
        for (int i = 0; i < N * W; ++i) {
            h[i] = h[i] * rstd * wt[i];
            if (EIGHT) top[0] = max_nan(top[0], fabsf(h[i]));
        }
        const long long oy = offset(a.y, now);
        if (!EIGHT) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (first + i * step >= count) continue;
                Pack<E, W> o;
                if (now.live) pack(o, h + i * W);
                else zero(o);
                store<E, W>(a.y.p, oy + (long long)(first + i * step) * W, o);
            }
        } else {
            reduce<MULTI, true>(top, slots[turn][1]);
            const float near = top[0] * (1.f / 448.f);
            const float exact = near < 3.4e38f ? fmaf(fmaf(-near, 448.f, top[0]), 1.f / 448.f, near) : near;  // its last bit
            const float scale = now.live ? exact : 0.f;
            if (first == 0) a.scales[here] = scale;
            // The quotient, correctly rounded: by 1 / scale and what is left of the value (73 us for 16384 x 4096, 89 by division)
            // where that is exact, 2^-48 of values down to scale / 1024 being no less than 2^-149; else by division. A row of
            // zeros stays 0.
            const bool plain = !(scale >= 1e-27f && scale < 3.4e38f);
            const float inv = plain ? 0.f : 1.f / scale;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (first + i * step >= count) continue;
                float q[W];
                const float* v = h + i * W;
                if (plain) {
#pragma unroll
                    for (int e = 0; e < W; ++e) q[e] = !now.live || scale == 0.f ? 0.f : v[e] / scale;
                } else if (W == 1) {
                    q[0] = v[0] * inv;
                    q[0] = fmaf(fmaf(-q[0], scale, v[0]), inv, q[0]);
                } else {
#pragma unroll
                    for (int e = 0; e + 1 < W; e += 2) {
                        const float2 x2 = pair(v[e], v[e + 1]), f = pair(inv, inv), near2 = mul2(x2, f);
                        const float2 r2 = fma2(fma2(near2, pair(-scale, -scale), x2), f, near2);
                        q[e] = r2.x, q[e + 1] = r2.y;
                    }
                }
                store8<W>(static_cast<uint8_t*>(a.y.p) + oy + (long long)(first + i * step) * W, q);
            }
        }
        if (row >= g.rows) return;
    }
}

// dweight's sums: a lane adds up its own channels over the CTA's tokens, then the CTA's warps in their order, and
// rms_sum the CTAs in theirs. What a lane holds (32 channels at most where a warp has a token) leaves room for 16 warps an
// SM, whose loads cover one another: fetching a token ahead takes the registers of half of them.
template <typename E, int W, int N, bool MULTI>
__global__ void __launch_bounds__(MULTI ? kMost : 32 * kWarps, MULTI ? 1 : 4) rms_bwd(const Args g) {
    extern __shared__ __align__(16) float sums[];
    __shared__ float slots[2][2 * 32];
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const RmsArgs& a = g.a;
    const int step = MULTI ? blockDim.x : 32, first = MULTI ? threadIdx.x : threadIdx.x & 31;
    const int count = a.d / W;
    const long long stride = MULTI ? gridDim.x : (long long)gridDim.x * kWarps;
    float acc[N * W];
#pragma unroll
    for (int i = 0; i < N * W; ++i) acc[i] = 0.f;
    const float inv_d = 1.f / a.d;
    // the weights of vector i, from the first-level cache
    auto weights = [&](int i, float* w) {
        const int c = (first + i * step) * W;
#pragma unroll
        for (int e = 0; e < W; ++e) w[e] = 1.f;
        if (!a.weight || c >= a.d) return;
        if (W % 4 == 0 && g.weight16) {
#pragma unroll
            for (int e = 0; e < W / 4; ++e) {
                const float4 v = *reinterpret_cast<const float4*>(a.weight + c + 4 * e);
                w[4 * e] = v.x, w[4 * e + 1] = v.y, w[4 * e + 2] = v.z, w[4 * e + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = a.weight[c + e];
        }
    };
    int turn = 0;
    for (long long row = MULTI ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); row < g.rows; row += stride, turn ^= 1) {
        const Row at = row_of(a, row);
        Line<E, W, N> x, dy, dh;
        x.fetch(a.x.p, offset(a.x, at), first, step, count, at.live);
        dy.fetch(a.dy.p, offset(a.dy, at), first, step, count, at.live);
        if (a.dh.p) dh.fetch(a.dh.p, offset(a.dh, at), first, step, count, at.live);
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[W];
            weights(i, w);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float h = elem(x.v[i], e), p = elem(dy.v[i], e) * w[e];
                s[0] = fmaf(h, h, s[0]);
                s[1] = fmaf(p, h, s[1]);
            }
        }
        reduce<MULTI, false>(s, slots[turn]);
        const float rstd = 1.f / sqrtf(fmaf(s[0], inv_d, a.eps)), k = rstd * rstd * (s[1] * inv_d);
        const long long o = offset(a.dx, at);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float v[W], w[W];
            weights(i, w);
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float h = elem(x.v[i], e), y = elem(dy.v[i], e);
                if (at.live) acc[i * W + e] = fmaf(y, h * rstd, acc[i * W + e]);
                v[e] = rstd * fmaf(-h, k, y * w[e]);
                if (a.dh.p) v[e] += elem(dh.v[i], e);
                if (!at.live) v[e] = 0.f;
            }
            if (first + i * step >= count) continue;
            Pack<E, W> u;
            pack(u, v);
            store<E, W>(a.dx.p, o + (long long)(first + i * step) * W, u);
        }
    }
    if (!a.ws) return;
    float* to = a.ws + (long long)blockIdx.x * a.d;
    if (!MULTI) {
        float* mine = sums + (threadIdx.x >> 5) * a.d;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const int c = (first + i * step) * W + e;
                if (c < a.d) mine[c] = acc[i * W + e];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += 32 * kWarps) {
            float v = sums[c];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += sums[w * a.d + c];
            to[c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const int c = (first + i * step) * W + e;
                if (c < a.d) to[c] = acc[i * W + e];
            }
    }
}

// A CTA has 32 channels, its warps every 32nd of the sums.
__global__ void __launch_bounds__(1024) rms_sum(const float* part, int splits, int d, float* out) {
    __shared__ float s[32][33];
    ptx::pdl_wait();  // launched while the CTAs whose sums it adds still run
    ptx::pdl_launch_dependents();
    const int l = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + l;
    float v = 0.f;
    if (c < d) {
#pragma unroll 16
        for (int i = w; i < splits; i += 32) v += part[(long long)i * d + c];
    }
    s[l][w] = v;
    __syncthreads();
    v = s[w][l];  // warp w: channel w
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    if (l == 0 && blockIdx.x * 32 + w < d) out[blockIdx.x * 32 + w] = v;
}

// Lanes of a token. A vector is 16 bytes where every access can be one, else an element, and a lane holds N of them: as
// few as keep a token in one warp, or in a CTA's most threads.
bool vec_ok(const RowView& v, int bytes, int es) {
    const long long m = bytes / es;
    return !v.p || (reinterpret_cast<uintptr_t>(v.p) % (uintptr_t)bytes == 0 && v.sb % m == 0 && v.st % m == 0);
}
int lanes_of(int d, int per) { return ((d + per - 1) / per + 31) / 32 * 32; }

// ONE: such tokens may fit a warp.
template <typename E, int W, int N, bool ONE = true>
int fwd(const Args& g, cudaStream_t s) {
    const int lanes = lanes_of(g.a.d, W * N);
    const bool multi = lanes > 32;
    const int threads = multi ? lanes : 32 * kWarps;
    // as many CTAs as are resident at up to 128 registers a thread: each warp goes on to its next token
    const long long most = (long long)kSms * (512 / threads);
    const long long want = multi ? g.rows : (g.rows + kWarps - 1) / kWarps;
    const unsigned grid = (unsigned)(want < most ? want : most);
    if constexpr (ONE) {
        if (!multi) return g.a.eight ? launch_ahead<rms_fwd<E, W, N, false, true>>(grid, threads, 0, s, g)
                                     : launch_ahead<rms_fwd<E, W, N, false, false>>(grid, threads, 0, s, g);
    }
    return g.a.eight ? launch_ahead<rms_fwd<E, W, N, true, true>>(grid, threads, 0, s, g)
                     : launch_ahead<rms_fwd<E, W, N, true, false>>(grid, threads, 0, s, g);
}
template <typename E, int W, int N, bool ONE = true>
int bwd(const Args& g, cudaStream_t s) {
    const int lanes = lanes_of(g.a.d, W * N);
    const unsigned grid = (unsigned)rms_bwd_splits(g.rows, g.a.d, g.a.bf16);
    if constexpr (ONE) {
        if (lanes == 32) return launch_ahead<rms_bwd<E, W, N, false>>(grid, 32 * kWarps, kSums, s, g);
    }
    return launch_ahead<rms_bwd<E, W, N, true>>(grid, lanes, 0, s, g);
}

bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
}  // namespace rms

int rms_bwd_splits(long long rows, int d, int bf16) {
    // as many CTAs as are resident, by the lanes of a token: one warp each, or 2 to 16 (fp32 of 1000 channels, four warps: 45 us
    // with 4 CTAs an SM, 39 with 6)
    const int per_sm = bf16 ? (d <= 2048 ? 4 : 2) : d <= 256 ? 4 : d <= 1024 ? 6 : d <= 2048 ? 3 : 2;
    const long long most = (long long)rms::kSms * per_sm;
    return (int)(rows < most ? rows : most);
}

int launch_rms_fwd(const RmsArgs& a, cudaStream_t s) {
    using namespace rms;
    const int es = a.bf16 ? 2 : 4, w = 16 / es;
    const bool vec = a.d % w == 0 && vec_ok(a.x, 16, es) && vec_ok(a.residual, 16, es) && vec_ok(a.h, 16, es) &&
                     (a.eight ? vec_ok(a.y, w, 1) : vec_ok(a.y, 16, es));
    const Args g = {a, a.B * a.T, al16(a.weight)};
    const bool wide = a.d > kMost * 16;
    if (a.bf16) return vec ? fwd<bf16, 8, 4>(g, s) : wide ? fwd<bf16, 1, 32, false>(g, s) : fwd<bf16, 1, 16>(g, s);
    if (vec) return wide ? fwd<float, 4, 8, false>(g, s) : fwd<float, 4, 4>(g, s);
    return wide ? fwd<float, 1, 32, false>(g, s) : fwd<float, 1, 16>(g, s);
}

int launch_rms_bwd(const RmsArgs& a, cudaStream_t s) {
    using namespace rms;
    const int es = a.bf16 ? 2 : 4, w = 16 / es, d = a.d;
    const bool vec = d % w == 0 && vec_ok(a.x, 16, es) && vec_ok(a.dy, 16, es) && vec_ok(a.dh, 16, es) && vec_ok(a.dx, 16, es);
    const Args g = {a, a.B * a.T, al16(a.weight)};
    const bool mid = d <= kMost * 8, wide = d > kMost * 16;  // 8, 16 or 32 channels a lane, in a CTA's most threads
    int st;
    if (a.bf16 && vec) {
        st = wide ? bwd<bf16, 8, 4, false>(g, s) : d > 1024 || d <= 512 ? bwd<bf16, 8, 2>(g, s) : d <= 768 ? bwd<bf16, 8, 3>(g, s) : bwd<bf16, 8, 4>(g, s);
    } else if (a.bf16) {
        st = mid ? bwd<bf16, 1, 8>(g, s) : wide ? bwd<bf16, 1, 32, false>(g, s) : bwd<bf16, 1, 16, false>(g, s);
    } else if (vec) {
        st = mid ? bwd<float, 4, 2>(g, s) : wide ? bwd<float, 4, 8, false>(g, s) : bwd<float, 4, 4, false>(g, s);
    } else {
        st = mid ? bwd<float, 1, 8>(g, s) : wide ? bwd<float, 1, 32, false>(g, s) : bwd<float, 1, 16, false>(g, s);
    }
    if (!a.ws || st != 0) return st;
    return launch_ahead<rms_sum>((d + 31) / 32, 1024, 0, s, (const float*)a.ws, rms_bwd_splits(g.rows, d, a.bf16), d, a.dweight);
}

}  // namespace falcon
