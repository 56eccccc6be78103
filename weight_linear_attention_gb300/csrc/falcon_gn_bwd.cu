// Group norm of a token's head with an activation and a gate, backward. With xh the normalised row,
// n = w xh + b, dn = dy act'(n) (or dy act(z), dz = dy n act'(z)) and p = dn w:
//   dx = rstd (p - mean(p) - xh mean(p xh)),  dw = sum over rows of dn xh,  db = sum over rows of dn.
//
// Memory bound: 3 (5 with a gate) tensors' bytes per element. A CTA takes rows of one head only, so a
// thread's channels stay the same and it sums dw and db in registers; the CTA adds its threads' sums up
// in shared memory and leaves one partial sum per split of the rows, which a second, small kernel adds
// in the order of the splits. Every order depends on the sizes alone: no atomics.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "falcon_gn.cuh"

namespace falcon {
namespace {

using namespace gn;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
#ifndef GNB_U
#define GNB_U 2
#endif
#ifndef GNB_PER
#define GNB_PER 4
#endif

struct BwdParams {
    const void* x;
    const void* z;
    const void* dy;
    void* dx;
    void* dz;
    const float* w;
    const float* b;
    const int32_t* lengths;
    float* ws;
    long long xb, xh, xt, zb, zh, zt, yb, yh, yt, dxb, dxh, dxt, dzb, dzh, dzt;
    uint32_t rows;  // B T
    FastDiv tokens;
    int T, d, H, act;
    float inv_d, eps;
};

template <int P>
__device__ __forceinline__ void slope_all(int a, const float2 (&v)[P], float2 (&f)[P], float2 (&df)[P]) {
    switch (a) {  // the same for the whole grid
        case kActNone:
#pragma unroll
            for (int i = 0; i < P; ++i) act_slope<kActNone>(v[i], f[i], df[i]);
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < P; ++i) act_slope<kActSilu>(v[i], f[i], df[i]);
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < P; ++i) act_slope<kActGelu>(v[i], f[i], df[i]);
            break;
        default:
#pragma unroll
            for (int i = 0; i < P; ++i) act_slope<kActSigmoid>(v[i], f[i], df[i]);
    }
}

template <typename E, int VW, int LPR, int NCH, bool GATED, bool FULL>
__global__ void __launch_bounds__(kThreads) gn_bwd_kernel(const __grid_constant__ BwdParams p) {
    using Q = Row<VW, LPR, NCH, FULL>;
    constexpr int P = Q::P;
    constexpr int G = kThreads / LPR;  // rows side by side
    constexpr int U = NCH == 1 ? GNB_U : 1;
    __shared__ float part[kWarps][LPR * NCH * VW];
    const Q q = {(int)threadIdx.x % LPR, p.d};
    const uint32_t grp = threadIdx.x / LPR, h = blockIdx.y;
    float2 w[P], bias[P], aw[P], ab[P];
    q.template params<1>(p.w ? p.w + (long long)h * p.d : nullptr, 1.f, w);
    q.template params<1>(p.b ? p.b + (long long)h * p.d : nullptr, 0.f, bias);
#pragma unroll
    for (int i = 0; i < P; ++i) aw[i] = ab[i] = pair(0.f, 0.f);
    const E* x0 = static_cast<const E*>(p.x) + h * p.xh + q.chan(0);
    const E* z0 = static_cast<const E*>(p.z) + (GATED ? h * p.zh + q.chan(0) : 0);
    const E* d0 = static_cast<const E*>(p.dy) + h * p.yh + q.chan(0);
    E* ox = static_cast<E*>(p.dx) + h * p.dxh + q.chan(0);
    E* oz = static_cast<E*>(p.dz) + (GATED ? h * p.dzh + q.chan(0) : 0);
    const uint32_t step = gridDim.x * G * U;
    for (uint32_t r0 = blockIdx.x * G * U; r0 < p.rows; r0 += step) {  // the same count for a whole CTA
        Pack<E, VW> px[U][NCH], pz[U][GATED ? NCH : 1], pd[U][NCH];
        uint32_t b[U], t[U];
        bool have[U], in[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t r = r0 + u * G + grp;
            have[u] = r < p.rows;
            b[u] = div(have[u] ? r : 0, p.tokens);
            t[u] = (have[u] ? r : 0) - b[u] * p.tokens.d;
            in[u] = have[u] && (!p.lengths || (int)t[u] < p.lengths[b[u]]);
#pragma unroll
            for (int k = 0; k < NCH; ++k) {
                zero(px[u][k]);
                zero(pd[u][k]);
                if (GATED) zero(pz[u][k]);
                if (in[u] && q.live(k)) {
                    px[u][k] = load<E, VW>(x0, b[u] * p.xb + t[u] * p.xt + LPR * k * VW);
                    pd[u][k] = load<E, VW>(d0, b[u] * p.yb + t[u] * p.yt + LPR * k * VW);
                    if (GATED) pz[u][k] = load<E, VW>(z0, b[u] * p.zb + t[u] * p.zt + LPR * k * VW);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 x[P], dn[P], f[P], df[P];
            q.get(px[u], x);
            q.get(pd[u], dn);
            const float rstd = q.normalise(x, p.inv_d, p.eps);
            if constexpr (GATED) {
                float2 z[P];
                q.get(pz[u], z);
                slope_all<P>(p.act, z, f, df);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    df[i] = ptx::mul2(ptx::mul2(dn[i], ptx::fma2(x[i], w[i], bias[i])), df[i]);  // dz
                    dn[i] = ptx::mul2(dn[i], f[i]);
                }
#pragma unroll
                for (int k = 0; k < NCH; ++k)
                    if (have[u] && q.live(k)) {
                        Pack<E, VW> po = q.template put<E>(df, k);
                        if (!in[u]) zero(po);
                        store(oz, b[u] * p.dzb + t[u] * p.dzt + LPR * k * VW, po);
                    }
            } else {
                float2 n[P];
#pragma unroll
                for (int i = 0; i < P; ++i) n[i] = ptx::fma2(x[i], w[i], bias[i]);
                slope_all<P>(p.act, n, f, df);
#pragma unroll
                for (int i = 0; i < P; ++i) dn[i] = ptx::mul2(dn[i], df[i]);
            }
            // rows behind the end were read as zeros: dy = 0, and no activation's slope at 0 is infinite
            float2 s1 = pair(0.f, 0.f), s2 = s1;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                aw[i] = ptx::fma2(dn[i], x[i], aw[i]);
                ab[i] = ptx::add2(ab[i], dn[i]);
                dn[i] = ptx::mul2(dn[i], w[i]);  // p; 0 behind d
                s1 = ptx::add2(s1, dn[i]);
                s2 = ptx::fma2(dn[i], x[i], s2);
            }
            const float m1 = -row_sum<LPR>(s1) * p.inv_d, m2 = -row_sum<LPR>(s2) * p.inv_d;
#pragma unroll
            for (int i = 0; i < P; ++i)
                dn[i] = ptx::mul2(ptx::fma2(x[i], pair(m2, m2), ptx::add2(dn[i], pair(m1, m1))), pair(rstd, rstd));
#pragma unroll
            for (int k = 0; k < NCH; ++k)
                if (have[u] && q.live(k)) {
                    Pack<E, VW> po = q.template put<E>(dn, k);
                    if (!in[u]) zero(po);
                    store(ox, b[u] * p.dxb + t[u] * p.dxt + LPR * k * VW, po);
                }
        }
    }
    if (!p.ws) return;
    // the warp's groups, then the CTA's warps; first dw, then db
    float* to = p.ws + (long long)blockIdx.x * 2 * p.H * p.d + (long long)h * p.d;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int e = 0; e < 2 * P; ++e) {
            const float2 a = which ? ab[e / 2] : aw[e / 2];
            float v = e % 2 ? a.y : a.x;
#pragma unroll
            for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (threadIdx.x % 32 < LPR) part[threadIdx.x / 32][q.chan(e / VW) + e % VW] = v;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.d; e += kThreads) {
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) v += part[i][e];
            to[(long long)which * p.H * p.d + e] = v;
        }
        __syncthreads();
    }
}

constexpr int kSumChannels = 32, kSumSlices = 8;

// out[c] = the sum of ws[s][c] over the splits s, for the channels of dw (c < n) and of db.
__global__ void __launch_bounds__(kSumChannels* kSumSlices)
    gn_sum_kernel(const float* __restrict__ ws, int splits, long long n, float* __restrict__ dw,
                  float* __restrict__ db) {
    __shared__ float part[kSumSlices][kSumChannels];
    const int lane = threadIdx.x % kSumChannels, slice = threadIdx.x / kSumChannels;
    const long long c = (long long)blockIdx.x * kSumChannels + lane;
    float v = 0.f;
    if (c < 2 * n)
        for (int s = slice; s < splits; s += kSumSlices) v += ws[(long long)s * 2 * n + c];
    part[slice][lane] = v;
    __syncthreads();
    if (slice == 0 && c < 2 * n) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < kSumSlices; ++i) v += part[i][lane];
        if (c < n) {
            if (dw) dw[c] = v;
        } else if (db) {
            db[c - n] = v;
        }
    }
}

template <typename E, int VW, int LPR, int NCH>
int launch(const BwdParams& p, int splits, cudaStream_t s) {
    const dim3 grid((unsigned)splits, (unsigned)p.H);
    const bool full = p.d == VW * LPR * NCH;
    if (p.z && full) gn_bwd_kernel<E, VW, LPR, NCH, true, true><<<grid, kThreads, 0, s>>>(p);
    else if (p.z) gn_bwd_kernel<E, VW, LPR, NCH, true, false><<<grid, kThreads, 0, s>>>(p);
    else if (full) gn_bwd_kernel<E, VW, LPR, NCH, false, true><<<grid, kThreads, 0, s>>>(p);
    else gn_bwd_kernel<E, VW, LPR, NCH, false, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : 4;
}

template <typename E, int VW>
int by_width(const BwdParams& p, int splits, cudaStream_t s) {
    const int nv = (p.d + VW - 1) / VW;
    if constexpr (VW > 1) {
        if (nv <= 4) return launch<E, VW, 4, 1>(p, splits, s);
        if (nv <= 8) return launch<E, VW, 8, 1>(p, splits, s);
        if (nv <= 16) return launch<E, VW, 16, 1>(p, splits, s);
        if (nv <= 32) return launch<E, VW, 32, 1>(p, splits, s);
    }
    if (nv <= 64) return launch<E, VW, 32, 2>(p, splits, s);
    if (nv <= 128) return launch<E, VW, 32, 4>(p, splits, s);
    if constexpr (VW * 256 <= kGnMaxD)
        if (nv <= 256) return launch<E, VW, 32, 8>(p, splits, s);
    if constexpr (VW == 1) return launch<E, VW, 32, 32>(p, splits, s);
    return 2;
}

}  // namespace

// As many CTAs as run at once (4 per SM), over the heads; no more than there are rows for.
int gn_bwd_splits(const SeqSizes& n) {
    const long long rows = n.B * n.T;
    long long s = (152 * GNB_PER + n.H - 1) / n.H;
    const long long most = (rows + 31) / 32;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

int launch_gn_bwd(const GnArgs& a, cudaStream_t s) {
    if (a.n.H > 65535 || (unsigned __int128)a.n.B * a.n.T >= ((unsigned __int128)1 << 31) - 65536) return 2;
    BwdParams p = {};
    p.x = a.x.p, p.z = a.z.p, p.dy = a.dy.p, p.dx = a.dx.p, p.dz = a.dz.p;
    p.w = a.w, p.b = a.b, p.lengths = a.lengths, p.ws = a.ws;
    p.xb = a.x.sb, p.xh = a.x.sh, p.xt = a.x.st;
    p.zb = a.z.sb, p.zh = a.z.sh, p.zt = a.z.st;
    p.yb = a.dy.sb, p.yh = a.dy.sh, p.yt = a.dy.st;
    p.dxb = a.dx.sb, p.dxh = a.dx.sh, p.dxt = a.dx.st;
    p.dzb = a.dz.sb, p.dzh = a.dz.sh, p.dzt = a.dz.st;
    p.rows = (uint32_t)(a.n.B * a.n.T);
    p.tokens = fast_div((uint32_t)a.n.T);
    p.T = a.n.T, p.d = a.n.d, p.H = (int)a.n.H, p.act = a.act;
    p.inv_d = 1.f / a.n.d, p.eps = a.eps;
    const int splits = gn_bwd_splits(a.n);
    const int es = a.n.bf16 ? 2 : 4;
    const bool vec = a.n.d % (16 / es) == 0 && seq_vec_ok(a.x, es, 16) && seq_vec_ok(a.z, es, 16) &&
                     seq_vec_ok(a.dy, es, 16) && seq_vec_ok(a.dx, es, 16) && seq_vec_ok(a.dz, es, 16);
    int st;
    if (a.n.bf16) st = vec ? by_width<bf16, 8>(p, splits, s) : by_width<bf16, 1>(p, splits, s);
    else st = vec ? by_width<float, 4>(p, splits, s) : by_width<float, 1>(p, splits, s);
    if (st != 0 || !a.ws) return st;
    const long long n = a.n.H * a.n.d;
    gn_sum_kernel<<<(unsigned)((2 * n + kSumChannels - 1) / kSumChannels), kSumChannels * kSumSlices, 0, s>>>(
        a.ws, splits, n, a.dw, a.db);
    return cudaGetLastError() == cudaSuccess ? 0 : 4;
}

}  // namespace falcon
