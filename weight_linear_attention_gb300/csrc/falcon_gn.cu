// Group norm of a token's head with an activation and a gate, forward:
// n = w (x - mean) / sqrt(var + eps) + b over the d channels of one (batch, head, token);
// y = act(n), or n act(z).
//
// A memory-bound transposition with arithmetic on the way: 2 (3 with a gate) tensors' bytes per element.
// LPR lanes hold a row in registers (16 bytes a lane), so the row is read once and the variance is that
// of the centred values; a thread takes UNR tokens of one head, so that weight and bias are fetched once
// for them and UNR (2 UNR) vector loads are in flight. Row blocks go over the heads first where y's heads
// are its closer axis (the projection's layout), else over the tokens, so that neighbouring CTAs write
// neighbouring memory.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "falcon_gn.cuh"

namespace falcon {
namespace {

using namespace gn;

constexpr int kThreads = 256;
#ifndef GN_UNR
#define GN_UNR (NCH == 1 ? 2 : 1)
#endif

struct FwdParams {
    const void* x;
    const void* z;
    void* y;
    const float* w;
    const float* b;
    const int32_t* lengths;
    long long xb, xh, xt, zb, zh, zt, yb, yh, yt;
    uint32_t total;      // row blocks
    FastDiv fast, slow;  // the sizes of the block index's fastest axis and of the next
    int heads_first;
    int T, d, act;
    float inv_d, eps;
};

template <int P>
__device__ __forceinline__ void act_all(int a, const float2 (&v)[P], float2 (&f)[P]) {
    switch (a) {  // the same for the whole grid
        case kActNone:
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = act<kActNone>(v[i]);
            break;
        case kActSilu:
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = act<kActSilu>(v[i]);
            break;
        case kActGelu:
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = act<kActGelu>(v[i]);
            break;
        default:
#pragma unroll
            for (int i = 0; i < P; ++i) f[i] = act<kActSigmoid>(v[i]);
    }
}

template <typename E, int VW, int LPR, int NCH, int UNR, bool GATED, bool FULL>
__global__ void __launch_bounds__(kThreads) gn_fwd_kernel(const __grid_constant__ FwdParams p) {
    using Q = Row<VW, LPR, NCH, FULL>;
    const Q q = {(int)threadIdx.x % LPR, p.d};
    const uint32_t i = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
    const bool have = i < p.total;  // a group without rows still takes part in the shuffles
    const uint32_t blk = have ? i : p.total - 1;
    const uint32_t q1 = div(blk, p.fast), f0 = blk - q1 * p.fast.d;
    const uint32_t q2 = div(q1, p.slow), f1 = q1 - q2 * p.slow.d;
    const long long b = q2;
    const uint32_t h = p.heads_first ? f0 : f1;
    const int t0 = (int)((p.heads_first ? f1 : f0) * UNR);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int c0 = q.chan(0);
    const E* x0 = static_cast<const E*>(p.x) + b * p.xb + h * p.xh + t0 * p.xt + c0;
    const E* z0 = static_cast<const E*>(p.z) + (GATED ? b * p.zb + h * p.zh + t0 * p.zt + c0 : 0);
    E* y0 = static_cast<E*>(p.y) + b * p.yb + h * p.yh + t0 * p.yt + c0;

    Pack<E, VW> px[UNR][NCH], pz[UNR][GATED ? NCH : 1];
#pragma unroll
    for (int u = 0; u < UNR; ++u)
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
            zero(px[u][k]);
            if (GATED) zero(pz[u][k]);
            if (have && t0 + u < len && q.live(k)) {
                px[u][k] = load<E, VW>(x0, u * p.xt + LPR * k * VW);
                if (GATED) pz[u][k] = load<E, VW>(z0, u * p.zt + LPR * k * VW);
            }
        }
    float2 w[Q::P], bias[Q::P];
    constexpr int FW = VW < 4 ? VW : 4;
    q.template params<FW>(p.w ? p.w + (long long)h * p.d : nullptr, 1.f, w);
    q.template params<FW>(p.b ? p.b + (long long)h * p.d : nullptr, 0.f, bias);
#pragma unroll
    for (int u = 0; u < UNR; ++u) {
        float2 x[Q::P], f[Q::P];
        q.get(px[u], x);
        q.normalise(x, p.inv_d, p.eps);
#pragma unroll
        for (int j = 0; j < Q::P; ++j) x[j] = ptx::fma2(x[j], w[j], bias[j]);
        if constexpr (GATED) {
            float2 z[Q::P];
            q.get(pz[u], z);
            act_all<Q::P>(p.act, z, f);
#pragma unroll
            for (int j = 0; j < Q::P; ++j) f[j] = ptx::mul2(f[j], x[j]);
        } else {
            act_all<Q::P>(p.act, x, f);
        }
        const int t = t0 + u;
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
            if (!have || t >= p.T || !q.live(k)) continue;
            Pack<E, VW> po = q.template put<E>(f, k);
            if (t >= len) zero(po);
            store(y0, u * p.yt + LPR * k * VW, po);
        }
    }
}

template <typename E, int VW, int LPR, int NCH>
int launch(FwdParams p, long long B, long long H, cudaStream_t s) {
    constexpr int UNR = GN_UNR;
    const long long TB = (p.T + UNR - 1) / UNR;
    const unsigned __int128 total = (unsigned __int128)B * H * TB;
    if (total >= ((unsigned __int128)1 << 31)) return 2;
    p.total = (uint32_t)total;
    p.heads_first = p.yh < p.yt || p.T == 1;
    p.fast = fast_div((uint32_t)(p.heads_first ? H : TB));
    p.slow = fast_div((uint32_t)(p.heads_first ? TB : H));
    constexpr int per = kThreads / LPR;
    const unsigned grid = (p.total + per - 1) / per;
    const bool full = p.d == VW * LPR * NCH;
    if (p.z && full) gn_fwd_kernel<E, VW, LPR, NCH, UNR, true, true><<<grid, kThreads, 0, s>>>(p);
    else if (p.z) gn_fwd_kernel<E, VW, LPR, NCH, UNR, true, false><<<grid, kThreads, 0, s>>>(p);
    else if (full) gn_fwd_kernel<E, VW, LPR, NCH, UNR, false, true><<<grid, kThreads, 0, s>>>(p);
    else gn_fwd_kernel<E, VW, LPR, NCH, UNR, false, false><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : 4;
}

template <typename E, int VW>
int by_width(const FwdParams& p, long long B, long long H, cudaStream_t s) {
    const int nv = (p.d + VW - 1) / VW;
    if constexpr (VW > 1) {
        if (nv <= 4) return launch<E, VW, 4, 1>(p, B, H, s);
        if (nv <= 8) return launch<E, VW, 8, 1>(p, B, H, s);
        if (nv <= 16) return launch<E, VW, 16, 1>(p, B, H, s);
        if (nv <= 32) return launch<E, VW, 32, 1>(p, B, H, s);
    }
    if (nv <= 64) return launch<E, VW, 32, 2>(p, B, H, s);
    if (nv <= 128) return launch<E, VW, 32, 4>(p, B, H, s);
    if constexpr (VW * 256 <= kGnMaxD)
        if (nv <= 256) return launch<E, VW, 32, 8>(p, B, H, s);
    if constexpr (VW == 1) return launch<E, VW, 32, 32>(p, B, H, s);
    return 2;
}

}  // namespace

int launch_gn_fwd(const GnArgs& a, cudaStream_t s) {
    FwdParams p = {};
    p.x = a.x.p, p.z = a.z.p, p.y = a.y.p;
    p.w = a.w, p.b = a.b, p.lengths = a.lengths;
    p.xb = a.x.sb, p.xh = a.x.sh, p.xt = a.x.st;
    p.zb = a.z.sb, p.zh = a.z.sh, p.zt = a.z.st;
    p.yb = a.y.sb, p.yh = a.y.sh, p.yt = a.y.st;
    p.T = a.n.T, p.d = a.n.d, p.act = a.act;
    p.inv_d = 1.f / a.n.d, p.eps = a.eps;
    long long B = a.n.B;
    if (p.T == 1 && !p.lengths && B < (1LL << 30)) {  // single tokens: the batch takes the tokens' place
        p.T = (int)B, B = 1;
        p.xt = p.xb, p.zt = p.zb, p.yt = p.yb;
    }
    const int es = a.n.bf16 ? 2 : 4;
    const bool vec = a.n.d % (16 / es) == 0 && seq_vec_ok(a.x, es, 16) && seq_vec_ok(a.z, es, 16) &&
                     seq_vec_ok(a.y, es, 16) && reinterpret_cast<uintptr_t>(a.w) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.b) % 16 == 0;
    if (a.n.bf16) return vec ? by_width<bf16, 8>(p, B, a.n.H, s) : by_width<bf16, 1>(p, B, a.n.H, s);
    return vec ? by_width<float, 4>(p, B, a.n.H, s) : by_width<float, 1>(p, B, a.n.H, s);
}

}  // namespace falcon
