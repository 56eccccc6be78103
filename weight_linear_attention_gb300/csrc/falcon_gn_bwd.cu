// Group norm of a token's head with an activation and a gate, backward. With xh the normalised row,
// n = w xh + b, dn = dy act'(n) (or dy act(z), dz = dy n act'(z)) and p = dn w:
//   dx = rstd (p - mean(p) - xh mean(p xh)),  dw = sum over rows of dn xh,  db = sum over rows of dn.
//
// Memory bound: 3 (5 with a gate) tensors' bytes per element. A CTA takes rows of one head only, so a
// thread's channels stay the same and it sums dw and db in registers; the CTA adds its threads' sums up
// in shared memory and leaves one partial sum per split of the rows, which a second, small kernel adds
// in the order of the splits. Every order depends on sizes and alignment alone: no atomics.
//
// What bounds it: memory ([16,16,4096,64] bf16 with a SiLU gate: 104 us, 95 % of the copy rate; [4,12,8192,64] fp32
// with a gate 82 us, 91 %); at [8,12,1024,64] bf16 (14.9 us with the sums' kernel, 62 %) filling, emptying and the sums.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "falcon_gn.cuh"
#include "sm103_ptx.cuh"

namespace falcon {
namespace {

using namespace gn;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

enum { kX, kZ, kDy, kDx, kDz };

struct BwdParams {
    Tensors<5> s;
    const float* w;
    const float* b;
    const int32_t* lengths;
    float* ws;
    uint32_t rows;  // B T
    int d, H, act;
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

// CTAs that an SM is given: what the registers of the row's width allow.
template <int VW, int NCH>
constexpr int kPerSm = NCH * VW <= 4 ? 3 : NCH * VW <= 8 ? 2 : 1;

// Bytes of a row of the CTA's groups, and the rows that its ring holds (0: registers). The ring keeps twice the bytes
// on their way that the registers have room for: [16,16,4096,64] bf16 104 instead of 128 us, [8,12,1024,64] 14.9 instead
// of 17.1. fp32 has as many on their way in registers up to 16 elements a lane ([4,12,8192,64] 82 us, with a ring 87).
template <typename E, int VW, int NCH, bool GATED>
constexpr int kRow = (GATED ? 3 : 2) * NCH * VW * (int)sizeof(E) * kThreads;
template <typename E, int VW, int LPR, int NCH, bool GATED>
constexpr int kRing = VW == 1 || (sizeof(E) == 4 && NCH * VW < 16)
                          ? 0
                          : depth(kRow<E, VW, NCH, GATED>, kPerSm<VW, NCH>, kWarps* LPR* NCH* VW * (int)sizeof(float));

template <typename E, int VW, int LPR, int NCH, bool GATED, bool FULL>
__global__ void __launch_bounds__(kThreads, kPerSm<VW, NCH>) gn_bwd_kernel(const __grid_constant__ BwdParams p) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    using Q = Row<VW, LPR, NCH, FULL>;
    constexpr int P = Q::P;
    constexpr int G = kThreads / LPR;  // rows side by side
    constexpr bool kHeld = NCH * VW <= 24;  // weight and bias stay in registers, else they come from the L1 cache
    using V = Pack<E, VW>;
    constexpr int CB = LPR * VW * sizeof(E), D = kRing<E, VW, LPR, NCH, GATED>;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float part[kWarps][LPR * NCH * VW];
    const Q q = {(int)threadIdx.x % LPR, p.d};
    const uint32_t h = blockIdx.y, i0 = blockIdx.x * G + threadIdx.x / LPR;
    Rows<E, VW, LPR, NCH, FULL, GATED, 3, 5, kThreads, D, NCH * VW * sizeof(E) <= 64> row;
    row.start(q, p.s, p.lengths, i0, h, ring);
    constexpr int FW = VW < 4 ? VW : 4;
    float2 w[P], bias[P], aw[P], ab[P];
    auto params = [&] {
        q.template params<FW>(p.w ? p.w + (long long)h * p.d : nullptr, 1.f, w);
        q.template params<FW>(p.b ? p.b + (long long)h * p.d : nullptr, 0.f, bias);
    };
    if (kHeld) params();
#pragma unroll
    for (int i = 0; i < P; ++i) aw[i] = ab[i] = pair(0.f, 0.f);
    // the same number of turns for a whole CTA; the next row's loads are on their way while this one is worked on
    for (uint32_t r = blockIdx.x * G; r < p.rows; r += p.s.by) {
        float2 x[P], dn[P], f[P], df[P], z[GATED ? P : 1];
        row.wait(q, p.s, p.lengths);
        row.get(q, kX, x);
        row.get(q, kDy, dn);
        if constexpr (GATED) row.get(q, kZ, z);
        const bool mine = row.mine, in = row.in;
        char *const to_x = row.out[0], *const to_z = row.out[1];
        if (D > 0 || r + p.s.by < p.rows) row.next(q, p.s, p.lengths);
        const float rstd = q.normalise(x, p.inv_d, p.eps);
        if (!kHeld) params();
        if constexpr (GATED) {
            slope_all<P>(p.act, z, f, df);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                df[i] = mul2(mul2(dn[i], fma2(x[i], w[i], bias[i])), df[i]);  // dz
                dn[i] = mul2(dn[i], f[i]);
            }
#pragma unroll
            for (int k = 0; k < NCH; ++k)
                if (mine && q.live(k)) {
                    V po;
                    if (in) po = q.template put<E>(df, k);
                    else zero(po);
                    *reinterpret_cast<V*>(to_z + k * CB) = po;
                }
        } else {
            float2 n[P];
#pragma unroll
            for (int i = 0; i < P; ++i) n[i] = fma2(x[i], w[i], bias[i]);
            slope_all<P>(p.act, n, f, df);
#pragma unroll
            for (int i = 0; i < P; ++i) dn[i] = mul2(dn[i], df[i]);
        }
        float2 s1 = pair(0.f, 0.f), s2 = s1;
        if (in) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                aw[i] = fma2(dn[i], x[i], aw[i]);
                ab[i] = add2(ab[i], dn[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            dn[i] = mul2(dn[i], w[i]);  // p; 0 behind d
            s1 = add2(s1, dn[i]);
            s2 = fma2(dn[i], x[i], s2);
        }
        const float m1 = -row_sum<LPR>(s1) * p.inv_d, m2 = -row_sum<LPR>(s2) * p.inv_d;
#pragma unroll
        for (int i = 0; i < P; ++i)
            dn[i] = mul2(fma2(x[i], pair(m2, m2), add2(dn[i], pair(m1, m1))), pair(rstd, rstd));
#pragma unroll
        for (int k = 0; k < NCH; ++k)
            if (mine && q.live(k)) {
                V po;
                if (in) po = q.template put<E>(dn, k);
                else zero(po);
                *reinterpret_cast<V*>(to_x + k * CB) = po;
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
    ptx::pdl_wait();  // launched while the CTAs whose sums it adds still run
    ptx::pdl_launch_dependents();
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

template <typename E, int VW, int LPR, int NCH, bool GATED, bool FULL>
int run(const BwdParams& p, dim3 grid, cudaStream_t s) {
    constexpr int kBytes = kRing<E, VW, LPR, NCH, GATED> * kRow<E, VW, NCH, GATED>;
    return launch_ahead<gn_bwd_kernel<E, VW, LPR, NCH, GATED, FULL>>(grid, kThreads, kBytes, s, p);
}

// Launches the row's width with `splits` (as many as the workspace has room for), or fewer if fewer CTAs run at once.
template <typename E, int VW, int LPR, int NCH>
int launch(BwdParams p, int& splits, cudaStream_t s) {
    splits = std::max(1, std::min(splits, kSms * kPerSm<VW, NCH> / p.H));
    set_step(p.s, (uint32_t)splits * (kThreads / LPR));
    const dim3 grid((unsigned)splits, (unsigned)p.H);
    const bool gated = p.s.base[kZ] != nullptr, full = p.d == VW * LPR * NCH;
    if (gated) return full ? run<E, VW, LPR, NCH, true, true>(p, grid, s) : run<E, VW, LPR, NCH, true, false>(p, grid, s);
    return full ? run<E, VW, LPR, NCH, false, true>(p, grid, s) : run<E, VW, LPR, NCH, false, false>(p, grid, s);
}

// Lanes and chunks of a row: 8 elements a lane (of fp32 4) with two or three CTAs an SM, or 24 with one where that
// leaves fewer lanes idle. The sums of dw and db take twice an element's registers, so the forward's 16 are slower (d =
// 64: 30.6 against 28.9 us for [8,12,2048,64] bf16), while fewer elements on more lanes pay a row's fixed part more
// often: [8,12,1310,100] bf16 takes 32 us with 8 on 16 lanes, 45 with 4 on 32; [8,12,3971,33] 46 us with 6 on 8
// lanes, 109 with 2 on 32; [4,1,32768,192] 49 us with 24 on 8 lanes, 60 with 8 on 32 (all without the ring).
template <typename E, int VW>
int by_width(const BwdParams& p, int& splits, cudaStream_t s) {
    const int nv = (p.d + VW - 1) / VW;
    if constexpr (VW * sizeof(E) == 16) {
        if (nv <= 2) return launch<E, VW, 2, 1>(p, splits, s);
        if (nv <= 4) return launch<E, VW, 4, 1>(p, splits, s);
        if (nv <= 8) return launch<E, VW, 8, 1>(p, splits, s);
        if constexpr (VW == 8)
            if (nv <= 12) return launch<E, VW, 4, 3>(p, splits, s);
        if (nv <= 16) return launch<E, VW, 16, 1>(p, splits, s);
        if constexpr (VW == 8)
            if (nv > 16 && nv <= 24) return launch<E, VW, 8, 3>(p, splits, s);
        if (nv <= 32) return launch<E, VW, 32, 1>(p, splits, s);
        if (nv <= 48) return launch<E, VW, 16, 3>(p, splits, s);
        if constexpr (VW == 4)
            if (nv <= 64) return launch<E, VW, 16, 4>(p, splits, s);
    } else if constexpr (VW == 4) {
        if (nv <= 4) return launch<E, VW, 2, 2>(p, splits, s);
        if (nv <= 8) return launch<E, VW, 4, 2>(p, splits, s);
        if (nv <= 16) return launch<E, VW, 8, 2>(p, splits, s);
        if (nv <= 32) return launch<E, VW, 16, 2>(p, splits, s);
    } else {
        if (nv <= 16) return launch<E, VW, 4, 4>(p, splits, s);
        if (nv <= 32) return launch<E, VW, 8, 4>(p, splits, s);
        if (nv <= 48) return launch<E, VW, 8, 6>(p, splits, s);
        if (nv <= 64) return launch<E, VW, 8, 8>(p, splits, s);
        if (nv <= 128) return launch<E, VW, 16, 8>(p, splits, s);
        if (nv <= 256) return launch<E, VW, 32, 8>(p, splits, s);
        return launch<E, VW, 32, 32>(p, splits, s);
    }
    if constexpr (VW > 1) {
        if (nv <= 64) return launch<E, VW, 32, 2>(p, splits, s);
        if (nv <= 96) return launch<E, VW, 32, 3>(p, splits, s);
        if (nv <= 128) return launch<E, VW, 32, 4>(p, splits, s);
    }
    if constexpr (VW == 4) {
        if (nv <= 192) return launch<E, VW, 32, 6>(p, splits, s);
        if (nv <= 256) return launch<E, VW, 32, 8>(p, splits, s);
    }
    return 2;
}

}  // namespace

// As many CTAs as run at once (a CTA more would wait for a whole turn: 24 against 17.5 us for [8,12,1024,64]
// bf16 with a gate), over the heads; no more than there are rows for.
int gn_bwd_splits(const SeqSizes& n) {
    const long long rows = n.B * n.T;
    const bool narrow = n.d * (n.bf16 ? 1 : 2) <= 256;  // a lane holds 16 bytes of a row or less
    long long s = kSms * (narrow ? n.bf16 ? 2 : 3 : 1) / n.H;
    const long long most = (rows + 31) / 32;
    if (s > most) s = most;
    return s < 1 ? 1 : (int)s;
}

int launch_gn_bwd(const GnArgs& a, cudaStream_t s) {
    if (a.n.H > 65535 || (unsigned __int128)a.n.B * a.n.T >= ((unsigned __int128)1 << 31) - 65536) return 2;
    BwdParams p = {};
    p.w = a.w, p.b = a.b, p.lengths = a.lengths, p.ws = a.ws;
    const SeqView* v[] = {&a.x, &a.z, &a.dy, &a.dx, &a.dz};
    const int es = a.n.bf16 ? 2 : 4;
    int vw = 16 / es;  // elements that every access can move at a time: 16 bytes, or 8, else one
    while (vw > 1 && a.n.d % vw) vw /= 2;
    for (int k = 0; k < 5; ++k) {
        p.s.base[k] = static_cast<char*>(v[k]->p);
        p.s.sb[k] = v[k]->sb * es, p.s.sh[k] = v[k]->sh * es, p.s.st[k] = v[k]->st * es;
        while (vw > 1 && !seq_vec_ok(*v[k], es, vw * es)) vw /= 2;
    }
    p.rows = (uint32_t)(a.n.B * a.n.T);
    p.s.tokens = fast_div((uint32_t)a.n.T);
    p.s.B = (uint32_t)a.n.B;
    p.d = a.n.d, p.H = (int)a.n.H, p.act = a.act;
    p.inv_d = 1.f / a.n.d, p.eps = a.eps;
    if (a.n.T == 1 && !p.lengths) {  // single tokens: the batch takes the tokens' place
        p.s.tokens = fast_div(p.rows);
        p.s.B = 1;
        for (int k = 0; k < 5; ++k) p.s.st[k] = p.s.sb[k];
    }
    if (reinterpret_cast<uintptr_t>(a.w) % 16 || reinterpret_cast<uintptr_t>(a.b) % 16) vw = 1;
    int splits = gn_bwd_splits(a.n);
    int st;
    if (a.n.bf16)
        st = vw == 8   ? by_width<bf16, 8>(p, splits, s)
             : vw == 4 ? by_width<bf16, 4>(p, splits, s)
                       : by_width<bf16, 1>(p, splits, s);
    else
        st = vw == 4 ? by_width<float, 4>(p, splits, s) : by_width<float, 1>(p, splits, s);
    if (st != 0 || !a.ws) return st;
    const long long n = a.n.H * a.n.d;
    return launch_ahead<gn_sum_kernel>(dim3((unsigned)((2 * n + kSumChannels - 1) / kSumChannels)),
                                       kSumChannels * kSumSlices, 0, s, (const float*)a.ws, splits, n, a.dw, a.db);
}

}  // namespace falcon
