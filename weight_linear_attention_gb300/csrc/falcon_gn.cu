// Group norm of a token's head with an activation and a gate, forward:
// n = w (x - mean) / sqrt(var + eps) + b over the d channels of one (batch, head, token);
// y = act(n), or n act(z).
//
// A memory-bound transposition with arithmetic on the way: 2 (3 with a gate) tensors' bytes per element.
// LPR lanes hold a row in registers (16 or 24 elements a lane), so the row is read once and the variance is that
// of the centred values. A group of lanes keeps one head, so that weight and bias stay in registers, and
// steps over the tokens, the next rows' loads on their way while it works on this one; neighbouring groups
// have neighbouring heads, so that a CTA writes whole lines of the projection's layout.
//
// What bounds it: memory ([16,16,4096,64] bf16 with a SiLU gate: 60 us, 99 % of the copy rate; [4,12,8192,64] fp32 46
// us, 97 %); at [8,12,2048,64] bf16 (13.4 us, 83 %) filling and emptying; without a gate GELU's arithmetic (the same 14.8
// us, 50 %; [8,12,8192,64] 48.6 us, 61 %, with 63 % of the issue slots busy, where SiLU takes 36.4).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <numeric>

#include "falcon_gn.cuh"

namespace falcon {
namespace {

using namespace gn;

constexpr int kThreads = 256;

enum { kX, kZ, kY };

struct FwdParams {
    Tensors<3> s;
    const float* w;
    const float* b;
    const int32_t* lengths;
    uint32_t rows, H;  // B T, heads
    int d, act;
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

// CTAs that an SM is given: what the registers of the row's width allow.
template <int VW, int NCH>
constexpr int kPerSm = NCH * VW <= 4 ? 4 : NCH * VW <= 8 ? 3 : NCH * VW <= 24 ? 2 : 1;

// Bytes of a row of the CTA's groups, and the rows that its ring holds (0: registers). The ring keeps twice the bytes
// on their way that the registers have room for: [16,16,4096,64] bf16 60 instead of 72 us, [8,12,2048,64] 13.4 instead
// of 16.0. fp32 has as many on their way in registers ([4,12,8192,64] 46 us, with a ring 47); with 24 elements a lane
// the ring's shared memory costs more than it gains ([4,1,8192,768] 28 against 26 us).
template <typename E, int VW, int NCH, bool GATED>
constexpr int kRow = (GATED ? 2 : 1) * NCH * VW * (int)sizeof(E) * kThreads;
template <typename E, int VW, int NCH, bool GATED>
constexpr int kRing =
    VW == 1 || sizeof(E) == 4 || NCH * VW > 16 ? 0 : depth(kRow<E, VW, NCH, GATED>, kPerSm<VW, NCH>, 0);

template <typename E, int VW, int LPR, int NCH, bool GATED, bool FULL>
__global__ void __launch_bounds__(kThreads, kPerSm<VW, NCH>) gn_fwd_kernel(const __grid_constant__ FwdParams p) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    using Q = Row<VW, LPR, NCH, FULL>;
    constexpr int P = Q::P, G = kThreads / LPR;
    constexpr bool kHeld = NCH * VW <= 16;  // weight and bias stay in registers, else they come from the L1 cache
    using V = Pack<E, VW>;
    constexpr int CB = LPR * VW * sizeof(E), D = kRing<E, VW, NCH, GATED>;
    extern __shared__ __align__(16) uint8_t ring[];
    const Q q = {(int)threadIdx.x % LPR, p.d};
    const uint32_t first = blockIdx.x * G, i = first + threadIdx.x / LPR;
    const uint32_t h = i % p.H;
    Rows<E, VW, LPR, NCH, FULL, GATED, 2, 3, kThreads, D, NCH * VW * sizeof(E) <= 64> row;
    row.start(q, p.s, p.lengths, i / p.H, h, ring);
    float2 w[P], bias[P];
    constexpr int FW = VW < 4 ? VW : 4;
    auto params = [&] {
        q.template params<FW>(p.w ? p.w + (long long)h * p.d : nullptr, 1.f, w);
        q.template params<FW>(p.b ? p.b + (long long)h * p.d : nullptr, 0.f, bias);
    };
    if (kHeld) params();
    // the CTA's first group has the first rows: all take as many turns as it has
    for (uint32_t r = first / p.H; r < p.rows; r += p.s.by) {
        float2 x[P], z[GATED ? P : 1], f[P];
        row.wait(q, p.s, p.lengths);
        row.get(q, kX, x);
        if constexpr (GATED) row.get(q, kZ, z);
        const bool mine = row.mine, in = row.in;
        char* const out = row.out[0];
        if (D > 0 || r + p.s.by < p.rows) row.next(q, p.s, p.lengths);
        q.normalise(x, p.inv_d, p.eps);
        if (!kHeld) params();
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = fma2(x[j], w[j], bias[j]);
        if constexpr (GATED) {
            act_all<P>(p.act, z, f);
#pragma unroll
            for (int j = 0; j < P; ++j) f[j] = mul2(f[j], x[j]);
        } else {
            act_all<P>(p.act, x, f);
        }
#pragma unroll
        for (int k = 0; k < NCH; ++k) {
            if (!mine || !q.live(k)) continue;
            V po;
            if (in) po = q.template put<E>(f, k);
            else zero(po);
            *reinterpret_cast<V*>(out + k * CB) = po;
        }
    }
}

template <typename E, int VW, int LPR, int NCH, bool GATED, bool FULL>
int run(const FwdParams& p, uint32_t grid, cudaStream_t s) {
    constexpr int kBytes = kRing<E, VW, NCH, GATED> * kRow<E, VW, NCH, GATED>;
    return launch_ahead<gn_fwd_kernel<E, VW, LPR, NCH, GATED, FULL>>(dim3(grid), kThreads, kBytes, s, p);
}

template <typename E, int VW, int LPR, int NCH>
int launch(FwdParams p, cudaStream_t s) {
    constexpr int G = kThreads / LPR;
    const unsigned __int128 groups = (unsigned __int128)p.rows * p.H;
    if (groups >= ((unsigned __int128)1 << 31)) return 2;
    // the grid's groups are a multiple of the heads, so that a group keeps its head; no more CTAs than run at once
    const uint32_t unit = p.H / std::gcd(p.H, (uint32_t)G);
    const uint32_t most = ((uint32_t)groups + G - 1) / G, slots = kSms * kPerSm<VW, NCH>;
    const uint32_t grid = most <= slots ? (most + unit - 1) / unit * unit : std::max(slots / unit, 1u) * unit;
    set_step(p.s, (uint32_t)((unsigned long long)grid * G / p.H));
    const bool gated = p.s.base[kZ] != nullptr, full = p.d == VW * LPR * NCH;
    if (gated) return full ? run<E, VW, LPR, NCH, true, true>(p, grid, s) : run<E, VW, LPR, NCH, true, false>(p, grid, s);
    return full ? run<E, VW, LPR, NCH, false, true>(p, grid, s) : run<E, VW, LPR, NCH, false, false>(p, grid, s);
}

// Lanes and chunks of a row: 16 elements a lane, or 24 where that leaves fewer lanes idle. What a row costs beside its
// elements (the reductions' shuffles, the walk, the loop) is paid once per lane, so few lanes with much each beat many
// with little: against 16 bytes a lane, both without the ring, [16,16,4096,64] bf16 takes 72 instead of 78 us,
// [4,12,8192,64] fp32 46 instead of 51, and rows whose length is no power of two [8,12,1310,100] bf16 17 instead of 23, [8,12,3971,33] 26 instead of
// 63, [4,1,32768,192] 26 instead of 31. 32 elements a lane leave one CTA an SM: 35 against 16 us at d = 64. Few rows
// (up to two CTAs an SM at 16 bytes a lane) are over sooner with a lane's least to fetch: single tokens
// [256,12,1,64] bf16 1.6 against 2.0 us, [2,12,256,64] 1.9 against 2.0.
template <typename E, int VW>
int by_width(const FwdParams& p, cudaStream_t s) {
    const int nv = (p.d + VW - 1) / VW;
    if constexpr (VW * sizeof(E) == 16) {
        const unsigned __int128 few = 2 * kSms * kThreads / ((unsigned __int128)p.rows * p.H);  // lanes a row may take
        if (nv > 2 && nv <= 4 && few >= 4) return launch<E, VW, 4, 1>(p, s);
        if (nv > 4 && nv <= 8 && few >= 8) return launch<E, VW, 8, 1>(p, s);
        if (nv > 8 && nv <= 16 && few >= 16) return launch<E, VW, 16, 1>(p, s);
        if (nv > 16 && nv <= 32 && few >= 32) return launch<E, VW, 32, 1>(p, s);
    }
    if constexpr (VW == 8) {
        if (nv <= 2) return launch<E, VW, 2, 1>(p, s);
        if (nv <= 4) return launch<E, VW, 2, 2>(p, s);
        if (nv <= 8) return launch<E, VW, 4, 2>(p, s);
        if (nv <= 12) return launch<E, VW, 4, 3>(p, s);
        if (nv <= 16) return launch<E, VW, 8, 2>(p, s);
        if (nv <= 24) return launch<E, VW, 8, 3>(p, s);
        if (nv <= 32) return launch<E, VW, 16, 2>(p, s);
        if (nv <= 48) return launch<E, VW, 16, 3>(p, s);
        if (nv <= 64) return launch<E, VW, 32, 2>(p, s);
        if (nv <= 96) return launch<E, VW, 32, 3>(p, s);
        if (nv <= 128) return launch<E, VW, 32, 4>(p, s);
    } else if constexpr (VW == 4) {
        if (nv <= 4) return launch<E, VW, 2, 2>(p, s);
        if (nv <= 8) return launch<E, VW, 4, 2>(p, s);
        if (nv <= 12) return launch<E, VW, 4, 3>(p, s);
        if (nv <= 16) return launch<E, VW, 4, 4>(p, s);
        if (nv <= 24) return launch<E, VW, 8, 3>(p, s);
        if (nv <= 32) return launch<E, VW, 8, 4>(p, s);
        if (nv <= 48) return launch<E, VW, 16, 3>(p, s);
        if (nv <= 64) return launch<E, VW, 16, 4>(p, s);
        if (nv <= 96) return launch<E, VW, 32, 3>(p, s);
        if (nv <= 128) return launch<E, VW, 32, 4>(p, s);
        if (nv <= 192) return launch<E, VW, 32, 6>(p, s);
        if (nv <= 256) return launch<E, VW, 32, 8>(p, s);
    } else {
        if (nv <= 16) return launch<E, VW, 4, 4>(p, s);
        if (nv <= 32) return launch<E, VW, 8, 4>(p, s);
        if (nv <= 48) return launch<E, VW, 8, 6>(p, s);
        if (nv <= 64) return launch<E, VW, 8, 8>(p, s);
        if (nv <= 128) return launch<E, VW, 16, 8>(p, s);
        if (nv <= 256) return launch<E, VW, 32, 8>(p, s);
        if (nv <= 1024) return launch<E, VW, 32, 32>(p, s);
    }
    return 2;
}

}  // namespace

int launch_gn_fwd(const GnArgs& a, cudaStream_t s) {
    if ((unsigned __int128)a.n.B * a.n.T >= ((unsigned __int128)1 << 31) || a.n.H >= 1LL << 30) return 2;
    FwdParams p = {};
    p.w = a.w, p.b = a.b, p.lengths = a.lengths;
    const SeqView* v[] = {&a.x, &a.z, &a.y};
    const int es = a.n.bf16 ? 2 : 4;
    int vw = 16 / es;  // elements that every access can move at a time: 16 bytes, or 8, else one
    while (vw > 1 && a.n.d % vw) vw /= 2;
    for (int k = 0; k < 3; ++k) {
        p.s.base[k] = static_cast<char*>(v[k]->p);
        p.s.sb[k] = v[k]->sb * es, p.s.sh[k] = v[k]->sh * es, p.s.st[k] = v[k]->st * es;
        while (vw > 1 && !seq_vec_ok(*v[k], es, vw * es)) vw /= 2;
    }
    p.d = a.n.d, p.act = a.act, p.H = (uint32_t)a.n.H;
    p.rows = (uint32_t)(a.n.B * a.n.T);
    p.s.tokens = fast_div((uint32_t)a.n.T);
    p.s.B = (uint32_t)a.n.B;
    p.inv_d = 1.f / a.n.d, p.eps = a.eps;
    if (a.n.T == 1 && !p.lengths) {  // single tokens: the batch takes the tokens' place
        p.s.tokens = fast_div(p.rows);
        p.s.B = 1;
        for (int k = 0; k < 3; ++k) p.s.st[k] = p.s.sb[k];
    }
    if (reinterpret_cast<uintptr_t>(a.w) % 16 || reinterpret_cast<uintptr_t>(a.b) % 16) vw = 1;
    if (a.n.bf16) return vw == 8 ? by_width<bf16, 8>(p, s) : vw == 4 ? by_width<bf16, 4>(p, s) : by_width<bf16, 1>(p, s);
    return vw == 4 ? by_width<float, 4>(p, s) : by_width<float, 1>(p, s);
}

}  // namespace falcon
