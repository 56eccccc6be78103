// Gated delta rule, forward: the chunks' maps (gdr_prep), the scan over them (gdr_scan), the outputs (gdr_out), and
// short sequences token by token (gdr_step). The algebra is in falcon_gdr.cuh.

#include <type_traits>

#include "falcon.h"
#include "falcon_gdr.cuh"
#include "falcon_gdr_bwd.cuh"

namespace falcon {
namespace gdr {
namespace {

// ---- outputs of one chunk: out = scale diag(e^G) Q S + P U, U = diag(beta) X (V - diag(e^G) K S), every
// fp32 operand in three planes.
template <typename E>
struct OutArgs {
    Sizes n;
    Ten<const E> q, k, v;
    Ten<E> out;
    Ten<float> beta, g;
    const uint8_t *X, *S;
};

// acc += K S and o += Q S (S stored [n][k]): S is fetched once; twice from fp32 inputs, whose small products come first.
template <int PA, int WHICH = kAll>
__device__ __forceinline__ void mm_both(float (&acc)[8][4], float (&o)[8][4], uint32_t K, uint32_t Q, int rb, uint32_t S, const Lane& ln) {
    if constexpr (PA == 3 && WHICH == kAll) {
        mm_both<PA, kSmall>(acc, o, K, Q, rb, S, ln);
        mm_both<PA, kGreat>(acc, o, K, Q, rb, S, ln);
        return;
    }
    constexpr int NA = WHICH == kGreat ? 1 : PA, NB = WHICH == kGreat ? 1 : 3;
#pragma unroll 1
    for (int kk = 0; kk < 4; ++kk) {
        uint32_t a[NA][4], q[NA][4];
        const uint32_t at = (16 * rb + ln.l7 + 8 * ln.l8) * 128 + (((2 * kk + ln.l16) ^ ln.l7) << 4);
#pragma unroll
        for (int m = 0; m < NA; ++m) {
            ldm<false>(a[m], K + at + m * kPlane);
            ldm<false>(q[m], Q + at + m * kPlane);
        }
        const uint32_t row = S + (8 * ln.l16 + ln.l7) * 128 + (((2 * kk + ln.l8) ^ ln.l7) << 4);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint32_t v[NB][4];
#pragma unroll
            for (int m = 0; m < NB; ++m) ldm<false>(v[m], row + m * kPlane + p * 2048);
#pragma unroll
            for (int s = NB - 1; s >= (WHICH == kSmall ? 1 : 0); --s)
#pragma unroll
                for (int ma = 0; ma < NA; ++ma) {
                    if (s < ma) continue;
                    mma(acc[2 * p], a[ma], v[s - ma][0], v[s - ma][1]);
                    mma(acc[2 * p + 1], a[ma], v[s - ma][2], v[s - ma][3]);
                    mma(o[2 * p], q[ma], v[s - ma][0], v[s - ma][1]);
                    mma(o[2 * p + 1], q[ma], v[s - ma][2], v[s - ma][3]);
                }
        }
    }
}

template <typename E, int NK>
__host__ __device__ constexpr int out_smem() { return (2 * NK * planes<E>() + 6) * kPlane; }

template <typename E, int NK>
__global__ void __launch_bounds__(kThreads, ctas_of(out_smem<E, NK>())) gdr_out(const OutArgs<E> a) {
    constexpr int PI = planes<E>();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Scal s;
    uint8_t* K = smem;
    uint8_t* Q = K + NK * PI * kPlane;
    uint8_t* X = Q + NK * PI * kPlane;
    uint8_t* W = X + 3 * kPlane;
    const uint32_t Ks = saddr(K), Qs = saddr(Q), Xs = saddr(X), Ws = saddr(W);
    const Lane ln;
    const unsigned ubh = blockIdx.x / (unsigned)a.n.NC, ub = ubh / (unsigned)a.n.H, uh = ubh % (unsigned)a.n.H;
    const long long bh = ubh, b = ub, h = uh, hk = uh / (unsigned)a.n.group;
    const int c = (int)(blockIdx.x % (unsigned)a.n.NC);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int rows = min(kC, a.n.T - c * kC), live = min(kC, length_of(a.n, b) - c * kC);
    const int rb = ((threadIdx.x >> 5) + blockIdx.x) & 3;
    const long long t0 = (long long)c * kC;
    const int NV = (a.n.dv + kC - 1) / kC;
    float acc[8][4];
    if (live <= 0) {
        zero(acc);
        for (int sb = 0; sb < NV; ++sb)
            write_rows(a.out.row0(b, h, t0) + sb * kC, a.out.st, a.out.pair, rb, acc, ln, rows, 0, a.n.dv - sb * kC);
        return;
    }
    const uint8_t* St = a.S + (bh * (a.n.NC + 1) + c) * ((long long)NV * NK * 3 * kPlane);
    const Gates gates = load_gates<false>(a.beta, a.g, b, h, t0, live);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) {
        load_planes(K + kb * PI * kPlane, a.k.row0(b, hk, t0) + kb * kC, a.k.st, live, a.n.dk - kb * kC, a.k.vec);
        load_planes(Q + kb * PI * kPlane, a.q.row0(b, hk, t0) + kb * kC, a.q.st, live, a.n.dk - kb * kC, a.q.vec);
    }
    commit();
    copy_planes<3>(Ws, St);
    copy_planes<3>(Xs, a.X + (bh * a.n.NC + c) * (3 * kPlane));
    commit();
    make_scal(s, gates);
    wait<1>();
    __syncthreads();
    float P[8][4];
    zero(P);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb)
        sum<NK * PI == 6>(P, [&](float (&x)[8][4]) { mm<PI, PI, false, false>(x, Qs + kb * PI * kPlane, rb, Ks + kb * PI * kPlane, ln, 0, 4, 0, rb + 1); });
    times_decay<false, false>(P, s, rb, ln, nullptr, a.n.scale);
#pragma unroll 1
    for (int sb = 0; sb < NV; ++sb) {
        float o[8][4];
        Rows<E> v;
        load_rows(v, a.v.row0(b, h, t0) + sb * kC, a.v.st, a.v.pair, rb, ln, live, a.n.dv - sb * kC);
        zero(acc);
        zero(o);
        auto state = [&](int kb, auto planes) {  // its tile (sb, kb) in W
            constexpr int N = decltype(planes)::value;
            if (sb + kb > 0 || N == 1) {
                __syncthreads();
                copy_planes<N>(Ws, St + (sb * NK + kb) * (3 * kPlane));
                commit();
            }
            wait<0>();
            __syncthreads();
        };
        if constexpr (NK * PI == 6) {  // fp32's wide heads: both tiles' small products first
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                state(kb, std::integral_constant<int, 3>{});
                mm_both<PI, kSmall>(acc, o, Ks + kb * PI * kPlane, Qs + kb * PI * kPlane, rb, Ws, ln);
            }
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                state(kb, std::integral_constant<int, 1>{});
                mm_both<PI, kGreat>(acc, o, Ks + kb * PI * kPlane, Qs + kb * PI * kPlane, rb, Ws, ln);
            }
        } else {
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                state(kb, std::integral_constant<int, 3>{});
                mm_both<PI>(acc, o, Ks + kb * PI * kPlane, Qs + kb * PI * kPlane, rb, Ws, ln);
            }
        }
        __syncthreads();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const float eG = s.eG[16 * rb + ln.r + 8 * hf];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 x = v.of(nt, hf);
                acc[nt][2 * hf] = fmaf(-eG, acc[nt][2 * hf], x.x);
                acc[nt][2 * hf + 1] = fmaf(-eG, acc[nt][2 * hf + 1], x.y);
                o[nt][2 * hf] *= eG * a.n.scale;
                o[nt][2 * hf + 1] *= eG * a.n.scale;
            }
        }
        const bool predicted = all_finite(acc);
        put_planes(W, rb, acc, ln);
        __syncthreads();
        zero(acc);
        mm_lower(acc, Xs, rb, Ws, ln, predicted);
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] *= s.beta[16 * rb + ln.r + 8 * (e >> 1)];
        const bool written = all_finite(acc);
        put_planes(W, rb, acc, ln);
        __syncthreads();
        sum<PI == 3>(o, [&](float (&x)[8][4]) { mmr_lower(x, P, Ws, rb, ln, written); });
        write_rows(a.out.row0(b, h, t0) + sb * kC, a.out.st, a.out.pair, rb, o, ln, rows, live, a.n.dv - sb * kC);
    }
}

// ---- short sequences: a CTA holds 64 columns of a head's state, a thread R rows x 4 columns of them (16 threads a row, a
// warp 2 R whole rows that lie together), and walks the tokens, k and q in shared memory. Bound by the state's bytes, read
// and written once: 256 x 12 states of 64 x 64 take 19.3 us, 78 % of the copy rate (a warp's rows 8 apart and k and q in
// registers took 23 % more).
template <typename E>
struct StepArgs {
    Sizes n;
    Ten<const E> q, k, v;
    Ten<E> out;
    Ten<float> beta, g;
    const float* S0;
    float* S;
    int cols;         // of 64 a head
    bool vec;         // states in 16-byte pieces
};

template <typename E, int R>
__global__ void __launch_bounds__(kThreads, R == 8 ? 6 : 4) gdr_step(const StepArgs<E> a) {
    __shared__ float part[2][kThreads / 32][9 * 16];
    __shared__ __align__(16) float ks[2][kGdrMaxD], qs[2][kGdrMaxD];  // zero from dk on
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31, rg = threadIdx.x >> 4, c = l & 15;
    const unsigned ubh = blockIdx.x / (unsigned)a.cols, ub = ubh / (unsigned)a.n.H, uh = ubh % (unsigned)a.n.H;
    const long long bh = ubh, b = ub, h = uh, hk = uh / (unsigned)a.n.group;
    const int c0 = 64 * (int)(blockIdx.x % (unsigned)a.cols) + 4 * c;
    const int dk = a.n.dk, dv = a.n.dv;
    float S[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = R * rg + i;
        S[i][0] = S[i][1] = S[i][2] = S[i][3] = 0.f;
        if (!a.S0 || row >= dk || c0 >= dv) continue;
        const float* p = a.S0 + (bh * dk + row) * dv + c0;
        if (a.vec) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            S[i][0] = x.x, S[i][1] = x.y, S[i][2] = x.z, S[i][3] = x.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c0 + e < dv) S[i][e] = p[e];
        }
    }
    const int live = length_of(a.n, b);
    for (int t = 0; t < a.n.T; ++t) {
        E* po = a.out.row0(b, h, t) + c0;
        if (t >= live) {
            if (rg == 0) store2(po, 0.f, 0.f, dv - c0, a.out.pair), store2(po + 2, 0.f, 0.f, dv - c0 - 2, a.out.pair);
            continue;
        }
        const E* pv = a.v.row0(b, h, t) + c0;
        const int id = threadIdx.x, now = t & 1;  // the other half is still read for the token before
        ks[now][id] = id < dk ? to_f(a.k.row0(b, hk, t)[id]) : 0.f;
        qs[now][id] = id < dk ? to_f(a.q.row0(b, hk, t)[id]) : 0.f;
        const float2 v0 = load2(pv, dv - c0, a.v.pair), v1 = load2(pv + 2, dv - c0 - 2, a.v.pair);
        const float v[4] = {v0.x, v0.y, v1.x, v1.y};
        const float beta = *a.beta.row0(b, h, t), dec = expf(*a.g.row0(b, h, t));
        __syncthreads();
        const float *k = ks[now] + R * rg, *q = qs[now] + R * rg;
        float x[9];  // S^T k, S^T q, k.q
#pragma unroll
        for (int e = 0; e < 9; ++e) x[e] = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                S[i][e] *= dec;
                x[e] = fmaf(S[i][e], k[i], x[e]);
                x[4 + e] = fmaf(S[i][e], q[i], x[4 + e]);
            }
            x[8] = fmaf(k[i], q[i], x[8]);
        }
        float* mine = part[now][w];
#pragma unroll
        for (int e = 0; e < 9; ++e) {
            x[e] += __shfl_xor_sync(0xffffffffu, x[e], 16);
            if (l < 16) mine[16 * e + c] = x[e];
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 9; ++e) {
            const float* p = part[now][0] + 16 * e + c;
            x[e] = (p[0] + p[9 * 16]) + (p[18 * 16] + p[27 * 16]);
        }
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = beta * (v[e] - x[e]);
            o[e] = a.n.scale * fmaf(x[8], u, x[4 + e]);
#pragma unroll
            for (int i = 0; i < R; ++i) S[i][e] = fmaf(k[i], u, S[i][e]);
        }
        if (rg == 0) store2(po, o[0], o[1], dv - c0, a.out.pair), store2(po + 2, o[2], o[3], dv - c0 - 2, a.out.pair);
    }
    if (!a.S) return;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = R * rg + i;
        if (row >= dk || c0 >= dv) continue;
        float* p = a.S + (bh * dk + row) * dv + c0;
        if (a.vec) {
            *reinterpret_cast<float4*>(p) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (c0 + e < dv) p[e] = S[i][e];
        }
    }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename E>
int launch_step(const GdrArgs& a, cudaStream_t st) {
    StepArgs<E> p = {};
    p.n = sizes_of(a, Layout{});
    p.q = ten<const E>(a.q, a.n.dk);
    p.k = ten<const E>(a.k, a.n.dk);
    p.v = ten<const E>(a.v, a.n.dv);
    p.out = ten<E>(a.out, a.n.dv);
    p.beta = ten<float>(a.beta, 1);
    p.g = ten<float>(a.g, 1);
    p.S0 = a.S0;
    p.S = a.S_final;
    p.cols = (a.n.dv + 63) / 64;
    p.vec = a.n.dv % 4 == 0 && al16(a.S0) && al16(a.S_final);
    const unsigned grid = (unsigned)(p.n.BH * p.cols);
    return a.n.dk <= 64 ? launch_ahead<gdr_step<E, 8>>(grid, kThreads, 0, st, p) : launch_ahead<gdr_step<E, 16>>(grid, kThreads, 0, st, p);
}

template <typename E, int NK>
int launch_chunks(const GdrArgs& a, const Layout& l, cudaStream_t st) {
    const Sizes n = sizes_of(a, l);
    PrepArgs<E> p = {};
    p.n = n;
    p.k = ten<const E>(a.k, a.n.dk);
    p.v = ten<const E>(a.v, a.n.dv);
    p.beta = ten<float>(a.beta, 1);
    p.g = ten<float>(a.g, 1);
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
    p.X = ws + l.X;
    p.M = ws + l.M;
    p.A = reinterpret_cast<float*>(ws + l.A);
    OutArgs<E> o = {};
    o.n = n;
    o.q = ten<const E>(a.q, a.n.dk);
    o.k = p.k;
    o.v = p.v;
    o.out = ten<E>(a.out, a.n.dv);
    o.beta = p.beta;
    o.g = p.g;
    o.X = p.X;
    o.S = ws + l.S;
    const unsigned grid = (unsigned)(n.BH * l.NC);
    int r = launch_ahead<gdr_prep<E, NK, false>>(grid, kThreads, prep_smem<E, NK, false>(), st, p);
    r |= run_scan<NK>(n, l, ws, a.S0, a.S_final, st);
    return r | launch_ahead<gdr_out<E, NK>>(grid, kThreads, out_smem<E, NK>(), st, o);
}

template <typename E>
int launch_fwd(const GdrArgs& a, cudaStream_t st) {
    if (a.n.T <= kGdrStepT) return launch_step<E>(a, st);
    const Layout l = layout_of(a.n, false);
    return l.NK == 1 ? launch_chunks<E, 1>(a, l, st) : launch_chunks<E, 2>(a, l, st);
}

}  // namespace
}  // namespace gdr

unsigned long long gdr_fwd_workspace(const GdrSizes& n) {
    return n.T <= kGdrStepT ? 0 : (unsigned long long)gdr::layout_of(n, false).total;
}

bool gdr_fits(const GdrSizes& n) {
    const long long BH = n.B * n.H, NC = (n.T + gdr::kC - 1) / gdr::kC;
    return BH < 1ll << 28 && (n.T <= kGdrStepT || BH * NC < 1ll << 27);
}

int launch_gdr_fwd(const GdrArgs& a, cudaStream_t s) { return a.n.bf16 ? gdr::launch_fwd<gdr::bf16>(a, s) : gdr::launch_fwd<float>(a, s); }

unsigned long long gdr_bwd_workspace(const GdrSizes& n) { return (unsigned long long)gdr::layout_of(n, true).total; }

int launch_gdr_bwd(const GdrArgs& a, cudaStream_t s) {
    const bool one = a.n.dk <= gdr::kC;
    if (a.n.bf16) return one ? gdr::launch_bwd<gdr::bf16, 1>(a, s) : gdr::launch_bwd<gdr::bf16, 2>(a, s);
    return one ? gdr::launch_bwd<float, 1>(a, s) : gdr::launch_bwd<float, 2>(a, s);
}

}  // namespace falcon
