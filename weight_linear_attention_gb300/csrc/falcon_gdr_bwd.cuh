// Gated delta rule, backward. With the notation of falcon_gdr.cuh, dO the output's adjoint, dS' that of the state
// behind a chunk:
//   dU = P^T dO + diag(w) K dS',   Z = X^T diag(beta) dU = dV,
//   dS = e^{G_C} dS' + scale Q^T diag(e^G) dO - K^T diag(e^G) Z = M^T dS' + dA,
//   dP_ij = scale D_ij beta_j dO_i.E_j (j <= i),   H_ij = -D_ij beta_j Z_i.E_j (j < i), H symmetric,
//   dQ = scale diag(e^G) dO S^T + dP K,
//   dK = dP^T Q + H K - diag(e^G) Z S^T + diag(w beta) E dS'^T,
//   dbeta_j = E_j.(dU - N^T Z)_j = E_j.Z_j / beta_j.
// The factor e^{G_i} stands before all that token i reads (out_i, what it predicts), e^{-G_i} before all that it
// writes, so dG_i = dO_i.out_i - dV_i.V_i = dQ_i.Q_i - dV_i.V_i, and G_C has <dS', S'> besides; dg is the sum of dG
// from its token to the chunk's end. Its error is 1e-6 of these terms, of which dg is the part e^g: where a token's decay is
// below kSteep, the chunk takes dg from what passes that token. gdr_prep leaves X, M, A and dA, two scans the states S and
// adjoints dS', and gdr_grad takes the gradients, all chunks at once: 18 products a chunk, two CTAs an SM (of their
// operands' 104 KB), bound by latency and by fetching its own instructions (8 x 12 x 1024 x 64 bf16: maps 103, scans 45,
// gradients 211 us).

#pragma once

#include <type_traits>

#include "falcon.h"
#include "falcon_gdr.cuh"

namespace falcon {
namespace gdr {

template <typename E>
struct GradArgs {
    Sizes n;
    Ten<const E> q, k, v, dout;
    Ten<float> beta, g, dbeta, dg;
    Ten<E> dq, dk, dv;
    float *pq, *pk;  // [B,H,T,dk] instead of dq and dk where heads share theirs, or null
    const uint8_t *X, *S, *dS;
};

// K, E, Z, what comes and goes, and dO. With one tile of S and dS' (and bf16) all of it is on its way early: S and dS'
// in E's and Z's places, X and Q in W, then S and dS' in W, whose last plane is dO's, and Q again; else these come one
// after the other. So does fp32's dO: 96 KB then let two CTAs of heads up to 64 run on an SM.
template <typename E>
__host__ __device__ constexpr bool grad_keeps() { return sizeof(E) == 2; }
template <typename E, int NK, int NV>
__host__ __device__ constexpr bool grad_one() { return NK * NV == 1 && sizeof(E) == 2; }
template <typename E, int NK, int NV>
__host__ __device__ constexpr int grad_smem() { return ((NK + (grad_keeps<E>() ? NV : 0)) * planes<E>() + 6 * NV + (grad_one<E, NK, NV>() ? 5 : 3)) * kPlane; }

// Above it the sums' 1e-6 of their terms is e^2 times that of dg at most or so (at -4 it was 2e-4 of dg, at -12 a tenth). What
// passes a token takes a third more of a call (8 x 12 x 1024 x 64 with all tokens below: 389 to 514 us).
constexpr float kSteep = -2.f;

// Summed over the four lanes that hold a row.
__device__ __forceinline__ float row_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}

template <typename E, int NK, int NV>
__global__ void __launch_bounds__(kThreads, ctas_of(grad_smem<E, NK, NV>())) gdr_grad(const GradArgs<E> a) {
    constexpr bool ONE = grad_one<E, NK, NV>(), KEEPS = grad_keeps<E>();
    constexpr int PI = planes<E>();
    constexpr bool SEP = PI == 3;  // what is added to a product's result is made by itself
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Scal s;
    __shared__ float own[kC], dbe[kC], part[kThreads / 32];
    __shared__ bool steep;
    uint8_t* K = smem;
    uint8_t* Et = K + NK * PI * kPlane;
    uint8_t* Zt = Et + NV * 3 * kPlane;
    uint8_t* W = Zt + NV * 3 * kPlane;
    uint8_t* dO = W + (ONE ? 5 : 3) * kPlane;  // KEEPS
    const uint32_t Ks = saddr(K), Os = saddr(dO), Es0 = saddr(Et), Zs0 = saddr(Zt), Ws = saddr(W);
    const Lane ln;
    const unsigned ubh = blockIdx.x / (unsigned)a.n.NC, ub = ubh / (unsigned)a.n.H, uh = ubh % (unsigned)a.n.H;
    const long long bh = ubh, b = ub, h = uh, hk = uh / (unsigned)a.n.group;
    const int c = (int)(blockIdx.x % (unsigned)a.n.NC);
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const int rows = min(kC, a.n.T - c * kC), live = min(kC, length_of(a.n, b) - c * kC);
    const int rb = ((threadIdx.x >> 5) + blockIdx.x) & 3;
    const int dk = a.n.dk, dv = a.n.dv;
    const long long t0 = (long long)c * kC;
    auto write_qk = [&](const Ten<E>& t, float* p, const float (&x)[8][4], int kb) {
        if (p) write_rows(p + (bh * a.n.T + t0) * dk + kb * kC, (long long)dk, dk % 2 == 0, rb, x, ln, rows, live, dk - kb * kC);
        else write_rows(t.row0(b, hk, t0) + kb * kC, t.st, t.pair, rb, x, ln, rows, live, dk - kb * kC);
    };
    float x[8][4], d[8][4];
    if (live <= 0) {
        zero(x);
        for (int kb = 0; kb < NK; ++kb) {
            write_qk(a.dq, a.pq, x, kb);
            write_qk(a.dk, a.pk, x, kb);
        }
        for (int sb = 0; sb < NV; ++sb) write_rows(a.dv.row0(b, h, t0) + sb * kC, a.dv.st, a.dv.pair, rb, x, ln, rows, 0, dv - sb * kC);
        if (threadIdx.x < rows) {
            *a.dbeta.row0(b, h, t0 + threadIdx.x) = 0.f;
            *a.dg.row0(b, h, t0 + threadIdx.x) = 0.f;
        }
        return;
    }
    const long long st = (long long)NV * NK * 3 * kPlane;
    const uint8_t* St = a.S + (bh * (a.n.NC + 1) + c) * st;
    const uint8_t* dSt = a.dS + (bh * a.n.NC + c) * st;
    const uint8_t* Xt = a.X + (bh * a.n.NC + c) * (3 * kPlane);
    auto load_q = [&](uint8_t* to, int kb) {
        load_planes(to, a.q.row0(b, hk, t0) + kb * kC, a.q.st, live, dk - kb * kC, a.q.vec);
    };
    // a warp's own rows, 64 channels of them
    auto rows_of = [&](float (&f)[8][4], const Ten<const E>& t, long long head, int blk, int width) {
        Rows<E> o;
        load_rows(o, t.row0(b, head, t0) + blk * kC, t.st, t.pair, rb, ln, live, width - blk * kC);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[nt][e] = e & 1 ? o.of(nt, e >> 1).y : o.of(nt, e >> 1).x;
    };
    // a tile of planes that every warp then reads
    auto bring = [&](uint32_t to, const uint8_t* from) {
        __syncthreads();
        copy_planes<3>(to, from);
        commit();
        wait<0>();
        __syncthreads();
    };
    // <dS', S'>: a tile of dS' in shared memory against the state's behind the chunk
    float ends = 0.f;
    auto meet = [&](const uint8_t* t, const uint8_t* S1) {
#pragma unroll 1
        for (int i = 0; i < kPlane / 16 / kThreads; ++i) {
            float x[8] = {}, y[8] = {};
#pragma unroll
            for (int m = 2; m >= 0; --m) {
                const int o = m * kPlane + 16 * (threadIdx.x + i * kThreads);
                const uint4 u = *reinterpret_cast<const uint4*>(t + o), v = *reinterpret_cast<const uint4*>(S1 + o);
                const uint32_t p[4] = {u.x, u.y, u.z, u.w}, q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] += __uint_as_float(p[e] << 16), x[2 * e + 1] += __uint_as_float(p[e] & 0xffff0000u);
                    y[2 * e] += __uint_as_float(q[e] << 16), y[2 * e + 1] += __uint_as_float(q[e] & 0xffff0000u);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ends = fmaf(x[e], y[e], ends);
        }
    };
    // dO's tile sb, where it is or brought
    auto adjoint = [&](int sb) {
        if (KEEPS) return Os + sb * PI * kPlane;
        __syncthreads();
        load_planes(W, a.dout.row0(b, h, t0) + sb * kC, a.dout.st, live, dv - sb * kC, a.dout.vec);
        commit();
        wait<0>();
        __syncthreads();
        return Ws;
    };
    const uint32_t Xs = ONE ? Ws + 2 * kPlane : Ws;
    const Gates gates = load_gates<true>(a.beta, a.g, b, h, t0, live);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) load_planes(K + kb * PI * kPlane, a.k.row0(b, hk, t0) + kb * kC, a.k.st, live, dk - kb * kC, a.k.vec);
    if (ONE) load_q(W, 0);
    commit();
#pragma unroll 1
    for (int sb = 0; KEEPS && sb < NV; ++sb) load_planes(dO + sb * PI * kPlane, a.dout.row0(b, h, t0) + sb * kC, a.dout.st, live, dv - sb * kC, a.dout.vec);
    if (ONE) {
        copy_planes<3>(Es0, St);
        copy_planes<3>(Zs0, dSt);
        copy_planes<3>(Xs, Xt);
    }
    commit();
    make_scal(s, gates);
    if (threadIdx.x < 32) {
        const bool any = __any_sync(0xffffffffu, gates.g[0] < kSteep || gates.g[1] < kSteep);
        if (threadIdx.x == 0) steep = any;
    }
    // P transposed: rows j, columns i >= j
    float P[8][4];
    zero(P);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) {
        if (!ONE) {
            if (kb > 0) __syncthreads();
            load_q(W, kb);
            commit();
            wait<0>();
        } else {
            wait<1>();
        }
        __syncthreads();
        sum<SEP && NK == 2>(P, [&](float (&t)[8][4]) { mm<PI, PI, false, false>(t, Ks + kb * PI * kPlane, rb, Ws, ln, 0, 4, rb, 4); });
    }
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        if (nt < 2 * rb) continue;  // 0 there
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 16 * rb + ln.r + 8 * (e >> 1), i = 8 * nt + 2 * ln.j + (e & 1);
            P[nt][e] = j <= i ? P[nt][e] * decay(s, i, j) * a.n.scale : 0.f;
        }
    }
    float q1[8][4];                                 // ONE: dO S^T, taken while S is there
    float sb_[2] = {0.f, 0.f}, sv[2] = {0.f, 0.f};  // the rows' E.Z and dV.V
    float back[2];                                  // what takes a gain's substitute out of Z again
    zero(q1);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int row = 16 * rb + ln.r + 8 * hf;
        const float t = row < live ? a.beta.row0(b, h, t0)[row * a.beta.st] : 0.f;
        back[hf] = fabsf(t) < kTiny ? t / kTiny : 1.f;
    }
#pragma unroll 1
    for (int sb = 0; sb < NV; ++sb) {
        const uint32_t Es = Es0 + sb * 3 * kPlane, Zs = Zs0 + sb * 3 * kPlane;
        Rows<E> v;
        load_rows(v, a.v.row0(b, h, t0) + sb * kC, a.v.st, a.v.pair, rb, ln, live, dv - sb * kC);
        zero(x);
        zero(d);
        if (ONE) {
            wait<0>();
            __syncthreads();
            mm<PI, 3, false, false, kOrdered>(x, Ks, rb, Es, ln);
            mm<PI, 3, false, true, kOrdered>(q1, Os, rb, Es, ln);
            mm<PI, 3, false, false, kOrdered>(d, Ks, rb, Zs, ln);
            meet(Zt, St + st);
        } else {
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                bring(Ws, St + (sb * NK + kb) * (3 * kPlane));
                sum<SEP && NK == 2>(x, [&](float (&t)[8][4]) { mm<PI, 3, false, false, kOrdered>(t, Ks + kb * PI * kPlane, rb, Ws, ln); });
                bring(Ws, dSt + (sb * NK + kb) * (3 * kPlane));
                sum<SEP && NK == 2>(d, [&](float (&t)[8][4]) { mm<PI, 3, false, false, kOrdered>(t, Ks + kb * PI * kPlane, rb, Ws, ln); });
                meet(W, St + st + (sb * NK + kb) * (3 * kPlane));
            }
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[nt][e] *= s.w[16 * rb + ln.r + 8 * (e >> 1)];
        const uint32_t Ob = adjoint(sb);
        sum<SEP>(d, [&](float (&t)[8][4]) { mmr<PI, true, true, kOrdered>(t, P, Ob, ln, rb, 4); });  // dU
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const float eG = s.eG[16 * rb + ln.r + 8 * hf];
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 u = v.of(nt, hf);
                x[nt][2 * hf] = fmaf(-eG, x[nt][2 * hf], u.x);
                x[nt][2 * hf + 1] = fmaf(-eG, x[nt][2 * hf + 1], u.y);
            }
        }
        if (ONE) __syncthreads();  // S and dS' are read
        else bring(Xs, Xt);
        put_planes(Et + sb * 3 * kPlane, rb, x, ln);
        float z[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[nt][e] = d[nt][e] * s.beta[16 * rb + ln.r + 8 * (e >> 1)];
        put_planes(Zt + sb * 3 * kPlane, rb, z, ln);
        __syncthreads();
        zero(x);
        zero(z);
        mm<3, 3, false, true>(x, Xs, rb, Es, ln, 0, rb + 1);  // E
        mm<3, 3, true, true>(z, Xs, rb, Zs, ln, rb, 4);       // Z
        __syncthreads();
        if (ONE) {  // for dK: what there is room for
            copy_planes<3>(Ws, St);
            copy_planes<2>(Ws + 3 * kPlane, dSt);
            commit();
        }
        put_planes(Et + sb * 3 * kPlane, rb, x, ln);
        put_planes(Zt + sb * 3 * kPlane, rb, z, ln);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sb_[e >> 1] = fmaf(x[nt][e], z[nt][e], sb_[e >> 1]);  // Z has beta as a factor
                z[nt][e] *= back[e >> 1];
            }
        write_rows(a.dv.row0(b, h, t0) + sb * kC, a.dv.st, a.dv.pair, rb, z, ln, rows, live, dv - sb * kC);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
                const float2 u = v.of(nt, hf);
                sv[hf] = fmaf(z[nt][2 * hf], u.x, fmaf(z[nt][2 * hf + 1], u.y, sv[hf]));
            }
        __syncthreads();
    }
    // dP, its transpose, and H
    float A1[8][4], A3[8][4], H[8][4];
    zero(A1);
    zero(A3);
    zero(H);
    zero(x);
#pragma unroll 1
    for (int sb = 0; sb < NV; ++sb) {
        const uint32_t Es = Es0 + sb * 3 * kPlane, Zs = Zs0 + sb * 3 * kPlane, Ob = adjoint(sb);
        sum<SEP && NV == 2>(A1, [&](float (&t)[8][4]) { mm<PI, 3, false, false, kOrdered>(t, Ob, rb, Es, ln, 0, 4, 0, rb + 1); });
        sum<SEP && NV == 2>(A3, [&](float (&t)[8][4]) { mm<3, PI, false, false>(t, Es, rb, Ob, ln, 0, 4, rb, 4); });
        sum<SEP && NV == 2>(H, [&](float (&t)[8][4]) { mm<3, 3, false, false>(t, Zs, rb, Es, ln, 0, 4, 0, rb + 1); });
        sum<SEP && NV == 2>(x, [&](float (&t)[8][4]) { mm<3, 3, false, false>(t, Es, rb, Zs, ln, 0, 4, rb, 4); });
    }
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int m = 16 * rb + ln.r + 8 * (e >> 1), n = 8 * nt + 2 * ln.j + (e & 1);
            const bool low = m >= n;
            const float f = decay(s, low ? m : n, low ? n : m) * s.beta[low ? n : m];
            A1[nt][e] = low ? A1[nt][e] * f * a.n.scale : 0.f;
            A3[nt][e] = m <= n ? A3[nt][e] * f * a.n.scale : 0.f;
            H[nt][e] = m == n ? 0.f : (low ? H[nt][e] : x[nt][e]) * -f;
        }
    float sq[2] = {0.f, 0.f};
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) {
        float t[8][4];
        zero(d);
        zero(t);
        if (ONE) {
            wait<0>();
            __syncthreads();
            copy_planes<1>(Ws + 5 * kPlane, dSt + 2 * kPlane);  // dO is read
            commit();
            mm<3, 3, false, true>(d, Zs0, rb, Ws, ln);
            wait<0>();
            __syncthreads();
            load_q(W, 0);
            commit();
            mm<3, 3, false, true>(t, Es0, rb, Ws + 3 * kPlane, ln);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[nt][e] = q1[nt][e];
        } else {
            zero(x);
            // SEP and two tiles: the small products of both come first (in registers of their own there is no room for them)
            auto tiles = [&](auto which) {
                constexpr int WH = decltype(which)::value;
#pragma unroll 1
                for (int sb = 0; sb < NV; ++sb) {
                    float f[8][4];
                    if (!KEEPS) rows_of(f, a.dout, h, sb, dv);
                    bring(Ws, St + (sb * NK + kb) * (3 * kPlane));
                    if (KEEPS) mm<PI, 3, false, true, WH == kAll ? kOrdered : WH>(x, Os + sb * PI * kPlane, rb, Ws, ln);
                    else mmr<3, true, true, WH>(x, f, Ws, ln);
                    mm<3, 3, false, true, WH>(d, Zs0 + sb * 3 * kPlane, rb, Ws, ln);
                    bring(Ws, dSt + (sb * NK + kb) * (3 * kPlane));
                    mm<3, 3, false, true, WH>(t, Es0 + sb * 3 * kPlane, rb, Ws, ln);
                }
            };
            if constexpr (SEP && NV == 2) {
                tiles(std::integral_constant<int, kSmall>{});
                tiles(std::integral_constant<int, kGreat>{});
            } else {
                tiles(std::integral_constant<int, kAll>{});
            }
            __syncthreads();
            load_q(W, kb);
            commit();
        }
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * rb + ln.r + 8 * (e >> 1);
                x[nt][e] *= s.eG[row] * a.n.scale;
                d[nt][e] = fmaf(s.bw[row], t[nt][e], -s.eG[row] * d[nt][e]);
            }
        const uint32_t Kb = Ks + kb * PI * kPlane;
        sum<SEP>(x, [&](float (&u)[8][4]) { mmr<PI, true, true, kOrdered>(u, A1, Kb, ln, 0, rb + 1); });
        write_qk(a.dq, a.pq, x, kb);
        sum<SEP>(d, [&](float (&u)[8][4]) {
            mmr<PI, true, true, SEP ? kSmall : kAll>(u, H, Kb, ln);
            wait<0>();
            __syncthreads();
            mmr<PI, true, true, SEP ? kSmall : kAll>(u, A3, Ws, ln, rb, 4);
            if constexpr (SEP) {
                mmr<PI, true, true, kGreat>(u, H, Kb, ln);
                mmr<PI, true, true, kGreat>(u, A3, Ws, ln, rb, 4);
            }
        });
        write_qk(a.dk, a.pk, d, kb);
        get_planes<PI>(W, rb, t, ln);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) sq[e >> 1] = fmaf(x[nt][e], t[nt][e], sq[e >> 1]);
    }
    // dg of tokens 2 l and 2 l + 1 in the first warp
    float dg[2];
    const int l = threadIdx.x;
    auto sum_ends = [&] {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) ends += __shfl_xor_sync(0xffffffffu, ends, m);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = ends;
    };
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
        const int row = 16 * rb + ln.r + 8 * hf;
        const float o = row_sum(sq[hf] - sv[hf]), e = row_sum(sb_[hf]) / s.beta[row];
        if (ln.j == 0) own[row] = o, dbe[row] = e;  // own = dQ.Q - dV.V
    }
    if (!steep) {
        sum_ends();
        __syncthreads();
        if (threadIdx.x >= 32) return;
        Two sum = add(Two{own[2 * l], 0.f}, Two{own[2 * l + 1], 0.f});  // pairs of floats: the sums may cancel
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const Two o = {__shfl_down_sync(0xffffffffu, sum.hi, m), __shfl_down_sync(0xffffffffu, sum.lo, m)};
            if (l + m < 32) sum = add(sum, o);
        }
        sum = add(sum, Two{(part[0] + part[1]) + (part[2] + part[3]), 0.f});
        dg[0] = sum.hi;
        dg[1] = add(sum, Two{-own[2 * l], 0.f}).hi;
    } else {
        // What passes token t, of which each part has e^g as a factor: with F_ij what token j writes and i > j reads,
        // F_i what i reads of the state before the chunk, F^j what is left of j's at the end, F that state's rest there,
        // dg_t = sum over i >= t, j < t of F_ij + sum over i >= t of F_i + sum over j < t of F^j + F.
        ends = 0.f;
        float f0[2] = {0.f, 0.f}, f1[2] = {0.f, 0.f};  // F_i, F^j
        auto dot = [&](float (&to)[2], const float (&p)[8][4], const float (&q)[8][4], const float* f, float one) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                float u = 0.f;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt) u = fmaf(p[nt][2 * hf], q[nt][2 * hf], fmaf(p[nt][2 * hf + 1], q[nt][2 * hf + 1], u));
                to[hf] = fmaf(u, f[16 * rb + ln.r + 8 * hf] * one, to[hf]);
            }
        };
        float f[8][4], t[8][4];
#pragma unroll 1
        for (int sb = 0; sb < NV; ++sb) {
            zero(x);
            zero(d);
            zero(t);
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                rows_of(f, a.q, hk, kb, dk);
                bring(Ws, St + (sb * NK + kb) * (3 * kPlane));
                mmr<3, false, true>(x, f, Ws, ln);
                mm<PI, 3, false, false>(d, Ks + kb * PI * kPlane, rb, Ws, ln);
                bring(Ws, dSt + (sb * NK + kb) * (3 * kPlane));
                mm<PI, 3, false, false>(t, Ks + kb * PI * kPlane, rb, Ws, ln);
                meet(W, St + (sb * NK + kb) * (3 * kPlane));
            }
            rows_of(f, a.dout, h, sb, dv);
            dot(f0, x, f, s.eG, a.n.scale);
            get_planes<3>(Zt + sb * 3 * kPlane, rb, f, ln);
            dot(f0, d, f, s.eG, -1.f);
            get_planes<3>(Et + sb * 3 * kPlane, rb, f, ln);
            dot(f1, t, f, s.bw, 1.f);
        }
        ends *= s.eC;
        sum_ends();
        zero(x);
        zero(d);
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) {
            rows_of(f, a.q, hk, kb, dk);
            mmr<PI, false, true>(x, f, Ks + kb * PI * kPlane, ln);
            mm<PI, PI, false, false>(d, Ks + kb * PI * kPlane, rb, Ks + kb * PI * kPlane, ln, 0, 4, 0, rb + 1);
        }
        zero(t);
        zero(H);
#pragma unroll 1
        for (int sb = 0; sb < NV; ++sb) {
            rows_of(f, a.dout, h, sb, dv);
            mmr<3, false, true>(t, f, Es0 + sb * 3 * kPlane, ln);
            mm<3, 3, false, false>(H, Zs0 + sb * 3 * kPlane, rb, Es0 + sb * 3 * kPlane, ln, 0, 4, 0, rb + 1);
        }
        f0[0] = row_sum(f0[0]), f0[1] = row_sum(f0[1]), f1[0] = row_sum(f1[0]), f1[1] = row_sum(f1[1]);
        __syncthreads();  // W is read
        float* at_t = reinterpret_cast<float*>(W);  // [4][kC], a warp's rows' part of dg
        float before[2] = {f0[0], f0[1]};           // F_i and the sum over columns before nt's
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int i = 16 * rb + ln.r + 8 * hf, j = 8 * nt + 2 * ln.j;
                float v[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    v[e] = j + e < i ? decay(s, i, j + e) * s.beta[j + e] * fmaf(t[nt][2 * hf + e] * a.n.scale, x[nt][2 * hf + e], -H[nt][2 * hf + e] * d[nt][2 * hf + e]) : 0.f;
                float upto = v[0] + v[1];
#pragma unroll
                for (int m = 1; m < 4; m <<= 1) {
                    const float o = __shfl_up_sync(0xffffffffu, upto, m, 4);
                    if (ln.j >= m) upto += o;
                }
                const float all = __shfl_sync(0xffffffffu, upto, 3, 4), prev = __shfl_up_sync(0xffffffffu, upto, 1, 4);
                const float c0 = before[hf] + (ln.j ? prev : 0.f);
                if (j <= i) sum[0] += c0;
                if (j + 1 <= i) sum[1] += c0 + v[0];
                before[hf] += all;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], m);
                if (ln.r == 0) at_t[rb * kC + 8 * nt + 2 * ln.j + e] = sum[e];
            }
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
            if (ln.j == 0) own[16 * rb + ln.r + 8 * hf] = f1[hf];
        __syncthreads();
        if (threadIdx.x >= 32) return;
        float upto = own[2 * l] + own[2 * l + 1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float o = __shfl_up_sync(0xffffffffu, upto, m);
            if (l >= m) upto += o;
        }
        float left = __shfl_up_sync(0xffffffffu, upto, 1);
        if (l == 0) left = 0.f;
        left += (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float* p = at_t + 2 * l + e;
            dg[e] = (p[0] + p[kC]) + (p[2 * kC] + p[3 * kC]) + left + (e ? own[2 * l] : 0.f);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * l + e;
        if (t >= rows) continue;
        const bool in = t < live;
        *a.dbeta.row0(b, h, t0 + t) = in ? dbe[t] : 0.f;
        // a decay of 0 keeps nothing: its gradient is 0, not what rounding leaves of the sum
        const bool kept = in && !(expf(*a.g.row0(b, h, t0 + t)) == 0.f);
        *a.dg.row0(b, h, t0 + t) = kept ? dg[e] : 0.f;
    }
}

// ---- dq and dk of shared heads: the sums over the heads that share them, in their order
template <typename E>
struct SumArgs {
    const float* part;  // [B,Hk,group,T,dk]
    Ten<E> to;
    long long count;    // rows: B Hk T
    int Hk, group, T, dk;
};
template <typename E>
__global__ void __launch_bounds__(256) gdr_sum(const SumArgs<E> a, const SumArgs<E> a2) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const SumArgs<E>& p = blockIdx.y ? a2 : a;
    const unsigned per = (p.dk + 3) / 4;  // of four channels, a thread each
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, row = id / per;
    if (row >= p.count) return;
    const int i = 4 * (int)(id % per), left = p.dk - i;
    const long long bk = row / p.T, t = row % p.T, next = (long long)p.T * p.dk;
    const float* src = p.part + (bk * p.group * p.T + t) * p.dk + i;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    const bool vec = p.dk % 4 == 0;
#pragma unroll 4
    for (int m = 0; m < p.group; ++m, src += next) {
        if (vec) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) s[e] += src[e];
        }
    }
    E* dst = p.to.row0(bk / p.Hk, bk % p.Hk, t) + i;
    store2(dst, s[0], s[1], left, p.to.pair);
    store2(dst + 2, s[2], s[3], left - 2, p.to.pair);
}

template <typename E, int NK>
int launch_bwd(const GdrArgs& a, cudaStream_t st) {
    const Layout l = layout_of(a.n, true);
    const Sizes n = sizes_of(a, l);
    const unsigned grid = (unsigned)(n.BH * l.NC);
    PrepArgs<E> p = {};
    p.n = n;
    p.q = ten<const E>(a.q, a.n.dk);
    p.k = ten<const E>(a.k, a.n.dk);
    p.v = ten<const E>(a.v, a.n.dv);
    p.dout = ten<const E>(a.dout, a.n.dv);
    p.beta = ten<float>(a.beta, 1);
    p.g = ten<float>(a.g, 1);
    uint8_t* ws = reinterpret_cast<uint8_t*>(a.ws);
    p.X = ws + l.X;
    p.M = ws + l.M;
    p.A = reinterpret_cast<float*>(ws + l.A);
    p.dA = reinterpret_cast<float*>(ws + l.dA);
    int r = 0;
    if (grid) r |= launch_ahead<gdr_prep<E, NK, true>>(grid, kThreads, prep_smem<E, NK, true>(), st, p);
    r |= run_scans<NK>(n, l, ws, a.S0, a.dS_final, a.dS0, st);
    if (!grid) return r;
    GradArgs<E> g = {};
    g.n = n;
    g.q = p.q, g.k = p.k, g.v = p.v, g.dout = p.dout, g.beta = p.beta, g.g = p.g;
    g.dbeta = ten<float>(a.dbeta, 1);
    g.dg = ten<float>(a.dg, 1);
    g.dq = ten<E>(a.dq, a.n.dk);
    g.dk = ten<E>(a.dk, a.n.dk);
    g.dv = ten<E>(a.dv, a.n.dv);
    const bool shared = n.group > 1;
    g.pq = shared ? reinterpret_cast<float*>(ws + l.dq) : nullptr;
    g.pk = shared ? reinterpret_cast<float*>(ws + l.dk) : nullptr;
    g.X = p.X;
    g.S = ws + l.S;
    g.dS = ws + l.dS;
    r |= l.NV == 1 ? launch_ahead<gdr_grad<E, NK, 1>>(grid, kThreads, grad_smem<E, NK, 1>(), st, g)
                   : launch_ahead<gdr_grad<E, NK, 2>>(grid, kThreads, grad_smem<E, NK, 2>(), st, g);
    if (shared) {
        SumArgs<E> q = {g.pq, g.dq, a.n.B * a.n.Hk * a.n.T, (int)a.n.Hk, n.group, a.n.T, a.n.dk}, k = q;
        k.part = g.pk;
        k.to = g.dk;
        r |= launch_ahead<gdr_sum<E>>(dim3((unsigned)((q.count * ((a.n.dk + 3) / 4) + 255) / 256), 2), 256, 0, st, q, k);
    }
    return r;
}

// One translation unit for each, to be compiled side by side.
extern template int launch_bwd<bf16, 1>(const GdrArgs&, cudaStream_t);
extern template int launch_bwd<bf16, 2>(const GdrArgs&, cudaStream_t);
extern template int launch_bwd<float, 1>(const GdrArgs&, cudaStream_t);
extern template int launch_bwd<float, 2>(const GdrArgs&, cudaStream_t);

}  // namespace gdr
}  // namespace falcon
