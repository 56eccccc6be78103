// Gated linear recurrence, h_t = a_t h_{t-1} + u_t per channel, forward and backward.
//
// A span of tokens acts on the state as the affine map h -> A h + H with A the product of its a and H
// what the span makes of a zero state; maps compose as (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2). The
// backward pass is the same scan over the tokens in reverse: with c the gradient that reaches the state
// before token t, dh_t = dout_t + c_{t+1} and c_t = a_t dh_t.
//
// One pass over the data. A CTA owns a tile of kTile tokens x 16 VW channels; each thread holds VW
// channels of R consecutive tokens in registers, loaded once (gates evaluated once), reduced to the
// thread's map, composed over the CTA's threads through shared memory and, for long sequences, over the
// CTAs of a cluster that lie side by side along the tokens: each CTA writes its tile's map into its
// peers' shared memory, and every CTA composes them all in the same order, so that the state that enters
// the next cluster-wide tile is known everywhere without another exchange. Then each thread replays its
// tokens from its entering state and stores them. No scratch in global memory, no atomics, no waits but
// the cluster barrier; the order of every sum is fixed by the sizes.
//
// What bounds it: 3 tensors' bytes per element forward, 5 or 6 backward; ~20 thread instructions per
// element, of which an SM has about 31 (bf16, forward) at the memory rate.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "falcon_internal.h"
#include "falcon_seq.cuh"
#include "falcon_seq.h"
#include "sm103_ptx.cuh"

namespace falcon {
namespace {

using namespace seq;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

struct Params {
    const void* x;
    const void* g;
    const void* out_in;  // backward: the forward's outputs
    const void* dout;
    void* out;           // forward: out; backward: dx
    void* dg;
    const float* h_in;   // forward: h0; backward: dh_final
    const float* h0;     // backward: h_{-1}
    float* h_out;        // forward: h_final; backward: dh0
    const int32_t* lengths;
    long long sb[6], sh[6], st[6];  // x, g, out_in, dout, out, dg
    int H, T, d, tiles;             // tiles: channel tiles of a head
};
enum { kX, kG, kOutIn, kDout, kOut, kDg };

// The maps of a CTA's warps and of a cluster's CTAs: [A | H] of 16 VW channels each.
template <int VW>
struct Smem {
    float warp[2][kWarps][2][16 * VW];
    float cta[2][kMaxCluster][2][16 * VW];
};

template <int VW>
__device__ __forceinline__ void ld_map(const float (*m)[16 * VW], int lane16, float (&A)[VW], float (&Hm)[VW]) {
    if (VW == 4) {
        const float4 a = *reinterpret_cast<const float4*>(&m[0][4 * lane16]);
        const float4 h = *reinterpret_cast<const float4*>(&m[1][4 * lane16]);
        A[0] = a.x, A[VW > 1 ? 1 : 0] = a.y, A[VW > 2 ? 2 : 0] = a.z, A[VW > 3 ? 3 : 0] = a.w;
        Hm[0] = h.x, Hm[VW > 1 ? 1 : 0] = h.y, Hm[VW > 2 ? 2 : 0] = h.z, Hm[VW > 3 ? 3 : 0] = h.w;
    } else {
        A[0] = m[0][lane16];
        Hm[0] = m[1][lane16];
    }
}
template <int VW>
__device__ __forceinline__ void st_map(float (*m)[16 * VW], int lane16, const float (&A)[VW], const float (&Hm)[VW]) {
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        m[0][VW * lane16 + i] = A[i];
        m[1][VW * lane16 + i] = Hm[i];
    }
}

// The state that enters this thread's tokens: composes the thread's map (A, Hm) over the CTA and the
// cluster; `carry` is the state entering the cluster's tile on entry and leaving it on return. Called
// by all threads of the cluster the same number of times; `it` counts the calls.
template <int VW>
__device__ __forceinline__ void scan_tile(Smem<VW>& sm, int it, int cs, int rank, const float (&A)[VW],
                                          const float (&Hm)[VW], float (&carry)[VW], float (&h)[VW]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lane16 = lane & 15;
    const bool upper = lane >= 16;  // the warp's second half holds the later tokens
    const int buf = it & 1;
    float oA[VW], oH[VW];  // the other half's map
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        oA[i] = __shfl_xor_sync(0xffffffffu, A[i], 16);
        oH[i] = __shfl_xor_sync(0xffffffffu, Hm[i], 16);
    }
    if (upper) {
        float wA[VW], wH[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            wA[i] = A[i] * oA[i];
            wH[i] = fmaf(A[i], oH[i], Hm[i]);
        }
        st_map<VW>(sm.warp[buf][warp], lane16, wA, wH);
    }
    __syncthreads();
    // compose the warps' maps: pA, pH those before this warp, tA, tH all of them
    float pA[VW], pH[VW], tA[VW], tH[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) tA[i] = 1.f, tH[i] = 0.f, pA[i] = 1.f, pH[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        float wA[VW], wH[VW];
        ld_map<VW>(sm.warp[buf][w], lane16, wA, wH);
        if (w == warp)
#pragma unroll
            for (int i = 0; i < VW; ++i) pA[i] = tA[i], pH[i] = tH[i];
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            tH[i] = fmaf(wA[i], tH[i], wH[i]);
            tA[i] *= wA[i];
        }
    }
    float in[VW];  // the state entering this CTA's tile
    if (cs > 1) {
        if (it == 0) cluster_wait();  // every peer runs: its shared memory may be written
        if (warp < cs) {              // warp w writes to peer w, A from the lower half, H from the upper
            const uint32_t to = peer(ptx::smem_u32(&sm.cta[buf][rank][upper ? 1 : 0][VW * lane16]), warp);
            if (VW == 4) st_peer4(to, upper ? tH : tA);
            else st_peer(to, upper ? tH[0] : tA[0]);
        }
        // a buffer is written again two tiles on: by then every peer has arrived for the tile between,
        // which it does after reading this one
        cluster_arrive();
        cluster_wait();
#pragma unroll
        for (int i = 0; i < VW; ++i) in[i] = carry[i];
        for (int r = 0; r < cs; ++r) {
            float rA[VW], rH[VW];
            ld_map<VW>(sm.cta[buf][r], lane16, rA, rH);
            if (r == rank)
#pragma unroll
                for (int i = 0; i < VW; ++i) in[i] = carry[i];
#pragma unroll
            for (int i = 0; i < VW; ++i) carry[i] = fmaf(rA[i], carry[i], rH[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            in[i] = carry[i];
            carry[i] = fmaf(tA[i], carry[i], tH[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < VW; ++i) {
        h[i] = fmaf(pA[i], in[i], pH[i]);
        if (upper) h[i] = fmaf(oA[i], h[i], oH[i]);
    }
}

__device__ __forceinline__ int length_of(const Params& p, long long b) {
    if (!p.lengths) return p.T;
    return min(max(p.lengths[b], 0), p.T);
}

// Where this thread works: channels c .. c + VW - 1 of head h of sequence b, tokens from `seg` R on.
struct Place {
    long long b, h;
    int c, seg;
    bool live;  // the channels exist (the last channel tile may be cut)
};
template <int VW>
__device__ __forceinline__ Place place(const Params& p, int cs) {
    Place q;
    const long long i = blockIdx.x / cs;
    const long long bh = i / p.tiles;
    q.c = (int)(i % p.tiles) * 16 * VW + (threadIdx.x & 15) * VW;
    q.b = bh / p.H;
    q.h = bh % p.H;
    q.seg = threadIdx.x >> 4;
    q.live = q.c < p.d;  // VW divides d, or is 1
    return q;
}

template <int VW>
__device__ __forceinline__ void ld_state(const float* s, long long off, bool live, float (&v)[VW]) {
#pragma unroll
    for (int i = 0; i < VW; ++i) v[i] = 0.f;
    if (!s || !live) return;
    const Pack<float, VW> w = load<float, VW>(s, off);
#pragma unroll
    for (int i = 0; i < VW; ++i) v[i] = elem(w, i);
}
template <int VW>
__device__ __forceinline__ void st_state(float* s, long long off, const float (&v)[VW]) {
    Pack<float, VW> w;
    pack(w, v);
    store(s, off, w);
}

template <typename E, int GATE, int VW, int R>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const __grid_constant__ Params p, int cs) {
    __shared__ Smem<VW> sm;
    constexpr int kTile = 2 * kWarps * R;
    const int rank = blockIdx.x % cs;
    if (cs > 1) cluster_arrive();
    const Place q = place<VW>(p, cs);
    const int len = length_of(p, q.b);
    const long long x0 = q.b * p.sb[kX] + q.h * p.sh[kX] + q.c, g0 = q.b * p.sb[kG] + q.h * p.sh[kG] + q.c,
                    o0 = q.b * p.sb[kOut] + q.h * p.sh[kOut] + q.c, s0 = (q.b * p.H + q.h) * p.d + q.c;
    float carry[VW];
    ld_state<VW>(p.h_in, s0, q.live, carry);
    const int step = cs * kTile;
    int it = 0;
    for (int t0 = 0; t0 < len; t0 += step, ++it) {
        const int t = t0 + rank * kTile + q.seg * R;  // far below 2^31: the host refuses T >= 2^30
        Pack<E, VW> px[R], pg[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (q.live && t + r < len) {
                px[r] = load<E, VW>(p.x, x0 + (t + r) * p.st[kX]);
                pg[r] = load<E, VW>(p.g, g0 + (t + r) * p.st[kG]);
            } else {
                zero(px[r]);
                zero(pg[r]);
            }
        }
        float a[R][VW], u[R][VW], A[VW], Hm[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) A[i] = 1.f, Hm[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = t + r < len;
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                float ga, gc;
                if (GATE == kGateDecay) ga = decay_exp(elem(pg[r], i));
                else logistic(elem(pg[r], i), ga, gc);
                a[r][i] = in ? ga : 1.f;
                u[r][i] = GATE == kGateMix ? gc * elem(px[r], i) : elem(px[r], i);  // 0 behind the end
                Hm[i] = fmaf(a[r][i], Hm[i], u[r][i]);
                A[i] *= a[r][i];
            }
        }
        float h[VW];
        scan_tile<VW>(sm, it, cs, rank, A, Hm, carry, h);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int i = 0; i < VW; ++i) h[i] = fmaf(a[r][i], h[i], u[r][i]);
            if (q.live && t + r < len) {
                Pack<E, VW> po;
                pack(po, h);
                store(p.out, o0 + (t + r) * p.st[kOut], po);
            }
        }
    }
    if (cs > 1 && it == 0) cluster_wait();
    if (p.h_out && rank == 0 && q.seg == 0 && q.live) st_state<VW>(p.h_out, s0, carry);
    if (q.live) {
        Pack<E, VW> z;
        zero(z);
        for (long long t = (long long)len + rank * 2 * kWarps + q.seg; t < p.T; t += cs * 2 * kWarps)
            store(p.out, o0 + t * p.st[kOut], z);
    }
}

template <typename E, int GATE, int VW, int R>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const __grid_constant__ Params p, int cs) {
    __shared__ Smem<VW> sm;
    constexpr int kTile = 2 * kWarps * R;
    const int rank = blockIdx.x % cs;
    if (cs > 1) cluster_arrive();
    const Place q = place<VW>(p, cs);
    const int len = length_of(p, q.b);
    long long o[6];
#pragma unroll
    for (int k = 0; k < 6; ++k) o[k] = q.b * p.sb[k] + q.h * p.sh[k] + q.c;
    const long long s0 = (q.b * p.H + q.h) * p.d + q.c;
    float carry[VW];
    ld_state<VW>(p.h_in, s0, q.live, carry);
    const int step = cs * kTile;
    int it = 0;
    for (int n0 = 0; n0 < len; n0 += step, ++it) {
        // the token of reversed position n is len - 1 - n; this thread's are t, t - 1, ..
        const int t = len - 1 - (n0 + rank * kTile + q.seg * R);
        Pack<E, VW> pd[R], pg[R], ph[R], px[GATE == kGateMix ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            zero(pd[r]);
            zero(pg[r]);
            zero(ph[r]);
            if (GATE == kGateMix) zero(px[r]);
            if (q.live && t - r >= 0) {
                pg[r] = load<E, VW>(p.g, o[kG] + (t - r) * p.st[kG]);
                pd[r] = load<E, VW>(p.dout, o[kDout] + (t - r) * p.st[kDout]);
                if (t - r > 0) ph[r] = load<E, VW>(p.out_in, o[kOutIn] + (t - r - 1) * p.st[kOutIn]);
                if (GATE == kGateMix) px[r] = load<E, VW>(p.x, o[kX] + (t - r) * p.st[kX]);
            }
        }
        // a (or, negated and with the sign bit set, 1 - a where that is the smaller): one register that
        // gives both without the cancellation of 1 - (1 - a)
        float a[R][VW], f[R][VW], A[VW], C[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) A[i] = 1.f, C[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool in = t - r >= 0;
            float before[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) before[i] = elem(ph[r], i);
            if (t - r == 0) ld_state<VW>(p.h0, s0, q.live, before);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                float ga, gc;
                if (GATE == kGateDecay) ga = decay_exp(elem(pg[r], i));
                else logistic(elem(pg[r], i), ga, gc);
                if (GATE == kGateDecay) f[r][i] = ga * before[i];
                else f[r][i] = ga * gc * (GATE == kGateMix ? before[i] - elem(px[r], i) : before[i]);
                if (GATE == kGateMix) a[r][i] = ga < gc ? ga : __uint_as_float(__float_as_uint(gc) | 0x80000000u);
                else a[r][i] = in ? ga : 1.f;
                if (!in) ga = 1.f;
                C[i] = ga * (C[i] + elem(pd[r], i));  // dout is 0 behind the end
                A[i] *= ga;
            }
        }
        float c[VW];
        scan_tile<VW>(sm, it, cs, rank, A, C, carry, c);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float dx[VW], dg[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                float ga = a[r][i], gc = 1.f;
                if (GATE == kGateMix) {
                    const float other = 1.f - fabsf(ga);
                    const bool comp = (__float_as_uint(ga) & 0x80000000u) != 0;
                    gc = comp ? fabsf(ga) : other;
                    ga = comp ? other : ga;
                }
                const float dh = elem(pd[r], i) + c[i];
                dx[i] = gc * dh;
                dg[i] = dh * f[r][i];
                c[i] = ga * dh;
            }
            if (q.live && t - r >= 0) {
                Pack<E, VW> po;
                pack(po, dx);
                store(p.out, o[kOut] + (t - r) * p.st[kOut], po);
                pack(po, dg);
                store(p.dg, o[kDg] + (t - r) * p.st[kDg], po);
            }
        }
    }
    if (cs > 1 && it == 0) cluster_wait();
    if (p.h_out && rank == 0 && q.seg == 0 && q.live) st_state<VW>(p.h_out, s0, carry);
    if (q.live) {
        Pack<E, VW> z;
        zero(z);
        for (long long t = (long long)len + rank * 2 * kWarps + q.seg; t < p.T; t += cs * 2 * kWarps) {
            store(p.out, o[kOut] + t * p.st[kOut], z);
            store(p.dg, o[kDg] + t * p.st[kDg], z);
        }
    }
}

// Few tokens (a decoding step): one thread per VW channels walks them.
template <typename E, int GATE, int VW>
__global__ void __launch_bounds__(128) glr_step_kernel(const __grid_constant__ Params p, long long lanes) {
    // a decoding loop's previous step wrote the state: wait for the grid before this one
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= lanes) return;
    const int per = p.d / VW;
    const long long bh = i / per;
    const int c = (int)(i % per) * VW;
    const long long b = bh / p.H, hd = bh % p.H;
    const long long s0 = bh * p.d + c;
    float h[VW];
    ld_state<VW>(p.h_in, s0, true, h);
    const int len = length_of(p, b);
    const long long x0 = b * p.sb[kX] + hd * p.sh[kX] + c, g0 = b * p.sb[kG] + hd * p.sh[kG] + c,
                    o0 = b * p.sb[kOut] + hd * p.sh[kOut] + c;
    for (int t = 0; t < p.T; ++t) {
        Pack<E, VW> po;
        zero(po);
        if (t < len) {
            const Pack<E, VW> px = load<E, VW>(p.x, x0 + t * p.st[kX]), pg = load<E, VW>(p.g, g0 + t * p.st[kG]);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
                float ga, gc = 1.f;
                if (GATE == kGateDecay) ga = decay_exp(elem(pg, j));
                else logistic(elem(pg, j), ga, gc);
                h[j] = fmaf(ga, h[j], GATE == kGateMix ? gc * elem(px, j) : elem(px, j));
            }
            pack(po, h);
        }
        store(p.out, o0 + t * p.st[kOut], po);
    }
    if (p.h_out) st_state<VW>(p.h_out, s0, h);
}

constexpr int kStepTokens = 4;  // up to this length the step kernel runs
constexpr long long kMaxGrid = 0x7fffffffLL;

void set_view(Params& p, int k, const SeqView& v) {
    p.sb[k] = v.sb;
    p.sh[k] = v.sh;
    p.st[k] = v.st;
}

// CTAs of a cluster along the tokens: as many as the sequence has tiles, while the grid is small.
int cluster_size(long long seqs, long long tiles_t) {
    int cs = 1;
    while (cs < kMaxCluster && cs < tiles_t && seqs * cs < 152 * 8) cs *= 2;
    return cs;
}

template <int VW, int R>
int launch_scan_kernel(void (*fn)(Params, int), Params p, long long B, cudaStream_t s) {
    p.tiles = (p.d + 16 * VW - 1) / (16 * VW);
    const long long seqs = B * p.H * p.tiles;
    const int cs = cluster_size(seqs, ((long long)p.T + 2 * kWarps * R - 1) / (2 * kWarps * R));
    if (seqs > kMaxGrid / cs) return 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(seqs * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, p, cs) == cudaSuccess ? 0 : 4;
}

template <typename E, int GATE, int VW>
int launch_fwd(const Params& p, long long B, cudaStream_t s) {
    if (p.T <= kStepTokens) {
        const long long lanes = B * p.H * (p.d / VW), blocks = (lanes + 127) / 128;
        if (blocks > kMaxGrid) return 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(128);
        cfg.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, glr_step_kernel<E, GATE, VW>, p, lanes) == cudaSuccess ? 0 : 4;
    }
    return launch_scan_kernel<VW, 8>(glr_fwd_kernel<E, GATE, VW, 8>, p, B, s);
}
template <typename E, int GATE, int VW>
int launch_bwd_t(const Params& p, long long B, cudaStream_t s) {
    constexpr int R = sizeof(E) == 2 ? 8 : 4;
    return launch_scan_kernel<VW, R>(glr_bwd_kernel<E, GATE, VW, R>, p, B, s);
}

template <typename E, int VW>
int by_gate(bool bwd, int gate, const Params& p, long long B, cudaStream_t s) {
    switch (gate) {
        case kGateDecay: return bwd ? launch_bwd_t<E, kGateDecay, VW>(p, B, s) : launch_fwd<E, kGateDecay, VW>(p, B, s);
        case kGateSigmoid:
            return bwd ? launch_bwd_t<E, kGateSigmoid, VW>(p, B, s) : launch_fwd<E, kGateSigmoid, VW>(p, B, s);
        default: return bwd ? launch_bwd_t<E, kGateMix, VW>(p, B, s) : launch_fwd<E, kGateMix, VW>(p, B, s);
    }
}

int launch(bool bwd, const GlrArgs& a, const SeqView* const* v, int nv, const Params& p, cudaStream_t s) {
    const int es = a.n.bf16 ? 2 : 4;
    bool vec = a.n.d % 4 == 0;
    for (int i = 0; i < nv; ++i) vec = vec && (!v[i]->p || seq_vec_ok(*v[i], es, 4 * es));
    for (const void* st : {(const void*)p.h_in, (const void*)p.h0, (const void*)p.h_out})
        vec = vec && reinterpret_cast<uintptr_t>(st) % 16 == 0;
    if (a.n.bf16) return vec ? by_gate<bf16, 4>(bwd, a.gate, p, a.n.B, s) : by_gate<bf16, 1>(bwd, a.gate, p, a.n.B, s);
    return vec ? by_gate<float, 4>(bwd, a.gate, p, a.n.B, s) : by_gate<float, 1>(bwd, a.gate, p, a.n.B, s);
}

}  // namespace

int launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    Params p = {};
    p.x = a.x.p, p.g = a.g.p, p.out = a.out.p;
    set_view(p, kX, a.x), set_view(p, kG, a.g), set_view(p, kOut, a.out);
    p.h_in = a.h0, p.h_out = a.h_final, p.lengths = a.lengths;
    p.H = (int)a.n.H, p.T = a.n.T, p.d = a.n.d;
    const SeqView* v[] = {&a.x, &a.g, &a.out};
    return launch(false, a, v, 3, p, s);
}

int launch_glr_bwd(const GlrArgs& a, cudaStream_t s) {
    Params p = {};
    p.x = a.x.p, p.g = a.g.p, p.out_in = a.out.p, p.dout = a.dout.p, p.out = a.dx.p, p.dg = a.dg.p;
    set_view(p, kX, a.x), set_view(p, kG, a.g), set_view(p, kOutIn, a.out), set_view(p, kDout, a.dout);
    set_view(p, kOut, a.dx), set_view(p, kDg, a.dg);
    p.h_in = a.dh_final, p.h0 = a.h0, p.h_out = a.dh0, p.lengths = a.lengths;
    p.H = (int)a.n.H, p.T = a.n.T, p.d = a.n.d;
    const SeqView* v[] = {&a.x, &a.g, &a.out, &a.dout, &a.dx, &a.dg};
    return launch(true, a, v, 6, p, s);
}

}  // namespace falcon
