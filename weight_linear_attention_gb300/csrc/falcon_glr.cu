// Gated linear recurrence, h_t = a_t h_{t-1} + u_t per channel, forward and backward.
//
// A span of tokens acts on the state as the affine map h -> A h + H with A the product of its a and H
// what the span makes of a zero state; maps compose as (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2). The
// backward pass is the same scan over the tokens in reverse: with c the gradient that reaches the state
// before token t, dh_t = dout_t + c_{t+1} and c_t = a_t dh_t. Tokens are counted by their position in the
// scan's direction: position n is token n forward and token len - 1 - n backward.
//
// One pass over the data. A CTA works through tiles of kTile positions x 2 LC channels; a thread owns two
// channels of R consecutive positions. Each warp keeps its own ring of tiles in shared memory, filled ahead
// by TMA (by cp.async, or through registers, where addresses do not allow it), evaluates the gates once
// into registers and reduces its tokens to their map; maps are composed over the warp (shuffles), the CTA
// (shared memory) and, for long sequences, the CTAs of a cluster that lie side by side along the tokens:
// each CTA sends its tile's map into its peers' shared memory (st.async, counted by an mbarrier there: no
// fence that would wait for the outputs on their way to memory), and every CTA composes them all in the
// same order, so that the state that enters the next cluster-wide tile is known everywhere without another
// exchange. Then each thread replays its tokens from its entering state into the ring, whence a TMA store
// takes them. No scratch in global memory, no atomics on data; the order of every sum is fixed by the
// sizes. Waits are bounded: one that runs out raises a flag (falcon_device_status) and is not repeated.
//
// What bounds it: 3 tensors' bytes per element forward, 5 or 6 backward; the thread instructions per
// element, of which an SM has about 33 (bf16, forward) at the memory rate.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdlib.h>

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
constexpr long long kTimeoutCycles = 4000000000LL;  // ~2 s

__device__ int g_glr_timeout_flag = 0;

struct Params {
    CUtensorMap tm[6];   // by tensor, for the TMA kernels
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
    long long items;                // sequences x channel tiles
    int H, T, d, tiles;             // tiles: channel tiles of a head
};
enum { kX, kG, kOutIn, kDout, kOut, kDg };

__device__ __forceinline__ int length_of(const Params& p, long long b) {
    if (!p.lengths) return p.T;
    return min(max(p.lengths[b], 0), p.T);
}

// ---- the tiles' geometry: LC lanes of two channels side by side, 32 / LC segments of R positions in a warp
template <int LC, int R>
struct Geo {
    static constexpr int kSegs = 32 / LC;           // of a warp
    static constexpr int kRows = kSegs * R;         // positions of a warp
    static constexpr int kTile = kWarps * kRows;    // positions of a CTA
    static constexpr int kChans = 2 * LC;
};

// A map of one lane's two channels.
struct __align__(16) Map {
    float2 A, H;
};
__device__ __forceinline__ Map shfl_up(const Map& m, int o) {
    Map r;
    r.A.x = __shfl_up_sync(0xffffffffu, m.A.x, o);
    r.A.y = __shfl_up_sync(0xffffffffu, m.A.y, o);
    r.H.x = __shfl_up_sync(0xffffffffu, m.H.x, o);
    r.H.y = __shfl_up_sync(0xffffffffu, m.H.y, o);
    return r;
}
// first `before`, then `m`
__device__ __forceinline__ Map compose(const Map& before, const Map& m) {
    return Map{ptx::mul2(m.A, before.A), ptx::fma2(m.A, before.H, m.H)};
}
__device__ __forceinline__ float2 apply(const Map& m, float2 h) { return ptx::fma2(m.A, h, m.H); }

template <int LC>
struct Maps {
    Map warp[2][kWarps][LC];
    Map cta[2][kMaxCluster][LC];
    uint64_t ready[2];  // the maps of a cluster-wide tile have arrived
};

// Bounded wait of a whole warp. After a wait that ran out the following ones are skipped: the outputs are
// lost, the flag tells, and the kernel comes to its end.
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, bool& dead) {
    if (dead) return;
    if (!ptx::mbar_wait_bounded(ptx::smem_u32(bar), parity, kTimeoutCycles)) {
        dead = true;
        atomicExch(&g_glr_timeout_flag, 1);
    }
    dead = __any_sync(0xffffffffu, dead);
}

// The state that enters this thread's positions: composes the thread's map over the warp, the CTA and the
// cluster; `carry` is the state entering the cluster's tile on entry and leaving it on return. Called by all
// threads of the cluster the same number of times; `it` counts the calls.
template <int LC>
__device__ __forceinline__ float2 scan_tile(Maps<LC>& sm, int it, int cs, int rank, const Map& own, float2& carry,
                                            bool& dead) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % LC;
    const int buf = it & 1;
    Map inc = own;  // over the segments up to this one
#pragma unroll
    for (int o = LC; o < 32; o *= 2) {
        const Map m = shfl_up(inc, o);
        if (lane >= o) inc = compose(m, inc);
    }
    if (lane >= 32 - LC) sm.warp[buf][warp][lc] = inc;
    Map exc = {pair(1.f, 1.f), pair(0.f, 0.f)};  // over the segments before it
    if (LC < 32) {
        const Map m = shfl_up(inc, LC);
        if (lane >= LC) exc = m;
    }
    // the state that was loaded for the first tile has arrived before any peer can know of this tile, and so
    // before the last tile's state may be written over it
    asm volatile("" ::"f"(carry.x), "f"(carry.y) : "memory");
    __syncthreads();
    Map before = {pair(1.f, 1.f), pair(0.f, 0.f)}, all = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = all;
        all = compose(all, sm.warp[buf][w][lc]);
    }
    float2 in;  // the state entering this CTA's tile
    if (cs > 1) {
        if (it == 0) cluster_wait();  // every peer runs and has set up its mbarriers
        const uint32_t bar = ptx::smem_u32(&sm.ready[buf]);
        if (threadIdx.x == 0) ptx::mbar_expect_tx(bar, cs * LC * (uint32_t)sizeof(Map));
        if (warp < cs && lane < LC)
            st_async4(peer(ptx::smem_u32(&sm.cta[buf][rank][lc]), warp), &all.A.x, peer(bar, warp));
        // A peer writes this buffer again two tiles on, after this CTA's map of the tile between has
        // reached it; that is sent behind the __syncthreads above, so behind the reads below.
        wait_for(&sm.ready[buf], (it >> 1) & 1, dead);
        in = carry;
#pragma unroll 4
        for (int r = 0; r < cs; ++r) {
            if (r == rank) in = carry;
            carry = apply(sm.cta[buf][r][lc], carry);
        }
    } else {
        in = carry;
        carry = apply(all, carry);
    }
    return apply(exc, apply(before, in));
}

// ---- the work list: items (sequence, channel tile) dealt to the clusters in turn, each of one or more tiles
struct Cursor {
    long long item;
    long long b, h;
    int c0, n0, len;  // first channel; first position of the cluster's tile; positions in all
};
template <int CHANS>
__device__ __forceinline__ void enter(const Params& p, Cursor& c) {
    c.n0 = 0;
    if (c.item >= p.items) return;
    const long long bh = c.item / p.tiles;
    c.c0 = (int)(c.item - bh * p.tiles) * CHANS;
    c.b = bh / p.H;
    c.h = bh - c.b * p.H;
    c.len = length_of(p, c.b);
}
template <int CHANS>
__device__ __forceinline__ void advance(const Params& p, Cursor& c, int step, int clusters) {
    c.n0 += step;  // far below 2^31: the host refuses T >= 2^30
    if (c.n0 >= c.len) {
        c.item += clusters;
        enter<CHANS>(p, c);
    }
}

// A warp copies its rows of tensor k: position n of the scan is token `first + sign n` (shifted for the
// backward's outputs). CB bytes at a time; 2 bytes (odd addresses of bf16) go through registers.
template <typename E, int LC, int R, int CB>
__device__ __forceinline__ void copy_rows(const Params& p, uint32_t dst, uint8_t* dst_p, const void* base, int k,
                                          const Cursor& c, int n, int t0, int sign, int shift) {
    constexpr int RB = Geo<LC, R>::kChans * sizeof(E), PAD = Geo<LC, R>::kSegs > 1 ? RB : 0;  // as Ring's
    constexpr int CPR = RB / CB, N = Geo<LC, R>::kRows * CPR / 32, EPC = CB / sizeof(E);
    const int lane = threadIdx.x & 31;
    const long long off = c.b * p.sb[k] + c.h * p.sh[k] + c.c0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int q = lane + 32 * j, row = q / CPR, col = q % CPR;
        const int t = t0 + sign * (n + row) + shift;
        const bool in = n + row < c.len && t >= 0 && c.c0 + col * EPC < p.d;
        const long long at = in ? off + t * p.st[k] + col * EPC : 0;
        const uint32_t o = row * RB + row / R * PAD + col * CB;
        if constexpr (CB >= 4) copy_async<CB>(dst + o, static_cast<const E*>(base) + at, in);
        else *reinterpret_cast<uint16_t*>(dst_p + o) = in ? static_cast<const uint16_t*>(base)[at] : (uint16_t)0;
    }
}
__device__ __forceinline__ float2 ld_pair(const float* s) { return *reinterpret_cast<const float2*>(s); }
__device__ __forceinline__ float2 ld_pair(const bf16* s) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(s);
    return pair(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two channels of one row to global memory; VS: both at once (they exist together and the address allows it).
template <typename E, bool VS>
__device__ __forceinline__ void st_pair(void* base, long long off, float2 v, bool second) {
    E* at = static_cast<E*>(base) + off;
    if constexpr (sizeof(E) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
        if (VS) {
            *reinterpret_cast<__nv_bfloat162*>(at) = h;
        } else {
            at[0] = h.x;
            if (second) at[1] = h.y;
        }
    } else {
        if (VS) {
            *reinterpret_cast<float2*>(at) = v;
        } else {
            at[0] = v.x;
            if (second) at[1] = v.y;
        }
    }
}
// The fp32 states: alignment of single elements.
__device__ __forceinline__ float2 ld_state2(const float* s, long long off, bool first, bool second) {
    return pair(s && first ? s[off] : 0.f, s && second ? s[off + 1] : 0.f);
}
__device__ __forceinline__ void st_state2(float* s, long long off, float2 v, bool first, bool second) {
    if (first) s[off] = v.x;
    if (second) s[off + 1] = v.y;
}

template <typename E, int GATE>
__device__ __forceinline__ void gates(float2 g, float2& a, float2& om) {
    if (GATE == kGateDecay) {
        a = decay_exp2(g);
        om = pair(1.f, 1.f);
    } else {
        logistic2(g, a, om);
    }
}

// How a kernel moves its rows: TMA boxes, or copies of 16, 4 or 2 bytes.
constexpr int kTma = 0;

template <typename E, int LC, int R, int CB>
struct Ring {
    using G = Geo<LC, R>;
    static constexpr bool kBoxes = CB == kTma;
    static constexpr bool VS = CB == kTma || CB == 16 || (CB == 4 && sizeof(E) == 2);
    static constexpr int RB = G::kChans * sizeof(E);                     // bytes of a row
    static constexpr int PAD = G::kSegs > 1 && !kBoxes ? RB : 0;         // between segments, against bank conflicts
    static constexpr int WB = G::kRows * RB + G::kSegs * PAD;            // one warp's rows of one tensor
    // where row r of segment seg lies
    static __device__ __forceinline__ int at(int seg, int r) { return (seg * R + r) * RB + seg * PAD; }
};

template <typename E, int GATE, int LC, int R, int CB, int S>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const __grid_constant__ Params p, int cs) {
    using G = Geo<LC, R>;
    using Q = Ring<E, LC, R, CB>;
    __shared__ Maps<LC> sm;
    __shared__ uint64_t full[S][kWarps];
    extern __shared__ __align__(128) uint8_t ring[];  // [S][warp][x, g][rows]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = lane / LC, lc = lane % LC;
    const int rank = blockIdx.x % cs, clusters = gridDim.x / cs, step = cs * G::kTile;
    const int row0 = (rank * kWarps + warp) * G::kRows;  // of the warp, in the cluster's tile
    uint8_t* const mine = ring + warp * 2 * Q::WB;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S * kWarps; ++i) ptx::mbar_init(ptx::smem_u32(&full[0][0] + i), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[1]), 1);
        ptx::mbar_init_fence();
    }
    __syncthreads();
    if (cs > 1) cluster_arrive();

    Cursor pre = {};
    pre.item = blockIdx.x / cs;
    enter<G::kChans>(p, pre);
    Cursor cur = pre;
    bool dead = false;
    int fetched = 0, landed = 0;
    auto fetch = [&](int stage) {
        if (pre.item < p.items && !dead) {
            uint8_t* to = mine + stage * kWarps * 2 * Q::WB;
            const uint32_t dst = ptx::smem_u32(to);
            const int n = pre.n0 + row0;
            if constexpr (Q::kBoxes) {
                if (lane == 0) {
                    const uint32_t bar = ptx::smem_u32(&full[stage][warp]);
                    ptx::bulk_wait_read<0>();  // outputs that lie in the stage have left it
                    ptx::mbar_expect_tx(bar, 2 * Q::WB);
                    tma_load_4d(dst, &p.tm[kX], pre.c0, n, (int)pre.h, (int)pre.b, bar);
                    tma_load_4d(dst + Q::WB, &p.tm[kG], pre.c0, n, (int)pre.h, (int)pre.b, bar);
                }
            } else {
                copy_rows<E, LC, R, CB>(p, dst, to, p.x, kX, pre, n, 0, 1, 0);
                copy_rows<E, LC, R, CB>(p, dst + Q::WB, to + Q::WB, p.g, kG, pre, n, 0, 1, 0);
            }
            advance<G::kChans>(p, pre, step, clusters);
            ++fetched;
        }
        if constexpr (!Q::kBoxes) copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    float2 carry = pair(0.f, 0.f);
    int it = 0, stage = 0;
    for (; cur.item < p.items; ++it) {
        const int c = cur.c0 + 2 * lc;
        const bool first = c < p.d, second = c + 1 < p.d;
        const long long s0 = (cur.b * p.H + cur.h) * p.d + c;
        if (cur.n0 == 0) carry = ld_state2(p.h_in, s0, first, second);
        if constexpr (Q::kBoxes) {
            wait_for(&full[stage][warp], it / S & 1, dead);
            landed += !dead;
        } else {
            copy_wait<S - 2>();
            __syncwarp();
        }
        const int t0 = cur.n0 + row0 + seg * R, left = cur.len - t0;  // this thread's rows inside the sequence
        uint8_t* const from = mine + stage * kWarps * 2 * Q::WB + Q::at(seg, 0) + lc * 2 * sizeof(E);
        float2 a[R], u[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 x = ld_pair(reinterpret_cast<const E*>(from + r * Q::RB));
            float2 om;
            gates<E, GATE>(ld_pair(reinterpret_cast<const E*>(from + Q::WB + r * Q::RB)), a[r], om);
            u[r] = GATE == kGateMix ? ptx::mul2(om, x) : x;
        }
        if (left < R) {  // rows behind the end change nothing, whatever they hold
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r >= left) a[r] = pair(1.f, 1.f), u[r] = pair(0.f, 0.f);
        }
        Map own = {a[0], u[0]};
#pragma unroll
        for (int r = 1; r < R; ++r) own = compose(own, Map{a[r], u[r]});
        __syncwarp();  // every lane has read the stage before this one, which is filled again
        fetch(stage == 0 ? S - 1 : stage - 1);
        float2 h = scan_tile<LC>(sm, it, cs, rank, own, carry, dead);
        const long long o0 = cur.b * p.sb[kOut] + cur.h * p.sh[kOut] + c;
        if constexpr (Q::kBoxes) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = ptx::fma2(a[r], h, u[r]);
                st_pair<E, true>(from + r * Q::RB, 0, h, true);
            }
            if (left < R) {
#pragma unroll
                for (int r = 0; r < R; ++r)
                    if (r >= left) st_pair<E, true>(from + r * Q::RB, 0, pair(0.f, 0.f), true);
            }
            ptx::fence_async_smem();
            __syncwarp();
            if (lane == 0 && cur.n0 + row0 < p.T) {  // a box that ends behind T is cut there
                tma_store_4d(&p.tm[kOut], ptx::smem_u32(mine + stage * kWarps * 2 * Q::WB), cur.c0, cur.n0 + row0,
                             (int)cur.h, (int)cur.b);
                ptx::bulk_commit();
            }
        } else if (first) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = ptx::fma2(a[r], h, u[r]);
                if (r < left) st_pair<E, Q::VS>(p.out, o0 + (t0 + r) * p.st[kOut], h, second);
            }
        }
        if (cur.n0 + step >= cur.len) {
            if (p.h_out && rank == 0 && threadIdx.x < LC) st_state2(p.h_out, s0, carry, first, second);
            // zeros behind the end; boxes have reached the end of the cluster's tile
            const int t1 = Q::kBoxes ? cur.n0 + step : cur.len;
            if (first)
                for (int t = t1 + (rank * kWarps + warp) * G::kSegs + seg; t < p.T; t += cs * kWarps * G::kSegs)
                    st_pair<E, Q::VS>(p.out, o0 + t * p.st[kOut], pair(0.f, 0.f), second);
        }
        advance<G::kChans>(p, cur, step, clusters);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    if constexpr (Q::kBoxes) {
        for (; landed < fetched; ++landed)  // after a wait that ran out: the loads on their way, once more
            ptx::mbar_wait_bounded(ptx::smem_u32(&full[landed % S][warp]), landed / S & 1, kTimeoutCycles);
        if (lane == 0) ptx::bulk_wait_all();
    }
    if (cs > 1) {  // no CTA leaves while a peer may still write to it
        if (it == 0) cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
}

template <typename E, int GATE, int LC, int R, int CB, int S>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const __grid_constant__ Params p, int cs) {
    using G = Geo<LC, R>;
    using Q = Ring<E, LC, R, CB>;
    constexpr int NT = GATE == kGateMix ? 4 : 3;  // g, dout, out, x
    __shared__ Maps<LC> sm;
    __shared__ uint64_t full[S][kWarps];
    extern __shared__ __align__(128) uint8_t ring[];  // [S][warp][tensor][rows]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = lane / LC, lc = lane % LC;
    const int rank = blockIdx.x % cs, clusters = gridDim.x / cs, step = cs * G::kTile;
    const int row0 = (rank * kWarps + warp) * G::kRows;
    uint8_t* const mine = ring + warp * NT * Q::WB;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S * kWarps; ++i) ptx::mbar_init(ptx::smem_u32(&full[0][0] + i), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[1]), 1);
        ptx::mbar_init_fence();
    }
    __syncthreads();
    if (cs > 1) cluster_arrive();

    Cursor pre = {};
    pre.item = blockIdx.x / cs;
    enter<G::kChans>(p, pre);
    Cursor cur = pre;
    bool dead = false;
    int fetched = 0, landed = 0;
    auto fetch = [&](int stage) {
        if (pre.item < p.items && !dead) {
            uint8_t* to = mine + stage * kWarps * NT * Q::WB;
            const uint32_t dst = ptx::smem_u32(to);
            const int n = pre.n0 + row0, last = pre.len - 1;
            if constexpr (Q::kBoxes) {
                if (lane == 0) {
                    // a box holds its tokens in ascending order; it may start before the first one
                    const int t = pre.len - n - G::kRows, h = (int)pre.h, b = (int)pre.b;
                    const uint32_t bar = ptx::smem_u32(&full[stage][warp]);
                    ptx::bulk_wait_read<0>();
                    ptx::mbar_expect_tx(bar, NT * Q::WB);
                    tma_load_4d(dst, &p.tm[kG], pre.c0, t, h, b, bar);
                    tma_load_4d(dst + Q::WB, &p.tm[kDout], pre.c0, t, h, b, bar);
                    tma_load_4d(dst + 2 * Q::WB, &p.tm[kOutIn], pre.c0, t - 1, h, b, bar);
                    if (GATE == kGateMix) tma_load_4d(dst + 3 * Q::WB, &p.tm[kX], pre.c0, t, h, b, bar);
                }
            } else {
                copy_rows<E, LC, R, CB>(p, dst, to, p.g, kG, pre, n, last, -1, 0);
                copy_rows<E, LC, R, CB>(p, dst + Q::WB, to + Q::WB, p.dout, kDout, pre, n, last, -1, 0);
                // h before the token; the first token's is h0
                copy_rows<E, LC, R, CB>(p, dst + 2 * Q::WB, to + 2 * Q::WB, p.out_in, kOutIn, pre, n, last, -1, -1);
                if (GATE == kGateMix)
                    copy_rows<E, LC, R, CB>(p, dst + 3 * Q::WB, to + 3 * Q::WB, p.x, kX, pre, n, last, -1, 0);
            }
            advance<G::kChans>(p, pre, step, clusters);
            ++fetched;
        }
        if constexpr (!Q::kBoxes) copy_commit();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);

    float2 carry = pair(0.f, 0.f);
    int it = 0, stage = 0;
    for (; cur.item < p.items; ++it) {
        const int c = cur.c0 + 2 * lc;
        const bool first = c < p.d, second = c + 1 < p.d;
        const long long s0 = (cur.b * p.H + cur.h) * p.d + c;
        if (cur.n0 == 0) carry = ld_state2(p.h_in, s0, first, second);
        if constexpr (Q::kBoxes) {
            wait_for(&full[stage][warp], it / S & 1, dead);
            landed += !dead;
        } else {
            copy_wait<S - 2>();
            __syncwarp();
        }
        const int n0 = cur.n0 + row0 + seg * R, left = cur.len - n0, t0 = left - 1;  // tokens t0, t0 - 1, ..
        uint8_t* const base = mine + stage * kWarps * NT * Q::WB + lc * 2 * sizeof(E);
        // boxes lie in ascending order of the tokens, copied rows in the scan's
        uint8_t* const from = base + (Q::kBoxes ? (G::kRows - 1 - seg * R) * Q::RB : Q::at(seg, 0));
        constexpr int RS = Q::kBoxes ? -Q::RB : Q::RB;
        float2 a[R], f[R], d[R], om[GATE == kGateMix ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 o, before = ld_pair(reinterpret_cast<const E*>(from + 2 * Q::WB + r * RS));
            gates<E, GATE>(ld_pair(reinterpret_cast<const E*>(from + r * RS)), a[r], o);
            d[r] = ld_pair(reinterpret_cast<const E*>(from + Q::WB + r * RS));
            if (t0 - r == 0) before = ld_state2(p.h0, s0, first, second);
            f[r] = ptx::mul2(a[r], before);
            if (GATE == kGateSigmoid) f[r] = ptx::mul2(f[r], o);
            if (GATE == kGateMix) {
                const float2 x = ld_pair(reinterpret_cast<const E*>(from + 3 * Q::WB + r * RS));
                f[r] = ptx::mul2(ptx::mul2(a[r], o), ptx::fma2(x, pair(-1.f, -1.f), before));
                om[r] = o;
            }
        }
        if (left < R) {  // positions behind the last: their rows are zeros
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r >= left) a[r] = pair(1.f, 1.f);
        }
        Map own = {a[0], ptx::mul2(a[0], d[0])};
#pragma unroll
        for (int r = 1; r < R; ++r) {
            own.H = ptx::mul2(a[r], ptx::add2(own.H, d[r]));
            own.A = ptx::mul2(own.A, a[r]);
        }
        __syncwarp();
        fetch(stage == 0 ? S - 1 : stage - 1);
        float2 g = scan_tile<LC>(sm, it, cs, rank, own, carry, dead);
        const long long x0 = cur.b * p.sb[kOut] + cur.h * p.sh[kOut] + c, g0 = cur.b * p.sb[kDg] + cur.h * p.sh[kDg] + c;
        const int low = cur.len - (cur.n0 + row0) - G::kRows;  // the warp's first token, if there are as many
        if (Q::kBoxes && low >= 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 dh = ptx::add2(d[r], g);
                g = ptx::mul2(a[r], dh);
                st_pair<E, true>(from + r * RS, 0, GATE == kGateMix ? ptx::mul2(om[GATE == kGateMix ? r : 0], dh) : dh,
                                 true);
                st_pair<E, true>(from + Q::WB + r * RS, 0, ptx::mul2(dh, f[r]), true);
            }
            ptx::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                const uint32_t src = ptx::smem_u32(mine + stage * kWarps * NT * Q::WB);
                tma_store_4d(&p.tm[kOut], src, cur.c0, low, (int)cur.h, (int)cur.b);
                tma_store_4d(&p.tm[kDg], src + Q::WB, cur.c0, low, (int)cur.h, (int)cur.b);
                ptx::bulk_commit();
            }
        } else if (first) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 dh = ptx::add2(d[r], g);
                g = ptx::mul2(a[r], dh);
                if (r < left) {
                    st_pair<E, Q::VS>(p.out, x0 + (t0 - r) * p.st[kOut],
                                      GATE == kGateMix ? ptx::mul2(om[GATE == kGateMix ? r : 0], dh) : dh, second);
                    st_pair<E, Q::VS>(p.dg, g0 + (t0 - r) * p.st[kDg], ptx::mul2(dh, f[r]), second);
                }
            }
        }
        if (cur.n0 + step >= cur.len) {
            if (p.h_out && rank == 0 && threadIdx.x < LC) st_state2(p.h_out, s0, carry, first, second);
            if (first)
                for (int t = cur.len + (rank * kWarps + warp) * G::kSegs + seg; t < p.T; t += cs * kWarps * G::kSegs) {
                    st_pair<E, Q::VS>(p.out, x0 + t * p.st[kOut], pair(0.f, 0.f), second);
                    st_pair<E, Q::VS>(p.dg, g0 + t * p.st[kDg], pair(0.f, 0.f), second);
                }
        }
        advance<G::kChans>(p, cur, step, clusters);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    if constexpr (Q::kBoxes) {
        for (; landed < fetched; ++landed)  // after a wait that ran out: the loads on their way, once more
            ptx::mbar_wait_bounded(ptx::smem_u32(&full[landed % S][warp]), landed / S & 1, kTimeoutCycles);
        if (lane == 0) ptx::bulk_wait_all();
    }
    if (cs > 1) {
        if (it == 0) cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
}

template <int VW>
__device__ __forceinline__ void ld_state(const float* s, long long off, float (&v)[VW]) {
#pragma unroll
    for (int i = 0; i < VW; ++i) v[i] = 0.f;
    if (!s) return;
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
    ld_state<VW>(p.h_in, s0, h);
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

// A kernel's shared memory beyond the default 48 KB, once per device.
bool allow_smem(const void* fn, int bytes) {
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

struct Shape {
    int lc, cs;
};

template <int R>
Shape shape_of(long long seqs, int d, int T, bool narrow) {
    Shape s = {32, 1};
    if (getenv("GLR_LC")) s.lc = atoi(getenv("GLR_LC"));
    if (getenv("GLR_CS")) s.cs = atoi(getenv("GLR_CS"));
    return s;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) ==
                            cudaSuccess &&
                        r == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiledFn>(q) : nullptr;
    }();
    return fn;
}

// Boxes of chans x rows of a [B,H,T,d] tensor; false where TMA does not take its address or strides.
bool encode_view(CUtensorMap* tm, const SeqView& v, const Params& p, long long B, int es, int chans, int rows) {
    const EncodeTiledFn fn = encode_fn();
    if (!fn || !seq_vec_ok(v, es, 16)) return false;
    const long long size[4] = {p.d, p.T, p.H, B}, st[3] = {v.st, v.sh, v.sb};
    cuuint64_t dims[4], strides[3];
    for (int i = 0; i < 4; ++i) {
        dims[i] = (cuuint64_t)size[i];
        if (i == 0) continue;
        if (size[i] > 1 && (st[i - 1] == 0 || st[i - 1] >= (1LL << 40) / es)) return false;
        strides[i - 1] = size[i] > 1 ? (cuuint64_t)st[i - 1] * es : 16;
    }
    const cuuint32_t box[4] = {(cuuint32_t)chans, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(tm, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, v.p, dims, strides,
              box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One call on its way to a kernel: the parameters and the views they were made of, by tensor index.
struct Call {
    Params p;
    SeqView view[6];
    bool used[6];
    long long B;
    int gate, es;
    bool bwd;
};

template <typename E, int LC, int R, int CB, int S>
int launch_scan_kernel(void (*fn)(Params, int), const Call& c, int cs, int tensors, cudaStream_t s) {
    Params p = c.p;
    p.tiles = (p.d + 2 * LC - 1) / (2 * LC);
    p.items = c.B * p.H * p.tiles;
    const int bytes = S * kWarps * tensors * Ring<E, LC, R, CB>::WB;
    if (p.items > kMaxGrid / cs) return 2;
    if (CB == kTma)
        for (int i = 0; i < 6; ++i)
            if (c.used[i] && !encode_view(&p.tm[i], c.view[i], p, c.B, c.es, 2 * LC, Geo<LC, R>::kRows)) return -1;
    if (!allow_smem(reinterpret_cast<const void*>(fn), bytes)) return 4;
    long long clusters = p.items;
    int per = getenv("GLR_PER") ? atoi(getenv("GLR_PER")) : 2;
    if (clusters > 152 * per / cs) clusters = 152 * per / cs;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
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
int launch_step(const Params& p, long long B, cudaStream_t s) {
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

template <typename E, int GATE, int LC, int CB>
int launch_lc(const Call& c, int cs, cudaStream_t s) {
    constexpr int RF = sizeof(E) == 2 ? 16 : 8, RB = sizeof(E) == 2 ? 8 : 4, S = 3;
    if (!c.bwd) return launch_scan_kernel<E, LC, RF, CB, S>(glr_fwd_kernel<E, GATE, LC, RF, CB, S>, c, cs, 2, s);
    return launch_scan_kernel<E, LC, RB, CB, S>(glr_bwd_kernel<E, GATE, LC, RB, CB, S>, c, cs, GATE == kGateMix ? 4 : 3, s);
}

template <typename E, int GATE>
int launch_gate(const Call& c, int cb, bool vec4, cudaStream_t s) {
    const Params& p = c.p;
    if (!c.bwd && p.T <= kStepTokens) return vec4 ? launch_step<E, GATE, 4>(p, c.B, s) : launch_step<E, GATE, 1>(p, c.B, s);
    const Shape sh = shape_of<16>(c.B * p.H, p.d, p.T, cb == 16);
    if (cb == 16) {
        const int st = sh.lc == 8    ? launch_lc<E, GATE, 8, kTma>(c, sh.cs, s)
                       : sh.lc == 16 ? launch_lc<E, GATE, 16, kTma>(c, sh.cs, s)
                                     : launch_lc<E, GATE, 32, kTma>(c, sh.cs, s);
        return st >= 0 ? st : launch_lc<E, GATE, 32, 16>(c, sh.cs, s);
    }
    if (cb >= 4) return launch_lc<E, GATE, 32, 4>(c, sh.cs, s);
    if constexpr (sizeof(E) == 2) return launch_lc<E, GATE, 32, 2>(c, sh.cs, s);
    return 2;
}

template <typename E>
int launch_type(const Call& c, int cb, bool vec4, cudaStream_t s) {
    switch (c.gate) {
        case kGateDecay: return launch_gate<E, kGateDecay>(c, cb, vec4, s);
        case kGateSigmoid: return launch_gate<E, kGateSigmoid>(c, cb, vec4, s);
        default: return launch_gate<E, kGateMix>(c, cb, vec4, s);
    }
}

int launch(Call& c, const GlrArgs& a, cudaStream_t s) {
    Params& p = c.p;
    p.H = (int)a.n.H, p.T = a.n.T, p.d = a.n.d, p.lengths = a.lengths;
    c.B = a.n.B, c.gate = a.gate, c.es = a.n.bf16 ? 2 : 4;
    int cb = 16;  // bytes that every access can move at a time
    bool vec4 = p.d % 4 == 0;
    for (int i = 0; i < 6; ++i) {
        const SeqView& v = c.view[i];
        c.used[i] = v.p != nullptr;
        p.sb[i] = v.sb, p.sh[i] = v.sh, p.st[i] = v.st;
        vec4 = vec4 && (!c.used[i] || seq_vec_ok(v, c.es, 4 * c.es));
        while (cb > c.es && (((long long)p.d * c.es) % cb != 0 || (c.used[i] && !seq_vec_ok(v, c.es, cb))))
            cb = cb == 16 ? 4 : cb / 2;
    }
    for (const void* st : {(const void*)p.h_in, (const void*)p.h0, (const void*)p.h_out})
        vec4 = vec4 && reinterpret_cast<uintptr_t>(st) % 16 == 0;
    return a.n.bf16 ? launch_type<bf16>(c, cb, vec4, s) : launch_type<float>(c, cb, vec4, s);
}

}  // namespace

int launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    Call c = {};
    c.view[kX] = a.x, c.view[kG] = a.g, c.view[kOut] = a.out;
    Params& p = c.p;
    p.x = a.x.p, p.g = a.g.p, p.out = a.out.p;
    p.h_in = a.h0, p.h_out = a.h_final;
    return launch(c, a, s);
}

int launch_glr_bwd(const GlrArgs& a, cudaStream_t s) {
    if (a.n.T == 0) {  // no tokens: the adjoint passes through
        if (!a.dh0) return 0;
        const size_t bytes = (size_t)a.n.B * a.n.H * a.n.d * sizeof(float);
        const cudaError_t e = a.dh_final ? cudaMemcpyAsync(a.dh0, a.dh_final, bytes, cudaMemcpyDeviceToDevice, s)
                                         : cudaMemsetAsync(a.dh0, 0, bytes, s);
        return e == cudaSuccess ? 0 : 4;
    }
    Call c = {};
    c.bwd = true;
    c.view[kX] = a.x, c.view[kG] = a.g, c.view[kOutIn] = a.out, c.view[kDout] = a.dout, c.view[kOut] = a.dx,
    c.view[kDg] = a.dg;
    Params& p = c.p;
    p.x = a.x.p, p.g = a.g.p, p.out_in = a.out.p, p.dout = a.dout.p, p.out = a.dx.p, p.dg = a.dg.p;
    p.h_in = a.dh_final, p.h0 = a.h0, p.h_out = a.dh0;
    return launch(c, a, s);
}

int glr_consume_timeout_flag(int* flag) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_glr_timeout_flag, sizeof(int)) != cudaSuccess) return 1;
    if (v && cudaMemcpyToSymbol(g_glr_timeout_flag, &zero, sizeof(int)) != cudaSuccess) return 1;
    *flag = v;
    return 0;
}

}  // namespace falcon
