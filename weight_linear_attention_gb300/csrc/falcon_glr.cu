// Gated linear recurrence, h_t = a_t h_{t-1} + u_t per channel, forward and backward.
//
// A span of tokens acts on the state as the affine map h -> A h + H with A the product of its a and H
// what the span makes of a zero state; maps compose as (A2, H2) o (A1, H1) = (A2 A1, A2 H1 + H2). The
// backward pass is the same scan over the tokens in reverse: with c the gradient that reaches the state
// before token t, dh_t = dout_t + c_{t+1} and c_t = a_t dh_t. Tokens are counted by their position in the
// scan's direction: position n is token n forward and token len - 1 - n backward.
//
// One pass over the data. A CTA works through tiles of kTile positions x 2 LC channels; a thread owns two
// channels of R consecutive positions. Tiles lie in a ring in shared memory, filled ahead by TMA
// (where addresses do not allow that, each warp copies its rows by cp.async, or through registers, and stores
// them itself). A warp evaluates the gates of its rows once into registers and reduces its tokens to their map;
// maps are composed over the warp (shuffles), the CTA (shared memory) and, for long sequences, the CTAs of a
// cluster that lie side by side along the tokens: each CTA sends its tile's map into its peers' shared memory
// (st.async, counted by an mbarrier there: no fence that would wait for the outputs on their way to memory), and
// every CTA composes them all in the same order, so that the state that enters the next cluster-wide tile is
// known everywhere without another exchange. Then each thread replays its tokens from its entering state into
// a buffer of their own, whence a TMA store takes them while the next tile is worked on. No scratch in global memory,
// no atomics on data; the order of every sum is fixed by sizes and alignment. Waits are bounded: one that runs out
// raises a flag (falcon_device_status) and is not repeated.
//
// What bounds it: 3 tensors' bytes per element forward, 5 or 6 backward, where there are tiles enough to hide
// the rest ([16,16,4096,64] bf16: 65 us forward, 92 % of the copy rate, 133 us backward, 90 %; 20 to 26 thread
// instructions per element, of which an SM has 33 at that rate). One long sequence ([1,12,131072,64] decay: 119 us,
// 75 %) is bound by the exchange (95 us without it), a training batch ([8,12,1024,64] mix: 12.2 us forward, 46 %, 18.1
// backward, 62 %) by filling and emptying three tiles per CTA (the same boxes without arithmetic: 8.5 us forward) and
// by arithmetic that does not overlap them (the other 3.7).

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "falcon_internal.h"
#include "falcon_seq.cuh"
#include "falcon_seq.h"
#include "sm103_ptx.cuh"

namespace falcon {
namespace {

using namespace seq;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
template <int LC>
constexpr int kMaxCluster = LC == 32 ? 8 : 16;  // CTAs of a cluster; a fuller tile has more maps to hold
constexpr int kStorer = 0, kLoader = 32;        // the threads that move boxes, in two warps: an issue takes ~130 cycles
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
    int items;                      // sequences x channel tiles
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
__device__ __forceinline__ Map shfl(const Map& m, int from) {
    Map r;
    r.A.x = __shfl_sync(0xffffffffu, m.A.x, from);
    r.A.y = __shfl_sync(0xffffffffu, m.A.y, from);
    r.H.x = __shfl_sync(0xffffffffu, m.H.x, from);
    r.H.y = __shfl_sync(0xffffffffu, m.H.y, from);
    return r;
}
// first `before`, then `m`
__device__ __forceinline__ Map compose(const Map& before, const Map& m) {
    return Map{mul2(m.A, before.A), fma2(m.A, before.H, m.H)};
}
__device__ __forceinline__ float2 apply(const Map& m, float2 h) { return fma2(m.A, h, m.H); }

template <int LC>
struct __align__(16) Maps {
    Map warp[2][kWarps][LC];
    Map cta[2][kMaxCluster<LC>][LC];
    float2 state[2][LC];  // behind a tile, where there is no cluster
    uint64_t ready[2];    // the maps of a cluster-wide tile have arrived
};

// Waits for a phase for at most about kTimeoutCycles; false when that runs out.
__device__ __forceinline__ bool bounded_wait(uint64_t* bar, uint32_t parity) {
    const uint32_t at = ptx::smem_u32(bar);
    if (ptx::mbar_try(at, parity)) return true;
    const long long t0 = clock64();
    do {
        if (ptx::mbar_try(at, parity)) return true;
    } while (clock64() - t0 <= kTimeoutCycles);
    return false;
}
// After a wait that ran out the thread skips its following ones: the outputs are lost, the flag tells, and the
// kernel comes to its end.
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, bool& dead) {
    if (!dead && !bounded_wait(bar, parity)) {
        dead = true;
        atomicExch(&g_glr_timeout_flag, 1);
    }
}

// The state that enters this thread's positions: composes the thread's map over the warp, the CTA and the
// cluster. `carry` is the state entering the cluster's tile (without a cluster only for an item's first tile,
// `fresh`; then sm.state has it) and, in a cluster, the one leaving it on return. Called by all scanning
// threads of the cluster the same number of times; `it` counts the calls.
// `behind_barrier` runs when every thread of the CTA has evaluated its gates and left the tile before this one.
template <int LC, typename F>
__device__ __forceinline__ float2 scan_tile(Maps<LC>& sm, int it, bool fresh, int cs, int rank, const Map& own,
                                            float2& carry, bool& dead, F behind_barrier) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, lc = lane % LC;
    const int buf = it & 1;
    Map inc = own;  // over the segments up to this one
#pragma unroll
    for (int o = LC; o < 32; o *= 2) {
        const Map m = shfl_up(inc, o);
        if (lane >= o) inc = compose(m, inc);
    }
    if (lane >= 32 - LC && warp < kWarps - 1) sm.warp[buf][warp][lc] = inc;
    Map exc = {pair(1.f, 1.f), pair(0.f, 0.f)};  // over the segments before it
    if (LC < 32) {
        const Map m = shfl_up(inc, LC);
        if (lane >= LC) exc = m;
    }
    // the state that was loaded for the first tile has arrived before any peer can know of this tile, and so
    // before the last tile's state may be written over it
    asm volatile("" ::"f"(carry.x), "f"(carry.y) : "memory");
    __syncthreads();
    behind_barrier();
    Map before = {pair(1.f, 1.f), pair(0.f, 0.f)};  // over the warps before this one
#pragma unroll
    for (int w0 = 0; w0 < kWarps - 1; w0 += 4) {
        if (w0 >= warp) break;
        Map m[4];
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (w0 + w < kWarps - 1) m[w] = sm.warp[buf][w0 + w][lc];  // those from `warp` on are not used
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (w0 + w < kWarps - 1 && w0 + w < warp) before = compose(before, m[w]);
    }
    float2 in = carry;  // the state entering this CTA's tile
    if (cs > 1) {
        const uint32_t bar = ptx::smem_u32(&sm.ready[buf]);
        // a thread whose wait ran out neither arrives again (the phase before may be open) nor sends any more: its
        // peers' waits run out as well, and all come to their end
        if (threadIdx.x == 0 && !dead) ptx::mbar_expect_tx(bar, cs * LC * (uint32_t)sizeof(Map));
        if (warp == kWarps - 1) {  // the CTA's map, to every peer: the lanes of a segment send to every kSegs-th
            Map all = compose(before, inc);
            if (LC < 32) all = shfl(all, 32 - LC + lc);
            const uint32_t at = ptx::smem_u32(&sm.cta[buf][rank][lc]);
            for (int r = dead ? cs : lane / LC; r < cs; r += 32 / LC) st_async4(peer(at, r), &all.A.x, peer(bar, r));
        }
        // A peer writes this buffer again two tiles on, after this CTA's map of the tile between has
        // reached it; that is sent behind the barrier above, so behind the reads below.
        wait_for(&sm.ready[buf], (it >> 1) & 1, dead);
#pragma unroll
        for (int r0 = 0; r0 < kMaxCluster<LC>; r0 += 4) {
            if (r0 >= cs) break;
            Map m[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) m[r] = sm.cta[buf][r0 + r][lc];  // those behind cs are not used
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (r0 + r >= cs) break;
                if (r0 + r == rank) in = carry;
                carry = apply(m[r], carry);
            }
        }
    } else if (!fresh) {
        in = sm.state[buf ^ 1][lc];
    }
    return apply(exc, apply(before, in));
}

// ---- the work list: items (sequence, channel tile) dealt to the clusters in turn, each of one or more tiles
struct Cursor {
    int item, b, h;
    int c0, n0, len;  // first channel; first position of the cluster's tile; positions in all
};
template <int CHANS>
__device__ __forceinline__ void enter(const Params& p, Cursor& c) {
    c.n0 = 0;
    if (c.item >= p.items) return;
    const int bh = c.item / p.tiles;
    c.c0 = (c.item - bh * p.tiles) * CHANS;
    c.b = bh / p.H;
    c.h = bh - c.b * p.H;
    c.len = length_of(p, c.b);
}
template <int CHANS>
__device__ __forceinline__ void advance(const Params& p, Cursor& c, int step, int clusters) {
    c.n0 += step;  // far below 2^31: the host refuses T >= 2^30
    if (c.n0 >= c.len) {
        c.item += clusters;  // so does this: fewer than 2^30 items
        enter<CHANS>(p, c);
    }
}

// A warp copies its rows of tensor k: position n of the scan is token `t0 + sign n` (shifted for the
// backward's outputs). CB bytes at a time; 2 bytes (odd addresses of bf16) go through registers. One pointer steps
// from row to row: with an address computed for every copy [8,12,3971,33] bf16 takes 103 us forward instead of 58.
template <typename E, int LC, int R, int CB>
__device__ __forceinline__ void copy_rows(const Params& p, uint32_t dst, uint8_t* dst_p, const void* base, int k,
                                          const Cursor& c, int n, int t0, int sign, int shift) {
    constexpr int RB = Geo<LC, R>::kChans * sizeof(E);
    constexpr int CPR = RB / CB, EPC = CB / sizeof(E);
    constexpr int RPS = CPR < 32 ? 32 / CPR : 1, CPL = CPR < 32 ? 1 : CPR / 32;  // rows a step, columns a lane
    const int lane = threadIdx.x & 31, row0 = lane / CPR % RPS, col0 = lane % CPR;
    int t = t0 + sign * (n + row0) + shift;
    const int left = c.len - n - row0;  // rows from this lane's first to the end
    const E* src = static_cast<const E*>(base) + ((long long)c.b * p.sb[k] + (long long)c.h * p.sh[k] + c.c0 +
                                                  t * p.st[k] + col0 * EPC);
    const long long inc = sign * RPS * p.st[k];
#pragma unroll
    for (int r = 0; r < Geo<LC, R>::kRows; r += RPS) {
        const bool row_in = r < left && t >= 0;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const bool in = row_in && c.c0 + (col0 + 32 * j) * EPC < p.d;
            const E* at = in ? src + 32 * j * EPC : static_cast<const E*>(base);
            const uint32_t o = (r + row0) * RB + (col0 + 32 * j) * CB;
            if constexpr (CB >= 4) copy_async<CB>(dst + o, at, in);
            else *reinterpret_cast<uint16_t*>(dst_p + o) = in ? *reinterpret_cast<const uint16_t*>(at) : (uint16_t)0;
        }
        src += inc;
        t += sign * RPS;
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

// A gate that keeps the state and adds nothing: a is 1 and 1 - a is 0, exactly.
template <int GATE>
__device__ __forceinline__ float2 idle_gate() {
    const float g = GATE == kGateDecay ? 0.f : __uint_as_float(0x7f800000u);
    return pair(g, g);
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

// How a kernel moves its rows: TMA boxes, or copies of 8, 4 or 2 bytes.
constexpr int kTma = 0;

template <typename E, int LC, int R, int CB>
struct Ring {
    using G = Geo<LC, R>;
    static constexpr bool kBoxes = CB == kTma;
    static constexpr bool VS = CB == kTma || CB == 2 * sizeof(E) || CB == 8;  // pairs of channels are aligned
    static constexpr int RB = G::kChans * sizeof(E);  // bytes of a row
    static constexpr int WB = G::kRows * RB;          // one warp's rows of one tensor
    static constexpr int TB = kWarps * WB;            // a tile's
    static constexpr int kBoxes1 = (G::kTile + 255) / 256, kBoxRows = G::kTile / kBoxes1;  // boxes of a tile, rows of a box
    static_assert(kBoxRows * kBoxes1 == G::kTile, "a tile is whole boxes");
    static __device__ __forceinline__ int at(int seg) { return seg * R * RB; }  // a segment's first row
};

// A tile's rows of one tensor, as boxes: from shared memory (`mine` its address) or to it.
template <typename Q>
__device__ __forceinline__ void load_tile(uint32_t to, const CUtensorMap* tm, const Cursor& c, int t, uint32_t bar) {
#pragma unroll
    for (int i = 0; i < Q::G::kTile; i += Q::kBoxRows)
        tma_load_4d(to + i * Q::RB, tm, c.c0, t + i, c.h, c.b, bar);
}
template <typename Q>
__device__ __forceinline__ void store_tile(const CUtensorMap* tm, uint32_t from, const Cursor& c, int t, int T) {
#pragma unroll
    for (int i = 0; i < Q::G::kTile; i += Q::kBoxRows)  // a box that reaches behind T is cut there
        if (t + i < T) tma_store_4d(tm, from + i * Q::RB, c.c0, t + i, c.h, c.b);
}

// Behind a tile: the thread with the last positions hands the state `h` on, or the cluster's rank 0 knows it
// as `carry`; after an item's last tile it goes to memory.
template <int LC>
__device__ __forceinline__ void leave_tile(const Params& p, Maps<LC>& sm, int it, int cs, int rank, const Cursor& c,
                                           int step, float2 h, float2 carry, bool first, bool second) {
    const int lc = threadIdx.x % LC;
    if (cs == 1 ? threadIdx.x < kThreads - LC : rank > 0 || threadIdx.x >= LC) return;
    if (cs == 1) sm.state[it & 1][lc] = h;
    if (p.h_out && c.n0 + step >= c.len)
        st_state2(p.h_out, ((long long)c.b * p.H + c.h) * p.d + c.c0 + 2 * lc, cs == 1 ? h : carry, first, second);
}

// What the threads that move boxes keep: a stage's boxes have landed (a barrier for each stage); the tile to be
// loaded next, the tile whose outputs lie in the ring.
template <int S>
struct Mover {
    uint64_t full[S];
    Cursor next, held;
    int loaded;
};
template <int LC, int S>
__device__ __forceinline__ void set_up(Mover<S>& mv, Maps<LC>& sm) {
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) ptx::mbar_init(ptx::smem_u32(&mv.full[i]), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&sm.ready[1]), 1);
        ptx::mbar_init_fence();
    }
    __syncthreads();
}

// Behind a wait that ran out nothing is loaded any more and nothing waited for, so what is still on its way into this
// CTA's shared memory is waited for at the end (each with the same limit). The boxes: each stage's last ones, whose
// phase no later one has followed.
template <int S>
__device__ __forceinline__ void drain_loads(Mover<S>& mv) {
    for (int i = max(mv.loaded - S, 0); i < mv.loaded; ++i) bounded_wait(&mv.full[i % S], i / S & 1);
}
// No CTA leaves while a peer may still write to it. Every map has been waited for, unless a wait ran out: then some may
// be on their way that no phase will count, and what is sent is given the time of a wait to arrive.
__device__ __forceinline__ void leave_cluster(int cs, bool dead) {
    if (cs == 1) return;
    cluster_arrive();
    cluster_wait();
    if (dead)
        for (const long long t0 = clock64(); clock64() - t0 <= kTimeoutCycles;) {
        }
}

template <typename E, int GATE, int LC, int R, int CB, int S>
__global__ void __launch_bounds__(kThreads, 2) glr_fwd_kernel(const __grid_constant__ Params p, int cs) {
    using G = Geo<LC, R>;
    using Q = Ring<E, LC, R, CB>;
    constexpr int SB = 2 * Q::TB;  // a stage: x, g
    __shared__ Maps<LC> sm;
    __shared__ Mover<S> mv;
    extern __shared__ __align__(128) uint8_t ring[];  // [S][x, g][warp][rows], then with boxes [2][out][warp][rows]
    constexpr int OB = Q::TB;
    uint8_t* const outs = ring + S * SB;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = lane / LC, lc = lane % LC;
    const int rank = blockIdx.x % cs, clusters = gridDim.x / cs, step = cs * G::kTile;
    const int row0 = (rank * kWarps + warp) * G::kRows;  // of the warp, in the cluster's tile
    set_up(mv, sm);
    if (cs > 1) cluster_arrive();
    ptx::pdl_wait();  // what the grids before this one wrote may be read from here on
    ptx::pdl_launch_dependents();
    Cursor pre = {};
    pre.item = blockIdx.x / cs;
    enter<G::kChans>(p, pre);

    // one thread fills the ring with boxes, another stores the outputs
    auto load = [&](int stage, const Cursor& c) {
        const uint32_t to = ptx::smem_u32(ring + stage * SB), bar = ptx::smem_u32(&mv.full[stage]);
        ptx::mbar_expect_tx(bar, SB);
        load_tile<Q>(to, &p.tm[kX], c, c.n0 + rank * G::kTile, bar);
        load_tile<Q>(to + Q::TB, &p.tm[kG], c, c.n0 + rank * G::kTile, bar);
    };
    auto store = [&](int tile, const Cursor& c) {
        store_tile<Q>(&p.tm[kOut], ptx::smem_u32(outs + (tile & 1) * OB), c, c.n0 + rank * G::kTile, p.T);
        ptx::bulk_commit();
    };
    if (Q::kBoxes && threadIdx.x == kLoader) {
        Cursor c = pre;
        int n = 0;
        for (; n < S && c.item < p.items; ++n) {
            load(n, c);
            advance<G::kChans>(p, c, step, clusters);
        }
        mv.next = c;
        mv.loaded = n;
    }

    Cursor cur = pre;
    auto fetch = [&](int stage) {
        if constexpr (!Q::kBoxes) {
            if (pre.item < p.items) {
                uint8_t* to = ring + stage * SB + warp * Q::WB;
                const int n = pre.n0 + row0;
                copy_rows<E, LC, R, CB>(p, ptx::smem_u32(to), to, p.x, kX, pre, n, 0, 1, 0);
                copy_rows<E, LC, R, CB>(p, ptx::smem_u32(to) + Q::TB, to + Q::TB, p.g, kG, pre, n, 0, 1, 0);
                advance<G::kChans>(p, pre, step, clusters);
            }
            copy_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    if (cs > 1) cluster_wait();  // every peer runs and has set up its mbarriers

    float2 carry = pair(0.f, 0.f);
    bool dead = false;
    int it = 0, stage = 0;
    for (; cur.item < p.items; ++it) {
        const int c = cur.c0 + 2 * lc;
        const bool first = c < p.d, second = c + 1 < p.d;
        if (cur.n0 == 0) carry = ld_state2(p.h_in, ((long long)cur.b * p.H + cur.h) * p.d + c, first, second);
        if constexpr (Q::kBoxes) {
            wait_for(&mv.full[stage], it / S & 1, dead);
        } else {
            copy_wait<S - 2>();
            __syncwarp();
        }
        const int t0 = cur.n0 + row0 + seg * R, left = cur.len - t0;  // this thread's rows inside the sequence
        uint8_t* const from = ring + stage * SB + warp * Q::WB + Q::at(seg) + lc * 2 * sizeof(E);
        const bool whole = left >= R;
        if (!whole) {  // rows behind the end change nothing, whatever they hold
#pragma unroll 1
            for (int r = max(left, 0); r < R; ++r) {
                st_pair<E, true>(from + r * Q::RB, 0, pair(0.f, 0.f), true);
                st_pair<E, true>(from + Q::TB + r * Q::RB, 0, idle_gate<GATE>(), true);
            }
            if (Q::kBoxes) ptx::fence_async_smem();  // before boxes overwrite it
        }
        float2 a[R], u[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float2 x = ld_pair(reinterpret_cast<const E*>(from + r * Q::RB));
            float2 om;
            gates<E, GATE>(ld_pair(reinterpret_cast<const E*>(from + Q::TB + r * Q::RB)), a[r], om);
            u[r] = GATE == kGateMix ? mul2(om, x) : x;
        }
        Map own = {a[0], u[0]};
#pragma unroll
        for (int r = 1; r < R; ++r) own = compose(own, Map{a[r], u[r]});
        __syncwarp();  // every lane has read the stage before this one, which is filled again
        fetch(stage == 0 ? S - 1 : stage - 1);
        if (Q::kBoxes && threadIdx.x == kStorer) ptx::bulk_wait_read<0>();  // this tile's outputs go where those two back lay
        float2 h = scan_tile<LC>(sm, it, cur.n0 == 0, cs, rank, own, carry, dead, [&] {
            if (!Q::kBoxes || dead) return;
            if (threadIdx.x == kStorer) {
                if (it > 0) store(it - 1, mv.held);
                mv.held = cur;
            }
            if (threadIdx.x == kLoader && mv.next.item < p.items) {  // into the stage that every warp has read
                Cursor n = mv.next;
                load(stage, n);
                advance<G::kChans>(p, n, step, clusters);
                mv.next = n;
                ++mv.loaded;
            }
        });
        if constexpr (Q::kBoxes) {
            uint8_t* const to = outs + (it & 1) * OB + warp * Q::WB + Q::at(seg) + lc * 2 * sizeof(E);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = fma2(a[r], h, u[r]);
                st_pair<E, true>(to + r * Q::RB, 0, h, true);
            }
            if (!whole) {
#pragma unroll 1
                for (int r = max(left, 0); r < R; ++r) st_pair<E, true>(to + r * Q::RB, 0, pair(0.f, 0.f), true);
            }
            ptx::fence_async_smem();
        } else if (first) {
            const long long o0 = cur.b * p.sb[kOut] + cur.h * p.sh[kOut] + c;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = fma2(a[r], h, u[r]);
                if (r < left) st_pair<E, Q::VS>(p.out, o0 + (t0 + r) * p.st[kOut], h, second);
            }
        }
        leave_tile<LC>(p, sm, it, cs, rank, cur, step, h, carry, first, second);
        if (cur.n0 + step >= cur.len) {
            // zeros behind the end; boxes have reached the end of the cluster's tile
            const long long o0 = cur.b * p.sb[kOut] + cur.h * p.sh[kOut] + c;
            if (first)
                for (int t = (Q::kBoxes ? cur.n0 + step : cur.len) + (rank * kWarps + warp) * G::kSegs + seg; t < p.T;
                     t += cs * kWarps * G::kSegs)
                    st_pair<E, Q::VS>(p.out, o0 + t * p.st[kOut], pair(0.f, 0.f), second);
        }
        advance<G::kChans>(p, cur, step, clusters);
        stage = stage == S - 1 ? 0 : stage + 1;
    }
    if constexpr (Q::kBoxes) {
        __syncthreads();
        if (threadIdx.x == kStorer) {
            if (it > 0 && !dead) store(it - 1, mv.held);
            ptx::bulk_wait_all();
        }
        if (threadIdx.x == kLoader && dead) drain_loads(mv);
    }
    leave_cluster(cs, dead);
}

template <typename E, int GATE, int LC, int R, int CB, int S>
__global__ void __launch_bounds__(kThreads, 2) glr_bwd_kernel(const __grid_constant__ Params p, int cs) {
    using G = Geo<LC, R>;
    using Q = Ring<E, LC, R, CB>;
    constexpr int NT = GATE == kGateMix ? 4 : 3, SB = NT * Q::TB;  // a stage: g, dout, out, x
    __shared__ Maps<LC> sm;
    __shared__ Mover<S> mv;
    extern __shared__ __align__(128) uint8_t ring[];  // [S][tensor][warp][rows], then with boxes [2][dx, dg][..][..]
    constexpr int OB = 2 * Q::TB;
    uint8_t* const outs = ring + S * SB;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = lane / LC, lc = lane % LC;
    const int rank = blockIdx.x % cs, clusters = gridDim.x / cs, step = cs * G::kTile;
    const int row0 = (rank * kWarps + warp) * G::kRows;
    set_up(mv, sm);
    if (cs > 1) cluster_arrive();
    ptx::pdl_wait();  // what the grids before this one wrote may be read from here on
    ptx::pdl_launch_dependents();
    Cursor pre = {};
    pre.item = blockIdx.x / cs;
    enter<G::kChans>(p, pre);
    // the first token of a CTA's tile, whose rows lie in ascending order; negative where the sequence begins
    // inside the tile
    auto low = [&](const Cursor& c) { return c.len - (c.n0 + rank * G::kTile) - G::kTile; };

    // one thread fills the ring with boxes, another stores the outputs
    auto load = [&](int stage, const Cursor& c) {
        const uint32_t to = ptx::smem_u32(ring + stage * SB), bar = ptx::smem_u32(&mv.full[stage]);
        const int t = low(c);
        ptx::mbar_expect_tx(bar, SB);
        load_tile<Q>(to, &p.tm[kG], c, t, bar);
        load_tile<Q>(to + Q::TB, &p.tm[kDout], c, t, bar);
        load_tile<Q>(to + 2 * Q::TB, &p.tm[kOutIn], c, t - 1, bar);  // h before the token
        if (GATE == kGateMix) load_tile<Q>(to + 3 * Q::TB, &p.tm[kX], c, t, bar);
    };
    auto store = [&](int tile, const Cursor& c) {
        if (low(c) < 0) return;  // the warps have stored such a tile themselves
        const uint32_t from = ptx::smem_u32(outs + (tile & 1) * OB);
        store_tile<Q>(&p.tm[kOut], from, c, low(c), p.T);
        store_tile<Q>(&p.tm[kDg], from + Q::TB, c, low(c), p.T);
        ptx::bulk_commit();
    };
    if (Q::kBoxes && threadIdx.x == kLoader) {
        Cursor c = pre;
        int n = 0;
        for (; n < S && c.item < p.items; ++n) {
            load(n, c);
            advance<G::kChans>(p, c, step, clusters);
        }
        mv.next = c;
        mv.loaded = n;
    }

    Cursor cur = pre;
    auto fetch = [&](int stage) {
        if constexpr (!Q::kBoxes) {
            if (pre.item < p.items) {
                uint8_t* to = ring + stage * SB + warp * Q::WB;
                const uint32_t dst = ptx::smem_u32(to);
                const int n = pre.n0 + row0, last = pre.len - 1;
                copy_rows<E, LC, R, CB>(p, dst, to, p.g, kG, pre, n, last, -1, 0);
                copy_rows<E, LC, R, CB>(p, dst + Q::TB, to + Q::TB, p.dout, kDout, pre, n, last, -1, 0);
                copy_rows<E, LC, R, CB>(p, dst + 2 * Q::TB, to + 2 * Q::TB, p.out_in, kOutIn, pre, n, last, -1, -1);
                if (GATE == kGateMix)
                    copy_rows<E, LC, R, CB>(p, dst + 3 * Q::TB, to + 3 * Q::TB, p.x, kX, pre, n, last, -1, 0);
                advance<G::kChans>(p, pre, step, clusters);
            }
            copy_commit();
        }
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) fetch(i);
    if (cs > 1) cluster_wait();

    float2 carry = pair(0.f, 0.f);
    bool dead = false;
    int it = 0, stage = 0;
    for (; cur.item < p.items; ++it) {
        const int c = cur.c0 + 2 * lc;
        const bool first = c < p.d, second = c + 1 < p.d;
        if (cur.n0 == 0) carry = ld_state2(p.h_in, ((long long)cur.b * p.H + cur.h) * p.d + c, first, second);
        if constexpr (Q::kBoxes) {
            wait_for(&mv.full[stage], it / S & 1, dead);
        } else {
            copy_wait<S - 2>();
            __syncwarp();
        }
        const int n0 = cur.n0 + row0 + seg * R, left = cur.len - n0, t0 = left - 1;  // tokens t0, t0 - 1, ..
        // boxes lie in ascending order of the tokens, copied rows in the scan's
        uint8_t* const from = ring + stage * SB + lc * 2 * sizeof(E) +
                              (Q::kBoxes ? (G::kTile - 1 - warp * G::kRows - seg * R) * Q::RB
                                         : warp * Q::WB + Q::at(seg));
        constexpr int RS = Q::kBoxes ? -Q::RB : Q::RB;
        const bool whole = left >= R;
        if (!whole) {  // positions behind the last: dout and out read as zeros there
#pragma unroll 1
            for (int r = max(left, 0); r < R; ++r) st_pair<E, true>(from + r * RS, 0, idle_gate<GATE>(), true);
            if (Q::kBoxes) ptx::fence_async_smem();
        }
        float2 a[R], f[R], d[R], om[GATE == kGateMix ? R : 1];
        Map own = {pair(1.f, 1.f), pair(0.f, 0.f)};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float2 o, before = ld_pair(reinterpret_cast<const E*>(from + 2 * Q::TB + r * RS));
            gates<E, GATE>(ld_pair(reinterpret_cast<const E*>(from + r * RS)), a[r], o);
            if (GATE == kGateMix)
                before = fma2(ld_pair(reinterpret_cast<const E*>(from + 3 * Q::TB + r * RS)), pair(-1.f, -1.f), before);
            f[r] = mul2(a[r], before);
            if (GATE != kGateDecay) f[r] = mul2(f[r], o);
            if (GATE == kGateMix) om[r] = o;
            d[r] = ld_pair(reinterpret_cast<const E*>(from + Q::TB + r * RS));
            own.H = mul2(a[r], add2(own.H, d[r]));
            own.A = mul2(own.A, a[r]);
        }
        if (t0 >= 0 && t0 < R) {  // the sequence's first token: h0 comes before it
            const float2 h0 = ld_state2(p.h0, ((long long)cur.b * p.H + cur.h) * p.d + c, first, second);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r != t0) continue;
                float2 ga, o, before = h0;
                gates<E, GATE>(ld_pair(reinterpret_cast<const E*>(from + r * RS)), ga, o);
                if (GATE == kGateMix)
                    before = fma2(ld_pair(reinterpret_cast<const E*>(from + 3 * Q::TB + r * RS)), pair(-1.f, -1.f),
                                       before);
                f[r] = mul2(ga, before);
                if (GATE != kGateDecay) f[r] = mul2(f[r], o);
            }
        }
        __syncwarp();
        fetch(stage == 0 ? S - 1 : stage - 1);
        if (Q::kBoxes && threadIdx.x == kStorer) ptx::bulk_wait_read<0>();
        float2 g = scan_tile<LC>(sm, it, cur.n0 == 0, cs, rank, own, carry, dead, [&] {
            if (!Q::kBoxes || dead) return;
            if (threadIdx.x == kStorer) {
                if (it > 0) store(it - 1, mv.held);
                mv.held = cur;
            }
            if (threadIdx.x == kLoader && mv.next.item < p.items) {  // into the stage that every warp has read
                Cursor n = mv.next;
                load(stage, n);
                advance<G::kChans>(p, n, step, clusters);
                mv.next = n;
                ++mv.loaded;
            }
        });
        const long long x0 = cur.b * p.sb[kOut] + cur.h * p.sh[kOut] + c, g0 = cur.b * p.sb[kDg] + cur.h * p.sh[kDg] + c;
        const bool boxes = Q::kBoxes && low(cur) >= 0;
        if (boxes) {
            uint8_t* const to = outs + (it & 1) * OB + lc * 2 * sizeof(E) + (G::kTile - 1 - warp * G::kRows - seg * R) * Q::RB;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 dh = add2(d[r], g);
                g = mul2(a[r], dh);
                st_pair<E, true>(to + r * RS, 0, GATE == kGateMix ? mul2(om[GATE == kGateMix ? r : 0], dh) : dh,
                                 true);
                st_pair<E, true>(to + Q::TB + r * RS, 0, mul2(dh, f[r]), true);
            }
            ptx::fence_async_smem();
        } else if (first) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 dh = add2(d[r], g);
                g = mul2(a[r], dh);
                if (r < left) {
                    st_pair<E, Q::VS>(p.out, x0 + (t0 - r) * p.st[kOut],
                                      GATE == kGateMix ? mul2(om[GATE == kGateMix ? r : 0], dh) : dh, second);
                    st_pair<E, Q::VS>(p.dg, g0 + (t0 - r) * p.st[kDg], mul2(dh, f[r]), second);
                }
            }
        }
        leave_tile<LC>(p, sm, it, cs, rank, cur, step, g, carry, first, second);
        if (cur.n0 + step >= cur.len) {
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
        __syncthreads();
        if (threadIdx.x == kStorer) {
            if (it > 0 && !dead) store(it - 1, mv.held);
            ptx::bulk_wait_all();
        }
        if (threadIdx.x == kLoader && dead) drain_loads(mv);
    }
    leave_cluster(cs, dead);
}

// ---- few tokens (a decoding step, short sequences): one thread per VW channels walks them, its rows loaded U at
// a time
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

constexpr int kWalkThreads = 128;

// The channels of one walking thread.
struct Lane {
    long long b, h, s0;  // s0: the state's offset
    int c;
};
template <int VW>
__device__ __forceinline__ Lane lane_of(const Params& p, long long i) {
    const int per = p.d / VW;
    const long long bh = i / per;
    Lane l;
    l.c = (int)(i - bh * per) * VW;
    l.b = bh / p.H;
    l.h = bh - l.b * p.H;
    l.s0 = bh * p.d + l.c;
    return l;
}
__device__ __forceinline__ long long offset(const Params& p, const Lane& l, int k) {
    return l.b * p.sb[k] + l.h * p.sh[k] + l.c;
}

template <typename E, int GATE, int VW, int U>
__global__ void __launch_bounds__(kWalkThreads) glr_walk_kernel(const __grid_constant__ Params p, long long lanes) {
    // a decoding loop's previous step wrote the state: wait for the grid before this one
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * kWalkThreads + threadIdx.x;
    if (i >= lanes) return;
    const Lane l = lane_of<VW>(p, i);
    const long long x0 = offset(p, l, kX), g0 = offset(p, l, kG), o0 = offset(p, l, kOut);
    const int len = length_of(p, l.b);
    float h[VW];
    ld_state<VW>(p.h_in, l.s0, h);
    for (int t0 = 0; t0 < p.T; t0 += U) {
        Pack<E, VW> px[U], pg[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t0 + u < len) {
                px[u] = load<E, VW>(p.x, x0 + (t0 + u) * p.st[kX]);
                pg[u] = load<E, VW>(p.g, g0 + (t0 + u) * p.st[kG]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t0 + u >= p.T) break;
            Pack<E, VW> po;
            zero(po);
            if (t0 + u < len) {
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    float ga, gc = 1.f;
                    if (GATE == kGateDecay) ga = decay_exp(elem(pg[u], j));
                    else logistic(elem(pg[u], j), ga, gc);
                    h[j] = fmaf(ga, h[j], GATE == kGateMix ? gc * elem(px[u], j) : elem(px[u], j));
                }
                pack(po, h);
            }
            store(p.out, o0 + (t0 + u) * p.st[kOut], po);
        }
    }
    if (p.h_out) st_state<VW>(p.h_out, l.s0, h);
}

template <typename E, int GATE, int VW, int U>
__global__ void __launch_bounds__(kWalkThreads) glr_walk_bwd_kernel(const __grid_constant__ Params p, long long lanes) {
    ptx::pdl_wait();
    ptx::pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * kWalkThreads + threadIdx.x;
    if (i >= lanes) return;
    const Lane l = lane_of<VW>(p, i);
    const long long x0 = offset(p, l, kX), g0 = offset(p, l, kG), h0 = offset(p, l, kOutIn), d0 = offset(p, l, kDout),
                    ox = offset(p, l, kOut), og = offset(p, l, kDg);
    const int len = length_of(p, l.b);
    float c[VW];
    ld_state<VW>(p.h_in, l.s0, c);
    for (int t1 = p.T - 1; t1 >= 0; t1 -= U) {
        Pack<E, VW> px[GATE == kGateMix ? U : 1], pg[U], ph[U], pd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t1 - u;
            if (t >= 0 && t < len) {
                pg[u] = load<E, VW>(p.g, g0 + t * p.st[kG]);
                pd[u] = load<E, VW>(p.dout, d0 + t * p.st[kDout]);
                if (t > 0) ph[u] = load<E, VW>(p.out_in, h0 + (t - 1) * p.st[kOutIn]);
                if (GATE == kGateMix) px[GATE == kGateMix ? u : 0] = load<E, VW>(p.x, x0 + t * p.st[kX]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t1 - u;
            if (t < 0) break;
            Pack<E, VW> po, pq;
            zero(po);
            zero(pq);
            if (t < len) {
                float before[VW], dx[VW], dg[VW];
#pragma unroll
                for (int j = 0; j < VW; ++j) before[j] = elem(ph[u], j);
                if (t == 0) ld_state<VW>(p.h0, l.s0, before);
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                    float ga, gc = 1.f;
                    if (GATE == kGateDecay) ga = decay_exp(elem(pg[u], j));
                    else logistic(elem(pg[u], j), ga, gc);
                    float f = ga * (GATE == kGateMix ? before[j] - elem(px[GATE == kGateMix ? u : 0], j) : before[j]);
                    if (GATE != kGateDecay) f *= gc;
                    const float dh = elem(pd[u], j) + c[j];
                    dx[j] = GATE == kGateMix ? gc * dh : dh;
                    dg[j] = dh * f;
                    c[j] = ga * dh;
                }
                pack(po, dx);
                pack(pq, dg);
            }
            store(p.out, ox + t * p.st[kOut], po);
            store(p.dg, og + t * p.st[kDg], pq);
        }
    }
    if (p.h_out) st_state<VW>(p.h_out, l.s0, c);
}

constexpr long long kMaxGrid = 0x7fffffffLL;
constexpr int kSms = 152;
constexpr int kMaxDevices = 64;

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
};

// What is known of one kernel on each device: its shared memory allowed, and how many clusters of each size run
// at once (0: not asked yet). Both are the same whoever asks first.
struct KernelInfo {
    std::atomic<int> ready[kMaxDevices];
    std::atomic<int> clusters[kMaxDevices][17];
};

// With programmatic stream serialisation: a call's launch and set-up overlap the end of the one before it.
void describe(cudaLaunchConfig_t* cfg, cudaLaunchAttribute (&at)[2], int cs, int bytes) {
    cfg->blockDim = dim3(kThreads);
    cfg->dynamicSmemBytes = bytes;
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = cs;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = at;
    cfg->numAttrs = 2;
}

// Clusters of cs CTAs that run at once on device `dev`, two CTAs an SM; 0 on an error.
template <typename Fn>
int resident(Fn fn, KernelInfo& info, int dev, int cs, int bytes) {
    if (!info.ready[dev].load(std::memory_order_acquire)) {
        const void* f = reinterpret_cast<const void*>(fn);
        if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess ||
            cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return 0;
        info.ready[dev].store(1, std::memory_order_release);
    }
    int n = info.clusters[dev][cs].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[2];
        cfg.gridDim = dim3(cs);
        describe(&cfg, at, cs, bytes);
        if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            (void)cudaGetLastError();  // a size that does not run is no error of the call's
            return 0;
        }
        info.clusters[dev][cs].store(n, std::memory_order_relaxed);
    }
    return n;
}

// A launch of one of the tile shapes, and what it would cost (sixteenths of a microsecond).
struct Plan {
    int cs = 0;           // 0: the kernel cannot run
    long long clusters = 0, cost = 0;
};

// The cluster size for a tile shape. A sequence's tiles are dealt to the cs CTAs of its cluster; every round of
// cluster-wide tiles lasts as long as a tile on the fullest SM, and in a cluster the exchange longer. Measured, in
// sixteenths of a microsecond (bf16; fp32 tiles, of half the elements, are a little quicker): a tile takes 16
// forward and 18 backward where each SM holds one CTA, 28 to 31 and 25 to 26 (the narrower the more: a box moves a
// row at a time) where one holds two; the exchange 6, and 7 and 12 where no second CTA covers it.
template <int LC, bool BWD, bool F32, typename Fn>
Plan plan_for(Fn fn, KernelInfo& info, int dev, int bytes, long long items, int T, int rows) {
    constexpr int kAlone = F32 ? 14 : BWD ? 18 : 16, kExchangeAlone = BWD ? 12 : 7, kExchange = 6;
    constexpr int kShared = (BWD ? LC == 8 ? 26 : 25 : LC == 8 ? 31 : LC == 16 ? 29 : 28) - (F32 ? 2 : 0);
    Plan best;
    const long long tiles = ((long long)T + rows - 1) / rows;
    for (int cs = 1; cs <= kMaxCluster<LC> && cs <= tiles; ++cs) {
        const long long most = resident(fn, info, dev, cs, bytes);
        if (most == 0) continue;
        const long long clusters = items < most ? items : most;
        const long long rounds = (items + clusters - 1) / clusters * ((tiles + cs - 1) / cs);
        const bool alone = clusters * cs <= kSms;
        const long long cost =
            rounds * ((alone ? kAlone : kShared) + (cs == 1 ? 0 : alone ? kExchangeAlone : kExchange));
        if (best.cs == 0 || cost < best.cost) {
            best.cs = cs;
            best.clusters = clusters;
            best.cost = cost;
        }
    }
    return best;
}

template <int LC>
bool items_of(const Call& c, int* tiles, long long* items) {
    *tiles = (int)(((long long)c.p.d + 2 * LC - 1) / (2 * LC));
    *items = c.B * c.p.H * *tiles;
    return *items < 1LL << 30;
}

// R: rows of a thread. Forward 16 (two fp32 values a row and channel stay in registers), backward 8 (four); half
// for fp32, whose tiles take twice the shared memory. In the narrow tiles one less: the segments of a warp then
// start in different banks (118 against 141 us for [1,12,131072,64] bf16 in tiles of 16 channels).
template <typename E, int LC, bool BWD>
constexpr int kR = (BWD ? 8 : 16) / (int)(sizeof(E) / 2) - (LC < 32 && sizeof(E) == 2 ? 1 : 0);

template <typename E, int GATE, int LC, int CB, bool BWD>
struct Kernel {
    static constexpr int R = kR<E, LC, BWD>;
    using Q = Ring<E, LC, R, CB>;
    // two tiles of inputs and two of outputs (boxes), or three of inputs: about 96 KB, two CTAs an SM
    static constexpr int kStages = Q::kBoxes ? 2 : 3;
    static constexpr int kBytes =
        (kStages * (BWD ? (GATE == kGateMix ? 4 : 3) : 2) + (Q::kBoxes ? (BWD ? 4 : 2) : 0)) * Q::TB;
    static KernelInfo& info() {
        static KernelInfo k;
        return k;
    }
    static void (*fn())(Params, int) {
        if constexpr (BWD) return glr_bwd_kernel<E, GATE, LC, R, CB, kStages>;
        else return glr_fwd_kernel<E, GATE, LC, R, CB, kStages>;
    }
    static Plan plan(const Call& c, int dev) {
        int tiles;
        long long items;
        if (!items_of<LC>(c, &tiles, &items)) return Plan{};
        return plan_for<LC, BWD, sizeof(E) == 4>(fn(), info(), dev, kBytes, items, c.p.T, Q::G::kTile);
    }
    // 0, a status, or -1: TMA does not take these tensors
    static int launch(const Call& c, const Plan& plan, cudaStream_t s) {
        Params p = c.p;
        long long items;
        if (!items_of<LC>(c, &p.tiles, &items)) return 2;
        p.items = (int)items;
        if (CB == kTma)
            for (int i = 0; i < 6; ++i)
                if (c.used[i] && !encode_view(&p.tm[i], c.view[i], p, c.B, c.es, 2 * LC, Q::kBoxRows)) return -1;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute at[2];
        describe(&cfg, at, plan.cs, kBytes);
        cfg.gridDim = dim3((unsigned)(plan.clusters * plan.cs));
        cfg.stream = s;
        return cudaLaunchKernelEx(&cfg, fn(), p, plan.cs) == cudaSuccess ? 0 : 4;
    }
};

// U: rows loaded at a time.
template <typename E, int GATE, int VW, int U, bool BWD>
int launch_walk_rows(const Call& c, cudaStream_t s) {
    const long long lanes = c.B * c.p.H * (c.p.d / VW), blocks = (lanes + kWalkThreads - 1) / kWalkThreads;
    if (blocks > kMaxGrid) return 2;
    void (*fn)(Params, long long);
    if constexpr (BWD) fn = glr_walk_bwd_kernel<E, GATE, VW, U>;
    else fn = glr_walk_kernel<E, GATE, VW, U>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kWalkThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, c.p, lanes) == cudaSuccess ? 0 : 4;
}

template <typename E, int GATE, int VW, bool BWD>
int launch_walk(const Call& c, cudaStream_t s) {
    if (c.p.T == 1) return launch_walk_rows<E, GATE, VW, 1, BWD>(c, s);
    return launch_walk_rows<E, GATE, VW, VW == 1 || !BWD ? 8 : 4, BWD>(c, s);
}

// Whether walking costs less than the plan. A token takes a walking thread 0.25 us forward and 0.63 us backward
// (half a load's latency, and a third of one's of four tensors) up to about 40,000 threads on the GPU, then in
// proportion to them; a plan has about 1 us of filling and emptying to it.
template <bool BWD>
bool walks(const Call& c, int vw, const Plan& plan) {
    const long long lanes = c.B * c.p.H * (c.p.d / vw);
    const long long token = BWD ? std::max(10LL, lanes / 4700) : std::max(4LL, lanes / 9300);
    return c.p.T <= 256 && c.p.T * token <= plan.cost + 16;
}

// The plan's kernel, unless walking is cheaper.
template <typename K, bool BWD, typename Walk>
int launch_copied(const Call& c, int dev, int vw, Walk walk, cudaStream_t s) {
    const Plan k = K::plan(c, dev);
    if (k.cs == 0) return 4;
    return walks<BWD>(c, vw, k) ? walk() : K::launch(c, k, s);
}

template <typename E, int GATE, bool BWD>
int launch_scan(const Call& c, int cb, int vw, cudaStream_t s) {
    auto walk = [&] { return vw == 4 ? launch_walk<E, GATE, 4, BWD>(c, s) : launch_walk<E, GATE, 1, BWD>(c, s); };
    if (c.p.T <= 8) return walk();
    int dev = 0, tiles;
    long long items;
    if (!items_of<32>(c, &tiles, &items)) return 2;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 4;
    if (cb == 16) {
        // narrower tiles split the channels where sequences are few and long
        using Wide = Kernel<E, GATE, 32, kTma, BWD>;
        using Half = Kernel<E, GATE, 16, kTma, BWD>;
        using Narrow = Kernel<E, GATE, 8, kTma, BWD>;
        const Plan plans[3] = {Wide::plan(c, dev), Half::plan(c, dev), Narrow::plan(c, dev)};
        int k = 0;
        for (int i = 1; i < 3; ++i)
            if (plans[i].cs > 0 && (plans[k].cs == 0 || plans[i].cost < plans[k].cost)) k = i;
        if (plans[k].cs == 0) return 4;
        if (walks<BWD>(c, vw, plans[k])) return walk();
        const int st = k == 0   ? Wide::launch(c, plans[0], s)
                       : k == 1 ? Half::launch(c, plans[1], s)
                                : Narrow::launch(c, plans[2], s);
        if (st >= 0) return st;
        cb = 8;
    }
    if (cb == 8) return launch_copied<Kernel<E, GATE, 32, 8, BWD>, BWD>(c, dev, vw, walk, s);
    if (cb == 4) return launch_copied<Kernel<E, GATE, 32, 4, BWD>, BWD>(c, dev, vw, walk, s);
    if constexpr (sizeof(E) == 2) return launch_copied<Kernel<E, GATE, 32, 2, BWD>, BWD>(c, dev, vw, walk, s);
    return 4;
}

template <typename E, bool BWD>
int launch_gate(const Call& c, int cb, int vw, cudaStream_t s) {
    switch (c.gate) {
        case kGateDecay: return launch_scan<E, kGateDecay, BWD>(c, cb, vw, s);
        case kGateSigmoid: return launch_scan<E, kGateSigmoid, BWD>(c, cb, vw, s);
        default: return launch_scan<E, kGateMix, BWD>(c, cb, vw, s);
    }
}

template <bool BWD>
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
            cb /= 2;
    }
    for (const void* st : {(const void*)p.h_in, (const void*)p.h0, (const void*)p.h_out})
        vec4 = vec4 && reinterpret_cast<uintptr_t>(st) % 16 == 0;
    const int vw = vec4 ? 4 : 1;
    return a.n.bf16 ? launch_gate<bf16, BWD>(c, cb, vw, s) : launch_gate<float, BWD>(c, cb, vw, s);
}

}  // namespace

int launch_glr_fwd(const GlrArgs& a, cudaStream_t s) {
    Call c = {};
    c.view[kX] = a.x, c.view[kG] = a.g, c.view[kOut] = a.out;
    Params& p = c.p;
    p.x = a.x.p, p.g = a.g.p, p.out = a.out.p;
    p.h_in = a.h0, p.h_out = a.h_final;
    return launch<false>(c, a, s);
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
    c.view[kX] = a.x, c.view[kG] = a.g, c.view[kOutIn] = a.out, c.view[kDout] = a.dout, c.view[kOut] = a.dx,
    c.view[kDg] = a.dg;
    Params& p = c.p;
    p.x = a.x.p, p.g = a.g.p, p.out_in = a.out.p, p.dout = a.dout.p, p.out = a.dx.p, p.dg = a.dg.p;
    p.h_in = a.dh_final, p.h0 = a.h0, p.h_out = a.dh0;
    return launch<true>(c, a, s);
}

int glr_consume_timeout_flag(int* flag) {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_glr_timeout_flag, sizeof(int)) != cudaSuccess) return 1;
    if (v && cudaMemcpyToSymbol(g_glr_timeout_flag, &zero, sizeof(int)) != cudaSuccess) return 1;
    *flag = v;
    return 0;
}

}  // namespace falcon
