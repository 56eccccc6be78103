// Device code that the gated delta rule's kernels share: tiles of 64 x 64, their products on the tensor cores, a chunk's
// decays, the inverse of a triangle, and the kernels of the chunk maps and of the scan over them.
//
// Per head, S [dk, dv]: S_t = a_t S_{t-1} + k_t (beta_t (v_t - a_t S_{t-1}^T k_t))^T, a_t = e^{g_t}. In a chunk of
// 64 tokens (rows i, j), G_i the sum of its log decays up to i, S the state before it, D_ij = e^{G_i - G_j}:
//   N_ij = D_ij k_i.k_j (j < i),  P_ij = scale D_ij q_i.k_j (j <= i),  X = (I + N diag(beta))^-1,
//   E = X (V - diag(e^G) K S)  what the state does not predict,  U = diag(beta) E,
//   out = scale diag(e^G) Q S + P U,
//   S' = e^{G_C} S + K^T diag(w) U,  w_j = e^{G_C - G_j}.
// So S' = M S + A with M = e^{G_C} I - K^T diag(w beta) X diag(e^G) K and A = K^T diag(w beta) X V: the chunk
// kernels run for all chunks at once, and only S' = M S + A goes along the sequence.
//
// Products: an fp32 operand x enters as bf16 planes of 8 bits each, x = h + m + l, and a product of two as h h + h m +
// m h + m m + h l + l h with fp32 sums, what is left out being a few units of 2^-24 of it. bf16 inputs are their own single
// plane. An operand is split once, where it is made; the warps' products are loads of matrices and nothing else. (As tf32
// pairs, split by every warp that reads them, the gradient kernel took 306 us for 8 x 12 x 1024 x 64, so 246.)
// They are mma.sync products. A chunk is a row of dependent ones of 64 x 64 x 64 with its own arithmetic between them, and
// what follows a product finds its result in registers; no pipe is busy more than half of the time, the tensor cores 30 % (44 with wide heads).
// On tcgen05, results in tensor memory, the chunk kernels of Falcon-1's backward do the same work with two planes an
// operand in 89 and 117 ns a chunk (the map, the gradients); these, with three, take 67 and 137.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "falcon_gdr.h"
#include "falcon_launch.h"
#include "sm103_ptx.cuh"

namespace falcon {
namespace gdr {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;              // tokens of a chunk, rows and columns of a tile
constexpr int kTile = kC * kC;      // floats of an fp32 tile
constexpr int kPlane = kC * kC * 2; // bytes of a bf16 plane
constexpr int kThreads = 128;

// An fp32 tile's element (row, col) lies at row * 64 + (col ^ 8 f(row)): reads of 4 consecutive rows x 8 columns and of
// every other one of 8 rows x 8 columns both touch 32 different banks. It lies in the workspace as in shared memory.
__device__ __forceinline__ int fsw(int row) { return (row ^ ((row >> 2) & 1)) & 3; }
__device__ __forceinline__ int at(int row, int col) { return row * kC + (col ^ (fsw(row) << 3)); }
// A plane's element lies at this byte: rows of 128 bytes, their pieces of 16 in an order that puts a column of
// pieces of 8 rows into 8 different bank groups.
__device__ __forceinline__ int pat(int row, int col) { return row * 128 + ((((col >> 3) ^ row) & 7) << 4) + 2 * (col & 7); }

struct Lane {
    int r, j, fr;       // of a product's result: rows r and r + 8, columns 2 j and 2 j + 1 of 8
    int l7, l8, l16;    // of a load of four 8 x 8 matrices
    __device__ Lane() {
        const int l = threadIdx.x & 31;
        r = l >> 2;
        j = l & 3;
        fr = fsw(r);
        l7 = l & 7;
        l8 = (l >> 3) & 1;
        l16 = l >> 4;
    }
};

__device__ __forceinline__ uint32_t saddr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// Not a barrier to the compiler: what is read was written before a barrier of all threads, and is overwritten behind one.
template <bool TRANS>
__device__ __forceinline__ void ldm(uint32_t (&v)[4], uint32_t addr) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two values as planes of packed pairs (x in the low half). A plane is the upper half of what is left, cut off: 8 bits
// each, so that three are the value itself.
__device__ __forceinline__ void split(float x, float y, uint32_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
        x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
        y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
    }
}

// Which products of planes: all of them, or those below the first two's, or theirs alone, or first the ones and then the
// other. The tensor cores cut sums off, a unit at a time: of fp32 operands the small products of all k steps come first,
// while the sums are small, and leave four cuts of the result instead of 24 (fp32's forward is off by 3e-7 of its norm
// instead of 6e-7). What is added to such a result is made by itself and added in fp32 (`sum`), or its small products would
// be cut by units of the whole (wide heads' results 7e-7 to 1.2e-6 so, 2 to 4e-7 by itself). kOrdered: the order for other
// operands, too, where a product goes into dg, in which what it is made of cancels (5e-7 instead of 1e-6; 4 % of the gradients' kernel).
enum { kAll = 0, kSmall = 1, kGreat = 2, kOrdered = 3 };

// One k step of 16: acc (16 rows x 64 columns, column groups of 16 in [p0, p1)) += a B. B, its planes at `b`, is stored
// [n][k], or [k][n] (BCOL).
template <int PA, int PB, bool BCOL, int WHICH = kAll>
__device__ __forceinline__ void step(float (&acc)[8][4], const uint32_t (&a)[PA][4], uint32_t b, const Lane& ln, int kk, int p0, int p1) {
    const uint32_t row = BCOL ? b + (16 * kk + ln.l7 + 8 * ln.l8) * 128 : b + (8 * ln.l16 + ln.l7) * 128 + (((2 * kk + ln.l8) ^ ln.l7) << 4);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (p1 <= 2 * q || p0 >= 2 * q + 2) continue;
        uint32_t v[2][PB][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int m = 0; m < (WHICH == kGreat ? 1 : PB); ++m) {
                const int p = 2 * q + i;
                ldm<BCOL>(v[i][m], row + m * kPlane + (BCOL ? (((2 * p + ln.l16) ^ ln.l7) << 4) : p * 2048));
            }
#pragma unroll
        for (int s = WHICH == kGreat ? 0 : (PA > PB ? PA : PB) - 1; s >= (WHICH == kSmall ? 1 : 0); --s)
#pragma unroll
            for (int ma = 0; ma < PA; ++ma) {
                const int mb = s - ma;
                if (mb < 0 || mb >= PB) continue;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mma(acc[4 * q + 2 * i], a[ma], v[i][mb][0], v[i][mb][1]);
                    mma(acc[4 * q + 2 * i + 1], a[ma], v[i][mb][2], v[i][mb][3]);
                }
            }
    }
}

// acc += A[16 rb ..][k] B over k steps [k0, k1). ACOL: A is stored [k][m].
template <int PA, int PB, bool ACOL, bool BCOL, int WHICH = kAll>
__device__ __forceinline__ void mm(float (&acc)[8][4], uint32_t A, int rb, uint32_t B, const Lane& ln, int k0 = 0, int k1 = 4,
                                   int p0 = 0, int p1 = 4) {
    if constexpr ((PA * PB == 9 && WHICH == kAll) || WHICH == kOrdered) {
        mm<PA, PB, ACOL, BCOL, kSmall>(acc, A, rb, B, ln, k0, k1, p0, p1);
        mm<PA, PB, ACOL, BCOL, kGreat>(acc, A, rb, B, ln, k0, k1, p0, p1);
        return;
    }
#pragma unroll 1
    for (int kk = k0; kk < k1; ++kk) {
        uint32_t a[PA][4];
#pragma unroll
        for (int m = 0; m < (WHICH == kGreat ? 1 : PA); ++m) {
            const uint32_t p = ACOL ? A + (16 * kk + ln.l7 + 8 * ln.l16) * 128 + (((2 * rb + ln.l8) ^ ln.l7) << 4)
                                    : A + (16 * rb + ln.l7 + 8 * ln.l8) * 128 + (((2 * kk + ln.l16) ^ ln.l7) << 4);
            ldm<ACOL>(a[m], p + m * kPlane);
        }
        step<PA, PB, BCOL, WHICH>(acc, a, B, ln, kk, p0, p1);
    }
}
// Registers of a product's result as one k step's operand.
__device__ __forceinline__ void split_a(uint32_t (&a)[3][4], const float (&x)[2][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t s[3];
        split(x[i >> 1][2 * (i & 1)], x[i >> 1][2 * (i & 1) + 1], s);
#pragma unroll
        for (int m = 0; m < 3; ++m) a[m][i] = s[m];
    }
}
// The same with A in registers, as a product leaves it. ROLL: the loop stays one, its registers chosen by selection, for the
// backward's long kernels, which wait for instructions as long as for anything else (gradients 220 us unrolled, 209 so;
// the forward's are shorter and lose 5 % by it).
template <int PB, bool BCOL, bool ROLL = false, int WHICH = kAll>
__device__ __forceinline__ void mmr(float (&acc)[8][4], const float (&A)[8][4], uint32_t B, const Lane& ln, int k0 = 0, int k1 = 4) {
    if constexpr ((PB == 3 && WHICH == kAll) || WHICH == kOrdered) {
        mmr<PB, BCOL, ROLL, kSmall>(acc, A, B, ln, k0, k1);
        mmr<PB, BCOL, ROLL, kGreat>(acc, A, B, ln, k0, k1);
        return;
    }
    if (!ROLL) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            if (kk < k0 || kk >= k1) continue;
            const float x[2][4] = {{A[2 * kk][0], A[2 * kk][1], A[2 * kk][2], A[2 * kk][3]}, {A[2 * kk + 1][0], A[2 * kk + 1][1], A[2 * kk + 1][2], A[2 * kk + 1][3]}};
            uint32_t a[3][4];
            split_a(a, x);
            step<3, PB, BCOL, WHICH>(acc, a, B, ln, kk, 0, 4);
        }
        return;
    }
#pragma unroll 1
    for (int kk = k0; kk < k1; ++kk) {
        float x[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float lo = kk & 1 ? A[2 + i][e] : A[i][e], hi = kk & 1 ? A[6 + i][e] : A[4 + i][e];
                x[i][e] = kk & 2 ? hi : lo;
            }
        uint32_t a[3][4];
        split_a(a, x);
        step<3, PB, BCOL, WHICH>(acc, a, B, ln, kk, 0, 4);
    }
}
// ---- values that are not finite. A row i of a triangle's product depends on rows j <= i of B, but the zeros above the diagonal
// meet the others' NaN in the k step on the diagonal. So where a warp's own 16 rows of B hold such a value, that step is
// made without it, and what a product of ones below the diagonal with ones in its places counts is made NaN.
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028234e38f; }
__device__ __forceinline__ bool all_finite(const float (&x)[8][4]) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fmaf(x[i][e], 0.f, s);
    return __all_sync(0xffffffffu, s == 0.f);
}
// acc += A B for the k step kk that holds the rows of acc, A (lower triangular) in registers, B stored [k][n].
__device__ __forceinline__ void step_diagonal(float (&acc)[8][4], const uint32_t (&a)[3][4], uint32_t b, const Lane& ln, int kk) {
    const uint32_t row = b + (16 * kk + ln.l7 + 8 * ln.l8) * 128;
    uint32_t ones[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = ln.r + 8 * (i & 1), k = 2 * ln.j + 8 * (i >> 1);
        ones[i] = (k <= m ? 0x3f80u : 0u) | (k + 1 <= m ? 0x3f800000u : 0u);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        uint32_t v[3][4], bad[4];
#pragma unroll
        for (int m = 0; m < 3; ++m) ldm<true>(v[m], row + m * kPlane + (((2 * p + ln.l16) ^ ln.l7) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // the first plane has the value's exponent
            const uint32_t lo = (v[0][i] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u, hi = (v[0][i] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
            bad[i] = (lo | hi) & 0x3f803f80u;
#pragma unroll
            for (int m = 0; m < 3; ++m) v[m][i] &= ~(lo | hi);
        }
#pragma unroll
        for (int s = 2; s >= 0; --s)
#pragma unroll
            for (int m = 0; m <= s; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) mma(acc[2 * p + i], a[m], v[s - m][2 * i], v[s - m][2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float n[4] = {0.f, 0.f, 0.f, 0.f};
            mma(n, ones, bad[2 * i], bad[2 * i + 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n[e] > 0.f) acc[2 * p + i][e] = __int_as_float(0x7fc00000);
        }
    }
}
// acc += A B, A's rows 16 rb .. lower triangular; `whole`: all of B's rows 16 rb .. are finite.
__device__ __forceinline__ void mm_lower(float (&acc)[8][4], uint32_t A, int rb, uint32_t B, const Lane& ln, bool whole) {
    mm<3, 3, false, true>(acc, A, rb, B, ln, 0, whole ? rb + 1 : rb);
    if (whole) return;
    uint32_t a[3][4];
#pragma unroll
    for (int m = 0; m < 3; ++m) ldm<false>(a[m], A + m * kPlane + (16 * rb + ln.l7 + 8 * ln.l8) * 128 + (((2 * rb + ln.l16) ^ ln.l7) << 4));
    step_diagonal(acc, a, B, ln, rb);
}
__device__ __forceinline__ void mmr_lower(float (&acc)[8][4], const float (&A)[8][4], uint32_t B, int rb, const Lane& ln, bool whole) {
    mmr<3, true>(acc, A, B, ln, 0, whole ? rb + 1 : rb);
    if (whole) return;
    float x[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = rb == 0 ? A[i][e] : rb == 1 ? A[2 + i][e] : rb == 2 ? A[4 + i][e] : A[6 + i][e];
    uint32_t a[3][4];
    split_a(a, x);
    step_diagonal(acc, a, B, ln, rb);
}
// The same with A[k][m] one plane in shared memory, each k scaled by f[k]: the products of planes are made here.
template <int PI, int PB, bool BCOL, int WHICH = kAll>
__device__ __forceinline__ void mms(float (&acc)[8][4], uint32_t A, const float* f, int rb, uint32_t B, const Lane& ln) {
    if constexpr (PB == 3 && WHICH == kAll) {
        mms<PI, PB, BCOL, kSmall>(acc, A, f, rb, B, ln);
        mms<PI, PB, BCOL, kGreat>(acc, A, f, rb, B, ln);
        return;
    }
#pragma unroll 1
    for (int kk = 0; kk < 4; ++kk) {
        float x[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll
        for (int m = PI - 1; m >= 0; --m) {
            uint32_t v[4];
            ldm<true>(v, A + m * kPlane + (16 * kk + ln.l7 + 8 * ln.l16) * 128 + (((2 * rb + ln.l8) ^ ln.l7) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i][0] += __uint_as_float(v[i] << 16), x[i][1] += __uint_as_float(v[i] & 0xffff0000u);
        }
        uint32_t a[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 s = *reinterpret_cast<const float2*>(f + 16 * kk + 8 * (i >> 1) + 2 * ln.j);
            uint32_t p[3];
            split(x[i][0] * s.x, x[i][1] * s.y, p);
#pragma unroll
            for (int m = 0; m < 3; ++m) a[m][i] = p[m];
        }
        step<3, PB, BCOL, WHICH>(acc, a, B, ln, kk, 0, 4);
    }
}

__device__ __forceinline__ void zero(float (&acc)[8][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
}
// acc += make(t), t from zero: SEP, or into acc.
template <bool SEP, typename F>
__device__ __forceinline__ void sum(float (&acc)[8][4], F make) {
    if constexpr (!SEP) {
        make(acc);
    } else {
        float t[8][4];
        zero(t);
        make(t);
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] += t[i][e];
    }
}
// Rows 16 rb .. of an fp32 tile from and to a product's registers: acc[nt][e] is row 16 rb + r + 8 (e / 2), column
// 8 nt + 2 j + e % 2.
__device__ __forceinline__ void put(float* T, int rb, const float (&acc)[8][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        float* p = T + (16 * rb + ln.r) * kC + (((nt & 3) ^ ln.fr) << 3) + ((nt >> 2) << 5) + 2 * ln.j;
        *reinterpret_cast<float2*>(p) = make_float2(acc[nt][0], acc[nt][1]);
        *reinterpret_cast<float2*>(p + 8 * kC) = make_float2(acc[nt][2], acc[nt][3]);
    }
}
__device__ __forceinline__ void get(const float* T, int rb, float (&acc)[8][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        const float* p = T + (16 * rb + ln.r) * kC + (((nt & 3) ^ ln.fr) << 3) + ((nt >> 2) << 5) + 2 * ln.j;
        const float2 x = *reinterpret_cast<const float2*>(p), y = *reinterpret_cast<const float2*>(p + 8 * kC);
        acc[nt][0] = x.x, acc[nt][1] = x.y, acc[nt][2] = y.x, acc[nt][3] = y.y;
    }
}
// The same transposed: acc's row is the tile's column.
__device__ __forceinline__ void get_cols(const float* T, int rb, float (&acc)[8][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][e] = T[at(8 * nt + 2 * ln.j + (e & 1), 16 * rb + ln.r + 8 * (e >> 1))];
}
// Rows 16 rb .. of planes, in shared or global memory: as they are made, three; as they are read, N.
__device__ __forceinline__ void put_planes(uint8_t* T, int rb, const float (&acc)[8][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t p[3];
            split(acc[nt][2 * h], acc[nt][2 * h + 1], p);
            uint8_t* to = T + (16 * rb + ln.r + 8 * h) * 128 + ((nt ^ ln.r) << 4) + 4 * ln.j;
#pragma unroll
            for (int m = 0; m < 3; ++m) *reinterpret_cast<uint32_t*>(to + m * kPlane) = p[m];
        }
}
template <int N>
__device__ __forceinline__ void get_planes(const uint8_t* T, int rb, float (&acc)[8][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint8_t* from = T + (16 * rb + ln.r + 8 * h) * 128 + ((nt ^ ln.r) << 4) + 4 * ln.j;
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int m = N - 1; m >= 0; --m) {
                const uint32_t u = *reinterpret_cast<const uint32_t*>(from + m * kPlane);
                x += __uint_as_float(u << 16);
                y += __uint_as_float(u & 0xffff0000u);
            }
            acc[nt][2 * h] = x, acc[nt][2 * h + 1] = y;
        }
}

// ---- asynchronous copies
// A warp's 16 rows of a result into the workspace: by bulk copies from a place in shared memory, or, DIRECT, as they lie in
// registers, a quarter of eight lines an instruction. The copies need the place: with wide heads they save the forward 8 %;
// the backward's kernel, which has no room for it beside a third CTA, loses 15 % by it.
// A copy still reads its place when the warp goes on, and only the thread that sent it can wait for that. So a warp's
// pieces are its own whatever they hold, rows of a plane or half of its rows of an fp32 tile, and no barrier is needed for them.
constexpr int kPiece = 2048, kPieces = 3;
__host__ __device__ constexpr int piece(int rb, int i) { return i * kPlane + rb * kPiece; }
constexpr bool pieces_apart() {
    for (int a = 0; a < 4 * kPieces; ++a)
        for (int b = 0; b < a; ++b) {
            const int x = piece(a & 3, a >> 2), y = piece(b & 3, b >> 2);
            if (x < y + kPiece && y < x + kPiece) return false;
        }
    return true;
}
static_assert(pieces_apart() && piece(3, kPieces - 1) + kPiece <= kPieces * kPlane && 2 * kPiece == 16 * kC * 4, "stages overlap");
__device__ __forceinline__ void bulk_out(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
template <bool DIRECT>
__device__ __forceinline__ void leave_planes(uint8_t* dst, uint8_t* stage, int rb, const float (&acc)[8][4], const Lane& ln) {
    if (DIRECT) return put_planes(dst, rb, acc, ln);
    if (ln.r + ln.j == 0) ptx::bulk_wait_read<0>();  // what these rows held before has left
    __syncwarp();
    put_planes(stage, rb, acc, ln);
    ptx::fence_async_smem();
    __syncwarp();
    if (ln.r + ln.j == 0) {
#pragma unroll
        for (int m = 0; m < kPieces; ++m) bulk_out(dst + m * kPlane + rb * kPiece, saddr(stage) + piece(rb, m), kPiece);
        ptx::bulk_commit();
    }
}
template <bool DIRECT>
__device__ __forceinline__ void leave_tile(float* dst, uint8_t* stage, int rb, const float (&acc)[8][4], const Lane& ln) {
    if (DIRECT) return put(dst, rb, acc, ln);
    if (ln.r + ln.j == 0) ptx::bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows 8 h .. 8 h + 7 of the 16
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            float* p = reinterpret_cast<float*>(stage + piece(rb, h)) + ln.r * kC + (((nt & 3) ^ ln.fr) << 3) + ((nt >> 2) << 5) + 2 * ln.j;
            *reinterpret_cast<float2*>(p) = make_float2(acc[nt][2 * h], acc[nt][2 * h + 1]);
        }
    ptx::fence_async_smem();
    __syncwarp();
    if (ln.r + ln.j == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) bulk_out(dst + rb * (16 * kC) + h * (8 * kC), saddr(stage) + piece(rb, h), kPiece);
        ptx::bulk_commit();
    }
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in = true) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// N planes as they lie.
template <int N>
__device__ __forceinline__ void copy_planes(uint32_t dst, const uint8_t* src) {
#pragma unroll
    for (int i = 0; i < N * kPlane / 16 / kThreads; ++i) {
        const int o = 16 * (threadIdx.x + i * kThreads);
        copy16(dst + o, src + o);
    }
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- the inputs: up to 64 rows x 64 columns of a strided tensor as planes (one of bf16, three of fp32), zero outside
// rows x cols. `vec`: rows start on 16 bytes and cols is whole vectors; bf16 then goes by asynchronous copies, which the
// caller commits and waits for.
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

__device__ __forceinline__ void load_planes(uint8_t* dst, const bf16* src, long long st, int rows, int cols, bool vec) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = threadIdx.x + i * kThreads, row = c >> 3, col = (c & 7) * 8;
            const bool in = row < rows && col < cols;
            copy16(saddr(dst) + pat(row, col), in ? src + row * st + col : src, in);
        }
    } else {
#pragma unroll 4
        for (int c = threadIdx.x; c < kTile; c += kThreads) {
            const int row = c >> 6, col = c & 63;
            *reinterpret_cast<bf16*>(dst + pat(row, col)) = row < rows && col < cols ? src[row * st + col] : __float2bfloat16_rn(0.f);
        }
    }
}
__device__ __forceinline__ void load_planes(uint8_t* dst, const float* src, long long st, int rows, int cols, bool vec) {
    if (vec) {
#pragma unroll 4
        for (int i = 0; i < 8; ++i) {
            const int c = threadIdx.x + i * kThreads, row = c >> 4, col = (c & 15) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < rows && col < cols) v = *reinterpret_cast<const float4*>(src + row * st + col);
            uint32_t x[3], y[3];
            split(v.x, v.y, x);
            split(v.z, v.w, y);
#pragma unroll
            for (int m = 0; m < 3; ++m) *reinterpret_cast<uint2*>(dst + m * kPlane + pat(row, col)) = make_uint2(x[m], y[m]);
        }
    } else {
#pragma unroll 2
        for (int c = threadIdx.x; c < kTile / 2; c += kThreads) {
            const int row = c >> 5, col = (c & 31) * 2;
            const float* p = src + row * st + col;
            uint32_t x[3];
            split(row < rows && col < cols ? p[0] : 0.f, row < rows && col + 1 < cols ? p[1] : 0.f, x);
#pragma unroll
            for (int m = 0; m < 3; ++m) *reinterpret_cast<uint32_t*>(dst + m * kPlane + pat(row, col)) = x[m];
        }
    }
}
// Two neighbouring elements; `pair`: they can be moved as one.
template <typename E>
__device__ __forceinline__ float2 load2(const E* p, int left, bool pair);
template <>
__device__ __forceinline__ float2 load2<float>(const float* p, int left, bool pair) {
    if (pair && left >= 2) return *reinterpret_cast<const float2*>(p);
    return make_float2(left > 0 ? p[0] : 0.f, left > 1 ? p[1] : 0.f);
}
template <>
__device__ __forceinline__ float2 load2<bf16>(const bf16* p, int left, bool pair) {
    if (pair && left >= 2) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    return make_float2(left > 0 ? to_f(p[0]) : 0.f, left > 1 ? to_f(p[1]) : 0.f);
}
__device__ __forceinline__ void store2(float* p, float x, float y, int left, bool pair) {
    if (pair && left >= 2) *reinterpret_cast<float2*>(p) = make_float2(x, y);
    else {
        if (left > 0) p[0] = x;
        if (left > 1) p[1] = y;
    }
}
__device__ __forceinline__ void store2(bf16* p, float x, float y, int left, bool pair) {
    if (pair && left >= 2) *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
    else {
        if (left > 0) p[0] = __float2bfloat16_rn(x);
        if (left > 1) p[1] = __float2bfloat16_rn(y);
    }
}

// Rows 16 rb .. of a tensor as a product's registers have them, kept as they come: on their way while a product runs.
template <typename E>
struct Rows;
template <>
struct Rows<float> {
    float2 v[8][2];
    __device__ __forceinline__ float2 of(int nt, int h) const { return v[nt][h]; }
    __device__ __forceinline__ void take(const float* p, int left, bool pair, int nt, int h) { v[nt][h] = load2(p, left, pair); }
};
template <>
struct Rows<bf16> {
    uint32_t v[8][2];
    __device__ __forceinline__ float2 of(int nt, int h) const {
        return make_float2(__uint_as_float(v[nt][h] << 16), __uint_as_float(v[nt][h] & 0xffff0000u));
    }
    __device__ __forceinline__ void take(const bf16* p, int left, bool pair, int nt, int h) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
        if (pair && left >= 2) v[nt][h] = *reinterpret_cast<const uint32_t*>(p);
        else v[nt][h] = (left > 0 ? q[0] : 0u) | (left > 1 ? (uint32_t)q[1] << 16 : 0u);
    }
};
template <typename E>
__device__ __forceinline__ void load_rows(Rows<E>& r, const E* p, long long st, bool pair, int rb, const Lane& ln, int live, int cols) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 16 * rb + ln.r + 8 * h;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const int col = 8 * nt + 2 * ln.j;
            r.take(p + row * st + col, row < live ? cols - col : 0, pair, nt, h);
        }
    }
}

// A tensor of the call. vec: 16-byte accesses hold everywhere, pair: those of two elements.
template <typename E>
struct Ten {
    E* p;
    long long sb, sh, st;
    bool vec, pair;
    __device__ E* row0(long long b, long long h, long long t) const { return p + b * sb + h * sh + t * st; }
};
template <typename E>
Ten<E> ten(const SeqView& v, int d) {
    const int es = sizeof(E);
    return Ten<E>{static_cast<E*>(v.p), v.sb, v.sh, v.st, seq_vec_ok(v, es, 16) && d % (16 / es) == 0, seq_vec_ok(v, es, 2 * es)};
}

// Rows 16 rb .. of a result (columns c0 .. of the tensor), rows from `live` on as zeros, rows from `rows` on not at all.
template <typename E>
__device__ __forceinline__ void write_rows(E* p, long long st, bool pair, int rb, const float (&acc)[8][4], const Lane& ln,
                                           int rows, int live, int cols) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int row = 16 * rb + ln.r + 8 * h;
        if (row >= rows) continue;
        const bool in = row < live;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt) {
            const int col = 8 * nt + 2 * ln.j;
            store2(p + row * st + col, in ? acc[nt][2 * h] : 0.f, in ? acc[nt][2 * h + 1] : 0.f, cols - col, pair);
        }
    }
}

// ---- a chunk's gains and decays. Sums of log decays are pairs of floats, hi + lo, 48 bits: a difference of two, at whatever
// size, keeps fp32's relative precision. (In double, whose units are few, this took 10,900 of a chunk's 36,600 cycles.)
struct Scal {
    float beta[kC], hi[kC], lo[kC];  // (backward: no gain below kTiny), G / ln 2 = hi + lo
    float eG[kC], w[kC], bw[kC];     // e^G, e^{G_C - G}, beta w
    // D_ij of a row block of 16 and columns before it as a product: with R the sum before the block, since[i] = e^{G_i - R}
    // and until[block][j] = e^{R - G_j}, neither above 1 where the decays are not
    float since[kC], until[4][kC];
    float eC;
};
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// 2^(hi + lo), lo being small.
__device__ __forceinline__ float ex2(float hi, float lo) {
    const float e = ex2(hi);
    return fmaf(e, lo * 0.69314718f, e);
}
__device__ __forceinline__ float decay(const Scal& s, int i, int j) { return ex2((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j])); }

struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two add(Two a, Two b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = ((a.hi - (s - t)) + (b.hi - t)) + (a.lo + b.lo);
    const float h = s + e;
    return Two{h, e - (h - s)};
}

// The backward divides by the gain what has it as a factor: where it is (nearly) 0, this takes its place, which moves nothing
// else, and dV is scaled back.
constexpr float kTiny = 5.421010862427522e-20f;  // 2^-64

// Below this a log decay's factor is 0 in fp32 and so are all that contain it; sums of 64 keep their lesser parts.
constexpr float kLeast = -1e5f;

// The gains and log decays of tokens 2 l and 2 l + 1, in the lanes of the first warp: read early, summed late.
struct Gates {
    float beta[2], g[2];
};
template <bool BWD>
__device__ __forceinline__ Gates load_gates(const Ten<float>& beta, const Ten<float>& g, long long b, long long h, long long t0, int live) {
    Gates r = {};
    if (threadIdx.x < 32) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int t = 2 * threadIdx.x + e;
            if (t < live) {
                r.beta[e] = beta.row0(b, h, t0)[t * beta.st];
                if (BWD && fabsf(r.beta[e]) < kTiny) r.beta[e] = kTiny;
                r.g[e] = g.row0(b, h, t0)[t * g.st];
            }
        }
    }
    return r;
}
__device__ __forceinline__ void make_scal(Scal& s, const Gates& r) {
    if (threadIdx.x >= 32) return;
    const int l = threadIdx.x;
    Two x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float g = r.g[e] < kLeast ? kLeast : r.g[e];
        x[e].hi = g * 1.44269502f;  // 1 / ln 2 = 1.44269502 + 1.92596299e-8
        x[e].lo = fmaf(g, 1.44269502f, -x[e].hi) + g * 1.92596299e-8f;
    }
    Two sum = add(x[0], x[1]);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Two o = {__shfl_up_sync(0xffffffffu, sum.hi, d), __shfl_up_sync(0xffffffffu, sum.lo, d)};
        if (l >= d) sum = add(o, sum);
    }
    const Two all = {__shfl_sync(0xffffffffu, sum.hi, 31), __shfl_sync(0xffffffffu, sum.lo, 31)};
    Two prev = {__shfl_up_sync(0xffffffffu, sum.hi, 1), __shfl_up_sync(0xffffffffu, sum.lo, 1)};
    if (l == 0) prev = Two{0.f, 0.f};
    const Two G[2] = {add(prev, x[0]), sum};  // (not sum - x[1], which a decay that is not finite would carry back)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * l + e;
        const Two left = add(all, Two{-G[e].hi, -G[e].lo});
        const float w = ex2(left.hi, left.lo);
        s.beta[t] = r.beta[e];
        s.hi[t] = G[e].hi;
        s.lo[t] = G[e].lo;
        s.eG[t] = ex2(G[e].hi, G[e].lo);
        s.w[t] = w;
        s.bw[t] = r.beta[e] * w;
    }
    if (l == 31) s.eC = ex2(all.hi, all.lo);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int t = l + 32 * h, first = t & ~15;
        const float rh = first ? s.hi[first - 1] : 0.f, rl = first ? s.lo[first - 1] : 0.f;
        s.since[t] = ex2((s.hi[t] - rh) + (s.lo[t] - rl));
#pragma unroll
        for (int b = 1; b < 4; ++b)
            if (t < 16 * b) s.until[b][t] = ex2((s.hi[16 * b - 1] - s.hi[t]) + (s.lo[16 * b - 1] - s.lo[t]));
    }
}

// (The far blocks so, and not by exponentials, save the chunk maps' kernel 2 us of 54 and the outputs' 2 as well; the gradients'
// kernel, which waits for its instructions, does better with fewer of them: 211 us against 241.)
// A product's rows times D, and times f of the column (of the row, UPPER) or f itself: rows i and columns j <= i, or rows
// j and columns i >= j (UPPER), STRICT without the diagonal; 0 elsewhere.
template <bool UPPER, bool STRICT>
__device__ __forceinline__ void times_decay(float (&acc)[8][4], const Scal& s, int rb, const Lane& ln, const float* f, float one) {
    const int r0 = 16 * rb + ln.r;
    const float a0 = UPPER ? (f ? f[r0] * one : one) : s.since[r0] * one, a1 = UPPER ? (f ? f[r0 + 8] * one : one) : s.since[r0 + 8] * one;
#pragma unroll
    for (int nt = 0; nt < 8; ++nt) {
        const int c = 8 * nt + 2 * ln.j;
        if ((nt >> 1) == rb) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = r0 + 8 * (e >> 1), col = c + (e & 1), i = UPPER ? col : row, j = UPPER ? row : col;
                const bool in = STRICT ? j < i : j <= i;
                acc[nt][e] = in ? acc[nt][e] * (decay(s, i, j) * (f ? f[j] * one : one)) : 0.f;
            }
        } else if (UPPER ? nt > 2 * rb : nt < 2 * rb) {
            float2 v = *reinterpret_cast<const float2*>(UPPER ? s.since + c : s.until[rb] + c);
            if (!UPPER && f) {
                const float2 u = *reinterpret_cast<const float2*>(f + c);
                v.x *= u.x, v.y *= u.y;
            }
            const float b0 = UPPER ? a0 * s.until[nt >> 1][r0] : a0, b1 = UPPER ? a1 * s.until[nt >> 1][r0 + 8] : a1;
            acc[nt][0] *= b0 * v.x, acc[nt][1] *= b0 * v.y;
            acc[nt][2] *= b1 * v.x, acc[nt][3] *= b1 * v.y;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        }
    }
}

// ---- the inverse of I + A, A strictly lower triangular in tile T, in its place: 16 x 16 diagonal blocks by
// substitution, then twice the corner of a block pair, -Y22 A21 Y11, as products of tf32 pairs (the blocks are
// too small for planes to pay; 22 bits, and with the product of both low parts no result's error is another). They are
// formed transposed, Y11^T A21^T first: its result is then the next product's A in registers.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = h + l, h its nearest tf32. The carry of a NaN's mantissa may leave the NaN out of h, never out of l.
__device__ __forceinline__ void split(float x, uint32_t& h, uint32_t& l) {
    h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    l = __float_as_uint(x - __uint_as_float(h));
}
// Columns o + 16 mb .. + 15 of the corner below the block of N rows at o, its rows 16 half .. + 15, transposed: res[nt][e]
// is column 16 mb + r + 8 (e / 2), row 16 half + 8 nt + 2 j + e % 2 of it.
template <int N>
__device__ __forceinline__ void corner(const float* T, int o, int mb, int half, float (&res)[2][4], const Lane& ln) {
    float x[N / 8][4];
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) res[e >> 2][e & 3] = 0.f;
    const int rows = 2 * half + 2;  // Y22[n][k] is 0 for k > n: rows of A21 Y11 that count, by 8
#pragma unroll
    for (int kk = 0; kk < N / 8; ++kk) {
        if (kk < 2 * mb) continue;  // Y11[k][m] is 0 for k < m
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(T[at(o + 8 * kk + 2 * ln.j + (e >> 1), o + 16 * mb + ln.r + 8 * (e & 1))], ah[e], al[e]);
#pragma unroll
        for (int nt = 0; nt < N / 8; ++nt) {
            if (nt >= rows) continue;
            const float2 v = *reinterpret_cast<const float2*>(T + at(o + N + 8 * nt + ln.r, o + 8 * kk + 2 * ln.j));
            uint32_t h0, l0, h1, l1;
            split(v.x, h0, l0);
            split(v.y, h1, l1);
            mma_tf32(x[nt], al, h0, h1);
            mma_tf32(x[nt], ah, l0, l1);
            mma_tf32(x[nt], ah, h0, h1);
        }
    }
#pragma unroll
    for (int kk = 0; kk < N / 8; ++kk) {
        if (kk >= rows) continue;
        float a[4] = {-x[kk][0], -x[kk][2], -x[kk][1], -x[kk][3]};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const int below = 2 * half + nt - kk;  // Y22's block
            if (below < 0) continue;
            uint32_t bad[4] = {0, 0, 0, 0};  // on the diagonal a row that is not finite leaves those before it alone
            if (below == 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!finite(a[e])) bad[e] = __float_as_uint(1.f);
            }
            uint32_t ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split(bad[e] ? 0.f : a[e], ah[e], al[e]);
            const float2 v = *reinterpret_cast<const float2*>(T + at(o + N + 16 * half + 8 * nt + ln.r, o + N + 8 * kk + 2 * ln.j));
            uint32_t h0, l0, h1, l1;
            split(v.x, h0, l0);
            split(v.y, h1, l1);
            mma_tf32(res[nt], al, h0, h1);
            mma_tf32(res[nt], ah, l0, l1);
            mma_tf32(res[nt], ah, h0, h1);
            if (below == 0 && __any_sync(0xffffffffu, bad[0] | bad[1] | bad[2] | bad[3])) {
                float n[4] = {0.f, 0.f, 0.f, 0.f};
                mma_tf32(n, bad, __float_as_uint(2 * ln.j <= ln.r ? 1.f : 0.f), __float_as_uint(2 * ln.j + 1 <= ln.r ? 1.f : 0.f));
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n[e] > 0.f) res[nt][e] = __int_as_float(0x7fc00000);
            }
        }
    }
}
template <int N>
__device__ __forceinline__ void put_corner(float* T, int o, int mb, int half, const float (&res)[2][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            T[at(o + N + 16 * half + 8 * nt + 2 * ln.j + (e & 1), o + 16 * mb + ln.r + 8 * (e >> 1))] = res[nt][e];
}
// All threads, w a warp's turn; the tile is written and read between barriers of its own. Two warps have a pair of diagonal
// blocks each, 16 lanes a block, and the corner between them; four share the last.
__device__ __forceinline__ void invert(float* T, int w, const Lane& ln) {
    const int l = threadIdx.x & 31;
    float res[2][4];
    __syncthreads();
    if (w < 2) {
        const int o = 32 * w + (l & 16), c = l & 15;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s[4] = {i == c ? 1.f : 0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < (i + 3) / 4; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(T + at(o + i, o + 4 * q));
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e < i) s[e] = fmaf(-a[e], y[4 * q + e], s[e]);
            }
            y[i] = (s[0] + s[1]) + (s[2] + s[3]);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) T[at(o + i, o + c)] = y[i];
        __syncwarp();
        corner<16>(T, 32 * w, 0, 0, res, ln);
        __syncwarp();
        put_corner<16>(T, 32 * w, 0, 0, res, ln);
    }
    __syncthreads();
    corner<32>(T, 0, w & 1, w >> 1, res, ln);
    __syncthreads();
    put_corner<32>(T, 0, w & 1, w >> 1, res, ln);
    __syncthreads();
}

// ---- the chunk kernels' common arguments
struct Sizes {
    long long BH;   // sequences
    int H, group;   // heads of v; heads that share one of q and k
    int T, dk, dv, NC;
    const int32_t* lengths;
    float scale;
};
__device__ __forceinline__ int length_of(const Sizes& n, long long b) {
    if (!n.lengths) return n.T;
    const int l = n.lengths[b];
    return l < 0 ? 0 : l > n.T ? n.T : l;
}

// Where a chunk's tiles lie in the workspace: X [BH][NC], M [BH][NC][NK][NK] (M[i][j]: rows 64 i of the new state,
// columns 64 j of the old) in planes, A [BH][NC][NV][NK] in fp32, the states transposed like A (tile (s, i): rows 64 s of
// dv, columns 64 i of dk), [BH][NC + 1], in planes.
template <typename E>
__host__ __device__ constexpr int planes() { return sizeof(E) == 2 ? 1 : 3; }
template <typename E>
struct PrepArgs {
    Sizes n;
    Ten<const E> q, k, v, dout;
    Ten<float> beta, g;
    uint8_t *X, *M;
    float *A, *dA;  // dA: backward, what the chunk adds to the adjoint of the state before it
};

// Whether the inverse keeps a tile of its own: else it leaves its place to Y, its rows, and backward its columns, being in
// registers (of which fp32's kernel, two CTAs an SM instead of one then, has enough).
template <typename E, bool BWD>
__host__ __device__ constexpr bool prep_keeps() { return BWD && sizeof(E) == 2; }
template <typename E, int NK, bool BWD>
__host__ __device__ constexpr int prep_smem() {
    return (NK * planes<E>() + 3 + (prep_keeps<E, BWD>() ? 2 : 0) + (BWD ? (NK + 1) * planes<E>() : 3)) * kPlane;
}

// CTAs that the shared memory of an SM holds, up to `most`: what the registers are to allow. 3 KiB a CTA are for its
// static arrays and what the system keeps.
__host__ __device__ constexpr int ctas_of(int smem, int most = 4) {
    return 226 * 1024 / (smem + 3 * 1024) < most ? 226 * 1024 / (smem + 3 * 1024) : most;
}

template <typename E, int NK, bool BWD>
__global__ void __launch_bounds__(kThreads, ctas_of(prep_smem<E, NK, BWD>())) gdr_prep(const PrepArgs<E> a) {
    constexpr int PI = planes<E>();
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Scal s;
    uint8_t* K = smem;
    float* T = reinterpret_cast<float*>(K + NK * PI * kPlane);
    constexpr bool KEEPS = prep_keeps<E, BWD>();
    uint8_t* Y = K + (NK * PI + (KEEPS ? 2 : 0)) * kPlane;
    uint8_t* Q = Y + 3 * kPlane;  // BWD; forward: results on their way out
    uint8_t* dO = Q + NK * PI * kPlane;
    const uint32_t Ks = saddr(K), Ys = saddr(Y), Qs = saddr(Q), Os = saddr(dO);
    const Lane ln;
    const unsigned ubh = blockIdx.x / (unsigned)a.n.NC, ub = ubh / (unsigned)a.n.H, uh = ubh % (unsigned)a.n.H;
    const long long bh = ubh, b = ub, h = uh, hk = uh / (unsigned)a.n.group;
    const int c = (int)(blockIdx.x % (unsigned)a.n.NC);
    // what the grids before this one wrote may be read from here on; the scan behind it is not let in early, or its few
    // CTAs share the first SMs that are free (144 us a forward call against 121)
    ptx::pdl_wait();
    const int live = min(kC, length_of(a.n, b) - c * kC);
    if (live <= 0) return;
    // the CTAs of an SM put the longest rows of a triangle on different quarters of it
    const int rb = ((threadIdx.x >> 5) + blockIdx.x) & 3;
    const long long t0 = (long long)c * kC;
    const Gates gates = load_gates<BWD>(a.beta, a.g, b, h, t0, live);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) {
        load_planes(K + kb * PI * kPlane, a.k.row0(b, hk, t0) + kb * kC, a.k.st, live, a.n.dk - kb * kC, a.k.vec);
        if (BWD) load_planes(Q + kb * PI * kPlane, a.q.row0(b, hk, t0) + kb * kC, a.q.st, live, a.n.dk - kb * kC, a.q.vec);
    }
    commit();
    make_scal(s, gates);
    wait<0>();
    __syncthreads();
    float acc[8][4];
    {  // N diag(beta)
        zero(acc);
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb)
            sum<NK * PI == 6>(acc, [&](float (&t)[8][4]) { mm<PI, PI, false, false>(t, Ks + kb * PI * kPlane, rb, Ks + kb * PI * kPlane, ln, 0, 4, 0, rb + 1); });
        times_decay<false, true>(acc, s, rb, ln, s.beta, 1.f);
        put(T, rb, acc, ln);
    }
    invert(T, rb, ln);
    const long long item = bh * a.n.NC + c;
    float t[8][4];
    get(T, rb, t, ln);
    leave_planes<BWD>(a.X + item * (3 * kPlane), Q, rb, t, ln);
    float tc[8][4];
    if (BWD && !KEEPS) get_cols(T, rb, tc, ln);
    if (!KEEPS) __syncthreads();
    const int k1 = rb + 1;  // X's rows end on the diagonal
#pragma unroll 1
    for (int cb = 0; cb < NK; ++cb) {  // M's columns 64 cb ..
        float f[8][4];
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) f[nt][e] = t[nt][e] * s.eG[8 * nt + 2 * ln.j + (e & 1)];
        zero(acc);
        mmr<PI, true, BWD>(acc, f, Ks + cb * PI * kPlane, ln, 0, k1);
        if (cb > 0) __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] *= s.bw[16 * rb + ln.r + 8 * (e >> 1)];
        put_planes(Y, rb, acc, ln);
        __syncthreads();
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) {
            zero(acc);
            mm<PI, 3, true, true>(acc, Ks + kb * PI * kPlane, rb, Ys, ln);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = -acc[nt][e];
                if (kb != cb || (nt >> 1) != rb) continue;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (ln.r + 8 * (e >> 1) == 8 * (nt & 1) + 2 * ln.j + (e & 1)) acc[nt][e] += s.eC;
            }
            leave_planes<BWD>(a.M + ((item * NK + kb) * NK + cb) * (3 * kPlane), Q, rb, acc, ln);
        }
    }
    const int NV = (a.n.dv + kC - 1) / kC;
#pragma unroll 1
    for (int sb = 0; sb < NV; ++sb) {
        __syncthreads();
        load_planes(Y, a.v.row0(b, h, t0) + sb * kC, a.v.st, live, a.n.dv - sb * kC, a.v.vec);
        if (BWD) load_planes(dO, a.dout.row0(b, h, t0) + sb * kC, a.dout.st, live, a.n.dv - sb * kC, a.dout.vec);
        commit();
        wait<0>();
        __syncthreads();
        zero(acc);
        mmr<PI, true, BWD>(acc, t, Ys, ln, 0, k1);
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] *= s.bw[16 * rb + ln.r + 8 * (e >> 1)];
        put_planes(Y, rb, acc, ln);
        __syncthreads();
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) {
            zero(acc);
            mm<3, PI, true, true>(acc, Ys, rb, Ks + kb * PI * kPlane, ln);
            leave_tile<BWD>(a.A + ((item * NV + sb) * NK + kb) * kTile, Q, rb, acc, ln);
        }
        if (BWD) {
            // local part of the adjoints: Z = X^T diag(beta) P^T dO; adds scale Q^T diag(e^G) dO - K^T diag(e^G) Z
            float P[8][4];  // scale D_ij q_i.k_j, transposed: rows j, columns i >= j
            zero(P);
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb)
                sum<NK * PI == 6>(P, [&](float (&x)[8][4]) { mm<PI, PI, false, false>(x, Ks + kb * PI * kPlane, rb, Qs + kb * PI * kPlane, ln, 0, 4, rb, 4); });
            times_decay<true, false>(P, s, rb, ln, nullptr, a.n.scale);
            zero(acc);
            mmr<PI, true, BWD>(acc, P, Os, ln, rb, 4);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] *= s.beta[16 * rb + ln.r + 8 * (e >> 1)];
            __syncthreads();
            put_planes(Y, rb, acc, ln);
            __syncthreads();
            if (KEEPS) get_cols(T, rb, P, ln);
            zero(acc);
            mmr<3, true, BWD>(acc, KEEPS ? P : tc, Ys, ln, rb, 4);
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] *= -s.eG[16 * rb + ln.r + 8 * (e >> 1)];
            put_planes(Y, rb, acc, ln);
            __syncthreads();
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                zero(acc);
                zero(P);
                mms<PI, PI, true>(acc, Os, s.eG, rb, Qs + kb * PI * kPlane, ln);
                mm<3, PI, true, true>(P, Ys, rb, Ks + kb * PI * kPlane, ln);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][e] = fmaf(acc[nt][e], a.n.scale, P[nt][e]);
                put(a.dA + ((item * NV + sb) * NK + kb) * kTile, rb, acc, ln);
            }
        }
    }
    if (!BWD) ptx::bulk_wait_all();
}

// ---- the scan over items (chunks, or segments of them): state = M_i state + A_i, or with REV state = M_i^T state +
// A_i from the last item to the first. A warp holds 16 rows of the transposed state, 16 x 64 NK, in registers: its own
// result is the next step's operand. S_i takes the state before the item (REV: behind it). With MAP a segment's own map is
// left instead of states: the state that it makes of nothing, and (rows NV ..) the product of its M.
// The chain of steps is what takes the time, so four warps do nothing but products and two bring M, block by block into a
// ring, and A, and carry the states away: a step takes 1.5 us, 1.95 with loads and stores in the products' warps (its
// 192 products a warp are 0.8).
struct ScanArgs {
    Sizes n;
    int NV;
    const uint8_t* M;      // [BH][items][NK][NK]
    const float* A;        // [BH][items][NV][NK]
    uint8_t* S;            // [BH][stride][NV][NK]
    long long stride;
    int items;             // items of a sequence (at most)
    int chunks;            // 1: an item is a chunk, and sequence lengths count; 0: an item is a segment
    int L, nseg;           // items of a segment (L * nseg >= items)
    const float* init;     // [BH][dk][dv], null: zero
    const uint8_t* init_tiles;  // or, of segments, [BH][nseg][NV][NK] in three planes
    float* last;           // [BH][dk][dv] or null
    int end_tile;          // leave the state behind the last chunk behind S's others, too
    uint8_t* mapM;         // MAP: [BH][nseg][NK][NK]
    float* mapA;           // MAP: [BH][nseg][NV][NK]
};

// Blocks of M in the ring; A's and S's places follow it. Two CTAs of one block a step fit an SM, one of four.
__host__ __device__ constexpr int ring_of(int NK) { return NK == 1 ? 2 : 4; }
__host__ __device__ constexpr int scan_smem(int NK) { return (ring_of(NK) * 3 + 2 * NK * 2 + NK * 3) * kPlane; }
constexpr int kScanThreads = kThreads + 64;

template <int NK, bool REV, bool MAP>
__device__ __forceinline__ void scan(const ScanArgs& a, uint8_t* smem) {
    constexpr int R = ring_of(NK), NB = NK * NK;
    const Lane ln;
    uint8_t* At = smem + R * 3 * kPlane;
    uint8_t* St = At + 2 * NK * 2 * kPlane;
    const int w = threadIdx.x >> 5;
    const unsigned ubh = blockIdx.x / (unsigned)a.nseg;
    const long long bh = ubh, b = ubh / (unsigned)a.n.H;
    const int seg = (int)(blockIdx.x % (unsigned)a.nseg), sb = blockIdx.y;
    const bool ident = MAP && sb >= a.NV;
    const int count = a.chunks ? (length_of(a.n, b) + kC - 1) / kC : a.items;
    const int i0 = min(count, seg * a.L), i1 = min(count, i0 + a.L), n = i1 - i0;
    auto item = [&](int i) { return REV ? i1 - 1 - i : i0 + i; };
    // block t of a step: rows kb, columns kc of M (REV: of its transpose)
    auto block = [&](int t) { return REV ? (t % NK) * NK + t / NK : t; };
    if (threadIdx.x >= kThreads) {
        const int id = threadIdx.x - kThreads;
        auto bring = [&](uint8_t* dst, const uint8_t* src, int bytes) {
            const uint32_t d = saddr(dst);
            for (int o = 16 * id; o < bytes; o += 16 * 64) copy16(d + o, src + o);
        };
        auto fetch = [&](int g) {
            const int i = g / NB;
            if (i < n) bring(smem + (g % R) * (3 * kPlane), a.M + ((bh * a.items + item(i)) * NB + block(g % NB)) * (3 * kPlane), 3 * kPlane);
        };
        auto fetch_a = [&](int i) {  // two places, each a step's
            if (i < n && !ident)
                bring(At + (i & 1) * (NK * 2 * kPlane), reinterpret_cast<const uint8_t*>(a.A + ((bh * a.items + item(i)) * a.NV + sb) * (NK * kTile)), NK * kTile * 4);
        };
        fetch_a(0);
        for (int g = 0; g < R - 1; ++g) {
            fetch(g);
            commit();
        }
        for (int i = 0; i < n; ++i) {
            for (int t = 0; t < NB; ++t) {
                wait<R - 2>();
                __syncthreads();  // block t has arrived (and A, a step ago), the one before it is read, and so is the state
                fetch(i * NB + t + R - 1);
                if (t == 0) fetch_a(i + 1);
                commit();
                if (t > 0 || MAP) continue;
                ptx::named_bar(1, kScanThreads);  // the state is in its place
                uint8_t* dst = a.S + ((bh * a.stride + item(i)) * a.NV + sb) * (NK * 3 * kPlane);
#pragma unroll 8
                for (int o = 16 * id; o < NK * 3 * kPlane; o += 16 * 64) *reinterpret_cast<uint4*>(dst + o) = *reinterpret_cast<const uint4*>(St + o);
            }
        }
        return;
    }
    float acc[NK][8][4];
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
        zero(acc[kb]);
        if (MAP) {
            if (ident && sb - a.NV == kb) {
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (16 * w + ln.r + 8 * (e >> 1) == 8 * nt + 2 * ln.j + (e & 1)) acc[kb][nt][e] = 1.f;
            }
        } else if (a.init_tiles) {
            get_planes<3>(a.init_tiles + (((bh * a.nseg + seg) * a.NV + sb) * NK + kb) * (3 * kPlane), w, acc[kb], ln);
        } else if (a.init) {
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int m = sb * kC + 16 * w + ln.r + 8 * (e >> 1), k = kb * kC + 8 * nt + 2 * ln.j + (e & 1);
                    if (m < a.n.dv && k < a.n.dk) acc[kb][nt][e] = a.init[(bh * a.n.dk + k) * a.n.dv + m];
                }
        }
    }
    for (int i = 0; i < n; ++i) {
        float nw[NK][8][4];
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const int kb = t / NK, kc = t % NK;
            __syncthreads();
            if (t == 0) {
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    if (!MAP) put_planes(St + k * (3 * kPlane), w, acc[k], ln);
                    zero(nw[k]);
                }
                if (!MAP) asm volatile("bar.arrive 1, %0;" ::"n"(kScanThreads) : "memory");
            }
            sum<(NK > 1)>(nw[kb], [&](float (&x)[8][4]) { mmr<3, REV>(x, acc[kc], saddr(smem) + ((i * NB + t) % R) * (3 * kPlane), ln); });
        }
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (ident) zero(acc[kb]);
            else get(reinterpret_cast<const float*>(At) + ((i & 1) * NK + kb) * kTile, w, acc[kb], ln);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[kb][nt][e] += nw[kb][nt][e];
        }
    }
    if (MAP) {
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (!ident) {
                put(a.mapA + (((bh * a.nseg + seg) * a.NV + sb) * NK + kb) * kTile, w, acc[kb], ln);
            } else {
                // rows of the transposed product: element (m, k) of the map is acc[k][m]
                uint8_t* t = a.mapM + (((bh * a.nseg + seg) * NK + kb) * NK + (sb - a.NV)) * (3 * kPlane);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t p[3];
                        split(acc[kb][nt][2 * h], acc[kb][nt][2 * h + 1], p);
#pragma unroll
                        for (int m = 0; m < 3; ++m) {
                            const int row = 8 * nt + 2 * ln.j, col = 16 * w + ln.r + 8 * h;
                            *reinterpret_cast<uint16_t*>(t + m * kPlane + pat(row, col)) = (uint16_t)p[m];
                            *reinterpret_cast<uint16_t*>(t + m * kPlane + pat(row + 1, col)) = (uint16_t)(p[m] >> 16);
                        }
                    }
            }
        }
        return;
    }
    const bool ends = i1 == count && (n > 0 || seg == 0);
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
        if (a.end_tile && ends) put_planes(a.S + (((bh * a.stride + count) * a.NV + sb) * NK + kb) * (3 * kPlane), w, acc[kb], ln);
        if (!a.last) continue;
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int m = sb * kC + 16 * w + ln.r + 8 * (e >> 1), k = kb * kC + 8 * nt + 2 * ln.j + (e & 1);
                if (m < a.n.dv && k < a.n.dk) a.last[(bh * a.n.dk + k) * a.n.dv + m] = acc[kb][nt][e];
            }
    }
}

// The states' scan.
template <int NK, bool MAP>
__global__ void __launch_bounds__(kScanThreads, NK == 1 ? 2 : 1) gdr_scan(const ScanArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::pdl_wait();
    if (!MAP && a.chunks) ptx::pdl_launch_dependents();
    scan<NK, false, MAP>(a, smem);
}
// The states' and the adjoints', side by side: neither needs the other.
template <int NK, bool MAP>
__global__ void __launch_bounds__(kScanThreads, NK == 1 ? 2 : 1) gdr_scans(const ScanArgs a, const ScanArgs r) {
    extern __shared__ __align__(128) uint8_t smem[];
    ptx::pdl_wait();
    if (!MAP && a.chunks) ptx::pdl_launch_dependents();
    if (blockIdx.z == 0) scan<NK, false, MAP>(a, smem);
    else if (!MAP || (int)blockIdx.y < r.NV) scan<NK, true, MAP>(r, smem);
}

// The scan's segments, for as few microseconds as the steps make: one of the states takes 1.5 with a CTA an SM, 2.8 with the
// two that fit, one of a segment's map, which writes nothing, 1.3 and 2.1; wide heads have an SM to themselves, 5.1 and 5.2. A
// scan over the segments' maps and two more launches come on top. (12 heads, 1024 chunks: 25 segments.) A backward call has two
// scans side by side, which share the map's product of M.
struct Cut {
    int L, nseg;
};
inline Cut cut_of(long long BH, int NC, int NK, int NV, int scans) {
    auto step = [&](long long ctas, double one, double two, double wide) {
        const long long n = (ctas + 151) / 152;  // of the fullest SM
        return NK == 1 ? (double)(n / 2) * two + (double)(n % 2) * one : (double)n * wide;
    };
    auto own = [&](long long ctas) { return step(ctas, 1.5, 2.8, 5.1); };
    auto map = [&](long long ctas) { return step(ctas, 1.3, 2.1, 5.2); };
    Cut best = {NC > 0 ? NC : 1, 1};
    double least = NC * own(BH * NV * scans);
    for (int s = 2; s <= 64 && s * 4 <= NC; ++s) {
        const int L = (NC + s - 1) / s, nseg = (NC + L - 1) / L;
        const double c = L * (map(BH * nseg * (NV * scans + NK)) + own(BH * nseg * NV * scans)) + own(BH * NV * scans) * nseg + 8;
        if (c < least) least = c, best = Cut{L, nseg};
    }
    return best;
}

// The workspace of one call, in bytes from its start.
struct Layout {
    int NK, NV, NC;
    Cut cut;
    long long X, M, A, S, P, Z, G, dA, dS, dZ, dG, dq, dk, total;
};
inline Layout layout_of(const GdrSizes& n, bool bwd) {
    Layout l = {};
    l.NK = (n.dk + kC - 1) / kC;
    l.NV = (n.dv + kC - 1) / kC;
    l.NC = (n.T + kC - 1) / kC;
    const long long BH = n.B * n.H, sq = (long long)l.NK * l.NK, st = (long long)l.NV * l.NK;
    l.cut = cut_of(BH, l.NC, l.NK, l.NV, bwd ? 2 : 1);
    long long at = 0;
    auto take = [&](long long bytes) {
        const long long o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const long long seg = l.cut.nseg > 1 ? l.cut.nseg : 0, tile = kTile * 4;
    l.X = take(BH * l.NC * 3 * kPlane);
    l.M = take(BH * l.NC * sq * 3 * kPlane);
    l.A = take(BH * l.NC * st * tile);
    l.S = take(BH * (l.NC + 1) * st * 3 * kPlane);
    l.P = take(BH * seg * sq * 3 * kPlane);
    l.Z = take(BH * seg * st * tile);
    l.G = take(BH * seg * st * 3 * kPlane);
    if (bwd) {
        l.dA = take(BH * l.NC * st * tile);
        l.dS = take(BH * l.NC * st * 3 * kPlane);
        l.dZ = take(BH * seg * st * tile);
        l.dG = take(BH * seg * st * 3 * kPlane);
        const long long shared = n.H != n.Hk ? BH * n.T * n.dk * 4 : 0;
        l.dq = take(shared);
        l.dk = take(shared);
    }
    l.total = at;
    return l;
}

inline Sizes sizes_of(const GdrArgs& a, const Layout& l) {
    return Sizes{a.n.B * a.n.H, (int)a.n.H, (int)(a.n.H / a.n.Hk), a.n.T, a.n.dk, a.n.dv, l.NC, a.lengths, a.scale};
}

// Arguments of the scan's three launches: the segments' maps, the scan over them, the states. Uncut, the last alone.
struct ScanSteps {
    ScanArgs map, over, own;
};
inline ScanSteps scan_steps(const Sizes& n, const Layout& l, uint8_t* ws, bool rev, const float* init, float* last) {
    ScanSteps r = {};
    ScanArgs& c = r.own;
    c.n = n;
    c.NV = l.NV;
    c.M = ws + l.M;
    c.A = reinterpret_cast<const float*>(ws + (rev ? l.dA : l.A));
    c.S = ws + (rev ? l.dS : l.S);
    c.stride = l.NC + (rev ? 0 : 1);
    c.items = l.NC;
    c.chunks = 1;
    c.L = l.cut.L;
    c.nseg = l.cut.nseg;
    if (l.cut.nseg > 1) {
        r.map = r.over = c;
        r.map.mapM = ws + l.P;
        r.map.mapA = reinterpret_cast<float*>(ws + (rev ? l.dZ : l.Z));
        ScanArgs& t = r.over;
        t.M = ws + l.P;
        t.A = r.map.mapA;
        t.S = ws + (rev ? l.dG : l.G);
        t.stride = t.items = t.L = l.cut.nseg;
        t.chunks = 0;
        t.nseg = 1;
        t.init = init;
        t.last = last;
        c.init_tiles = t.S;
    } else {
        c.init = init;
        c.last = last;
    }
    return r;
}
// The states' scan of a forward call.
template <int NK>
int run_scan(const Sizes& n, const Layout& l, uint8_t* ws, const float* init, float* last, cudaStream_t s) {
    const ScanSteps f = scan_steps(n, l, ws, false, init, last);
    const unsigned x = (unsigned)(n.BH * l.cut.nseg);
    int st = 0;
    if (l.cut.nseg > 1) {
        st |= launch_ahead<gdr_scan<NK, true>>(dim3(x, l.NV + NK), kScanThreads, scan_smem(NK), s, f.map);
        st |= launch_ahead<gdr_scan<NK, false>>(dim3((unsigned)n.BH, l.NV), kScanThreads, scan_smem(NK), s, f.over);
    }
    return st | launch_ahead<gdr_scan<NK, false>>(dim3(x, l.NV), kScanThreads, scan_smem(NK), s, f.own);
}
// Both of a backward call's. The segments' products of M are the forward's: the other reads them transposed.
template <int NK>
int run_scans(const Sizes& n, const Layout& l, uint8_t* ws, const float* S0, const float* dS_final, float* dS0, cudaStream_t s) {
    ScanSteps f = scan_steps(n, l, ws, false, S0, nullptr), r = scan_steps(n, l, ws, true, dS_final, dS0);
    f.own.end_tile = 1;  // the state behind the last chunk, too
    const unsigned x = (unsigned)(n.BH * l.cut.nseg);
    int st = 0;
    if (l.cut.nseg > 1) {
        st |= launch_ahead<gdr_scans<NK, true>>(dim3(x, l.NV + NK, 2), kScanThreads, scan_smem(NK), s, f.map, r.map);
        st |= launch_ahead<gdr_scans<NK, false>>(dim3((unsigned)n.BH, l.NV, 2), kScanThreads, scan_smem(NK), s, f.over, r.over);
    }
    return st | launch_ahead<gdr_scans<NK, false>>(dim3(x, l.NV, 2), kScanThreads, scan_smem(NK), s, f.own, r.own);
}

}  // namespace gdr
}  // namespace falcon
