// Device code that the gated delta rule's chunk kernels share: 64 x 64 fp32 tiles in shared memory, products of
// them in three tf32 passes, a chunk's decays, and the kernels of the chunk maps and of the scan over them.
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
// Products: operands are fp32, a value x enters as x = h + l, h its nearest tf32, and a product as
// l h + h l + h h with fp32 sums: what is left out is below 2^-22 of it. bf16 inputs are tf32 values, so
// their l is nothing and the pass falls away.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "falcon_gdr.h"

namespace falcon {
namespace gdr {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;          // tokens of a chunk, rows and columns of a tile
constexpr int kTile = kC * kC;  // floats
constexpr int kThreads = 128;

// A tile's element (row, col) lies at row * 64 + (col ^ 8 f(row)): reads of 4 consecutive rows x 8 columns and of
// every other one of 8 rows x 8 columns both touch 32 different banks. Groups of 8 columns stay together, so a tile
// is copied in pieces of 16 bytes, and lies in the workspace as it does in shared memory.
__device__ __forceinline__ int fsw(int row) { return (row ^ ((row >> 2) & 1)) & 3; }
__device__ __forceinline__ int at(int row, int col) { return row * kC + (col ^ (fsw(row) << 3)); }

struct Lane {
    int r, j, fr, f0, f1;
    __device__ Lane() {
        const int l = threadIdx.x & 31;
        r = l >> 2;
        j = l & 3;
        fr = fsw(r);
        f0 = fsw(2 * j);
        f1 = fsw(2 * j + 1);
    }
};

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// x = h + l. The carry of a NaN's mantissa may leave the NaN out of h, never out of l.
__device__ __forceinline__ void split(float x, uint32_t& h, uint32_t& l) {
    h = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    l = __float_as_uint(x - __uint_as_float(h));
}

// How an operand enters: kExact, a value that is tf32 as it is; kRound, its nearest tf32 alone; kFull, both parts.
enum { kExact = 0, kRound = 1, kFull = 2 };
template <int P>
__device__ __forceinline__ void part(float x, uint32_t& h, uint32_t& l) {
    if (P == kFull) split(x, h, l);
    else h = P == kRound ? tf32(x) : __float_as_uint(x);
}

// Operand B of k step kk for four column groups: B[n][k] (COL false) or B[k][n] (COL true). Contraction index j of the
// instruction is column 2j of the k step and j + 4 column 2j + 1, for A and B alike, so that a lane's two values
// lie together in a row, and so that a product's own result can be the next one's A.
template <int PB, bool COL>
__device__ __forceinline__ void load_b(const float* B, const Lane& ln, int kk, int nt0, uint32_t (&h)[4][2], uint32_t (&l)[4][2]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int nt = nt0 + i;
        float x, y;
        if (!COL) {
            const float2 v = *reinterpret_cast<const float2*>(B + (8 * nt + ln.r) * kC + (((kk & 3) ^ ln.fr) << 3) +
                                                              ((kk >> 2) << 5) + 2 * ln.j);
            x = v.x;
            y = v.y;
        } else {
            const float* p = B + (8 * kk + 2 * ln.j) * kC + ((nt >> 2) << 5) + ln.r;
            x = p[((nt & 3) ^ ln.f0) << 3];
            y = p[kC + (((nt & 3) ^ ln.f1) << 3)];
        }
        part<PB>(x, h[i][0], l[i][0]);
        part<PB>(y, h[i][1], l[i][1]);
    }
}

// One k step: acc (16 rows x 64 columns, column groups [n0, n1)) += a B.
template <int PA, int PB, bool BCOL>
__device__ __forceinline__ void step(float (&acc)[8][4], const float (&a)[4], const float* B, const Lane& ln, int kk, int n0, int n1) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part<PA>(a[i], ah[i], al[i]);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (n1 <= 4 * q || n0 >= 4 * q + 4) continue;
        uint32_t bh[4][2], bl[4][2];
        load_b<PB, BCOL>(B, ln, kk, 4 * q, bh, bl);
        if (PA == kFull) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(acc[4 * q + i], al, bh[i][0], bh[i][1]);
        }
        if (PB == kFull) {
#pragma unroll
            for (int i = 0; i < 4; ++i) mma(acc[4 * q + i], ah, bl[i][0], bl[i][1]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) mma(acc[4 * q + i], ah, bh[i][0], bh[i][1]);
    }
}

// acc += A[16 rb ..][k] B over k steps [k0, k1). ACOL: A is stored [k][m]. `scale`: a factor for each k, or null.
template <int PA, int PB, bool ACOL, bool BCOL>
__device__ __forceinline__ void mm(float (&acc)[8][4], const float* A, int rb, const float* B, const Lane& ln, int k0 = 0,
                                   int k1 = 8, int n0 = 0, int n1 = 8, const float* scale = nullptr) {
#pragma unroll 2
    for (int kk = k0; kk < k1; ++kk) {
        float a[4];
        if (!ACOL) {
            const float* p = A + (16 * rb + ln.r) * kC + (((kk & 3) ^ ln.fr) << 3) + ((kk >> 2) << 5) + 2 * ln.j;
            const float2 x = *reinterpret_cast<const float2*>(p), y = *reinterpret_cast<const float2*>(p + 8 * kC);
            a[0] = x.x, a[1] = y.x, a[2] = x.y, a[3] = y.y;
        } else {
            const int nt = 2 * rb;
            const float* p = A + (8 * kk + 2 * ln.j) * kC + ((nt >> 2) << 5) + ln.r;
            a[0] = p[((nt & 3) ^ ln.f0) << 3], a[1] = p[(((nt + 1) & 3) ^ ln.f0) << 3];
            a[2] = p[kC + (((nt & 3) ^ ln.f1) << 3)], a[3] = p[kC + ((((nt + 1) & 3) ^ ln.f1) << 3)];
        }
        if (scale) {
            const float s0 = scale[8 * kk + 2 * ln.j], s1 = scale[8 * kk + 2 * ln.j + 1];
            a[0] *= s0, a[1] *= s0, a[2] *= s1, a[3] *= s1;
        }
        step<PA, PB, BCOL>(acc, a, B, ln, kk, n0, n1);
    }
}
// The same with A in registers, as a product leaves it.
template <int PA, int PB, bool BCOL>
__device__ __forceinline__ void mmr(float (&acc)[8][4], const float (&A)[8][4], const float* B, const Lane& ln, int k0 = 0,
                                    int k1 = 8) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
        if (kk < k0 || kk >= k1) continue;
        const float a[4] = {A[kk][0], A[kk][2], A[kk][1], A[kk][3]};
        step<PA, PB, BCOL>(acc, a, B, ln, kk, 0, 8);
    }
}

__device__ __forceinline__ void zero(float (&acc)[8][4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
}
// Rows 16 rb .. of a tile from and to a product's registers: acc[nt][e] is row 16 rb + r + 8 (e / 2), column
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

// ---- copies of whole tiles, global to shared
__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_tile(float* dst, const float* src) {
#pragma unroll
    for (int i = 0; i < kTile / 4 / kThreads; ++i) {
        const int o = 4 * (threadIdx.x + i * kThreads);
        copy16(dst + o, src + o);
    }
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- the inputs: up to 64 rows x 64 columns of a strided tensor as a tile, zero outside rows x cols. `vec`: rows
// start on 16 bytes and cols is whole vectors.
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

template <typename E>
__device__ __forceinline__ void load_tile(float* dst, const E* src, long long st, int rows, int cols, bool vec) {
    if (vec) {
        constexpr int W = 16 / sizeof(E), PER = kC / W, N = kC * PER / kThreads;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = threadIdx.x + i * kThreads, row = c / PER, col = (c % PER) * W;
            v[i] = make_uint4(0, 0, 0, 0);
            if (row < rows && col < cols) v[i] = *reinterpret_cast<const uint4*>(src + row * st + col);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = threadIdx.x + i * kThreads, row = c / PER, col = (c % PER) * W;
            float* p = dst + at(row, col);
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            if (sizeof(E) == 4) {
                *reinterpret_cast<uint4*>(p) = v[i];
            } else {
                *reinterpret_cast<uint4*>(p) = make_uint4(u[0] << 16, u[0] & 0xffff0000u, u[1] << 16, u[1] & 0xffff0000u);
                *reinterpret_cast<uint4*>(p + 4) = make_uint4(u[2] << 16, u[2] & 0xffff0000u, u[3] << 16, u[3] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll 4
        for (int c = threadIdx.x; c < kTile; c += kThreads) {
            const int row = c >> 6, col = c & 63;
            dst[at(row, col)] = row < rows && col < cols ? to_f(src[row * st + col]) : 0.f;
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

// ---- a chunk's gains and decays
struct Scal {
    float beta[kC], hi[kC], lo[kC];  // G = hi + lo: a difference of two keeps fp32's relative precision
    float eG[kC], w[kC], bw[kC];     // e^G, e^{G_C - G}, beta w
    float eC;
};
__device__ __forceinline__ float exp_sum(float hi, float lo) {
    const float e = expf(hi);
    return fmaf(e, lo, e);
}
__device__ __forceinline__ float decay(const Scal& s, int i, int j) { return expf((s.hi[i] - s.hi[j]) + (s.lo[i] - s.lo[j])); }

// Below this a log decay's factor is 0 in fp32 and so are all that contain it; sums of 64 stay exact enough in double.
constexpr float kLeast = -1e5f;

__device__ __forceinline__ void load_scal(Scal& s, const Ten<float>& beta, const Ten<float>& g, long long b, long long h,
                                          long long t0, int live) {
    if (threadIdx.x >= 32) return;
    const int l = threadIdx.x;
    const float* pb = beta.row0(b, h, t0);
    const float* pg = g.row0(b, h, t0);
    float v[2];
    double x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * l + e;
        const bool in = t < live;
        v[e] = in ? pb[t * beta.st] : 0.f;
        float y = in ? pg[t * g.st] : 0.f;
        y = y < kLeast ? kLeast : y;
        x[e] = y;
    }
    double sum = x[0] + x[1];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, sum, d);
        if (l >= d) sum += o;
    }
    const double all = __shfl_sync(0xffffffffu, sum, 31);
    const double G[2] = {sum - x[1], sum};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int t = 2 * l + e;
        const float hi = (float)G[e], lo = (float)(G[e] - hi);
        const double left = all - G[e];
        const float lh = (float)left, w = exp_sum(lh, (float)(left - lh));
        s.beta[t] = v[e];
        s.hi[t] = hi;
        s.lo[t] = lo;
        s.eG[t] = exp_sum(hi, lo);
        s.w[t] = w;
        s.bw[t] = v[e] * w;
    }
    if (l == 31) s.eC = exp_sum((float)all, (float)(all - (float)all));
}

// ---- the inverse of I + A, A strictly lower triangular in tile T, in its place: 16 x 16 diagonal blocks by
// substitution, then twice the corner of a block pair, -Y22 A21 Y11, as products. They are formed transposed,
// Y11^T A21^T first: its result is then the next product's A in registers.
__device__ __forceinline__ void corner(const float* T, int o, int n, int mb, float (&res)[4][4], const Lane& ln) {
    // columns o + 16 mb .. + 15 of the corner below the block of n rows at o, transposed: res[nt][e] is column
    // 16 mb + r + 8 (e / 2), row 8 nt + 2j + e % 2 of it
    float x[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = 0.f, res[i][e] = 0.f;
    const int nn = n / 8;
    for (int kk = 2 * mb; kk < nn; ++kk) {  // Y11[k][m] is 0 for k < m
        float a[4];
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            a[e] = T[at(o + 8 * kk + 2 * ln.j + (e >> 1), o + 16 * mb + ln.r + 8 * (e & 1))];
            split(a[e], ah[e], al[e]);
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt >= nn) continue;
            const float2 v = *reinterpret_cast<const float2*>(T + at(o + n + 8 * nt + ln.r, o + 8 * kk + 2 * ln.j));
            uint32_t h0, l0, h1, l1;
            split(v.x, h0, l0);
            split(v.y, h1, l1);
            mma(x[nt], al, h0, h1);
            mma(x[nt], ah, l0, l1);
            mma(x[nt], ah, h0, h1);
        }
    }
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        if (kk >= nn) continue;
        const float a[4] = {-x[kk][0], -x[kk][2], -x[kk][1], -x[kk][3]};
        uint32_t ah[4], al[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split(a[e], ah[e], al[e]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt >= nn || nt < kk) continue;  // Y22[n][k] is 0 for k > n
            const float2 v = *reinterpret_cast<const float2*>(T + at(o + n + 8 * nt + ln.r, o + n + 8 * kk + 2 * ln.j));
            uint32_t h0, l0, h1, l1;
            split(v.x, h0, l0);
            split(v.y, h1, l1);
            mma(res[nt], al, h0, h1);
            mma(res[nt], ah, l0, l1);
            mma(res[nt], ah, h0, h1);
        }
    }
}
__device__ __forceinline__ void put_corner(float* T, int o, int n, int mb, const float (&res)[4][4], const Lane& ln) {
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt >= n / 8) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) T[at(o + n + 8 * nt + 2 * ln.j + (e & 1), o + 16 * mb + ln.r + 8 * (e >> 1))] = res[nt][e];
    }
}
// All threads; the tile is written and read between barriers of its own.
__device__ __forceinline__ void invert(float* T, const Lane& ln) {
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    __syncthreads();
    {
        const int o = 16 * w, c = l & 15;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == c ? 1.f : 0.f;
#pragma unroll
            for (int q = 0; q < (i + 3) / 4; ++q) {
                const float4 v = *reinterpret_cast<const float4*>(T + at(o + i, o + 4 * q));
                const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * q + e < i) s = fmaf(-a[e], y[4 * q + e], s);
            }
            y[i] = s;
        }
        __syncwarp();
        if (l < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) T[at(o + i, o + c)] = y[i];
        }
    }
    __syncthreads();
    float res[4][4];
    if (!(w & 1)) {
        corner(T, 16 * w, 16, 0, res, ln);
        __syncwarp();
        put_corner(T, 16 * w, 16, 0, res, ln);
    }
    __syncthreads();
    if (w < 2) corner(T, 0, 32, w, res, ln);
    __syncthreads();
    if (w < 2) put_corner(T, 0, 32, w, res, ln);
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

// Where a chunk's tiles lie, in floats: X [BH][NC] tiles, M [BH][NC][NK][NK] (M[i][j]: rows 64 i of the new state,
// columns 64 j of the old), states transposed [BH][NC + 1][NV][NK] (tile (s, i): rows 64 s of dv, columns 64 i of dk).
template <typename E>
struct PrepArgs {
    Sizes n;
    Ten<const E> q, k, v, dout;
    Ten<float> beta, g;
    float *X, *M, *A, *dA;  // dA: backward, what the chunk adds to the adjoint of the state before it
};

// Strict lower triangle of D * (K K^T) * beta_col into tile T (rows 16 rb ..).
template <int PI, int NK>
__device__ __forceinline__ void gram(float* T, const float* K, const Scal& s, int rb, const Lane& ln) {
    float acc[8][4];
    zero(acc);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) mm<PI, PI, false, false>(acc, K + kb * kTile, rb, K + kb * kTile, ln, 0, 8, 0, 2 * rb + 2);
#pragma unroll
    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * rb + ln.r + 8 * (e >> 1), j = 8 * nt + 2 * ln.j + (e & 1);
            acc[nt][e] = j < i ? acc[nt][e] * decay(s, i, j) * s.beta[j] : 0.f;
        }
    put(T, rb, acc, ln);
}

template <typename E, int NK, bool BWD>
__global__ void __launch_bounds__(kThreads) gdr_prep(const PrepArgs<E> a) {
    constexpr int PI = sizeof(E) == 2 ? kExact : kFull;
    extern __shared__ __align__(16) float smem[];
    __shared__ Scal s;
    float* K = smem;
    float* T = K + NK * kTile;
    float* Y = T + kTile;
    float* Q = Y + kTile;      // BWD
    float* dO = Q + NK * kTile;
    const Lane ln;
    const long long bh = blockIdx.x / (unsigned)a.n.NC, b = bh / a.n.H, h = bh % a.n.H, hk = h / a.n.group;
    const int c = (int)(blockIdx.x % (unsigned)a.n.NC);
    const int live = min(kC, length_of(a.n, b) - c * kC);
    if (live <= 0) return;
    // the CTAs of an SM put the longest rows of a triangle on different quarters of it
    const int rb = ((threadIdx.x >> 5) + blockIdx.x) & 3;
    const long long t0 = (long long)c * kC;
    load_scal(s, a.beta, a.g, b, h, t0, live);
#pragma unroll 1
    for (int kb = 0; kb < NK; ++kb) load_tile(K + kb * kTile, a.k.row0(b, hk, t0) + kb * kC, a.k.st, live, a.n.dk - kb * kC, a.k.vec);
    if (BWD) {
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) load_tile(Q + kb * kTile, a.q.row0(b, hk, t0) + kb * kC, a.q.st, live, a.n.dk - kb * kC, a.q.vec);
    }
    __syncthreads();
    gram<PI, NK>(T, K, s, rb, ln);
    invert(T, ln);
    const long long item = bh * a.n.NC + c;
    {
        float* out = a.X + item * kTile;
        // a forward call reads X as a tf32 operand only
        constexpr bool ROUND = !BWD && PI == kExact;
#pragma unroll
        for (int i = 0; i < kTile / 4 / kThreads; ++i) {
            const int o = 4 * (threadIdx.x + i * kThreads);
            float4 v = *reinterpret_cast<const float4*>(T + o);
            if (ROUND) {
                v.x = __uint_as_float(tf32(v.x)), v.y = __uint_as_float(tf32(v.y));
                v.z = __uint_as_float(tf32(v.z)), v.w = __uint_as_float(tf32(v.w));
            }
            *reinterpret_cast<float4*>(out + o) = v;
        }
    }
    float acc[8][4];
    const int k1 = 2 * rb + 2;  // X's rows end on the diagonal
#pragma unroll 1
    for (int cb = 0; cb < NK; ++cb) {  // M's columns 64 cb ..
        zero(acc);
        mm<kFull, PI, false, true>(acc, T, rb, K + cb * kTile, ln, 0, k1, 0, 8, s.eG);
        if (cb > 0) __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] *= s.bw[16 * rb + ln.r + 8 * (e >> 1)];
        put(Y, rb, acc, ln);
        __syncthreads();
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) {
            zero(acc);
            mm<PI, kFull, true, true>(acc, K + kb * kTile, rb, Y, ln);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[nt][e] = (kb == cb && 16 * rb + ln.r + 8 * (e >> 1) == 8 * nt + 2 * ln.j + (e & 1) ? s.eC : 0.f) - acc[nt][e];
            put(a.M + ((item * NK + kb) * NK + cb) * kTile, rb, acc, ln);
        }
    }
    const int NV = (a.n.dv + kC - 1) / kC;
    float P[8][4];  // BWD: scale D_ij q_i.k_j, transposed: rows j, columns i >= j
    if (BWD) {
        zero(P);
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) mm<PI, PI, false, false>(P, K + kb * kTile, rb, Q + kb * kTile, ln, 0, 8, 2 * rb, 8);
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = 16 * rb + ln.r + 8 * (e >> 1), i = 8 * nt + 2 * ln.j + (e & 1);
                P[nt][e] = j <= i ? P[nt][e] * decay(s, i, j) * a.n.scale : 0.f;
            }
    }
#pragma unroll 1
    for (int sb = 0; sb < NV; ++sb) {
        __syncthreads();
        load_tile(Y, a.v.row0(b, h, t0) + sb * kC, a.v.st, live, a.n.dv - sb * kC, a.v.vec);
        if (BWD) load_tile(dO, a.dout.row0(b, h, t0) + sb * kC, a.dout.st, live, a.n.dv - sb * kC, a.dout.vec);
        __syncthreads();
        zero(acc);
        mm<kFull, PI, false, true>(acc, T, rb, Y, ln, 0, k1);
        __syncthreads();
#pragma unroll
        for (int nt = 0; nt < 8; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] *= s.bw[16 * rb + ln.r + 8 * (e >> 1)];
        put(Y, rb, acc, ln);
        __syncthreads();
#pragma unroll 1
        for (int kb = 0; kb < NK; ++kb) {
            zero(acc);
            mm<kFull, PI, true, true>(acc, Y, rb, K + kb * kTile, ln);
            put(a.A + (((bh * (a.n.NC + 1) + c) * NV + sb) * NK + kb) * kTile, rb, acc, ln);
        }
        if (BWD) {
            // local part of the adjoints: Z = X^T diag(beta) P^T dO; adds scale Q^T diag(e^G) dO - K^T diag(e^G) Z
            zero(acc);
            mmr<kFull, PI, true>(acc, P, dO, ln, 2 * rb, 8);
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] *= s.beta[16 * rb + ln.r + 8 * (e >> 1)];
            __syncthreads();
            put(Y, rb, acc, ln);
            __syncthreads();
            zero(acc);
            mm<kFull, kFull, true, true>(acc, T, rb, Y, ln, 2 * rb, 8);
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] *= -s.eG[16 * rb + ln.r + 8 * (e >> 1)];
            put(Y, rb, acc, ln);
            __syncthreads();
#pragma unroll 1
            for (int kb = 0; kb < NK; ++kb) {
                zero(acc);
                mm<kFull, PI, true, true>(acc, dO, rb, Q + kb * kTile, ln, 0, 8, 0, 8, s.eG);
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[nt][e] *= a.n.scale;
                mm<kFull, PI, true, true>(acc, Y, rb, K + kb * kTile, ln);
                put(a.dA + (((bh * a.n.NC + c) * NV + sb) * NK + kb) * kTile, rb, acc, ln);
            }
        }
    }
}

// ---- the scan over items (chunks, or segments of them): state = M_i state + A_i, or with REV state = M_i^T state +
// A_i from the last item to the first. A warp holds 16 rows of the transposed state, 16 x 64 NK, in registers: its own
// result is the next step's operand, and nothing but M goes through shared memory. A_i's place takes the state before
// the item (REV: behind it). With MAP a segment's own map is left instead of states: the state that it makes of
// nothing, and (rows NV ..) the product of its M.
struct ScanArgs {
    Sizes n;
    int NV;
    const float* M;        // [BH][items][NK][NK]
    float* A;              // [BH][stride][NV][NK]
    long long stride;      // items of A a sequence
    int items;             // items of a sequence (at most)
    int chunks;            // 1: an item is a chunk, and sequence lengths count; 0: an item is a segment
    int L, nseg;           // items of a segment (L * nseg >= items)
    const float* init;     // [BH][dk][dv], null: zero; with nseg > 1 the segments' states
    const float* init_tiles;  // [BH][init_stride][NV][NK]
    long long init_stride;
    float* last;           // [BH][dk][dv] or null
    int end_tile;          // leave the state behind the last chunk in A's place after it, too
    int round;             // states are read as tf32 operands only
    float *mapM, *mapA;    // MAP: [BH][nseg][NK][NK], [BH][map_stride][NV][NK]
    long long map_stride;
};

__host__ __device__ constexpr int scan_stages(int NK) { return NK == 1 ? 3 : 2; }
__host__ __device__ constexpr int scan_smem(int NK) { return scan_stages(NK) * NK * NK * kTile * 4; }

template <int NK, bool REV, bool MAP>
__global__ void __launch_bounds__(kThreads) gdr_scan(const ScanArgs a) {
    constexpr int STAGES = scan_stages(NK);
    extern __shared__ __align__(16) float smem[];
    const Lane ln;
    const int w = threadIdx.x >> 5;
    const long long bh = blockIdx.x / (unsigned)a.nseg, b = bh / a.n.H;
    const int seg = (int)(blockIdx.x % (unsigned)a.nseg), sb = blockIdx.y;
    const bool ident = MAP && sb >= a.NV;
    const int count = a.chunks ? (length_of(a.n, b) + kC - 1) / kC : a.items;
    const int i0 = min(count, seg * a.L), i1 = min(count, i0 + a.L), n = i1 - i0;
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
            get(a.init_tiles + (((bh * a.init_stride + seg) * a.NV + sb) * NK + kb) * kTile, w, acc[kb], ln);
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
    auto item = [&](int i) { return REV ? i1 - 1 - i : i0 + i; };
    auto fetch = [&](int i) {
        if (i < n) {
            const float* src = a.M + (bh * a.items + item(i)) * (NK * NK * kTile);
            float* dst = smem + (i % STAGES) * (NK * NK * kTile);
#pragma unroll 1
            for (int t = 0; t < NK * NK; ++t) copy_tile(dst + t * kTile, src + t * kTile);
        }
        commit();
    };
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);
    for (int i = 0; i < n; ++i) {
        float* tile = ident ? nullptr : a.A + ((bh * a.stride + item(i)) * a.NV + sb) * (NK * kTile);
        float add[NK][8][4];
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (ident) zero(add[kb]);
            else get(tile + kb * kTile, w, add[kb], ln);
        }
        wait<STAGES - 2>();
        __syncthreads();  // item i has arrived for every warp, and item i - 1 is read by every warp
        fetch(i + STAGES - 1);
        if (!MAP) {
#pragma unroll
            for (int kb = 0; kb < NK; ++kb) {
                if (a.round) {
                    float t[8][4];
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[nt][e] = __uint_as_float(tf32(acc[kb][nt][e]));
                    put(tile + kb * kTile, w, t, ln);
                } else {
                    put(tile + kb * kTile, w, acc[kb], ln);
                }
            }
        }
        const float* M = smem + (i % STAGES) * (NK * NK * kTile);
        float nw[NK][8][4];
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            zero(nw[kb]);
#pragma unroll
            for (int kc = 0; kc < NK; ++kc) {
                if (!REV) mmr<kFull, kFull, false>(nw[kb], acc[kc], M + (kb * NK + kc) * kTile, ln);
                else mmr<kFull, kFull, true>(nw[kb], acc[kc], M + (kc * NK + kb) * kTile, ln);
            }
        }
#pragma unroll
        for (int kb = 0; kb < NK; ++kb)
#pragma unroll
            for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[kb][nt][e] = nw[kb][nt][e] + add[kb][nt][e];
    }
    if (MAP) {
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            if (!ident) {
                put(a.mapA + (((bh * a.map_stride + seg) * a.NV + sb) * NK + kb) * kTile, w, acc[kb], ln);
            } else {
                // rows of the transposed product: element (m, k) of the map is acc[k][m]
                float* t = a.mapM + (((bh * a.nseg + seg) * NK + kb) * NK + (sb - a.NV)) * kTile;
#pragma unroll
                for (int nt = 0; nt < 8; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        t[at(8 * nt + 2 * ln.j + (e & 1), 16 * w + ln.r + 8 * (e >> 1))] = acc[kb][nt][e];
            }
        }
        return;
    }
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
        const bool ends = i1 == count && (n > 0 || seg == 0);
        if (a.end_tile && ends) put(a.A + (((bh * a.stride + count) * a.NV + sb) * NK + kb) * kTile, w, acc[kb], ln);
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

// The scan's segments. In units of 1000 cycles: a step along the chain takes 1.7 alone, and an SM's tensor cores take
// 1.55 for each CTA's step. Cut into segments, the segments' maps come first (as many steps, for dk more rows), then a
// scan over them, then the segments' own states. 8: what two more launches cost.
struct Cut {
    int L, nseg;
};
inline Cut cut_of(long long BH, int NC, int NK, int NV) {
    auto steps = [](double ctas) { return ctas / 152 * 1.55 > 1.7 ? ctas / 152 * 1.55 : 1.7; };
    Cut best = {NC > 0 ? NC : 1, 1};
    double least = NC * steps((double)BH * NV);
    for (int s = 2; s <= 128 && s * 4 <= NC; s += s < 16 ? 1 : 8) {
        const int L = (NC + s - 1) / s, nseg = (NC + L - 1) / L;
        const double c = L * (steps((double)BH * nseg * (NV + NK)) + steps((double)BH * nseg * NV)) + 1.7 * nseg + 8;
        if (c < least) least = c, best = Cut{L, nseg};
    }
    return best;
}

// The workspace of one call, in floats from its start.
struct Layout {
    int NK, NV, NC;
    Cut cut;
    long long X, M, S, P, Z, dA, dZ, dq, dk, total;
};
inline Layout layout_of(const GdrSizes& n, bool bwd) {
    Layout l = {};
    l.NK = (n.dk + kC - 1) / kC;
    l.NV = (n.dv + kC - 1) / kC;
    l.NC = (n.T + kC - 1) / kC;
    const long long BH = n.B * n.H, sq = (long long)l.NK * l.NK * kTile, st = (long long)l.NV * l.NK * kTile;
    l.cut = cut_of(BH, l.NC, l.NK, l.NV);
    long long at = 0;
    auto take = [&](long long count) {
        const long long o = at;
        at += (count + 63) / 64 * 64;
        return o;
    };
    const long long seg = l.cut.nseg > 1 ? l.cut.nseg : 0;
    l.X = take(BH * l.NC * kTile);
    l.M = take(BH * l.NC * sq);
    l.S = take(BH * (l.NC + 1) * st);
    l.P = take(BH * seg * sq);
    l.Z = take(BH * seg * st);
    if (bwd) {
        l.dA = take(BH * l.NC * st);
        l.dZ = take(BH * seg * st);
        const long long shared = n.H != n.Hk ? BH * n.T * n.dk : 0;
        l.dq = take(shared);
        l.dk = take(shared);
    }
    l.total = at;
    return l;
}

template <typename K>
inline bool want_smem(K* kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}
inline Sizes sizes_of(const GdrArgs& a, const Layout& l) {
    return Sizes{a.n.B * a.n.H, (int)a.n.H, (int)(a.n.H / a.n.Hk), a.n.T, a.n.dk, a.n.dv, l.NC, a.lengths, a.scale};
}

// The states' scan (REV: the adjoints'), in one pass or by segments. The segments' products of M are the forward
// pass's: the backward one reads them transposed.
template <int NK, bool REV>
bool run_scan(const Sizes& n, const Layout& l, float* ws, const float* init, float* last, bool end_tile, bool round, cudaStream_t s) {
    ScanArgs c = {};
    c.n = n;
    c.NV = l.NV;
    c.M = ws + l.M;
    c.A = ws + (REV ? l.dA : l.S);
    c.stride = l.NC + (REV ? 0 : 1);
    c.items = l.NC;
    c.chunks = 1;
    c.L = l.cut.L;
    c.nseg = l.cut.nseg;
    const int smem = scan_smem(NK);
    if (!want_smem(gdr_scan<NK, REV, false>, smem) || !want_smem(gdr_scan<NK, REV, true>, smem)) return false;
    const unsigned x = (unsigned)(n.BH * l.cut.nseg);
    if (l.cut.nseg > 1) {
        ScanArgs m = c;
        m.mapM = ws + l.P;
        m.mapA = ws + (REV ? l.dZ : l.Z);
        m.map_stride = l.cut.nseg;
        gdr_scan<NK, REV, true><<<dim3(x, l.NV + (REV ? 0 : NK)), kThreads, smem, s>>>(m);
        ScanArgs t = c;
        t.M = ws + l.P;
        t.A = ws + (REV ? l.dZ : l.Z);
        t.stride = t.items = t.L = l.cut.nseg;
        t.chunks = 0;
        t.nseg = 1;
        t.init = init;
        t.last = last;
        gdr_scan<NK, REV, false><<<dim3((unsigned)n.BH, l.NV), kThreads, smem, s>>>(t);
        c.init_tiles = t.A;
        c.init_stride = l.cut.nseg;
    } else {
        c.init = init;
        c.last = last;
    }
    c.end_tile = end_tile;
    c.round = round;
    gdr_scan<NK, REV, false><<<dim3(x, l.NV), kThreads, smem, s>>>(c);
    return true;
}

}  // namespace gdr
}  // namespace falcon
