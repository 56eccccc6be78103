// Which bytes a call's strided tensors touch, and whether two of them may share one: the argument checks of the
// operators beside the scan. Host only.
#pragma once

#include <stdint.h>

#include "falcon.h"
#include "falcon_seq.h"

namespace falcon {
namespace check {

typedef unsigned __int128 u128;

constexpr int64_t kMax = (int64_t)1 << 31;        // every size is below it, T below half of it
constexpr uint64_t kSpan = (uint64_t)1 << 62;     // every view's extent in bytes is below it

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline uint64_t gcd(uint64_t a, uint64_t b) {
    while (b) {
        const uint64_t t = a % b;
        a = b;
        b = t;
    }
    return a;
}

// The bytes that a view touches: runs of `run` contiguous bytes whose starts differ by multiples of
// `step` (0: one run), all inside [lo, lo + extent).
struct Span {
    uint64_t lo = 0, extent = 0, run = 0, step = 0;
};

inline Span dense_span(const void* p, uint64_t bytes) {
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.extent = s.run = p ? bytes : 0;
    return s;
}

// Sizes of a [B,H,T,d] tensor of elements of es bytes.
struct Shape {
    int64_t B, H, T, d;
    int es;
    bool some() const { return B * H > 0 && T > 0; }
};

// False if the view's extent overflows. `own`: every element has an address of its own.
inline bool view_span(const SeqView& v, const Shape& n, Span* out, bool* own) {
    const uint64_t es = n.es;
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(v.p);
    *own = true;
    if (!v.p || !n.some()) {
        *out = Span{};
        return true;
    }
    uint64_t size[3] = {(uint64_t)n.B, (uint64_t)n.H, (uint64_t)n.T};
    uint64_t stride[3] = {(uint64_t)v.sb, (uint64_t)v.sh, (uint64_t)v.st};
    s.run = (uint64_t)n.d * es;
    u128 extent = s.run;
    // axes from the smallest stride up: each either continues the run or steps over what lies below it
    bool merged = true;
    for (int k = 0; k < 3; ++k) {
        int m = k;
        for (int j = k + 1; j < 3; ++j)
            if (stride[j] < stride[m]) m = j;
        const uint64_t sz = size[m], st = stride[m];
        size[m] = size[k], stride[m] = stride[k];
        size[k] = sz, stride[k] = st;
        if (sz <= 1) continue;
        const u128 sb = (u128)st * es;
        if (sb < extent) *own = false;
        if (merged && sb == s.run) {
            const u128 run = (u128)s.run * sz;
            if (run >= kSpan) return false;
            s.run = (uint64_t)run;
            extent = run;
            continue;
        }
        merged = false;
        extent += sb * (sz - 1);
        if (extent >= kSpan) return false;
        s.step = gcd(s.step, (uint64_t)sb);
    }
    s.extent = (uint64_t)extent;
    *out = s;
    return s.lo <= UINT64_MAX - s.extent;
}

// Whether the two may share a byte (a sound test: false only when they cannot).
inline bool may_share(const Span& a, const Span& b) {
    if (a.extent == 0 || b.extent == 0) return false;
    if (a.lo + a.extent <= b.lo || b.lo + b.extent <= a.lo) return false;
    const uint64_t m = gcd(a.step, b.step);
    if (m == 0 || a.run > m || b.run > m) return true;
    // run starts of a lie at phase 0 modulo m, those of b at phase `delta`
    const uint64_t delta = b.lo >= a.lo ? (b.lo - a.lo) % m : (m - (a.lo - b.lo) % m) % m;
    return delta < a.run || delta + b.run > m;
}

// Collects the tensors of one call: their views, alignment, and which may share memory.
struct Checker {
    int status = FALCON_OK;
    int nin = 0, nout = 0;
    Span in[12], out[12];

    void fail(int s) {
        if (status == FALCON_OK) status = s;
    }
    // The tensor at p with strides s (batch, head, token), null: dense.
    SeqView view(const void* p, const Shape& n, const int64_t* s, bool written, bool required = true) {
        SeqView v = {const_cast<void*>(p), 0, 0, 0};
        if (!p) {
            if (required && n.some()) fail(FALCON_ERR_INVALID_ARG);
            return v;
        }
        if (!aligned(p, n.es)) fail(FALCON_ERR_MISALIGNED);
        if (s) {
            if ((n.B > 1 && s[0] < 0) || (n.H > 1 && s[1] < 0) || (n.T > 1 && s[2] < 0)) {
                fail(FALCON_ERR_INVALID_ARG);
                return v;
            }
            v.sb = n.B > 1 ? s[0] : 0;
            v.sh = n.H > 1 ? s[1] : 0;
            v.st = n.T > 1 ? s[2] : 0;
        } else {
            // dense: the products stay below 2^62 or the span check below refuses the call
            const u128 sh = (u128)n.T * (uint64_t)n.d, sb = sh * (uint64_t)n.H;
            if (sb * (uint64_t)n.B >= kSpan / 4) {
                fail(FALCON_ERR_UNSUPPORTED);
                return v;
            }
            v.sb = n.B > 1 ? (long long)sb : 0;
            v.sh = n.H > 1 ? (long long)sh : 0;
            v.st = n.T > 1 ? n.d : 0;
        }
        Span span;
        bool own;
        if (!view_span(v, n, &span, &own)) {
            fail(FALCON_ERR_INVALID_ARG);
            return v;
        }
        if (written && !own) fail(FALCON_ERR_INVALID_ARG);
        if (written) out[nout++] = span;
        else in[nin++] = span;
        return v;
    }
    // a dense fp32 or int32 array
    void dense(const void* p, uint64_t count, bool written) {
        if (!p) return;
        if (!aligned(p, 4)) fail(FALCON_ERR_MISALIGNED);
        const Span s = dense_span(p, count * 4);
        if (s.lo > UINT64_MAX - s.extent) return fail(FALCON_ERR_INVALID_ARG);
        if (written) out[nout++] = s;
        else in[nin++] = s;
    }
    int finish() {
        if (status != FALCON_OK) return status;
        for (int i = 0; i < nout; ++i) {
            for (int j = 0; j < nin; ++j)
                if (may_share(out[i], in[j])) return FALCON_ERR_INVALID_ARG;
            for (int j = i + 1; j < nout; ++j)
                if (may_share(out[i], out[j])) return FALCON_ERR_INVALID_ARG;
        }
        return FALCON_OK;
    }
};

// eps > 0, and not NaN or infinite
inline bool good_eps(float eps) { return eps > 0.f && eps < 3.4e38f; }

// A call's status. What CUDA refused is told by it alone: the runtime's last error, which the program's other
// launches are checked by, is cleared.
inline int result(int status) {
    if (status == FALCON_ERR_CUDA) (void)cudaGetLastError();
    return status;
}

}  // namespace check
}  // namespace falcon
