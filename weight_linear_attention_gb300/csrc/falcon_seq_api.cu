// C-ABI front end of the strided [B,H,T,d] operators: argument checking for falcon_glr_fwd,
// falcon_glr_bwd, falcon_gn_fwd and falcon_gn_bwd. The contract is documented in include/falcon.h.

#include <cuda_runtime.h>
#include <stdint.h>

#include "falcon.h"
#include "falcon_seq.h"

namespace {

using falcon::SeqSizes;
using falcon::SeqView;
typedef unsigned __int128 u128;

constexpr int64_t kMax = (int64_t)1 << 31;        // every size is below it, T below half of it
constexpr uint64_t kSpan = (uint64_t)1 << 62;     // every view's extent in bytes is below it

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uint64_t gcd(uint64_t a, uint64_t b) {
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

Span dense_span(const void* p, uint64_t bytes) {
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.extent = s.run = p ? bytes : 0;
    return s;
}

// False if the view's extent overflows. `own`: every element has an address of its own.
bool view_span(const SeqView& v, const SeqSizes& n, Span* out, bool* own) {
    const uint64_t es = n.bf16 ? 2 : 4;
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(v.p);
    *own = true;
    if (!v.p || n.B * n.H == 0 || n.T == 0) {
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
bool may_share(const Span& a, const Span& b) {
    if (a.extent == 0 || b.extent == 0) return false;
    if (a.lo + a.extent <= b.lo || b.lo + b.extent <= a.lo) return false;
    const uint64_t m = gcd(a.step, b.step);
    if (m == 0 || a.run > m || b.run > m) return true;
    // run starts of a lie at phase 0 modulo m, those of b at phase `delta`
    const uint64_t delta = b.lo >= a.lo ? (b.lo - a.lo) % m : (m - (a.lo - b.lo) % m) % m;
    return delta < a.run || delta + b.run > m;
}

int sizes_of(const falcon_seq_dims_t* d, SeqSizes* n) {
    if (!d || d->batch < 0 || d->heads < 0 || d->seqlen < 0 || d->d <= 0 || d->reserved != 0)
        return FALCON_ERR_INVALID_ARG;
    if (d->dtype != FALCON_F32 && d->dtype != FALCON_BF16) return FALCON_ERR_UNSUPPORTED;
    if (d->batch >= kMax || d->heads >= kMax || d->seqlen >= kMax / 2 || d->d >= kMax) return FALCON_ERR_UNSUPPORTED;
    // [B,H,d] fp32 states and everything counted from them stay below 2^62 bytes
    if ((u128)d->batch * (uint64_t)d->heads * (uint64_t)d->d * 4 >= kSpan) return FALCON_ERR_UNSUPPORTED;
    n->B = d->batch;
    n->H = d->heads;
    n->T = (int)d->seqlen;
    n->d = (int)d->d;
    n->bf16 = d->dtype == FALCON_BF16;
    return FALCON_OK;
}

// Collects the tensors of one call: their views, alignment, and which may share memory.
struct Checker {
    SeqSizes n;
    const int64_t* strides;
    int status = FALCON_OK;
    int nin = 0, nout = 0;
    Span in[8], out[8];

    void fail(int s) {
        if (status == FALCON_OK) status = s;
    }
    // the k-th tensor of the stride list
    SeqView view(const void* p, int k, bool written, bool required = true) {
        SeqView v = {const_cast<void*>(p), 0, 0, 0};
        const bool some = n.B * n.H > 0 && n.T > 0;
        if (!p) {
            if (required && some) fail(FALCON_ERR_INVALID_ARG);
            return v;
        }
        if (!aligned(p, n.bf16 ? 2 : 4)) fail(FALCON_ERR_MISALIGNED);
        if (strides) {
            const int64_t* s = strides + 3 * k;
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
        Span s;
        bool own;
        if (!view_span(v, n, &s, &own)) {
            fail(FALCON_ERR_INVALID_ARG);
            return v;
        }
        if (written && !own) fail(FALCON_ERR_INVALID_ARG);
        if (written) out[nout++] = s;
        else in[nin++] = s;
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

// Where every given tensor's heads follow each other without a gap (the projection's layout), the head
// axis is part of the channels: fewer, fuller channel tiles.
void merge_heads(SeqSizes* n, SeqView** v, int nv) {
    if (n->H <= 1 || n->H * n->d >= kMax) return;
    for (int i = 0; i < nv; ++i)
        if (v[i]->p && v[i]->sh != n->d) return;
    for (int i = 0; i < nv; ++i) v[i]->sh = 0;
    n->d = (int)(n->H * n->d);
    n->H = 1;
}

// A call's status. What CUDA refused is told by it alone: the runtime's last error, which the program's other
// launches are checked by, is cleared.
int result(int status) {
    if (status == FALCON_ERR_CUDA) (void)cudaGetLastError();
    return status;
}

}  // namespace

extern "C" {

int falcon_glr_fwd(int gate, const void* x, const void* g, const float* h0, const int32_t* lengths, void* out,
                   float* h_final, const falcon_seq_dims_t* dims, const int64_t* strides, void* stream) {
    if (gate < FALCON_GATE_DECAY || gate > FALCON_GATE_MIX) return FALCON_ERR_INVALID_ARG;
    Checker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    c.strides = strides;
    const uint64_t state = (uint64_t)c.n.B * c.n.H * c.n.d;
    falcon::GlrArgs a = {};
    a.gate = gate;
    a.x = c.view(x, 0, false);
    a.g = c.view(g, 1, false);
    a.out = c.view(out, 2, true);
    if (h0 != h_final) c.dense(h0, state, false);  // equal: the state is updated in place
    c.dense(lengths, c.n.B, false);
    c.dense(h_final, state, true);
    st = c.finish();
    if (st != FALCON_OK) return st;
    if (state == 0) return FALCON_OK;
    a.n = c.n;
    a.h0 = h0;
    a.lengths = lengths;
    a.h_final = h_final;
    SeqView* v[] = {&a.x, &a.g, &a.out};
    merge_heads(&a.n, v, 3);
    return result(falcon::launch_glr_fwd(a, static_cast<cudaStream_t>(stream)));
}

int falcon_glr_bwd(int gate, const void* x, const void* g, const void* out, const float* h0, const int32_t* lengths,
                   const void* dout, const float* dh_final, void* dx, void* dg, float* dh0,
                   const falcon_seq_dims_t* dims, const int64_t* strides, void* stream) {
    if (gate < FALCON_GATE_DECAY || gate > FALCON_GATE_MIX) return FALCON_ERR_INVALID_ARG;
    Checker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    c.strides = strides;
    const uint64_t state = (uint64_t)c.n.B * c.n.H * c.n.d;
    falcon::GlrArgs a = {};
    a.gate = gate;
    a.x = c.view(x, 0, false, gate == FALCON_GATE_MIX);
    a.g = c.view(g, 1, false);
    a.out = c.view(out, 2, false);
    a.dout = c.view(dout, 3, false);
    a.dx = c.view(dx, 4, true);
    a.dg = c.view(dg, 5, true);
    c.dense(h0, state, false);
    c.dense(lengths, c.n.B, false);
    c.dense(dh_final, state, false);
    c.dense(dh0, state, true);
    st = c.finish();
    if (st != FALCON_OK) return st;
    if (state == 0) return FALCON_OK;
    a.n = c.n;
    a.h0 = h0;
    a.lengths = lengths;
    a.dh_final = dh_final;
    a.dh0 = dh0;
    if (gate != FALCON_GATE_MIX) a.x.p = nullptr;  // not read
    SeqView* v[] = {&a.x, &a.g, &a.out, &a.dout, &a.dx, &a.dg};
    merge_heads(&a.n, v, 6);
    return result(falcon::launch_glr_bwd(a, static_cast<cudaStream_t>(stream)));
}

// eps > 0, and not NaN or infinite
static bool good_eps(float eps) { return eps > 0.f && eps < 3.4e38f; }

int falcon_gn_fwd(int act, const void* x, const void* z, const float* weight, const float* bias,
                  const int32_t* lengths, void* y, const falcon_seq_dims_t* dims, const int64_t* strides, float eps,
                  void* stream) {
    if (act < FALCON_ACT_NONE || act > FALCON_ACT_SIGMOID || !good_eps(eps)) return FALCON_ERR_INVALID_ARG;
    Checker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    if (c.n.d > falcon::kGnMaxD) return FALCON_ERR_UNSUPPORTED;
    c.strides = strides;
    const uint64_t chans = (uint64_t)c.n.H * c.n.d;
    falcon::GnArgs a = {};
    a.act = act;
    a.x = c.view(x, 0, false);
    a.z = c.view(z, 1, false, false);
    a.y = c.view(y, 2, true);
    c.dense(weight, chans, false);
    c.dense(bias, chans, false);
    c.dense(lengths, c.n.B, false);
    st = c.finish();
    if (st != FALCON_OK) return st;
    a.n = c.n;
    a.w = weight;
    a.b = bias;
    a.lengths = lengths;
    a.eps = eps;
    if (c.n.B * c.n.H == 0 || c.n.T == 0) return FALCON_OK;
    return result(falcon::launch_gn_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t falcon_gn_bwd_workspace_bytes(const falcon_seq_dims_t* dims) {
    SeqSizes n;
    if (sizes_of(dims, &n) != FALCON_OK || n.d > falcon::kGnMaxD || n.B * n.H == 0 || n.T == 0) return 0;
    return (size_t)falcon::gn_bwd_splits(n) * 2 * (size_t)n.H * n.d * sizeof(float);
}

int falcon_gn_bwd(int act, const void* x, const void* z, const float* weight, const float* bias,
                  const int32_t* lengths, const void* dy, void* dx, void* dz, float* dweight, float* dbias,
                  const falcon_seq_dims_t* dims, const int64_t* strides, float eps, void* workspace,
                  size_t workspace_bytes, void* stream) {
    if (act < FALCON_ACT_NONE || act > FALCON_ACT_SIGMOID || !good_eps(eps)) return FALCON_ERR_INVALID_ARG;
    if ((z == nullptr) != (dz == nullptr)) return FALCON_ERR_INVALID_ARG;
    Checker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    if (c.n.d > falcon::kGnMaxD) return FALCON_ERR_UNSUPPORTED;
    c.strides = strides;
    const uint64_t chans = (uint64_t)c.n.H * c.n.d;
    falcon::GnArgs a = {};
    a.act = act;
    a.x = c.view(x, 0, false);
    a.z = c.view(z, 1, false, false);
    a.dy = c.view(dy, 2, false);
    a.dx = c.view(dx, 3, true);
    a.dz = c.view(dz, 4, true, false);
    c.dense(weight, chans, false);
    c.dense(bias, chans, false);
    c.dense(lengths, c.n.B, false);
    c.dense(dweight, chans, true);
    c.dense(dbias, chans, true);
    const bool sums = dweight || dbias;
    const size_t need = sums ? falcon_gn_bwd_workspace_bytes(dims) : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FALCON_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return FALCON_ERR_MISALIGNED;
        c.dense(workspace, need / 4, true);
    }
    st = c.finish();
    if (st != FALCON_OK) return st;
    a.n = c.n;
    a.w = weight;
    a.b = bias;
    a.lengths = lengths;
    a.dw = dweight;
    a.db = dbias;
    a.eps = eps;
    a.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    if (c.n.B * c.n.H == 0 || c.n.T == 0) {  // no rows: the sums are zero
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        for (float* p : {dweight, dbias})
            if (p && chans && cudaMemsetAsync(p, 0, chans * 4, s) != cudaSuccess) return result(FALCON_ERR_CUDA);
        return FALCON_OK;
    }
    return result(falcon::launch_gn_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
