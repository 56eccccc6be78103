// C-ABI front end of the gated delta rule and the root-mean-square norm: argument checking for falcon_gdr_fwd,
// falcon_gdr_bwd, falcon_rms_fwd and falcon_rms_bwd. The contract is documented in include/falcon.h.

#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "falcon.h"
#include "falcon_check.h"
#include "falcon_gdr.h"
#include "falcon_rms.h"

namespace {

using namespace falcon::check;
using falcon::GdrSizes;
using falcon::RowView;
using falcon::SeqView;

int sizes_of(const falcon_gdr_dims_t* d, GdrSizes* n) {
    if (!d || d->batch < 0 || d->heads < 0 || d->qk_heads < 0 || d->seqlen < 0 || d->dk <= 0 || d->dv <= 0 || d->reserved != 0)
        return FALCON_ERR_INVALID_ARG;
    if (d->heads > 0 && (d->qk_heads == 0 || d->heads % d->qk_heads != 0)) return FALCON_ERR_INVALID_ARG;
    if (d->dtype != FALCON_F32 && d->dtype != FALCON_BF16) return FALCON_ERR_UNSUPPORTED;
    if (d->dk > falcon::kGdrMaxD || d->dv > falcon::kGdrMaxD) return FALCON_ERR_UNSUPPORTED;
    if (d->batch >= kMax || d->heads >= kMax || d->qk_heads >= kMax || d->seqlen >= kMax / 2) return FALCON_ERR_UNSUPPORTED;
    n->B = d->batch;
    n->H = d->heads;
    n->Hk = d->heads > 0 ? d->qk_heads : 0;
    n->T = (int)d->seqlen;
    n->dk = (int)d->dk;
    n->dv = (int)d->dv;
    n->bf16 = d->dtype == FALCON_BF16;
    return falcon::gdr_fits(*n) ? FALCON_OK : FALCON_ERR_UNSUPPORTED;
}

struct GdrChecker : Checker {
    GdrSizes n;
    const int64_t* strides;

    const int64_t* at(int k) const { return strides ? strides + 3 * k : nullptr; }
    int es() const { return n.bf16 ? 2 : 4; }
    SeqView qk(const void* p, int k, bool written) { return view(p, Shape{n.B, n.Hk, n.T, n.dk, es()}, at(k), written); }
    SeqView v(const void* p, int k, bool written) { return view(p, Shape{n.B, n.H, n.T, n.dv, es()}, at(k), written); }
    SeqView token(const void* p, int k, bool written) { return view(p, Shape{n.B, n.H, n.T, 1, 4}, at(k), written); }
    uint64_t state() const { return (uint64_t)n.B * n.H * n.dk * n.dv; }
    void workspace(const void* p, size_t bytes, unsigned long long need) {
        if (need == 0) return;
        if (!p || bytes < need) return fail(FALCON_ERR_INVALID_ARG);
        if (!aligned(p, 256)) return fail(FALCON_ERR_MISALIGNED);
        dense(p, need / 4, true);
    }
};

bool good_scale(float s) { return std::isfinite(s); }

int sizes_of(const falcon_rms_dims_t* d, falcon::RmsArgs* a) {
    if (!d || d->batch < 0 || d->seqlen < 0 || d->d <= 0) return FALCON_ERR_INVALID_ARG;
    if (d->dtype != FALCON_F32 && d->dtype != FALCON_BF16) return FALCON_ERR_UNSUPPORTED;
    if (d->out_dtype != d->dtype && d->out_dtype != FALCON_E4M3) return FALCON_ERR_UNSUPPORTED;
    if (d->d > falcon::kRmsMaxD || d->batch >= kMax || d->seqlen >= kMax / 2) return FALCON_ERR_UNSUPPORTED;
    if ((u128)d->batch * (uint64_t)d->seqlen >= (uint64_t)kMax) return FALCON_ERR_UNSUPPORTED;
    a->B = d->batch;
    a->T = (int)d->seqlen;
    a->d = (int)d->d;
    a->bf16 = d->dtype == FALCON_BF16;
    a->eight = d->out_dtype == FALCON_E4M3;
    return FALCON_OK;
}

struct RmsChecker : Checker {
    int64_t B, T, d;
    const int64_t* strides;

    RowView row(const void* p, int k, int es, bool written, bool required = true, bool count = true) {
        int64_t s[3];
        if (strides) s[0] = strides[2 * k], s[1] = 0, s[2] = strides[2 * k + 1];
        const int i = nin;
        const SeqView v = view(p, Shape{B, 1, T, d, es}, strides ? s : nullptr, written, required);
        if (!count) nin = i;
        return RowView{v.p, v.sb, v.st};
    }
};
bool same(const RowView& a, const RowView& b) { return a.p == b.p && a.sb == b.sb && a.st == b.st; }

}  // namespace

extern "C" {

size_t falcon_gdr_workspace_bytes(const falcon_gdr_dims_t* dims, int backward) {
    GdrSizes n = {};
    if (sizes_of(dims, &n) != FALCON_OK || n.B * n.H == 0) return 0;
    return (size_t)(backward ? falcon::gdr_bwd_workspace(n) : falcon::gdr_fwd_workspace(n));
}

int falcon_gdr_fwd(const void* q, const void* k, const void* v, const float* beta, const float* g, const float* S0,
                   const int32_t* lengths, void* out, float* S_final, const falcon_gdr_dims_t* dims,
                   const int64_t* strides, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!good_scale(scale)) return FALCON_ERR_INVALID_ARG;
    GdrChecker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    c.strides = strides;
    falcon::GdrArgs a = {};
    a.q = c.qk(q, 0, false);
    a.k = c.qk(k, 1, false);
    a.v = c.v(v, 2, false);
    a.beta = c.token(beta, 3, false);
    a.g = c.token(g, 4, false);
    a.out = c.v(out, 5, true);
    if (S0 != S_final) c.dense(S0, c.state(), false);  // equal: the state is updated in place
    c.dense(lengths, c.n.B, false);
    c.dense(S_final, c.state(), true);
    const bool some = c.n.B * c.n.H > 0;
    c.workspace(workspace, workspace_bytes, some ? falcon::gdr_fwd_workspace(c.n) : 0);
    st = c.finish();
    if (st != FALCON_OK || !some) return st;
    a.n = c.n;
    a.S0 = S0;
    a.lengths = lengths;
    a.S_final = S_final;
    a.scale = scale;
    a.ws = static_cast<float*>(workspace);
    return result(falcon::launch_gdr_fwd(a, static_cast<cudaStream_t>(stream)));
}

int falcon_gdr_bwd(const void* q, const void* k, const void* v, const float* beta, const float* g, const float* S0,
                   const int32_t* lengths, const void* dout, const float* dS_final, void* dq, void* dk, void* dv,
                   float* dbeta, float* dg, float* dS0, const falcon_gdr_dims_t* dims, const int64_t* strides,
                   float scale, void* workspace, size_t workspace_bytes, void* stream) {
    if (!good_scale(scale)) return FALCON_ERR_INVALID_ARG;
    GdrChecker c = {};
    int st = sizes_of(dims, &c.n);
    if (st != FALCON_OK) return st;
    c.strides = strides;
    falcon::GdrArgs a = {};
    a.q = c.qk(q, 0, false);
    a.k = c.qk(k, 1, false);
    a.v = c.v(v, 2, false);
    a.beta = c.token(beta, 3, false);
    a.g = c.token(g, 4, false);
    a.dout = c.v(dout, 5, false);
    a.dq = c.qk(dq, 6, true);
    a.dk = c.qk(dk, 7, true);
    a.dv = c.v(dv, 8, true);
    a.dbeta = c.token(dbeta, 9, true);
    a.dg = c.token(dg, 10, true);
    c.dense(S0, c.state(), false);
    c.dense(lengths, c.n.B, false);
    c.dense(dS_final, c.state(), false);
    c.dense(dS0, c.state(), true);
    const bool some = c.n.B * c.n.H > 0;
    c.workspace(workspace, workspace_bytes, some ? falcon::gdr_bwd_workspace(c.n) : 0);
    st = c.finish();
    if (st != FALCON_OK || !some) return st;
    a.n = c.n;
    a.S0 = S0;
    a.lengths = lengths;
    a.dS_final = dS_final;
    a.dS0 = dS0;
    a.scale = scale;
    a.ws = static_cast<float*>(workspace);
    return result(falcon::launch_gdr_bwd(a, static_cast<cudaStream_t>(stream)));
}

int falcon_rms_fwd(const void* x, const void* residual, const float* weight, const int32_t* lengths, void* h, void* y,
                   float* scales, const falcon_rms_dims_t* dims, const int64_t* strides, float eps, void* stream) {
    if (!good_eps(eps) || (h && !residual)) return FALCON_ERR_INVALID_ARG;
    falcon::RmsArgs a = {};
    int st = sizes_of(dims, &a);
    if (st != FALCON_OK) return st;
    if ((scales != nullptr) != (a.eight != 0) && a.B * a.T > 0) return FALCON_ERR_INVALID_ARG;
    RmsChecker c = {};
    c.B = a.B, c.T = a.T, c.d = a.d;
    c.strides = strides;
    const int es = a.bf16 ? 2 : 4;
    a.h = c.row(h, 2, es, true, false);
    // h may be x or residual: a token is read whole before it is written
    a.x = c.row(x, 0, es, false, true, h == nullptr || h != x);
    a.residual = c.row(residual, 1, es, false, false, h == nullptr || h != residual);
    if (c.status == FALCON_OK && h && ((h == x && !same(a.h, a.x)) || (h == residual && !same(a.h, a.residual))))
        return FALCON_ERR_INVALID_ARG;
    a.y = c.row(y, 3, a.eight ? 1 : es, true);
    c.dense(weight, a.d, false);
    c.dense(lengths, a.B, false);
    c.dense(scales, (uint64_t)a.B * a.T, true);
    st = c.finish();
    if (st != FALCON_OK || a.B * a.T == 0) return st;
    a.weight = weight;
    a.lengths = lengths;
    a.scales = scales;
    a.eps = eps;
    return result(falcon::launch_rms_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t falcon_rms_bwd_workspace_bytes(const falcon_rms_dims_t* dims) {
    falcon::RmsArgs a = {};
    if (sizes_of(dims, &a) != FALCON_OK || a.B * a.T == 0) return 0;
    return (size_t)falcon::rms_bwd_splits(a.B * a.T, a.d, a.bf16) * a.d * sizeof(float);
}

int falcon_rms_bwd(const void* h, const float* weight, const int32_t* lengths, const void* dy, const void* dh, void* dx,
                   float* dweight, const falcon_rms_dims_t* dims, const int64_t* strides, float eps, void* workspace,
                   size_t workspace_bytes, void* stream) {
    if (!good_eps(eps)) return FALCON_ERR_INVALID_ARG;
    falcon::RmsArgs a = {};
    int st = sizes_of(dims, &a);
    if (st != FALCON_OK) return st;
    if (a.eight) return FALCON_ERR_UNSUPPORTED;  // the gradient is of the sums, not of the 8-bit values
    RmsChecker c = {};
    c.B = a.B, c.T = a.T, c.d = a.d;
    c.strides = strides;
    const int es = a.bf16 ? 2 : 4;
    a.x = c.row(h, 0, es, false);
    a.dy = c.row(dy, 1, es, false);
    a.dx = c.row(dx, 3, es, true);
    a.dh = c.row(dh, 2, es, false, false, dh == nullptr || dh != dx);  // dx may be dh: the stream's gradient in place
    if (c.status == FALCON_OK && dh && dh == dx && !same(a.dh, a.dx)) return FALCON_ERR_INVALID_ARG;
    c.dense(weight, a.d, false);
    c.dense(lengths, a.B, false);
    c.dense(dweight, a.d, true);
    const size_t need = dweight ? falcon_rms_bwd_workspace_bytes(dims) : 0;
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return FALCON_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return FALCON_ERR_MISALIGNED;
        c.dense(workspace, need / 4, true);
    }
    st = c.finish();
    if (st != FALCON_OK) return st;
    a.weight = weight;
    a.lengths = lengths;
    a.dweight = dweight;
    a.eps = eps;
    a.ws = need > 0 ? static_cast<float*>(workspace) : nullptr;
    if (a.B * a.T == 0) {  // no tokens: the sum is zero
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        if (dweight && cudaMemsetAsync(dweight, 0, (size_t)a.d * 4, s) != cudaSuccess) return result(FALCON_ERR_CUDA);
        return FALCON_OK;
    }
    return result(falcon::launch_rms_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
