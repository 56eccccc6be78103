// C-ABI front end of the strided [B,H,T,d] operators: argument checking for falcon_glr_fwd,
// falcon_glr_bwd, falcon_gn_fwd and falcon_gn_bwd. The contract is documented in include/falcon.h.

#include <cuda_runtime.h>
#include <stdint.h>

#include "falcon.h"
#include "falcon_check.h"
#include "falcon_seq.h"

namespace {

using falcon::SeqSizes;
using falcon::SeqView;
using namespace falcon::check;

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

// The tensors of one call, by their place in its list of strides.
struct SeqChecker : Checker {
    SeqSizes n;
    const int64_t* strides;

    SeqView view(const void* p, int k, bool written, bool required = true) {
        return Checker::view(p, Shape{n.B, n.H, n.T, n.d, n.bf16 ? 2 : 4}, strides ? strides + 3 * k : nullptr, written,
                             required);
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

}  // namespace

extern "C" {

int falcon_glr_fwd(int gate, const void* x, const void* g, const float* h0, const int32_t* lengths, void* out,
                   float* h_final, const falcon_seq_dims_t* dims, const int64_t* strides, void* stream) {
    if (gate < FALCON_GATE_DECAY || gate > FALCON_GATE_MIX) return FALCON_ERR_INVALID_ARG;
    SeqChecker c = {};
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
    SeqChecker c = {};
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

int falcon_gn_fwd(int act, const void* x, const void* z, const float* weight, const float* bias,
                  const int32_t* lengths, void* y, const falcon_seq_dims_t* dims, const int64_t* strides, float eps,
                  void* stream) {
    if (act < FALCON_ACT_NONE || act > FALCON_ACT_SIGMOID || !good_eps(eps)) return FALCON_ERR_INVALID_ARG;
    SeqChecker c = {};
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
    SeqChecker c = {};
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
