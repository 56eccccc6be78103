// Internal interface of the strided [B,H,T,d] operators (gated linear recurrence, head norm): what
// falcon_seq_api.cu hands to the kernels after checking it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace falcon {

enum Gate { kGateDecay = 0, kGateSigmoid = 1, kGateMix = 2 };
enum Act { kActNone = 0, kActSilu = 1, kActGelu = 2, kActSigmoid = 3 };

// A [B,H,T,d] tensor: strides in elements, channels contiguous; the stride of an axis of length 1 is 0.
struct SeqView {
    void* p;
    long long sb, sh, st;
};

struct SeqSizes {
    long long B, H;
    int T, d;
    int bf16;
};

struct GlrArgs {
    int gate;
    SeqSizes n;
    SeqView x, g, out, dout, dx, dg;  // forward: x, g, out
    const float* h0;                  // [B,H,d]; may be null, as may all below
    const int32_t* lengths;
    float* h_final;                   // forward
    const float* dh_final;            // backward
    float* dh0;
};
int launch_glr_fwd(const GlrArgs& a, cudaStream_t s);
int launch_glr_bwd(const GlrArgs& a, cudaStream_t s);
// Reads and clears the kernels' timeout flag (synchronous).
int glr_consume_timeout_flag(int* flag);

struct GnArgs {
    int act;
    SeqSizes n;
    SeqView x, z, y, dy, dx, dz;  // z.p, dz.p null without a gate; forward: x, z, y
    const float* w;               // [H,d] or null
    const float* b;
    const int32_t* lengths;
    float* dw;
    float* db;
    float eps;
    float* ws;                    // partial sums, gn_bwd_splits x 2 x H x d
};
constexpr int kGnMaxD = 1024;
int launch_gn_fwd(const GnArgs& a, cudaStream_t s);
int launch_gn_bwd(const GnArgs& a, cudaStream_t s);
// CTAs per head in falcon_gn_bwd; a function of the sizes alone, so that sums keep their order.
int gn_bwd_splits(const SeqSizes& n);

// Whether every access through `v` can move `bytes` at a time.
inline bool seq_vec_ok(const SeqView& v, int es, int bytes) {
    const long long m = bytes / es;
    return (reinterpret_cast<uintptr_t>(v.p) % (uintptr_t)bytes) == 0 && v.sb % m == 0 && v.sh % m == 0 &&
           v.st % m == 0;
}

}  // namespace falcon
