// Internal interface of the gated delta rule: what falcon_block_api.cu hands to the kernels after checking it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "falcon_seq.h"

namespace falcon {

constexpr int kGdrMaxD = 128;   // dk, dv
constexpr int kGdrStepT = 32;   // sequences up to this long are walked token by token, without a workspace: 12 us for 16
                                // tokens of 8 x 12 x 64 and 96 of 256 x 12, 23 and 210 in chunks whatever their number

struct GdrSizes {
    long long B, H, Hk;  // Hk heads of q and k, each shared by H / Hk consecutive heads of v
    int T, dk, dv;
    int bf16;
};

struct GdrArgs {
    GdrSizes n;
    SeqView q, k, v, out;              // [B,Hk,T,dk], [B,Hk,T,dk], [B,H,T,dv], [B,H,T,dv]
    SeqView beta, g;                   // fp32 [B,H,T]
    SeqView dout, dq, dk, dv;          // backward
    SeqView dbeta, dg;
    const float* S0;                   // fp32 [B,H,dk,dv]; may be null, as may all below
    const int32_t* lengths;
    float* S_final;
    const float* dS_final;
    float* dS0;
    float scale;
    float* ws;
};

// Workspace of one call in bytes, a function of the sizes alone; 0 where none is needed.
unsigned long long gdr_fwd_workspace(const GdrSizes& n);
unsigned long long gdr_bwd_workspace(const GdrSizes& n);
// Whether the launch shapes hold these sizes.
bool gdr_fits(const GdrSizes& n);
int launch_gdr_fwd(const GdrArgs& a, cudaStream_t s);
int launch_gdr_bwd(const GdrArgs& a, cudaStream_t s);

}  // namespace falcon
