// Internal interface of the root-mean-square norm: what falcon_block_api.cu hands to the kernels after checking it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace falcon {

// A [B,T,d] tensor: strides in elements, channels contiguous; the stride of an axis of length 1 is 0.
struct RowView {
    void* p;
    long long sb, st;
};

constexpr int kRmsMaxD = 16384;  // channels: 32 in each of 512 lanes

struct RmsArgs {
    long long B;
    int T, d;
    int bf16;
    int eight;                  // y holds e4m3 values, scales their factors
    RowView x, residual, h, y;  // forward; residual.p and h.p may be null
    RowView dy, dh, dx;         // backward, x the normalised sum; dh.p may be null
    const float* weight;        // [d] or null, as may all below
    const int32_t* lengths;
    float* scales;              // [B,T]
    float* dweight;             // [d]
    float eps;
    float* ws;                  // partial sums, rms_bwd_splits x d
};
int launch_rms_fwd(const RmsArgs& a, cudaStream_t s);
int launch_rms_bwd(const RmsArgs& a, cudaStream_t s);
// CTAs of the backward pass; a function of the sizes alone, so that sums keep their order.
int rms_bwd_splits(long long rows, int d, int bf16);

}  // namespace falcon
