// Gated delta rule, backward: float32 inputs, dk up to 128. See falcon_gdr_bwd.cuh.

#include "falcon_gdr_bwd.cuh"

namespace falcon {
namespace gdr {

template int launch_bwd<float, 2>(const GdrArgs&, cudaStream_t);

}  // namespace gdr
}  // namespace falcon
