// attnres_cached_wide8.cu -- the read over many tokens of wide rows held in 8 bits.
#include "attnres_cached_wide.cuh"

namespace attnres {

unsigned take_cached_wide8_error() { return take_error(); }

cudaError_t launch_cached_wide8(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    return launch_bits<8>(a, sm_count, stream);
}

}  // namespace attnres
