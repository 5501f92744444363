// attnres_cached_wide4.cu -- the read over many tokens of wide rows held in 4 bits.
#include "attnres_cached_wide.cuh"

namespace attnres {

unsigned take_cached_wide4_error() { return take_error(); }

cudaError_t launch_cached_wide4(const CachedArgs& a, int sm_count, cudaStream_t stream) {
    return launch_bits<4>(a, sm_count, stream);
}

}  // namespace attnres
