// sv_attend_tiles_8bit.cu -- the kernels of sv_attend_tiles.cuh over a cache held in 8 bits, with or
// without sinks.
#include "sv_attend_tiles.cuh"

namespace sv {

cudaError_t launch_attend_tiles_8bit(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    return tiles_of_type<true, true>(dtype, dim, rm, p, s);
}

}  // namespace sv
