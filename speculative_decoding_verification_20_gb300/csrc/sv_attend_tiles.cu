// sv_attend_tiles.cu -- the kernels of sv_attend_tiles.cuh without sinks.
#include "sv_attend_tiles.cuh"

namespace sv {

cudaError_t launch_attend_tiles(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    return tiles_of_type<false, false>(dtype, dim, rm, p, s);
}

}  // namespace sv
