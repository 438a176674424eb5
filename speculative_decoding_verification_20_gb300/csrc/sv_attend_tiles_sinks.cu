// sv_attend_tiles_sinks.cu -- the kernels of sv_attend_tiles.cuh with sinks behind a window.
#include "sv_attend_tiles.cuh"

namespace sv {

cudaError_t launch_attend_tiles_sinks(int dtype, int dim, int rm, const AttendArgs& p, cudaStream_t s) {
    return tiles_of_type<true, false>(dtype, dim, rm, p, s);
}

}  // namespace sv
