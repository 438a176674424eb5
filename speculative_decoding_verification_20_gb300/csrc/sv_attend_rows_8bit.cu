// sv_attend_rows_8bit.cu -- the kernels of sv_attend_rows.cuh over a cache held in 8 bits, with or without sinks.
#include "sv_attend_rows.cuh"

namespace sv {

cudaError_t launch_attend_rows_8bit(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    return rows_of_type<true, true>(dtype, dim, mt, p, s);
}

}  // namespace sv
