// sv_attend_rows_sinks.cu -- the kernels of sv_attend_rows.cuh with sinks behind a window.
#include "sv_attend_rows.cuh"

namespace sv {

cudaError_t launch_attend_rows_sinks(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    return rows_of_type<true, false>(dtype, dim, mt, p, s);
}

}  // namespace sv
