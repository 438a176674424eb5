// sv_attend_rows.cu -- the kernels of sv_attend_rows.cuh without sinks.
#include "sv_attend_rows.cuh"

namespace sv {

cudaError_t launch_attend_rows(int dtype, int dim, int mt, const AttendArgs& p, cudaStream_t s) {
    return rows_of_type<false, false>(dtype, dim, mt, p, s);
}

}  // namespace sv
