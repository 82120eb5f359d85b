// attend_wide_sinks.cu — the wide kernel of dspark_attend_sinks.
#include "attend_wide.cuh"

namespace dspark {

template int launch_attend_wide<kSinks>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
