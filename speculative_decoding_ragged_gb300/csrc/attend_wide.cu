// attend_wide.cu — the wide kernel of dspark_attend.
#include "attend_wide.cuh"

namespace dspark {

template int launch_attend_wide<kAll>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
