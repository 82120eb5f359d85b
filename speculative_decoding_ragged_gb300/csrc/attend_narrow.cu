// attend_narrow.cu — the narrow kernel of dspark_attend.
#include "attend_narrow.cuh"

namespace dspark {

template int launch_attend_narrow<kAll>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
