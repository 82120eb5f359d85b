// attend_narrow_sinks.cu — the narrow kernel of dspark_attend_sinks.
#include "attend_narrow.cuh"

namespace dspark {

template int launch_attend_narrow<kSinks>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
