// attend_narrow_suffix.cu — the narrow kernel of dspark_attend_shared's own tokens.
#include "attend_narrow.cuh"

namespace dspark {

template int launch_attend_narrow<kSuffix>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
