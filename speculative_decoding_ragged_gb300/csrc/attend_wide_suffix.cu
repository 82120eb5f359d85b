// attend_wide_suffix.cu — the wide kernel of dspark_attend_shared's own tokens.
#include "attend_wide.cuh"

namespace dspark {

template int launch_attend_wide<kSuffix>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
