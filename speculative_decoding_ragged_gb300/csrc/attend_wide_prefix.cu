// attend_wide_prefix.cu — the wide kernel of dspark_attend_shared's prefixes.
#include "attend_wide.cuh"

namespace dspark {

template int launch_attend_wide<kPrefix>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
