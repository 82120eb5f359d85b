// attend_narrow_prefix.cu — the narrow kernel of dspark_attend_shared's prefixes.
#include "attend_narrow.cuh"

namespace dspark {

template int launch_attend_narrow<kPrefix>(const AttendCall& A, int ctas, int device, cudaStream_t stream);

}  // namespace dspark
