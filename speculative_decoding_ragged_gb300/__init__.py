"""GB300-native (sm_103a) DSpark ragged-verification hot path.

Four calls make one decode step of confidence-driven variable-length speculative
verification ("DSpark in SGLang: Speculative Decoding with Confidence-Driven, Variable-Length
Verification"): dspark_schedule -> dspark_pack -> dspark_verify -> dspark_scatter. They are
implemented as hand-written CUDA kernels in libdspark.so (C ABI: include/dspark.h); this
package is the ctypes binding (`_binding`), the in-tree build (`build`), a buffer-owning step
runner (`step`) and the seeded synthetic workloads (`synth`).
"""
from ._binding import (BF16, CAP_ACCEPT, COMPACT, F32, MODES, STATIC, Adjustments, CostTable, DSparkError,  # noqa: F401
                       PagedCache, Rope, dspark_adjust, dspark_append, dspark_attend, dspark_attend_shared,
                       dspark_attend_shared_workspace_bytes, dspark_attend_sinks,
                       dspark_attend_workspace_bytes, dspark_pack, dspark_rotate, dspark_scatter, dspark_schedule, dspark_verify,
                       dspark_verify_workspace_bytes, last_error, lib, version)
