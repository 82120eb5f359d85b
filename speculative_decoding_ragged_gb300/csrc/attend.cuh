// attend.cuh — what the two attention kernels share: the call's arguments and a request's rows.
#pragma once

#include "cache.cuh"

namespace dspark {

struct AttendCall {
    dspark_cache c;
    const void* q;
    int64_t q_stride;
    void* out;
    int64_t out_stride;
    int q_heads, group;        // group: query heads per cache head
    int rows;
    const int32_t* cu;
    const int32_t* lengths;
    int B;
    float scale;
    int window;
    float* lse;
    int reach;                 // tokens that the page table reaches
    int last_tile;             // the last 128-token tile of them
    void* ws;
    int32_t* status;
};

size_t attend_workspace_bytes(int dim);
int launch_attend(const AttendCall& A, int dtype, cudaStream_t stream);
// The tensor-core kernel: whether it serves a call, and its launch.
bool attend_mma_serves(const AttendCall& A, int dtype);
int launch_attend_mma(const AttendCall& A, cudaStream_t stream);

// Request b's packed rows [row0, row0 + w) and its length, checked: w = 0 for one whose rows are
// not within the buffer. *bits collects what was wrong, tokens past the page table included.
__device__ __forceinline__ void request_rows(const AttendCall& A, int b, int* row0, int* w,
                                             int* len, int* bits)
{
    const int r0 = A.cu[b], r1 = A.cu[b + 1];
    int n = A.lengths[b];
    if (n < 0) { n = 0; *bits |= DSPARK_STATUS_BAD_LENGTH; }
    *row0 = r0;
    *w = r1 - r0;
    *len = n;
    if (r0 < 0 || r1 < r0 || r1 > A.rows) { *w = 0; *bits |= DSPARK_STATUS_BAD_ROWS; }
    else if (n > INT32_MAX - 256 - *w) { *w = 0; *bits |= DSPARK_STATUS_BAD_LENGTH; }
    else if (*w > 0 && n + *w > A.reach) *bits |= DSPARK_STATUS_BAD_PAGE;
}

}  // namespace dspark
