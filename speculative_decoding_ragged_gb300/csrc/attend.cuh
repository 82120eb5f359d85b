// attend.cuh — what the attention kernels share: the call's arguments, what a row sees, a request's rows.
#pragma once

#include "cache.cuh"

namespace dspark {

// What the rows of a call see, a template argument of the tensor-core kernels:
//   kAll     every token up to the row's own, or the last `window` of them
//   kSinks   the last `window` tokens, and of those before them the first `sinks`
//   kSuffix  a request's own tokens, those behind its group's prefix; results of a request that has
//            one are partial, for
//   kPrefix  the rows of a whole group of requests see its shared tokens, all of them: a "request" is
//            a group, its length the prefix. Results are joined with the partial ones.
enum See { kAll = 0, kSinks = 1, kPrefix = 2, kSuffix = 3 };

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
    int sinks;                 // kSinks, and their blocks
    int sink_blocks;
    // kPrefix, kSuffix. In a kPrefix call B is the number of groups.
    int requests;
    const int32_t* group_cu;   // a group's requests: group_cu[g] .. group_cu[g + 1] - 1
    const int32_t* prefix;     // its shared tokens
    int32_t* from;             // [requests + 1] a request's first token that is its own; 0: all are, and
                               // so where negative, which a group's first request only is: minus the
                               // group's first request that has the prefix (group_lead).
                               // The last: whether prefixes are computed apart at all
    float* part_lse;           // [rows * q_heads] what the own tokens give each row: log2 of the sum
    float* part;               // [rows * q_heads, dim] and the quotient
};

size_t attend_workspace_bytes(int dim);
size_t attend_shared_workspace_bytes(int rows, int q_heads, int dim, int B);
// kAll or kSinks.
int launch_attend(const AttendCall& A, See see, int dtype, cudaStream_t stream);
int launch_attend_shared(const AttendCall& A, const int32_t* group_cu, const int32_t* prefix, int groups, int dtype,
                         cudaStream_t stream);
// The tensor-core kernel: whether it serves a call, whether its line of tiles can hold it, and its launch.
bool attend_mma_serves(const AttendCall& A, int dtype);
bool attend_mma_fits(const AttendCall& A);
int launch_attend_mma(const AttendCall& A, See see, cudaStream_t stream);

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

// A group's rows [row0, row0 + w) and its shared tokens in whole pages; w = 0 where they cannot be
// computed apart: a group of one, no whole page, rows or requests that are none.
__device__ __forceinline__ void group_shape(const AttendCall& A, int g, int* row0, int* w, int* len)
{
    const int b0 = A.group_cu[g], b1 = A.group_cu[g + 1];
    const int n = A.prefix[g] / A.c.page * A.c.page;
    *row0 = *w = 0;
    *len = n;
    // in an order in which no difference passes 32 bits, whatever the numbers are
    if (b0 < 0 || b1 < b0 || b1 > A.requests || b1 - b0 < 2 || n <= 0 || n > A.reach) return;
    const int r0 = A.cu[b0], r1 = A.cu[b1];
    if (r0 < 0 || r1 < r0 || r1 > A.rows) return;
    *row0 = r0;
    *w = r1 - r0;
}
// Whose table row a group's prefix is read by: its first request that has the prefix and rows. What stands
// in the others' rows is not known (an emptied slot's may be another request's pages by now). -1: none has.
__device__ __forceinline__ int group_lead(const AttendCall& A, int g)
{
    const int b0 = A.group_cu[g], x = A.from[b0];
    return x < 0 ? -x : x > 0 ? b0 : -1;
}
// The same of the groups that are computed apart: those that some request joins, none where it does not
// pay (all of `from` is 0). *lead: see above.
__device__ __forceinline__ void group_rows(const AttendCall& A, int g, int* row0, int* w, int* len, int* lead)
{
    group_shape(A, g, row0, w, len);
    if (*w <= 0) return;
    *lead = group_lead(A, g);
    if (*lead < 0) *w = 0;
}
// What a call takes as its requests; *from: the first token that is seen at all (kSuffix), the request that
// is read (kPrefix).
template <int SEE>
__device__ __forceinline__ void rows_of(const AttendCall& A, int b, int* row0, int* w, int* len, int* from, int* bits)
{
    if constexpr (SEE == kPrefix) {
        group_rows(A, b, row0, w, len, from);
    } else {
        request_rows(A, b, row0, w, len, bits);
        if constexpr (SEE == kSuffix) *from = max(A.from[b], 0);
    }
}
// The tokens of a "request" that are in the cache, whose table row it reads (from: rows_of's), a row's position.
template <int SEE>
__device__ __forceinline__ int stored_tokens(int len, int w) { return SEE == kPrefix ? len : len + w; }
template <int SEE>
__device__ __forceinline__ int table_of(int b, int from) { return SEE == kPrefix ? from : b; }
template <int SEE>
__device__ __forceinline__ int position(int len, int i) { return SEE == kPrefix ? len - 1 : len + i; }
// The first token that a row at this position sees, sinks apart.
template <int SEE>
__device__ __forceinline__ int first_seen_at(const AttendCall& A, int pos, int from)
{
    if constexpr (SEE == kPrefix) return 0;
    if constexpr (SEE == kSuffix) return from;
    return A.window > 0 && pos >= A.window ? pos - A.window + 1 : 0;
}

}  // namespace dspark
