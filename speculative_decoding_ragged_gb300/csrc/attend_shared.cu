// attend_shared.cu — dspark_attend_shared: what is computed apart, and the calls of the attention kernels.
//
// With own tokens o and a prefix p, a row's result is (2^(lse_o - t) O_o + 2^(lse_p - t) O_p) / (2^(lse_o - t)
// + 2^(lse_p - t)), t the larger log2 sum. The own tokens go first, request by request in units of few
// rows, and leave each row's quotient and log2 sum in the workspace; the prefixes follow, group by group
// in units of up to 128 rows of any of its requests, and join. So the join is paid by the kernel with
// few, long units, whose parts are joined from the workspace anyway: with the own tokens last, each of
// their many short units waited for 16 KB of the prefix's results (own tokens of 256 windows of 1 to 8 rows:
// 136 us, now 78).
#include "attend_mma.cuh"

namespace dspark {
namespace {

// A prefix computed apart costs a kernel's start and its join, about 25 us; a tile of 128 tokens and a
// head that is not read again saves about 4 ns (2500 cycles on 304 CTAs). 84 answers in 12 groups behind
// 300 to 5000 tokens, 3800 tiles saved: 40 us alone, 47 apart; 192 single tokens behind 16384, 195 thousand
// tiles: 573 and 125.
constexpr int64_t kWorth = 6000;

// Whether the groups' prefixes are worth it; every request's first own token, and whose pages are read for
// a group (the first CTA); no row has a part yet (the others).
// A request joins its group where its rows are the group's too and all of the prefix lies before them: the
// prefix is then in its table. What stands in the table of one that does not join is not known. The first
// that joins is the one before which the last that does lies in front of the group; requests are taken in
// order, a thread each.
// Groups that are not in order, or whose rows are not, are not computed apart at all: the cut of the prefixes'
// kernels counts on rows that are no more than the call's.
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(AttendCall A)
{
    __shared__ int saved[kPlanWarps];
    __shared__ int last[2][kPlanWarps];          // the last request of each warp's that joins, or -1
    pdl_wait_and_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x > 0) {
        const int step = (gridDim.x - 1) * kPlanThreads;
        for (int i = (blockIdx.x - 1) * kPlanThreads + tid; i < A.rows * A.q_heads; i += step)
            A.part_lse[i] = __uint_as_float(kNoPart);
        return;
    }
    int tiles = 0;                               // saved; times the heads no more than the line may have
    bool orderly = true;
    for (int g = tid; g < A.B; g += kPlanThreads) {
        const int b0 = A.group_cu[g], b1 = A.group_cu[g + 1];
        orderly = orderly && b0 >= 0 && b1 >= b0 && b1 <= A.requests && A.cu[b0] <= A.cu[b1];
    }
    int before = -1;                             // the last request of earlier rounds that joins
    for (int base = 0; base < A.requests; base += kPlanThreads) {
        const int b = base + tid, round = base / kPlanThreads & 1;
        int b0 = 0, n = 0;
        bool joins = false;
        if (b < A.requests) {
            int row0, w, len, bits = 0;          // their loads under the search's
            request_rows(A, b, &row0, &w, &len, &bits);
            int lo = 0, hi = A.B;                // the last group that starts at or before b
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (A.group_cu[mid] <= b) lo = mid; else hi = mid;
            }
            b0 = A.group_cu[lo];
            if (b0 <= b && b < A.group_cu[lo + 1]) {
                int r0, group_w;
                group_shape(A, lo, &r0, &group_w, &n);
                joins = group_w > 0 && w > 0 && row0 >= r0 && row0 + w <= r0 + group_w && len >= n;
            }
            A.from[b] = joins ? n : 0;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, joins);
        if (lane == 0) last[round][warp] = mask != 0 ? base + warp * 32 + 31 - __clz(mask) : -1;
        __syncthreads();
        const int its = lane < kPlanWarps ? last[round][lane] : -1;
        int earlier = max(before, __reduce_max_sync(0xffffffffu, lane < warp ? its : -1));
        before = max(before, __reduce_max_sync(0xffffffffu, its));
        const uint32_t below = mask & ((1u << lane) - 1);
        if (below != 0) earlier = base + warp * 32 + 31 - __clz(below);
        if (joins && earlier >= b0) tiles += (n + kTile - 1) / kTile;    // what it does not read again
        else if (joins && b > b0) A.from[b0] = -b;
    }
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    if (lane == 0) saved[warp] = tiles;
    orderly = __syncthreads_and(orderly);
    tiles = __reduce_add_sync(0xffffffffu, lane < kPlanWarps ? saved[lane] : 0);
    const bool worth = orderly && static_cast<int64_t>(tiles) * A.c.heads >= kWorth;
    if (tid == 0) A.from[A.requests] = worth;
    for (int b = tid; !worth && b < A.requests; b += kPlanThreads) A.from[b] = 0;
}

}  // namespace

// After the parts: each row's own tokens' quotient and log2 sum, the requests' first own tokens.
size_t attend_shared_workspace_bytes(int rows, int q_heads, int dim, int B)
{
    const size_t parts = attend_workspace_bytes(dim);
    if (dim != 64 && dim != 128) return parts;
    return parts + static_cast<size_t>(rows) * q_heads * (dim + 1) * sizeof(float) +
           (static_cast<size_t>(B) + 1) * sizeof(int32_t);
}

// Types and head sizes of the fp32 kernel have no such form: it attends over the whole contexts. So do
// calls whose page tables are too small for any prefix to be worth computing apart (4 windows of 4 rows
// behind 1000 tokens: 14 us alone, 33 apart, 21 with a plan that says so), and calls with so many groups
// that the prefixes' line could not hold them. All of that is known before anything is enqueued.
int launch_attend_shared(const AttendCall& A, const int32_t* group_cu, const int32_t* prefix, int groups, int dtype,
                         cudaStream_t stream)
{
    const int64_t most = (A.B - 1ll) * ((A.reach + kTile - 1ll) / kTile) * A.c.heads;
    AttendCall own = A;
    own.requests = A.B;
    own.group_cu = group_cu;
    own.prefix = prefix;
    own.part = reinterpret_cast<float*>(static_cast<char*>(A.ws) + attend_workspace_bytes(A.c.dim));
    own.part_lse = own.part + static_cast<int64_t>(A.rows) * A.q_heads * A.c.dim;
    own.from = reinterpret_cast<int32_t*>(own.part_lse + static_cast<int64_t>(A.rows) * A.q_heads);
    AttendCall shared = own;
    shared.B = groups;
    if (groups == 0 || most < kWorth || !attend_mma_serves(A, dtype) || !attend_mma_fits(own) || !attend_mma_fits(shared))
        return launch_attend(A, kAll, dtype, stream);
    const int64_t ctas = ceil_div(static_cast<int64_t>(A.rows) * A.q_heads, kPlanThreads);
    int rc = launch_pdl("attend plan", plan_kernel, dim3(static_cast<unsigned>(ctas < 64 ? ctas : 64) + 1),
                        dim3(kPlanThreads), 0, stream, shared);
    if (rc == DSPARK_OK) rc = launch_attend_mma(own, kSuffix, stream);
    return rc == DSPARK_OK ? launch_attend_mma(shared, kPrefix, stream) : rc;
}

}  // namespace dspark
