// append.cu — dspark_append: a step's keys and values, rotated, quantised and written to the
// paged 8-bit cache, its queries rotated on the way.
//
// A block is one page's slots of one kv head; its scale is a power of two, so that growing it
// rescales the codes already there by an exact shift of their exponent (only codes that leave
// e4m3's normal range round again), and multiplying by it is exact. The step's rows that fall
// into one block are consecutive packed rows; the first of them leads. One CTA owns a block: it
// finds the block's rows, their largest magnitude, hence the scale, requantises the retained
// codes if the scale grew, and writes the rows' codes. No two CTAs touch one block, so there are
// no atomics and the result does not depend on any order.
//
// Bound by memory for prompts, by the chain of dependent loads (row owner, length, page id,
// scale, retained codes) for a step.
#include "cache.cuh"
#include "rope.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTable = 1024;       // shared rope factors (8 KB)

struct AppendArgs {
    dspark_cache c;
    Rope rope;
    RowsIn k, v, q;
    RowsOut q_out;
    const int32_t* row_req;
    const int32_t* row_pos;
    const int32_t* lengths;
    int rows, B, q_heads;
    int kv_ctas;          // first of the grid: (row chunk, head, K or V)
    int chunk;            // rows a kv CTA looks for leaders in
    int q_rows;           // rows a query CTA rotates
    int32_t* status;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Elements 2i, 2i+1 of a pair slot: pair i of the rotated part, or two neighbours past it.
__device__ __forceinline__ int2 pair_at(const Rope& r, int i)
{
    if (i < r.half) return r.interleaved ? make_int2(2 * i, 2 * i + 1) : make_int2(i, i + r.half);
    return make_int2(2 * i, 2 * i + 1);
}

template <int DT>
__device__ __forceinline__ float2 load_pair(const AppendArgs& A, RowsIn x, const Rope& r,
                                            int64_t row, int h, int i, int pos, int* bad)
{
    const int2 at = pair_at(r, i);
    const int64_t base = row * x.row_stride + static_cast<int64_t>(h) * A.c.dim;
    float2 p = make_float2(load1<DT>(x.base, base + at.x), load1<DT>(x.base, base + at.y));
    if (!finite(p.x)) { p.x = 0.0f; *bad = 1; }
    if (!finite(p.y)) { p.y = 0.0f; *bad = 1; }
    if (i < r.half) {
        p = rope_turn(p.x, p.y, rope_factor(r, r.turns[i], pos));
        if (!finite(p.x)) { p.x = 0.0f; *bad = 1; }   // the sum of two products overflowed
        if (!finite(p.y)) { p.y = 0.0f; *bad = 1; }
    }
    return p;
}

template <int DT>
__device__ void append_block(const AppendArgs& A, int which, int h, int64_t row0, int b, int pos0,
                             int n, float* red)
{
    const dspark_cache& c = A.c;
    const int slot0 = pos0 % c.page;
    const int block = pos0 / c.page;
    const int page = block < c.width ? c.table[static_cast<int64_t>(b) * c.width + block] : -1;
    if (page < 0 || page >= c.n_pages) {
        if (threadIdx.x == 0) raise_status(A.status, DSPARK_STATUS_BAD_PAGE);
        return;
    }
    Rope r = A.rope;
    if (which) r.half = 0;                 // values are not rotated
    const RowsIn x = which ? A.v : A.k;
    const int64_t bh = static_cast<int64_t>(page) * c.heads + h;
    uint8_t* codes = static_cast<uint8_t*>(which ? c.v : c.k) + bh * c.page * c.dim;
    float* scale = (which ? c.v_scale : c.k_scale) + bh;

    int bad = 0;
    float amax = 0.0f;
    const int pairs = c.dim / 2;
    for (int u = threadIdx.x; u < n * pairs; u += kThreads) {
        const int k = u / pairs, i = u - k * pairs;
        const float2 p = load_pair<DT>(A, x, r, row0 + k, h, i, pos0 + k, &bad);
        amax = fmaxf(amax, fmaxf(fabsf(p.x), fabsf(p.y)));
    }
    for (int off = 16; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    const float old = slot0 > 0 ? *scale : 0.0f;     // read by all before thread 0 writes it
    __syncthreads();
    amax = red[0];
    for (int w = 1; w < kWarps; ++w) amax = fmaxf(amax, red[w]);
    const float fresh = exp2i(scale_exponent(amax));
    const float s = slot0 > 0 ? fmaxf(old, fresh) : fresh;
    if (threadIdx.x == 0) *scale = s;

    if (slot0 > 0 && s > old) {
        const float ratio = old / s;
        uint32_t* kept = reinterpret_cast<uint32_t*>(codes);
        for (int u = threadIdx.x; u < slot0 * c.dim / 4; u += kThreads) {
            float f[4];
            e4m3x4_to_f32(kept[u], f);
            kept[u] = e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
        }
    }
    const float inv = 1.0f / s;            // exact: s is a power of two unless the caller's was not
    for (int u = threadIdx.x; u < n * pairs; u += kThreads) {
        const int k = u / pairs, i = u - k * pairs;
        const float2 p = load_pair<DT>(A, x, r, row0 + k, h, i, pos0 + k, &bad);
        const uint32_t e = e4m3x4(p.x * inv, p.y * inv, 0.0f, 0.0f);
        const int2 at = pair_at(r, i);
        uint8_t* to = codes + static_cast<int64_t>(slot0 + k) * c.dim;
        to[at.x] = static_cast<uint8_t>(e & 0xff);
        to[at.y] = static_cast<uint8_t>((e >> 8) & 0xff);
    }
    if (bad) raise_status(A.status, DSPARK_STATUS_BAD_VALUE);
}

// The request of packed row r and its position, or -1 (padding, or an owner outside [0, B):
// *bits tells).
__device__ __forceinline__ int row_owner(const AppendArgs& A, int64_t r, int* pos, int* bits)
{
    const int b = A.row_req[r];
    if (b < 0) return -1;
    const int i = A.row_pos[r];
    if (b >= A.B || i < 0) { *bits |= DSPARK_STATUS_BAD_ROWS; return -1; }
    const int len = A.lengths[b];
    if (len < 0 || len > INT32_MAX - i) { *bits |= DSPARK_STATUS_BAD_LENGTH; return -1; }
    *pos = len + i;
    return b;
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs A)
{
    __shared__ float2 tab[kTable];
    __shared__ int32_t own[64], at[64];
    __shared__ float red[kWarps];
    pdl_wait_and_trigger();
    int bits = 0;
    if (static_cast<int>(blockIdx.x) >= A.kv_ctas) {              // queries
        const int64_t row0 = static_cast<int64_t>(blockIdx.x - A.kv_ctas) * A.q_rows;
        const int n = min(static_cast<int64_t>(A.q_rows), A.rows - row0);
        for (int k = threadIdx.x; k < n; k += kThreads) own[k] = row_owner(A, row0 + k, &at[k], &bits);
        __syncthreads();
        for (int i = threadIdx.x; i < n * A.rope.half; i += kThreads) {
            const int k = i / A.rope.half;
            if (own[k] >= 0)
                tab[i] = rope_factor(A.rope, A.rope.turns[i - k * A.rope.half], at[k]);
        }
        __syncthreads();
        const bool copy = !(A.q.base == A.q_out.base && A.q.row_stride == A.q_out.row_stride);
        rotate_rows<DT, VEC>(A.rope, tab, A.q, A.q_out, row0, n, A.q_heads, A.c.dim, copy, own);
        raise_status(A.status, bits);
        return;
    }
    const int heads2 = A.c.heads * 2;
    const int hv = blockIdx.x % heads2;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / heads2) * A.chunk;
    const int n = min(static_cast<int64_t>(A.chunk), A.rows - row0);
    for (int k = threadIdx.x; k < n; k += kThreads) own[k] = row_owner(A, row0 + k, &at[k], &bits);
    __syncthreads();
    for (int k = 0; k < n; ++k) {
        const int b = own[k];
        if (b < 0) continue;
        const int pos = at[k];
        if (pos % A.c.page != 0 && pos != A.lengths[b]) continue;       // not the block's first
        // the block's rows: the packed rows that follow, while they are b's next positions
        const int most = A.c.page - pos % A.c.page;
        int m = 1;
        for (int j0 = 1; j0 < most; j0 += kThreads) {
            const int j = j0 + threadIdx.x;
            const int64_t r = row0 + k + j;
            const bool mine = j < most && r < A.rows && A.row_req[r] == b &&
                              A.row_pos[r] == pos - A.lengths[b] + j;
            const int run = __syncthreads_count(mine);
            m += run;
            if (run < kThreads) break;
        }
        append_block<DT>(A, hv & 1, hv >> 1, row0 + k, b, pos, m, red);
    }
    raise_status(A.status, bits);
}

}  // namespace

int launch_append(const dspark_cache& cache, const Rope& rope, const void* k, int64_t ks,
                  const void* v, int64_t vs, const void* q, int64_t qs, void* q_out, int64_t os,
                  int q_heads, int dtype, int rows, int B, const int32_t* row_req,
                  const int32_t* row_pos, const int32_t* lengths, int32_t* status,
                  cudaStream_t stream)
{
    AppendArgs A;
    A.c = cache;
    A.rope = rope;
    A.k = {k, ks};
    A.v = {v, vs};
    A.q = {q, qs};
    A.q_out = {q_out, os};
    A.row_req = row_req;
    A.row_pos = row_pos;
    A.lengths = lengths;
    A.rows = rows;
    A.B = B;
    A.q_heads = q_heads;
    A.status = status;
    A.chunk = rows <= 4096 ? 1 : 16;
    A.q_rows = rows >= 152 * 8 && rope.half > 0 ? (rope.half <= 64 ? 4 : 2) : 1;
    A.kv_ctas = static_cast<int>(ceil_div(rows, A.chunk)) * cache.heads * 2;
    const int q_ctas = q != nullptr ? static_cast<int>(ceil_div(rows, A.q_rows)) : 0;
    const bool bf = dtype == DSPARK_BF16;
    const bool vec = rotate_vec(rope, q, qs, q_out, os, cache.dim, bf ? 2 : 4);
    auto kernel = bf ? (vec ? append_kernel<DSPARK_BF16, true> : append_kernel<DSPARK_BF16, false>)
                     : (vec ? append_kernel<DSPARK_F32, true> : append_kernel<DSPARK_F32, false>);
    return launch_pdl("append", kernel, dim3(static_cast<unsigned>(A.kv_ctas + q_ctas)),
                      dim3(kThreads), 0, stream, A);
}

}  // namespace dspark
