// append.cu — dspark_append: a step's keys and values, rotated, quantised and written to the
// paged 8-bit cache, its queries rotated on the way.
//
// A block is one page's slots of one kv head; its scale is a power of two, so that growing it
// rescales the codes already there by an exact shift of their exponent (only codes that leave
// e4m3's normal range round again), and multiplying by it is exact. The step's rows that fall
// into one block are consecutive packed rows; the first of them leads. One warp owns a block (of
// keys or of values): it finds the block's rows, their largest magnitude, hence the scale,
// requantises the retained codes if the scale grew, and writes the rows' codes. No two warps touch
// one block, so there are no atomics and the result does not depend on any order.
//
// A CTA takes one packed row (several where there are many rows) and the blocks of four heads'
// keys and values that it leads; the rotation's factors of the block's rows are computed once per
// CTA in shared memory. A window's few rows stay in registers between the maximum and the codes; a
// prompt's are read again, from L1 or L2, and the factors kept.
// Bound by memory for prompts, by the chain of dependent loads (row owner, length, page id,
// scale, retained codes) for a step.
#include "cache.cuh"
#include "rope.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTable = 4096;       // shared rope factors (32 KB): 64 rows of 64 pairs
constexpr int kKeep = 4;           // units of a lane that stay in registers

struct AppendArgs {
    dspark_cache c;
    Rope rope;
    RowsIn k, v, q;
    RowsOut q_out;
    const int32_t* row_req;
    const int32_t* row_pos;
    const int32_t* lengths;
    int rows, B, q_heads;
    int kv_ctas;          // first of the grid: (rows, eight blocks)
    int per_row;          // of them for the same rows
    int chunk;            // rows a kv CTA looks for leaders in
    int q_rows;           // rows a query CTA rotates
    int32_t* status;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Unit u of a row: N elements that are loaded, turned and stored together.
//   VEC (N = 8): four pairs of the rotated part, or eight neighbours past it;
//   else (N = 2): one pair, or two neighbours.
template <bool VEC>
struct Unit {
    static constexpr int N = VEC ? 8 : 2;
    int a, b;             // first element of either half of the unit
    int pair;             // first pair, or -1: not rotated
    bool split;           // the halves are apart: (a + j, b + j) are pairs
    __device__ __forceinline__ Unit(const Rope& r, int u)
    {
        const int p = u * (N / 2);
        pair = p < r.half ? p : -1;
        split = pair >= 0 && !r.interleaved;
        a = split ? p : u * N;
        b = split ? p + r.half : a + N / 2;
    }
};

template <int DT, bool VEC>
__device__ __forceinline__ void load_unit(const void* base, int64_t at, const Unit<VEC>& un, float* x)
{
    if (!VEC) {
        x[0] = load1<DT>(base, at + un.a);
        x[1] = load1<DT>(base, at + un.b);
    } else if (DT == DSPARK_BF16) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        const uint2 a = *reinterpret_cast<const uint2*>(p + un.a), b = *reinterpret_cast<const uint2*>(p + un.b);
        x[0] = bf16_lo(a.x); x[1] = bf16_hi(a.x); x[2] = bf16_lo(a.y); x[3] = bf16_hi(a.y);
        x[4] = bf16_lo(b.x); x[5] = bf16_hi(b.x); x[6] = bf16_lo(b.y); x[7] = bf16_hi(b.y);
    } else {
        const float* p = static_cast<const float*>(base) + at;
        const float4 a = *reinterpret_cast<const float4*>(p + un.a), b = *reinterpret_cast<const float4*>(p + un.b);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

// Non-finite elements count as 0; the rotated ones turn. Returns whether anything was not finite.
template <bool VEC>
__device__ __forceinline__ bool turn_unit(const Rope& r, const Unit<VEC>& un, const float2* tab, float* x)
{
    constexpr int N = Unit<VEC>::N;
    bool bad = false;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (!finite(x[j])) { x[j] = 0.0f; bad = true; }
    if (un.pair < 0) return bad;
    if (un.split) {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 t = rope_turn(x[j], x[j + N / 2], tab[un.pair + j]);
            x[j] = t.x;
            x[j + N / 2] = t.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            const float2 t = rope_turn(x[2 * j], x[2 * j + 1], tab[un.pair + j]);
            x[2 * j] = t.x;
            x[2 * j + 1] = t.y;
        }
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (!finite(x[j])) { x[j] = 0.0f; bad = true; }      // the sum of two products overflowed
    return bad;
}

template <bool VEC>
__device__ __forceinline__ float amax_unit(const float* x, float m)
{
#pragma unroll
    for (int j = 0; j < Unit<VEC>::N; ++j) m = fmaxf(m, fabsf(x[j]));
    return m;
}

template <bool VEC>
__device__ __forceinline__ void store_unit(uint8_t* row, const Unit<VEC>& un, const float* x, float inv)
{
    if (VEC) {
        const uint32_t a = e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        const uint32_t b = e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv);
        if (un.split) {
            *reinterpret_cast<uint32_t*>(row + un.a) = a;
            *reinterpret_cast<uint32_t*>(row + un.b) = b;
        } else {
            *reinterpret_cast<uint2*>(row + un.a) = make_uint2(a, b);
        }
    } else {
        const uint32_t e = e4m3x4(x[0] * inv, x[1] * inv, 0.0f, 0.0f);
        row[un.a] = static_cast<uint8_t>(e & 0xff);
        row[un.b] = static_cast<uint8_t>((e >> 8) & 0xff);
    }
}

// A block's scale from its rows' largest magnitude; the retained codes follow it. One warp.
__device__ __forceinline__ float settle_scale(float amax, float* scale, uint8_t* codes, int retained, int lane)
{
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const float fresh = exp2i(scale_exponent(amax));
    if (retained == 0) {
        if (lane == 0) *scale = fresh;
        return fresh;
    }
    const float old = *scale;
    __syncwarp();                          // read by all before one writes it
    const float s = fmaxf(old, fresh);
    if (s > old) {
        if (lane == 0) *scale = s;
        const float ratio = old / s;
        uint4* kept = reinterpret_cast<uint4*>(codes);
#pragma unroll 2
        for (int i = lane; i < retained / 16; i += 32) {
            const uint4 c = kept[i];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[4];
                e4m3x4_to_f32(w[k], f);
                o[k] = e4m3x4(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
            }
            kept[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    return s;
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

// The blocks that packed row r (request b's row i0, at position pos) leads: eight of them from hv0,
// one per warp. Returns status bits.
template <int DT, bool VEC>
__device__ __forceinline__ int append_blocks(const AppendArgs& A, int64_t r, int b, int i0, int pos, int hv0,
                                             float2* tab)
{
    const dspark_cache& c = A.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slot0 = pos & (c.page - 1), block = pos / c.page;
    const int page = block < c.width ? c.table[static_cast<int64_t>(b) * c.width + block] : -1;
    if (page < 0 || page >= c.n_pages) return DSPARK_STATUS_BAD_PAGE;
    // the block's rows: the packed rows that follow, while they are b's next positions
    const int most = c.page - slot0;
    int n = 1;
    for (int j0 = 1; j0 < most; j0 += 32) {
        const int j = j0 + lane;
        const bool mine = j < most && r + j < A.rows && A.row_req[r + j] == b && A.row_pos[r + j] == i0 + j;
        const unsigned run = __ballot_sync(0xffffffffu, mine);
        n += run == 0xffffffffu ? 32 : __ffs(~run) - 1;
        if (run != 0xffffffffu) break;
    }
    const int hv = hv0 + warp;
    const bool works = hv < 2 * c.heads, value = hv & 1;
    const int h = hv >> 1;
    const int half = A.rope.half;
    const int units = c.dim / Unit<VEC>::N;
    // Lanes over units, `step` rows at a time; a head wider than a warp's units (scalar accesses
    // only) takes several turns over a row.
    const int wide = units > 32 ? 32 : units, step = 32 / wide;
    const int k0 = lane / wide, u0 = lane - k0 * wide;
    const bool has = works && k0 < step;
    Rope rope = A.rope;
    if (value) rope.half = 0;
    const RowsIn in = value ? A.v : A.k;
    const int64_t bh = static_cast<int64_t>(page) * c.heads + h;
    uint8_t* codes = static_cast<uint8_t*>(value ? c.v : c.k) + bh * c.page * c.dim;
    float* scale = (value ? c.v_scale : c.k_scale) + bh;
    const int64_t first = r * in.row_stride + static_cast<int64_t>(h) * c.dim;
    bool bad = false;
    float amax = 0.0f;

    const int rows_at_once = half > 0 ? kTable / half : n;       // factors for so many rows fit
    auto factors = [&](int from, int m) {
        __syncthreads();
        for (int i = threadIdx.x; i < m * half; i += kThreads) {
            const int k = i / half;
            tab[i] = rope_factor(A.rope, A.rope.turns[i - k * half], pos + from + k);
        }
        __syncthreads();
    };
    if (n <= kKeep * step && n <= rows_at_once && units <= 32) {
        // a window: its values stay in registers
        float x[kKeep][Unit<VEC>::N];
        const Unit<VEC> un(rope, u0);
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (has && k0 + i * step < n) load_unit<DT, VEC>(in.base, first + (k0 + i * step) * in.row_stride, un, x[i]);
        if (half > 0) factors(0, n);
        if (!works) return 0;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (has && k0 + i * step < n) {
                bad |= turn_unit<VEC>(rope, un, tab + (k0 + i * step) * half, x[i]);
                amax = amax_unit<VEC>(x[i], amax);
            }
        const float inv = 1.0f / settle_scale(amax, scale, codes, slot0 * c.dim, lane);
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (has && k0 + i * step < n)
                store_unit<VEC>(codes + static_cast<int64_t>(slot0 + k0 + i * step) * c.dim, un, x[i], inv);
    } else {
        float inv = 0.0f;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
            for (int from = 0; from < n; from += rows_at_once) {
                const int m = min(rows_at_once, n - from);
                if (half > 0 && (pass == 0 || rows_at_once < n)) factors(from, m);
                if (!has) continue;
#pragma unroll 1
                for (int u = u0; u < units; u += wide) {
                    const Unit<VEC> un(rope, u);
#pragma unroll 4
                    for (int k = k0; k < m; k += step) {
                        float x[Unit<VEC>::N];
                        load_unit<DT, VEC>(in.base, first + (from + k) * in.row_stride, un, x);
                        bad |= turn_unit<VEC>(rope, un, tab + k * half, x);
                        if (pass == 0) amax = amax_unit<VEC>(x, amax);
                        else store_unit<VEC>(codes + static_cast<int64_t>(slot0 + from + k) * c.dim, un, x, inv);
                    }
                }
            }
            if (pass == 0 && works) inv = 1.0f / settle_scale(amax, scale, codes, slot0 * c.dim, lane);
        }
    }
    return bad ? DSPARK_STATUS_BAD_VALUE : 0;
}

template <int DT, bool VEC, bool QVEC>
__global__ void __launch_bounds__(kThreads) append_kernel(AppendArgs A)
{
    __shared__ float2 tab[kTable];
    __shared__ int32_t own[8], at[8];
    pdl_wait_and_trigger();
    int bits = 0;
    if (static_cast<int>(blockIdx.x) >= A.kv_ctas) {              // queries
        const int64_t row0 = static_cast<int64_t>(blockIdx.x - A.kv_ctas) * A.q_rows;
        const int n = min(static_cast<int64_t>(A.q_rows), A.rows - row0);
        if (threadIdx.x < n) own[threadIdx.x] = row_owner(A, row0 + threadIdx.x, &at[threadIdx.x], &bits);
        __syncthreads();
        for (int i = threadIdx.x; i < n * A.rope.half; i += kThreads) {
            const int k = i / A.rope.half;
            if (own[k] >= 0)
                tab[i] = rope_factor(A.rope, A.rope.turns[i - k * A.rope.half], at[k]);
        }
        __syncthreads();
        const bool copy = !(A.q.base == A.q_out.base && A.q.row_stride == A.q_out.row_stride);
        rotate_rows<DT, QVEC>(A.rope, tab, A.q, A.q_out, row0, n, A.q_heads, A.c.dim, copy, own);
    } else {
        const int64_t row0 = static_cast<int64_t>(blockIdx.x / A.per_row) * A.chunk;
        const int hv0 = (blockIdx.x % A.per_row) * kWarps;
        // each warp looks at the rows side by side; those that lead a block are the same for all
        const int lane = threadIdx.x & 31;
        int b = -1, pos = 0, i = 0;
        if (lane < A.chunk && row0 + lane < A.rows) {
            b = row_owner(A, row0 + lane, &pos, &bits);
            if (b >= 0) i = A.row_pos[row0 + lane];
        }
        unsigned leads = __ballot_sync(0xffffffffu, b >= 0 && (i == 0 || (pos & (A.c.page - 1)) == 0));
#pragma unroll 1
        while (leads != 0) {
            const int k = __ffs(leads) - 1;
            leads &= leads - 1;
            bits |= append_blocks<DT, VEC>(A, row0 + k, __shfl_sync(0xffffffffu, b, k),
                                           __shfl_sync(0xffffffffu, i, k), __shfl_sync(0xffffffffu, pos, k), hv0, tab);
        }
    }
    if (bits) raise_status(A.status, bits);
}

bool vector_rows(const Rope& r, const void* base, int64_t stride, int dim, int elem)
{
    return dim % 8 == 0 && r.half % 4 == 0 && stride % 4 == 0 &&
           (reinterpret_cast<uintptr_t>(base) & static_cast<uintptr_t>(4 * elem - 1)) == 0;
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
    // One row per kv CTA gives a step's windows the shortest chains; of a prompt's rows only one in a
    // page leads, so a CTA looks at 16.
    A.chunk = rows <= 4096 ? 1 : 16;
    A.q_rows = rows >= 152 * 8 && rope.half > 0 ? (rope.half <= 64 ? 4 : 2) : 1;
    A.per_row = static_cast<int>(ceil_div(2 * cache.heads, kWarps));
    A.kv_ctas = static_cast<int>(ceil_div(rows, A.chunk)) * A.per_row;
    const int q_ctas = q != nullptr ? static_cast<int>(ceil_div(rows, A.q_rows)) : 0;
    const bool bf = dtype == DSPARK_BF16;
    const int e = bf ? 2 : 4;
    const bool qvec = rotate_vec(rope, q, qs, q_out, os, cache.dim, e);
    const bool vec = vector_rows(rope, k, ks, cache.dim, e) && vector_rows(rope, v, vs, cache.dim, e);
    auto kernel = bf ? (vec ? (qvec ? append_kernel<DSPARK_BF16, true, true> : append_kernel<DSPARK_BF16, true, false>)
                            : (qvec ? append_kernel<DSPARK_BF16, false, true> : append_kernel<DSPARK_BF16, false, false>))
                     : (vec ? (qvec ? append_kernel<DSPARK_F32, true, true> : append_kernel<DSPARK_F32, true, false>)
                            : (qvec ? append_kernel<DSPARK_F32, false, true> : append_kernel<DSPARK_F32, false, false>));
    return launch_pdl("append", kernel, dim3(static_cast<unsigned>(A.kv_ctas + q_ctas)),
                      dim3(kThreads), 0, stream, A);
}

}  // namespace dspark
