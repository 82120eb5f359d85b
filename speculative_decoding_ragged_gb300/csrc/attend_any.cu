// attend_any.cu — dspark_attend and dspark_attend_sinks in fp32 on the ordinary cores: any supported
// head size and type.
//
// One CTA takes one packed row and one cache head, up to four of its query heads at a time; its
// warps take 32-token pieces of the row's visible tokens in turn, each with its own running
// maximum m and sum l (a piece that raises m rescales by 2^(m_old - m)), and the CTA joins them
// at the end. For the scores a lane holds one token: it reads the token's codes 16 bytes at a
// time against the queries in shared memory. For the values a lane holds dim / 32 elements and
// the weights arrive by shuffle.
// Bound by instruction issue (about 2 FMAs per code and query head plus the decoding); it serves
// the types and sizes that the tensor-core kernel does not.
#include "attend.cuh"
#include "rope.cuh"

namespace dspark {
namespace {

constexpr int kWarps = 8;
constexpr int kHeads = 4;                       // query heads per pass
constexpr int kMaxDim = DSPARK_MAX_CACHE_HEAD;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int DT, int SEE>
__global__ void __launch_bounds__(kWarps * 32) attend_any_kernel(AttendCall A)
{
    __shared__ __align__(16) float qs[kHeads][kMaxDim];
    __shared__ float acc_s[kWarps][kMaxDim];
    __shared__ float ml_s[kWarps][kHeads][2];
    __shared__ int job[4];
    pdl_wait_and_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, h = blockIdx.y;
    const int D = A.c.dim, page = A.c.page;
    if (threadIdx.x == 0) {
        int b = -1;
        if (row >= A.cu[0] && row < A.cu[A.B]) {      // the last b with cu[b] <= row
            int lo = 0, hi = A.B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (A.cu[mid] <= row) lo = mid; else hi = mid;
            }
            b = lo;
        }
        int row0 = 0, w = 0, len = 0, bits = 0;
        if (b >= 0) request_rows(A, b, &row0, &w, &len, &bits);
        if (row >= row0 + w || row < row0) b = -1;
        raise_status(A.status, bits);
        job[0] = b;
        job[1] = len + (row - row0);
    }
    __syncthreads();
    const int b = job[0];
    if (b < 0) return;
    const int pos = job[1];
    const int first = A.window > 0 && pos >= A.window ? pos - A.window + 1 : 0;
    const int32_t* table = A.c.table + static_cast<int64_t>(b) * A.c.width;

    for (int g0 = 0; g0 < A.group; g0 += kHeads) {
        const int ng = min(kHeads, A.group - g0);
        const int64_t head0 = static_cast<int64_t>(h) * A.group + g0;
        __syncthreads();
        for (int i = threadIdx.x; i < kHeads * D; i += blockDim.x) {
            const int g = i / D, d = i - g * D;
            qs[g][d] = g < ng ? load1<DT>(A.q, row * A.q_stride + (head0 + g) * D + d) *
                                    (A.scale * kLog2e) : 0.0f;
        }
        __syncthreads();
        float m[kHeads], l[kHeads], acc[kHeads][kMaxDim / 32];
        for (int g = 0; g < kHeads; ++g) {
            m[g] = -INFINITY;
            l[g] = 0.0f;
            for (int j = 0; j < kMaxDim / 32; ++j) acc[g][j] = 0.0f;
        }
        int bits = 0;
        // kSinks: the pieces from the sinks' last to the window's first are left out
        const int sink_pieces = SEE == kSinks ? (min(A.sinks, first) + 31) / 32 : 0;
        const int64_t skip = SEE == kSinks ? max(0, first / 32 - sink_pieces) * 32 : 0;
        const int from = SEE == kSinks ? 0 : (first / 32) * 32;
        for (int64_t t0 = from + static_cast<int64_t>(warp) * 32; t0 + skip <= pos || t0 < sink_pieces * 32;
             t0 += kWarps * 32) {
            const int64_t t = t0 + lane + (t0 < sink_pieces * 32 ? 0 : skip);
            bool see = (t >= first || (SEE == kSinks && t < A.sinks)) && t <= pos;
            const int block = static_cast<int>(t / page), slot = static_cast<int>(t % page);
            int64_t base = 0;
            float ks = 0.0f, vs = 0.0f;
            if (see) {
                const int id = block < A.c.width ? table[block] : -1;
                see = id >= 0 && id < A.c.n_pages;
                if (see) {
                    const int64_t bh = static_cast<int64_t>(id) * A.c.heads + h;
                    base = (bh * page + slot) * D;
                    ks = A.c.k_scale[bh];
                    vs = A.c.v_scale[bh];
                } else {
                    bits |= DSPARK_STATUS_BAD_PAGE;
                }
            }
            float s[kHeads] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (see) {
                const uint4* kp = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(A.c.k) + base);
                for (int d = 0; d < D; d += 16) {
                    const uint4 c = kp[d / 16];
                    float x[16];
                    e4m3x4_to_f32(c.x, x);
                    e4m3x4_to_f32(c.y, x + 4);
                    e4m3x4_to_f32(c.z, x + 8);
                    e4m3x4_to_f32(c.w, x + 12);
#pragma unroll
                    for (int g = 0; g < kHeads; ++g)
#pragma unroll
                        for (int j = 0; j < 16; ++j) s[g] = fmaf(qs[g][d + j], x[j], s[g]);
                }
            }
#pragma unroll
            for (int g = 0; g < kHeads; ++g) {
                s[g] = see ? s[g] * ks : -INFINITY;
                float top = s[g];
                for (int off = 16; off > 0; off >>= 1)
                    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
                const float mn = max_nan(m[g], top);
                // m = -inf: nothing seen yet, every weight and the old sum are 0
                const float shrink = m[g] == -INFINITY ? 0.0f : exp2f(m[g] - mn);
                const float p = mn == -INFINITY ? 0.0f : exp2f(s[g] - mn);
                m[g] = mn;
                l[g] = l[g] * shrink + p;
                s[g] = see ? p * vs : 0.0f;
                for (int j = 0; j < kMaxDim / 32; ++j) acc[g][j] *= shrink;
            }
            unsigned seen = __ballot_sync(0xffffffffu, see);
            while (seen != 0) {
                const int k = __ffs(seen) - 1;
                seen &= seen - 1;
                const int64_t vb = __shfl_sync(0xffffffffu, base, k);
                float p[kHeads];
#pragma unroll
                for (int g = 0; g < kHeads; ++g) p[g] = __shfl_sync(0xffffffffu, s[g], k);
                const uint8_t* vp = static_cast<const uint8_t*>(A.c.v) + vb;
#pragma unroll
                for (int j = 0; j < kMaxDim / 128; ++j) {
                    const int d = j * 128 + lane * 4;
                    if (d < D) {
                        float x[4];
                        e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(vp + d), x);
#pragma unroll
                        for (int g = 0; g < kHeads; ++g)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[g][j * 4 + i] = fmaf(p[g], x[i], acc[g][j * 4 + i]);
                    }
                }
            }
        }
        if (bits) raise_status(A.status, bits);
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
            float lg = l[g];
            for (int off = 16; off > 0; off >>= 1) lg += __shfl_xor_sync(0xffffffffu, lg, off);
            if (lane == 0) { ml_s[warp][g][0] = m[g]; ml_s[warp][g][1] = lg; }
        }
#pragma unroll
        for (int g = 0; g < kHeads; ++g) {
            __syncthreads();
            if (g >= ng) continue;                    // the same for every thread
#pragma unroll
            for (int j = 0; j < kMaxDim / 128; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = j * 128 + lane * 4 + i;
                    if (d < D) acc_s[warp][d] = acc[g][j * 4 + i];
                }
            __syncthreads();
            float top = -INFINITY, sum = 0.0f, f[kWarps];
            for (int w = 0; w < kWarps; ++w) top = max_nan(top, ml_s[w][g][0]);
            for (int w = 0; w < kWarps; ++w) {
                f[w] = ml_s[w][g][0] == -INFINITY ? 0.0f : exp2f(ml_s[w][g][0] - top);
                sum += f[w] * ml_s[w][g][1];
            }
            for (int d = threadIdx.x; d < D; d += blockDim.x) {
                float o = 0.0f;
                for (int w = 0; w < kWarps; ++w) o += f[w] * acc_s[w][d];
                store1<DT>(A.out, row * A.out_stride + (head0 + g) * D + d,
                           top == -INFINITY ? 0.0f : o / sum);
            }
            if (threadIdx.x == 0 && A.lse != nullptr)
                A.lse[static_cast<int64_t>(row) * A.q_heads + head0 + g] =
                    top == -INFINITY ? -INFINITY : (top + log2f(sum)) * kLn2;
        }
    }
}

}  // namespace

int launch_attend(const AttendCall& A, See see, int dtype, cudaStream_t stream)
{
    if (attend_mma_serves(A, dtype)) return launch_attend_mma(A, see, stream);
    const bool bf = dtype == DSPARK_BF16;
    auto kernel = see == kSinks
                      ? (bf ? attend_any_kernel<DSPARK_BF16, kSinks> : attend_any_kernel<DSPARK_F32, kSinks>)
                      : (bf ? attend_any_kernel<DSPARK_BF16, kAll> : attend_any_kernel<DSPARK_F32, kAll>);
    return launch_pdl("attend", kernel, dim3(static_cast<unsigned>(A.rows), static_cast<unsigned>(A.c.heads)),
                      dim3(kWarps * 32), 0, stream, A);
}

}  // namespace dspark
