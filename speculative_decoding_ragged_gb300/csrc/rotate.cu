// rotate.cu — dspark_rotate (rotary positions over rows of heads, and their inverse) and the
// host function that makes a rope's frequencies.
//
// y = m R(position) x for each pair, or m R(-position) x: the inverse is also the gradient, since
// a rotation's transpose is the rotation back. Bound by memory: 2 e bytes and 3 flops per
// element. A CTA takes a few rows, computes their factors once in shared memory (one sincospif
// per pair and row, shared by all heads: 40 heads would otherwise spend 40 of them) and then
// streams the rows' heads, two 16-byte accesses a thread at a time.
// 8192 rows of 40 heads of 128 in bf16: 31.2 us, 5.4 TB/s; a gradient of 4999 rows of 24 heads of 96,
// 64 rotated in pairs, fp32: 16.6 us, 5.5 TB/s. One window's 16 rows: 3.2 us, the launch.
#include <cmath>

#include "rope.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 128;   // 8192 rows of 40 heads: 31.3 us; 32.6 with 256, 37.9 with 512 and more rows each
constexpr int kTable = 512;        // shared factors: at least one row's, at most kTable entries

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
rotate_kernel(Turns t, const int32_t* __restrict__ positions, int rows, int per_cta)
{
    __shared__ __align__(16) float2 tab[kTable];
    pdl_wait_and_trigger();
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * per_cta;
    const int n = min(static_cast<int64_t>(per_cta), rows - row0);
    rotate_rows<DT, VEC>(t, tab, row0, n, nullptr, [&]() {
        for (int i = threadIdx.x; i < n * t.r.half; i += kThreads) {
            const int k = i / t.r.half;
            tab[i] = rope_factor(t.r, t.r.turns[i - k * t.r.half], positions[row0 + k]);
        }
        __syncthreads();
    });
}

}  // namespace

int launch_rotate(const Rope& r, const void* x, int64_t xs, void* y, int64_t ys, int dtype,
                  int rows, int heads, int dim, const int32_t* positions, cudaStream_t stream)
{
    const bool bf = dtype == DSPARK_BF16;
    const bool vec = rotate_vec(r, x, xs, y, ys, dim, bf ? 2 : 4);
    int per_cta = 1;
    if (rows >= 152 * 8 && r.half > 0) {
        per_cta = kThreads / r.half;
        per_cta = per_cta < 1 ? 1 : per_cta > 4 ? 4 : per_cta;
    }
    const Turns t = turns_of(r, x, xs, y, ys, heads, dim, vec, bf ? 2 : 4, per_cta);
    const dim3 grid(static_cast<unsigned>(ceil_div(rows, per_cta)));
    auto kernel = bf ? (vec ? rotate_kernel<DSPARK_BF16, true> : rotate_kernel<DSPARK_BF16, false>)
                     : (vec ? rotate_kernel<DSPARK_F32, true> : rotate_kernel<DSPARK_F32, false>);
    return launch_pdl("rotate", kernel, grid, dim3(kThreads), 0, stream, t, positions, rows, per_cta);
}

int check_rope(const char* fn, const dspark_rope* rope, int dim)
{
    if (rope == nullptr) return DSPARK_OK;
    if (rope->rot < 0 || rope->rot > dim || rope->rot % 2 != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: rot = %d must be even and within the head's %d",
                    fn, rope->rot, dim);
    if (rope->rot > 0 && (rope->turns == nullptr ||
                          (reinterpret_cast<uintptr_t>(rope->turns) & 7u) != 0))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: the rope's 8-byte aligned turns are required", fn);
    if (rope->interleaved != 0 && rope->interleaved != 1)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: interleaved = %d is neither 0 nor 1", fn,
                    rope->interleaved);
    if (!std::isfinite(rope->mscale))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: mscale must be finite", fn);
    return DSPARK_OK;
}

}  // namespace dspark

using dspark::fail;

extern "C" {

int dspark_rope_turns(int rot, double base, dspark_rope_scaling scaling, double factor,
                      double trained, double slow, double fast, uint64_t* turns)
{
    const char* fn = "dspark_rope_turns";
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    if (rot < 0 || rot % 2 != 0 || rot > DSPARK_MAX_HEAD)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: rot = %d must be even and in [0, %d]", fn, rot,
                    DSPARK_MAX_HEAD);
    if (!(base > 1.0) || !std::isfinite(base))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: base must be finite and above 1", fn);
    if (scaling != DSPARK_ROPE_PLAIN && scaling != DSPARK_ROPE_LINEAR &&
        scaling != DSPARK_ROPE_BY_PARTS)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: unknown scaling %d", fn, static_cast<int>(scaling));
    if (scaling != DSPARK_ROPE_PLAIN && !(factor >= 1.0 && std::isfinite(factor)))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: factor must be finite and at least 1", fn);
    if (scaling == DSPARK_ROPE_BY_PARTS &&
        !(trained > 0.0 && std::isfinite(trained) && slow >= 0.0 && fast > slow && std::isfinite(fast)))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: by parts needs trained > 0 and 0 <= slow < fast", fn);
    if (rot > 0 && turns == nullptr)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: turns is required", fn);
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(base, -2.0 * j / rot) / kTwoPi;     // turns per position
        if (scaling == DSPARK_ROPE_LINEAR) f /= factor;
        if (scaling == DSPARK_ROPE_BY_PARTS) {
            double keep = (trained * f - slow) / (fast - slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = (1.0 - keep) * (f / factor) + keep * f;
        }
        turns[j] = static_cast<uint64_t>(std::ldexp(f, 64));    // f < 1/6: no overflow
    }
    return DSPARK_OK;
}

int dspark_rotate(const void* x, int64_t x_stride, void* y, int64_t y_stride, dspark_dtype dtype,
                  int rows, int heads, int dim, const int32_t* positions,
                  const dspark_rope* rope, int inverse, cudaStream_t stream)
{
    const char* fn = "dspark_rotate";
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows < 0 || heads < 1 || dim < 1 || dim > DSPARK_MAX_HEAD ||
        static_cast<int64_t>(heads) * dim > INT32_MAX / 8)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: bad sizes rows=%d heads=%d dim=%d", fn, rows,
                    heads, dim);
    const int64_t width = static_cast<int64_t>(heads) * dim;
    if (x_stride < width || y_stride < width)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: row strides %lld, %lld below heads*dim = %lld", fn,
                    static_cast<long long>(x_stride), static_cast<long long>(y_stride),
                    static_cast<long long>(width));
    if (rope == nullptr)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: rope is required", fn);
    const int rc = dspark::check_rope(fn, rope, dim);
    if (rc != DSPARK_OK || rows == 0) return rc;
    const uintptr_t e = dtype == DSPARK_BF16 ? 2 : 4;
    if (x == nullptr || y == nullptr || positions == nullptr ||
        reinterpret_cast<uintptr_t>(x) % e != 0 || reinterpret_cast<uintptr_t>(y) % e != 0 ||
        reinterpret_cast<uintptr_t>(positions) % 4 != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: x, y and positions are required, aligned to their elements", fn);
    return dspark::launch_rotate(dspark::rope_of(rope, inverse != 0), x, x_stride, y, y_stride,
                                 static_cast<int>(dtype), rows, heads, dim, positions, stream);
}

}  // extern "C"
