// rope.cuh — rotary positions: the angle of a (position, pair) and the rotation of a pair.
//
// Pair j of a head turns by angle = position * f_j. f_j is held as a 64-bit fraction of a turn
// per position (turns[j] = f_j / (2 pi) * 2^64), so the product modulo 2^64 is the angle
// modulo one turn, exactly: positions of any size cost one integer multiply and lose nothing,
// where position * f_j in fp32 is off by whole radians at a few million. The top 32 bits then
// go through sincospif: cos and sin are within about 2e-7 for every position.
#pragma once

#include "common.cuh"

namespace dspark {

struct Rope {
    const uint64_t* turns;
    int half;          // rotated pairs: rot / 2 (0: nothing is rotated)
    int interleaved;   // pairs (2j, 2j+1); else (j, j + half)
    float mscale;
    float sign;        // +1, or -1 for the inverse
};

// Host: a dspark_rope as the kernels take it. Checks nothing.
inline Rope rope_of(const dspark_rope* r, bool inverse)
{
    Rope out;
    out.turns = r ? r->turns : nullptr;
    out.half = r ? r->rot / 2 : 0;
    out.interleaved = r ? r->interleaved : 0;
    out.mscale = r ? r->mscale : 1.0f;
    out.sign = inverse ? -1.0f : 1.0f;
    return out;
}
// Checks a caller's rope against a head of `dim` elements (NULL: fine, no rotation).
int check_rope(const char* fn, const dspark_rope* rope, int dim);

// (mscale cos, mscale sign sin) of pair j at `position`.
__device__ __forceinline__ float2 rope_factor(const Rope& r, uint64_t turn, int position)
{
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(position)) * turn;
    const float x = __int2float_rn(static_cast<int>(phase >> 32)) * 0x1p-31f;   // half turns
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * r.mscale, s * r.mscale * r.sign);
}

// (a, b) turned by f = (cos, sin).
__device__ __forceinline__ float2 rope_turn(float a, float b, float2 f)
{
    return make_float2(a * f.x - b * f.y, b * f.x + a * f.y);
}

// Eight elements of type DT at p (16-byte aligned) as fp32, and back.
template <int DT>
__device__ __forceinline__ void load8(const void* p, float* x)
{
    if (DT == DSPARK_BF16) {
        const uint4 v = *static_cast<const uint4*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    } else {
        const float4 a = static_cast<const float4*>(p)[0], b = static_cast<const float4*>(p)[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

// Two fp32 as packed bf16, rounded to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int DT>
__device__ __forceinline__ void store8(void* p, const float* x)
{
    if (DT == DSPARK_BF16) {
        *static_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                             pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    } else {
        static_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        static_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i)
{
    if (DT == DSPARK_BF16)
        return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
    return static_cast<const float*>(p)[i];
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float x)
{
    if (DT == DSPARK_BF16)
        static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16(x, 0.0f));
    else
        static_cast<float*>(p)[i] = x;
}

// Rows of heads as the rotation reads or writes them: element d of (row, head) is at
// base + (row * row_stride + head * dim + d) elements.
struct RowsIn { const void* base; int64_t row_stride; };
struct RowsOut { void* base; int64_t row_stride; };

// One CTA's part of a rotation: rows [row0, row0 + n) of `heads` heads of `dim` elements, with
// the factors of those rows in `tab` (n * half entries of shared memory, row-major).
// VEC: units of eight pairs (16-byte accesses; dim, half and the strides multiples of 8, bases
// 16-byte aligned), a unit past the rotated part being 16 copied elements (dim - rot a multiple
// of 16); else one pair, or two copied elements, at a time.
// `live` (shared, one flag per row; NULL: all): rows to touch. `copy`: also write the elements
// past the rotated ones (not needed in place).
template <int DT, bool VEC>
__device__ __forceinline__ void rotate_rows(const Rope& r, const float2* tab, RowsIn x, RowsOut y,
                                            int64_t row0, int n, int heads, int dim, bool copy,
                                            const int* live)
{
    constexpr int P = VEC ? 8 : 1;
    constexpr int E = DT == DSPARK_BF16 ? 2 : 4;
    const int rot_units = r.half / P;                     // a head's rotated units
    const int all_units = copy ? (dim + 2 * P - 1) / (2 * P) : rot_units;
    const int per_row = heads * all_units;
    for (int u = threadIdx.x; u < n * per_row; u += blockDim.x) {
        const int k = u / per_row;
        const int in_row = u - k * per_row;
        const int h = in_row / all_units;
        const int o = in_row - h * all_units;
        if (live != nullptr && live[k] < 0) continue;
        const int64_t xi = (row0 + k) * x.row_stride + static_cast<int64_t>(h) * dim;
        const int64_t yi = (row0 + k) * y.row_stride + static_cast<int64_t>(h) * dim;
        if (VEC) {
            const char* xp = static_cast<const char*>(x.base) + xi * E;
            char* yp = static_cast<char*>(y.base) + yi * E;
            float a[8], b[8];
            if (o < rot_units) {
                const int ia = r.interleaved ? o * 16 : o * 8;
                const int ib = r.interleaved ? o * 16 + 8 : r.half + o * 8;
                load8<DT>(xp + ia * E, a);
                load8<DT>(xp + ib * E, b);
                const float2* f = tab + k * r.half + o * 8;
                if (r.interleaved) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 t = rope_turn(a[2 * q], a[2 * q + 1], f[q]);
                        const float2 s = rope_turn(b[2 * q], b[2 * q + 1], f[q + 4]);
                        a[2 * q] = t.x; a[2 * q + 1] = t.y;
                        b[2 * q] = s.x; b[2 * q + 1] = s.y;
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float2 t = rope_turn(a[q], b[q], f[q]);
                        a[q] = t.x;
                        b[q] = t.y;
                    }
                }
                store8<DT>(yp + ia * E, a);
                store8<DT>(yp + ib * E, b);
            } else {
                const int i = 2 * r.half + (o - rot_units) * 16;
                load8<DT>(xp + i * E, a);
                load8<DT>(xp + (i + 8) * E, b);
                store8<DT>(yp + i * E, a);
                store8<DT>(yp + (i + 8) * E, b);
            }
        } else if (o < rot_units) {
            const int ia = r.interleaved ? 2 * o : o;
            const int ib = r.interleaved ? 2 * o + 1 : o + r.half;
            const float2 t = rope_turn(load1<DT>(x.base, xi + ia), load1<DT>(x.base, xi + ib),
                                       tab[k * r.half + o]);
            store1<DT>(y.base, yi + ia, t.x);
            store1<DT>(y.base, yi + ib, t.y);
        } else {
            const int i = 2 * o;
            store1<DT>(y.base, yi + i, load1<DT>(x.base, xi + i));
            if (i + 1 < dim) store1<DT>(y.base, yi + i + 1, load1<DT>(x.base, xi + i + 1));
        }
    }
}

// Whether rotate_rows<., true> may run.
inline bool rotate_vec(const Rope& r, const void* x, int64_t xs, const void* y, int64_t ys,
                       int dim, int elem)
{
    const int64_t per16 = 16 / elem;
    return dim % 16 == 0 && r.half % 8 == 0 && xs % per16 == 0 && ys % per16 == 0 &&
           (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (reinterpret_cast<uintptr_t>(y) & 15u) == 0;
}

}  // namespace dspark
