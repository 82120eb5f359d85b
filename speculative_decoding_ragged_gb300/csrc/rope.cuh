// rope.cuh — rotary positions: the angle of a (position, pair) and the rotation of a pair.
//
// Pair j of a head turns by angle = position * f_j. f_j is held as a 64-bit fraction of a turn
// per position (turns[j] = f_j / (2 pi) * 2^64), so the product modulo 2^64 is the angle
// modulo one turn, exactly: positions of any size cost one integer multiply and lose nothing,
// where position * f_j in fp32 is off by whole radians at a few million. What it lies off the
// nearest quarter turn then goes through sincospif, at most 1/4 in its half turns, which fp32 holds
// to 2^-27: cos and sin are within 8.4e-8 for every position. (The whole turn's fraction rounds at
// 2^-25: 1.13e-7, and fp32 rotations were off by 4.1e-8 relative where they now are by 3.1e-8.)
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
    // the nearest quarter turn, and what is left: at most an eighth, in units of 2^-33 half turns
    const uint64_t near = phase + (1ull << 61);
    const int left = static_cast<int>(static_cast<int64_t>((near & ~(3ull << 62)) - (1ull << 61)) >> 30);
    float s, c;
    sincospif(__int2float_rn(left) * 0x1p-33f, &s, &c);
    const int quarter = static_cast<int>(near >> 62);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    return make_float2((quarter == 1 || quarter == 2 ? -x : x) * r.mscale,
                       (quarter >= 2 ? -y : y) * r.mscale * r.sign);
}

// (a, b) turned by f = (cos, sin).
__device__ __forceinline__ float2 rope_turn(float a, float b, float2 f)
{
    return make_float2(a * f.x - b * f.y, b * f.x + a * f.y);
}

// Two fp32 as packed bf16, rounded to nearest even; `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// 16 bytes: eight bf16 or four fp32.
template <int DT>
__device__ __forceinline__ void load16(const uint4& v, float* x)
{
    if (DT == DSPARK_BF16) {
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
    } else {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
}
template <int DT>
__device__ __forceinline__ uint4 store16(const float* x)
{
    if (DT == DSPARK_BF16)
        return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
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

// n / d for small n by one multiplication: exact while n * d < 2^32 (the host checks).
struct Divider {
    uint32_t d, magic;     // magic 0: divide
    __device__ __forceinline__ int operator()(int n) const
    {
        return magic != 0 ? static_cast<int>(__umulhi(static_cast<uint32_t>(n), magic))
                          : static_cast<int>(static_cast<uint32_t>(n) / d);
    }
};
inline Divider divider(int64_t d, int64_t most)
{
    Divider r;
    r.d = static_cast<uint32_t>(d);
    r.magic = d > 1 && d * most < (1ll << 32) ? static_cast<uint32_t>(((1ull << 32) + d - 1) / d) : 0;
    return r;
}

// How a rotation cuts its rows: units of two 16-byte accesses (VEC: eight pairs of bf16, four of
// fp32, so that a warp's accesses lie side by side; with eight of fp32 the gradient of 4999 rows
// took 22.0 us; dim, half and the strides multiples of 8, bases 16-byte aligned), a unit past the
// rotated part being as many copied elements; else one pair, or two copied elements, at a time.
struct Turns {
    Rope r;
    RowsIn x;
    RowsOut y;
    int heads, dim;
    int rot_units;         // of a head
    Divider units, per_row;    // units of a head, of a row
};
inline Turns turns_of(const Rope& r, const void* x, int64_t xs, void* y, int64_t ys, int heads, int dim,
                      bool vec, int elem, int rows_per_cta)
{
    const int P = vec ? 16 / elem : 1;
    const bool copy = !(x == y && xs == ys);       // in place the rest stays where it is
    Turns t;
    t.r = r;
    t.x = {x, xs};
    t.y = {y, ys};
    t.heads = heads;
    t.dim = dim;
    t.rot_units = r.half / P;
    const int64_t units = copy ? (dim + 2 * P - 1) / (2 * P) : t.rot_units;
    t.units = divider(units, units * heads);
    t.per_row = divider(units * heads, units * heads * rows_per_cta);
    return t;
}

// A vector unit: where it is, and its elements as loaded.
template <int DT>
struct TurnUnit {
    static constexpr int E = DT == DSPARK_BF16 ? 2 : 4, N = 16 / E;     // elements of an access
    uint4 v[2];
    int64_t y;
    int a, b, f;             // offsets of the two accesses in the head; first factor, or -1: copied
    __device__ __forceinline__ void load(const Turns& t, int64_t row0, int u)
    {
        const int k = t.per_row(u), in_row = u - k * static_cast<int>(t.per_row.d);
        const int h = t.units(in_row), o = in_row - h * static_cast<int>(t.units.d);
        const int64_t head = static_cast<int64_t>(h) * t.dim;
        if (o < t.rot_units) {
            a = t.r.interleaved ? o * 2 * N : o * N;
            b = t.r.interleaved ? a + N : t.r.half + o * N;
            f = k * t.r.half + o * N;
        } else {
            a = 2 * t.r.half + (o - t.rot_units) * 2 * N;
            b = a + N;
            f = -1 - k;
        }
        y = (row0 + k) * t.y.row_stride + head;
        const char* x = static_cast<const char*>(t.x.base) + ((row0 + k) * t.x.row_stride + head) * E;
        v[0] = *reinterpret_cast<const uint4*>(x + a * E);
        v[1] = *reinterpret_cast<const uint4*>(x + b * E);
    }
    // live: one flag per row (NULL: all), negative: leave the row alone
    __device__ __forceinline__ void turn(const Turns& t, const float2* tab, const int* live)
    {
        if (live != nullptr && live[f >= 0 ? f / t.r.half : -1 - f] < 0) return;
        char* out = static_cast<char*>(t.y.base) + y * E;
        if (f >= 0) {
            float x[2 * N];
            load16<DT>(v[0], x);
            load16<DT>(v[1], x + N);
            const float4* c = reinterpret_cast<const float4*>(tab + f);
#pragma unroll
            for (int j = 0; j < N; j += 2) {
                const float4 g = c[j / 2];           // factors j and j + 1
                if (t.r.interleaved) {
                    float* z = x + 2 * j;
                    const float2 s = rope_turn(z[0], z[1], make_float2(g.x, g.y));
                    const float2 w = rope_turn(z[2], z[3], make_float2(g.z, g.w));
                    z[0] = s.x; z[1] = s.y; z[2] = w.x; z[3] = w.y;
                } else {
                    const float2 s = rope_turn(x[j], x[N + j], make_float2(g.x, g.y));
                    const float2 w = rope_turn(x[j + 1], x[N + j + 1], make_float2(g.z, g.w));
                    x[j] = s.x; x[N + j] = s.y;
                    x[j + 1] = w.x; x[N + j + 1] = w.y;
                }
            }
            v[0] = store16<DT>(x);
            v[1] = store16<DT>(x + N);
        }
        *reinterpret_cast<uint4*>(out + a * E) = v[0];
        *reinterpret_cast<uint4*>(out + b * E) = v[1];
    }
};

// One CTA's rows [row0, row0 + n): `table` fills the factors of the rows (n * half entries of
// shared memory, row-major, 16-byte aligned) and synchronises; it runs after the first loads are
// on their way.
template <int DT, bool VEC, class Table>
__device__ __forceinline__ void rotate_rows(const Turns& t, const float2* tab, int64_t row0, int n,
                                            const int* live, Table&& table)
{
    const int total = n * static_cast<int>(t.per_row.d), step = blockDim.x;
    if (VEC) {
        TurnUnit<DT> now;
        int u = threadIdx.x;
        if (u < total) now.load(t, row0, u);
        table();
#pragma unroll 1
        for (; u < total; u += step) {
            TurnUnit<DT> next;
            if (u + step < total) next.load(t, row0, u + step);
            now.turn(t, tab, live);
            now = next;
        }
    } else {
        table();
#pragma unroll 1
        for (int u = threadIdx.x; u < total; u += step) {
            const int k = t.per_row(u), in_row = u - k * static_cast<int>(t.per_row.d);
            const int h = t.units(in_row), o = in_row - h * static_cast<int>(t.units.d);
            if (live != nullptr && live[k] < 0) continue;
            const int64_t xi = (row0 + k) * t.x.row_stride + static_cast<int64_t>(h) * t.dim;
            const int64_t yi = (row0 + k) * t.y.row_stride + static_cast<int64_t>(h) * t.dim;
            if (o < t.rot_units) {
                const int ia = t.r.interleaved ? 2 * o : o;
                const int ib = t.r.interleaved ? 2 * o + 1 : o + t.r.half;
                const float2 s = rope_turn(load1<DT>(t.x.base, xi + ia), load1<DT>(t.x.base, xi + ib),
                                           tab[k * t.r.half + o]);
                store1<DT>(t.y.base, yi + ia, s.x);
                store1<DT>(t.y.base, yi + ib, s.y);
            } else {
                const int i = 2 * o;
                store1<DT>(t.y.base, yi + i, load1<DT>(t.x.base, xi + i));
                if (i + 1 < t.dim) store1<DT>(t.y.base, yi + i + 1, load1<DT>(t.x.base, xi + i + 1));
            }
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
