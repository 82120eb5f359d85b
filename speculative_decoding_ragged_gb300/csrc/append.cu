// append.cu — dspark_append: a step's keys and values, rotated, quantised and written to the
// paged 8-bit cache, its queries rotated on the way.
//
// A block is one page's slots of one kv head; the scale given to it is a power of two, so that growing it
// rescales the codes already there by an exact shift of their exponent (only codes that leave
// e4m3's normal range round again), and multiplying by it is exact. The step's rows that fall
// into one block are consecutive packed rows; the first of them leads. One warp, or for prompts a
// team of four, owns a block (of keys or of values): it finds the block's rows, their largest
// magnitude, hence the scale, requantises the retained codes if the scale grew, and writes the
// rows' codes. No two touch one block, so there are no atomics and the result does not depend on
// any order.
//
// The rotation's factors of the block's rows are computed once per CTA in shared memory, for four
// heads' keys (a prompt's: two teams, each two heads in turn). The rows' elements stay in registers
// between the maximum and the codes where they fit (8 rows of 128 for a warp, 64 for a prompt's
// four); else they are read again.
// Bound for a step by the chain of dependent loads (row owner, length, page id, scale, retained
// codes): one window of 4 rows, 8 heads of 128 and 32 query heads, 4.4 us, 256 windows 12.8 us (3.9 at
// the copy rate). For prompts by bandwidth in the queries (36 us of 200 MB), which start when the
// keys' and values' CTAs are all running, and by the chain and the factors in those (40 us of 74 MB):
// three prompts, 12 thousand rows in all, 73.9 us. Both kinds of CTAs mixed in one launch took 90 us:
// the queries need more warps than the others leave.
#include "cache.cuh"
#include "rope.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;      // of a step's CTA
constexpr int kWarps = kThreads / 32;
constexpr int kTeam = 4;           // warps that take a prompt's block together
constexpr int kPromptWarps = 8;    // of a CTA: two heads' blocks side by side
constexpr int kGroups = 2;         // heads of keys that a prompt's team takes in turn
constexpr int kTable = 4096;       // shared rope factors (32 KB): 64 rows of 64 pairs
constexpr int keep_of(int T) { return T > 1 ? 8 : 4; }     // units of a lane that stay in registers
constexpr int kQueryRows = 4;      // most rows of a CTA that rotates queries
constexpr int kQueryThreads = 128; // of a prompts' CTA that rotates queries
constexpr int kQueryFactors = 512; // their factors

struct AppendArgs {
    dspark_cache c;
    Rope rope;
    RowsIn k, v;
    Turns q;
    const int32_t* row_req;
    const int32_t* row_pos;
    const int32_t* lengths;
    int rows, B;
    int kv_ctas;          // first of the grid: (rows, eight blocks)
    int per_row;          // of them for the same rows
    int key_shares;       // of a prompt's: those with keys
    int chunk;            // rows a kv CTA looks for leaders in
    int q_rows;           // rows a query CTA rotates
    int32_t* status;
};

// Scales are powers of two unless the cache was filled elsewhere: products and quotients are then
// exact in fp32. Else these give an fp32 number on the exact value's side of every border between two
// codes (which have five bits at most), so that its code is the exact value's.
__device__ __forceinline__ bool power_of_two(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0; }
// x s: cut off, the last bit set where that lost anything.
__device__ __forceinline__ float sided_product(float x, float s)
{
    const float p = __fmul_rz(x, s);
    return fmaf(x, s, -p) != 0.0f ? __uint_as_float(__float_as_uint(p) | 1u) : p;
}
// x / s, inv = 1 / s: the product, off by a few last places, goes to the nearest multiple of 64 of
// them, then one step towards what the exact remainder says.
__device__ __forceinline__ float sided_quotient(float x, float s, float inv)
{
    const uint32_t near = (__float_as_uint(x * inv) + 32u) & ~63u;
    const float rest = fmaf(-__uint_as_float(near), s, x);
    return __uint_as_float(rest == 0.0f ? near : (rest < 0.0f) == (x < 0.0f) ? near + 1u : near - 1u);
}

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

// A unit as it was loaded, and its elements in fp32.
template <int DT, bool VEC>
struct Raw {
    static constexpr int W = VEC ? (DT == DSPARK_BF16 ? 4 : 8) : 2;
    uint32_t w[W];
    __device__ __forceinline__ void load(const void* base, int64_t at, const Unit<VEC>& un)
    {
        if (!VEC) {
            w[0] = __float_as_uint(load1<DT>(base, at + un.a));
            w[1] = __float_as_uint(load1<DT>(base, at + un.b));
        } else if (DT == DSPARK_BF16) {
            const uint16_t* p = static_cast<const uint16_t*>(base) + at;
            const uint2 a = *reinterpret_cast<const uint2*>(p + un.a), b = *reinterpret_cast<const uint2*>(p + un.b);
            w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
        } else {
            const uint32_t* p = static_cast<const uint32_t*>(base) + at;
            const uint4 a = *reinterpret_cast<const uint4*>(p + un.a), b = *reinterpret_cast<const uint4*>(p + un.b);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[W - 4] = b.x; w[W - 3] = b.y; w[W - 2] = b.z; w[W - 1] = b.w;
        }
    }
    __device__ __forceinline__ void get(float* x) const
    {
        if (VEC && DT == DSPARK_BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
};

// The rotated elements turn. CHECK: non-finite elements count as 0, before and after; returns
// whether there were any.
template <bool VEC, bool CHECK>
__device__ __forceinline__ bool turn_unit(const Rope& r, const Unit<VEC>& un, const float2* tab, float* x)
{
    constexpr int N = Unit<VEC>::N;
    bool bad = false;
    if (CHECK)
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
    if (CHECK)
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (!finite(x[j])) { x[j] = 0.0f; bad = true; }  // the sum of two products overflowed
    return bad;
}

template <bool VEC>
__device__ __forceinline__ float amax_unit(const float* x, float m)
{
#pragma unroll
    for (int j = 0; j < Unit<VEC>::N; ++j) m = max_nan(m, fabsf(x[j]));
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

// The same for any scale.
template <bool VEC>
__device__ __forceinline__ void store_exact(uint8_t* row, const Unit<VEC>& un, float* x, float scale)
{
    float inv = 1.0f / scale;
    if (!power_of_two(scale)) {
#pragma unroll
        for (int j = 0; j < Unit<VEC>::N; ++j) x[j] = sided_quotient(x[j], scale, inv);
        inv = 1.0f;
    }
    store_unit<VEC>(row, un, x, inv);
}

// A team: T warps that share a block, 1 or 4.
template <int T>
__device__ __forceinline__ void team_sync()
{
    if (T == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + static_cast<int>(threadIdx.x) / (32 * T)), "n"(32 * T) : "memory");
}
// The team's largest, NaN above all. `red`: T floats of the team's own.
template <int T>
__device__ __forceinline__ float team_max(float amax, float* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if (T > 1) {
        team_sync<T>();                    // the last use of red is over
        if ((threadIdx.x & 31) == 0) red[(threadIdx.x >> 5) & (T - 1)] = amax;
    }
    team_sync<T>();
    if (T > 1)
#pragma unroll
        for (int w = 0; w < T; ++w) amax = max_nan(amax, red[w]);
    return amax;
}

// A block's scale from its rows' largest magnitude; the retained codes follow it. `old`: the scale
// as every thread of the team read it before.
template <int T>
__device__ __forceinline__ float settle_scale(float amax, float old, float* scale, uint8_t* codes, int retained,
                                              int me)
{
    const float fresh = exp2i(scale_exponent(amax));
    if (retained == 0) {
        if (me == 0) *scale = fresh;
        return fresh;
    }
    const float s = fmaxf(old, fresh);
    if (s > old) {
        if (me == 0) *scale = s;
        const float ratio = old / s;
        uint4* kept = reinterpret_cast<uint4*>(codes);
#pragma unroll 2
        for (int i = me; i < retained / 16; i += 32 * T) {
            const uint4 c = kept[i];
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[4];
                e4m3x4_to_f32(w[k], f);
                o[k] = e4m3x4(sided_product(f[0], ratio), sided_product(f[1], ratio),
                              sided_product(f[2], ratio), sided_product(f[3], ratio));
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

// The blocks that packed row r (request b's row i0, at position pos) leads. T = 1: eight of them
// from hv0 (head, K or V), one per warp; T = 4: the keys' or the values' of two heads from hv0.
// again: the factors are those of the call before. Returns status bits.
template <int DT, bool VEC, int T>
__device__ __forceinline__ int append_blocks(const AppendArgs& A, int64_t r, int b, int i0, int pos, int hv0,
                                             bool again, float2* tab, float* reds)
{
    constexpr int kKeep = keep_of(T), kAll = T > 1 ? 32 * kPromptWarps : kThreads;
    const dspark_cache& c = A.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = warp / T;
    const int slot0 = pos & (c.page - 1), block = pos / c.page, most = c.page - slot0;
    const int me = threadIdx.x & (32 * T - 1);
    const int hv = hv0 + (T > 1 ? 2 * team : team);
    const bool works = hv < 2 * c.heads, value = hv & 1;
    const int h = hv >> 1;
    const int half = T > 1 && value ? 0 : A.rope.half;
    const int units = c.dim / Unit<VEC>::N;
    float* red = reds + team * T;
    // Lanes over units, `step` rows at a time; a head wider than a warp's units (scalar accesses
    // only) takes several turns over a row.
    const int wide = units > 32 ? 32 : units, per_warp = 32 / wide, step = per_warp * T;
    const int in_warp = lane / wide, u0 = lane - in_warp * wide;
    const int k0 = in_warp + per_warp * (warp & (T - 1));
    const bool has = works && in_warp < per_warp;
    Rope rope = A.rope;
    if (value) rope.half = 0;
    const RowsIn in = value ? A.v : A.k;
    const Unit<VEC> un(rope, u0);
    constexpr int E = DT == DSPARK_BF16 ? 2 : 4;
    // this lane's first row, and the bytes from one of its rows to the next
    const char* mine0 = static_cast<const char*>(in.base) +
                        ((r + k0) * in.row_stride + static_cast<int64_t>(h) * c.dim) * E;
    const int64_t hop = step * in.row_stride * E;
    // the rows that may be the block's, before it is known which are
    const int may = static_cast<int>(min(static_cast<int64_t>(most), A.rows - r));
    Raw<DT, VEC> raw[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
        if (has && k0 + i * step < may) raw[i].load(mine0 + i * hop, 0, un);
    const int page = block < c.width ? c.table[static_cast<int64_t>(b) * c.width + block] : -1;
    // the block's rows: the packed rows that follow, while they are b's next positions
    int n = 1;
    for (int j0 = 1; j0 < most; j0 += 32) {
        const int j = j0 + lane;
        const bool mine = j < may && A.row_req[r + j] == b && A.row_pos[r + j] == i0 + j;
        const unsigned run = __ballot_sync(0xffffffffu, mine);
        n += run == 0xffffffffu ? 32 : __ffs(~run) - 1;
        if (run != 0xffffffffu) break;
    }
    if (page < 0 || page >= c.n_pages) return DSPARK_STATUS_BAD_PAGE;

    const int rows_at_once = half > 0 ? kTable / half : n;       // factors for so many rows fit
    auto factors = [&](int from, int m) {
        __syncthreads();
        for (int i = threadIdx.x; i < m * half; i += kAll) {
            const int k = i / half;
            tab[i] = rope_factor(A.rope, A.rope.turns[i - k * half], pos + from + k);
        }
        __syncthreads();
    };
    const bool keep = n <= kKeep * step && n <= rows_at_once && units <= 32;
    if (keep && half > 0 && !again) factors(0, n);
    const int64_t bh = static_cast<int64_t>(page) * c.heads + h;
    uint8_t* codes = static_cast<uint8_t*>(value ? c.v : c.k) + bh * c.page * c.dim;
    float* scale = (value ? c.v_scale : c.k_scale) + bh;
    uint8_t* to = codes + (slot0 + k0) * c.dim;          // within a block: 32 bits
    float x[Unit<VEC>::N], amax = 0.0f;
    bool bad = false;
    if (keep) {
        if (!works) return 0;
        const float old = slot0 > 0 ? *scale : 0.0f;
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
            if (has && k0 + i * step < n) {
                raw[i].get(x);
                turn_unit<VEC, false>(rope, un, tab + (k0 + i * step) * half, x);
                amax = amax_unit<VEC>(x, amax);
            }
        amax = team_max<T>(amax, red);
        const bool clean = finite(amax);         // the same for the team
        if (!clean) {                            // rare: the offenders count as 0
            amax = 0.0f;
#pragma unroll 1
            for (int k = k0, i = 0; has && k < n; k += step, ++i) {
                Raw<DT, VEC> one;
                one.load(mine0 + i * hop, 0, un);
                one.get(x);
                bad |= turn_unit<VEC, true>(rope, un, tab + k * half, x);
                amax = amax_unit<VEC>(x, amax);
            }
            amax = team_max<T>(amax, red);
        }
        const float s = settle_scale<T>(amax, old, scale, codes, slot0 * c.dim, me), inv = 1.0f / s;
        if (clean && power_of_two(s)) {
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (has && k0 + i * step < n) {
                    raw[i].get(x);
                    turn_unit<VEC, false>(rope, un, tab + (k0 + i * step) * half, x);
                    store_unit<VEC>(to + i * step * c.dim, un, x, inv);
                }
        } else {
#pragma unroll 1
            for (int k = k0, i = 0; has && k < n; k += step, ++i) {
                Raw<DT, VEC> one;
                one.load(mine0 + i * hop, 0, un);
                one.get(x);
                turn_unit<VEC, true>(rope, un, tab + k * half, x);
                store_exact<VEC>(to + i * step * c.dim, un, x, s);
            }
        }
        return bad ? DSPARK_STATUS_BAD_VALUE : 0;
    }
    float s = 1.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int from = 0; from < n; from += rows_at_once) {
            const int m = min(rows_at_once, n - from);
            if (half > 0 && (pass == 0 || rows_at_once < n)) factors(from, m);
            if (!has) continue;
#pragma unroll 1
            for (int u = u0; u < units; u += wide) {
                const Unit<VEC> at(rope, u);
#pragma unroll 2
                for (int k = k0; k < m; k += step) {
                    Raw<DT, VEC> one;
                    one.load(mine0 + (from + k - k0) * (in.row_stride * E), 0, at);
                    one.get(x);
                    bad |= turn_unit<VEC, true>(rope, at, tab + k * half, x);
                    if (pass == 0) amax = amax_unit<VEC>(x, amax);
                    else store_exact<VEC>(to + (from + k - k0) * c.dim, at, x, s);
                }
            }
        }
        if (pass == 0 && works) {
            const float old = slot0 > 0 ? *scale : 0.0f;
            amax = team_max<T>(amax, red);
            s = settle_scale<T>(amax, old, scale, codes, slot0 * c.dim, me);
        }
    }
    return bad ? DSPARK_STATUS_BAD_VALUE : 0;
}

// A CTA's part of the keys and values: the rows [row0, row0 + chunk) and its share of their blocks.
template <int DT, bool VEC, int T>
__device__ __forceinline__ int append_rows(const AppendArgs& A, float2* tab, float* red)
{
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / A.per_row) * A.chunk;
    const int share = blockIdx.x % A.per_row;
    constexpr int kTeams = kPromptWarps / kTeam;
    // a prompt's CTA of keys takes kGroups times its teams' heads, one after the other: the factors
    // are theirs all; the values have none
    [[maybe_unused]] const bool value = share >= A.key_shares;
    [[maybe_unused]] const int head0 = value ? (share - A.key_shares) * kTeams : share * kTeams * kGroups;
    // each warp looks at the rows side by side; those that lead a block are the same for all
    const int lane = threadIdx.x & 31;
    int bits = 0;
#pragma unroll 1
    for (int from = 0; from < A.chunk; from += 32) {
        const int64_t r = row0 + from + lane;
        int b = -1, pos = 0, i = 0, before_b = -1, before_i = 0;
        if (from + lane < A.chunk && r < A.rows) {
            if (share == 0 && r > 0) {
                before_b = A.row_req[r - 1];
                before_i = A.row_pos[r - 1];
            }
            b = row_owner(A, r, &pos, &bits);
            if (b >= 0) i = A.row_pos[r];
        }
        const bool lead = b >= 0 && (i == 0 || (pos & (A.c.page - 1)) == 0);
        // a row that neither leads nor follows its request's last one is nobody's: not stored
        if (share == 0 && b >= 0 && !lead && (before_b != b || before_i != i - 1)) bits |= DSPARK_STATUS_BAD_ROWS;
        unsigned leads = __ballot_sync(0xffffffffu, lead);
#pragma unroll 1
        while (leads != 0) {
            const int k = __ffs(leads) - 1;
            leads &= leads - 1;
            const int bk = __shfl_sync(0xffffffffu, b, k), ik = __shfl_sync(0xffffffffu, i, k);
            const int pk = __shfl_sync(0xffffffffu, pos, k);
            if constexpr (T == 1) {
                bits |= append_blocks<DT, VEC, T>(A, row0 + from + k, bk, ik, pk, share * kWarps, false, tab, red);
            } else {
#pragma unroll 1
                for (int g = 0; g < (value ? 1 : kGroups); ++g)
                    if (head0 + g * kTeams < A.c.heads)
                        bits |= append_blocks<DT, VEC, T>(A, row0 + from + k, bk, ik, pk,
                                                          2 * (head0 + g * kTeams) + value, g > 0, tab, red);
            }
        }
    }
    return bits;
}

// A CTA's part of the queries, `block` of them.
template <int DT, bool QVEC>
__device__ __forceinline__ int rotate_queries(const AppendArgs& A, int block, float2* tab, int32_t* own, int32_t* at)
{
    int bits = 0;
    const int64_t row0 = static_cast<int64_t>(block) * A.q_rows;
    const int n = min(static_cast<int64_t>(A.q_rows), A.rows - row0);
    rotate_rows<DT, QVEC>(A.q, tab, row0, n, own, [&]() {
        if (threadIdx.x < n) own[threadIdx.x] = row_owner(A, row0 + threadIdx.x, &at[threadIdx.x], &bits);
        __syncthreads();
        for (int i = threadIdx.x; i < n * A.rope.half; i += blockDim.x) {
            const int k = i / A.rope.half;
            if (own[k] >= 0) tab[i] = rope_factor(A.rope, A.rope.turns[i - k * A.rope.half], at[k]);
        }
        __syncthreads();
    });
    return bits;
}

// A step: keys and values, and after them queries, in one launch.
template <int DT, bool VEC, bool QVEC>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(AppendArgs A)
{
    __shared__ __align__(16) float2 tab[kTable];
    __shared__ int32_t own[kQueryRows], at[kQueryRows];
    pdl_wait_and_trigger();
    int bits;
    if (static_cast<int>(blockIdx.x) >= A.kv_ctas)
        bits = rotate_queries<DT, QVEC>(A, blockIdx.x - A.kv_ctas, tab, own, at);
    else
        bits = append_rows<DT, VEC, 1>(A, tab, nullptr);
    if (bits) raise_status(A.status, bits);
}

// Prompts: the keys and values.
template <int DT, bool VEC>
__global__ void __launch_bounds__(32 * kPromptWarps, 2) append_prompt_kernel(AppendArgs A)
{
    __shared__ __align__(16) float2 tab[kTable];
    __shared__ float red[kPromptWarps];
    pdl_wait_and_trigger();
    const int bits = append_rows<DT, VEC, kTeam>(A, tab, red);
    if (bits) raise_status(A.status, bits);
}

// Prompts: the queries, beside the kernel above. It starts when that one has triggered its
// dependents, that is after everything before the call is done, touches nothing that one writes,
// and waits for it at its own end, so that what follows on the stream waits for both.
template <int DT, bool QVEC>
__global__ void __launch_bounds__(kQueryThreads) append_query_kernel(AppendArgs A)
{
    __shared__ __align__(16) float2 tab[kQueryFactors];
    __shared__ int32_t own[kQueryRows], at[kQueryRows];
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int bits = rotate_queries<DT, QVEC>(A, blockIdx.x, tab, own, at);
    if (bits) raise_status(A.status, bits);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
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
    A.row_req = row_req;
    A.row_pos = row_pos;
    A.lengths = lengths;
    A.rows = rows;
    A.B = B;
    A.status = status;
    // Steps: a warp per block, one row per CTA for the shortest chains in a small one (4 rows: 4.42 us
    // and 4.51 with four), four in a larger one, where about one row in four leads (2048 rows in 256
    // windows: 25 us, 33 with one). Prompts: four warps per block, so that a page's rows are read once
    // and stay in registers; by the rows that a block gets, which the page and the requests' average
    // bound. Pages of 64: one prompt of 64 rows 23 us, 40 the other way, 2048 rows 25 and 54; 64 windows
    // of 32 27 and 27, 256 of 8 53 and 25. One prompt of 2048 rows in pages of 32: 27 and 35, of 16: 33 and 25.
    const bool prompts = rows > 32ll * B && cache.page >= 32;
    A.chunk = prompts ? cache.page : rows <= 128 ? 1 : 4;
    A.q_rows = rows >= 152 * 8 && rope.half > 0 ? (rope.half <= 64 ? 4 : 2) : 1;
    A.key_shares = static_cast<int>(ceil_div(cache.heads, kPromptWarps / kTeam * kGroups));
    A.per_row = static_cast<int>(prompts ? A.key_shares + ceil_div(cache.heads, kPromptWarps / kTeam)
                                         : ceil_div(2 * cache.heads, kWarps));
    A.kv_ctas = static_cast<int>(ceil_div(rows, A.chunk)) * A.per_row;
    const int q_ctas = q != nullptr ? static_cast<int>(ceil_div(rows, A.q_rows)) : 0;
    const bool bf = dtype == DSPARK_BF16;
    const int e = bf ? 2 : 4;
    const bool qvec = rotate_vec(rope, q, qs, q_out, os, cache.dim, e);
    const bool vec = vector_rows(rope, k, ks, cache.dim, e) && vector_rows(rope, v, vs, cache.dim, e);
    A.q = turns_of(rope, q, qs, q_out, os, q != nullptr ? q_heads : 1, cache.dim, qvec, e, A.q_rows);
    if (prompts) {
        auto kv = bf ? (vec ? append_prompt_kernel<DSPARK_BF16, true> : append_prompt_kernel<DSPARK_BF16, false>)
                     : (vec ? append_prompt_kernel<DSPARK_F32, true> : append_prompt_kernel<DSPARK_F32, false>);
        const int rc = launch_pdl("append", kv, dim3(static_cast<unsigned>(A.kv_ctas)), dim3(32 * kPromptWarps), 0, stream, A);
        if (rc != DSPARK_OK || q == nullptr) return rc;
        auto turn = bf ? (qvec ? append_query_kernel<DSPARK_BF16, true> : append_query_kernel<DSPARK_BF16, false>)
                       : (qvec ? append_query_kernel<DSPARK_F32, true> : append_query_kernel<DSPARK_F32, false>);
        return launch_pdl("append queries", turn, dim3(static_cast<unsigned>(q_ctas)), dim3(kQueryThreads), 0, stream, A);
    }
    auto kernel = bf ? (vec ? (qvec ? append_kernel<DSPARK_BF16, true, true> : append_kernel<DSPARK_BF16, true, false>)
                            : (qvec ? append_kernel<DSPARK_BF16, false, true> : append_kernel<DSPARK_BF16, false, false>))
                     : (vec ? (qvec ? append_kernel<DSPARK_F32, true, true> : append_kernel<DSPARK_F32, true, false>)
                            : (qvec ? append_kernel<DSPARK_F32, false, true> : append_kernel<DSPARK_F32, false, false>));
    return launch_pdl("append", kernel, dim3(static_cast<unsigned>(A.kv_ctas + q_ctas)), dim3(kThreads), 0, stream, A);
}

}  // namespace dspark
