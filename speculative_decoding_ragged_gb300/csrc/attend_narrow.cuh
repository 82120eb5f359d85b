// attend_narrow.cuh — dspark_attend and its kin on the tensor cores for decode and verify: units of at most 32
// rows (window positions x query heads of one cache head): 8, 16 or 32, by the call.
//
// With few rows the products are turned round: the tile's 128 tokens (for the scores) and the
// head's elements (for the sums) fill the 128 lanes of the instruction, the rows are its columns:
//   S^T [128 tokens, 2 R] = K [128, D] (Q_1, Q_2)^T       O^T [D, 3 R] += V^T [D, 128] (W_1, W_2, W_3)
// so the products cost what the rows need, where 128 row lanes cost 1600 cycles a tile, and K and V
// are read from shared memory once. The pieces are separate columns and are added when they are read;
// at R = 32, where TMEM has no room for three sets of columns twice, the weights' are three products
// into one set. The weights' pieces are e5m2 for its range; in two e4m3 pieces, which end at 2^-16 of
// the largest, the batch below took 109 us, and a dominant token over 8192 others lost up to all of them.
// A thread's lane is a token: block scales are per-thread scalars, the rows' factors and
// references broadcast reads. The softmax needs no reduction over lanes in the common case: every
// thread checks its own exponents against the rows' references (one barrier with a vote), and
// only a tile that passes one by kBehind, a unit's first, or one that may lie far below finds the
// true maxima. The row sums stay in registers, one partial sum per row and thread, until the unit ends.
//
// A CTA: two groups of four warps do the softmax, a thread per token with half of the rows (groups
// of eight rows, four of them at R = 32, were 10 to 15 % slower) and prepare the queries of the
// pieces to come (a warp for that alone could not keep up: 140 us for 109 below); one warp loads
// pages with TMA, one issues the products one tile of scores ahead, one walks the run's units and
// describes them to the others. Scores and sums are double buffered in TMEM (256 columns), the ring
// holds 2.5 tiles of K and V, two CTAs per SM.
//
// Bound by HBM: 2 D bytes per token and cache head. What else showed in clock stamps was cold
// code (about 16 cycles per instruction the first time), hence one walker, rolled loops where
// registers allow them. 192 single tokens over 1 to 8 thousand, 8 heads of 128: 6.5 TB/s, 97 % of a
// copy. 256 windows of 1 to 8 over 128 to 2048: 113 us, 3.4 TB/s: a unit has about nine tiles, of about
// 2500 cycles each, and changing units costs 9000, the start 15 to 25 thousand.
#pragma once

#include "attend_mma.cuh"

namespace dspark {
namespace {

// Softmax threads: two groups of four warps (a thread per token), half of the rows each.
constexpr int group_rows(int R) { return R / 2; }
constexpr int groups(int R) { return R / group_rows(R); }
constexpr int soft_threads(int R) { return 128 * groups(R); }
constexpr int all_threads(int R) { return soft_threads(R) + 96; }
constexpr int kPieces = 8;                   // described pieces
// The weights' products: sets of R columns of sums, one for each of the three pieces or (R = 32) one
// for all; products for each 32 tokens; their columns, a multiple of 16; bytes of a token's row of weights.
constexpr int sum_sets(int R) { return R == 32 ? 1 : 3; }
constexpr int weight_products(int R) { return R == 32 ? 3 : 1; }
constexpr int weight_cols(int R) { return (sum_sets(R) * R + 15) / 16 * 16; }
constexpr int weight_row(int R) { return R == 32 ? 32 : 64; }

// A run's part of one unit.
struct Piece {
    int b, h, len, w;    // b: the row of the page table
    int row0, flat0;     // the request's first packed row; the unit's first (position, head)
    int rows;
    int k0, n;           // tiles
    int first_seen;
    int whole;           // nothing of the unit is elsewhere
    int last;
    int i0, g0;          // position and head of the unit's first row
    int from;            // the walk's
};
struct RowInfo {
    int prow, head;      // the row's packed row and query head
};

template <int D, int R, int SEE>
struct Smem {
    static constexpr int kSlot = kTile * D;              // one tile's K or V
    static constexpr int kSlots = D == 128 ? 5 : 10;     // K and V alternate
    static constexpr int kNums = kSlots / 2 + 2;         // tiles whose numbers may still be read
    uint8_t ring[kSlots][kSlot];
    uint8_t q[2][2 * R * D];                         // two units' queries: hi rows, lo rows
    uint8_t p[weight_products(R)][kTile * weight_row(R)];    // the weights, a row per token
    BlockNums nums[kNums][kBlocks];
    Piece piece[kPieces];
    RowInfo info[4][R];                                  // four units' rows
    __align__(16) int2 see[4][R];                    // first token seen, and how many past it
    __align__(16) float f[4][R];                     // score factors: scale log2(e) 2^e
    __align__(16) float ref[R];                      // kUp - reference (0: nothing seen yet)
    __align__(16) float grow[R];                     // 2^(old reference - new)
    float peak[R];                                   // kUp - the largest reference so far
    float4 part[R];                                  // the four warps' maxima or sums
    int look[groups(R)];                                 // the next tile that finds the maxima in any case
    int changed[groups(R)];                              // the last one that did changed a reference
    uint64_t full[kSlots], empty[kSlots];
    uint64_t piece_full[kPieces], q_full[2];
    uint64_t s_full[2], pv_done[2], p_full;
    Cut<R, SEE> cut;
    uint32_t tmem;
    int softened;        // pieces whose tiles the softmax is done with
    int stalled;         // a wait gave up: every role leaves its loop
};

// TMEM columns: scores at 64 * (tile & 1), sums at 128 + 64 * (unit & 1).
constexpr uint32_t kSums = 128;

// V^T as the first operand: its 128 lanes are the head's elements. Of a 64-wide head the second 64
// lanes read the first ones again (the stride between swizzle atoms is 0) and are ignored.
template <int D>
__device__ __forceinline__ uint64_t v_operand(uint64_t v)
{
    return D == 128 ? v : v & ~(0x3fffull << 16);
}

template <int N>
__device__ __forceinline__ void tc_ld(uint32_t addr, float* x)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    if (N == 4)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st4(uint32_t addr, const float* x)
{
    const uint32_t* r = reinterpret_cast<const uint32_t*>(x);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// The four warps of a group: a barrier, and a barrier with a vote.
__device__ __forceinline__ void group_sync(int grp) { asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory"); }
__device__ __forceinline__ bool group_any(int grp, bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n"
        " .reg .pred p, q;\n"
        " setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, %2, 128, p;\n"
        " selp.u32 %0, 1, 0, q;\n"
        "}\n" : "=r"(r) : "r"(static_cast<uint32_t>(yes)), "r"(5 + grp) : "memory");
    return r != 0;
}

// v[0..N) of every lane, combined over the warp's 32 lanes: lane i gets row i % N. Each step
// halves the rows a lane keeps, so N - 1 exchanges do what N full reductions would.
template <int N, bool MAX>
__device__ __forceinline__ float reduce_some(float* v, int lane)
{
    auto both = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int h = N / 2; h > 0; h >>= 1) {
        const bool up = (lane & h) != 0;
#pragma unroll
        for (int j = 0; j < h; ++j) {
            const float send = up ? v[j] : v[j + h], keep = up ? v[j + h] : v[j];
            v[j] = both(keep, __shfl_xor_sync(0xffffffffu, send, h));
        }
    }
    float y = v[0];
#pragma unroll
    for (int off = N; off < 32; off <<= 1) y = both(y, __shfl_xor_sync(0xffffffffu, y, off));
    return y;
}
// HR rows' values of a warp -> its column of part[r0 ..].
template <int HR, bool MAX>
__device__ __forceinline__ void reduce_rows(float4* part, float* v, int lane, int warp)
{
    const float y = reduce_some<HR, MAX>(v, lane);
    if (lane < HR) reinterpret_cast<float*>(part + lane)[warp] = y;
}

struct Token {
    BlockNums n;
    int t;
};

// One tile, this thread's token, one group's rows: scores in TMEM -> weights in shared memory;
// l += this token's weights.
template <int D, int R, int SEE>
__device__ __forceinline__ bool soften(Smem<D, R, SEE>& sm, int grp, int slot, uint64_t* l, uint32_t s_addr,
                                       uint32_t o_addr, const Token& k, bool mask, int tile, int it,
                                       int sinks, volatile int* stalled)
{
    constexpr int HR = group_rows(R);
    const int tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) & 3;
    const int r0 = grp * HR;
    const float4* f4 = reinterpret_cast<const float4*>(sm.f[slot] + r0);
    const float4* ref4 = reinterpret_cast<const float4*>(sm.ref + r0);
    const uint64_t ks2 = pack2(k.n.ks, k.n.ks), bias2 = pack2(k.n.bias, k.n.bias);
    uint64_t x[HR / 2];                       // pairs of rows
#pragma unroll 1
    for (int pass = 0;; ++pass) {
        constexpr int N = HR < 8 ? HR : 8;
#pragma unroll
        for (int c = 0; c < HR; c += N) {        // the two pieces' columns, added
            float hi[N], lo[N];
            tc_ld<N>(s_addr + r0 + c, hi);
            tc_ld<N>(s_addr + R + r0 + c, lo);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < N; j += 2)
                x[(c + j) / 2] = add2(pack2(hi[j], hi[j + 1]), pack2(lo[j], lo[j + 1]));
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
                const float4 f = f4[r / 4], ref = ref4[r / 4];
                x[r / 2] = fma2(x[r / 2], mul2(pack2(f.x, f.y), ks2), add2(bias2, pack2(ref.x, ref.y)));
                x[r / 2 + 1] = fma2(x[r / 2 + 1], mul2(pack2(f.z, f.w), ks2), add2(bias2, pack2(ref.z, ref.w)));
                const float2 a = unpack2(x[r / 2]), b = unpack2(x[r / 2 + 1]);
                top = fmaxf(top, fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y)));
            }
        if (mask) {
            top = -INFINITY;
            const int4* see2 = reinterpret_cast<const int4*>(sm.see[slot] + r0);
#pragma unroll
            for (int r = 0; r < HR; r += 2) {
                    const int4 s = see2[r / 2];
                    float2 a = unpack2(x[r / 2]);
                    if constexpr (SEE == kSinks) {
                        const bool sink = k.t < sinks;
                        if ((!sink && k.t < s.x) || k.t > s.x + s.y) a.x = -INFINITY;
                        if ((!sink && k.t < s.z) || k.t > s.z + s.w) a.y = -INFINITY;
                    } else {
                        if (static_cast<uint32_t>(k.t - s.x) > static_cast<uint32_t>(s.y)) a.x = -INFINITY;
                        if (static_cast<uint32_t>(k.t - s.z) > static_cast<uint32_t>(s.w)) a.y = -INFINITY;
                    }
                    x[r / 2] = pack2(a.x, a.y);
                    top = fmaxf(top, fmaxf(a.x, a.y));
                }
        }
        if (pass) break;
        const bool first = tile == 0;
        if (!first && !group_any(grp, top > kUp + kBehind || tile == sm.look[grp])) break;
        // The rows' maxima, as exponents over the present references; new references for the rows
        // that passed theirs by too much or lie far below, and those that see their first tokens.
        float v[HR];
#pragma unroll
        for (int r = 0; r < HR; r += 2) {
            const float2 a = unpack2(x[r / 2]);
            v[r] = a.x;
            v[r + 1] = a.y;
        }
        reduce_rows<HR, true>(sm.part + r0, v, lane, warp);
        group_sync(grp);
        if ((tid & 127) < 32) {
            const int r = r0 + min(lane, HR - 1);
            const float4 q = sm.part[r];
            const float over = fmaxf(fmaxf(q.x, q.y), fmaxf(q.z, q.w));
            const float old = sm.ref[r];
            const bool none = old == 0.0f;
            const float peak = sm.peak[r];
            float y = old;
            if (over > -INFINITY && (none || over > kUp + kBehind || over < kUp - kBelow)) {
                y = old - over + kUp;
                if (!none) y = fminf(y, peak + kDown);
                if (y == 0.0f) y = 1e-30f;       // 0 stands for none
            }
            __syncwarp();
            if (lane < HR) {
                sm.grow[r] = none ? 1.0f : ex2_approx(y - old);
                sm.ref[r] = y;
                sm.peak[r] = none ? y : fminf(peak, y);
            }
            // the next tile finds the maxima too where a row has seen nothing yet, or where a quarter of
            // this one lies far below another
            const float least = fminf(fminf(q.x, q.y), fminf(q.z, q.w));
            const bool next = __any_sync(0xffffffffu, y == 0.0f || over - least > kBelow);
            const bool changed = __any_sync(0xffffffffu, y != old);
            if (lane == 0) {
                sm.look[grp] = next ? tile + 1 : (tile | (kLook - 1)) + 1;
                sm.changed[grp] = changed;
            }
        }
        group_sync(grp);
        if (first) {                             // the present references were 0
#pragma unroll
            for (int r = 0; r < HR; r += 4) {
                    const float4 ref = ref4[r / 4];
                    x[r / 2] = add2(x[r / 2], pack2(ref.x, ref.y));
                    x[r / 2 + 1] = add2(x[r / 2 + 1], pack2(ref.z, ref.w));
                }
            break;
        }
        if (!sm.changed[grp]) break;
        // the tiles before this one have to be in the sums before these are scaled
        if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.pv_done[(it - 1) & 1]), ((it - 1) >> 1) & 1, stalled)))
            return false;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HR; c += 4) {
            float o[sum_sets(R)][4];
#pragma unroll
            for (int i = 0; i < sum_sets(R); ++i) tc_ld<4>(o_addr + i * R + r0 + c, o[i]);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < sum_sets(R); ++i) {
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][j] *= sm.grow[r0 + c + j];
                tc_st4(o_addr + i * R + r0 + c, o[i]);
            }
        }
        tc_wait_st();
#pragma unroll
        for (int r = 0; r < HR; r += 2)
            l[r / 2] = mul2(l[r / 2], pack2(sm.grow[r0 + r], sm.grow[r0 + r + 1]));
    }
    // the last tile's products read the weights that these replace
    if (it > 0 && !__all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.pv_done[(it - 1) & 1]),
                                                     ((it - 1) >> 1) & 1, stalled)))
        return false;
    const int token = tid & 127;
    // piece i of the rows from r0 on: the 64- or 32-byte swizzle of 16-byte chunks
    auto place = [&](int i) -> uint8_t* {
        if (weight_products(R) == 3)
            return &sm.p[i % weight_products(R)][token * 32 + (((r0 >> 4) ^ ((token >> 2) & 1)) << 4)];
        const int byte = i * R + r0;
        return &sm.p[0][token * 64 + (((byte >> 4) ^ ((token >> 1) & 3)) << 4) + (byte & 15)];
    };
    const uint64_t inv2 = pack2(k.n.inv, k.n.inv);
    uint32_t w[HR / 4][3];
#pragma unroll
    for (int c = 0; c < HR / 4; ++c)
        if (4 * c < HR) {
            float2 a = unpack2(x[2 * c]), b = unpack2(x[2 * c + 1]);
            a.x = ex2_approx(a.x);
            a.y = ex2_approx(a.y);
            b.x = ex2_approx(b.x);
            b.y = ex2_approx(b.y);
            l[2 * c] = fma2(pack2(a.x, a.y), inv2, l[2 * c]);
            l[2 * c + 1] = fma2(pack2(b.x, b.y), inv2, l[2 * c + 1]);
            split3(a.x, a.y, b.x, b.y, w[c]);
        }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (HR == 16)
            *reinterpret_cast<uint4*>(place(i)) = make_uint4(w[0][i], w[HR / 16][i], w[HR / 8][i], w[HR / 4 - 1][i]);
        else if (HR == 8)
            *reinterpret_cast<uint2*>(place(i)) = make_uint2(w[0][i], w[HR / 4 - 1][i]);
        else
            *reinterpret_cast<uint32_t*>(place(i)) = w[0][i];
    }
    return true;
}

// A finished piece, after its row sums are in part: results or a part written. Lane d holds
// element d. `partial` (kSuffix): the row has a prefix, whose kernel joins them.
template <int D, int R, int SEE>
__device__ __forceinline__ void finish(const AttendCall& A, Smem<D, R, SEE>& sm, int grp, int slot, uint32_t o_addr,
                                       int rows, bool whole, bool partial, int part, const Workspace& ws)
{
    const int tid = threadIdx.x;
    constexpr int HR = group_rows(R);
    const int r0 = grp * HR;
    const int d = tid & 127;
    if constexpr (SEE == kPrefix) {
        if (whole) {                             // the shares of every row to all its threads
            if (d < HR && r0 + d < rows) {
                const int64_t at = static_cast<int64_t>(sm.info[slot][r0 + d].prow) * A.q_heads + sm.info[slot][r0 + d].head;
                const float4 q = sm.part[r0 + d];
                const float sum = (q.x + q.y) + (q.z + q.w), own = A.part_lse[at];
                const Shares sh = shares_of(sum == 0.0f ? -INFINITY : log2f(sum) - sm.ref[r0 + d], own);
                sm.grow[r0 + d] = sum == 0.0f ? 0.0f : __fdividef(sh.s, sum);
                sm.peak[r0 + d] = is_part(own) ? sh.p : own;
                if (A.lse != nullptr && is_part(own)) A.lse[at] = sh.lse * kLn2;
            }
            group_sync(grp);
        }
    }
    uint16_t* out = static_cast<uint16_t*>(A.out) + d;
    float* po = ws.o + static_cast<int64_t>(part) * kTile * D + d;
#pragma unroll 1
    for (int c = r0; c < r0 + HR && c < rows; c += 4) {
        float o[sum_sets(R)][4];
#pragma unroll
        for (int i = 0; i < sum_sets(R); ++i) tc_ld<4>(o_addr + i * R + c, o[i]);
        int64_t at[4];
        float g[4], gp[4];                       // kPrefix: the own tokens' share
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 q = sm.part[c + j];
            const float sum = (q.x + q.y) + (q.z + q.w);
            const RowInfo in = sm.info[slot][c + j];
            at[j] = in.prow * A.out_stride + static_cast<int64_t>(in.head) * D;
            g[j] = !whole ? 1.0f : sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);      // nothing seen: zeros
            if (SEE == kSuffix && partial) at[j] = (static_cast<int64_t>(in.prow) * A.q_heads + in.head) * D + d;
            if constexpr (SEE == kPrefix) {
                gp[j] = sm.peak[c + j];
                if (whole) {
                    g[j] = sm.grow[c + j];
                    if (c + j < rows && is_part(gp[j]) && (D == 128 || d < D))
                        gp[j] *= A.part[(static_cast<int64_t>(in.prow) * A.q_heads + in.head) * D + d];
                }
            }
        }
        tc_wait_ld();
        if (D == 128 || d < D) {                 // D = 64: lanes 64.. repeat the first ones
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y = o[sum_sets(R) - 1][j];
#pragma unroll
                for (int i = sum_sets(R) - 2; i >= 0; --i) y += o[i][j];
                y *= g[j];
                if (SEE == kPrefix) {
                    if (whole && c + j < rows && is_part(sm.peak[c + j])) store1<DSPARK_BF16>(out, at[j], y + gp[j]);
                } else if (SEE == kSuffix && partial) {
                    if (whole && c + j < rows) A.part[at[j]] = y;
                } else if (whole && c + j < rows) store1<DSPARK_BF16>(out, at[j], y);
                if (!whole && c + j < rows) po[(c + j) * D] = y;
            }
        }
    }
    const int r = r0 + d;
    if (d < HR && r < rows) {
        const float4 q = sm.part[r];
        const float sum = (q.x + q.y) + (q.z + q.w);
        const float m = -sm.ref[r];              // reference - kUp, as the weights are
        const int64_t at = static_cast<int64_t>(sm.info[slot][r].prow) * A.q_heads + sm.info[slot][r].head;
        if (!whole)
            ws.ml[part * kTile + r] = make_float2(sum == 0.0f ? kNone : m, sum);
        else if (SEE == kSuffix && partial)
            A.part_lse[at] = sum == 0.0f ? -INFINITY : m + log2f(sum);
        else if (A.lse != nullptr && SEE != kPrefix)
            A.lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * kLn2;
    }
}

// A lane's share of a unit's queries: 16 elements of row `row`, one of its D / 16 segments.
struct QueryAt {
    int64_t prow;                                // the row's packed row and head
    int head, pos;
};
__device__ __forceinline__ QueryAt query_at(const AttendCall& A, const Piece& pc, int row)
{
    QueryAt q;
    int i = pc.i0, g = pc.g0 + min(row, pc.rows - 1);
    if (g >= A.group) {
        const int more = g / A.group;
        i += more;
        g -= more * A.group;
    }
    q.prow = pc.row0 + i;
    q.head = pc.h * A.group + g;
    q.pos = pc.len + i;
    return q;
}
template <int D>
__device__ __forceinline__ void fetch_query(const AttendCall& A, const QueryAt& q, uint4* v)
{
    const uint16_t* at = static_cast<const uint16_t*>(A.q) + q.prow * A.q_stride +
                         static_cast<int64_t>(q.head) * D + (threadIdx.x & (D / 16 - 1)) * 16;
    if ((reinterpret_cast<uintptr_t>(at) & 15u) == 0) {
        v[0] = reinterpret_cast<const uint4*>(at)[0];
        v[1] = reinterpret_cast<const uint4*>(at)[1];
    } else {
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = at[8 * j + 2 * k] | (static_cast<uint32_t>(at[8 * j + 2 * k + 1]) << 16);
            (j ? v[1] : v[0]) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}
// The fetched elements as two pieces in shared memory; the row's factor and what the softmax needs
// to know of it go to slot `slot`. Rows past the unit's are zeros. All 32 lanes.
template <int D, int R, int SEE>
static __device__ __noinline__ void put_query(const AttendCall& A, Smem<D, R, SEE>& sm, const Piece& pc, int slot,
                                              uint8_t* q, int row, uint4 v0, uint4 v1)
{
    constexpr int S = D / 16;
    const int seg = threadIdx.x & (S - 1);
    uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t top = 0;                            // magnitudes' bits order like them, NaN above all
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        if (row >= pc.rows) w[k] = 0;
        top = max(top, max(w[k] & 0x7fffu, (w[k] >> 16) & 0x7fffu));
    }
#pragma unroll
    for (int off = 1; off < S; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
    const bool fine = top < 0x7f80u;
    const int e = fine ? scale_exponent(__uint_as_float(top << 16)) : 0;
    const float inv = exp2i(-e);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float y[4] = {bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv,
                            bf16_lo(w[2 * k + 1]) * inv, bf16_hi(w[2 * k + 1]) * inv};
        float z[4];
        hi[k] = e4m3x4(y[0], y[1], y[2], y[3]);
        e4m3x4_to_f32(hi[k], z);
        lo[k] = e4m3x4(y[0] - z[0], y[1] - z[1], y[2] - z[2], y[3] - z[3]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int rr = p * R + row;
        const int chunk = seg ^ (D == 128 ? rr & 7 : (rr >> 1) & 3);
        *reinterpret_cast<uint4*>(q + rr * D + chunk * 16) =
            p ? make_uint4(lo[0], lo[1], lo[2], lo[3]) : make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    if (seg == 0) {
        const QueryAt at = query_at(A, pc, row);
        const int pos = SEE == kPrefix ? pc.len - 1 : at.pos;
        const int first = first_seen_at<SEE>(A, pos, pc.from);
        sm.info[slot][row] = {static_cast<int>(at.prow), at.head};
        sm.see[slot][row] = make_int2(first, pos - first);
        // a query that is not finite makes its row's factor, hence its results, NaN
        sm.f[slot][row] = fine ? A.scale * kLog2e * exp2i(e) : __int_as_float(0x7fc00000);
    }
}

template <int R, int SEE>
__device__ __forceinline__ void describe(const AttendCall& A, const Walk<R, SEE>& wk, Piece& p)
{
    p.b = table_of<SEE>(wk.b, wk.from);
    p.h = wk.h;
    p.len = wk.len;
    p.w = wk.w;
    p.row0 = wk.row0;
    p.flat0 = wk.qt * R;
    p.rows = wk.rows(A);
    p.i0 = p.flat0 == 0 ? 0 : p.flat0 / A.group;
    p.g0 = p.flat0 - p.i0 * A.group;
    p.k0 = wk.k0;
    p.n = wk.n;
    p.first_seen = wk.first_seen(A);
    p.whole = wk.whole();
    if constexpr (SEE == kSinks || SEE == kSuffix) p.from = wk.from;
    p.last = wk.last();
}

template <int D, int R, int SEE>
__global__ void __launch_bounds__(all_threads(R), 2)
attend_narrow_kernel(const __grid_constant__ AttendCall A, const __grid_constant__ CUtensorMap k_map,
                     const __grid_constant__ CUtensorMap v_map)
{
    extern __shared__ __align__(kSmemAlign) unsigned char raw[];
    typedef Smem<D, R, SEE> S;
    S& sm = *reinterpret_cast<S*>(raw);
    static_assert(sizeof(S) <= kSmemTwo, "two CTAs per SM");
    constexpr int kSlots = S::kSlots;
    constexpr int kNums = S::kNums;
    constexpr int G = groups(R), kLoader = 4 * G, kIssuer = kLoader + 1, kWalker = kLoader + 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Workspace ws = workspace_of(A.ws);
    if (!smem_aligned(A, ws, raw)) return;
    if constexpr (SEE == kPrefix) {              // a call that computes no prefix apart ends here
        pdl_wait_and_trigger();
        if (A.from[A.requests] == 0) {
            if (threadIdx.x == 0) ws.meta[blockIdx.x].rows = 0;
            return;
        }
    }

    if (tid < kSlots) {
        mbar_init(smem_addr(&sm.full[tid]), 1);
        mbar_init(smem_addr(&sm.empty[tid]), 1);
    } else if (tid >= 32 && tid < 32 + kPieces) {
        const int s = tid - 32;
        mbar_init(smem_addr(&sm.piece_full[s]), 1);
        if (s < 2) {
            mbar_init(smem_addr(&sm.q_full[s]), soft_threads(R));
            mbar_init(smem_addr(&sm.s_full[s]), 1);
            mbar_init(smem_addr(&sm.pv_done[s]), 1);
        }
        if (s == 2) mbar_init(smem_addr(&sm.p_full), soft_threads(R));
        if (s == 3) sm.stalled = sm.softened = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;"
                     ::"r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    pdl_wait_and_trigger();
    const int run = cut_line<R, SEE, all_threads(R)>(A, sm.cut);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    volatile int* stalled = &sm.stalled;
    if (tid == 0) write_meta<R, SEE>(A, ws, sm.cut.walk, run);
    if (sm.cut.walk.n > 0) {
        if (warp == kWalker) {
            // ---- the walk: pieces described to the others, and their queries fetched into L2 ----
            Walk<R, SEE> wk = sm.cut.walk;
#pragma unroll 1
            for (int d = 0;; ++d) {
                // the slot's last piece, and the one after it, are behind every role
                const long long deadline = clock64() + kWaitCycles;
                while (d >= kPieces - 2 && *reinterpret_cast<volatile int*>(&sm.softened) < d - (kPieces - 2) + 1) {
                    if (*stalled || clock64() > deadline) { *stalled = 1; break; }
                    __nanosleep(100);
                }
                if (__any_sync(0xffffffffu, *stalled)) break;
                Piece& pc = sm.piece[d & (kPieces - 1)];
                if (lane == 0) {
                    describe<R, SEE>(A, wk, pc);
                    mbar_arrive(smem_addr(&sm.piece_full[d & (kPieces - 1)]));
                }
                __syncwarp();
                if (lane < pc.rows) {
                    const QueryAt at = query_at(A, pc, lane);
                    const char* q = reinterpret_cast<const char*>(static_cast<const uint16_t*>(A.q) + at.prow * A.q_stride +
                                                                  static_cast<int64_t>(at.head) * D);
#pragma unroll
                    for (int o = 0; o < D * 2; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + o));
                }
                if (wk.last()) break;
                wk.next(A);
            }
        } else if (warp == kLoader) {
            // ---- pages in ----
            const int per_tile = kTile / A.c.page;
            const uint32_t box = static_cast<uint32_t>(A.c.page) * D;
            const int beyond = A.c.n_pages * A.c.heads * A.c.page;     // a row past the tensor: zeros
            int bad = 0, issued = 0, slot = 0, num = 0;
            uint32_t phase = 0;                              // parity of this use of the slot
            bool ok = true, ahead = false;
            int ahead_id = -1;
            float2 ahead_sc = make_float2(0.0f, 0.0f);
            auto scales_of = [&](int id, int h) -> float2 {
                if (id < 0) return make_float2(0.0f, 0.0f);
                const int64_t bh = static_cast<int64_t>(id) * A.c.heads + h;
                return make_float2(A.c.k_scale[bh], A.c.v_scale[bh]);
            };
            auto id_of = [&](const Piece& p, int n) -> int {        // -1: dead, not there, or not a page
                const int j = real_block<SEE>(A, n, p.from);
                if (n >= (p.k0 + p.n) * per_tile ||
                    j >= (stored_tokens<SEE>(p.len, p.w) + A.c.page - 1) / A.c.page ||
                    ((j + 1) * A.c.page <= p.first_seen && !(SEE == kSinks && j * A.c.page < A.sinks))) return -1;
                const int id = j < A.c.width ? A.c.table[static_cast<int64_t>(p.b) * A.c.width + j] : -1;
                if (id < 0 || id >= A.c.n_pages) { bad = 1; return -1; }
                return id;
            };
#pragma unroll 1
            for (int piece = 0; ok; ++piece) {
                const Piece& pc = sm.piece[piece & (kPieces - 1)];
                ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.piece_full[piece & (kPieces - 1)]),
                                                       (piece / kPieces) & 1, stalled));
                if (!ok) break;
                const int h = pc.h, n = pc.n;
                const bool last = pc.last;
                const int total_blocks = (stored_tokens<SEE>(pc.len, pc.w) + A.c.page - 1) / A.c.page;
                // 32 blocks at a time, one per lane; the next 32, or the next piece's first, are
                // fetched while these load
                int base = pc.k0 * per_tile;
                int id = -1, next_id = ahead_id, j0 = 32;
                if (!ahead) next_id = id_of(pc, base + lane);
                bool have = ahead;               // the first blocks' scales
                ahead = false;
                float2 sc = make_float2(0.0f, 0.0f);
                base -= 32;
#pragma unroll 1
                for (int k = 0; k < n; ++k) {
                    if (j0 == 32) {                          // the next 32 blocks
                        j0 = 0;
                        base += 32;
                        id = next_id;
                        sc = have ? ahead_sc : scales_of(id, h);
                        have = false;
                        if (base + 32 < (pc.k0 + n) * per_tile) {
                            next_id = id_of(pc, base + 32 + lane);
                        } else if (!last) {
                            const int s = (piece + 1) & (kPieces - 1);
                            ahead = __all_sync(0xffffffffu, mbar_test(smem_addr(&sm.piece_full[s]),
                                                                      ((piece + 1) / kPieces) & 1));
                            if (ahead) ahead_id = id_of(sm.piece[s], sm.piece[s].k0 * per_tile + lane);
                        }
                    }
                    const int src = j0 + (lane & (per_tile - 1));
                    const int my_id = __shfl_sync(0xffffffffu, id, src);
                    const bool there = lane < per_tile && real_block<SEE>(A, base + src, pc.from) < total_blocks;
                    const int count = __popc(__ballot_sync(0xffffffffu, there));
                    const int row = my_id < 0 ? beyond : (my_id * A.c.heads + h) * A.c.page;
#pragma unroll 1
                    for (int kv = 0; kv < 2; ++kv) {
                        if (issued >= kSlots)
                            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.empty[slot]), phase ^ 1u, stalled));
                        if (!ok) break;
                        const uint32_t full = smem_addr(&sm.full[slot]);
                        if (kv == 1) {
                            const float ks = __shfl_sync(0xffffffffu, sc.x, src);
                            const float vs = __shfl_sync(0xffffffffu, sc.y, src);
                            BlockNums b;
                            b.ks = my_id < 0 ? 0.0f : ks;
                            b.bias = my_id < 0 ? -INFINITY : __log2f(vs);
                            b.inv = my_id < 0 ? 0.0f : ex2_approx(-b.bias);
                            b.pad = 0.0f;
                            if (lane < per_tile) sm.nums[num][lane] = b;
                            if (++num == kNums) num = 0;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(full, count * box);
                        __syncwarp();
                        if (there)
                            tma_load(smem_addr(sm.ring[slot]) + lane * box, kv ? &v_map : &k_map, row, full);
                        ++issued;
                        if (++slot == kSlots) { slot = 0; phase ^= 1u; }
                    }
                    if (!ok) break;
                    j0 += per_tile;
                }
                if (ahead) ahead_sc = scales_of(ahead_id, sm.piece[(piece + 1) & (kPieces - 1)].h);
                if (last) break;
            }
            if (bad) raise_status(A.status, DSPARK_STATUS_BAD_PAGE);
            // every started copy lands before the CTA may leave
            __syncwarp();
#pragma unroll 1
            for (int s = 0; s < kSlots && s < issued; ++s)
                drain(smem_addr(&sm.full[s]), ((issued - 1 - s) / kSlots) & 1, stalled);
        } else if (warp == kIssuer) {
            // ---- products: the warp runs as one, an elected lane issues ----
            const bool leader = elect_one();
            constexpr uint32_t kIdesc = (1u << 4) | (kTile / 16 << 24) | (R / 4 << 17);      // 2 R columns
            // V^T: the head's elements are contiguous, and so are the weights' rows
            // by e5m2
            constexpr uint32_t kIdescPV = (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) |
                                          (weight_cols(R) / 8 << 17) | (kTile / 16 << 24);
            const uint32_t tmem = sm.tmem;
            const uint64_t ring0 = operand<D>(smem_addr(sm.ring[0]));
            const uint64_t q_op = operand<D>(smem_addr(sm.q[0]));
            constexpr int kP = weight_row(R);
            const uint64_t p_op = operand<kP>(smem_addr(sm.p));
            constexpr uint32_t kStep = S::kSlot / 16;
            constexpr uint32_t kQStep = sizeof(sm.q[0]) / 16;
            // the scores run one tile ahead of the sums: their own place in the pieces
            int pa = -1, left_a = 0, it_a = 0, slot_a = 0;
            uint32_t phase_a = 0;
            bool last_a = false, ready = true, ok = true;
            auto test = [&](uint32_t bar, uint32_t parity, bool wait) -> bool {
                return __all_sync(0xffffffffu, wait ? mbar_wait(bar, parity, stalled) : mbar_test(bar, parity));
            };
            // the scores of tile it_a; unless `wait`, only if everything is there already
            auto scores = [&](bool wait) -> bool {
                if (left_a == 0) {
                    if (ready) { ++pa; ready = false; }
                    const int s = pa & (kPieces - 1);
                    if (!test(smem_addr(&sm.piece_full[s]), (pa / kPieces) & 1, wait)) return false;
                    if (!test(smem_addr(&sm.q_full[pa & 1]), (pa >> 1) & 1, wait)) return false;
                    ready = true;
                    left_a = sm.piece[s].n;
                    last_a = sm.piece[s].last;
                }
                if (!test(smem_addr(&sm.full[slot_a]), phase_a, wait)) return false;
                tc_fence_after();
                --left_a;
                if (leader) {
                    const uint64_t a = ring0 + slot_a * kStep, b = q_op + (pa & 1) * kQStep;
#pragma unroll
                    for (int s = 0; s < D / 32; ++s)
                        mma_ss(tmem + 64 * (it_a & 1), a + 2 * s, b + 2 * s, kIdesc, s > 0);
                    tc_commit(smem_addr(&sm.s_full[it_a & 1]));
                    tc_commit(smem_addr(&sm.empty[slot_a]));
                }
                __syncwarp();
                slot_a += 2;
                if (slot_a >= kSlots) { slot_a -= kSlots; phase_a ^= 1u; }
                ++it_a;
                return true;
            };
            int it = 0, piece = -1, left = 0, slot = 1;
            uint32_t phase = 0, o_addr = 0;
            bool last = false, fresh = true;
#pragma unroll 1
            while (true) {
                // this tile's scores by all means, the next one's if they can start
#pragma unroll 1
                while (it_a <= it + 1 && !(last_a && left_a == 0)) {
                    const bool must = it_a == it;
                    if (!scores(must)) { ok = !must; break; }
                }
                if (!ok) break;
                if (left == 0) {
                    const Piece& pc = sm.piece[++piece & (kPieces - 1)];
                    left = pc.n;
                    last = pc.last;
                    o_addr = tmem + kSums + 64 * (piece & 1);
                    fresh = true;
                }
                ok = test(smem_addr(&sm.p_full), it & 1, true) && test(smem_addr(&sm.full[slot]), phase, true);
                if (!ok) break;
                tc_fence_after();
                if (leader) {
                    const uint64_t a = v_operand<D>(ring0 + slot * kStep);
#pragma unroll
                    for (int s = 0; s < kTile / 32; ++s)
#pragma unroll
                        for (int i = 0; i < weight_products(R); ++i)
                            mma_ss(o_addr, a + s * (32 * D / 16), p_op + i * (kTile * kP / 16) + s * (32 * kP / 16),
                                   kIdescPV, !fresh || s > 0 || i > 0);
                    tc_commit(smem_addr(&sm.pv_done[it & 1]));
                    tc_commit(smem_addr(&sm.empty[slot]));
                }
                __syncwarp();
                fresh = false;
                slot += 2;
                if (slot >= kSlots) { slot -= kSlots; phase ^= 1u; }
                ++it;
                if (--left == 0 && last) break;
            }
            // the last products' arrivals on the barriers land before the CTA leaves
            if (it > 0) {
                const int uk = 2 * (it - 1), uv = uk + 1;
                drain(smem_addr(&sm.empty[uk % kSlots]), (uk / kSlots) & 1, stalled);
                drain(smem_addr(&sm.empty[uv % kSlots]), (uv / kSlots) & 1, stalled);
            }
            __syncwarp();
        } else {
            // ---- softmax ----
            const int grp = warp >> 2;
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int token = tid & 127;
            const int my_block = token / A.c.page;
            int it = 0, piece = 0, slot = 1, num = 0;
            uint32_t phase = 0;
            bool ok = true;
            // Piece `p`'s queries: fetched here, put into shared memory by put() some time later.
            constexpr int kSegments = D / 16;
            const bool carries = warp * 32 / kSegments < R;
            uint4 v[2];
            auto fetch = [&](int p) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.piece_full[p & (kPieces - 1)]),
                                                             (p / kPieces) & 1, stalled));
                if (ok && carries) fetch_query<D>(A, query_at(A, sm.piece[p & (kPieces - 1)], tid / kSegments), v);
            };
            auto put = [&](int p) {
                if (ok && carries)
                    put_query<D, R, SEE>(A, sm, sm.piece[p & (kPieces - 1)], p & 3, sm.q[p & 1], tid / kSegments, v[0], v[1]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_addr(&sm.q_full[p & 1]));
            };
#pragma unroll 1
            for (int p = 0; p < 2; ++p) {
                fetch(p);
                put(p);
                if (!ok || sm.piece[p].last) break;
            }
            auto run_piece = [&]() -> bool {
                const Piece& pc = sm.piece[piece & (kPieces - 1)];
                constexpr int HR = group_rows(R);
                const int n = pc.n, rows = pc.rows;
                uint64_t l[HR / 2];
#pragma unroll
                for (int r = 0; r < HR / 2; ++r) l[r] = 0;
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.q_full[piece & 1]),
                                                             (piece >> 1) & 1, stalled));
                if (token < HR) sm.ref[grp * HR + token] = 0.0f;
                // tiles that every row sees whole need no mask
                const int first_pos = sm.see[piece & 3][0].x + sm.see[piece & 3][0].y;
                const int last_lo = sm.see[piece & 3][rows - 1].x;
                const int stored = stored_tokens<SEE>(pc.len, pc.w);
                group_sync(grp);
                const uint32_t o_addr = sm.tmem + lanes + kSums + 64 * (piece & 1);
                // a warp whose wait gave up goes on to the piece's end, where the warps agree on it:
                // they share the barriers within
                Token t;
                t.t = pc.k0 * kTile + token;
#pragma unroll 1
                for (int k = 0; k < n; ++k, ++it, t.t += kTile) {
                    if constexpr (SEE == kSinks) t.t = real_token<SEE>(A, (pc.k0 + k) * kTile + token, pc.from);
                    const int token0 = t.t - token;
                    ok = ok && mbar_wait(smem_addr(&sm.full[slot]), phase, stalled) &&
                         mbar_wait(smem_addr(&sm.s_full[it & 1]), (it >> 1) & 1, stalled);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    t.n = sm.nums[num][my_block];
                    if (++num == kNums) num = 0;
                    const bool mask = SEE == kSinks ? masked_tile<SEE>(A, pc.k0 + k, pc.from, last_lo, first_pos)
                                                    : token0 + kTile - 1 > first_pos || token0 < last_lo;
                    ok = soften<D, R, SEE>(sm, grp, piece & 3, l, sm.tmem + lanes + 64 * (it & 1), o_addr, t, mask, k, it,
                                           A.sinks, stalled) && ok;
                    tc_fence_before();
                    if (t.t >= stored) {         // a slot past the last token: 0 x NaN is NaN
                        uint4* v = reinterpret_cast<uint4*>(&sm.ring[slot][token * D + grp * (D / G)]);
#pragma unroll
                        for (int c = 0; c < D / G / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    if (ok) mbar_arrive(smem_addr(&sm.p_full));
                    slot += 2;
                    if (slot >= kSlots) { slot -= kSlots; phase ^= 1u; }
                }
                // the queries of the piece after the next go where this one's were
                if (tid == 0) *reinterpret_cast<volatile int*>(&sm.softened) = piece + 1;
                const bool more = !pc.last && !sm.piece[(piece + 1) & (kPieces - 1)].last;
                if (more) fetch(piece + 2);
                float sums[HR];
#pragma unroll
                for (int r = 0; r < HR; r += 2) {
                    const float2 a = unpack2(l[r / 2]);
                    sums[r] = a.x;
                    sums[r + 1] = a.y;
                }
                reduce_rows<HR, false>(sm.part + grp * HR, sums, lane, warp & 3);
                if (more) put(piece + 2);
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.pv_done[(it - 1) & 1]),
                                                             ((it - 1) >> 1) & 1, stalled));
                if (group_any(grp, !ok)) return false;
                tc_fence_after();
                finish<D, R, SEE>(A, sm, grp, piece & 3, o_addr, rows, pc.whole, SEE == kSuffix && pc.from > 0,
                                  blockIdx.x * 2 + (piece > 0), ws);
                return true;
            };
#pragma unroll 1
            for (;; ++piece) {
                const Piece& pc = sm.piece[piece & (kPieces - 1)];
                if (group_any(grp, !ok)) break;
                ok = run_piece();
                if (!ok) break;
                if (pc.last) break;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sm.stalled) raise_status(A.status, DSPARK_STATUS_STALL);
    if (warp == kIssuer)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(sm.tmem));
}

template <int D, int R, int SEE>
int launch(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    const size_t smem = sizeof(Smem<D, R, SEE>);
    // opt-in to large shared memory, once per device and host thread: threads share no state
    static thread_local int ready_device = -1;
    if (ready_device != device) {
        const cudaError_t e = cudaFuncSetAttribute(attend_narrow_kernel<D, R, SEE>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(DSPARK_ERR_CUDA, "dspark attend: %s", cudaGetErrorString(e));
        }
        ready_device = device;
    }
    CUtensorMap k_map, v_map;
    int rc = encode_cache(&k_map, A.c.k, A.c);
    if (rc == DSPARK_OK) rc = encode_cache(&v_map, A.c.v, A.c);
    if (rc != DSPARK_OK) return rc;
    return launch_pdl("attend", attend_narrow_kernel<D, R, SEE>, dim3(ctas), dim3(all_threads(R)), smem, stream, A,
                      k_map, v_map);
}

}  // namespace

template <int SEE>
int launch_attend_narrow(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    const int rows = unit_rows(A);
    if (A.c.dim == 128)
        return rows == 8 ? launch<128, 8, SEE>(A, ctas, device, stream)
             : rows == 16 ? launch<128, 16, SEE>(A, ctas, device, stream)
                          : launch<128, 32, SEE>(A, ctas, device, stream);
    return rows == 8 ? launch<64, 8, SEE>(A, ctas, device, stream)
         : rows == 16 ? launch<64, 16, SEE>(A, ctas, device, stream)
                      : launch<64, 32, SEE>(A, ctas, device, stream);
}

}  // namespace dspark
