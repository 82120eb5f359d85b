// attend_wide.cu — dspark_attend on the tensor cores for prompts and large groups: units of up to
// 128 rows, one row per TMEM lane.
//   S [128 rows, 128 tokens] = (Q_1 + Q_2) K^T       O [128 rows, D] += W V
// the queries' pieces adding up in the same columns, the weights in fp16.
//
// A CTA: warps 0-3 do the softmax, a thread per row, warp 4 loads pages with TMA (one box per page
// and K or V, swizzled), warp 5 issues the products. As in the narrow kernel a row's weights are
// taken over a reference that may lag its maximum: the scores pass through registers once, and
// only a tile in which some row of a warp passes its reference by kBehind or, where that is looked
// at, lies far below it, or a unit's first, stops to change references and rescale the sums. Two or
// four threads per row were slower (617 and 677 us, where one took 570): what a warp does once per
// tile, waits, votes, numbers, costs it as much as its elements, and one row's threads have to agree
// on a reference.
// The values are widened to fp16 in shared memory (exact), a token by each softmax thread, while the
// weights are one fp16 number each. Here the rows are many: for 128 of them three e5m2 pieces per
// weight cost 610 us for 507 (splitting them), and two e4m3 pieces, 508, end at 2^-16 of the largest.
// The weights go through shared memory, so that a tile's scores leave TMEM as soon as they are read
// and the next tile's products run under this one's softmax (as an operand in TMEM they overlaid
// the scores: 705 us for 641); 128 + D columns, so two CTAs fit and one's softmax runs under the
// other's. What a piece needs to be known by lives in shared memory: a thread holds 128 scores.
//
// Bound: sixteen products of about 101 cycles a tile at D = 128, 1616 cycles a tile and SM, and the
// softmax, which takes a CTA about 4250 cycles a tile, 2100 with two of them. Two prompts' pieces of
// about 2000 rows, 32 query heads of 128 over 8 heads, after 4 to 8 thousand tokens: 507 us, 0.93
// PFLOP/s of the plain form's 16-bit products. Its registers are tight: ptxas places the same
// source's scores well or badly (640 us with the queries loaded in two halves).
#include "attend_mma.cuh"

namespace dspark {
namespace {

constexpr int kRows = 128;
constexpr int kSoft = kRows;                 // softmax threads: one per row
constexpr int kThreads = kSoft + 64;

template <int D>
struct Smem {
    static constexpr int kSlot = kTile * D;              // one tile's K or V; 1024-byte aligned in order
    // K and V alternate. One of each suffices at D = 128, where two CTAs leave no room for more: K's
    // slot is free for a whole softmax, V's until the end of the next one.
    static constexpr int kSlots = D == 128 ? 2 : 4;
    uint8_t q[2][kTile * D];                             // the queries' two pieces
    uint8_t w[2][kRows * kTile];                         // the weights in fp16, 64 tokens each
    uint8_t ring[kSlots][kSlot];
    // The tile's values in fp16, 64 elements each. At D = 128 the first 64 take the place of V's codes in
    // the ring: a thread widens the 128 bytes of its own token, there and here.
    uint8_t wide[kTile * 128];
    // A tile's numbers are written once K's slot is free, kSlots / 2 tiles ahead at most, and read
    // until the tile's softmax ends: kNums slots cover kSlots / 2 + 1 tiles and the one being written.
    static constexpr int kNums = kSlots / 2 + 2;
    BlockNums nums[kNums][kBlocks];
    int8_t e[kRows];                                     // the rows' exponents; kNotFine: a query that is not finite
    uint8_t after[kRows];                                // their positions after the unit's first
    uint64_t full[kSlots], empty[kSlots];
    uint64_t s_full, s_read, p_full, pv_done, q_full;
    Cut<kRows> cut;        // its scan: afterwards how far the rows' references went down
    // The softmax threads' piece: here rather than in registers, which the scores need.
    Walk<kRows> soft;
    struct {
        int k0, n;         // its tiles
        int lo, hi;        // tokens from lo to hi are seen by all its rows; hi is the first row's position
    } span;
    int stored;            // the request's tokens
    uint32_t tmem;
    int stalled;       // a wait gave up: every role leaves its loop
};

constexpr int kNotFine = 127;

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// A barrier of the softmax threads, which says whether any of them says yes.
__device__ __forceinline__ bool soft_any(bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n"
        " .reg .pred p, q;\n"
        " setp.ne.u32 p, %1, 0;\n"
        " barrier.cta.red.or.pred q, 1, 128, p;\n"
        " selp.u32 %0, 1, 0, q;\n"
        "}\n" : "=r"(r) : "r"(static_cast<uint32_t>(yes)) : "memory");
    return r != 0;
}

struct Row {
    float f;              // score factor: scale log2(e) 2^e of the row's pieces
    float ref;            // kUp - reference; 0: nothing seen yet
    float l;              // the sum
    bool watch;           // a reference of the warp changed in the last tile
};

// One tile of this thread's row: scores in TMEM -> weights in shared memory.
// False once a wait gave up.
template <int D>
__device__ __forceinline__ bool soften(Smem<D>& sm, Row& r, uint32_t lanes, int row,
                                       const BlockNums* nums, int shift_page, int window, int k, int it, bool ok,
                                       volatile int* stalled)
{
    const uint32_t s_addr = sm.tmem + lanes;
    float x[kTile];
#pragma unroll
    for (int c = 0; c < kTile; c += 32) tc_ld32(s_addr + c, x + c);
    float2 num[kBlocks];
#pragma unroll
    for (int g = 0; g < kBlocks; ++g)
        num[g] = *reinterpret_cast<const float2*>(&nums[(g * 16) >> shift_page]);
    tc_wait_ld();
    tc_fence_before();
    __syncwarp();
    if (ok && (threadIdx.x & 31) == 0) mbar_arrive(smem_addr(&sm.s_read));
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < kTile; g += 16) {
        const float f = r.f * num[g / 16].x, add = num[g / 16].y + r.ref;
        const uint64_t f2 = pack2(f, f), a2 = pack2(add, add);
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
            const float2 y = unpack2(fma2(pack2(x[g + j], x[g + j + 1]), f2, a2));
            x[g + j] = y.x;
            x[g + j + 1] = y.y;
        }
    }
    const int token0 = (sm.span.k0 + k) * kTile;
    if (token0 + kTile - 1 > sm.span.hi || token0 < sm.span.lo) {
        const int pos = sm.span.hi + sm.after[row];
        const int first = window > 0 && pos >= window ? pos - window + 1 : 0;
        const uint32_t at = static_cast<uint32_t>(token0 - first), span = static_cast<uint32_t>(pos - first);
#pragma unroll
        for (int j = 0; j < kTile; ++j)
            if (at + j > span) x[j] = -INFINITY;
    }
    {
        float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int j = 4; j < kTile; ++j) m[j & 3] = fmaxf(m[j & 3], x[j]);
        top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    }
    const bool down = r.watch || look_down(k);
    const bool stop = __any_sync(0xffffffffu, top > kUp + kBehind || r.ref == 0.0f || (down && top < kUp - kBelow));
    r.watch = false;
    // the last tile's products read the weights' place and write the sums
    if (it > 0) ok = ok && mbar_wait(smem_addr(&sm.pv_done), (it - 1) & 1, stalled);
    ok = __all_sync(0xffffffffu, ok);
    if (stop) {
        float shift = 0.0f, g = 1.0f;
        if (top > -INFINITY && (r.ref == 0.0f || top > kUp + kBehind || top < kUp - kBelow)) {
            // how far the reference lies under the row's largest, in whole steps, at most kDown
            uint8_t& lowered = reinterpret_cast<uint8_t*>(sm.cut.scan)[row];
            shift = kUp - top;
            if (r.ref == 0.0f) {
                lowered = 0;
            } else {
                if (shift > 0.0f) shift = floorf(fminf(shift, kDown - lowered));
                lowered = static_cast<uint8_t>(max(0, lowered + static_cast<int>(ceilf(shift))));
            }
            float ref = r.ref + shift;
            if (ref == 0.0f) ref = 1e-30f;       // 0 stands for none
            shift = ref - r.ref;
            if (r.ref != 0.0f) {
                g = ex2_approx(shift);
                r.l *= g;
            }
            r.ref = ref;
        }
        r.watch = __any_sync(0xffffffffu, shift != 0.0f);
#pragma unroll
        for (int j = 0; j < kTile; j += 2) {
            const float2 y = unpack2(add2(pack2(x[j], x[j + 1]), pack2(shift, shift)));
            x[j] = y.x;
            x[j + 1] = y.y;
        }
        if (k > 0 && __any_sync(0xffffffffu, g != 1.0f)) {
            tc_fence_after();
            const uint32_t o_addr = sm.tmem + lanes + kTile;
#pragma unroll 1
            for (int d = 0; d < D; d += 16) {
                float o[16];
                tc_ld16(o_addr + d, o);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] *= g;
                tc_st16(o_addr + d, reinterpret_cast<const uint32_t*>(o));
            }
            tc_wait_st();
        }
    }
    // A group's weights, its part of the sum, and the pieces: 16 bytes of each, swizzled. The tile's
    // sum comes first: a thousand equal tiles added up group by group are off by 3e-4, tile by tile by 3e-5 at most.
    float sum = 0.0f;
#pragma unroll
    for (int g = 0; g < kTile; g += 16) {
        const float inv = nums[(g) >> shift_page].inv;
        float* y = x + g;
        uint32_t p[8];
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) y[j + k] = ex2_approx(y[j + k]);
            s2 = add2(s2, add2(pack2(y[j], y[j + 1]), pack2(y[j + 2], y[j + 3])));
            p[j / 2] = pack_f16(y[j], y[j + 1]);
            p[j / 2 + 1] = pack_f16(y[j + 2], y[j + 3]);
        }
        const float2 s = unpack2(s2);
        sum = fmaf(s.x + s.y, inv, sum);
        uint8_t* to = &sm.w[g / 64][row * kTile];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            *reinterpret_cast<uint4*>(to + (((g % 64) / 8 + i) ^ (row & 7)) * 16) =
                make_uint4(p[4 * i], p[4 * i + 1], p[4 * i + 2], p[4 * i + 3]);
    }
    r.l += sum;
    return ok;
}

// This thread's token of V's tile as fp16 (exact). Slots past the last token become zeros, whatever they
// hold: 0 x NaN is NaN.
template <int D>
__device__ __forceinline__ void widen(Smem<D>& sm, uint8_t* slot, int token, bool live)
{
    uint4 c[D / 16];
    const uint8_t* raw = slot + token * D;
    const int swz = D == 128 ? token & 7 : (token >> 1) & 3;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        c[i] = *reinterpret_cast<const uint4*>(raw + ((i ^ swz) << 4));
        if (!live) c[i] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
        const uint32_t in[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
        uint32_t o[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * k]) : "h"(static_cast<uint16_t>(in[k] & 0xffffu)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(o[2 * k + 1]) : "h"(static_cast<uint16_t>(in[k] >> 16)));
        }
        uint8_t* to = (D == 128 && i < 4 ? slot : sm.wide) + token * 128;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(to + (((2 * i + k) ^ token) & 7) * 16) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
    }
}

// A unit's queries as two pieces in shared memory, and their rows' exponents: eight (four) lanes per
// row with 16 elements each. Rows past the unit's are zeros. All loads come first.
template <int D>
__device__ __forceinline__ void load_queries(const AttendCall& A, Smem<D>& sm, const Walk<kRows>& wk, int rows)
{
    constexpr int S = D / 16, kStep = kSoft / S;             // lanes per row, rows per pass
    const int seg = threadIdx.x & (S - 1);
    const bool vec = ((reinterpret_cast<uintptr_t>(A.q) | static_cast<uintptr_t>(A.q_stride * 2)) & 15u) == 0;
    auto fetch = [&](int row, uint4* v) {
        const int flat = wk.qt * kRows + min(row, rows - 1);
        const int i = flat / A.group;
        const uint16_t* at = static_cast<const uint16_t*>(A.q) + (wk.row0 + i) * A.q_stride +
                             static_cast<int64_t>(wk.h * A.group + flat - i * A.group) * D + seg * 16;
        if (vec) {
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
    };
    auto place = [&](int row, const uint4* v) {
        uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        uint32_t top2 = 0;                       // magnitudes' bits order like them, NaN above all
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (row >= rows) w[k] = 0;
            top2 = __vmaxu2(top2, w[k] & 0x7fff7fffu);
        }
        uint32_t top = max(top2 & 0xffffu, top2 >> 16);
#pragma unroll
        for (int off = 1; off < S; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
        const bool fine = top < 0x7f80u;
        const int e = fine ? scale_exponent(__uint_as_float(top << 16)) : 0;
        const float inv = exp2i(-e);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {            // through fp16: it holds a bf16's 8 bits, down to 2^-24
            uint16_t h0, h1, l0, l1;
            split2(bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv, &h0, &l0);
            split2(bf16_lo(w[2 * k + 1]) * inv, bf16_hi(w[2 * k + 1]) * inv, &h1, &l1);
            hi[k] = join16(h0, h1);
            lo[k] = join16(l0, l1);
        }
        const int chunk = seg ^ (D == 128 ? row & 7 : (row >> 1) & 3);
        *reinterpret_cast<uint4*>(&sm.q[0][row * D + chunk * 16]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(&sm.q[1][row * D + chunk * 16]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (seg == 0) sm.e[row] = static_cast<int8_t>(fine ? e : kNotFine);
    };
    constexpr int kPasses = kRows / kStep;
    uint4 v[kPasses][2];
    const int row = threadIdx.x / S;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) fetch(row + i * kStep, v[i]);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) place(row + i * kStep, v[i]);
}

// A finished piece: results or a part written. Out of line: the tiles' loop gets better registers
// (521 -> 508 us).
template <int D>
static __device__ __noinline__ void finish(const AttendCall& A, const Row& r, uint32_t o_addr, int row,
                                       const Walk<kRows>& wk, int part, const Workspace& ws)
{
    const int rows = wk.rows(A);
    const bool whole = wk.whole();
    const float l = r.l;
    const float m = -r.ref;             // reference - kUp, as the weights are
    const float g = !whole ? 1.0f : l == 0.0f ? 0.0f : __fdividef(1.0f, l);      // nothing seen: zeros
    const bool live = row < rows;
    const int flat = wk.qt * kRows + min(row, rows - 1);
    const int64_t prow = wk.row0 + flat / A.group;
    const int head = wk.h * A.group + flat % A.group;
    if (live) {
        if (!whole)
            ws.ml[part * kTile + row] = make_float2(l == 0.0f ? kNone : m, l);
        else if (A.lse != nullptr)
            A.lse[prow * A.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    uint16_t* out = static_cast<uint16_t*>(A.out) + prow * A.out_stride + static_cast<int64_t>(head) * D;
    float* po = ws.o + (static_cast<int64_t>(part) * kTile + row) * D;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
#pragma unroll 1
    for (int d = 0; d < D; d += 16) {
        float o[16];
        tc_ld16(o_addr + d, o);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) o[j] *= g;
        if (!live) continue;
        if (!whole) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                *reinterpret_cast<float4*>(po + d + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        } else if (vec) {
            *reinterpret_cast<uint4*>(out + d) = store16<DSPARK_BF16>(o);
            *reinterpret_cast<uint4*>(out + d + 8) = store16<DSPARK_BF16>(o + 8);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) store1<DSPARK_BF16>(out, d + j, o[j]);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
attend_wide_kernel(const __grid_constant__ AttendCall A, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map)
{
    extern __shared__ __align__(kSmemAlign) unsigned char raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    static_assert(sizeof(Smem<D>) <= kSmemTwo, "two CTAs per SM");
    constexpr int kSlots = Smem<D>::kSlots, kNums = Smem<D>::kNums;
    constexpr int kLoader = kSoft / 32, kIssuer = kLoader + 1;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Workspace ws = workspace_of(A.ws);
    if (!smem_aligned(A, ws, raw)) return;

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        mbar_init(smem_addr(&sm.s_full), 2);
        mbar_init(smem_addr(&sm.s_read), kSoft / 32);
        mbar_init(smem_addr(&sm.p_full), kSoft / 32);
        mbar_init(smem_addr(&sm.pv_done), 1);
        mbar_init(smem_addr(&sm.q_full), kSoft);
        sm.stalled = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;"
                     ::"r"(smem_addr(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        tc_fence_before();
    }
    pdl_wait_and_trigger();
    const int run = cut_line<kRows, kThreads>(A, sm.cut);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    volatile int* stalled = &sm.stalled;
    Walk<kRows> wk = sm.cut.walk;
    auto next_piece = [&]() -> bool {
        if (wk.last()) return false;
        wk.next(A);
        return true;
    };
    if (tid == 0) write_meta<kRows>(A, ws, wk, run);
    if (wk.n > 0) {
        if (warp == kLoader) {
            // ---- pages in ----
            const int per_tile = kTile / A.c.page;
            const uint32_t box = static_cast<uint32_t>(A.c.page) * D;
            const int beyond = A.c.n_pages * A.c.heads * A.c.page;     // a row past the tensor: zeros
            int it = 0;
            int bad = 0, issued = 0;
            bool ok = true;
            do {
                const int32_t* table = A.c.table + static_cast<int64_t>(wk.b) * A.c.width;
                const int total_blocks = (wk.len + wk.w + A.c.page - 1) / A.c.page;
                const int lo = wk.first_seen(A);
                // 32 blocks at a time, one per lane; the next 32 are fetched while these load
                const int first_block = wk.k0 * per_tile;
                int base = first_block;
                auto id_of = [&](int j) -> int {        // -1: dead, not there, or not a page
                    if (j >= total_blocks || (j + 1) * A.c.page <= lo) return -1;
                    const int id = j < A.c.width ? table[j] : -1;
                    if (id < 0 || id >= A.c.n_pages) { bad = 1; return -1; }
                    return id;
                };
                auto nums_of = [&](int id) -> float2 {
                    if (id < 0) return make_float2(0.0f, 0.0f);
                    const int64_t bh = static_cast<int64_t>(id) * A.c.heads + wk.h;
                    return make_float2(A.c.k_scale[bh], A.c.v_scale[bh]);
                };
                const int end_block = (wk.k0 + wk.n) * per_tile;
                int id = base + lane < end_block ? id_of(base + lane) : -1;
                float2 sc = nums_of(id);
                int next_id = -1;
                float2 next_sc = make_float2(0.0f, 0.0f);
                for (int k = 0; ok && k < wk.n; ++k, ++it) {
                    const int j0 = first_block + k * per_tile - base;   // this tile's first lane
                    if (j0 == 0 && base + 32 + lane < end_block) next_id = id_of(base + 32 + lane);
                    if (j0 == per_tile) next_sc = nums_of(next_id);
                    const int src = j0 + (lane & (per_tile - 1));
                    const int my_id = __shfl_sync(0xffffffffu, id, src);
                    const float ks = __shfl_sync(0xffffffffu, sc.x, src);
                    const float vs = __shfl_sync(0xffffffffu, sc.y, src);
                    const int block = base + src;
                    const bool there = lane < per_tile && block < total_blocks;
                    const int count = __popc(__ballot_sync(0xffffffffu, there));
                    const int row = my_id < 0 ? beyond : (my_id * A.c.heads + wk.h) * A.c.page;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int use = 2 * it + kv;
                        const int s = use % kSlots;
                        const uint32_t full = smem_addr(&sm.full[s]);
                        if (use >= kSlots)
                            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.empty[s]),
                                                                   ((use / kSlots) & 1) ^ 1, stalled));
                        if (!ok) break;
                        if (kv == 0 && lane < per_tile) {
                            BlockNums n;
                            n.ks = my_id < 0 ? 0.0f : ks;
                            n.bias = my_id < 0 ? -INFINITY : log2f(vs);
                            n.inv = my_id < 0 ? 0.0f : 1.0f / vs;
                            n.pad = 0.0f;
                            sm.nums[it % kNums][lane] = n;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(full, count * box);
                        __syncwarp();
                        if (there)
                            tma_load(smem_addr(sm.ring[s]) + lane * box, kv ? &v_map : &k_map, row, full);
                        issued = use + 1;
                    }
                    if (j0 + per_tile == 32) {
                        base += 32;
                        id = next_id;
                        sc = next_sc;
                        next_id = -1;
                    }
                }
            } while (ok && next_piece());
            if (bad) raise_status(A.status, DSPARK_STATUS_BAD_PAGE);
            // every started copy lands before the CTA may leave
            __syncwarp();
            for (int s = 0; s < kSlots && s < issued; ++s)
                drain(smem_addr(&sm.full[s]), ((issued - 1 - s) / kSlots) & 1, stalled);
        } else if (warp == kIssuer) {
            // ---- products: the warp runs as one, an elected lane issues ----
            const bool leader = elect_one();
            constexpr uint32_t kIdesc = (1u << 4) | (kTile / 16 << 24);
            constexpr uint32_t kIdescQK = kIdesc | (kTile / 8 << 17);
            constexpr uint32_t kIdescPV = kIdesc | (D / 8 << 17) | (1u << 16);   // fp16; V: dim contiguous
            const uint32_t s_addr = sm.tmem, o_addr = sm.tmem + kTile;
            const uint64_t ring0 = operand<D>(smem_addr(sm.ring[0])), q_op = operand<D>(smem_addr(sm.q[0]));
            const uint64_t w_op = operand<kTile>(smem_addr(sm.w[0]));
            // V in fp16: 64 elements at the ring's slot, the next 64 one slot on, which is `wide`
            static_assert(D == 64 || (Smem<D>::kSlots == 2 && Smem<D>::kSlot == kTile * 128), "V's slot is the last");
            const uint64_t v_op = operand<128>(smem_addr(D == 128 ? sm.ring[kSlots - 1] : sm.wide)) &
                                  ~(0x3fffull << 16) | (static_cast<uint64_t>(kTile * 128 / 16) << 16);
            constexpr uint32_t kStep = Smem<D>::kSlot / 16;
            int it = 0, piece = 0;
            bool ok = true;
            auto wait = [&](uint64_t& bar, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait(smem_addr(&bar), parity, stalled));
            };
            do {
                ok = wait(sm.q_full, piece & 1);
                // scores of tile k, then the sums of tile k - 1: it counts the tiles before k
#pragma unroll 1
                for (int k = 0; ok && k <= wk.n; ++k) {
                    if (k < wk.n) {
                        const int use = 2 * it, s = use % kSlots;
                        ok = wait(sm.full[s], (use / kSlots) & 1) && (k == 0 || wait(sm.s_read, (it - 1) & 1));
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
                            const uint64_t kb = ring0 + s * kStep;
#pragma unroll
                            for (int p = 0; p < 2; ++p)
#pragma unroll
                                for (int i = 0; i < D / 32; ++i)
                                    mma_ss(s_addr, q_op + p * kStep + 2 * i, kb + 2 * i, kIdescQK, p > 0 || i > 0);
                            tc_commit(smem_addr(&sm.s_full));
                            mbar_arrive(smem_addr(&sm.s_full));      // hands on the tile's numbers too
                            tc_commit(smem_addr(&sm.empty[s]));
                        }
                        __syncwarp();
                        ++it;
                    }
                    if (k > 0) {
                        const int last = k < wk.n ? it - 2 : it - 1;
                        const int use = 2 * last + 1, s = use % kSlots;
                        ok = wait(sm.p_full, last & 1) && wait(sm.full[s], (use / kSlots) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int i = 0; i < kTile / 16; ++i)
                                mma_ss_f16(o_addr, w_op + i / 4 * (kRows * kTile / 16) + i % 4 * 2,
                                           v_op + i * (16 * 128 / 16), kIdescPV, k > 1 || i > 0);
                            tc_commit(smem_addr(&sm.pv_done));
                            tc_commit(smem_addr(&sm.empty[s]));
                        }
                        __syncwarp();
                    }
                }
                ++piece;
            } while (ok && next_piece());
            // the last products' arrivals on the slots' barriers land before the CTA leaves
            if (it > 0) {
                const int use = 2 * (it - 1);
                drain(smem_addr(&sm.empty[use % kSlots]), (use / kSlots) & 1, stalled);
                drain(smem_addr(&sm.empty[(use + 1) % kSlots]), (use / kSlots) & 1, stalled);
            }
            __syncwarp();
        } else {
            // ---- softmax ----
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            const int row = tid;
            const int shift_page = __ffs(A.c.page) - 1;      // a power of two
            int it = 0, piece = 0;
            bool ok = true, more = true;
            if (tid == 0) sm.soft = wk;
            while (more) {
                soft_sync();
                {
                    const Walk<kRows> now = sm.soft;
                    const int rows = now.rows(A);
                    load_queries<D>(A, sm, now, rows);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    mbar_arrive(smem_addr(&sm.q_full));
                    const int i0 = now.qt * kRows / A.group;
                    sm.after[row] = static_cast<uint8_t>((now.qt * kRows + min(row, rows - 1)) / A.group - i0);
                    // tiles that every row sees whole need no mask: those within [hi lo, lo pos]
                    if (tid == 0) {
                        const int p0 = now.len + i0;
                        const int p1 = now.len + (now.qt * kRows + rows - 1) / A.group;
                        const int lo1 = A.window > 0 && p1 >= A.window ? p1 - A.window + 1 : 0;
                        sm.span.k0 = now.k0;
                        sm.span.n = now.n;
                        sm.span.lo = lo1;
                        sm.span.hi = p0;
                        sm.stored = now.len + now.w;
                    }
                }
                soft_sync();
                // a query that is not finite makes its row's factor, hence its results, NaN
                const int e = sm.e[row];
                Row r = {e == kNotFine ? __int_as_float(0x7fc00000) : A.scale * kLog2e * exp2i(e), 0.0f, 0.0f,
                         false};
                const int n = sm.span.n;
                // a warp whose wait gave up goes on to the piece's end, where the warps agree on it:
                // they share the barriers within
#pragma unroll 1
                for (int k = 0; k < n; ++k, ++it) {
                    ok = ok && mbar_wait(smem_addr(&sm.s_full), it & 1, stalled);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    ok = soften<D>(sm, r, lanes, row, sm.nums[it % kNums], shift_page, A.window, k, it, ok,
                                   stalled);
                    const int use = 2 * it + 1, s = use % kSlots;
                    ok = ok && mbar_wait(smem_addr(&sm.full[s]), (use / kSlots) & 1, stalled);
                    ok = __all_sync(0xffffffffu, ok);
                    if (ok) widen<D>(sm, sm.ring[s], row, (sm.span.k0 + k) * kTile + row < sm.stored);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    tc_fence_before();
                    __syncwarp();
                    if (ok && (tid & 31) == 0) mbar_arrive(smem_addr(&sm.p_full));
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.pv_done), (it - 1) & 1, stalled));
                const Walk<kRows> now = sm.soft;
                more = !now.last();
                if (soft_any(!ok)) break;
                if (tid == 0 && more) {
                    Walk<kRows> next = now;
                    next.next(A);
                    sm.soft = next;
                }
                tc_fence_after();
                finish<D>(A, r, sm.tmem + lanes + kTile, row, now, blockIdx.x * 2 + (piece > 0), ws);
                tc_fence_before();
                ++piece;
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

template <int D>
int launch(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    const size_t smem = sizeof(Smem<D>);
    // opt-in to large shared memory, once per device and host thread: threads share no state
    static thread_local int ready_device = -1;
    if (ready_device != device) {
        const cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel<D>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(DSPARK_ERR_CUDA, "dspark attend: %s", cudaGetErrorString(e));
        }
        ready_device = device;
    }
    if (!places_fit<kRows>(A))
        return fail(DSPARK_ERR_UNSUPPORTED, "dspark_attend: rows, heads and pages beyond what one call can cut");
    CUtensorMap k_map, v_map;
    int rc = encode_cache(&k_map, A.c.k, A.c);
    if (rc == DSPARK_OK) rc = encode_cache(&v_map, A.c.v, A.c);
    if (rc != DSPARK_OK) return rc;
    return launch_pdl("attend", attend_wide_kernel<D>, dim3(ctas), dim3(kThreads), smem, stream, A,
                      k_map, v_map);
}

}  // namespace

int launch_attend_wide(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    return A.c.dim == 128 ? launch<128>(A, ctas, device, stream) : launch<64>(A, ctas, device, stream);
}

}  // namespace dspark
