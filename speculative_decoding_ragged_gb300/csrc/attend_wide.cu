// attend_wide.cu — dspark_attend on the tensor cores for prompts and large groups: units of up to
// 128 rows, one row per TMEM lane.
//
// A CTA: warp 4 loads pages with TMA (one box per page and K or V, swizzled), warp 5 issues the
// products, warps 0-3 do the softmax with one TMEM lane (row) per thread. A unit of at most 64 or
// 32 rows puts 2 or 4 copies of them in the lanes and each copy takes 1/2 or 1/4 of every tile's
// tokens, so all four warps share the softmax; the copies' products write their own lanes only
// (the instruction's lane mask) and join at the unit's end like parts.
// The weights overlay the scores in TMEM: 128 + dim columns, so two CTAs fit and one's softmax
// runs under the other's products.
#include "attend_mma.cuh"

namespace dspark {
namespace {

constexpr int kRows = 128;
constexpr int kSoftThreads = 128;
constexpr int kThreads = 192;

template <int D>
struct Smem {
    static constexpr int kSlot = kTile * D;              // one tile's K or V; 1024-byte aligned in order
    static constexpr int kSlots = D == 128 ? 4 : 8;      // K and V alternate
    uint8_t q[2][kTile * D];                             // the queries' two pieces
    uint8_t ring[kSlots][kSlot];
    BlockNums nums[kSlots / 2][kBlocks];
    float2 ml[kTile];
    uint64_t full[kSlots], empty[kSlots];
    uint64_t s_full, p_full, pv_done, q_full;
    Cut<kRows> cut;
    uint32_t tmem;
    int stalled;       // a wait gave up: every role leaves its loop
    int quit;          // the same, as the softmax warps agreed on it at a barrier
};

// ---- softmax -------------------------------------------------------------------------------
struct Row {
    float f;              // score factor: scale log2(e) 2^e of the row's pieces
    int lo, span;         // sees tokens [lo, lo + span]
    float m, l;
};

// One chunk's (32 tokens) exponents from its scores, in place.
template <bool MASK>
__device__ __forceinline__ void exponents(float* x, const Row& r, const BlockNums& n0,
                                          const BlockNums& n1, int token)
{
    const float f0 = r.f * n0.ks, f1 = r.f * n1.ks;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        x[j] = fmaf(x[j], f0, n0.bias);
        x[j + 16] = fmaf(x[j + 16], f1, n1.bias);
    }
    if (MASK) {
        const uint32_t at = static_cast<uint32_t>(token - r.lo), span = static_cast<uint32_t>(r.span);
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (at + j > span) x[j] = -INFINITY;
    }
}
__device__ __forceinline__ float max32(const float* x)
{
    float a = x[0], b = x[1], c = x[2], d = x[3];
#pragma unroll
    for (int j = 4; j < 32; j += 4) {
        a = fmaxf(a, x[j]);
        b = fmaxf(b, x[j + 1]);
        c = fmaxf(c, x[j + 2]);
        d = fmaxf(d, x[j + 3]);
    }
    return fmaxf(fmaxf(a, b), fmaxf(c, d));
}
// Exponents -> weights, their sum, and the pieces (8 words each) at p[0..7], p[8..15].
__device__ __forceinline__ void weights(float* x, Row& r, const BlockNums& n0, const BlockNums& n1,
                                        uint32_t* p)
{
    const float ref = r.m - kShift;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        x[j] = ex2_approx(x[j] - ref);
        s0 += x[j];
    }
#pragma unroll
    for (int j = 16; j < 32; ++j) {
        x[j] = ex2_approx(x[j] - ref);
        s1 += x[j];
    }
    r.l += s0 * n0.inv + s1 * n1.inv;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t h0, h1, l0, l1;
        split2(x[4 * k], x[4 * k + 1], &h0, &l0);
        split2(x[4 * k + 2], x[4 * k + 3], &h1, &l1);
        p[k] = h0 | (h1 << 16);
        p[8 + k] = l0 | (l1 << 16);
    }
}

// One tile for one row copy: scores in TMEM -> weights in TMEM. C copies: this thread's chunks
// are [q0, q0 + 4 / C).
template <int D, int C>
__device__ __forceinline__ void soften(Smem<D>& sm, Row& r, uint32_t lanes, const BlockNums* nums,
                                       int page, int token0, int q0, bool mask, bool first)
{
    constexpr int N = 4 / C;
    const uint32_t s_addr = sm.tmem + lanes;
    float x[32];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int q = q0 + i;
        tc_ld32(s_addr + 32 * q, x);
        tc_wait_ld();
        const BlockNums n0 = nums[32 * q / page], n1 = nums[(32 * q + 16) / page];
        if (mask) exponents<true>(x, r, n0, n1, token0 + 32 * q);
        else exponents<false>(x, r, n0, n1, 0);
        top = fmaxf(top, max32(x));
    }
    if (first) {
        r.m = fmaxf(top, kNone);
    } else {
        const bool grow = top > r.m + kLag;
        if (__any_sync(0xffffffffu, grow)) {
            float g = 1.0f;
            if (grow) {
                g = ex2_approx(r.m - top);
                r.m = top;
                r.l *= g;
            }
            const uint32_t o_addr = sm.tmem + lanes + kTile;
            float o[32];
#pragma unroll 1
            for (int d = 0; d < D; d += 32) {
                tc_ld32(o_addr + d, o);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] *= g;
                tc_st32(o_addr + d, o);
            }
            tc_wait_st();
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int q = q0 + i;
        const BlockNums n0 = nums[32 * q / page], n1 = nums[(32 * q + 16) / page];
        if (N > 1) {
            tc_ld32(s_addr + 32 * q, x);
            tc_wait_ld();
            if (mask) exponents<true>(x, r, n0, n1, token0 + 32 * q);
            else exponents<false>(x, r, n0, n1, 0);
        }
        uint32_t p[16];
        weights(x, r, n0, n1, p);
        tc_st16(s_addr + 16 * q, p);       // behind every chunk still to be read
    }
    tc_wait_st();
}

// This thread's row of the queries as two pieces in shared memory; returns the row's exponent.
template <int D>
__device__ __forceinline__ int load_query(const AttendCall& A, Smem<D>& sm, int t, bool live,
                                          int64_t row, int head)
{
    uint4 v[D / 8];
    const uint16_t* src = static_cast<const uint16_t*>(A.q) + row * A.q_stride +
                          static_cast<int64_t>(head) * D;
    if (!live) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = make_uint4(0, 0, 0, 0);
    } else if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = reinterpret_cast<const uint4*>(src)[i];
    } else {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = src[8 * i + 2 * k] | (static_cast<uint32_t>(src[8 * i + 2 * k + 1]) << 16);
            v[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    // the magnitudes' bits order like the magnitudes, NaN above all
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            top = max(top, w[k] & 0x7fffu);
            top = max(top, (w[k] >> 16) & 0x7fffu);
        }
    }
    const bool fine = top < 0x7f80u;
    const int e = fine ? scale_exponent(__uint_as_float(top << 16)) : 0;
    const float inv = exp2i(-e);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 u = v[2 * c + k / 2];
            const uint32_t w0 = (k & 1) ? u.z : u.x, w1 = (k & 1) ? u.w : u.y;
            const float y[4] = {bf16_lo(w0) * inv, bf16_hi(w0) * inv, bf16_lo(w1) * inv, bf16_hi(w1) * inv};
            float z[4];
            hi[k] = e4m3x4(y[0], y[1], y[2], y[3]);
            e4m3x4_to_f32(hi[k], z);
            lo[k] = e4m3x4(y[0] - z[0], y[1] - z[1], y[2] - z[2], y[3] - z[3]);
            if (!fine) hi[k] = 0x7f7f7f7fu;          // NaN: the row answers NaN
        }
        const int swz = D == 128 ? (c ^ (t & 7)) : (c ^ ((t >> 1) & 3));
        *reinterpret_cast<uint4*>(&sm.q[0][t * D + swz * 16]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(&sm.q[1][t * D + swz * 16]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return e;
}

// A finished piece: the copies' sums joined and written, as results or as a part.
template <int D>
__device__ __forceinline__ void finish(const AttendCall& A, Smem<D>& sm, const Row& r, uint32_t lanes,
                                       int t, int copies, const Walk<kRows>& wk, bool whole, int part,
                                       const Workspace& ws)
{
    const int RT = kTile / copies;
    const int row = t % RT, sub = t / RT;
    float m = r.m, l = r.l;
    if (copies > 1) {
        sm.ml[t] = make_float2(r.m, r.l);
        soft_sync();
        for (int c = 0; c < copies; ++c) m = fmaxf(m, sm.ml[row + c * RT].x);
        l = 0.0f;
        for (int c = 0; c < copies; ++c) {
            const float2 o = sm.ml[row + c * RT];
            l += o.y * ex2_approx(o.x - m);
        }
    }
    float g = copies > 1 ? ex2_approx(r.m - m) : 1.0f;
    if (whole) g = l == 0.0f ? 0.0f : g / l;       // a row that saw nothing: zeros
    const bool live = row < wk.rows(A);
    const int flat = wk.qt * kTile + row;
    const int64_t prow = wk.row0 + flat / A.group;
    const int head = wk.h * A.group + flat % A.group;
    if (live && sub == 0) {
        if (!whole)
            ws.ml[part * kTile + row] = make_float2(m - kShift, l);
        else if (A.lse != nullptr)
            A.lse[prow * A.q_heads + head] = l == 0.0f ? -INFINITY : (m - kShift + log2f(l)) * kLn2;
    }
    uint16_t* out = static_cast<uint16_t*>(A.out) + prow * A.out_stride + static_cast<int64_t>(head) * D;
    float* po = ws.o + (static_cast<int64_t>(part) * kTile + row) * D;
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    float4* stage = reinterpret_cast<float4*>(sm.q[0]);    // 128 x 32 floats: the queries are done
    const uint32_t o_addr = sm.tmem + lanes + kTile;
#pragma unroll 1
    for (int d0 = 0; d0 < D; d0 += 32) {
        float o[32];
        tc_ld32(o_addr + d0, o);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] *= g;
        int n = 32, d = d0;
        if (copies > 1) {
            n = 32 / copies;
            d = d0 + sub * n;
            soft_sync();                       // the stage's last readers are done
#pragma unroll
            for (int j = 0; j < 8; ++j)
                stage[t * 8 + (j ^ (t & 7))] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            soft_sync();
#pragma unroll
            for (int j = 0; j < 4; ++j) {      // 16 or 8 of the chunk's columns
                if (j * 4 >= n) break;
                float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (int c = 0; c < copies; ++c) {
                    const int from = row + c * RT;
                    const float4 v = stage[from * 8 + ((sub * (n / 4) + j) ^ (from & 7))];
                    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
                }
                o[4 * j] = s.x; o[4 * j + 1] = s.y; o[4 * j + 2] = s.z; o[4 * j + 3] = s.w;
            }
        }
        if (!live) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j * 8 >= n) break;
            const float* y = o + 8 * j;
            if (!whole) {
                *reinterpret_cast<float4*>(po + d + 8 * j) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(po + d + 8 * j + 4) = make_float4(y[4], y[5], y[6], y[7]);
            } else if (vec) {
                store8<DSPARK_BF16>(out + d + 8 * j, y);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) store1<DSPARK_BF16>(out, d + 8 * j + i, y[i]);
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
attend_wide_kernel(AttendCall A, const __grid_constant__ CUtensorMap k_map,
                  const __grid_constant__ CUtensorMap v_map)
{
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(
        raw + ((kSmemAlign - (smem_addr(raw) & (kSmemAlign - 1))) & (kSmemAlign - 1)));
    constexpr int kSlots = Smem<D>::kSlots;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Workspace ws = workspace_of(A.ws);

    if (tid == 0) {
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(smem_addr(&sm.full[s]), 1);
            mbar_init(smem_addr(&sm.empty[s]), 1);
        }
        mbar_init(smem_addr(&sm.s_full), 1);
        mbar_init(smem_addr(&sm.p_full), kSoftThreads);
        mbar_init(smem_addr(&sm.pv_done), 1);
        mbar_init(smem_addr(&sm.q_full), kSoftThreads);
        sm.stalled = 0;
        sm.quit = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5) {
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
        if (warp == 4) {
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
                    if (j0 == per_tile || (per_tile == 32 && j0 == 0)) next_sc = nums_of(next_id);
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
                        if (kv == 1 && lane < per_tile) {
                            BlockNums n;
                            n.ks = my_id < 0 ? 0.0f : ks;
                            n.bias = my_id < 0 ? -INFINITY : log2f(vs);
                            n.inv = my_id < 0 ? 0.0f : 1.0f / vs;
                            n.pad = 0.0f;
                            sm.nums[it % (kSlots / 2)][lane] = n;
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
        } else if (warp == 5) {
            // ---- products ----
            if (lane == 0) {
                constexpr uint32_t kIdesc = (1u << 4) | (kTile / 16 << 24);
                constexpr uint32_t kIdescQK = kIdesc | (kTile / 8 << 17);
                constexpr uint32_t kIdescPV = kIdesc | (D / 8 << 17) | (1u << 16);   // V: dim contiguous
                const uint32_t s_addr = sm.tmem, o_addr = sm.tmem + kTile;
                int it = 0, piece = 0;
                bool ok = true;
                do {
                    const int rows = wk.rows(A);
                    const int copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
                    ok = mbar_wait(smem_addr(&sm.q_full), piece & 1, stalled);
                    for (int k = 0; ok && k < wk.n; ++k, ++it) {
                        const int use = 2 * it;
                        const int sk = use % kSlots, sv = (use + 1) % kSlots;
                        const uint32_t round = (use / kSlots) & 1;
                        // the scores' columns hold the last tile's weights until its products end
                        ok = mbar_wait(smem_addr(&sm.full[sk]), round, stalled) &&
                             (it == 0 || mbar_wait(smem_addr(&sm.pv_done), (it - 1) & 1, stalled));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t kb = operand<D>(smem_addr(sm.ring[sk]));
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const uint64_t qa = operand<D>(smem_addr(sm.q[p]));
#pragma unroll
                            for (int s = 0; s < D / 32; ++s)
                                mma_ss(s_addr, qa + 2 * s, kb + 2 * s, kIdescQK, p > 0 || s > 0);
                        }
                        tc_commit(smem_addr(&sm.empty[sk]));
                        tc_commit(smem_addr(&sm.s_full));
                        ok = mbar_wait(smem_addr(&sm.p_full), it & 1, stalled) &&
                             mbar_wait(smem_addr(&sm.full[sv]), round, stalled);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vb = operand<D>(smem_addr(sm.ring[sv]));
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            // chunk s belongs to copy s * copies / 4
                            uint32_t off[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                off[i] = i * copies / 4 == s * copies / 4 ? 0u : 0xffffffffu;
                            const uint32_t fresh = k == 0 && (s * copies) % 4 == 0;
#pragma unroll
                            for (int p = 0; p < 2; ++p)
                                mma_ts(o_addr, s_addr + 16 * s + 8 * p, vb + s * (32 * D / 16), kIdescPV,
                                       p > 0 || !fresh, off[0], off[1], off[2], off[3]);
                        }
                        tc_commit(smem_addr(&sm.empty[sv]));
                        tc_commit(smem_addr(&sm.pv_done));
                    }
                    ++piece;
                } while (ok && next_piece());
                // the last products' arrivals on the slots' barriers land before the CTA leaves
                if (it > 0) {
                    const int use = 2 * (it - 1);
                    drain(smem_addr(&sm.empty[use % kSlots]), (use / kSlots) & 1, stalled);
                    drain(smem_addr(&sm.empty[(use + 1) % kSlots]), (use / kSlots) & 1, stalled);
                }
            }
            __syncwarp();
        } else {
            // ---- softmax ----
            const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
            int it = 0, piece = 0;
            bool ok = true;
            do {
                const int rows = wk.rows(A);
                const int copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
                const int RT = kTile / copies;
                const int row = min(tid % RT, rows - 1);
                const int flat = wk.qt * kTile + row;
                const int i = flat / A.group;
                const int e = load_query<D>(A, sm, tid, tid % RT < rows, wk.row0 + i,
                                            wk.h * A.group + flat - i * A.group);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_addr(&sm.q_full));
                Row r;
                r.f = A.scale * kLog2e * exp2i(e);
                const int pos = wk.len + i;
                r.lo = A.window > 0 && pos >= A.window ? pos - A.window + 1 : 0;
                r.span = pos - r.lo;
                r.m = kNone;
                r.l = 0.0f;
                // tiles that every row sees whole need no mask: those within [hi lo, lo pos]
                const int i0 = wk.qt * kTile / A.group;
                const int i1 = (wk.qt * kTile + rows - 1) / A.group;
                const int p0 = wk.len + i0, p1 = wk.len + i1;
                const int lo1 = A.window > 0 && p1 >= A.window ? p1 - A.window + 1 : 0;
                const int stored = wk.len + wk.w;
                for (int k = 0; k < wk.n; ++k, ++it) {
                    const int token0 = (wk.k0 + k) * kTile;
                    const int use = 2 * it + 1;
                    const int s = use % kSlots;
                    ok = mbar_wait(smem_addr(&sm.full[s]), (use / kSlots) & 1, stalled) &&
                         mbar_wait(smem_addr(&sm.s_full), it & 1, stalled);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const BlockNums* nums = sm.nums[it % (kSlots / 2)];
                    const bool mask = token0 + kTile - 1 > p0 || token0 < lo1;
                    const bool first = k == 0;
                    if (copies == 4)
                        soften<D, 4>(sm, r, lanes, nums, A.c.page, token0, warp, mask, first);
                    else if (copies == 2)
                        soften<D, 2>(sm, r, lanes, nums, A.c.page, token0, (warp >> 1) * 2, mask, first);
                    else
                        soften<D, 1>(sm, r, lanes, nums, A.c.page, token0, 0, mask, first);
                    tc_fence_before();
                    if (token0 + kTile > stored) {      // slots past the last token: 0 x NaN is NaN
                        if (token0 + tid >= stored) {
                            uint4* v = reinterpret_cast<uint4*>(&sm.ring[s][tid * D]);
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) v[c] = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    }
                    mbar_arrive(smem_addr(&sm.p_full));
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(&sm.pv_done), (it - 1) & 1, stalled));
                // a warp whose waits gave up leaves; agree on it before finish()'s barriers
                if (lane == 0 && !ok) *reinterpret_cast<volatile int*>(&sm.quit) = 1;
                soft_sync();
                if (*reinterpret_cast<volatile int*>(&sm.quit)) break;
                tc_fence_after();
                const bool whole = wk.whole();
                const int part = blockIdx.x * 2 + (piece > 0);
                finish<D>(A, sm, r, lanes, tid, copies, wk, whole, part, ws);
                ++piece;
                soft_sync();                   // the stage is free before the next queries enter it
            } while (next_piece());
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && sm.stalled) raise_status(A.status, DSPARK_STATUS_STALL);
    if (warp == 5)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(sm.tmem));
}

template <int D>
int launch(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    const size_t smem = sizeof(Smem<D>) + kSmemAlign;
    static bool ready[64] = {};               // opt-in to large shared memory, once per device
    if (!ready[device]) {
        const cudaError_t e = cudaFuncSetAttribute(attend_wide_kernel<D>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem));
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(DSPARK_ERR_CUDA, "dspark attend: %s", cudaGetErrorString(e));
        }
        ready[device] = true;
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
