// attend_mma.cuh — what the two tensor-core attention kernels share: the PTX they are written in,
// the cut of the work into equal runs, the parts left in the workspace.
//
// Mathematics. For a row r (one position, one query head) and tokens t with block scales ks, vs:
//   x_t = log2(e) scale q.K_t + log2 vs_t,   w_t = 2^(x_t - m),   O = sum_t w_t Vcode_t,
//   l = sum_t w_t / vs_t,   out = O / l,     lse = ln 2 (m + log2 l).
// Putting the value's scale into the exponent makes every product of the value side a plain
// product of codes, bounds w_t whatever the blocks' scales, and costs nothing: it is the
// addend of the multiply-add that scales the score.
//
// K stays in its 8 bits all the way into the tensor cores (kind::f8f6f4), and so does V where the rows
// are few. What is not 8-bit is split into pieces of 8 bits whose products add up in fp32. A bf16 query
// element has 8 significant bits, an e4m3 piece 4, so two pieces (over a power of two per row) hold it
// exactly down to 2^-17 of the row's largest. What counts for a weight is range, since one dominant
// token over a long context leaves the others small weights and much of the mass: it is three e5m2
// pieces (see split3) or, where there are rows enough to pay for widening V, one fp16 number. Compared
// with widening K too this moves half the shared-memory bytes; 8-bit products run at twice the 16-bit
// rate.
//
// Work. A unit is (request, cache head, up to R of its rows); its visible tokens come in tiles of
// 128. All tiles of all units form one line, which the persistent grid (two CTAs per SM) cuts
// into equal runs, so one long request and many short ones balance alike; every CTA computes the
// cut from cu_seqlens and lengths on the device. A unit cut by a run's end leaves (m, l, O) parts
// in the workspace that attend_join_kernel joins, in a fixed order: no atomics, the same bits
// every time.
#pragma once

#include <cuda.h>

#include "attend.cuh"
#include "rope.cuh"

namespace dspark {

constexpr int kTile = 128;                   // tokens per tile
constexpr int kMaxCtas = 304;                // parts the workspace holds: two CTAs on 152 SMs
constexpr int kBlocks = kTile / 16;          // most blocks in a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -1e30f;              // a row's reference before it has seen a token
// Weights are 2^(x - m + kUp), where the reference m may lag the row's true maximum by kBehind: at
// most 2^15.75, under fp16's largest and e5m2's. Less room for the lag rescales more often: 2.75 took
// 129 us where 6.5 took 115 (256 windows of 1 to 8 over 128 to 2048), 515 and 505 (two prompts' pieces).
constexpr float kUp = 9.25f;
constexpr float kBehind = 6.5f;
// What a weight may be off by is absolute under 2^-8 (see split3; fp16: under 2^-17), 2^-17 of the
// largest. So that a long tail of small weights after a dominant token keeps its bits, the reference
// also goes down, to a tile whose maximum lies kBelow under it: looked at after a tile that makes that
// likely, and every kLook tiles. The sums grow then: by at most 2^kDown in all over what the largest
// reference made them. It costs 2 us of 116 and 3 us of 507 in the two cases above.
constexpr float kBelow = 9.0f;
constexpr float kDown = 32.0f;
constexpr int kLook = 16;
__device__ __forceinline__ bool look_down(int k) { return k > 0 && (k & (kLook - 1)) == 0; }
constexpr long long kWaitCycles = 1ll << 31;
constexpr uint32_t kSmemAlign = 1024;        // the 128-byte swizzle's period
constexpr size_t kSmemTwo = 115712;          // of an SM's 228 KB, 1 KB reserved per CTA, for each of two CTAs

// What the join needs to know of the unit that a run's start cut.
struct RunMeta {
    int unit, end;      // the unit's places on the line
    int first;          // its first tile's
    int run;            // places per run
    int row0, rows;     // the request's first packed row; the unit's rows (position, head): 0 where
                        // the run starts with a unit's beginning, or holds no tile ...
    int flat0, head0;   // ... from this flat index on, first query head
};

struct Workspace {
    RunMeta* meta;      // [kMaxCtas]
    float2* ml;         // [kMaxCtas][2][kTile]
    float* o;           // [kMaxCtas][2][kTile][dim]
};
__host__ __device__ inline Workspace workspace_of(void* ws)
{
    char* p = static_cast<char*>(ws);
    Workspace w;
    w.meta = reinterpret_cast<RunMeta*>(p);
    w.ml = reinterpret_cast<float2*>(p + kMaxCtas * sizeof(RunMeta));
    w.o = reinterpret_cast<float*>(p + kMaxCtas * (sizeof(RunMeta) + 2 * kTile * sizeof(float2)));
    return w;
}

int encode_cache(CUtensorMap* map, void* codes, const dspark_cache& c);
int launch_attend_join(const AttendCall& A, int ctas, cudaStream_t stream);
int launch_attend_narrow(const AttendCall& A, int ctas, int device, cudaStream_t stream);
int launch_attend_wide(const AttendCall& A, int ctas, int device, cudaStream_t stream);

// ---- PTX -----------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
// The same without waiting at all (try_wait may suspend the thread for some microseconds).
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}
// Bounded wait for the phase of this parity. Once any thread of the CTA has given up (about a
// second), *stalled is set and every wait returns false, so that all roles leave their loops.
// The loop is out of line: the kernels run each part of their code a few times from a cold
// instruction cache, which costs about 16 cycles an instruction, so code size is time.
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, volatile int* stalled)
{
    const long long deadline = clock64() + kWaitCycles;
    while (!mbar_try(bar, parity)) {
        if (*stalled) return false;
        if (clock64() > deadline) { *stalled = 1; return false; }
    }
    return true;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* stalled)
{
    return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, stalled);
}
// The same bound, but not cut short by another wait's end: for what is in flight.
static __device__ __noinline__ void drain(uint32_t bar, uint32_t parity, volatile int* stalled)
{
    const long long deadline = clock64() + kWaitCycles;
    while (!mbar_try(bar, parity))
        if (clock64() > deadline) { *stalled = 1; return; }
}
// The tiles' swizzle needs shared memory that starts at its period, which the declaration asks for.
// Were it not so, the call would report a stall and write nothing.
__device__ __forceinline__ bool smem_aligned(const AttendCall& A, const Workspace& ws, const void* raw)
{
    const bool yes = (smem_addr(raw) & (kSmemAlign - 1)) == 0;
    if (!yes) {
        pdl_wait_and_trigger();
        if (threadIdx.x == 0) {
            ws.meta[blockIdx.x].rows = 0;        // nothing for the join
            raise_status(A.status, DSPARK_STATUS_STALL);
        }
    }
    return yes;
}
// True in one lane of the warp, which runs converged here.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " elect.sync _|p, 0xffffffff;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n" : "=r"(yes));
    return yes != 0;
}
// A page's box of the [rows, dim] tensor of codes -> shared memory.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(map), "r"(0), "r"(row), "r"(bar) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The barrier's arrival follows the completion of every product this thread issued before.
__device__ __forceinline__ void tc_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(bar) : "memory");
}
// D[tmem] (+)= A[smem] B[smem], 8-bit types; and fp16 by fp16
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma_ss_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
        "}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, float* x)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, "
        "%8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t addr, float* x)
{
    uint32_t* r = reinterpret_cast<uint32_t*>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]) : "memory");
}

// K-major and MN-major operands share the TMA swizzle: rows of BYTES (128, 64 or 32), groups of 8 rows.
template <int BYTES>
__device__ __forceinline__ uint64_t operand(uint32_t addr)
{
    constexpr uint64_t swizzle = BYTES == 128 ? 2 : BYTES == 64 ? 4 : 6;   // 128-, 64- or 32-byte
    return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (1ull << 16) |
           (static_cast<uint64_t>(8 * BYTES / 16) << 32) | (1ull << 46) | (swizzle << 61);
}

// A block's numbers in a tile: score factor, exponent addend, 1 / value scale.
struct __align__(16) BlockNums {
    float ks, bias, inv, pad;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Two query elements (under 448 in magnitude) in two e4m3 pieces each, through fp16, which holds a
// bf16's 8 bits down to 2^-17; the remainder is exact there.
__device__ __forceinline__ void split2(float a, float b, uint16_t* hi, uint16_t* lo)
{
    const uint32_t w = pack_f16(a, b);
    uint32_t back, rest;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(*hi) : "r"(w));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(*hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(rest) : "r"(w), "r"(back));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(*lo) : "r"(rest));
}
// Four weights in three e5m2 pieces each: p[i] holds the i-th pieces of a, b, c, d in order of bytes.
// An e5m2 number is the upper byte of an fp16 one. So the weight goes through fp16; the first piece is
// its upper byte, the second and third are those of what remains, rounded to nearest by adding half of
// the last place kept. Remainders are exact in fp16, of either sign after the second piece. From 2^-8
// up the three are within 2^-8.6 of the weight (3.7e-4 rms); below it the third piece ends at e5m2's
// smallest step, and they are off by 2^-16.8 at most. NaN stays NaN (first piece).
__device__ __forceinline__ void split3(float a, float b, float c, float d, uint32_t* p)
{
    uint32_t w0 = pack_f16(a, b), w1 = pack_f16(c, d), r0, r1;
    p[0] = __byte_perm(w0, w1, 0x7531);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r0) : "r"(w0), "r"(w0 & 0xff00ff00u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(w1), "r"(w1 & 0xff00ff00u));
    w0 = r0 + 0x00800080u;
    w1 = r1 + 0x00800080u;
    p[1] = __byte_perm(w0, w1, 0x7531);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r0) : "r"(r0), "r"(w0 & 0xff00ff00u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r1) : "r"(r1), "r"(w1 & 0xff00ff00u));
    p[2] = __byte_perm(r0 + 0x00800080u, r1 + 0x00800080u, 0x7531);
}
__device__ __forceinline__ uint32_t join16(uint16_t a, uint16_t b)
{
    uint32_t r;
    asm("mov.b32 %0, {%1, %2};" : "=r"(r) : "h"(a), "h"(b));
    return r;
}

// Packed fp32 pairs: one instruction for two.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// ---- the line of tiles ---------------------------------------------------------------------
// A unit of n tiles takes kUnitCost + n places on the line: starting and finishing a unit costs a
// CTA about as much as that many tiles, and runs of equal length should take equal time. Tile k is
// at place kUnitCost + k of its unit. Run i holds the places [i * run, (i + 1) * run). The host
// makes sure that a line's length fits an int (places_fit).
template <int R>
constexpr int kUnitCost = R < kTile ? 4 : 6;

struct Shape {                   // a unit's visible tiles [a, z]
    int a, z;
};
// The tiles that some row of a request's qt-th R rows sees and the page table reaches (one tile at
// least). The divisions by the group are spared where the unit holds the request's first or last
// rows: for decode and verify, always.
template <int R>
static __device__ __noinline__ Shape some_unit_tiles(const AttendCall& A, int w, int len, int qt)
{
    const int i0 = qt == 0 ? 0 : qt * R / A.group;
    const int i1 = static_cast<int64_t>(qt + 1) * R >= static_cast<int64_t>(w) * A.group
                       ? w - 1 : ((qt + 1) * R - 1) / A.group;
    const int p0 = len + i0;
    const int lo = A.window > 0 && p0 >= A.window ? p0 - A.window + 1 : 0;
    return {min(lo / kTile, A.last_tile), min((len + i1) / kTile, A.last_tile)};
}
template <int R>
__device__ __forceinline__ Shape unit_tiles(const AttendCall& A, int w, int len, int qt)
{
    if (static_cast<int64_t>(w) * A.group > R) return some_unit_tiles<R>(A, w, len, qt);
    const int lo = A.window > 0 && len >= A.window ? len - A.window + 1 : 0;      // the only unit
    return {min(lo / kTile, A.last_tile), min((len + w - 1) / kTile, A.last_tile)};
}
template <int R>
__device__ __forceinline__ int row_tiles(const AttendCall& A, int w)
{
    return static_cast<int>((static_cast<int64_t>(w) * A.group + R - 1) / R);
}
// The places that one head of a request takes on the line.
template <int R>
__device__ __forceinline__ int head_places(const AttendCall& A, int w, int len)
{
    int n = 0;
    const int nq = row_tiles<R>(A, w);
#pragma unroll 1
    for (int qt = 0; qt < nq; ++qt) {
        const Shape s = unit_tiles<R>(A, w, len, qt);
        n += s.z - s.a + 1 + kUnitCost<R>;
    }
    return n;
}
// Whether a call's line fits an int, whatever the lengths.
template <int R>
inline bool places_fit(const AttendCall& A)
{
    const int64_t units = (static_cast<int64_t>(A.rows) * A.q_heads) / R + static_cast<int64_t>(A.B) * A.c.heads;
    return units * (A.last_tile + 1 + kUnitCost<R>) <= INT32_MAX / 2;
}

// The units of one run in order.
template <int R>
struct Walk {
    int b, h, qt, nq;
    int row0, w, len;
    int a, z, k0, n;             // the unit's tiles [a, z]; this piece: n tiles from k0
    int unit;                    // the unit's first place on the line
    int stop;                    // the run's end on the line

    __device__ __forceinline__ void piece(const AttendCall& A, int from)
    {
        const Shape s = unit_tiles<R>(A, w, len, qt);
        a = s.a;
        z = s.z;
        const int first = unit + kUnitCost<R>;                          // the place of the first tile
        const int k = from > first ? from - first : 0;
        k0 = a + k;
        n = min(stop - first, z - a + 1) - k;                        // <= 0: nothing of it here
    }
    __device__ __forceinline__ int end() const { return unit + kUnitCost<R> + z - a + 1; }
    __device__ __forceinline__ bool last() const { return stop - end() <= kUnitCost<R>; }
    // The next unit of the run; only if !last().
    __device__ __forceinline__ void next(const AttendCall& A)
    {
        unit = end();
        if (++qt == nq) {
            qt = 0;
            if (++h == A.c.heads) {
                h = 0;
                int bits = 0;
#pragma unroll 1
                do {             // there is one with rows before the run's end
                    ++b;
                    request_rows(A, b, &row0, &w, &len, &bits);
                } while (w <= 0 && b + 1 < A.B);
                nq = row_tiles<R>(A, w);
            }
        }
        piece(A, unit);
    }
    __device__ __forceinline__ int rows(const AttendCall& A) const
    {
        return static_cast<int>(min(static_cast<int64_t>(R),
                                    static_cast<int64_t>(w) * A.group - static_cast<int64_t>(qt) * R));
    }
    __device__ __forceinline__ bool whole() const { return k0 == a && n == z - a + 1; }
    // The first token that some row of the unit sees.
    __device__ __forceinline__ int first_seen(const AttendCall& A) const
    {
        const int p0 = len + (qt == 0 ? 0 : qt * R / A.group);
        return A.window > 0 && p0 >= A.window ? p0 - A.window + 1 : 0;
    }
};

// The cut, by a whole CTA of NT threads: a group of threads counts the places of a stretch of
// requests, a scan over the groups gives the total and the stretch that holds the run's first
// place; that group finds the walk's start (n <= 0: the run holds no tile). The caller synchronises
// before the walk is read. Returns the places per run.
// A group is one thread where units are small: their requests have few units each, and the code is
// short. Where units are prompts' 128 rows, a few requests can have hundreds each: a group is then
// up to a warp, whose lanes take a request's units in turn (two prompts of 2000 rows and 32 heads:
// 66,600 cycles with single threads).
template <int R>
struct Cut {
    int scan[32];
    Walk<R> walk;
};
// A group: its lane, size and lanes' mask.
struct Group {
    int g, size;
    uint32_t mask;
    template <class T>
    __device__ __forceinline__ T from(T x, int lane_of) const { return __shfl_sync(mask, x, lane_of, size); }
};
template <int R>
__device__ __forceinline__ int group_places(const AttendCall& A, int w, int len, const Group& gr)
{
    if constexpr (R < kTile) return head_places<R>(A, w, len);
    int n = 0;
    const int nq = row_tiles<R>(A, w);
#pragma unroll 1
    for (int qt = gr.g; qt < nq; qt += gr.size) {
        const Shape s = unit_tiles<R>(A, w, len, qt);
        n += s.z - s.a + 1 + kUnitCost<R>;
    }
    for (int d = 1; d < gr.size; d <<= 1) n += __shfl_xor_sync(gr.mask, n, d);
    return n;
}
// By one group: the run [t0, t1) starts `off` places into the requests from b on. `k` holds request
// b already, and `per_head` its places per head.
template <int R>
__device__ __forceinline__ void find_start(const AttendCall& A, Walk<R>& k, int per_head, int off, int t0, int t1,
                                           const Group& gr)
{
    int bits = 0;
#pragma unroll 1
    while (off >= per_head * A.c.heads) {        // only where a group counts several requests
        off -= per_head * A.c.heads;
        ++k.b;
        request_rows(A, k.b, &k.row0, &k.w, &k.len, &bits);
        per_head = group_places<R>(A, k.w, k.len, gr);
    }
    k.h = static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(per_head));
    off -= k.h * per_head;
    k.nq = row_tiles<R>(A, k.w);
    k.stop = t1;
    k.qt = 0;
    k.unit = t0 - off;
    if constexpr (R < kTile) {
        k.piece(A, t0);
#pragma unroll 1
        while (k.end() <= t0) {                  // several units of rows: the one that holds t0
            ++k.qt;
            k.unit = k.end();
            k.piece(A, t0);
        }
    } else {
#pragma unroll 1
        for (;; k.qt += gr.size) {               // the group's units at once: off < per_head ends it
            const int qt = k.qt + gr.g;
            int n = 0;
            if (qt < k.nq) {
                const Shape s = unit_tiles<R>(A, k.w, k.len, qt);
                n = s.z - s.a + 1 + kUnitCost<R>;
            }
            int upto = n;
            for (int d = 1; d < gr.size; d <<= 1) {
                const int y = __shfl_up_sync(gr.mask, upto, d, gr.size);
                if (gr.g >= d) upto += y;
            }
            const uint32_t past = __ballot_sync(gr.mask, off < upto) & gr.mask;
            if (past || k.qt + gr.size >= k.nq) {
                const int at = past ? (__ffs(past) - 1) & (gr.size - 1) : 0;
                k.unit += gr.from(upto - n, at);
                k.qt += at;
                break;
            }
            const int all = gr.from(upto, gr.size - 1);
            off -= all;
            k.unit += all;
        }
        k.piece(A, t0);
    }
}
template <int R, int NT>
__device__ __forceinline__ int cut_line(const AttendCall& A, Cut<R>& cut)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int bits = 0;
    Group gr = {0, 1, 1u << lane};
    if constexpr (R >= kTile) {
        while (gr.size < 32 && static_cast<int64_t>(2 * gr.size) * A.B <= NT) gr.size *= 2;
        gr.g = lane & (gr.size - 1);
        gr.mask = (gr.size == 32 ? 0xffffffffu : (1u << gr.size) - 1) << (lane - gr.g);
    }
    const int groups = NT / gr.size;
    const int per = (A.B + groups - 1) / groups;
    const int b0 = min(tid / gr.size * per, A.B), b1 = min(b0 + per, A.B);
    int mine = 0, per_head = 1;
    Walk<R> k;
    if (tid == 0) cut.walk.n = 0;
#pragma unroll 1
    for (int b = b1 - 1; b >= b0; --b) {         // downwards: the walk is left at the first one
        k.b = b;
        request_rows(A, b, &k.row0, &k.w, &k.len, &bits);
        per_head = group_places<R>(A, k.w, k.len, gr);
        mine += gr.g == 0 ? per_head * A.c.heads : 0;
    }
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 31) cut.scan[warp] = upto;
    __syncthreads();
    int sums = lane < NT / 32 ? cut.scan[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sums, d);
        if (lane >= d) sums += y;
    }
    const int total = __shfl_sync(0xffffffffu, sums, NT / 32 - 1);
    const int before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
    int from = (warp > 0 ? before : 0) + upto - mine;
    const int run = static_cast<int>((static_cast<uint32_t>(total) + gridDim.x - 1) / gridDim.x);
    const int t0 = min(static_cast<int>(blockIdx.x) * run, total), t1 = min(t0 + run, total);
    if constexpr (R >= kTile) {
        mine = gr.from(mine, 0);
        from = gr.from(from, 0);
    }
    if (t0 < t1 && t0 >= from && t0 < from + mine) {
        find_start<R>(A, k, per_head, t0 - from, t0, t1, gr);
        if (gr.g == 0) cut.walk = k;
    }
    if (blockIdx.x == 0 && bits) raise_status(A.status, bits);
    return run;
}
// The run's entry for the join, by one thread.
template <int R>
__device__ __forceinline__ void write_meta(const AttendCall& A, const Workspace& ws, const Walk<R>& k, int run)
{
    RunMeta m;
    m.unit = k.unit;
    m.end = k.end();
    m.first = k.unit + kUnitCost<R>;
    m.run = run;
    m.row0 = k.row0;
    m.rows = k.n > 0 && k.k0 > k.a ? k.rows(A) : 0;
    m.flat0 = k.qt * R;
    m.head0 = k.h * A.group;
    ws.meta[blockIdx.x] = m;
}

}  // namespace dspark
