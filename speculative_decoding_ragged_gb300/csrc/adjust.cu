// adjust.cu — dspark_adjust: penalties for repeated tokens, biases and grammar masks on the packed
// rows' logits, between the target forward and verify.
//
// A row's adjustment differs from the next row's of its request by one draft, so a CTA takes one
// request and one slice of the vocabulary. It counts the request's tokens that fall into the slice
// once, in shared memory: a word per token (its uses, whether the prompt has it, its bias) and lists of
// the tokens met, one for each part of the slice. Its warps stream the slice of every row part by part,
// masked on the way, and a warp that has written a part then adjusts its listed tokens, a lane each.
// No sort, no hash, no order that matters: counts are integers, and of several biases for one token the
// last one counts.
//
// Bound by HBM: a row is read and written once. 256 windows of 1 to 8 rows over 151936 tokens in bf16: a copy
// takes 105 us, with drafts 106, with 150 biases a request too 111, with histories of 64 to 4096 tokens 123-126
// (5.6 TB/s). What the histories add is the adjusting of the listed tokens (a warp's instructions, whose
// logits come from L1 or L2) and the counting's round trips; the first of each array is therefore fetched
// before its length is known, and the counting runs under the warps' first loads. 320 rows under grammars:
// 28.8 us, 7 TB/s of the bytes counted with every logit read; parts that are forbidden whole are not (4.6 TB/s
// of what must move). In place, where what changes is written only, 77 and 24 us. One
// window of 8 rows: 5.0 us, launch and three dependent loads.
// Tried and slower for the 256 windows: four warps that count for eight that stream in a persistent grid
// (187 to 295 us: what waits for the counts then reads back what was written), the rows through shared
// memory by bulk copies (151), granules of 512 bytes dealt out to the slices, so that common tokens do not
// lie in one (150), all rows of a part adjusted together (162), a lane for each word of a bit array in place
// of lists (157, and 23 us for one window: common tokens lie together).
//
#include <cmath>
#include <type_traits>

#include "common.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                      // 16-byte units a thread has in flight
constexpr int64_t kFewCtas = 4;                // per SM, where requests are few
constexpr int kEach = 2;                       // listed tokens a lane adjusts at a time
constexpr int kMaxSlice = 7168, kMinSlice = 1024;
static_assert(kMinSlice % (32 * kUnits * 8) == 0 && kMaxSlice % kMinSlice == 0, "slices of whole parts");
// A token's word: uses in the answer, whether the prompt has it, whether it is a draft, 1 + the index of
// its bias.
constexpr uint32_t kUses = (1u << 19) - 1;
constexpr uint32_t kPrompt = 1u << 19;
constexpr uint32_t kDraft = 1u << 20;
constexpr int kBiasShift = 21;
static_assert(DSPARK_MAX_HISTORY + DSPARK_MAX_GAMMA <= static_cast<int>(kUses), "uses fit their bits");
static_assert(DSPARK_MAX_BIAS < (1 << (32 - kBiasShift)), "biases fit their bits");
// A word and a place in a list for each token of a slice.
constexpr size_t slice_bytes(int slice) { return slice * 6; }
static_assert(slice_bytes(kMaxSlice) <= 48 * 1024, "no opt-in to large shared memory");

struct AdjustCall {
    const void* x;
    int64_t xs;
    void* y;
    int64_t ys;
    int rows, V, B, gamma;
    const int32_t* cu;
    const int32_t* tokens;
    dspark_adjustments h;
    int slice, slices;
    int32_t* status;
};

struct Penalties {
    float rep, presence, frequency;
};

// A penalty as given, or the neutral one.
__device__ __forceinline__ float penalty_of(const float* p, int b, float neutral, bool positive, int* bits)
{
    if (p == nullptr) return neutral;
    const float x = p[b];
    if (isfinite(x) && (!positive || x > 0.0f)) return x;
    *bits |= DSPARK_STATUS_BAD_VALUE;
    return neutral;
}
__device__ __forceinline__ int clamped(int x, int hi, int* bits)
{
    if (x >= 0 && x <= hi) return x;
    *bits |= DSPARK_STATUS_BAD_LENGTH;
    return x < 0 ? 0 : hi;
}
// N bits from v on of a mask row, which ends with bit V - 1's word.
template <int N>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int v)
{
    const uint32_t lo = __ldg(row + (v >> 5)) >> (v & 31);
    return (v & 31) + N > 32 ? lo | __ldg(row + (v >> 5) + 1) << (32 - (v & 31)) : lo;
}

// Four tokens of a history at a 16-byte boundary, those outside [0, cap) left out.
struct Four {
    int v[4];
};
__device__ __forceinline__ Four four_of(const int32_t* history, int j, int cap)
{
    Four f;
    if (j >= 0 && j <= cap - 4) {
        const int4 x = *reinterpret_cast<const int4*>(history + j);
        f.v[0] = x.x, f.v[1] = x.y, f.v[2] = x.z, f.v[3] = x.w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[e] = static_cast<uint32_t>(j + e) < static_cast<uint32_t>(cap) ? history[j + e] : -1;
    }
    return f;
}

template <int DT>
struct Element;
template <>
struct Element<DSPARK_BF16> {
    typedef uint16_t type;
    static constexpr int kPer = 8;             // in 16 bytes
    static constexpr uint16_t kLowest = 0xff80;
    static __device__ __forceinline__ float up(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
    static __device__ __forceinline__ uint16_t down(float x)
    {
        uint16_t r;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(r) : "f"(x));
        return r;
    }
    // Word k of a unit whose elements are allowed by the bits of `allow`.
    static __device__ __forceinline__ uint32_t blend(uint32_t x, uint32_t allow, int k)
    {
        const uint32_t keep = (allow >> 2 * k & 1 ? 0xffffu : 0) | (allow >> (2 * k + 1) & 1 ? 0xffff0000u : 0);
        return (x & keep) | (0xff80ff80u & ~keep);
    }
};
template <>
struct Element<DSPARK_F32> {
    typedef uint32_t type;
    static constexpr int kPer = 4;
    static constexpr uint32_t kLowest = 0xff800000u;
    static __device__ __forceinline__ float up(uint32_t x) { return __uint_as_float(x); }
    static __device__ __forceinline__ uint32_t down(float x) { return __float_as_uint(x); }
    static __device__ __forceinline__ uint32_t blend(uint32_t x, uint32_t allow, int k)
    {
        return allow >> k & 1 ? x : kLowest;
    }
};
// COUNTING: the call has penalties or biases, MASKED: it has masks. A call without one of them is spared
// its code and registers: 256 windows without masks 143 -> 124 us, grammars alone 35 -> 29 us.
template <int DT, bool COUNTING, bool MASKED, bool IN_PLACE>
__global__ void __launch_bounds__(kThreads, COUNTING ? 4 : 5)
adjust_kernel(const __grid_constant__ AdjustCall A)
{
    typedef Element<DT> E;
    typedef typename E::type T;
    constexpr int N = E::kPer;
    constexpr uint32_t kAll = (1u << N) - 1;
    constexpr int kPart = 32 * kUnits * N;     // a warp's tokens at a time
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ int draft[DSPARK_MAX_GAMMA];    // the drafts' places in the slice
    __shared__ int listed[kMaxSlice / kPart];  // tokens met in each part of the slice
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / A.slices, slice = blockIdx.x - b * A.slices;
    const int v0 = slice * A.slice, nv = min(A.slice, A.V - v0);
    uint32_t* word = sm;                       // these only where something counts
    uint16_t* list = reinterpret_cast<uint16_t*>(word + A.slice);
    if constexpr (COUNTING) {
        for (int i = tid; i < A.slice / 4; i += kThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
        if (tid < kMaxSlice / kPart) listed[tid] = 0;
        __syncthreads();
    }
    pdl_wait_and_trigger();

    const dspark_adjustments& h = A.h;
    int bits = 0;
    // Everything the call says of the request, in one round of loads: the first of its history too.
    int r0 = static_cast<int64_t>(b) * A.gamma, w = A.gamma;
    if (A.cu != nullptr) {
        r0 = A.cu[b];
        const int r1 = A.cu[b + 1];
        w = r1 - r0;
        if (r0 < 0 || r1 < r0 || r1 > A.rows || w > A.gamma) { w = 0; bits |= DSPARK_STATUS_BAD_ROWS; }
    }
    float rep = 1.0f, presence = 0.0f, frequency = 0.0f;
    int n = 0, n_prompt = 0, n_bias = 0, shift = 0, my_draft = -1;
    const int32_t* history = nullptr;
    const float* bias = h.bias_values + static_cast<int64_t>(b) * h.bias_cap;
    Four first;
    int first_id = -1;
    float first_bias = 0.0f;
    if constexpr (COUNTING) {
        rep = penalty_of(h.repetition, b, 1.0f, true, &bits);
        presence = penalty_of(h.presence, b, 0.0f, false, &bits);
        frequency = penalty_of(h.frequency, b, 0.0f, false, &bits);
        if (A.tokens != nullptr && tid > 0 && tid < A.gamma) my_draft = A.tokens[static_cast<int64_t>(b) * A.gamma + tid];
        if (h.history != nullptr) {
            history = h.history + static_cast<int64_t>(b) * h.history_cap;
            shift = static_cast<int>(reinterpret_cast<uintptr_t>(history) / 4 & 3);
            first = four_of(history, 4 * tid - shift, h.history_cap);
            n = clamped(h.history_len[b], h.history_cap, &bits);
            if (h.prompt_len != nullptr) n_prompt = clamped(h.prompt_len[b], n, &bits);
        }
        if (h.bias_tokens != nullptr) {
            if (tid < h.bias_cap) {
                first_id = h.bias_tokens[static_cast<int64_t>(b) * h.bias_cap + tid];
                first_bias = bias[tid];
            }
            n_bias = clamped(h.bias_len[b], h.bias_cap, &bits);
        }
    }
    const bool penalties = rep != 1.0f || presence != 0.0f || frequency != 0.0f;
    const bool counts = COUNTING && w > 0 && (penalties || n_bias > 0);

    auto count = [&]() {
        // the place of token v in the slice, or -1
        auto place = [&](int v) -> int {
            if (static_cast<uint32_t>(v - v0) < static_cast<uint32_t>(nv)) return v - v0;
            if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(A.V)) bits |= DSPARK_STATUS_BAD_TOKEN;
            return -1;
        };
        // the one that finds a word empty lists its token
        auto meet = [&](int t, uint32_t before) {
            if (before == 0) list[t / kPart * kPart + atomicAdd(&listed[t / kPart], 1)] = static_cast<uint16_t>(t);
        };
        const int32_t* ids = h.bias_tokens + static_cast<int64_t>(b) * h.bias_cap;
        for (int j = tid; j < n_bias; j += kThreads) {
            const int t = place(j == tid ? first_id : ids[j]);
            if (t < 0) continue;
            if (!((j == tid ? first_bias : bias[j]) < INFINITY)) { bits |= DSPARK_STATUS_BAD_VALUE; continue; }      // -inf bans a token
            meet(t, atomicMax(&word[t], static_cast<uint32_t>(j + 1) << kBiasShift));
        }
        if (n_bias > 0) __syncthreads();       // the maximum is over biases alone
        if (tid < w) {
            const int t = penalties && tid > 0 ? place(my_draft) : -1;
            draft[tid] = t;
            if (t >= 0) meet(t, atomicOr(&word[t], kDraft));
        }
        Four now = first;
#pragma unroll 1
        for (int j = 4 * tid - shift; penalties && j < n; j += 4 * kThreads) {
            Four next = now;
            if (j + 4 * kThreads < n) next = four_of(history, j + 4 * kThreads, h.history_cap);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (static_cast<uint32_t>(j + e) >= static_cast<uint32_t>(n)) continue;
                const int t = place(now.v[e]);
                if (t >= 0) meet(t, j + e < n_prompt ? atomicOr(&word[t], kPrompt) : atomicAdd(&word[t], 1u));
            }
            now = next;
        }
        __syncthreads();
    };
    // The mask row of packed row r, or none.
    auto mask_of = [&](int r) -> const uint32_t* {
        if (!MASKED) return nullptr;
        const int m = h.mask_row != nullptr ? h.mask_row[r] : r;
        if (m >= 0 && m < h.mask_rows) return h.mask + m * h.mask_stride;
        if (m != -1) bits |= DSPARK_STATUS_BAD_ROWS;
        return nullptr;
    };
    // A warp takes kPart tokens of a row at a time; its part of the mask row is fetched one part ahead,
    // and the counting runs under its first loads.
    const int parts = IN_PLACE && !MASKED && !counts ? 0 : (nv + kPart - 1) / kPart;
    int i = 0, part = tid >> 5;
    const uint32_t* mask = nullptr;
    uint32_t ahead = 0;
    auto settle = [&]() {
        if (parts == 0) i = w;
        while (i < w && part >= parts) { part -= parts; ++i; }
        if (!MASKED || i >= w) return;
        mask = mask_of(r0 + i);
        const int v = part * kPart + lane * 32;
        ahead = mask != nullptr && v < min(nv, (part + 1) * kPart) ? __ldg(mask + (v0 + v) / 32) : 0;
    };
    settle();
    bool to_count = counts;
#pragma unroll 1
    while (i < w || to_count) {
        const bool some = i < w;
        const int r = r0 + i, p0 = part * kPart, now_i = i, now_part = part;
        const uint32_t* row_mask = MASKED ? mask : nullptr;
        const uint32_t mine = ahead;           // word `lane` of the part's mask
        const T* x = static_cast<const T*>(A.x) + r * A.xs + v0;
        T* y = static_cast<T*>(A.y) + r * A.ys + v0;
        const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ay = reinterpret_cast<uintptr_t>(y);
        // the common case: a whole part on 16-byte boundaries
        const bool plain = some && ((ax | ay) & 15) == 0 && p0 + kPart <= nv;
        uint32_t allow[kUnits];
        uint4 e[kUnits];
        if (plain) {
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                allow[k] = kAll;
                if (MASKED && row_mask != nullptr)
                    allow[k] = __shfl_sync(0xffffffffu, mine, (k * 32 + lane) * N / 32) >> (lane * N & 31) & kAll;
            }
#pragma unroll
            for (int k = 0; k < kUnits; ++k)
                if (allow[k] != 0 && !(IN_PLACE && allow[k] == kAll))
                    e[k] = *(reinterpret_cast<const uint4*>(x + p0) + k * 32 + lane);
        }
        if (COUNTING && to_count) {
            count();
            to_count = false;
        }
        if (!some) continue;
        part += kThreads / 32;
        settle();

        // Elements before the first 16-byte boundary and after the last one go one at a time, and so
        // do all where rows and results lie differently to the boundaries.
        int head = p0, tail = p0 + kPart;
        if (!plain) {
            const int end = min(nv, tail);
            const bool alike = ((ax ^ ay) & 15) == 0;
            head = alike ? min(end, p0 + static_cast<int>(((16 - (ay & 15)) & 15) / sizeof(T))) : end;
            tail = head + (end - head) / N * N;
            auto single = [&](int t) {
                const bool allowed = !MASKED || row_mask == nullptr || (mask_bits<1>(row_mask, v0 + t) & 1);
                if (!allowed) y[t] = E::kLowest;
                else if (!IN_PLACE) y[t] = x[t];
            };
            for (int t = p0 + lane; t < head; t += 32) single(t);
            if (tail + lane < end) single(tail + lane);
#pragma unroll
            for (int k = 0; k < kUnits; ++k) {
                const int t = head + (k * 32 + lane) * N;
                allow[k] = t >= tail || !MASKED || row_mask == nullptr ? kAll : mask_bits<N>(row_mask, v0 + t) & kAll;
                if (t < tail && allow[k] != 0 && !(IN_PLACE && allow[k] == kAll))
                    e[k] = *reinterpret_cast<const uint4*>(x + t);
            }
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int t = head + (k * 32 + lane) * N;
            if (t >= tail || (IN_PLACE && allow[k] == kAll)) continue;
            if (allow[k] != kAll) {
                e[k].x = E::blend(e[k].x, allow[k], 0);
                e[k].y = E::blend(e[k].y, allow[k], 1);
                e[k].z = E::blend(e[k].z, allow[k], 2);
                e[k].w = E::blend(e[k].w, allow[k], 3);
            }
            *reinterpret_cast<uint4*>(y + t) = e[k];
        }
        if (!COUNTING || !counts) continue;
        // the part's listed tokens, over what the warp wrote: kEach a lane at a time, their loads at once
        const int m = listed[now_part];
        __syncwarp();
#pragma unroll 1
        for (int k0 = lane; k0 < m; k0 += 32 * kEach) {
            int t[kEach];
            uint32_t its[kEach], uses[kEach];
            bool apply[kEach];
            T old[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int k = k0 + 32 * e;
                t[e] = list[p0 + min(k, m - 1)];
                its[e] = word[t[e]] & ~kDraft;
                uses[e] = its[e] & kUses;
                // not: a token that is not allowed
                apply[e] = k < m && (!MASKED || row_mask == nullptr || (mask_bits<1>(row_mask, v0 + t[e]) & 1));
                old[e] = x[t[e]];
            }
            for (int j = 1; j <= now_i; ++j) {
                const int d = draft[j];
#pragma unroll
                for (int e = 0; e < kEach; ++e) uses[e] += d == t[e];
            }
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (!apply[e] || (its[e] | uses[e]) == 0) continue;        // nor: a later row's draft
                const uint32_t entry = its[e] >> kBiasShift;
                float z = E::up(old[e]);
                const float add = entry ? bias[entry - 1] : 0.0f;
                if ((its[e] & kPrompt) | uses[e]) z = z > 0.0f ? z / rep : z * rep;
                if (uses[e]) z -= fmaf(frequency, static_cast<float>(uses[e]), presence);
                if (entry) z = add == -INFINITY ? add : z + add;     // a ban holds for +inf and NaN too
                y[t[e]] = E::down(z);
            }
        }
    }
    // Masks that allow nothing: row i's is looked at by slice i % slices.
    if constexpr (MASKED) {
        const int words = (A.V + 31) / 32;
        const uint32_t last = A.V % 32 ? (1u << (A.V % 32)) - 1 : 0xffffffffu;     // bits of the last word
        for (int i = slice; i < w; i += A.slices) {
            const uint32_t* mask = mask_of(r0 + i);
            uint32_t any = 0;
            if (mask != nullptr) {
#pragma unroll 8
                for (int k = tid; k < words; k += kThreads) any |= mask[k] & (k == words - 1 ? last : 0xffffffffu);
            }
            if (!__syncthreads_or(any != 0) && mask != nullptr) bits |= DSPARK_STATUS_NO_TOKEN;
        }
    }
    raise_status(A.status, bits);
}

int launch_adjust(AdjustCall& A, int dtype, cudaStream_t stream)
{
    DeviceInfo dev;
    int rc = current_device(&dev);
    if (rc != DSPARK_OK) return rc;
    const bool counting = A.h.repetition != nullptr || A.h.presence != nullptr || A.h.frequency != nullptr ||
                          A.h.bias_tokens != nullptr;
    // Slices of one size, in steps of kMinSlice: as few as kMaxSlice allows, since each counts the whole
    // history (4096 tokens instead of 7168: 140 -> 161 us for the 256 windows), or, where requests are few, so
    // many that there are kFewCtas CTAs for each SM (33 requests over 32003 tokens: 20 us, 28 with two).
    const int64_t least = ceil_div(A.V, kMaxSlice), wanted = ceil_div(kFewCtas * dev.sm_count, A.B);
    A.slice = static_cast<int>(ceil_div(ceil_div(A.V, least > wanted ? least : wanted), kMinSlice) * kMinSlice);
    A.slices = static_cast<int>(ceil_div(A.V, A.slice));           // each holds a token
    const bool masked = A.h.mask != nullptr;
    auto pick = [&](auto dt, auto in_place) {
        constexpr int DT = decltype(dt)::value;
        constexpr bool P = decltype(in_place)::value;
        return counting ? (masked ? adjust_kernel<DT, true, true, P> : adjust_kernel<DT, true, false, P>)
                        : (masked ? adjust_kernel<DT, false, true, P> : adjust_kernel<DT, false, false, P>);
    };
    const std::integral_constant<int, DSPARK_BF16> bf16;
    const std::integral_constant<int, DSPARK_F32> f32;
    auto kernel = A.x == A.y ? (dtype == DSPARK_BF16 ? pick(bf16, std::true_type{}) : pick(f32, std::true_type{}))
                             : (dtype == DSPARK_BF16 ? pick(bf16, std::false_type{}) : pick(f32, std::false_type{}));
    return launch_pdl("adjust", kernel, dim3(static_cast<unsigned>(A.B) * A.slices), dim3(kThreads),
                      counting ? slice_bytes(A.slice) : 0, stream, A);
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace
}  // namespace dspark

using dspark::aligned;
using dspark::fail;

extern "C" int dspark_adjust(const void* logits, int64_t stride, void* out, int64_t out_stride,
                             dspark_dtype dtype, int rows, int V, const int32_t* cu_seqlens,
                             const int32_t* block_tokens, int B, int gamma,
                             const dspark_adjustments* how, int32_t* status, cudaStream_t stream)
{
    const char* fn = "dspark_adjust";
    if (how == nullptr) return fail(DSPARK_ERR_INVALID_ARG, "%s: how is required", fn);
    const dspark_adjustments& h = *how;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows < 0 || V < 1 || B < 0 || gamma < 1 || gamma > DSPARK_MAX_GAMMA)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: bad sizes rows=%d V=%d B=%d gamma=%d", fn, rows, V, B, gamma);
    if (B > DSPARK_MAX_BATCH || V > INT32_MAX / 4)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: B = %d above %d or V = %d too large", fn, B, DSPARK_MAX_BATCH, V);
    if (stride < V || out_stride < V)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: row strides %lld, %lld below V = %d", fn,
                    static_cast<long long>(stride), static_cast<long long>(out_stride), V);
    if (logits == out && logits != nullptr && stride != out_stride)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: in place needs one row stride, got %lld and %lld", fn,
                    static_cast<long long>(stride), static_cast<long long>(out_stride));
    if (cu_seqlens == nullptr && rows < static_cast<int64_t>(B) * gamma)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: without cu_seqlens rows = %d must hold B*gamma = %lld", fn, rows,
                    static_cast<long long>(B) * gamma);
    const bool penalties = h.repetition != nullptr || h.presence != nullptr || h.frequency != nullptr;
    if (h.history_cap < 0 || h.history_cap > DSPARK_MAX_HISTORY)
        return fail(h.history_cap < 0 ? DSPARK_ERR_INVALID_ARG : DSPARK_ERR_UNSUPPORTED,
                    "%s: history_cap = %d outside [0, %d]", fn, h.history_cap, DSPARK_MAX_HISTORY);
    if (h.history != nullptr && h.history_len == nullptr)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: a history needs history_len", fn);
    if (h.bias_tokens != nullptr && (h.bias_cap < 0 || h.bias_cap > DSPARK_MAX_BIAS))
        return fail(h.bias_cap < 0 ? DSPARK_ERR_INVALID_ARG : DSPARK_ERR_UNSUPPORTED,
                    "%s: bias_cap = %d outside [0, %d]", fn, h.bias_cap, DSPARK_MAX_BIAS);
    if (h.bias_tokens != nullptr && (h.bias_values == nullptr || h.bias_len == nullptr))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: biases need their values and bias_len", fn);
    if (h.mask != nullptr && (h.mask_rows < 0 || h.mask_stride < dspark::ceil_div(V, 32)))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: mask of %d rows of %lld words, %lld needed", fn, h.mask_rows,
                    static_cast<long long>(h.mask_stride), static_cast<long long>(dspark::ceil_div(V, 32)));
    if (h.mask != nullptr && h.mask_row == nullptr && h.mask_rows < rows)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: without mask_row the mask needs %d rows, got %d", fn, rows,
                    h.mask_rows);
    if (rows == 0 || B == 0) return DSPARK_OK;
    const uintptr_t e = dtype == DSPARK_BF16 ? 2 : 4;
    if (logits == nullptr || out == nullptr || !aligned(logits, e) || !aligned(out, e) ||
        (penalties && block_tokens == nullptr))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: logits and out (and for penalties block_tokens) are required, "
                    "aligned to their elements", fn);
    for (const void* p : {static_cast<const void*>(cu_seqlens), static_cast<const void*>(block_tokens),
                          static_cast<const void*>(h.history), static_cast<const void*>(h.history_len),
                          static_cast<const void*>(h.prompt_len), static_cast<const void*>(h.repetition),
                          static_cast<const void*>(h.presence), static_cast<const void*>(h.frequency),
                          static_cast<const void*>(h.bias_tokens), static_cast<const void*>(h.bias_values),
                          static_cast<const void*>(h.bias_len), static_cast<const void*>(h.mask),
                          static_cast<const void*>(h.mask_row)})
        if (!aligned(p, 4)) return fail(DSPARK_ERR_INVALID_ARG, "%s: arrays must be 4-byte aligned", fn);
    dspark::AdjustCall A = {logits, stride, out, out_stride, rows, V, B, gamma, cu_seqlens, block_tokens, h, 0, 0,
                            status};
    return dspark::launch_adjust(A, static_cast<int>(dtype), stream);
}
