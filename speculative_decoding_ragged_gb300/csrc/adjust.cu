// adjust.cu — dspark_adjust: penalties for repeated tokens, biases and grammar masks on the packed
// rows' logits, between the target forward and verify.
//
// A row's adjustment differs from the next row's of its request by one draft, so a CTA takes one
// request and one slice of the vocabulary: it counts the request's tokens that fall into the slice
// once, in shared memory, a word per token (its uses, whether the prompt has it, its bias), and
// streams the slice of every row. A bit per token says which words are not zero, so that untouched
// logits are copied without looking at words; the drafts before a row are counted where a touched
// token is met. No sort, no hash, no order that matters: counts are integers, and of several
// biases for one token the last one counts.
//
#include <cmath>

#include "common.cuh"

namespace dspark {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;                      // 16-byte units a thread has in flight
constexpr int kMaxSlice = 4096, kMinSlice = 1024;
// A token's word: uses in the answer, whether the prompt has it, 1 + the index of its bias.
constexpr uint32_t kUses = (1u << 20) - 1;
constexpr uint32_t kPrompt = 1u << 20;
constexpr int kBiasShift = 21;
static_assert(DSPARK_MAX_HISTORY + DSPARK_MAX_GAMMA <= static_cast<int>(kUses), "uses fit their bits");
static_assert((kMaxSlice + kMaxSlice / 32 + 4) * sizeof(uint32_t) <= 48 * 1024, "no opt-in to large shared memory");
static_assert(DSPARK_MAX_BIAS < (1 << (32 - kBiasShift)), "biases fit their bits");

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
// A bias that counts: -inf bans a token.
__device__ __forceinline__ bool bias_counts(float v) { return v < INFINITY; }

// Bits t .. t + 31 of a bit array in shared memory (one word past its end may be read).
__device__ __forceinline__ uint32_t bits_at(const uint32_t* words, int t)
{
    return __funnelshift_r(words[t >> 5], words[(t >> 5) + 1], t & 31);
}
// N bits from v on of a mask row, which ends with bit V - 1's word.
template <int N>
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* row, int v)
{
    const uint32_t lo = __ldg(row + (v >> 5)) >> (v & 31);
    return (v & 31) + N > 32 ? lo | __ldg(row + (v >> 5) + 1) << (32 - (v & 31)) : lo;
}

// What a CTA knows of its request.
struct Request {
    float rep, presence, frequency;
    const float* bias;
    const uint32_t* word;
    const int* draft;                          // slice-relative tokens of the drafts 1 .. i
};
__device__ __forceinline__ float adjusted(float x, int t, int i, const Request& q)
{
    const uint32_t word = q.word[t];
    uint32_t uses = word & kUses;
    for (int j = 1; j <= i; ++j) uses += q.draft[j] == t;
    if ((word & kPrompt) | uses) x = x > 0.0f ? x / q.rep : x * q.rep;
    if (uses) x -= fmaf(q.frequency, static_cast<float>(uses), q.presence);
    const uint32_t entry = word >> kBiasShift;
    if (entry) x += q.bias[entry - 1];
    return x;
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
// Element j of a unit of 16 bytes, which stays in registers, replaced.
template <int DT>
__device__ __forceinline__ void replace(uint4& q, int j, int t, int i, const Request& rq)
{
    typedef Element<DT> E;
    constexpr int kIn = E::kPer / 4;           // elements of a word
    const int k = j / kIn, shift = j % kIn * 16;
    const uint32_t w = k < 2 ? (k == 0 ? q.x : q.y) : (k == 2 ? q.z : q.w);
    const uint32_t y = E::down(adjusted(E::up(static_cast<typename E::type>(w >> shift)), t, i, rq));
    const uint32_t field = kIn == 1 ? 0xffffffffu : 0xffffu << shift;
    const uint32_t z = (w & ~field) | (y << shift & field);
    if (k == 0) q.x = z;
    if (k == 1) q.y = z;
    if (k == 2) q.z = z;
    if (k == 3) q.w = z;
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
adjust_kernel(const __grid_constant__ AdjustCall A, bool counting, bool in_place)
{
    typedef Element<DT> E;
    typedef typename E::type T;
    constexpr int N = E::kPer;
    constexpr uint32_t kAll = (1u << N) - 1;
    constexpr int kPart = 32 * kUnits * N;     // a warp's tokens at a time
    extern __shared__ __align__(16) uint32_t sm[];
    __shared__ int draft[DSPARK_MAX_GAMMA];
    const int tid = threadIdx.x, lane = tid & 31;
    const int b = blockIdx.x / A.slices, slice = blockIdx.x - b * A.slices;
    const int v0 = slice * A.slice, nv = min(A.slice, A.V - v0);
    uint32_t* word = sm;                       // both only where something counts
    uint32_t* touched = word + A.slice;        // tokens whose word is not zero, or that are drafts
    pdl_wait_and_trigger();

    const dspark_adjustments& h = A.h;
    int bits = 0;
    int r0 = static_cast<int64_t>(b) * A.gamma, w = A.gamma;
    if (A.cu != nullptr) {
        r0 = A.cu[b];
        const int r1 = A.cu[b + 1];
        w = r1 - r0;
        if (r0 < 0 || r1 < r0 || r1 > A.rows || w > A.gamma) { w = 0; bits |= DSPARK_STATUS_BAD_ROWS; }
    }
    Request q;
    q.word = word;
    q.draft = draft;
    bool counts = false;
    if (counting) {
        q.rep = penalty_of(h.repetition, b, 1.0f, true, &bits);
        q.presence = penalty_of(h.presence, b, 0.0f, false, &bits);
        q.frequency = penalty_of(h.frequency, b, 0.0f, false, &bits);
        const bool penalties = q.rep != 1.0f || q.presence != 0.0f || q.frequency != 0.0f;
        int n = 0, n_prompt = 0, n_bias = 0;
        if (penalties && h.history != nullptr) {
            n = clamped(h.history_len[b], h.history_cap, &bits);
            if (h.prompt_len != nullptr) n_prompt = clamped(h.prompt_len[b], n, &bits);
        }
        if (h.bias_tokens != nullptr) n_bias = clamped(h.bias_len[b], h.bias_cap, &bits);
        q.bias = h.bias_values + static_cast<int64_t>(b) * h.bias_cap;
        counts = w > 0 && (penalties || n_bias > 0);
        // where token v of this request has its word: -1 outside the slice
        auto place = [&](int v) -> int {
            if (static_cast<uint32_t>(v) >= static_cast<uint32_t>(A.V)) { bits |= DSPARK_STATUS_BAD_TOKEN; return -1; }
            return static_cast<uint32_t>(v - v0) < static_cast<uint32_t>(nv) ? v - v0 : -1;
        };
        auto touch = [&](int t) { atomicOr(&touched[t >> 5], 1u << (t & 31)); };
        if (counts) {
            for (int i = tid; i < (A.slice + A.slice / 32 + 4) / 4; i += kThreads)
                reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            const int32_t* ids = h.bias_tokens + static_cast<int64_t>(b) * h.bias_cap;
            for (int j = tid; j < n_bias; j += kThreads) {
                const int t = place(ids[j]);
                if (t < 0) continue;
                if (!bias_counts(q.bias[j])) { bits |= DSPARK_STATUS_BAD_VALUE; continue; }
                atomicMax(&word[t], static_cast<uint32_t>(j + 1) << kBiasShift);
                touch(t);
            }
            if (n_bias > 0) __syncthreads();   // the maximum is over biases alone
            if (tid < w) {
                const int t = penalties && tid > 0 ? place(A.tokens[static_cast<int64_t>(b) * A.gamma + tid]) : -1;
                draft[tid] = t;
                if (t >= 0) touch(t);
            }
            const int32_t* history = h.history + static_cast<int64_t>(b) * h.history_cap;
#pragma unroll 4
            for (int j = tid; j < n; j += kThreads) {
                const int t = place(history[j]);
                if (t < 0) continue;
                if (j < n_prompt) atomicOr(&word[t], kPrompt);
                else atomicAdd(&word[t], 1u);
                touch(t);
            }
            __syncthreads();
        }
    }
    // The mask row of packed row r, or none.
    auto mask_of = [&](int r) -> const uint32_t* {
        if (h.mask == nullptr) return nullptr;
        const int m = h.mask_row != nullptr ? h.mask_row[r] : r;
        if (m >= 0 && m < h.mask_rows) return h.mask + m * h.mask_stride;
        if (m != -1) bits |= DSPARK_STATUS_BAD_ROWS;
        return nullptr;
    };
    // A warp takes kPart tokens of a row at a time.
    const int parts = (nv + kPart - 1) / kPart;
    int i = 0, part = tid >> 5;
    while (part >= parts) { part -= parts; ++i; }
#pragma unroll 1
    while (i < w) {
        const int r = r0 + i;
        const uint32_t* mask = mask_of(r);
        const T* x = static_cast<const T*>(A.x) + r * A.xs + v0;
        T* y = static_cast<T*>(A.y) + r * A.ys + v0;
        // elements before the first 16-byte boundary and after the last one go one at a time, and so
        // do all where rows and results lie differently to the boundaries
        const uintptr_t ax = reinterpret_cast<uintptr_t>(x), ay = reinterpret_cast<uintptr_t>(y);
        const bool alike = ((ax ^ ay) & 15) == 0;
        const int head = alike ? min(nv, static_cast<int>(((16 - (ay & 15)) & 15) / sizeof(T))) : 0;
        const int units = alike ? (nv - head) / N : 0, tail = head + units * N;
        auto single = [&](int t) {
            const bool allowed = mask == nullptr || (mask_bits<1>(mask, v0 + t) & 1);
            if (!allowed) y[t] = E::kLowest;
            else if (counts && (touched[t >> 5] >> (t & 31) & 1)) y[t] = E::down(adjusted(E::up(x[t]), t, i, q));
            else if (!in_place) y[t] = x[t];
        };
        if (!alike) {
            const int end = min(nv, (part + 1) * kPart);
            for (int t = part * kPart + lane; t < end; t += 32) single(t);
        } else if (part == 0 && lane < nv - units * N) {
            single(lane < head ? lane : tail + lane - head);
        }
        const int u0 = part * (32 * kUnits) + lane;
        uint4 e[kUnits];
        uint32_t allow[kUnits], touch[kUnits];
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int u = u0 + k * 32;
            allow[k] = u < units && mask != nullptr ? mask_bits<N>(mask, v0 + head + u * N) & kAll : kAll;
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int u = u0 + k * 32, t = head + u * N;
            touch[k] = counts && u < units ? bits_at(touched, t) & allow[k] : 0;
            if (u < units && allow[k] != 0 && !(in_place && allow[k] == kAll && touch[k] == 0))
                e[k] = in_place ? *reinterpret_cast<const uint4*>(x + t) : ld_stream16(x + t);
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
            const int u = u0 + k * 32, t = head + u * N;
            if (u >= units || (in_place && allow[k] == kAll && touch[k] == 0)) continue;
#pragma unroll 1
            for (uint32_t m = touch[k]; m != 0; m &= m - 1) {
                const int j = __ffs(m) - 1;
                replace<DT>(e[k], j, t + j, i, q);
            }
            if (allow[k] != kAll) {
                e[k].x = E::blend(e[k].x, allow[k], 0);
                e[k].y = E::blend(e[k].y, allow[k], 1);
                e[k].z = E::blend(e[k].z, allow[k], 2);
                e[k].w = E::blend(e[k].w, allow[k], 3);
            }
            *reinterpret_cast<uint4*>(y + t) = e[k];
        }
        part += kThreads / 32;
        while (part >= parts) { part -= parts; ++i; }
    }
    // Masks that allow nothing: row i's is looked at by slice i % slices.
    if (h.mask != nullptr) {
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
    A.slice = kMaxSlice;
    while (A.slice > kMinSlice && A.B * ceil_div(A.V, A.slice) < 2ll * dev.sm_count) A.slice /= 2;
    A.slices = static_cast<int>(ceil_div(A.V, A.slice));
    const size_t smem = counting ? (A.slice + A.slice / 32 + 4) * sizeof(uint32_t) : 0;
    auto kernel = dtype == DSPARK_BF16 ? adjust_kernel<DSPARK_BF16> : adjust_kernel<DSPARK_F32>;
    return launch_pdl("adjust", kernel, dim3(static_cast<unsigned>(A.B) * A.slices), dim3(kThreads), smem, stream,
                      A, counting, A.x == A.y);
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
