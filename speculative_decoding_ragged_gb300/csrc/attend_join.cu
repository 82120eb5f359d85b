// attend_join.cu — the second kernel of dspark_attend on the tensor cores: joins the parts of the
// units that a run's end cut; and the host side that both first kernels share.
#include "attend_mma.cuh"

namespace dspark {
namespace {

// Joins the parts of each cut unit: the runs that a unit's places cross, but the first, share its
// rows (a unit cut once is joined by one CTA, one cut 37 times by 37). A warp takes a row, or four
// where the parts are few: its lanes read the parts' references and sums, dim / 4 lanes add up the
// parts, up to 16 loads in flight. Prompts' units have 128 rows and mostly two parts, so that a warp's
// time is its rows' round trips: with a row at a time, its references read before its parts, two
// prompts' pieces took 37 us, now 12.
constexpr int kJoinWarps = 8;
constexpr int kFewParts = 4, kFewRows = 4;

// A unit's row: where its result goes, and (kPrefix) what it is joined with.
struct JoinRow {
    int64_t prow, at;
    int head;
    float own_lse;
    float4 own;
};
template <int D, int SEE>
__device__ __forceinline__ JoinRow join_row(const AttendCall& A, const RunMeta& m, int row, int lane)
{
    JoinRow r;
    const int flat = m.flat0 + row;
    r.prow = m.row0 + flat / A.group;
    r.head = m.head0 + flat % A.group;
    r.at = r.prow * A.q_heads + r.head;
    if constexpr (SEE == kPrefix) {
        r.own_lse = A.part_lse[r.at];
        r.own = lane * 4 < D ? *reinterpret_cast<const float4*>(A.part + r.at * D + lane * 4)
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    return r;
}
// Its parts added up: written out.
template <int D, int SEE>
__device__ __forceinline__ void put_row(const AttendCall& A, const JoinRow& r, bool partial, int lane, float top,
                                        float sum, float4 acc)
{
    float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    float lse = sum == 0.0f ? -INFINITY : top + log2f(sum);
    if (SEE == kSuffix && partial) {
        if (lane * 4 < D)
            *reinterpret_cast<float4*>(A.part + r.at * D + lane * 4) =
                make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
        if (lane == 0) A.part_lse[r.at] = lse;
        return;
    }
    if constexpr (SEE == kPrefix) {
        if (!is_part(r.own_lse)) return;                 // none of this call's rows
        const Shares sh = shares_of(lse, r.own_lse);
        inv *= sh.s;
        lse = sh.lse;
        acc = make_float4(fmaf(acc.x, inv, sh.p * r.own.x), fmaf(acc.y, inv, sh.p * r.own.y),
                          fmaf(acc.z, inv, sh.p * r.own.z), fmaf(acc.w, inv, sh.p * r.own.w));
        inv = 1.0f;
    }
    if (lane * 4 < D) {
        uint16_t* out = static_cast<uint16_t*>(A.out) + r.prow * A.out_stride +
                        static_cast<int64_t>(r.head) * D + lane * 4;
        const uint32_t a = pack_bf16(acc.x * inv, acc.y * inv), b = pack_bf16(acc.z * inv, acc.w * inv);
        out[0] = static_cast<uint16_t>(a);
        out[1] = static_cast<uint16_t>(a >> 16);
        out[2] = static_cast<uint16_t>(b);
        out[3] = static_cast<uint16_t>(b >> 16);
    }
    if (lane == 0 && A.lse != nullptr) A.lse[r.at] = lse * kLn2;
}
__device__ __forceinline__ void add_part(float4& acc, float f, const float4& o)
{
    acc.x = fmaf(f, o.x, acc.x);
    acc.y = fmaf(f, o.y, acc.y);
    acc.z = fmaf(f, o.z, acc.z);
    acc.w = fmaf(f, o.w, acc.w);
}

template <int D, int SEE>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) attend_join_kernel(AttendCall A)
{
    pdl_wait_and_trigger();
    const Workspace ws = workspace_of(A.ws);
    RunMeta m = ws.meta[blockIdx.x];
    if (m.rows == 0) return;
    const bool partial = SEE == kSuffix && (m.rows & kPartial) != 0;
    if constexpr (SEE == kSuffix) m.rows &= ~kPartial;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = m.first / m.run;                          // the run of the unit's first tile
    const int c1 = (m.end + m.run - 1) / m.run;              // one past the run of its last
    // in the first run an earlier unit's piece may come before
    const int part0 = 2 * c0 + (c0 * m.run < m.unit ? 1 : 0);
    const int shares = c1 - c0 - 1, share = static_cast<int>(blockIdx.x) - c0 - 1;
    const int step = shares * kJoinWarps;
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto slot = [&](int c, int row) -> int64_t { return static_cast<int64_t>(c == c0 ? part0 : 2 * c) * kTile + row; };
    if (c1 - c0 <= kFewParts) {
        constexpr int kLanes = 32 / kFewRows;
#pragma unroll 1
        for (int row0 = share * kJoinWarps + warp; row0 < m.rows; row0 += kFewRows * step) {
            // lane kLanes j + k: row j's part k
            const int mine = row0 + lane / kLanes * step, c = c0 + lane % kLanes;
            float2 ml = make_float2(kNone, 0.0f);
            if (mine < m.rows && c < c1) ml = ws.ml[slot(c, mine)];
            JoinRow r[kFewRows];
            float4 o[kFewRows][kFewParts];
#pragma unroll
            for (int j = 0; j < kFewRows; ++j) {
                const int row = min(row0 + j * step, m.rows - 1);
                r[j] = join_row<D, SEE>(A, m, row, lane);
#pragma unroll
                for (int k = 0; k < kFewParts; ++k)
                    o[j][k] = c0 + k < c1 && lane * 4 < D
                                  ? *reinterpret_cast<const float4*>(ws.o + slot(c0 + k, row) * D + lane * 4) : zero;
            }
            float top = ml.x;
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float f = c < c1 ? exp2f(ml.x - top) : 0.0f;
            float sum = f * ml.y;
#pragma unroll
            for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
            for (int j = 0; j < kFewRows; ++j) {
                float4 acc = zero;
#pragma unroll
                for (int k = 0; k < kFewParts; ++k) add_part(acc, __shfl_sync(0xffffffffu, f, kLanes * j + k), o[j][k]);
                const float its_top = __shfl_sync(0xffffffffu, top, kLanes * j);
                const float its_sum = __shfl_sync(0xffffffffu, sum, kLanes * j);
                if (row0 + j * step < m.rows) put_row<D, SEE>(A, r[j], partial, lane, its_top, its_sum, acc);
            }
        }
        return;
    }
#pragma unroll 1
    for (int row = share * kJoinWarps + warp; row < m.rows; row += step) {
        const JoinRow r = join_row<D, SEE>(A, m, row, lane);
        float top = kNone, sum = 0.0f;
#pragma unroll 1
        for (int c = c0 + lane; c < c1; c += 32) top = fmaxf(top, ws.ml[slot(c, row)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float4 acc = zero;
#pragma unroll 1
        for (int cb = c0; cb < c1; cb += 32) {
            const int c = cb + lane;
            float f = 0.0f;
            if (c < c1) {
                const float2 ml = ws.ml[slot(c, row)];
                f = exp2f(ml.x - top);
                sum += f * ml.y;
            }
            const int n = min(32, c1 - cb);
            const int d = lane * 4 < D ? lane * 4 : 0;
#pragma unroll 1
            for (int k0 = 0; k0 < n; k0 += 16) {
                float4 o[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int ck = min(cb + k0 + k, c1 - 1);
                    o[k] = k0 + k < n ? *reinterpret_cast<const float4*>(ws.o + slot(ck, row) * D + d) : zero;
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) add_part(acc, __shfl_sync(0xffffffffu, f, (k0 + k) & 31), o[k]);
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        put_row<D, SEE>(A, r, partial, lane, top, sum, acc);
    }
}

// cuTensorMapEncodeTiled, found through the runtime (the library does not link libcuda).
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                             CUtensorMapFloatOOBfill);
EncodeFn encode_fn()
{
    static const EncodeFn fn = []() -> EncodeFn {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess || q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

}  // namespace

int encode_cache(CUtensorMap* map, void* codes, const dspark_cache& c)
{
    const EncodeFn fn = encode_fn();
    if (fn == nullptr) return fail(DSPARK_ERR_CUDA, "dspark attend: cuTensorMapEncodeTiled not found");
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.dim),
                                static_cast<cuuint64_t>(c.n_pages) * c.heads * c.page};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.dim)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(c.dim), static_cast<cuuint32_t>(c.page)};
    const cuuint32_t ones[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          c.dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(DSPARK_ERR_CUDA, "dspark attend: cuTensorMapEncodeTiled returned %d", static_cast<int>(r));
    return DSPARK_OK;
}

bool attend_mma_serves(const AttendCall& A, int dtype)
{
    return dtype == DSPARK_BF16 && (A.c.dim == 64 || A.c.dim == 128) && A.c.n_pages > 0;
}

// Whether a call's line fits an int, whatever the lengths.
bool attend_mma_fits(const AttendCall& A)
{
    const int R = unit_rows(A), cost = R < kTile ? kUnitCost<8> : kUnitCost<kTile>;
    const int64_t units = static_cast<int64_t>(A.rows) * A.q_heads / R + static_cast<int64_t>(A.B) * A.c.heads;
    return units * (A.last_tile + 1 + cost) <= INT32_MAX / 2;
}

size_t attend_workspace_bytes(int dim)
{
    if (dim != 64 && dim != 128) return 16;
    return kMaxCtas * (sizeof(RunMeta) + 2 * kTile * (sizeof(float2) + dim * sizeof(float)));
}

namespace {
template <int SEE>
int launch_both(const AttendCall& A, int ctas, int device, cudaStream_t stream)
{
    const int rc = unit_rows(A) < kTile ? launch_attend_narrow<SEE>(A, ctas, device, stream)
                                        : launch_attend_wide<SEE>(A, ctas, device, stream);
    if (rc != DSPARK_OK) return rc;
    return launch_pdl("attend join", A.c.dim == 128 ? attend_join_kernel<128, SEE> : attend_join_kernel<64, SEE>,
                      dim3(ctas), dim3(kJoinWarps * 32), 0, stream, A);
}
}  // namespace

int launch_attend_mma(const AttendCall& A, See see, cudaStream_t stream)
{
    if (!attend_mma_fits(A))
        return fail(DSPARK_ERR_UNSUPPORTED, "dspark_attend: rows, heads and pages beyond what one call can cut");
    DeviceInfo dev;
    const int rc = current_device(&dev);
    if (rc != DSPARK_OK) return rc;
    const int ctas = dev.sm_count * 2 < kMaxCtas ? dev.sm_count * 2 : kMaxCtas;
    switch (see) {
    case kSinks: return launch_both<kSinks>(A, ctas, dev.device, stream);
    case kPrefix: return launch_both<kPrefix>(A, ctas, dev.device, stream);
    case kSuffix: return launch_both<kSuffix>(A, ctas, dev.device, stream);
    default: return launch_both<kAll>(A, ctas, dev.device, stream);
    }
}

}  // namespace dspark
