// attend_join.cu — the second kernel of dspark_attend on the tensor cores: joins the parts of the
// units that a run's end cut; and the host side that both first kernels share.
#include "attend_mma.cuh"

namespace dspark {
namespace {

// Joins the parts of each cut unit: the runs that a unit's places cross, but the first, share its
// rows (a unit cut once is joined by one CTA, one cut 37 times by 37). A warp takes a row: its
// lanes first read the parts' references and sums, then dim / 4 lanes add up the parts, 16 loads
// in flight.
constexpr int kJoinWarps = 16;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(AttendCall A)
{
    pdl_wait_and_trigger();
    const Workspace ws = workspace_of(A.ws);
    const RunMeta m = ws.meta[blockIdx.x];
    if (m.rows == 0) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = m.first / m.run;                          // the run of the unit's first tile
    const int c1 = (m.end + m.run - 1) / m.run;              // one past the run of its last
    // in the first run an earlier unit's piece may come before
    const int part0 = 2 * c0 + (c0 * m.run < m.unit ? 1 : 0);
    const int shares = c1 - c0 - 1, share = static_cast<int>(blockIdx.x) - c0 - 1;
#pragma unroll 1
    for (int row = share * kJoinWarps + warp; row < m.rows; row += shares * kJoinWarps) {
        float top = kNone, sum = 0.0f;
#pragma unroll 1
        for (int c = c0 + lane; c < c1; c += 32)
            top = fmaxf(top, ws.ml[(c == c0 ? part0 : 2 * c) * kTile + row].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int cb = c0; cb < c1; cb += 32) {
            const int c = cb + lane;
            float f = 0.0f;
            if (c < c1) {
                const float2 ml = ws.ml[(c == c0 ? part0 : 2 * c) * kTile + row];
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
                    if (k0 + k < n)
                        o[k] = *reinterpret_cast<const float4*>(
                            ws.o + (static_cast<int64_t>(ck == c0 ? part0 : 2 * ck) * kTile + row) * D + d);
                    else
                        o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float fk = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
                    acc.x = fmaf(fk, o[k].x, acc.x);
                    acc.y = fmaf(fk, o[k].y, acc.y);
                    acc.z = fmaf(fk, o[k].z, acc.z);
                    acc.w = fmaf(fk, o[k].w, acc.w);
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int flat = m.flat0 + row;
        const int64_t prow = m.row0 + flat / A.group;
        const int head = m.head0 + flat % A.group;
        if (lane * 4 < D) {
            uint16_t* out = static_cast<uint16_t*>(A.out) + prow * A.out_stride +
                            static_cast<int64_t>(head) * D + lane * 4;
            const uint32_t a = pack_bf16(acc.x * inv, acc.y * inv), b = pack_bf16(acc.z * inv, acc.w * inv);
            out[0] = static_cast<uint16_t>(a);
            out[1] = static_cast<uint16_t>(a >> 16);
            out[2] = static_cast<uint16_t>(b);
            out[3] = static_cast<uint16_t>(b >> 16);
        }
        if (lane == 0 && A.lse != nullptr)
            A.lse[prow * A.q_heads + head] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
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

int launch_attend_join(const AttendCall& A, int ctas, cudaStream_t stream)
{
    return launch_pdl("attend join", A.c.dim == 128 ? attend_join_kernel<128> : attend_join_kernel<64>,
                      dim3(ctas), dim3(kJoinWarps * 32), 0, stream, A);
}

bool attend_mma_serves(const AttendCall& A, int dtype)
{
    return dtype == DSPARK_BF16 && (A.c.dim == 64 || A.c.dim == 128) && A.c.n_pages > 0;
}

size_t attend_workspace_bytes(int dim)
{
    if (dim != 64 && dim != 128) return 16;
    return kMaxCtas * (sizeof(RunMeta) + 2 * kTile * (sizeof(float2) + dim * sizeof(float)));
}

int launch_attend_mma(const AttendCall& A, cudaStream_t stream)
{
    DeviceInfo dev;
    int rc = current_device(&dev);
    if (rc != DSPARK_OK) return rc;
    const int ctas = dev.sm_count * 2 < kMaxCtas ? dev.sm_count * 2 : kMaxCtas;
    // By the requests' average of (position, head) rows: up to 32 the narrow kernel (64 requests over
    // 2048 tokens, 8 heads of 128: at 16 rows 74 us, wide 120; at 32 87 and 126), where it takes one
    // unit per request and head. From 33 on, two units and more, wide (48 rows: 138 and 131; 256 requests
    // over 512: 206 and 175; 128 rows: 248 and 155).
    const bool narrow = static_cast<int64_t>(A.rows) * A.group <= 32ll * A.B;
    rc = narrow ? launch_attend_narrow(A, ctas, dev.device, stream)
                : launch_attend_wide(A, ctas, dev.device, stream);
    return rc == DSPARK_OK ? launch_attend_join(A, ctas, stream) : rc;
}

}  // namespace dspark
