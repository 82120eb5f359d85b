// attend_join.cu — the second kernel of dspark_attend on the tensor cores: joins the parts of the
// units that a run's end cut; and the host side that both first kernels share.
#include "attend_mma.cuh"

namespace dspark {
namespace {

// Joins the parts of each cut unit: one warp per row, each CTA of a column takes every kJoinY-th
// group of rows.
constexpr int kJoinWarps = 4;
constexpr int kJoinY = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(AttendCall A, int ctas)
{
    pdl_wait_and_trigger();
    const Workspace ws = workspace_of(A.ws);
    const RunMeta m = ws.meta[blockIdx.x];
    if (!m.cut) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c0 = blockIdx.x;
    auto start = [&](int c) -> int64_t { return run_start(m.total, c, ctas); };
    int c1 = c0 + 1;                          // one past the last run that holds a part
    {
        int lo = c0 + 1, hi = ctas;           // the first run that starts at or past the unit's end
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (start(mid) < m.unit_end) lo = mid + 1; else hi = mid;
        }
        c1 = lo;
    }
    auto part = [&](int c) -> int { return c * 2 + (c == c0 ? m.slot : 0); };
    for (int row = blockIdx.y * kJoinWarps + warp; row < m.rows; row += kJoinY * kJoinWarps) {
        float top = kNone, sum = 0.0f;
        for (int c = c0 + lane; c < c1; c += 32)
            if (start(c) < start(c + 1)) top = fmaxf(top, ws.ml[part(c) * kTile + row].x);
        for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int cb = c0; cb < c1; cb += 32) {
            const int c = cb + lane;
            float f = 0.0f;
            int p = -1;
            if (c < c1 && start(c) < start(c + 1)) {
                p = part(c);
                const float2 ml = ws.ml[p * kTile + row];
                f = exp2f(ml.x - top);
                sum += f * ml.y;
            }
            const int n = min(32, c1 - cb);
#pragma unroll 4
            for (int k = 0; k < n; ++k) {
                const int pk = __shfl_sync(0xffffffffu, p, k);
                const float fk = __shfl_sync(0xffffffffu, f, k);
                if (pk < 0 || lane * 4 >= D) continue;
                const float4 o = *reinterpret_cast<const float4*>(
                    ws.o + (static_cast<int64_t>(pk) * kTile + row) * D + lane * 4);
                acc.x = fmaf(fk, o.x, acc.x);
                acc.y = fmaf(fk, o.y, acc.y);
                acc.z = fmaf(fk, o.z, acc.z);
                acc.w = fmaf(fk, o.w, acc.w);
            }
        }
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
                      dim3(ctas, kJoinY), dim3(kJoinWarps * 32), 0, stream, A, ctas);
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
    const bool narrow = static_cast<int64_t>(A.rows) * A.group <= 32ll * A.B;
    rc = narrow ? launch_attend_narrow(A, ctas, dev.device, stream)
                : launch_attend_wide(A, ctas, dev.device, stream);
    return rc == DSPARK_OK ? launch_attend_join(A, ctas, stream) : rc;
}

}  // namespace dspark
