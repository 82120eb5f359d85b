// cache_abi.cu — host-side argument checks and dispatch of dspark_append, dspark_attend and its kin.
// Every check happens before anything is enqueued; see include/dspark.h for the contract.
#include <cmath>

#include "attend.cuh"
#include "cache.cuh"
#include "rope.cuh"

namespace dspark {

namespace {
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
}  // namespace

int check_cache(const char* fn, const dspark_cache* c)
{
    if (c == nullptr) return fail(DSPARK_ERR_INVALID_ARG, "%s: cache is required", fn);
    if (c->n_pages < 0 || c->heads < 1 || c->width < 0 || c->dim < 1)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: bad cache sizes n_pages=%d heads=%d dim=%d width=%d",
                    fn, c->n_pages, c->heads, c->dim, c->width);
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: page = %d is none of 16, 32, 64, 128", fn, c->page);
    if (c->dim % 16 != 0 || c->dim > DSPARK_MAX_CACHE_HEAD)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: dim = %d is not a multiple of 16 up to %d", fn,
                    c->dim, DSPARK_MAX_CACHE_HEAD);
    if (c->heads > 65535)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: heads = %d above 65535", fn, c->heads);
    if (static_cast<int64_t>(c->n_pages) * c->heads * c->page > INT32_MAX - 256)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: n_pages*heads*page = %lld overflows int32", fn,
                    static_cast<long long>(c->n_pages) * c->heads * c->page);
    if (c->n_pages > 0 && (c->k == nullptr || c->v == nullptr || c->k_scale == nullptr ||
                           c->v_scale == nullptr))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: the cache's pages and scales are required", fn);
    if (c->width > 0 && c->table == nullptr)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: the cache's page table is required", fn);
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
        !aligned(c->v_scale, 4) || !aligned(c->table, 4))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: pages must be 16-byte, scales and table 4-byte aligned", fn);
    return DSPARK_OK;
}

// The checks that the attention calls share, and the call they describe. *go: there is work to do.
int attend_call(const char* fn, const dspark_cache* cache, const void* q, int64_t q_stride, void* out,
                int64_t out_stride, int q_heads, dspark_dtype dtype, int rows, const int32_t* cu_seqlens,
                const int32_t* lengths, int B, float scale, int window, float* lse, void* workspace,
                size_t workspace_bytes, int32_t* status, AttendCall* call, bool* go)
{
    *go = false;
    const int rc = check_cache(fn, cache);
    if (rc != DSPARK_OK) return rc;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows < 0 || B < 0 || window < 0)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: bad sizes rows=%d B=%d window=%d", fn, rows, B,
                    window);
    if (q_heads < 1 || q_heads % cache->heads != 0)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: q_heads = %d is not a multiple of the cache's %d",
                    fn, q_heads, cache->heads);
    if (static_cast<int64_t>(rows) * q_heads > INT32_MAX / 2)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: rows*q_heads = %lld is too large", fn,
                    static_cast<long long>(rows) * q_heads);
    const int64_t width = static_cast<int64_t>(q_heads) * cache->dim;
    if (q_stride < width || out_stride < width)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: row strides %lld, %lld below q_heads*dim = %lld",
                    fn, static_cast<long long>(q_stride), static_cast<long long>(out_stride),
                    static_cast<long long>(width));
    if (!std::isfinite(scale))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: scale must be finite", fn);
    if (rows == 0 || B == 0) return DSPARK_OK;
    const uintptr_t e = dtype == DSPARK_BF16 ? 2 : 4;
    if (q == nullptr || out == nullptr || cu_seqlens == nullptr || lengths == nullptr ||
        !aligned(q, e) || !aligned(out, e) || !aligned(cu_seqlens, 4) || !aligned(lengths, 4) ||
        !aligned(lse, 4))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: q, out, cu_seqlens and lengths are required, "
                    "aligned to their elements", fn);
    const size_t need = attend_workspace_bytes(cache->dim);
    if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: a 16-byte aligned workspace of %zu bytes is needed, got %zu",
                    fn, need, workspace_bytes);
    AttendCall A = {};
    A.c = *cache;
    A.q = q;
    A.q_stride = q_stride;
    A.out = out;
    A.out_stride = out_stride;
    A.q_heads = q_heads;
    A.group = q_heads / cache->heads;
    A.rows = rows;
    A.cu = cu_seqlens;
    A.lengths = lengths;
    A.B = B;
    A.scale = scale;
    A.window = window;
    A.lse = lse;
    const int64_t reach = static_cast<int64_t>(cache->width) * cache->page;
    A.reach = static_cast<int>(reach < INT32_MAX ? reach : INT32_MAX);
    A.last_tile = static_cast<int>((reach > 0 ? reach - 1 : 0) / 128);
    A.ws = workspace;
    A.status = status;
    *call = A;
    *go = true;
    return DSPARK_OK;
}

}  // namespace dspark

using dspark::aligned;
using dspark::fail;

extern "C" {

int dspark_append(const dspark_cache* cache, const dspark_rope* rope, const void* k,
                  int64_t k_stride, const void* v, int64_t v_stride, const void* q,
                  int64_t q_stride, void* q_out, int64_t q_out_stride, int q_heads,
                  dspark_dtype dtype, int rows, const int32_t* row_req, const int32_t* row_pos,
                  const int32_t* lengths, int B, int32_t* status, cudaStream_t stream)
{
    const char* fn = "dspark_append";
    int rc = dspark::check_cache(fn, cache);
    if (rc == DSPARK_OK) rc = dspark::check_rope(fn, rope, cache->dim);
    if (rc != DSPARK_OK) return rc;
    if (dtype != DSPARK_BF16 && dtype != DSPARK_F32)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, static_cast<int>(dtype));
    if (rows < 0 || B < 0)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: bad sizes rows=%d B=%d", fn, rows, B);
    const int64_t width = static_cast<int64_t>(cache->heads) * cache->dim;
    if (k_stride < width || v_stride < width)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: row strides %lld, %lld below heads*dim = %lld", fn,
                    static_cast<long long>(k_stride), static_cast<long long>(v_stride),
                    static_cast<long long>(width));
    if ((q == nullptr) != (q_out == nullptr))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: give both q and q_out or neither", fn);
    const int64_t q_width = static_cast<int64_t>(q_heads) * cache->dim;
    if (q != nullptr && (q_heads < 1 || q_width > INT32_MAX / 8 || q_stride < q_width ||
                         q_out_stride < q_width))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: q_heads = %d, row strides %lld, %lld", fn, q_heads,
                    static_cast<long long>(q_stride), static_cast<long long>(q_out_stride));
    if ((static_cast<int64_t>(rows) + 16) * cache->heads * 2 > INT32_MAX / 2)
        return fail(DSPARK_ERR_UNSUPPORTED, "%s: rows*heads = %lld is too large", fn,
                    static_cast<long long>(rows) * cache->heads);
    if (rows == 0) return DSPARK_OK;
    const uintptr_t e = dtype == DSPARK_BF16 ? 2 : 4;
    if (k == nullptr || v == nullptr || row_req == nullptr || row_pos == nullptr ||
        (B > 0 && lengths == nullptr) || !aligned(k, e) || !aligned(v, e) || !aligned(q, e) ||
        !aligned(q_out, e) || !aligned(row_req, 4) || !aligned(row_pos, 4) || !aligned(lengths, 4))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: k, v, row_req, row_pos and lengths are required, "
                    "aligned to their elements", fn);
    return dspark::launch_append(*cache, dspark::rope_of(rope, false), k, k_stride, v, v_stride, q,
                                 q_stride, q_out, q_out_stride, q_heads, static_cast<int>(dtype),
                                 rows, B, row_req, row_pos, lengths, status, stream);
}

size_t dspark_attend_workspace_bytes(int heads, int dim)
{
    if (heads < 1 || dim < 16 || dim % 16 != 0 || dim > DSPARK_MAX_CACHE_HEAD) {
        fail(DSPARK_ERR_INVALID_ARG, "dspark_attend_workspace_bytes: bad sizes heads=%d dim=%d",
             heads, dim);
        return 0;
    }
    return dspark::attend_workspace_bytes(dim);
}

int dspark_attend(const dspark_cache* cache, const void* q, int64_t q_stride, void* out,
                  int64_t out_stride, int q_heads, dspark_dtype dtype, int rows,
                  const int32_t* cu_seqlens, const int32_t* lengths, int B, float scale,
                  int window, float* lse, void* workspace, size_t workspace_bytes,
                  int32_t* status, cudaStream_t stream)
{
    dspark::AttendCall A;
    bool go;
    const int rc = dspark::attend_call("dspark_attend", cache, q, q_stride, out, out_stride, q_heads, dtype, rows,
                                       cu_seqlens, lengths, B, scale, window, lse, workspace, workspace_bytes,
                                       status, &A, &go);
    return rc == DSPARK_OK && go ? dspark::launch_attend(A, dspark::kAll, static_cast<int>(dtype), stream) : rc;
}

int dspark_attend_sinks(const dspark_cache* cache, const void* q, int64_t q_stride, void* out,
                        int64_t out_stride, int q_heads, dspark_dtype dtype, int rows,
                        const int32_t* cu_seqlens, const int32_t* lengths, int B, float scale,
                        int window, int sinks, float* lse, void* workspace, size_t workspace_bytes,
                        int32_t* status, cudaStream_t stream)
{
    const char* fn = "dspark_attend_sinks";
    dspark::AttendCall A;
    bool go;
    const int rc = dspark::attend_call(fn, cache, q, q_stride, out, out_stride, q_heads, dtype, rows, cu_seqlens,
                                       lengths, B, scale, window, lse, workspace, workspace_bytes, status, &A, &go);
    if (rc != DSPARK_OK) return rc;
    if (sinks < 0 || sinks > INT32_MAX - 256)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: sinks = %d outside [0, %d]", fn, sinks, INT32_MAX - 256);
    if (!go) return DSPARK_OK;
    A.sinks = sinks;
    A.sink_blocks = (sinks + cache->page - 1) / cache->page;
    // without a window every row sees its first tokens anyway
    return dspark::launch_attend(A, window > 0 && sinks > 0 ? dspark::kSinks : dspark::kAll, static_cast<int>(dtype),
                                 stream);
}

size_t dspark_attend_shared_workspace_bytes(int rows, int q_heads, int heads, int dim, int B)
{
    if (rows < 0 || q_heads < 1 || heads < 1 || q_heads % heads != 0 || dim < 16 || dim % 16 != 0 ||
        dim > DSPARK_MAX_CACHE_HEAD || B < 0 || static_cast<int64_t>(rows) * q_heads > INT32_MAX / 2) {
        fail(DSPARK_ERR_INVALID_ARG,
             "dspark_attend_shared_workspace_bytes: bad sizes rows=%d q_heads=%d heads=%d dim=%d B=%d", rows, q_heads,
             heads, dim, B);
        return 0;
    }
    return dspark::attend_shared_workspace_bytes(rows, q_heads, dim, B);
}

int dspark_attend_shared(const dspark_cache* cache, const void* q, int64_t q_stride, void* out,
                         int64_t out_stride, int q_heads, dspark_dtype dtype, int rows,
                         const int32_t* cu_seqlens, const int32_t* lengths, int B,
                         const int32_t* group_cu, const int32_t* prefix, int groups, float scale,
                         float* lse, void* workspace, size_t workspace_bytes, int32_t* status,
                         cudaStream_t stream)
{
    const char* fn = "dspark_attend_shared";
    dspark::AttendCall A;
    bool go;
    const int rc = dspark::attend_call(fn, cache, q, q_stride, out, out_stride, q_heads, dtype, rows, cu_seqlens,
                                       lengths, B, scale, 0, lse, workspace, workspace_bytes, status, &A, &go);
    if (rc != DSPARK_OK) return rc;
    if (groups < 0 || groups > INT32_MAX / 2)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: groups = %d", fn, groups);
    if (!go) return DSPARK_OK;
    if (groups > 0 && (group_cu == nullptr || prefix == nullptr || !aligned(group_cu, 4) || !aligned(prefix, 4)))
        return fail(DSPARK_ERR_INVALID_ARG, "%s: group_cu and prefix are required, 4-byte aligned", fn);
    const size_t need = dspark::attend_shared_workspace_bytes(rows, q_heads, cache->dim, B);
    if (workspace_bytes < need)
        return fail(DSPARK_ERR_INVALID_ARG, "%s: a workspace of %zu bytes is needed, got %zu", fn, need, workspace_bytes);
    return dspark::launch_attend_shared(A, group_cu, prefix, groups, static_cast<int>(dtype), stream);
}

}  // extern "C"
