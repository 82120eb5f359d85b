/* A plain C caller of the calls that take structs and many sizes: dspark_adjust with every field of
 * dspark_adjustments, dspark_attend_sinks and dspark_attend_shared over a small paged cache in fp32.
 * Device buffers come from cudaMalloc, the calls go on the legacy default stream, and the results are
 * compared with the formulas in double. Exit status 0 and "ok" when everything matches. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda_runtime.h>

#include "dspark.h"

#define CUDA(x)                                                                              \
    do {                                                                                     \
        cudaError_t e_ = (x);                                                                \
        if (e_ != cudaSuccess) {                                                             \
            fprintf(stderr, "%s failed: %s\n", #x, cudaGetErrorString(e_));                  \
            exit(2);                                                                         \
        }                                                                                    \
    } while (0)

#define DSPARK(x)                                                                            \
    do {                                                                                     \
        int r_ = (x);                                                                        \
        if (r_ != DSPARK_OK) {                                                               \
            fprintf(stderr, "%s returned %d: %s\n", #x, r_, dspark_last_error());            \
            exit(3);                                                                         \
        }                                                                                    \
    } while (0)

static int failures = 0;

/* 64-bit linear congruential generator (Knuth's MMIX constants): the inputs' only source */
static uint64_t lcg_state = 0x2545F4914F6CDD1Dull;
static uint32_t rnd32(void)
{
    lcg_state = lcg_state * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(lcg_state >> 32);
}
static float rnd01(void) { return (float)(rnd32() >> 8) * (1.0f / 16777216.0f); }

static void* dev_copy(const void* host, size_t bytes)
{
    void* d = NULL;
    CUDA(cudaMalloc(&d, bytes));
    CUDA(cudaMemcpy(d, host, bytes, cudaMemcpyHostToDevice));
    return d;
}

static void check(const char* what, int i, double got, double want, double tol)
{
    if (!(fabs(got - want) <= tol) && got != want) {
        fprintf(stderr, "%s[%d]: library %.9g, formula %.9g\n", what, i, got, want);
        ++failures;
    }
}

/* ---- dspark_adjust: two requests, 3 and 2 rows of 70 tokens ------------------------------- */
enum { V = 70, B = 2, GAMMA = 3, ROWS = 5, CAP = 8, NB = 3, WORDS = 4, MASKS = 2 };

static void adjust(int32_t* d_status)
{
    static float x[ROWS * V], out[ROWS * V];
    for (int i = 0; i < ROWS * V; ++i) x[i] = 6.0f * (rnd01() - 0.5f);
    const int32_t cu[B + 1] = {0, 3, 5}, tokens[B * GAMMA] = {9, 4, 4, 20, 5, 0};
    const int32_t history[B * CAP] = {1, 2, 4, 4, 9, 0, 0, 0, 5, 5, 20, 0, 0, 0, 0, 0};
    const int32_t length[B] = {5, 3}, prompt[B] = {2, 1};
    const float repetition[B] = {1.25f, 0.8f}, presence[B] = {0.5f, 0.0f}, frequency[B] = {0.25f, 1.0f};
    const int32_t bias_tokens[B * NB] = {4, 60, 4, 5, 6, 0}, bias_len[B] = {3, 2};
    const float bias_values[B * NB] = {9.0f, -INFINITY, 1.5f, -2.0f, 3.0f, 0.0f};
    uint32_t mask[MASKS * WORDS];
    for (int i = 0; i < MASKS * WORDS; ++i) mask[i] = rnd32() | 0x70u;     /* 4, 5 and 6 stay allowed */
    const int32_t mask_row[ROWS] = {0, -1, 1, 0, -1};
    dspark_adjustments how;
    memset(&how, 0, sizeof(how));
    how.history = (const int32_t*)dev_copy(history, sizeof(history));
    how.history_len = (const int32_t*)dev_copy(length, sizeof(length));
    how.prompt_len = (const int32_t*)dev_copy(prompt, sizeof(prompt));
    how.history_cap = CAP;
    how.bias_cap = NB;
    how.repetition = (const float*)dev_copy(repetition, sizeof(repetition));
    how.presence = (const float*)dev_copy(presence, sizeof(presence));
    how.frequency = (const float*)dev_copy(frequency, sizeof(frequency));
    how.bias_tokens = (const int32_t*)dev_copy(bias_tokens, sizeof(bias_tokens));
    how.bias_values = (const float*)dev_copy(bias_values, sizeof(bias_values));
    how.bias_len = (const int32_t*)dev_copy(bias_len, sizeof(bias_len));
    how.mask = (const uint32_t*)dev_copy(mask, sizeof(mask));
    how.mask_row = (const int32_t*)dev_copy(mask_row, sizeof(mask_row));
    how.mask_stride = WORDS;
    how.mask_rows = MASKS;
    void *d_x = dev_copy(x, sizeof(x)), *d_out;
    CUDA(cudaMalloc(&d_out, sizeof(out)));
    DSPARK(dspark_adjust(d_x, V, d_out, V, DSPARK_F32, ROWS, V, (const int32_t*)dev_copy(cu, sizeof(cu)),
                         (const int32_t*)dev_copy(tokens, sizeof(tokens)), B, GAMMA, &how, d_status, 0));
    CUDA(cudaDeviceSynchronize());
    CUDA(cudaMemcpy(out, d_out, sizeof(out), cudaMemcpyDeviceToHost));
    for (int b = 0; b < B; ++b)
        for (int r = cu[b]; r < cu[b + 1]; ++r)
            for (int v = 0; v < V; ++v) {
                int uses = 0, seen = 0;
                for (int j = 0; j < length[b]; ++j)
                    if (history[b * CAP + j] == v) { seen = 1; uses += j >= prompt[b]; }
                for (int j = 1; j <= r - cu[b]; ++j) uses += tokens[b * GAMMA + j] == v;
                double y = x[r * V + v];
                if (seen || uses) y = y > 0 ? y / repetition[b] : y * repetition[b];
                if (uses) y -= (double)frequency[b] * uses + presence[b];
                double bias = 0.0;
                for (int j = 0; j < bias_len[b]; ++j)
                    if (bias_tokens[b * NB + j] == v) bias = bias_values[b * NB + j];
                y += bias;
                if (mask_row[r] >= 0 && !(mask[mask_row[r] * WORDS + v / 32] >> (v % 32) & 1)) y = -INFINITY;
                /* four roundings to fp32 of magnitudes up to 16 */
                check("adjust", r * V + v, out[r * V + v], y, 4 * 16 * 0x1p-24);
            }
}

/* ---- attention: three requests of 2, 1 and 3 rows, 2 heads to each of 2 cache heads, dim 16 ---- */
enum { REQ = 3, QROWS = 6, HEADS = 2, HQ = 4, DIM = 16, PAGE = 16, PAGES = 9, WIDTH = 4 };

static double code_value(uint8_t c)
{
    const int e = c >> 3 & 15, m = c & 7;
    const double a = e == 0 ? m * 0x1p-9 : (8 + m) * ldexp(1.0, e - 10);
    return c & 0x80 ? -a : a;
}

static void attend(int shared, int32_t* d_status)
{
    static uint8_t k[PAGES * HEADS * PAGE * DIM], v[PAGES * HEADS * PAGE * DIM];
    static float ks[PAGES * HEADS], vs[PAGES * HEADS], q[QROWS * HQ * DIM], out[QROWS * HQ * DIM], lse[QROWS * HQ];
    /* codes of magnitudes up to 1 (exponents 1 to 7, either sign) */
    for (size_t i = 0; i < sizeof(k); ++i) {
        k[i] = (uint8_t)((rnd32() & 0x80) | (8 + rnd32() % 49));
        v[i] = (uint8_t)((rnd32() & 0x80) | (8 + rnd32() % 49));
    }
    for (int i = 0; i < PAGES * HEADS; ++i) { ks[i] = 0.5f + rnd01(); vs[i] = 0.5f + rnd01(); }
    for (int i = 0; i < QROWS * HQ * DIM; ++i) q[i] = 2.0f * rnd01() - 1.0f;
    /* the first two pages are common to all */
    const int32_t table[REQ * WIDTH] = {7, 2, 0, 1, 7, 2, 3, -1, 7, 2, 4, 5};
    const int32_t cu[REQ + 1] = {0, 2, 3, 6}, lengths[REQ] = {45, 33, 60};
    const int32_t group_cu[2] = {0, REQ}, prefix[1] = {32};
    const int window = 11, sinks = 18;
    const float scale = 0.25f;
    dspark_cache cache;
    memset(&cache, 0, sizeof(cache));
    cache.k = dev_copy(k, sizeof(k));
    cache.v = dev_copy(v, sizeof(v));
    cache.k_scale = (float*)dev_copy(ks, sizeof(ks));
    cache.v_scale = (float*)dev_copy(vs, sizeof(vs));
    cache.table = (const int32_t*)dev_copy(table, sizeof(table));
    cache.n_pages = PAGES;
    cache.heads = HEADS;
    cache.page = PAGE;
    cache.dim = DIM;
    cache.width = WIDTH;
    const int32_t *d_cu = (const int32_t*)dev_copy(cu, sizeof(cu)),
                  *d_lengths = (const int32_t*)dev_copy(lengths, sizeof(lengths));
    void *d_q = dev_copy(q, sizeof(q)), *d_out, *d_ws;
    float* d_lse;
    CUDA(cudaMalloc(&d_out, sizeof(out)));
    CUDA(cudaMalloc((void**)&d_lse, sizeof(lse)));
    const size_t bytes = shared ? dspark_attend_shared_workspace_bytes(QROWS, HQ, HEADS, DIM, REQ)
                                : dspark_attend_workspace_bytes(HEADS, DIM);
    CUDA(cudaMalloc(&d_ws, bytes));
    if (shared)
        DSPARK(dspark_attend_shared(&cache, d_q, HQ * DIM, d_out, HQ * DIM, HQ, DSPARK_F32, QROWS, d_cu, d_lengths, REQ,
                                    (const int32_t*)dev_copy(group_cu, sizeof(group_cu)),
                                    (const int32_t*)dev_copy(prefix, sizeof(prefix)), 1, scale, d_lse, d_ws, bytes,
                                    d_status, 0));
    else
        DSPARK(dspark_attend_sinks(&cache, d_q, HQ * DIM, d_out, HQ * DIM, HQ, DSPARK_F32, QROWS, d_cu, d_lengths, REQ,
                                   scale, window, sinks, d_lse, d_ws, bytes, d_status, 0));
    CUDA(cudaDeviceSynchronize());
    CUDA(cudaMemcpy(out, d_out, sizeof(out), cudaMemcpyDeviceToHost));
    CUDA(cudaMemcpy(lse, d_lse, sizeof(lse), cudaMemcpyDeviceToHost));
    for (int b = 0; b < REQ; ++b)
        for (int r = cu[b]; r < cu[b + 1]; ++r)
            for (int h = 0; h < HQ; ++h) {
                const int p = lengths[b] + r - cu[b], g = h / (HQ / HEADS);
                const float* x = q + (r * HQ + h) * DIM;
                double sum = 0.0, o[DIM] = {0.0};
                for (int t = 0; t <= p; ++t) {
                    if (!shared && t <= p - window && t >= sinks) continue;
                    const int block = (table[b * WIDTH + t / PAGE] * HEADS + g), at = (block * PAGE + t % PAGE) * DIM;
                    double s = 0.0;
                    for (int d = 0; d < DIM; ++d) s += x[d] * code_value(k[at + d]);
                    const double w = exp(scale * ks[block] * s);
                    sum += w;
                    for (int d = 0; d < DIM; ++d) o[d] += w * vs[block] * code_value(v[at + d]);
                }
                /* scores are under 0.25 x 1.5 x 16 = 6, off by (16 + 8) 2^-24 of that; a weight is off by
                   twice the exponential of it, times values under 1.5 */
                for (int d = 0; d < DIM; ++d)
                    check(shared ? "shared" : "sinks", (r * HQ + h) * DIM + d, out[(r * HQ + h) * DIM + d], o[d] / sum,
                          4e-5);
                check("lse", r * HQ + h, lse[r * HQ + h], log(sum), 4e-5);
            }
}

int main(void)
{
    int32_t status = 0, *d_status = (int32_t*)dev_copy(&status, 4);
    adjust(d_status);
    attend(0, d_status);
    attend(1, d_status);
    CUDA(cudaMemcpy(&status, d_status, 4, cudaMemcpyDeviceToHost));
    if (status != 0) {
        fprintf(stderr, "status %d\n", status);
        ++failures;
    }
    if (failures) return 1;
    printf("ok\n");
    return 0;
}
