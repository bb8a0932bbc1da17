/*
 * attention_abi_check.c -- drives the attention operators of libar.so from
 * plain C with raw device pointers: no PyTorch, no Python in the call path.
 * Test helper, built by the package's build step and run by
 * tests/test_gpu_attention_abi.py.
 *
 * usage: attention_abi_check in.bin out.bin
 *   in.bin   TOKENS x (HEADS + 2 KV_HEADS) x DIM bf16: queries, keys, values of
 *            each token; then TOKENS x DIM floats: cosines and sines
 *   out.bin  written: q and k after ar_qk_norm_rope (in place), keys and
 *            values read back from the cache, the attention's output (bf16),
 *            then lse and the gradient of the queries' weight for q as its own
 *            gradient (floats)
 * Exit status 0 when every call succeeds and bad calls are refused.
 */
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "ar.h"

#define HIP_OK(x)                                                                  \
    do {                                                                           \
        hipError_t e_ = (x);                                                       \
        if (e_ != hipSuccess) {                                                    \
            fprintf(stderr, "%s failed: %s\n", #x, hipGetErrorString(e_));         \
            return 2;                                                              \
        }                                                                          \
    } while (0)

#define AR_IS(x, code)                                                             \
    do {                                                                           \
        int rc_ = (x);                                                             \
        if (rc_ != (code)) {                                                       \
            fprintf(stderr, "%s gave: %s\n", #x, ar_strerror(rc_));                \
            return 3;                                                              \
        }                                                                          \
    } while (0)

enum { TOKENS = 70, HEADS = 4, KV_HEADS = 2, DIM = 64, PAGE = 32, PAGES = 5 };
enum { ROW = (HEADS + 2 * KV_HEADS) * DIM, QN = TOKENS * HEADS * DIM, KN = TOKENS * KV_HEADS * DIM };

int main(int argc, char **argv)
{
    if (argc != 3) return 1;
    static uint16_t qkv[TOKENS * ROW], ones[DIM], res[QN];
    static float cs[TOKENS * DIM], stats[TOKENS * HEADS];
    static int64_t at[TOKENS], slot[TOKENS];
    const int32_t pages[3] = {4, 0, 2}, start[2] = {0, TOKENS}, len[1] = {TOKENS};
    FILE *f = fopen(argv[1], "rb");
    if (!f || fread(qkv, 2, TOKENS * ROW, f) != TOKENS * ROW || fread(cs, 4, TOKENS * DIM, f) != TOKENS * DIM) return 1;
    fclose(f);
    for (int i = 0; i < DIM; ++i) ones[i] = 0x3F80;
    for (int i = 0; i < TOKENS; ++i) at[i] = i, slot[i] = (int64_t)pages[i / PAGE] * PAGE + i % PAGE;

    const int64_t cache_bytes = ar_kv4_cache_bytes(PAGES, KV_HEADS, DIM, PAGE);
    const int64_t bwd_bytes = ar_qk_norm_rope_bwd_workspace(TOKENS, HEADS, KV_HEADS, DIM);
    const int64_t attn_bytes = ar_kv4_attention_workspace(1, TOKENS, TOKENS, TOKENS, HEADS, KV_HEADS, DIM);
    if (cache_bytes < 0 || bwd_bytes < 0 || attn_bytes < 0) return 3;
    /* one block of memory, cut into buffers of 1 MiB */
    uint8_t *m;
    const size_t part = 1 << 20;
    if ((size_t)cache_bytes > part || (size_t)bwd_bytes > part || (size_t)attn_bytes > part) return 1;
    HIP_OK(hipMalloc((void **)&m, 16 * part));
    HIP_OK(hipMemset(m, 0, 16 * part));
    uint8_t *d_qkv = m, *d_cs = m + part, *d_at = m + 2 * part, *d_slot = m + 3 * part, *d_w = m + 4 * part,
            *cache = m + 5 * part, *d_pages = m + 6 * part, *d_start = m + 7 * part, *d_len = m + 8 * part,
            *d_k = m + 9 * part, *d_v = m + 10 * part, *out = m + 11 * part, *lse = m + 12 * part,
            *ws = m + 13 * part, *d_dw = m + 14 * part, *d_raw = m + 15 * part;
    HIP_OK(hipMemcpy(d_qkv, qkv, sizeof qkv, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_raw, qkv, sizeof qkv, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_cs, cs, sizeof cs, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_at, at, sizeof at, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_slot, slot, sizeof slot, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_w, ones, sizeof ones, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_pages, pages, sizeof pages, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_start, start, sizeof start, hipMemcpyHostToDevice));
    HIP_OK(hipMemcpy(d_len, len, sizeof len, hipMemcpyHostToDevice));
    hipStream_t s;
    HIP_OK(hipStreamCreate(&s));

    const ar_rows q = {d_qkv, ROW, DIM}, k = {d_qkv + 2 * HEADS * DIM, ROW, DIM},
                  v = {d_qkv + 2 * (HEADS + KV_HEADS) * DIM, ROW, DIM}, k_out = {d_k, KV_HEADS * DIM, DIM},
                  v_out = {d_v, KV_HEADS * DIM, DIM}, o = {out, HEADS * DIM, DIM},
                  raw = {d_raw, ROW, DIM}, none = {0, 0, 0};
    /* the gradient goes where the output will be written later */
    AR_IS(ar_qk_norm_rope_bwd(raw, none, raw, none, d_w, 0, d_cs, d_at, o, none, d_dw, 0, ws, TOKENS, HEADS, 0, DIM, DIM, TOKENS,
                              1e-6f, 0, s), AR_OK);
    AR_IS(ar_qk_norm_rope(q, k, d_w, d_w, d_cs, d_at, q, k, TOKENS, HEADS, KV_HEADS, DIM, DIM, TOKENS, 1e-6f, 0, s), AR_OK);
    AR_IS(ar_qk_norm_rope(q, k, d_w, d_w, d_cs, d_at, k, q, TOKENS, HEADS, KV_HEADS, DIM, DIM, TOKENS, 1e-6f, 0, s), AR_EALIAS);
    AR_IS(ar_kv4_write(k, v, d_slot, cache, TOKENS, KV_HEADS, DIM, PAGES, PAGE, s), AR_OK);
    AR_IS(ar_kv4_write(k, v, d_slot, cache, TOKENS, KV_HEADS, DIM, PAGES, PAGE + 1, s), AR_EINVAL);
    AR_IS(ar_kv4_read(cache, d_slot, k_out, v_out, TOKENS, KV_HEADS, DIM, PAGES, PAGE, s), AR_OK);
    AR_IS(ar_kv4_attention(q, cache, d_pages, 3, d_start, d_len, o, lse, ws, TOKENS, 1, HEADS, KV_HEADS, DIM, PAGES, PAGE, 3, TOKENS,
                           TOKENS, 0, 0.125f, s), AR_OK);
    AR_IS(ar_kv4_attention(q, cache, d_pages, 3, d_start, d_len, o, lse, 0, TOKENS, 1, HEADS, KV_HEADS, DIM, PAGES, PAGE, 3, TOKENS,
                           TOKENS, 0, 0.125f, s), AR_EINVAL);
    HIP_OK(hipStreamSynchronize(s));

    f = fopen(argv[2], "wb");
    if (!f) return 1;
    HIP_OK(hipMemcpy(qkv, d_qkv, sizeof qkv, hipMemcpyDeviceToHost));
    for (int i = 0; i < TOKENS; ++i) fwrite(qkv + i * ROW, 2, HEADS * DIM, f);
    for (int i = 0; i < TOKENS; ++i) fwrite(qkv + i * ROW + HEADS * DIM, 2, KV_HEADS * DIM, f);
    HIP_OK(hipMemcpy(res, d_k, 2 * KN, hipMemcpyDeviceToHost));
    fwrite(res, 2, KN, f);
    HIP_OK(hipMemcpy(res, d_v, 2 * KN, hipMemcpyDeviceToHost));
    fwrite(res, 2, KN, f);
    HIP_OK(hipMemcpy(res, out, 2 * QN, hipMemcpyDeviceToHost));
    fwrite(res, 2, QN, f);
    HIP_OK(hipMemcpy(stats, lse, sizeof stats, hipMemcpyDeviceToHost));
    fwrite(stats, 4, TOKENS * HEADS, f);
    HIP_OK(hipMemcpy(stats, d_dw, 4 * DIM, hipMemcpyDeviceToHost));
    fwrite(stats, 4, DIM, f);
    fclose(f);
    HIP_OK(hipStreamDestroy(s));
    HIP_OK(hipFree(m));
    return 0;
}
