/*
 * block_abi_check.c -- drives the operators around a block of libar.so from plain
 * C with raw device pointers: no PyTorch, no Python in the call path.  Test
 * helper, built by the package's build step and run by
 * tests/test_gpu_block_abi.py.
 *
 * usage: block_abi_check in.bin out.bin
 *   in.bin   bf16: PARTS parts and x, TOKENS x DIM each; post_weight, gate and
 *            pre_weight, DIM each; a matrix OUT x DIM; a router EXPERTS x DIM;
 *            of each expert gate and up, 2 INNER x DIM; of each expert down,
 *            DIM x INNER
 *   out.bin  written: h, z (bf16); with h, z as their own gradients and part 0 as
 *            the sum of the parts dx, dy (bf16), the gradients of gate,
 *            post_weight and pre_weight (floats); the matrix unpacked, its
 *            product with z, the experts' output for z (bf16), their choice
 *            (int32) and weights (floats)
 * Exit status 0 when every call succeeds and bad calls are refused.
 */
#include <hip/hip_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

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

enum { TOKENS = 5, DIM = 320, PARTS = 3, OUT = 100, EXPERTS = 6, INNER = 96, TOP_K = 2 };
enum { ROWS = TOKENS * DIM, UP = 2 * INNER * DIM, DOWN = DIM * INNER };
enum { IN = (PARTS + 1) * ROWS + 3 * DIM + OUT * DIM + EXPERTS * (DIM + UP + DOWN) };

static uint8_t host[1 << 20];

static int save(FILE *f, const void *device, size_t bytes)
{
    return hipMemcpy(host, device, bytes, hipMemcpyDeviceToHost) == hipSuccess && fwrite(host, 1, bytes, f) == bytes;
}

int main(int argc, char **argv)
{
    if (argc != 3) return 1;
    uint16_t *in = malloc(2 * IN);
    FILE *f = fopen(argv[1], "rb");
    if (!in || !f || fread(in, 2, IN, f) != IN) return 1;
    fclose(f);

    const int64_t matrix = ar_w4_bytes(OUT, DIM), up = ar_w4_bytes(2 * INNER, DIM), down = ar_w4_bytes(DIM, INNER);
    const int64_t bwd_bytes = ar_block_norm_bwd_workspace(TOKENS, DIM);
    const int64_t experts_bytes = ar_w4_experts_workspace(TOKENS, DIM, INNER, EXPERTS, TOP_K);
    if (matrix < 0 || up < 0 || down < 0 || bwd_bytes < 0 || experts_bytes < 0) return 3;
    /* one block of memory, cut into buffers of 4 MiB */
    uint8_t *m;
    const size_t part = 4 << 20;
    if (2 * (size_t)IN > part || (size_t)(EXPERTS * up) > part || (size_t)bwd_bytes > part || (size_t)experts_bytes > part) return 1;
    HIP_OK(hipMalloc((void **)&m, 16 * part));
    HIP_OK(hipMemset(m, 0xFF, 16 * part));
    uint16_t *d = (uint16_t *)m;
    HIP_OK(hipMemcpy(d, in, 2 * IN, hipMemcpyHostToDevice));
    const uint16_t *x = d + PARTS * ROWS, *post = x + ROWS, *gate_w = post + DIM, *pre = gate_w + DIM, *w = pre + DIM,
                   *router = w + OUT * DIM, *w_up = router + EXPERTS * DIM, *w_down = w_up + EXPERTS * UP;
    uint8_t *packed = m + part, *p_up = m + 2 * part, *p_down = m + 3 * part, *ws = m + 4 * part, *h = m + 5 * part, *z = m + 6 * part,
            *dx = m + 7 * part, *dy = m + 8 * part, *sums = m + 9 * part, *back = m + 10 * part, *y = m + 11 * part, *out = m + 12 * part,
            *choice = m + 13 * part, *weight = m + 14 * part;
    hipStream_t s;
    HIP_OK(hipStreamCreate(&s));

    ar_ptrs parts = {{0}};
    for (int p = 0; p < PARTS; ++p) parts.p[p] = d + p * ROWS;
    const ar_rows rx = {(void *)x, DIM, 0}, rh = {h, DIM, 0}, rz = {z, DIM, 0}, rdx = {dx, DIM, 0}, rdy = {dy, DIM, 0},
                  gate = {(void *)gate_w, 0, 0}, part0 = {d, DIM, 0}, dgate = {sums, 0, 0}, ry = {y, OUT, 0}, ro = {out, DIM, 0};
    AR_IS(ar_block_norm(parts, DIM, PARTS, rx, post, gate, pre, rh, rz, TOKENS, DIM, 1.0f, 1e-6f, s), AR_OK);
    AR_IS(ar_block_norm(parts, DIM, PARTS, rx, post, gate, pre, rh, rh, TOKENS, DIM, 1.0f, 1e-6f, s), AR_EALIAS);
    AR_IS(ar_block_norm_bwd(rh, rz, part0, rx, post, gate, pre, rdx, rdy, dgate, sums + 4 * DIM, sums + 8 * DIM, ws, TOKENS, DIM, 1.0f,
                            1e-6f, s), AR_OK);
    AR_IS(ar_block_norm_bwd(rh, rz, part0, rx, post, gate, pre, rdx, rdy, dgate, sums, sums + 8 * DIM, ws, TOKENS, DIM, 1.0f, 1e-6f, s),
          AR_EALIAS);
    AR_IS(ar_w4_pack(w, DIM, packed, OUT, DIM, s), AR_OK);
    AR_IS(ar_w4_pack(w, DIM, packed, OUT, DIM - 1, s), AR_EINVAL);
    AR_IS(ar_w4_unpack(packed, back, DIM, OUT, DIM, s), AR_OK);
    for (int e = 0; e < EXPERTS; ++e) {
        AR_IS(ar_w4_pack(w_up + e * UP, DIM, p_up + e * up, 2 * INNER, DIM, s), AR_OK);
        AR_IS(ar_w4_pack(w_down + e * DOWN, INNER, p_down + e * down, DIM, INNER, s), AR_OK);
    }
    AR_IS(ar_w4_linear(rz, packed, ry, TOKENS, OUT, DIM, s), AR_OK);
    AR_IS(ar_w4_linear(rz, packed, rz, TOKENS, DIM, DIM, s), AR_EALIAS);
    AR_IS(ar_w4_experts(rz, router, p_up, p_down, ro, choice, weight, ws, TOKENS, DIM, INNER, EXPERTS, TOP_K, 1.5f, s), AR_OK);
    AR_IS(ar_w4_experts(rz, router, p_up, p_down, ro, choice, weight, 0, TOKENS, DIM, INNER, EXPERTS, TOP_K, 1.5f, s), AR_EINVAL);
    HIP_OK(hipStreamSynchronize(s));

    f = fopen(argv[2], "wb");
    if (!f) return 1;
    if (!save(f, h, 2 * ROWS) || !save(f, z, 2 * ROWS) || !save(f, dx, 2 * ROWS) || !save(f, dy, 2 * ROWS) || !save(f, sums, 12 * DIM) ||
        !save(f, back, 2 * OUT * DIM) || !save(f, y, 2 * TOKENS * OUT) || !save(f, out, 2 * ROWS) || !save(f, choice, 4 * TOKENS * TOP_K) ||
        !save(f, weight, 4 * TOKENS * TOP_K))
        return 2;
    fclose(f);
    HIP_OK(hipStreamDestroy(s));
    HIP_OK(hipFree(m));
    free(in);
    return 0;
}
