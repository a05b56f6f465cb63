/*
 * Hardware self-checks for the sm_103a building blocks of the attention
 * kernels (libfa_selftest.so). These are not part of the attention method;
 * they isolate one fact each so that a failing attention parity test can be
 * traced to a tcgen05 operand layout or to the bounded-wait machinery.
 */
#ifndef IO_AWARE_EXACT_FA_SELFTEST_H
#define IO_AWARE_EXACT_FA_SELFTEST_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FA_SELFTEST_A_MN 1   /* A stored [K][128] (M contiguous) instead of [128][K] */
#define FA_SELFTEST_B_MN 2   /* B stored [K][N] (N contiguous) instead of [N][K] */
#define FA_SELFTEST_A_TMEM 4 /* A copied to tensor memory, read by the MMA from there ([128][K] storage) */

/* d[128][N] (fp32, device) = A (128 x K) * B (K x N), one CTA, bf16 operands
 * in device memory (16-byte aligned), N and K in {64, 128}. The layouts are
 * selected by `mode` as above. `status` is a device int[4], zeroed by the
 * caller; a wait that runs out writes FA_ERR_TIMEOUT there. */
FA_API int fa_selftest_mma(const void* a, const void* b, float* d, int N, int K, int mode, int* status,
                    fa_stream_t stream);

/* The same in 8 bits, D[128 x N] (fp32): a is e4m3, b e4m3 or (e5m2 = 1) e5m2, b stored
 * [N][K]. a_mn = 0: a stored [128][d], K = d; a_mn = 1: a stored [128][d] as well, but
 * taken as K rows of d elements of M (rows d and up of D mean nothing), K = 128.
 * d = 64 or 128 (64- or 128-byte swizzle); N a multiple of 16, at most 256.
 * b_mn: 0, or (a_mn = 1) the bytes of a row, 64 or 128, of b stored [128][b_mn], of which
 * the N from b_from (a multiple of 16) are taken. */
FA_API int fa_selftest_mma8(const void* a, const void* b, float* d_out, int N, int d, int a_mn, int e5m2, int b_mn,
                            int b_from, int* status, fa_stream_t stream);

/* Launches one thread that waits on a shared-memory barrier nothing arrives
 * on, with a limit of limit_us microseconds (1 .. 5e6). Afterwards status[0]
 * (device int[4], zeroed by the caller) must read FA_ERR_TIMEOUT. */
FA_API int fa_selftest_wait_timeout(int* status, unsigned int limit_us, fa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif
