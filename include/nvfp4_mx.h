/*
 * nvfp4_mx.h -- MXFP4: the 4-bit format whose block scales gfx950's matrix
 * instructions take themselves, with its quantizers, product and
 * routed-expert layer.  Part of the C ABI of nvfp4.h, which includes this
 * file; the conventions there (device pointers, bf16 as uint16_t patterns,
 * tensors 16-byte aligned, checks on the host before any HIP call, stream
 * order, status codes, zero-sized problems) hold here too.
 *
 * MXFP4 (OCP Microscaling Formats 1.0): E2M1 codes packed as in NVFP4 (two a
 * byte, the even element in the low nibble), one E8M0 byte s per 32
 * consecutive elements along a row, worth 2^(s - 127) (255: NaN), no global
 * scale.  A value decodes as q * 2^(s - 127), which bf16 holds exactly.
 * Encoding: s - 127 = floor(log2(largest magnitude)) - 2, at least -127
 * (which a block of zeros gets); codes round x / 2^(s - 127) to nearest,
 * ties to the even code, saturating at 6, and keep the sign.  A block that
 * holds an infinity or a NaN gets s = 255: all of it decodes as NaN.
 */
#ifndef NVFP4_MX_H
#define NVFP4_MX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Quantize and dequantize.
 * nvfp4_mx_quantize: x bf16 [rows, cols] -> codes [rows, cols/2], scales
 * [rows, cols/32].  cols % 32 == 0 (else SHAPE).
 * nvfp4_mx_quantize_columnwise: the MXFP4 of x^T, blocks along rows: codes_t
 * [cols, rows/2], scales_t [cols, rows/32].  rows % 32 == 0 (else SHAPE),
 * any cols.  It packs the operands of a linear layer's gradients: with dY
 * [M, N], X [M, K] and W [N, K], dX = dY W is the product of dY's rows with
 * W's columnwise copy, and dW = dY^T X that of both columnwise copies.
 * nvfp4_mx_dequantize: y[r, c] = q * 2^(s - 127) as bf16, exact (finite
 * values past bf16's range become infinities).
 * No workspace.  Outputs are bit-identical to the definition above.
 * ------------------------------------------------------------------------ */
int32_t nvfp4_mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                          void* stream);
int32_t nvfp4_mx_quantize_columnwise(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t,
                                     uint8_t* scales_t, void* stream);
int32_t nvfp4_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* y,
                            void* stream);

/* ------------------------------------------------------------------------
 * Product of two MXFP4 operands, K innermost on both:
 *   y[m, n] = bf16( sum_k a[m, k] * w[n, k] ), fp32 accumulation.
 * nvfp4_mx_gemm_packed: a_codes [M, K/2], a_scales [M, K/32]; w_codes
 * [N, K/2], w_scales [N, K/32]; y bf16 [M, N].
 * nvfp4_mx_gemm: the same on nvfp4_mx_quantize of x bf16 [M, K], quantized
 * within the call.
 * K % 32 == 0 and K > 0 (else SHAPE), any M and N; K < 2^24, M < 2^30, N <
 * 2^28 and M * N <= 2^36 (else UNSUPPORTED).  Workspace: the sizes below (0:
 * none, and then workspace may be NULL).
 * ------------------------------------------------------------------------ */
size_t nvfp4_mx_gemm_workspace_size(int64_t M, int64_t N, int64_t K);
int32_t nvfp4_mx_gemm(const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                      const uint8_t* w_scales, uint16_t* y, void* workspace, size_t workspace_bytes, void* stream);
size_t nvfp4_mx_gemm_packed_workspace_size(int64_t M, int64_t N, int64_t K);
int32_t nvfp4_mx_gemm_packed(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M, int64_t N, int64_t K,
                             const uint8_t* w_codes, const uint8_t* w_scales, uint16_t* y, void* workspace,
                             size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * Routed-expert layer with MXFP4 experts and activations.  For each token t
 * and slot j < top_k with expert e = topk_ids[t, j] (slots whose id lies
 * outside [0, E) are skipped, as nvfp4_moe_gate leaves them):
 *   x^ = MXFP4(x[t]);  [g | u] = x^ * W13_e^T  (gate rows 0..I-1, then up)
 *   h = bf16(silu(g) * u);  h^ = MXFP4(h)
 *   out[t] = bf16( sum_j topk_weights[t, j] * (h^ * W2_e^T) )
 * products and sums in fp32, slots in order; a token without a slot gets 0.
 * x bf16 [T, H]; topk_ids int32 [T, top_k]; topk_weights fp32 [T, top_k];
 * w13_codes [E, 2I, H/2], w13_scales [E, 2I, H/32]; w2_codes [E, H, I/2],
 * w2_scales [E, H, I/32]; out bf16 [T, H].
 * H % 32 == 0 and I % 32 == 0 (else SHAPE); E <= 4096, T * top_k <= 2^30
 * and every operand that the products read below 2 GiB (T * H / 2,
 * T * top_k * I / 2, the codes of one expert's W13 and W2), else
 * UNSUPPORTED.  Workspace: nvfp4_mx_moe_workspace_size(p) bytes.
 * ------------------------------------------------------------------------ */
typedef struct nvfp4_mx_moe_problem {
    int64_t T;      /* tokens */
    int64_t E;      /* routed experts */
    int64_t top_k;  /* experts per token */
    int64_t H;      /* hidden size */
    int64_t I;      /* expert intermediate size */
} nvfp4_mx_moe_problem;

typedef struct nvfp4_mx_moe_tensors {
    const uint16_t* x;
    const int32_t* topk_ids;
    const float* topk_weights;
    const uint8_t* w13_codes;
    const uint8_t* w13_scales;
    const uint8_t* w2_codes;
    const uint8_t* w2_scales;
    uint16_t* out;
} nvfp4_mx_moe_tensors;

size_t nvfp4_mx_moe_workspace_size(const nvfp4_mx_moe_problem* p);
int32_t nvfp4_mx_moe(const nvfp4_mx_moe_problem* p, const nvfp4_mx_moe_tensors* t, void* workspace,
                     size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_MX_H */
