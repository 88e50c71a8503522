/*
 * nvfp4_gate.h -- the expert gate in front of the routed-expert layers, and
 * its gradient.  Part of the C ABI of nvfp4.h, which includes this file; the
 * conventions there (device pointers, checks on the host before any HIP
 * call, stream order, status codes, zero-sized problems) hold here too.
 */
#ifndef NVFP4_GATE_H
#define NVFP4_GATE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define NVFP4_GATE_F32 0  /* logits (and their gradient) fp32 */
#define NVFP4_GATE_BF16 1 /* ... bf16 */

#define NVFP4_GATE_SOFTMAX 0
#define NVFP4_GATE_SIGMOID 1

/* ------------------------------------------------------------------------
 * For every token t, with l_e = logits[t, e]:
 *   candidates  experts with l_e > -inf (NaN is none) and, with a bias, a
 *               choice value > -inf; l_e = +inf counts as the largest
 *               finite fp32.
 *   score       s = softmax(l) over the row, or s_e = sigmoid(l_e).
 *   choice      c_e = l_e when there is no bias and group_top = 1 (both
 *               scores grow with the logit), else s_e + bias_e in 64 bits.
 *   groups      n_group > 1: the experts form n_group runs of E / n_group;
 *               a run's rank is the sum of its group_top (1 or 2) largest
 *               choice values (of those it has) and only the topk_group
 *               highest-ranked runs keep their candidates.
 *   ids         the top_k candidates of largest choice value, in that order.
 *   weights     scale * s_id, or with renormalize scale * s_id / (sum of the
 *               selected s).
 * Ties, between experts and between runs, go to the lower index.  A row with
 * fewer candidates than top_k fills its last slots with id -1 and weight 0,
 * which the routed-expert layers skip.
 *
 * logits fp32 or bf16 [T, E]; bias fp32 [E] or NULL (enters the choice only,
 * so it has no gradient); ids int32 [T, top_k]; weights fp32 [T, top_k].
 * SHAPE: T < 0, E < 1, top_k < 1, n_group < 1 or not dividing E, topk_group
 * outside [1, n_group], top_k > topk_group * (E / n_group), group_top not 1
 * or 2, a score or dtype outside the values above, a scale that is not
 * finite or not > 0.  UNSUPPORTED: E > 4096, top_k > 64, T >= 2^26.
 * logits are 16-byte aligned, the other arrays 4-byte.  No workspace; the
 * choice needs no host round trip.  ids do not depend on how the sums of the
 * weights are rounded.
 * ------------------------------------------------------------------------ */
typedef struct nvfp4_gate_config {
    int64_t T;             /* tokens */
    int64_t E;             /* experts */
    int64_t top_k;         /* experts per token */
    int64_t n_group;       /* runs of experts (1: none) */
    int64_t topk_group;    /* runs kept */
    int32_t group_top;     /* choice values in a run's rank: 1 or 2 */
    int32_t score;         /* NVFP4_GATE_SOFTMAX or NVFP4_GATE_SIGMOID */
    int32_t renormalize;   /* 0 or 1 */
    int32_t logits_dtype;  /* NVFP4_GATE_F32 or NVFP4_GATE_BF16 */
    float scale;
} nvfp4_gate_config;

int32_t nvfp4_moe_gate(const nvfp4_gate_config* c, const void* logits, const float* bias, int32_t* ids,
                       float* weights, void* stream);

/* ------------------------------------------------------------------------
 * The gradient of the weights with respect to the logits, at the ids that
 * the forward call chose (the choice itself has none):
 *   softmax                 dl_e = p_e * (scale [e selected] dw_e - D)
 *   softmax, renormalized   dl_e = w_e * (dw_e - D / scale)
 *   sigmoid                 dl_e = w_e * (1 - s_e) * dw_e
 *   sigmoid, renormalized   dl_e = w_e * (1 - s_e) * (dw_e - D / scale)
 * with D = sum over the selected of w dw, and 0 for every expert the formula
 * does not reach.  logits, ids, dweights fp32 [T, top_k] as in the forward
 * call; dlogits [T, E] in the type of the logits, rounded once.  Slots whose
 * id lies outside [0, E), or whose logit is no candidate, take no part; an
 * id that a row names twice counts once per slot.  Of the config T, E,
 * top_k, score, renormalize, logits_dtype and scale are read.  Limits,
 * alignment (dlogits as logits) as above.
 * ------------------------------------------------------------------------ */
int32_t nvfp4_moe_gate_backward(const nvfp4_gate_config* c, const void* logits, const int32_t* ids,
                                const float* dweights, void* dlogits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GATE_H */
