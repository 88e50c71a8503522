// mx_api.cpp -- the C ABI of include/nvfp4_gate.h and include/nvfp4_mx.h:
// argument checks on the host, workspace layout, and the launch sequence of
// each entry point.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "mx_internal.hpp"

using namespace nvfp4;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
template <typename T>
T* at(void* base, size_t off) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(base) + off);
}

// --------------------------------------------------------------------- gate --

int32_t check_gate(const nvfp4_gate_config* c, bool backward) {
    if (!c) return api_fail(NVFP4_ERR_NULL_ARG, "moe_gate: a config is required");
    if (c->T < 0 || c->E < 1 || c->top_k < 1 || c->top_k > c->E || (c->score != 0 && c->score != 1) ||
        (c->logits_dtype != 0 && c->logits_dtype != 1) || (c->renormalize != 0 && c->renormalize != 1) ||
        !std::isfinite(c->scale) || !(c->scale > 0.0f))
        return api_fail(NVFP4_ERR_SHAPE,
                        "moe_gate: need T >= 0, 1 <= top_k <= E, a known score and dtype, renormalize 0 or 1 and a "
                        "finite scale > 0");
    if (!backward) {
        if (c->n_group < 1 || c->n_group > c->E || c->E % c->n_group != 0 || c->topk_group < 1 ||
            c->topk_group > c->n_group || (c->group_top != 1 && c->group_top != 2) ||
            c->top_k > c->topk_group * (c->E / c->n_group))
            return api_fail(NVFP4_ERR_SHAPE,
                            "moe_gate: n_group divides E, 1 <= topk_group <= n_group, group_top is 1 or 2 and the "
                            "kept groups hold at least top_k experts");
    }
    if (c->E > 4096 || c->top_k > 64 || c->T >= ((int64_t)1 << 26))
        return api_fail(NVFP4_ERR_UNSUPPORTED, "moe_gate: at most 4096 experts, top_k 64 and 2^26 - 1 tokens");
    return NVFP4_OK;
}

// ---------------------------------------------------------------- product --

int32_t check_product(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K <= 0 || K % 32 != 0)
        return api_fail(NVFP4_ERR_SHAPE, "mx_gemm: need M, N >= 0, K > 0 and K % 32 == 0");
    // (few rows: a workgroup of 256 threads for 32 or more columns, where N is large)
    if (K >= ((int64_t)1 << 24) || M >= ((int64_t)1 << 30) || N >= ((int64_t)1 << 28) ||
        (N > 0 && M > (((int64_t)1 << 36) / N)))
        return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_gemm: K below 2^24, M below 2^30, N below 2^28, M * N up to 2^36");
    return NVFP4_OK;
}

// A bf16 activation that the streaming kernel quantizes itself.
bool one_launch(int64_t M, int64_t N, int64_t K) { return mx_stream_takes(M, N, K) && mx_stream_quantizes(M, K); }

size_t partial_bytes(int64_t M, int64_t N, int64_t K) {
    int steps;
    const int splits = mx_stream_takes(M, N, K) ? 1 : mx_gemm_splits(M, N, K, &steps);
    return splits > 1 ? align_up((size_t)splits * (size_t)(M * N) * 4) : 0;
}

hipError_t run_product(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M, int64_t N, int64_t K,
                       const uint8_t* w_codes, const uint8_t* w_scales, uint16_t* y, float* partial, hipStream_t s) {
    if (mx_stream_takes(M, N, K)) {
        MxStreamArgs g;
        g.a_codes = a_codes;
        g.a_scales = a_scales;
        g.b_codes = w_codes;
        g.b_scales = w_scales;
        g.M = M;
        g.N = N;
        g.K = K;
        g.y = y;
        return launch_mx_stream(g, s);
    }
    MxGemmArgs g;
    g.a_codes = a_codes;
    g.a_scales = a_scales;
    g.b_codes = w_codes;
    g.b_scales = w_scales;
    g.M = M;
    g.N = N;
    g.K = K;
    g.out = y;
    g.ldo = N;
    if (partial_bytes(M, N, K) > 0) return launch_mx_gemm_split(g, partial, s);
    return launch_mx_gemm(g, MxEpi::kStoreBf16, 0, s);
}

size_t packed_codes_bytes(int64_t rows, int64_t cols) { return align_up((size_t)(rows * (cols / 2))); }
size_t packed_scales_bytes(int64_t rows, int64_t cols) { return align_up((size_t)(rows * (cols / 32))); }

// ---------------------------------------------------------------- experts --

struct MxMoeLayout {
    size_t row_off = 0, tile_off = 0, perm = 0, inv = 0, pos_group = 0, route = 0;
    size_t xc = 0, xs = 0, hc = 0, hs = 0, y = 0, total = 0;
};

// How the layer runs: slot by slot (no sorting, two launches) while few slots
// can meet on an expert, else sorted by expert, in row tiles of 16 on the
// streaming kernel or of kMxMoeBM on the LDS tiles.  Measured on MI355X (us,
// slots / 16 rows / LDS tiles), E experts of H x I, uniform routing:
//   E = 256, 6144 x 2048, top 8   4 tokens 121 / 140 / 153, 8: 240 / 240 / 266,
//     64: 1761 / 838 / 842, 128: - / 1009 / 980, 512: - / 1441 / 1040
//   256, 2048 x 1024, top 8       8: 52 / 59 / 83, 16: 91 / 88 / 121,
//     256: - / 202 / 223, 512: - / 276 / 233
//   64, 2048 x 1408, top 6        4: 30 / 36 / 59, 8: 50 / 50 / 84,
//     128: - / 84 / 105, 256: - / 126 / 108
//   32, 2048 x 1024, top 4        8: 32 / 29 / 52, 128: - / 49 / 62,
//     256: - / 68 / 64
//   8, 4096 x 2048, top 2         4: 28 / 33 / 51, 8: 50 / 36 / 60,
//     64: - / 47 / 62, 128: - / 66 / 64
enum class MoePlan { kSlots, kStream, kTiles };
MoePlan plan_mx_moe(const nvfp4_mx_moe_problem& p) {
    const int64_t S = p.T * p.top_k, expert = p.I * p.H / 2 * 3;  // an expert's codes, in bytes
    // Two slots of different tokens share an expert about S (S - top_k) / 2E
    // times, and its second reading costs more than sorting does from about 55 MB
    // on.
    if (S <= 128 && mx_slots_fit(p.H) && S * (S - p.top_k) * expert <= p.E * 110000000) return MoePlan::kSlots;
    // Beyond 16 rows the streaming kernel reads an expert again, out of the
    // caches while all of them are small.
    return S <= p.E * std::min<int64_t>(24, 3 + ((int64_t)1 << 32) / (p.E * expert)) ? MoePlan::kStream
                                                                                    : MoePlan::kTiles;
}

MxMoeLayout layout_mx_moe(const nvfp4_mx_moe_problem& p) {
    MxMoeLayout l;
    const int64_t S = p.T * p.top_k;
    size_t off = 0;
    if (plan_mx_moe(p) == MoePlan::kSlots) {
        l.hc = off; off += packed_codes_bytes(S, p.I);
        l.hs = off; off += packed_scales_bytes(S, p.I);
        l.total = off;
        return l;
    }
    l.row_off = off; off += align_up((size_t)(p.E + 1) * 4);
    l.tile_off = off; off += align_up((size_t)(p.E + 1) * 4);
    l.perm = off; off += align_up((size_t)S * 4);
    l.inv = off; off += align_up((size_t)S * 4);
    if (S > kMxPrepareSlots) {
        l.pos_group = off; off += align_up((size_t)S * 4);
        l.route = off; off += align_up(moe_route_scratch_bytes(S, (int32_t)p.E));
    }
    l.xc = off; off += packed_codes_bytes(p.T, p.H);
    l.xs = off; off += packed_scales_bytes(p.T, p.H);
    l.hc = off; off += packed_codes_bytes(S, p.I);
    l.hs = off; off += packed_scales_bytes(S, p.I);
    l.y = off; off += align_up((size_t)S * (size_t)p.H * 4);
    l.total = off;
    return l;
}

int32_t check_mx_moe(const nvfp4_mx_moe_problem* p) {
    if (!p) return api_fail(NVFP4_ERR_NULL_ARG, "mx_moe: a problem is required");
    if (p->T < 0 || p->E <= 0 || p->top_k <= 0 || p->H <= 0 || p->I <= 0 || p->H % 32 || p->I % 32)
        return api_fail(NVFP4_ERR_SHAPE, "mx_moe: need T >= 0, E, top_k, H, I > 0, H and I multiples of 32");
    constexpr int64_t kBytes = kMaxOperandBytes, kSlots = (int64_t)1 << 30;
    if (p->E > 4096 || p->T > kSlots || p->top_k > kSlots || p->T * p->top_k > kSlots)
        return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_moe: at most 4096 experts and 2^30 slots");
    const int64_t S = p->T * p->top_k;
    if (p->H >= kBytes || p->I >= kBytes || p->T * (p->H / 2) >= kBytes || S * (p->I / 2) >= kBytes ||
        p->I * p->H >= kBytes)
        return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_moe: an operand of 2 GiB or more");
    // workgroups of the grouped products: fewer than 2^32 threads in all (256 each;
    // the streaming forms: row tiles of 16, 32 columns of h or 16 of H)
    const int64_t mt = S / kMxMoeBM + p->E + 1, nt = std::max(p->I / 64, p->H / 128) + 1;
    const int64_t ms = std::min(S, 16 * p->E) / 16 + p->E + 64, ns = std::max(p->I / 32, p->H / 16) + 1;
    if (mt * nt >= ((int64_t)1 << 24) || ms * ns >= ((int64_t)1 << 23))
        return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_moe: too many tiles");
    return NVFP4_OK;
}

}  // namespace

extern "C" {

int32_t nvfp4_moe_gate(const nvfp4_gate_config* c, const void* logits, const float* bias, int32_t* ids,
                       float* weights, void* stream) {
    api_clear();
    if (int32_t st = check_gate(c, false)) return st;
    if (c->T == 0) return NVFP4_OK;
    if (!logits || !ids || !weights) return api_fail(NVFP4_ERR_NULL_ARG, "moe_gate: logits, ids and weights are required");
    if (!aligned16(logits) || (bias && !aligned4(bias)) || !aligned4(ids) || !aligned4(weights))
        return api_fail(NVFP4_ERR_ALIGN, "moe_gate: logits must be 16-byte aligned, the other arrays 4-byte");
    return api_hip(launch_gate(*c, logits, bias, ids, weights, as_stream(stream)), "moe_gate");
}

int32_t nvfp4_moe_gate_backward(const nvfp4_gate_config* c, const void* logits, const int32_t* ids,
                                const float* dweights, void* dlogits, void* stream) {
    api_clear();
    if (int32_t st = check_gate(c, true)) return st;
    if (c->T == 0) return NVFP4_OK;
    if (!logits || !ids || !dweights || !dlogits)
        return api_fail(NVFP4_ERR_NULL_ARG, "moe_gate_backward: logits, ids, dweights and dlogits are required");
    if (!aligned16(logits) || !aligned16(dlogits) || !aligned4(ids) || !aligned4(dweights))
        return api_fail(NVFP4_ERR_ALIGN,
                        "moe_gate_backward: logits and dlogits must be 16-byte aligned, the other arrays 4-byte");
    return api_hip(launch_gate_backward(*c, logits, ids, dweights, dlogits, as_stream(stream)), "moe_gate_backward");
}

int32_t nvfp4_mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                          void* stream) {
    api_clear();
    if (rows < 0 || cols <= 0 || cols % 32 != 0)
        return api_fail(NVFP4_ERR_SHAPE, "mx_quantize: need rows >= 0, cols > 0 and cols % 32 == 0");
    if (!mx_quantize_fits(rows, cols)) return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_quantize: more than 2^37 elements");
    if (rows == 0) return NVFP4_OK;
    if (!x || !codes || !scales) return api_fail(NVFP4_ERR_NULL_ARG, "mx_quantize: x, codes and scales are required");
    if (!aligned16(x) || !aligned16(codes) || !aligned16(scales))
        return api_fail(NVFP4_ERR_ALIGN, "mx_quantize: pointers must be 16-byte aligned");
    return api_hip(launch_mx_quantize(x, rows, cols, codes, scales, as_stream(stream)), "mx_quantize");
}

int32_t nvfp4_mx_quantize_columnwise(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t,
                                     uint8_t* scales_t, void* stream) {
    api_clear();
    if (rows < 0 || cols < 0 || rows % 32 != 0)
        return api_fail(NVFP4_ERR_SHAPE, "mx_quantize_columnwise: need rows, cols >= 0 and rows % 32 == 0");
    if (!mx_quantize_cols_fits(rows, cols))
        return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_quantize_columnwise: more than 2^24 tiles of 256 x 64");
    if (rows == 0 || cols == 0) return NVFP4_OK;
    if (!x || !codes_t || !scales_t)
        return api_fail(NVFP4_ERR_NULL_ARG, "mx_quantize_columnwise: x, codes_t and scales_t are required");
    if (!aligned16(x) || !aligned16(codes_t) || !aligned16(scales_t))
        return api_fail(NVFP4_ERR_ALIGN, "mx_quantize_columnwise: pointers must be 16-byte aligned");
    return api_hip(launch_mx_quantize_cols(x, rows, cols, codes_t, scales_t, as_stream(stream)),
                   "mx_quantize_columnwise");
}

int32_t nvfp4_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* y,
                            void* stream) {
    api_clear();
    if (rows < 0 || cols <= 0 || cols % 32 != 0)
        return api_fail(NVFP4_ERR_SHAPE, "mx_dequantize: need rows >= 0, cols > 0 and cols % 32 == 0");
    if (!mx_quantize_fits(rows, cols)) return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_dequantize: more than 2^37 elements");
    if (rows == 0) return NVFP4_OK;
    if (!codes || !scales || !y) return api_fail(NVFP4_ERR_NULL_ARG, "mx_dequantize: codes, scales and y are required");
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(y))
        return api_fail(NVFP4_ERR_ALIGN, "mx_dequantize: pointers must be 16-byte aligned");
    return api_hip(launch_mx_dequantize(codes, scales, rows, cols, y, as_stream(stream)), "mx_dequantize");
}

size_t nvfp4_mx_gemm_packed_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || check_product(M, N, K) != NVFP4_OK) return 0;
    return partial_bytes(M, N, K);
}

int32_t nvfp4_mx_gemm_packed(const uint8_t* a_codes, const uint8_t* a_scales, int64_t M, int64_t N, int64_t K,
                             const uint8_t* w_codes, const uint8_t* w_scales, uint16_t* y, void* workspace,
                             size_t workspace_bytes, void* stream) {
    api_clear();
    if (int32_t st = check_product(M, N, K)) return st;
    if (M == 0 || N == 0) return NVFP4_OK;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !y)
        return api_fail(NVFP4_ERR_NULL_ARG, "mx_gemm_packed: both operands and y are required");
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        (workspace && !aligned16(workspace)))
        return api_fail(NVFP4_ERR_ALIGN, "mx_gemm_packed: pointers must be 16-byte aligned");
    const size_t need = nvfp4_mx_gemm_packed_workspace_size(M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return api_fail(NVFP4_ERR_WORKSPACE, "mx_gemm_packed: workspace smaller than nvfp4_mx_gemm_packed_workspace_size");
    return api_hip(run_product(a_codes, a_scales, M, N, K, w_codes, w_scales, y, at<float>(workspace, 0),
                               as_stream(stream)),
                   "mx_gemm_packed");
}

size_t nvfp4_mx_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || check_product(M, N, K) != NVFP4_OK) return 0;
    if (one_launch(M, N, K)) return 0;
    return packed_codes_bytes(M, K) + packed_scales_bytes(M, K) + partial_bytes(M, N, K);
}

int32_t nvfp4_mx_gemm(const uint16_t* x, int64_t M, int64_t N, int64_t K, const uint8_t* w_codes,
                      const uint8_t* w_scales, uint16_t* y, void* workspace, size_t workspace_bytes, void* stream) {
    api_clear();
    if (int32_t st = check_product(M, N, K)) return st;
    if (!mx_quantize_fits(M, K)) return api_fail(NVFP4_ERR_UNSUPPORTED, "mx_gemm: more than 2^37 activations");
    if (M == 0 || N == 0) return NVFP4_OK;
    if (!x || !w_codes || !w_scales || !y) return api_fail(NVFP4_ERR_NULL_ARG, "mx_gemm: x, weights and y are required");
    if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        (workspace && !aligned16(workspace)))
        return api_fail(NVFP4_ERR_ALIGN, "mx_gemm: pointers must be 16-byte aligned");
    const size_t need = nvfp4_mx_gemm_workspace_size(M, N, K);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return api_fail(NVFP4_ERR_WORKSPACE, "mx_gemm: workspace smaller than nvfp4_mx_gemm_workspace_size");
    hipStream_t s = as_stream(stream);
    if (one_launch(M, N, K)) {
        MxStreamArgs g;
        g.x = x;
        g.b_codes = w_codes;
        g.b_scales = w_scales;
        g.M = M;
        g.N = N;
        g.K = K;
        g.y = y;
        return api_hip(launch_mx_stream(g, s), "mx_gemm stream");
    }
    uint8_t* const xc = at<uint8_t>(workspace, 0);
    uint8_t* const xs = at<uint8_t>(workspace, packed_codes_bytes(M, K));
    if (int32_t st = api_hip(launch_mx_quantize(x, M, K, xc, xs, s), "mx_gemm quantize")) return st;
    float* const partial = at<float>(workspace, packed_codes_bytes(M, K) + packed_scales_bytes(M, K));
    return api_hip(run_product(xc, xs, M, N, K, w_codes, w_scales, y, partial, s), "mx_gemm");
}

size_t nvfp4_mx_moe_workspace_size(const nvfp4_mx_moe_problem* p) {
    if (check_mx_moe(p) != NVFP4_OK || p->T == 0) return 0;
    return layout_mx_moe(*p).total;
}

int32_t nvfp4_mx_moe(const nvfp4_mx_moe_problem* p, const nvfp4_mx_moe_tensors* t, void* workspace,
                     size_t workspace_bytes, void* stream) {
    api_clear();
    if (!p || !t) return api_fail(NVFP4_ERR_NULL_ARG, "mx_moe: problem and tensors are required");
    if (int32_t st = check_mx_moe(p)) return st;
    if (p->T == 0) return NVFP4_OK;
    if (!t->x || !t->topk_ids || !t->topk_weights || !t->w13_codes || !t->w13_scales || !t->w2_codes ||
        !t->w2_scales || !t->out)
        return api_fail(NVFP4_ERR_NULL_ARG, "mx_moe: a required tensor is NULL");
    const void* tensors[] = {t->x, t->w13_codes, t->w13_scales, t->w2_codes, t->w2_scales, t->out};
    for (const void* q : tensors)
        if (!aligned16(q)) return api_fail(NVFP4_ERR_ALIGN, "mx_moe: tensor pointers must be 16-byte aligned");
    if (!aligned4(t->topk_ids) || !aligned4(t->topk_weights))
        return api_fail(NVFP4_ERR_ALIGN, "mx_moe: ids and weights must be 4-byte aligned");
    if (workspace && !aligned16(workspace)) return api_fail(NVFP4_ERR_ALIGN, "mx_moe: workspace must be 16-byte aligned");
    const MxMoeLayout l = layout_mx_moe(*p);
    if (!workspace || workspace_bytes < l.total)
        return api_fail(NVFP4_ERR_WORKSPACE, "mx_moe: workspace smaller than nvfp4_mx_moe_workspace_size");

    hipStream_t s = as_stream(stream);
    const int64_t S = p->T * p->top_k;
    const int32_t E = (int32_t)p->E;
    const MoePlan plan = plan_mx_moe(*p);
    MxStreamArgs up, down;
    up.b_codes = t->w13_codes;
    up.b_scales = t->w13_scales;
    up.M = S;
    up.N = 2 * p->I;
    up.K = p->H;
    up.E = down.E = E;
    up.top_k = down.top_k = (int32_t)p->top_k;
    up.h_codes = at<uint8_t>(workspace, l.hc);
    up.h_scales = at<uint8_t>(workspace, l.hs);
    down.a_codes = up.h_codes;
    down.a_scales = up.h_scales;
    down.b_codes = t->w2_codes;
    down.b_scales = t->w2_scales;
    down.M = S;
    down.N = p->H;
    down.K = p->I;
    if (plan == MoePlan::kSlots) {
        up.x = t->x;
        up.ids = down.ids = t->topk_ids;
        down.slot_w = t->topk_weights;
        down.y = t->out;
        if (int32_t e = api_hip(launch_mx_slot_up(up, S, s), "mx_moe gate/up")) return e;
        return api_hip(launch_mx_slot_down(down, p->T, s), "mx_moe down");
    }
    const int bm = plan == MoePlan::kStream ? 16 : kMxMoeBM;
    int32_t* row_off = at<int32_t>(workspace, l.row_off);
    int32_t* tile_off = at<int32_t>(workspace, l.tile_off);
    int32_t* perm = at<int32_t>(workspace, l.perm);
    int32_t* inv = at<int32_t>(workspace, l.inv);
    uint8_t* xc = at<uint8_t>(workspace, l.xc);
    uint8_t* xs = at<uint8_t>(workspace, l.xs);
    uint8_t* hc = at<uint8_t>(workspace, l.hc);
    uint8_t* hs = at<uint8_t>(workspace, l.hs);
    float* Y = at<float>(workspace, l.y);
    int32_t st;
    if (S <= kMxPrepareSlots) {
        const MxPrepareArgs a = {t->topk_ids, (int32_t)S, E, bm, row_off, tile_off, perm, inv, t->x, p->T * (p->H / 8),
                                 xc, xs};
        st = api_hip(launch_mx_prepare(a, s), "mx_moe prepare");
        if (st) return st;
    } else {
        st = api_hip(launch_moe_route(t->topk_ids, S, E, bm, row_off, tile_off, perm, inv,
                                      at<int32_t>(workspace, l.pos_group), at<int32_t>(workspace, l.route), s),
                     "mx_moe route");
        if (st) return st;
        st = api_hip(launch_mx_quantize(t->x, p->T, p->H, xc, xs, s), "mx_moe quantize");
        if (st) return st;
    }
    const int grid_m = (int)((S + bm - 1) / bm + std::min<int64_t>(E, S));
    if (plan == MoePlan::kStream) {
        up.a_codes = xc;
        up.a_scales = xs;
        up.perm = perm;
        up.row_off = down.row_off = row_off;
        up.tile_off = down.tile_off = tile_off;
        down.slot_y = Y;
        st = api_hip(launch_mx_group_up(up, grid_m, s), "mx_moe gate/up");
        if (st) return st;
        st = api_hip(launch_mx_group_down(down, grid_m, s), "mx_moe down");
        if (st) return st;
        return api_hip(launch_mx_combine(Y, inv, t->topk_weights, p->T, (int32_t)p->top_k, p->H, t->out, s),
                       "mx_moe combine");
    }
    MxGemmArgs g1;
    g1.a_codes = xc;
    g1.a_scales = xs;
    g1.a_rows = perm;
    g1.a_div = (int32_t)p->top_k;
    g1.a_src_rows = p->T;
    g1.b_codes = t->w13_codes;
    g1.b_scales = t->w13_scales;
    g1.M = S;
    g1.N = 2 * p->I;
    g1.K = p->H;
    g1.row_off = row_off;
    g1.tile_off = tile_off;
    g1.groups = E;
    g1.out = hc;
    g1.out_scales = hs;
    g1.ldo = p->I;
    st = api_hip(launch_mx_gemm(g1, MxEpi::kGateUp, grid_m, s), "mx_moe gate/up");
    if (st) return st;
    MxGemmArgs g2;
    g2.a_codes = hc;
    g2.a_scales = hs;
    g2.a_src_rows = S;
    g2.b_codes = t->w2_codes;
    g2.b_scales = t->w2_scales;
    g2.M = S;
    g2.N = p->H;
    g2.K = p->I;
    g2.row_off = row_off;
    g2.tile_off = tile_off;
    g2.groups = E;
    g2.out = Y;
    g2.ldo = p->H;
    st = api_hip(launch_mx_gemm(g2, MxEpi::kStoreF32, grid_m, s), "mx_moe down");
    if (st) return st;
    return api_hip(launch_mx_combine(Y, inv, t->topk_weights, p->T, (int32_t)p->top_k, p->H, t->out, s),
                   "mx_moe combine");
}

}  // extern "C"
