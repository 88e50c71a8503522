// mx_internal.hpp -- launchers of the MXFP4 and gate kernels, shared between
// the C ABI (mx_api.cpp) and the kernel translation units.
#pragma once

#include "nvfp4.h"
#include "nvfp4_internal.hpp"

namespace nvfp4 {

// ------------------------------------------------------------ quantization --

// Whether a tensor's flat pass (tile grid) fits one launch.
bool mx_quantize_fits(int64_t rows, int64_t cols);
bool mx_quantize_cols_fits(int64_t rows, int64_t cols);
hipError_t launch_mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream);
hipError_t launch_mx_quantize_cols(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t, uint8_t* scales_t,
                                   hipStream_t stream);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* y,
                                hipStream_t stream);

// ---------------------------------------------------------------- products --

enum class MxEpi : int {
    kStoreBf16 = 0,  // y = bf16(acc)
    kGateUp = 1,     // h = bf16(silu(g) * u), stored as MXFP4
    kPartialF32 = 2, // partial[split] = acc (K split, joined afterwards)
    kStoreF32 = 3,   // y = acc (grouped: slot outputs, summed afterwards)
};

struct MxGemmArgs {
    const uint8_t* a_codes = nullptr;   // activation [*, K/2] (gathered when a_rows is set)
    const uint8_t* a_scales = nullptr;  // [*, K/32]
    const int32_t* a_rows = nullptr;    // A row of output row r = a_rows[r] / a_div
    int32_t a_div = 1;
    int64_t a_src_rows = 0;             // rows of the source tensor (gathered operands)
    const uint8_t* b_codes = nullptr;   // weights [N, K/2] per group
    const uint8_t* b_scales = nullptr;
    int64_t M = 0, N = 0, K = 0;
    // grouping: rows of group e are [row_off[e], row_off[e+1]), its row tiles
    // [tile_off[e], tile_off[e+1])
    const int32_t* row_off = nullptr;
    const int32_t* tile_off = nullptr;
    int32_t groups = 0;
    int32_t ntiles = 0;                 // set by the launcher
    int32_t ksplit = 1, ksteps = 0;     // kPartialF32: K splits and the steps of each
    void* out = nullptr;                // kStoreBf16, kStoreF32: bf16, fp32 [M, ldo]; kGateUp: codes [M, ldo/2]
    uint8_t* out_scales = nullptr;      // kGateUp: [M, ldo/32]
    int64_t ldo = 0;
};

// Row tile of the grouped launches.
constexpr int kMxMoeBM = 192;
// grid_m bounds the row tiles of a grouped launch (ungrouped: ignored).
hipError_t launch_mx_gemm(const MxGemmArgs& g, MxEpi epi, int grid_m, hipStream_t stream);
// The K splits that launch_mx_gemm_split makes of a plain product (1: none) and
// the steps of each; it holds that many [M, N] fp32 sums in `partial`.
int mx_gemm_splits(int64_t M, int64_t N, int64_t K, int* steps);
hipError_t launch_mx_gemm_split(const MxGemmArgs& g, float* partial, hipStream_t stream);

// Few activation rows (mx_stream.hip).
struct MxStreamArgs {
    const uint16_t* x = nullptr;        // bf16 activation, quantized by the kernel; or
    const uint8_t* a_codes = nullptr;   // packed activation [*, K/2], [*, K/32]
    const uint8_t* a_scales = nullptr;
    const uint8_t* b_codes = nullptr;   // weights [E, N, K/2], [E, N, K/32] (plain: E = 1)
    const uint8_t* b_scales = nullptr;
    int64_t M = 0, N = 0, K = 0;
    int32_t E = 1, top_k = 1;
    const int32_t* ids = nullptr;       // slot forms: [T, top_k]
    const float* slot_w = nullptr;      // kSlotDown: [T, top_k]
    const int32_t* perm = nullptr;      // grouped forms: slot of each expert row,
    const int32_t* row_off = nullptr;   // row and tile offsets as in MxGemmArgs
    const int32_t* tile_off = nullptr;
    uint16_t* y = nullptr;              // bf16 outputs
    float* slot_y = nullptr;            // kGroupDown: fp32 outputs [S, N]
    uint8_t* h_codes = nullptr;         // gate/up forms: MXFP4 h [S, N/4], [S, N/64]
    uint8_t* h_scales = nullptr;
    int32_t ntiles = 0, slice = 0, rt = 16;  // set by the launcher
};
// Whether the plain form is the one to run (at most 64 activation rows), and
// whether it takes bf16 activations of this size, and the slot forms tokens of
// this width (they quantize them into LDS).
bool mx_stream_takes(int64_t M, int64_t N, int64_t K);
bool mx_stream_quantizes(int64_t M, int64_t K);
bool mx_slots_fit(int64_t H);
hipError_t launch_mx_stream(const MxStreamArgs& g, hipStream_t stream);
hipError_t launch_mx_slot_up(const MxStreamArgs& g, int64_t slots, hipStream_t stream);
hipError_t launch_mx_slot_down(const MxStreamArgs& g, int64_t tokens, hipStream_t stream);
// Row tiles of 16; mtiles bounds them.
hipError_t launch_mx_group_up(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream);
hipError_t launch_mx_group_down(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream);

// The sorted routed layer's first launch (mx_route.hip): row_off and tile_off
// [E + 1] (tiles of bm rows), the slot of each expert row perm [slots] and the
// row of each slot inv [slots] (-1 for an id outside [0, E)); and the MXFP4 of
// the tokens x, n8 pieces of 8 elements.  E <= 4096.  One workgroup sorts, so
// at most kMxPrepareSlots slots (its scattered stores take 32 us at 32768,
// where three launches and the quantizer take 25).
struct MxPrepareArgs {
    const int32_t* ids;
    int32_t slots, E, bm;
    int32_t* row_off;
    int32_t* tile_off;
    int32_t* perm;
    int32_t* inv;
    const uint16_t* x;
    int64_t n8;
    uint8_t* codes;
    uint8_t* scales;
};
constexpr int64_t kMxPrepareSlots = 1 << 13;
hipError_t launch_mx_prepare(const MxPrepareArgs& a, hipStream_t stream);

// out[t] = bf16(sum_j w[t, j] * Y[inv[t * top_k + j]]) over expert-sorted fp32
// rows Y [S, H], slots in order, inv < 0 skipped; H % 32 == 0.
hipError_t launch_mx_combine(const float* Y, const int32_t* inv, const float* w, int64_t T, int32_t top_k, int64_t H,
                             uint16_t* out, hipStream_t stream);

// -------------------------------------------------------------------- gate --

hipError_t launch_gate(const nvfp4_gate_config& c, const void* logits, const float* bias, int32_t* ids,
                       float* weights, hipStream_t stream);
hipError_t launch_gate_backward(const nvfp4_gate_config& c, const void* logits, const int32_t* ids,
                                const float* dweights, void* dlogits, hipStream_t stream);

// ------------------------------------------------------------------ errors --

// Sets the calling thread's error text and returns `status` (api.cpp).
int32_t api_fail(int32_t status, const char* text);
int32_t api_hip(hipError_t e, const char* where);
void api_clear();

}  // namespace nvfp4
