// mx_combine.hip -- the weighted sum over a token's slots of the sorted routed
// layer: out[t] = bf16(sum_j w[t, j] * Y[row of slot j]), fp32, slots in order.
//
// Y is bf16: each slot's product is rounded once (2^-9 relative) before the
// fp32 sum and the output's own rounding, which halves the largest tensor of
// the layer (4096 x 8 slots of 6144: 403 MB written and read instead of 805).
// Bound by that read.
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace nvfp4 {

namespace {

// A thread sums 8 columns of one token; the rows of 8 slots are in flight
// together (a skipped slot reads row 0 and is not added).
__global__ __launch_bounds__(256) void k_mx_combine(const uint16_t* __restrict__ Y, const int32_t* __restrict__ inv,
                                                    const float* __restrict__ w, int64_t total, int32_t top_k,
                                                    int32_t h8, uint16_t* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / h8, c = (i - t * h8) * 8, H = (int64_t)h8 * 8;
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        int32_t pos[8];
        float wj[8];
        u32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = j0 + u < top_k;
            pos[u] = in ? inv[t * top_k + j0 + u] : -1;
            wj[u] = in ? w[t * top_k + j0 + u] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(Y + (int64_t)max(pos[u], 0) * H + c));
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (pos[u] < 0) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                s[2 * q] = __builtin_fmaf(wj[u], __uint_as_float(v[u][q] << 16), s[2 * q]);
                s[2 * q + 1] = __builtin_fmaf(wj[u], __uint_as_float(v[u][q] & 0xFFFF0000u), s[2 * q + 1]);
            }
        }
    }
    *reinterpret_cast<uint4*>(out + t * H + c) =
        make_uint4(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]), pack_bf16(s[4], s[5]), pack_bf16(s[6], s[7]));
}

}  // namespace

hipError_t launch_mx_combine(const uint16_t* Y, const int32_t* inv, const float* w, int64_t T, int32_t top_k, int64_t H,
                             uint16_t* out, hipStream_t stream) {
    const int64_t total = T * (H / 8);
    if (total >= (int64_t)1 << 32) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_mx_combine, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream, Y, inv, w, total,
                       top_k, (int32_t)(H / 8), out);
    return hipGetLastError();
}

}  // namespace nvfp4
