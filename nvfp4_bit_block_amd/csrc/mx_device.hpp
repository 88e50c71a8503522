// mx_device.hpp -- MXFP4 on gfx950: E8M0 scales, the block encoder, and the
// scaled matrix instructions.
//
// MXFP4 (OCP Microscaling Formats 1.0): E2M1 codes, one E8M0 byte s per 32
// elements along a row, value q * 2^(s - 127).
#pragma once

#include "nvfp4_device.hpp"

namespace nvfp4 {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// The byte's value as fp32, exact: 2^-127 is a subnormal pattern, 255 is NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// Scale byte of a block from its largest |x| as a bf16 magnitude pattern:
// floor(log2 amax) - 2 is the exponent field less 2 + 127, clamped at 0 (a
// subnormal's field is 0 and so clamps too, like zero); field 255 (an
// infinity or a NaN in the block) stays 255.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
    const uint32_t f = amax >> 7;
    return f == 255 ? 255u : f > 2 ? f - 2 : 0u;
}

// Eight bf16 (four words) -> eight codes under the scale value 2^(s - 127)
// (its fp32 form; the conversion rounds to nearest even on the E2M1 grid,
// saturates at 6 and keeps the sign, also of a zero; checked for every bf16
// under every scale).
__device__ __forceinline__ uint32_t mx_encode8(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, float d) {
    uint32_t o = 0;
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w0), d, 0);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w1), d, 1);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w2), d, 2);
    o = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o, __builtin_bit_cast(bf16x2, w3), d, 3);
    return o;
}
// Two fp32 -> two bf16 patterns in a word, round to nearest even (one
// instruction; a NaN, which a block of scale byte 255 makes, stays one).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// silu(g) * u from the hardware's exponential and reciprocal: a few parts in
// 2^22 for the gate values a layer meets, against the half step of 2^-9 that
// rounding h to bf16 takes.  (With the library's exponential and a correctly
// rounded division this took 200 of the 1000 us of the gate/up product at
// 4096 tokens x 8 of 256 experts, 6144 x 2048.)
__device__ __forceinline__ float silu_mul(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g)) * u;
}

// The scale the encoder divides by: a block of byte 255 decodes as NaN
// whatever its codes, so any finite value serves there.
__device__ __forceinline__ float mx_divisor(uint32_t s) { return e8m0_to_f32(s == 255 ? 127u : s); }

// Largest magnitude of a word's two bf16, as a pattern, folded into m.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t m, uint32_t w) {
    return max(max(m, w & 0x7FFFu), (w >> 16) & 0x7FFFu);
}

// Eight elements per lane, a block per quad of lanes (all four active): this
// lane's codes and the block's scale byte.
__device__ __forceinline__ void mx_encode_quad(const uint4& v, uint32_t& code, uint32_t& s) {
    uint32_t m = max_bf16x2(max_bf16x2(max_bf16x2(max_bf16x2(0, v.x), v.y), v.z), v.w);
    m = max(m, dpp_u32<0xB1>(m));  // quad_perm [1,0,3,2]
    m = max(m, dpp_u32<0x4E>(m));  // quad_perm [2,3,0,1]
    s = mx_scale_byte(m);
    code = mx_encode8(v.x, v.y, v.z, v.w, mx_divisor(s));
}

// The group whose row tiles [tile_off[e], tile_off[e + 1]) hold tile `mt`
// (which some group's do): a wave compares 64 bounds at a time, so 4096
// groups take two dependent loads.
__device__ __forceinline__ int group_of_tile(const int32_t* __restrict__ tile_off, int groups, int mt) {
    const int lane = threadIdx.x & 63, stride = (groups + 63) / 64;
    int lo = 0, e = lane * stride;
    if (stride > 1) {
        const bool le = e < groups && tile_off[e] <= mt;
        lo = (__popcll(__ballot(le)) - 1) * stride;  // the bounds ascend; tile_off[0] = 0
    }
    e = lo + lane;
    const bool le = lane < stride + (stride == 1 ? 63 : 0) && e < groups && tile_off[e] <= mt;
    return __builtin_amdgcn_readfirstlane(lo + __popcll(__ballot(le)) - 1);
}

// D += A B on the scaled matrix instructions.  32x32x64: lane l holds row
// (column) l % 32 and the 32 K positions [32 (l / 32), + 32), one MX block,
// as 16 code bytes; 16x16x128: row l % 16, block l / 16.  Byte SEL of the
// lane's scale word is that block's E8M0 byte.  D: lane l holds column l % 32
// (l % 16), rows 8 (r / 4) + 4 (l / 32) + r % 4 (4 (l / 16) + r).
template <int SEL_A, int SEL_B>
__device__ __forceinline__ f32x16 mx_mfma32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
    const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(A, B, c, 4, 4, SEL_A, (int)sa, SEL_B, (int)sb);
}
template <int SEL_A, int SEL_B>
__device__ __forceinline__ f32x4 mx_mfma16(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
    const i32x8 A = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
    const i32x8 B = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(A, B, c, 4, 4, SEL_A, (int)sa, SEL_B, (int)sb);
}

}  // namespace nvfp4
