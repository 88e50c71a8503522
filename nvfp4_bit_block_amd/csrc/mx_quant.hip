// mx_quant.hip -- MXFP4 quantize (along rows and along columns) and
// dequantize.
//
// Rows are whole blocks, so the rowwise passes run over the flat tensor: a
// lane takes 8 elements (16 bytes), a quad of lanes one block.  Bound by
// memory: 2 bytes read and 17/32 written per element (the reverse for
// dequantize).
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // 16-byte pieces in flight per lane

__global__ __launch_bounds__(kThreads) void k_mx_quantize(const uint16_t* __restrict__ x, int64_t n8,
                                                          uint32_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
    // n8 (pieces of 8 elements) is a multiple of 4, and so is every quad's
    // first index: the lanes of a quad leave together
    const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        v[u] = make_uint4(0, 0, 0, 0);
        if (i < n8) v[u] = load_nt16(x + 8 * i);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        uint32_t m = 0;
        m = max_bf16x2(m, v[u].x);
        m = max_bf16x2(m, v[u].y);
        m = max_bf16x2(m, v[u].z);
        m = max_bf16x2(m, v[u].w);
        m = max(m, dpp_u32<0xB1>(m));  // quad_perm [1,0,3,2]
        m = max(m, dpp_u32<0x4E>(m));  // quad_perm [2,3,0,1]
        const uint32_t s = mx_scale_byte(m);
        if (i < n8) {
            codes[i] = mx_encode8(v[u].x, v[u].y, v[u].z, v[u].w, mx_divisor(s));
            if ((threadIdx.x & 3) == 0) scales[i >> 2] = (uint8_t)s;
        }
    }
}

__global__ __launch_bounds__(kThreads) void k_mx_dequantize(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t n8,
                                                            uint16_t* __restrict__ y) {
    const int64_t base = (int64_t)blockIdx.x * (kThreads * kUnroll) + threadIdx.x;
    uint32_t c[kUnroll], s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        c[u] = s[u] = 0;
        if (i < n8) {
            c[u] = __builtin_nontemporal_load(codes + i);
            s[u] = scales[i >> 2];
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        if (i >= n8) return;
        const float d = e8m0_to_f32(s[u]);
        f32x2 q[4];
        fp4x8_to_f32(c[u], q);
        u32x4 o;
        // q * d is exact in bf16 (at most two significant bits, 2^-128 the
        // least magnitude), so the fp32 pattern's low half is zero
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[j] = (__float_as_uint(q[j].x * d) >> 16) | (__float_as_uint(q[j].y * d) & 0xFFFF0000u);
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(y + 8 * i));
    }
}

// Columnwise: a tile of 256 rows x 64 columns of x goes through LDS; a lane
// encodes one 32-row block of one column, the eight blocks of a column in
// eight neighbouring lanes, so that a wave stores 128 contiguous code bytes
// of eight columns.  LDS keeps word w (columns 2w, 2w + 1) of row r at
// w ^ (4 ((r / 32) % 8)): the eight blocks then read eight different groups
// of four banks, and the 16-byte row pieces stay whole.
constexpr int kCR = 256, kCC = 64, kCW = kCC / 2;
__device__ __forceinline__ int col_word(int r, int w) { return r * kCW + (w ^ (((r >> 5) & 7) << 2)); }

__global__ __launch_bounds__(kThreads) void k_mx_quantize_cols(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                               int64_t ctiles, uint8_t* __restrict__ codes_t,
                                                               uint8_t* __restrict__ scales_t) {
    __shared__ __align__(16) uint32_t tile[kCR * kCW];
    const int64_t rt = blockIdx.x / ctiles, ct = blockIdx.x - rt * ctiles;
    const int64_t r0 = rt * kCR, c0 = ct * kCC;
#pragma unroll
    for (int pass = 0; pass < kCR / 32; ++pass) {
        const int lr = pass * 32 + (threadIdx.x >> 3), lc = (threadIdx.x & 7) * 8;
        const int64_t r = r0 + lr, c = c0 + lc;
        uint32_t w[4] = {0, 0, 0, 0};
        if (r < R && c < C) {
            const uint16_t* p = x + r * C + c;
            if (c + 8 <= C) {
                __builtin_memcpy(w, p, 16);  // rows of an odd width start at any even address
            } else {
                for (int j = 0; j < (int)(C - c); ++j) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            }
        }
        *reinterpret_cast<uint4*>(tile + col_word(lr, lc / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    const int blk = threadIdx.x & 7;
    const int64_t rb = r0 + 32 * blk;
    if (rb >= R) return;  // R is a multiple of 32: a block is whole or absent
    const uint16_t* t16 = reinterpret_cast<const uint16_t*>(tile);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int col = (threadIdx.x >> 3) + 32 * half;
        const int64_t c = c0 + col;
        if (c >= C) continue;
        uint32_t w[16], m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t lo = t16[2 * col_word(32 * blk + 2 * i, col >> 1) + (col & 1)];
            const uint32_t hi = t16[2 * col_word(32 * blk + 2 * i + 1, col >> 1) + (col & 1)];
            w[i] = lo | (hi << 16);
            m = max_bf16x2(m, w[i]);
        }
        const uint32_t s = mx_scale_byte(m);
        const float d = mx_divisor(s);
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = mx_encode8(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3], d);
        *reinterpret_cast<u32x4*>(codes_t + c * (R / 2) + rb / 2) = o;
        scales_t[c * (R / 32) + rb / 32] = (uint8_t)s;
    }
}

int64_t flat_grid(int64_t n8) { return (n8 + kThreads * kUnroll - 1) / (kThreads * kUnroll); }

}  // namespace

// (a launch holds fewer than 2^32 threads)
constexpr int64_t kMaxGrid = ((int64_t)1 << 32) / kThreads;

bool mx_quantize_fits(int64_t rows, int64_t cols) {
    return rows < ((int64_t)1 << 40) / (cols / 8 + 1) && flat_grid(rows * (cols / 8)) < kMaxGrid;
}

hipError_t launch_mx_quantize(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                              hipStream_t stream) {
    const int64_t n8 = rows * (cols / 8);
    hipLaunchKernelGGL(k_mx_quantize, dim3((unsigned)flat_grid(n8)), dim3(kThreads), 0, stream, x, n8,
                       reinterpret_cast<uint32_t*>(codes), scales);
    return hipGetLastError();
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, uint16_t* y,
                                hipStream_t stream) {
    const int64_t n8 = rows * (cols / 8);
    hipLaunchKernelGGL(k_mx_dequantize, dim3((unsigned)flat_grid(n8)), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint32_t*>(codes), scales, n8, y);
    return hipGetLastError();
}

bool mx_quantize_cols_fits(int64_t rows, int64_t cols) {
    const int64_t rt = (rows + kCR - 1) / kCR, ct = (cols + kCC - 1) / kCC;
    return rt < kMaxGrid && ct < kMaxGrid && rt * ct < kMaxGrid;
}

hipError_t launch_mx_quantize_cols(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t, uint8_t* scales_t,
                                   hipStream_t stream) {
    const int64_t rt = (rows + kCR - 1) / kCR, ct = (cols + kCC - 1) / kCC;
    hipLaunchKernelGGL(k_mx_quantize_cols, dim3((unsigned)(rt * ct)), dim3(kThreads), 0, stream, x, rows, cols, ct,
                       codes_t, scales_t);
    return hipGetLastError();
}

}  // namespace nvfp4
