// mx_quant.hip -- MXFP4 quantize (along rows and along columns) and
// dequantize.
//
// Rows are whole blocks, so the rowwise passes run over the flat tensor: a
// lane takes 8 elements (16 bytes), a quad of lanes one block.  Bound by
// memory: 2 bytes read and 17/32 written per element (the reverse for
// dequantize); 65536 x 6144, 1.02 GB, takes 148 us each on MI355X, 6.9 TB/s with
// what the cache keeps, against 5.0 TB/s of a large copy.
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
        uint32_t code, s;
        mx_encode_quad(v[u], code, s);
        if (i < n8) {
            codes[i] = code;
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

// Columnwise: a tile of CR rows x CC columns of x goes through LDS; a lane
// encodes one 32-row block of one column, the CR / 32 blocks of a column in
// neighbouring lanes, so that 256 rows give stores of 128 contiguous code
// bytes.  LDS keeps word w (columns 2w, 2w + 1) of row r at w ^ (S ((r / 32) %
// (CR / 32))), S = 1024 / CR: the blocks of a column then read different
// groups of banks, and the 16-byte row pieces stay whole.
template <int CR, int CC, int NT>
__global__ __launch_bounds__(NT) void k_mx_quantize_cols(const uint16_t* __restrict__ x, int64_t R, int64_t C,
                                                         int64_t ctiles, uint8_t* __restrict__ codes_t,
                                                         uint8_t* __restrict__ scales_t) {
    constexpr int kBlk = CR / 32, kW = CC / 2, kPer = NT / (CC / 8);  // rows loaded per pass
    static_assert(CR % kPer == 0 && (CC * kBlk) % NT == 0 && CC >= 64, "tile");
    __shared__ __align__(16) uint32_t tile[CR * kW];
    auto word = [](int r, int w) { return r * kW + (w ^ (((r >> 5) & (kBlk - 1)) * (32 / kBlk))); };
    const int64_t rt = blockIdx.x / ctiles, ct = blockIdx.x - rt * ctiles;
    const int64_t r0 = rt * CR, c0 = ct * CC;
#pragma unroll
    for (int pass = 0; pass < CR / kPer; ++pass) {
        const int lr = pass * kPer + threadIdx.x / (CC / 8), lc = (threadIdx.x % (CC / 8)) * 8;
        const int64_t r = r0 + lr, c = c0 + lc;
        uint32_t w[4] = {0, 0, 0, 0};
        if (r < R && c < C) {
            const uint16_t* p = x + r * C + c;
            if (c + 8 <= C) {
                __builtin_memcpy(w, p, 16);  // rows of an odd width start at any even address
            } else {
#pragma unroll
                for (int j = 0; j < 7; ++j)
                    if (c + j < C) w[j >> 1] |= (uint32_t)p[j] << (16 * (j & 1));
            }
        }
        *reinterpret_cast<uint4*>(tile + word(lr, lc / 2)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    const int blk = threadIdx.x % kBlk;
    const int64_t rb = r0 + 32 * blk;
    if (rb >= R) return;  // R is a multiple of 32: a block is whole or absent
    const uint16_t* t16 = reinterpret_cast<const uint16_t*>(tile);
#pragma unroll
    for (int part = 0; part < CC * kBlk / NT; ++part) {
        const int col = threadIdx.x / kBlk + part * (NT / kBlk);
        const int64_t c = c0 + col;
        if (c >= C) continue;
        uint32_t w[16], m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t lo = t16[2 * word(32 * blk + 2 * i, col >> 1) + (col & 1)];
            const uint32_t hi = t16[2 * word(32 * blk + 2 * i + 1, col >> 1) + (col & 1)];
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

template <int CR, int CC, int NT>
hipError_t launch_cols(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t, uint8_t* scales_t,
                       hipStream_t stream) {
    const int64_t rt = (rows + CR - 1) / CR, ct = (cols + CC - 1) / CC;
    hipLaunchKernelGGL((k_mx_quantize_cols<CR, CC, NT>), dim3((unsigned)(rt * ct)), dim3(NT), 0, stream, x, rows, cols,
                       ct, codes_t, scales_t);
    return hipGetLastError();
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
    if (rows > 256 * kMaxGrid || cols > 64 * kMaxGrid) return false;  // (the sums and the product below stay in range)
    return (rows + 255) / 256 * ((cols + 63) / 64) < kMaxGrid;
}

// 256-row tiles write whole cache lines of codes; below two of them per CU,
// 32-row tiles give eight times the workgroups (1056 x 1021: 11.0 -> 4.9 us).
// 4096 x 6144 takes 14.3 us, 4.5 TB/s (along rows 12.5), 65536 x 6144 246 us, 4.2
// TB/s (155): a lane reads its column from LDS two bytes at a time.
hipError_t launch_mx_quantize_cols(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes_t, uint8_t* scales_t,
                                   hipStream_t stream) {
    const int64_t rt = (rows + 255) / 256, ct = (cols + 63) / 64;
    return rt * ct < 512 ? launch_cols<32, 128, 128>(x, rows, cols, codes_t, scales_t, stream)
                         : launch_cols<256, 64, 256>(x, rows, cols, codes_t, scales_t, stream);
}

}  // namespace nvfp4
