// mx_gemm.hip -- MXFP4 x MXFP4 products on the scaled matrix instructions:
// Y = A W^T, A [M, K] and W [N, K], both packed codes with one E8M0 byte per
// 32 elements along K; plain, or grouped by expert for the routed layer.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the packed codes and their scale
// bytes as they are stored, so nothing is decoded: a K step moves bytes from
// memory to LDS and from LDS to the matrix units.
//
// Roles: the weights are the instruction's A operand and the activations its
// B operand, so a lane's results are 4-element runs along N of one activation
// row: rows leave as whole pieces, and a block of 32 outputs of one row lies
// in two lanes, which is what requantizing h needs.
//
// K step: 256 elements (128 code bytes, 8 scale bytes a row).  A K
// permutation applied to both operands leaves the product unchanged: lane
// half hf = lane / 32 takes blocks 4 hf + kk of the step in instruction kk, so
// its four scale bytes are one word and byte kk is selected by the
// instruction.
//
// Codes go from global memory straight into LDS (buffer_load ... lds, 1 KB =
// 8 rows per instruction), two stages, one barrier per step.  LDS rows are
// not padded: row r keeps its 16-byte chunk c in slot c ^ ((r / 2) % 8), so
// that 16 consecutive rows' fragment reads cover all banks.  Blocks past K
// and rows past the operand load zeros with scale byte 0.
#include "mx_device.hpp"
#include "mx_internal.hpp"
#include "nvfp4_dma.hpp"

#include <type_traits>

namespace nvfp4 {

namespace {

constexpr int kGroupM = 8;  // row tiles per band in the ungrouped tile order

template <int SEL>
__device__ __forceinline__ f32x16 mfma_kk(u32x4 w, u32x4 a, f32x16 c, uint32_t sw, uint32_t sa) {
    return mx_mfma32<SEL, SEL>(w, a, c, sw, sa);
}

// TM, TN: 32-row blocks of activations and of weights per wave; WM x WN
// waves.  ALIGNED: K % 256 == 0, so a row's 8 scale bytes of a step are one
// aligned word pair (else they are read byte by byte).
template <int TM, int TN, int WM, int WN, MxEpi EP, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm(MxGemmArgs g) {
    constexpr int NW = WM * WN, NT = 64 * NW;
    constexpr int WTM = 32 * TM, WTN = 32 * TN, BM = WTM * WM, BN = WTN * WN;
    constexpr int A_SLABS = BM / 8, B_SLABS = BN / 8;
    constexpr int A_PER_W = A_SLABS / NW, B_PER_W = B_SLABS / NW;
    static_assert(A_SLABS % NW == 0 && B_SLABS % NW == 0, "copy");
    constexpr int SC_OFF = (BM + BN) * 128;
    constexpr int STAGE = SC_OFF + (BM + BN) * 8;
    constexpr int SC_PER_T = (BM + BN + NT - 1) / NT;
    static_assert(2 * STAGE <= 160 * 1024, "LDS");
    constexpr bool kGateUp = EP == MxEpi::kGateUp;
    static_assert(!kGateUp || TN % 2 == 0, "gate/up pairs column blocks");
    __shared__ __align__(1024) uint8_t smem[2 * STAGE];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int c32 = lane & 31, hf = lane >> 5;

    // ---- tile.  Workgroups reach the 8 XCDs round-robin by id; renumber so
    // that each XCD has a contiguous run of the real tiles.
    const int gm_tiles = g.groups > 0 ? g.tile_off[g.groups] : (int)((g.M + BM - 1) / BM);
    const int64_t total = (int64_t)gm_tiles * g.ntiles;
    int64_t id = blockIdx.x;
    if ((gridDim.x & 7) == 0) {
        const int64_t per = (total + 7) >> 3, j = id >> 3;
        if (j >= per) return;
        id = (id & 7) * per + j;
    }
    if (id >= total) return;
    int grp = 0, tn;
    int64_t row_beg, row_end;
    if (g.groups > 0) {
        const int mt = (int)(id / g.ntiles);
        tn = (int)(id - (int64_t)mt * g.ntiles);
        int lo = 0, hi = g.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g.tile_off[mid] <= mt) lo = mid; else hi = mid;
        }
        grp = lo;
        row_beg = (int64_t)g.row_off[grp] + (int64_t)(mt - g.tile_off[grp]) * BM;
        row_end = min((int64_t)g.row_off[grp + 1], row_beg + BM);
    } else {
        const int64_t per_band = (int64_t)kGroupM * g.ntiles;
        const int64_t band = id / per_band;
        const int first_m = (int)(band * kGroupM);
        const int gsz = min(gm_tiles - first_m, kGroupM);
        const int64_t r = id - band * per_band;
        tn = (int)(r / gsz);
        row_beg = (int64_t)(first_m + (int)(r % gsz)) * BM;
        row_end = min(g.M, row_beg + BM);
    }

    const uint32_t KB = (uint32_t)(g.K / 2), KS = (uint32_t)(g.K / 32);
    const int nsteps = (int)((g.K + 255) / 256);
    const int tail = (int)(KS - 8 * (uint32_t)(nsteps - 1));  // blocks of the last step, 1 .. 8

    // First weight row of the tile, and tile row n's row relative to it (-1
    // past the end).  Gate/up: each wave holds gate blocks, then the matching
    // up blocks, I rows further.
    const int64_t n0 = (int64_t)tn * (kGateUp ? BN / 2 : BN);
    const int64_t nlim = kGateUp ? g.N / 2 : g.N;
    auto b_row = [&](int n) -> int64_t {
        if constexpr (kGateUp) {
            const int w = n / WTN, j = (n % WTN) / 32;
            const int64_t h = w * (WTN / 2) + 32 * (j % (TN / 2)) + n % 32;
            if (n0 + h >= nlim) return -1;
            return j < TN / 2 ? h : h + nlim;
        } else {
            return n0 + n < nlim ? n : -1;
        }
    };
    const bool gather = g.a_rows != nullptr;
    auto a_row = [&](int r) -> int64_t {
        const int64_t row = row_beg + r;
        if (row >= row_end) return -1;
        return gather ? (int64_t)(g.a_rows[row] / g.a_div) : (int64_t)r;
    };
    const int64_t a0 = gather ? 0 : row_beg;
    const u32x4 ra = make_rsrc(g.a_codes + a0 * KB, (uint64_t)(gather ? g.a_src_rows : row_end - row_beg) * KB);
    const int64_t brows = (kGateUp ? 2 * nlim : nlim) - n0;
    const u32x4 rb = make_rsrc(g.b_codes + ((int64_t)grp * g.N + n0) * KB,
                               (uint64_t)(kGateUp || brows < BN ? brows : BN) * KB);
    const uint8_t* const as = g.a_scales + a0 * KS;
    const uint8_t* const bs = g.b_scales + ((int64_t)grp * g.N + n0) * KS;

    // ---- copy assignments.  A code slab: tile rows 8 s + lane / 8, slot
    // lane % 8, which holds chunk slot ^ ((r / 2) % 8).
    uint32_t va[A_PER_W], vb[B_PER_W];
    const int chunk0 = (lane & 7);
#pragma unroll
    for (int u = 0; u < A_PER_W; ++u) {
        const int r = 8 * (A_PER_W * wave + u) + (lane >> 3);
        const int64_t src = a_row(r);
        va[u] = src < 0 ? kOob : (uint32_t)src * KB + 16u * (chunk0 ^ ((r >> 1) & 7));
    }
#pragma unroll
    for (int u = 0; u < B_PER_W; ++u) {
        const int r = 8 * (B_PER_W * wave + u) + (lane >> 3);
        const int64_t src = b_row(r);
        vb[u] = src < 0 ? kOob : (uint32_t)src * KB + 16u * (chunk0 ^ ((r >> 1) & 7));
    }
    // scales: thread t handles tile rows t, t + NT, ..: activations, then weights
    const uint8_t* sp[SC_PER_T];
#pragma unroll
    for (int u = 0; u < SC_PER_T; ++u) {
        const int r = tid + u * NT;
        sp[u] = nullptr;
        if (r < BM) {
            const int64_t src = a_row(r);
            if (src >= 0) sp[u] = as + src * KS;
        } else if (r < BM + BN) {
            const int64_t src = b_row(r - BM);
            if (src >= 0) sp[u] = bs + src * KS;
        }
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
    uint2 sv[SC_PER_T];
    auto load_scales = [&](int kc) {
#pragma unroll
        for (int u = 0; u < SC_PER_T; ++u) {
            sv[u] = make_uint2(0, 0);
            if (sp[u] == nullptr) continue;
            if constexpr (ALIGNED) {
                sv[u] = *reinterpret_cast<const uint2*>(sp[u] + 8 * kc);
            } else {
                const int nb = kc + 1 < nsteps ? 8 : tail;
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int b = 0; b < 8; ++b)
                    if (b < nb) w[b >> 2] |= (uint32_t)sp[u][8 * kc + b] << (8 * (b & 3));
                sv[u] = make_uint2(w[0], w[1]);
            }
        }
    };
    auto store_scales = [&](int st) {
#pragma unroll
        for (int u = 0; u < SC_PER_T; ++u) {
            const int r = tid + u * NT;
            if (r < BM + BN) *reinterpret_cast<uint2*>(smem + st * STAGE + SC_OFF + 8 * r) = sv[u];
        }
    };
    auto issue = [&](int kc, int st) {
        const uint32_t b = lds0 + (uint32_t)(st * STAGE);
        const bool cut = !ALIGNED && kc + 1 == nsteps;  // the last step may lack blocks
#pragma unroll
        for (int u = 0; u < A_PER_W; ++u) {
            const int sl = A_PER_W * wave + u;
            uint32_t v = va[u];
            if (cut && (chunk0 ^ (((8 * sl + (lane >> 3)) >> 1) & 7)) >= tail) v = kOob;
            lds_load16(ra, v, (uint32_t)kc * 128u, b + (uint32_t)(sl * 1024));
        }
#pragma unroll
        for (int u = 0; u < B_PER_W; ++u) {
            const int sl = B_PER_W * wave + u;
            uint32_t v = vb[u];
            if (cut && (chunk0 ^ (((8 * sl + (lane >> 3)) >> 1) & 7)) >= tail) v = kOob;
            lds_load16(rb, v, (uint32_t)kc * 128u, b + (uint32_t)(BM * 128 + sl * 1024));
        }
    };

    f32x16 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    uint32_t off_k[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) off_k[kk] = (uint32_t)(c32 * 128 + 16 * ((4 * hf + kk) ^ ((c32 >> 1) & 7)));
    auto compute = [&](int st) {
        const uint8_t* const base = smem + st * STAGE;
        const uint8_t* const ab = base + wm * WTM * 128;
        const uint8_t* const bb = base + BM * 128 + wn * WTN * 128;
        const uint8_t* const sab = base + SC_OFF + 8 * (wm * WTM + c32) + 4 * hf;
        const uint8_t* const sbb = base + SC_OFF + 8 * (BM + wn * WTN + c32) + 4 * hf;
        uint32_t sa[TM], sb[TN];
#pragma unroll
        for (int i = 0; i < TM; ++i) sa[i] = *reinterpret_cast<const uint32_t*>(sab + 256 * i);
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = *reinterpret_cast<const uint32_t*>(sbb + 256 * j);
        auto group = [&](auto kkc) {
            constexpr int kk = decltype(kkc)::value;
            u32x4 a[TM], b[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) a[i] = *reinterpret_cast<const u32x4*>(ab + off_k[kk] + 4096 * i);
#pragma unroll
            for (int j = 0; j < TN; ++j) b[j] = *reinterpret_cast<const u32x4*>(bb + off_k[kk] + 4096 * j);
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i) acc[j][i] = mfma_kk<kk>(b[j], a[i], acc[j][i], sb[j], sa[i]);
        };
        group(std::integral_constant<int, 0>{});
        group(std::integral_constant<int, 1>{});
        group(std::integral_constant<int, 2>{});
        group(std::integral_constant<int, 3>{});
    };

    load_scales(0);
    issue(0, 0);
    store_scales(0);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
    for (int s = 0; s < nsteps; ++s) {
        const int st = s & 1;
        const bool more = s + 1 < nsteps;
        if (more) {
            load_scales(s + 1);
            issue(s + 1, st ^ 1);
        }
        compute(st);
        if (more) store_scales(st ^ 1);
        __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
        __syncthreads();
    }

    // ---- epilogue: acc[j][i][r] is weight row 32 j + 8 (r / 4) + 4 hf + r % 4
    // of the wave, activation row 32 i + c32.
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t row = row_beg + wm * WTM + 32 * i + c32;
        if constexpr (kGateUp) {
            // (rows past the end take part in the exchange and store nothing)
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                const int64_t hc = n0 + wn * (WTN / 2) + 32 * j;
                uint32_t w[8], m = 0;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    uint32_t pair = 0;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float gv = acc[j][i][2 * p + b], uv = acc[j + TN / 2][i][2 * p + b];
                        pair |= f32_to_bf16(gv / (1.0f + expf(-gv)) * uv) << (16 * b);
                    }
                    w[p] = pair;
                    m = max_bf16x2(m, pair);
                }
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, kWave));
                const uint32_t s = mx_scale_byte(m);
                const float d = mx_divisor(s);
                // this lane's codes: four runs of 4 elements (2 bytes) at 4 (2 q + hf)
                const uint32_t lo = mx_encode8(w[0], w[1], w[2], w[3], d), hi = mx_encode8(w[4], w[5], w[6], w[7], d);
                if (row < row_end && hc < nlim) {
                    uint8_t* const dst = reinterpret_cast<uint8_t*>(g.out) + row * (g.ldo / 2) + hc / 2 + 2 * hf;
                    *reinterpret_cast<uint16_t*>(dst) = (uint16_t)lo;
                    *reinterpret_cast<uint16_t*>(dst + 4) = (uint16_t)(lo >> 16);
                    *reinterpret_cast<uint16_t*>(dst + 8) = (uint16_t)hi;
                    *reinterpret_cast<uint16_t*>(dst + 12) = (uint16_t)(hi >> 16);
                    if (hf == 0) g.out_scales[row * (g.ldo / 32) + hc / 32] = (uint8_t)s;
                }
            }
        } else {
            if (row >= row_end) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int64_t col = n0 + wn * WTN + 32 * j + 8 * p + 4 * hf;
                    if (col >= nlim) continue;
                    const float v0 = acc[j][i][4 * p], v1 = acc[j][i][4 * p + 1], v2 = acc[j][i][4 * p + 2],
                                v3 = acc[j][i][4 * p + 3];
                    if constexpr (EP == MxEpi::kDown) {
                        // (N is the hidden size, a multiple of 32)
                        *reinterpret_cast<float4*>(reinterpret_cast<float*>(g.out) + row * g.ldo + col) =
                            make_float4(v0, v1, v2, v3);
                    } else {
                        uint16_t* const dst = reinterpret_cast<uint16_t*>(g.out) + row * g.ldo + col;
                        const uint32_t lo = f32_to_bf16(v0) | (f32_to_bf16(v1) << 16);
                        const uint32_t hi = f32_to_bf16(v2) | (f32_to_bf16(v3) << 16);
                        if ((g.ldo & 3) == 0) {
                            *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
                        } else {
                            dst[0] = (uint16_t)lo;
                            if (col + 1 < nlim) dst[1] = (uint16_t)(lo >> 16);
                            if (col + 2 < nlim) dst[2] = (uint16_t)hi;
                            if (col + 3 < nlim) dst[3] = (uint16_t)(hi >> 16);
                        }
                    }
                }
            }
        }
    }
}

template <int TM, int TN, int WM, int WN, MxEpi EP>
hipError_t launch_cfg(const MxGemmArgs& g0, int grid_m, hipStream_t stream) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    MxGemmArgs g = g0;
    const int64_t ncols = EP == MxEpi::kGateUp ? g.N / 2 : g.N, bn = EP == MxEpi::kGateUp ? BN / 2 : BN;
    g.ntiles = (int32_t)((ncols + bn - 1) / bn);
    const int64_t mt = g.groups > 0 ? grid_m : (g.M + BM - 1) / BM;
    int64_t wgs = mt * g.ntiles;
    if (g.groups > 0) wgs = (wgs + 7) / 8 * 8;  // a multiple of 8 for the XCD renumbering
    if (wgs < 1 || wgs >= ((int64_t)1 << 32) / (64 * WM * WN)) return hipErrorInvalidValue;
    if (g.K % 256 == 0)
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, EP, true>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    else
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, EP, false>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& g, MxEpi epi, int grid_m, hipStream_t stream) {
    switch (epi) {
        case MxEpi::kStoreBf16: return launch_cfg<2, 2, 2, 2, MxEpi::kStoreBf16>(g, grid_m, stream);
        case MxEpi::kGateUp: return launch_cfg<2, 2, 2, 2, MxEpi::kGateUp>(g, grid_m, stream);
        default: return launch_cfg<2, 2, 2, 2, MxEpi::kDown>(g, grid_m, stream);
    }
}

}  // namespace nvfp4
