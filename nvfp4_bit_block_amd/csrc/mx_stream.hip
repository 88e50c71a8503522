// mx_stream.hip -- MXFP4 products for few activation rows: every weight byte
// is read once, straight from memory into the matrix instruction's operand
// registers, and nothing else is large.  Bound by the weight stream.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, weights as the A operand (16 weight
// rows), activations as the B operand (16 rows, fewer are padded with copies
// that are never stored).  A workgroup owns NR tiles of 16 weight rows; its
// waves split K and their sums meet in LDS.  In a K unit of 256 elements lane
// group g = lane / 16 takes blocks g and 4 + g, so an instruction reads 64
// contiguous code bytes of each row; the unit's 8 scale bytes of a row are
// one load, and the lane shifts its byte down.
//
// Forms (Mode):
//   kPlain     y = bf16(A W^T).
//   kSlotUp    routed layer, one workgroup per (slot, 32 columns of h): the
//              token is quantized by the waves themselves, gate and up rows
//              are multiplied, and h leaves as one MXFP4 block.
//   kSlotDown  one workgroup per (token, 16 NR columns): the waves walk the
//              token's slots in order and weigh them, so the weighted sum
//              leaves as bf16 without a pass of its own.
//   kGroupUp, kGroupDown  the same products on expert-sorted rows (up to
//              16 MB of one expert per workgroup).
#include <algorithm>
#include <type_traits>

#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace nvfp4 {

namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

// One operand's rows as a lane sees them: the lane's row offset (bytes) into
// codes and scales, from uniform bases.
struct RowPtr {
    const uint8_t* codes;
    const uint8_t* scales;
};

// codes and scale words of one 128-element step for this lane.
struct Step {
    u32x4 c;
    uint32_t s;
};

// FAST: K % 256 == 0 (whole units, 8-byte scale loads); otherwise units of
// one 128-element step, scale bytes loaded one by one and blocks past K read
// as zeros.
template <bool FAST>
struct Unit {
    static constexpr int kSteps = FAST ? 2 : 1;
    Step st[kSteps];
};

template <bool FAST, bool NT>
__device__ __forceinline__ Unit<FAST> load_unit(const RowPtr& r, int unit, int g, int nblk) {
    Unit<FAST> u;
    if constexpr (FAST) {
        const uint8_t* c = r.codes + (size_t)unit * 128 + 16 * g;
        u.st[0].c = NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c)) : *reinterpret_cast<const u32x4*>(c);
        u.st[1].c = NT ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c + 64))
                       : *reinterpret_cast<const u32x4*>(c + 64);
        const uint2 s = *reinterpret_cast<const uint2*>(r.scales + (size_t)unit * 8);
        u.st[0].s = s.x >> (8 * g);
        u.st[1].s = s.y >> (8 * g);
    } else {
        const int b = 4 * unit + g;
        u.st[0].c = u32x4{0, 0, 0, 0};
        u.st[0].s = 0;
        if (b < nblk) {
            u.st[0].c = *reinterpret_cast<const u32x4*>(r.codes + (size_t)b * 16);
            u.st[0].s = r.scales[b];
        }
    }
    return u;
}

// Quantizes `blocks` blocks of one bf16 row (from block b0) into this wave's
// LDS: codes 16 bytes a block, then scale bytes.
__device__ __forceinline__ void quantize_slice(const uint16_t* x, int b0, int blocks, uint8_t* lc, uint8_t* ls) {
    const int lane = threadIdx.x & 63;
    for (int b = lane; b < blocks; b += 64) {
        const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)(b0 + b) * 32);
        uint4 v[4];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = max_bf16x2(m, v[i].x);
            m = max_bf16x2(m, v[i].y);
            m = max_bf16x2(m, v[i].z);
            m = max_bf16x2(m, v[i].w);
        }
        const uint32_t s = mx_scale_byte(m);
        const float d = mx_divisor(s);
        u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mx_encode8(v[i].x, v[i].y, v[i].z, v[i].w, d);
        *reinterpret_cast<u32x4*>(lc + 16 * b) = o;
        ls[b] = (uint8_t)s;
    }
}

enum class Mode : int { kPlain = 0, kSlotUp = 1, kSlotDown = 2, kGroupUp = 3, kGroupDown = 4 };

// acc += W A^T over units [u0, u1) of one activation operand.
template <int NR, int MB, bool FAST, int UC>
__device__ __forceinline__ void run_units(f32x4 (&acc)[NR][MB], const RowPtr (&w)[NR], const RowPtr (&a)[MB], int u0,
                                          int u1, int g, int nblk) {
    Unit<FAST> wb[2][UC][NR];
    auto fetch = [&](int u, int buf) {
#pragma unroll
        for (int c = 0; c < UC; ++c)
            if (u + c < u1)
#pragma unroll
                for (int i = 0; i < NR; ++i) wb[buf][c][i] = load_unit<FAST, true>(w[i], u + c, g, nblk);
    };
    auto use = [&](int u, int buf) {
#pragma unroll
        for (int c = 0; c < UC; ++c) {
            if (u + c >= u1) break;
            Unit<FAST> ab[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) ab[m] = load_unit<FAST, false>(a[m], u + c, g, nblk);
#pragma unroll
            for (int s = 0; s < Unit<FAST>::kSteps; ++s)
#pragma unroll
                for (int i = 0; i < NR; ++i)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[i][m] = mx_mfma16<0, 0>(wb[buf][c][i].st[s].c, ab[m].st[s].c, acc[i][m],
                                                    wb[buf][c][i].st[s].s, ab[m].st[s].s);
        }
    };
    if (u0 >= u1) return;
    fetch(u0, 0);
    for (int u = u0; u < u1; u += 2 * UC) {
        fetch(u + UC, 1);
        use(u, 0);
        fetch(u + 2 * UC, 0);
        use(u + UC, 1);
    }
}

// QUANT: the activation is bf16 and each wave quantizes its K slice into
// LDS (kPlain: up to 16 rows; kSlotUp).  The LDS of a wave: `slice` blocks
// per row.
template <int NR, int MB, bool FAST, Mode MODE, bool QUANT>
__global__ __launch_bounds__(kThreads) void k_mx_stream(MxStreamArgs g) {
    constexpr bool kUp = MODE == Mode::kSlotUp || MODE == Mode::kGroupUp;
    static_assert(!kUp || NR == 4, "gate/up: two tiles each");
    constexpr int UC = NR * MB >= 4 ? 1 : NR >= 2 ? 2 : 4;
    extern __shared__ __align__(16) uint8_t smem[];
    float* const red = reinterpret_cast<float*>(smem);  // [wave][tile][lane][4]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, lg = lane >> 4;

    const int64_t KB = g.K / 2, KS = g.K / 32;
    const int nblk = (int)KS;
    const int units = FAST ? (int)(g.K / 256) : (int)((g.K + 127) / 128);

    // ---- tile
    const int nt = g.ntiles;
    int64_t id = blockIdx.x;
    int64_t row_beg = 0, row_end = g.M;  // activation (output) rows
    int64_t expert = 0;
    int tn = 0;
    if constexpr (MODE == Mode::kPlain) {
        tn = (int)id;
    } else if constexpr (MODE == Mode::kSlotUp || MODE == Mode::kSlotDown) {
        // slot (token) major: the workgroups of one slot share its expert
        const int64_t s = id / nt;
        tn = (int)(id - s * nt);
        row_beg = s;
        row_end = s + 1;
        if constexpr (MODE == Mode::kSlotUp) {
            expert = g.ids[s];
            if (expert < 0 || expert >= g.E) return;
        }
    } else {
        const int64_t mt = id / nt;
        tn = (int)(id - mt * nt);
        if (mt >= g.tile_off[g.E]) return;
        const int lo = group_of_tile(g.tile_off, g.E, (int)mt);
        expert = lo;
        row_beg = (int64_t)g.row_off[lo] + (mt - g.tile_off[lo]) * (16 * MB);
        row_end = min((int64_t)g.row_off[lo + 1], row_beg + 16 * MB);
    }
    const int64_t n0 = (int64_t)tn * (kUp ? 32 : 16 * NR);
    const int64_t half = g.N / 2;  // kUp: I
    // weight rows of tile i; rows past N repeat row n0's tile (never stored)
    auto w_row = [&](int i) -> int64_t {
        if constexpr (kUp) return (i < 2 ? 0 : half) + n0 + 16 * (i & 1) + l16;
        const int64_t n = n0 + 16 * i + l16;
        return n < g.N ? n : g.N - 1;
    };

    f32x4 acc[NR][MB];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int m = 0; m < MB; ++m) acc[i][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    if constexpr (MODE == Mode::kSlotDown) {
        // this wave's share of the token's top_k * units K units, slot by slot
        const int total = g.top_k * units;
        int p = wave * total / kWaves;
        const int end = (wave + 1) * total / kWaves;
        while (p < end) {
            const int j = p / units, u0 = p - j * units, u1 = min(units, u0 + end - p);
            p += u1 - u0;
            const int64_t s = row_beg * g.top_k + j;
            const int32_t e = g.ids[s];
            if (e < 0 || e >= g.E) continue;
            const float wj = g.slot_w[s];
            RowPtr w[NR], a[1];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int64_t r = (int64_t)e * g.N + w_row(i);
                w[i] = {g.b_codes + r * KB, g.b_scales + r * KS};
            }
            a[0] = {g.a_codes + s * KB, g.a_scales + s * KS};
            f32x4 part[NR][1];
#pragma unroll
            for (int i = 0; i < NR; ++i) part[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            run_units<NR, 1, FAST, UC>(part, w, a, u0, u1, lg, nblk);
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][0][r] = __builtin_fmaf(wj, part[i][0][r], acc[i][0][r]);
        }
    } else {
        const int u0 = wave * units / kWaves, u1 = (wave + 1) * units / kWaves;
        RowPtr w[NR], a[MB];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int64_t r = expert * g.N + w_row(i);
            w[i] = {g.b_codes + r * KB, g.b_scales + r * KS};
        }
        if constexpr (QUANT) {
            // this wave's slice of every row, quantized into its own LDS; the
            // operand reads below see it through pointers that start at unit 0
            constexpr int kBpu = FAST ? 8 : 4;  // blocks per unit
            const int b0 = u0 * kBpu, blocks = min(u1 * kBpu, nblk) - b0;
            const int rows = MODE == Mode::kPlain ? (int)g.M : 1;
            const int cap = g.slice;  // blocks a wave's row may hold, a multiple of 8
            uint8_t* const lc = smem + (size_t)wave * rows * cap * 17;
            uint8_t* const ls = lc + (size_t)rows * cap * 16;
            for (int m = 0; m < rows; ++m) {
                const int64_t src = MODE == Mode::kPlain ? m : row_beg / g.top_k;
                quantize_slice(g.x + src * g.K, b0, blocks, lc + (size_t)m * cap * 16, ls + (size_t)m * cap);
            }
            const int mr = l16 < rows ? l16 : 0;
            a[0] = {lc + ((size_t)mr * cap - b0) * 16, ls + (size_t)mr * cap - b0};
            __builtin_amdgcn_wave_barrier();
        } else {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                int64_t r = row_beg + 16 * m + l16;
                if (r >= row_end) r = row_beg;
                if constexpr (MODE == Mode::kGroupUp) r = g.perm[r] / g.top_k;
                a[m] = {g.a_codes + r * KB, g.a_scales + r * KS};
            }
        }
        run_units<NR, MB, FAST, UC>(acc, w, a, u0, u1, lg, nblk);
        if constexpr (QUANT) __syncthreads();  // the sums below reuse the slices' LDS
    }

    // ---- the waves' sums, in wave order
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            *reinterpret_cast<f32x4*>(red + ((size_t)(wave * NR * MB + i * MB + m) * 64 + lane) * 4) = acc[i][m];
    __syncthreads();
    // tile t of NR MB, lane ln: weight rows 4 (ln / 16) + r, activation row ln % 16
    auto total = [&](int t, int ln) -> f32x4 {
        f32x4 s = *reinterpret_cast<const f32x4*>(red + ((size_t)t * 64 + ln) * 4);
#pragma unroll
        for (int v = 1; v < kWaves; ++v)
            s += *reinterpret_cast<const f32x4*>(red + ((size_t)(v * NR * MB + t) * 64 + ln) * 4);
        return s;
    };
    if constexpr (kUp) {
        // thread: activation row m, columns 4 q .. 4 q + 3 of the 32 (eight
        // neighbouring lanes share a row, and so its block)
        for (int p = threadIdx.x; p < 16 * MB * 8; p += kThreads) {
            const int m = p >> 3, q = p & 7;
            const int ln = 16 * (q & 3) + (m & 15), tile = q >> 2;
            const f32x4 gv = total(tile * MB + (m >> 4), ln), uv = total((2 + tile) * MB + (m >> 4), ln);
            const uint32_t w[2] = {pack_bf16(silu_mul(gv[0], uv[0]), silu_mul(gv[1], uv[1])),
                                   pack_bf16(silu_mul(gv[2], uv[2]), silu_mul(gv[3], uv[3]))};
            uint32_t mx = max_bf16x2(max_bf16x2(0, w[0]), w[1]);
            mx = max(mx, dpp_u32<0xB1>(mx));
            mx = max(mx, dpp_u32<0x4E>(mx));
            mx = max(mx, dpp_u32<0x141>(mx));  // the 8 lanes of a row
            const uint32_t s = mx_scale_byte(mx);
            const uint32_t code = mx_encode8(w[0], w[1], 0, 0, mx_divisor(s));
            const int64_t row = row_beg + m;
            if (row < row_end) {
                *reinterpret_cast<uint16_t*>(g.h_codes + row * (half / 2) + n0 / 2 + 2 * q) = (uint16_t)code;
                if (q == 0) g.h_scales[row * (half / 32) + n0 / 32] = (uint8_t)s;
            }
        }
    } else {
        for (int p = threadIdx.x; p < NR * MB * 64; p += kThreads) {
            const int t = p >> 6, ln = p & 63;
            const int64_t row = row_beg + 16 * (t % MB) + (ln & 15);
            const int64_t col = n0 + 16 * (t / MB) + 4 * (ln >> 4);
            if (row >= row_end || col >= g.N) continue;
            const f32x4 v = total(t, ln);
            {
                uint16_t* const dst = g.y + row * g.N + col;
                const uint32_t lo = pack_bf16(v[0], v[1]), hi = pack_bf16(v[2], v[3]);
                if ((g.N & 3) == 0) {
                    *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
                } else {
                    dst[0] = (uint16_t)lo;
                    if (col + 1 < g.N) dst[1] = (uint16_t)(lo >> 16);
                    if (col + 2 < g.N) dst[2] = (uint16_t)hi;
                    if (col + 3 < g.N) dst[3] = (uint16_t)(hi >> 16);
                }
            }
        }
    }
}

template <int NR, int MB, bool FAST, Mode MODE, bool QUANT>
hipError_t launch_one(MxStreamArgs g, int64_t mtiles, hipStream_t stream) {
    constexpr bool kUp = MODE == Mode::kSlotUp || MODE == Mode::kGroupUp;
    g.ntiles = (int32_t)(kUp ? (g.N / 2 + 31) / 32 : (g.N + 16 * NR - 1) / (16 * NR));
    const int64_t wgs = mtiles * g.ntiles;
    if (wgs < 1 || wgs >= ((int64_t)1 << 32) / kThreads) return hipErrorInvalidValue;
    size_t lds = (size_t)kWaves * NR * MB * 1024;
    if (QUANT) {
        g.slice = mx_stream_slice(g.K);
        lds = std::max(lds, (size_t)kWaves * (MODE == Mode::kPlain ? (size_t)g.M : 1) * g.slice * 17);
    }
    if (lds > 64 * 1024) return hipErrorInvalidValue;
    hipLaunchKernelGGL((k_mx_stream<NR, MB, FAST, MODE, QUANT>), dim3((unsigned)wgs), dim3(kThreads), lds, stream, g);
    return hipGetLastError();
}

template <int NR, int MB, Mode MODE, bool QUANT>
hipError_t launch_k(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream) {
    return g.K % 256 == 0 ? launch_one<NR, MB, true, MODE, QUANT>(g, mtiles, stream)
                          : launch_one<NR, MB, false, MODE, QUANT>(g, mtiles, stream);
}

}  // namespace

int mx_stream_slice(int64_t K) {
    // the largest share of a wave, in blocks, rounded up to whole units of 8
    const int64_t units = K % 256 == 0 ? K / 256 : (K + 127) / 128, bpu = K % 256 == 0 ? 8 : 4;
    const int64_t b = (units + kWaves - 1) / kWaves * bpu;
    return (int)((b + 7) / 8 * 8);
}
bool mx_stream_quantizes(int64_t M, int64_t K) {
    return M <= 4 && K <= ((int64_t)1 << 20) && (int64_t)kWaves * M * mx_stream_slice(K) * 17 <= 64 * 1024;
}

hipError_t launch_mx_stream(const MxStreamArgs& g, hipStream_t stream) {
    // 16-row weight tiles a workgroup: one while that gives at most 1024
    // workgroups or the rows are long, else two or four
    const int64_t t1 = (g.N + 15) / 16;
    const int nr = t1 <= 512 || g.K >= 8192 ? 1 : t1 <= 1024 ? 2 : 4;
    if (g.x != nullptr)
        return nr == 1 ? launch_k<1, 1, Mode::kPlain, true>(g, 1, stream)
                       : nr == 2 ? launch_k<2, 1, Mode::kPlain, true>(g, 1, stream)
                                 : launch_k<4, 1, Mode::kPlain, true>(g, 1, stream);
    if (g.M <= 16)
        return nr == 1 ? launch_k<1, 1, Mode::kPlain, false>(g, 1, stream)
                       : nr == 2 ? launch_k<2, 1, Mode::kPlain, false>(g, 1, stream)
                                 : launch_k<4, 1, Mode::kPlain, false>(g, 1, stream);
    if (g.M <= 32)
        return nr == 1 ? launch_k<1, 2, Mode::kPlain, false>(g, 1, stream)
                       : launch_k<2, 2, Mode::kPlain, false>(g, 1, stream);
    if (g.M <= 64)
        return nr == 1 ? launch_k<1, 4, Mode::kPlain, false>(g, 1, stream)
                       : launch_k<2, 4, Mode::kPlain, false>(g, 1, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_mx_slot_up(const MxStreamArgs& g, int64_t slots, hipStream_t stream) {
    return launch_k<4, 1, Mode::kSlotUp, true>(g, slots, stream);
}
hipError_t launch_mx_slot_down(const MxStreamArgs& g, int64_t tokens, hipStream_t stream) {
    return launch_k<1, 1, Mode::kSlotDown, false>(g, tokens, stream);
}
hipError_t launch_mx_group_up(const MxStreamArgs& g, int bm, int64_t mtiles, hipStream_t stream) {
    return bm == 16 ? launch_k<4, 1, Mode::kGroupUp, false>(g, mtiles, stream)
                    : launch_k<4, 2, Mode::kGroupUp, false>(g, mtiles, stream);
}
hipError_t launch_mx_group_down(const MxStreamArgs& g, int bm, int64_t mtiles, hipStream_t stream) {
    return bm == 16 ? launch_k<4, 1, Mode::kGroupDown, false>(g, mtiles, stream)
                    : launch_k<2, 2, Mode::kGroupDown, false>(g, mtiles, stream);
}

}  // namespace nvfp4
