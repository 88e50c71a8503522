// mx_stream.hip -- MXFP4 products for few activation rows: every weight byte
// is read once, straight from memory into the matrix instruction's operand
// registers, and nothing else is large.  Bound by the weight stream, and by a
// launch's ramp and tail where that is short.  On MI355X, kernel times over
// eight sets of weights in turn, so that they come from memory: one token
// through 6144 x 16384 13.0 us (53.5 MB, 4.1 TB/s; 10.4 while three sets stay in
// the last-level cache), the gate/up product of its 8 experts of 6144 x 2048
// 24.1 us (107 MB, 4.4 TB/s) and the down product 12.0 us (53.5 MB, 4.5 TB/s).
// The figures below are times per call in a graph, weights of 0.4 GB or more in
// turn where one set is larger than 16 MB.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, weights as the A operand (16 weight
// rows), activations as the B operand (16 rows, fewer are padded with copies
// that are never stored).  A workgroup owns NR tiles of 16 weight rows; its
// waves split K and their sums meet in LDS.  In a step of 128 elements lane
// group g = lane / 16 takes block g, so an instruction reads 64 contiguous
// code bytes of each row; the scale bytes of a row are loaded for two or four
// steps at once, and the lane shifts its byte down.
//
// Forms (Mode):
//   kPlain     y = bf16(A W^T).
//   kSlotUp    routed layer, one workgroup per (slot, 32 columns of h): the
//              token is quantized by the waves themselves, gate and up rows
//              are multiplied, and h leaves as one MXFP4 block.
//   kSlotDown  one workgroup per (token, 16 NR columns): the waves walk the
//              token's slots in order and weigh them, so the weighted sum
//              leaves as bf16 without a pass of its own.
//   kGroupUp, kGroupDown  the same products on expert-sorted rows (up to 16
//              of one expert per workgroup); kGroupDown's leave as fp32.
#include <algorithm>
#include <type_traits>

#include "mx_device.hpp"
#include "mx_internal.hpp"
#include "nvfp4_dma.hpp"

namespace nvfp4 {

namespace {

// Waves of a workgroup: eight, or four where a wave has four weight tiles and
// more than 128 registers, so that several workgroups share a CU (one loads
// while another adds up).
constexpr int waves_of(int nr) { return nr == 4 ? 4 : 8; }
// Waves per SIMD: four, or three where a wave has four tiles, between what the
// large layers and the small ones like best (two / three / four; 64 tokens, 8 of
// 256 experts, 6144 x 2048: 823 / 840 / 889 us, 2048 x 1024: 162 / 163 / 157).
constexpr int wpe_of(int nr, int mb) { return nr * mb <= 2 ? 4 : 3; }

// One operand: uniform bases of codes and scales and the bytes that are
// reached from them, all below 2 GiB.
struct Rows {
    const uint8_t* codes;
    const uint8_t* scales;
    uint32_t code_bytes, scale_bytes;
};
// A row of it as a lane sees it: offsets of its piece of the codes and of the
// row's scales.
struct RowAt {
    uint32_t c, s;
};

// codes and scale words of one 128-element step for this lane.
struct Step {
    u32x4 c;
    uint32_t s;
};

// A unit of K: USTEPS steps of 128 elements whose scale bytes of a row are
// one aligned load (4: 16 bytes, 2: 8 bytes); 1: K is no multiple of 256 and
// the scale bytes are loaded one by one.
template <int USTEPS>
struct Unit {
    Step st[USTEPS];
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const uint8_t* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)bytes, (int)kRsrcWord3);
}

// A unit that is not live, and blocks past K, are pushed out of range: they
// read as zeros, without a memory access.  (The scalar offset stays inside the
// buffer, so that the range check holds whichever way it counts it.)  Loads
// that keep their lines, not non-temporal ones: an instruction reads half a
// cache line of each row and the next one the other half, which a line that is
// not kept fetches again (one token's layer of 8 experts, 6144 x 2048: 41.0
// against 36.4 us; 64 tokens, 8 of 256: 1092 against 868).
template <int USTEPS>
__device__ __forceinline__ Unit<USTEPS> load_unit(const Rows& r, const RowAt& at, int unit, bool live, int g, int nblk) {
    Unit<USTEPS> u;
    const auto rc = buffer(r.codes, r.code_bytes), rs = buffer(r.scales, r.scale_bytes);
    if constexpr (USTEPS > 1) {
        const uint32_t dead = live ? 0u : kOob;
        unit = live ? unit : 0;
        const int vc = (int)(at.c | dead), vs = (int)(at.s | dead);
#pragma unroll
        for (int i = 0; i < USTEPS; ++i)
            u.st[i].c = __builtin_amdgcn_raw_buffer_load_b128(rc, vc + 64 * i, unit * (64 * USTEPS), 0);
        if constexpr (USTEPS == 4) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, vs, unit * 16, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) u.st[i].s = v[i];
        } else {
            const auto v = __builtin_amdgcn_raw_buffer_load_b64(rs, vs, unit * 8, 0);
            u.st[0].s = v[0];
            u.st[1].s = v[1];
        }
    } else {
        const uint32_t dead = live && 4 * unit + g < nblk ? 0u : kOob;
        unit = live ? unit : 0;
        u.st[0].c = __builtin_amdgcn_raw_buffer_load_b128(rc, (int)(at.c | dead), unit * 64, 0);
        u.st[0].s = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)((at.s + g) | dead), unit * 4, 0);
    }
    return u;
}
// The same of an activation in LDS (a live unit).
template <int USTEPS>
__device__ __forceinline__ Unit<USTEPS> lds_unit(const uint8_t* codes, const uint8_t* scales, int unit, int g, int nblk) {
    Unit<USTEPS> u;
    if constexpr (USTEPS > 1) {
        const uint8_t* c = codes + unit * (64 * USTEPS) + 16 * g;
#pragma unroll
        for (int i = 0; i < USTEPS; ++i) {
            u.st[i].c = *reinterpret_cast<const u32x4*>(c + 64 * i);
            u.st[i].s = *reinterpret_cast<const uint32_t*>(scales + unit * (4 * USTEPS) + 4 * i);
        }
    } else {
        const int b = 4 * unit + g;
        u.st[0].c = u32x4{0, 0, 0, 0};
        u.st[0].s = 0;
        if (b < nblk) {
            u.st[0].c = *reinterpret_cast<const u32x4*>(codes + b * 16);
            u.st[0].s = scales[b];
        }
    }
    return u;
}

// A wave quantizes its K slice of `rows` bf16 rows (blocks [b0, b0 + blocks) of
// each) into its own LDS: codes, `cap` 16-byte blocks a row, then scale bytes.
// Item i is block i % blocks of row i / blocks.  load() is apart from store()
// so that the first items can be asked for before the weights, whose loads
// would otherwise have to return first.
struct SliceItem {
    uint4 v[4];
    __device__ __forceinline__ void load(const uint16_t* x, int64_t K, int b0, int blocks, int i) {
        const int m = i / blocks, b = i - m * blocks;
        const uint4* p = reinterpret_cast<const uint4*>(x + m * K + (int64_t)(b0 + b) * 32);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = p[q];
    }
    __device__ __forceinline__ void store(uint8_t* lc, uint8_t* ls, int cap, int blocks, int i) {
        const int m = i / blocks, b = i - m * blocks;
        uint32_t mx = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            asm("" : "+v"(v[q].x), "+v"(v[q].y), "+v"(v[q].z), "+v"(v[q].w));  // (opaque until here, as in Stream)
            mx = max_bf16x2(mx, v[q].x);
            mx = max_bf16x2(mx, v[q].y);
            mx = max_bf16x2(mx, v[q].z);
            mx = max_bf16x2(mx, v[q].w);
        }
        const uint32_t s = mx_scale_byte(mx);
        const float d = mx_divisor(s);
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = mx_encode8(v[q].x, v[q].y, v[q].z, v[q].w, d);
        *reinterpret_cast<u32x4*>(lc + ((size_t)m * cap + b) * 16) = o;
        ls[(size_t)m * cap + b] = (uint8_t)s;
    }
};

// The same for packed rows, which are only copied: a lane then loads its piece
// of the activation once, where the operand's layout has every 16 lanes load a
// row again with each unit of weights (one packed row through 6144 x 16384 15.8
// -> 12.5 us, four 16.4 -> 14.3, a token's layer of 8 experts 39.1 -> 36.4).
struct PackedItem {
    u32x4 c;
    uint32_t s;
    __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int64_t KB, int b0, int blocks, int i) {
        const int m = i / blocks, b = b0 + i - m * blocks;
        c = *reinterpret_cast<const u32x4*>(codes + m * KB + (int64_t)b * 16);
        s = scales[m * (KB / 16) + b];
    }
    __device__ __forceinline__ void store(uint8_t* lc, uint8_t* ls, int cap, int blocks, int i) {
        const int m = i / blocks, b = i - m * blocks;
        asm("" : "+v"(s));
        *reinterpret_cast<u32x4*>(lc + ((size_t)m * cap + b) * 16) = c;
        ls[(size_t)m * cap + b] = (uint8_t)s;
    }
};

// D units in flight: their weights, and the packed activations (A_LDS: these
// are in LDS, and read when they are used).
//
// The compiler counts the loads in flight where it needs one of them, but past
// a branch around a load it cannot, and waits for all; and it moves arithmetic
// on a loaded word up to the load, and waits there.  So no load is branched
// around, and the scale words are opaque until they are used.
template <int NR, int MB, int USTEPS, int D, bool A_LDS>
struct Stream {
    Rows wr, ar;                // weights, activations
    RowAt w_at[NR], a_at[MB];
    const uint8_t* a_codes;     // A_LDS: the row in LDS, from unit 0
    const uint8_t* a_scales;
    Unit<USTEPS> w[D][NR];
    Unit<USTEPS> a[A_LDS ? 1 : D][A_LDS ? 1 : MB];

    __device__ __forceinline__ void fetch(int u, int u1, int slot, int g, int nblk) {
        __builtin_amdgcn_sched_barrier(0);
        const bool live = u < u1;
#pragma unroll
        for (int i = 0; i < NR; ++i) w[slot][i] = load_unit<USTEPS>(wr, w_at[i], u, live, g, nblk);
        if constexpr (!A_LDS)
#pragma unroll
            for (int m = 0; m < MB; ++m) a[slot][m] = load_unit<USTEPS>(ar, a_at[m], u, live, g, nblk);
        __builtin_amdgcn_sched_barrier(0);
    }
    __device__ __forceinline__ void start(int u0, int u1, int g, int nblk) {
#pragma unroll
        for (int c = 0; c < D; ++c) fetch(u0 + c, u1, c, g, nblk);
    }
    __device__ __forceinline__ void use(f32x4 (&acc)[NR][MB], int u, int slot, int g, int nblk) {
        auto scale = [&](uint32_t s) -> uint32_t {
            asm("" : "+v"(s));
            return USTEPS > 1 ? s >> (8 * g) : s;
        };
        Unit<USTEPS> av[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if constexpr (A_LDS) av[m] = lds_unit<USTEPS>(a_codes, a_scales, u, g, nblk);
            else av[m] = a[slot][m];
        }
#pragma unroll
        for (int s = 0; s < USTEPS; ++s) {
            uint32_t sa[MB];
#pragma unroll
            for (int m = 0; m < MB; ++m) sa[m] = scale(av[m].st[s].s);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const uint32_t sw = scale(w[slot][i].st[s].s);
#pragma unroll
                for (int m = 0; m < MB; ++m)
                    acc[i][m] = mx_mfma16<0, 0>(w[slot][i].st[s].c, av[m].st[s].c, acc[i][m], sw, sa[m]);
            }
        }
    }
    // acc += W A^T over units [u0, u1), the first D of which start() asked for
    __device__ __forceinline__ void run(f32x4 (&acc)[NR][MB], int u0, int u1, int g, int nblk) {
        int u = u0;
        for (; u + D < u1; u += D)
#pragma unroll
            for (int c = 0; c < D; ++c) {
                use(acc, u + c, c, g, nblk);
                fetch(u + c + D, u1, c, g, nblk);
            }
#pragma unroll
        for (int c = 0; c < D; ++c)
            if (u + c < u1) use(acc, u + c, c, g, nblk);
    }
};

enum class Mode : int { kPlain = 0, kSlotUp = 1, kSlotDown = 2, kGroupUp = 3, kGroupDown = 4 };

// SRC: each wave reads the activation, packed, from memory as it goes; or
// first quantizes its K slice of a bf16 activation into LDS, or copies that of
// a packed one.  The LDS of a wave: `slice` blocks per row.
enum class Src : int { kMemory = 0, kQuantize = 1, kCopy = 2 };

template <int NR, int MB, int USTEPS, Mode MODE, Src SRC, int D>
__global__ __launch_bounds__(64 * waves_of(NR)) __attribute__((amdgpu_waves_per_eu(wpe_of(NR, MB))))
void k_mx_stream(MxStreamArgs g) {
    constexpr int kWaves = waves_of(NR), kThreads = 64 * kWaves;
    constexpr bool kUp = MODE == Mode::kSlotUp || MODE == Mode::kGroupUp;
    static_assert(!kUp || NR == 4, "gate/up: two tiles each");
    constexpr bool kLds = SRC != Src::kMemory;
    static_assert(MB == 1 || !kLds, "LDS holds up to 16 rows");
    Stream<NR, MB, USTEPS, D, kLds> st;
    extern __shared__ __align__(16) uint8_t smem[];
    float* const red = reinterpret_cast<float*>(smem);  // [wave][tile][lane][4]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int l16 = lane & 15, lg = lane >> 4;

    const int64_t KB = g.K / 2, KS = g.K / 32;
    const int nblk = (int)KS;
    const int units = (int)((g.K + 128 * USTEPS - 1) / (128 * USTEPS));

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
    const int64_t n0 = (int64_t)tn * (kUp ? 32 : g.rt * NR);
    const int64_t half = g.N / 2;  // kUp: I
    // weight rows of tile i, of which the first rt are the tile's (see
    // rows_per_tile); others, and rows past N, repeat one and are never stored
    const int rt = kUp ? 16 : g.rt;
    auto w_row = [&](int i) -> uint32_t {  // from n0 on
        if constexpr (kUp) return (uint32_t)(i < 2 ? 0 : half) + 16 * (i & 1) + l16;
        return (uint32_t)min((int64_t)(rt * i + min(l16, rt - 1)), g.N - 1 - n0);
    };
    auto weights = [&](int64_t e) {
        const int64_t r0 = e * g.N + n0, rows = kUp ? half + 32 : min((int64_t)(16 * NR), g.N - n0);
        st.wr = {g.b_codes + r0 * KB, g.b_scales + r0 * KS, (uint32_t)(rows * KB), (uint32_t)(rows * KS)};
#pragma unroll
        for (int i = 0; i < NR; ++i) st.w_at[i] = {w_row(i) * (uint32_t)KB + 16u * lg, w_row(i) * (uint32_t)KS};
    };

    // units [u0, u1) of `rows` activation rows into this wave's own LDS, the
    // first loads of them before those of the weights and stored after; the
    // operand reads see them through pointers that start at unit 0
    auto stage = [&](int rows, int u0, int u1, const uint16_t* x, const uint8_t* codes, const uint8_t* scales) {
        constexpr int kBpu = 4 * USTEPS;  // blocks per unit
        const int b0 = u0 * kBpu, blocks = max(min(u1 * kBpu, nblk) - b0, 0);
        const int cap = g.slice;  // blocks a wave's row may hold, a multiple of 16
        uint8_t* const lc = smem + (size_t)wave * rows * cap * 17;
        uint8_t* const ls = lc + (size_t)rows * cap * 16;
        const int items = rows * blocks;
        auto copy = [&](auto item, auto load) {
            if (lane < items) load(item, lane);
            st.start(u0, u1, lg, nblk);
            if (lane < items) item.store(lc, ls, cap, blocks, lane);
            for (int i = lane + 64; i < items; i += 64) {
                load(item, i);
                item.store(lc, ls, cap, blocks, i);
            }
        };
        if constexpr (SRC == Src::kQuantize)
            copy(SliceItem(), [&](SliceItem& it, int i) { it.load(x, g.K, b0, blocks, i); });
        else
            copy(PackedItem(), [&](PackedItem& it, int i) { it.load(codes, scales, KB, b0, blocks, i); });
        const int mr = l16 < rows ? l16 : 0;
        st.a_codes = lc + (mr * cap - b0) * 16;
        st.a_scales = ls + mr * cap - b0;
        __builtin_amdgcn_wave_barrier();
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
            weights(e);
            if constexpr (!kLds) {
                st.ar = {g.a_codes + s * KB, g.a_scales + s * KS, (uint32_t)KB, (uint32_t)KS};
                st.a_at[0] = {16u * lg, 0u};
            }
            f32x4 part[NR][1];
#pragma unroll
            for (int i = 0; i < NR; ++i) part[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (kLds) stage(1, u0, u1, nullptr, g.a_codes + s * KB, g.a_scales + s * KS);
            else st.start(u0, u1, lg, nblk);
            st.run(part, u0, u1, lg, nblk);
#pragma unroll
            for (int i = 0; i < NR; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][0][r] = __builtin_fmaf(wj, part[i][0][r], acc[i][0][r]);
        }
    } else {
        const int u0 = wave * units / kWaves, u1 = (wave + 1) * units / kWaves;
        weights(expert);
        if constexpr (SRC == Src::kQuantize)
            stage(MODE == Mode::kPlain ? (int)g.M : 1, u0, u1, g.x + (MODE == Mode::kPlain ? 0 : row_beg / g.top_k) * g.K,
                  nullptr, nullptr);
        else if constexpr (SRC == Src::kCopy) {
            stage((int)g.M, u0, u1, nullptr, g.a_codes, g.a_scales);
        } else {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                int64_t r = row_beg + 16 * m + l16;
                if (r >= row_end) r = row_beg;
                if constexpr (MODE == Mode::kGroupUp) r = g.perm[r] / g.top_k;
                st.a_at[m] = {(uint32_t)(r * KB) + 16u * lg, (uint32_t)(r * KS)};
            }
            st.ar = {g.a_codes, g.a_scales, kOob, kOob};  // (rows below 2 GiB, all of them there)
            st.start(u0, u1, lg, nblk);
        }
        st.run(acc, u0, u1, lg, nblk);
    }
    if constexpr (kLds) __syncthreads();  // the sums below reuse the slices' LDS

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
            const int64_t col = n0 + rt * (t / MB) + 4 * (ln >> 4);
            if (row >= row_end || col >= g.N || 4 * (ln >> 4) >= rt) continue;
            const f32x4 v = total(t, ln);
            if constexpr (MODE == Mode::kGroupDown) {
                *reinterpret_cast<f32x4*>(g.slot_y + row * g.N + col) = v;  // (N is a multiple of 32)
            } else {
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

// The largest share of one row that a wave quantizes, in blocks, rounded up to
// 16.
int slice_of(int64_t K, int usteps, int waves) {
    const int64_t units = (K + 128 * usteps - 1) / (128 * usteps);
    return (int)(((units + waves - 1) / waves * 4 * usteps + 15) / 16 * 16);
}

// Weight rows of a tile: 16, or 12 or 8 where that spreads the tiles more
// evenly over the 256 CUs (6144 rows: 384 tiles of 16 leave half the CUs with
// two and half with one; 512 of 12 give each two: one token through 6144 x
// 16384 14.4 -> 13.2 us, packed 13.5 -> 12.5, through 8 experts of 6144 x 2048
// 38.5 -> 36.4).  With more than 16 activation rows a workgroup's reads of
// them count, and fewer, whole tiles win (37 x 4099 x 2080: 6.0 against 7.1).
int rows_per_tile(int64_t N, int nr) {
    auto most = [&](int64_t rt) { return ((N + rt * nr - 1) / (rt * nr) + 255) / 256 * rt; };  // rows of the fullest CU
    int rt = 16;
    for (int r = 12; r >= 8; r -= 4)
        if (most(r) < most(rt)) rt = r;
    return rt;
}

// Units in flight: 16 code loads a lane of weights alone, 8 and their
// activation's (4 where the scale bytes come one by one); at least two units.
template <int NR, int MB, int USTEPS, Src SRC>
constexpr int units_in_flight() {
    constexpr int steps = USTEPS == 1 ? 2 : SRC != Src::kMemory ? 16 : MB == 1 ? 8 : 4;
    return std::max(2, steps / (USTEPS * NR));
}

template <int NR, int MB, int USTEPS, Mode MODE, Src SRC>
hipError_t launch_one(MxStreamArgs g, int64_t mtiles, hipStream_t stream) {
    constexpr int kWaves = waves_of(NR), kThreads = 64 * kWaves;
    constexpr bool kUp = MODE == Mode::kSlotUp || MODE == Mode::kGroupUp;
    g.rt = kUp || MODE == Mode::kGroupDown || MB > 1 ? 16 : rows_per_tile(g.N, NR);
    g.ntiles = (int32_t)(kUp ? (g.N / 2 + 31) / 32 : (g.N + g.rt * NR - 1) / (g.rt * NR));
    const int64_t wgs = mtiles * g.ntiles;
    if (wgs < 1 || wgs >= ((int64_t)1 << 32) / kThreads) return hipErrorInvalidValue;
    size_t lds = (size_t)kWaves * NR * MB * 1024;
    if (SRC != Src::kMemory) {
        g.slice = slice_of(g.K, USTEPS, MODE == Mode::kSlotDown ? 1 : kWaves);  // (a wave may have a slot's whole row)
        lds = std::max(lds, (size_t)kWaves * (MODE == Mode::kPlain ? (size_t)g.M : 1) * g.slice * 17);
    }
    if (lds > 64 * 1024) return hipErrorInvalidValue;
    // (a unit past a wave's last still issues its loads: two where it has no
    // more; 37 x 4099 x 2080 with four 11.5, with two 9.6 us)
    constexpr int D = units_in_flight<NR, MB, USTEPS, SRC>();
    if constexpr (MODE == Mode::kPlain && D > 2)
        if (g.K <= (int64_t)2 * kWaves * 128 * USTEPS) {
            hipLaunchKernelGGL((k_mx_stream<NR, MB, USTEPS, MODE, SRC, 2>), dim3((unsigned)wgs), dim3(kThreads), lds,
                               stream, g);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((k_mx_stream<NR, MB, USTEPS, MODE, SRC, D>), dim3((unsigned)wgs), dim3(kThreads), lds, stream, g);
    return hipGetLastError();
}

template <int NR, int MB, Mode MODE, Src SRC>
hipError_t launch_k(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream) {
    // units of four steps where one tile's waves then share them evenly
    if constexpr (NR == 1 && MB == 1 && MODE == Mode::kPlain)
        if (g.K % (512 * 8) == 0) return launch_one<NR, MB, 4, MODE, SRC>(g, mtiles, stream);
    if (g.K % 256 == 0) return launch_one<NR, MB, 2, MODE, SRC>(g, mtiles, stream);
    return launch_one<NR, MB, 1, MODE, SRC>(g, mtiles, stream);
}

}  // namespace

// Every workgroup quantizes the rows for itself: through 6144 x 16384 two rows
// take 15.9 us that way (14.3 for four packed ones), three 17.4 against 16.7
// with a launch of its own, four 18.7 against 17.4.  (LDS: the
// largest of the forms, four waves, units of up to four steps.)
static bool fits_lds(int64_t M, int64_t K) {
    return K <= ((int64_t)1 << 20) && M * (K / 32 + 16 * 8) * 17 <= 64 * 1024;
}
bool mx_stream_quantizes(int64_t M, int64_t K) { return M <= 2 && fits_lds(M, K); }
bool mx_slots_fit(int64_t H) { return mx_stream_quantizes(1, H); }

// 16-row weight tiles of a wave in the plain form: one while that gives at most
// 512 workgroups or the rows are long (and a launch holds them: fewer than 2^23
// workgroups of 512 threads, two to a tile at most), else two or (up to 16
// activation rows) four.
static int plain_tiles(int64_t M, int64_t N, int64_t K) {
    const int64_t t1 = (N + 15) / 16;
    const int nr = t1 <= 512 || (K >= 8192 && t1 < (1 << 22)) ? 1 : t1 <= 1024 ? 2 : 4;
    return M <= 16 ? nr : M <= 32 ? std::min(nr, 2) : 1;
}

// Every workgroup reads the activation, so with more rows that becomes the
// larger stream.  Streaming against the LDS tiles, us: 6144 x 16384 4 rows 13.7
// / 20.8, 8 16.9 / 21.0, 16 19.9 / 21.1, 32 35.6 / 22.3, 64 58.0 / 25.0; 16384 x
// 2048 16 rows 7.1 / 12.1, 32 9.6 / 12.4, 64 20.9 / 12.6.  (The border was set
// with the weights in the last-level cache, where the tiles take 17 at 6144 x
// 16384: from memory 8 and 16 rows of it lie on the wrong side, by 4 and 1 us.)
bool mx_stream_takes(int64_t M, int64_t N, int64_t K) {
    if (M > 64) return false;
    if (M <= 4) return true;
    const int64_t nr = plain_tiles(M, N, K), wgs = (N + 16 * nr - 1) / (16 * nr);
    return wgs <= ((int64_t)20 << 20) / (M * (K / 2));
}

hipError_t launch_mx_stream(const MxStreamArgs& g, hipStream_t stream) {
    const int nr = plain_tiles(g.M, g.N, g.K);
    auto rows16 = [&](auto src) {
        constexpr Src S = decltype(src)::value;
        return nr == 1 ? launch_k<1, 1, Mode::kPlain, S>(g, 1, stream)
                       : nr == 2 ? launch_k<2, 1, Mode::kPlain, S>(g, 1, stream)
                                 : launch_k<4, 1, Mode::kPlain, S>(g, 1, stream);
    };
    if (g.x != nullptr) return rows16(std::integral_constant<Src, Src::kQuantize>{});
    if (g.M <= 16)
        return fits_lds(g.M, g.K) ? rows16(std::integral_constant<Src, Src::kCopy>{})
                                  : rows16(std::integral_constant<Src, Src::kMemory>{});
    if (g.M <= 32)
        return nr == 1 ? launch_k<1, 2, Mode::kPlain, Src::kMemory>(g, 1, stream)
                       : launch_k<2, 2, Mode::kPlain, Src::kMemory>(g, 1, stream);
    if (g.M <= 64)
        return launch_k<1, 4, Mode::kPlain, Src::kMemory>(g, 1, stream);
    return hipErrorInvalidValue;
}

hipError_t launch_mx_slot_up(const MxStreamArgs& g, int64_t slots, hipStream_t stream) {
    return launch_k<4, 1, Mode::kSlotUp, Src::kQuantize>(g, slots, stream);
}
hipError_t launch_mx_slot_down(const MxStreamArgs& g, int64_t tokens, hipStream_t stream) {
    return fits_lds(8, g.K) ? launch_k<1, 1, Mode::kSlotDown, Src::kCopy>(g, tokens, stream)
                            : launch_k<1, 1, Mode::kSlotDown, Src::kMemory>(g, tokens, stream);
}
hipError_t launch_mx_group_up(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream) {
    return launch_k<4, 1, Mode::kGroupUp, Src::kMemory>(g, mtiles, stream);
}
hipError_t launch_mx_group_down(const MxStreamArgs& g, int64_t mtiles, hipStream_t stream) {
    return launch_k<4, 1, Mode::kGroupDown, Src::kMemory>(g, mtiles, stream);
}

}  // namespace nvfp4
