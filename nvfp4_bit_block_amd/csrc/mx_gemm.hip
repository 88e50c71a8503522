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
// K step: 256 elements (128 code bytes, a cache line, and 8 scale bytes a
// row), four instructions deep.  A K permutation applied to both operands
// leaves the product unchanged: lane half hf = lane / 32 takes blocks
// 4 hf + kk of the step in instruction kk, so its four scale bytes are one
// word and byte kk is selected by the instruction.
//
// Codes go from global memory straight into LDS (buffer_load ... lds, 1 KB =
// 8 rows per instruction) through NS stages, one barrier per step.  LDS rows
// are not padded: row r keeps its 16-byte chunk c in slot c ^ ((r / 2) % 8),
// so that 16 consecutive rows' fragment reads cover all banks.  Blocks past K
// and rows past the operand load as zeros.
#include "mx_device.hpp"
#include "mx_internal.hpp"
#include "nvfp4_dma.hpp"

#include <type_traits>

namespace nvfp4 {

namespace {

constexpr int kWaitAll = vmcnt_imm(0) & ~0xF00;  // vector memory and LDS
constexpr int kGroupM = 8;  // row tiles per band in the ungrouped tile order

template <int SEL>
__device__ __forceinline__ f32x16 mfma_kk(u32x4 w, u32x4 a, f32x16 c, uint32_t sw, uint32_t sa) {
    return mx_mfma32<SEL, SEL>(w, a, c, sw, sa);
}

// TM, TN: 32-row blocks of activations and of weights per wave; WM x WN
// waves; NS stages.  The activation blocks are dealt to the wave rows in turn
// (wave row wm has blocks wm, wm + WM, ..), and a tile of fewer rows runs a
// main loop of as many blocks as its fullest wave has.  ALIGNED: K % 128 == 0,
// so a row's scale bytes are whole words (else they are read byte by byte).
template <int TM, int TN, int WM, int WN, int NS, MxEpi EP, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm(MxGemmArgs g) {
    constexpr int NW = WM * WN, NT = 64 * NW;
    constexpr int WTN = 32 * TN, BM = 32 * TM * WM, BN = WTN * WN;
    constexpr int SLABS = (BM + BN) / 8, CODES = SLABS / NW;  // code slabs of 1 KB: activations, then weights
    static_assert(SLABS % NW == 0, "copy");
    constexpr int SC_OFF = (BM + BN) * 128;
    constexpr int STAGE = SC_OFF + (BM + BN) * 8;
    constexpr int SC_SLABS = (BM + BN) / 32, SC_PER_W = (SC_SLABS + NW - 1) / NW;
    constexpr int SC_PER_T = (BM + BN + NT - 1) / NT;
    constexpr int LOADS = CODES + (ALIGNED ? SC_PER_W : 0);  // of a wave, per step
    static_assert(NS >= 2 && NS <= 3 && NS * STAGE <= 160 * 1024 && LOADS * (NS - 1) <= 63, "stages");
    constexpr bool kGateUp = EP == MxEpi::kGateUp;
    static_assert(!kGateUp || TN % 2 == 0, "gate/up pairs column blocks");
    __shared__ __align__(1024) uint8_t smem[NS * STAGE];

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
        // group by group, and within a group its row tiles of one column tile
        // together: they read the same weights
        const int mt = (int)(id / g.ntiles);
        int lo = 0, hi = g.groups;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (g.tile_off[mid] <= mt) lo = mid; else hi = mid;
        }
        grp = lo;
        const int r = (int)(id - (int64_t)g.tile_off[grp] * g.ntiles), mts = g.tile_off[grp + 1] - g.tile_off[grp];
        tn = r / mts;
        row_beg = (int64_t)g.row_off[grp] + (int64_t)(r - tn * mts) * BM;
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

    // ---- copy assignments.  Code slab sl: tile rows 8 sl + lane / 8 (the
    // activations', then the weights'), slot lane % 8, which holds chunk
    // slot ^ ((r / 2) % 8).
    auto tile_row = [&](int r) -> int64_t { return r < BM ? a_row(r) : r < BM + BN ? b_row(r - BM) : -1; };
    uint32_t vc[CODES];
    // (r / 2) % 8 of row 8 sl + lane / 8 depends on sl's parity
    const int slot = lane & 7, rhalf = lane >> 4;
#pragma unroll
    for (int u = 0; u < CODES; ++u) {
        const int sl = CODES * wave + u;
        const int64_t src = tile_row(8 * sl + (lane >> 3));
        vc[u] = src < 0 ? kOob : (uint32_t)src * KB + 16u * (slot ^ (4 * (sl & 1) + rhalf));
    }
    // scales.  ALIGNED: slab sl holds tile rows 32 sl + lane / 2, word lane %
    // 2.  Otherwise thread t carries tile rows t, t + NT, .. of one step
    // through registers.
    const u32x4 rsa = make_rsrc(g.a_scales + a0 * KS, (uint64_t)(gather ? g.a_src_rows : row_end - row_beg) * KS);
    const u32x4 rsb = make_rsrc(g.b_scales + ((int64_t)grp * g.N + n0) * KS,
                                (uint64_t)(kGateUp || brows < BN ? brows : BN) * KS);
    // (slabs beyond an even deal repeat the last one)
    auto sc_slab = [&](int u) { return min(SC_PER_W * wave + u, SC_SLABS - 1); };
    uint32_t vs[ALIGNED ? SC_PER_W : 1];
    const uint8_t* sp[ALIGNED ? 1 : SC_PER_T];
    bool sok[ALIGNED ? 1 : SC_PER_T];
    uint2 sv[ALIGNED ? 1 : SC_PER_T];
    if constexpr (ALIGNED) {
#pragma unroll
        for (int u = 0; u < SC_PER_W; ++u) {
            const int64_t src = tile_row(32 * sc_slab(u) + (lane >> 1));
            vs[u] = src < 0 ? kOob : (uint32_t)src * KS + 4u * (lane & 1);
        }
    } else {
        const uint8_t* const as = g.a_scales + a0 * KS;
        const uint8_t* const bs = g.b_scales + ((int64_t)grp * g.N + n0) * KS;
#pragma unroll
        for (int u = 0; u < SC_PER_T; ++u) {
            const int r = tid + u * NT;
            const int64_t src = tile_row(r);
            sp[u] = (r < BM ? as : bs) + max(src, (int64_t)0) * KS;  // (a row that is there, if none is meant)
            sok[u] = src >= 0;
        }
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
    auto load_scales = [&](int kc) {
        if constexpr (!ALIGNED) {
            const int nb = kc + 1 < nsteps ? 8 : tail;
#pragma unroll
            for (int u = 0; u < SC_PER_T; ++u) {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const uint32_t v = sp[u][8 * kc + min(b, nb - 1)];
                    w[b >> 2] |= (sok[u] && b < nb ? v : 0u) << (8 * (b & 3));
                }
                sv[u] = make_uint2(w[0], w[1]);
            }
        }
    };
    auto store_scales = [&](uint32_t stage) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int u = 0; u < SC_PER_T; ++u) {
                const int r = tid + u * NT;
                if (r < BM + BN) *reinterpret_cast<uint2*>(smem + stage + SC_OFF + 8 * r) = sv[u];
            }
        }
    };
    // Load p (0 .. LOADS - 1) of this wave for step kc into a stage.  In the
    // last step the chunks (and scale words) past K are pushed out of range,
    // and steps past the last load nothing: a resource of no bytes, at offset
    // zero so that the range check holds whichever way it counts the offset.
    auto issue = [&](int p, int kc, uint32_t stage) {
        const bool live = kc < nsteps, last = kc + 1 == nsteps;
        const bool code = p < CODES;
        const int sl = code ? CODES * wave + p : sc_slab(p - CODES);
        const bool isa = code ? 8 * sl < BM : 32 * sl < BM;
        u32x4 r = code ? (isa ? ra : rb) : (isa ? rsa : rsb);
        r.x = __builtin_amdgcn_readfirstlane(r.x);
        r.y = __builtin_amdgcn_readfirstlane(r.y);
        r.z = __builtin_amdgcn_readfirstlane(live ? r.z : 0u);
        r.w = kRsrcWord3;
        const uint32_t k = live ? (uint32_t)kc : 0u;
        if (code) {
            const uint32_t cut = last && (slot ^ (4 * (sl & 1) + rhalf)) >= tail ? kOob : 0u;
            lds_load16(r, vc[code ? p : 0] | cut, k * 128u, lds0 + stage + (uint32_t)(sl * 1024));
        } else {
            const uint32_t cut = last && 4 * (lane & 1) >= tail ? kOob : 0u;
            lds_load4(r, vs[code ? 0 : p - CODES] | cut, k * 8u, lds0 + stage + (uint32_t)(SC_OFF + 256 * sl));
        }
    };

    f32x16 acc[TN][TM];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    // ---- main loop.  The fragments of the next instruction are read among
    // the instructions of this one, into the other half of the fragment
    // registers.  The step's barrier stands before its last quarter: by then
    // every fragment of the step is in registers, so the stage is free, and
    // the next step has landed (only the loads of the steps after it may be
    // out); the last quarter's instructions cover the first reads of the next
    // step and the issue of the loads into the freed stage.  The scheduling
    // barriers keep that order, and the body must not branch: the matrix
    // instructions, which the compiler sees without side effects, otherwise
    // sink below the last branch and nothing overlaps (325 us against 239 us
    // at 4096 x 6144 x 16384, tiles of 256 x 256).
    uint32_t off_k[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) off_k[kk] = (uint32_t)(c32 * 128 + 16 * ((4 * hf + kk) ^ ((c32 >> 1) & 7)));
    const uint32_t a_off = (uint32_t)(wm * 32 * 128), b_off = (uint32_t)((BM + wn * WTN) * 128);
    const uint32_t sa_off = (uint32_t)(SC_OFF + 8 * (32 * wm + c32) + 4 * hf);
    const uint32_t sb_off = (uint32_t)(SC_OFF + 8 * (BM + wn * WTN + c32) + 4 * hf);
    load_scales(0);
    store_scales(0);
    load_scales(min(1, nsteps - 1));
#pragma unroll
    for (int t = 0; t < NS; ++t)
#pragma unroll
        for (int p = 0; p < LOADS; ++p) issue(p, t, t * STAGE);
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (NS - 1)) & ~0xF00);
    __syncthreads();
    auto main_loop = [&](auto tmc) {
        constexpr int TA = decltype(tmc)::value;  // activation blocks in use
        u32x4 fa[2][TA], fb[2][TN];
        uint32_t sa[TA], sb[TN];
        auto read_frag = [&](int q, uint32_t stage, int kk, int buf) {  // q: 0 .. TA + TN - 1
            if (q < TA)
                fa[buf][q] = *reinterpret_cast<const u32x4*>(smem + (stage + off_k[kk] + a_off) + 4096 * WM * q);
            else
                fb[buf][q - TA] = *reinterpret_cast<const u32x4*>(smem + (stage + off_k[kk] + b_off) + 4096 * (q - TA));
        };
        auto read_scales = [&](uint32_t stage, uint32_t (&da)[TA], uint32_t (&db)[TN]) {
#pragma unroll
            for (int i = 0; i < TA; ++i)
                da[i] = *reinterpret_cast<const uint32_t*>(smem + (stage + sa_off) + 256 * WM * i);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                db[j] = *reinterpret_cast<const uint32_t*>(smem + (stage + sb_off) + 256 * j);
        };
        read_scales(0, sa, sb);
#pragma unroll
        for (int q = 0; q < TA + TN; ++q) read_frag(q, 0, 0, 0);
        uint32_t cur = 0;
        for (int s = 0; s < nsteps; ++s) {
            const uint32_t nxt = cur + STAGE == NS * STAGE ? 0 : cur + STAGE;
            uint32_t na[TA], nb[TN];
            auto group = [&](auto kkc) {
                constexpr int kk = decltype(kkc)::value, buf = kk & 1;
                if constexpr (kk == 3) {
                    __builtin_amdgcn_s_waitcnt(vmcnt_imm(LOADS * (NS - 2)) & ~0xF00);
                    store_scales(nxt);
                    __syncthreads();
                    read_scales(nxt, na, nb);
                    load_scales(min(s + 2, nsteps - 1));
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    constexpr int kR = (TA + TN + TN - 1) / TN, kL = (LOADS + TN - 1) / TN;
#pragma unroll
                    for (int q = j * kR; q < (j + 1) * kR && q < TA + TN; ++q)
                        read_frag(q, kk < 3 ? cur : nxt, (kk + 1) & 3, buf ^ 1);
#pragma unroll
                    for (int i = 0; i < TA; ++i)
                        acc[j][i] = mfma_kk<kk>(fb[buf][j], fa[buf][i], acc[j][i], sb[j], sa[i]);
                    if constexpr (kk == 3) {
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int p = j * kL; p < (j + 1) * kL && p < LOADS; ++p) issue(p, s + NS, cur);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            group(std::integral_constant<int, 2>{});
            group(std::integral_constant<int, 3>{});
#pragma unroll
            for (int i = 0; i < TA; ++i) sa[i] = na[i];
#pragma unroll
            for (int j = 0; j < TN; ++j) sb[j] = nb[j];
            cur = nxt;
        }
    };
    // blocks of the fullest wave row
    const int used = (int)((row_end - row_beg + 32 * WM - 1) / (32 * WM));
    if (TM >= 2 && used == 1) main_loop(std::integral_constant<int, 1>{});
    else if (TM >= 3 && used == 2) main_loop(std::integral_constant<int, TM >= 3 ? 2 : TM>{});
    else if (TM >= 4 && used == 3) main_loop(std::integral_constant<int, TM >= 4 ? 3 : TM>{});
    else main_loop(std::integral_constant<int, TM>{});
    __builtin_amdgcn_s_waitcnt(kWaitAll);

    // (the slabs below reuse the stages, which other waves may still read)
    if constexpr (EP == MxEpi::kStoreBf16) __syncthreads();

    // ---- epilogue: acc[j][i][r] is weight row 32 j + 8 (r / 4) + 4 hf + r % 4
    // of the wave, activation row 32 (i WM + wm) + c32.
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t row = row_beg + 32 * (i * WM + wm) + c32;
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
        } else if constexpr (EP == MxEpi::kDown) {
            if (row >= row_end) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    // (N is the hidden size, a multiple of 32)
                    const int64_t col = n0 + wn * WTN + 32 * j + 8 * p + 4 * hf;
                    if (col < nlim)
                        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(g.out) + row * g.ldo + col) =
                            f32x4{acc[j][i][4 * p], acc[j][i][4 * p + 1], acc[j][i][4 * p + 2], acc[j][i][4 * p + 3]};
                }
        } else {
            // a 32-row slab of the wave's tile meets in LDS and leaves as
            // 16-byte pieces of rows (pitch: 16 rows' 8-byte writes fall on
            // different banks)
            constexpr int kPitch = WTN * 2 + 16;
            static_assert(NW * 32 * kPitch <= NS * STAGE, "epilogue slabs");
            uint8_t* const slab = smem + wave * 32 * kPitch;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p)
                    *reinterpret_cast<uint2*>(slab + c32 * kPitch + 2 * (32 * j + 8 * p + 4 * hf)) =
                        make_uint2(f32_to_bf16(acc[j][i][4 * p]) | (f32_to_bf16(acc[j][i][4 * p + 1]) << 16),
                                   f32_to_bf16(acc[j][i][4 * p + 2]) | (f32_to_bf16(acc[j][i][4 * p + 3]) << 16));
            __builtin_amdgcn_wave_barrier();
            const int64_t row0 = row_beg + 32 * (i * WM + wm);
            const bool vec = (g.ldo & 7) == 0;
#pragma unroll
            for (int p = 0; p < 2 * TN; ++p) {
                const int e = 64 * p + lane, rr = e / (4 * TN), ch = e % (4 * TN);
                const uint4 v = *reinterpret_cast<const uint4*>(slab + rr * kPitch + 16 * ch);
                const int64_t col = n0 + wn * WTN + 8 * ch;
                if (row0 + rr >= row_end || col >= nlim) continue;
                uint16_t* const dst = reinterpret_cast<uint16_t*>(g.out) + (row0 + rr) * g.ldo + col;
                if (vec && col + 8 <= nlim) {
                    *reinterpret_cast<uint4*>(dst) = v;
                } else {
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        if (col + q < nlim) dst[q] = (uint16_t)(w[q >> 1] >> (16 * (q & 1)));
                }
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

template <int TM, int TN, int WM, int WN, int NS, MxEpi EP>
hipError_t launch_cfg(const MxGemmArgs& g0, int grid_m, hipStream_t stream) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    MxGemmArgs g = g0;
    const int64_t ncols = EP == MxEpi::kGateUp ? g.N / 2 : g.N, bn = EP == MxEpi::kGateUp ? BN / 2 : BN;
    g.ntiles = (int32_t)((ncols + bn - 1) / bn);
    const int64_t mt = g.groups > 0 ? grid_m : (g.M + BM - 1) / BM;
    int64_t wgs = mt * g.ntiles;
    if (g.groups > 0) wgs = (wgs + 7) / 8 * 8;  // a multiple of 8 for the XCD renumbering
    if (wgs < 1 || wgs >= ((int64_t)1 << 32) / (64 * WM * WN)) return hipErrorInvalidValue;
    if (g.K % 128 == 0)
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, NS, EP, true>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    else
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, NS, EP, false>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& g, MxEpi epi, int grid_m, hipStream_t stream) {
    switch (epi) {
        case MxEpi::kStoreBf16: return launch_cfg<2, 2, 2, 2, 2, MxEpi::kStoreBf16>(g, grid_m, stream);
        case MxEpi::kGateUp: return launch_cfg<2, 2, 2, 2, 2, MxEpi::kGateUp>(g, grid_m, stream);
        default: return launch_cfg<2, 2, 2, 2, 2, MxEpi::kDown>(g, grid_m, stream);
    }
}

}  // namespace nvfp4
