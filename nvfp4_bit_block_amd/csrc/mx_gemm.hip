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
// 8 rows per instruction), one barrier per step: activations through two
// stages, weights, which mostly come from farther away, through NS.  LDS rows
// are not padded: row r keeps its 16-byte chunk c in slot c ^ ((r / 2) % 8),
// so that 16 consecutive rows' fragment reads cover all banks.  A step's 8
// scale bytes of a row would cost a request to L2 like the 128 bytes of its
// codes; they come for RSTEP steps at a time into a ring of their own.
// Blocks past K and rows past the operand load as zeros.
//
// Bound by the matrix units' power on large plain products (4096 x 6144 x
// 16384 on MI355X: 220 to 230 us, 3.6 to 3.75 PFLOP/s; the instruction alone
// keeps 3.8 to 4.0 on random codes), by the weights on the routed layer (4096 tokens, 8 of 256
// experts of 6144 x 2048: 807 to 836 us for 3.8 GB and 530 to 541 us for 2.6 GB,
// read and written).
#include "mx_device.hpp"
#include "mx_internal.hpp"
#include "nvfp4_dma.hpp"

#include <algorithm>
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
// waves; NS weight stages; scales for RSTEP steps at a time.  The activation
// blocks are dealt to the wave rows in turn (wave row wm has blocks wm,
// wm + WM, ..), and a tile of fewer rows runs a main loop of as many blocks
// as its fullest wave has.  ALIGNED: K % 128 == 0,
// so a row's scale bytes are whole words (else each step's are shifted into
// place on their way through registers).
template <int TM, int TN, int WM, int WN, int NS, int RSTEP, MxEpi EP, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm(MxGemmArgs g) {
    constexpr int NW = WM * WN, NT = 64 * NW;
    constexpr int WTN = 32 * TN, BM = 32 * TM * WM, BN = WTN * WN;
    // code slabs of 1 KB, and how many of them a wave loads
    constexpr int CA = BM / 8 / NW, CB = BN / 8 / NW, CODES = CA + CB;
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "copy");
    constexpr int A_STAGE = BM * 128, B_STAGE = BN * 128, B_OFF = 2 * A_STAGE;
    // scale ring: two halves, each RSTEP steps' bytes of every row, in slabs
    // of 1 KB, one per wave and phase
    constexpr int SCB = 8 * RSTEP, SC_OFF = B_OFF + NS * B_STAGE, SC_HALF = (BM + BN) * SCB;
    constexpr int SCR = 1024 / SCB, LPR = SCB / 16;  // rows of a slab, lanes of a row
    constexpr int SC_SLABS = (BM + BN) / SCR, PHASES = (SC_SLABS + NW - 1) / NW;
    constexpr int SC_PER_T = (BM + BN + NT - 1) / NT;
    static_assert((RSTEP == 2 || RSTEP == 4) && BM % SCR == 0 && BN % SCR == 0 && PHASES <= RSTEP, "scales");
    static_assert(NS == 2 || NS == 3, "stages");
    constexpr int LDS = SC_OFF + 2 * SC_HALF;
    static_assert(LDS <= 160 * 1024, "LDS");
    constexpr bool kGateUp = EP == MxEpi::kGateUp;
    constexpr bool kSplit = EP == MxEpi::kPartialF32;
    static_assert(!kGateUp || TN % 2 == 0, "gate/up pairs column blocks");
    __shared__ __align__(1024) uint8_t smem[LDS];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int c32 = lane & 31, hf = lane >> 5;

    // ---- tile.  Workgroups reach the 8 XCDs round-robin by id; renumber so
    // that each XCD has a contiguous run of the real tiles.
    const int gm_tiles = g.groups > 0 ? g.tile_off[g.groups] : (int)((g.M + BM - 1) / BM);
    const int64_t tiles = (int64_t)gm_tiles * g.ntiles, total = tiles * (kSplit ? g.ksplit : 1);
    int64_t id = blockIdx.x;
    if ((gridDim.x & 7) == 0) {
        const int64_t per = (total + 7) >> 3, j = id >> 3;
        if (j >= per) return;
        id = (id & 7) * per + j;
    }
    if (id >= total) return;
    int kz = 0;
    if constexpr (kSplit) {
        kz = (int)(id / tiles);
        id -= kz * tiles;
    }
    int grp = 0, tn;
    int64_t row_beg, row_end;
    if (g.groups > 0) {
        // group by group, and within a group its row tiles of one column tile
        // together: they read the same weights
        grp = group_of_tile(g.tile_off, g.groups, (int)(id / g.ntiles));
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
    // this workgroup's K steps [k0, k0 + nsteps) of ksteps (k0 a multiple of
    // RSTEP)
    const int ksteps = (int)((KS + 7) / 8), k0 = kSplit ? kz * g.ksteps : 0;
    const int nsteps = kSplit ? min(g.ksteps, ksteps - k0) : ksteps;
    const int tail = (int)(KS - 8 * (uint32_t)(ksteps - 1));  // blocks of the last step, 1 .. 8

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

    // ---- copy assignments.  Code slab sl of an operand: its rows 8 sl +
    // lane / 8, slot lane % 8.  Load p of a wave: CA slabs of activations,
    // then CB of weights.
    auto tile_row = [&](int r) -> int64_t { return r < BM ? a_row(r) : r < BM + BN ? b_row(r - BM) : -1; };
    auto slab = [&](int p) { return p < CA ? CA * wave + p : CB * wave + p - CA; };
    // the chunk in this lane's slot of slab sl
    auto chunk_of = [&](int sl) { return (lane & 7) ^ (((8 * sl + (lane >> 3)) >> 1) & 7); };
    uint32_t vc[CODES];
#pragma unroll
    for (int p = 0; p < CODES; ++p) {
        const int r = 8 * slab(p) + (lane >> 3);
        const int64_t src = p < CA ? a_row(r) : b_row(r);
        vc[p] = src < 0 ? kOob : (uint32_t)src * KB + 16u * chunk_of(slab(p));
    }
    // scales.  ALIGNED: slab sl holds tile rows SCR sl + lane / LPR (the
    // activations', then the weights'), 16 bytes lane % LPR of theirs; in
    // phase p a wave loads slab p NW + wave.  Otherwise thread t carries tile
    // rows t, t + NT, .. of one step through registers, as the aligned words
    // that hold its bytes (so up to three bytes next to the tensor's are read).
    const uint8_t* const as = g.a_scales + a0 * KS;
    const uint8_t* const bs = g.b_scales + ((int64_t)grp * g.N + n0) * KS;
    const uint32_t da = ALIGNED ? 0u : (uint32_t)(uintptr_t)as & 3u, db = ALIGNED ? 0u : (uint32_t)(uintptr_t)bs & 3u;
    const u32x4 rsa = make_rsrc(as - da, ((uint64_t)(gather ? g.a_src_rows : row_end - row_beg) * KS + da + 3) & ~3ull);
    const u32x4 rsb = make_rsrc(bs - db, ((uint64_t)(kGateUp || brows < BN ? brows : BN) * KS + db + 3) & ~3ull);
    auto sc_slab = [&](int ph) { return min(ph * NW + wave, SC_SLABS - 1); };  // (one too many repeats the last)
    uint32_t vs[ALIGNED ? PHASES : SC_PER_T];
    uint2 sv[ALIGNED ? 1 : SC_PER_T];
#pragma unroll
    for (int u = 0; u < (ALIGNED ? PHASES : SC_PER_T); ++u) {
        const int r = ALIGNED ? SCR * sc_slab(u) + lane / LPR : tid + u * NT;
        const int64_t src = tile_row(r);
        vs[u] = src < 0 ? kOob : (uint32_t)src * KS + (ALIGNED ? 16u * (lane % LPR) : r < BM ? da : db);
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_address(smem));
    // Phase ph of the scales of steps RSTEP q .. RSTEP (q + 1) - 1 (a phase too
    // many repeats the last).  The bytes may run past the row, whose
    // neighbour's bytes no step uses, and past the tensor, where the range
    // check, made word by word, gives zeros.
    auto issue_scales = [&](int ph, int q) {
        if constexpr (ALIGNED) {
            ph = min(ph, PHASES - 1);
            const int sl = sc_slab(ph);
            uint32_t v = vs[0];
#pragma unroll
            for (int u = 1; u < PHASES; ++u) v = ph == u ? vs[u] : v;
            const bool isa = SCR * sl < BM;
            u32x4 r = isa ? rsa : rsb;
            r.x = __builtin_amdgcn_readfirstlane(r.x);
            r.y = __builtin_amdgcn_readfirstlane(r.y);
            r.z = __builtin_amdgcn_readfirstlane(r.z);
            r.w = kRsrcWord3;
            lds_load16(r, v + (uint32_t)(SCB * q + 8 * k0), 0u, lds0 + (uint32_t)(SC_OFF + (q & 1) * SC_HALF + 1024 * sl));
        }
    };
    auto load_scales = [&](int kc) {
        if constexpr (!ALIGNED) {
            const int nb = k0 + kc + 1 < ksteps ? 8 : tail;
            const uint32_t m0 = nb >= 4 ? ~0u : (1u << (8 * nb)) - 1u;
            const uint32_t m1 = nb >= 8 ? ~0u : nb <= 4 ? 0u : (1u << (8 * (nb - 4))) - 1u;
#pragma unroll
            for (int u = 0; u < SC_PER_T; ++u) {
                // (rows of one wave are all activations or all weights)
                const u32x4 rr = __builtin_amdgcn_readfirstlane(tid + u * NT) < BM ? rsa : rsb;
                const uint32_t at = vs[u] + 8u * (uint32_t)(k0 + kc), sh = 8u * (at & 3u);
                const u32x4 d = __builtin_amdgcn_raw_buffer_load_b128(
                    __builtin_amdgcn_make_buffer_rsrc((void*)(((uint64_t)rr.y << 32) | rr.x), 0, (int)rr.z, (int)rr.w),
                    (int)(at & ~3u), 0, 0);
                sv[u].x = __builtin_amdgcn_alignbit(d.y, d.x, sh) & m0;
                sv[u].y = __builtin_amdgcn_alignbit(d.z, d.y, sh) & m1;
            }
        }
    };
    auto store_scales = [&](int kc) {
        if constexpr (!ALIGNED) {
#pragma unroll
            for (int u = 0; u < SC_PER_T; ++u) {
                const int r = tid + u * NT;
                if (r < BM + BN)
                    *reinterpret_cast<uint2*>(smem + SC_OFF + ((kc / RSTEP) & 1) * SC_HALF + SCB * r + 8 * (kc % RSTEP)) =
                        sv[u];
            }
        }
    };
    // Code load p (0 .. CODES - 1) of this wave for step kc, into the stage at
    // `at`.  In the last step the chunks past K are pushed out of range, and
    // steps past the last load nothing: a resource of no bytes, at offset zero
    // so that the range check holds whichever way it counts the offset.
    auto issue = [&](int p, int kc, uint32_t at) {
        const bool live = kc < nsteps, last = k0 + kc + 1 == ksteps;
        u32x4 r = p < CA ? ra : rb;
        r.z = __builtin_amdgcn_readfirstlane(live ? r.z : 0u);
        const uint32_t cut = last && chunk_of(slab(p)) >= tail ? kOob : 0u;
        lds_load16(r, vc[p] | cut, live ? (uint32_t)(k0 + kc) * 128u : 0u, lds0 + at + (uint32_t)(slab(p) * 1024));
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
    // registers.  The step's barrier stands before its last instructions: by
    // then every fragment of the step is in registers, so the stage is free,
    // and the next step has landed (only the loads of the steps after it may
    // be out); those last instructions cover the first reads of the next step
    // and the issue of the loads into the freed stage.  The scheduling
    // barriers keep that order, and the body must not branch: the matrix
    // instructions, which the compiler sees without side effects, otherwise
    // sink below the last branch and nothing overlaps (325 us against 239 us
    // at 4096 x 6144 x 16384, tiles of 256 x 256).
    uint32_t off_k[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) off_k[kk] = (uint32_t)(c32 * 128 + 16 * ((4 * hf + kk) ^ ((c32 >> 1) & 7)));
    const uint32_t a_off = (uint32_t)(wm * 32 * 128), b_off = (uint32_t)(wn * WTN * 128);
    const uint32_t sa_off = (uint32_t)(SC_OFF + SCB * (32 * wm + c32) + 4 * hf);
    const uint32_t sb_off = (uint32_t)(SC_OFF + SCB * (BM + wn * WTN + c32) + 4 * hf);
#pragma unroll
    for (int ph = 0; ph < PHASES; ++ph) issue_scales(ph, 0);
    load_scales(0);
    store_scales(0);
    load_scales(min(1, nsteps - 1));
    // In the order that the waits count on: a step's scales and activations
    // before its weights, and with NS = 3 the weights of a step further on.
#pragma unroll
    for (int p = CA; p < CODES; ++p) issue(p, 0, B_OFF);
    if constexpr (NS == 3)
#pragma unroll
        for (int p = CA; p < CODES; ++p) issue(p, 1, B_OFF + B_STAGE);
#pragma unroll
    for (int p = 0; p < CA; ++p) issue(p, 0, 0);
    issue_scales(0, 1);
#pragma unroll
    for (int p = 0; p < CODES; ++p)
        issue(p, p < CA ? 1 : NS - 1, p < CA ? (uint32_t)A_STAGE : (uint32_t)(B_OFF + (NS - 1) * B_STAGE));
    // (step 0: everything before that last set, whose activations are step 1's)
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(CODES + (ALIGNED ? 1 : 0)) & ~0xF00);
    __syncthreads();
    auto main_loop = [&](auto tmc) {
        constexpr int TA = decltype(tmc)::value;  // activation blocks in use
        u32x4 fa[2][TA], fb[2][TN];
        uint32_t sa[TA], sb[TN];
        // fragment q (TA activations, then TN weights) of the stages at sta, stb
        auto read_frag = [&](int q, uint32_t sta, uint32_t stb, int kk, int buf) {
            if (q < TA)
                fa[buf][q] = *reinterpret_cast<const u32x4*>(smem + (sta + off_k[kk] + a_off) + 4096 * WM * q);
            else
                fb[buf][q - TA] = *reinterpret_cast<const u32x4*>(smem + (stb + off_k[kk] + b_off) + 4096 * (q - TA));
        };
        auto read_scales = [&](int kc, uint32_t (&xa)[TA], uint32_t (&xb)[TN]) {
            const uint32_t at = (uint32_t)(((kc / RSTEP) & 1) * SC_HALF + 8 * (kc % RSTEP));
            // (blocks 4 .. 7 of a last step without them: zero, not the bytes
            // after the row)
            const uint32_t keep = k0 + kc + 1 == ksteps && 4 * hf >= tail ? 0u : ~0u;
#pragma unroll
            for (int i = 0; i < TA; ++i)
                xa[i] = *reinterpret_cast<const uint32_t*>(smem + (at + sa_off) + 32 * SCB * WM * i) & keep;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                xb[j] = *reinterpret_cast<const uint32_t*>(smem + (at + sb_off) + 32 * SCB * j) & keep;
        };
        read_scales(0, sa, sb);
#pragma unroll
        for (int q = 0; q < TA + TN; ++q) read_frag(q, 0, B_OFF, 0, 0);
        uint32_t ca = 0, cb = B_OFF;  // this step's stages
        for (int s = 0; s < nsteps; ++s) {
            const uint32_t xa = A_STAGE - ca, xb = cb + B_STAGE == SC_OFF ? B_OFF : cb + B_STAGE;  // the next one's
            uint32_t na[TA], nb[TN];
            auto group = [&](auto kkc) {
                constexpr int kk = decltype(kkc)::value, buf = kk & 1;
                if constexpr (kk == 3) {
                    // (NS = 3: the weights issued last, a step ahead, may be out)
                    __builtin_amdgcn_s_waitcnt(vmcnt_imm(NS == 3 ? CB : 0) & ~0xF00);
                    store_scales(s + 1);
                    __syncthreads();
                    read_scales(s + 1, na, nb);
                    load_scales(min(s + 2, nsteps - 1));
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    __builtin_amdgcn_sched_barrier(0);
                    constexpr int kR = (TA + TN + TN - 1) / TN;
#pragma unroll
                    for (int q = j * kR; q < (j + 1) * kR && q < TA + TN; ++q)
                        read_frag(q, kk < 3 ? ca : xa, kk < 3 ? cb : xb, (kk + 1) & 3, buf ^ 1);
#pragma unroll
                    for (int i = 0; i < TA; ++i) {
                        acc[j][i] = mfma_kk<kk>(fb[buf][j], fa[buf][i], acc[j][i], sb[j], sa[i]);
                        // (a matrix instruction takes 32 cycles of its unit,
                        // about what one load takes to issue)
                        if constexpr (kk == 3) {
                            constexpr int kM = TN * TA, kL = CODES + 1;
                            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                            for (int p = (j * TA + i) * kL / kM; p < (j * TA + i + 1) * kL / kM; ++p) {
                                if (p == 0) issue_scales((s + 1) % RSTEP, (s + 1) / RSTEP + 1);
                                else if (p <= CA) issue(p - 1, s + 2, ca);
                                else issue(p - 1, s + NS, cb);
                            }
                            __builtin_amdgcn_sched_barrier(0);
                        }
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
            ca = xa;
            cb = xb;
        }
    };
    // blocks of the fullest wave row
    const int used = (int)((row_end - row_beg + 32 * WM - 1) / (32 * WM));
    if (TM >= 2 && used == 1) main_loop(std::integral_constant<int, 1>{});
    else if (TM >= 3 && used == 2) main_loop(std::integral_constant<int, TM >= 3 ? 2 : TM>{});
    else if (TM >= 4 && used == 3) main_loop(std::integral_constant<int, TM >= 4 ? 3 : TM>{});
    else if (TM >= 5 && used == 4) main_loop(std::integral_constant<int, TM >= 5 ? 4 : TM>{});
    else if (TM >= 6 && used == 5) main_loop(std::integral_constant<int, TM >= 6 ? 5 : TM>{});
    else main_loop(std::integral_constant<int, TM>{});
    __builtin_amdgcn_s_waitcnt(kWaitAll);

    // (the slabs below reuse the stages, which other waves may still read)
    if constexpr (EP == MxEpi::kStoreBf16 || EP == MxEpi::kStoreF32) __syncthreads();

    // ---- epilogue: acc[j][i][r] is weight row 32 j + 8 (r / 4) + 4 hf + r % 4
    // of the wave, activation row 32 (i WM + wm) + c32.
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        if (i >= used) break;
        const int64_t row = row_beg + 32 * (i * WM + wm) + c32;
        if constexpr (kGateUp) {
            // (rows past the end take part in the exchange and store nothing)
#pragma unroll
            for (int j = 0; j < TN / 2; ++j) {
                const int64_t hc = n0 + wn * (WTN / 2) + 32 * j;
                uint32_t w[8], m = 0;
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                    w[p] = pack_bf16(silu_mul(acc[j][i][2 * p], acc[j + TN / 2][i][2 * p]),
                                     silu_mul(acc[j][i][2 * p + 1], acc[j + TN / 2][i][2 * p + 1]));
                    m = max_bf16x2(m, w[p]);
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
        } else if constexpr (kSplit) {
            if (row >= row_end) continue;
            float* const out = reinterpret_cast<float*>(g.out) + ((int64_t)kz * g.M + row) * g.ldo;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int64_t col = n0 + wn * WTN + 32 * j + 8 * p + 4 * hf;
                    if ((g.ldo & 3) == 0) {
                        if (col < nlim)
                            *reinterpret_cast<f32x4*>(out + col) = f32x4{acc[j][i][4 * p], acc[j][i][4 * p + 1],
                                                                         acc[j][i][4 * p + 2], acc[j][i][4 * p + 3]};
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (col + q < nlim) out[col + q] = acc[j][i][4 * p + q];
                    }
                }
        } else {
            // a 32-row slab of the wave's tile meets in LDS and leaves as
            // 16-byte pieces of rows (pitch: 16 rows' 8-byte writes fall on
            // different banks)
            constexpr bool kF32 = EP == MxEpi::kStoreF32;
            constexpr int kPitch = WTN * (kF32 ? 4 : 2) + 16;
            static_assert(NW * 32 * kPitch <= SC_OFF, "epilogue slabs");
            uint8_t* const slab = smem + wave * 32 * kPitch;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                    const int at = 32 * j + 8 * p + 4 * hf;
                    const float v0 = acc[j][i][4 * p], v1 = acc[j][i][4 * p + 1];
                    const float v2 = acc[j][i][4 * p + 2], v3 = acc[j][i][4 * p + 3];
                    if constexpr (kF32)
                        *reinterpret_cast<f32x4*>(slab + c32 * kPitch + 4 * at) = f32x4{v0, v1, v2, v3};
                    else
                        *reinterpret_cast<uint2*>(slab + c32 * kPitch + 2 * at) =
                            make_uint2(pack_bf16(v0, v1), pack_bf16(v2, v3));
                }
            __builtin_amdgcn_wave_barrier();
            const int64_t row0 = row_beg + 32 * (i * WM + wm);
            const bool vec = (g.ldo & 7) == 0;
            constexpr int kPieces = WTN * (kF32 ? 4 : 2) / 16;  // of a row
#pragma unroll
            for (int p = 0; p < kPieces / 2; ++p) {
                const int e = 64 * p + lane, rr = e / kPieces, ch = e % kPieces;
                const uint4 v = *reinterpret_cast<const uint4*>(slab + rr * kPitch + 16 * ch);
                const int64_t col = n0 + wn * WTN + (kF32 ? 4 : 8) * ch;
                if (row0 + rr >= row_end || col >= nlim) continue;
                if constexpr (kF32) {  // (ldo is a multiple of 32)
                    *reinterpret_cast<uint4*>(reinterpret_cast<float*>(g.out) + (row0 + rr) * g.ldo + col) = v;
                    continue;
                }
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

// ONLY_ALIGNED: built for K % 128 == 0 alone.
template <int TM, int TN, int WM, int WN, int NS, int RSTEP, MxEpi EP, bool ONLY_ALIGNED = false>
hipError_t launch_cfg(const MxGemmArgs& g0, int grid_m, hipStream_t stream) {
    constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN;
    MxGemmArgs g = g0;
    const int64_t ncols = EP == MxEpi::kGateUp ? g.N / 2 : g.N, bn = EP == MxEpi::kGateUp ? BN / 2 : BN;
    g.ntiles = (int32_t)((ncols + bn - 1) / bn);
    const int64_t mt = g.groups > 0 ? grid_m : (g.M + BM - 1) / BM;
    int64_t wgs = mt * g.ntiles * (EP == MxEpi::kPartialF32 ? g.ksplit : 1);
    if (g.groups > 0) wgs = (wgs + 7) / 8 * 8;  // a multiple of 8 for the XCD renumbering
    if (wgs < 1 || wgs >= ((int64_t)1 << 32) / (64 * WM * WN)) return hipErrorInvalidValue;
    if (ONLY_ALIGNED && g.K % 128 != 0) return hipErrorInvalidValue;
    if (ONLY_ALIGNED || g.K % 128 == 0)
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, NS, RSTEP, EP, true>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    else
        hipLaunchKernelGGL((k_mx_gemm<TM, TN, WM, WN, NS, RSTEP, EP, ONLY_ALIGNED>), dim3((unsigned)wgs), dim3(64 * WM * WN), 0, stream, g);
    return hipGetLastError();
}

// y[i] = bf16(sum over the K splits, in order); four elements a thread.
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int ksplit, int64_t n,
                                                 uint16_t* __restrict__ y) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    if ((n & 3) == 0) {
        f32x4 s = *reinterpret_cast<const f32x4*>(part + i);
        for (int k = 1; k < ksplit; ++k) s += *reinterpret_cast<const f32x4*>(part + k * n + i);
        *reinterpret_cast<uint2*>(y + i) = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
    } else {
        for (int64_t e = i; e < n && e < i + 4; ++e) {
            float s = part[e];
            for (int k = 1; k < ksplit; ++k) s += part[k * n + e];
            y[e] = (uint16_t)pack_bf16(s, 0.0f);
        }
    }
}

}  // namespace

// K splits of the 128 x 128 tiles: while the tiles leave CUs without one and
// every split keeps eight K steps (64 rows x 6144 x 16384 in 8 splits: 25 us;
// 256 rows x 16384 x 2048, 256 tiles of 8 steps, in two: 26 us against 14
// unsplit; weights from memory).
int mx_gemm_splits(int64_t M, int64_t N, int64_t K, int* steps) {
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128), ksteps = (K + 255) / 256;
    int64_t s = std::min<int64_t>({512 / std::max<int64_t>(tiles, 1), ksteps / 8, 16});
    if (s < 2 || tiles >= 256) return 1;
    const int64_t per = ((ksteps + s - 1) / s + 3) / 4 * 4;  // a multiple of the scale ring's four steps
    *steps = (int)per;
    return (int)((ksteps + per - 1) / per);
}

hipError_t launch_mx_gemm_split(const MxGemmArgs& g0, float* partial, hipStream_t stream) {
    MxGemmArgs g = g0;
    g.ksplit = mx_gemm_splits(g.M, g.N, g.K, &g.ksteps);
    g.out = partial;
    hipError_t e = launch_cfg<2, 2, 2, 2, 2, 4, MxEpi::kPartialF32>(g, 0, stream);
    if (e != hipSuccess) return e;
    const int64_t n = g.M * g.N;
    hipLaunchKernelGGL(k_mx_join, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, stream, partial, g.ksplit, n,
                       reinterpret_cast<uint16_t*>(g0.out));
    return hipGetLastError();
}

// Tiles, measured on MI355X with random codes (TFLOP/s; N x K 6144 x 16384 at
// M = 4096 and 1024, 16384 x 2048 at M = 4096):
//                      256 x 192   256 x 256   128 x 128 (two workgroups a CU)
//   4096 x 6144 x 16384     3836        3545        3547
//   1024 x 6144 x 16384     2276        2100        3066
//   4096 x 16384 x 2048     2172        3000        2668
// The large tiles need one workgroup per CU and few partly filled rounds; on
// short rows 256 x 192's odd tile count and longer tail lose.
// Grouped: 192 x 256, each wave all the rows and 64 weight rows, so that the
// main loop counts an expert's rows by 32.  Gate/up and down of 256 experts of
// 6144 x 2048, top 8 (us; 2 x 2 waves, which count them by 64, in brackets):
// 4096 tokens 831 and 486 (846, 486), 2560 738 and 415 (752, 426), 640 648 and
// 368 (659, 375), the down product with bf16 stores; fp32 ones make the 486 530.
hipError_t launch_mx_gemm(const MxGemmArgs& g, MxEpi epi, int grid_m, hipStream_t stream) {
    if (g.groups > 0)
        return epi == MxEpi::kGateUp ? launch_cfg<6, 2, 1, 4, 3, 2, MxEpi::kGateUp>(g, grid_m, stream)
                                     : launch_cfg<6, 2, 1, 4, 3, 2, MxEpi::kStoreF32>(g, grid_m, stream);
    // share of the CUs' time that a tile's rounds fill
    auto fill = [&](int64_t bm, int64_t bn, int64_t slots) {
        const int64_t t = ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn);
        return (double)t / (double)((t + slots - 1) / slots * slots) * (double)(g.M * g.N) /
               (double)(t * bm * bn);
    };
    // (256 x 256 leaves no registers for the scales of an unaligned K)
    const double f192 = fill(256, 192, 256) * (g.K >= 8192 ? 1.05 : 0.8), f256 = g.K % 128 ? 0.0 : fill(256, 256, 256);
    const double f128 = fill(128, 128, 512) * 0.9;
    if (f192 > f256 && f192 > f128) return launch_cfg<4, 3, 2, 2, 3, 2, MxEpi::kStoreBf16>(g, grid_m, stream);
    if (f256 > f128) return launch_cfg<2, 4, 4, 2, 2, 4, MxEpi::kStoreBf16, true>(g, grid_m, stream);
    return launch_cfg<2, 2, 2, 2, 2, 4, MxEpi::kStoreBf16>(g, grid_m, stream);
}

}  // namespace nvfp4
