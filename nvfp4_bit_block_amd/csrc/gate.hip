// gate.hip -- the expert gate (scores, groups, top-k, weights) and the
// gradient of its weights.
//
// LPT lanes share one token, each holding NPL of its E logits in registers: 16
// lanes, four tokens a wave, for many tokens of up to 256 experts and top_k
// 16, the whole wave otherwise.  Few tokens are bound by the chain of
// dependent steps, which a whole wave shortens (one token of 256 experts,
// sigmoid, bias and groups: 14.3 -> 6.1 us); many by their instructions, of
// which a quarter wave needs half as many per token.  Lane q of the token has
// experts 4 LPT (i / 4) + 4 q + i % 4, i < NPL, so that four neighbours load
// as one piece.  top_k rounds of "largest key, lowest expert among equals"
// pick the experts; every lane of the token sees each winner, and lane j
// keeps slot j's.
//
// Measured on MI355X: 4096 x 256 fp32, top 8, 6.8 us (a launch takes about 2):
// each of the rounds scans a lane's keys twice and reduces twice, one after the
// other.  65536 tokens 34 us, 2.1 TB/s; 4096 x 1024 12.7 us.  The dense gradient
// of 65536 x 256 bf16, 71 MB read and written, 17.8 us, 4.0 TB/s, bound by its
// exponentials and the passes through LDS.
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace nvfp4 {

namespace {

constexpr float kNegInf = -__builtin_inff();
constexpr float kF32Max = 3.402823466e38f;
// Threads of a workgroup: 16 tokens, or one token of more than 256 experts
// (whose keys may take 64 KB of LDS).
constexpr int gate_threads(int lpt) { return lpt == 16 ? 256 : 64; }

struct GateArgs {
    const void* logits;
    const float* bias;
    const int32_t* ids_in;
    const float* dw;
    int32_t* ids;
    float* weights;
    void* dlogits;
    int64_t T;
    int32_t E, top_k, n_group, topk_group, members, group_top;
    float scale;
};

// Reductions over the LPT lanes of a token, the result in all of them: DPP
// steps within rows of 16 lanes, then the four rows' values through scalars.
struct OpMax {
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct OpAdd {
    template <typename T>
    __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct OpMin {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return min(a, b); }
};
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) { return dpp_u32<CTRL>(v); }
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return dpp_f32<CTRL>(v); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)dpp_u32<CTRL>((uint32_t)b) |
                                          ((uint64_t)dpp_u32<CTRL>((uint32_t)(b >> 32)) << 32));
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ float lane_value(float v, int l) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)lane_value((uint32_t)b, l) |
                                          ((uint64_t)lane_value((uint32_t)(b >> 32), l) << 32));
}
template <int LPT, typename T, typename Op>
__device__ __forceinline__ T tok_reduce(T v, Op op) {
    v = op(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
    v = op(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
    v = op(v, dpp<0x141>(v));  // row_half_mirror
    v = op(v, dpp<0x140>(v));  // row_mirror
    if constexpr (LPT == 64)
        v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
    return v;
}
template <int LPT, typename T>
__device__ __forceinline__ T tok_max(T v) { return tok_reduce<LPT>(v, OpMax()); }
template <int LPT, typename T>
__device__ __forceinline__ T tok_sum(T v) { return tok_reduce<LPT>(v, OpAdd()); }
template <int LPT>
__device__ __forceinline__ uint32_t tok_min(uint32_t v) { return tok_reduce<LPT>(v, OpMin()); }

template <int LPT>
__device__ __forceinline__ int expert_of(int q, int i) {
    return (i >> 2) * (4 * LPT) + 4 * q + (i & 3);
}

// Logit as a candidate's fp32 value: NaN -> -inf, +inf -> the largest finite.
__device__ __forceinline__ float clean(float l) { return l > kNegInf ? fminf(l, kF32Max) : kNegInf; }

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* logits, int64_t i) {
    if constexpr (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(logits)[i]);
    else return reinterpret_cast<const float*>(logits)[i];
}

// This lane's NPL logits of token t (-inf past E).
template <int LPT, int NPL, bool BF16>
__device__ __forceinline__ void load_row(const void* logits, int64_t t, int E, int q, float (&l)[NPL]) {
    const int64_t row = t * E;
    if ((E & 3) == 0) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4) {
            const int e = expert_of<LPT>(q, i);
#pragma unroll
            for (int c = 0; c < 4; ++c) l[i + c] = kNegInf;
            if (e < E) {
                if constexpr (BF16) {
                    const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(logits) + row + e);
                    l[i] = clean(__uint_as_float(w.x << 16));
                    l[i + 1] = clean(__uint_as_float(w.x & 0xFFFF0000u));
                    l[i + 2] = clean(__uint_as_float(w.y << 16));
                    l[i + 3] = clean(__uint_as_float(w.y & 0xFFFF0000u));
                } else {
                    const float4 w = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(logits) + row + e);
                    l[i] = clean(w.x);
                    l[i + 1] = clean(w.y);
                    l[i + 2] = clean(w.z);
                    l[i + 3] = clean(w.w);
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = expert_of<LPT>(q, i);
            l[i] = e < E ? clean(load_logit<BF16>(logits, row + e)) : kNegInf;
        }
    }
}

// Slot weights of a token: lane j < top_k holds slot j, `take` if it has an
// expert, l its logit; m and z the row's softmax statistics (softmax without
// renormalisation only).  Renormalised weights are a softmax over the slots:
// of the logits, or of the logarithm of the sigmoid, so that no sum vanishes
// whatever the logits.
template <int LPT, bool SIGMOID, bool RENORM>
__device__ __forceinline__ float slot_weight(bool take, float l, float m, float z, float scale) {
    if constexpr (!RENORM) {
        float w;
        if constexpr (SIGMOID) {
            const float e = expf(-fabsf(l));
            w = (l >= 0.0f ? 1.0f : e) / (1.0f + e);
        } else {
            w = expf(l - m) / z;
        }
        return take ? scale * w : 0.0f;
    } else {
        const float u = SIGMOID ? fminf(l, 0.0f) - log1pf(expf(-fabsf(l))) : l;
        const float um = tok_max<LPT>(take ? u : kNegInf);
        const float e = take ? expf(u - um) : 0.0f;
        const float s = tok_sum<LPT>(e);
        return take ? scale * e / s : 0.0f;
    }
}

// Key: float orders by the logit; double by the 64-bit choice value (a bias,
// or a rank of two values; near-equal scores then order as the definition
// says).  Dead experts hold -inf, and -0 is made +0 so that it ties with it.
template <int LPT, int NPL, bool BF16, bool SIGMOID, bool RENORM, typename Key>
__global__ __launch_bounds__(gate_threads(LPT)) void k_gate(GateArgs a) {
    constexpr int kTok = gate_threads(LPT) / LPT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int q = threadIdx.x % LPT, tl = threadIdx.x / LPT;
    const int64_t t_ = (int64_t)blockIdx.x * kTok + tl;
    const bool live_row = t_ < a.T;
    const int64_t t = live_row ? t_ : a.T - 1;  // surplus tokens repeat the last one and store nothing
    float l[NPL];
    load_row<LPT, NPL, BF16>(a.logits, t, a.E, q, l);

    float m = 0.0f, z = 1.0f;
    if constexpr (!SIGMOID && (!RENORM || sizeof(Key) == 8)) {
        float mm = l[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) mm = fmaxf(mm, l[i]);
        m = fmaxf(tok_max<LPT>(mm), -kF32Max);
        if constexpr (!RENORM) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NPL; ++i) s += expf(l[i] - m);
            z = fmaxf(tok_sum<LPT>(s), 1e-30f);
        }
    }

    Key key[NPL];
    if constexpr (sizeof(Key) == 4) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = l[i] + 0.0f;
    } else {
        double zd = 1.0;
        if constexpr (!SIGMOID) {
            double s = 0.0;
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                key[i] = exp((double)l[i] - (double)m);
                s += key[i];
            }
            zd = fmax(tok_sum<LPT>(s), 1e-300);
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = expert_of<LPT>(q, i);
            const double b = a.bias != nullptr && e < a.E ? (double)a.bias[e] : 0.0;
            const double s = SIGMOID ? 1.0 / (1.0 + exp(-(double)l[i])) : key[i] / zd;
            const double c = s + b;
            key[i] = l[i] > kNegInf && c > -__builtin_inf() ? c + 0.0 : -__builtin_inf();
        }
    }

    if (a.n_group > a.topk_group) {
        // ranks of the groups, from the keys in LDS: P lanes per group (a power
        // of two, as many as the groups leave), lane p takes members p, p + P, ..
        Key* const ks = reinterpret_cast<Key*>(smem) + (size_t)tl * (a.E + a.n_group);
        Key* const rank = ks + a.E;
        const Key none = -(Key)__builtin_inf();
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = expert_of<LPT>(q, i);
            if (e < a.E) ks[e] = key[i];
        }
        __syncthreads();
        int P = LPT;
        while (P > 1 && P * a.n_group > LPT) P >>= 1;
        const int gq = q / P, p = q & (P - 1);
        for (int g0 = 0; g0 < a.n_group; g0 += LPT / P) {
            const int g = g0 + gq;
            Key b1 = none, b2 = none;
            if (g < a.n_group)
                for (int i = p; i < a.members; i += P) {
                    const Key v = ks[g * a.members + i];
                    b2 = v > b1 ? b1 : (v > b2 ? v : b2);
                    b1 = v > b1 ? v : b1;
                }
            for (int off = 1; off < P; off <<= 1) {
                const Key o1 = __shfl_xor(b1, off, kWave), o2 = __shfl_xor(b2, off, kWave);
                b2 = o1 > b1 ? (b1 > o2 ? b1 : o2) : (o1 > b2 ? o1 : b2);
                b1 = o1 > b1 ? o1 : b1;
            }
            if (a.group_top == 2 && b2 > none) b1 += b2;
            if (p == 0 && g < a.n_group) rank[g] = b1;
        }
        __syncthreads();
        // a group stays if fewer than topk_group groups come before it
        for (int g = q; g < a.n_group; g += LPT) {
            const Key r = rank[g];
            int before = 0;
            for (int h = 0; h < a.n_group; ++h) {
                const Key o = rank[h];
                before += o > r || (o == r && h < g);
            }
            ks[g] = (Key)(before < a.topk_group ? 1 : 0);  // (the keys are in registers)
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = expert_of<LPT>(q, i);
            if (e < a.E && ks[(uint32_t)e / (uint32_t)a.members] == (Key)0) key[i] = none;
        }
    }

    int32_t mine = -1;
    for (int j = 0; j < a.top_k; ++j) {
        Key best = key[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) best = key[i] > best ? key[i] : best;
        best = tok_max<LPT>(best);
        if (!(best > -(Key)__builtin_inf())) {
            // (all lanes of the token agree; other tokens of the wave go on)
            continue;
        }
        int at = NPL;
#pragma unroll
        for (int i = NPL - 1; i >= 0; --i) at = key[i] == best ? i : at;
        const uint32_t e = at < NPL ? (uint32_t)expert_of<LPT>(q, at) : 0xFFFFFFFFu;
        const uint32_t win = tok_min<LPT>(e);
        const int drop = e == win ? at : NPL;
#pragma unroll
        for (int i = 0; i < NPL; ++i) key[i] = i == drop ? -(Key)__builtin_inf() : key[i];
        if (q == j) mine = (int32_t)win;
    }
    const bool take = mine >= 0;
    float ls = 0.0f;
    if (take) ls = clean(load_logit<BF16>(a.logits, t * a.E + mine));
    const float w = slot_weight<LPT, SIGMOID, RENORM>(take, ls, m, z, a.scale);
    if (live_row && q < a.top_k) {
        a.ids[t * a.top_k + q] = mine;
        a.weights[t * a.top_k + q] = w;
    }
}

// The gradient: the selected experts' values meet the row in LDS (E floats a
// token), which leaves as whole pieces; only the softmax without
// renormalisation reads the row itself.
template <int LPT, int NPL, bool BF16, bool SIGMOID, bool RENORM>
__global__ __launch_bounds__(gate_threads(LPT)) void k_gate_backward(GateArgs a) {
    constexpr int kTok = gate_threads(LPT) / LPT;
    extern __shared__ __align__(16) uint8_t smem[];
    const int q = threadIdx.x % LPT, tl = threadIdx.x / LPT;
    const int64_t t_ = (int64_t)blockIdx.x * kTok + tl;
    const bool live_row = t_ < a.T;
    const int64_t t = live_row ? t_ : a.T - 1;
    float* const row = reinterpret_cast<float*>(smem) + (size_t)tl * ((a.E + 3) / 4 * 4);

    int32_t id = -1;
    float dw = 0.0f, ls = kNegInf;
    if (q < a.top_k) {
        id = a.ids_in[t * a.top_k + q];
        dw = a.dw[t * a.top_k + q];
        if (id >= 0 && id < a.E) ls = clean(load_logit<BF16>(a.logits, t * a.E + id));
    }
    const bool take = ls > kNegInf;
    if (!take) id = -1;
    ls = take ? ls : 0.0f;

    constexpr bool kDense = !SIGMOID && !RENORM;
    float l[NPL], m = 0.0f, z = 1.0f;
    if constexpr (kDense) {
        load_row<LPT, NPL, BF16>(a.logits, t, a.E, q, l);
        float mm = l[0];
#pragma unroll
        for (int i = 1; i < NPL; ++i) mm = fmaxf(mm, l[i]);
        m = fmaxf(tok_max<LPT>(mm), -kF32Max);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            // (a bf16 gradient keeps 8 bits: the hardware's exponential, a few
            // parts in 2^22 at the arguments that matter, is exact enough)
            l[i] = BF16 ? __builtin_amdgcn_exp2f(1.44269504f * (l[i] - m)) : expf(l[i] - m);
            s += l[i];
        }
        z = fmaxf(tok_sum<LPT>(s), 1e-30f);
    }
    const float w = slot_weight<LPT, SIGMOID, RENORM>(take, ls, m, z, a.scale);
    const float dot = tok_sum<LPT>(take ? w * dw : 0.0f);
    float g = take ? w * (RENORM ? dw - dot / a.scale : dw) : 0.0f;
    if constexpr (SIGMOID) g *= 1.0f / (1.0f + expf(ls));  // 1 - sigmoid(l)

    // an expert that several slots name gets their sum, from each of them
    float gs = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
        const int src = (threadIdx.x & (kWave - 1) & ~(LPT - 1)) + j;
        const int32_t oid = __shfl(id, src, kWave);
        const float og = __shfl(g, src, kWave);
        gs += oid == id ? og : 0.0f;
    }
    const float share = kDense ? -dot / z : 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
        const int e = expert_of<LPT>(q, i);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (kDense) v = make_float4(share * l[i], share * l[i + 1], share * l[i + 2], share * l[i + 3]);
        if (e < a.E) *reinterpret_cast<float4*>(row + e) = v;  // (rows are padded to fours)
    }
    __syncthreads();
    if (id >= 0) row[id] += gs;  // equal ids store equal sums
    __syncthreads();
    if (!live_row) return;
    const int64_t base = t * a.E;
    if ((a.E & 3) == 0) {
        for (int e = 4 * q; e < a.E; e += 4 * LPT) {
            const float4 v = *reinterpret_cast<const float4*>(row + e);
            if constexpr (BF16)
                *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.dlogits) + base + e) =
                    make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.dlogits) + base + e) = v;
        }
    } else {
        for (int e = q; e < a.E; e += LPT) {
            if constexpr (BF16)
                reinterpret_cast<uint16_t*>(a.dlogits)[base + e] = (uint16_t)pack_bf16(row[e], 0.0f);
            else
                reinterpret_cast<float*>(a.dlogits)[base + e] = row[e];
        }
    }
}

template <int LPT, int NPL, bool BF16, bool SIGMOID, bool RENORM>
hipError_t gate_launch(const GateArgs& a, bool wide_key, bool backward, hipStream_t s) {
    constexpr int kTok = gate_threads(LPT) / LPT;
    const unsigned grid = (unsigned)((a.T + kTok - 1) / kTok);
    if (backward) {
        const size_t lds = (size_t)kTok * ((a.E + 3) / 4 * 4) * 4;
        hipLaunchKernelGGL((k_gate_backward<LPT, NPL, BF16, SIGMOID, RENORM>), dim3(grid), dim3(gate_threads(LPT)), lds, s, a);
    } else {
        const bool grouped = a.n_group > a.topk_group;
        const size_t lds = grouped ? (size_t)kTok * (a.E + a.n_group) * (wide_key ? 8 : 4) : 0;
        if (wide_key)
            hipLaunchKernelGGL((k_gate<LPT, NPL, BF16, SIGMOID, RENORM, double>), dim3(grid), dim3(gate_threads(LPT)), lds, s, a);
        else
            hipLaunchKernelGGL((k_gate<LPT, NPL, BF16, SIGMOID, RENORM, float>), dim3(grid), dim3(gate_threads(LPT)), lds, s, a);
    }
    return hipGetLastError();
}

template <int LPT, int NPL>
hipError_t gate_types(const nvfp4_gate_config& c, const GateArgs& a, bool backward, hipStream_t s) {
    // (group_top = 2 orders by the score even where every group is kept: scores
    // that are equal in 64 bits go by index, whatever their logits)
    const bool wide = a.bias != nullptr || c.group_top == 2;
    const int which = (c.logits_dtype == NVFP4_GATE_BF16 ? 4 : 0) + (c.score == NVFP4_GATE_SIGMOID ? 2 : 0) +
                      (c.renormalize ? 1 : 0);
    switch (which) {
        case 0: return gate_launch<LPT, NPL, false, false, false>(a, wide, backward, s);
        case 1: return gate_launch<LPT, NPL, false, false, true>(a, wide, backward, s);
        case 2: return gate_launch<LPT, NPL, false, true, false>(a, wide, backward, s);
        case 3: return gate_launch<LPT, NPL, false, true, true>(a, wide, backward, s);
        case 4: return gate_launch<LPT, NPL, true, false, false>(a, wide, backward, s);
        case 5: return gate_launch<LPT, NPL, true, false, true>(a, wide, backward, s);
        case 6: return gate_launch<LPT, NPL, true, true, false>(a, wide, backward, s);
        default: return gate_launch<LPT, NPL, true, true, true>(a, wide, backward, s);
    }
}

hipError_t gate_dispatch(const nvfp4_gate_config& c, GateArgs a, bool backward, hipStream_t s) {
    a.T = c.T;
    a.E = (int32_t)c.E;
    a.top_k = (int32_t)c.top_k;
    a.scale = c.scale;
    // A whole wave per token / four tokens a wave, us on MI355X, fp32, top_k 8,
    // softmax and (in brackets) sigmoid with a bias and 8 groups:
    //   E = 64   1024 tokens 4.1 / 3.7 (7.0 / 6.7), 2048 4.8 / 3.7 (8.1 / 6.7),
    //     16384 17.3 / 5.9 (34.0 / 11.1)
    //   128      1024 4.1 / 4.4 (6.9 / 9.1), 2048 4.7 / 4.5 (8.2 / 9.1), 4096 6.7
    //     / 5.1 (11.9 / 9.9), 16384 17.3 / 7.7 (34.3 / 17.1)
    //   256      2048 5.0 / 6.8 (8.8 / 15.4), 4096 6.8 / 6.9 (12.3 / 15.5), 16384
    //     18.1 / 12.1 (36.0 / 29.6)
    // One border between them, where 128 experts cross; 256 would cross at 4096
    // (8192 and more with groups).  The gradient's row passes want whole waves of
    // tokens at any T.
    if (c.E <= 256 && c.top_k <= 16 && (backward || c.T > 2048)) {
        if (c.E <= 64) return gate_types<16, 4>(c, a, backward, s);
        if (c.E <= 128) return gate_types<16, 8>(c, a, backward, s);
        return gate_types<16, 16>(c, a, backward, s);
    }
    if (c.E <= 256) return gate_types<64, 4>(c, a, backward, s);
    if (c.E <= 512) return gate_types<64, 8>(c, a, backward, s);
    if (c.E <= 1024) return gate_types<64, 16>(c, a, backward, s);
    return gate_types<64, 64>(c, a, backward, s);
}

}  // namespace

hipError_t launch_gate(const nvfp4_gate_config& c, const void* logits, const float* bias, int32_t* ids,
                       float* weights, hipStream_t stream) {
    GateArgs a = {};
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.n_group = (int32_t)c.n_group;
    a.topk_group = (int32_t)c.topk_group;
    a.members = (int32_t)(c.E / c.n_group);
    a.group_top = c.group_top;
    return gate_dispatch(c, a, false, stream);
}

hipError_t launch_gate_backward(const nvfp4_gate_config& c, const void* logits, const int32_t* ids,
                                const float* dweights, void* dlogits, hipStream_t stream) {
    GateArgs a = {};
    a.logits = logits;
    a.ids_in = ids;
    a.dw = dweights;
    a.dlogits = dlogits;
    a.n_group = a.topk_group = 1;
    return gate_dispatch(c, a, true, stream);
}

}  // namespace nvfp4
