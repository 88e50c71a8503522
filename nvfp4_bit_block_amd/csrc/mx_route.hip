// mx_route.hip -- what surrounds the products of the sorted routed layer: the
// slots sorted by expert and the tokens quantized, in one launch, and the
// weighted sum over a token's slots.
//
// Sum: out[t] = bf16(sum_j w[t, j] * Y[row of slot j]), fp32, slots in order.
// Y is fp32, so that the output's own rounding is the only one, as in the slot
// form (bf16 rows, 1389 against 1488 us for the layer at 4096 tokens, take the
// output's error from 0.0017 to 0.0023 relative).  Bound by that read: 4096 x 8
// slots of 6144, 805 MB, take 139 to 153 us on MI355X, up to 6.1 TB/s.
#include "mx_device.hpp"
#include "mx_internal.hpp"

namespace nvfp4 {

namespace {

constexpr int kPrepThreads = 1024;
constexpr int kMaxExperts = 4096;
constexpr int kBatch = 8;
constexpr int kPieces = 2;  // 16-byte pieces of x per thread

// Workgroup 0 sorts the slots, the others quantize the tokens meanwhile.
// Sorting: slots counted per expert in LDS, a scan over the experts for the
// first row and first row tile of each, then every slot takes the next row of
// its expert.  Which of an expert's rows a slot gets depends on the order of
// the LDS atomics; every row is computed on its own, so the layer's output
// does not.  (366 slots of 61 tokens: 4.5 us against 12 for three launches of
// the sort and one for the tokens.)
__global__ __launch_bounds__(kPrepThreads) void k_mx_prepare(MxPrepareArgs a) {
    if (blockIdx.x > 0) {
        const int64_t base = (int64_t)(blockIdx.x - 1) * (kPrepThreads * kPieces) + threadIdx.x;
        uint4 v[kPieces];
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int64_t i = base + u * kPrepThreads;
            v[u] = make_uint4(0, 0, 0, 0);
            if (i < a.n8) v[u] = load_nt16(a.x + 8 * i);
        }
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            const int64_t i = base + u * kPrepThreads;
            uint32_t code, s;
            mx_encode_quad(v[u], code, s);
            if (i < a.n8) {
                reinterpret_cast<uint32_t*>(a.codes)[i] = code;
                if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = (uint8_t)s;
            }
        }
        return;
    }
    __shared__ int32_t cnt[kMaxExperts];
    __shared__ int32_t part[2][kPrepThreads / kWave];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < a.E; e += kPrepThreads) cnt[e] = 0;
    __syncthreads();
    // kBatch slots of a thread at a time, so that their loads (and below
    // their LDS atomics) are in flight together; -1 past the end
    auto batch = [&](int p0, int32_t (&e)[kBatch]) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int p = p0 + u * kPrepThreads + tid;
            e[u] = p < a.slots ? a.ids[p] : -1;
            if (e[u] >= a.E) e[u] = -1;
        }
    };
    for (int p0 = 0; p0 < a.slots; p0 += kBatch * kPrepThreads) {
        int32_t e[kBatch];
        batch(p0, e);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (e[u] >= 0) atomicAdd(&cnt[e[u]], 1);
    }
    __syncthreads();
    // thread i scans experts [4 i, 4 i + 4)
    int32_t rows[4], tiles[4], sr = 0, st = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int e = 4 * tid + q;
        rows[q] = e < a.E ? cnt[e] : 0;
        tiles[q] = (rows[q] + a.bm - 1) / a.bm;
        sr += rows[q];
        st += tiles[q];
    }
    int32_t ir = sr, it = st;  // inclusive over the wave, then over the waves
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int32_t r = __shfl_up(ir, off, kWave), t = __shfl_up(it, off, kWave);
        if (lane >= off) {
            ir += r;
            it += t;
        }
    }
    if (lane == kWave - 1) {
        part[0][wave] = ir;
        part[1][wave] = it;
    }
    __syncthreads();
    int32_t r = ir - sr, t = it - st;
    for (int w = 0; w < wave; ++w) {
        r += part[0][w];
        t += part[1][w];
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int e = 4 * tid + q;
        if (e < a.E) {
            cnt[e] = r;  // the expert's next row
            a.row_off[e] = r;
            a.tile_off[e] = t;
        }
        r += rows[q];
        t += tiles[q];
    }
    if (tid == kPrepThreads - 1) {
        a.row_off[a.E] = r;
        a.tile_off[a.E] = t;
    }
    __syncthreads();
    for (int p0 = 0; p0 < a.slots; p0 += kBatch * kPrepThreads) {
        int32_t e[kBatch], pos[kBatch];
        batch(p0, e);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) pos[u] = e[u] >= 0 ? atomicAdd(&cnt[e[u]], 1) : -1;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int p = p0 + u * kPrepThreads + tid;
            if (p >= a.slots) continue;
            a.inv[p] = pos[u];
            if (pos[u] >= 0) a.perm[pos[u]] = p;
        }
    }
}

// A thread sums 4 columns of one token; the rows of 8 slots are in flight
// together (a skipped slot reads row 0 and is not added).  The NVFP4 layer's
// sum rounds finite values only; this one keeps a NaN of any pattern.
__global__ __launch_bounds__(256) void k_mx_combine(const float* __restrict__ Y, const int32_t* __restrict__ inv,
                                                    const float* __restrict__ w, int64_t total, int32_t top_k,
                                                    int32_t h4, uint16_t* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t t = i / h4, c = (i - t * h4) * 4, H = (int64_t)h4 * 4;
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < top_k; j0 += 8) {
        int32_t pos[8];
        float wj[8];
        f32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const bool in = j0 + u < top_k;
            pos[u] = in ? inv[t * top_k + j0 + u] : -1;
            wj[u] = in ? w[t * top_k + j0 + u] : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(Y + (int64_t)max(pos[u], 0) * H + c));
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (pos[u] < 0) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) s[q] = __builtin_fmaf(wj[u], v[u][q], s[q]);
        }
    }
    *reinterpret_cast<uint2*>(out + t * H + c) = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
}

}  // namespace

hipError_t launch_mx_prepare(const MxPrepareArgs& a, hipStream_t stream) {
    const int64_t wgs = 1 + (a.n8 + kPrepThreads * kPieces - 1) / (kPrepThreads * kPieces);
    if (a.E < 1 || a.E > kMaxExperts || a.slots < 1 || wgs >= ((int64_t)1 << 32) / kPrepThreads)
        return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_mx_prepare, dim3((unsigned)wgs), dim3(kPrepThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_mx_combine(const float* Y, const int32_t* inv, const float* w, int64_t T, int32_t top_k, int64_t H,
                             uint16_t* out, hipStream_t stream) {
    const int64_t total = T * (H / 4);
    if (total >= (int64_t)1 << 32) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_mx_combine, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream, Y, inv, w, total,
                       top_k, (int32_t)(H / 4), out);
    return hipGetLastError();
}

}  // namespace nvfp4
