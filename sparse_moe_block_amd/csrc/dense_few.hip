// The forward products for few rows (single tokens, decode batches): bound by
// the weights' bytes, each of which is read once per 16 NQ rows of its expert.
//
// A workgroup takes 16 weight rows of one expert (gated: 8 gate rows and the 8
// up rows of the same features) and all of the reduction, an eighth of it per
// wavefront.  The weights are the MFMA's first operand, loaded straight from
// memory in its layout (lane l: row l % 16, steps 8 (l / 16) .. + 7, 16 bytes),
// four loads in flight per wavefront; NQ groups of 16 rows of x are the second.
// The eight partial tiles meet in LDS and are summed in order.
//
// Measured (graph replays): 128 rows over 128 experts, 2048 -> 2 x 768, 511 MB of
// weights: 81.5 us (6.3 TB/s); 102 us as 64-row tiles through LDS, 120 us with
// eight loads in flight (half the workgroups a CU).  One row, 7168 -> 2 x 2048, 59
// MB: 11.2 us (5.2 TB/s); 13.7 us with four wavefronts of eight loads, 33 us as
// 64-row tiles.
#include "dense_core.h"

namespace fw {
namespace {

constexpr int kFewWaves = 8;

template <bool GLU, int NQ>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(RowsArgs a,
                                                             const int32_t *__restrict__ offsets) {
    constexpr int U = 4;   // steps in flight
    __shared__ f4 part[kFewWaves][NQ][64];
    const int e = blockIdx.y, lane = threadIdx.x % kWave, wave = wave_id();
    int b = 0, n = a.R;
    if (offsets) {
        const int rb = ld_const(offsets + e), rn = ld_const(offsets + e + 1);
        if (blockIdx.x == 0 && threadIdx.x == 0 &&
            ((e == 0 && rb != 0) || rb < 0 || rb > a.R || rn < rb || rn > a.R))
            atomicOr(&a.hdr->status, FW_STATUS_BAD_OFFSETS);
        b = min(max(rb, 0), a.R);
        n = min(max(rn, b), a.R);
    }
    if (b == n) return;
    const int K = a.Kd, p = lane & 15, k8 = 8 * (lane >> 4);
    // the lane's weight row (linear: past the last one, the last)
    const int f0 = blockIdx.x * (GLU ? 8 : 16);
    const uint16_t *w = GLU ? (p < 8 ? a.w0 : a.w1) : a.w0;
    const int wrow = GLU ? f0 + (p & 7) : min(f0 + p, a.Np - 1);
    w += (size_t)e * a.w_stride + (size_t)wrow * K + k8;
    // whole 32-step slices, an eighth per wavefront; the rest with the last
    const int slices = K / 32, per = (slices + kFewWaves - 1) / kFewWaves;
    const int s0 = min(wave * per, slices), s1 = min(s0 + per, slices);
    const bool rest = wave == kFewWaves - 1 && K % 32 != 0;
    for (int rb = b; rb < n; rb += 16 * NQ) {
        const uint16_t *x[NQ];
        f4 acc[NQ];
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
            x[q] = a.q + (size_t)min(rb + 16 * q + p, n - 1) * K + k8;
            acc[q] = f4{0.f, 0.f, 0.f, 0.f};
        }
        // what the thread's outputs need besides the sums, on its way meanwhile.
        // Lane l of group q: row rb + 16 q + l % 16, weight rows 4 (l / 16) .. + 3;
        // gated: lanes below 32 hold the gate rows, those above the up rows
        constexpr int T = GLU ? 32 : 64;
        const int oq = threadIdx.x / T, ol = threadIdx.x % T;
        const int row = rb + 16 * oq + (ol & 15), col = f0 + 4 * (ol >> 4);
        const bool mine = (int)threadIdx.x < T * NQ && row < n && col < a.Np;
        const size_t at = (size_t)row * a.Np + col;
        float4 bias{0.f, 0.f, 0.f, 0.f};
        uint4 res{0, 0, 0, 0};
        if constexpr (!GLU) {
            if (mine && a.bias) bias = *(const float4 *)(a.bias + (size_t)e * a.Np + col);
            if (mine && a.residual) {
                if (a.out_f32) {
                    res = *(const uint4 *)((const float *)a.residual + at);
                } else {
                    const uint2 r = *(const uint2 *)((const uint16_t *)a.residual + at);
                    res = uint4{r.x << 16, r.x & 0xFFFF0000u, r.y << 16, r.y & 0xFFFF0000u};
                }
            }
        }
        for (int s = s0; s < s1; s += U) {
            uint4 wv[U], xv[U][NQ];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < s1) {
                    wv[u] = *(const uint4 *)(w + 32 * (s + u));
#pragma unroll
                    for (int q = 0; q < NQ; ++q) xv[u][q] = *(const uint4 *)(x[q] + 32 * (s + u));
                }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (s + u < s1) {
#pragma unroll
                    for (int q = 0; q < NQ; ++q)
                        acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf8, wv[u]), __builtin_bit_cast(bf8, xv[u][q]),
                            acc[q], 0, 0, 0);
                }
        }
        if (rest) {
            const bool in = 32 * slices + k8 < K;   // K is a multiple of 8
            const uint4 zero = {0, 0, 0, 0};
            const uint4 wv = in ? *(const uint4 *)(w + 32 * slices) : zero;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                const uint4 xv = in ? *(const uint4 *)(x[q] + 32 * slices) : zero;
                acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf8, wv), __builtin_bit_cast(bf8, xv), acc[q], 0, 0, 0);
            }
        }
#pragma unroll
        for (int q = 0; q < NQ; ++q) part[wave][q][lane] = acc[q];
        __syncthreads();
        if (mine) {
            f4 z = part[0][oq][ol], u{};
#pragma unroll
            for (int i = 1; i < kFewWaves; ++i) z += part[i][oq][ol];
            if constexpr (GLU) {
                u = part[0][oq][ol + 32];
#pragma unroll
                for (int i = 1; i < kFewWaves; ++i) u += part[i][oq][ol + 32];
            }
            const float b4[4] = {bias.x, bias.y, bias.z, bias.w};
            const uint32_t r4[4] = {res.x, res.y, res.z, res.w};
            float v[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if constexpr (GLU) {
                    v[t] = act_value(a.fn, z[t]) * u[t];
                } else {
                    v[t] = act_value(a.fn, z[t] + b4[t]);
                    if (a.residual) v[t] += __uint_as_float(r4[t]);
                }
            }
            if (a.out_f32)
                *(float4 *)((float *)a.out + at) = float4{v[0], v[1], v[2], v[3]};
            else
                *(uint2 *)((uint16_t *)a.out + at) =
                    uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        }
        __syncthreads();
    }
}

}  // namespace

hipError_t launch_few(bool glu, const RowsArgs &a, const int32_t *offsets, hipStream_t s) {
    const dim3 grid(glu ? a.Np / 8 : (a.Np + 15) / 16, a.E);
    auto go = [&](auto k) { k<<<grid, 64 * kFewWaves, 0, s>>>(a, offsets); };
    if (a.E == 1 && a.R > 16)
        glu ? go(few_kernel<true, 2>) : go(few_kernel<false, 2>);
    else
        glu ? go(few_kernel<true, 1>) : go(few_kernel<false, 1>);
    return hipGetLastError();
}

}  // namespace fw
