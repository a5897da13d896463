// Activation checkpoints in 8 bits: the layer's own 8-bit activation blocks
// (32 values along a row; MXFP8 or int8), written to caller-owned memory and
// read back as bf16 or fp32.
//
// Four lanes hold one block, eight consecutive values each, so that a
// wavefront's loads and stores are contiguous (16 bytes of bf16 source and 8
// bytes of codes per lane); the block maximum is two quad permutations.  Bound
// by memory: 2 (bf16) or 4 (fp32) + 1 + 1/32 or 1/8 bytes a value.
//
// A block that holds a NaN or an infinity is written as a NaN block (scale
// byte 255, or d = NaN, codes 0) and sets FW_STATUS_RANGE: gradients formed
// from it are NaN, as from the values themselves, rather than quietly wrong.
#include "dense.h"
#include "stages.h"

namespace fw {
namespace {

constexpr int kCkptThreads = 256;

// E8M0 exponent of a block of largest magnitude amax > 0 (finite):
// floor(log2 amax) - 8 in -127 .. 127; the E4M3 element is v 2^-e, clamped to
// 448 (the conversion returns NaN above 464), nearest-even.
__device__ __forceinline__ int block_exp(float amax) {
    return min(max(__builtin_amdgcn_frexp_expf(amax) - 1 - 8, -127), 127);
}
__device__ __forceinline__ float e4m3_in(float v, int e) {
    return fminf(fmaxf(__builtin_amdgcn_ldexpf(v, -e), -448.0f), 448.0f);
}
// round(v / d), halves away from zero, the division correctly rounded.
__device__ __forceinline__ uint32_t int8_code(float v, float d) {
    return (uint32_t)(int)fminf(fmaxf(roundf(v / d), -127.0f), 127.0f) & 0xFFu;
}

template <int FMT, bool BF16>
__global__ __launch_bounds__(kCkptThreads) void pack_kernel(const void *__restrict__ src,
                                                            int64_t blocks,
                                                            uint2 *__restrict__ codes,
                                                            void *__restrict__ scales,
                                                            WsHeader *__restrict__ hdr) {
    const int64_t i = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x, b = i >> 2;
    if (b >= blocks) return;   // the four lanes of a block leave together
    float v[8];
    if constexpr (BF16) {
        const uint4 r = ((const uint4 *)src)[i];
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = bf16_lo(w[q]);
            v[2 * q + 1] = bf16_hi(w[q]);
        }
    } else {
        const float4 lo = ((const float4 *)src)[2 * i], hi = ((const float4 *)src)[2 * i + 1];
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    }
    // |v| as fp32 bits orders like |v| (NaN above +inf)
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, __float_as_uint(v[q]) & 0x7FFFFFFFu);
    m = max(m, dpp<0xB1>(m));   // quad_perm [1,0,3,2]
    m = max(m, dpp<0x4E>(m));   // quad_perm [2,3,0,1]
    const bool bad = m >= 0x7F800000u, zero = m == 0;
    const float amax = __uint_as_float(m);
    uint32_t o[2] = {0u, 0u};
    if constexpr (FMT == FW_ACT_MXFP8) {
        const int e = zero || bad ? -127 : block_exp(amax);
        if (!bad) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                int w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_in(v[4 * q], e),
                                                        e4m3_in(v[4 * q + 1], e), 0, false);
                w = __builtin_amdgcn_cvt_pk_fp8_f32(e4m3_in(v[4 * q + 2], e),
                                                    e4m3_in(v[4 * q + 3], e), w, true);
                o[q] = (uint32_t)w;
            }
        }
        if ((i & 3) == 0) ((uint8_t *)scales)[b] = (uint8_t)(bad ? 255 : zero ? 0 : e + 127);
    } else {
        const float d = amax / 127.0f;
        if (!bad && d != 0.0f) {
#pragma unroll
            for (int q = 0; q < 8; ++q) o[q / 4] |= int8_code(v[q], d) << (8 * (q % 4));
        }
        if ((i & 3) == 0) ((float *)scales)[b] = bad ? __builtin_nanf("") : d;
    }
    codes[i] = uint2{o[0], o[1]};
    if (bad && (i & 3) == 0) atomicOr(&hdr->status, FW_STATUS_RANGE);
}

template <int FMT, bool BF16>
__global__ __launch_bounds__(kCkptThreads) void unpack_kernel(const uint2 *__restrict__ codes,
                                                              const void *__restrict__ scales,
                                                              int64_t blocks,
                                                              void *__restrict__ dst) {
    const int64_t i = (int64_t)blockIdx.x * kCkptThreads + threadIdx.x, b = i >> 2;
    if (b >= blocks) return;
    const uint2 c = codes[i];
    const uint32_t w[2] = {c.x, c.y};
    float v[8];
    if constexpr (FMT == FW_ACT_MXFP8) {
        const int sb = ((const uint8_t *)scales)[b];
        const float nan = __builtin_nanf("");
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], false);
            const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[q], true);
            const float f[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
            for (int t = 0; t < 4; ++t)
                v[4 * q + t] = sb == 255 ? nan : __builtin_amdgcn_ldexpf(f[t], sb - 127);
        }
    } else {
        const float d = ((const float *)scales)[b];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = (float)(int8_t)((w[q / 4] >> (8 * (q % 4))) & 0xFFu) * d;
    }
    // the checkpoint's values are bf16 (MXFP8: exactly); fp32 outputs hold the same
    const uint4 r = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7])};
    if constexpr (BF16) {
        ((uint4 *)dst)[i] = r;
    } else {
        ((float4 *)dst)[2 * i] = float4{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
        ((float4 *)dst)[2 * i + 1] = float4{bf16_lo(r.z), bf16_hi(r.z), bf16_lo(r.w), bf16_hi(r.w)};
    }
}

}  // namespace

hipError_t launch_ckpt_pack(int format, int64_t blocks, const void *src, int src_bf16,
                            void *codes, void *scales, WsHeader *hdr, hipStream_t s) {
    const unsigned grid = (unsigned)((4 * blocks + kCkptThreads - 1) / kCkptThreads);
    auto go = [&](auto k) { k<<<grid, kCkptThreads, 0, s>>>(src, blocks, (uint2 *)codes, scales, hdr); };
    if (format == FW_ACT_MXFP8)
        src_bf16 ? go(pack_kernel<FW_ACT_MXFP8, true>) : go(pack_kernel<FW_ACT_MXFP8, false>);
    else
        src_bf16 ? go(pack_kernel<FW_ACT_INT8, true>) : go(pack_kernel<FW_ACT_INT8, false>);
    return hipGetLastError();
}

hipError_t launch_ckpt_unpack(int format, int64_t blocks, const void *codes, const void *scales,
                              void *dst, int dst_bf16, hipStream_t s) {
    const unsigned grid = (unsigned)((4 * blocks + kCkptThreads - 1) / kCkptThreads);
    auto go = [&](auto k) {
        k<<<grid, kCkptThreads, 0, s>>>((const uint2 *)codes, scales, blocks, dst);
    };
    if (format == FW_ACT_MXFP8)
        dst_bf16 ? go(unpack_kernel<FW_ACT_MXFP8, true>) : go(unpack_kernel<FW_ACT_MXFP8, false>);
    else
        dst_bf16 ? go(unpack_kernel<FW_ACT_INT8, true>) : go(unpack_kernel<FW_ACT_INT8, false>);
    return hipGetLastError();
}

}  // namespace fw
