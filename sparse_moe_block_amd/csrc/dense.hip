// The bf16 training products: the gated feed-forward products and the linear
// product with their epilogues, their input gradients and their weight and
// bias gradients, for one matrix or one per expert (rows grouped by
// expert_offsets).  Every product runs on v_mfma_f32_32x32x16_bf16 with fp32
// accumulators (dense_core.h).
//
// Backward.  g, u (and z) are formed again from x instead of being kept: their
// product's epilogue turns the accumulators and the arriving gradient straight
// into dg, du (dz), so neither g nor u ever reaches memory.  dg, du and dz are
// rounded to bf16 there (half a step, at most 2^-8 relative), the only way into the
// bf16 products that follow; the bias gradient is summed before that rounding.
#include <math.h>

#include "dense_core.h"
#include "stages.h"

namespace fw {
namespace {

// Four consecutive output values at p (bf16 or fp32).
__device__ __forceinline__ void store4(void *out, int f32, size_t at, const float *v) {
    if (f32)
        *(float4 *)((float *)out + at) = float4{v[0], v[1], v[2], v[3]};
    else
        *(uint2 *)((uint16_t *)out + at) = uint2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ __forceinline__ void load4(const void *in, int f32, size_t at, float *v) {
    if (f32) {
        const float4 f = *(const float4 *)((const float *)in + at);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
        const uint2 u = *(const uint2 *)((const uint16_t *)in + at);
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x); v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
    }
}

__global__ __launch_bounds__(kPrepThreads) void dense_schedule_kernel(
    const int32_t *__restrict__ offsets, int E, int R, int tile_rows, int max_tiles,
    int4 *__restrict__ active, int4 *__restrict__ tiles, int *__restrict__ split_cnt,
    WsHeader *__restrict__ hdr) {
    build_schedule(offsets, E, R, tile_rows, max_tiles, active, tiles, split_cnt, hdr);
}

// The tile of a workgroup of one dense product: XCD b % 8 takes an eighth of
// the tile list, which walks blocks of kBlockRows row tiles column by column,
// so that an XCD's workgroups in flight share few weight and few row panels in
// its L2.  -1: none.
constexpr int kBlockRows = 8;
__device__ __forceinline__ int dense_tile(int row_tiles, int col_tiles, int &ct) {
    const int total = row_tiles * col_tiles, per = (total + 7) / 8;
    const int idx = blockIdx.x / 8, id = (blockIdx.x % 8) * per + idx;
    ct = 0;
    if (idx >= per || id >= total) return -1;
    const int block = id / (kBlockRows * col_tiles), in = id % (kBlockRows * col_tiles);
    const int r0 = block * kBlockRows, n = min(kBlockRows, row_tiles - r0);
    ct = in / n;
    return r0 + in % n;
}

template <DenseOp OP> struct RowShape {
    using T = Shape<128, 128, 2, 2, OP == kInput, false, OP == kGlu || OP == kGluGrad>;
};

// One (row tile, column tile).
template <DenseOp OP>
__global__ __launch_bounds__(256, 2) void rows_kernel(RowsArgs a, int col_tiles, int row_tiles) {
    using S = typename RowShape<OP>::T;
    __shared__ uint4 P0[S::PChunks];
    __shared__ uint4 P1[S::PChunks];
    __shared__ uint4 Q0[S::QChunks];
    __shared__ uint4 Q1[S::QChunks];
    constexpr int BC = S::DUAL ? S::BP / 2 : S::BP;   // output columns of a tile
    int ct, rt;
    if (a.tiles)
        rt = xcd_row_tile(a.hdr, col_tiles, row_tiles, 0, 0, ct);
    else
        rt = dense_tile(row_tiles, col_tiles, ct);
    if (rt < 0) return;
    int expert = 0, rb = rt * S::BQ, rows = min(S::BQ, a.R - rb);
    if (a.tiles) {
        const int4 tl = ld_const(a.tiles + rt);
        expert = tl.x;
        rb = tl.y;
        rows = tl.z;
    }
    const int lane = threadIdx.x % kWave, wave = wave_id();
    const int c0 = ct * BC, cols = min(BC, a.Np - c0);
    const size_t we = (size_t)expert * a.w_stride;
    const uint32_t qpitch = 2u * (uint32_t)a.Kd;
    auto q = [&](int seg) {
        return Operand{(const char *)(a.q + seg * a.q_seg + (size_t)rb * a.Kd), rows, qpitch, 0};
    };
    auto p = [&](int seg) {
        const uint16_t *w = seg ? a.w1 : a.w0;
        if (OP == kInput)   // w [Kd][Np], read across
            return Operand{(const char *)(w + we + c0), 0, 2u * (uint32_t)a.Np, 2u * (uint32_t)c0};
        return Operand{(const char *)(w + we + (size_t)c0 * a.Kd), cols, qpitch, 0};
    };
    auto pb = [&](int) {
        return Operand{(const char *)(a.w1 + we + (size_t)c0 * a.Kd), cols, qpitch, 0};
    };
    f16v acc[S::PI][S::QJ];
    tile_product<S>(acc, P0, P1, Q0, Q1, wave, lane, a.Kd, a.nseg, p, pb, q);

    // acc[i][j][4 m + t]: row qrow(wq, j) + lane % 32, column prow(wp, i) +
    // 8 m + 4 (lane / 32) + t
    const int wp = wave % S::WP, wq = wave / S::WP, g4 = 4 * (lane >> 5);
    const size_t dzu = (size_t)a.R * a.Np;   // du behind dg
    if constexpr (OP == kLinGrad) {
        // per-column sums over the tile's rows, through LDS
        __syncthreads();
    }
    float colsum[S::PI][16];
    if constexpr (OP == kLinGrad) {
#pragma unroll
        for (int i = 0; i < S::PI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) colsum[i][v] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < S::QJ; ++j) {
        const int row = S::qrow(wq, j) + (lane & 31);
        const size_t at0 = (size_t)(rb + row) * a.Np;
#pragma unroll
        for (int i = 0; i < (S::DUAL ? 1 : S::PI); ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int col = c0 + S::prow(wp, i) + 8 * m + g4;
                if (row >= rows || col >= a.Np || col >= c0 + cols) continue;
                const size_t at = at0 + col;
                float v[4];
                if constexpr (OP == kGlu) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        v[t] = act_value(a.fn, acc[0][j][4 * m + t]) * acc[1][j][4 * m + t];
                    store4(a.out, a.out_f32, at, v);
                } else if constexpr (OP == kGluGrad) {
                    float dh[4], dg[4], du[4];
                    load4(a.dy, 0, at, dh);
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        float f, df;
                        const float u = acc[1][j][4 * m + t];
                        act_both(a.fn, acc[0][j][4 * m + t], f, df);
                        v[t] = f * u;
                        dg[t] = dh[t] * u * df;
                        du[t] = dh[t] * f;
                    }
                    store4(a.dz, 0, at, dg);
                    store4(a.dz, 0, dzu + at, du);
                    if (a.out) store4(a.out, 0, at, v);
                } else if constexpr (OP == kLinear || OP == kLinGrad) {
                    float b[4] = {0.f, 0.f, 0.f, 0.f};
                    if (a.bias) load4(a.bias, 1, (size_t)expert * a.Np + col, b);
                    if constexpr (OP == kLinear) {
                        float r[4] = {0.f, 0.f, 0.f, 0.f};
                        if (a.residual) load4(a.residual, a.out_f32, at, r);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            v[t] = act_value(a.fn, acc[i][j][4 * m + t] + b[t]);
                            if (a.residual) v[t] += r[t];
                        }
                        store4(a.out, a.out_f32, at, v);
                    } else {
                        float dy[4];
                        load4(a.dy, 0, at, dy);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            float f, df;
                            act_both(a.fn, acc[i][j][4 * m + t] + b[t], f, df);
                            v[t] = dy[t] * df;
                            colsum[i][4 * m + t] += v[t];
                        }
                        store4(a.dz, 0, at, v);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t) v[t] = acc[i][j][4 * m + t];
                    store4(a.out, a.out_f32, at, v);
                }
            }
    }
    if constexpr (OP == kLinGrad) {
        if (!a.bpart) return;
        // over the 32 rows a lane group holds, then over the wavefronts of the
        // column, in a fixed order
        float *part = (float *)P0;   // [WQ][BP]
#pragma unroll
        for (int i = 0; i < S::PI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                float s = colsum[i][v];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor(s, o);
                if ((lane & 31) == 0)
                    part[wq * S::BP + S::prow(wp, i) + 8 * (v >> 2) + g4 + (v & 3)] = s;
            }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += S::Threads) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < S::WQ; ++w) s += part[w * S::BP + c];
            a.bpart[(size_t)rt * a.Np + c0 + c] = s;
        }
    }
}

// dw tiles: Q = output features (rows of dw), P = input features.
using GradShape = Shape<128, 128, 2, 2, true, true, false>;

__global__ __launch_bounds__(256, 2) void grad_kernel(GradArgs a, int nt, int kt, int tiles) {
    using S = GradShape;
    __shared__ uint4 P0[S::PChunks];
    __shared__ uint4 P1[S::PChunks];
    __shared__ uint4 Q0[S::QChunks];
    __shared__ uint4 Q1[S::QChunks];
    // XCD x takes an eighth of the tile list (k tiles fastest)
    const int per = (tiles + 7) / 8;
    const int id = (blockIdx.x % 8) * per + blockIdx.x / 8;
    if (id >= tiles || (int)(blockIdx.x / 8) >= per) return;
    const int k0 = id % kt * S::BP, n_all = id / kt;
    const int n0 = n_all % nt * S::BQ, em = n_all / nt;
    const int mat = em % a.mats, expert = em / a.mats;
    int b = 0, e = a.R;
    if (a.offsets) {
        b = min(max(ld_const(a.offsets + expert), 0), a.R);
        e = min(max(ld_const(a.offsets + expert + 1), b), a.R);
    }
    const int lane = threadIdx.x % kWave, wave = wave_id();
    const uint16_t *dz = a.dz + (size_t)mat * a.R * a.N + (size_t)b * a.N + n0;
    const uint16_t *x = a.x + (size_t)b * a.K + k0;
    auto q = [&](int) {
        return Operand{(const char *)dz, 0, 2u * (uint32_t)a.N, 2u * (uint32_t)n0};
    };
    auto p = [&](int) {
        return Operand{(const char *)x, 0, 2u * (uint32_t)a.K, 2u * (uint32_t)k0};
    };
    f16v acc[S::PI][S::QJ];
    tile_product<S>(acc, P0, P1, Q0, Q1, wave, lane, e - b, 1, p, p, q);

    const int wp = wave % S::WP, wq = wave / S::WP, g4 = 4 * (lane >> 5);
    void *dw = mat ? a.dw1 : a.dw0;
#pragma unroll
    for (int j = 0; j < S::QJ; ++j) {
        const int n = n0 + S::qrow(wq, j) + (lane & 31);
        const size_t at0 = ((size_t)expert * a.N + n) * a.K;
#pragma unroll
        for (int i = 0; i < S::PI; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const int k = k0 + S::prow(wp, i) + 8 * m + g4;
                if (n >= a.N || k >= a.K) continue;
                float v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) v[t] = acc[i][j][4 * m + t];
                if (a.accumulate) {
                    float o[4];
                    load4(dw, a.out_f32, at0 + k, o);
#pragma unroll
                    for (int t = 0; t < 4; ++t) v[t] += o[t];
                }
                store4(dw, a.out_f32, at0 + k, v);
            }
    }
}

// Column sums of one row tile of bf16 rows.
__global__ __launch_bounds__(256) void colsum_kernel(const uint16_t *__restrict__ dy, int R,
                                                     int N, const int4 *__restrict__ tiles,
                                                     const WsHeader *__restrict__ hdr,
                                                     int max_tiles, float *__restrict__ bpart) {
    const int rt = blockIdx.y, c = 2 * (blockIdx.x * 256 + threadIdx.x);
    int rb = rt * kDenseMinTileRows, rows = min(kDenseMinTileRows, R - rb);
    if (tiles) {
        if (rt >= min(ld_const(&hdr->n_tiles), max_tiles)) return;
        const int4 tl = ld_const(tiles + rt);
        rb = tl.y;
        rows = tl.z;
    }
    if (c >= N) return;
    float s0 = 0.f, s1 = 0.f;
    const uint16_t *p = dy + (size_t)rb * N + c;
    for (int r = 0; r < rows; ++r, p += N) {
        const uint32_t v = *(const uint32_t *)p;
        s0 += bf16_lo(v);
        s1 += bf16_hi(v);
    }
    *(float2 *)(bpart + (size_t)rt * N + c) = float2{s0, s1};
}

// db[e] = the sum of e's row tiles' partials, in tile order (the schedule
// lists each expert's tiles in row order, experts ascending).
__global__ __launch_bounds__(256) void bias_grad_kernel(const float *__restrict__ bpart,
                                                        const int32_t *__restrict__ offsets,
                                                        int R, int N, int max_tiles,
                                                        float *__restrict__ db, int accumulate) {
    const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    int first = 0, n = (R + kDenseMinTileRows - 1) / kDenseMinTileRows;
    if (offsets) {
        for (int i = 0; i <= e; ++i) {
            first += i ? n : 0;
            const int b = min(max(ld_const(offsets + i), 0), R);
            const int t = min(max(ld_const(offsets + i + 1), b), R);
            n = (t - b + kDenseMinTileRows - 1) / kDenseMinTileRows;
        }
        first = min(first, max_tiles);
        n = min(n, max_tiles - first);
    }
    if (c >= N) return;
    float s = accumulate ? db[(size_t)e * N + c] : 0.f;
    float sum = 0.f;
    for (int i = 0; i < n; ++i) sum += bpart[(size_t)(first + i) * N + c];
    db[(size_t)e * N + c] = s + sum;
}

template <DenseOp OP> hipError_t run_rows(const RowsArgs &a, hipStream_t s) {
    using S = typename RowShape<OP>::T;
    constexpr int BC = S::DUAL ? S::BP / 2 : S::BP;
    const int ct = (a.Np + BC - 1) / BC;
    const int rt = a.tiles ? a.max_tiles : (a.R + S::BQ - 1) / S::BQ;
    const int per = a.tiles ? xcd_tile_cap(a.R, a.E, S::BQ, a.max_tiles) * ct : (rt * ct + 7) / 8;
    rows_kernel<OP><<<8 * per, S::Threads, 0, s>>>(a, ct, rt);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rows(DenseOp op, const RowsArgs &a, hipStream_t s) {
    switch (op) {
        case kGlu: return run_rows<kGlu>(a, s);
        case kGluGrad: return run_rows<kGluGrad>(a, s);
        case kLinear: return run_rows<kLinear>(a, s);
        case kLinGrad: return run_rows<kLinGrad>(a, s);
        default: return run_rows<kInput>(a, s);
    }
}

int64_t rows_tiles(int R, int E, int Np) {
    return (int64_t)((R + 127) / 128 + E + 8) * ((Np + 63) / 64);
}

int64_t grad_tiles(int E, int N, int K, int mats) {
    return (int64_t)E * mats * ((N + GradShape::BQ - 1) / GradShape::BQ) *
           ((K + GradShape::BP - 1) / GradShape::BP);
}

hipError_t launch_grad(const GradArgs &a, hipStream_t s) {
    const int nt = (a.N + GradShape::BQ - 1) / GradShape::BQ;
    const int kt = (a.K + GradShape::BP - 1) / GradShape::BP;
    const int tiles = a.E * a.mats * nt * kt;
    grad_kernel<<<(tiles + 7) / 8 * 8, GradShape::Threads, 0, s>>>(a, nt, kt, tiles);
    return hipGetLastError();
}

hipError_t launch_colsum(const uint16_t *dy, int R, int N, const int4 *tiles, WsHeader *hdr,
                         int max_tiles, float *bpart, hipStream_t s) {
    const int rt = tiles ? max_tiles : (R + kDenseMinTileRows - 1) / kDenseMinTileRows;
    colsum_kernel<<<dim3((N / 2 + 255) / 256, rt), 256, 0, s>>>(dy, R, N, tiles, hdr, max_tiles,
                                                                bpart);
    return hipGetLastError();
}

hipError_t launch_bias_grad(const float *bpart, const int32_t *offsets, int R, int E, int N,
                            float *db, int accumulate, hipStream_t s) {
    const int max_tiles = (R + kDenseMinTileRows - 1) / kDenseMinTileRows + E;
    bias_grad_kernel<<<dim3((N + 255) / 256, E), 256, 0, s>>>(bpart, offsets, R, N, max_tiles, db,
                                                              accumulate);
    return hipGetLastError();
}

hipError_t launch_dense_schedule(const int32_t *offsets, int E, int R, const DenseWs &L, char *ws,
                                 hipStream_t s) {
    dense_schedule_kernel<<<1, kPrepThreads, 0, s>>>(
        offsets, E, R, kDenseMinTileRows, L.max_tiles, (int4 *)(ws + L.active),
        (int4 *)(ws + L.tiles), (int *)(ws + L.split_cnt), (WsHeader *)ws);
    return hipGetLastError();
}

}  // namespace fw
