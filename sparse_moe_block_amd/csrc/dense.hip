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

#include <type_traits>

#include "dense_core.h"
#include "stages.h"

namespace fw {
namespace {

// Eight consecutive values in memory, bf16 or fp32.
struct Eight {
    uint4 r[2];   // bf16: r[0]
};
__device__ __forceinline__ void load8(Eight &e, const void *in, int f32, size_t at) {
    if (f32) {
        const uint4 *p = (const uint4 *)((const float *)in + at);
        e.r[0] = p[0];
        e.r[1] = p[1];
    } else {
        e.r[0] = *(const uint4 *)((const uint16_t *)in + at);
    }
}
__device__ __forceinline__ void values8(const Eight &e, int f32, float *v) {
    const uint32_t w[8] = {e.r[0].x, e.r[0].y, e.r[0].z, e.r[0].w,
                           e.r[1].x, e.r[1].y, e.r[1].z, e.r[1].w};
#pragma unroll
    for (int t = 0; t < 8; ++t)
        v[t] = f32 ? __uint_as_float(w[t]) : (t & 1) ? bf16_hi(w[t / 2]) : bf16_lo(w[t / 2]);
}
__device__ __forceinline__ void store8(void *out, int f32, size_t at, const float *v) {
    if (f32) {
        float4 *p = (float4 *)((float *)out + at);
        p[0] = float4{v[0], v[1], v[2], v[3]};
        p[1] = float4{v[4], v[5], v[6], v[7]};
    } else {
        *(uint4 *)((uint16_t *)out + at) = uint4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                 pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
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
__device__ __forceinline__ int dense_block(int row_tiles, int col_tiles, int &ct) {
    const int total = row_tiles * col_tiles, per = (total + 7) / 8;
    const int idx = blockIdx.x / 8, id = (blockIdx.x % 8) * per + idx;
    ct = 0;
    if (idx >= per || id >= total) return -1;
    const int block = id / (kBlockRows * col_tiles), in = id % (kBlockRows * col_tiles);
    const int r0 = block * kBlockRows, n = min(kBlockRows, row_tiles - r0);
    ct = in / n;
    return r0 + in % n;
}

// Tile shapes.
//  kTile256   256 x 256, eight wavefronts of 64 x 128 outputs, two stages, one
//             workgroup a CU: the fewest bytes from L2 and LDS an output
//  kTile128   128 x 128, four wavefronts of 64 x 64, two stages, two workgroups
//             a CU
//  kTile128D  128 x 128, eight wavefronts of 32 x 64, four stages, one workgroup
//             a CU: for products whose tiles do not fill the CUs twice
//  kTile64    64 x 64, four wavefronts of 32 x 32, four stages, two workgroups a
//             CU: for products of few tiles
template <DenseTile TILE, bool PX, bool QX, bool DUAL>
using TileShape = std::conditional_t<
    TILE == kTile256, Shape<256, 256, 4, 2, 2, PX, QX, DUAL>,
    std::conditional_t<TILE == kTile128, Shape<128, 128, 2, 2, 2, PX, QX, DUAL>,
                       std::conditional_t<TILE == kTile128D, Shape<128, 128, 4, 2, 4, PX, QX, DUAL>,
                                          Shape<64, 64, 2, 2, 4, PX, QX, DUAL>>>>;
template <DenseOp OP, DenseTile TILE>
using RowShape = TileShape<TILE, OP == kInput, false, OP == kGlu || OP == kGluGrad>;
template <DenseTile TILE>
constexpr int kThreads = TILE == kTile256 || TILE == kTile128D ? 512 : 256;
template <DenseTile TILE> constexpr int kBlocksPerCu = kThreads<TILE> == 512 ? 1 : 2;

// One (row tile, column tile).
template <DenseOp OP, DenseTile TILE>
__global__ __launch_bounds__(kThreads<TILE>, kBlocksPerCu<TILE>) void rows_kernel(
    RowsArgs a, int col_tiles, int row_tiles) {
    using S = RowShape<OP, TILE>;
    FW_RING(S, ring);
    constexpr int BC = S::DUAL ? S::BP / 2 : S::BP;   // output columns of a tile
    int ct, rt;
    if (a.tiles)
        rt = xcd_row_tile(a.hdr, col_tiles, row_tiles, 0, 0, ct);
    else
        rt = dense_block(row_tiles, col_tiles, ct);
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
    f4 acc[S::PI][S::QJ];
    tile_product<S>(acc, ring, wave, lane, a.Kd, a.nseg, p, pb, q);

    const size_t dzu = (size_t)a.R * a.Np;   // du behind dg
    float bias[8], colsum[8];
    {
        // the columns a lane is handed are the same for every row
        const int col = c0 + wave % S::WP * kOutCols<S> + lane % (kOutCols<S> / 8) * 8;
        Eight e{};
        if ((OP == kLinear || OP == kLinGrad) && a.bias && col < c0 + cols)
            load8(e, a.bias, 1, (size_t)expert * a.Np + col);
        values8(e, 1, bias);
#pragma unroll
        for (int t = 0; t < 8; ++t) colsum[t] = 0.f;
    }
    auto inside = [&](int row, int col) { return row < rows && col < cols; };
    auto place = [&](int row, int col) { return (size_t)(rb + row) * a.Np + c0 + col; };
    auto fetch = [&](int row, int col) {
        Eight e{};
        if constexpr (OP == kGluGrad || OP == kLinGrad) {
            if (inside(row, col)) load8(e, a.dy, 0, place(row, col));
        } else if constexpr (OP == kLinear) {
            if (a.residual && inside(row, col)) load8(e, a.residual, a.out_f32, place(row, col));
        }
        return e;
    };
    hand_out<S>(acc, ring.p[0], wave, lane, fetch,
                [&](int row, int col, float *v, const float *u, const Eight &e) {
        if (!inside(row, col)) return;
        const size_t at = place(row, col);
        if constexpr (OP == kGlu) {
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] = act_value(a.fn, v[t]) * u[t];
            store8(a.out, a.out_f32, at, v);
        } else if constexpr (OP == kGluGrad) {
            float dh[8], dg[8], du[8];
            values8(e, 0, dh);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                float f, df;
                act_both(a.fn, v[t], f, df);
                v[t] = f * u[t];
                dg[t] = dh[t] * u[t] * df;
                du[t] = dh[t] * f;
            }
            store8(a.dz, 0, at, dg);
            store8(a.dz, 0, dzu + at, du);
            if (a.out) store8(a.out, 0, at, v);
        } else if constexpr (OP == kLinear) {
            float r[8];
            values8(e, a.out_f32, r);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                v[t] = act_value(a.fn, v[t] + bias[t]);
                if (a.residual) v[t] += r[t];
            }
            store8(a.out, a.out_f32, at, v);
        } else if constexpr (OP == kLinGrad) {
            float dy[8];
            values8(e, 0, dy);
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                float f, df;
                act_both(a.fn, v[t] + bias[t], f, df);
                v[t] = dy[t] * df;
                colsum[t] += v[t];
            }
            store8(a.dz, 0, at, v);
        } else {
            store8(a.out, a.out_f32, at, v);
        }
    });
    if constexpr (OP == kLinGrad) {
        if (!a.bpart) return;
        // over the lanes that hold the same columns, then over the wavefronts
        // of the column, in a fixed order
        constexpr int CW = kOutCols<S>, LR = CW / 8;
        const int wp = wave % S::WP, wq = wave / S::WP;
        float *part = (float *)ring.q[0];   // [WQ][BP]
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            float s = colsum[t];
#pragma unroll
            for (int o = 32; o >= LR; o >>= 1) s += __shfl_xor(s, o);
            if (lane < LR) part[wq * S::BP + wp * CW + 8 * lane + t] = s;
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
template <DenseTile TILE>
__global__ __launch_bounds__(kThreads<TILE>, kBlocksPerCu<TILE>) void grad_kernel(
    GradArgs a, int nt, int kt, int tiles) {
    using S = TileShape<TILE, true, true, false>;
    FW_RING(S, ring);
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
    f4 acc[S::PI][S::QJ];
    tile_product<S>(acc, ring, wave, lane, e - b, 1, p, p, q);

    void *dw = mat ? a.dw1 : a.dw0;
    auto inside = [&](int n, int k) { return n0 + n < a.N && k0 + k < a.K; };
    auto place = [&](int n, int k) { return ((size_t)expert * a.N + n0 + n) * a.K + k0 + k; };
    auto fetch = [&](int n, int k) {
        Eight e{};
        if (a.accumulate && inside(n, k)) load8(e, dw, a.out_f32, place(n, k));
        return e;
    };
    hand_out<S>(acc, ring.p[0], wave, lane, fetch,
                [&](int n, int k, float *v, const float *, const Eight &e) {
        if (!inside(n, k)) return;
        if (a.accumulate) {
            float o[8];
            values8(e, a.out_f32, o);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[t] += o[t];
        }
        store8(dw, a.out_f32, place(n, k), v);
    });
}

// Column sums of one row tile of bf16 rows: a workgroup takes 64 columns,
// eight lanes (16 bytes each) a row and 32 rows at a time, so that the rows'
// loads are in flight together; the 32 partial sums meet in LDS, in order.
__global__ __launch_bounds__(256) void colsum_kernel(const uint16_t *__restrict__ dy, int R,
                                                     int N, const int4 *__restrict__ tiles,
                                                     const WsHeader *__restrict__ hdr,
                                                     int max_tiles, int tile_rows,
                                                     float *__restrict__ bpart) {
    __shared__ float part[32][64];
    const int rt = blockIdx.y, c0 = blockIdx.x * 64;
    int rb = rt * tile_rows, rows = min(tile_rows, R - rb);
    if (tiles) {
        if (rt >= min(ld_const(&hdr->n_tiles), max_tiles)) return;
        const int4 tl = ld_const(tiles + rt);
        rb = tl.y;
        rows = tl.z;
    }
    const int c = 8 * (threadIdx.x % 8), r0 = threadIdx.x / 8;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c0 + c < N) {
        const uint16_t *p = dy + (size_t)rb * N + c0 + c;
#pragma unroll 4
        for (int r = r0; r < rows; r += 32) {
            Eight e;
            float v[8];
            load8(e, p, 0, (size_t)r * N);
            e.r[1] = uint4{0, 0, 0, 0};
            values8(e, 0, v);
#pragma unroll
            for (int t = 0; t < 8; ++t) s[t] += v[t];
        }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) part[r0][c + t] = s[t];
    __syncthreads();
    if (threadIdx.x < 64 && c0 + (int)threadIdx.x < N) {
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) sum += part[r][threadIdx.x];
        bpart[(size_t)rt * N + c0 + threadIdx.x] = sum;
    }
}

// db[e] = the sum of e's row tiles' partials, in tile order (the schedule
// lists each expert's tiles in row order, experts ascending).
__global__ __launch_bounds__(256) void bias_grad_kernel(const float *__restrict__ bpart,
                                                        const int32_t *__restrict__ offsets,
                                                        int R, int N, int max_tiles,
                                                        int tile_rows, float *__restrict__ db,
                                                        int accumulate) {
    __shared__ int before[256], own;
    const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    int first = 0, n = (R + tile_rows - 1) / tile_rows;
    if (offsets) {
        int mine = 0;
        for (int i = threadIdx.x; i <= e; i += 256) {
            const int b = min(max(offsets[i], 0), R), t = min(max(offsets[i + 1], b), R);
            const int nt = (t - b + tile_rows - 1) / tile_rows;
            if (i == e) own = nt;
            else mine += nt;
        }
        before[threadIdx.x] = mine;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if ((int)threadIdx.x < o) before[threadIdx.x] += before[threadIdx.x + o];
            __syncthreads();
        }
        first = min(before[0], max_tiles);
        n = min(own, max_tiles - first);
    }
    if (c >= N) return;
    const float s = accumulate ? db[(size_t)e * N + c] : 0.f;
    const float *p = bpart + (size_t)first * N + c;
    float sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) sum += p[(size_t)i * N];
    db[(size_t)e * N + c] = s + sum;
}

template <DenseOp OP, DenseTile TILE> hipError_t run_rows(const RowsArgs &a, hipStream_t s) {
    using S = RowShape<OP, TILE>;
    constexpr int BC = S::DUAL ? S::BP / 2 : S::BP;
    const int ct = (a.Np + BC - 1) / BC;
    const int rt = a.tiles ? a.max_tiles : (a.R + S::BQ - 1) / S::BQ;
    const int per = a.tiles ? xcd_tile_cap(a.R, a.E, S::BQ, a.max_tiles) * ct : (rt * ct + 7) / 8;
    rows_kernel<OP, TILE><<<8 * per, S::Threads, 0, s>>>(a, ct, rt);
    return hipGetLastError();
}
template <DenseOp OP> hipError_t pick_rows(const RowsArgs &a, hipStream_t s) {
    switch (a.tile) {
        case kTile256: return run_rows<OP, kTile256>(a, s);
        case kTile128: return run_rows<OP, kTile128>(a, s);
        case kTile128D: return run_rows<OP, kTile128D>(a, s);
        default: return run_rows<OP, kTile64>(a, s);
    }
}

template <DenseTile TILE> hipError_t run_grad(const GradArgs &a, hipStream_t s) {
    constexpr int B = tile_rows(TILE);
    const int nt = (a.N + B - 1) / B, kt = (a.K + B - 1) / B;
    const int tiles = a.E * a.mats * nt * kt;
    grad_kernel<TILE><<<(tiles + 7) / 8 * 8, kThreads<TILE>, 0, s>>>(a, nt, kt, tiles);
    return hipGetLastError();
}

// The tile shape that takes the least time for `tiles(rows)` tiles, in percent
// of a round of 256-row tiles.
template <class F> DenseTile best_tile(F &&tiles) {
    const int64_t large = tiles(256), small = tiles(128), tiny = tiles(64);
    auto rounds = [](int64_t n, int64_t per) { return (n + per - 1) / per; };
    const int64_t l = rounds(large, kCus) * 100;
    const int64_t s = small <= kCus ? 40 : rounds(small, 2 * kCus) * 65;
    const int64_t t = rounds(tiny, 2 * kCus) * 31;
    return l <= s && l <= t ? kTile256 : s <= t ? (small <= kCus ? kTile128D : kTile128) : kTile64;
}

}  // namespace

DenseTile dense_tile(int R, int E, int cols, bool grouped) {
    if (grouped) return R >= E * 256LL ? kTile256 : R >= E * 64LL ? kTile128 : kTile64;
    return best_tile([&](int r) { return (int64_t)((R + r - 1) / r) * ((cols + r - 1) / r); });
}

hipError_t launch_rows(DenseOp op, const RowsArgs &a, hipStream_t s) {
    switch (op) {
        case kGlu: return pick_rows<kGlu>(a, s);
        case kGluGrad: return pick_rows<kGluGrad>(a, s);
        case kLinear: return pick_rows<kLinear>(a, s);
        case kLinGrad: return pick_rows<kLinGrad>(a, s);
        default: return pick_rows<kInput>(a, s);
    }
}

int64_t rows_tiles(int R, int E, int Np) {
    return (int64_t)((R + 63) / 64 + E + 8) * ((Np + 31) / 32);
}

int64_t grad_tiles(int E, int N, int K, int mats, int rows) {
    return (int64_t)E * mats * ((N + rows - 1) / rows) * ((K + rows - 1) / rows);
}

hipError_t launch_grad(const GradArgs &a, hipStream_t s) {
    switch (best_tile([&](int r) { return grad_tiles(a.E, a.N, a.K, a.mats, r); })) {
        case kTile256: return run_grad<kTile256>(a, s);
        case kTile128: return run_grad<kTile128>(a, s);
        case kTile128D: return run_grad<kTile128D>(a, s);
        default: return run_grad<kTile64>(a, s);
    }
}

hipError_t launch_colsum(const uint16_t *dy, int R, int N, const int4 *tiles, WsHeader *hdr,
                         int max_tiles, int tile_rows, float *bpart, hipStream_t s) {
    const int rt = tiles ? max_tiles : (R + tile_rows - 1) / tile_rows;
    colsum_kernel<<<dim3((N + 63) / 64, rt), 256, 0, s>>>(dy, R, N, tiles, hdr, max_tiles,
                                                                tile_rows, bpart);
    return hipGetLastError();
}

hipError_t launch_bias_grad(const float *bpart, const int32_t *offsets, int R, int E, int N,
                            int max_tiles, int tile_rows, float *db, int accumulate,
                            hipStream_t s) {
    bias_grad_kernel<<<dim3((N + 255) / 256, E), 256, 0, s>>>(bpart, offsets, R, N, max_tiles,
                                                              tile_rows, db, accumulate);
    return hipGetLastError();
}

hipError_t launch_dense_schedule(const int32_t *offsets, int E, int R, int tile_rows,
                                 const DenseWs &L, char *ws, hipStream_t s) {
    dense_schedule_kernel<<<1, kPrepThreads, 0, s>>>(
        offsets, E, R, tile_rows, L.max_tiles, (int4 *)(ws + L.active), (int4 *)(ws + L.tiles),
        (int *)(ws + L.split_cnt), (WsHeader *)ws);
    return hipGetLastError();
}

}  // namespace fw
