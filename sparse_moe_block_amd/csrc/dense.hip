// The bf16 training products: the gated feed-forward products and the linear
// product with their epilogues, their input gradients and their weight and
// bias gradients, for one matrix or one per expert (rows grouped by
// expert_offsets).  Every product runs on v_mfma_f32_16x16x32_bf16 with fp32
// accumulators (dense_core.h).
//
// Backward.  g, u (and z) are formed again from x instead of being kept: their
// product's epilogue turns the accumulators and the arriving gradient straight
// into dg, du (dz), so neither g nor u ever reaches memory.  dg, du and dz are
// rounded to bf16 there (half a step, at most 2^-8 relative), the only way into the
// bf16 products that follow; the bias gradient is summed before that rounding.
#include <math.h>

#include <algorithm>
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

// Stores past the caches, for outputs larger than they are.  A wavefront's store
// has to fill whole lines then: fp32 values with eight a lane took 964 us where
// 16 bytes a lane side by side take 621 (16384 rows over 128 experts, 2048 -> 1536,
// dW of 1.6 GB, whole call).
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store16(void *p, bool past, u4 v) {
    // of different types, or the compiler makes one plain store of the two
    if (past) __builtin_nontemporal_store(v, (u4 *)p);
    else *(uint4 *)p = uint4{v.x, v.y, v.z, v.w};
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
constexpr int kBlockRows = 4;   // 8: up to 3 % slower
__device__ __forceinline__ int dense_block(int block_id, int row_tiles, int col_tiles, int &ct) {
    const int total = row_tiles * col_tiles, per = (total + 7) / 8;
    const int idx = block_id / 8, id = (block_id % 8) * per + idx;
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
//  kTileWide  256 columns x 128 rows, eight wavefronts of 64 x 64, three stages,
//             one workgroup a CU (row products only)
//  kTile128   128 x 128, four wavefronts of 64 x 64, two stages, two workgroups
//             a CU
//  kTile128D  128 x 128, eight wavefronts of 32 x 64, four stages, one workgroup
//             a CU: for products whose tiles do not fill the CUs twice
//  kTile64    64 x 64, four wavefronts of 32 x 32, four stages, two workgroups a
//             CU: for products of few tiles
template <DenseTile TILE, bool PX, bool QX, bool DUAL>
using TileShape = std::conditional_t<
    TILE == kTile256, Shape<256, 256, 4, 2, 2, PX, QX, DUAL>,
    std::conditional_t<
        TILE == kTileWide, Shape<256, 128, 4, 2, 3, PX, QX, DUAL>,
        std::conditional_t<TILE == kTile128, Shape<128, 128, 2, 2, 2, PX, QX, DUAL>,
                           std::conditional_t<TILE == kTile128D,
                                              Shape<128, 128, 4, 2, 4, PX, QX, DUAL>,
                                              Shape<64, 64, 2, 2, 4, PX, QX, DUAL>>>>>;
template <DenseOp OP, DenseTile TILE>
using RowShape = TileShape<TILE, OP == kInput, false, OP == kGlu || OP == kGluGrad>;
template <DenseTile TILE>
constexpr int kThreads = TILE == kTile128 || TILE == kTile64 ? 256 : 512;
template <DenseTile TILE> constexpr int kBlocksPerCu = kThreads<TILE> == 512 ? 1 : 2;

// One (row tile rt, column tile ct).
template <DenseOp OP, class S>
__device__ __forceinline__ void rows_tile(const RowsArgs &a, const Ring<S::NS> &ring, int rt,
                                          int ct) {
    constexpr int BC = S::DUAL ? S::BP / 2 : S::BP;   // output columns of a tile
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

template <DenseOp OP, DenseTile TILE>
__global__ __launch_bounds__(kThreads<TILE>, kBlocksPerCu<TILE>) void rows_kernel(
    RowsArgs a, int col_tiles, int row_tiles) {
    using S = RowShape<OP, TILE>;
    FW_RING(S, ring);
    int ct, rt;
    if (a.tiles) {
        rt = xcd_row_tile(a.hdr, col_tiles, row_tiles, 0, 0, ct);
        // dx takes the experts from the last to the first: the weights that the
        // recomputation before it read last are still in the memory-side cache
        // (4096 rows over 128 experts, 2048 -> 2 x 768, whole call: 562 -> 534 us)
        if (OP == kInput && rt >= 0) {
            const int xcd = blockIdx.x % 8, n = min(ld_const(&a.hdr->n_tiles), row_tiles);
            rt = ld_const(&a.hdr->xcd_first[xcd]) +
                 min(ld_const(&a.hdr->xcd_first[xcd + 1]), n) - 1 - rt;
        }
    } else {
        rt = dense_block(blockIdx.x, row_tiles, col_tiles, ct);
    }
    if (rt >= 0) rows_tile<OP, S>(a, ring, rt, ct);
}

// XCD x takes an eighth of a list of `tiles`; -1: none.
__device__ __forceinline__ int grad_block(int block, int tiles) {
    const int per = (tiles + 7) / 8, id = (block % 8) * per + block / 8;
    return block / 8 < per && id < tiles ? id : -1;
}

// dw tile id (k tiles fastest): Q = output features (rows of dw), P = input
// features.
template <class S>
__device__ __forceinline__ void grad_tile(const GradArgs &a, const Ring<S::NS> &ring, int nt,
                                          int kt, int id) {
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
    if (a.out_f32) {
        constexpr int gap = kOutCols<S> / 2;   // from a lane's first four to its second
        auto half = [&](int n, int k) { return (u4 *)((float *)dw + place(n, k)); };
        auto fetch = [&](int n, int k) {
            Eight e{};
            if (a.accumulate && inside(n, k)) e.r[0] = *(const uint4 *)half(n, k);
            if (a.accumulate && inside(n, k + gap)) e.r[1] = *(const uint4 *)half(n, k + gap);
            return e;
        };
        hand_out<S, true>(acc, ring.p[0], wave, lane, fetch,
                          [&](int n, int k, float *v, const float *, const Eight &e) {
            float o[8];
            values8(e, 1, o);
            uint32_t b[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) b[t] = __float_as_uint(a.accumulate ? v[t] + o[t] : v[t]);
            if (inside(n, k)) store16(half(n, k), a.stream, u4{b[0], b[1], b[2], b[3]});
            if (inside(n, k + gap)) store16(half(n, k + gap), a.stream, u4{b[4], b[5], b[6], b[7]});
        });
    } else {
        auto at = [&](int n, int k) { return (uint16_t *)dw + place(n, k); };
        auto fetch = [&](int n, int k) {
            Eight e{};
            if (a.accumulate && inside(n, k)) load8(e, at(n, k), 0, 0);
            return e;
        };
        hand_out<S>(acc, ring.p[0], wave, lane, fetch,
                    [&](int n, int k, float *v, const float *, const Eight &e) {
            if (!inside(n, k)) return;
            if (a.accumulate) {
                float o[8];
                values8(e, 0, o);
#pragma unroll
                for (int t = 0; t < 8; ++t) v[t] += o[t];
            }
            store16(at(n, k), a.stream,
                    u4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                       pack_bf16(v[6], v[7])});
        });
    }
}

template <DenseTile TILE>
__global__ __launch_bounds__(kThreads<TILE>, kBlocksPerCu<TILE>) void grad_kernel(
    GradArgs a, int nt, int kt, int tiles) {
    using S = TileShape<TILE, true, true, false>;
    FW_RING(S, ring);
    const int id = grad_block(blockIdx.x, tiles);
    if (id >= 0) grad_tile<S>(a, ring, nt, kt, id);
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

// db[e][c] = the sum of n row tiles' partials from tile `first` on, in order.
__device__ __forceinline__ void bias_column(const BiasArgs &b, int e, int c, int first, int n) {
    if (c >= b.N) return;
    const float s = b.accumulate ? b.db[(size_t)e * b.N + c] : 0.f;
    const float *p = b.part + (size_t)first * b.N + c;
    float sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) sum += p[(size_t)i * b.N];
    b.db[(size_t)e * b.N + c] = s + sum;
}

// Expert e's tiles: the schedule lists each expert's in row order, experts
// ascending.
__global__ __launch_bounds__(256) void bias_grad_kernel(BiasArgs b) {
    __shared__ int before[256], own;
    const int e = blockIdx.y;
    int first = 0, n = (b.R + b.tile_rows - 1) / b.tile_rows;
    if (b.offsets) {
        int mine = 0;
        for (int i = threadIdx.x; i <= e; i += 256) {
            const int r = min(max(b.offsets[i], 0), b.R), t = min(max(b.offsets[i + 1], r), b.R);
            const int nt = (t - r + b.tile_rows - 1) / b.tile_rows;
            if (i == e) own = nt;
            else mine += nt;
        }
        before[threadIdx.x] = mine;
        __syncthreads();
        for (int o = 128; o > 0; o >>= 1) {
            if ((int)threadIdx.x < o) before[threadIdx.x] += before[threadIdx.x + o];
            __syncthreads();
        }
        first = min(before[0], b.max_tiles);
        n = min(own, b.max_tiles - first);
    }
    bias_column(b, e, blockIdx.x * 256 + threadIdx.x, first, n);
}

// dx, dw and the bias gradient of one matrix in one launch: they depend on dz
// alone, and the tiles of one fill the CUs that the other's leave idle.  Blocks:
// the product with the longer reduction, the other one, the bias columns.
// Measured, all three together against launches of their own: 777 rows, 1536 ->
// 4096: 51 us against 63; 1023 rows, 2048 -> 2 x 1376: 59 us against 63 (whole calls).
template <DenseTile TILE>
__global__ __launch_bounds__(kThreads<TILE>, kBlocksPerCu<TILE>) void pair_kernel(
    RowsArgs a, GradArgs g, BiasArgs b, int ct_n, int rt_n, int nt, int kt, int dx_blocks,
    int dw_blocks, int dw_first) {
    using SR = RowShape<kInput, TILE>;
    using SG = TileShape<TILE, true, true, false>;
    static_assert(SR::PChunks == SG::PChunks && SR::QChunks == SG::QChunks, "one ring for both");
    FW_RING(SR, ring);
    int i = blockIdx.x;
    const bool first = i < (dw_first ? dw_blocks : dx_blocks);
    if (!first) i -= dw_first ? dw_blocks : dx_blocks;
    if (i >= (dw_first ? dx_blocks : dw_blocks) && !first) {
        i -= dw_first ? dx_blocks : dw_blocks;
        bias_column(b, 0, i * kThreads<TILE> + threadIdx.x, 0,
                    (b.R + b.tile_rows - 1) / b.tile_rows);
        return;
    }
    if (first == (dw_first != 0)) {
        const int id = grad_block(i, g.mats * nt * kt);
        if (id >= 0) grad_tile<SG>(g, ring, nt, kt, id);
    } else {
        int ct;
        const int rt = dense_block(i, rt_n, ct_n, ct);
        if (rt >= 0) rows_tile<kInput, SR>(a, ring, rt, ct);
    }
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
        case kTileWide: return run_rows<OP, kTileWide>(a, s);
        case kTile128D: return run_rows<OP, kTile128D>(a, s);
        default: return run_rows<OP, kTile64>(a, s);
    }
}

template <DenseTile TILE>
hipError_t run_pair(const RowsArgs &a, const GradArgs &g, const BiasArgs &b, hipStream_t s) {
    using SR = RowShape<kInput, TILE>;
    using SG = TileShape<TILE, true, true, false>;
    const int ct = (a.Np + SR::BP - 1) / SR::BP, rt = (a.R + SR::BQ - 1) / SR::BQ;
    const int nt = (g.N + SG::BQ - 1) / SG::BQ, kt = (g.K + SG::BP - 1) / SG::BP;
    const int dx = (rt * ct + 7) / 8 * 8, dw = (g.mats * nt * kt + 7) / 8 * 8;
    const int db = b.db ? (b.N + kThreads<TILE> - 1) / kThreads<TILE> : 0;
    pair_kernel<TILE><<<dx + dw + db, kThreads<TILE>, 0, s>>>(
        a, g, b, ct, rt, nt, kt, dx, dw, g.R > a.nseg * a.Kd);
    return hipGetLastError();
}

template <DenseTile TILE> hipError_t run_grad(const GradArgs &a, hipStream_t s) {
    constexpr int B = tile_rows(TILE);
    const int nt = (a.N + B - 1) / B, kt = (a.K + B - 1) / B;
    const int tiles = a.E * a.mats * nt * kt;
    grad_kernel<TILE><<<(tiles + 7) / 8 * 8, kThreads<TILE>, 0, s>>>(a, nt, kt, tiles);
    return hipGetLastError();
}

int64_t rounds(int64_t tiles, int64_t per) { return (tiles + per - 1) / per; }

}  // namespace

// The shape that takes the least time, in percent of a round of 256-row tiles.
// Measured: 2048 x 4096 -> 1536 in 76 us with 48 tiles of 256, 44 us with 192 of
// 128 two to a CU, 30 us one to a CU; 4096 x 7168 -> 2048 in 136 us with 128
// tiles of 256, 105 us with 512 of 128, 95 us with 256 wide ones; 777 x 4096 ->
// 1536 in 27.4 us with 84 tiles of 128, 25.6 us with 312 of 64; 777 x 1536 ->
// 4096 in 16.1 us with 224 tiles of 128, 22.7 us with 832 of 64.  Rows in groups
// of about 128 (2048 -> 2 x 768, 128 groups): 254 us with wide tiles, 265 us with
// 128 x 128; backwards, 300 rows over 3 experts: 68 us with tiles of 256 rows, 41
// us with 64; forward, 1000 rows over 4: 34 us with 256, 22 us with 128.
//
// Rows by expert take one row count a call, for the schedule: the best one for
// `widest` columns if the experts have equal rows; the shape with that many rows
// is the product's own choice.
DenseTile dense_tile(int R, int E, int cols, int widest) {
    auto tiles = [&](int r, int c, int n) {
        const int64_t rt = widest ? (int64_t)E * (((R + E - 1) / E + r - 1) / r) : (R + r - 1) / r;
        return rt * ((n + c - 1) / c);
    };
    auto mid = [&](int n) {
        return tiles(128, 128, n) <= kCus ? 40 : rounds(tiles(128, 256, n), kCus) * 60;
    };
    const int n = widest ? widest : cols;
    if (widest && R <= 64LL * E) return kTile64;   // 32 rows an expert: 165 us, 192 us wide
    // experts of unequal rows leave more of a smaller tile's last one empty
    const int64_t l = rounds(tiles(256, 256, n), kCus) * (widest ? 87 : 100), m = mid(n);
    const int64_t t = rounds(tiles(64, 64, n), 2 * kCus) * 31;
    return l <= m && l <= t ? kTile256
           : m <= t         ? (tiles(128, 128, cols) <= kCus ? kTile128D : kTileWide)
                            : kTile64;
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
    // as in dense_tile
    auto tiles = [&](int r) { return grad_tiles(a.E, a.N, a.K, a.mats, r); };
    const int64_t l = rounds(tiles(256), kCus) * 100;
    const int64_t m = tiles(128) <= kCus ? 40 : rounds(tiles(128), 2 * kCus) * 65;
    const int64_t t = rounds(tiles(64), 2 * kCus) * 31;
    return l <= m && l <= t ? run_grad<kTile256>(a, s)
           : m > t          ? run_grad<kTile64>(a, s)
           : tiles(128) <= kCus ? run_grad<kTile128D>(a, s)
                                : run_grad<kTile128>(a, s);
}

hipError_t launch_pair(const RowsArgs &a, const GradArgs &g, const BiasArgs &b, hipStream_t s) {
    // Time in percent of a 256-row tile's step: all tile steps at the rate of a
    // full CU (`full` a tile) over the CUs, or the longest tile at the rate of a
    // tile alone on its CU, and half of a shorter one for the end; `more` steps a
    // tile for its start and epilogue.  Fitted to nine shapes from 100 x 4096 ->
    // 4096 to 4096 x 7168 -> 2 x 2048, on each of which it picks the fastest or
    // one within 1 %.
    const int64_t sx = a.nseg * ((a.Kd + kStepK - 1) / kStepK), sw = (g.R + kStepK - 1) / kStepK;
    auto time = [&](int r, int more, int full, int alone) {
        const int64_t nx = (int64_t)((a.R + r - 1) / r) * ((a.Np + r - 1) / r);
        const int64_t nw = grad_tiles(1, g.N, g.K, g.mats, r);
        const int64_t work = (nx * (sx + more) + nw * (sw + more)) * full / kCus;
        return std::max(work, (std::max(sx, sw) + more) * alone) +
               (std::min(sx, sw) + more) * full / 2;
    };
    const int64_t l = time(256, 4, 100, 85), m = time(128, 3, 40, 45), d = time(128, 3, 42, 27),
                  t = time(64, 2, 20, 12);
    const int64_t best = std::min({l, m, d, t});
    return best == l   ? run_pair<kTile256>(a, g, b, s)
           : best == m ? run_pair<kTile128>(a, g, b, s)
           : best == d ? run_pair<kTile128D>(a, g, b, s)
                       : run_pair<kTile64>(a, g, b, s);
}

hipError_t launch_colsum(const uint16_t *dy, int R, int N, const int4 *tiles, WsHeader *hdr,
                         int max_tiles, int tile_rows, float *bpart, hipStream_t s) {
    const int rt = tiles ? max_tiles : (R + tile_rows - 1) / tile_rows;
    colsum_kernel<<<dim3((N + 63) / 64, rt), 256, 0, s>>>(dy, R, N, tiles, hdr, max_tiles,
                                                                tile_rows, bpart);
    return hipGetLastError();
}

hipError_t launch_bias_grad(const BiasArgs &b, int E, hipStream_t s) {
    bias_grad_kernel<<<dim3((b.N + 255) / 256, E), 256, 0, s>>>(b);
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
