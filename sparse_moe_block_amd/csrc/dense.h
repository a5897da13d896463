// Internal declarations of the bf16 training products (fw_moe_glu_*,
// fw_moe_linear_*): workspace layout, launch arguments, launchers, and the
// activation functions of their epilogues.
#pragma once

#include "common.h"

namespace fw {

// Row tiles are at least this long, so R / kDenseMinTileRows + E bounds them.
constexpr int kDenseMinTileRows = 64;

// Byte offsets of the scratch areas of one call inside its workspace.
struct DenseWs {
    size_t active;     // int4 [E + 1]           (build_schedule's active experts)
    size_t tiles;      // int4 [max_tiles]       (expert, first row, rows) per row tile
    size_t split_cnt;  // int [kSplitTiles]      (cleared by build_schedule)
    size_t xq;         // bf16 [R][K]            the checkpoint's values (backward, 8-bit x)
    size_t dz;         // bf16 [mats][R][N]      dg then du, or dz
    size_t bpart;      // f32 [max_tiles][N]     per-row-tile column sums of dz
    size_t total;
    int max_tiles;
};
// mats: 2 for the gated products, 1 for the linear one; the larger area
// serves both.
DenseWs dense_ws(const fw_moe_dense_desc &d, int R);

// Tile shapes (dense.hip) and their rows.
enum DenseTile { kTile64, kTile128D, kTile128, kTileWide, kTile256 };
constexpr int tile_rows(DenseTile t) { return t == kTile256 ? 256 : t == kTile64 ? 64 : 128; }

// One product over row tiles: out rows from rows of q (bf16 [R][Kd], row pitch
// Kd) times weights, with an epilogue.
//   kGlu      h = f(q Wg^T) * (q Wu^T)
//   kGluGrad  the same g and u; dg = dh u f'(g), du = dh f(g) (and h if set)
//   kLinear   y = f(q W^T + b) + residual
//   kLinGrad  z = q W^T + b; dz = dy f'(z), and the tile's column sums of dz
//   kInput    dx = sum over nseg of q_seg W_seg (the weights read along their
//             rows: reduction over out_features)
enum DenseOp { kGlu, kGluGrad, kLinear, kLinGrad, kInput };

struct RowsArgs {
    const uint16_t *q;         // bf16 rows (kInput: dz, segment s at q + s * q_seg)
    size_t q_seg;
    const uint16_t *w0, *w1;   // bf16 weights (expert stride w_stride elements)
    size_t w_stride;
    int Kd;                    // reduction length (of a segment)
    int nseg;                  // 1, or 2: the reduction runs over two row / weight pairs
    int Np;                    // output features
    int R, E, fn;
    const int4 *tiles;         // row tiles, or nullptr: all R rows of expert 0
    WsHeader *hdr;
    int max_tiles;
    DenseTile tile;
    const float *bias;         // [E][Np] or nullptr
    const void *residual;      // out's type, or nullptr
    const uint16_t *dy;        // bf16 [R][Np]: the arriving gradient
    void *out;                 // h, y or dx; kGluGrad: bf16 h or nullptr
    int out_f32;
    uint16_t *dz;              // kGluGrad: dg, then du at + R * Np; kLinGrad: dz
    float *bpart;              // kLinGrad: [row tile][Np] or nullptr
};
constexpr int kCus = 256;      // the MI355X's compute units
// The tile shape of a product with `cols` output columns; widest: the most columns
// of the call's products where the row tiles come from a schedule, 0 otherwise.
DenseTile dense_tile(int R, int E, int cols, int widest);
hipError_t launch_rows(DenseOp op, const RowsArgs &a, hipStream_t s);

// kGlu and kLinear for few rows an expert (dense_few.hip), straight from
// offsets.  Several experts: up to 8 rows on average (128 experts, 2048 -> 1024:
// 96 us against the tiles' 119 at 4 rows, 126 against 127 at 8, 176 against 129
// at 16).  One matrix: up to 16 rows, and up to 32 of a long reduction, which is
// what the tiles' time grows with (32 rows, 7168 -> 2 x 2048: 22 us against 35;
// 2048 -> 7168: 14 us against 10.5).
constexpr bool few_rows(int R, int E, int K) {
    return E > 1 ? R <= 8 * E : R <= 16 || (R <= 32 && K >= 4096);
}
hipError_t launch_few(bool glu, const RowsArgs &a, const int32_t *offsets, hipStream_t s);

// Weight gradients: dw[e][n][k] = sum over the rows r of e of dz[r][n] x[r][k].
struct GradArgs {
    const uint16_t *dz;        // bf16 [mats][R][N]
    const uint16_t *x;         // bf16 [R][K]
    int R, E, N, K, mats;
    const int32_t *offsets;    // [E + 1] or nullptr: all rows
    void *dw0, *dw1;           // [E][N][K]
    int out_f32, accumulate;
    // gradients that outgrow the 256 MB Infinity Cache are stored past it (128
    // experts' 2 x 768 x 2048, 805 MB: the whole backward 783 -> 737 us)
    int stream;
};
hipError_t launch_grad(const GradArgs &a, hipStream_t s);
// Number of workgroups of that launch (the ABI refuses grids HIP cannot hold).
int64_t grad_tiles(int E, int N, int K, int mats, int rows);
int64_t rows_tiles(int R, int E, int Np);

// db[e][n] = sum over e's rows of dz: per row tile (colsum: from bf16 rows
// dy; kLinGrad writes the same partials itself), then over e's tiles in order.
hipError_t launch_colsum(const uint16_t *dy, int R, int N, const int4 *tiles, WsHeader *hdr,
                         int max_tiles, int tile_rows, float *bpart, hipStream_t s);
struct BiasArgs {
    const float *part;         // [row tile][N]
    const int32_t *offsets;    // as in GradArgs
    int R, N, max_tiles, tile_rows;
    float *db;                 // [E][N] (launch_pair: nullptr if not wanted)
    int accumulate;
};
hipError_t launch_bias_grad(const BiasArgs &b, int E, hipStream_t s);
// dx (kInput), dw and db of one matrix without offsets in one launch.
hipError_t launch_pair(const RowsArgs &a, const GradArgs &g, const BiasArgs &b, hipStream_t s);

hipError_t launch_dense_schedule(const int32_t *offsets, int E, int R, int tile_rows,
                                 const DenseWs &L, char *ws, hipStream_t s);

// 8-bit blocks (ckpt.hip)
hipError_t launch_ckpt_pack(int format, int64_t blocks, const void *src, int src_bf16,
                            void *codes, void *scales, WsHeader *hdr, hipStream_t s);
hipError_t launch_ckpt_unpack(int format, int64_t blocks, const void *codes, const void *scales,
                              void *dst, int dst_bf16, hipStream_t s);

// f(z) and f'(z).  gelu (tanh form): z s(2 c (z + 0.044715 z^3)), c =
// sqrt(2 / pi), s the logistic function, which is 0.5 z (1 + tanh(c (...))).
// NaN stays NaN; the polynomial's z is bounded so that 0 * polynomial is 0 at
// any finite z.
__device__ __forceinline__ float logistic(float z) { return 1.0f / (1.0f + __expf(-z)); }
constexpr float kGelu2C = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
__device__ __forceinline__ float act_value(int fn, float z) {
    if (fn == FW_FN_SILU) return z * logistic(z);
    if (fn == FW_FN_GELU_TANH) return z * logistic(kGelu2C * fmaf(kGeluA * z * z, z, z));
    if (fn == FW_FN_RELU) return z <= 0.0f ? 0.0f : z;
    return z;
}
__device__ __forceinline__ void act_both(int fn, float z, float &f, float &df) {
    if (fn == FW_FN_SILU) {
        const float s = logistic(z);
        f = z * s;
        df = fmaf(f, 1.0f - s, s);
    } else if (fn == FW_FN_GELU_TANH) {
        const float b = fminf(fmaxf(z, -1e15f), 1e15f);
        const float s = logistic(kGelu2C * fmaf(kGeluA * b * b, b, b));
        f = z * s;
        df = fmaf(f * (1.0f - s), kGelu2C * fmaf(3.0f * kGeluA * b, b, 1.0f), s);
    } else if (fn == FW_FN_RELU) {
        f = z <= 0.0f ? 0.0f : z;
        df = z > 0.0f ? 1.0f : 0.0f;
    } else {
        f = z;
        df = 1.0f;
    }
}

// bf16 from fp32, nearest-even (NaN stays NaN)
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return __builtin_bit_cast(uint32_t, b2{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ float bf16_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

}  // namespace fw
