// The bf16 MFMA tile product of the training kernels: one workgroup forms a
// BP x BQ tile of P Q^T over a reduction of any length, operands staged HBM/L2
// -> LDS by range-checked DMA, 64 reduction steps at a time, into one of two
// buffers while the other is used.
//
// Each operand is either stored along the reduction (its rows are the tile's
// rows, "along") or across it (its rows are reduction steps, "across": weight
// rows in dx, activation and gradient rows in dW).  Along: LDS holds [rows][64]
// in 16-byte chunks, chunk c of row r at c ^ (r % 8), and a lane's MFMA operand
// (row l % 32, steps 8 (l / 32) .. + 7 of a 16-step slice) is one ds_read_b128
// whose eight-lane groups touch eight different chunk columns.  Across: LDS
// holds [64][cols] with the 64-byte column blocks of row k moved by xor k % 4,
// and the operand is two ds_read_b64_tr_b16, each 16-lane group reading four
// rows x 32 bytes and receiving them transposed (four steps of one column per
// lane); the xor puts the four rows' blocks into different banks.
//
// The first MFMA operand is P and the accumulator holds, per lane, four
// consecutive P indices of one Q index: P is the output's contiguous dimension.
#pragma once

#include "dense.h"

namespace fw {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kStepK = 64;                  // reduction steps per stage
constexpr uint32_t kNoChunk = 0x80000000u;  // an offset beyond every range

// BP x BQ tile by WP x WQ wavefronts; PX / QX: the operand is stored across.
template <int BP_, int BQ_, int WP_, int WQ_, bool PX_, bool QX_, bool DUAL_> struct Shape {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_;
    static constexpr bool PX = PX_, QX = QX_;
    // the P tile is half of one matrix and half of another, so that a wavefront
    // holds the same columns of both
    static constexpr bool DUAL = DUAL_;
    static constexpr int NW = WP * WQ, Threads = 64 * NW;
    static constexpr int PI = BP / WP / 32, QJ = BQ / WQ / 32;
    static constexpr int PChunks = BP * kStepK / 8, QChunks = BQ * kStepK / 8;
    static_assert(!DUAL || PI == 2, "a dual tile holds one column group of each matrix");
    static_assert(PChunks % Threads == 0 && QChunks % Threads == 0, "whole DMA instructions");
    // tile index of the first row of wavefront wp's P group i
    static __device__ __forceinline__ int prow(int wp, int i) {
        return DUAL ? i * (BP / 2) + 32 * wp : wp * (BP / WP) + 32 * i;
    }
    static __device__ __forceinline__ int qrow(int wq, int j) { return wq * (BQ / WQ) + 32 * j; }
};

// One operand as the tile sees it.  along: base = the tile's first row, `rows`
// rows of `pitch` bytes, reduction length Kd along them.  across: base = the
// tile's first column at reduction step 0, steps `pitch` bytes apart, `rows`
// unused.  Chunks outside (rows past the end, steps past Kd) read as zero.
struct Operand {
    const char *base;
    int rows;
    uint32_t pitch;
    uint32_t tail;   // across: bytes of a row in front of the tile's first column
};

typedef __amdgpu_buffer_rsrc_t rsrc_t;
__device__ __forceinline__ rsrc_t make_rsrc(const char *p, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes;
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, (int)n, 0x00020000);
}

// The DMA of one operand's stage: ROWS tile rows (columns when ACROSS), in a
// dual tile the first half of one matrix and the second of another.
template <int ROWS, bool ACROSS, int NW, bool DUAL = false> struct Stager {
    static_assert(!ACROSS || (ROWS >= 128 && !DUAL), "four 64-byte blocks to permute");
    static constexpr int kInstr = ROWS * kStepK / 8 / (64 * NW);
    static constexpr int kRowChunks = ACROSS ? ROWS / 8 : kStepK / 8;
    uint32_t off[kInstr];
    int kc;   // along: the lane's first reduction step within the stage

    __device__ __forceinline__ void init(int wave, int lane, uint32_t pitch) {
#pragma unroll
        for (int i = 0; i < kInstr; ++i) {
            const int idx = (i * NW + wave) * 64 + lane;
            const int r = idx / kRowChunks, p = idx % kRowChunks;
            if constexpr (ACROSS) {
                off[i] = (uint32_t)r * pitch + 16u * (uint32_t)(p ^ ((r & 3) << 2));
            } else {
                const int c = p ^ (r & 7);
                off[i] = (uint32_t)(DUAL ? r % (ROWS / 2) : r) * pitch + 16u * (uint32_t)c;
                if (i == 0) kc = 8 * c;   // r % 8 = lane / 8 in every instruction
            }
        }
    }
    // rows row0 .. row0 + n of the operand's stage that starts at step k
    __device__ __forceinline__ rsrc_t rsrc(const Operand &o, int k, int Kd) const {
        if constexpr (ACROSS) {
            const int left = min(Kd - k, kStepK);
            return make_rsrc(o.base + (int64_t)k * o.pitch, (int64_t)left * o.pitch - o.tail);
        } else {
            return make_rsrc(o.base + 2 * (int64_t)k,
                             k < Kd ? (int64_t)o.rows * o.pitch - 2 * (int64_t)k : 0);
        }
    }
    __device__ __forceinline__ void issue(rsrc_t r, uint4 *lds, int wave, int k, int Kd,
                                          int i) const {
        const uint32_t o = ACROSS || k + kc < Kd ? off[i] : kNoChunk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + (i * NW + wave) * 64), 16,
                                                 o, 0, 0, 0);
    }
};

// A lane's MFMA operands: slice s of the N groups of 32 tile rows (columns)
// that start at the rows init is given.
template <int ROWS, bool ACROSS, int N> struct Reader {
    uint32_t at[N];            // byte offset per group
    uint32_t in[4];            // along: the lane's chunk in a row, per slice
    template <class F> __device__ __forceinline__ void init(int lane, F &&row0) {
        if constexpr (ACROSS) {
            const int j = lane & 15, q = lane >> 4;
            // the lane reads step 8 (q / 2) + j / 4 (+ 4), columns
            // 16 (q % 2) + 4 (j % 4) .. + 3; its 64-byte block index is xored
            // with step % 4 = j / 4
            const uint32_t row = (uint32_t)(8 * (q >> 1) + (j >> 2)) * (2 * ROWS);
#pragma unroll
            for (int i = 0; i < N; ++i)
                at[i] = row + 64u * (uint32_t)((row0(i) >> 5) ^ (j >> 2)) + 32u * (q & 1) +
                        8u * (j & 3);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i] = 128u * (uint32_t)(row0(i) + (lane & 31));
#pragma unroll
            for (int s = 0; s < 4; ++s) in[s] = 16u * (uint32_t)((2 * s + (lane >> 5)) ^ (lane & 7));
        }
    }
    __device__ __forceinline__ bf8 read(const uint4 *lds, int i, int s) const {
        if constexpr (ACROSS) {
            const char *p = (const char *)lds + at[i] + (uint32_t)s * (16 * 2 * ROWS);
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * 2 * ROWS));
            return __builtin_bit_cast(
                bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(const bf8 *)((const char *)lds + at[i] + in[s]);
        }
    }
};

// acc[i][j] (PI x QJ groups of 32 x 32) = the tile product over nseg segments
// of Kd steps; p(seg) / pb(seg) and q(seg) give the operands (pb: the second
// matrix of a dual P tile).
template <class S, class PF, class PBF, class QF>
__device__ __forceinline__ void tile_product(f16v (&acc)[S::PI][S::QJ], uint4 *P0, uint4 *P1,
                                             uint4 *Q0, uint4 *Q1, int wave, int lane, int Kd,
                                             int nseg, PF &&p, PBF &&pb, QF &&q) {
    const int wp = wave % S::WP, wq = wave / S::WP;
    Stager<S::BP, S::PX, S::NW, S::DUAL> ps;
    Stager<S::BQ, S::QX, S::NW> qs;
    ps.init(wave, lane, p(0).pitch);
    qs.init(wave, lane, q(0).pitch);
    Reader<S::BP, S::PX, S::PI> pr;
    Reader<S::BQ, S::QX, S::QJ> qr;
    pr.init(lane, [&](int i) { return S::prow(wp, i); });
    qr.init(lane, [&](int j) { return S::qrow(wq, j); });
#pragma unroll
    for (int i = 0; i < S::PI; ++i)
#pragma unroll
        for (int j = 0; j < S::QJ; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.f;

    const int per = (Kd + kStepK - 1) / kStepK, steps = per * nseg;
    if (steps == 0) return;
    auto load = [&](int st, uint4 *pl, uint4 *ql) {
        const int seg = st >= per, k = (st - seg * per) * kStepK;   // nseg <= 2
        const int kd = st < steps ? Kd : 0;   // past the end: zeros
        const rsrc_t rq = qs.rsrc(q(seg), k, kd);
#pragma unroll
        for (int i = 0; i < qs.kInstr; ++i) qs.issue(rq, ql, wave, k, kd, i);
        const rsrc_t ra = ps.rsrc(p(seg), k, kd);
        if constexpr (S::DUAL) {
            const rsrc_t rb = ps.rsrc(pb(seg), k, kd);
#pragma unroll
            for (int i = 0; i < ps.kInstr; ++i) ps.issue(2 * i < ps.kInstr ? ra : rb, pl, wave, k, kd, i);
        } else {
#pragma unroll
            for (int i = 0; i < ps.kInstr; ++i) ps.issue(ra, pl, wave, k, kd, i);
        }
    };
    auto step = [&](const uint4 *pl, const uint4 *ql) {
#pragma unroll
        for (int s = 0; s < kStepK / 16; ++s) {
            bf8 a[S::PI], b[S::QJ];
#pragma unroll
            for (int i = 0; i < S::PI; ++i) a[i] = pr.read(pl, i, s);
#pragma unroll
            for (int j = 0; j < S::QJ; ++j) b[j] = qr.read(ql, j, s);
#pragma unroll
            for (int i = 0; i < S::PI; ++i)
#pragma unroll
                for (int j = 0; j < S::QJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[i], b[j], acc[i][j], 0,
                                                                        0, 0);
        }
    };
    // everything issued so far has landed and every wavefront is here: the
    // buffer read before may be refilled
    auto sync = [&]() {
        __builtin_amdgcn_s_waitcnt(7 << 4);   // vmcnt(0) lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    load(0, P0, Q0);
    sync();
    // Two steps per turn, so that each buffer keeps its name (the compiler then
    // knows that a pending DMA and a read touch different arrays).  Past the
    // last step the loads are out of range and write zeros.
    int st = 0;
    for (; st + 1 < steps; st += 2) {
        load(st + 1, P1, Q1);
        step(P0, Q0);
        sync();
        load(st + 2, P0, Q0);
        step(P1, Q1);
        sync();
    }
    if (st < steps) step(P0, Q0);
}

}  // namespace fw
