// The bf16 MFMA tile product of the training kernels: one workgroup forms a
// BP x BQ tile of P Q^T over a reduction of any length, operands staged HBM/L2
// -> LDS by range-checked DMA, 64 reduction steps a stage, in a ring of two to
// four stages.
//
// Each operand is either stored along the reduction (its rows are the tile's
// rows, "along") or across it (its rows are reduction steps, "across": weight
// rows in dx, activation and gradient rows in dW).  Along: LDS holds [rows][64]
// in 16-byte chunks, chunk c of row r at c ^ (r / 2 % 8), and a lane's MFMA
// operand (row l % 16, steps 8 (l / 16) .. + 7 of a 32-step slice) is one
// ds_read_b128: the sixteen lanes served at once read sixteen rows, two rows to
// a 256-byte turn of the banks, at sixteen different places in it (with
// c ^ (r % 8) rows eight apart met: half of the LDS cycles were conflicts).
// Across: LDS holds [64][cols] with the 32-byte column blocks of a row moved by
// xor (across_key), and the operand is two ds_read_b64_tr_b16, each 16-lane
// group reading four rows x 32 bytes and receiving them transposed (four steps
// of one column per lane); the xor puts the eight rows that 32 lanes read at
// once into different banks.
//
// v_mfma_f32_16x16x32_bf16 rather than the 32x32x16 form: the large tiles run at
// the clock that power allows, and it moves half as many accumulator registers a
// flop (4096 x 7168 -> 2 x 2048: 178 us against 190).
//
// The first MFMA operand is P and the accumulator holds, per lane, four
// consecutive P indices of one Q index: P is the output's contiguous dimension.
#pragma once

#include <type_traits>

#include "dense.h"

namespace fw {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kStepK = 64;                  // reduction steps per stage
constexpr int kSlices = kStepK / 32;        // of 32, one MFMA deep
constexpr uint32_t kNoChunk = 0x80000000u;  // an offset beyond every range

// BP x BQ tile by WP x WQ wavefronts, NS stages of 64 reduction steps; PX / QX:
// the operand is stored across.
template <int BP_, int BQ_, int WP_, int WQ_, int NS_, bool PX_, bool QX_, bool DUAL_>
struct Shape {
    static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NS = NS_;
    static constexpr bool PX = PX_, QX = QX_;
    // the P tile is half of one matrix and half of another, so that a wavefront
    // holds the same columns of both
    static constexpr bool DUAL = DUAL_;
    static constexpr int NW = WP * WQ, Threads = 64 * NW;
    static constexpr int PI = BP / WP / 16, QJ = BQ / WQ / 16;
    // 16-byte chunks of a stage
    static constexpr int PChunks = BP * kStepK / 8, QChunks = BQ * kStepK / 8;
    static_assert(!DUAL || PI % 2 == 0, "a dual tile's wavefront holds as many groups of each matrix");
    static_assert(PChunks % Threads == 0 && QChunks % Threads == 0, "whole DMA instructions");
    // tile index of the first row of wavefront wp's P group i
    static __device__ __forceinline__ int prow(int wp, int i) {
        return DUAL ? i / (PI / 2) * (BP / 2) + wp * (BP / 2 / WP) + 16 * (i % (PI / 2))
                    : wp * (BP / WP) + 16 * i;
    }
    static __device__ __forceinline__ int qrow(int wq, int j) { return wq * (BQ / WQ) + 16 * j; }
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
// At most 256 rows of 131072 bytes: 32-bit lengths; none if negative.
__device__ __forceinline__ rsrc_t make_rsrc(const char *p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, max(bytes, 0), 0x00020000);
}

// The 32-byte column block of an across operand's row is moved by xor this key:
// the eight rows that 32 lanes read at once (r % 4, r / 8 % 2) differ in it, or,
// in rows of 64 columns (two to a turn of the banks), four pairs of them do.
template <int ROWS> __device__ __forceinline__ int across_key(int r) {
    return ROWS >= 128 ? (r & 3) | ((r >> 1) & 4) : ((r >> 1) & 1) | ((r >> 2) & 2);
}

// The DMA of one operand's stage: ROWS tile rows (columns when ACROSS), in a
// dual tile the first half of one matrix and the second of another.
template <int ROWS, bool ACROSS, int NW, bool DUAL = false> struct Stager {
    static_assert(!ACROSS || (ROWS >= 128 && !DUAL) || ROWS == 64, "whole column blocks");
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
                off[i] = (uint32_t)r * pitch + 16u * (uint32_t)(p ^ (across_key<ROWS>(r) << 1));
            } else {
                const int c = p ^ ((r >> 1) & 7);
                off[i] = (uint32_t)(DUAL ? r % (ROWS / 2) : r) * pitch + 16u * (uint32_t)c;
                if (i == 0) kc = 8 * c;   // r / 2 % 8 is the same in every instruction
            }
        }
    }
    // rows row0 .. row0 + n of the operand's stage that starts at step k
    __device__ __forceinline__ rsrc_t rsrc(const Operand &o, int k, int Kd) const {
        if constexpr (ACROSS) {
            const int left = min(Kd - k, kStepK);
            return make_rsrc(o.base + (int64_t)k * o.pitch, left * (int)o.pitch - (int)o.tail);
        } else {
            return make_rsrc(o.base + 2 * (int64_t)k, k < Kd ? o.rows * (int)o.pitch - 2 * k : 0);
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void issue(rsrc_t r, uint4 *lds, int wave, int k, int Kd,
                                          int i) const {
        const uint32_t o = WHOLE || ACROSS || k + kc < Kd ? off[i] : kNoChunk;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)(lds + (i * NW + wave) * 64), 16,
                                                 o, 0, 0, 0);
    }
};

// A lane's MFMA operands: slice s of the N groups of 16 tile rows (columns)
// that start at the rows init is given.
template <int ROWS, bool ACROSS, int N> struct Reader {
    uint32_t at[N];         // byte offset per group
    uint32_t in[kSlices];   // along: the lane's chunk in a row, per slice
    template <class F> __device__ __forceinline__ void init(int lane, F &&row0) {
        const int q = lane >> 4, j = lane & 15;
        if constexpr (ACROSS) {
            // the lane reads step 8 q + j / 4 (+ 4, + 32 s), columns 4 (j % 4) .. + 3
            // of the group: in-group lane i then holds column i, four steps
            const int r = 8 * q + (j >> 2);
#pragma unroll
            for (int i = 0; i < N; ++i)
                at[i] = (uint32_t)r * (2 * ROWS) +
                        32u * (uint32_t)((row0(i) >> 4) ^ across_key<ROWS>(r)) + 8u * (j & 3);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) at[i] = 2u * kStepK * (uint32_t)(row0(i) + j);
#pragma unroll
            for (int s = 0; s < kSlices; ++s) in[s] = 16u * (uint32_t)((4 * s + q) ^ ((j >> 1) & 7));
        }
    }
    __device__ __forceinline__ bf8 read(const uint4 *lds, int i, int s) const {
        if constexpr (ACROSS) {
            const char *p = (const char *)lds + at[i] + (uint32_t)s * (32 * 2 * ROWS);
            const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)p);
            const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * 2 * ROWS));
            return __builtin_bit_cast(
                bf8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return *(const bf8 *)((const char *)lds + at[i] + in[s]);
        }
    }
};

// The stages' LDS: arrays of their own, so that the compiler knows that a
// pending DMA and a read touch different ones.
template <int NS> struct Ring {
    uint4 *p[NS], *q[NS];
};
#define FW_STAGE(S, n)                                          \
    __shared__ uint4 fw_p##n[S::NS > n ? S::PChunks : 1];       \
    __shared__ uint4 fw_q##n[S::NS > n ? S::QChunks : 1];       \
    if constexpr (S::NS > n) {                                  \
        fw_ring.p[n] = fw_p##n;                                 \
        fw_ring.q[n] = fw_q##n;                                 \
    }
#define FW_RING(S, name)   \
    Ring<S::NS> fw_ring;   \
    FW_STAGE(S, 0)         \
    FW_STAGE(S, 1)         \
    FW_STAGE(S, 2)         \
    FW_STAGE(S, 3)         \
    const Ring<S::NS> &name = fw_ring

// acc[i][j] (PI x QJ groups of 16 x 16) = the tile product over nseg segments
// of Kd steps; p(seg) / pb(seg) and q(seg) give the operands (pb: the second
// matrix of a dual P tile).
template <class S, class PF, class PBF, class QF>
__device__ __forceinline__ void tile_product(f4 (&acc)[S::PI][S::QJ], const Ring<S::NS> &ring,
                                             int wave, int lane, int Kd, int nseg, PF &&p,
                                             PBF &&pb, QF &&q) {
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
            for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.f;

    const int per = (Kd + kStepK - 1) / kStepK, steps = per * nseg;
    if (steps == 0) return;
    // The addresses of step st's stage.  `whole`: all of its 64 reduction steps
    // are there, which lets the DMA do without the test of each chunk; otherwise
    // chunks outside (and past the last step everything) read as zeros.
    struct Next {
        rsrc_t q, p, pb;
        int k, kd;
    };
    auto prepare = [&](int st) {
        const int seg = st >= per, k = (st - seg * per) * kStepK;   // nseg <= 2
        const int kd = st < steps ? Kd : 0;
        return Next{qs.rsrc(q(seg), k, kd), ps.rsrc(p(seg), k, kd),
                    S::DUAL ? ps.rsrc(pb(seg), k, kd) : ps.rsrc(p(seg), k, kd), k, kd};
    };
    // The same for whole stages, one after the other from `at` on: a few scalar
    // additions (the general form's fifty scalar instructions took a tenth of a
    // large tile's step and a quarter of a small one's).
    struct {
        const char *q, *p, *pb;
        int qn, pn;   // range lengths
    } at;
    auto start = [&](int seg, int k) {
        const Operand oq = q(seg), op = p(seg);
        const int64_t qk = S::QX ? (int64_t)k * oq.pitch : 2 * (int64_t)k;
        const int64_t pk = S::PX ? (int64_t)k * op.pitch : 2 * (int64_t)k;
        at.q = oq.base + qk;
        at.p = op.base + pk;
        at.pb = S::DUAL ? pb(seg).base + pk : nullptr;
        at.qn = S::QX ? kStepK * (int)oq.pitch - (int)oq.tail : oq.rows * (int)oq.pitch - 2 * k;
        at.pn = S::PX ? kStepK * (int)op.pitch - (int)op.tail : op.rows * (int)op.pitch - 2 * k;
    };
    const int64_t qstep = S::QX ? kStepK * (int64_t)q(0).pitch : 2 * kStepK;
    const int64_t pstep = S::PX ? kStepK * (int64_t)p(0).pitch : 2 * kStepK;
    auto advance = [&]() {
        const Next n{make_rsrc(at.q, at.qn), make_rsrc(at.p, at.pn),
                     make_rsrc(S::DUAL ? at.pb : at.p, at.pn), 0, 0};
        at.q += qstep;
        at.p += pstep;
        if (S::DUAL) at.pb += pstep;
        if (!S::QX) at.qn -= 2 * kStepK;
        if (!S::PX) at.pn -= 2 * kStepK;
        return n;
    };
    // DMA instruction i of a stage (buffer x): Q's, then P's
    constexpr int kDma = ps.kInstr + qs.kInstr;
    auto issue = [&](const Next &n, int x, int i, auto whole) {
        constexpr bool W = decltype(whole)::value;
        if (i < qs.kInstr) {
            qs.template issue<W>(n.q, ring.q[x], wave, n.k, n.kd, i);
        } else if (i < kDma) {
            const int j = i - qs.kInstr;
            ps.template issue<W>(S::DUAL && 2 * j >= ps.kInstr ? n.pb : n.p, ring.p[x], wave, n.k,
                                 n.kd, j);
        }
    };
    // The slice's operands.  P's are held twice, the next slice's read during
    // this one; each Q operand is replaced by the next slice's right behind its
    // MFMAs, S::QJ - 1 groups before it is needed.
    static_assert(S::PI <= S::QJ, "one P operand read behind each group");
    bf8 a[2][S::PI], b[S::QJ];
    auto group = [&](int s, int j) {
#pragma unroll
        for (int i = 0; i < S::PI; ++i)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[s][i], b[j], acc[i][j], 0, 0, 0);
    };
    // the next step's stage has landed (those behind it may be in flight) and
    // every wavefront is here
    constexpr int kBehind = (S::NS - 2) * kDma;
    static_assert(kBehind < 64, "vmcnt");
    auto sync = [&]() {
        __builtin_amdgcn_s_waitcnt(7 << 4 | kBehind % 16 | kBehind / 16 << 14);   // lgkmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // The MFMAs of the present slice (P operands a[x]), behind each group the
    // reads of slice s of buffer `from`.
    auto slice = [&](int x, int from, int s, auto &&behind) {
#pragma unroll
        for (int j = 0; j < S::QJ; ++j) {
            group(x, j);
            behind(j);
            b[j] = qr.read(ring.q[from], j, s);
            if (j < S::PI) a[x ^ 1][j] = pr.read(ring.p[from], j, s);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // One step (buffer x): two 32-step slices.  The rendezvous comes behind the
    // second slice's first group, when all of this buffer is in registers and its
    // MFMAs cover the wait: from there on the reads are of the next buffer and
    // this one is refilled with step st + NS's stage, a few DMA instructions
    // behind each group (a burst of them would fill the memory pipeline's queue
    // and hold up the MFMAs behind it).
    static_assert(kSlices == 2, "a step's slices alternate the P operands");
    auto step = [&](int st, int x, auto whole) {
        slice(0, x, 1, [](int) {});
        const Next n = decltype(whole)::value ? advance() : prepare(st + S::NS);
        constexpr int kPer = (kDma + S::QJ - 1) / S::QJ;
        slice(1, (x + 1) % S::NS, 0, [&](int j) {
            if (j == 0) sync();
#pragma unroll
            for (int d = 0; d < kPer; ++d) issue(n, x, j * kPer + d, whole);
        });
    };
    constexpr auto whole = std::true_type{};
    constexpr auto partial = std::false_type{};
#pragma unroll
    for (int x = 0; x < S::NS; ++x) {
        const Next n = prepare(x);
#pragma unroll
        for (int i = 0; i < kDma; ++i) issue(n, x, i, partial);
    }
    constexpr int kFirst = (S::NS - 1) * kDma;   // all but the first stage
    static_assert(kFirst < 64, "vmcnt");
    __builtin_amdgcn_s_waitcnt(7 << 4 | kFirst % 16 | kFirst / 16 << 14);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < S::PI; ++i) a[0][i] = pr.read(ring.p[0], i, 0);
#pragma unroll
    for (int j = 0; j < S::QJ; ++j) b[j] = qr.read(ring.q[0], j, 0);
    // NS steps per turn, so that each buffer keeps its name; step st issues stage
    // st + NS.  Per segment: turns that issue whole stages of it only, then turns
    // of any stages up to where the next segment's begin (the end).
    int st = 0;
    for (int seg = 0; seg < nseg; ++seg) {
        const int first = seg * per, full = first + Kd / kStepK;
        start(seg, (st + S::NS - first) * kStepK);
        for (; st + 2 * S::NS <= full; st += S::NS) {
#pragma unroll
            for (int x = 0; x < S::NS; ++x) step(st + x, x, whole);
        }
        const int until = seg + 1 < nseg ? first + per - S::NS : steps - S::NS + 1;
        for (; st < until; st += S::NS) {
#pragma unroll
            for (int x = 0; x < S::NS; ++x) step(st + x, x, partial);
        }
    }
#pragma unroll
    for (int x = 0; x + 1 < S::NS; ++x)
        if (st + x < steps) step(st + x, x, partial);
    // the last DMA has landed in every wavefront: the buffers are free
    __builtin_amdgcn_s_waitcnt(7 << 4);   // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// Hands the accumulators out by rows: emit(row, col, v, u, e) gets eight
// consecutive columns of one tile row (u: the same columns of a dual tile's
// second matrix), with e = fetch(row, col) issued for half of the tile at a
// time, ahead of its use.  Lanes of a wavefront cover whole rows of its part of
// the tile, so loads and stores are runs of 64 or 128 bytes (16 or more) of a
// row instead of the accumulators' 32.  The way there is LDS, 16 rows at a
// time, private to the wavefront, the 16-byte columns of a row moved by an xor
// of the row against bank conflicts.  lds: a buffer of the product, free again.
// APART: v[4..7] lie kOutCols / 2 columns behind v[0..3], so that each half of
// eight fp32 values is a run of whole cache lines over the lanes of a row.
template <class S> constexpr int kOutCols = S::BP / S::WP / (S::DUAL ? 2 : 1);

template <class S, bool APART = false, class Fetch, class Emit>
__device__ __forceinline__ void hand_out(const f4 (&acc)[S::PI][S::QJ], void *lds, int wave,
                                         int lane, Fetch &&fetch, Emit &&emit) {
    constexpr int CW = kOutCols<S>, LR = CW / 8;   // lanes a row
    static_assert(S::NW * (S::DUAL ? 2 : 1) * 16 * CW * 4 <= S::PChunks * 16, "LDS");
    static_assert(CW == 64 || CW == 32 || CW == 16, "4, 8 or 16 columns of 16 bytes");
    // rows a pass, passes per 16 rows (16 columns: half of the lanes have a row)
    constexpr int RP = LR < 4 ? 16 : 64 / LR, NP = 16 / RP;
    constexpr int HALF = S::QJ / 2, PG = S::DUAL ? S::PI / 2 : S::PI;
    static_assert(RP <= 16 && S::QJ % 2 == 0, "wave tile");
    const int wp = wave % S::WP, wq = wave / S::WP;
    f4 *mine = (f4 *)lds + wave * (S::DUAL ? 2 : 1) * 4 * CW;
    // 16-byte column c of row r: sixteen rows of one c, and a row's neighbours,
    // lie in different banks
    auto cell = [&](int r, int c) {
        return r * (CW / 4) + (c ^ (CW == 64 ? r : CW == 32 ? r >> 1 : r >> 2));
    };
    const int rr = lane / LR % RP, rc = (APART ? 4 : 8) * (lane % LR);
    const int rc2 = rc + (APART ? CW / 2 : 4);
    const bool idle = lane / LR >= RP;
    const int col = wp * CW + rc;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        decltype(fetch(0, 0)) e[HALF][NP];
#pragma unroll
        for (int j = 0; j < HALF; ++j)
#pragma unroll
            for (int p = 0; p < NP; ++p)
                if (!idle) e[j][p] = fetch(S::qrow(wq, h * HALF + j) + p * RP + rr, col);
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
            const int jj = h * HALF + j;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int i = 0; i < S::PI; ++i)
                mine[i / PG * 4 * CW + cell(lane & 15, 4 * (i % PG) + (lane >> 4))] = acc[i][jj];
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int lo = cell(p * RP + rr, rc / 4), hi = cell(p * RP + rr, rc2 / 4);
                float v[8], u[8];
                *(f4 *)v = mine[lo];
                *(f4 *)(v + 4) = mine[hi];
                if constexpr (S::DUAL) {
                    *(f4 *)u = mine[4 * CW + lo];
                    *(f4 *)(u + 4) = mine[4 * CW + hi];
                }
                if (!idle) emit(S::qrow(wq, jj) + p * RP + rr, col, v, u, e[j][p]);
            }
        }
    }
}

}  // namespace fw
