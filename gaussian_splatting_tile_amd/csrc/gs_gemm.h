// Matrix products on the CDNA4 matrix cores, the engine of the linear layer
// and of the orthogonalised update (internal; the public interface is
// include/gs.h).
//
//   out[q][p] = epilogue( sum_k P(p, k) Q(q, k) ),   p contiguous in memory
//
// One block computes a BP x BQ tile; its waves form a WP x WQ grid, each with
// a (BP / WP) x (BQ / WQ) tile of 16x16 accumulators in registers.  An operand
// is stored either with k contiguous ("rows") or with its own index contiguous
// ("columns", PT / QT): the second kind is kept as it is in LDS and transposed
// on the way to the registers by ds_read_b64_tr_b16, so a product and both its
// gradients read the same arrays, with no transposed copies.
//
// fp32 operands use the 16-bit matrix instructions too: x = x0 + x1 + x2 with
// each limb a bf16 (8 bits) of what the previous left, so three limbs hold all
// 24 bits, and x y = sum of x_i y_j.  With NL = 3 the six products i + j <= 2
// are formed, the rest is below 2^-25 of x y; with NL = 2 three, the rest below
// 2^-16 (for results that are rounded to 16 bits).  Six bf16 products run at
// 2.6 times the rate of the fp32 matrix instruction.  Small products are
// accumulated first.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gs.h"
#include "gs_numeric.h"

namespace gsi {
namespace gemm {

enum Kind { kBF16 = 0, kF16 = 1, kMX8 = 2 };          // what the matrix instructions multiply

struct Args {
    // operands: element (i, k) of P is p[i * ldp + k] (rows) or p[k * ldp + i]
    // (columns); limb l starts plane_p elements further, matrix b of a batch
    // batch_p elements
    const void *p, *q;
    int64_t ldp, ldq, plane_p, plane_q, batch_p, batch_q;
    int P, Q, K;
    int Pl, Ql;                                        // rows that may be read: P, Q, or padded up to a multiple of 8
    // staged loads only: element types (gs_dtype) and whether 8 consecutive
    // elements of a row may be read with 16-byte accesses
    int p_type, q_type, p_vec, q_vec;
    // kMX8: scale bytes, one per 32 k, and their row strides
    const uint8_t *ps, *qs;
    int64_t ldps, ldqs;
    int tiles_p, tiles_q;
    int k_split;                                       // k range of one split (a multiple of the k tile), grid.y splits
};

typedef float f4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));
typedef int i8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef short s4 __attribute__((ext_vector_type(4)));

template <int KIND> __device__ __forceinline__ f4 mfma32(i4 a, i4 b, f4 c)
{
    if constexpr (KIND == kF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

// 128 k of e4m3 values with one e8m0 scale per 32 (byte 0 of sa / sb).  Lane
// group g = lane / 16 holds k = 16 g .. 16 g + 15 in a.lo and 64 more in a.hi,
// and the scale of k = 32 g .. 32 g + 31.
__device__ __forceinline__ f4 mfma_mx(i4 alo, i4 ahi, int sa, i4 blo, i4 bhi, int sb, f4 c)
{
    const i8v a = __builtin_shufflevector(alo, ahi, 0, 1, 2, 3, 4, 5, 6, 7);
    const i8v b = __builtin_shufflevector(blo, bhi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, sa, 0, sb);
}

// ---- one operand's LDS tile -------------------------------------------------
// Rows: [BX][CH] chunks of 16 bytes, CH = 8 (64 values of 16 bits or 128 of 8)
// or 4; chunk c of row r sits at c ^ swz(r), so the 16 rows a fragment reads
// spread over all banks.  Columns: [BK][BX] with the chunks (8 rows) of line k
// at c ^ swz(k).  Direct loads write LDS in lane order, so the exchange is
// applied to the address a lane reads from.
template <int BX, int BK, bool T> struct Tile {
    static constexpr int kBytes = BX * BK * 2;
    static constexpr int kChunks = kBytes / 16;
    static constexpr int CH = T ? BX / 8 : BK / 8;     // chunks per line

    __device__ static __forceinline__ int swz(int line)
    {
        if constexpr (T) return (((line & 3) << 1) | (line & 8)) & (CH - 1);
        else if constexpr (CH == 8) return line & 7;
        else return (line >> 1) & 3;
    }
    // Fragment f (rows row0 + 16 f ..), k = 32 kk .. 32 kk + 31: lane group
    // g = lane / 16 holds row lane % 16, k = 32 kk + 8 g + (0..7).
    __device__ static __forceinline__ i4 frag(const char *lds, int row0, int f, int kk, int lane)
    {
        const int g = lane >> 4, r = lane & 15;
        if constexpr (!T) {
            const int x = row0 + f * 16 + r;
            return *reinterpret_cast<const i4 *>(lds + x * (CH * 16) + (((kk * 4 + g) ^ swz(x)) << 4));
        } else {
            // 16 lanes read 4 lines of k x 16 rows, and each gets its row's 4 k
            const int x = row0 + f * 16 + (r & 3) * 4;
            i4 v;
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int k = kk * 32 + g * 8 + j * 4 + (r >> 2);
                const char *a = lds + k * (CH * 16) + (((x >> 3) ^ swz(k)) << 4) + (x & 4) * 2;
                const int2 h = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                                            (__attribute__((address_space(3))) s4 *)a));
                v[2 * j] = h.x;
                v[2 * j + 1] = h.y;
            }
            return v;
        }
    }
};

// Direct loads of one operand: 16-byte pieces from global memory into LDS,
// no registers between.  The buffer's base is the tile's first element and
// moves with k; rows past the operand's end are read from its last row (their
// products are not stored); k past the end gets an offset beyond the buffer's
// size, which reads as zeros.
constexpr uint32_t kBufferBytes = 0x80000000u;          // of every buffer descriptor: offsets stay below

template <class TL, int THREADS, bool T, int ES> struct Direct {
    static constexpr int kLoads = TL::kChunks / THREADS;
    static_assert(TL::kChunks % THREADS == 0, "tile and block size");
    static constexpr int kPer = 16 / ES;                // elements per chunk
    static constexpr int kLineStep = THREADS / TL::CH;  // lines between a thread's loads
    static_assert(THREADS % TL::CH == 0 && kLineStep % 16 == 0, "a thread's chunks sit alike in their lines");
    uint32_t off[kLoads];                               // bytes from the tile's base
    int k0;                                             // first k of the thread's first chunk within the tile

    __device__ __forceinline__ void init(int x0, int X, int64_t ld, int tid)
    {
        const int line0 = tid / TL::CH, c = (tid % TL::CH) ^ TL::swz(line0);
        k0 = T ? line0 : c * kPer;
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int line = line0 + j * kLineStep;
            if constexpr (!T)
                off[j] = (uint32_t)min(line, X - 1 - x0) * (uint32_t)(ld * ES) + (uint32_t)c * 16u;
            else
                off[j] = (uint32_t)line * (uint32_t)(ld * ES) + (uint32_t)(min(c * kPer, X - kPer - x0) * ES);
        }
    }
    // left: k values from the tile's base to the end
    __device__ __forceinline__ void issue(const char *base, char *lds, int left, int wave) const
    {
        const __amdgpu_buffer_rsrc_t rsrc =
            __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(base), 0, (int)kBufferBytes, 0x00020000);
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int k = T ? k0 + j * kLineStep : k0;
            const uint32_t o = k < left ? off[j] : kBufferBytes;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(lds + (j * THREADS + wave * 64) * 16), 16, o, 0, 0, 0);
        }
    }
};

// Staged loads: any type, stride, alignment and size; converted (and split
// into limbs) in registers, then written to LDS.
template <class TL, int THREADS, bool T, int NL, int KIND> struct Staged {
    static constexpr int kLoads = TL::kChunks / THREADS;
    static_assert(TL::kChunks % THREADS == 0, "tile and block size");
    float v[kLoads][8];

    __device__ __forceinline__ void load(const void *p, int type, bool vec, const uint8_t *scales, int64_t lds_scale,
                                         int x0, int X, int64_t ld, int k0, int K, int tid)
    {
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int id = j * THREADS + tid;
            const int line = id / TL::CH, c = id % TL::CH;
            const int x = T ? x0 + c * 8 : x0 + line, k = T ? k0 + line : k0 + c * 8;
            int valid = T ? (k < K ? X - x : 0) : (x < X ? K - k : 0);
            valid = max(0, min(8, valid));
            const int64_t i = T ? (int64_t)k * ld + x : (int64_t)x * ld + k;
            if (type == GS_DTYPE_MXFP8) {
                const uint8_t *b = static_cast<const uint8_t *>(p);
                const float s = valid ? e8m0_value(scales[(int64_t)x * lds_scale + (k >> 5)]) : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) v[j][e] = e < valid ? e4m3_value(b[i + e]) * s : 0.0f;
            } else {
                load8(p, type, i, valid, vec, v[j]);
            }
        }
    }
    __device__ __forceinline__ void write(char *lds, int tid) const
    {
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int id = j * THREADS + tid;
            const int line = id / TL::CH, c = (id % TL::CH) ^ TL::swz(line);
            union { uint16_t h[8]; uint4 u; } w[NL];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                if constexpr (NL == 1) {
                    w[0].h[e] = KIND == kF16 ? __builtin_bit_cast(uint16_t, (_Float16)v[j][e])
                                             : __builtin_bit_cast(uint16_t, (__bf16)v[j][e]);
                } else {
                    uint16_t limb[NL];
                    split_limbs<NL>(v[j][e], limb);
#pragma unroll
                    for (int l = 0; l < NL; l++) w[l].h[e] = limb[l];
                }
            }
#pragma unroll
            for (int l = 0; l < NL; l++)
                *reinterpret_cast<uint4 *>(lds + l * TL::kBytes + (line * TL::CH + c) * 16) = w[l].u;
        }
    }
};

// Which tile a block takes.  Blocks go to the 8 dies in turn, so block b of
// nb becomes (b % 8)-th die's next tile of a contiguous eighth: the tiles of a
// die share operands in its L2.  Within that order, 8 tiles down q by all of p.
__device__ __forceinline__ void tile_of(int b, int tiles_p, int tiles_q, int &tp, int &tq)
{
    const int nb = tiles_p * tiles_q, die = b & 7, at = b >> 3, per = nb >> 3, more = nb & 7;
    const int t = die * per + min(die, more) + at;
    const int group = 8 * tiles_p, g = t / group, r = t - g * group;
    const int h = min(8, tiles_q - g * 8);
    tp = r / h;
    tq = g * 8 + r - tp * h;
}

// Orders a wave's own LDS writes and reads across its lanes (the lanes run in
// lockstep and LDS serves a wave in order: only the compiler has to be held).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// EPI::store(e, p, q, valid, v, batch, split): v[0 .. valid - 1] (LDS, 16-byte
// aligned) are the sums of p .. at q.
template <int KIND, int NL, int BK, int BP, int BQ, int WP, int WQ, bool PT, bool QT, bool STAGED, class EPI>
__global__ __launch_bounds__(WP *WQ * 64, NL == 3 && BP == 128 ? 1 : 2) void product_kernel(Args a, typename EPI::Args e)
{
    constexpr int kThreads = WP * WQ * 64;
    constexpr int FP = BP / WP / 16, FQ = BQ / WQ / 16, KK = BK / 32;
    constexpr int ES = KIND == kMX8 ? 1 : 2;
    constexpr int kStepK = KIND == kMX8 ? 2 * BK : BK;  // k per tile
    static_assert(KIND != kMX8 || (!PT && !QT && !STAGED && NL == 1 && BK == 64), "8-bit operands");
    using TP = Tile<BP, BK, PT>;
    using TQ = Tile<BQ, BK, QT>;
    constexpr int kStage = NL * (TP::kBytes + TQ::kBytes);
    // after the last product each wave turns its sums round in LDS, 16 q at a time
    constexpr int kTurnLd = FP * 16 + 4, kTurn = WP * WQ * 16 * kTurnLd * 4;
    __shared__ __align__(128) char lds0[kStage > kTurn ? kStage : kTurn];
    __shared__ __align__(128) char lds1[kStage];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave / WQ, wq = wave % WQ;
    int tp, tq;
    tile_of(blockIdx.x, a.tiles_p, a.tiles_q, tp, tq);
    const int p0 = tp * BP, q0 = tq * BQ;
    const int kbeg = blockIdx.y * a.k_split, kend = min(a.K, kbeg + a.k_split);
    const char *pb = static_cast<const char *>(a.p), *qb = static_cast<const char *>(a.q);

    f4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; i++)
#pragma unroll
        for (int j = 0; j < FQ; j++) acc[i][j] = f4{0, 0, 0, 0};

    auto compute = [&](const char *s, const int *sp, const int *sq) {
        if constexpr (KIND == kMX8) {
            i4 qf[FQ][2];
#pragma unroll
            for (int j = 0; j < FQ; j++)
#pragma unroll
                for (int h = 0; h < 2; h++) qf[j][h] = TQ::frag(s + TP::kBytes, wq * FQ * 16, j, h, lane);
#pragma unroll
            for (int i = 0; i < FP; i++) {
                const i4 lo = TP::frag(s, wp * FP * 16, i, 0, lane), hi = TP::frag(s, wp * FP * 16, i, 1, lane);
#pragma unroll
                for (int j = 0; j < FQ; j++) acc[i][j] = mfma_mx(lo, hi, sp[i], qf[j][0], qf[j][1], sq[j], acc[i][j]);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < KK; kk++) {
                if (kk) __builtin_amdgcn_sched_barrier(0);      // one slice's fragments in registers at a time
                i4 pf[NL][FP], qf[NL][FQ];
#pragma unroll
                for (int l = 0; l < NL; l++) {
#pragma unroll
                    for (int i = 0; i < FP; i++) pf[l][i] = TP::frag(s + l * TP::kBytes, wp * FP * 16, i, kk, lane);
#pragma unroll
                    for (int j = 0; j < FQ; j++)
                        qf[l][j] = TQ::frag(s + NL * TP::kBytes + l * TQ::kBytes, wq * FQ * 16, j, kk, lane);
                }
#pragma unroll
                for (int order = NL - 1; order >= 0; order--)
#pragma unroll
                    for (int l = 0; l <= order; l++)
#pragma unroll
                        for (int i = 0; i < FP; i++)
#pragma unroll
                            for (int j = 0; j < FQ; j++)
                                acc[i][j] = mfma32<KIND>(pf[l][i], qf[order - l][j], acc[i][j]);
            }
        }
    };

    if constexpr (!STAGED) {
        pb += (int64_t)blockIdx.z * a.batch_p * ES;
        qb += (int64_t)blockIdx.z * a.batch_q * ES;
        Direct<TP, kThreads, PT, ES> dp;
        Direct<TQ, kThreads, QT, ES> dq;
        dp.init(p0, a.Pl, a.ldp, tid);
        dq.init(q0, a.Ql, a.ldq, tid);
        // first elements of the tile at k = kbeg, and the step to the next
        pb += (PT ? (int64_t)kbeg * a.ldp + p0 : (int64_t)p0 * a.ldp + kbeg) * ES;
        qb += (QT ? (int64_t)kbeg * a.ldq + q0 : (int64_t)q0 * a.ldq + kbeg) * ES;
        const int64_t step_p = (PT ? a.ldp : 1) * (int64_t)kStepK * ES, step_q = (QT ? a.ldq : 1) * (int64_t)kStepK * ES;
        const int nt = (kend - kbeg + kStepK - 1) / kStepK;

        // scale bytes of a lane's rows, by buffers that start at the tile's rows
        constexpr int NS = KIND == kMX8 ? 1 : 0;
        int sp0[NS ? FP : 1], sq0[NS ? FQ : 1], sp1[NS ? FP : 1], sq1[NS ? FQ : 1];
        uint32_t sp_off[NS ? FP : 1], sq_off[NS ? FQ : 1];
        if constexpr (NS) {
#pragma unroll
            for (int i = 0; i < FP; i++)
                sp_off[i] = (uint32_t)min((wp * FP + i) * 16 + (lane & 15), a.P - 1 - p0) * (uint32_t)a.ldps;
#pragma unroll
            for (int j = 0; j < FQ; j++)
                sq_off[j] = (uint32_t)min((wq * FQ + j) * 16 + (lane & 15), a.Q - 1 - q0) * (uint32_t)a.ldqs;
        }
        auto scales = [&](int t, int *sp, int *sq) {
            if constexpr (NS) {
                const __amdgpu_buffer_rsrc_t rp = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<uint8_t *>(a.ps + p0 * a.ldps), 0, (int)kBufferBytes, 0x00020000);
                const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
                    const_cast<uint8_t *>(a.qs + q0 * a.ldqs), 0, (int)kBufferBytes, 0x00020000);
                // blocks past the end of k: their values are 0, any finite scale does
                const int b = kbeg / 32 + t * 4 + (lane >> 4);
                const uint32_t bo = (uint32_t)min(b, (a.K >> 5) - 1);
                const bool in = b < (a.K >> 5);
#pragma unroll
                for (int i = 0; i < FP; i++) {
                    const int v = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rp, sp_off[i] + bo, 0, 0);
                    sp[i] = in ? v : 127;
                }
#pragma unroll
                for (int j = 0; j < FQ; j++) {
                    const int v = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rq, sq_off[j] + bo, 0, 0);
                    sq[j] = in ? v : 127;
                }
            }
        };
        auto issue = [&](int t, char *s) {
            const int left = kend - kbeg - t * kStepK;
            const char *pt = pb + t * step_p, *qt = qb + t * step_q;
#pragma unroll
            for (int l = 0; l < NL; l++) {
                dp.issue(pt + l * a.plane_p * ES, s + l * TP::kBytes, left, wave);
                dq.issue(qt + l * a.plane_q * ES, s + NL * TP::kBytes + l * TQ::kBytes, left, wave);
            }
        };
        // two LDS stages: while one is multiplied the next is on its way
        issue(0, lds0);
        scales(0, sp0, sq0);
        int t = 0;
        for (; t + 1 < nt; t += 2) {
            __syncthreads();                            // stage 0 has landed, stage 1 is free
            issue(t + 1, lds1);
            scales(t + 1, sp1, sq1);
            compute(lds0, sp0, sq0);
            __syncthreads();
            issue(t + 2, lds0);                         // zeros when there is no such tile
            scales(t + 2, sp0, sq0);
            compute(lds1, sp1, sq1);
        }
        if (t < nt) {
            __syncthreads();
            compute(lds0, sp0, sq0);
        }
    } else {
        Staged<TP, kThreads, PT, NL, KIND> sp;
        Staged<TQ, kThreads, QT, NL, KIND> sq;
        pb += (int64_t)blockIdx.z * a.batch_p * dtype_bytes(a.p_type);
        qb += (int64_t)blockIdx.z * a.batch_q * dtype_bytes(a.q_type);
        auto load = [&](int k0) {
            sp.load(pb, a.p_type, a.p_vec, a.ps, a.ldps, p0, a.P, a.ldp, k0, kend, tid);
            sq.load(qb, a.q_type, a.q_vec, a.qs, a.ldqs, q0, a.Q, a.ldq, k0, kend, tid);
        };
        load(kbeg);
        for (int k0 = kbeg; k0 < kend; k0 += kStepK) {
            char *s = ((k0 - kbeg) / kStepK) & 1 ? lds1 : lds0;
            sp.write(s, tid);
            sq.write(s + NL * TP::kBytes, tid);
            __syncthreads();                            // also: every wave is done with this stage's last use
            if (k0 + kStepK < kend) load(k0 + kStepK);
            compute(s, nullptr, nullptr);
        }
    }

    // sums to the epilogue, 8 consecutive p at a time; a lane's accumulator holds
    // p = 16 i + 4 g + (0..3) at q = 16 j + r
    __syncthreads();
    float *turn = reinterpret_cast<float *>(lds0) + wave * (16 * kTurnLd);
    constexpr int kLanesP = FP * 2, kRowsQ = 64 / kLanesP;      // lanes along p, q rows at a time
#pragma unroll
    for (int j = 0; j < FQ; j++) {
#pragma unroll
        for (int i = 0; i < FP; i++)
            *reinterpret_cast<f4 *>(turn + (lane & 15) * kTurnLd + i * 16 + (lane >> 4) * 4) = acc[i][j];
        wave_fence();
#pragma unroll 1
        for (int h = 0; h < 16; h += kRowsQ) {
            const int qr = h + lane / kLanesP, pr = lane % kLanesP * 8;
            const int p = p0 + wp * FP * 16 + pr, q = q0 + (wq * FQ + j) * 16 + qr;
            if (p >= a.P || q >= a.Q) continue;
            EPI::store(e, p, q, min(8, a.P - p), turn + qr * kTurnLd + pr, blockIdx.z, blockIdx.y);
        }
        wave_fence();
    }
}

inline bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Whether an operand may be loaded directly: 16-byte pieces must not cross
// its edges and their offsets within a tile must fit 32 bits.  extent: k (rows)
// or the operand's own count (columns), padded where the array is.
inline bool direct_ok(const void *p, int es, int64_t ld, int64_t extent)
{
    const int per = 16 / es;
    return al16(p) && ld % per == 0 && extent % per == 0 && ld * es < (1 << 23);
}

template <int KIND, int NL, int BK, int BP, int BQ, int WP, int WQ, bool PT, bool QT, bool STAGED, class EPI>
hipError_t launch(Args a, const typename EPI::Args &e, int splits, int batch, hipStream_t s)
{
    constexpr int kStepK = KIND == kMX8 ? 2 * BK : BK;
    a.tiles_p = (a.P + BP - 1) / BP;
    a.tiles_q = (a.Q + BQ - 1) / BQ;
    const int nt = (a.K + kStepK - 1) / kStepK, per = (nt + splits - 1) / splits;
    if ((nt + per - 1) / per != splits) return hipErrorInvalidValue;       // every split has at least one tile
    a.k_split = per * kStepK;
    const dim3 grid((unsigned)(a.tiles_p * a.tiles_q), (unsigned)splits, (unsigned)batch);
    product_kernel<KIND, NL, BK, BP, BQ, WP, WQ, PT, QT, STAGED, EPI><<<grid, WP * WQ * 64, 0, s>>>(a, e);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace gsi
