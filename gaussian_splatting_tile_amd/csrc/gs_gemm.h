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
//
// Measured on large squares (8192): 1.32 PFLOP/s of bf16 by 256 tiles, where the
// card's power limit holds the clock near 1.8 GHz, and 2.2 PFLOP/s of 8-bit
// values; fp32 4096 x 4096 x 1024 in 192 us (179 TFLOP/s).  With a short k the
// epilogue's writes and arithmetic add to that: one block of 256 x 256 fills a
// CU's registers, and pairs of smaller blocks, which could cover for each other,
// were no faster (4096 x 16384 x 1024 with GELU and z: 173 us by 256 x 256, 174 to 195
// by 256 x 128 and 128 x 128 in every wave layout, with and without priorities).
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
    int p_type, q_type;                                // staged loads only: element types (gs_dtype)
    // kMX8: scale bytes, one per 32 k, and their row strides
    const uint8_t *ps, *qs;
    int64_t ldps, ldqs;
    int tiles_p, tiles_q;
    int k_split;                                       // k range of one split (a multiple of the k tile), grid.y splits
    int symmetric;                                     // the result is: only tiles with p tile <= q tile are formed
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

// The descriptor's words: base, no stride, size, 32-bit raw data.
__device__ __forceinline__ i4 buffer_at(const void *base)
{
    const uint64_t b = (uint64_t)(uintptr_t)base;
    return i4{(int)__builtin_amdgcn_readfirstlane((int)b), (int)__builtin_amdgcn_readfirstlane((int)(b >> 32) & 0xFFFF),
              (int)kBufferBytes, 0x00020000};
}
// 64 lanes' pieces of 16 bytes, or bytes widened to words, to consecutive
// places from `lds` (the same in all lanes) on.  Written as assembly because the
// compiler cannot tell which stage a transposing LDS read touches and would
// wait for every load in flight before each; the loads have no result
// registers, and stage_barrier waits for them.  (m0 cannot be named as
// clobbered: it is reserved.  Nothing else in these kernels uses it.)
__device__ __forceinline__ void load_lds16(i4 buffer, uint32_t off, const char *lds)
{
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(buffer)
                 : "memory");
}
__device__ __forceinline__ void load_lds1(i4 buffer, uint32_t off, const char *lds)
{
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_ubyte %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(buffer)
                 : "memory");
}

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
        const i4 buffer = buffer_at(base);
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int k = T ? k0 + j * kLineStep : k0;
            const uint32_t o = k < left ? off[j] : kBufferBytes;
            load_lds16(buffer, o, lds + (j * THREADS + wave * 64) * 16);
        }
    }
};

// Scale bytes of a kMX8 tile: 4 blocks of 32 k per row, each widened to a word
// in LDS, [BX][4].  Blocks past the end of k read as 0, a finite scale.
template <int BX, int THREADS> struct Scales {
    static constexpr int kLoads = BX * 4 >= THREADS ? BX * 4 / THREADS : 1;
    uint32_t off[kLoads];

    __device__ __forceinline__ void init(int x0, int X, int64_t ld, int tid)
    {
#pragma unroll
        for (int j = 0; j < kLoads; j++)
            off[j] = (uint32_t)min((j * THREADS + tid) >> 2, X - 1 - x0) * (uint32_t)ld + (tid & 3);
    }
    __device__ __forceinline__ void issue(const uint8_t *base, char *lds, int blocks, int wave) const
    {
        const i4 buffer = buffer_at(base);
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const uint32_t o = (int)(threadIdx.x & 3) < blocks ? off[j] : kBufferBytes;
            load_lds1(buffer, o, lds + (j * THREADS + wave * 64) * 4);
        }
    }
};

// Staged loads: any type, stride, alignment and size.  A chunk waits in
// registers as it was loaded, so that the loads of the next tile are under way
// while a tile is multiplied, and is converted (and split into limbs) on its
// way to LDS.
template <class TL, int THREADS, bool T, int NL, int KIND> struct Staged {
    static constexpr int kLoads = TL::kChunks / THREADS;
    static_assert(TL::kChunks % THREADS == 0, "tile and block size");
    static constexpr int kWords = NL > 1 ? 8 : 4;
    uint32_t raw[kLoads][kWords];                       // 8 values each: fp32, or in pairs, or (MXFP8) in fours
    float scale[kLoads];                                // MXFP8

    __device__ __forceinline__ void load(const void *p, int type, const uint8_t *scales, int64_t lds_scale, int x0, int X, int64_t ld,
                                         int k0, int K, int tid)
    {
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int id = j * THREADS + tid;
            const int line = id / TL::CH, c = id % TL::CH;
            const int x = T ? x0 + c * 8 : x0 + line, k = T ? k0 + line : k0 + c * 8;
            int valid = T ? (k < K ? X - x : 0) : (x < X ? K - k : 0);
            valid = max(0, min(8, valid));
            const int64_t i = T ? (int64_t)k * ld + x : (int64_t)x * ld + k;
#pragma unroll
            for (int e = 0; e < kWords; e++) raw[j][e] = 0;
            if constexpr (NL > 1) {                     // fp32
                const uint32_t *f = static_cast<const uint32_t *>(p) + i;
                if (valid == 8) {
                    const auto v = *reinterpret_cast<const Vec<uint32_t, 8> *>(f);
#pragma unroll
                    for (int e = 0; e < 8; e++) raw[j][e] = v.v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (e < valid) raw[j][e] = f[e];
                }
            } else if (type == GS_DTYPE_MXFP8) {        // k is a multiple of 32
                if (valid == 8) {
                    const auto v = *reinterpret_cast<const Vec<uint8_t, 8> *>(static_cast<const uint8_t *>(p) + i);
                    const auto u = __builtin_bit_cast(uint2, v);
                    raw[j][0] = u.x;
                    raw[j][1] = u.y;
                }
                scale[j] = valid ? e8m0_value(scales[(int64_t)x * lds_scale + (k >> 5)]) : 0.0f;
            } else {
                const uint16_t *h = static_cast<const uint16_t *>(p) + i;
                if (valid == 8) {
                    const auto v = *reinterpret_cast<const Vec<uint16_t, 8> *>(h);
                    const auto u = __builtin_bit_cast(uint4, v);
                    raw[j][0] = u.x;
                    raw[j][1] = u.y;
                    raw[j][2] = u.z;
                    raw[j][3] = u.w;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (e < valid) raw[j][e >> 1] |= (uint32_t)h[e] << (16 * (e & 1));
                }
            }
        }
    }
    __device__ __forceinline__ void write(char *lds, int type, int tid) const
    {
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const int id = j * THREADS + tid;
            const int line = id / TL::CH, c = (id % TL::CH) ^ TL::swz(line);
            Vec<uint16_t, 8> w[NL];
            if constexpr (NL == 1) {
                w[0] = __builtin_bit_cast(Vec<uint16_t, 8>, make_uint4(raw[j][0], raw[j][1], raw[j][2], raw[j][3]));
                if (type == GS_DTYPE_MXFP8) {
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        w[0].v[e] = __builtin_bit_cast(uint16_t, (__bf16)(e4m3_value((uint8_t)(raw[j][e >> 2] >> (8 * (e & 3)))) * scale[j]));
                }
            } else {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; e++) v[e] = __uint_as_float(raw[j][e]);
                split_all<NL, 8>(v, w);
            }
#pragma unroll
            for (int l = 0; l < NL; l++)
                *reinterpret_cast<uint4 *>(lds + l * TL::kBytes + (line * TL::CH + c) * 16) = __builtin_bit_cast(uint4, w[l]);
        }
    }
};

// Which tile and split of k a block takes.  Blocks go to the 8 dies in turn, so
// block b of nb becomes the (b % 8)-th die's next item of a contiguous eighth of
// the list of matrices of a batch, splits and tiles: a die's blocks share
// operands in its L2 (with splits, only a range of k of them: half a 1024 x
// 1024 x 4096 product of two limbs in 7 splits takes 19.5 us, 28.8 us where every
// die read all k).
__device__ __forceinline__ int die_order(int b, int nb)
{
    const int die = b & 7, at = b >> 3, per = nb >> 3, more = nb & 7;
    return die * per + min(die, more) + at;
}
// The t-th tile: 8 tiles down q by all of p, and so on.
__device__ __forceinline__ void tile_of(int t, int tiles_p, int tiles_q, int &tp, int &tq)
{
    const int group = 8 * tiles_p, g = t / group, r = t - g * group;
    const int h = min(8, tiles_q - g * 8);
    tp = r / h;
    tq = g * 8 + r - tp * h;
}
// The t-th tile of the triangle tp <= tq, row by row.
__device__ __forceinline__ void triangle_of(int t, int &tp, int &tq)
{
    tq = (int)((sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
    while ((tq + 1) * (tq + 2) / 2 <= t) tq++;
    while (tq * (tq + 1) / 2 > t) tq--;
    tp = t - tq * (tq + 1) / 2;
}

// Waits until at most LEFT of the wave's loads are outstanding and its LDS
// reads are done, then for the other waves.
template <int LEFT> __device__ __forceinline__ void stage_barrier()
{
    static_assert(LEFT >= 0 && LEFT < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
}

// The same for LDS reads alone.
__device__ __forceinline__ void slice_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Orders a wave's own LDS writes and reads across its lanes (the lanes run in
// lockstep and LDS serves a wave in order: only the compiler has to be held).
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Fragments along p that the waves turn at once within `bytes` of LDS, [16 q][16
// p each]; the 16-byte chunks of row q at c ^ (q & 7), so that neither the
// writes (16 rows of a chunk) nor the reads (a row) meet in a bank.
constexpr int turn_part(int fp, int waves, int bytes)
{
    while (fp > 1 && waves * 16 * fp * 16 * 4 > bytes) fp /= 2;
    return fp;
}
template <int PART> __device__ __forceinline__ int turn_at(int q, int p)
{
    return q * (PART * 16) + (((p >> 2) ^ (q & 7 & (PART * 4 - 1))) << 2) + (p & 3);
}

// Waves on a SIMD that the register budget has to leave room for: of two blocks
// where the LDS holds two.
constexpr int waves_per_simd(int waves, int lds) { return (2 * lds <= 160 * 1024 ? 2 : 1) * waves / 4; }

// The epilogue takes 8 sums of consecutive p at a time, EPI::store8(e, p, q, v,
// part, ahead, batch, split), which leaves the final values in v and finds in
// `part` and `ahead` what EPI::part(e, p, ..) and EPI::look_ahead(e, p, q, ..)
// loaded for it; at the end of p single ones, EPI::store1.  A tile that also
// stands for its transpose (EPI::kMirror) hands those on to EPI::store_mirror.
template <int KIND, int NL, int NS, int BK, int BP, int BQ, int WP, int WQ, bool PT, bool QT, bool STAGED, bool PING, class EPI>
__global__ __launch_bounds__(WP *WQ * 64, waves_per_simd(WP * WQ, NS * NL * (BP + BQ) * BK * 2)) void product_kernel(Args a, typename EPI::Args e)
{
    constexpr int kThreads = WP * WQ * 64;
    constexpr int FP = BP / WP / 16, FQ = BQ / WQ / 16, KK = BK / 32;
    constexpr int ES = KIND == kMX8 ? 1 : 2;
    constexpr int kStepK = KIND == kMX8 ? 2 * BK : BK;  // k per tile
    static_assert(NS == 2 || NS == 3, "stages");
    static_assert(!PING || (WP * WQ == 8 && !STAGED), "two waves on every SIMD");
    static_assert(KIND != kMX8 || (!PT && !QT && !STAGED && NL == 1 && BK == 64), "8-bit operands");
    using TP = Tile<BP, BK, PT>;
    using TQ = Tile<BQ, BK, QT>;
    constexpr int kScaleAt = NL * (TP::kBytes + TQ::kBytes);
    constexpr int kStage = kScaleAt + (KIND == kMX8 ? (BP + BQ) * 16 : 0);
    // after the last product each wave turns its sums round in a stage's place,
    // 16 q by as many p as fit there at a time
    constexpr int kPart = turn_part(FP, WP * WQ, kStage);
    __shared__ __align__(128) char lds0[kStage];
    __shared__ __align__(128) char lds1[kStage];
    __shared__ __align__(128) char lds2[NS > 2 ? kStage : 16];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wp = wave / WQ, wq = wave % WQ;
    int tp, tq;
    const int per_matrix = gridDim.x * gridDim.y;
    const int item = die_order(blockIdx.z * per_matrix + blockIdx.y * gridDim.x + blockIdx.x, per_matrix * gridDim.z);
    const int batch = item / per_matrix, split = item % per_matrix / gridDim.x, tile = item % gridDim.x;
    if (a.symmetric)
        triangle_of(tile, tp, tq);
    else
        tile_of(tile, a.tiles_p, a.tiles_q, tp, tq);
    const int p0 = tp * BP, q0 = tq * BQ;
    const int kbeg = split * a.k_split, kend = min(a.K, kbeg + a.k_split);
    const char *pb = static_cast<const char *>(a.p), *qb = static_cast<const char *>(a.q);

    f4 acc[FP][FQ];
#pragma unroll
    for (int i = 0; i < FP; i++)
#pragma unroll
        for (int j = 0; j < FQ; j++) acc[i][j] = f4{0, 0, 0, 0};

    // A tile's products in slices: 32 k each, or (kMX8, 128 k at once) half of
    // the P side each.  fetch() reads a slice's fragments, multiply() uses them.
    constexpr bool MX = KIND == kMX8;
    constexpr int kSlices = MX ? (FP > 1 ? 2 : 1) : KK, kHalf = MX ? FP / kSlices : FP;
    i4 pf[MX ? 2 : NL][kHalf], qf[MX ? 2 : NL][FQ];
    int sp[MX ? kHalf : 1], sq[MX ? FQ : 1];
    auto fetch = [&](const char *s, int slice) {
        const char *t = s + NL * TP::kBytes;
        if constexpr (MX) {
            const int *cp = reinterpret_cast<const int *>(s + kScaleAt) + (wp * FP * 16 + (lane & 15)) * 4 + (lane >> 4);
            const int *cq = reinterpret_cast<const int *>(s + kScaleAt + BP * 16) + (wq * FQ * 16 + (lane & 15)) * 4 + (lane >> 4);
            if (slice == 0) {
#pragma unroll
                for (int j = 0; j < FQ; j++) {
                    sq[j] = cq[j * 64];
#pragma unroll
                    for (int h = 0; h < 2; h++) qf[h][j] = TQ::frag(t, wq * FQ * 16, j, h, lane);
                }
            }
#pragma unroll
            for (int i = 0; i < kHalf; i++) {
                sp[i] = cp[(slice * kHalf + i) * 64];
#pragma unroll
                for (int h = 0; h < 2; h++) pf[h][i] = TP::frag(s, wp * FP * 16, slice * kHalf + i, h, lane);
            }
        } else {
#pragma unroll
            for (int l = 0; l < NL; l++) {
#pragma unroll
                for (int i = 0; i < FP; i++) pf[l][i] = TP::frag(s + l * TP::kBytes, wp * FP * 16, i, slice, lane);
#pragma unroll
                for (int j = 0; j < FQ; j++) qf[l][j] = TQ::frag(t + l * TQ::kBytes, wq * FQ * 16, j, slice, lane);
            }
        }
    };
    auto multiply = [&](int slice) {
        if constexpr (MX) {
#pragma unroll
            for (int i = 0; i < kHalf; i++)
#pragma unroll
                for (int j = 0; j < FQ; j++)
                    acc[slice * kHalf + i][j] = mfma_mx(pf[0][i], pf[1][i], sp[i], qf[0][j], qf[1][j], sq[j], acc[slice * kHalf + i][j]);
        } else {
#pragma unroll
            for (int order = NL - 1; order >= 0; order--)
#pragma unroll
                for (int l = 0; l <= order; l++)
#pragma unroll
                    for (int i = 0; i < FP; i++)
#pragma unroll
                        for (int j = 0; j < FQ; j++) acc[i][j] = mfma32<KIND>(pf[l][i], qf[order - l][j], acc[i][j]);
        }
    };

    if constexpr (!STAGED) {
        pb += (int64_t)batch * a.batch_p * ES;
        qb += (int64_t)batch * a.batch_q * ES;
        Direct<TP, kThreads, PT, ES> dp;
        Direct<TQ, kThreads, QT, ES> dq;
        Scales<BP, kThreads> cp;
        Scales<BQ, kThreads> cq;
        dp.init(p0, a.Pl, a.ldp, tid);
        dq.init(q0, a.Ql, a.ldq, tid);
        if constexpr (KIND == kMX8) {
            static_assert(BP * 4 % kThreads == 0 && BQ * 4 % kThreads == 0, "tile and block size");
            cp.init(p0, a.P, a.ldps, tid);
            cq.init(q0, a.Q, a.ldqs, tid);
        }
        constexpr int kLoadsPerTile = NL * (dp.kLoads + dq.kLoads) + (KIND == kMX8 ? cp.kLoads + cq.kLoads : 0);
        // first elements of the tile at k = kbeg, and the step to the next
        pb += (PT ? (int64_t)kbeg * a.ldp + p0 : (int64_t)p0 * a.ldp + kbeg) * ES;
        qb += (QT ? (int64_t)kbeg * a.ldq + q0 : (int64_t)q0 * a.ldq + kbeg) * ES;
        const int64_t step_p = (PT ? a.ldp : 1) * (int64_t)kStepK * ES, step_q = (QT ? a.ldq : 1) * (int64_t)kStepK * ES;
        const int nt = (kend - kbeg + kStepK - 1) / kStepK;

        auto issue = [&](int t, char *s) {
            const int left = kend - kbeg - t * kStepK;
            const char *pt = pb + t * step_p, *qt = qb + t * step_q;
#pragma unroll
            for (int l = 0; l < NL; l++) {
                dp.issue(pt + l * a.plane_p * ES, s + l * TP::kBytes, left, wave);
                dq.issue(qt + l * a.plane_q * ES, s + NL * TP::kBytes + l * TQ::kBytes, left, wave);
            }
            if constexpr (KIND == kMX8) {
                const int b = kbeg / 32 + t * 4, blocks = (a.K >> 5) - b;
                cp.issue(a.ps + (int64_t)p0 * a.ldps + b, s + kScaleAt, blocks, wave);
                cq.issue(a.qs + (int64_t)q0 * a.ldqs + b, s + kScaleAt + BP * 16, blocks, wave);
            }
        };
        // NS stages in LDS: tile t is multiplied while the next NS - 1 are on
        // their way.  A wave's loads land in order, so waiting until only the
        // later tiles' are outstanding leaves tile t complete; the barrier then
        // makes it so for every wave, and frees the stage of tile t - 1.  Every
        // tile counts the same loads: past the end they read zeros.
        //
        // PING: the block's two halves of waves (one wave of each on every SIMD)
        // work half a slice apart, so that one half's LDS reads run beside the
        // other's matrix instructions.  The 256 tile of 16-bit operands gains 1 to
        // 5 per cent (1024 x 16384 x 4096 110.5 -> 108 us); with 128 tiles or 8-bit
        // operands it made no difference and is left off.  A half
        // reads a tile while the other half's pieces must already be there, so
        // each waits for its own one phase early.
        constexpr int kAhead = kLoadsPerTile * (NS - 2);
        auto turn_stage = [&](int t, char *now, char *next) {
            if constexpr (!PING) stage_barrier<kAhead>();
#pragma unroll
            for (int c = 0; c < kSlices; c++) {
                if (!PING && c) __builtin_amdgcn_sched_barrier(0);      // one slice's fragments in registers at a time
                fetch(now, c);
                // the next tile's loads start once the first fragments are on
                // their way: the wave's LDS reads do not queue behind them
                if (c == 0) issue(t + NS - 1, next);
                if constexpr (PING) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (c == kSlices - 1) stage_barrier<kAhead>();
                    else slice_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                }
                multiply(c);
                if constexpr (PING) {
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        char *const stage[3] = {lds0, lds1, lds2};
#pragma unroll
        for (int t = 0; t < NS - 1; t++) issue(t, stage[t]);
        const bool late = wave >= WP * WQ / 2;
        if constexpr (PING) {
            stage_barrier<kAhead>();
            if (late) __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        }
        int t = 0;
        for (; t + NS <= nt; t += NS)
#pragma unroll
            for (int i = 0; i < NS; i++) turn_stage(t + i, stage[i], stage[(i + NS - 1) % NS]);
        if (t < nt) turn_stage(t, stage[0], stage[NS - 1]);
        if (NS > 2 && t + 1 < nt) turn_stage(t + 1, stage[1], stage[0]);
        if (PING && !late) __builtin_amdgcn_s_barrier();
    } else {
        // a stage's next tile but one is on its way while it is multiplied
        constexpr int kSets = 2;
        Staged<TP, kThreads, PT, NL, KIND> sp[kSets];
        Staged<TQ, kThreads, QT, NL, KIND> sq[kSets];
        pb += (int64_t)batch * a.batch_p * dtype_bytes(a.p_type);
        qb += (int64_t)batch * a.batch_q * dtype_bytes(a.q_type);
        auto load = [&](int k0, int set) {
            if (k0 >= kend) return;
            sp[set].load(pb, a.p_type, a.ps, a.ldps, p0, a.P, a.ldp, k0, kend, tid);
            sq[set].load(qb, a.q_type, a.qs, a.ldqs, q0, a.Q, a.ldq, k0, kend, tid);
        };
#pragma unroll
        for (int i = 0; i < kSets; i++) load(kbeg + i * kStepK, i);
        for (int k0 = kbeg; k0 < kend; k0 += kSets * kStepK) {
#pragma unroll
            for (int i = 0; i < kSets; i++) {
                if (k0 + i * kStepK >= kend) continue;
                char *s = i ? lds1 : lds0;
                sp[i].write(s, a.p_type, tid);
                sq[i].write(s + NL * TP::kBytes, a.q_type, tid);
                __syncthreads();                        // also: every wave is done with this stage's last use
                load(k0 + (i + kSets) * kStepK, i);
#pragma unroll
                for (int c = 0; c < kSlices; c++) {
                    fetch(s, c);
                    multiply(c);
                }
            }
        }
    }

    // sums to the epilogue, 8 consecutive p at a time; a lane's accumulator holds
    // p = 16 i + 4 g + (0..3) at q = 16 j + r
    stage_barrier<0>();
    float *turn = reinterpret_cast<float *>(lds0) + wave * (256 * kPart);
    constexpr int kLanesP = kPart * 2, kRowsQ = 64 / kLanesP;   // lanes along p, q rows at a time
    constexpr int kParts = FQ * (FP / kPart), kIts = kRowsQ < 16 ? 16 / kRowsQ : 1;
    const bool mirror = EPI::kMirror && a.symmetric && tp != tq;
    // what the epilogue reads for a part is on its way while its sums turn
    typename EPI::Ahead ahead[kIts];
    auto part_p = [&](int u) { return p0 + (wp * FP + u % (FP / kPart) * kPart) * 16; };
    auto part_q = [&](int u) { return q0 + (wq * FQ + u / (FP / kPart)) * 16; };
    auto look_ahead = [&](int u) {
#pragma unroll
        for (int it = 0; it < kIts; it++) {
            const int qr = it * kRowsQ + lane / kLanesP, p = part_p(u) + lane % kLanesP * 8, q = part_q(u) + qr;
            if (qr < 16 && q < a.Q && p + 8 <= a.P) EPI::look_ahead(e, p, q, batch, ahead[it]);
        }
    };
#pragma unroll 1
    for (int u = 0; u < kParts; u++) {
        typename EPI::Part part;
        look_ahead(u);
        const int part_at = part_p(u) + lane % kLanesP * 8;
        if (part_at + 8 <= a.P) EPI::part(e, part_at, part);
        // accumulators have no run-time index: one of kParts branches
#pragma unroll
        for (int c = 0; c < kParts; c++)
            if (u == c) {
#pragma unroll
                for (int i = 0; i < kPart; i++)
                    *reinterpret_cast<f4 *>(turn + turn_at<kPart>(lane & 15, i * 16 + (lane >> 4) * 4)) =
                        acc[c % (FP / kPart) * kPart + i][c / (FP / kPart)];
            }
        wave_fence();
        const int pb0 = part_p(u), qb0 = part_q(u);
#pragma unroll
        for (int it = 0; it < kIts; it++) {
            const int qr = it * kRowsQ + lane / kLanesP, pr = lane % kLanesP * 8;
            const int p = pb0 + pr, q = qb0 + qr;
            if (qr >= 16 || q >= a.Q) continue;     // two lanes a row would reach 32 rows
            if (p + 8 <= a.P) {
                f4 *const lo = reinterpret_cast<f4 *>(turn + turn_at<kPart>(qr, pr));
                f4 *const hi = reinterpret_cast<f4 *>(turn + turn_at<kPart>(qr, pr + 4));
                float v[8] = {(*lo)[0], (*lo)[1], (*lo)[2], (*lo)[3], (*hi)[0], (*hi)[1], (*hi)[2], (*hi)[3]};
                EPI::store8(e, p, q, v, part, ahead[it], batch, split);
                if (mirror) {
                    *lo = f4{v[0], v[1], v[2], v[3]};
                    *hi = f4{v[4], v[5], v[6], v[7]};
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < a.P - p; i++) EPI::store1(e, p + i, q, turn[turn_at<kPart>(qr, pr + i)], batch, split);
            }
        }
        if constexpr (EPI::kMirror) {
            if (mirror) {               // the transposed tile: 8 q of a p to a lane
                wave_fence();
#pragma unroll 1
                for (int x = lane; x < 32 * kPart; x += 64) {
                    const int pr = x % (16 * kPart), qr = x / (16 * kPart) * 8;
                    if (pb0 + pr >= a.P || qb0 + qr >= a.Q) continue;
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) v[i] = turn[turn_at<kPart>(qr + i, pr)];
                    EPI::store_mirror(e, qb0 + qr, pb0 + pr, v, batch, split);
                }
            }
        }
        wave_fence();
    }
}

// Tiles of one launch: HIP takes fewer than 2^32 threads along a dimension, and
// blocks have up to 512.
constexpr int64_t kMaxTiles = (1 << 23) - 1;

inline bool al16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Whether an operand may be loaded directly: 16-byte pieces must not cross
// its edges and their offsets within a tile must fit 32 bits.  extent: k (rows)
// or the operand's own count (columns), padded where the array is.
inline bool direct_ok(const void *p, int es, int64_t ld, int64_t extent)
{
    const int per = 16 / es;
    return al16(p) && ld % per == 0 && extent % per == 0 && ld * es < (1 << 23);
}

template <int KIND, int NL, int NS, int BK, int BP, int BQ, int WP, int WQ, bool PT, bool QT, bool STAGED, bool PING, class EPI>
hipError_t launch(Args a, const typename EPI::Args &e, int splits, int batch, hipStream_t s)
{
    constexpr int kStepK = KIND == kMX8 ? 2 * BK : BK;
    a.tiles_p = (a.P + BP - 1) / BP;
    a.tiles_q = (a.Q + BQ - 1) / BQ;
    const int nt = (a.K + kStepK - 1) / kStepK, per = (nt + splits - 1) / splits;
    if ((nt + per - 1) / per != splits) return hipErrorInvalidValue;       // every split has at least one tile
    a.k_split = per * kStepK;
    const int64_t tiles = a.symmetric ? (int64_t)a.tiles_p * (a.tiles_p + 1) / 2 : (int64_t)a.tiles_p * a.tiles_q;
    if (tiles > kMaxTiles || tiles * splits * batch > INT32_MAX) return hipErrorInvalidValue;
    const dim3 grid((unsigned)tiles, (unsigned)splits, (unsigned)batch);
    product_kernel<KIND, NL, NS, BK, BP, BQ, WP, WQ, PT, QT, STAGED, PING, EPI><<<grid, WP * WQ * 64, 0, s>>>(a, e);
    return hipGetLastError();
}

}  // namespace gemm
}  // namespace gsi
