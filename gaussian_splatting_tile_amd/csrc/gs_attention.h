// Cross attention: what its kernels share (internal; the public interface is
// gs_attention_fwd and gs_attention_bwd in include/gs.h).
//
// Every product is formed with one operand's rows down the accumulators and 32
// columns across the lanes: a wave owns 32 columns (queries in the forward and
// in dq, keys in dk and dv) and walks over tiles of the other side's rows in
// LDS.  v_mfma_32x32x16 leaves lane l with column l % 32 and, in register i,
// row (i & 3) + 8 (i >> 2) + 4 (l / 32): everything that a softmax does to a
// column stays inside a lane and its partner l ^ 32, and a tile of scores is
// already the second operand of the next product, whose contraction runs over
// those rows: its 16 slots per instruction only have to be filled from the same
// rows on the other side, which the transposing LDS read takes from any four
// lines.  So probabilities go from one product to the next without leaving
// their lane.
#pragma once

#include "gs_gemm.h"

namespace gsi {
namespace attn {

using gemm::i4;
typedef float f16v __attribute__((ext_vector_type(16)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
// fp16 probabilities of the backward are held times 2^14: softmax over many
// keys has values far below fp16's smallest normal, 2^-14, and none above 1.
constexpr float kHalfShift = 14.0f;

// A tensor [batch][rows][heads][d]; strides in elements.
struct Tensor {
    const void *p;
    int64_t sb, sr, sh;
};
// A 16-bit operand as the tiles are loaded: limb l starts `plane` bytes further;
// strides in bytes.
struct Operand {
    const char *p;
    int64_t sb, sr, sh, plane;
};

// How a kernel's blocks are laid out: tiles of columns of a pair (batch element and
// head of k and v), each in `splits` of the other side's rows.
struct Grid {
    int tiles, splits, run, waves;              // run: tiles that stay on a die; waves of a block
    uint32_t blocks;                            // a multiple of 8
};

struct Args {
    Tensor q, out, dout;                        // read as they are, row by row
    Operand k, v, qt, dot;                      // read in tiles
    Tensor kt, vt;                              // k and v row by row (gradients)
    Tensor dq, dk, dv;                          // results
    Grid t, tk;                                 // of the forward or of dq, and of dk and dv
    float *lse;                                 // [batch][heads][nq], or NULL
    const float *lse2, *delta;                  // backward: [batch][heads][nq_pad]; lse times log2 e, of fp32 as it is
    // of splits, as the waves hold them: sums [split][wave][DP / 8][64][4] of out or dq, of
    // dk and of dv, and (forward) maxima, as power() takes them, and sums of exponentials
    // [split][wave][32][2];
    // wave = (pair * tiles + tile) * waves + wave of the block
    float *part, *part_k, *part_v, *ml;
    const int32_t *lengths;
    const uint8_t *mask;
    int64_t mask_stride;
    int batch, heads, kv, group, nq, nk, nq_pad, d, rows;       // rows = nq * group
    int type;                                   // gs_dtype of the tensors
    float c, scale;                             // scale * log2 e, scale
};

// exp(S - x) of a score s, S = scale s.  x is in units of log 2; fp32's in natural ones: the
// difference from it is rounded once, and small where the result is not, while the
// products' own roundings, of the size of S, would go into lse and gradients (S = 60:
// 5e-6 of them).  The second product costs fp32 1 % (2048 x 8192 x 8 heads x 64 188 -> 191 us, backward
// over 4096 states 350 -> 354); 16-bit types save it.
template <int NL> __device__ __forceinline__ float unit(const Args &a) { return NL > 1 ? a.scale : a.c; }
template <int NL> __device__ __forceinline__ float power(float x) { return __builtin_amdgcn_exp2f(NL > 1 ? x * kLog2e : x); }
template <int NL> __device__ __forceinline__ float power(const Args &a, float s, float x) { return power<NL>(fmaf(s, unit<NL>(a), -x)); }
// lse from a maximum in those units and the sum of exponentials of differences from it.
template <int NL> __device__ __forceinline__ float lse_of(float m, float sum) { return NL > 1 ? fmaf(log2f(sum), kLn2, m) : (m + log2f(sum)) * kLn2; }

// ---- tiles --------------------------------------------------------------------
// [rows][CH] chunks of 16 bytes (8 values); chunk c of row r sits at c ^ swz(r).
// Eight neighbouring rows have eight different places for a chunk, and so have the
// 4 rows x 2 chunks of a transposing read.  Sixteen places would leave no bank
// conflict at all (as it is they are 33 % of the cycles of LDS at d = 64, 50 % at
// 128), but LDS is not what bounds the kernels: no time gained, and the addresses'
// registers cost the backward at d = 128 a sixth.
template <int DP> struct HeadTile {
    static constexpr int CH = DP <= 32 ? 4 : DP <= 64 ? 8 : 16;
    static constexpr int kRowBytes = CH * 16;

    __device__ static __forceinline__ int swz(int row)
    {
        if constexpr (CH == 4) return (row >> 1) & 3;
        else return (row & 1) | ((row & 2) << 1) | ((row >> 1) & 2);
    }
    // First operand, rows row0 .. row0 + 31 (a multiple of 32), d = 16 s .. 16 s + 15.
    __device__ static __forceinline__ i4 rows(const char *lds, int row0, int s, int lane)
    {
        const int r = lane & 31, x = swz(r) ^ (lane >> 5);
        const int at = r * kRowBytes + ((((2 * s) & (CH == 4 ? 2 : 6)) ^ x) << 4);
        return *reinterpret_cast<const i4 *>(lds + at + row0 * kRowBytes + (CH == 4 ? 0 : (s >> 2) * 128));
    }
    // First operand of a contraction over rows row0 .. row0 + 15 (a multiple of
    // 16): its 32 rows are d = 32 t .. 32 t + 31, ordered so that register i of
    // the result's lane half h is d = 32 t + 16 h + i; slots 0-3 and 4-7 of lane
    // half h are rows row0 + 4 h + (0..3) and row0 + 8 + 4 h + (0..3), those of
    // the registers of a product with rows().
    __device__ static __forceinline__ i4 cols(const char *lds, int row0, int t, int lane)
    {
        const int r = lane & 15, g = ((lane >> 4) & 1) * 4 + (r & 3);           // four rows of the operand
        const int dg = (g & 1) * 4 + (g >> 1);                                  // are d = 32 t + 4 dg ..
        const int line = (lane >> 5) * 4 + (r >> 2), x = swz(line) ^ (dg >> 1);
        i4 v;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            // lines 8 apart are swizzled alike where a row has 8 chunks or more, and also where it has 4
            const char *a = lds + (row0 + line + j * 8) * kRowBytes + ((x ^ ((t & 1) * (CH == 4 ? 0 : 4))) << 4) + (t >> 1) * 128 + (dg & 1) * 8;
            const int2 h = __builtin_bit_cast(int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) gemm::s4 *)a));
            v[2 * j] = h.x;
            v[2 * j + 1] = h.y;
        }
        return v;
    }
};

// Keys (or queries) of a tile in LDS: 64, or 32 where two stages of three limbs of
// them would be 96 KB (d = 64) or 192.
template <int NL, int DP> constexpr int kTileRows = NL > 1 && DP > 32 ? 32 : 64;

// Waves on a SIMD that the register budget leaves room for: the limbs of fp32 and
// single waves (more loads each) take what there is.
constexpr int room_for(int limbs, int waves, int most) { return limbs > 1 || waves == 1 ? 1 : most; }

// Loads of a tile of ROWS rows of one operand, straight into LDS.
template <int DP, int ROWS, int THREADS> struct Loader {
    using TL = HeadTile<DP>;
    static constexpr int kChunks = ROWS * TL::CH, kLoads = kChunks / THREADS, kStep = THREADS / TL::CH;
    static constexpr int kBytes = kChunks * 16;
    // a thread's chunks sit alike in their rows, or (rows 4 apart) in every other of them
    static constexpr int kKinds = kStep % 8 ? 2 : 1;
    static_assert(kChunks % THREADS == 0 && kStep % 4 == 0, "tile and block size");
    int line0;
    uint32_t off[kKinds], step;                 // bytes from the tile's first row; kBufferBytes: past d

    __device__ __forceinline__ void init(int64_t sr, int d, int tid)
    {
        line0 = tid / TL::CH;
#pragma unroll
        for (int i = 0; i < kKinds; i++) {
            const int c = (tid % TL::CH) ^ TL::swz(line0 + i * kStep);
            off[i] = c * 8 < d ? (uint32_t)line0 * (uint32_t)sr + (uint32_t)c * 16u : gemm::kBufferBytes;
        }
        step = (uint32_t)kStep * (uint32_t)sr;
    }
    // Rows whose bit in `seen` is 0 and columns past d arrive as zeros.
    __device__ __forceinline__ void issue(const char *base, char *lds, uint64_t seen, int wave) const
    {
        const i4 buffer = gemm::buffer_at(base);
#pragma unroll
        for (int j = 0; j < kLoads; j++) {
            const uint32_t at = off[j % kKinds];
            const bool there = (seen >> (line0 + j * kStep)) & 1;
            gemm::load_lds16(buffer, there && at != gemm::kBufferBytes ? at + (uint32_t)j * step : gemm::kBufferBytes,
                             lds + (j * THREADS + wave * 64) * 16);
        }
    }
};

// 64 consecutive floats to LDS, a lane each.
__device__ __forceinline__ void load_lds4(i4 buffer, uint32_t off, const char *lds)
{
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char *)lds);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(buffer)
                 : "memory");
}

// ---- products -------------------------------------------------------------------
template <int KIND> __device__ __forceinline__ f16v mfma(i4 a, i4 b, f16v c)
{
    if constexpr (KIND == gemm::kF16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(gemm::h8, a), __builtin_bit_cast(gemm::h8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(gemm::bf8, a), __builtin_bit_cast(gemm::bf8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f16v zeros()
{
    return f16v{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
}

// Second operands from eight fp32 values: rounded to nearest even, or as limbs.
template <int KIND, int NL> __device__ __forceinline__ void pack8(const float v[8], i4 w[NL])
{
    if constexpr (NL > 1) {
        Vec<uint16_t, 8> l[NL];
        split_all<NL, 8>(v, l);
#pragma unroll
        for (int i = 0; i < NL; i++) w[i] = __builtin_bit_cast(i4, l[i]);
    } else {
        typedef float f2 __attribute__((ext_vector_type(2)));
        typedef __bf16 b2 __attribute__((ext_vector_type(2)));
        typedef _Float16 h2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const f2 x = {v[2 * i], v[2 * i + 1]};
            if constexpr (KIND == gemm::kF16) w[0][i] = __builtin_bit_cast(int, __builtin_convertvector(x, h2));
            else w[0][i] = __builtin_bit_cast(int, __builtin_convertvector(x, b2));
        }
    }
}

template <int NL> struct Elements { typedef float type; };
template <> struct Elements<1> { typedef uint16_t type; };

// A wave's own 32 columns: lane l holds row `row` (its column), d = 16 s + 8 (l / 32) + (0..7).
// Loads are whole vectors that no branch waits for (past d: of the last values,
// unused; a row that is not there is one that is), but for the last values of a d
// that is no multiple of 8.
template <int KIND, int NL, int STEPS> __device__ __forceinline__ void load_columns(const char *row, bool there, int d, int lane, i4 f[NL][STEPS])
{
    using E = typename Elements<NL>::type;
    const E *p = reinterpret_cast<const E *>(row);
    Vec<E, 8> w[STEPS] = {};
    const int mine = (lane >> 5) * 8, whole = d & ~7;
    if (whole) {
#pragma unroll
        for (int s = 0; s < STEPS; s++) w[s] = *reinterpret_cast<const Vec<E, 8> *>(p + min(s * 16 + mine, whole - 8));
    }
#pragma unroll
    for (int s = 0; s < STEPS; s++)
#pragma unroll
        for (int j = 0; j < 8; j++) w[s].v[j] = there && s * 16 + mine < whole ? w[s].v[j] : E(0);
    if (d != whole) {
        E last[8];
#pragma unroll
        for (int j = 0; j < 8; j++) last[j] = p[min(whole + j, d - 1)];
#pragma unroll
        for (int s = 0; s < STEPS; s++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (there && s * 16 + mine == whole && whole + j < d) w[s].v[j] = last[j];
    }
#pragma unroll
    for (int s = 0; s < STEPS; s++) {
        if constexpr (NL > 1) {
            i4 l[NL];
            pack8<KIND, NL>(w[s].v, l);
#pragma unroll
            for (int i = 0; i < NL; i++) f[i][s] = l[i];
        } else {
            f[0][s] = __builtin_bit_cast(i4, w[s]);
        }
    }
}

// 32 rows of a tile times the wave's columns, contracted over d.
template <int KIND, int NL, int DP, int TILE> __device__ __forceinline__ f16v over_d(const char *lds, int row0, const i4 (&f)[NL][DP / 16], int lane)
{
    f16v acc = zeros();
#pragma unroll
    for (int s = 0; s < DP / 16; s++) {
        i4 a[NL];
#pragma unroll
        for (int l = 0; l < NL; l++) a[l] = HeadTile<DP>::rows(lds + l * TILE, row0, s, lane);
#pragma unroll
        for (int order = NL - 1; order >= 0; order--)
#pragma unroll
            for (int l = 0; l <= order; l++) acc = mfma<KIND>(a[l], f[order - l][s], acc);
    }
    return acc;
}
// acc[t] += (32 rows of a tile)^T times their weights w (those of registers 8 j ..
// 8 j + 7 in w[..][j]).
template <int KIND, int NL, int DP, int TILE> __device__ __forceinline__ void over_rows(const char *lds, int row0, const i4 (&w)[2][NL], f16v (&acc)[DP / 32], int lane)
{
#pragma unroll
    for (int j = 0; j < 2; j++)
#pragma unroll
        for (int t = 0; t < DP / 32; t++) {
            i4 a[NL];
#pragma unroll
            for (int l = 0; l < NL; l++) a[l] = HeadTile<DP>::cols(lds + l * TILE, row0 + 16 * j, t, lane);
#pragma unroll
            for (int order = NL - 1; order >= 0; order--)
#pragma unroll
                for (int l = 0; l <= order; l++) acc[t] = mfma<KIND>(a[l], w[j][order - l], acc[t]);
        }
}

// The larger and the sum of a lane's value and its partner's (lane ^ 32).
__device__ __forceinline__ float pair_max(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// A lane's 16 values d = 32 t + 16 h .. of each t, times f, to a row.
template <int DP> __device__ __forceinline__ void store_columns(void *row, int type, int64_t at, const f16v (&acc)[DP / 32], float f, int d, int lane)
{
#pragma unroll
    for (int t = 0; t < DP / 32; t++)
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int x = t * 32 + (lane >> 5) * 16 + j * 8;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = acc[t][j * 8 + i] * f;
            if (x + 8 <= d) {
                store8_vec(row, type, at + x, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++)
                    if (x + i < d) store_from_float(row, type, at + x + i, v[i]);
            }
        }
}

// A wave's sums as they are, for the joining of splits: 16 bytes a lane, in order.
template <int DP> __device__ __forceinline__ void store_part(float *part, int64_t at, const f16v (&acc)[DP / 32], float f, int lane)
{
    gemm::f4 *to = reinterpret_cast<gemm::f4 *>(part) + at * (DP / 8 * 64) + lane;
#pragma unroll
    for (int t = 0; t < DP / 32; t++)
#pragma unroll
        for (int i = 0; i < 4; i++) to[(t * 4 + i) * 64] = gemm::f4{acc[t][4 * i], acc[t][4 * i + 1], acc[t][4 * i + 2], acc[t][4 * i + 3]} * f;
}

// Which of 64 keys from k0 on are attended.  `byte`: the lane's mask byte (lane =
// key), prefetched; 1 without a mask.
__device__ __forceinline__ uint64_t attended(int k0, int length, uint32_t byte, int lane)
{
    return __ballot(k0 + lane < length && byte != 0);
}
__device__ __forceinline__ uint32_t mask_byte(const Args &a, int batch, int64_t key, int length)
{
    return a.mask && key < length ? a.mask[(int64_t)batch * a.mask_stride + key] : 1u;
}
__device__ __forceinline__ int length_of(const Args &a, int batch)
{
    return a.lengths ? max(0, min(a.lengths[batch], a.nk)) : a.nk;
}

// What a block works on.  Blocks go to the 8 dies in turn; runs of tiles that share
// a head's operands and a split stay on one die, whose second-level cache then
// serves them, and neighbouring runs go to different dies, so that batch elements
// of different lengths keep all of them busy (4 x 1000 x 2777 of ragged lengths: 72 us
// before this and partial sums in the waves' own order, 54 with both).
struct Item {
    int batch, head, split, tile;               // head: of k and v
};
__device__ __forceinline__ bool item_of(const Args &a, const Grid &g, uint32_t b, Item &it)
{
    const uint32_t at = b >> 3, run = at / (uint32_t)g.run * 8 + (b & 7), parts = ((uint32_t)g.tiles + g.run - 1) / g.run;
    const uint32_t pair = run / parts, group = pair / (uint32_t)g.splits;
    it.tile = (int)((run - pair * parts) * g.run + at % g.run);
    it.split = (int)(pair - group * g.splits);
    it.batch = (int)(group / (uint32_t)a.kv);
    it.head = (int)(group - (uint32_t)it.batch * a.kv);
    return it.batch < a.batch && it.tile < g.tiles;
}
// The wave's place among the partial sums.
__device__ __forceinline__ int64_t part_at(const Args &a, const Grid &g, const Item &it, int wave)
{
    const int64_t pairs = (int64_t)a.batch * a.kv;
    return ((it.split * pairs + (int64_t)it.batch * a.kv + it.head) * g.tiles + it.tile) * g.waves + wave;
}

}  // namespace attn
}  // namespace gsi
