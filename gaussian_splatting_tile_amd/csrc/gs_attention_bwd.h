// The backward's kernels, instantiated once per kind of operand.
//
//   P = exp(S - lse),  dP = dout v,  dS = P (dP - delta),
//   dq = scale dS k,   dk = scale dS^T q,   dv = P^T dout
//
// by two kinds of blocks of one launch, each of which forms S and dP itself: some
// walk over keys and sum dq, the others over queries and sum dk and dv.  Two of
// seven products are formed twice; in exchange nothing is added to memory from
// many blocks, so the results do not depend on an order, and a card that one kind
// would not fill has the other's blocks too (with one launch each for what comes
// before, for both kinds and for all joins, 2048 x 8192 took 271 us, not 286, and
// 1 x 300 x 2000 27, not 45).
//
// P and dS are rounded to the operands' type for the last products: bf16's gradients are
// 2.4e-3 of their norm off, 1.7e-3 of it by their own rounding.  Two limbs of each leave just that
// and take 352 us, not 257, for 2048 x 8192 x 64, and 777, not 548, for 4096 x 4096 x 128.
//
// Bound by the products and what makes P and dS out of them, as the forward:
// 2048 x 8192 x 16 heads x 64 245 us for seven products, 0.98 PFLOP/s (256 with what is
// before and after); 4096 x 4096 x 16 x 128 548 us, 0.88 PFLOP/s.
#pragma once

#include "gs_attention.h"

namespace gsi {
namespace attn {

// fp16 holds a column of dS times a power of two of its own, which shrinks as
// larger values come (like a softmax's maximum): gradients are small, P of many
// keys too, and their product would be subnormal in fp16, or vanish.  bf16 and
// the limbs of fp32 have fp32's exponents.
template <int KIND> struct ColumnScale {
    float f = KIND == gemm::kF16 ? 0x1p100f : 1.0f;

    // Brings v (16 values of the lane's column) to this scale; acc are the sums so far.
    template <int T> __device__ __forceinline__ void apply(float v[16], f16v (&acc)[T])
    {
        if constexpr (KIND == gemm::kF16) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(v[i]));
            if (__any(top * f > 32768.0f)) {
                top = pair_max(top);
                if (top * f > 32768.0f) {       // to 2^10 .. 2^11
                    const int e = max(-100, min(100, (int)(__float_as_uint(top) >> 23) - 127 - 10));
                    const float now = __uint_as_float((uint32_t)(127 - e) << 23), less = now / f;
                    f = now;
#pragma unroll
                    for (int t = 0; t < T; t++) acc[t] *= less;
                }
            }
#pragma unroll
            for (int i = 0; i < 16; i++) v[i] *= f;
        }
    }
    __device__ __forceinline__ float inverse() const { return KIND == gemm::kF16 ? 1.0f / f : 1.0f; }
};

template <int KIND, int NL> __device__ __forceinline__ void pack16(const float v[16], i4 (&w)[2][NL])
{
#pragma unroll
    for (int j = 0; j < 2; j++) pack8<KIND, NL>(v + j * 8, w[j]);
}

// The second half of a tile is left out where nothing is in it, but not of 128 wide
// heads: the branch keeps the halves' instructions apart, and with two waves on a
// SIMD nothing else fills the gap (4096 x 4096 x 128: 545 -> 619 us; x 64: 271 -> 260).
template <int DP> constexpr bool kSkip = DP <= 96;

// dq: a wave owns 32 queries and walks over tiles of keys.
template <int KIND, int NL, int DP, int NW> __device__ __forceinline__ void dq_block(const Args &a, uint32_t block, char *lds)
{
    constexpr int KT = kTileRows<NL, DP>, KS = KT / 32;
    using LD = Loader<DP, KT, NW * 64>;
    constexpr int kStage = 2 * NL * LD::kBytes, ES = NL > 1 ? 4 : 2;

    Item it;
    if (!item_of(a, a.t, block, it)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int length = length_of(a, it.batch);
    const int tiles = (length + KT - 1) / KT, per = (tiles + a.t.splits - 1) / a.t.splits;
    const int t0 = it.split * per, t1 = min(tiles, t0 + per);

    const int row = (it.tile * NW + wave) * 32 + (lane & 31);
    const bool there = row < a.rows;
    const int token = there ? row / a.group : 0, head = it.head * a.group + (there ? row - token * a.group : 0);
    i4 q[NL][DP / 16], g[NL][DP / 16];
    load_columns<KIND, NL, DP / 16>(static_cast<const char *>(a.q.p) + (it.batch * a.q.sb + token * a.q.sr + head * a.q.sh) * ES, there, a.d, lane, q);
    load_columns<KIND, NL, DP / 16>(static_cast<const char *>(a.dout.p) + (it.batch * a.dout.sb + token * a.dout.sr + head * a.dout.sh) * ES, there, a.d, lane, g);
    const int64_t stat = ((int64_t)it.batch * a.heads + head) * a.nq_pad + token;
    const float lse = there ? a.lse2[stat] : INFINITY, delta = there ? a.delta[stat] : 0.0f;

    LD lk, lv;
    lk.init(a.k.sr, a.d, tid);
    lv.init(a.v.sr, a.d, tid);
    const char *kb = a.k.p + it.batch * a.k.sb + it.head * a.k.sh, *vb = a.v.p + it.batch * a.v.sb + it.head * a.v.sh;
    auto issue = [&](int t, uint64_t seen) {
        char *s = lds + (t & 1) * kStage;
#pragma unroll
        for (int l = 0; l < NL; l++) {
            lk.issue(kb + l * a.k.plane + (int64_t)t * KT * a.k.sr, s + l * LD::kBytes, seen, wave);
            lv.issue(vb + l * a.v.plane + (int64_t)t * KT * a.v.sr, s + (NL + l) * LD::kBytes, seen, wave);
        }
    };
    const uint64_t whole = KT == 64 ? ~0ull : 0xFFFFFFFFull;
    auto byte_of = [&](int t) { return t < t1 ? mask_byte(a, it.batch, (int64_t)t * KT + lane, length) : 0u; };
    auto seen_in = [&](int t, uint32_t byte) { return t < t1 ? attended(t * KT, length, byte, lane) & whole : 0ull; };

    f16v acc[DP / 32];
#pragma unroll
    for (int t = 0; t < DP / 32; t++) acc[t] = zeros();
    ColumnScale<KIND> scale;
    uint64_t seen = seen_in(t0, byte_of(t0)), next = 0;
    uint32_t byte = byte_of(t0 + 1);
    if (t0 < t1) issue(t0, seen);
    for (int t = t0; t < t1; t++, seen = next) {
        gemm::stage_barrier<0>();
        next = seen_in(t + 1, byte);
        byte = byte_of(t + 2);
        if (t + 1 < t1) issue(t + 1, next);
        if (!seen) continue;
        const char *kt = lds + (t & 1) * kStage, *vt = kt + NL * LD::kBytes;
#pragma unroll
        for (int u = 0; u < KS; u++) {
            if (kSkip<DP> && u && !(seen >> 32)) break;
            const f16v s = over_d<KIND, NL, DP, LD::kBytes>(kt, u * 32, q, lane);
            const f16v dp = over_d<KIND, NL, DP, LD::kBytes>(vt, u * 32, g, lane);
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; i++) v[i] = power<NL>(a, s[i], lse) * (dp[i] - delta);
            if (seen != whole) {
                const uint32_t bits = (uint32_t)(seen >> (u * 32)) >> (4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 16; i++)
                    if (!((bits >> ((i & 3) + 8 * (i >> 2))) & 1)) v[i] = 0.0f;
            }
            scale.apply(v, acc);
            i4 w[2][NL];
            pack16<KIND, NL>(v, w);
            over_rows<KIND, NL, DP, LD::kBytes>(kt, u * 32, w, acc, lane);
        }
    }
    const float f = a.scale * scale.inverse() * (KIND == gemm::kF16 ? 1.0f / (float)(1 << (int)kHalfShift) : 1.0f);
    if (a.t.splits > 1) {
        store_part<DP>(a.part, part_at(a, a.t, it, wave), acc, f, lane);
    } else if (there) {
        store_columns<DP>(const_cast<void *>(a.dq.p), a.type, it.batch * a.dq.sb + token * a.dq.sr + head * a.dq.sh, acc, f, a.d, lane);
    }
}

// dk and dv: a wave owns 32 keys and walks over tiles of queries of every head
// that shares them.
template <int KIND, int NL, int DP, int NW> __device__ __forceinline__ void dkv_block(const Args &a, uint32_t block, char *lds)
{
    constexpr int RT = kTileRows<NL, DP>, RS = RT / 32;
    using LD = Loader<DP, RT, NW * 64>;
    constexpr int kOperands = 2 * NL * LD::kBytes, kStage = kOperands + 512, ES = NL > 1 ? 4 : 2;

    Item it;
    if (!item_of(a, a.tk, block, it)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int length = length_of(a, it.batch);
    const int key = (it.tile * NW + wave) * 32 + (lane & 31);
    const bool there = key < a.nk, seen = key < length && mask_byte(a, it.batch, key, length);
    const bool all = __all(seen);
    // a block without an attended key has only zeros to write
    const bool any = __syncthreads_or(seen);

    // tiles of queries of one head after the other
    const int per_head = (a.nq + RT - 1) / RT;
    const int64_t tiles = any ? (int64_t)per_head * a.group : 0, per = (tiles + a.tk.splits - 1) / a.tk.splits;
    const int64_t t0 = it.split * per, t1 = min(tiles, t0 + per);

    i4 k[NL][DP / 16], v[NL][DP / 16];
    load_columns<KIND, NL, DP / 16>(static_cast<const char *>(a.kt.p) + (it.batch * a.kt.sb + (seen ? key : 0) * a.kt.sr + it.head * a.kt.sh) * ES, seen, a.d, lane, k);
    load_columns<KIND, NL, DP / 16>(static_cast<const char *>(a.vt.p) + (it.batch * a.vt.sb + (seen ? key : 0) * a.vt.sr + it.head * a.vt.sh) * ES, seen, a.d, lane, v);

    LD lq, lg;
    lq.init(a.qt.sr, a.d, tid);
    lg.init(a.dot.sr, a.d, tid);
    const char *qb = a.qt.p + it.batch * a.qt.sb + (int64_t)it.head * a.group * a.qt.sh, *gb = a.dot.p + it.batch * a.dot.sb + (int64_t)it.head * a.group * a.dot.sh;
    const int64_t stat = ((int64_t)it.batch * a.heads + it.head * a.group) * a.nq_pad;
    auto issue = [&](int64_t t) {
        char *s = lds + (t & 1) * kStage;
        const int head = (int)(t / per_head), r0 = (int)(t - (int64_t)head * per_head) * RT;
        const int left = a.nq - r0;
        const uint64_t rows = left >= 64 ? ~0ull : (1ull << left) - 1;
#pragma unroll
        for (int l = 0; l < NL; l++) {
            lq.issue(qb + l * a.qt.plane + head * a.qt.sh + r0 * a.qt.sr, s + l * LD::kBytes, rows, wave);
            lg.issue(gb + l * a.dot.plane + head * a.dot.sh + r0 * a.dot.sr, s + (NL + l) * LD::kBytes, rows, wave);
        }
        if (wave == 0) {                        // the rows' lse and delta; nq_pad is a multiple of 64
            const int64_t at = stat + (int64_t)head * a.nq_pad + r0;
            const uint32_t mine = lane < RT ? lane * 4u : gemm::kBufferBytes;
            load_lds4(gemm::buffer_at(a.lse2 + at), mine, s + kOperands);
            load_lds4(gemm::buffer_at(a.delta + at), mine, s + kOperands + 256);
        }
    };

    f16v dk[DP / 32], dv[DP / 32];
#pragma unroll
    for (int t = 0; t < DP / 32; t++) dk[t] = dv[t] = zeros();
    ColumnScale<KIND> scale;
    int in_head = (int)(t0 % max(per_head, 1));             // the tile's number in its head
    if (t0 < t1) issue(t0);
    for (int64_t t = t0; t < t1; t++) {
        gemm::stage_barrier<0>();
        if (t + 1 < t1) issue(t + 1);
        const char *qt = lds + (t & 1) * kStage, *gt = qt + NL * LD::kBytes;
        const float *lse = reinterpret_cast<const float *>(qt + kOperands), *delta = lse + 64;
#pragma unroll
        for (int u = 0; u < RS; u++) {
            if (kSkip<DP> && u && a.nq - in_head * RT <= 32) break;
            const f16v s = over_d<KIND, NL, DP, LD::kBytes>(qt, u * 32, k, lane);
            float p[16], ds[16];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const gemm::f4 l = *reinterpret_cast<const gemm::f4 *>(lse + u * 32 + j * 8 + (lane >> 5) * 4);
#pragma unroll
                for (int i = 0; i < 4; i++) p[j * 4 + i] = power<NL>(a, s[j * 4 + i], l[i]);
            }
            const f16v dp = over_d<KIND, NL, DP, LD::kBytes>(gt, u * 32, v, lane);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const gemm::f4 d = *reinterpret_cast<const gemm::f4 *>(delta + u * 32 + j * 8 + (lane >> 5) * 4);
#pragma unroll
                for (int i = 0; i < 4; i++) ds[j * 4 + i] = p[j * 4 + i] * (dp[j * 4 + i] - d[i]);
            }
            if (!all) {
#pragma unroll
                for (int i = 0; i < 16; i++) {
                    p[i] = seen ? p[i] : 0.0f;
                    ds[i] = seen ? ds[i] : 0.0f;
                }
            }
            i4 w[2][NL];
            pack16<KIND, NL>(p, w);
            over_rows<KIND, NL, DP, LD::kBytes>(gt, u * 32, w, dv, lane);
            scale.apply(ds, dk);
            pack16<KIND, NL>(ds, w);
            over_rows<KIND, NL, DP, LD::kBytes>(qt, u * 32, w, dk, lane);
        }
        in_head = in_head + 1 == per_head ? 0 : in_head + 1;
    }
    const float down = KIND == gemm::kF16 ? 1.0f / (float)(1 << (int)kHalfShift) : 1.0f, f = a.scale * scale.inverse() * down;
    if (a.tk.splits > 1) {
        const int64_t at = part_at(a, a.tk, it, wave);
        store_part<DP>(a.part_k, at, dk, f, lane);
        store_part<DP>(a.part_v, at, dv, down, lane);
    } else if (there) {
        if (a.dk.p) store_columns<DP>(const_cast<void *>(a.dk.p), a.type, it.batch * a.dk.sb + key * a.dk.sr + it.head * a.dk.sh, dk, f, a.d, lane);
        if (a.dv.p) store_columns<DP>(const_cast<void *>(a.dv.p), a.type, it.batch * a.dv.sb + key * a.dv.sr + it.head * a.dv.sh, dv, down, a.d, lane);
    }
}

template <int KIND, int NL, int DP, int NW> __global__ __launch_bounds__(NW * 64, room_for(NL, NW, DP <= 32 ? 4 : DP <= 64 ? 3 : 2)) void attention_bwd(Args a)
{
    using LD = Loader<DP, kTileRows<NL, DP>, NW * 64>;
    __shared__ __align__(128) char lds[2 * (2 * NL * LD::kBytes + 512)];
    const uint32_t b = (uint32_t)block_of();
    if (b < a.tk.blocks) dkv_block<KIND, NL, DP, NW>(a, b, lds);
    else dq_block<KIND, NL, DP, NW>(a, b - a.tk.blocks, lds);
}

template <int KIND, int NL, int DP> hipError_t launch_bwd_waves(const Args &a, int waves, hipStream_t s)
{
    const dim3 grid = grid_of((int64_t)a.tk.blocks + a.t.blocks, waves * 64);
    if (waves == 1) attention_bwd<KIND, NL, DP, 1><<<grid, 64, 0, s>>>(a);
    else attention_bwd<KIND, NL, DP, 4><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}
// Blocks of `waves` waves, of one kind or both.
template <int KIND, int NL> hipError_t launch_bwd_kind(const Args &a, int waves, hipStream_t s)
{
    if (a.d <= 32) return launch_bwd_waves<KIND, NL, 32>(a, waves, s);
    if (a.d <= 64) return launch_bwd_waves<KIND, NL, 64>(a, waves, s);
    if (a.d <= 96) return launch_bwd_waves<KIND, NL, 96>(a, waves, s);
    return launch_bwd_waves<KIND, NL, 128>(a, waves, s);
}

}  // namespace attn
}  // namespace gsi
