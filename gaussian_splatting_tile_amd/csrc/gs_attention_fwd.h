// The forward's kernel, instantiated once per kind of operand.
#pragma once

#include "gs_attention.h"

namespace gsi {
namespace attn {

// Online softmax over tiles of keys.  A column's scores are the lane's and its
// partner's registers.  What is subtracted from them is the maximum of the first
// tile, and a later one's only where probabilities have grown so large that a
// tile's sum passes 2^13 (fp16 holds 2^16): then the tile is done again and the
// sums so far are rescaled.  So the usual tile looks for no maximum.
// Probabilities are rounded to the operands' type for the second product (half
// an ulp each, unbiased), which leaves bf16's out 2.3e-3 of its norm off; out's own
// rounding alone is 1.7e-3, and what two limbs of each would leave takes 2048 x 16384 x 64
// from 176 to 244 us, 4096 x 4096 x 128 from 136 to 188.  Their sum takes them
// unrounded, as lse has to be good to fp32.  fp16 ones are held times 2^6, 64 of which still stay below 2^13: it is
// 2^-20 of the maximum, not 2^-14, where they begin to lose bits, which many keys of
// little weight would feel (262143 of 2^-20.5: 0.4 % of out).
//
// Bound by the two kinds of instructions one after the other: 4096 x 4096 x 16
// heads take 64 us at d = 32, 86 at 64 and 136 at 128 (1.0 PFLOP/s), which is 40 us
// for a score's fused multiply-add, exponential, sum and rounding, and 0.75 us per d
// for the products.  A fourth wave on a SIMD (128 registers: 175 -> 178 us for
// 2048 x 16384 x 64), priorities for either kind (174 -> 181) and LDS without bank
// conflicts change nothing; leaving out the maximum of the usual tile gave 186 -> 174.
constexpr float kMostSum = 8192.0f;
template <int KIND> constexpr float kBelow = KIND == gemm::kF16 ? 6.0f : 0.0f;

template <int KIND, int NL, int DP, int NW> __global__ __launch_bounds__(NW * 64, room_for(NL, NW, DP <= 32 ? 4 : DP <= 64 ? 3 : 2)) void attention_fwd(Args a)
{
    constexpr int KT = kTileRows<NL, DP>, KS = KT / 32;
    using LD = Loader<DP, KT, NW * 64>;
    constexpr int kStage = 2 * NL * LD::kBytes;
    __shared__ __align__(128) char lds[2 * kStage];

    Item it;
    if (!item_of(a, a.t, (uint32_t)block_of(), it)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int length = length_of(a, it.batch);
    // this split's tiles
    const int tiles = (length + KT - 1) / KT, per = (tiles + a.t.splits - 1) / a.t.splits;
    const int t0 = it.split * per, t1 = min(tiles, t0 + per);

    const int row = (it.tile * NW + wave) * 32 + (lane & 31);
    const bool there = row < a.rows;
    const int token = there ? row / a.group : 0, head = it.head * a.group + (there ? row - token * a.group : 0);
    i4 q[NL][DP / 16];
    load_columns<KIND, NL, DP / 16>(static_cast<const char *>(a.q.p) +
                                        (it.batch * a.q.sb + token * a.q.sr + head * a.q.sh) * (NL > 1 ? 4 : 2),
                                    there, a.d, lane, q);

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

    f16v o[DP / 32];
#pragma unroll
    for (int t = 0; t < DP / 32; t++) o[t] = zeros();
    float m = -INFINITY, base = 0.0f, sum = 0.0f;          // m: what is subtracted; base: the same, or 0 before there is one
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
        f16v s[KS];
#pragma unroll
        for (int u = 0; u < KS; u++) {
            s[u] = over_d<KIND, NL, DP, LD::kBytes>(kt, u * 32, q, lane);
            if (seen != whole) {
                const uint32_t bits = (uint32_t)(seen >> (u * 32)) >> (4 * (lane >> 5));
#pragma unroll
                for (int i = 0; i < 16; i++)
                    if (!((bits >> ((i & 3) + 8 * (i >> 2))) & 1)) s[u][i] = -INFINITY;
            }
        }
        i4 w[KS][2][NL];
        float more;                             // of this tile's probabilities
        auto exponentials = [&]() {
            more = 0.0f;
#pragma unroll
            for (int u = 0; u < KS; u++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        v[i] = power<NL>(a, s[u][j * 8 + i], base);
                        more += v[i];
                    }
                    pack8<KIND, NL>(v, w[u][j]);
                }
        };
        bool again = __any(m == -INFINITY);
        if (!again) {
            exponentials();
            again = __any(!(more < kMostSum));
        }
        if (again) {
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < KS; u++)
#pragma unroll
                for (int i = 0; i < 16; i++) top = fmaxf(top, s[u][i]);
            const float up = fmaxf(m, pair_max(top * unit<NL>(a)) - kBelow<KIND>), now = up == -INFINITY ? 0.0f : up, f = power<NL>(m - now);
            m = up;
            base = now;
            sum *= f;
#pragma unroll
            for (int t = 0; t < DP / 32; t++) o[t] *= f;
            exponentials();
        }
        sum += more;
#pragma unroll
        for (int u = 0; u < KS; u++) over_rows<KIND, NL, DP, LD::kBytes>(vt, u * 32, w[u], o, lane);
    }

    sum = pair_sum(sum);
    if (a.t.splits > 1) {                         // as they are, for join_splits
        const int64_t at = part_at(a, a.t, it, wave);
        store_part<DP>(a.part, at, o, 1.0f, lane);
        if (lane < 32) *reinterpret_cast<float2 *>(a.ml + (at * 32 + lane) * 2) = float2{m, sum};
        return;
    }
    if (!there) return;
    const float f = m == -INFINITY && sum == 0.0f ? 0.0f : 1.0f / sum;
    store_columns<DP>(const_cast<void *>(a.out.p), a.type, it.batch * a.out.sb + token * a.out.sr + head * a.out.sh, o, f, a.d, lane);
    if (a.lse && lane < 32) a.lse[((int64_t)it.batch * a.heads + head) * a.nq + token] = lse_of<NL>(m, sum);
}

template <int KIND, int NL, int DP> hipError_t launch_fwd_waves(const Args &a, hipStream_t s)
{
    const dim3 grid = grid_of(a.t.blocks, a.t.waves * 64);
    if (a.t.waves == 1) attention_fwd<KIND, NL, DP, 1><<<grid, 64, 0, s>>>(a);
    else attention_fwd<KIND, NL, DP, 4><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}
template <int KIND, int NL> hipError_t launch_fwd_kind(const Args &a, hipStream_t s)
{
    if (a.d <= 32) return launch_fwd_waves<KIND, NL, 32>(a, s);
    if (a.d <= 64) return launch_fwd_waves<KIND, NL, 64>(a, s);
    if (a.d <= 96) return launch_fwd_waves<KIND, NL, 96>(a, s);
    return launch_fwd_waves<KIND, NL, 128>(a, s);
}

}  // namespace attn
}  // namespace gsi
