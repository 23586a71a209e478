// Cross attention: argument checks, the choice of launches, and the small
// kernels around the main ones (gs_attention_fwd.h, gs_attention_bwd.h): packed
// copies of operands that cannot be loaded directly, the backward's row
// statistics, and the joining of splits.
#include "gs_attention.h"

#include <math.h>

#include <algorithm>

namespace gsi {
namespace attn {

hipError_t launch_fwd_bf16(const Args &, int, hipStream_t);
hipError_t launch_fwd_f16(const Args &, int, hipStream_t);
hipError_t launch_fwd_f32(const Args &, int, hipStream_t);
hipError_t launch_dq_bf16(const Args &, int, hipStream_t);
hipError_t launch_dq_f16(const Args &, int, hipStream_t);
hipError_t launch_dq_f32(const Args &, int, hipStream_t);
hipError_t launch_dkv_bf16(const Args &, int, hipStream_t);
hipError_t launch_dkv_f16(const Args &, int, hipStream_t);
hipError_t launch_dkv_f32(const Args &, int, hipStream_t);

namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 128;

gs_status from_hip(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }
bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
constexpr size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// ---- packed operands ------------------------------------------------------------
// [limb][batch][heads][n][dp] of 16 bits from a tensor of any strides, d padded
// with zeros to a multiple of 8; fp32 in three limbs.
struct PackArgs {
    Tensor from;
    char *to;
    int64_t plane;                              // values of a limb
    int n, heads, pairs, d, chunks, type;       // pairs: batch * heads; chunks: of 8 values in a row
};
template <int NL> __global__ __launch_bounds__(kThreads) void pack(PackArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= (int64_t)a.n * a.chunks) return;
    const int row = (int)(i / a.chunks), at = (int)(i - (int64_t)row * a.chunks) * 8;
    for (int pair = blockIdx.y; pair < a.pairs; pair += gridDim.y) {
        const int batch = pair / a.heads, head = pair - batch * a.heads;
        const int64_t from = batch * a.from.sb + row * a.from.sr + head * a.from.sh + at;
        const int64_t to = (((int64_t)pair * a.n + row) * a.chunks) * 8 + at;
        const int valid = min(8, a.d - at);
        if constexpr (NL > 1) {
            float v[8];
            load8(a.from.p, GS_DTYPE_F32, from, valid, v);
            Vec<uint16_t, 8> w[NL];
            split_all<NL, 8>(v, w);
#pragma unroll
            for (int l = 0; l < NL; l++) *reinterpret_cast<Vec<uint16_t, 8> *>(a.to + (l * a.plane + to) * 2) = w[l];
        } else {
            Vec<uint16_t, 8> w = {{0, 0, 0, 0, 0, 0, 0, 0}};
            const uint16_t *p = static_cast<const uint16_t *>(a.from.p) + from;
            if (valid == 8) w = *reinterpret_cast<const Vec<uint16_t, 8> *>(p);
            else
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (j < valid) w.v[j] = p[j];
            *reinterpret_cast<Vec<uint16_t, 8> *>(a.to + to * 2) = w;
        }
    }
}

// ---- row statistics of the backward ------------------------------------------------
// delta = dout . out, and lse in units of log 2 with what keeps P of an empty or
// absent row at 0; 16 lanes a row.
__global__ __launch_bounds__(kThreads) void row_statistics(Args a, float *lse2, float *delta, float shift)
{
    const int lane = threadIdx.x & 15;
    const int64_t token = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
    if (token >= a.nq_pad) return;
    const int pairs = a.batch * a.heads;
    for (int pair = blockIdx.y; pair < pairs; pair += gridDim.y) {
        const int batch = pair / a.heads, head = pair - batch * a.heads;
        float dot = 0.0f;
        if (token < a.nq && lane * 8 < a.d) {
            float x[8], y[8];
            load8(a.out.p, a.type, batch * a.out.sb + token * a.out.sr + head * a.out.sh + lane * 8, a.d - lane * 8, x);
            load8(a.dout.p, a.type, batch * a.dout.sb + token * a.dout.sr + head * a.dout.sh + lane * 8, a.d - lane * 8, y);
#pragma unroll
            for (int i = 0; i < 8; i++) dot = fmaf(x[i], y[i], dot);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
        if (lane == 0) {
            const float l = token < a.nq ? a.lse[(int64_t)pair * a.nq + token] : -INFINITY;
            const int64_t at = (int64_t)pair * a.nq_pad + token;
            lse2[at] = l == -INFINITY ? INFINITY : fmaf(l, kLog2e, -shift);
            delta[at] = dot;
        }
    }
}

// ---- splits -----------------------------------------------------------------------
// A unit is 16 bytes a lane of the 64 lanes that hold 32 rows' sums; its SW waves
// take every SW-th split, the first of them adds theirs, in order.
struct JoinArgs {
    const float *part, *ml;
    Tensor to;
    float *lse;
    int64_t waves, units;                       // waves' places in a split, units = waves * per
    int per, rows, tiles, wide, group, heads, splits, d, type;      // per: units of a wave; wide: waves of a block; rows: of a pair
};
// Where a unit's lane writes: its row's place in the tensor, or not.
struct Target {
    bool there;
    int at;                                     // first of four d
    int64_t row, stat;                          // elements; index into lse
};
__device__ __forceinline__ Target target_of(const JoinArgs &a, int64_t wave, int unit, int lane)
{
    const int64_t tile = wave / a.wide, pair = tile / a.tiles;
    const int row = (int)((tile - pair * a.tiles) * a.wide + (wave - tile * a.wide)) * 32 + (lane & 31);
    const int kv = a.heads / a.group;
    const int64_t batch = pair / kv;
    const int token = row / a.group, head = (int)(pair - batch * kv) * a.group + row - token * a.group;
    Target t;
    t.there = row < a.rows;
    t.at = (unit >> 2) * 32 + (lane >> 5) * 16 + (unit & 3) * 4;
    t.row = batch * a.to.sb + token * a.to.sr + head * a.to.sh;
    t.stat = (batch * a.heads + head) * (a.rows / a.group) + token;
    return t;
}
__device__ __forceinline__ void store4(const JoinArgs &a, const Target &t, const gemm::f4 &v)
{
    void *to = const_cast<void *>(a.to.p);
    if (!t.there) return;
    if (t.at + 4 <= a.d) {
        const int64_t i = t.row + t.at;
        if (a.type == GS_DTYPE_F32) *reinterpret_cast<Vec<float, 4> *>(static_cast<float *>(to) + i) = Vec<float, 4>{{v[0], v[1], v[2], v[3]}};
        else if (a.type == GS_DTYPE_F16) *reinterpret_cast<Vec<_Float16, 4> *>(static_cast<_Float16 *>(to) + i) = Vec<_Float16, 4>{{(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]}};
        else *reinterpret_cast<Vec<__bf16, 4> *>(static_cast<__bf16 *>(to) + i) = Vec<__bf16, 4>{{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]}};
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; j++)
        if (t.at + j < a.d) store_from_float(to, a.type, t.row + t.at + j, v[j]);
}

// Partial softmaxes (SOFT: sums relative to their own maxima), or plain sums.
template <int SW, bool SOFT> __global__ __launch_bounds__(kThreads) void join_splits(JoinArgs a)
{
    constexpr int kUnits = kThreads / 64 / SW;
    __shared__ gemm::f4 turn[SW > 1 ? kThreads : 1];
    __shared__ float2 stats[SW > 1 ? kThreads : 1];
    const int lane = threadIdx.x & 63, sub = (threadIdx.x >> 6) % SW;
    const int64_t u = block_of() * kUnits + (threadIdx.x >> 6) / SW;
    const bool works = u < a.units;
    const int64_t wave = works ? u / a.per : 0;
    const int unit = works ? (int)(u - wave * a.per) : 0, splits = works ? a.splits : 0;
    const gemm::f4 *part = reinterpret_cast<const gemm::f4 *>(a.part) + (wave * a.per + unit) * 64 + lane;
    const float2 *ml = reinterpret_cast<const float2 *>(a.ml) + wave * 32 + (lane & 31);
    const int64_t next = a.waves * a.per * 64, next_ml = a.waves * 32;
    gemm::f4 v = {0, 0, 0, 0};
    float sum = 0.0f, m = -INFINITY, base = 0.0f;
    if constexpr (SOFT) {
        for (int s = sub; s < splits; s += 8 * SW) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = s + i * SW < splits ? ml[(s + i * SW) * next_ml].x : -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; i++) m = fmaxf(m, x[i]);
        }
        if constexpr (SW > 1) {
            stats[threadIdx.x].x = m;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < SW; i++) m = fmaxf(m, stats[(threadIdx.x / (64 * SW) * SW + i) * 64 + lane].x);
            __syncthreads();
        }
        base = m == -INFINITY ? 0.0f : m;
    }
    for (int s = sub; s < splits; s += 8 * SW) {
        gemm::f4 x[8];
        float2 w[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (s + i * SW < splits) {
                x[i] = part[(s + i * SW) * next];
                if constexpr (SOFT) w[i] = ml[(s + i * SW) * next_ml];
            }
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (s + i * SW < splits) {
                if constexpr (SOFT) {
                    // NaN scores have no maximum, but a sum: it goes on
                    const float f = w[i].x == -INFINITY && w[i].y != 0.0f ? 1.0f : __builtin_amdgcn_exp2f(w[i].x - base);
                    sum = fmaf(w[i].y, f, sum);
                    v += x[i] * f;
                } else {
                    v += x[i];
                }
            }
    }
    if constexpr (SW > 1) {
        turn[threadIdx.x] = v;
        stats[threadIdx.x].y = sum;
        __syncthreads();
        if (sub) return;
#pragma unroll
        for (int i = 1; i < SW; i++) {
            v += turn[threadIdx.x + i * 64];
            sum += stats[threadIdx.x + i * 64].y;
        }
    }
    if (!works) return;
    const Target t = target_of(a, wave, unit, lane);
    if constexpr (SOFT) {
        v *= m == -INFINITY && sum == 0.0f ? 0.0f : 1.0f / sum;
        if (a.lse && t.there && unit == 0 && lane < 32) a.lse[t.stat] = (m + log2f(sum)) * kLn2;
    }
    store4(a, t, v);
}

// ---- plan ----------------------------------------------------------------------------
struct Tiling {
    int waves, tiles, splits;
};
// Waves of a block, blocks along the columns, and splits of the `other` tiles
// where the blocks alone would not fill the card.
Tiling tile_columns(int64_t columns, int64_t pairs, int64_t other)
{
    Tiling t;
    t.waves = columns <= 32 ? 1 : 4;
    t.tiles = (int)((columns + t.waves * 32 - 1) / (t.waves * 32));
    const int64_t blocks = std::max<int64_t>(1, pairs * t.tiles), target = t.waves == 1 ? 1024 : 512;
    t.splits = (int)std::max<int64_t>(1, std::min<int64_t>({target / blocks, other / 2, 256}));
    return t;
}

int tile_rows(const gs_attention *p) { return p->dtype == GS_DTYPE_F32 && p->d > 32 ? 32 : 64; }

bool direct_ok(const gs_attention *p, const void *t, int64_t sb, int64_t sr, int64_t sh, int rows, int heads)
{
    if (p->dtype == GS_DTYPE_F32 || p->d % 8 || !aligned_to(t, 16)) return false;
    if ((p->batch > 1 && sb % 8) || (heads > 1 && sh % 8)) return false;
    return rows <= 1 || (sr % 8 == 0 && sr < (1 << 23));
}

struct Piece {                                  // an operand of the tiles: in place, or where it is packed
    bool packed;
    size_t at;
};
struct Plan {
    Tiling t;                                   // of the forward, or of dq
    Tiling tkv;
    Piece k, v, q, g;
    size_t lse2, delta, part, part2, ml, bytes;
    int nq_pad;
};

size_t packed_bytes(const gs_attention *p, int rows, int heads)
{
    return round256((size_t)p->batch * heads * rows * ((p->d + 7) / 8 * 8) * 2 * (p->dtype == GS_DTYPE_F32 ? 3 : 1));
}

void place(Plan &w, Piece &piece, const gs_attention *p, const void *t, int64_t sb, int64_t sr, int64_t sh, int rows, int heads)
{
    piece.packed = rows > 0 && !direct_ok(p, t, sb, sr, sh, rows, heads);
    piece.at = w.bytes;
    if (piece.packed) w.bytes += packed_bytes(p, rows, heads);
}

// Places of partial sums in a split, and the bytes of all.
size_t places(const gs_attention *p, const Tiling &t) { return (size_t)p->batch * p->kv_heads * t.tiles * t.waves; }
int padded(int d) { return (d + 31) / 32 * 32; }
size_t part_bytes(const gs_attention *p, const Tiling &t) { return t.splits * places(p, t) * 32 * padded(p->d) * 4; }

Plan plan_fwd(const gs_attention *p)
{
    Plan w = {};
    const int kt = tile_rows(p);
    w.t = tile_columns((int64_t)p->nq * (p->heads / p->kv_heads), (int64_t)p->batch * p->kv_heads, (p->nk + kt - 1) / kt);
    place(w, w.k, p, p->k, p->k_batch, p->k_row, p->k_head, p->nk, p->kv_heads);
    place(w, w.v, p, p->v, p->v_batch, p->v_row, p->v_head, p->nk, p->kv_heads);
    if (w.t.splits > 1) {
        w.part = w.bytes;
        w.bytes += part_bytes(p, w.t);
        w.ml = w.bytes;
        w.bytes += (size_t)w.t.splits * places(p, w.t) * 32 * 8;
    }
    return w;
}

Plan plan_bwd(const gs_attention *p, const gs_attention_grads *g)
{
    Plan w = {};
    const int kt = tile_rows(p), group = p->heads / p->kv_heads;
    const int64_t pairs = (int64_t)p->batch * p->kv_heads;
    w.nq_pad = (p->nq + 63) / 64 * 64;
    w.t = tile_columns((int64_t)p->nq * group, pairs, (p->nk + kt - 1) / kt);
    w.tkv = tile_columns(p->nk, pairs, (int64_t)(p->nq + kt - 1) / kt * group);
    w.lse2 = 0;
    const size_t stat = round256((size_t)p->batch * p->heads * w.nq_pad * 4);
    w.delta = stat;
    w.bytes = 2 * stat;
    size_t part = 0;
    if (g->dq) {
        place(w, w.k, p, p->k, p->k_batch, p->k_row, p->k_head, p->nk, p->kv_heads);
        place(w, w.v, p, p->v, p->v_batch, p->v_row, p->v_head, p->nk, p->kv_heads);
        if (w.t.splits > 1) part = part_bytes(p, w.t);
    }
    w.part = w.part2 = w.bytes;
    if (g->dk || g->dv) {
        place(w, w.q, p, p->q, p->q_batch, p->q_row, p->q_head, p->nq, p->heads);
        place(w, w.g, p, g->dout, g->dout_batch, g->dout_row, g->dout_head, p->nq, p->heads);
        w.part = w.part2 = w.bytes;
        if (w.tkv.splits > 1) {
            const size_t one = part_bytes(p, w.tkv);
            part = std::max(part, 2 * one);
            w.part2 = w.part + one;
        }
    }
    w.bytes += part;
    return w;
}

// ---- checks ----------------------------------------------------------------------------
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }

bool strides_ok(const void *p, int es, int64_t sb, int64_t sr, int64_t sh) { return aligned_to(p, es) && sb >= 0 && sr >= 0 && sh >= 0; }

// Whether the elements of a result all have places of their own.
bool apart(const gs_attention *p, int64_t sb, int64_t sr, int64_t sh, int rows, int heads)
{
    struct {
        int64_t stride, count;
    } dim[3] = {{sb, p->batch}, {sr, rows}, {sh, heads}};
    std::sort(dim, dim + 3, [](const auto &x, const auto &y) { return x.stride < y.stride; });
    __int128 extent = p->d;
    for (const auto &x : dim) {
        if (x.count <= 1) continue;
        if (x.stride < extent) return false;
        extent += (__int128)x.stride * (x.count - 1);
    }
    return true;
}

gs_status check(const gs_attention *p)
{
    if (!p) return GS_ERR_INVALID_ARG;
    if (p->batch < 0 || p->batch > 65535 || p->heads < 1 || p->heads > 65535 || p->kv_heads < 1 || p->heads % p->kv_heads) return GS_ERR_INVALID_ARG;
    if (p->nq < 0 || p->nq > (1 << 30) || p->nk < 0 || p->nk > (1 << 30) || p->d < 1 || !float_type(p->dtype)) return GS_ERR_INVALID_ARG;
    if (!(p->scale > 0.0f) || !(p->scale < INFINITY)) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(p->dtype);
    if (!strides_ok(p->q, es, p->q_batch, p->q_row, p->q_head) || !strides_ok(p->k, es, p->k_batch, p->k_row, p->k_head) ||
        !strides_ok(p->v, es, p->v_batch, p->v_row, p->v_head) || !strides_ok(p->out, es, p->out_batch, p->out_row, p->out_head))
        return GS_ERR_INVALID_ARG;
    if (!aligned_to(p->lse, 4) || !aligned_to(p->kv_lengths, 4) || (p->kv_mask && p->kv_mask_stride < 0)) return GS_ERR_INVALID_ARG;
    if (p->batch > 0 && p->nk > 0 && (!p->k || !p->v)) return GS_ERR_INVALID_ARG;
    if (p->batch > 0 && p->nq > 0 && (!p->q || !p->out)) return GS_ERR_INVALID_ARG;
    if (p->d > kMaxD || (int64_t)p->nq * (p->heads / p->kv_heads) > (1 << 30)) return GS_ERR_UNSUPPORTED;
    if ((int64_t)p->batch * p->heads * std::max(p->nq, p->nk) > ((int64_t)1 << 40)) return GS_ERR_UNSUPPORTED;
    return GS_OK;
}

gs_status check_grads(const gs_attention *p, const gs_attention_grads *g)
{
    const gs_status st = check(p);
    if (st != GS_OK) return st;
    if (!g) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(p->dtype);
    if (p->batch > 0 && p->nq > 0 && (!g->dout || !p->lse)) return GS_ERR_INVALID_ARG;
    if (!strides_ok(g->dout, es, g->dout_batch, g->dout_row, g->dout_head) || !strides_ok(g->dq, es, g->dq_batch, g->dq_row, g->dq_head) ||
        !strides_ok(g->dk, es, g->dk_batch, g->dk_row, g->dk_head) || !strides_ok(g->dv, es, g->dv_batch, g->dv_row, g->dv_head))
        return GS_ERR_INVALID_ARG;
    if ((g->dq && !apart(p, g->dq_batch, g->dq_row, g->dq_head, p->nq, p->heads)) ||
        (g->dk && !apart(p, g->dk_batch, g->dk_row, g->dk_head, p->nk, p->kv_heads)) ||
        (g->dv && !apart(p, g->dv_batch, g->dv_row, g->dv_head, p->nk, p->kv_heads)))
        return GS_ERR_INVALID_ARG;
    return GS_OK;
}

// ---- launches ----------------------------------------------------------------------------
Args args_of(const gs_attention *p)
{
    Args a = {};
    a.q = {p->q, p->q_batch, p->q_row, p->q_head};
    a.out = {p->out, p->out_batch, p->out_row, p->out_head};
    a.kt = {p->k, p->k_batch, p->k_row, p->k_head};
    a.vt = {p->v, p->v_batch, p->v_row, p->v_head};
    a.lse = p->lse;
    a.lengths = p->kv_lengths;
    a.mask = p->kv_mask;
    a.mask_stride = p->kv_mask_stride;
    a.batch = p->batch;
    a.heads = p->heads;
    a.kv = p->kv_heads;
    a.group = p->heads / p->kv_heads;
    a.nq = p->nq;
    a.nk = p->nk;
    a.nq_pad = (p->nq + 63) / 64 * 64;
    a.d = p->d;
    a.rows = p->nq * a.group;
    a.type = p->dtype;
    a.scale = p->scale;
    a.c = p->scale * kLog2e;
    return a;
}

// The operand as the tiles are loaded, packed first where it has to be.
hipError_t operand(const gs_attention *p, const Tensor &t, int rows, int heads, const Piece &piece, char *ws, Operand &o, hipStream_t s)
{
    if (!piece.packed) {
        o = {static_cast<const char *>(t.p), t.sb * 2, t.sr * 2, t.sh * 2, 0};
        return hipSuccess;
    }
    const int dp = (p->d + 7) / 8 * 8;
    const int64_t row = dp * 2, plane = (int64_t)p->batch * heads * rows * row;
    o = {ws + piece.at, heads * (int64_t)rows * row, row, (int64_t)rows * row, plane};
    PackArgs a = {t, ws + piece.at, plane / 2, rows, heads, p->batch * heads, p->d, dp / 8, p->dtype};
    const dim3 grid((unsigned)(((int64_t)rows * a.chunks + kThreads - 1) / kThreads), (unsigned)std::min(a.pairs, 65535));
    if (p->dtype == GS_DTYPE_F32) pack<3><<<grid, kThreads, 0, s>>>(a);
    else pack<1><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

void tile(Args &a, const Tiling &t)
{
    a.tiles = t.tiles;
    a.splits = t.splits;
    a.waves = t.waves;
    const int64_t pairs = (int64_t)a.batch * a.kv * t.splits, want = (64 + pairs - 1) / pairs;      // runs: 64 or more
    a.run = (int)((t.tiles + want - 1) / want);
    const int64_t parts = (t.tiles + a.run - 1) / a.run;
    a.blocks = (pairs * parts + 7) / 8 * 8 * a.run;
}

// Joins the splits of what `t` tiled: `rows` rows of a pair, `group` heads of them
// to a token, into `to`.
hipError_t launch_join(const Args &a, const float *part, const float *ml, const Tensor &to, int rows, int group, int heads, hipStream_t s)
{
    JoinArgs j = {part, ml, to, ml ? a.lse : nullptr, 0, 0, padded(a.d) / 8, rows, a.tiles, a.waves, group, heads, a.splits, a.d, a.type};
    j.waves = (int64_t)a.batch * a.kv * a.tiles * a.waves;
    j.units = j.waves * j.per;
    const bool wide = a.splits > 8;             // four waves to a unit
    const dim3 grid = grid_of(wide ? j.units : (j.units + 3) / 4, kThreads);
    if (ml && wide) join_splits<4, true><<<grid, kThreads, 0, s>>>(j);
    else if (ml) join_splits<1, true><<<grid, kThreads, 0, s>>>(j);
    else if (wide) join_splits<4, false><<<grid, kThreads, 0, s>>>(j);
    else join_splits<1, false><<<grid, kThreads, 0, s>>>(j);
    return hipGetLastError();
}

}  // namespace
}  // namespace attn
}  // namespace gsi

using namespace gsi;
using namespace gsi::attn;

extern "C" {

size_t gs_attention_fwd_workspace_bytes(const gs_attention *p)
{
    return check(p) == GS_OK && p->batch > 0 && p->nq > 0 ? plan_fwd(p).bytes : 0;
}

gs_status gs_attention_fwd(const gs_attention *p, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = check(p);
    if (st != GS_OK) return st;
    if (!apart(p, p->out_batch, p->out_row, p->out_head, p->nq, p->heads)) return GS_ERR_INVALID_ARG;
    if (p->batch == 0 || p->nq == 0) return GS_OK;
    const Plan w = plan_fwd(p);
    if (workspace_bytes < w.bytes) return GS_ERR_WORKSPACE;
    if (w.bytes && (!workspace || !aligned_to(workspace, 16))) return GS_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    char *ws = static_cast<char *>(workspace);
    Args a = args_of(p);
    hipError_t e = operand(p, a.kt, p->nk, p->kv_heads, w.k, ws, a.k, s);
    if (e == hipSuccess) e = operand(p, a.vt, p->nk, p->kv_heads, w.v, ws, a.v, s);
    if (e != hipSuccess) return from_hip(e);
    tile(a, w.t);
    a.part = reinterpret_cast<float *>(ws + w.part);
    a.ml = reinterpret_cast<float *>(ws + w.ml);
    e = p->dtype == GS_DTYPE_F32 ? launch_fwd_f32(a, w.t.waves, s) : p->dtype == GS_DTYPE_F16 ? launch_fwd_f16(a, w.t.waves, s) : launch_fwd_bf16(a, w.t.waves, s);
    if (e == hipSuccess && a.splits > 1) e = launch_join(a, a.part, a.ml, a.out, a.rows, a.group, a.heads, s);
    return from_hip(e);
}

size_t gs_attention_bwd_workspace_bytes(const gs_attention *p, const gs_attention_grads *g)
{
    return check_grads(p, g) == GS_OK && p->batch > 0 ? plan_bwd(p, g).bytes : 0;
}

gs_status gs_attention_bwd(const gs_attention *p, const gs_attention_grads *g, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = check_grads(p, g);
    if (st != GS_OK) return st;
    if (p->batch == 0) return GS_OK;
    const Plan w = plan_bwd(p, g);
    if (workspace_bytes < w.bytes) return GS_ERR_WORKSPACE;
    if (w.bytes && (!workspace || !aligned_to(workspace, 16))) return GS_ERR_INVALID_ARG;
    hipStream_t s = (hipStream_t)stream;
    char *ws = static_cast<char *>(workspace);
    Args a = args_of(p);
    a.dout = {g->dout, g->dout_batch, g->dout_row, g->dout_head};
    a.dq = {g->dq, g->dq_batch, g->dq_row, g->dq_head};
    a.dk = {g->dk, g->dk_batch, g->dk_row, g->dk_head};
    a.dv = {g->dv, g->dv_batch, g->dv_row, g->dv_head};
    a.lse2 = reinterpret_cast<float *>(ws + w.lse2);
    a.delta = reinterpret_cast<float *>(ws + w.delta);
    a.part = reinterpret_cast<float *>(ws + w.part);
    a.part2 = reinterpret_cast<float *>(ws + w.part2);
    hipError_t e = hipSuccess;
    if (p->nq > 0) {
        const dim3 grid((unsigned)(a.nq_pad / (kThreads / 16)), (unsigned)std::min<int64_t>((int64_t)p->batch * p->heads, 65535));
        row_statistics<<<grid, kThreads, 0, s>>>(a, reinterpret_cast<float *>(ws + w.lse2), reinterpret_cast<float *>(ws + w.delta),
                                                 p->dtype == GS_DTYPE_F16 ? kHalfShift : 0.0f);
        e = hipGetLastError();
    }
    if (e == hipSuccess && g->dq && p->nq > 0) {
        e = operand(p, a.kt, p->nk, p->kv_heads, w.k, ws, a.k, s);
        if (e == hipSuccess) e = operand(p, a.vt, p->nk, p->kv_heads, w.v, ws, a.v, s);
        tile(a, w.t);
        if (e == hipSuccess)
            e = p->dtype == GS_DTYPE_F32 ? launch_dq_f32(a, w.t.waves, s) : p->dtype == GS_DTYPE_F16 ? launch_dq_f16(a, w.t.waves, s) : launch_dq_bf16(a, w.t.waves, s);
        if (e == hipSuccess && a.splits > 1) e = launch_join(a, a.part, nullptr, a.dq, a.rows, a.group, a.heads, s);
    }
    if (e == hipSuccess && (g->dk || g->dv) && p->nk > 0) {
        e = operand(p, a.q, p->nq, p->heads, w.q, ws, a.qt, s);
        if (e == hipSuccess) e = operand(p, a.dout, p->nq, p->heads, w.g, ws, a.dot, s);
        tile(a, w.tkv);
        if (e == hipSuccess)
            e = p->dtype == GS_DTYPE_F32 ? launch_dkv_f32(a, w.tkv.waves, s) : p->dtype == GS_DTYPE_F16 ? launch_dkv_f16(a, w.tkv.waves, s) : launch_dkv_bf16(a, w.tkv.waves, s);
        if (e == hipSuccess && a.splits > 1) {
            if (g->dk) e = launch_join(a, a.part, nullptr, a.dk, p->nk, 1, a.kv, s);
            if (e == hipSuccess && g->dv) e = launch_join(a, a.part2, nullptr, a.dv, p->nk, 1, a.kv, s);
        }
    }
    return from_hip(e);
}

}  // extern "C"
