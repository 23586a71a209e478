// Cross attention: argument checks, the choice of launches, and the small
// kernels around the main ones (gs_attention_fwd.h, gs_attention_bwd.h): packed
// copies of operands that cannot be loaded directly, the backward's row
// statistics, and the joining of splits.
#include "gs_attention.h"

#include <math.h>

#include <algorithm>

namespace gsi {
namespace attn {

hipError_t launch_fwd_bf16(const Args &, hipStream_t);
hipError_t launch_fwd_f16(const Args &, hipStream_t);
hipError_t launch_fwd_f32(const Args &, hipStream_t);
hipError_t launch_bwd_bf16(const Args &, int, hipStream_t);
hipError_t launch_bwd_f16(const Args &, int, hipStream_t);
hipError_t launch_bwd_f32(const Args &, int, hipStream_t);

namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 128;
constexpr int kCus = 256;

gs_status from_hip(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }
bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
constexpr size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

// ---- what comes before the products ---------------------------------------------
// One launch for up to four packed operands and the backward's row statistics; a
// row is 2^lanes lanes', eight values each.  4 to 5 us, most of it the launch.  fp32
// limbs are made here once: split by every workgroup that stages them, the main
// kernels took up to twice as long.
struct PackJob {                                // [limb][batch][heads][n][dp] of 16 bits from any strides
    Tensor from;
    char *to;
    int64_t plane;                              // values of a limb
    int n, heads;
    uint32_t first, per;                        // first block; blocks of a batch element and head
};
struct Prepare {
    PackJob jobs[4];
    int count, d, chunks, lanes, type;          // chunks: of eight values in a packed row
    // statistics: delta = dout . out, and lse (of 16-bit types in units of log 2, times
    // `shift` powers of it) with what keeps P of an empty or absent row at 0
    Tensor out, dout;
    const float *lse;
    float *lse2, *delta;
    float shift;
    int nq, nq_pad, heads;
    uint32_t first, per, blocks;                // blocks: of the launch
};

template <int NL> __device__ __forceinline__ void pack_row(const Prepare &a, const PackJob &job, uint32_t block)
{
    const uint32_t pair = block / job.per;
    const int at = (int)(threadIdx.x & ((1u << a.lanes) - 1)) * 8;
    const int64_t row = (int64_t)(block - pair * job.per) * (kThreads >> a.lanes) + (threadIdx.x >> a.lanes);
    if (row >= job.n || at >= a.chunks * 8) return;
    const uint32_t batch = pair / (uint32_t)job.heads, head = pair - batch * job.heads;
    const int64_t from = batch * job.from.sb + row * job.from.sr + head * job.from.sh + at;
    const int64_t to = ((int64_t)pair * job.n + row) * a.chunks * 8 + at;
    const int valid = min(8, a.d - at);
    if constexpr (NL > 1) {
        float v[8];
        load8(job.from.p, GS_DTYPE_F32, from, valid, v);
        Vec<uint16_t, 8> w[NL];
        split_all<NL, 8>(v, w);
#pragma unroll
        for (int l = 0; l < NL; l++) *reinterpret_cast<Vec<uint16_t, 8> *>(job.to + (l * job.plane + to) * 2) = w[l];
    } else {
        Vec<uint16_t, 8> w = {{0, 0, 0, 0, 0, 0, 0, 0}};
        const uint16_t *p = static_cast<const uint16_t *>(job.from.p) + from;
        if (valid == 8) w = *reinterpret_cast<const Vec<uint16_t, 8> *>(p);
        else
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j < valid) w.v[j] = p[j];
        *reinterpret_cast<Vec<uint16_t, 8> *>(job.to + to * 2) = w;
    }
}

__global__ __launch_bounds__(kThreads) void prepare(Prepare a)
{
    uint32_t b = (uint32_t)block_of();
    if (b < a.first) {
        int k = 0;
#pragma unroll
        for (int i = 1; i < 4; i++)
            if (i < a.count && b >= a.jobs[i].first) k = i;
        const PackJob &job = a.jobs[k];
        if (a.type == GS_DTYPE_F32) pack_row<3>(a, job, b - job.first);
        else pack_row<1>(a, job, b - job.first);
        return;
    }
    b -= a.first;
    if (!a.per) return;
    const uint32_t pair = b / a.per;
    const int64_t token = (int64_t)(b - pair * a.per) * (kThreads >> a.lanes) + (threadIdx.x >> a.lanes);
    const uint32_t batch = pair / (uint32_t)a.heads, head = pair - batch * a.heads;
    if (token >= a.nq_pad || a.first + b >= a.blocks) return;
    const int at = (int)(threadIdx.x & ((1u << a.lanes) - 1)) * 8;
    float dot = 0.0f;
    if (token < a.nq && at < a.d) {
        float x[8], y[8];
        load8(a.out.p, a.type, batch * a.out.sb + token * a.out.sr + head * a.out.sh + at, a.d - at, x);
        load8(a.dout.p, a.type, batch * a.dout.sb + token * a.dout.sr + head * a.dout.sh + at, a.d - at, y);
#pragma unroll
        for (int i = 0; i < 8; i++) dot = fmaf(x[i], y[i], dot);
    }
    for (int o = 1 << a.lanes >> 1; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
    if (at == 0) {
        const float l = token < a.nq ? a.lse[(int64_t)pair * a.nq + token] : -INFINITY;
        const int64_t to = (int64_t)pair * a.nq_pad + token;
        a.lse2[to] = l == -INFINITY ? INFINITY : a.type == GS_DTYPE_F32 ? l : fmaf(l, kLog2e, -a.shift);
        a.delta[to] = dot;
    }
}

// ---- splits -----------------------------------------------------------------------
// A unit is 16 bytes a lane of the 64 lanes that hold 32 rows' sums; its SW waves
// take every SW-th split, the first of them adds theirs, in order.  Bound by reading
// sums that other dies have just written: 34 MB in 12.6 us, 2.8 TB/s.
struct JoinJob {
    const float *part, *ml;
    Tensor to;
    float *lse;
    int64_t waves, first;                       // waves' places in a split; first unit
    int rows, tiles, wide, group, heads, splits;        // rows of a pair; wide: waves of a block
};
struct JoinArgs {
    JoinJob jobs[3];
    int64_t units;                              // of all jobs
    int count, per, d, type;                    // per: units of a wave
};
// Where a unit's lane writes: its row's place in the tensor, or not.
struct Target {
    bool there;
    int at;                                     // first of four d
    int64_t row, stat;                          // elements; index into lse
};
__device__ __forceinline__ Target target_of(const JoinJob &a, int64_t wave, int unit, int lane)
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
__device__ __forceinline__ void store4(const JoinArgs &a, const Tensor &tensor, const Target &t, const gemm::f4 &v)
{
    void *to = const_cast<void *>(tensor.p);
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

// Partial softmaxes (sums relative to their own maxima; NL as power() takes it), or plain sums (NL 0).
template <int SW, int NL> __global__ __launch_bounds__(kThreads) void join_splits(JoinArgs a)
{
    constexpr int kUnits = kThreads / 64 / SW;
    __shared__ gemm::f4 turn[SW > 1 ? kThreads : 1];
    __shared__ float2 stats[SW > 1 ? kThreads : 1];
    const int lane = threadIdx.x & 63, sub = (threadIdx.x >> 6) % SW;
    const int64_t u = block_of() * kUnits + (threadIdx.x >> 6) / SW;
    const bool works = u < a.units;
    int k = 0;
#pragma unroll
    for (int i = 1; i < 3; i++)
        if (i < a.count && u >= a.jobs[i].first) k = i;
    const JoinJob &job = a.jobs[__builtin_amdgcn_readfirstlane(k)];         // a wave is of one unit
    const int64_t wave = works ? (u - job.first) / a.per : 0;
    const int unit = works ? (int)(u - job.first - wave * a.per) : 0, splits = works ? job.splits : 0;
    const gemm::f4 *part = reinterpret_cast<const gemm::f4 *>(job.part) + (wave * a.per + unit) * 64 + lane;
    const float2 *ml = reinterpret_cast<const float2 *>(job.ml) + wave * 32 + (lane & 31);
    const int64_t next = job.waves * a.per * 64, next_ml = job.waves * 32;
    gemm::f4 v = {0, 0, 0, 0};
    constexpr bool SOFT = NL > 0;
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
                    const float f = w[i].x == -INFINITY && w[i].y != 0.0f ? 1.0f : power<NL>(w[i].x - base);
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
    const Target t = target_of(job, wave, unit, lane);
    if constexpr (SOFT) {
        v *= m == -INFINITY && sum == 0.0f ? 0.0f : 1.0f / sum;
        if (job.lse && t.there && unit == 0 && lane < 32) job.lse[t.stat] = lse_of<NL>(m, sum);
    }
    store4(a, job.to, t, v);
}

// ---- plan ----------------------------------------------------------------------------
struct Tiling {
    int waves, tiles, splits;
};
// Time of one tile of the other side's rows on a CU that holds one block, and per
// tile where it holds two or more (us; blocks of four waves; 64 rows, or 32 of fp32
// above d = 32), and how many it holds.  Measured.
struct Cost {
    double alone, shared;
    int hold;
};
enum Product { kForward, kQueries, kStates };

Cost cost_of(const gs_attention *p, Product what)
{
    static const Cost h[3][4] = {{{0.8, 0.52, 4}, {1.05, 0.7, 3}, {1.3, 0.95, 2}, {1.45, 1.1, 2}},
                                 {{0.95, 0.63, 4}, {1.25, 0.95, 3}, {1.8, 1.35, 2}, {1.95, 1.63, 2}},
                                 {{1.35, 0.77, 4}, {2.0, 1.29, 3}, {2.2, 1.6, 2}, {4.7, 2.5, 2}}};
    static const Cost f[3][4] = {{{2.1, 1.58, 2}, {1.65, 1.32, 2}, {2.25, 2.25, 1}, {2.8, 2.8, 1}},
                                 {{2.5, 2.1, 2}, {2.2, 2.2, 1}, {3.15, 3.15, 1}, {4.05, 4.05, 1}},
                                 {{3.7, 2.95, 2}, {3.0, 3.0, 1}, {4.1, 4.1, 1}, {5.1, 5.1, 1}}};
    const int i = p->d <= 32 ? 0 : p->d <= 64 ? 1 : p->d <= 96 ? 2 : 3;
    return p->dtype == GS_DTYPE_F32 ? f[what][i] : h[what][i];
}

// A wave has 32 columns.
int waves_for(int64_t columns) { return columns <= 32 ? 1 : 4; }

int padded(int d) { return (d + 31) / 32 * 32; }

// One kind of blocks: `blocks` of them, each of whose splits walks over a share of
// the `other` side's tiles.
struct Work {
    Tiling t;
    Cost cost;
    int64_t blocks, other;
    double part;                                // us to write and join a split's partial sums
};
Work work_of(const gs_attention *p, Product what, int waves, int64_t columns, int64_t pairs, int64_t other)
{
    Work w = {};
    w.t = {waves, (int)((columns + waves * 32 - 1) / (waves * 32)), 1};
    w.cost = cost_of(p, what);
    // single waves: a quarter of the work, and less to hide it behind.  One estimate for every
    // type and width, though LDS lets four and more of 16 bits and d <= 64 share a CU, three
    // of fp32 and d <= 64, two of 16 bits above and one of fp32 above
    if (waves == 1) w.cost = {1.2, w.cost.shared / 4, 4};
    w.blocks = pairs * w.t.tiles;
    w.other = other;
    w.part = 0.03 + (double)w.blocks * waves * 32 * padded(p->d) * 4 * 2 * (what == kStates ? 2 : 1) / 7e6;
    return w;
}
int64_t tiles_of(int64_t other, int64_t splits) { return (other + splits - 1) / splits; }

// Time of w's blocks in s splits each and then of v's in u: blocks go to the first
// place that is free, as many to a CU as it holds.
double time_of(const Work &w, int64_t s, const Work *v, int64_t u)
{
    const int64_t n = w.blocks * s, m = v ? v->blocks * u : 0;
    const int64_t hold = std::min<int64_t>(v ? std::min(w.cost.hold, v->cost.hold) : w.cost.hold, (n + m + kCus - 1) / kCus), places = kCus * std::max<int64_t>(1, hold);
    auto one = [&](const Work &x, int64_t splits) { return tiles_of(x.other, splits) * (hold <= 1 ? x.cost.alone : std::max(x.cost.alone, x.cost.shared * hold)) + 2.0; };
    const double dn = one(w, s), dm = v ? one(*v, u) : 0.0;
    const int64_t rounds = n / places, left = n % places;
    double early = rounds * dn, late = early + (left ? dn : 0.0);       // when `places - left` and `left` places are free
    int64_t rest = m;
    while (rest > 0) {
        if (left == 0 || early <= late) {
            rest -= places - left;
            early += dm;
        } else {
            rest -= left;
            late += dm;
        }
    }
    double time = std::max(early, late);
    if (s > 1 || u > 1) time += 3.5;
    if (s > 1) time += s * w.part;
    if (u > 1) time += u * v->part;
    return time;
}

// Splits of one or both kinds of blocks (v: NULL, or the second kind) where the blocks
// alone would not fill the card: those of the least estimated time.
void choose_splits(Work *w, Work *v)
{
    static const int tried[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64, 96, 128, 192, 256};
    constexpr int64_t kMostBlocks = 2048;       // more need no splits
    double best = 0;
    const Work a = *w, b = v ? *v : Work{};
    for (int s : tried) {
        const int64_t ss = (a.other + tiles_of(a.other, s) - 1) / std::max<int64_t>(1, tiles_of(a.other, s));
        if (s > 1 && (s > a.other || a.blocks * s > kMostBlocks || (ss != s && s <= 4))) continue;
        for (int u : tried) {
            if (u > 1 && (!v || u > b.other || b.blocks * u > kMostBlocks)) break;
            const int64_t uu = v ? (b.other + tiles_of(b.other, u) - 1) / std::max<int64_t>(1, tiles_of(b.other, u)) : 1;
            const double time = time_of(a, std::max<int64_t>(1, ss), v ? &b : nullptr, std::max<int64_t>(1, uu));
            if (best == 0 || time < best) {
                best = time;
                w->t.splits = (int)std::max<int64_t>(1, ss);
                if (v) v->t.splits = (int)std::max<int64_t>(1, uu);
            }
        }
    }
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
    Tiling tk;
    Piece k, v, q, g;
    size_t lse2, delta, part, part_k, part_v, ml, bytes;
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
size_t part_bytes(const gs_attention *p, const Tiling &t) { return t.splits * places(p, t) * 32 * padded(p->d) * 4; }

Plan plan_fwd(const gs_attention *p)
{
    Plan w = {};
    const int kt = tile_rows(p);
    const int64_t rows = (int64_t)p->nq * (p->heads / p->kv_heads);
    Work fwd = work_of(p, kForward, waves_for(rows), rows, (int64_t)p->batch * p->kv_heads, (p->nk + kt - 1) / kt);
    choose_splits(&fwd, nullptr);
    w.t = fwd.t;
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
    const size_t stat = round256((size_t)p->batch * p->heads * w.nq_pad * 4);
    w.delta = stat;
    w.bytes = 2 * stat;
    const bool queries = g->dq && p->nq > 0, states = (g->dk || g->dv) && p->nk > 0;
    // one launch: blocks of as many waves, first those of dk and dv
    const int waves = std::max(queries ? waves_for((int64_t)p->nq * group) : 1, states ? waves_for(p->nk) : 1);
    Work dq = work_of(p, kQueries, waves, (int64_t)p->nq * group, pairs, (p->nk + kt - 1) / kt);
    Work dkv = work_of(p, kStates, waves, p->nk, pairs, (int64_t)(p->nq + kt - 1) / kt * group);
    if (states) choose_splits(&dkv, queries ? &dq : nullptr);
    else if (queries) choose_splits(&dq, nullptr);
    if (queries) {
        w.t = dq.t;
        place(w, w.k, p, p->k, p->k_batch, p->k_row, p->k_head, p->nk, p->kv_heads);
        place(w, w.v, p, p->v, p->v_batch, p->v_row, p->v_head, p->nk, p->kv_heads);
        w.part = w.bytes;
        if (w.t.splits > 1) w.bytes += part_bytes(p, w.t);
    }
    if (states) {
        w.tk = dkv.t;
        place(w, w.q, p, p->q, p->q_batch, p->q_row, p->q_head, p->nq, p->heads);
        place(w, w.g, p, g->dout, g->dout_batch, g->dout_row, g->dout_head, p->nq, p->heads);
        w.part_k = w.part_v = w.bytes;
        if (w.tk.splits > 1) {
            w.part_v += part_bytes(p, w.tk);
            w.bytes += 2 * part_bytes(p, w.tk);
        }
    }
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
    if ((int64_t)p->batch * p->heads * std::max(std::max(p->nq, p->nk), 32) > ((int64_t)1 << 33)) return GS_ERR_UNSUPPORTED;   // block numbers have 32 bits
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

// The operand as the tiles are loaded, with its packing among the jobs where it
// has to be packed first.
Operand operand(const gs_attention *p, const Tensor &t, int rows, int heads, const Piece &piece, char *ws, Prepare &pre)
{
    if (!piece.packed) return {static_cast<const char *>(t.p), t.sb * 2, t.sr * 2, t.sh * 2, 0};
    const int64_t row = pre.chunks * 16, plane = (int64_t)p->batch * heads * rows * row, lines = kThreads >> pre.lanes;
    PackJob &job = pre.jobs[pre.count++];
    job = {t, ws + piece.at, plane / 2, rows, heads, pre.blocks, (uint32_t)((rows + lines - 1) / lines)};
    pre.blocks += job.per * (uint32_t)(p->batch * heads);
    pre.first = pre.blocks;
    return {ws + piece.at, heads * (int64_t)rows * row, row, (int64_t)rows * row, plane};
}
Prepare prepare_of(const gs_attention *p)
{
    Prepare pre = {};
    pre.d = p->d;
    pre.type = p->dtype;
    pre.chunks = (p->d + 7) / 8;
    while ((1 << pre.lanes) < pre.chunks) pre.lanes++;
    pre.heads = p->heads;
    return pre;
}
hipError_t launch_prepare(const Prepare &pre, hipStream_t s)
{
    if (!pre.blocks) return hipSuccess;
    prepare<<<grid_of(pre.blocks, kThreads), kThreads, 0, s>>>(pre);
    return hipGetLastError();
}

Grid grid_for(const gs_attention *p, const Tiling &t)
{
    const int64_t pairs = (int64_t)p->batch * p->kv_heads * t.splits, want = (64 + pairs - 1) / pairs;       // runs: 64 or more
    Grid g = {t.tiles, t.splits, (int)((t.tiles + want - 1) / want), t.waves, 0};
    const int64_t parts = (t.tiles + g.run - 1) / g.run;
    g.blocks = (uint32_t)((pairs * parts + 7) / 8 * 8 * g.run);
    return g;
}

// Adds the join of what `g` laid out to the jobs: `rows` rows of a pair, `group` heads
// of them to a token, into `to`.
void add_join(JoinArgs &j, const Args &a, const Grid &g, const float *part, const float *ml, const Tensor &to, int rows, int group, int heads)
{
    if (g.splits <= 1 || !to.p) return;
    JoinJob &job = j.jobs[j.count++];
    job = {part, ml, to, ml ? a.lse : nullptr, (int64_t)a.batch * a.kv * g.tiles * g.waves, j.units, rows, g.tiles, g.waves, group, heads, g.splits};
    j.units += job.waves * j.per;
}
hipError_t launch_join(const JoinArgs &j, bool soft, hipStream_t s)
{
    if (!j.count) return hipSuccess;
    bool wide = false;                          // four waves to a unit
    for (int i = 0; i < j.count; i++) wide = wide || j.jobs[i].splits > 8;
    const dim3 grid = grid_of(wide ? j.units : (j.units + 3) / 4, kThreads);
    if (soft && j.type == GS_DTYPE_F32) {
        if (wide) join_splits<4, 3><<<grid, kThreads, 0, s>>>(j);
        else join_splits<1, 3><<<grid, kThreads, 0, s>>>(j);
    } else if (soft) {
        if (wide) join_splits<4, 1><<<grid, kThreads, 0, s>>>(j);
        else join_splits<1, 1><<<grid, kThreads, 0, s>>>(j);
    } else if (wide) {
        join_splits<4, 0><<<grid, kThreads, 0, s>>>(j);
    } else {
        join_splits<1, 0><<<grid, kThreads, 0, s>>>(j);
    }
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
    Prepare pre = prepare_of(p);
    a.k = operand(p, a.kt, p->nk, p->kv_heads, w.k, ws, pre);
    a.v = operand(p, a.vt, p->nk, p->kv_heads, w.v, ws, pre);
    a.t = grid_for(p, w.t);
    a.part = reinterpret_cast<float *>(ws + w.part);
    a.ml = reinterpret_cast<float *>(ws + w.ml);
    JoinArgs j = {};
    j.per = padded(p->d) / 8;
    j.d = p->d;
    j.type = p->dtype;
    add_join(j, a, a.t, a.part, a.ml, a.out, a.rows, a.group, a.heads);
    hipError_t e = launch_prepare(pre, s);
    if (e == hipSuccess) e = p->dtype == GS_DTYPE_F32 ? launch_fwd_f32(a, s) : p->dtype == GS_DTYPE_F16 ? launch_fwd_f16(a, s) : launch_fwd_bf16(a, s);
    if (e == hipSuccess) e = launch_join(j, true, s);
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
    a.part_k = reinterpret_cast<float *>(ws + w.part_k);
    a.part_v = reinterpret_cast<float *>(ws + w.part_v);
    Prepare pre = prepare_of(p);
    JoinArgs j = {};
    j.per = padded(p->d) / 8;
    j.d = p->d;
    j.type = p->dtype;
    if (w.t.waves) {
        a.k = operand(p, a.kt, p->nk, p->kv_heads, w.k, ws, pre);
        a.v = operand(p, a.vt, p->nk, p->kv_heads, w.v, ws, pre);
        a.t = grid_for(p, w.t);
        add_join(j, a, a.t, a.part, nullptr, a.dq, a.rows, a.group, a.heads);
    }
    if (w.tk.waves) {
        a.qt = operand(p, a.q, p->nq, p->heads, w.q, ws, pre);
        a.dot = operand(p, a.dout, p->nq, p->heads, w.g, ws, pre);
        a.tk = grid_for(p, w.tk);
        add_join(j, a, a.tk, a.part_k, nullptr, a.dk, p->nk, 1, a.kv);
        add_join(j, a, a.tk, a.part_v, nullptr, a.dv, p->nk, 1, a.kv);
    }
    if (p->nq > 0) {
        const int lines = kThreads >> pre.lanes;
        pre.out = a.out;
        pre.dout = a.dout;
        pre.lse = a.lse;
        pre.lse2 = reinterpret_cast<float *>(ws + w.lse2);
        pre.delta = reinterpret_cast<float *>(ws + w.delta);
        pre.shift = p->dtype == GS_DTYPE_F16 ? kHalfShift : 0.0f;
        pre.nq = p->nq;
        pre.nq_pad = a.nq_pad;
        pre.per = (uint32_t)((a.nq_pad + lines - 1) / lines);
        pre.blocks += pre.per * (uint32_t)(p->batch * p->heads);
    }
    const int waves = std::max(w.t.waves, w.tk.waves);
    hipError_t e = launch_prepare(pre, s);
    if (e == hipSuccess && a.t.blocks + a.tk.blocks) e = p->dtype == GS_DTYPE_F32 ? launch_bwd_f32(a, waves, s) : p->dtype == GS_DTYPE_F16 ? launch_bwd_f16(a, waves, s) : launch_bwd_bf16(a, waves, s);
    if (e == hipSuccess) e = launch_join(j, false, s);
    return from_hip(e);
}

}  // extern "C"
