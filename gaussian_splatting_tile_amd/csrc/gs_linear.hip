// Linear layer: argument checks, choice of tile and split, and the passes
// around its products (see gs_gemm.h for the products themselves).
//
// Forward: one product, out[q][p] with p the contiguous index of y: rows take
// p = outputs (P = w, Q = x), planes take p = rows of x (P = x, Q = w), so both
// layouts are written with full-width stores and neither is transposed.
// Backward: dz = dy act'(z) and the partial sums of db in one pass over dy and
// z (skipped when dz is dy as it stands), then dx[m][k] = dz w and
// dw[n][k] = dz^T x, whose operands are read by columns where k is theirs.
//
// 16-bit operands: dz is rounded to their type, which lets both products load it
// straight into LDS.  That is as much error again as dx's own rounding (16384 x 4096 x
// 1024 with GELU in bf16: 2.3e-3 of the norm, 1.7e-3 with dz unrounded); two limbs of
// dz would keep it at twice the products' time, 240 us more of that call's 333.
//
// Operands that cannot be loaded into LDS as they stand (fp32, odd sizes,
// strides or alignments of 16-bit ones, 8-bit values for an fp32 result) go one
// of two ways.  Staged, the product converts while loading, once per tile
// across the result; packed, one pass first writes both operands as padded
// 16-bit planes (three bf16 limbs of fp32).  Staged is taken where the result's
// smaller side is at most 1024 (fp32; by columns 512), 256 (16 bits; by columns
// never) or 128 (8 bits).  Staged against packed in us: fp32 16384 x 1024 x 512
// 112 / 116, 4096 x 4096 x 1024 205 / 189, by columns 72519 x 512 x 832 465 / 466 and
// 20000 x 768 x 768 182 / 159; bf16 of odd sizes 72519 x 250 x 830 97 / 132, by columns
// 189 / 133; 8-bit 30000 x 91 x 192 17 / 25, 72519 x 250 x 800 129 / 99.
#include <string.h>

#include "gs_linear.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;

bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }
bool al16(const void *p) { return aligned_to(p, 16); }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// ---- choice of tile and split -----------------------------------------------
// Estimated time in microseconds of a tile choice: rounds of blocks over the
// 256 CUs, each CU working through its resident blocks at `rate`, plus what a
// split of k costs to reduce.  The rates are measured ones at full occupancy;
// one block by itself reaches `alone` of them.  What a block does before and
// after its product counts as 64 more of k, or `around` where blocks share or follow
// one another on a CU and all write at once (40000 x 1000 x 64 in bf16: 43 us by
// 256 tiles, 32 by 128, 48 by 64; 72519 x 512 x 832: 88, 81, 101).
struct TileRate { int size, resident; float mflop_us, alone; int around; };     // per CU

double product_cost(const TileRate &t, int64_t P, int64_t Q, int64_t K, int splits, float work)
{
    const double blocks = (double)((P + t.size - 1) / t.size) * (double)((Q + t.size - 1) / t.size) * splits;
    // many small blocks even out over the CUs
    const double per_cu = blocks > 512.0 * t.resident ? blocks / 256.0 + 0.5 : ceil(blocks / 256.0);
    const double tile = 2e-6 * t.size * t.size * (ceil((double)K / splits) + (per_cu >= t.resident ? t.around : 64)) * work;
    // the last few blocks of a CU leave some of its rate unused
    const double whole = floor(per_cu / t.resident) * t.resident, rest = per_cu - whole;
    const double filled = t.resident > 1 ? t.alone + (1.0 - t.alone) * (rest > 1.0 ? rest - 1.0 : 0.0) / (t.resident - 1.0) : 1.0;
    double us = tile / t.mflop_us * (whole + rest / filled);
    if (splits > 1) us += 3.0 + splits * (0.1 + (double)P * (double)Q * 4.0 / 6e6);
    return us;
}

ProductPlan make_plan(int64_t P, int64_t Q, int64_t K, bool pt, bool qt, bool staged, bool f32, int step_k, float work)
{
    static const TileRate direct[3] = {{256, 1, 4.9f, 1.0f, 350}, {128, 2, 4.1f, 0.68f, 300}, {64, 3, 2.4f, 0.87f, 200}};
    static const TileRate limbs[3] = {{256, 1, 0.0f, 1.0f, 64}, {128, 1, 4.8f, 1.0f, 64}, {64, 2, 3.9f, 0.6f, 64}};
    static const TileRate staged_[3] = {{256, 1, 0.0f, 1.0f, 64}, {128, 1, 4.4f, 1.0f, 128}, {64, 3, 3.7f, 0.38f, 64}};
    ProductPlan best{pt, qt, staged, 2, 1, 0.0};
    double least = 1e30;
    const int64_t nt = (K + step_k - 1) / step_k;
    // three limbs of a 256 tile exceed the LDS
    for (int tile = staged || f32 ? 1 : 0; tile < 3; tile++) {
        const TileRate &t = staged ? staged_[tile] : f32 ? limbs[tile] : direct[tile];
        for (int64_t want = 1; want <= 64 && want <= nt; want = want < 4 ? want + 1 : want * 2) {
            const int64_t per = (nt + want - 1) / want;
            const int splits = (int)((nt + per - 1) / per);
            const double us = product_cost(t, P, Q, K, splits, work);
            if (us < least * 0.98) {
                least = us;
                best.tile = tile;
                best.splits = splits;
            }
        }
    }
    best.us = least;
    return best;
}

// The same of the way for few rows, as measured: a workgroup takes 16 outputs,
// so without enough of them for every CU a long k is better split over tiles.
// One row of 16384 to 64 outputs in bf16 takes 20 us against 9.0 by tiles, to
// 4096 outputs 26 against 24.5; of 1024 to 4096 4.2 against 6.5.
double few_rows_cost(const gs_linear &l)
{
    const double per_k = l.dtype == GS_DTYPE_F32 ? 2.6e-3 : l.dtype == GS_DTYPE_MXFP8 ? 0.9e-3 : 1.3e-3;
    return 2.2 + per_k * l.k * (l.n > 4096 ? l.n / 4096.0 : 1.0);
}

// ---- operands as padded 16-bit planes -----------------------------------------
struct PackJob {
    const void *src;                    // [rows][cols] of `type`
    const uint8_t *scales;              // MXFP8
    int64_t ld, ld_scales, rows;
    int type, cols;
    uint16_t *dst;                      // [limbs][rows][ld_dst], zeros past cols
    int64_t ld_dst;
    int limbs, half;                    // 3: bf16 limbs of fp32; 1: bf16, or fp16 if half
    int64_t first;                      // the job's first thread
};
struct PackJobs {
    PackJob job[2];
    int count;
    int64_t threads;
};

__device__ __forceinline__ void store_planes(uint16_t *dst, int64_t plane, int64_t at, int limbs, int half, const float v[8])
{
    if (limbs == 1) {
        Vec<uint16_t, 8> w;
#pragma unroll
        for (int i = 0; i < 8; i++)
            w.v[i] = half ? __builtin_bit_cast(uint16_t, (_Float16)v[i]) : __builtin_bit_cast(uint16_t, (__bf16)v[i]);
        *reinterpret_cast<Vec<uint16_t, 8> *>(dst + at) = w;
        return;
    }
    Vec<uint16_t, 8> w[3];
    split_all<3, 8>(v, w);
#pragma unroll
    for (int l = 0; l < 3; l++) *reinterpret_cast<Vec<uint16_t, 8> *>(dst + l * plane + at) = w[l];
}

// A thread per 8 columns of a row.
__global__ __launch_bounds__(kThreads) void pack_operands(PackJobs jobs)
{
    const int64_t id = block_of() * kThreads + threadIdx.x;
    if (id >= jobs.threads) return;
    const PackJob j = jobs.count > 1 && id >= jobs.job[1].first ? jobs.job[1] : jobs.job[0];
    const int64_t groups = j.ld_dst / 8, at = id - j.first, r = at / groups;
    const int c = (int)(at - r * groups) * 8, valid = min(8, j.cols - c);
    float v[8];
    if (j.type == GS_DTYPE_MXFP8) {
        const uint8_t *b = static_cast<const uint8_t *>(j.src) + r * j.ld + c;
        const float f = e8m0_value(j.scales[r * j.ld_scales + (c >> 5)]);       // cols is a multiple of 32
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = e4m3_value(b[i]) * f;
    } else {
        load8(j.src, j.type, r * j.ld + c, valid, v);
    }
    store_planes(j.dst, j.rows * j.ld_dst, r * j.ld_dst + c, j.limbs, j.half, v);
}

void add_job(PackJobs &jobs, const void *src, int type, const uint8_t *scales, int64_t ld, int64_t ld_scales, int64_t rows, int cols,
             void *dst)
{
    PackJob &j = jobs.job[jobs.count++];
    j.src = src;
    j.scales = scales;
    j.ld = ld;
    j.ld_scales = ld_scales;
    j.rows = rows;
    j.type = type;
    j.cols = cols;
    j.dst = static_cast<uint16_t *>(dst);
    j.ld_dst = ((int64_t)cols + 7) & ~(int64_t)7;
    j.limbs = type == GS_DTYPE_F32 ? 3 : 1;
    j.half = type == GS_DTYPE_F16;
    j.first = jobs.threads;
    jobs.threads += rows * (j.ld_dst / 8);
}

hipError_t run_jobs(const PackJobs &jobs, hipStream_t s)
{
    if (jobs.count == 0) return hipSuccess;
    pack_operands<<<grid_of((jobs.threads + kThreads - 1) / kThreads, kThreads), kThreads, 0, s>>>(jobs);
    return hipGetLastError();
}

size_t packed_bytes(int type, int64_t rows, int64_t cols)
{
    return round256((size_t)(type == GS_DTYPE_F32 ? 3 : 1) * rows * ((cols + 7) & ~(int64_t)7) * 2);
}

// One product with its plan; everything but the workspace addresses.
enum Way { kDirect, kPacked, kStaged, kFew };

struct Product {
    gemm::Args a;
    LinearEpilogue::Args e;
    ProductPlan plan;
    int type;                           // gs_dtype of the operands as given
    Way way;
    bool pack_p, pack_q;
    size_t partial_bytes;
};

bool exact_results(const LinearEpilogue::Args &e) { return e.y_type == GS_DTYPE_F32 || (e.z && e.z_type == GS_DTYPE_F32); }

// The way of a product whose operands can (p_ok, q_ok) or cannot be loaded
// directly, then its tile and splits.
void finish_plan(Product &r, bool p_ok, bool q_ok)
{
    const bool pt = r.plan.pt, qt = r.plan.qt;
    const int least = r.a.P < r.a.Q ? r.a.P : r.a.Q;
    const int staged_up_to = r.type == GS_DTYPE_F32 ? (pt ? 512 : 1024) : r.type == GS_DTYPE_MXFP8 ? 128 : pt ? 0 : 256;
    r.way = p_ok && q_ok ? kDirect : least <= staged_up_to ? kStaged : kPacked;
    r.pack_p = r.way == kPacked && (!p_ok || r.type == GS_DTYPE_MXFP8);
    r.pack_q = r.way == kPacked && (!q_ok || r.type == GS_DTYPE_MXFP8);
    const bool mx = r.type == GS_DTYPE_MXFP8 && r.way == kDirect, f32 = r.type == GS_DTYPE_F32;
    const int step = mx ? 128 : r.way == kStaged || f32 ? 32 : 64;
    r.plan = make_plan(r.a.P, r.a.Q, r.a.K, pt, qt, r.way == kStaged, f32, step, f32 ? 6.0f : r.way == kStaged ? 3.0f : mx ? 0.6f : 1.0f);
    r.e.ld_partial = (r.a.P + 7) & ~7;
    r.e.split_stride = r.e.ld_partial * r.a.Q;
    r.partial_bytes = r.plan.splits > 1 ? (size_t)r.plan.splits * r.e.split_stride * 4 : 0;
    r.e.exact = exact_results(r.e);
}

// Points an operand at its packed planes.
void use_planes(const void *planes, int64_t rows, int64_t cols, const void *&p, int64_t &ld, int64_t &plane, int &extent, bool columns)
{
    p = planes;
    ld = (cols + 7) & ~(int64_t)7;
    plane = rows * ld;
    if (columns) extent = (int)ld;
}

// Sum of the splits in their order, then the epilogue: a thread per 8
// consecutive p, or per one where the result's layout allows no vectors.
constexpr int kReduceThreads = 64;              // a wave a block: the few threads of a small result on many CUs

// A few partial rows of db, whose sum shares a launch with that of dw's splits: so
// few take longer to launch than to add (1001 x 59 x 333 in fp32 21.0 us a call,
// 23.2 with a launch of their own).
struct RowSum {
    const float *part;
    float *out;
    int n, rows, accumulate;
};
constexpr int kSharedRows = 128;

// 16 columns a wave, 4 lanes of rows each, added in a fixed order.
__device__ __forceinline__ void sum_few_rows(const RowSum &d, int block)
{
    const int c = block * 16 + (threadIdx.x & 15);
    float s = 0.0f;
    if (c < d.n) {
#pragma unroll 8
        for (int r = threadIdx.x >> 4; r < d.rows; r += 4) s += d.part[(int64_t)r * d.n + c];
    }
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (threadIdx.x < 16 && c < d.n) d.out[c] = d.accumulate ? d.out[c] + s : s;
}

template <bool VEC>
__global__ __launch_bounds__(kReduceThreads) void reduce_splits(LinearEpilogue::Args e, int P, int Q, int splits, int blocks, RowSum rows)
{
    if ((int)blockIdx.x >= blocks) return sum_few_rows(rows, (int)blockIdx.x - blocks);
    const int64_t groups = VEC ? P / 8 : P, id = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x;
    if (id >= groups * Q) return;
    const int q = (int)(id / groups), p = (int)(id - q * groups) * (VEC ? 8 : 1);
    const float *src = e.partial + (int64_t)q * e.ld_partial + p;
    if constexpr (VEC) {
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        e.partial = nullptr;
        LinearEpilogue::Ahead ahead;
        LinearEpilogue::look_ahead(e, p, q, 0, ahead);
        LinearEpilogue::Part part;
        LinearEpilogue::part(e, p, part);
#pragma unroll 4
        for (int s = 0; s < splits; s++) {
            float w[8];
            load8_vec(src + s * e.split_stride, w);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] += w[i];
        }
        LinearEpilogue::finish8(e, p, q, v, part, ahead);
    } else {
        float v = 0.0f;
#pragma unroll 8
        for (int s = 0; s < splits; s++) v += src[s * e.split_stride];
        LinearEpilogue::finish1(e, p, q, v);
    }
}

// `count` of the product's columns (along p) or rows (along q) of results, from `at` on.
Product band_of(const Product &whole, bool along_p, int at, int count)
{
    Product r = whole;
    gemm::Args &a = r.a;
    LinearEpilogue::Args &e = r.e;
    const auto move = [](auto &base, int64_t bytes) {
        if (base) base = reinterpret_cast<std::remove_reference_t<decltype(base)>>(reinterpret_cast<uintptr_t>(base) + (uintptr_t)bytes);
    };
    const int es = r.way == kPacked ? 2 : dtype_bytes(r.type), ys = dtype_bytes(e.y_type), zs = dtype_bytes(e.z_type);
    if (along_p) {
        move(a.p, (r.plan.pt ? at : at * a.ldp) * es);
        move(a.ps, at * a.ldps);
        a.P = count;
        a.Pl -= at;
        if (!e.bias_on_q) move(e.bias, at * (int64_t)4);
        move(e.residual, (int64_t)at * ys);
        move(e.y, (int64_t)at * ys);
        move(e.z, at * e.z_p * zs);
    } else {
        move(a.q, (r.plan.qt ? at : at * a.ldq) * es);
        move(a.qs, at * a.ldqs);
        a.Q = count;
        a.Ql -= at;
        if (e.bias_on_q) move(e.bias, at * (int64_t)4);
        move(e.residual, at * e.ldr * ys);
        move(e.y, at * e.ldy * ys);
        move(e.z, at * e.z_q * zs);
    }
    return r;
}

hipError_t run_product(Product &r, void *partial, hipStream_t s, const RowSum &rows = RowSum{})
{
    // more tiles than one launch takes: in bands along the longer side
    const int tile = 256 >> r.plan.tile;
    const int64_t tiles_p = (r.a.P + tile - 1) / tile, tiles_q = (r.a.Q + tile - 1) / tile;
    if (tiles_p * tiles_q > gemm::kMaxTiles) {
        const bool along_p = tiles_p > tiles_q;
        const int64_t whole = along_p ? r.a.P : r.a.Q, band = gemm::kMaxTiles / (along_p ? tiles_q : tiles_p) * tile;
        for (int64_t at = 0; at < whole; at += band) {
            Product part = band_of(r, along_p, (int)at, (int)(band < whole - at ? band : whole - at));
            const hipError_t err = run_product(part, partial, s, at == 0 ? rows : RowSum{});
            if (err != hipSuccess) return err;
        }
        return hipSuccess;
    }
    r.e.partial = r.plan.splits > 1 ? static_cast<float *>(partial) : nullptr;
    hipError_t err;
    if (r.type == GS_DTYPE_MXFP8 && r.way == kDirect) err = launch_product_mx8(r.a, r.e, r.plan, s);
    else if (r.type == GS_DTYPE_F32) err = launch_product_f32(r.a, r.e, r.plan, s);
    else if (r.type == GS_DTYPE_F16) err = launch_product_f16(r.a, r.e, r.plan, s);
    else err = launch_product_bf16(r.a, r.e, r.plan, s);        // widened 8-bit operands too
    if (err != hipSuccess || r.plan.splits == 1) return err;
    const bool vec = r.a.P % 8 == 0;            // whole chunks
    const int64_t n = (int64_t)(vec ? r.a.P / 8 : r.a.P) * r.a.Q;
    const int blocks = (int)((n + kReduceThreads - 1) / kReduceThreads), more = (rows.n + 15) / 16;
    if (vec) reduce_splits<true><<<(unsigned)(blocks + more), kReduceThreads, 0, s>>>(r.e, r.a.P, r.a.Q, r.plan.splits, blocks, rows);
    else reduce_splits<false><<<(unsigned)(blocks + more), kReduceThreads, 0, s>>>(r.e, r.a.P, r.a.Q, r.plan.splits, blocks, rows);
    return hipGetLastError();
}

// ---- forward ------------------------------------------------------------------
gs_status linear_ok(const gs_linear *l)
{
    if (!l) return GS_ERR_INVALID_ARG;
    if (l->m < 0 || l->m > ((int64_t)1 << 30) || l->n < 1 || l->n > (1 << 20) || l->k < 1 || l->k > (1 << 20))
        return GS_ERR_INVALID_ARG;
    if (!float_type(l->dtype) && l->dtype != GS_DTYPE_MXFP8) return GS_ERR_INVALID_ARG;
    if (l->y_dtype == GS_DTYPE_MXFP8) return GS_ERR_UNSUPPORTED;
    if (!float_type(l->y_dtype)) return GS_ERR_INVALID_ARG;
    if (l->activation < GS_ACT_NONE || l->activation > GS_ACT_GELU) return GS_ERR_INVALID_ARG;
    if (l->dtype == GS_DTYPE_MXFP8 && (l->k % 32 != 0 || l->z)) return GS_ERR_UNSUPPORTED;
    if ((l->m + 63) / 64 * ((l->n + 63) / 64) > INT32_MAX) return GS_ERR_UNSUPPORTED;
    const int es = dtype_bytes(l->dtype);
    if (l->x_stride < l->k || l->w_stride < l->k) return GS_ERR_INVALID_ARG;
    if (l->m > 0 && (!l->x || !l->w)) return GS_ERR_INVALID_ARG;
    if (!aligned_to(l->x, es) || !aligned_to(l->w, es) || !aligned_to(l->bias, 4)) return GS_ERR_INVALID_ARG;
    if (l->dtype == GS_DTYPE_MXFP8 && ((l->m > 0 && (!l->x_scales || !l->w_scales)) || l->x_scales_stride < l->k / 32 ||
                                       l->w_scales_stride < l->k / 32))
        return GS_ERR_INVALID_ARG;
    if (l->z && (l->z_stride < l->n || !aligned_to(l->z, es))) return GS_ERR_INVALID_ARG;
    return GS_OK;
}

gs_status linear_fwd_ok(const gs_linear *l)
{
    const gs_status st = linear_ok(l);
    if (st != GS_OK) return st;
    const int64_t row = l->planes ? l->m : l->n;
    const int ys = dtype_bytes(l->y_dtype);
    if ((l->m > 0 && !l->y) || l->y_stride < row || !aligned_to(l->y, ys)) return GS_ERR_INVALID_ARG;
    if (l->residual && (l->residual_stride < row || !aligned_to(l->residual, ys))) return GS_ERR_INVALID_ARG;
    return GS_OK;
}

struct FwdPlan {
    Product product;
    size_t p_at, q_at, partial_at, bytes;
};

FwdPlan plan_fwd(const gs_linear &l)
{
    FwdPlan f;
    memset(&f, 0, sizeof f);
    Product &r = f.product;
    const int es = dtype_bytes(l.dtype);
    const bool px = l.planes != 0;              // the P operand is x
    gemm::Args &a = r.a;
    a.p = px ? l.x : l.w;
    a.q = px ? l.w : l.x;
    a.ldp = px ? l.x_stride : l.w_stride;
    a.ldq = px ? l.w_stride : l.x_stride;
    a.ps = px ? l.x_scales : l.w_scales;
    a.qs = px ? l.w_scales : l.x_scales;
    a.ldps = px ? l.x_scales_stride : l.w_scales_stride;
    a.ldqs = px ? l.w_scales_stride : l.x_scales_stride;
    a.P = a.Pl = (int)(px ? l.m : l.n);
    a.Q = a.Ql = (int)(px ? l.n : l.m);
    a.K = l.k;
    a.p_type = a.q_type = l.dtype;
    r.type = l.dtype;
    LinearEpilogue::Args &e = r.e;
    e.bias = l.bias;
    e.bias_on_q = px;
    e.act = l.activation;
    e.residual = l.residual;
    e.ldr = l.residual_stride;
    e.y = l.y;
    e.ldy = l.y_stride;
    e.y_type = l.y_dtype;
    e.z = l.z;
    e.z_type = l.dtype;
    e.z_q = px ? 1 : l.z_stride;
    e.z_p = px ? l.z_stride : 1;
    bool p_ok = l.dtype != GS_DTYPE_F32 && gemm::direct_ok(a.p, es, a.ldp, a.K), q_ok = l.dtype != GS_DTYPE_F32 && gemm::direct_ok(a.q, es, a.ldq, a.K);
    // 8-bit matrix instructions only for 16-bit results: they keep fewer bits
    // of a sum than fp32 holds
    if (l.dtype == GS_DTYPE_MXFP8)
        p_ok = q_ok = p_ok && q_ok && l.y_dtype != GS_DTYPE_F32 && a.ldps < (1 << 22) && a.ldqs < (1 << 22);
    finish_plan(r, p_ok, q_ok);
    if (l.m <= kFewRows && !(l.dtype == GS_DTYPE_MXFP8 && l.y_dtype == GS_DTYPE_F32) &&
        few_rows_cost(l) < r.plan.us + 1.8) {
        r.way = kFew;                           // no workspace
        return f;
    }
    if (r.pack_p) {
        f.p_at = f.bytes;
        f.bytes += packed_bytes(l.dtype, a.P, l.k);
    }
    if (r.pack_q) {
        f.q_at = f.bytes;
        f.bytes += packed_bytes(l.dtype, a.Q, l.k);
    }
    f.partial_at = f.bytes;
    f.bytes += r.partial_bytes;
    return f;
}

hipError_t run_fwd(const gs_linear &l, FwdPlan &f, char *ws, hipStream_t s)
{
    Product &r = f.product;
    if (r.way == kFew) return launch_few_rows(l, r.e, s);
    gemm::Args &a = r.a;
    PackJobs jobs;
    memset(&jobs, 0, sizeof jobs);
    if (r.pack_p) {
        add_job(jobs, a.p, l.dtype, a.ps, a.ldp, a.ldps, a.P, l.k, ws + f.p_at);
        use_planes(ws + f.p_at, a.P, l.k, a.p, a.ldp, a.plane_p, a.Pl, false);
    }
    if (r.pack_q) {
        add_job(jobs, a.q, l.dtype, a.qs, a.ldq, a.ldqs, a.Q, l.k, ws + f.q_at);
        use_planes(ws + f.q_at, a.Q, l.k, a.q, a.ldq, a.plane_q, a.Ql, false);
    }
    const hipError_t err = run_jobs(jobs, s);
    return err == hipSuccess ? run_product(r, ws + f.partial_at, s) : err;
}

// ---- backward: dz and the sums of db -------------------------------------------
struct DzArgs {
    const void *dy, *z;
    int64_t lddy, ldz;
    int dy_type, type, act, exact;
    void *dz;                           // [m][ld_dz] of `type`, zeros past n; NULL: not wanted
    uint16_t *limbs;                    // fp32: [3][m][ld_dz] bf16 limbs of dz; NULL: not wanted
    int64_t ld_dz;
    float *part;                        // [row blocks][n] partial sums of db, or NULL
    int64_t m;
    int n, rows_per_block;
};

// A block's sums of its columns over its row lanes, in order, to its partial row.
__device__ __forceinline__ void column_sums(const DzArgs &d, int groups, const float acc[8], float (*sums)[8])
{
    if (!d.part) return;
    const int lanes = kThreads / groups;
#pragma unroll
    for (int i = 0; i < 8; i++) sums[threadIdx.x][i] = acc[i];
    __syncthreads();
    for (int i = threadIdx.x; i < groups * 8; i += kThreads) {
        const int c = blockIdx.x * groups * 8 + i;
        float s = 0.0f;
        for (int l = 0; l < lanes; l++) s += sums[l * groups + i / 8][i % 8];
        if (c < d.n) d.part[(int64_t)blockIdx.y * d.n + c] = s;
    }
}

// dy in rows.  A block takes `rows_per_block` rows of up to 512 columns: a
// thread owns 8 columns and every (256 / groups)-th row.
__global__ __launch_bounds__(kThreads) void dz_rows(DzArgs d, int groups)
{
    __shared__ float sums[kThreads][8];
    const int cg = threadIdx.x % groups, rl = threadIdx.x / groups, lanes = kThreads / groups;
    const int c0 = (blockIdx.x * groups + cg) * 8, valid = max(0, min(8, d.n - c0));
    const int64_t r0 = (int64_t)blockIdx.y * d.rows_per_block, r1 = min(d.m, r0 + d.rows_per_block);
    const bool room = c0 < d.ld_dz;             // ld_dz is a multiple of 8
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t r = r0 + rl; r < r1; r += lanes) {
        float v[8];
        load8(d.dy, d.dy_type, r * d.lddy + c0, valid, v);
        if (d.act != GS_ACT_NONE) {
            float z[8];
            load8(d.z, d.type, r * d.ldz + c0, valid, z);
            if (d.exact) scale_by_slope<8, true>(v, z, d.act);      // past n: 0 times the slope at 0
            else scale_by_slope<8, false>(v, z, d.act);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] += v[i];
        if (room && d.dz) store8_vec(d.dz, d.type, r * d.ld_dz + c0, v);
        if (room && d.limbs) store_planes(d.limbs, d.m * d.ld_dz, r * d.ld_dz + c0, 3, 0, v);
    }
    column_sums(d, groups, acc, sums);
}

// The same where dy, z and dz are of one 16-bit type in whole chunks of 8: the next row is on its way, unconverted, while a row is worked on
// (16384 x 4096 with GELU in bf16: 79 us, 5.1 TB/s; 103 us without).
template <typename T> __global__ __launch_bounds__(kThreads) void dz_rows_ahead(DzArgs d, int groups)
{
    __shared__ float sums[kThreads][8];
    using Row = Vec<T, 8>;
    const int cg = threadIdx.x % groups, rl = threadIdx.x / groups, lanes = kThreads / groups;
    const int c0 = (blockIdx.x * groups + cg) * 8;
    const int64_t r0 = (int64_t)blockIdx.y * d.rows_per_block, r1 = min(d.m, r0 + d.rows_per_block);
    const T *dy = static_cast<const T *>(d.dy) + c0, *z = static_cast<const T *>(d.z) + c0;
    T *dz = static_cast<T *>(d.dz) + c0;
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    Row ny{}, nz{};
    auto fetch = [&](int64_t r) {
        if (r >= r1 || c0 >= d.n) return;
        ny = *reinterpret_cast<const Row *>(dy + r * d.lddy);
        nz = *reinterpret_cast<const Row *>(z + r * d.ldz);
    };
    fetch(r0 + rl);
    for (int64_t r = r0 + rl; r < r1; r += lanes) {
        float v[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            v[i] = (float)ny.v[i];
            w[i] = (float)nz.v[i];
        }
        fetch(r + lanes);
        scale_by_slope<8, false>(v, w, d.act);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] += v[i];
        if (c0 < d.n) store8_vec(dz + r * d.ld_dz, v);
    }
    column_sums(d, groups, acc, sums);
}

// dy in planes [n][m]: tiles of 64 columns x 32 rows, read 8 rows of a column at
// a time, turned round in LDS and written 8 columns of a row at a time; the
// next tile is on its way meanwhile.  HBM-bound: 58091 x 192 with GELU in bf16 22 us
// (4.1 TB/s; 47 with single elements an access), 1001 x 59 in fp32 3.9 us.
constexpr int kPlaneRows = 32;

template <bool EXACT> __global__ __launch_bounds__(kThreads) void dz_planes(DzArgs d)
{
    __shared__ float tile[64][kPlaneRows + 1];
    __shared__ float sums[kThreads][8];
    constexpr int kGroups = 8;                  // of 8 columns
    const int cg = threadIdx.x % kGroups, rl = threadIdx.x / kGroups;
    const int c0 = (blockIdx.x * kGroups + cg) * 8, valid = max(0, min(8, d.n - c0));
    const int column = blockIdx.x * 64 + threadIdx.x / 4, rows_at = threadIdx.x % 4 * 8;
    const int64_t r0 = (int64_t)blockIdx.y * d.rows_per_block, r1 = min(d.m, r0 + d.rows_per_block);
    const bool room = c0 < d.ld_dz;             // ld_dz is a multiple of 8
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0}, in[8], z[8];
    auto fetch = [&](int64_t r) {
        const int there = column < d.n ? (int)max((int64_t)0, min((int64_t)8, r1 - r - rows_at)) : 0;
        load8(d.dy, d.dy_type, (int64_t)column * d.lddy + r + rows_at, there, in);
        if (d.act != GS_ACT_NONE) load8(d.z, d.type, (r + rl) * d.ldz + c0, r + rl < r1 ? valid : 0, z);
    };
    fetch(r0);
    for (int64_t r = r0; r < r1; r += kPlaneRows) {
#pragma unroll
        for (int j = 0; j < 8; j++) tile[threadIdx.x / 4][rows_at + j] = in[j];
        __syncthreads();
        float v[8], at_z[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            v[j] = tile[cg * 8 + j][rl];
            at_z[j] = z[j];
        }
        __syncthreads();
        if (r + kPlaneRows < r1) fetch(r + kPlaneRows);
        if (d.act != GS_ACT_NONE) {
            scale_by_slope<8, EXACT>(v, at_z, d.act);   // outside: 0 times the slope at 0
        }
#pragma unroll
        for (int j = 0; j < 8; j++) acc[j] += v[j];
        if (!room || r + rl >= r1) continue;
        if (d.dz) store8_vec(d.dz, d.type, (r + rl) * d.ld_dz + c0, v);
        if (d.limbs) store_planes(d.limbs, d.m * d.ld_dz, (r + rl) * d.ld_dz + c0, 3, 0, v);
    }
    column_sums(d, kGroups, acc, sums);
}

// Rows of x that one row block of the pass takes: 128 x 256 x 512 12.5 us against
// 13.9 with partial sums and their own launch, 256 x 1024 x 256 20.4 against 19.2.
constexpr int kOneRowBlock = 128;

// Everything a backward call does, with its places in the workspace.
struct BwdPlan {
    bool own_dz;                        // dz is written to the workspace in `dtype` (else dz is dy where that is read)
    bool limbs;                         // dz is written as limbs
    bool pass;                          // the dz / db pass runs
    int row_blocks, rows_per_block;
    int64_t ld_dz;
    size_t dz_at, limbs_at, part_at, w_at, x_at, split_at, bytes;
    Product dx, dw;
};

BwdPlan plan_bwd(const gs_linear &l, const gs_linear_grads &g)
{
    BwdPlan b;
    memset(&b, 0, sizeof b);
    const int es = dtype_bytes(l.dtype);
    const bool f32 = l.dtype == GS_DTYPE_F32;
    b.ld_dz = ((int64_t)l.n + 7) & ~(int64_t)7;
    // dz is dy itself when nothing has to be done to it; a 16-bit dz is always
    // loadable directly, written that way if dy is not
    const bool same = l.activation == GS_ACT_NONE && !l.planes && l.y_dtype == l.dtype;
    const bool as_is = same && (f32 || gemm::direct_ok(g.dy, es, g.dy_stride, l.n));

    auto product = [&](Product &r, const void *p, int64_t ldp, int Q, int K, bool qt, void *y, int64_t ldy, int y_type, bool add) {
        r.type = l.dtype;
        r.plan.pt = true;
        r.plan.qt = qt;
        r.a.p = p;
        r.a.ldp = ldp;
        r.a.p_type = r.a.q_type = l.dtype;
        r.a.q = as_is ? g.dy : nullptr;                 // else: the workspace, aligned to 16 bytes
        r.a.ldq = as_is ? g.dy_stride : b.ld_dz;
        r.a.P = r.a.Pl = l.k;
        r.a.Q = r.a.Ql = Q;
        r.a.K = K;
        r.e.y = y;
        r.e.ldy = ldy;
        r.e.y_type = y_type;
        r.e.accumulate = add;
        finish_plan(r, !f32 && gemm::direct_ok(p, es, ldp, l.k), !f32);
        if (qt && !as_is) r.a.Ql = (int)b.ld_dz;        // its padding may be read
        r.pack_q = false;                               // dz comes from the pass in the form it is needed in
    };
    if (g.dx) product(b.dx, l.w, l.w_stride, (int)l.m, l.n, false, g.dx, g.dx_stride, l.dtype, false);
    if (g.dw) product(b.dw, l.x, l.x_stride, l.n, (int)l.m, true, g.dw, g.dw_stride, g.dw_dtype, g.accumulate != 0);
    const bool staged_f32 = f32 && ((g.dx && b.dx.way == kStaged) || (g.dw && b.dw.way == kStaged));
    b.limbs = f32 && ((g.dx && b.dx.way == kPacked) || (g.dw && b.dw.way == kPacked));
    b.own_dz = !as_is && (f32 ? staged_f32 : g.dx || g.dw);
    b.pass = b.own_dz || b.limbs || g.db;

    // row blocks of the pass: enough for the device, at most 1024 (the partial
    // sums are read once more); one for few rows, whose sums are then db itself
    // and save a launch
    const int64_t cols = l.planes ? (l.n + 63) / 64 : (l.n + 511) / 512;
    int64_t want = 2048 / cols;
    want = want < 1 ? 1 : want > 1024 ? 1024 : want;
    int64_t per = (l.m + want - 1) / want;
    const int64_t whole = l.planes ? kPlaneRows : 8;    // rows that a block works on at a time
    per = (per + whole - 1) / whole * whole;
    if (per < whole) per = whole;
    if (l.m <= kOneRowBlock) per = kOneRowBlock;
    b.rows_per_block = (int)per;
    b.row_blocks = (int)((l.m + per - 1) / per);
    auto take = [&](size_t bytes) {
        const size_t at = b.bytes;
        b.bytes += round256(bytes);
        return at;
    };
    if (b.own_dz) b.dz_at = take((size_t)l.m * b.ld_dz * es);
    if (b.limbs) b.limbs_at = take((size_t)3 * l.m * b.ld_dz * 2);
    if (g.db) b.part_at = take((size_t)b.row_blocks * l.n * 4);
    if (b.dx.pack_p) b.w_at = take(packed_bytes(l.dtype, l.n, l.k));
    if (b.dw.pack_p) b.x_at = take(packed_bytes(l.dtype, l.m, l.k));
    // the two products run one after the other and share their partial sums' place
    b.split_at = take(b.dx.partial_bytes > b.dw.partial_bytes ? b.dx.partial_bytes : b.dw.partial_bytes);
    return b;
}

gs_status linear_bwd_ok(const gs_linear *l, const gs_linear_grads *g)
{
    const gs_status st = linear_ok(l);
    if (st != GS_OK) return st;
    if (!g) return GS_ERR_INVALID_ARG;
    if (l->dtype == GS_DTYPE_MXFP8) return GS_ERR_UNSUPPORTED;
    if (l->activation != GS_ACT_NONE && l->m > 0 && !l->z) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(l->dtype);
    if ((l->m > 0 && !g->dy) || g->dy_stride < (l->planes ? l->m : l->n) || !aligned_to(g->dy, dtype_bytes(l->y_dtype)))
        return GS_ERR_INVALID_ARG;
    if (g->dx && (g->dx_stride < l->k || !aligned_to(g->dx, es))) return GS_ERR_INVALID_ARG;
    if (g->dw && ((g->dw_dtype != GS_DTYPE_F32 && g->dw_dtype != l->dtype) || g->dw_stride < l->k ||
                  !aligned_to(g->dw, dtype_bytes(g->dw_dtype))))
        return GS_ERR_INVALID_ARG;
    if (!aligned_to(g->db, 4)) return GS_ERR_INVALID_ARG;
    return GS_OK;
}

__global__ __launch_bounds__(kThreads) void zero_rows(void *p, int type, int64_t ld, int rows, int cols)
{
    const int64_t id = block_of() * kThreads + threadIdx.x;
    if (id >= (int64_t)rows * cols) return;
    store_from_float(p, type, id / cols * ld + id % cols, 0.0f);
}

hipError_t run_bwd(const gs_linear &l, const gs_linear_grads &g, BwdPlan &b, char *ws, hipStream_t s)
{
    hipError_t err = hipSuccess;
    if (l.m == 0) {                             // sums over no rows
        if (g.dw && !g.accumulate) {
            const int64_t blocks = ((int64_t)l.n * l.k + kThreads - 1) / kThreads;
            zero_rows<<<grid_of(blocks, kThreads), kThreads, 0, s>>>(g.dw, g.dw_dtype, g.dw_stride, l.n, l.k);
            if ((err = hipGetLastError()) != hipSuccess) return err;
        }
        if (g.db && !g.accumulate) {
            zero_rows<<<(unsigned)((l.n + kThreads - 1) / kThreads), kThreads, 0, s>>>(g.db, GS_DTYPE_F32, l.n, 1, l.n);
            err = hipGetLastError();
        }
        return err;
    }
    RowSum rows = {};                           // left to the launch after dw
    if (b.pass) {
        DzArgs d;
        d.dy = g.dy;
        d.z = l.z;
        d.lddy = g.dy_stride;
        d.ldz = l.z_stride;
        d.dy_type = l.y_dtype;
        d.type = l.dtype;
        d.act = l.activation;
        d.exact = l.dtype == GS_DTYPE_F32;
        d.dz = b.own_dz ? ws + b.dz_at : nullptr;
        d.limbs = b.limbs ? reinterpret_cast<uint16_t *>(ws + b.limbs_at) : nullptr;
        d.ld_dz = b.ld_dz;
        const bool sum = g.db && (b.row_blocks > 1 || g.accumulate);
        d.part = sum ? reinterpret_cast<float *>(ws + b.part_at) : g.db;
        d.m = l.m;
        d.n = l.n;
        d.rows_per_block = b.rows_per_block;
        if (l.planes) {
            const dim3 grid((unsigned)((l.n + 63) / 64), (unsigned)b.row_blocks);
            if (d.exact) dz_planes<true><<<grid, kThreads, 0, s>>>(d);
            else dz_planes<false><<<grid, kThreads, 0, s>>>(d);
        } else {
            // of 8 columns: a power of two, at most 64; few where one block takes all rows
            const int most = l.m <= kOneRowBlock ? 8 : 64;
            int groups = 1;
            while (groups < most && groups * 8 < l.n) groups *= 2;
            const dim3 grid((unsigned)((l.n + groups * 8 - 1) / (groups * 8)), (unsigned)b.row_blocks);
            const bool ahead = d.dz && !d.limbs && l.n % 8 == 0 && l.activation != GS_ACT_NONE && l.y_dtype == l.dtype;
            if (ahead && l.dtype == GS_DTYPE_BF16) dz_rows_ahead<__bf16><<<grid, kThreads, 0, s>>>(d, groups);
            else if (ahead && l.dtype == GS_DTYPE_F16) dz_rows_ahead<_Float16><<<grid, kThreads, 0, s>>>(d, groups);
            else dz_rows<<<grid, kThreads, 0, s>>>(d, groups);
        }
        if ((err = hipGetLastError()) != hipSuccess) return err;
        if (sum && g.dw && b.dw.plan.splits > 1 && b.row_blocks <= kSharedRows)
            rows = {d.part, g.db, l.n, b.row_blocks, g.accumulate};
        else if (sum && (err = launch_sum_rows(d.part, g.db, l.n, b.row_blocks, g.accumulate, s)) != hipSuccess)
            return err;
    }
    PackJobs jobs;
    memset(&jobs, 0, sizeof jobs);
    auto operands = [&](Product &r, bool packed_at, size_t at, int64_t rows, bool qt) {
        gemm::Args &a = r.a;
        if (packed_at) {
            add_job(jobs, a.p, l.dtype, nullptr, a.ldp, 0, rows, l.k, ws + at);
            use_planes(ws + at, rows, l.k, a.p, a.ldp, a.plane_p, a.Pl, true);
        }
        if (b.limbs && r.way == kPacked) {
            use_planes(ws + b.limbs_at, l.m, l.n, a.q, a.ldq, a.plane_q, a.Ql, qt);
        } else if (b.own_dz) {
            a.q = ws + b.dz_at;
        }
    };
    if (g.dx) operands(b.dx, b.dx.pack_p, b.w_at, l.n, false);
    if (g.dw) operands(b.dw, b.dw.pack_p, b.x_at, l.m, true);
    if ((err = run_jobs(jobs, s)) != hipSuccess) return err;
    if (g.dx && (err = run_product(b.dx, ws + b.split_at, s)) != hipSuccess) return err;
    if (g.dw && (err = run_product(b.dw, ws + b.split_at, s, rows)) != hipSuccess) return err;
    return hipSuccess;
}

gs_status from_hip(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }

}  // namespace
}  // namespace gsi

using namespace gsi;

extern "C" {

size_t gs_linear_fwd_workspace_bytes(const gs_linear *l)
{
    if (linear_fwd_ok(l) != GS_OK || l->m == 0) return 0;
    return plan_fwd(*l).bytes;
}

gs_status gs_linear_fwd(const gs_linear *l, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = linear_fwd_ok(l);
    if (st != GS_OK) return st;
    if (l->m == 0) return GS_OK;
    FwdPlan f = plan_fwd(*l);
    if (f.bytes > 0) {
        if (workspace_bytes < f.bytes) return GS_ERR_WORKSPACE;
        if (!workspace || !al16(workspace)) return GS_ERR_INVALID_ARG;
    }
    return from_hip(run_fwd(*l, f, static_cast<char *>(workspace), (hipStream_t)stream));
}

size_t gs_linear_bwd_workspace_bytes(const gs_linear *l, const gs_linear_grads *g)
{
    if (linear_bwd_ok(l, g) != GS_OK || l->m == 0) return 0;
    return plan_bwd(*l, *g).bytes;
}

gs_status gs_linear_bwd(const gs_linear *l, const gs_linear_grads *g, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = linear_bwd_ok(l, g);
    if (st != GS_OK) return st;
    BwdPlan b = plan_bwd(*l, *g);
    if (l->m > 0 && b.bytes > 0) {
        if (workspace_bytes < b.bytes) return GS_ERR_WORKSPACE;
        if (!workspace || !al16(workspace)) return GS_ERR_INVALID_ARG;
    }
    return from_hip(run_bwd(*l, *g, b, static_cast<char *>(workspace), (hipStream_t)stream));
}

}  // extern "C"
