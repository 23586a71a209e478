// Root-mean-square norm with the residual's addition, output in the input's
// type or in 8-bit blocks, and its backward; 8-bit quantisation of a matrix.
//
// HBM-bound: the forward reads x and the residual and writes the sum and y
// once, the backward reads the sum, dy and dsum and writes dx.  A row is held
// in registers between its reduction and its outputs, 8 consecutive elements
// (16 bytes of a 16-bit type) per lane and access.  Forward: rows of up to 128
// by 16 lanes, up to 256 by 32, up to 2048 by a wave (4 rows per workgroup, no barrier), up to
// 8192 by a workgroup, longer ones in two passes.  An 8-bit block of 32 values is
// 4 neighbouring lanes.  Backward: as few elements per lane as cover the row, 8
// or (512 < n <= 1024) 16, as it also holds the next row and its columns' sums.
//
// bf16 with a residual: 16384 x 1024 in 27.4 us (134 MB, 4.9 TB/s; fp32 53.7), 100000 x
// 2048 to 8 bits in 264 us (1.44 GB, 5.4 TB/s), the backward of 16384 x 1024 in 33 us
// (4.1 TB/s, 4 us of them the sum of the partial dgammas; fp32 65).  Quantisation
// alone: bf16 65536 x 2048 in 76.5 us (5.3 TB/s).
#include "gs_linear.h"

#include <math.h>

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRegRow = 8192;

bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }
gs_status from_hip(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }

template <typename T> __device__ __forceinline__ void load_chunk(const T *p, int64_t i, int valid, float v[8])
{
    if (valid == 8) {
        load8_vec(p + i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = j < valid ? (float)p[i + j] : 0.0f;
}
template <typename T> __device__ __forceinline__ void store_chunk(T *p, int64_t i, int valid, const float v[8])
{
    if (valid == 8) {
        store8_vec(p + i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < valid) p[i + j] = (T)v[j];
}

// Sum over the LANES threads of a row: (part of) a wave, or the workgroup by LDS.
template <int LANES> __device__ __forceinline__ float row_sum(float x, float *lds)
{
#pragma unroll
    for (int o = min(LANES, 64) / 2; o > 0; o >>= 1) x += __shfl_xor(x, o);
    if constexpr (LANES > 64) {
        __syncthreads();                        // the last use of lds is over
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
        __syncthreads();
        x = 0.0f;
#pragma unroll
        for (int w = 0; w < LANES / 64; w++) x += lds[w];
    }
    return x;
}

struct NormArgs {
    const void *x, *residual;
    const float *gamma;
    void *sum, *y;
    uint8_t *scales;
    float *rstd;
    int64_t m, ldx, ldr, lds, ldy, ldsc;
    int n, q8, norm;                            // norm 0: y is x (quantisation alone)
    float eps;
};

__device__ __forceinline__ float inverse_rms(float sum_sq, int n, float eps) { return 1.0f / sqrtf(sum_sq / (float)n + eps); }

template <typename T>
__device__ __forceinline__ void emit(const NormArgs &a, int64_t row, int c, int valid, float v[8], float rstd)
{
    if (a.norm) {
        float g[8];
        if (a.gamma) load_chunk(a.gamma, c, valid, g);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = a.gamma ? v[j] * rstd * g[j] : v[j] * rstd;
    }
    if (a.q8)
        quantize_chunk(v, static_cast<uint8_t *>(a.y) + row * a.ldy + c, (threadIdx.x & 3) == 0 ? a.scales + row * a.ldsc + (c >> 5) : nullptr);
    else
        store_chunk(static_cast<T *>(a.y), row * a.ldy + c, valid, v);
}

// Rows of up to LANES * 8 * V elements.  WIDE, rows of at least 8: the last chunk
// of a row takes its last 8 elements, so that every access is a whole vector;
// those that are also the chunk's before it count once and are written twice
// alike, after the whole row was read.
template <typename T, int LANES, int V, bool WIDE> __global__ __launch_bounds__(kThreads) void norm_rows(NormArgs a)
{
    __shared__ float lds[kThreads / 64];
    const int lane = threadIdx.x % LANES;
    const int64_t row = block_of() * (kThreads / LANES) + threadIdx.x / LANES;
    if (row >= a.m) return;                     // a row's lanes together
    auto chunk = [&](int k) { return (k * LANES + lane) * 8; };
    auto start = [&](int c) { return WIDE ? min(c, a.n - 8) : c; };
    auto inside = [&](int at) { return WIDE ? 8 : min(8, a.n - at); };
    float v[V][8], sq = 0.0f;
#pragma unroll
    for (int k = 0; k < V; k++) {
        const int c = chunk(k), at = start(c);
#pragma unroll
        for (int j = 0; j < 8; j++) v[k][j] = 0.0f;
        if (c >= a.n) continue;
        load_chunk(static_cast<const T *>(a.x), row * a.ldx + at, inside(at), v[k]);
        if (a.residual) {
            float r[8];
            load_chunk(static_cast<const T *>(a.residual), row * a.ldr + at, inside(at), r);
#pragma unroll
            for (int j = 0; j < 8; j++) v[k][j] += r[j];
        }
    }
#pragma unroll
    for (int k = 0; k < V; k++) {
        const int shared = WIDE ? max(0, min(8, chunk(k) - (a.n - 8))) : 0;
#pragma unroll
        for (int j = 0; j < 8; j++) {           // not times 0: an infinity would make the row NaN
            const float own = j >= shared ? v[k][j] : 0.0f;
            sq = fmaf(own, own, sq);
        }
    }
    const float rstd = inverse_rms(row_sum<LANES>(sq, lds), a.n, a.eps);
    if (a.rstd && lane == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int k = 0; k < V; k++) {
        const int c = chunk(k), at = start(c);
        if (c >= a.n) continue;                 // whole 8-bit blocks: n is a multiple of 32 there
        if (a.sum) store_chunk(static_cast<T *>(a.sum), row * a.lds + at, inside(at), v[k]);
        emit<T>(a, row, at, inside(at), v[k], rstd);
    }
}

// Rows of any length, a workgroup each, read twice.
template <typename T> __global__ __launch_bounds__(kThreads) void norm_long(NormArgs a)
{
    __shared__ float lds[kThreads / 64];
    const int64_t row = block_of();
    if (row >= a.m) return;
    auto sum_at = [&](int c, int valid, float v[8]) {
        load_chunk(static_cast<const T *>(a.x), row * a.ldx + c, valid, v);
        if (a.residual) {
            float r[8];
            load_chunk(static_cast<const T *>(a.residual), row * a.ldr + c, valid, r);
#pragma unroll
            for (int j = 0; j < 8; j++) v[j] += r[j];
        }
    };
    float sq = 0.0f, rstd = 0.0f;
    if (a.norm) {
        for (int c = threadIdx.x * 8; c < a.n; c += kThreads * 8) {
            float v[8];
            sum_at(c, min(8, a.n - c), v);
#pragma unroll
            for (int j = 0; j < 8; j++) sq = fmaf(v[j], v[j], sq);
        }
        rstd = inverse_rms(row_sum<kThreads>(sq, lds), a.n, a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x * 8; c < a.n; c += kThreads * 8) {
        const int valid = min(8, a.n - c);
        float v[8];
        sum_at(c, valid, v);
        if (a.sum) store_chunk(static_cast<T *>(a.sum), row * a.lds + c, valid, v);
        emit<T>(a, row, c, valid, v, rstd);
    }
}

template <typename T> hipError_t launch_norm(const NormArgs &a, hipStream_t s)
{
    const dim3 rows16 = grid_of((a.m + 15) / 16, kThreads), rows8 = grid_of((a.m + 7) / 8, kThreads), rows4 = grid_of((a.m + 3) / 4, kThreads),
               rows1 = grid_of(a.m, kThreads);
    if (a.n < 8) norm_rows<T, 16, 1, false><<<rows16, kThreads, 0, s>>>(a);
    else if (a.n <= 128) norm_rows<T, 16, 1, true><<<rows16, kThreads, 0, s>>>(a);
    else if (a.n <= 256) norm_rows<T, 32, 1, true><<<rows8, kThreads, 0, s>>>(a);
    else if (a.n <= 512) norm_rows<T, 64, 1, true><<<rows4, kThreads, 0, s>>>(a);
    else if (a.n <= 1024) norm_rows<T, 64, 2, true><<<rows4, kThreads, 0, s>>>(a);
    else if (a.n <= 2048) norm_rows<T, 64, 4, true><<<rows4, kThreads, 0, s>>>(a);
    else if (a.n <= 4096) norm_rows<T, 256, 2, true><<<rows1, kThreads, 0, s>>>(a);
    else if (a.n <= kMaxRegRow) norm_rows<T, 256, 4, true><<<rows1, kThreads, 0, s>>>(a);
    else norm_long<T><<<rows1, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_norm(const NormArgs &a, int dtype, hipStream_t s)
{
    if (dtype == GS_DTYPE_F32) return launch_norm<float>(a, s);
    if (dtype == GS_DTYPE_F16) return launch_norm<_Float16>(a, s);
    return launch_norm<__bf16>(a, s);
}

// ---- backward -------------------------------------------------------------------
struct GradArgs {
    const void *sum, *dy, *dsum;
    const float *rstd, *gamma;
    void *dx;
    float *part;                                // [grid][n] partial sums of dgamma, or NULL
    int64_t m, lds, ldy, ldds, ldx;
    int n;
};

template <int LANES> constexpr int kGradThreads = LANES <= 64 ? kThreads : LANES;

// Each workgroup strides over the rows; a thread keeps the dgamma sums of its
// columns in registers and the workgroup writes one partial row at the end.  The
// next row's sum and dy are on their way, unconverted, while a row is worked on.
// WIDE, rows of at least 8: the last chunk of a row takes its last 8 elements,
// so that every load is a whole vector, and leaves those of them that are the
// chunk's before it alone (62846 x 118 in bf16: 18 us, 27 with loads of single
// elements there).
template <typename T, int LANES, int V, bool WIDE> __global__ __launch_bounds__(kGradThreads<LANES>) void grad_rows(GradArgs a)
{
    constexpr int kRows = kGradThreads<LANES> / LANES;
    __shared__ float lds[LANES > 64 ? LANES / 64 : 1];
    __shared__ float turn[kRows > 1 ? kThreads : 1][8];
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    auto chunk = [&](int k, int l) { return (k * LANES + l) * 8; };
    auto start = [&](int c) { return WIDE ? min(c, a.n - 8) : c; };      // of a chunk's 8 elements
    // element j of a chunk that starts at `at` is its own
    auto own = [&](int c, int at, int j) { return WIDE ? at + j >= c : c + j < a.n; };
    auto load = [&](auto *p, int at, float v[8]) {
        if constexpr (WIDE) load8_vec(p + at, v);
        else load_chunk(p, at, a.n - at, v);
    };
    float dg[V][8];
    Vec<T, 8> nh[V], ng[V];
#pragma unroll
    for (int k = 0; k < V; k++) {
        nh[k] = ng[k] = Vec<T, 8>{};
#pragma unroll
        for (int j = 0; j < 8; j++) dg[k][j] = 0.0f;
    }
    auto fetch = [&](int64_t row) {
        if (row >= a.m) return;
#pragma unroll
        for (int k = 0; k < V; k++) {
            const int c = chunk(k, lane), at = start(c);
            if (c >= a.n) continue;
            const T *h = static_cast<const T *>(a.sum) + row * a.lds + at, *g = static_cast<const T *>(a.dy) + row * a.ldy + at;
            if constexpr (WIDE) {
                nh[k] = *reinterpret_cast<const Vec<T, 8> *>(h);
                ng[k] = *reinterpret_cast<const Vec<T, 8> *>(g);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (c + j < a.n) {
                        nh[k].v[j] = h[j];
                        ng[k].v[j] = g[j];
                    }
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * kRows;
    int64_t row = (int64_t)blockIdx.x * kRows + sub;
    fetch(row);
    for (; row < a.m; row += step) {
        const float rstd = a.rstd[row];
        float h[V][8], g[V][8], dot = 0.0f;
#pragma unroll
        for (int k = 0; k < V; k++)
#pragma unroll
            for (int j = 0; j < 8; j++) {
                h[k][j] = (float)nh[k].v[j];
                g[k][j] = (float)ng[k].v[j];
            }
        fetch(row + step);
#pragma unroll
        for (int k = 0; k < V; k++) {
            const int c = chunk(k, lane), at = start(c);
            if (c >= a.n) continue;
            if (WIDE && at < c) {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (!own(c, at, j)) h[k][j] = g[k][j] = 0.0f;
            }
            float w[8];
            if (a.gamma) load(a.gamma, at, w);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                h[k][j] *= rstd;
                dg[k][j] = fmaf(g[k][j], h[k][j], dg[k][j]);
                if (a.gamma) g[k][j] *= w[j];
                dot = fmaf(g[k][j], h[k][j], dot);
            }
        }
        dot = row_sum<LANES>(dot, lds) / (float)a.n;
#pragma unroll
        for (int k = 0; k < V; k++) {
            const int c = chunk(k, lane), at = start(c);
            if (c >= a.n) continue;
            float d[8];
            if (a.dsum) load(static_cast<const T *>(a.dsum) + row * a.ldds, at, d);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float v = rstd * fmaf(-h[k][j], dot, g[k][j]);
                d[j] = a.dsum ? v + d[j] : v;
            }
            T *dx = static_cast<T *>(a.dx) + row * a.ldx + at;
            if (WIDE && at == c) {
                store8_vec(dx, d);
            } else {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    if (own(c, at, j)) dx[j] = (T)d[j];
            }
        }
    }
    if (!a.part) return;
    float *out = a.part + (int64_t)blockIdx.x * a.n;
#pragma unroll
    for (int k = 0; k < V; k++) {
        if constexpr (kRows > 1) {              // a column's sums over the workgroup's rows, in order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; j++) turn[threadIdx.x][j] = dg[k][j];
            __syncthreads();
            for (int i = threadIdx.x; i < LANES * 8; i += kThreads) {
                const int c = chunk(k, i / 8), at = start(c);
                float sum = turn[i / 8][i % 8];
#pragma unroll
                for (int r = 1; r < kRows; r++) sum += turn[r * LANES + i / 8][i % 8];
                if (c < a.n && own(c, at, i % 8)) out[at + i % 8] = sum;
            }
        } else {
            const int c = chunk(k, lane), at = start(c);
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (c < a.n && own(c, at, j)) out[at + j] = dg[k][j];
        }
    }
}

// Rows of any length: dx, a workgroup each.
template <typename T> __global__ __launch_bounds__(kThreads) void grad_long(GradArgs a)
{
    __shared__ float lds[kThreads / 64];
    const int64_t row = block_of();
    if (row >= a.m) return;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    auto at = [&](int c, int valid, float h[8], float g[8]) {
        float w[8];
        load_chunk(static_cast<const T *>(a.sum), row * a.lds + c, valid, h);
        load_chunk(static_cast<const T *>(a.dy), row * a.ldy + c, valid, g);
        if (a.gamma) load_chunk(a.gamma, c, valid, w);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            h[j] *= rstd;
            if (a.gamma) g[j] *= w[j];
        }
    };
    for (int c = threadIdx.x * 8; c < a.n; c += kThreads * 8) {
        float h[8], g[8];
        at(c, min(8, a.n - c), h, g);
#pragma unroll
        for (int j = 0; j < 8; j++) dot = fmaf(g[j], h[j], dot);
    }
    dot = row_sum<kThreads>(dot, lds) / (float)a.n;
    for (int c = threadIdx.x * 8; c < a.n; c += kThreads * 8) {
        const int valid = min(8, a.n - c);
        float h[8], g[8], d[8];
        at(c, valid, h, g);
        if (a.dsum) load_chunk(static_cast<const T *>(a.dsum), row * a.ldds + c, valid, d);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float v = rstd * fmaf(-h[j], dot, g[j]);
            d[j] = a.dsum ? v + d[j] : v;
        }
        store_chunk(static_cast<T *>(a.dx), row * a.ldx + c, valid, d);
    }
}

// Rows of any length: partial sums of dgamma, 2048 columns by every grid.y-th row.
template <typename T> __global__ __launch_bounds__(kThreads) void dgamma_long(GradArgs a)
{
    const int c = (blockIdx.x * kThreads + threadIdx.x) * 8, valid = max(0, min(8, a.n - c));
    float dg[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int64_t row = blockIdx.y; row < a.m; row += gridDim.y) {
        float h[8], g[8];
        load_chunk(static_cast<const T *>(a.sum), row * a.lds + c, valid, h);
        load_chunk(static_cast<const T *>(a.dy), row * a.ldy + c, valid, g);
        const float rstd = a.rstd[row];
#pragma unroll
        for (int j = 0; j < 8; j++) dg[j] = fmaf(g[j], h[j] * rstd, dg[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < valid) a.part[(int64_t)blockIdx.y * a.n + c + j] = dg[j];
}

// Column sums of partial rows: 16 columns (64 bytes) a block, 64 lanes of rows
// with 8 loads under way each, then a tree over the lanes.
constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void sum_rows(const float *part, float *out, int n, int rows, int accumulate)
{
    __shared__ float sums[64][17];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, c = blockIdx.x * 16 + tx;
    float s = 0.0f;
    if (c < n) {
#pragma unroll 8
        for (int r = ty; r < rows; r += 64) s += part[(int64_t)r * n + c];
    }
    sums[ty][tx] = s;
#pragma unroll
    for (int h = 32; h > 0; h >>= 1) {
        __syncthreads();
        if (ty < h) sums[ty][tx] += sums[ty + h][tx];
    }
    if (ty == 0 && c < n) out[c] = accumulate ? out[c] + sums[0][tx] : sums[0][tx];
}

// Workgroups of the backward, each with one partial row of dgamma: one per CU
// before any takes a second pass over the rows, then at least two passes each
// (four of the one row of wide workgroups) while that gives each CU as many as
// it runs best with.  In bf16 with 512 / 1024: 60000 x 512 takes 75.3 / 53.5 us,
// 16384 x 1024 37.7 / 32.7, 16384 x 2048 82.5 / 64.2, 16384 x 4096 121 / 128;
// 2000 x 2048 17.3 with 512 and 20.7 with 1024.
int grad_blocks(int64_t m, int n)
{
    if (n > kMaxRegRow) return (int)(m < 64 ? m : 64);
    const int64_t rows = n <= 128 ? 16 : n <= 256 ? 8 : n <= 1024 ? 4 : 1;
    const int64_t passes = (m + rows - 1) / rows, most = n <= 2048 ? 1024 : 512;
    // its partial row is dgamma and saves a launch: 4 x 2034 7.8 us against 7.2 on
    // the GPU, but a call takes 10.7 against 13.1
    if (passes <= 4) return 1;
    if (passes <= 256) return (int)passes;
    const int64_t each = n <= 1024 ? 2 : 4, want = passes / each > 256 ? passes / each : 256;
    return (int)(want < most ? want : most);
}

template <typename T> hipError_t launch_grad(const GradArgs &a, hipStream_t s)
{
    const unsigned g = (unsigned)grad_blocks(a.m, a.n);
    if (a.n < 8) grad_rows<T, 16, 1, false><<<g, kThreads, 0, s>>>(a);
    else if (a.n <= 128) grad_rows<T, 16, 1, true><<<g, kThreads, 0, s>>>(a);
    else if (a.n <= 256) grad_rows<T, 32, 1, true><<<g, kThreads, 0, s>>>(a);
    else if (a.n <= 512) grad_rows<T, 64, 1, true><<<g, kThreads, 0, s>>>(a);
    else if (a.n <= 1024) grad_rows<T, 64, 2, true><<<g, kThreads, 0, s>>>(a);
    else if (a.n <= 2048) grad_rows<T, 256, 1, true><<<g, 256, 0, s>>>(a);
    else if (a.n <= 4096) grad_rows<T, 512, 1, true><<<g, 512, 0, s>>>(a);
    else if (a.n <= kMaxRegRow) grad_rows<T, 1024, 1, true><<<g, 1024, 0, s>>>(a);
    else {
        // dgamma first: dx may be written over dy
        if (a.part) dgamma_long<T><<<dim3((unsigned)((a.n + 2047) / 2048), g), kThreads, 0, s>>>(a);
        grad_long<T><<<grid_of(a.m, kThreads), kThreads, 0, s>>>(a);
    }
    return hipGetLastError();
}

gs_status norm_ok(const gs_rms_norm *a)
{
    if (!a) return GS_ERR_INVALID_ARG;
    if (a->m < 0 || a->m > ((int64_t)1 << 30) || a->n < 1 || a->n > (1 << 20)) return GS_ERR_INVALID_ARG;
    if (!float_type(a->dtype)) return GS_ERR_INVALID_ARG;
    if (a->y_dtype != a->dtype && a->y_dtype != GS_DTYPE_MXFP8) return GS_ERR_UNSUPPORTED;
    const bool q8 = a->y_dtype == GS_DTYPE_MXFP8;
    if (q8 && a->n % 32 != 0) return GS_ERR_INVALID_ARG;
    if (!isfinite(a->eps) || a->eps < 0.0f) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(a->dtype), ys = dtype_bytes(a->y_dtype);
    if (a->m > 0 && (!a->x || !a->y || (q8 && !a->y_scales))) return GS_ERR_INVALID_ARG;
    if (a->x_stride < a->n || a->y_stride < a->n || (a->residual && a->residual_stride < a->n) ||
        (a->sum && a->sum_stride < a->n) || (q8 && a->y_scales_stride < a->n / 32))
        return GS_ERR_INVALID_ARG;
    if (!aligned_to(a->x, es) || !aligned_to(a->residual, es) || !aligned_to(a->sum, es) || !aligned_to(a->y, ys) ||
        !aligned_to(a->gamma, 4) || !aligned_to(a->rstd, 4))
        return GS_ERR_INVALID_ARG;
    return GS_OK;
}

gs_status grads_ok(const gs_rms_norm_grads *a)
{
    if (!a) return GS_ERR_INVALID_ARG;
    if (a->m < 0 || a->m > ((int64_t)1 << 30) || a->n < 1 || a->n > (1 << 20)) return GS_ERR_INVALID_ARG;
    if (!float_type(a->dtype)) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(a->dtype);
    if (a->m > 0 && (!a->sum || !a->rstd || !a->dy || !a->dx)) return GS_ERR_INVALID_ARG;
    if (a->sum_stride < a->n || a->dy_stride < a->n || a->dx_stride < a->n || (a->dsum && a->dsum_stride < a->n))
        return GS_ERR_INVALID_ARG;
    if (!aligned_to(a->sum, es) || !aligned_to(a->dy, es) || !aligned_to(a->dsum, es) || !aligned_to(a->dx, es) ||
        !aligned_to(a->rstd, 4) || !aligned_to(a->gamma, 4) || !aligned_to(a->dgamma, 4))
        return GS_ERR_INVALID_ARG;
    return GS_OK;
}

__global__ __launch_bounds__(kThreads) void zero_floats(float *p, int n)
{
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

}  // namespace

hipError_t launch_sum_rows(const float *part, float *out, int n, int rows, int accumulate, hipStream_t s)
{
    sum_rows<<<(unsigned)((n + 15) / 16), kSumThreads, 0, s>>>(part, out, n, rows, accumulate);
    return hipGetLastError();
}

}  // namespace gsi

using namespace gsi;

extern "C" {

gs_status gs_rms_norm_fwd(const gs_rms_norm *p, void *stream)
{
    const gs_status st = norm_ok(p);
    if (st != GS_OK) return st;
    if (p->m == 0) return GS_OK;
    const bool q8 = p->y_dtype == GS_DTYPE_MXFP8;
    NormArgs a;
    a.x = p->x;
    a.residual = p->residual;
    a.gamma = p->gamma;
    a.sum = p->sum;
    a.y = p->y;
    a.scales = p->y_scales;
    a.rstd = p->rstd;
    a.m = p->m;
    a.ldx = p->x_stride;
    a.ldr = p->residual_stride;
    a.lds = p->sum_stride;
    a.ldy = p->y_stride;
    a.ldsc = p->y_scales_stride;
    a.n = p->n;
    a.q8 = q8;
    a.norm = 1;
    a.eps = p->eps;
    return from_hip(launch_norm(a, p->dtype, (hipStream_t)stream));
}

gs_status gs_mxfp8_quantize(const void *x, int32_t dtype, int64_t m, int32_t n, int64_t x_stride, uint8_t *codes,
                            int64_t codes_stride, uint8_t *scales, int64_t scales_stride, void *stream)
{
    gs_rms_norm p = {};
    p.m = m;
    p.n = n;
    p.dtype = dtype;
    p.y_dtype = GS_DTYPE_MXFP8;
    p.x = x;
    p.x_stride = x_stride;
    p.y = codes;
    p.y_stride = codes_stride;
    p.y_scales = scales;
    p.y_scales_stride = scales_stride;
    const gs_status st = norm_ok(&p);
    if (st != GS_OK) return st;
    if (m == 0) return GS_OK;
    NormArgs a = {};
    a.x = x;
    a.y = codes;
    a.scales = scales;
    a.m = m;
    a.ldx = x_stride;
    a.ldy = codes_stride;
    a.ldsc = scales_stride;
    a.n = n;
    a.q8 = 1;
    return from_hip(launch_norm(a, dtype, (hipStream_t)stream));
}

size_t gs_rms_norm_bwd_workspace_bytes(int64_t m, int32_t n)
{
    if (m <= 0 || m > ((int64_t)1 << 30) || n < 1 || n > (1 << 20)) return 0;
    return (size_t)grad_blocks(m, n) * n * 4;
}

gs_status gs_rms_norm_bwd(const gs_rms_norm_grads *p, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = grads_ok(p);
    if (st != GS_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    if (p->m == 0) {
        if (!p->dgamma || p->accumulate) return GS_OK;
        zero_floats<<<(p->n + kThreads - 1) / kThreads, kThreads, 0, s>>>(p->dgamma, p->n);
        return from_hip(hipGetLastError());
    }
    if (p->dgamma) {
        if (workspace_bytes < gs_rms_norm_bwd_workspace_bytes(p->m, p->n)) return GS_ERR_WORKSPACE;
        if (!workspace || !aligned_to(workspace, 16)) return GS_ERR_INVALID_ARG;
    }
    GradArgs a;
    a.sum = p->sum;
    a.dy = p->dy;
    a.dsum = p->dsum;
    a.rstd = p->rstd;
    a.gamma = p->gamma;
    a.dx = p->dx;
    const int blocks = grad_blocks(p->m, p->n);
    const bool add = p->dgamma && (blocks > 1 || p->accumulate);
    a.part = add ? static_cast<float *>(workspace) : p->dgamma;
    a.m = p->m;
    a.lds = p->sum_stride;
    a.ldy = p->dy_stride;
    a.ldds = p->dsum_stride;
    a.ldx = p->dx_stride;
    a.n = p->n;
    hipError_t e = p->dtype == GS_DTYPE_F32 ? launch_grad<float>(a, s)
                   : p->dtype == GS_DTYPE_F16 ? launch_grad<_Float16>(a, s) : launch_grad<__bf16>(a, s);
    if (e == hipSuccess && add) e = launch_sum_rows(a.part, p->dgamma, p->n, blocks, p->accumulate, s);
    return from_hip(e);
}

}  // extern "C"
