// Group norm with an activation over feature maps whose channels are
// contiguous, its input kept in 8-bit blocks for the backward, and the backward.
//
// HBM-bound: the forward has to read x and write y, the backward to read x (or
// its 8-bit checkpoint) and dy and write dx; both need sums over a whole image
// first, so what they read is read twice, the second time out of the last-level
// cache while it fits.  A thread keeps eight consecutive channels (16 bytes of a
// 16-bit type) and walks over pixels, so that statistics, gamma and beta stay in
// registers and any group size costs the same.  Images of up to 16K values (64K of
// many) are one workgroup's, in one launch; larger ones take two or three: sums
// of blocks of pixels, joined per group, then the results.
//
// A channel's values are taken as differences from a shift, the mean of eight of its
// pixels spread over the image, which every workgroup forms alike: an offset that
// is large beside the spread costs no bits.  The shift need not be typical (all eight
// may lie on a border): a part of the pixels is its sum S and its squares M about its own
// mean, and parts of n_i values with the mean m join as S = sum S_i,
// M = sum (M_i + n_i (S_i / n_i - m)^2), so that M never holds more than the spread
// itself; single values are the smallest part.  (Sums of squares about the shift, two
// operations a value less: with those eight pixels at 0 and 65528 at 4096 +- 1
// rstd was off by 1.2e-3, now by 2e-7; 8 x 65536 x 128 with checkpoint took 110 us, now 112.)
// Channels are joined in fp64, relative to their group's first one.  Everything is summed in
// a fixed order.
#include "gs_numeric.h"

#include <algorithm>

namespace gsi {
namespace {

constexpr int kThreads = 256, kOneThreads = 512;
// Four workgroups to a CU, one round (8 x 16384 x 256 backward from 8 bits 66 us, 68 with
// two; 8 x 65536 x 128 forward 112 and 117, and 151 with five for four).
constexpr int kBlocks = 1024;
// Results that the second-level caches do not hold are written past them
// (8 x 16384 x 256 backward 79 -> 73 us); smaller ones stay for who reads them next.
constexpr int64_t kStreamBytes = 32 << 20;
// Channels of a workgroup, in eights, where an image is many workgroups': more
// would leave each few pixels, and sums as large as what they are sums of.
constexpr int kTileChunks = 32;
constexpr int kJoinChannels = 1024, kJoinBlocks = 32;
constexpr int kTurn = 17;                       // a thread's 16 sums in LDS, in banks of their own (one workgroup, 256 x 64: 9.2 -> 8.8 us)
constexpr int kHeld = 4;                        // pixels a thread of a single workgroup keeps
constexpr int64_t kOneChunks = 8192;            // of eight channels: an image of one workgroup

bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }
gs_status from_hip(hipError_t e) { return e == hipSuccess ? GS_OK : GS_ERR_HIP; }

struct Args {
    const void *x, *dy;
    const uint8_t *x_scales;                    // x in 8-bit blocks, or NULL
    void *y;                                    // y, or dx
    uint8_t *kept, *kept_scales;
    const float *gamma, *beta;
    float *mean, *rstd;                         // [n][groups]
    float *part;                                // [n][blocks][c][2] sums of blocks of pixels (forward: S and M)
    float *shift;                               // forward: [n][c] what the sums' values are relative to
    float *sums;                                // [n][c][2] those of an image
    float *means;                               // backward: [n][groups][2] means of g and g h
    float *dgamma, *dbeta;
    int64_t x_image, x_pixel, xs_image, xs_pixel, dy_image, dy_pixel, y_image, y_pixel, k_image, k_pixel, ks_image, ks_pixel;
    int64_t p, per, per_out;                    // pixels of an image, of a block that sums, of one that writes
    int n, c, groups, cg, ct, tiles;            // ct: chunks of a block's channels; tiles of them
    int blocks, blocks_out, act, accumulate;
    int stream;                                 // results are written past the caches
    float eps;
};

// A thread's place: eight channels from `at` on, pixels sub, sub + step, ..  The
// last chunk of c channels (8 or more) takes the last eight, so that every load is
// a whole vector: its first `skip` are the chunk's before it and go no further.
struct Place {
    int at, skip, sub, step;
    bool works;
};
template <int THREADS> __device__ __forceinline__ Place place_of(const Args &a, int tile)
{
    Place t;
    t.step = THREADS / a.ct;
    t.sub = threadIdx.x / a.ct;
    const int c = (tile * a.ct + threadIdx.x - t.sub * a.ct) * 8;
    t.works = t.sub < t.step && c < a.c;
    t.at = max(0, min(c, a.c - 8));
    t.skip = t.works ? c - t.at : 0;
    return t;
}

template <typename T> __device__ __forceinline__ Vec<T, 8> load(const T *p, const Args &a)
{
    if (a.c >= 8) return *reinterpret_cast<const Vec<T, 8> *>(p);
    Vec<T, 8> w = {};
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < a.c) w.v[j] = p[j];
    return w;
}
template <typename T> constexpr int type_of() { return sizeof(T) == 4 ? GS_DTYPE_F32 : __is_same(T, _Float16) ? GS_DTYPE_F16 : GS_DTYPE_BF16; }
template <typename T> __device__ __forceinline__ void store(T *p, const Place &t, const Args &a, const float v[8])
{
    if (t.skip == 0 && a.c >= 8) {
        if (a.stream) store8_stream(p, type_of<T>(), 0, v);
        else store8_vec(p, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j >= t.skip && j < a.c) p[j] = (T)v[j];
}
// x of the backward as it is stored: its own type, or 8-bit blocks.
template <typename T, bool Q8> struct Stored {
    Vec<T, 8> w;
    __device__ __forceinline__ void values(float v[8]) const
    {
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = (float)w.v[j];
    }
};
template <typename T> struct Stored<T, true> {
    Vec<uint8_t, 8> w;
    uint8_t s;
    __device__ __forceinline__ void values(float v[8]) const
    {
        typedef float f2 __attribute__((ext_vector_type(2)));
        const float scale = e8m0_value(s);
        const uint2 u = __builtin_bit_cast(uint2, w);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int x = (int)(j ? u.y : u.x);
            const f2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(x, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(x, true);
            v[4 * j] = lo[0] * scale;
            v[4 * j + 1] = lo[1] * scale;
            v[4 * j + 2] = hi[0] * scale;
            v[4 * j + 3] = hi[1] * scale;
        }
    }
};

// For every pixel of the thread in [p0, p1): fetch(pixel) of up to N of them, then
// use(pixel, what was fetched) of each.
template <int N, class F, class U> __device__ __forceinline__ void each_pixel(const Place &t, int64_t p0, int64_t p1, F fetch, U use)
{
    int64_t p = p0 + t.sub;
    for (; p + (int64_t)(N - 1) * t.step < p1; p += (int64_t)N * t.step) {
        decltype(fetch(p)) w[N];
#pragma unroll
        for (int i = 0; i < N; i++) w[i] = fetch(p + (int64_t)i * t.step);
#pragma unroll
        for (int i = 0; i < N; i++) use(p + (int64_t)i * t.step, w[i]);
    }
    if (p >= p1) return;
    decltype(fetch(p)) w[N];                    // the last ones, fewer than N
#pragma unroll
    for (int i = 0; i < N; i++)
        if (p + (int64_t)i * t.step < p1) w[i] = fetch(p + (int64_t)i * t.step);
#pragma unroll
    for (int i = 0; i < N; i++)
        if (p + (int64_t)i * t.step < p1) use(p + (int64_t)i * t.step, w[i]);
}

// ---- forward -------------------------------------------------------------------
// One over a number of pixels (of none: 1), to an ulp.
__device__ __forceinline__ float one_over(float n) { return __builtin_amdgcn_rcpf(fmaxf(n, 1.0f)); }

// A part of the pixels, n of them, or {}: none.
struct Moments {
    float s, q, n, mean;

    __device__ __forceinline__ void add(const Moments &w)
    {
        const float share = one_over(n + w.n), e = w.mean - mean;
        q = fmaf(e * (n * w.n * share), e, q + w.q);
        s += w.s;
        n += w.n;
        mean = s * share;
    }
    // K parts at once.
    template <int K> __device__ __forceinline__ void add(const Moments (&w)[K])
    {
        Moments t = {};
#pragma unroll
        for (int i = 0; i < K; i++) {
            t.s += w[i].s;
            t.q += w[i].q;
            t.n += w[i].n;
        }
        t.mean = t.s * one_over(t.n);
#pragma unroll
        for (int i = 0; i < K; i++) {
            const float e = w[i].mean - t.mean;
            t.q = fmaf(e * w[i].n, e, t.q);
        }
        add(t);
    }
};

// What the sums of the thread's channels are relative to.
template <typename T> __device__ __forceinline__ void shift_of(const Args &a, int64_t image, const Place &t, float shift[8])
{
    Vec<T, 8> v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = load(static_cast<const T *>(a.x) + image * a.x_image + ((a.p * i) >> 3) * a.x_pixel + t.at, a);
#pragma unroll
    for (int j = 0; j < 8; j++) {
        shift[j] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) shift[j] += (float)v[i].v[j];
        shift[j] *= 0.125f;
    }
}

// One more pixel in S and M of a thread's channels: with its difference e from the mean
// of the n before, M grows by n / (n + 1) e^2.
template <typename T> struct ThreadMoments {
    float s[8], q[8], n, share;                 // share: one over n

    __device__ __forceinline__ void add(const Vec<T, 8> &w, const float shift[8])
    {
        const float before = share;
        n += 1.0f;
        share = one_over(n);
        const float weight = 1.0f - share;
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float d = (float)w.v[j] - shift[j], e = fmaf(-s[j], before, d);
            q[j] = fmaf(e * weight, e, q[j]);
            s[j] += d;
        }
    }
};

// Adds what the threads of a workgroup that share a chunk have for its
// channels: channel i's two sums in LDS out[2 i ..].  MOMENTS: they are S and M of the
// thread's share of `pixels`, and of all of these in the end.
template <int THREADS, bool MOMENTS> __device__ __forceinline__ void join_threads(const Args &a, const Place &t, int c0, int64_t pixels, const float s[8], const float q[8], float (*turn)[kTurn], float *out)
{
#pragma unroll
    for (int j = 0; j < 8; j++) {
        turn[threadIdx.x][j] = s[j];
        turn[threadIdx.x][8 + j] = q[j];
    }
    // the first `more` rows of threads have one pixel more than the others
    const int each = (int)pixels / t.step, more = (int)pixels - each * t.step;
    const float share = one_over((float)each), share_more = one_over((float)(each + 1));
    __syncthreads();
    // a channel's rows by as many threads as there are to a channel, a power of
    // two of neighbours
    const int all = a.ct * 8;
    int parts = 1;
    while (parts < 8 && parts * 2 * all <= THREADS) parts *= 2;
    for (int k = threadIdx.x; k < all * parts; k += THREADS) {
        const int i = k / parts, chunk = i >> 3, j = (i & 7) + max(0, min(c0 + chunk * 8, a.c) + 8 - max(a.c, 8));
        const int rows = c0 + i < a.c ? t.step : 0;
        float u = 0.0f, v = 0.0f;
        if constexpr (MOMENTS) {
            Moments sum = {};
            for (int r = k & (parts - 1); r < rows; r += 4 * parts) {
                Moments w[4] = {};
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int row = r + h * parts;
                    if (row >= rows) continue;
                    const float x = turn[row * a.ct + chunk][j];
                    w[h] = {x, turn[row * a.ct + chunk][8 + j], (float)(each + (row < more)), x * (row < more ? share_more : share)};
                }
                sum.add(w);
            }
            u = sum.s;
            for (int o = parts / 2; o > 0; o >>= 1) u += __shfl_xor(u, o);
            const float e = sum.mean - u * one_over((float)(int)pixels);
            v = fmaf(e * sum.n, e, sum.q);
        } else {
            for (int r = k & (parts - 1); r < rows; r += parts) {
                u += turn[r * a.ct + chunk][j];
                v += turn[r * a.ct + chunk][8 + j];
            }
            for (int o = parts / 2; o > 0; o >>= 1) u += __shfl_xor(u, o);
        }
        for (int o = parts / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
        if ((k & (parts - 1)) == 0) {
            out[2 * i] = u;
            out[2 * i + 1] = v;
        }
    }
    __syncthreads();
}

// One block of pixels by one tile of channels.
struct Part {
    int64_t image;
    int block, tile;
    bool there;
};
__device__ __forceinline__ Part part_of(const Args &a, int blocks)
{
    int64_t b = block_of();
    Part w;
    w.there = b < (int64_t)a.n * blocks * a.tiles;
    w.tile = (int)(b % a.tiles);
    b /= a.tiles;
    w.block = (int)(b % blocks);
    w.image = b / blocks;
    return w;
}

template <typename T> __global__ __launch_bounds__(kThreads, 4) void sum_moments(Args a)
{
    __shared__ float turn[kThreads][kTurn], out[kTileChunks * 16];
    const Part w = part_of(a, a.blocks);
    if (!w.there) return;
    const int64_t p0 = w.block * a.per, p1 = min(a.p, p0 + a.per);
    const Place t = place_of<kThreads>(a, w.tile);
    float shift[8];
    ThreadMoments<T> m = {};
    if (t.works) {
        shift_of<T>(a, w.image, t, shift);
        const T *x = static_cast<const T *>(a.x) + w.image * a.x_image + t.at;
        each_pixel<8>(t, p0, p1, [&](int64_t p) { return load(x + p * a.x_pixel, a); }, [&](int64_t, const Vec<T, 8> &v) { m.add(v, shift); });
        if (w.block == 0 && t.sub == 0)
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j >= t.skip && j < a.c) a.shift[w.image * a.c + t.at + j] = shift[j];
    }
    const int c0 = w.tile * a.ct * 8, wide = 2 * min(a.ct * 8, a.c - c0);
    join_threads<kThreads, true>(a, t, c0, p1 - p0, m.s, m.q, turn, out);
    float *part = a.part + ((w.image * a.blocks + w.block) * a.c + c0) * 2;
    for (int i = threadIdx.x; i < wide; i += kThreads) part[i] = out[i];
}

// Sum over the threads of a workgroup.
template <int THREADS, typename T> __device__ __forceinline__ T block_sum(T x, T *lds)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
    __syncthreads();                            // the last use of lds is over
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 64; w++) x += lds[w];
    return x;
}

// A group's channels: the sums of their means' distances from the first channel's shift and of
// their squares about it.  In fp64, as channels may lie far apart and the mean is good to
// its own rounding then (in fp32 it was off by 4e-5 for channels of -1000 to 1000).
struct Group {
    double m, q;

    __device__ __forceinline__ void add(float shift, float first, float s, float q1, double pixels, double share)
    {
        const double far = (double)shift - (double)first + (double)s * share;
        m += far;
        q += fma(far * far, pixels, (double)q1);
    }
    // mean and rstd of cg channels
    __device__ __forceinline__ float2 statistics(float first, int cg, double pixels, double share, float eps) const
    {
        const double part = 1.0 / (double)cg, far = m * part;
        const float var = (float)(fma(q * part, share, -far * far));
        return float2{(float)((double)first + far), 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps)};
    }
};

// S and M of a channel over the blocks of pixels b, b + step, .. , eight loads on their way at once.
__device__ __forceinline__ Moments block_moments(const Args &a, const float2 *part, int b, int step)
{
    const float pixels = (float)(int)a.per, last = (float)(int)(a.p - (a.blocks - 1) * a.per), share = one_over(pixels), share_last = one_over(last);
    Moments sum = {};
    for (; b < a.blocks; b += 8 * step) {
        Moments w[8] = {};
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int k = b + i * step;
            const float2 x = k < a.blocks ? part[(int64_t)k * a.c] : float2{0.0f, 0.0f};
            w[i] = {x.x, x.y, k < a.blocks - 1 ? pixels : k < a.blocks ? last : 0.0f, x.x * (k < a.blocks - 1 ? share : share_last)};
        }
        sum.add(w);
    }
    return sum;
}

// Adds a group's channels' two sums over the blocks of pixels, up to 256 channels
// at a time by as many rows of threads as fit; each(channel, sums) in one thread.
template <class F> __device__ __forceinline__ void join_blocks(const Args &a, int64_t image, int g, float (*turn)[2], F each)
{
    const float *part = a.part + (image * a.blocks * a.c + (int64_t)g * a.cg) * 2;
    for (int c0 = 0; c0 < a.cg; c0 += kThreads) {
        const int wide = min(kThreads, a.cg - c0), step = kThreads / wide, sub = threadIdx.x / wide, c = c0 + threadIdx.x - sub * wide;
        float u = 0.0f, v = 0.0f;
        if (sub < step)
            for (int b = sub; b < a.blocks; b += step) {
                u += part[((int64_t)b * a.c + c) * 2];
                v += part[((int64_t)b * a.c + c) * 2 + 1];
            }
        __syncthreads();
        turn[threadIdx.x][0] = u;
        turn[threadIdx.x][1] = v;
        __syncthreads();
        if (sub) continue;
        for (int r = 1; r < step; r++) {
            u += turn[r * wide + threadIdx.x][0];
            v += turn[r * wide + threadIdx.x][1];
        }
        each(g * a.cg + c, u, v);
    }
}
// Their S and M in the same way.
template <class F> __device__ __forceinline__ void join_block_moments(const Args &a, int64_t image, int g, Moments *turn, F each)
{
    const float2 *part = reinterpret_cast<const float2 *>(a.part) + image * a.blocks * a.c + (int64_t)g * a.cg;
    for (int c0 = 0; c0 < a.cg; c0 += kThreads) {
        const int wide = min(kThreads, a.cg - c0), step = min(kThreads / wide, (a.blocks + 7) / 8), sub = threadIdx.x / wide, c = c0 + threadIdx.x - sub * wide;
        Moments sum = {};
        if (sub < step) sum = block_moments(a, part + c, sub, step);
        __syncthreads();
        turn[threadIdx.x] = sum;
        __syncthreads();
        if (sub) continue;
        for (int r = 1; r < step; r += 4) {
            Moments w[4] = {};
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (r + i < step) w[i] = turn[(r + i) * wide + threadIdx.x];
            sum.add(w);
        }
        each(g * a.cg + c, sum.s, sum.q);
    }
}

// A group's statistics by a workgroup, where those that write do not join them themselves.
__global__ __launch_bounds__(kThreads) void join_groups(Args a)
{
    __shared__ Moments turn[kThreads];
    __shared__ double lds[kThreads / 64];
    const int64_t item = block_of();
    if (item >= (int64_t)a.n * a.groups) return;
    const int64_t image = item / a.groups;
    const int g = (int)(item - image * a.groups);
    const float *shift = a.shift + image * a.c, first = shift[(int64_t)g * a.cg];
    const double pixels = (double)a.p, share = 1.0 / pixels;
    Group sum = {};
    join_block_moments(a, image, g, turn, [&](int c, float s, float q) { sum.add(shift[c], first, s, q, pixels, share); });
    sum.m = block_sum<kThreads>(sum.m, lds);
    sum.q = block_sum<kThreads>(sum.q, lds);
    if (threadIdx.x) return;
    const float2 w = sum.statistics(first, a.cg, pixels, share, a.eps);
    a.mean[item] = w.x;
    a.rstd[item] = w.y;
}

// y (and the 8-bit x) of one pixel's eight channels.
template <typename T, int G> __device__ __forceinline__ void emit_one(const Args &a, int64_t image, int64_t p, const Place &t, const Vec<T, 8> &w, const float mean[G], const float scale[8], const float shift[8])
{
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = (float)w.v[j];
    if (a.kept)
        quantize_chunk(v, a.kept + image * a.k_image + p * a.k_pixel + t.at,
                       (threadIdx.x & 3) == 0 ? a.kept_scales + image * a.ks_image + p * a.ks_pixel + (t.at >> 5) : nullptr);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = fmaf(v[j] - mean[j * G / 8], scale[j], shift[j]);
    activate_all<8, sizeof(T) == 4>(v, a.act);
    store(static_cast<T *>(a.y) + image * a.y_image + p * a.y_pixel + t.at, t, a, v);
}
// Those of the thread's pixels of [p0, p1).
template <typename T, int G> __device__ __forceinline__ void emit(const Args &a, int64_t image, int64_t p0, int64_t p1, const Place &t, const float mean[G],
                                                           const float scale[8], const float shift[8])
{
    const T *x = static_cast<const T *>(a.x) + image * a.x_image + t.at;
    each_pixel<4>(t, p0, p1, [&](int64_t p) { return load(x + p * a.x_pixel, a); },
                  [&](int64_t p, const Vec<T, 8> &w) { emit_one<T, G>(a, image, p, t, w, mean, scale, shift); });
}

// A thread keeps G values of each statistic: 2 where every four channels from a
// multiple of four on are of one group, else 8; channel j's is number j * G / 8.
// Each of them, and its group g: f(i, g).
template <int G, class F> __device__ __forceinline__ void each_group(const Args &a, const Place &t, F f)
{
    int g = t.at / a.cg, left = (g + 1) * a.cg - t.at;
#pragma unroll
    for (int i = 0; i < G; i++) {
        f(i, min(g, a.groups - 1));
        left -= 8 / G;
        if (left <= 0) {
            g++;
            left += a.cg;
        }
    }
}
// Eight values from p[t.at] on, or `other`.
__device__ __forceinline__ void load_channels(const Args &a, const float *p, const Place &t, float other, float v[8])
{
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = other;
    if (!p) return;
    if (a.c >= 8) {
        load8_vec(p + t.at, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (j < a.c) v[j] = p[j];
}
// mean, and rstd gamma in gamma's place, of the thread's channels.
template <int G> __device__ __forceinline__ void coefficients(const Args &a, const float *means, const float *rstds, const Place &t, float mean[G], float scale[8])
{
    float rstd[G];
    each_group<G>(a, t, [&](int i, int g) {
        mean[i] = means[g];
        rstd[i] = rstds[g];
    });
#pragma unroll
    for (int j = 0; j < 8; j++) scale[j] *= rstd[j * G / 8];
}

// Statistics of an image's groups from its channels' sums, a wave per group; all in
// LDS, and in mean and rstd (`keep`).
template <int THREADS> __device__ __forceinline__ void group_statistics(const Args &a, int64_t image, const float *shifts, const float *sums, float *means, float *rstds, bool keep)
{
    const double pixels = (double)a.p, share = 1.0 / pixels;
    for (int g = threadIdx.x >> 6; g < a.groups; g += THREADS / 64) {
        const int c0 = g * a.cg;
        const float first = shifts[c0];
        Group sum = {};
        for (int c = c0 + (threadIdx.x & 63); c < c0 + a.cg; c += 64) sum.add(shifts[c], first, sums[2 * c], sums[2 * c + 1], pixels, share);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            sum.m += __shfl_xor(sum.m, o);
            sum.q += __shfl_xor(sum.q, o);
        }
        if (threadIdx.x & 63) continue;
        const float2 w = sum.statistics(first, a.cg, pixels, share, a.eps);
        means[g] = w.x;
        rstds[g] = w.y;
        if (keep && a.mean) a.mean[image * a.groups + g] = w.x;
        if (keep && a.rstd) a.rstd[image * a.groups + g] = w.y;
    }
    __syncthreads();
}
// An image's channels' sums over its few blocks of pixels, in LDS.
__device__ __forceinline__ void image_sums(const Args &a, int64_t image, float *sums)
{
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
        float u = 0.0f, v = 0.0f;
        const float2 *part = reinterpret_cast<const float2 *>(a.part) + image * a.blocks * a.c + c;
        for (int b = 0; b < a.blocks; b += 8) {            // eight loads on their way at once
            float2 w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = b + i < a.blocks ? part[(int64_t)(b + i) * a.c] : float2{0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                u += w[i].x;
                v += w[i].y;
            }
        }
        sums[2 * c] = u;
        sums[2 * c + 1] = v;
    }
}

// Its channels' S and M over as few.
__device__ __forceinline__ void image_moments(const Args &a, int64_t image, float *sums)
{
    for (int c = threadIdx.x; c < a.c; c += kThreads) {
        const Moments m = block_moments(a, reinterpret_cast<const float2 *>(a.part) + image * a.blocks * a.c + c, 0, 1);
        sums[2 * c] = m.s;
        sums[2 * c + 1] = m.q;
    }
}

// JOIN: every workgroup forms the statistics itself, from few blocks' sums.
template <typename T, int G, bool JOIN> __global__ __launch_bounds__(kThreads, 4) void write_norm(Args a)
{
    __shared__ float sums[JOIN ? 2 * kJoinChannels : 1], shifts[JOIN ? kJoinChannels : 1], means[JOIN ? kJoinChannels : 1], rstds[JOIN ? kJoinChannels : 1];
    const Part w = part_of(a, a.blocks_out);
    if (!w.there) return;
    const Place t = place_of<kThreads>(a, w.tile);
    float mean[G], scale[8], shift[8];
    load_channels(a, a.gamma, t, 1.0f, scale);
    load_channels(a, a.beta, t, 0.0f, shift);
    if constexpr (JOIN) {
        image_moments(a, w.image, sums);
        for (int c = threadIdx.x; c < a.c; c += kThreads) shifts[c] = a.shift[w.image * a.c + c];
        __syncthreads();
        group_statistics<kThreads>(a, w.image, shifts, sums, means, rstds, w.block == 0);
    }
    if (!t.works) return;
    coefficients<G>(a, JOIN ? means : a.mean + w.image * a.groups, JOIN ? rstds : a.rstd + w.image * a.groups, t, mean, scale);
    const int64_t p0 = w.block * a.per_out;
    emit<T, G>(a, w.image, p0, min(a.p, p0 + a.per_out), t, mean, scale, shift);
}

// An image per workgroup; with HELD its values wait in registers, up to kHeld
// pixels a thread, else they are read again.
template <typename T, int G, bool HELD> __global__ __launch_bounds__(kOneThreads) void norm_image(Args a)
{
    __shared__ float turn[kOneThreads][kTurn], out[kOneThreads * 4], shifts[kOneThreads * 2], means[kOneThreads * 2], rstds[kOneThreads * 2];
    const int64_t image = block_of();
    if (image >= a.n) return;
    const Place t = place_of<kOneThreads>(a, 0);
    const T *x = static_cast<const T *>(a.x) + image * a.x_image + t.at;
    Vec<T, 8> held[HELD ? kHeld : 1];
    float near[8], scale[8], shift[8], mean[G];
    ThreadMoments<T> m = {};
    load_channels(a, a.gamma, t, 1.0f, scale);              // on their way early
    load_channels(a, a.beta, t, 0.0f, shift);
    if (t.works) {
        if constexpr (HELD) {
#pragma unroll
            for (int i = 0; i < kHeld; i++)
                if (t.sub + i * t.step < a.p) held[i] = load(x + (int64_t)(t.sub + i * t.step) * a.x_pixel, a);
            shift_of<T>(a, image, t, near);
#pragma unroll
            for (int i = 0; i < kHeld; i++)
                if (t.sub + i * t.step < a.p) m.add(held[i], near);
        } else {
            shift_of<T>(a, image, t, near);
            each_pixel<8>(t, 0, a.p, [&](int64_t p) { return load(x + p * a.x_pixel, a); }, [&](int64_t, const Vec<T, 8> &v) { m.add(v, near); });
        }
        if (t.sub == 0)
#pragma unroll
            for (int j = 0; j < 8; j++)
                if (j >= t.skip && j < a.c) shifts[t.at + j] = near[j];
    }
    join_threads<kOneThreads, true>(a, t, 0, a.p, m.s, m.q, turn, out);
    group_statistics<kOneThreads>(a, image, shifts, out, means, rstds, true);
    if (!t.works) return;
    coefficients<G>(a, means, rstds, t, mean, scale);
    if constexpr (HELD) {
#pragma unroll
        for (int i = 0; i < kHeld; i++)
            if (t.sub + i * t.step < a.p) emit_one<T, G>(a, image, t.sub + i * t.step, t, held[i], mean, scale, shift);
    } else {
        emit<T, G>(a, image, 0, a.p, t, mean, scale, shift);
    }
}

// ---- backward --------------------------------------------------------------------
// What a pixel's eight channels need: x and dy as they are stored.
template <typename T, bool Q8> struct Pair {
    Stored<T, Q8> x;
    Vec<T, 8> dy;
};
// The thread's channels, and the first of its values.
template <typename T, bool Q8, int G> struct Channels {
    float mean[G], rstd[G], gamma[8], beta[8];
    const void *x;
    const uint8_t *scale;
    const T *dy;

    __device__ __forceinline__ void init(const Args &a, int64_t image, const Place &t)
    {
        load_channels(a, a.gamma, t, 1.0f, gamma);
        load_channels(a, a.beta, t, 0.0f, beta);
        each_group<G>(a, t, [&](int i, int g) {
            mean[i] = a.mean[image * a.groups + g];
            rstd[i] = a.rstd[image * a.groups + g];
        });
        dy = static_cast<const T *>(a.dy) + image * a.dy_image + t.at;
        if constexpr (Q8) {
            x = static_cast<const uint8_t *>(a.x) + image * a.x_image + t.at;
            scale = a.x_scales + image * a.xs_image + (t.at >> 5);
        } else {
            x = static_cast<const T *>(a.x) + image * a.x_image + t.at;
        }
    }
    __device__ __forceinline__ Pair<T, Q8> fetch(const Args &a, int64_t p) const
    {
        Pair<T, Q8> w;
        if constexpr (Q8) {                     // c is a multiple of 32
            w.x.w = *reinterpret_cast<const Vec<uint8_t, 8> *>(static_cast<const uint8_t *>(x) + p * a.x_pixel);
            w.x.s = scale[p * a.xs_pixel];
        } else {
            w.x.w = load(static_cast<const T *>(x) + p * a.x_pixel, a);
        }
        w.dy = load(dy + p * a.dy_pixel, a);
        return w;
    }
    // h and dz of a pixel
    __device__ __forceinline__ void gradient(const Args &a, const Pair<T, Q8> &w, float h[8], float dz[8]) const
    {
        float z[8];
        w.x.values(h);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            h[j] = (h[j] - mean[j * G / 8]) * rstd[j * G / 8];
            z[j] = fmaf(h[j], gamma[j], beta[j]);
            dz[j] = (float)w.dy.v[j];
        }
        scale_by_slope<8, sizeof(T) == 4>(dz, z, a.act);
    }
};

// Sums of dz and dz h of a range, per channel, in LDS out[2 i ..].
template <typename T, bool Q8, int G, int THREADS> __device__ __forceinline__ void gradient_sums(const Args &a, const Channels<T, Q8, G> &ch, int64_t p0, int64_t p1, const Place &t, int c0, float (*turn)[kTurn], float *out)
{
    float s[8], sh[8];
#pragma unroll
    for (int j = 0; j < 8; j++) s[j] = sh[j] = 0.0f;
    if (t.works)
        each_pixel<2>(t, p0, p1, [&](int64_t p) { return ch.fetch(a, p); },
                      [&](int64_t, const Pair<T, Q8> &w) {
                          float h[8], dz[8];
                          ch.gradient(a, w, h, dz);
#pragma unroll
                          for (int j = 0; j < 8; j++) {
                              s[j] += dz[j];
                              sh[j] = fmaf(dz[j], h[j], sh[j]);
                          }
                      });
    join_threads<THREADS, false>(a, t, c0, p1 - p0, s, sh, turn, out);
}

template <typename T, bool Q8, int G> __global__ __launch_bounds__(kThreads, 4) void sum_gradients(Args a)
{
    __shared__ float turn[kThreads][kTurn], out[kTileChunks * 16];
    const Part w = part_of(a, a.blocks);
    if (!w.there) return;
    const int64_t p0 = w.block * a.per, p1 = min(a.p, p0 + a.per);
    const Place t = place_of<kThreads>(a, w.tile);
    Channels<T, Q8, G> ch;
    ch.init(a, w.image, t);
    const int c0 = w.tile * a.ct * 8, wide = 2 * min(a.ct * 8, a.c - c0);
    gradient_sums<T, Q8, G, kThreads>(a, ch, p0, p1, t, c0, turn, out);
    float *part = a.part + ((w.image * a.blocks + w.block) * a.c + c0) * 2;
    for (int i = threadIdx.x; i < wide; i += kThreads) part[i] = out[i];
}

// A group's channels' sums over the blocks of pixels, and its means of g and g h.
__global__ __launch_bounds__(kThreads) void join_gradients(Args a)
{
    __shared__ float turn[kThreads][2], lds[kThreads / 64];
    const int64_t item = block_of();
    if (item >= (int64_t)a.n * a.groups) return;
    const int64_t image = item / a.groups;
    const int g = (int)(item - image * a.groups);
    float mg = 0.0f, mgh = 0.0f;
    join_blocks(a, image, g, turn, [&](int c, float s, float sh) {
        a.sums[(image * a.c + c) * 2] = s;
        a.sums[(image * a.c + c) * 2 + 1] = sh;
        const float gamma = a.gamma ? a.gamma[c] : 1.0f;
        mg = fmaf(gamma, s, mg);
        mgh = fmaf(gamma, sh, mgh);
    });
    const float values = (float)a.p * (float)a.cg;
    mg = block_sum<kThreads>(mg, lds);
    mgh = block_sum<kThreads>(mgh, lds);
    if (threadIdx.x) return;
    a.means[2 * item] = mg / values;
    a.means[2 * item + 1] = mgh / values;
}

// dx = rstd (g - mean g - h mean(g h)) of the thread's pixels of [p0, p1).
template <typename T, bool Q8, int G> __device__ __forceinline__ void emit_gradient(const Args &a, const Channels<T, Q8, G> &ch, int64_t image, int64_t p0, int64_t p1, const Place &t, const float *means)
{
    float mg[G], mgh[G];
    each_group<G>(a, t, [&](int i, int g) {
        mg[i] = means[2 * g];
        mgh[i] = means[2 * g + 1];
    });
    T *dx = static_cast<T *>(a.y) + image * a.y_image + t.at;
    each_pixel<2>(t, p0, p1, [&](int64_t p) { return ch.fetch(a, p); },
                  [&](int64_t p, const Pair<T, Q8> &w) {
                      float h[8], dz[8];
                      ch.gradient(a, w, h, dz);
#pragma unroll
                      for (int j = 0; j < 8; j++) dz[j] = ch.rstd[j * G / 8] * fmaf(-h[j], mgh[j * G / 8], fmaf(dz[j], ch.gamma[j], -mg[j * G / 8]));
                      store(dx + p * a.y_pixel, t, a, dz);
                  });
}

// Means of g and g h of an image's groups from its channels' sums, a wave per
// group, in LDS.
template <int THREADS> __device__ __forceinline__ void group_means(const Args &a, const float *sums, float *means)
{
    const float values = (float)a.p * (float)a.cg;
    for (int g = threadIdx.x >> 6; g < a.groups; g += THREADS / 64) {
        float mg = 0.0f, mgh = 0.0f;
        for (int i = threadIdx.x & 63; i < a.cg; i += 64) {
            const int c = g * a.cg + i;
            const float w = a.gamma ? a.gamma[c] : 1.0f;
            mg = fmaf(w, sums[2 * c], mg);
            mgh = fmaf(w, sums[2 * c + 1], mgh);
        }
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) {
            mg += __shfl_xor(mg, o);
            mgh += __shfl_xor(mgh, o);
        }
        if (threadIdx.x & 63) continue;
        means[2 * g] = mg / values;
        means[2 * g + 1] = mgh / values;
    }
    __syncthreads();
}

// The sum over rows of [rows][c] pairs of 16 channels, c0 .. : 16 rows of threads,
// eight loads on their way at once; the result in the first 16 threads.
__device__ __forceinline__ float2 sum_rows_of(const float2 *part, int64_t rows, int c0, int channels, float2 *turn)
{
    const int c = c0 + (threadIdx.x & 15);
    float2 s = {0.0f, 0.0f};
    if (c < channels)
        for (int64_t b = threadIdx.x >> 4; b < rows; b += 8 * 16) {
            float2 w[8];
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = b + i * 16 < rows ? part[(b + i * 16) * channels + c] : float2{0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 8; i++) {
                s.x += w[i].x;
                s.y += w[i].y;
            }
        }
    turn[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x < 16)
#pragma unroll
        for (int r = 1; r < 16; r++) {
            s.x += turn[r * 16 + threadIdx.x].x;
            s.y += turn[r * 16 + threadIdx.x].y;
        }
    return s;
}
// S and M of 16 channels over an image's blocks in the same way.
__device__ __forceinline__ float2 join_rows_of(const Args &a, const float2 *part, int c0, Moments *turn)
{
    const int c = c0 + (threadIdx.x & 15);
    Moments s = {};
    if (c < a.c) s = block_moments(a, part + c, threadIdx.x >> 4, 16);
    turn[threadIdx.x] = s;
    __syncthreads();
    Moments sum = {};
    if (threadIdx.x < 16) {
        Moments w[16] = {};
#pragma unroll
        for (int r = 0; r < 16; r++) w[r] = turn[r * 16 + threadIdx.x];
        sum.add(w);
    }
    return float2{sum.s, sum.q};
}

// A channel's sums over an image's blocks (MOMENTS: S and M): what the workgroups
// that write then join as one block's.
template <bool MOMENTS> __global__ __launch_bounds__(kThreads) void join_channels(Args a, float *to)
{
    __shared__ __align__(16) Moments turn[kThreads];
    const int64_t slices = (a.c + 15) / 16, item = block_of();
    if (item >= a.n * slices) return;
    const int64_t image = item / slices;
    const int c0 = (int)(item - image * slices) * 16;
    const float2 *part = reinterpret_cast<const float2 *>(a.part) + image * a.blocks * a.c;
    const float2 s = MOMENTS ? join_rows_of(a, part, c0, turn) : sum_rows_of(part, a.blocks, c0, a.c, reinterpret_cast<float2 *>(turn));
    if (threadIdx.x < 16 && c0 + (int)threadIdx.x < a.c) reinterpret_cast<float2 *>(to)[image * a.c + c0 + threadIdx.x] = s;
}

// dgamma and dbeta of 16 channels: sums over the `rows` of images, or of images'
// blocks.
__device__ __forceinline__ void sum_images(const Args &a, const float *sums, int64_t rows, int64_t block, float2 *turn)
{
    if (block * 16 >= a.c) return;
    const float2 s = sum_rows_of(reinterpret_cast<const float2 *>(sums), rows, (int)block * 16, a.c, turn);
    const int64_t c = block * 16 + threadIdx.x;
    if (threadIdx.x >= 16 || c >= a.c) return;
    if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + s.x : s.x;
    if (a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + s.y : s.y;
}

template <typename T, bool Q8, int G, bool JOIN> __global__ __launch_bounds__(kThreads, 4) void write_gradient(Args a)
{
    __shared__ __align__(8) float sums[JOIN ? 2 * kJoinChannels : 2 * kThreads], means[JOIN ? 2 * kJoinChannels : 1];
    const Part w = part_of(a, a.blocks_out);
    if (!w.there) {
        sum_images(a, JOIN ? a.part : a.sums, JOIN ? (int64_t)a.n * a.blocks : a.n, block_of() - (int64_t)a.n * a.blocks_out * a.tiles,
                   reinterpret_cast<float2 *>(sums));
        return;
    }
    const Place t = place_of<kThreads>(a, w.tile);
    Channels<T, Q8, G> ch;
    ch.init(a, w.image, t);
    if constexpr (JOIN) {
        image_sums(a, w.image, sums);
        __syncthreads();
        group_means<kThreads>(a, sums, means);
    }
    if (!t.works) return;
    const int64_t p0 = w.block * a.per_out;
    emit_gradient<T, Q8, G>(a, ch, w.image, p0, min(a.p, p0 + a.per_out), t, JOIN ? means : a.means + w.image * a.groups * 2);
}

// An image per workgroup; dgamma and dbeta of a single image at once.
template <typename T, bool Q8, int G> __global__ __launch_bounds__(kOneThreads) void gradient_image(Args a)
{
    __shared__ float turn[kOneThreads][kTurn], out[kOneThreads * 4], means[kOneThreads * 4];
    const int64_t image = block_of();
    if (image >= a.n) return;
    const Place t = place_of<kOneThreads>(a, 0);
    Channels<T, Q8, G> ch;
    ch.init(a, image, t);
    gradient_sums<T, Q8, G, kOneThreads>(a, ch, 0, a.p, t, 0, turn, out);
    group_means<kOneThreads>(a, out, means);
    for (int c = threadIdx.x; c < a.c; c += kOneThreads) {
        if (a.sums) {
            a.sums[(image * a.c + c) * 2] = out[2 * c];
            a.sums[(image * a.c + c) * 2 + 1] = out[2 * c + 1];
        } else {
            if (a.dbeta) a.dbeta[c] = a.accumulate ? a.dbeta[c] + out[2 * c] : out[2 * c];
            if (a.dgamma) a.dgamma[c] = a.accumulate ? a.dgamma[c] + out[2 * c + 1] : out[2 * c + 1];
        }
    }
    if (t.works) emit_gradient<T, Q8, G>(a, ch, image, 0, a.p, t, means);
}

__global__ __launch_bounds__(kThreads) void sum_images_alone(Args a)
{
    __shared__ float2 turn[kThreads];
    sum_images(a, a.sums, a.n, blockIdx.x, turn);
}

__global__ __launch_bounds__(kThreads) void zero_two(float *p, float *q, int n)
{
    const int i = blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    if (p) p[i] = 0.0f;
    if (q) q[i] = 0.0f;
}

// ---- plan -------------------------------------------------------------------------
constexpr size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

struct Shape {
    int64_t n, p;
    int c, groups;
};
struct Plan {
    bool one;                                   // an image per workgroup
    int ct, tiles, blocks, blocks_out;
    int64_t per, per_out;
};
// Blocks of pixels so that about `want` workgroups run, each thread with at least
// `least` pixels.
void cut(const Shape &s, const Plan &w, int64_t want, int least, int &blocks, int64_t &per)
{
    const int64_t step = kThreads / w.ct, rows = (s.p + step * least - 1) / (step * least);
    const int64_t b = std::max<int64_t>(1, std::min<int64_t>(rows, want / std::max<int64_t>(1, s.n * w.tiles)));
    per = (s.p + b - 1) / b;
    blocks = (int)((s.p + per - 1) / per);
}
Plan plan_of(const Shape &s)
{
    Plan w;
    const int chunks = (s.c + 7) / 8;
    // one workgroup per image: its values held in registers, or many images
    w.one = chunks <= kOneThreads / 4 && (s.p <= (int64_t)kHeld * (kOneThreads / chunks) || (s.p * chunks <= kOneChunks && s.n >= 128));
    w.tiles = w.one ? 1 : (chunks + kTileChunks - 1) / kTileChunks;
    w.ct = (chunks + w.tiles - 1) / w.tiles;
    if (w.tiles > 1) w.ct = (w.ct + 3) / 4 * 4;                         // whole 8-bit blocks
    if (w.one) {
        w.blocks = w.blocks_out = 1;
        w.per = w.per_out = s.p;
    } else {
        cut(s, w, kBlocks, 2, w.blocks, w.per);
        cut(s, w, kBlocks, 1, w.blocks_out, w.per_out);
    }
    return w;
}

bool shape_ok(int64_t n, int64_t p, int64_t c, int64_t groups)
{
    return n >= 0 && n <= 65535 && p >= 0 && p <= ((int64_t)1 << 30) && c >= 1 && c <= 65536 && groups >= 1 && groups <= c && c % groups == 0;
}

void set_shape(Args &a, const Shape &s, const Plan &w, int es)
{
    a.n = (int)s.n;
    a.p = s.p;
    a.c = s.c;
    a.groups = s.groups;
    a.cg = s.c / s.groups;
    a.ct = w.ct;
    a.tiles = w.tiles;
    a.blocks = w.blocks;
    a.blocks_out = w.blocks_out;
    a.per = w.per;
    a.per_out = w.per_out;
    a.stream = s.n * s.p * s.c * es > kStreamBytes;
}

// Whether the workgroups that write join an image's channels themselves: few blocks'
// sums as they are (3 x 1001 x 90: 17 -> 14 us for the launch less), or, where groups
// are too few or too wide to be joined by a workgroup each, added up per channel
// first.  Else a workgroup joins each group (8 x 65536 x 128: 112 us, 122 by channels).
bool few_blocks(const Args &a) { return a.blocks <= kJoinBlocks && (int64_t)a.n * a.blocks <= 1024; }
bool by_channels(const Args &a) { return a.c <= kJoinChannels && (few_blocks(a) || a.cg > 64 || (int64_t)a.n * a.groups < 64); }
template <bool MOMENTS> Args joined(const Args &a, hipStream_t s)
{
    Args b = a;
    if (few_blocks(a)) return b;
    join_channels<MOMENTS><<<grid_of((int64_t)a.n * ((a.c + 15) / 16), kThreads), kThreads, 0, s>>>(a, a.sums);
    b.part = a.sums;
    b.blocks = 1;
    return b;
}

template <typename T, int G> hipError_t launch_fwd(const Args &a, bool one, hipStream_t s)
{
    if (one) {
        if (a.p <= (int64_t)kHeld * (kOneThreads / a.ct)) norm_image<T, G, true><<<grid_of(a.n, kOneThreads), kOneThreads, 0, s>>>(a);
        else norm_image<T, G, false><<<grid_of(a.n, kOneThreads), kOneThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    sum_moments<T><<<grid_of((int64_t)a.n * a.blocks * a.tiles, kThreads), kThreads, 0, s>>>(a);
    const dim3 out = grid_of((int64_t)a.n * a.blocks_out * a.tiles, kThreads);
    if (by_channels(a)) {
        write_norm<T, G, true><<<out, kThreads, 0, s>>>(joined<true>(a, s));
        return hipGetLastError();
    }
    join_groups<<<grid_of((int64_t)a.n * a.groups, kThreads), kThreads, 0, s>>>(a);
    write_norm<T, G, false><<<out, kThreads, 0, s>>>(a);
    return hipGetLastError();
}
// Two values of a statistic to a thread, or eight (see each_group).
bool by_fours(const Args &a) { return a.cg % 4 == 0; }
template <typename T> hipError_t launch_fwd(const Args &a, bool one, hipStream_t s) { return by_fours(a) ? launch_fwd<T, 2>(a, one, s) : launch_fwd<T, 8>(a, one, s); }

template <typename T, bool Q8, int G> hipError_t launch_bwd(const Args &a, bool one, hipStream_t s)
{
    const bool wanted = a.dgamma || a.dbeta;
    const int sums = (a.c + 15) / 16;
    if (one) {
        gradient_image<T, Q8, G><<<grid_of(a.n, kOneThreads), kOneThreads, 0, s>>>(a);
        if (wanted && a.n > 1) sum_images_alone<<<sums, kThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    sum_gradients<T, Q8, G><<<grid_of((int64_t)a.n * a.blocks * a.tiles, kThreads), kThreads, 0, s>>>(a);
    const dim3 out = grid_of((int64_t)a.n * a.blocks_out * a.tiles + (wanted ? sums : 0), kThreads);
    if (by_channels(a)) {
        write_gradient<T, Q8, G, true><<<out, kThreads, 0, s>>>(joined<false>(a, s));
        return hipGetLastError();
    }
    join_gradients<<<grid_of((int64_t)a.n * a.groups, kThreads), kThreads, 0, s>>>(a);
    write_gradient<T, Q8, G, false><<<out, kThreads, 0, s>>>(a);
    return hipGetLastError();
}
template <typename T, bool Q8> hipError_t launch_bwd(const Args &a, bool one, hipStream_t s) { return by_fours(a) ? launch_bwd<T, Q8, 2>(a, one, s) : launch_bwd<T, Q8, 8>(a, one, s); }
template <typename T> hipError_t launch_bwd(const Args &a, bool one, hipStream_t s) { return a.x_scales ? launch_bwd<T, true>(a, one, s) : launch_bwd<T, false>(a, one, s); }

bool strides_ok(const void *p, int es, int64_t image, int64_t pixel) { return aligned_to(p, es) && image >= 0 && pixel >= 0; }
// Whether the values of a result [n][p][wide] all have places of their own.
bool apart(int64_t n, int64_t p, int64_t wide, int64_t image, int64_t pixel)
{
    __int128 extent = wide;
    const bool pixels_first = pixel <= image;
    for (int i = 0; i < 2; i++) {
        const bool pixels = pixels_first == (i == 0);
        const int64_t count = pixels ? p : n, stride = pixels ? pixel : image;
        if (count <= 1) continue;
        if (stride < extent) return false;
        extent += (__int128)stride * (count - 1);
    }
    return true;
}

gs_status check(const gs_group_norm *a)
{
    if (!a || !shape_ok(a->n, a->p, a->c, a->groups) || !float_type(a->dtype) || a->activation < GS_ACT_NONE || a->activation > GS_ACT_GELU) return GS_ERR_INVALID_ARG;
    if (!(a->eps >= 0.0f) || !(a->eps < INFINITY)) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(a->dtype);
    if (!strides_ok(a->x, es, a->x_image, a->x_pixel) || !strides_ok(a->y, es, a->y_image, a->y_pixel) || !apart(a->n, a->p, a->c, a->y_image, a->y_pixel))
        return GS_ERR_INVALID_ARG;
    if (!aligned_to(a->gamma, 4) || !aligned_to(a->beta, 4) || !aligned_to(a->mean, 4) || !aligned_to(a->rstd, 4)) return GS_ERR_INVALID_ARG;
    if (a->n > 0 && a->p > 0 && (!a->x || !a->y)) return GS_ERR_INVALID_ARG;
    if (!a->kept != !a->kept_scales) return GS_ERR_INVALID_ARG;
    if (a->kept && (a->c % 32 || !strides_ok(a->kept, 1, a->kept_image, a->kept_pixel) || !strides_ok(a->kept_scales, 1, a->kept_scales_image, a->kept_scales_pixel) ||
                    !apart(a->n, a->p, a->c, a->kept_image, a->kept_pixel) || !apart(a->n, a->p, a->c / 32, a->kept_scales_image, a->kept_scales_pixel)))
        return GS_ERR_INVALID_ARG;
    return GS_OK;
}

gs_status check(const gs_group_norm_grads *a)
{
    if (!a || !shape_ok(a->n, a->p, a->c, a->groups) || !float_type(a->dtype) || a->activation < GS_ACT_NONE || a->activation > GS_ACT_GELU) return GS_ERR_INVALID_ARG;
    const int es = dtype_bytes(a->dtype);
    if (a->x_dtype != a->dtype && a->x_dtype != GS_DTYPE_MXFP8) return a->x_dtype >= 0 && a->x_dtype <= GS_DTYPE_MXFP8 ? GS_ERR_UNSUPPORTED : GS_ERR_INVALID_ARG;
    const bool q8 = a->x_dtype == GS_DTYPE_MXFP8;
    if (!strides_ok(a->x, q8 ? 1 : es, a->x_image, a->x_pixel) || !strides_ok(a->dy, es, a->dy_image, a->dy_pixel) || !strides_ok(a->dx, es, a->dx_image, a->dx_pixel) ||
        !apart(a->n, a->p, a->c, a->dx_image, a->dx_pixel))
        return GS_ERR_INVALID_ARG;
    if (q8 && (a->c % 32 || !strides_ok(a->x_scales, 1, a->x_scales_image, a->x_scales_pixel))) return GS_ERR_INVALID_ARG;
    if (!aligned_to(a->gamma, 4) || !aligned_to(a->beta, 4) || !aligned_to(a->mean, 4) || !aligned_to(a->rstd, 4) || !aligned_to(a->dgamma, 4) || !aligned_to(a->dbeta, 4))
        return GS_ERR_INVALID_ARG;
    if (a->n > 0 && a->p > 0 && (!a->x || !a->dy || !a->dx || !a->mean || !a->rstd || (q8 && !a->x_scales))) return GS_ERR_INVALID_ARG;
    return GS_OK;
}

// Partial sums, and what the calls keep per image: statistics (forward), or sums
// and means (backward).
size_t part_bytes(const Shape &s, const Plan &w) { return w.one ? 0 : round256((size_t)s.n * w.blocks * s.c * 8); }

}  // namespace
}  // namespace gsi

using namespace gsi;

extern "C" {

size_t gs_group_norm_fwd_workspace_bytes(int64_t n, int64_t p, int32_t c, int32_t groups)
{
    if (!shape_ok(n, p, c, groups) || n == 0 || p == 0) return 0;
    const Shape s = {n, p, c, groups};
    const Plan w = plan_of(s);
    return w.one ? 0 : part_bytes(s, w) + 2 * round256((size_t)n * groups * 4) + round256((size_t)n * c * 4) + round256((size_t)n * c * 8);
}

gs_status gs_group_norm_fwd(const gs_group_norm *p, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = check(p);
    if (st != GS_OK) return st;
    if (p->n == 0 || p->p == 0) return GS_OK;
    const Shape shape = {p->n, p->p, p->c, p->groups};
    const Plan w = plan_of(shape);
    const size_t need = gs_group_norm_fwd_workspace_bytes(p->n, p->p, p->c, p->groups);
    if (workspace_bytes < need) return GS_ERR_WORKSPACE;
    if (need && (!workspace || !aligned_to(workspace, 16))) return GS_ERR_INVALID_ARG;
    Args a = {};
    set_shape(a, shape, w, dtype_bytes(p->dtype));
    a.x = p->x;
    a.x_image = p->x_image;
    a.x_pixel = p->x_pixel;
    a.y = p->y;
    a.y_image = p->y_image;
    a.y_pixel = p->y_pixel;
    a.kept = p->kept;
    a.k_image = p->kept_image;
    a.k_pixel = p->kept_pixel;
    a.kept_scales = p->kept_scales;
    a.ks_image = p->kept_scales_image;
    a.ks_pixel = p->kept_scales_pixel;
    a.gamma = p->gamma;
    a.beta = p->beta;
    a.mean = p->mean;
    a.rstd = p->rstd;
    a.act = p->activation;
    a.eps = p->eps;
    if (!w.one) {
        char *ws = static_cast<char *>(workspace);
        a.part = reinterpret_cast<float *>(ws);
        const size_t at = part_bytes(shape, w), one = round256((size_t)p->n * p->groups * 4);
        if (!a.mean) a.mean = reinterpret_cast<float *>(ws + at);
        if (!a.rstd) a.rstd = reinterpret_cast<float *>(ws + at + one);
        a.shift = reinterpret_cast<float *>(ws + at + 2 * one);
        a.sums = reinterpret_cast<float *>(ws + at + 2 * one + round256((size_t)p->n * p->c * 4));
    }
    hipStream_t s = (hipStream_t)stream;
    return from_hip(p->dtype == GS_DTYPE_F32 ? launch_fwd<float>(a, w.one, s) : p->dtype == GS_DTYPE_F16 ? launch_fwd<_Float16>(a, w.one, s) : launch_fwd<__bf16>(a, w.one, s));
}

size_t gs_group_norm_bwd_workspace_bytes(int64_t n, int64_t p, int32_t c, int32_t groups)
{
    if (!shape_ok(n, p, c, groups) || n == 0 || p == 0) return 0;
    const Shape s = {n, p, c, groups};
    const Plan w = plan_of(s);
    if (w.one && n == 1) return 0;
    return part_bytes(s, w) + round256((size_t)n * c * 8) + (w.one ? 0 : round256((size_t)n * groups * 8));
}

gs_status gs_group_norm_bwd(const gs_group_norm_grads *p, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = check(p);
    if (st != GS_OK) return st;
    hipStream_t s = (hipStream_t)stream;
    if (p->n == 0 || p->p == 0) {
        if (p->accumulate || (!p->dgamma && !p->dbeta)) return GS_OK;
        zero_two<<<(p->c + kThreads - 1) / kThreads, kThreads, 0, s>>>(p->dgamma, p->dbeta, p->c);
        return from_hip(hipGetLastError());
    }
    const Shape shape = {p->n, p->p, p->c, p->groups};
    const Plan w = plan_of(shape);
    const size_t need = gs_group_norm_bwd_workspace_bytes(p->n, p->p, p->c, p->groups);
    if (workspace_bytes < need) return GS_ERR_WORKSPACE;
    if (need && (!workspace || !aligned_to(workspace, 16))) return GS_ERR_INVALID_ARG;
    Args a = {};
    set_shape(a, shape, w, dtype_bytes(p->dtype));
    a.x = p->x;
    a.x_image = p->x_image;
    a.x_pixel = p->x_pixel;
    if (p->x_dtype == GS_DTYPE_MXFP8) {
        a.x_scales = p->x_scales;
        a.xs_image = p->x_scales_image;
        a.xs_pixel = p->x_scales_pixel;
    }
    a.dy = p->dy;
    a.dy_image = p->dy_image;
    a.dy_pixel = p->dy_pixel;
    a.y = p->dx;
    a.y_image = p->dx_image;
    a.y_pixel = p->dx_pixel;
    a.gamma = p->gamma;
    a.beta = p->beta;
    a.mean = const_cast<float *>(p->mean);
    a.rstd = const_cast<float *>(p->rstd);
    a.dgamma = p->dgamma;
    a.dbeta = p->dbeta;
    a.act = p->activation;
    a.accumulate = p->accumulate;
    char *ws = static_cast<char *>(workspace);
    const size_t at = part_bytes(shape, w);
    a.part = reinterpret_cast<float *>(ws);
    a.sums = need ? reinterpret_cast<float *>(ws + at) : nullptr;
    a.means = reinterpret_cast<float *>(ws + at + round256((size_t)p->n * p->c * 8));
    return from_hip(p->dtype == GS_DTYPE_F32 ? launch_bwd<float>(a, w.one, s) : p->dtype == GS_DTYPE_F16 ? launch_bwd<_Float16>(a, w.one, s) : launch_bwd<__bf16>(a, w.one, s));
}

}  // extern "C"
