// Orthogonalised update (Newton-Schulz iterations) of a batch of weight
// matrices, alone and as the momentum step of the weights.
//
// With r = min(rows, cols) and f = max, X is [r][f] (U^T when U is tall) and
// an iteration is three products: A = X X^T, B = b A + c A A^T (A is
// symmetric) and X' = a X + B X.  A and B are formed on one side of the diagonal.  X, A and B
// live in the workspace as bf16 limbs, padded with zeros to multiples of 32,
// and every epilogue writes its result as limbs, so no product converts
// anything: B X reads X by columns, and a tall U is turned round once at each
// end.  fp32 results take three limbs, 16-bit results two: an iteration
// amplifies an error in a weak direction up to |a| times, 2^-16 grows to about
// 2^-11 in five, where one bf16 limb would lose the direction.
//
// A matrix that fits the LDS of a CU is iterated by one workgroup from its
// gradient to its weight.
//
// 4096 x 1024 in bf16, 5 iterations: 352 us (up to 364 with the card's clock; fp16 353, fp32
// 535), each A 20 us and its splits' sum 6, B 11 and X' 30 (860 TFLOP/s of the three
// limb products), momentum, norm and first limbs 24.  8 x 256 x 256 in fp32: 106 us (bf16
// 95), 17 launches of 5 to 7 us; the products are bound by their starts and ends, which
// 32 x 32 tiles on more CUs shorten.
#include <string.h>

#include "gs_gemm.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxNormBlocks = 512;             // partial sums of squares per matrix

bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Update {
    const void *grad;
    const float *momentum;                      // NULL: U = grad
    float *momentum_out;
    int grad_type, nesterov;
    float beta;
    int vec;                                    // size is a multiple of 4
    int64_t size;                               // rows * cols
};

__device__ __forceinline__ void load4(const void *p, int t, int64_t i, float v[4])
{
    if (t == GS_DTYPE_F32) {
        const Vec<float, 4> w = *reinterpret_cast<const Vec<float, 4> *>(static_cast<const float *>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; k++) v[k] = w.v[k];
    } else if (t == GS_DTYPE_F16) {
        const Vec<_Float16, 4> w = *reinterpret_cast<const Vec<_Float16, 4> *>(static_cast<const _Float16 *>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; k++) v[k] = (float)w.v[k];
    } else {
        const Vec<__bf16, 4> w = *reinterpret_cast<const Vec<__bf16, 4> *>(static_cast<const __bf16 *>(p) + i);
#pragma unroll
        for (int k = 0; k < 4; k++) v[k] = (float)w.v[k];
    }
}

// Element i of U once momentum_out is written.
__device__ __forceinline__ float update_at(const Update &u, int64_t i)
{
    if (!u.momentum) return load_as_float(u.grad, u.grad_type, i);
    const float m = u.momentum_out[i];
    return u.nesterov ? fmaf(u.beta, m, load_as_float(u.grad, u.grad_type, i)) : m;
}

// Momentum and the sums of squares of U, one partial sum per workgroup.
// The norm scales every singular value alike and the iterations' polynomial is
// steep between its plateaus, so it is kept in fp64: an fp32 norm's error was
// the largest part of the fp32 result's.
__global__ __launch_bounds__(kThreads) void momentum_and_norm(Update u, double *part)
{
    // 4 consecutive elements a thread and pass where the matrices allow it
    __shared__ double lds[kThreads / 64];
    const int64_t base = (int64_t)blockIdx.y * u.size, stride = (int64_t)gridDim.x * kThreads;
    double sq = 0.0;
    if (u.vec) {
        for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4; i < u.size; i += stride * 4) {
            float g[4];
            load4(u.grad, u.grad_type, base + i, g);
            if (u.momentum) {
                float m[4];
                load4(u.momentum, GS_DTYPE_F32, base + i, m);
#pragma unroll
                for (int k = 0; k < 4; k++) m[k] = fmaf(u.beta, m[k], g[k]);
                *reinterpret_cast<Vec<float, 4> *>(u.momentum_out + base + i) = Vec<float, 4>{{m[0], m[1], m[2], m[3]}};
#pragma unroll
                for (int k = 0; k < 4; k++) g[k] = u.nesterov ? fmaf(u.beta, m[k], g[k]) : m[k];
            }
#pragma unroll
            for (int k = 0; k < 4; k++) sq = fma((double)g[k], (double)g[k], sq);
        }
    } else {
        for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < u.size; i += stride) {
            if (u.momentum)
                u.momentum_out[base + i] = fmaf(u.beta, u.momentum[base + i], load_as_float(u.grad, u.grad_type, base + i));
            const double x = update_at(u, base + i);
            sq = fma(x, x, sq);
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sq += __shfl_xor(sq, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = sq;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.y * gridDim.x + blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

// X = U / (|U| + eps) as limbs [r_pad][f_pad], zeros in the padding; tiles of
// 32 x 32 turned round in LDS when U is tall.
template <int NL>
__global__ __launch_bounds__(kThreads) void normalised_limbs(Update u, const double *part, int parts, float eps, int rows, int cols, int tall,
                                                             uint16_t *x, int64_t ldx, int64_t plane, int64_t batch)
{
    __shared__ float tile[32][33];
    __shared__ double lds[kThreads / 64];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    double sq = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) sq += part[blockIdx.z * parts + i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sq += __shfl_xor(sq, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = sq;
    __syncthreads();
    sq = lds[0] + lds[1] + lds[2] + lds[3];
    const double inv = 1.0 / (sqrt(sq) + (double)eps);
    const int64_t base = (int64_t)blockIdx.z * u.size;
    const int f0 = blockIdx.x * 32, r0 = blockIdx.y * 32;
    // U's rows are f (tall) or r
    const int u0 = tall ? f0 : r0, v0 = tall ? r0 : f0;
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        const int a = u0 + ty + i, b = v0 + tx;
        tile[ty + i][tx] = a < rows && b < cols ? (float)(update_at(u, base + (int64_t)a * cols + b) * inv) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        const float v = tall ? tile[tx][ty + i] : tile[ty + i][tx];
        uint16_t limb[NL];
        split_limbs<NL>(v, limb);
#pragma unroll
        for (int l = 0; l < NL; l++) x[blockIdx.z * batch + l * plane + (int64_t)(r0 + ty + i) * ldx + f0 + tx] = limb[l];
    }
}

// v = alpha sum + beta C, written as limbs or, in the last product, as the
// result.
template <int NL> struct NsEpilogue {
    struct Args {
        float *partial;                         // [batch][splits][q][ld_partial], or NULL: one split
        int64_t ld_partial, split_stride;
        int splits;
        float alpha, beta;
        const uint16_t *c;                      // limbs at q * ld + p, or NULL
        uint16_t *o;
        int64_t ldc, plane_c, batch_c, ldo, plane_o, batch_o;
        // last product
        void *out;
        const void *weight;
        int out_type, tall, rows, cols;
        float decay, rate;                      // weight * decay - rate * v
    };

    __device__ static __forceinline__ void write_limbs(const Args &e, int p, int q, const float v[8], int batch)
    {
        Vec<uint16_t, 8> h[NL];
        split_all<NL, 8>(v, h);
        uint16_t *o = e.o + batch * e.batch_o + (int64_t)q * e.ldo + p;
#pragma unroll
        for (int l = 0; l < NL; l++) *reinterpret_cast<Vec<uint16_t, 8> *>(o + l * e.plane_o) = h[l];
    }

    struct Part {};
    __device__ static __forceinline__ void part(const Args &, int, Part &) {}
    struct Ahead { Vec<uint16_t, 8> c[NL]; };   // the limbs of C
    __device__ static __forceinline__ void look_ahead(const Args &e, int p, int q, int batch, Ahead &a)
    {
        if (!e.c || e.partial) return;
        const uint16_t *c = e.c + batch * e.batch_c + (int64_t)q * e.ldc + p;
#pragma unroll
        for (int l = 0; l < NL; l++) a.c[l] = *reinterpret_cast<const Vec<uint16_t, 8> *>(c + l * e.plane_c);
    }

    // v = alpha sum + beta C, in place
    __device__ static __forceinline__ void combine(const Args &e, float v[8], const Ahead &a)
    {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] *= e.alpha;
        if (!e.c) return;
        float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int l = NL - 1; l >= 0; l--)
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] += limb_value(a.c[l].v[i]);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = fmaf(e.beta, w[i], v[i]);
    }

    __device__ static __forceinline__ void write_result(const Args &e, int p, int q, const float v[8], int batch)
    {
        const int64_t base = (int64_t)batch * e.rows * e.cols;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int row = e.tall ? p + i : q, col = e.tall ? q : p + i;
            if (row >= e.rows || col >= e.cols) continue;
            const int64_t at = base + (int64_t)row * e.cols + col;
            float x = v[i];
            if (e.weight) x = load_as_float(e.weight, e.out_type, at) * e.decay - e.rate * x;
            store_from_float(e.out, e.out_type, at, x);
        }
    }

    static constexpr bool kMirror = true;

    __device__ static __forceinline__ void store8(const Args &e, int p, int q, float v[8], const Part &, const Ahead &a, int batch, int split)
    {
        if (e.partial) {
            store8_vec(e.partial + ((int64_t)batch * e.splits + split) * e.split_stride + (int64_t)q * e.ld_partial + p, v);
            return;
        }
        combine(e, v, a);
        if (e.out) write_result(e, p, q, v, batch);
        else write_limbs(e, p, q, v, batch);
    }
    __device__ static __forceinline__ void store_mirror(const Args &e, int p, int q, const float v[8], int batch, int)
    {
        if (!e.partial) write_limbs(e, p, q, v, batch);
    }
    __device__ static __forceinline__ void store1(const Args &, int, int, float, int, int) {}  // never: 8 | P
};

// Sum of the splits of k in their order and the epilogue, 32 rows q of a 64 x 64
// tile a workgroup, 8 p a thread; a symmetric result is summed on one side of
// the diagonal and turned round in LDS for the other.
template <int NL>
__global__ __launch_bounds__(kThreads) void reduce_splits(typename NsEpilogue<NL>::Args e, int P, int Q, int symmetric)
{
    using E = NsEpilogue<NL>;
    __shared__ float tile[32][65];
    int tp, tq;
    const int tiles_p = (P + 63) / 64, t = blockIdx.x / 2, half = blockIdx.x % 2 * 32;
    if (symmetric) {
        gemm::triangle_of(t, tp, tq);
    } else {
        tp = t % tiles_p;
        tq = t / tiles_p;
    }
    const int pl = threadIdx.x % 8 * 8, ql = threadIdx.x / 8, p = tp * 64 + pl, q = tq * 64 + half + ql;
    if (p < P && q < Q) {
        const float *part = e.partial + (int64_t)blockIdx.y * e.splits * e.split_stride + (int64_t)q * e.ld_partial + p;
        typename E::Args whole = e;
        whole.partial = nullptr;
        typename E::Ahead ahead;
        E::look_ahead(whole, p, q, blockIdx.y, ahead);
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 8
        for (int s = 0; s < e.splits; s++) {
            float w[8];
            load8_vec(part + s * e.split_stride, w);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] += w[i];
        }
        E::combine(e, v, ahead);
        if (e.out) E::write_result(e, p, q, v, blockIdx.y);
        else E::write_limbs(e, p, q, v, blockIdx.y);
#pragma unroll
        for (int i = 0; i < 8; i++) tile[ql][pl + i] = v[i];
    }
    if (!symmetric || tp == tq) return;
    __syncthreads();
    // the mirrored tile: p and q change places
    const int mp = tq * 64 + half + threadIdx.x % 4 * 8, mq = tp * 64 + threadIdx.x / 4;
    if (mp >= P || mq >= Q) return;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = tile[threadIdx.x % 4 * 8 + i][threadIdx.x / 4];
    E::write_limbs(e, mp, mq, v, blockIdx.y);
}

// Tile and splits of one product of a batch.
struct NsProduct {
    int tile;                                   // 128, 64 or 32
    int splits;
    double us;                                  // estimated time
};
NsProduct choose(int P, int Q, int K, int batch, bool symmetric, int nl);

// Whether a symmetric product's tiles are multiplied on one side of the diagonal
// only: the sums of splits are taken by 64 x 64, so smaller tiles of them all.
bool one_side(int tile, int splits) { return tile >= 64 || splits == 1; }

// ---- small matrices: all iterations in one workgroup --------------------------
// X and A (then B in its place) stay in LDS as limbs, rows padded by 16 bytes so
// that neither 16 rows of a chunk nor 4 lines of a transposed read meet in a
// bank.  A wave takes pairs of 16 x 16 results side by side; the sums wait in
// registers until every wave has read what they replace.  Bound by LDS reads (9
// fragments for 12 products of fp32) and the barriers' latency: 64 x 64 in fp32
// 35 us, 2 us a product.
constexpr int kSmallThreads = 1024, kSmallWaves = kSmallThreads / 64;
constexpr int kSmallLds = 158 * 1024;
constexpr int kSmallPairs = 4;                  // pairs of results of X per wave

struct Small {
    Update u;
    int rows, cols, tall, r, f, steps;
    float a, b, c, eps, decay, rate;
    void *out;
    const void *weight;
    int out_type;
};

struct LdsMatrix {                              // [limbs][rows][pitch]
    uint16_t *at;
    int pitch, plane;
};

// Limbs of rows x0 .. x0 + 15 at k = 32 kk .. 32 kk + 31; T: of columns x0 ..
template <int NL, bool T> __device__ __forceinline__ void small_fragment(const LdsMatrix &m, int x0, int kk, int lane, gemm::i4 v[NL])
{
    const int g = lane >> 4, r = lane & 15;
#pragma unroll
    for (int l = 0; l < NL; l++) {
        const uint16_t *p = m.at + l * m.plane;
        if constexpr (!T) {
            v[l] = *reinterpret_cast<const gemm::i4 *>(p + (x0 + r) * m.pitch + kk * 32 + g * 8);
        } else {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint16_t *a = p + (kk * 32 + g * 8 + h * 4 + (r >> 2)) * m.pitch + x0 + (r & 3) * 4;
                const int2 w = __builtin_bit_cast(
                    int2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) gemm::s4 *)a));
                v[l][2 * h] = w.x;
                v[l][2 * h + 1] = w.y;
            }
        }
    }
}

// acc[j] = this wave's j-th pair of results, q0[j] .. + 15 by p0[j] .. + 31
template <int NL, int PAIRS, bool PT>
__device__ __forceinline__ void small_product(const LdsMatrix &P, const LdsMatrix &Q, int K, int mine, const int p0[PAIRS], const int q0[PAIRS], int lane,
                                              gemm::f4 acc[PAIRS][2])
{
#pragma unroll
    for (int j = 0; j < PAIRS; j++) acc[j][0] = acc[j][1] = gemm::f4{0, 0, 0, 0};
    asm volatile("" : "+v"(lane));
#pragma unroll 1
    for (int kk = 0; kk < K / 32; kk++) {
#pragma unroll
        for (int j = 0; j < PAIRS; j++) {
            __builtin_amdgcn_sched_barrier(0);          // one pair's fragments in registers at a time
            if (j >= mine) continue;
            gemm::i4 q[NL], p[2][NL];
            small_fragment<NL, false>(Q, q0[j], kk, lane, q);
            small_fragment<NL, PT>(P, p0[j], kk, lane, p[0]);
            small_fragment<NL, PT>(P, p0[j] + 16, kk, lane, p[1]);
#pragma unroll
            for (int order = NL - 1; order >= 0; order--)
#pragma unroll
                for (int l = 0; l <= order; l++)
#pragma unroll
                    for (int i = 0; i < 2; i++) acc[j][i] = gemm::mfma32<gemm::kBF16>(p[i][l], q[order - l], acc[j][i]);
        }
    }
}

// A lane's sums hold p + (0..3) of one q.
template <int NL> __device__ __forceinline__ void small_read(const LdsMatrix &m, int p, int q, float v[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++) v[i] = 0.0f;
#pragma unroll
    for (int l = NL - 1; l >= 0; l--) {
        const gemm::s4 w = *reinterpret_cast<const gemm::s4 *>(m.at + l * m.plane + q * m.pitch + p);
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] += limb_value((uint16_t)w[i]);
    }
}
template <int NL> __device__ __forceinline__ void small_write(const LdsMatrix &m, int p, int q, const gemm::f4 &v)
{
    const float x[4] = {v[0], v[1], v[2], v[3]};
    Vec<uint16_t, 4> w[NL];
    split_all<NL, 4>(x, w);
#pragma unroll
    for (int l = 0; l < NL; l++) *reinterpret_cast<gemm::s4 *>(m.at + l * m.plane + q * m.pitch + p) = __builtin_bit_cast(gemm::s4, w[l]);
}

template <int NL> __global__ __launch_bounds__(kSmallThreads) void small_matrices(Small s)
{
    __shared__ __align__(16) uint16_t lds[kSmallLds / 2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Update &u = s.u;
    const int64_t base = (int64_t)blockIdx.x * u.size;
    const int size = (int)u.size;
    const LdsMatrix X{lds, s.f + 8, s.r * (s.f + 8)}, A{lds + NL * X.plane, s.r + 8, s.r * (s.r + 8)};

    // momentum and the norm in fp64, as for larger matrices
    double sq = 0.0;
#pragma unroll 4
    for (int i = tid; i < size; i += kSmallThreads) {
        if (u.momentum) u.momentum_out[base + i] = fmaf(u.beta, u.momentum[base + i], load_as_float(u.grad, u.grad_type, base + i));
        const double x = update_at(u, base + i);
        sq = fma(x, x, sq);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sq += __shfl_xor(sq, o);
    double *sums = reinterpret_cast<double *>(A.at);
    if (lane == 0) sums[wave] = sq;
    for (int i = tid; i < NL * X.plane / 8; i += kSmallThreads) reinterpret_cast<uint4 *>(X.at)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    sq = 0.0;
#pragma unroll
    for (int w = 0; w < kSmallWaves; w++) sq += sums[w];
    const double inv = 1.0 / (sqrt(sq) + (double)s.eps);
#pragma unroll 4
    for (int i = tid; i < size; i += kSmallThreads) {
        const int row = i / s.cols, col = i - row * s.cols;
        uint16_t limb[NL];
        split_limbs<NL>((float)(update_at(u, base + i) * inv), limb);
        const int at = s.tall ? col * X.pitch + row : row * X.pitch + col;
#pragma unroll
        for (int l = 0; l < NL; l++) X.at[l * X.plane + at] = limb[l];
    }
    __syncthreads();

    // this wave's pairs of results of A and of X
    constexpr int kPairsA = 2;                  // r up to 128
    int ap[kPairsA], aq[kPairsA], xp[kSmallPairs], xq[kSmallPairs], mine_a = 0, mine_x = 0;
    const int across_a = s.r / 32, across_x = s.f / 32;
#pragma unroll
    for (int j = 0; j < kPairsA; j++) {
        const int t = wave + j * kSmallWaves;
        aq[j] = t / across_a * 16;
        ap[j] = t % across_a * 32;
        mine_a += aq[j] < s.r;
    }
#pragma unroll
    for (int j = 0; j < kSmallPairs; j++) {
        const int t = wave + j * kSmallWaves;
        xq[j] = t / across_x * 16;
        xp[j] = t % across_x * 32;
        mine_x += xq[j] < s.r;
    }
    int lp = (lane >> 4) * 4, lq = lane & 15;
    // the last sums take X's place, unsplit
    float *const result = reinterpret_cast<float *>(lds);
    const int pitch = s.f + 4;
    for (int it = 0; it < s.steps; it++) {
        // addresses are made anew: kept over the iterations they would take the registers of the sums
        asm volatile("" : "+v"(lp), "+v"(lq));
        {
            gemm::f4 acc[kPairsA][2];
            small_product<NL, kPairsA, false>(X, X, s.f, mine_a, ap, aq, lane, acc);
#pragma unroll
            for (int j = 0; j < kPairsA; j++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (j < mine_a) small_write<NL>(A, ap[j] + i * 16 + lp, aq[j] + lq, acc[j][i]);
            __syncthreads();
            small_product<NL, kPairsA, false>(A, A, s.r, mine_a, ap, aq, lane, acc);
#pragma unroll
            for (int j = 0; j < kPairsA; j++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (j < mine_a) {
                        float v[4];
                        small_read<NL>(A, ap[j] + i * 16 + lp, aq[j] + lq, v);
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[j][i][e] = fmaf(s.b, v[e], s.c * acc[j][i][e]);
                    }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kPairsA; j++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (j < mine_a) small_write<NL>(A, ap[j] + i * 16 + lp, aq[j] + lq, acc[j][i]);
            __syncthreads();
        }
        gemm::f4 acc[kSmallPairs][2];
        small_product<NL, kSmallPairs, true>(X, A, s.r, mine_x, xp, xq, lane, acc);
#pragma unroll
        for (int j = 0; j < kSmallPairs; j++)
#pragma unroll
            for (int i = 0; i < 2; i++)
                if (j < mine_x) {
                    float v[4];
                    small_read<NL>(X, xp[j] + i * 16 + lp, xq[j] + lq, v);
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[j][i][e] = fmaf(s.a, v[e], acc[j][i][e]);
                    __builtin_amdgcn_sched_barrier(0);
                }
        __syncthreads();
        if (it < s.steps - 1) {
#pragma unroll
            for (int j = 0; j < kSmallPairs; j++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (j < mine_x) small_write<NL>(X, xp[j] + i * 16 + lp, xq[j] + lq, acc[j][i]);
                }
        } else {
#pragma unroll
            for (int j = 0; j < kSmallPairs; j++)
#pragma unroll
                for (int i = 0; i < 2; i++)
                    if (j < mine_x) *reinterpret_cast<gemm::f4 *>(result + (xq[j] + lq) * pitch + xp[j] + i * 16 + lp) = acc[j][i];
        }
        __syncthreads();
    }
#pragma unroll 4
    for (int i = tid; i < size; i += kSmallThreads) {
        const int row = i / s.cols, col = i - row * s.cols;
        float x = result[s.tall ? col * pitch + row : row * pitch + col];
        if (s.weight) x = load_as_float(s.weight, s.out_type, base + i) * s.decay - s.rate * x;
        store_from_float(s.out, s.out_type, base + i, x);
    }
}

struct MuonPlan {
    int r, f;                                   // padded
    int nl;
    bool small;                                 // one workgroup a matrix
    int64_t x_size, a_size;                     // elements of one limb plane
    int norm_blocks;
    size_t part_at, x_at[2], a_at, b_at, split_at, bytes;
};

// Whether a matrix fits the LDS of one workgroup and that is the faster way: a
// wave's steps of 32 k in the three products, as measured, against the products'
// estimates and what their launches cost.  In us, small against products: fp32
// 64 x 64 35 / 67, 64 x 256 65 / 73, 300 of 64 x 64 72 / 149; 16-bit 96 x 96 51 / 65,
// 128 x 128 85 / 64, 300 of them 181 / 297.
bool small_way(const MuonPlan &p, const gs_muon &m)
{
    const int64_t lds = 2 * p.nl * ((int64_t)p.r * (p.f + 8) + (int64_t)p.r * (p.r + 8));
    if (p.r > 128 || p.r * (int64_t)p.f > kSmallWaves * kSmallPairs * 512 || lds > kSmallLds) return false;
    const int pairs_a = (p.r / 16 * (p.r / 32) + kSmallWaves - 1) / kSmallWaves, pairs_x = (p.r / 16 * (p.f / 32) + kSmallWaves - 1) / kSmallWaves;
    const int turns = pairs_a * (p.f / 32 + p.r / 32) + pairs_x * (p.r / 32);
    const double one = 12.0 + m.steps * (0.6 + turns * (p.nl == 3 ? 0.65 : 0.58));
    const double products = choose(p.r, p.r, p.f, m.batch, true, p.nl).us + choose(p.r, p.r, p.r, m.batch, true, p.nl).us +
                            choose(p.f, p.r, p.r, m.batch, false, p.nl).us;
    const double many = 8.0 + m.steps * products, launches = 3.9 * (2 + 3 * m.steps);
    return one * ((m.batch + 255) / 256) < (many > launches ? many : launches);
}

MuonPlan plan_muon(const gs_muon &m)
{
    MuonPlan p;
    const int lo = m.rows < m.cols ? m.rows : m.cols, hi = m.rows < m.cols ? m.cols : m.rows;
    p.r = (lo + 31) & ~31;
    p.f = (hi + 31) & ~31;
    p.nl = m.out_dtype == GS_DTYPE_F32 ? 3 : 2;
    p.x_size = (int64_t)p.r * p.f;
    p.a_size = (int64_t)p.r * p.r;
    p.small = small_way(p, m);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    // a workgroup per 4096 elements of a matrix
    const int64_t blocks = ((int64_t)m.rows * m.cols + 4095) / 4096;
    p.norm_blocks = (int)(blocks < kMaxNormBlocks ? blocks : kMaxNormBlocks);
    p.part_at = take((size_t)m.batch * p.norm_blocks * sizeof(double));
    const size_t xb = (size_t)m.batch * p.nl * p.x_size * 2, ab = (size_t)m.batch * p.nl * p.a_size * 2;
    p.x_at[0] = take(xb);
    p.x_at[1] = take(xb);
    p.a_at = take(ab);
    p.b_at = take(ab);
    // sums of split products, one product at a time
    const NsProduct g[3] = {choose(p.r, p.r, p.f, m.batch, true, p.nl), choose(p.r, p.r, p.r, m.batch, true, p.nl),
                            choose(p.f, p.r, p.r, m.batch, false, p.nl)};
    size_t most = 0;
    for (int i = 0; i < 3; i++) {
        const size_t b = g[i].splits > 1 ? (size_t)m.batch * g[i].splits * (i == 2 ? p.x_size : p.a_size) * 4 : 0;
        most = b > most ? b : most;
    }
    p.split_at = take(most);
    p.bytes = at;
    return p;
}

// Estimated time in microseconds: rounds of blocks over the 256 CUs, each with
// its start and end and so many 64 k; a split costs a launch and its sums' way to
// memory and back.  A product of the iteration, on average over its three, in
// us by tiles of 128 / 64 / 32: 256 x 256 in three limbs 16.7 / 7.5 / 5.9, 8 of them
// 16.8 / 7.7 / 7.2, 1024 x 1024 41.3 / 16.9 / 23.9, 4 of them 46.6 / 52.0 / 68.4; in two
// limbs 256 x 256 12.0 / 6.0 / 5.0, 4 of 1024 x 1024 29.2 / 34.6 / 42.4.
NsProduct choose(int P, int Q, int K, int batch, bool symmetric, int nl)
{
    static const struct { int tile, step_k; float start, us3, us2; } kTiles[3] = {{128, 32, 3.0f, 2.3f, 1.3f}, {64, 64, 1.2f, 0.77f, 0.46f}, {32, 64, 0.5f, 0.62f, 0.38f}};
    NsProduct best{64, 1, 0.0};
    double least = 1e30;
    for (const auto &t : kTiles) {
        const int tp = (P + t.tile - 1) / t.tile, tq = (Q + t.tile - 1) / t.tile, nt = (K + t.step_k - 1) / t.step_k;
        for (int want = 1; want <= 8 && want <= nt; want++) {
            const int per = (nt + want - 1) / want, splits = (nt + per - 1) / per;
            const double tiles = (double)(symmetric && one_side(t.tile, splits) ? tp * (tp + 1) / 2 : tp * tq) * batch;
            double rounds = tiles * splits / 256.0;
            // one block a CU, or (32) several that share its time
            rounds = t.tile > 32 ? ceil(rounds) : rounds > 1.0 ? rounds : 1.0;
            double us = 3.2 + rounds * (t.start + per * t.step_k / 64.0 * (nl == 3 ? t.us3 : t.us2));
            if (splits > 1) us += 5.0 + tiles * splits * t.tile * t.tile * 8.0 / 6e6;
            if (us < least * 0.97) {
                least = us;
                best.tile = t.tile;
                best.splits = splits;
            }
        }
    }
    best.us = least;
    return best;
}

template <int NL, bool PT>
hipError_t launch_product(gemm::Args a, typename NsEpilogue<NL>::Args e, float *partial, int batch, bool symmetric, hipStream_t s)
{
    using E = NsEpilogue<NL>;
    const NsProduct c = choose(a.P, a.Q, a.K, batch, symmetric, NL);
    a.symmetric = symmetric && one_side(c.tile, c.splits);
    e.splits = c.splits;
    e.partial = c.splits > 1 ? partial : nullptr;
    e.ld_partial = a.P;
    e.split_stride = (int64_t)a.P * a.Q;
    hipError_t err = c.tile == 128  ? gemm::launch<gemm::kBF16, NL, 3, 32, 128, 128, 2, 4, PT, false, false, false, E>(a, e, c.splits, batch, s)
                     : c.tile == 64 ? gemm::launch<gemm::kBF16, NL, 3, 64, 64, 64, 2, 4, PT, false, false, false, E>(a, e, c.splits, batch, s)
                                    : gemm::launch<gemm::kBF16, NL, 3, 64, 32, 32, 2, 2, PT, false, false, false, E>(a, e, c.splits, batch, s);
    if (err != hipSuccess || c.splits == 1) return err;
    const int tp = (a.P + 63) / 64, tq = (a.Q + 63) / 64;
    reduce_splits<NL><<<dim3((unsigned)(symmetric ? tp * (tp + 1) : 2 * tp * tq), (unsigned)batch), kThreads, 0, s>>>(e, a.P, a.Q, symmetric);
    return hipGetLastError();
}

template <int NL> hipError_t run_muon(const gs_muon &m, bool step, char *ws, hipStream_t s)
{
    const MuonPlan p = plan_muon(m);
    const bool tall = m.rows > m.cols;
    double *part = reinterpret_cast<double *>(ws + p.part_at);
    uint16_t *x[2] = {reinterpret_cast<uint16_t *>(ws + p.x_at[0]), reinterpret_cast<uint16_t *>(ws + p.x_at[1])};
    float *split = reinterpret_cast<float *>(ws + p.split_at);
    uint16_t *A = reinterpret_cast<uint16_t *>(ws + p.a_at), *B = reinterpret_cast<uint16_t *>(ws + p.b_at);
    Update u;
    u.grad = m.grad;
    u.momentum = step ? m.momentum : nullptr;
    u.momentum_out = m.momentum_out;
    u.grad_type = m.grad_dtype;
    u.nesterov = m.nesterov;
    u.beta = m.beta;
    u.size = (int64_t)m.rows * m.cols;
    u.vec = u.size % 4 == 0;
    if (p.small) {
        Small q;
        q.u = u;
        q.rows = m.rows;
        q.cols = m.cols;
        q.tall = tall;
        q.r = p.r;
        q.f = p.f;
        q.steps = m.steps;
        q.a = m.a;
        q.b = m.b;
        q.c = m.c;
        q.eps = m.eps;
        q.decay = 1.0f - m.lr * m.weight_decay;
        q.rate = m.lr * m.scale;
        q.out = step ? m.weight_out : m.out;
        q.weight = step ? m.weight : nullptr;
        q.out_type = m.out_dtype;
        small_matrices<NL><<<(unsigned)m.batch, kSmallThreads, 0, s>>>(q);
        return hipGetLastError();
    }
    momentum_and_norm<<<dim3((unsigned)p.norm_blocks, (unsigned)m.batch), kThreads, 0, s>>>(u, part);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    normalised_limbs<NL><<<dim3((unsigned)(p.f / 32), (unsigned)(p.r / 32), (unsigned)m.batch), kThreads, 0, s>>>(
        u, part, p.norm_blocks, m.eps, m.rows, m.cols, tall, x[0], p.f, p.x_size, NL * p.x_size);
    if ((err = hipGetLastError()) != hipSuccess) return err;

    // products of limb arrays: [r][f] for X, [r][r] for A and B
    auto args = [&](const uint16_t *P, int64_t ldp, int64_t plane_p, const uint16_t *Q, int64_t ldq, int64_t plane_q, int np, int K) {
        gemm::Args a;
        memset(&a, 0, sizeof a);
        a.p = P;
        a.q = Q;
        a.ldp = ldp;
        a.ldq = ldq;
        a.plane_p = plane_p;
        a.plane_q = plane_q;
        a.batch_p = NL * plane_p;
        a.batch_q = NL * plane_q;
        a.P = a.Pl = np;
        a.Q = a.Ql = p.r;
        a.K = K;
        return a;
    };
    for (int it = 0; it < m.steps; it++) {
        const uint16_t *X = x[it & 1];
        typename NsEpilogue<NL>::Args e;
        memset(&e, 0, sizeof e);
        e.alpha = 1.0f;
        e.o = A;
        e.ldo = p.r;
        e.plane_o = p.a_size;
        e.batch_o = NL * p.a_size;
        if ((err = launch_product<NL, false>(args(X, p.f, p.x_size, X, p.f, p.x_size, p.r, p.f), e, split, m.batch, true, s)) != hipSuccess) return err;
        e.alpha = m.c;
        e.beta = m.b;
        e.c = A;
        e.ldc = p.r;
        e.plane_c = p.a_size;
        e.batch_c = NL * p.a_size;
        e.o = B;
        if ((err = launch_product<NL, false>(args(A, p.r, p.a_size, A, p.r, p.a_size, p.r, p.r), e, split, m.batch, true, s)) != hipSuccess) return err;
        e.alpha = 1.0f;
        e.beta = m.a;
        e.c = X;
        e.ldc = p.f;
        e.plane_c = p.x_size;
        e.batch_c = NL * p.x_size;
        e.o = x[(it & 1) ^ 1];
        e.ldo = p.f;
        e.plane_o = p.x_size;
        e.batch_o = NL * p.x_size;
        if (it == m.steps - 1) {
            e.out = step ? m.weight_out : m.out;
            e.weight = step ? m.weight : nullptr;
            e.out_type = m.out_dtype;
            e.tall = tall;
            e.rows = m.rows;
            e.cols = m.cols;
            e.decay = 1.0f - m.lr * m.weight_decay;
            e.rate = m.lr * m.scale;
        }
        if ((err = launch_product<NL, true>(args(X, p.f, p.x_size, B, p.r, p.a_size, p.f, p.r), e, split, m.batch, false, s)) != hipSuccess) return err;
    }
    return hipSuccess;
}

gs_status muon_ok(const gs_muon *m)
{
    if (!m) return GS_ERR_INVALID_ARG;
    if (m->batch < 0 || m->batch > 65535 || m->rows < 1 || m->rows > 16384 || m->cols < 1 || m->cols > 16384) return GS_ERR_INVALID_ARG;
    if (!float_type(m->grad_dtype) || !float_type(m->out_dtype)) return GS_ERR_INVALID_ARG;
    if (m->steps < 1 || m->steps > 64) return GS_ERR_INVALID_ARG;
    if (!isfinite(m->a) || !isfinite(m->b) || !isfinite(m->c) || !isfinite(m->eps) || !(m->eps > 0.0f)) return GS_ERR_INVALID_ARG;
    if ((m->batch > 0 && !m->grad) || !aligned_to(m->grad, dtype_bytes(m->grad_dtype))) return GS_ERR_INVALID_ARG;
    return GS_OK;
}

gs_status run(const gs_muon &m, bool step, void *workspace, size_t workspace_bytes, void *stream)
{
    if (m.batch == 0) return GS_OK;
    if (workspace_bytes < plan_muon(m).bytes) return GS_ERR_WORKSPACE;
    if (!workspace || !aligned_to(workspace, 16)) return GS_ERR_INVALID_ARG;
    char *ws = static_cast<char *>(workspace);
    hipStream_t s = (hipStream_t)stream;
    const hipError_t e = m.out_dtype == GS_DTYPE_F32 ? run_muon<3>(m, step, ws, s) : run_muon<2>(m, step, ws, s);
    return e == hipSuccess ? GS_OK : GS_ERR_HIP;
}

}  // namespace
}  // namespace gsi

using namespace gsi;

extern "C" {

size_t gs_muon_workspace_bytes(const gs_muon *m)
{
    if (muon_ok(m) != GS_OK || m->batch == 0) return 0;
    return plan_muon(*m).bytes;
}

gs_status gs_orthogonalize(const gs_muon *m, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = muon_ok(m);
    if (st != GS_OK) return st;
    if ((m->batch > 0 && !m->out) || !aligned_to(m->out, dtype_bytes(m->out_dtype))) return GS_ERR_INVALID_ARG;
    return run(*m, false, workspace, workspace_bytes, stream);
}

gs_status gs_muon_step(const gs_muon *m, void *workspace, size_t workspace_bytes, void *stream)
{
    const gs_status st = muon_ok(m);
    if (st != GS_OK) return st;
    const int os = dtype_bytes(m->out_dtype);
    if (m->batch > 0 && (!m->momentum || !m->momentum_out || !m->weight || !m->weight_out)) return GS_ERR_INVALID_ARG;
    if (!aligned_to(m->momentum, 4) || !aligned_to(m->momentum_out, 4) || !aligned_to(m->weight, os) || !aligned_to(m->weight_out, os))
        return GS_ERR_INVALID_ARG;
    if (!isfinite(m->lr) || !isfinite(m->beta) || !isfinite(m->weight_decay) || !isfinite(m->scale)) return GS_ERR_INVALID_ARG;
    return run(*m, true, workspace, workspace_bytes, stream);
}

}  // extern "C"
