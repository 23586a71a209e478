// Orthogonalised update (Newton-Schulz iterations) of a batch of weight
// matrices, alone and as the momentum step of the weights.
//
// With r = min(rows, cols) and f = max, X is [r][f] (U^T when U is tall) and
// an iteration is three products: A = X X^T, B = b A + c A A^T (A is
// symmetric) and X' = a X + B X, 2 r^2 (2 f + r) multiply-adds.  X, A and B
// live in the workspace as bf16 limbs, padded with zeros to multiples of 32,
// and every epilogue writes its result as limbs, so no product converts
// anything: B X reads X by columns, and a tall U is turned round once at each
// end.  fp32 results take three limbs, 16-bit results two: an iteration
// amplifies an error in a weak direction up to |a| times, 2^-16 grows to about
// 2^-11 in five, where one bf16 limb would lose the direction.
#include <string.h>

#include "gs_gemm.h"

namespace gsi {
namespace {

constexpr int kThreads = 256;
constexpr int kNormBlocks = 64;                 // partial sums of squares per matrix

bool aligned_to(const void *p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }
bool float_type(int t) { return t == GS_DTYPE_F32 || t == GS_DTYPE_F16 || t == GS_DTYPE_BF16; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Update {
    const void *grad;
    const float *momentum;                      // NULL: U = grad
    float *momentum_out;
    int grad_type, nesterov;
    float beta;
    int64_t size;                               // rows * cols
};

// Element i of U once momentum_out is written.
__device__ __forceinline__ float update_at(const Update &u, int64_t i)
{
    if (!u.momentum) return load_as_float(u.grad, u.grad_type, i);
    const float m = u.momentum_out[i];
    return u.nesterov ? fmaf(u.beta, m, load_as_float(u.grad, u.grad_type, i)) : m;
}

// Momentum and the sums of squares of U, kNormBlocks workgroups per matrix.
// The norm scales every singular value alike and the iterations' polynomial is
// steep between its plateaus, so it is kept in fp64: an fp32 norm's error was
// the largest part of the fp32 result's.
__global__ __launch_bounds__(kThreads) void momentum_and_norm(Update u, double *part)
{
    __shared__ double lds[kThreads / 64];
    const int64_t base = (int64_t)blockIdx.y * u.size;
    double sq = 0.0;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < u.size; i += (int64_t)kNormBlocks * kThreads) {
        if (u.momentum)
            u.momentum_out[base + i] = fmaf(u.beta, u.momentum[base + i], load_as_float(u.grad, u.grad_type, base + i));
        const double x = update_at(u, base + i);
        sq = fma(x, x, sq);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sq += __shfl_xor(sq, o);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = sq;
    __syncthreads();
    if (threadIdx.x == 0) part[blockIdx.y * kNormBlocks + blockIdx.x] = lds[0] + lds[1] + lds[2] + lds[3];
}

// X = U / (|U| + eps) as limbs [r_pad][f_pad], zeros in the padding; tiles of
// 32 x 32 turned round in LDS when U is tall.
template <int NL>
__global__ __launch_bounds__(kThreads) void normalised_limbs(Update u, const double *part, float eps, int rows, int cols, int tall,
                                                             uint16_t *x, int64_t ldx, int64_t plane, int64_t batch)
{
    __shared__ float tile[32][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    double sq = 0.0;
    for (int i = 0; i < kNormBlocks; i++) sq += part[blockIdx.z * kNormBlocks + i];
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

    __device__ static __forceinline__ void store(const Args &e, int p, int q, int, const float *s, int batch, int)
    {
        float v[8];
        load8_vec(s, v);
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] *= e.alpha;
        if (e.c) {
            const uint16_t *c = e.c + batch * e.batch_c + (int64_t)q * e.ldc + p;
            float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int l = NL - 1; l >= 0; l--) {
                const Vec<uint16_t, 8> h = *reinterpret_cast<const Vec<uint16_t, 8> *>(c + l * e.plane_c);
#pragma unroll
                for (int i = 0; i < 8; i++) w[i] += limb_value(h.v[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] = fmaf(e.beta, w[i], v[i]);
        }
        if (!e.out) {
            Vec<uint16_t, 8> h[NL];
#pragma unroll
            for (int i = 0; i < 8; i++) {
                uint16_t limb[NL];
                split_limbs<NL>(v[i], limb);
#pragma unroll
                for (int l = 0; l < NL; l++) h[l].v[i] = limb[l];
            }
            uint16_t *o = e.o + batch * e.batch_o + (int64_t)q * e.ldo + p;
#pragma unroll
            for (int l = 0; l < NL; l++) *reinterpret_cast<Vec<uint16_t, 8> *>(o + l * e.plane_o) = h[l];
            return;
        }
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
};

struct MuonPlan {
    int r, f;                                   // padded
    int nl;
    int64_t x_size, a_size;                     // elements of one limb plane
    size_t part_at, x_at[2], a_at, b_at, bytes;
};

MuonPlan plan_muon(const gs_muon &m)
{
    MuonPlan p;
    const int lo = m.rows < m.cols ? m.rows : m.cols, hi = m.rows < m.cols ? m.cols : m.rows;
    p.r = (lo + 31) & ~31;
    p.f = (hi + 31) & ~31;
    p.nl = m.out_dtype == GS_DTYPE_F32 ? 3 : 2;
    p.x_size = (int64_t)p.r * p.f;
    p.a_size = (int64_t)p.r * p.r;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round256(bytes);
        return here;
    };
    p.part_at = take((size_t)m.batch * kNormBlocks * sizeof(double));
    const size_t xb = (size_t)m.batch * p.nl * p.x_size * 2, ab = (size_t)m.batch * p.nl * p.a_size * 2;
    p.x_at[0] = take(xb);
    p.x_at[1] = take(xb);
    p.a_at = take(ab);
    p.b_at = take(ab);
    p.bytes = at;
    return p;
}

template <int NL, bool PT>
hipError_t launch_product(const gemm::Args &a, const typename NsEpilogue<NL>::Args &e, int batch, hipStream_t s)
{
    using E = NsEpilogue<NL>;
    const int64_t blocks = (int64_t)((a.P + 127) / 128) * ((a.Q + 127) / 128) * batch;
    if (blocks >= 192) return gemm::launch<gemm::kBF16, NL, 32, 128, 128, 2, 2, PT, false, false, E>(a, e, 1, batch, s);
    return gemm::launch<gemm::kBF16, NL, 32, 64, 64, 2, 2, PT, false, false, E>(a, e, 1, batch, s);
}

template <int NL> hipError_t run_muon(const gs_muon &m, bool step, char *ws, hipStream_t s)
{
    const MuonPlan p = plan_muon(m);
    const bool tall = m.rows > m.cols;
    double *part = reinterpret_cast<double *>(ws + p.part_at);
    uint16_t *x[2] = {reinterpret_cast<uint16_t *>(ws + p.x_at[0]), reinterpret_cast<uint16_t *>(ws + p.x_at[1])};
    uint16_t *A = reinterpret_cast<uint16_t *>(ws + p.a_at), *B = reinterpret_cast<uint16_t *>(ws + p.b_at);
    Update u;
    u.grad = m.grad;
    u.momentum = step ? m.momentum : nullptr;
    u.momentum_out = m.momentum_out;
    u.grad_type = m.grad_dtype;
    u.nesterov = m.nesterov;
    u.beta = m.beta;
    u.size = (int64_t)m.rows * m.cols;
    momentum_and_norm<<<dim3(kNormBlocks, (unsigned)m.batch), kThreads, 0, s>>>(u, part);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    normalised_limbs<NL><<<dim3((unsigned)(p.f / 32), (unsigned)(p.r / 32), (unsigned)m.batch), kThreads, 0, s>>>(
        u, part, m.eps, m.rows, m.cols, tall, x[0], p.f, p.x_size, NL * p.x_size);
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
        if ((err = launch_product<NL, false>(args(X, p.f, p.x_size, X, p.f, p.x_size, p.r, p.f), e, m.batch, s)) != hipSuccess) return err;
        e.alpha = m.c;
        e.beta = m.b;
        e.c = A;
        e.ldc = p.r;
        e.plane_c = p.a_size;
        e.batch_c = NL * p.a_size;
        e.o = B;
        if ((err = launch_product<NL, false>(args(A, p.r, p.a_size, A, p.r, p.a_size, p.r, p.r), e, m.batch, s)) != hipSuccess) return err;
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
        if ((err = launch_product<NL, true>(args(X, p.f, p.x_size, B, p.r, p.a_size, p.f, p.r), e, m.batch, s)) != hipSuccess) return err;
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
