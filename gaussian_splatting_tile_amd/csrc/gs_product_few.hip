// Linear layer for few rows of x (single tokens up to 16).
//
// The weights are read once and nothing else is large, so the call is bound by
// their bytes and, below a few MB, by latency: a workgroup takes 16 outputs for
// all rows, its waves share k, and every weight goes from memory straight into
// the matrix instruction's registers.  A lane's two 16-byte pieces of a row are
// neighbours, four lanes make 128 bytes of it; which k a lane holds is the same
// for both operands, so the order within the sum is all that changes.  The
// waves' sums are added in their order.  One row, 1024 inputs, 4096 outputs in
// bf16: 4.1 us (8.4 MB of weights, 2.0 TB/s) of a call's 10.2, against 6.5 by 64 x 64
// tiles.  A call takes 10.1 in fp32, 12.1 with 8-bit blocks; 16 rows 11.1 in bf16, 10.7 in
// fp32.
#include "gs_linear.h"

namespace gsi {
namespace {

using namespace gemm;

constexpr int kOutputs = 16;                    // per workgroup

struct FewArgs {
    const void *x, *w;
    int64_t ldx, ldw;
    const uint8_t *xs, *ws;                     // kMX8
    int64_t ldxs, ldws;
    int m, n, k, planes;
};

template <int KIND, int NL> struct Piece {      // what one lane holds of 64 k (kMX8: 128 k) of a row
    i4 v[NL][2];
    int scale;
};

template <int KIND, int NL>
__device__ __forceinline__ void load_piece(Piece<KIND, NL> &f, const void *base, int64_t ld, const uint8_t *scales, int64_t lds, int row,
                                           int k0, int K, int g)
{
    if constexpr (KIND == kMX8) {                       // k is a multiple of 32
        const uint8_t *p = static_cast<const uint8_t *>(base) + row * ld + k0;
        using V = Vec<uint8_t, 16>;
        f.v[0][0] = f.v[0][1] = i4{0, 0, 0, 0};
        if (k0 + g * 16 < K) f.v[0][0] = __builtin_bit_cast(i4, *reinterpret_cast<const V *>(p + g * 16));
        if (k0 + 64 + g * 16 < K) f.v[0][1] = __builtin_bit_cast(i4, *reinterpret_cast<const V *>(p + 64 + g * 16));
        f.scale = k0 + g * 32 < K ? scales[row * lds + (k0 >> 5) + g] : 127;
    } else if constexpr (NL == 1) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + row * ld;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int k = k0 + g * 16 + h * 8;
            Vec<uint16_t, 8> v{};
            if (k + 8 <= K) {
                v = *reinterpret_cast<const Vec<uint16_t, 8> *>(p + k);
            } else if (k < K) {
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (k + e < K) v.v[e] = p[k + e];
            }
            f.v[0][h] = __builtin_bit_cast(i4, v);
        }
    } else {
        const float *p = static_cast<const float *>(base) + row * ld;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int k = k0 + g * 16 + h * 8;
            float v[8];
            load8(p, GS_DTYPE_F32, k, min(8, K - k), v);
            Vec<uint16_t, 8> limb[NL];
            split_all<NL, 8>(v, limb);
#pragma unroll
            for (int i = 0; i < NL; i++) f.v[i][h] = __builtin_bit_cast(i4, limb[i]);
        }
    }
}

template <int KIND, int NL>
__device__ __forceinline__ f4 product(const Piece<KIND, NL> &a, const Piece<KIND, NL> &b, f4 c)
{
    if constexpr (KIND == kMX8) return mfma_mx(a.v[0][0], a.v[0][1], a.scale, b.v[0][0], b.v[0][1], b.scale, c);
#pragma unroll
    for (int order = NL - 1; order >= 0; order--)
#pragma unroll
        for (int l = 0; l <= order; l++)
#pragma unroll
            for (int h = 0; h < 2; h++) c = mfma32<KIND>(a.v[l][h], b.v[order - l][h], c);
    return c;
}

constexpr int at_once(int NL) { return NL == 1 ? 4 : 1; }       // pieces of weights on their way together

template <int KIND, int NL, int WAVES> __global__ __launch_bounds__(WAVES * 64) void few_rows_kernel(FewArgs a, LinearEpilogue::Args e)
{
    constexpr int kStep = KIND == kMX8 ? 128 : 64, kAtOnce = at_once(NL);
    __shared__ float sums[WAVES][kFewRows][kOutputs + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * kOutputs, row = min(n0 + r, a.n - 1);
    f4 acc = {0, 0, 0, 0};
    for (int k0 = wave * kStep; k0 < a.k; k0 += kAtOnce * WAVES * kStep) {
        Piece<KIND, NL> w[kAtOnce], x[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; u++) {
            const int k = k0 + u * WAVES * kStep;
            load_piece(w[u], a.w, a.ldw, a.ws, a.ldws, row, k, a.k, g);
            load_piece(x[u], a.x, a.ldx, a.xs, a.ldxs, min(r, a.m - 1), k, a.k, g);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; u++) acc = product(w[u], x[u], acc);
    }
#pragma unroll
    for (int i = 0; i < 4; i++) sums[wave][r][g * 4 + i] = acc[i];
    __syncthreads();
    const int id = threadIdx.x;
    if (id >= kFewRows * kOutputs) return;
    // neighbouring threads along the contiguous index of y
    const int o = a.planes ? id / kFewRows : id % kOutputs, t = a.planes ? id % kFewRows : id / kOutputs;
    if (t >= a.m || n0 + o >= a.n) return;
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; i++) v += sums[i][t][o];
    if (a.planes) LinearEpilogue::finish1(e, t, n0 + o, v);
    else LinearEpilogue::finish1(e, n0 + o, t, v);
}

template <int KIND, int NL> hipError_t launch_few(const FewArgs &a, const LinearEpilogue::Args &e, hipStream_t s)
{
    const unsigned blocks = (unsigned)((a.n + kOutputs - 1) / kOutputs);
    // 16 waves where 4 would go round more than once
    if (a.k <= (KIND == kMX8 ? 512 : 256) * at_once(NL)) few_rows_kernel<KIND, NL, 4><<<blocks, 4 * 64, 0, s>>>(a, e);
    else few_rows_kernel<KIND, NL, 16><<<blocks, 16 * 64, 0, s>>>(a, e);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_few_rows(const gs_linear &l, const LinearEpilogue::Args &e, hipStream_t s)
{
    FewArgs a;
    a.x = l.x;
    a.w = l.w;
    a.ldx = l.x_stride;
    a.ldw = l.w_stride;
    a.xs = l.x_scales;
    a.ws = l.w_scales;
    a.ldxs = l.x_scales_stride;
    a.ldws = l.w_scales_stride;
    a.m = (int)l.m;
    a.n = l.n;
    a.k = l.k;
    a.planes = l.planes != 0;
    if (l.dtype == GS_DTYPE_F32) return launch_few<kBF16, 3>(a, e, s);
    if (l.dtype == GS_DTYPE_F16) return launch_few<kF16, 1>(a, e, s);
    if (l.dtype == GS_DTYPE_BF16) return launch_few<kBF16, 1>(a, e, s);
    return launch_few<kMX8, 1>(a, e, s);
}

}  // namespace gsi
