// Internal declarations of the linear layer: the epilogue of its products and
// the launchers of each kind of operand (public interface: gs_linear_fwd and
// gs_linear_bwd in include/gs.h).
#pragma once

#include "gs_gemm.h"

namespace gsi {

// What becomes of a product's sums.  With `partial` they are stored as they
// are, one fp32 array [q][ld_partial] per split, and reduced by a second
// kernel; otherwise
//   z = sum + bias;  y = act(z) + residual (+ y if accumulate).
struct LinearEpilogue {
    struct Args {
        float *partial;
        int64_t ld_partial, split_stride;
        const float *bias;
        int bias_on_q;                  // bias[q] (planes) or bias[p]
        int act, exact;                 // exact: fp32 results
        const void *residual;
        int64_t ldr;
        void *y;                        // residual and y: element q * ld + p
        int64_t ldy;
        int y_type, accumulate;
        void *z;                        // element q * z_q + p * z_p
        int64_t z_q, z_p;
        int z_type;
    };

    // One value, any layout.
    __device__ static __forceinline__ void finish1(const Args &e, int p, int q, float v)
    {
        const int64_t at = (int64_t)q * e.ldy + p;
        if (e.bias) v += e.bias[e.bias_on_q ? q : p];
        if (e.z) store_from_float(e.z, e.z_type, (int64_t)q * e.z_q + (int64_t)p * e.z_p, v);
        if (e.exact) activate_all<1, true>(&v, e.act);
        else activate_all<1, false>(&v, e.act);
        if (e.residual) v += load_as_float(e.residual, e.y_type, (int64_t)q * e.ldr + p);
        if (e.accumulate) v += load_as_float(e.y, e.y_type, at);
        store_from_float(e.y, e.y_type, at, v);
    }

    struct Part { float bias[8]; };                 // of eight p
    struct Ahead { Vec<uint16_t, 8> residual; };    // of eight values of a 16-bit type, unconverted

    __device__ static __forceinline__ void part(const Args &e, int p, Part &b)
    {
        if (e.partial || !e.bias || e.bias_on_q) return;
        load8_vec(e.bias + p, b.bias);
    }
    __device__ static __forceinline__ void look_ahead(const Args &e, int p, int q, int, Ahead &a)
    {
        if (!e.partial && e.residual && e.y_type != GS_DTYPE_F32)
            a.residual = *reinterpret_cast<const Vec<uint16_t, 8> *>(static_cast<const uint16_t *>(e.residual) + (int64_t)q * e.ldr + p);
    }

    // Eight values p .. p + 7.
    __device__ static __forceinline__ void finish8(const Args &e, int p, int q, float v[8], const Part &b, const Ahead &a)
    {
        const int64_t at = (int64_t)q * e.ldy + p;
        if (e.bias) {
            if (e.bias_on_q) {
                const float b = e.bias[q];
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += b;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += b.bias[i];
            }
        }
        if (e.z) {
            if (e.z_p == 1) {
                store8_stream(e.z, e.z_type, (int64_t)q * e.z_q + p, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; i++) store_from_float(e.z, e.z_type, (int64_t)q * e.z_q + (int64_t)(p + i) * e.z_p, v[i]);
            }
        }
        if (e.exact) activate_all<8, true>(v, e.act);
        else activate_all<8, false>(v, e.act);
        float r[8];
        if (e.residual) {
            if (e.y_type == GS_DTYPE_F32) {
                load8_vec(static_cast<const float *>(e.residual) + (int64_t)q * e.ldr + p, r);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += r[i];
            } else if (e.y_type == GS_DTYPE_F16) {
                const gemm::h8 h = __builtin_bit_cast(gemm::h8, a.residual);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += (float)h[i];
            } else {
                const gemm::bf8 h = __builtin_bit_cast(gemm::bf8, a.residual);
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] += (float)h[i];
            }
        }
        if (e.accumulate) {
            load8_vec(e.y, e.y_type, at, r);
#pragma unroll
            for (int i = 0; i < 8; i++) v[i] += r[i];
        }
        store8_vec(e.y, e.y_type, at, v);
    }

    static constexpr bool kMirror = false;

    __device__ static __forceinline__ void store8(const Args &e, int p, int q, float v[8], const Part &b, const Ahead &a, int, int split)
    {
        if (e.partial)                                          // rows of partial sums are padded to 8
            store8_vec(e.partial + split * e.split_stride + (int64_t)q * e.ld_partial + p, v);
        else
            finish8(e, p, q, v, b, a);
    }
    __device__ static __forceinline__ void store1(const Args &e, int p, int q, float v, int, int split)
    {
        if (e.partial)
            e.partial[split * e.split_stride + (int64_t)q * e.ld_partial + p] = v;
        else
            finish1(e, p, q, v);
    }
};

// One product of the linear layer: which operands are stored by columns,
// which tile and how many splits of k.
struct ProductPlan {
    bool pt, qt;
    bool staged;
    int tile;                           // 0: 256 x 256, 1: 128 x 128, 2: 64 x 64 (staged and fp32: 1, 2)
    int splits;                         // of k, each with at least one tile of k
    double us;                          // estimated time
};

// out[c] (+)= sum over rows r of part[r][c], in a fixed order (gs_norm.hip).
hipError_t launch_sum_rows(const float *part, float *out, int n, int rows, int accumulate, hipStream_t s);

hipError_t launch_product_bf16(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s);
hipError_t launch_product_f16(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s);
hipError_t launch_product_f32(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s);
// At most 16 rows of x (8-bit operands: for a 16-bit y).
constexpr int kFewRows = 16;
hipError_t launch_few_rows(const gs_linear &l, const LinearEpilogue::Args &e, hipStream_t s);
hipError_t launch_product_mx8(const gemm::Args &a, const LinearEpilogue::Args &e, const ProductPlan &plan, hipStream_t s);

}  // namespace gsi
