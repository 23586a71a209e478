// Number formats and elementwise functions shared by the norm, the matrix
// products and the orthogonalised update (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gs.h"

namespace gsi {

__host__ __device__ constexpr int dtype_bytes(int t) { return t == GS_DTYPE_F32 ? 4 : t == GS_DTYPE_MXFP8 ? 1 : 2; }

// HIP takes fewer than 2^32 threads along a dimension of a launch: more blocks
// than that are spread over y too, and those past the last find nothing to do.
inline dim3 grid_of(int64_t blocks, int threads)
{
    const int64_t most = 0xFFFFFFFFll / threads, y = (blocks + most - 1) / most;
    return dim3((unsigned)((blocks + y - 1) / y), (unsigned)y);
}
__device__ __forceinline__ int64_t block_of() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Consecutive values as one vector access of up to 16 bytes.  Only the elements'
// own alignment is asked for: the hardware takes the wide accesses at any
// address of global memory, so odd strides and offsets need no other path.
template <typename T, int N> struct __attribute__((packed, aligned(sizeof(T)))) Vec { T v[N]; };

// Element i of an array of type t (not GS_DTYPE_MXFP8).
__device__ __forceinline__ float load_as_float(const void *p, int t, int64_t i)
{
    if (t == GS_DTYPE_F32) return static_cast<const float *>(p)[i];
    if (t == GS_DTYPE_F16) return (float)static_cast<const _Float16 *>(p)[i];
    return (float)static_cast<const __bf16 *>(p)[i];
}
__device__ __forceinline__ void store_from_float(void *p, int t, int64_t i, float x)
{
    if (t == GS_DTYPE_F32) static_cast<float *>(p)[i] = x;
    else if (t == GS_DTYPE_F16) static_cast<_Float16 *>(p)[i] = (_Float16)x;
    else static_cast<__bf16 *>(p)[i] = (__bf16)x;
}

template <typename T> __device__ __forceinline__ void load8_vec(const T *p, float v[8])
{
    const Vec<T, 8> w = *reinterpret_cast<const Vec<T, 8> *>(p);
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = (float)w.v[i];
}
template <typename T> __device__ __forceinline__ void store8_vec(T *p, const float v[8])
{
    Vec<T, 8> w;
#pragma unroll
    for (int i = 0; i < 8; i++) w.v[i] = (T)v[i];
    *reinterpret_cast<Vec<T, 8> *>(p) = w;
}
// Elements i .. i + 7 of an array of type t.
__device__ __forceinline__ void load8_vec(const void *p, int t, int64_t i, float v[8])
{
    if (t == GS_DTYPE_F32) load8_vec(static_cast<const float *>(p) + i, v);
    else if (t == GS_DTYPE_F16) load8_vec(static_cast<const _Float16 *>(p) + i, v);
    else load8_vec(static_cast<const __bf16 *>(p) + i, v);
}
// The same for results that are not read again soon: written past the caches.
__device__ __forceinline__ void store8_stream(void *p, int t, int64_t i, const float v[8])
{
    typedef int any4 __attribute__((ext_vector_type(4), aligned(2)));     // at any element's address
    if (t == GS_DTYPE_F32) {
        float *q = static_cast<float *>(p) + i;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const Vec<float, 4> w = {{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]}};
            __builtin_nontemporal_store(__builtin_bit_cast(any4, w), reinterpret_cast<any4 *>(q + 4 * h));
        }
        return;
    }
    union { Vec<_Float16, 8> h; Vec<__bf16, 8> b; } w;
#pragma unroll
    for (int k = 0; k < 8; k++) {
        if (t == GS_DTYPE_F16) w.h.v[k] = (_Float16)v[k];
        else w.b.v[k] = (__bf16)v[k];
    }
    __builtin_nontemporal_store(__builtin_bit_cast(any4, w), reinterpret_cast<any4 *>(static_cast<uint16_t *>(p) + i));
}
__device__ __forceinline__ void store8_vec(void *p, int t, int64_t i, const float v[8])
{
    if (t == GS_DTYPE_F32) store8_vec(static_cast<float *>(p) + i, v);
    else if (t == GS_DTYPE_F16) store8_vec(static_cast<_Float16 *>(p) + i, v);
    else store8_vec(static_cast<__bf16 *>(p) + i, v);
}
// Elements past the first `valid` do not exist and read as 0.
__device__ __forceinline__ void load8(const void *p, int t, int64_t i, int valid, float v[8])
{
    if (valid >= 8) {
        load8_vec(p, t, i, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = j < valid ? load_as_float(p, t, i + j) : 0.0f;
}

// x = limb 0 + limb 1 + limb 2, each what is left rounded to bf16 (8 bits): a
// rounded limb leaves a remainder of either sign, so three hold all 24 bits
// and what a product of limbs drops does not pile up on one side.  A finite x
// that would round to an infinity is truncated instead; an infinity or NaN
// stays alone in the first limb.  Limbs below the smallest bf16 vanish, so
// values under 2^-110 keep fewer bits.
template <int NL> __device__ __forceinline__ void split_limbs(float x, uint16_t limb[NL])
{
    limb[0] = __builtin_bit_cast(uint16_t, (__bf16)x);
    float head = __uint_as_float((uint32_t)limb[0] << 16);
    if (!(fabsf(head) < INFINITY) && fabsf(x) < INFINITY) {
        head = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
        limb[0] = (uint16_t)(__float_as_uint(head) >> 16);
    }
    float rest = fabsf(x) < INFINITY ? x - head : 0.0f;
#pragma unroll
    for (int l = 1; l < NL; l++) {
        limb[l] = __builtin_bit_cast(uint16_t, (__bf16)rest);
        rest -= __uint_as_float((uint32_t)limb[l] << 16);
    }
}
// The same for N values at once, the hardware's conversions taking two each:
// half the instructions, which bound the loads that convert.  Infinities and
// values that would round to one go the way above.
template <int NL, int N> __device__ __forceinline__ void split_all(const float v[N], Vec<uint16_t, N> w[NL])
{
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i++) top = fmaxf(top, fabsf(v[i]));
    if (__builtin_expect(!(top < 0x1.FFp127f), 0)) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            uint16_t limb[NL];
            split_limbs<NL>(v[i], limb);
#pragma unroll
            for (int l = 0; l < NL; l++) w[l].v[i] = limb[l];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        f2 rest = {v[i], v[i + 1]};
#pragma unroll
        for (int l = 0; l < NL; l++) {
            const uint32_t two = __builtin_bit_cast(uint32_t, __builtin_convertvector(rest, b2));
            w[l].v[i] = (uint16_t)two;
            w[l].v[i + 1] = (uint16_t)(two >> 16);
            if (l == NL - 1) break;
            rest[0] -= __uint_as_float(two << 16);
            rest[1] -= __uint_as_float(two & 0xFFFF0000u);
        }
    }
}
__device__ __forceinline__ float limb_value(uint16_t l) { return __uint_as_float((uint32_t)l << 16); }

// e4m3 (1 sign, 4 exponent, 3 mantissa bits, bias 7, no infinities, 0x7F NaN).
__device__ __forceinline__ float e4m3_value(uint8_t b)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)b, 0);
}
// 2^(s - 127); 255 is NaN, 0 is 2^-127.
__device__ __forceinline__ float e8m0_value(uint32_t s)
{
    return s == 255u ? NAN : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// ---- activations -------------------------------------------------------------
// Phi(-|z|) of the standard normal distribution and e = exp(-z^2 / 2): both as t
// times a polynomial in t = 1 / (1 + p |z| / sqrt 2) times e.
// For results rounded to 16 bits the five terms of Abramowitz and Stegun 7.1.26:
// absolute error 7.5e-8, relative 5e-5 at |z| = 3, 5e-4 at 4, 1.6e-3 at 5 and 3.6e-3 at 6,
// where half an ulp is 5e-4 of fp16 (but values under 6e-5 are subnormal there)
// and 2e-3 of bf16.  For fp32 results (EXACT) nine, fitted for this to
// the scaled complementary error function: relative error 4e-8 before rounding,
// 7e-7 up to |z| = 4 in fp32, where a sum 1 + erf has lost all of the tail.  The
// library's erfc, with its branches, took most of an epilogue's time.
template <bool EXACT> __device__ __forceinline__ float normal_tail(float z, float &e)
{
    e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
    if constexpr (EXACT) {
        const float d = fmaf(fminf(fabsf(z), 16.0f), 0.5f * 0.70710678118654752f, 1.0f);
        float t = __builtin_amdgcn_rcpf(d);
        t = fmaf(fmaf(-d, t, 1.0f), t, t);
        constexpr float k[9] = {0.141044193f, 0.141170635f, 0.121674233f, 0.100864183f, -0.0121898435f, 0.137415421f, -0.242194546f, 0.141612519f, -0.0293968155f};
        float p = k[8];
#pragma unroll
        for (int i = 7; i >= 0; i--) p = fmaf(t, p, k[i]);
        return t * p * e;
    }
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752f, 1.0f));
    const float p = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, -0.5f * 1.453152027f), 0.5f * 1.421413741f),
                                     -0.5f * 0.284496736f), 0.5f * 0.254829592f);
    return p * e;
}
// 1 / (1 + exp(-z)); EXACT carries what the exponent's product rounds off and
// corrects the reciprocal once.
template <bool EXACT> __device__ __forceinline__ float logistic(float z)
{
    if constexpr (EXACT) {
        const float x = -fminf(fmaxf(z, -87.0f), 87.0f), u = x * 1.4426950408889634f;
        const float rest = fmaf(x, 1.4426950408889634f, -u) + x * 1.9259629911266175e-8f;     // log2 e to 48 bits
        float e = __builtin_amdgcn_exp2f(u);
        e = fmaf(e, rest * 0.69314718055994531f, e);
        const float d = 1.0f + e, s = __builtin_amdgcn_rcpf(d);
        return z < -87.0f ? 0.0f : fmaf(fmaf(-d, s, 1.0f), s, s);       // under 2^-125
    }
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.4426950408889634f));
}
template <int ACT, bool EXACT> __device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == GS_ACT_RELU) return z < 0.0f ? 0.0f : z;     // a NaN stays one
    if constexpr (ACT == GS_ACT_SILU) return z * logistic<EXACT>(z);
    if constexpr (ACT == GS_ACT_GELU) {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|); the bound keeps an infinite z from
        // meeting the tail's 0
        float e;
        const float h = normal_tail<EXACT>(z, e);
        return fmaf(-fminf(fabsf(z), 64.0f), h, fmaxf(z, 0.0f));
    }
    return z;
}
template <int ACT, bool EXACT> __device__ __forceinline__ float activate_slope(float z)
{
    if constexpr (ACT == GS_ACT_RELU) return z > 0.0f ? 1.0f : z == z ? 0.0f : z;
    if constexpr (ACT == GS_ACT_SILU) {
        const float s = logistic<EXACT>(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    if constexpr (ACT == GS_ACT_GELU) {
        float e;
        const float h = normal_tail<EXACT>(z, e);
        return fmaf(z * 0.39894228040143268f, e, z >= 0.0f ? 1.0f - h : h);
    }
    return 1.0f;
}

// The choice of activation is made once for N values: a branch in front of
// each would put their exponentials and reciprocals one after the other.
template <int N, bool EXACT> __device__ __forceinline__ void activate_all(float v[N], int act)
{
    if (act == GS_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = activate<GS_ACT_RELU, EXACT>(v[i]);
    } else if (act == GS_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = activate<GS_ACT_SILU, EXACT>(v[i]);
    } else if (act == GS_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = activate<GS_ACT_GELU, EXACT>(v[i]);
    }
}
// v *= act'(z)
template <int N, bool EXACT> __device__ __forceinline__ void scale_by_slope(float v[N], const float z[N], int act)
{
    if (act == GS_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= activate_slope<GS_ACT_RELU, EXACT>(z[i]);
    } else if (act == GS_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= activate_slope<GS_ACT_SILU, EXACT>(z[i]);
    } else if (act == GS_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] *= activate_slope<GS_ACT_GELU, EXACT>(z[i]);
    }
}

}  // namespace gsi
