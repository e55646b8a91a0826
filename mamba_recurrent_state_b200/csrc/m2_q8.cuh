// m2_q8.cuh -- the 8-bit state cache: what its kernels and entry points share.
//
// A state row (the N values of one (head, p)) is stored as N signed codes and
// one fp32 scale. With a = max |v| over the row:
//   a < 2^-100        scale = 0, codes 0 (127 / a would overflow)
//   a inf or NaN      scale = NaN: the whole row reads back as NaN
//   else              scale = a / 127, code = round_half_even(v * (127 / a))
//                     (the scale one float lower where 127 of it would pass the largest float)
// both quotients rounded to fp32, the product not rounded before the code.
// A value reads back as code * scale, at most scale / 2 from v (1 + 2^-22).
//
// Why integers and a scale a row: the rows of a recurrent state are close to
// normally distributed, and at equal size (8 bits a value) e4m3 codes round
// every value by up to 2^-4 of itself (2.6% rms) where these round by up to
// 1/254 of the row's maximum (0.6% of its rms). The rounding matters twice as
// a decode step stores the state every token: what one step rounds the next
// ones carry on.
#pragma once

#include "m2_device.cuh"
#include "m2_internal.cuh"

namespace m2 {

struct Q8CopyArgs {  // between a 16/32-bit cache and an 8-bit one
    void* ssm;       // [slots, R, N] fp32 or bf16
    void* conv;
    int32_t* error;
    int64_t num_slots;
    int8_t* q;       // [q_slots, R, N]
    float* scale;    // [q_slots, R]
    void* q_conv;
    int32_t* q_error;
    int64_t q_num_slots;
    int rows;        // R = H * P
    int N;
    int state_bf16;
    int64_t conv_bytes;  // per slot, a multiple of 16
    int n;
    const int32_t* src_idx;
    const int32_t* dst_idx;
};
cudaError_t launch_q8_store(const Q8CopyArgs& a, cudaStream_t stream);
cudaError_t launch_q8_load(const Q8CopyArgs& a, cudaStream_t stream);

struct Q8UpdateArgs {
    int8_t* ssm;
    float* scale;
    void* conv;
    int32_t* error;
    int64_t num_slots;
    int H, P, N, G, K;
    int64_t conv_dim;
    int act_bf16;
    const float* A_log;
    const float* dt_bias;
    const float* D;
    const void* conv_w;
    const void* conv_b;
    int activation;
    int batch;
    const void* xBC;
    int64_t xBC_stride;
    const void* dt;
    int64_t dt_stride;
    const void* z;
    int64_t z_stride;
    void* y;
    int64_t y_stride;
    const int32_t* slot_idx;
    const void* norm_w;  // gated RMSNorm weight [H*P] act dtype, or NULL
    float norm_eps;
    int tile_rows;       // state rows per CTA (plan_q8_update)
    int group_ctas;      // CTAs per SSM group: the thread-block cluster
    int group_rows, hpg; // rows and heads of a group
    uint32_t inv_P;      // 2^22 / P, rounded up
};
// Shape check of the decode step (host arithmetic): M2_OK or M2_ERR_UNSUPPORTED.
m2_status q8_shape_supported(int H, int P, int N, int G);
cudaError_t launch_q8_update(Q8UpdateArgs a, cudaStream_t stream);

// max that keeps a NaN of either side.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The largest scale: the float below the largest finite one over 127, whose
// product with 127 would round to an infinity.
constexpr float kQ8TopScale = 0x1.020406p+121f;

// Scale and inverse of a row whose largest magnitude is a.
__device__ __forceinline__ void q8_scale(float a, float& scale, float& inv) {
    const bool finite = a <= 3.402823466e38f;   // false for inf and NaN
    const bool live = finite && a >= 7.888609052e-31f;  // 2^-100
    const float d = live ? a : 1.f;
    inv = live ? __fdiv_rn(127.f, d) : 0.f;
    scale = live ? fminf(__fdiv_rn(d, 127.f), kQ8TopScale) : (finite ? 0.f : __int_as_float(0x7fc00000));
}

// The largest of m and the magnitudes of a and b; a NaN stays.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}

// q8_scale for the decode step: a product with 1/127 and the reciprocal of the
// special-function unit, each within 2^-22 of the quotient. It takes the
// quotients only where the reciprocal would leave the normal range.
__device__ __forceinline__ void q8_scale_fast(float a, float& scale, float& inv) {
    if (a >= 7.888609052e-31f && a <= 1.329227996e36f) {  // 2^-100 .. 2^120
        scale = a * (1.f / 127.f);
        inv = 127.f * rcp_approx(a);
    } else {
        q8_scale(a, scale, inv);
    }
}

// 1.5 * 2^23: fma(v, inv, kQ8Magic) rounds the exact product half to even to
// an integer k, |k| < 2^22, and its low byte is k in two's complement.
constexpr float kQ8Magic = 12582912.f;

// Four codes, the low bytes of four such floats, in one word.
__device__ __forceinline__ uint32_t q8_pack(float c0, float c1, float c2, float c3) {
    const uint32_t lo = __byte_perm(__float_as_uint(c0), __float_as_uint(c1), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(c2), __float_as_uint(c3), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
}

// Four codes of a word as floats. code + 128 is put in the low byte of 2^23
// (so the float is 2^23 + 128 + code), and the constant subtracted: exact.
__device__ __forceinline__ void q8_unpack(uint32_t word, float2& lo, float2& hi) {
    const uint32_t u = word ^ 0x80808080u;
    const float2 c = make_float2(-8388736.f, -8388736.f);
    lo = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)),
                                __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441))), c);
    hi = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)),
                                __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443))), c);
}

}  // namespace m2
