// m2_sel.cuh -- the per-channel selective scan: what its kernels and entry
// points share.
//
// D channels of N states each, B and C shared by the D/G channels of a group:
//   dt = softplus(dt_raw[d] + dt_bias[d]),  A = -exp(A_log[d, n])
//   h[d,n] <- h[d,n] * exp(dt * A[d,n]) + (dt * x[d]) * B[g,n]
//   y[d]    = sum_n h[d,n] * C[g,n] + D[d] * x[d],  times silu(z[d]) if z
// Every (token, channel, state) needs an exponential of its own; nothing of it
// is a matrix product, because the decay depends on the state index.
#pragma once

#include "m2_device.cuh"
#include "m2_internal.cuh"

namespace m2 {

struct SelArgs {
    void* ssm;  // [slots, D, N]
    int32_t* error;
    int64_t num_slots;
    int D, N, G;
    int state_bf16, act_bf16;
    const float* A_log;    // [D, N]
    const float* dt_bias;  // [D]
    const float* skip;     // [D]
    int nseq;              // sequences (scan) or rows (one token each)
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int max_seqlen;
    const void* x;
    int64_t x_stride;
    const void* dt;
    int64_t dt_stride;
    const void* B;
    int64_t B_stride;
    const void* C;
    int64_t C_stride;
    const void* z;
    int64_t z_stride;
    void* y;
    int64_t y_stride;
    const int32_t* slot_idx;
    const uint8_t* has_init;
};
bool sel_state_size_supported(int N);
cudaError_t launch_sel_scan(const SelArgs& a, cudaStream_t stream);
cudaError_t launch_sel_update(const SelArgs& a, cudaStream_t stream);

constexpr float kLog2E = 1.4426950408889634f;

// How exact the factors are goes by the activations' type. fp32 ones get the
// library's expf and log1pf on dt * A itself, within an ulp or two each; for
// 16-bit ones, whose own rounding is 2^-8, the special-function unit's 2^x
// (2^-22) of dt * (A log2 e) and the softplus below do: a decay is within 3e-7 +
// |dt A| (1e-6 + (|v| + |A_log|) 2^-23) of itself, v = dt_raw + dt_bias.
template <typename AT>
struct Decay {
    static constexpr bool kExact = sizeof(AT) == 4;
    // what a state keeps of its A, and the decay over dt by it
    // (kept finite, so that a dt of zero leaves the state as it is)
    __device__ static __forceinline__ float factor(float A_log) {
        const float f = kExact ? -expf(A_log) : -kLog2E * ex2_approx(A_log * kLog2E);
        return f < -3e38f ? -3e38f : f;
    }
    __device__ static __forceinline__ float over(float x) { return kExact ? expf(x) : ex2_approx(x); }  // x = dt * factor
    __device__ static __forceinline__ float2 softplus(float2 v);
};

// softplus of a pair: max(v, 0) + log1p(u), u = exp(-|v|) in (0, 1], with
// log1p(u) = u (1 + u r(u)), r the minimax polynomial of degree 7 on [0, 1]
// (fitted by exchange for the relative error: 5.0e-8 as its constants are printed,
// 1.6e-7 with its fp32 roundings). One special-function operation a value; expf and
// log1pf of the library take more, and a reciprocal for a series in u / (2 + u) one
// more. Within 5e-7 + |v| 2^-23 of the value: the second part is the rounding of
// -|v| log2 e, at v = -64 4e-6, where dt itself is 2e-28 (a bf16 v is known to |v| 2^-8).
// Below v = -87 it is 0.
__device__ __forceinline__ float2 softplus2_fast(float2 v) {
    const float2 u = make_float2(ex2_approx(-fabsf(v.x) * kLog2E), ex2_approx(-fabsf(v.y) * kLog2E));
    auto both = [](float c) { return make_float2(c, c); };
    float2 p = __ffma2_rn(u, both(0.0053648232f), both(-0.030065788f));
    p = __ffma2_rn(p, u, both(0.07920452f));
    p = __ffma2_rn(p, u, both(-0.13753802f));
    p = __ffma2_rn(p, u, both(0.19153655f));
    p = __ffma2_rn(p, u, both(-0.24857163f));
    p = __ffma2_rn(p, u, both(0.33321324f));
    p = __ffma2_rn(p, u, both(-0.49999648f));
    p = __ffma2_rn(p, u, both(1.f));
    return __ffma2_rn(p, u, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// silu of a pair with one special-function operation a value, within 1e-6 + |z| 2^-23
// of itself (the rounding of the exponent; 0 below z = -87): with u = exp(-|z|) in (0, 1] it is
// z / (1 + u), below zero z u / (1 + u). The reciprocal of d = 1 + u starts from
// (98 - 80 u + 32 u^2) / 99, the quadratic for which 1 - d r is the Chebyshev
// polynomial T3(2 u - 1) over 99, and takes two Newton steps r += r (1 - d r), each of
// which squares that error: 99^-4 = 1.0e-8. (8 x 2048 tokens of 8192 channels: 769 us;
// with the unit's reciprocal, silu2_f32, 780; 740 with the hardware tanh, which is
// off by 2^-12 of z, more than all of the value below z = -9.)
__device__ __forceinline__ float2 silu2_newton(float2 z) {
    const float2 u = make_float2(ex2_approx(-fabsf(z.x) * kLog2E), ex2_approx(-fabsf(z.y) * kLog2E));
    auto both = [](float c) { return make_float2(c, c); };
    const float2 minus_d = __ffma2_rn(u, both(-1.f), both(-1.f));
    float2 r = __ffma2_rn(u, both(32.f / 99.f), both(-80.f / 99.f));
    r = __ffma2_rn(r, u, both(98.f / 99.f));
#pragma unroll
    for (int i = 0; i < 2; ++i) r = __ffma2_rn(r, __ffma2_rn(minus_d, r, both(1.f)), r);
    const float2 zu = __fmul2_rn(z, u);
    return __fmul2_rn(make_float2(z.x < 0.f ? zu.x : z.x, z.y < 0.f ? zu.y : z.y), r);
}

template <typename AT>
__device__ __forceinline__ float2 Decay<AT>::softplus(float2 v) {
    return kExact ? make_float2(softplus_f32(v.x), softplus_f32(v.y)) : softplus2_fast(v);
}

}  // namespace m2
