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

// softplus(v) = max(v, 0) + log1p(exp(-|v|)). With u = exp(-|v|) in (0, 1],
// log1p(u) = 2 atanh(s), s = u / (2 + u) <= 1/3, by the series
// s + s^3/3 + s^5/5 + ... in s^2 <= 1/9 up to s^15 (what is left out is below
// 2e-9 of the sum). Two special-function operations and 11 FMAs or so in place
// of the library's expf and log1pf; within 4e-7 of the value, small ones
// included (v down to -87, below which it is 0).
__device__ __forceinline__ float softplus_fast(float v) {
    const float u = ex2_approx(-fabsf(v) * kLog2E);
    const float s = u * rcp_approx(2.f + u);
    const float q = s * s;
    float p = fmaf(q, 1.f / 15.f, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    const float s2 = s + s;
    return fmaxf(v, 0.f) + fmaf(s2 * q, p, s2);
}

}  // namespace m2
