// m2_sel_update.cu -- one token of the per-channel selective scan for a batch
// of sequences, on the slot-indexed cache in place.
//
// HBM-bound: a sequence's state [D, N] is read and written once (all but a few
// percent of the bytes). A lane owns one 16-byte vector of a channel's states,
// LPC = N * sizeof(state) / 16 lanes a channel, and works on kChannels
// channels, whose vectors it loads before it uses the first; y goes over the
// LPC lanes with xor shuffles. exp(A_log) is formed anew each call, as the
// framework's other decode steps do.
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_sel.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 256;
constexpr int kChannels = 4;  // channels per lane

template <typename AT, typename ST, int N>
__global__ void __launch_bounds__(kThreads) sel_update_kernel(const SelArgs a) {
    constexpr int EPV = Vec16<ST>::n;
    constexpr int LPC = N / EPV;
    constexpr int CPP = kThreads / LPC;  // channels the CTA covers once
    static_assert(LPC >= 1 && LPC <= 32, "a channel's lanes are in one warp");
    const int tid = threadIdx.x;
    const int l = tid % LPC;
    const int gch = a.D / a.G;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int64_t b = blockIdx.y;
    const int32_t slot = a.slot_idx[b];
    const int c_first = blockIdx.x * CPP * kChannels + tid / LPC;
    AT* y = static_cast<AT*>(a.y) + b * a.y_stride;
    if (slot < 0) {
        for (int u = 0; u < kChannels; ++u) {
            const int c = c_first + u * CPP;
            if (c < a.D && l == 0) y[c] = from_f32<AT>(0.f);
        }
        return;
    }
    if (slot >= a.num_slots) {
        if (tid == 0 && blockIdx.x == 0) record_error(a.error, M2_ERR_BAD_SLOT);
        return;
    }
    ST* state = static_cast<ST*>(a.ssm) + static_cast<int64_t>(slot) * a.D * N;
    uint4 raw[kChannels];
#pragma unroll
    for (int u = 0; u < kChannels; ++u) {
        const int c = min(c_first + u * CPP, a.D - 1);
        raw[u] = ld_stream(state + static_cast<int64_t>(c) * N + l * EPV);
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const AT* x = static_cast<const AT*>(a.x) + b * a.x_stride;
    const AT* dtp = static_cast<const AT*>(a.dt) + b * a.dt_stride;
    const AT* z = a.z ? static_cast<const AT*>(a.z) + b * a.z_stride : nullptr;
#pragma unroll
    for (int u = 0; u < kChannels; ++u) {
        const int c_true = c_first + u * CPP;
        const int c = min(c_true, a.D - 1);
        const int g = c / gch;
        const AT* Bp = static_cast<const AT*>(a.B) + b * a.B_stride + g * N + l * EPV;
        const AT* Cp = static_cast<const AT*>(a.C) + b * a.C_stride + g * N + l * EPV;
        const float dt = softplus_f32(to_f32(dtp[c]) + a.dt_bias[c]);
        const float xv = to_f32(x[c]);
        const float dtx = dt * xv;
        float h[EPV];
        unpack16<ST>(raw[u], h);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < EPV; ++e) {
            const float A = -expf(__ldg(a.A_log + static_cast<int64_t>(c) * N + l * EPV + e));
            h[e] = fmaf(h[e], expf(dt * A), dtx * to_f32(Bp[e]));
            s = fmaf(h[e], to_f32(Cp[e]), s);
        }
#pragma unroll
        for (int off = LPC / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        if (c_true < a.D) {
            st_stream(state + static_cast<int64_t>(c) * N + l * EPV, pack16<ST>(h));
            if (l == 0) {
                float yv = fmaf(a.skip[c], xv, s);
                if (z) yv *= silu_f32(to_f32(z[c]));
                y[c] = from_f32<AT>(yv);
            }
        }
    }
}

template <typename AT, typename ST, int N>
cudaError_t launch_one(const SelArgs& a, cudaStream_t s) {
    constexpr int per_cta = kThreads / (N / Vec16<ST>::n) * kChannels;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.D + per_cta - 1) / per_cta, a.nseq, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sel_update_kernel<AT, ST, N>, a);
}

template <typename AT, typename ST>
cudaError_t update_by_n(const SelArgs& a, cudaStream_t s) {
    switch (a.N) {
        case 8: return launch_one<AT, ST, 8>(a, s);
        case 16: return launch_one<AT, ST, 16>(a, s);
        case 32: return launch_one<AT, ST, 32>(a, s);
        case 64: return launch_one<AT, ST, 64>(a, s);
        case 128: return launch_one<AT, ST, 128>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_sel_update(const SelArgs& a, cudaStream_t s) {
    if (a.act_bf16) return a.state_bf16 ? update_by_n<bf16_t, bf16_t>(a, s) : update_by_n<bf16_t, float>(a, s);
    return a.state_bf16 ? update_by_n<float, bf16_t>(a, s) : update_by_n<float, float>(a, s);
}

}  // namespace m2
