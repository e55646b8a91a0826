// m2_sel_update.cu -- one token of the per-channel selective scan for a batch
// of sequences, on the slot-indexed cache in place.
//
// HBM-bound: a sequence's state [D, N] is read and written once (all but a few
// percent of the bytes). A CTA keeps one block of channels, 8 KB of a state,
// and walks rows of the batch: A = -exp(A_log), the bias and the skip of its
// channels are formed once. A producer warp brings a row's block of the state
// (one contiguous run of the slot), its x, dt and z and its B and C into a ring
// of shared-memory stages with bulk copies, kStages rows ahead, so that the copies
// never wait for the arithmetic; 256 threads run the update out of a stage,
// 16 bytes of a channel's states a lane, LPC = N * sizeof(state) / 16 lanes a
// channel, and store the new state straight from registers. y goes over the
// LPC lanes with xor shuffles. Waits are bounded as in m2_state_update.cu.
//
// 256 rows of 8192 channels of 16 states: fp32 states 50.1 us (0.88 of the copy
// bandwidth), bf16 ones 38.7 us (floor 23.5): the same arithmetic on half the bytes,
// bound by instruction issue (eight states a lane, 28 to 52 bytes of spill at 56
// registers). With fp32 activations, whose decays call expf, 60.1 us (46.9) and 47.7
// us (26.1).
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_sel.cuh"

namespace m2 {
namespace {

constexpr int kUpdate = 256;              // threads that compute
constexpr int kThreads = kUpdate + 32;    // and the producer warp
// Stages of the ring and resident CTAs per SM. 256 rows of 8192 x 16 fp32
// states (44.3 us at the copy bandwidth): 2 stages, 4 CTAs 50.2 us; 3, 4 53.4;
// 4, 4 57.0; 3, 3 54.3; 2, 3 58.4; 1, 4 65.2; 6, 2 69.7 us. Every thread reading
// its own vectors, 4 in flight and no ring: 85 us.
constexpr int kStages = 2;
constexpr int kMinBlocks = 4;
constexpr int kVectors = 2;               // 16-byte state vectors of a thread
constexpr uint64_t kWaitLimitNs = 1000000000ull;

template <typename AT, typename ST, int N>
struct Block {
    static constexpr int EPV = Vec16<ST>::n;
    static constexpr int LPC = N / EPV;
    static constexpr int CPP = kUpdate / LPC;      // channels the threads cover once
    static constexpr int CH = CPP * kVectors;      // channels of a block
    struct Stage {
        ST state[CH * N];
        AT x[CH], dt[CH], z[CH];
        AT B[N], C[N];
    };
    static_assert(LPC >= 1 && LPC <= 32, "a channel's lanes are in one warp");
    static_assert(sizeof(Stage) % 16 == 0, "stages start on 16 bytes");
};

template <typename AT, typename ST, int N>
__global__ void __launch_bounds__(kThreads, kMinBlocks) sel_update_kernel(const SelArgs a) {
    using K = Block<AT, ST, N>;
    constexpr int EPV = K::EPV, LPC = K::LPC, CPP = K::CPP;
    extern __shared__ __align__(128) uint8_t s_dyn[];
    typename K::Stage* stages = reinterpret_cast<typename K::Stage*>(s_dyn);
    __shared__ __align__(8) uint64_t s_full[kStages], s_empty[kStages];
    __shared__ int s_slot[kStages];

    const int tid = threadIdx.x;
    const int g = blockIdx.y;
    const int gch = a.D / a.G;
    const int c_in_group = blockIdx.x * K::CH;
    const int nch = min(K::CH, gch - c_in_group);  // whole 16-byte vectors of activations
    const int64_t c0 = static_cast<int64_t>(g) * gch + c_in_group;
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], kUpdate / 32);
        }
        fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    const int rows = (a.nseq - static_cast<int>(blockIdx.z) + gridDim.z - 1) / gridDim.z;  // of this CTA: blockIdx.z + i * gridDim.z
    if (tid >= kUpdate) {
        // ======== the producer warp; lane 0 issues
        const int lane = tid - kUpdate;
        int slots_of_lane = 0;
        for (int i = 0; i < rows; ++i) {
            if ((i & 31) == 0) {
                const int64_t mine = blockIdx.z + static_cast<int64_t>(i + lane) * gridDim.z;
                slots_of_lane = mine < a.nseq ? a.slot_idx[mine] : -1;
            }
            const int slot = __shfl_sync(0xffffffffu, slots_of_lane, i & 31);
            const int s = i % kStages;
            bool ok = true;
            if (lane == 0) {
                if (i >= kStages) ok = mbar_wait_bounded(&s_empty[s], (i / kStages - 1) & 1, kWaitLimitNs);
                if (ok) {
                    s_slot[s] = slot;
                    if (slot >= 0 && slot < a.num_slots) {
                        typename K::Stage& st = stages[s];
                        const int64_t b = blockIdx.z + static_cast<int64_t>(i) * gridDim.z;
                        const uint32_t act = nch * sizeof(AT), bc = N * sizeof(AT), full = nch * N * sizeof(ST);
                        mbar_arrive_expect_tx(&s_full[s], full + act * (a.z ? 3 : 2) + 2 * bc);
                        bulk_g2s(st.state, static_cast<const ST*>(a.ssm) + (static_cast<int64_t>(slot) * a.D + c0) * N, full, &s_full[s]);
                        bulk_g2s(st.x, static_cast<const AT*>(a.x) + b * a.x_stride + c0, act, &s_full[s]);
                        bulk_g2s(st.dt, static_cast<const AT*>(a.dt) + b * a.dt_stride + c0, act, &s_full[s]);
                        if (a.z) bulk_g2s(st.z, static_cast<const AT*>(a.z) + b * a.z_stride + c0, act, &s_full[s]);
                        bulk_g2s(st.B, static_cast<const AT*>(a.B) + b * a.B_stride + static_cast<int64_t>(g) * N, bc, &s_full[s]);
                        bulk_g2s(st.C, static_cast<const AT*>(a.C) + b * a.C_stride + static_cast<int64_t>(g) * N, bc, &s_full[s]);
                    } else {
                        mbar_arrive(&s_full[s]);
                    }
                }
            }
            if (i == 0) asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
            if (!__shfl_sync(0xffffffffu, static_cast<int>(ok), 0)) break;  // the others have given up
        }
        return;
    }

    // ======== the update
    const int l = tid % LPC;
    float A[kVectors][EPV], bias[kVectors], skip[kVectors];
#pragma unroll
    for (int u = 0; u < kVectors; ++u) {
        const int c = min(tid / LPC + u * CPP, nch - 1);
        bias[u] = a.dt_bias[c0 + c];
        skip[u] = a.skip[c0 + c];
#pragma unroll
        for (int e = 0; e < EPV; e += 4) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(a.A_log + (c0 + c) * N + l * EPV + e));
            A[u][e] = Decay<AT>::factor(v.x);
            A[u][e + 1] = Decay<AT>::factor(v.y);
            A[u][e + 2] = Decay<AT>::factor(v.z);
            A[u][e + 3] = Decay<AT>::factor(v.w);
        }
    }
    for (int i = 0; i < rows; ++i) {
        const int s = i % kStages;
        if (!mbar_wait_bounded(&s_full[s], (i / kStages) & 1, kWaitLimitNs)) {
            record_error(a.error, M2_ERR_TIMEOUT);
            // this CTA's copies land (bounded) before its shared memory goes
            for (int j = i; j < min(i + kStages, rows); ++j) mbar_wait_bounded(&s_full[j % kStages], (j / kStages) & 1, kWaitLimitNs);
            break;
        }
        const int64_t b = blockIdx.z + static_cast<int64_t>(i) * gridDim.z;
        AT* y = static_cast<AT*>(a.y) + b * a.y_stride + c0;
        const int slot = s_slot[s];
        if (slot >= 0 && slot < a.num_slots) {
            const typename K::Stage& st = stages[s];
            ST* out = static_cast<ST*>(a.ssm) + (static_cast<int64_t>(slot) * a.D + c0) * N;
            float Bv[EPV], Cv[EPV];
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                Bv[e] = to_f32(st.B[l * EPV + e]);
                Cv[e] = to_f32(st.C[l * EPV + e]);
            }
#pragma unroll
            for (int u = 0; u < kVectors; ++u) {
                const int c = tid / LPC + u * CPP;
                const int cc = min(c, nch - 1);  // (a lane past the end computes the last channel again)
                const float xv = to_f32(st.x[cc]);
                const float dt = Decay<AT>::softplus(make_float2(to_f32(st.dt[cc]) + bias[u], 0.f)).x, dtx = dt * xv;
                float h[EPV];
                unpack16<ST>(*reinterpret_cast<const uint4*>(st.state + cc * N + l * EPV), h);
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < EPV; ++e) {
                    h[e] = fmaf(h[e], Decay<AT>::over(dt * A[u][e]), dtx * Bv[e]);
                    sum = fmaf(h[e], Cv[e], sum);
                }
#pragma unroll
                for (int off = LPC / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (c < nch) {
                    st_stream(out + static_cast<int64_t>(c) * N + l * EPV, pack16<ST>(h));
                    if (l == 0) {
                        float yv = fmaf(skip[u], xv, sum);
                        if (a.z) yv *= silu_f32(to_f32(st.z[cc]));
                        y[c] = from_f32<AT>(yv);
                    }
                }
            }
        } else if (slot < 0) {
            for (int c = tid; c < nch; c += kUpdate) y[c] = from_f32<AT>(0.f);
        } else if (tid == 0 && blockIdx.x == 0 && g == 0) {
            record_error(a.error, M2_ERR_BAD_SLOT);
        }
        __syncwarp();
        if (tid % 32 == 0) mbar_arrive(&s_empty[s]);
    }
}

template <typename AT, typename ST, int N>
cudaError_t launch_one(const SelArgs& a, cudaStream_t s) {
    using K = Block<AT, ST, N>;
    constexpr int smem = static_cast<int>(sizeof(typename K::Stage)) * kStages;
    auto kern = sel_update_kernel<AT, ST, N>;
    static AttrOnce attrs;
    const cudaError_t e =
        attrs.ensure([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    // as many rows at once as the GPU holds CTAs for, the rows spread evenly over the rounds
    const int blocks = (a.D / a.G + K::CH - 1) / K::CH;
    const int64_t at_once = std::max<int64_t>(1, static_cast<int64_t>(kMinBlocks) * sms / (static_cast<int64_t>(blocks) * a.G));
    const int64_t rounds = (a.nseq + at_once - 1) / at_once;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, a.G, static_cast<unsigned>((a.nseq + rounds - 1) / rounds));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
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
