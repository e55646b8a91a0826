// m2_sel_scan.cu -- the per-channel selective scan over packed prompts.
//
// A channel is handled by LPC lanes of a warp, SPL states a lane in registers;
// a CTA of 128 threads has CB = 128 / LPC channels of one sequence and walks
// its tokens in tiles of TT. Per tile:
//  * every thread takes NV 16-byte vectors of (token, channels) of x, dt and z
//    (loaded into registers a tile ahead), forms dt = softplus(..) and dt * x
//    and leaves them in shared memory; B and C of the tile go there as floats;
//  * the lanes run the tile's tokens: h = h * 2^(dt * A log2 e) + (dt x) B,
//    four tokens at a time, whose sums over the channel's lanes are exchanged
//    together (3 shuffles for 4 tokens of 4 lanes in place of 8);
//  * every thread adds D x, gates and stores y for the vectors that it loaded.
// There is no pass over the sequence but this one and no scratch memory.
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_sel.cuh"

namespace m2 {
namespace {

constexpr int kThreads = 128;

// Tokens of a tile: one 16-bit vector a thread where B and C of the tile
// (2 * TT * N floats) stay within 32 KB.
constexpr int tile_tokens(int lpc, int spl) {
    const int t = lpc >= 2 ? 8 * lpc : 16, most = 4096 / (lpc * spl);
    return t < most ? t : most;
}

template <typename AT, typename ST, int LPC, int SPL>
__global__ void __launch_bounds__(kThreads) sel_scan_kernel(const SelArgs a, const int blocks_per_group) {
    constexpr int N = LPC * SPL;
    constexpr int CB = kThreads / LPC;
    constexpr int VEC = Vec16<AT>::n;
    constexpr int TT = tile_tokens(LPC, SPL);
    constexpr int VPR = (CB + VEC - 1) / VEC;          // vectors of a token's channels
    constexpr int NV = (TT * VPR + kThreads - 1) / kThreads;
    constexpr int YP = CB + 8;                         // pitch of s_y: the four tokens that lanes write fall in other banks
    constexpr int BCV = N / VEC;                       // vectors of B (or C) of a token
    static_assert(TT % 4 == 0, "four tokens at a time");

    __shared__ __align__(16) float2 s_in[TT][CB];      // dt, dt * x
    __shared__ __align__(16) float s_y[TT][YP];
    __shared__ __align__(16) float s_B[TT][N];
    __shared__ __align__(16) float s_C[TT][N];

    const int tid = threadIdx.x;
    const int b = blockIdx.y;
    const int gch = a.D / a.G;
    const int g = blockIdx.x / blocks_per_group;
    const int c_in_group = (blockIdx.x % blocks_per_group) * CB;
    const int64_t c0 = static_cast<int64_t>(g) * gch + c_in_group;
    const int nch = min(CB, gch - c_in_group);          // a multiple of VEC
    const int64_t row0 = a.cu_seqlens[b];
    const int T = a.cu_seqlens[b + 1] - static_cast<int>(row0);
    if (T <= 0) return;
    const AT* x = static_cast<const AT*>(a.x) + row0 * a.x_stride + c0;
    const AT* dt = static_cast<const AT*>(a.dt) + row0 * a.dt_stride + c0;
    const AT* z = a.z ? static_cast<const AT*>(a.z) + row0 * a.z_stride + c0 : nullptr;
    const AT* Bp = static_cast<const AT*>(a.B) + row0 * a.B_stride + static_cast<int64_t>(g) * N;
    const AT* Cp = static_cast<const AT*>(a.C) + row0 * a.C_stride + static_cast<int64_t>(g) * N;
    AT* y = static_cast<AT*>(a.y) + row0 * a.y_stride + c0;

    const int32_t slot = a.slot_idx[b];
    // the vectors (token, channels) of this thread within a tile
    auto vec_of = [&](int i, int& t, int& c) -> bool {
        const int v = i * kThreads + tid;
        t = v / VPR;
        c = (v % VPR) * VEC;
        return t < TT && c < nch;
    };
    if (slot < 0) {  // padding: y = 0, the caches stay
        for (int t0 = 0; t0 < T; t0 += TT)
            for (int i = 0; i < NV; ++i) {
                int t, c;
                if (vec_of(i, t, c) && t0 + t < T)
                    *reinterpret_cast<uint4*>(y + (t0 + t) * a.y_stride + c) = make_uint4(0, 0, 0, 0);
            }
        return;
    }
    if (slot >= a.num_slots) {
        if (tid == 0 && blockIdx.x == 0) record_error(a.error, M2_ERR_BAD_SLOT);
        return;
    }

    // ---- this lane's channel and states
    const int lc = tid / LPC;                  // channel within the block
    const int l = tid % LPC;
    const bool live = lc < nch;
    const int64_t ch = c0 + (live ? lc : 0);
    ST* state = static_cast<ST*>(a.ssm) + (static_cast<int64_t>(slot) * a.D + ch) * N + l * SPL;
    float A2[SPL], h[SPL];
    const bool init = a.has_init && a.has_init[b];
#pragma unroll
    for (int i = 0; i < SPL; ++i) {
        A2[i] = -expf(a.A_log[ch * N + l * SPL + i]) * kLog2E;
        h[i] = init ? to_f32(state[i]) : 0.f;
    }
    float bias[NV][VEC], skip[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        int t, c;
        const bool ok = vec_of(i, t, c);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            bias[i][e] = ok ? a.dt_bias[c0 + c + e] : 0.f;
            skip[i][e] = ok ? a.skip[c0 + c + e] : 0.f;
        }
    }

    uint4 xr[NV], dr[NV], zr[NV];
    auto load_tile = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int t, c;
            const bool ok = vec_of(i, t, c) && t0 + t < T;
            const int64_t tt = t0 + t;
            xr[i] = ok ? ld_stream(x + tt * a.x_stride + c) : make_uint4(0, 0, 0, 0);
            dr[i] = ok ? ld_stream(dt + tt * a.dt_stride + c) : make_uint4(0, 0, 0, 0);
            zr[i] = ok && z ? ld_stream(z + tt * a.z_stride + c) : make_uint4(0, 0, 0, 0);
        }
    };
    load_tile(0);
    for (int t0 = 0; t0 < T; t0 += TT) {
        uint4 xc[NV], zc[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int t, c;
            const bool ok = vec_of(i, t, c);
            xc[i] = xr[i];
            zc[i] = zr[i];
            if (t < TT && c < CB) {
                float xv[VEC], dv[VEC];
                unpack16<AT>(xr[i], xv);
                unpack16<AT>(dr[i], dv);
                const bool real = ok && t0 + t < T;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float d = real ? softplus_fast(dv[e] + bias[i][e]) : 0.f;
                    s_in[t][c + e] = make_float2(d, d * xv[e]);
                }
            }
        }
        for (int v = tid; v < 2 * TT * BCV; v += kThreads) {
            const int which = v / (TT * BCV), r = v % (TT * BCV);
            const int t = r / BCV, n = (r % BCV) * VEC;
            float f[VEC];
            const int64_t tt = t0 + t;
            if (tt < T) {
                unpack16<AT>(__ldg(reinterpret_cast<const uint4*>(which ? Cp + tt * a.C_stride + n : Bp + tt * a.B_stride + n)), f);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = 0.f;
            }
            float* to = which ? &s_C[t][n] : &s_B[t][n];
#pragma unroll
            for (int e = 0; e < VEC; ++e) to[e] = f[e];
        }
        __syncthreads();
        if (t0 + TT < T) load_tile(t0 + TT);
#pragma unroll 1
        for (int t = 0; t < TT; t += 4) {
            float acc[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 in = s_in[t + j][lc];
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < SPL; ++i) {
                    h[i] = fmaf(h[i], ex2_approx(in.x * A2[i]), in.y * s_B[t + j][l * SPL + i]);
                    s = fmaf(h[i], s_C[t + j][l * SPL + i], s);
                }
                acc[j] = s;
            }
            if constexpr (LPC >= 4) {
                int which;
                const float sum = reduce_rows<LPC, 4>(acc, tid & 31, which);
                if (l % (LPC / 4) == 0) s_y[t + which][lc] = sum;
            } else if constexpr (LPC == 2) {
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float mine = (l ? acc[j + 1] : acc[j]) + __shfl_xor_sync(0xffffffffu, l ? acc[j] : acc[j + 1], 1);
                    s_y[t + j + l][lc] = mine;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) s_y[t + j][lc] = acc[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            int t, c;
            if (!vec_of(i, t, c) || t0 + t >= T) continue;
            float xv[VEC], zv[VEC], out[VEC];
            unpack16<AT>(xc[i], xv);
            unpack16<AT>(zc[i], zv);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                out[e] = fmaf(skip[i][e], xv[e], s_y[t][c + e]);
                if (z) out[e] *= silu_f32(zv[e]);
            }
            st_stream(y + static_cast<int64_t>(t0 + t) * a.y_stride + c, pack16<AT>(out));
        }
    }
    if (live) {
#pragma unroll
        for (int i = 0; i < SPL; ++i) state[i] = from_f32<ST>(h[i]);
    }
}

template <typename AT, typename ST, int LPC, int SPL>
cudaError_t launch_one(const SelArgs& a, cudaStream_t s) {
    constexpr int CB = kThreads / LPC;
    const int bpg = (a.D / a.G + CB - 1) / CB;
    const dim3 grid(static_cast<unsigned>(bpg) * a.G, static_cast<unsigned>(a.nseq));
    sel_scan_kernel<AT, ST, LPC, SPL><<<grid, kThreads, 0, s>>>(a, bpg);
    return cudaGetLastError();
}

template <typename AT, typename ST>
cudaError_t scan_by_n(const SelArgs& a, cudaStream_t s) {
    switch (a.N) {
        case 8: return launch_one<AT, ST, 2, 4>(a, s);
        case 16: return launch_one<AT, ST, 4, 4>(a, s);
        case 32: return launch_one<AT, ST, 8, 4>(a, s);
        case 64: return launch_one<AT, ST, 8, 8>(a, s);
        case 128: return launch_one<AT, ST, 16, 8>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

bool sel_state_size_supported(int N) { return N == 8 || N == 16 || N == 32 || N == 64 || N == 128; }

cudaError_t launch_sel_scan(const SelArgs& a, cudaStream_t s) {
    if (a.act_bf16) return a.state_bf16 ? scan_by_n<bf16_t, bf16_t>(a, s) : scan_by_n<bf16_t, float>(a, s);
    return a.state_bf16 ? scan_by_n<float, bf16_t>(a, s) : scan_by_n<float, float>(a, s);
}

}  // namespace m2
