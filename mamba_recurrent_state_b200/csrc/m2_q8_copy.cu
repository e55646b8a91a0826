// m2_q8_copy.cu -- states between a 16/32-bit slot cache and an 8-bit one:
// quantised as they are written (store), as values as they are read (load).
// The conv rows of a slot are copied as they are.
//
// Both kernels are streams: store reads R*N*s + writes R*(N + 4) bytes a
// sequence, load the reverse. A row of N values is handled by N/16 lanes of
// one warp, 16 values each, so a row's maximum is a few shuffles; a lane takes
// its values as 16-byte vectors a row-width apart, so every load and store of
// a warp is contiguous. A CTA has kUnroll passes of rows in flight before it
// uses the first.
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_q8.cuh"

namespace m2 {
namespace {

// 128 Nemotron-H sequences (422 MB either way, 65.3 us at the copy bandwidth):
// store 68.7 us, load 69.2 us with 128 threads and four passes; 256 threads and
// four 70.7 / 77.1, one 77.0 / 69.8, eight 74.8 / 79.3; 64 and four 70.1 / 69.7 us.
constexpr int kThreads = 128;
constexpr int kUnroll = 4;

template <int EPV>
__device__ __forceinline__ void put_codes(int8_t* p, const uint32_t* w) {
    if constexpr (EPV == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// The slots of copy i; false where it has nothing to do (recording bad slots).
__device__ __forceinline__ bool copy_slots(const Q8CopyArgs& a, int i, bool store, int64_t& full, int64_t& q8) {
    const int32_t s = a.src_idx[i], d = a.dst_idx[i];
    const int32_t f = store ? s : d, q = store ? d : s;
    const bool first = threadIdx.x == 0 && blockIdx.x == 0;
    if (f < 0 || q < 0) return false;
    if (f >= a.num_slots) {
        if (first) record_error(a.error, M2_ERR_BAD_SLOT);
        return false;
    }
    if (q >= a.q_num_slots) {
        if (first) record_error(a.q_error, M2_ERR_BAD_SLOT);
        return false;
    }
    full = f;
    q8 = q;
    return true;
}

// The CTAs past the row blocks copy the conv rows.
__device__ __forceinline__ void copy_conv(const void* src, void* dst, int64_t bytes, int part, int parts) {
    const uint4* s = static_cast<const uint4*>(src);
    uint4* d = static_cast<uint4*>(dst);
    for (int64_t i = static_cast<int64_t>(part) * kThreads + threadIdx.x; i < bytes / 16;
         i += static_cast<int64_t>(parts) * kThreads)
        st_stream(d + i, ld_stream(s + i));
}

template <typename ST, int N>
__global__ void __launch_bounds__(kThreads) q8_store_kernel(const Q8CopyArgs a, const int row_blocks) {
    constexpr int EPV = Vec16<ST>::n;
    constexpr int LPR = N / 16;
    constexpr int V = 16 / EPV;  // vectors per lane
    constexpr int RPP = kThreads / LPR;
    const int tid = threadIdx.x;
    for (int i = blockIdx.y; i < a.n; i += gridDim.y) {
        int64_t full, q8;
        if (!copy_slots(a, i, true, full, q8)) continue;
        if (static_cast<int>(blockIdx.x) >= row_blocks) {
            copy_conv(static_cast<const char*>(a.conv) + full * a.conv_bytes, static_cast<char*>(a.q_conv) + q8 * a.conv_bytes,
                      a.conv_bytes, blockIdx.x - row_blocks, gridDim.x - row_blocks);
            continue;
        }
        const ST* src = static_cast<const ST*>(a.ssm) + full * a.rows * N;
        int8_t* dst = a.q + q8 * a.rows * N;
        const int lane = tid % LPR;
        const int r0 = blockIdx.x * (RPP * kUnroll) + tid / LPR;
        uint4 raw[kUnroll][V];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * RPP;
#pragma unroll
            for (int v = 0; v < V; ++v)
                raw[u][v] = r < a.rows ? ld_stream(src + static_cast<int64_t>(r) * N + (v * LPR + lane) * EPV)
                                       : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * RPP;
            float f[V][EPV];
            float m = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                unpack16<ST>(raw[u][v], f[v]);
#pragma unroll
                for (int e = 0; e < EPV; ++e) m = max_nan(m, fabsf(f[v][e]));
            }
#pragma unroll
            for (int off = LPR / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
            float scale, inv;
            q8_scale(m, scale, inv);
            if (r < a.rows) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    uint32_t w[EPV / 4];
#pragma unroll
                    for (int e = 0; e < EPV; e += 4)
                        w[e / 4] = q8_pack(fmaf(f[v][e], inv, kQ8Magic), fmaf(f[v][e + 1], inv, kQ8Magic),
                                           fmaf(f[v][e + 2], inv, kQ8Magic), fmaf(f[v][e + 3], inv, kQ8Magic));
                    put_codes<EPV>(dst + static_cast<int64_t>(r) * N + (v * LPR + lane) * EPV, w);
                }
                if (lane == 0) a.scale[q8 * a.rows + r] = scale;
            }
        }
    }
}

template <typename ST, int N>
__global__ void __launch_bounds__(kThreads) q8_load_kernel(const Q8CopyArgs a, const int row_blocks) {
    constexpr int EPV = Vec16<ST>::n;
    constexpr int LPR = N / 16;
    constexpr int V = 16 / EPV;
    constexpr int RPP = kThreads / LPR;
    const int tid = threadIdx.x;
    for (int i = blockIdx.y; i < a.n; i += gridDim.y) {
        int64_t full, q8;
        if (!copy_slots(a, i, false, full, q8)) continue;
        if (static_cast<int>(blockIdx.x) >= row_blocks) {
            copy_conv(static_cast<const char*>(a.q_conv) + q8 * a.conv_bytes, static_cast<char*>(a.conv) + full * a.conv_bytes,
                      a.conv_bytes, blockIdx.x - row_blocks, gridDim.x - row_blocks);
            continue;
        }
        const int8_t* src = a.q + q8 * a.rows * N;
        ST* dst = static_cast<ST*>(a.ssm) + full * a.rows * N;
        const int lane = tid % LPR;
        const int r0 = blockIdx.x * (RPP * kUnroll) + tid / LPR;
        uint32_t w[kUnroll][V][EPV / 4];
        float scale[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = min(r0 + u * RPP, a.rows - 1);
            scale[u] = __ldg(a.scale + q8 * a.rows + r);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int8_t* p = src + static_cast<int64_t>(r) * N + (v * LPR + lane) * EPV;
                if constexpr (EPV == 8) {
                    const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
                    w[u][v][0] = t.x;
                    w[u][v][1] = t.y;
                } else {
                    w[u][v][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int r = r0 + u * RPP;
            if (r >= a.rows) break;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[EPV];
#pragma unroll
                for (int e = 0; e < EPV; e += 4) {
                    float2 lo, hi;
                    q8_unpack(w[u][v][e / 4], lo, hi);
                    f[e] = lo.x * scale[u];
                    f[e + 1] = lo.y * scale[u];
                    f[e + 2] = hi.x * scale[u];
                    f[e + 3] = hi.y * scale[u];
                }
                st_stream(dst + static_cast<int64_t>(r) * N + (v * LPR + lane) * EPV, pack16<ST>(f));
            }
        }
    }
}

template <typename ST, int N>
cudaError_t launch_copy(const Q8CopyArgs& a, bool store, cudaStream_t s) {
    constexpr int rows = kThreads / (N / 16) * kUnroll;  // per CTA
    const int row_blocks = (a.rows + rows - 1) / rows;
    const int conv_blocks = static_cast<int>(std::min<int64_t>(8, (a.conv_bytes / 16 + kThreads * 4 - 1) / (kThreads * 4)));
    const dim3 grid(static_cast<unsigned>(row_blocks + conv_blocks), static_cast<unsigned>(std::min(a.n, 65535)));
    if (store) q8_store_kernel<ST, N><<<grid, kThreads, 0, s>>>(a, row_blocks);
    else q8_load_kernel<ST, N><<<grid, kThreads, 0, s>>>(a, row_blocks);
    return cudaGetLastError();
}

template <typename ST>
cudaError_t copy_by_n(const Q8CopyArgs& a, bool store, cudaStream_t s) {
    switch (a.N) {
        case 64: return launch_copy<ST, 64>(a, store, s);
        case 128: return launch_copy<ST, 128>(a, store, s);
        case 256: return launch_copy<ST, 256>(a, store, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_q8_store(const Q8CopyArgs& a, cudaStream_t s) {
    return a.state_bf16 ? copy_by_n<bf16_t>(a, true, s) : copy_by_n<float>(a, true, s);
}
cudaError_t launch_q8_load(const Q8CopyArgs& a, cudaStream_t s) {
    return a.state_bf16 ? copy_by_n<bf16_t>(a, false, s) : copy_by_n<float>(a, false, s);
}

}  // namespace m2
