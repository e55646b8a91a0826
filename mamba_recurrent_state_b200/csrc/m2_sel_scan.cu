// m2_sel_scan.cu -- the per-channel selective scan over packed prompts.
//
// Bound by the special-function unit: N + 2 exponentials a (token, channel), at 16 a
// cycle and SM, against 8 bytes of HBM traffic.
//
// A channel is handled by LPC lanes of a warp, SPL states a lane in registers.
// A CTA has CB = 128 / LPC channels of one sequence and walks its tokens in
// tiles of TT, in two halves that work on different tiles at a time:
//  * the helpers (128 threads) bring the inputs a tile ahead: they take 16-byte
//    vectors of (token, channels) of x and dt, form dt = softplus(..) and dt * x,
//    and leave both in shared memory, B and C beside them as floats; and they
//    finish the tile that the scan has done: D x is added, y gated and stored;
//  * the scan (128 threads) runs h = h * exp(dt A) + (dt x) B and sums
//    h * C, four tokens at a time: shared memory holds every channel's (and
//    every state's) tokens side by side, so that a lane reads four tokens at
//    once and the packed f32x2 arithmetic takes pairs of tokens. The sums of
//    four tokens over a channel's lanes are exchanged together.
//
// Long prompts of few channels leave SMs idle. There the sequence is cut into
// as many segments as a thread-block cluster has CTAs. Each CTA runs its
// segment from a zero state without y, the cluster exchanges the segments'
// final states and sums of dt through distributed shared memory (the decay of
// a whole segment is exp(A * sum of dt)), and each CTA runs its segment again
// from the state that the ones before it leave. One launch, no scratch memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "m2_sel.cuh"

namespace m2 {
namespace {

constexpr int kScan = 128;      // threads that run the recurrence
constexpr int kHelp = 128;      // threads that bring the inputs and finish y
constexpr int kThreads = kScan + kHelp;
// Resident CTAs per SM that the registers are sized for (128 each, where eight states
// a lane spill 8 to 40 bytes a thread with 16-bit activations and four states up to 20
// with 32-bit ones; with three CTAs eight states took 1870 us in place of 762 us for
// 8 x 2048 tokens of 8192 channels), and blocks of four tokens that the scan
// unrolls (two: 926 us) where a tile is longer than 32 tokens or the decays call
// expf; otherwise it unrolls the tile, so that places in it are constants.
constexpr int kMinBlocks = 2;
constexpr int kUnroll4 = 4;

// Named barriers between the two halves of a CTA, one of each per buffer.
__device__ __forceinline__ void bar_arrive(int id) {
    asm volatile("barrier.cta.arrive %0, %1;\n" ::"r"(id), "n"(kThreads) : "memory");
}
__device__ __forceinline__ void bar_sync(int id) {
    asm volatile("barrier.cta.sync %0, %1;\n" ::"r"(id), "n"(kThreads) : "memory");
}
constexpr int kFull = 1, kDone = 3;  // + buffer

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// A float of cluster CTA `rank`, at the place of `local` in its shared memory.
__device__ __forceinline__ float ld_cluster_f32(const float* local, uint32_t rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

template <typename AT, int LPC, int SPL>
struct Scan {
    using Factors = Decay<AT>;
    static constexpr int N = LPC * SPL;
    static constexpr int CB = kScan / LPC;
    static constexpr int VEC = Vec16<AT>::n;
    // tokens of a tile: one 16-bit vector a helper where B and C stay within 16 KB
    static constexpr int TT = 8 * LPC < 2048 / N ? 8 * LPC : 2048 / N;
    static constexpr int P = TT + 4;                          // pitch of a channel's (or state's) tokens
    static constexpr int VPR = CB / VEC;                      // vectors of a token's channels
    static constexpr int VT = kHelp / VPR;                    // tokens from one vector of a helper to its next
    static constexpr int NV = (TT + VT - 1) / VT;
    static constexpr int BCV = N / VEC;                       // vectors of B (or C) of a token
    static constexpr int NBC = (2 * TT * BCV + kHelp - 1) / kHelp;
    static constexpr int ROT = 32 / VPR > 4 ? 32 / VPR : 4;
    static_assert(TT % 4 == 0 && (TT & (TT - 1)) == 0 && CB % VEC == 0 && kHelp % VPR == 0,
                  "four tokens at a time; a helper keeps its channels");
    // Where token t of channel c lies in the channel's row: rows of other
    // vectors are rotated (by multiples of four tokens), so that the helpers,
    // who write and read a token's channels, meet other banks.
    __device__ static __forceinline__ int place(int c, int t) { return (t + ROT * (c / VEC)) & (TT - 1); }
    // The same for the states' rows of B and C: the helpers of a warp write
    // BCV vectors of 32 / BCV tokens (1649 tokens of 4096 channels of 64 states:
    // 248 us without, 182 to 188 us with). With fp32 activations, whose scan is bound by
    // expf and where a vector holds fewer states than a channel has lanes, the
    // places cost more than the conflicts (334 us without, 350 us with).
    static constexpr int BC_ROT = Factors::kExact ? 0 : (32 / BCV > 4 ? 32 / BCV : 4);
    __device__ static __forceinline__ int bc_place(int vec, int t) { return (t + BC_ROT * vec) & (TT - 1); }
    struct Buffer {
        float d[CB][P];     // dt
        float u[CB][P];     // dt * x
        float y[CB][P];
        float bc[2][N][P];  // B, C
    };
    struct Shared {
        Buffer buf[2];
        float bias[CB];
        float skip[CB];
        float end_h[CB][N];  // a segment's final state from zero, and its sum of dt
        float end_dt[CB];
    };
};

// Four tokens' sums over a channel's lanes, to the tokens t .. t + 3 of its row of y.
template <int LPC>
__device__ __forceinline__ void put_sums(float* y, float2 y01, float2 y23, int l, int lane) {
    if constexpr (LPC >= 4) {
        const float four[4] = {y01.x, y01.y, y23.x, y23.y};
        int which;
        const float sum = reduce_rows<LPC, 4>(four, lane, which);
        if (l % (LPC / 4) == 0) y[which] = sum;
    } else {
        const float2 keep = l ? y23 : y01, give = l ? y01 : y23;
        *reinterpret_cast<float2*>(y + 2 * l) =
            make_float2(keep.x + __shfl_xor_sync(0xffffffffu, give.x, 1), keep.y + __shfl_xor_sync(0xffffffffu, give.y, 1));
    }
}

// The tokens of one tile for a lane's states s * LPC + l of channel lc. Y: y is
// wanted; otherwise the sum of dt is.
template <bool Y, int SPL, int LPC, typename K>
__device__ __forceinline__ void scan_tile(typename K::Buffer& buf, const float (&A)[SPL], float (&h)[SPL], float& sum_dt, int lc, int l,
                                          int lane) {
    constexpr int TT = K::TT, P = K::P;
    const float* d_of = buf.d[lc];
    const float* u_of = buf.u[lc];
    const float* B = buf.bc[0][l];
    const float* C = buf.bc[1][l];
    float* y = buf.y[lc];
    auto load4 = [](const float* p) { return *reinterpret_cast<const float4*>(p); };
    // the vector that holds state s * LPC + l (a constant unless a vector is shorter than LPC)
    const int lane_vec = K::BC_ROT != 0 && LPC > K::VEC ? l / K::VEC : 0;
    auto at = [&](int s, int t) { return s * LPC * P + K::bc_place(s * LPC / K::VEC + lane_vec, t); };
    float4 d = load4(d_of + K::place(lc, 0)), u = load4(u_of + K::place(lc, 0)), b[SPL], c[SPL];
#pragma unroll
    for (int s = 0; s < SPL; ++s) {
        b[s] = load4(B + at(s, 0));
        if constexpr (Y) c[s] = load4(C + at(s, 0));
    }
    float2 last01 = make_float2(0.f, 0.f), last23 = last01;
    constexpr int kUnroll = TT <= 32 && !K::Factors::kExact ? TT / 4 : kUnroll4;
#pragma unroll kUnroll
    for (int t = 0; t < TT; t += 4) {
        const float2 d01 = make_float2(d.x, d.y), d23 = make_float2(d.z, d.w), u01 = make_float2(u.x, u.y), u23 = make_float2(u.z, u.w);
        if constexpr (!Y) sum_dt += (d.x + d.y) + (d.z + d.w);
        // the next four tokens' inputs, before anything is stored
        const int tn = t + 4 < TT ? t + 4 : t;
        float4 nb[SPL], nc[SPL];
        d = load4(d_of + K::place(lc, tn));
        u = load4(u_of + K::place(lc, tn));
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            nb[s] = load4(B + at(s, tn));
            if constexpr (Y) nc[s] = load4(C + at(s, tn));
        }
        float2 y01, y23;
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            const float2 a2 = make_float2(A[s], A[s]);
            const float2 x01 = __fmul2_rn(d01, a2), x23 = __fmul2_rn(d23, a2);
            const float2 v01 = __fmul2_rn(u01, make_float2(b[s].x, b[s].y)), v23 = __fmul2_rn(u23, make_float2(b[s].z, b[s].w));
            const float h0 = fmaf(h[s], K::Factors::over(x01.x), v01.x);
            const float h1 = fmaf(h0, K::Factors::over(x01.y), v01.y);
            const float h2 = fmaf(h1, K::Factors::over(x23.x), v23.x);
            h[s] = fmaf(h2, K::Factors::over(x23.y), v23.y);
            if constexpr (Y) {
                const float2 c01 = make_float2(c[s].x, c[s].y), c23 = make_float2(c[s].z, c[s].w);
                y01 = s == 0 ? __fmul2_rn(make_float2(h0, h1), c01) : __ffma2_rn(make_float2(h0, h1), c01, y01);
                y23 = s == 0 ? __fmul2_rn(make_float2(h2, h[s]), c23) : __ffma2_rn(make_float2(h2, h[s]), c23, y23);
            }
        }
        if constexpr (Y) {
            // the sums of the four tokens before: their exchange runs beside this block's arithmetic
            if (t > 0) put_sums<LPC>(y + K::place(lc, t - 4), last01, last23, l, lane);
            last01 = y01;
            last23 = y23;
        }
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            b[s] = nb[s];
            if constexpr (Y) c[s] = nc[s];
        }
    }
    if constexpr (Y) put_sums<LPC>(y + K::place(lc, TT - 4), last01, last23, l, lane);
}

template <typename AT, typename ST, int LPC, int SPL>
__global__ void __launch_bounds__(kThreads, kMinBlocks) sel_scan_kernel(const SelArgs a, const int blocks, const int segments) {
    using K = Scan<AT, LPC, SPL>;
    constexpr int N = K::N, CB = K::CB, VEC = K::VEC, TT = K::TT, VT = K::VT, NV = K::NV, BCV = K::BCV, NBC = K::NBC;
    extern __shared__ __align__(16) uint8_t s_dyn[];
    typename K::Shared& sm = *reinterpret_cast<typename K::Shared*>(s_dyn);

    const int b = blockIdx.z;
    const int gch = a.D / a.G;
    const int g = blockIdx.y;
    const int rank = segments > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int c_in_group = (segments > 1 ? blockIdx.x / segments : blockIdx.x) * CB;
    const int64_t c0 = static_cast<int64_t>(g) * gch + c_in_group;
    const int nch = min(CB, gch - c_in_group);          // a multiple of VEC
    const int64_t row0 = a.cu_seqlens[b];
    const int T = a.cu_seqlens[b + 1] - static_cast<int>(row0);
    const int32_t slot = a.slot_idx[b];
    if (T <= 0) return;  // here and below: the whole cluster alike
    if (slot >= a.num_slots) {
        if (threadIdx.x == 0 && blockIdx.x == 0 && g == 0) record_error(a.error, M2_ERR_BAD_SLOT);
        return;
    }
    const int all_tiles = T / TT + (T % TT != 0);
    const int per_segment = segments > 1 ? (all_tiles + segments - 1) / segments : all_tiles;
    const int first = rank * per_segment, last = min(first + per_segment, all_tiles);  // this CTA's tiles
    const bool ahead = segments > 1 && last < all_tiles;  // a later segment needs this one's end

    for (int c = threadIdx.x; c < CB; c += kThreads) {
        sm.bias[c] = c < nch ? a.dt_bias[c0 + c] : 0.f;
        sm.skip[c] = c < nch ? a.skip[c0 + c] : 0.f;
    }
    __syncthreads();

    if (threadIdx.x < kScan) {
        // ======== the recurrence: this lane's channel and states
        if (slot < 0) return;
        const int tid = threadIdx.x;
        const int lc = tid / LPC;                  // channel within the block
        const int l = tid % LPC;
        const bool live = lc < nch;
        const int64_t ch = c0 + (live ? lc : 0);
        ST* state = static_cast<ST*>(a.ssm) + (static_cast<int64_t>(slot) * a.D + ch) * N + l;  // states s * LPC + l
        float A[SPL], h[SPL];  // (A: as Decay keeps it)
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            A[s] = K::Factors::factor(a.A_log[ch * N + s * LPC + l]);
            h[s] = 0.f;
        }
        float sum_dt = 0.f;
        int q = 0;  // tiles so far: their buffer is q & 1
        if (ahead) {
            for (int i = first; i < last; ++i, ++q) {
                bar_sync(kFull + (q & 1));
                scan_tile<false, SPL, LPC, K>(sm.buf[q & 1], A, h, sum_dt, lc, l, tid & 31);
                bar_arrive(kDone + (q & 1));
            }
#pragma unroll
            for (int s = 0; s < SPL; ++s) sm.end_h[lc][s * LPC + l] = h[s];
            if (l == 0) sm.end_dt[lc] = sum_dt;
        }
        if (segments > 1) {
            cluster_arrive();
            cluster_wait();
        }
        const bool init = a.has_init && a.has_init[b];
#pragma unroll
        for (int s = 0; s < SPL; ++s) h[s] = init ? to_f32(state[s * LPC]) : 0.f;
        if (segments > 1) {
            for (int r = 0; r < rank && r * per_segment < all_tiles; ++r) {
                const float dt = ld_cluster_f32(&sm.end_dt[lc], r);
#pragma unroll
                for (int s = 0; s < SPL; ++s)
                    h[s] = fmaf(h[s], K::Factors::over(dt * A[s]), ld_cluster_f32(&sm.end_h[lc][s * LPC + l], r));
            }
            cluster_arrive();  // done with the others' shared memory and with the slot's initial state
        }
        for (int i = first; i < last; ++i, ++q) {
            bar_sync(kFull + (q & 1));
            scan_tile<true, SPL, LPC, K>(sm.buf[q & 1], A, h, sum_dt, lc, l, tid & 31);
            bar_arrive(kDone + (q & 1));
        }
        // The arrive above releases this CTA's reads of the others' shared memory and
        // of the slot: after the wait the last segment may write the slot, and
        // every CTA may leave.
        if (segments > 1) cluster_wait();
        if (live && first < last && last == all_tiles) {
#pragma unroll
            for (int s = 0; s < SPL; ++s) state[s * LPC] = from_f32<ST>(h[s]);
        }
        return;
    }

    // ======== the helpers: inputs a tile ahead, y a tile behind
    const int tid = threadIdx.x - kScan;
    const int vt = tid / K::VPR, vc = (tid % K::VPR) * VEC;  // this thread's vectors: tokens vt + i * VT, channels vc ..
    const bool vc_ok = vc < nch;
    const AT* x = static_cast<const AT*>(a.x) + row0 * a.x_stride + c0 + vc;
    const AT* dt = static_cast<const AT*>(a.dt) + row0 * a.dt_stride + c0 + vc;
    const AT* z = a.z ? static_cast<const AT*>(a.z) + row0 * a.z_stride + c0 + vc : nullptr;
    AT* y = static_cast<AT*>(a.y) + row0 * a.y_stride + c0 + vc;
    if (slot < 0) {  // padding: y = 0, the caches stay
        const int64_t end = min(static_cast<int64_t>(last) * TT, static_cast<int64_t>(T));
        for (int64_t t = static_cast<int64_t>(first) * TT + vt; t < end && vc_ok; t += VT)
            *reinterpret_cast<uint4*>(y + t * a.y_stride) = make_uint4(0, 0, 0, 0);
        return;
    }
    const AT* Bp = static_cast<const AT*>(a.B) + row0 * a.B_stride + static_cast<int64_t>(g) * N;
    const AT* Cp = static_cast<const AT*>(a.C) + row0 * a.C_stride + static_cast<int64_t>(g) * N;

    uint4 xr[NV], dr[NV], zr[NV], bcr[NBC];  // the raw inputs of the next tile
    auto load_tile = [&](int i, bool full) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int64_t t = i * TT + vt + v * VT;
            const bool ok = vc_ok && t < T && vt + v * VT < TT;
            xr[v] = ok ? ld_stream(x + t * a.x_stride) : make_uint4(0, 0, 0, 0);
            dr[v] = ok ? ld_stream(dt + t * a.dt_stride) : make_uint4(0, 0, 0, 0);
            zr[v] = ok && full && z ? ld_stream(z + t * a.z_stride) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int v = 0; v < NBC; ++v) {
            const int q = v * kHelp + tid, which = q / (TT * BCV), t = q % (TT * BCV) / BCV, n = q % BCV * VEC;
            const int64_t tt = i * TT + t;
            bcr[v] = which < 2 && tt < T
                         ? __ldg(reinterpret_cast<const uint4*>(which ? Cp + tt * a.C_stride + n : Bp + tt * a.B_stride + n))
                         : make_uint4(0, 0, 0, 0);
        }
    };
    uint4 xc[NV], zc[NV];  // x and z of the tile that the scan is at
    uint4 xn[NV], zn[NV];  // and of the one after it
    auto prepare = [&](int i, int q) {
        typename K::Buffer& buf = sm.buf[q & 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int t = vt + v * VT;
            xn[v] = xr[v];
            zn[v] = zr[v];
            if (t < TT) {
                float xv[VEC], dv[VEC];
                unpack16<AT>(xr[v], xv);
                unpack16<AT>(dr[v], dv);
                const bool real = i * TT + t < T;  // past the end dt = 0: the state stays
                const int at = K::place(vc, t);
#pragma unroll
                for (int e = 0; e < VEC; e += 2) {
                    const float2 bias = *reinterpret_cast<const float2*>(&sm.bias[vc + e]);
                    float2 d = K::Factors::softplus(__fadd2_rn(make_float2(dv[e], dv[e + 1]), bias));
                    if (!real) d = make_float2(0.f, 0.f);
                    const float2 u = __fmul2_rn(d, make_float2(xv[e], xv[e + 1]));
                    buf.d[vc + e][at] = d.x;
                    buf.d[vc + e + 1][at] = d.y;
                    buf.u[vc + e][at] = u.x;
                    buf.u[vc + e + 1][at] = u.y;
                }
            }
        }
#pragma unroll
        for (int v = 0; v < NBC; ++v) {
            const int p = v * kHelp + tid, which = p / (TT * BCV), t = p % (TT * BCV) / BCV, n = p % BCV * VEC;
            if (which < 2) {
                float f[VEC];
                unpack16<AT>(bcr[v], f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) buf.bc[which][n + e][K::bc_place(n / VEC, t)] = f[e];
            }
        }
        bar_arrive(kFull + (q & 1));
    };
    auto finish = [&](int i, int q) {
        typename K::Buffer& buf = sm.buf[q & 1];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int t = vt + v * VT;
            if (t >= TT || i * TT + t >= T || !vc_ok) continue;
            float xv[VEC], zv[VEC], out[VEC];
            unpack16<AT>(xc[v], xv);
            unpack16<AT>(zc[v], zv);
            const int at = K::place(vc, t);
#pragma unroll
            for (int e = 0; e < VEC; e += 2) {
                const float2 skip = *reinterpret_cast<const float2*>(&sm.skip[vc + e]);
                float2 o = __ffma2_rn(skip, make_float2(xv[e], xv[e + 1]), make_float2(buf.y[vc + e][at], buf.y[vc + e + 1][at]));
                if (z) {
                    const float2 zz = make_float2(zv[e], zv[e + 1]);
                    o = __fmul2_rn(o, K::Factors::kExact ? silu2_f32(zz) : silu2_newton(zz));
                }
                out[e] = o.x;
                out[e + 1] = o.y;
            }
            st_stream(y + static_cast<int64_t>(i * TT + t) * a.y_stride, pack16<AT>(out));
        }
    };

    int q = 0;
    auto run = [&](bool full) {
        load_tile(first, full);
        prepare(first, q);
        if (first + 1 < last) load_tile(first + 1, full);
        for (int i = first; i < last; ++i, ++q) {
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                xc[v] = xn[v];
                zc[v] = zn[v];
            }
            if (i + 1 < last) {
                prepare(i + 1, q + 1);
                if (i + 2 < last) load_tile(i + 2, full);
            }
            bar_sync(kDone + (q & 1));
            if (full) finish(i, q);
        }
    };
    if (ahead) run(false);
    if (segments > 1) {
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
    }
    if (first < last) run(true);
    if (segments > 1) cluster_wait();
}

template <typename AT, typename ST, int LPC, int SPL>
cudaError_t launch_one(const SelArgs& a, int segments, cudaStream_t s) {
    using K = Scan<AT, LPC, SPL>;
    constexpr int smem = static_cast<int>(sizeof(typename K::Shared));
    auto kern = sel_scan_kernel<AT, ST, LPC, SPL>;
    static AttrOnce attrs;
    const cudaError_t e =
        attrs.ensure([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    const int blocks = (a.D / a.G + K::CB - 1) / K::CB;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks * segments), static_cast<unsigned>(a.G), static_cast<unsigned>(a.nseq));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = segments;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = segments > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a, blocks, segments);
}

// How the channels are spread: lanes a channel and segments a sequence. Fewer
// states a lane make a token shorter and need more CTAs; segments run every
// token twice. Measured, ns a token of a CTA by the states that a lane has, for
// 16- and 32-bit activations: with one CTA an SM, with two; and the two runs of a
// segment's token with few clusters (up to half the SMs in CTAs) and with
// many (two CTAs an SM; 33 clusters of 8 fit). A segment's exchange and second
// start take 1 us, a round of CTAs 3 us to start and one of clusters 5. The plan
// is the cheapest by these; a batch counts as many of its longest sequence as its tokens
// make, and shorter ones fill the last round of CTAs. What that gives at 16384
// tokens of 16 states: 512 channels 143 us (two states a lane in segments), 1024 228
// (four, segments), 2048 438 (eight, segments), 4096 600 (four), 8192 982 (four). The
// table and the other choices were timed with a gate of the hardware tanh, 2 to 4%
// faster throughout: 512 channels 140 us, 459 without segments; 1024 222, 390 with
// eight states a lane; 4096 578, 676 with two; 8192 944, 1060 with eight. Over 60 drawn
// shapes the plan took 1.04 times the best one's time in the geometric mean, 1.43 times
// at worst: prompts of a few tokens, where what a CTA takes to start decides.
constexpr int kSegments = 8;
struct Plan {
    int lpc, segments;
};
Plan plan_scan(const SelArgs& a) {
    static const struct {
        int states;
        double one, two, few, many;
    } kTimes[2][3] = {{{8, 62, 97, 118, 200}, {4, 36, 58, 65, 106}, {2, 29, 41, 46, 68}},
                      {{8, 122, 188, 219, 355}, {4, 65, 105, 110, 187}, {2, 36, 56, 60, 97}}};
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    const double T = static_cast<double>(std::max<int64_t>(1, std::min<int64_t>(a.max_seqlen, a.total_tokens)));
    const double seqs = std::min<double>(a.nseq, std::max(1., a.total_tokens / T));  // of the longest's length
    Plan best{};
    double best_ns = 0.;
    auto offer = [&](int lpc, int segments, double ns) {
        if (best.lpc == 0 || ns < best_ns) {
            best = {lpc, segments};
            best_ns = ns;
        }
    };
    for (auto k : kTimes[a.act_bf16 ? 0 : 1]) {
        const int lpc = a.N / k.states;
        if (lpc < 2 || lpc > 16) continue;
        if (lpc == 2) {  // 64 channels a CTA: no shorter than the helpers' work
            k.one = std::max(k.one, 58.);
            k.two = std::max(k.two, 72.);
            k.few = std::max(k.few, 76.);
            k.many = std::max(k.many, 129.);
        }
        const double blocks = static_cast<double>(a.G) * ((a.D / a.G + kScan / lpc - 1) / (kScan / lpc));
        const double all = blocks * a.nseq, full = blocks * seqs, in_segments = all * kSegments;
        const bool ragged = seqs < a.nseq;
        auto rounds = [&](double ctas, double places) { return std::max(1., ragged ? ctas / places : std::ceil(ctas / places)); };
        const double places = 2. * sms, in_clusters = places * 8 / 9;
        const double shared = k.one + (k.two - k.one) * std::min(1., std::max(.5, full / places));
        offer(lpc, 1, 3000. * std::max(1., all / places) + T * (all <= sms ? k.one : shared * rounds(full, places)));
        const double twice = in_segments <= sms / 2 ? k.few : k.many * rounds(full * kSegments, in_clusters);
        offer(lpc, kSegments, 1000. + 5000. * std::max(1., in_segments / in_clusters) + T / kSegments * twice);
    }
    return best;
}

template <typename AT, typename ST>
cudaError_t scan_by_n(const SelArgs& a, cudaStream_t s) {
    const Plan p = plan_scan(a);
    switch (a.N * 100 + p.lpc) {
        case 802: return launch_one<AT, ST, 2, 4>(a, p.segments, s);
        case 804: return launch_one<AT, ST, 4, 2>(a, p.segments, s);
        case 1602: return launch_one<AT, ST, 2, 8>(a, p.segments, s);
        case 1604: return launch_one<AT, ST, 4, 4>(a, p.segments, s);
        case 1608: return launch_one<AT, ST, 8, 2>(a, p.segments, s);
        case 3204: return launch_one<AT, ST, 4, 8>(a, p.segments, s);
        case 3208: return launch_one<AT, ST, 8, 4>(a, p.segments, s);
        case 3216: return launch_one<AT, ST, 16, 2>(a, p.segments, s);
        case 6408: return launch_one<AT, ST, 8, 8>(a, p.segments, s);
        case 6416: return launch_one<AT, ST, 16, 4>(a, p.segments, s);
        case 12816: return launch_one<AT, ST, 16, 8>(a, p.segments, s);
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
