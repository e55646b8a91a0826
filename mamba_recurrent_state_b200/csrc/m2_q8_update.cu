// m2_q8_update.cu -- the one-token decode step on an 8-bit state cache: the
// conv tap and the selective state update of m2_state_update.cu, with the
// state read as codes * scale, updated in fp32 and stored as codes and a new
// scale per row, all in one launch. Per head h, group g = h / (H/G):
//   S = code * scale, S' = S*dA + (dt*x)*B[g], y = sum_n S'*C[g] + D*x
//   a = max_n |S'|, scale' = a / 127, code' = rne(S' * (127 / a))
// y comes from the unrounded S'. All of it is fp32 between the codes.
//
// Work decomposition:
//  * A sequence's state is H*P rows of N codes. The rows of an SSM group are
//    cut into tiles of tile_rows rows (the last may be short), a CTA of 128
//    threads each, the group's CTAs one thread-block cluster.
//  * One thread puts the slot's conv rows, the tile's scales and the codes in
//    flight as bulk copies before anything else is computed.
//  * LPR = N/16 lanes share a row, 16 codes (one 16-byte vector) a lane. A
//    thread works on two rows at once: their S' stay in registers while the
//    sums y and the maxima a go over the LPR lanes, both with the first level
//    exchanging halves, so that one lane in two ends with one row's result and
//    forms one row's scale and inverse only (a product with 1/127 and the
//    special-function unit's reciprocal, within 2^-22 of the quotients); the
//    inverses come back with one shuffle a row.
//  * Codes become floats by a byte permute into 2^23 and one exact subtraction
//    and are rounded by one FMA with 1.5 * 2^23 (m2_q8.cuh): no conversion
//    instructions, which issue at a quarter of the FMA rate.
//  * Conv, cluster and waits as in m2_state_update.cu: every CTA computes the
//    conv of its x channels and of the group's B and C; cluster rank 0 alone
//    rolls the group's B/C conv rows, after all have read them.
//
// Bound by instruction issue beside HBM: a code takes 0.34 warp instructions, all
// included (unpack, update, y, maximum, round, pack, exchanges, conv), which for
// 64 Nemotron-H rows is 20 us of the SMs' issue slots beside 23 us of HBM time,
// and a CTA's wait for its rows overlaps only with other CTAs' arithmetic.
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_q8.cuh"

namespace m2 {
namespace {

// Threads of a CTA, rows of its tile, the resident CTAs per SM that the
// registers are sized for (five do reside: 90 registers, 43 KB), passes over the
// tile that one copy brings. 64 Nemotron-H rows (23.2 us at the copy bandwidth):
// 128, 256, 4, 8 passes 35.8 us; sized for three CTAs 39.1 (126 registers, four
// reside), for five 42.1 (the compiler trades registers for instructions); 192
// rows 43.4; 256 threads 57.5, with 512 rows 52.3 us; two rings of 256 rows, the
// next row's copies under this one's arithmetic, 54.3 us.
constexpr int kThreads = 128;
constexpr int kTileRows = 256;
constexpr int kMinBlocks = 4;
constexpr int kWarps = kThreads / 32;
constexpr int kRowsPerThread = 2;
constexpr int kMaxPasses = 16;
constexpr int kCopyPasses = 8;
constexpr int kMaxCopies = kMaxPasses / kCopyPasses;
constexpr int kMaxHeads = 66;       // heads that a tile of 512 rows can touch (P >= 8)
constexpr int kMaxCluster = 16;
constexpr uint64_t kWaitLimitNs = 1000000000ull;

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_release() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_cluster_f32(float* local, uint32_t rank, float v) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(remote) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(remote), "f"(v) : "memory");
}

// One 32-bit word of activations: two bf16 channels or one fp32.
template <typename AT>
__device__ __forceinline__ void unpack_word(uint32_t u, float* out) {
    if constexpr (sizeof(AT) == 2) {
        out[0] = __uint_as_float(u << 16);
        out[1] = __uint_as_float(u & 0xFFFF0000u);
    } else {
        out[0] = __uint_as_float(u);
    }
}

// Byte offsets of the dynamic shared memory of a CTA.
struct Layout {
    int scale, conv_x, conv_bc, rp, y, B, C, raw_bc, bytes;
    __host__ __device__ Layout(int tile, int N, int K, int as) {
        scale = tile * N;                       // the old scales, later the new ones
        conv_x = scale + tile * 4;              // [K-1][tile]
        conv_bc = conv_x + (K - 1) * tile * as; // [2][K-1][N]
        rp = conv_bc + 2 * (K - 1) * N * as;    // per row {dt*x, scale*dA}
        y = rp + tile * 8;                      // D*x, later y
        B = y + tile * 4;
        C = B + N * 4;
        raw_bc = C + N * 4;                     // this step's raw B and C inputs
        bytes = raw_bc + 2 * N * as;
    }
};

// The sum (or largest) of two rows over their LPR lanes: lanes with the upper
// half bit end with row 1, the others with row 0.
template <int LPR, typename Op>
__device__ __forceinline__ float reduce_two(float v0, float v1, bool upper, Op op) {
    float v = op(upper ? v1 : v0, __shfl_xor_sync(0xffffffffu, upper ? v0 : v1, LPR / 2));
#pragma unroll
    for (int off = LPR / 4; off > 0; off >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// Where B and C of state n are kept: the 16 of a lane as four 16-byte vectors,
// vector q of all lanes side by side (no bank conflicts).
template <int LPR>
__device__ __forceinline__ int bc_place(int n) {
    return ((n / 4 % 4) * LPR + n / 16) * 4 + n % 4;
}

template <typename AT, int N, bool NORM>
__global__ void __launch_bounds__(kThreads, kMinBlocks) q8_update_kernel(const Q8UpdateArgs a) {
    constexpr int LPR = N / 16;
    constexpr int RPP = kThreads / LPR;              // rows a CTA covers once
    constexpr int PASS = RPP * kRowsPerThread;       // rows of one pass
    constexpr int CW = 4 / sizeof(AT);               // channels per 32-bit word
    constexpr int AS = sizeof(AT);
    constexpr int kPre = (kTileRows + 2 * N) / CW >= 3 * kThreads ? 3 : ((kTileRows + 2 * N) / CW >= 2 * kThreads ? 2 : 1);

    extern __shared__ __align__(128) uint8_t s_dyn[];
    __shared__ __align__(8) uint64_t s_bar[kMaxCopies + 1];
    __shared__ float s_dt[kMaxHeads], s_dA[kMaxHeads], s_D[kMaxHeads];
    __shared__ int s_fail;
    __shared__ float s_red[kWarps], s_parts[kMaxCluster], s_rstd;

    const int tid = threadIdx.x;
    const int K = a.K, P = a.P;
    const int64_t HP = static_cast<int64_t>(a.H) * P;
    const int group_rows = a.group_rows;
    const int g = blockIdx.y;
    const int off = blockIdx.x * a.tile_rows;              // first row within the group
    const int nrows = min(a.tile_rows, group_rows - off);  // a multiple of 8, at least 8
    const int64_t r0 = static_cast<int64_t>(g) * group_rows + off;
    // rows to heads: v / P for v < 2^13 by the host's reciprocal 2^22 / P
    auto head_of = [&](uint32_t v) -> int { return static_cast<int>((v * a.inv_P) >> 22); };
    const int h_in_group = head_of(off);
    const int h_first = g * a.hpg + h_in_group;
    const int rr0 = off - h_in_group * P;
    const int n_heads = head_of(rr0 + nrows - 1) + 1;
    const int64_t cd = a.conv_dim;
    const int64_t cB = HP + static_cast<int64_t>(g) * N;
    const int64_t cC = cB + static_cast<int64_t>(a.G) * N;
    const Layout L(a.tile_rows, N, K, AS);
    const uint8_t* s_codes = s_dyn;
    float* s_scale = reinterpret_cast<float*>(s_dyn + L.scale);
    const AT* s_cx = reinterpret_cast<const AT*>(s_dyn + L.conv_x);
    const AT* s_cbc = reinterpret_cast<const AT*>(s_dyn + L.conv_bc);
    float2* s_rp = reinterpret_cast<float2*>(s_dyn + L.rp);
    float* s_y = reinterpret_cast<float*>(s_dyn + L.y);
    float* s_B = reinterpret_cast<float*>(s_dyn + L.B);
    float* s_C = reinterpret_cast<float*>(s_dyn + L.C);
    uint32_t* s_rawbc = reinterpret_cast<uint32_t*>(s_dyn + L.raw_bc);

    constexpr int COPY = PASS * kCopyPasses;  // rows of one copy
    const int passes = (nrows + PASS - 1) / PASS;
    const int copies = (nrows + COPY - 1) / COPY;
    uint64_t* bar_conv = &s_bar[kMaxCopies];
    if (tid == 0) {
        s_fail = 0;
        for (int c = 0; c < copies; ++c) mbar_init(&s_bar[c], 1);
        mbar_init(bar_conv, 1);
        fence_mbar_init();
    }
    __syncthreads();

    // A programmatic dependent of the previous kernel: nothing is read before.
    asm volatile("griddepcontrol.wait;\n" ::: "memory");

    const int64_t b = blockIdx.z;
    const AT* xrow = static_cast<const AT*>(a.xBC) + b * a.xBC_stride;
    const AT* zrow = a.z ? static_cast<const AT*>(a.z) + b * a.z_stride : nullptr;
    AT* yrow = static_cast<AT*>(a.y) + b * a.y_stride;
    // ---- what does not depend on the slot is loaded before the slot is read:
    // its latency hides behind the slot's and the copies'
    const int n_words = (nrows + 2 * N) / CW;  // conv words: x of the tile, then B and C
    const int nx = nrows / CW;
    const AT* w = static_cast<const AT*>(a.conv_w);
    const AT* bias = static_cast<const AT*>(a.conv_b);
    auto word_channel = [&](int q) -> int64_t {
        if (q < nx) return r0 + q * CW;
        const int j = (q - nx) * CW;
        return j < N ? cB + j : cC + (j - N);
    };
    uint32_t raw_in[kPre], bias_in[kPre];
    uint4 w_in[kPre];
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
        const int q = i * kThreads + tid;
        raw_in[i] = bias_in[i] = 0;
        w_in[i] = make_uint4(0, 0, 0, 0);
        if (q < n_words) {
            const int64_t c0 = word_channel(q);
            raw_in[i] = *reinterpret_cast<const uint32_t*>(xrow + c0);
            if (bias) bias_in[i] = __ldg(reinterpret_cast<const uint32_t*>(bias + c0));
            if (K == 4) w_in[i] = __ldg(reinterpret_cast<const uint4*>(w + c0 * 4));
        }
    }
    float hs_dt = 0.f, hs_bias = 0.f, hs_alog = 0.f, hs_D = 0.f;
    if (tid < n_heads) {
        hs_dt = to_f32(static_cast<const AT*>(a.dt)[b * a.dt_stride + h_first + tid]);
        hs_bias = a.dt_bias[h_first + tid];
        hs_alog = a.A_log[h_first + tid];
        hs_D = a.D[h_first + tid];
    }
    const int32_t slot = a.slot_idx[b];
    // skipped rows are skipped by the whole cluster
    if (slot < 0) {
        for (int i = tid; i < nrows; i += kThreads) yrow[r0 + i] = from_f32<AT>(0.f);
        return;
    }
    if (slot >= a.num_slots) {
        if (tid == 0) record_error(a.error, M2_ERR_BAD_SLOT);
        return;
    }
    const int64_t row_base = static_cast<int64_t>(slot) * HP + r0;
    int8_t* tile = a.ssm + row_base * N;
    float* scales = a.scale + row_base;
    AT* conv0 = static_cast<AT*>(a.conv) + static_cast<int64_t>(slot) * (K - 1) * cd;
    if (tid == 0) {
        mbar_arrive_expect_tx(bar_conv, static_cast<uint32_t>((K - 1) * (nrows + 2 * N) * AS + nrows * 4));
        bulk_g2s(s_dyn + L.scale, scales, nrows * 4, bar_conv);
        for (int k = 0; k < K - 1; ++k) {
            bulk_g2s(s_dyn + L.conv_x + k * a.tile_rows * AS, conv0 + k * cd + r0, nrows * AS, bar_conv);
            bulk_g2s(s_dyn + L.conv_bc + k * N * AS, conv0 + k * cd + cB, N * AS, bar_conv);
            bulk_g2s(s_dyn + L.conv_bc + (K - 1 + k) * N * AS, conv0 + k * cd + cC, N * AS, bar_conv);
        }
        for (int c = 0; c < copies; ++c) {
            const int rows = min(COPY, nrows - c * COPY);
            mbar_arrive_expect_tx(&s_bar[c], rows * N);
            bulk_g2s(s_dyn + c * COPY * N, tile + static_cast<int64_t>(c) * COPY * N, rows * N, &s_bar[c]);
        }
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid < n_heads) {
        const float dt = softplus_f32(hs_dt + hs_bias);
        s_dt[tid] = dt;
        s_dA[tid] = expf(dt * -expf(hs_alog));
        s_D[tid] = hs_D;
    }
    __syncthreads();

    // ---- conv: one word of channels at a time, x of the tile, then B and C
    {
        auto conv_word = [&](int q, uint32_t raw, uint32_t bias_w, uint4 wv) {
            const bool is_x = q < nx;
            const int j = is_x ? q * CW : (q - nx) * CW;  // channel within the segment(s)
            const int seg = j >= N ? 1 : 0;               // (B, C) 0 or 1
            const int64_t c0 = word_channel(q);
            const AT* rows = is_x ? s_cx + j : s_cbc + seg * (K - 1) * N + (j - seg * N);
            const int pitch = is_x ? a.tile_rows : N;
            float out[CW];
            unpack_word<AT>(bias_w, out);
            if (K == 4) {  // the CW x 4 weights are one 16-byte vector
                float w4[Vec16<AT>::n], xv[CW];
                unpack16<AT>(wv, w4);
                unpack_word<AT>(raw, xv);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    float rv[CW];
                    unpack_word<AT>(*reinterpret_cast<const uint32_t*>(rows + k * pitch), rv);
#pragma unroll
                    for (int e = 0; e < CW; ++e) out[e] = fmaf(w4[e * 4 + k], rv[e], out[e]);
                }
#pragma unroll
                for (int e = 0; e < CW; ++e) out[e] = fmaf(w4[e * 4 + 3], xv[e], out[e]);
            } else {
                for (int k = 0; k < K; ++k) {
                    float rv[CW];
                    unpack_word<AT>(k < K - 1 ? *reinterpret_cast<const uint32_t*>(rows + k * pitch) : raw, rv);
#pragma unroll
                    for (int e = 0; e < CW; ++e) out[e] = fmaf(to_f32(__ldg(w + (c0 + e) * K + k)), rv[e], out[e]);
                }
            }
            if (a.activation) {
#pragma unroll
                for (int e = 0; e < CW; ++e) out[e] = silu_f32(out[e]);
            }
            if (is_x) {
                for (int k = 0; k < K - 1; ++k)  // roll this CTA's own conv rows
                    *reinterpret_cast<uint32_t*>(conv0 + k * cd + c0) =
                        k < K - 2 ? *reinterpret_cast<const uint32_t*>(rows + (k + 1) * pitch) : raw;
                const int hl = head_of(rr0 + j);  // CW channels lie in one head
                const float dtv = s_dt[hl], dAv = s_dA[hl], Dv = s_D[hl];
#pragma unroll
                for (int e = 0; e < CW; ++e) {
                    s_rp[j + e] = make_float2(dtv * out[e], s_scale[j + e] * dAv);
                    s_y[j + e] = Dv * out[e];
                }
            } else {
                float* dst = (seg ? s_C : s_B) + bc_place<LPR>(j - seg * N);
#pragma unroll
                for (int e = 0; e < CW; ++e) dst[e] = out[e];
                s_rawbc[j / CW] = raw;
            }
        };
        if (mbar_wait_bounded(bar_conv, 0, kWaitLimitNs)) {
#pragma unroll
            for (int i = 0; i < kPre; ++i) {
                const int q = i * kThreads + tid;
                if (q < n_words) conv_word(q, raw_in[i], bias_in[i], w_in[i]);
            }
            for (int q = kPre * kThreads + tid; q < n_words; q += kThreads) {
                const int64_t c0 = word_channel(q);
                conv_word(q, *reinterpret_cast<const uint32_t*>(xrow + c0),
                          bias ? __ldg(reinterpret_cast<const uint32_t*>(bias + c0)) : 0u,
                          K == 4 ? __ldg(reinterpret_cast<const uint4*>(w + c0 * 4)) : make_uint4(0, 0, 0, 0));
            }
        } else {
            record_error(a.error, M2_ERR_TIMEOUT);
            s_fail = 1;
        }
        cluster_arrive_relaxed();  // this CTA has read the group's B/C conv rows
    }
    __syncthreads();
    bool ok = s_fail == 0;

    // ---- the state, two rows a thread at a time
    const int lane = tid & 31;
    const int l = lane % LPR;
    const bool upper = (lane & (LPR / 2)) != 0;
    float2 B2[8], C2[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float4 vb = *reinterpret_cast<const float4*>(s_B + (q * LPR + l) * 4);
        const float4 vc = *reinterpret_cast<const float4*>(s_C + (q * LPR + l) * 4);
        B2[2 * q] = make_float2(vb.x, vb.y);
        B2[2 * q + 1] = make_float2(vb.z, vb.w);
        C2[2 * q] = make_float2(vc.x, vc.y);
        C2[2 * q + 1] = make_float2(vc.z, vc.w);
    }
    // row (c * 2 + i) * RPP + tid / LPR of the tile is codes ((c * 2 + i) * kThreads + tid) * 16 .. + 15
    const float2* rps = s_rp + tid / LPR;
    const uint8_t* codes = s_codes + tid * 16;
    int8_t* out = tile + tid * 16;
    const int end = nrows * N - tid * 16;  // codes of this thread's rows that exist lie below
#pragma unroll 1
    for (int c = 0; c < passes; ++c) {
        if (c % kCopyPasses == 0 && !mbar_wait_bounded(&s_bar[c / kCopyPasses], 0, kWaitLimitNs)) {
            record_error(a.error, M2_ERR_TIMEOUT);
            ok = false;
            break;
        }
        float2 S[kRowsPerThread][8];
        float sum[kRowsPerThread], big[kRowsPerThread];
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const float2 rp = rps[(c * kRowsPerThread + i) * RPP];
            const uint4 w = *reinterpret_cast<const uint4*>(codes + (c * kRowsPerThread + i) * (kThreads * 16));
            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
            const float2 dtx = make_float2(rp.x, rp.x), k2 = make_float2(rp.y, rp.y);
            float2 acc;
            float m = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 lo, hi;
                q8_unpack(words[q], lo, hi);
                lo = __ffma2_rn(lo, k2, __fmul2_rn(dtx, B2[2 * q]));
                hi = __ffma2_rn(hi, k2, __fmul2_rn(dtx, B2[2 * q + 1]));
                acc = q == 0 ? __fmul2_rn(lo, C2[0]) : __ffma2_rn(lo, C2[2 * q], acc);
                acc = __ffma2_rn(hi, C2[2 * q + 1], acc);
                m = max_abs(m, lo.x, lo.y);
                m = max_abs(m, hi.x, hi.y);
                S[i][2 * q] = lo;
                S[i][2 * q + 1] = hi;
            }
            sum[i] = acc.x + acc.y;
            big[i] = m;
        }
        const float ysum = reduce_two<LPR>(sum[0], sum[1], upper, [](float u, float v) { return u + v; });
        const float amax = reduce_two<LPR>(big[0], big[1], upper, [](float u, float v) { return max_nan(u, v); });
        float scale, inv;
        q8_scale_fast(amax, scale, inv);
        if (l % (LPR / 2) == 0) {
            const int row = (c * kRowsPerThread + (upper ? 1 : 0)) * RPP + tid / LPR;  // < tile_rows
            s_y[row] += ysum;
            s_scale[row] = scale;
        }
        float inv_of[kRowsPerThread];
        inv_of[0] = __shfl_sync(0xffffffffu, inv, lane & ~(LPR / 2));
        inv_of[1] = __shfl_sync(0xffffffffu, inv, lane | (LPR / 2));
#pragma unroll
        for (int i = 0; i < kRowsPerThread; ++i) {
            const float2 iv = make_float2(inv_of[i], inv_of[i]), mg = make_float2(kQ8Magic, kQ8Magic);
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float2 lo = __ffma2_rn(S[i][2 * q], iv, mg), hi = __ffma2_rn(S[i][2 * q + 1], iv, mg);
                o[q] = q8_pack(lo.x, lo.y, hi.x, hi.y);
            }
            const int at = (c * kRowsPerThread + i) * (kThreads * 16);
            if (at < end) st_stream(out + at, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    if (!ok) {  // let this CTA's copies land before its shared memory goes
        for (int c = 0; c < copies; ++c) mbar_wait_bounded(&s_bar[c], 0, kWaitLimitNs);
        mbar_wait_bounded(bar_conv, 0, kWaitLimitNs);
    }
    __syncthreads();

    if (ok) {
        for (int i = tid; i < nrows; i += kThreads) scales[i] = s_scale[i];
    }
    if constexpr (!NORM) {
        if (ok) {
            for (int i = tid; i < nrows; i += kThreads) {
                float yv = s_y[i];
                if (zrow) yv *= silu_f32(to_f32(zrow[r0 + i]));
                yrow[r0 + i] = from_f32<AT>(yv);
            }
        }
    } else {
        // gated RMSNorm over the group's rows, which are this cluster's
        float ss = 0.f;
        if (ok) {
            for (int i = tid; i < nrows; i += kThreads) {
                float yv = s_y[i];
                if (zrow) yv *= silu_f32(to_f32(zrow[r0 + i]));
                s_y[i] = yv;
                ss = fmaf(yv, yv, ss);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) s_red[tid >> 5] = ss;
        __syncthreads();
        cluster_wait();  // the phase of the conv's arrive: every CTA is running
        if (tid < a.group_ctas) {
            float part = 0.f;
            for (int w = 0; w < kWarps; ++w) part += s_red[w];
            st_cluster_f32(&s_parts[cluster_rank()], static_cast<uint32_t>(tid), part);
        }
        cluster_arrive_release();
        cluster_wait();
        if (tid == 0) {
            float total = 0.f;
            for (int q = 0; q < a.group_ctas; ++q) total += s_parts[q];
            s_rstd = rsqrtf(total / static_cast<float>(group_rows) + a.norm_eps);
        }
        __syncthreads();
        if (ok) {
            const AT* nw = static_cast<const AT*>(a.norm_w);
            for (int i = tid; i < nrows; i += kThreads)
                yrow[r0 + i] = from_f32<AT>(s_y[i] * s_rstd * to_f32(nw[r0 + i]));
        }
    }

    // ---- cluster rank 0 rolls the group's B and C conv rows
    if (!NORM && cluster_rank() == 0) cluster_wait();
    if (ok && cluster_rank() == 0) {
        for (int q = tid; q < 2 * N / CW; q += kThreads) {
            const int j = q * CW, seg = j / N;
            const int64_t c0 = (seg ? cC : cB) + (j - seg * N);
            const AT* rows = s_cbc + seg * (K - 1) * N + (j - seg * N);
            for (int k = 0; k < K - 1; ++k)
                *reinterpret_cast<uint32_t*>(conv0 + k * cd + c0) =
                    k < K - 2 ? *reinterpret_cast<const uint32_t*>(rows + (k + 1) * N) : s_rawbc[q];
        }
    }
}

template <typename AT, int N, bool NORM>
cudaError_t launch_one(const Q8UpdateArgs& a, cudaStream_t stream) {
    auto kern = q8_update_kernel<AT, N, NORM>;
    static AttrOnce attrs;
    const cudaError_t e = attrs.ensure([&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (r == cudaSuccess) r = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        return r;
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.group_ctas, a.G, a.batch);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Layout(a.tile_rows, N, a.K, sizeof(AT)).bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.group_ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename AT, int N>
cudaError_t by_norm(const Q8UpdateArgs& a, cudaStream_t s) {
    return a.norm_w ? launch_one<AT, N, true>(a, s) : launch_one<AT, N, false>(a, s);
}

template <typename AT>
cudaError_t by_n(const Q8UpdateArgs& a, cudaStream_t s) {
    switch (a.N) {
        case 64: return by_norm<AT, 64>(a, s);
        case 128: return by_norm<AT, 128>(a, s);
        case 256: return by_norm<AT, 256>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

// Rows of one pass and the largest tile of a CTA.
int pass_rows(int N) { return kThreads / (N / 16) * kRowsPerThread; }
int max_tile(int N) { return std::min(512, pass_rows(N) * kMaxPasses); }

}  // namespace

m2_status q8_shape_supported(int H, int P, int N, int G) {
    if (N != 64 && N != 128 && N != 256) return M2_ERR_UNSUPPORTED;
    if (P < 8 || P > 256 || P % 8 != 0) return M2_ERR_UNSUPPORTED;
    const int64_t group_rows = static_cast<int64_t>(H / G) * P;
    if (group_rows > static_cast<int64_t>(kMaxCluster) * max_tile(N)) return M2_ERR_UNSUPPORTED;
    return M2_OK;
}

cudaError_t launch_q8_update(Q8UpdateArgs a, cudaStream_t stream) {
    const int group_rows = a.H / a.G * a.P;
    int tile = std::min(kTileRows, max_tile(a.N));
    if (group_rows < tile) tile = (group_rows + pass_rows(a.N) - 1) / pass_rows(a.N) * pass_rows(a.N);
    while ((group_rows + tile - 1) / tile > kMaxCluster) tile *= 2;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    // few rows: halve the tiles as long as that brings idle SMs in and the
    // cluster stays portable (one Nemotron-H row: 6.2 us with 256 rows a tile, 4.9
    // with 128; five 7.2 and 6.2)
    while (tile % (2 * pass_rows(a.N)) == 0 && 2 * ((group_rows + tile - 1) / tile) <= 8 &&
           static_cast<int64_t>(a.G) * ((group_rows + tile - 1) / tile) * a.batch < 2 * sms)
        tile /= 2;
    a.group_rows = group_rows;
    a.hpg = a.H / a.G;
    a.inv_P = ((1u << 22) + a.P - 1) / a.P;
    a.tile_rows = tile;
    a.group_ctas = (group_rows + tile - 1) / tile;
    return a.act_bf16 ? by_n<bf16_t>(a, stream) : by_n<float>(a, stream);
}

}  // namespace m2
