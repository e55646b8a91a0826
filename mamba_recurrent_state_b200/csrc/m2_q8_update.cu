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
//  * One thread puts the tile's codes in flight as one bulk copy as soon as the
//    slot is known; the slot's conv rows and scales go to registers, four
//    channels a thread, the parameters before them (with the conv rows as bulk
//    copies too, one thread's nine more issues held up the codes: 35.9 us in
//    place of 33.1 for 64 Nemotron-H rows).
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
// Bound by instruction issue beside HBM: a warp takes 9.4 instructions for 32
// codes (5 for unpack, update, y, maximum, round and pack; a row's exchanges and
// a tile's conv and output the rest), for 64 Nemotron-H rows 18 us of the
// SMs' issue slots beside 23 us of HBM time, and a CTA's wait for its codes
// overlaps only with other CTAs' arithmetic. 64 rows 32.1 us (floor 23.2), 384 rows
// 165 us, 0.84 of the copy bandwidth; one row 3.4 us. With the norm 38.0 and 209 us:
// two more cluster phases, and a CTA's tile waits for its group's. fp32 activations
// 37.7 us for 64 rows (floor 25.0). K != 4 takes its taps one by one: K = 3 37.0 us
// (22.8), K = 8 53.8 us (24.8).
#include <cuda_runtime.h>

#include <algorithm>

#include "m2_q8.cuh"

namespace m2 {
namespace {

// Threads of a CTA, codes of its tile, the resident CTAs per SM that the
// registers are sized for (five do reside: 96 registers, 40 KB), passes over the
// tile that one copy brings. 64 Nemotron-H rows (23.2 us at the copy bandwidth):
// 128, 256 rows, 4, 8 passes 32.0 us; sized for five CTAs 34.7 (fewer registers, more
// instructions); four passes a copy 32.9; tiles of 128 rows 36.7, of 512 45.2;
// 256 threads with 512 rows 38.1, 64 threads with 128 38.8 us. A persistent CTA
// with two rings, the next row's copies under this one's arithmetic, took half
// as long again. Rows of 64 codes: 512 a tile 70.0 us for 256 rows of 128 heads,
// 256 74.6; of 256 codes: 128 a tile 240 us, 256 255 us.
constexpr int kThreads = 128;
constexpr int kTileCodes = 32768;
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

// Four channels of activations as one vector.
template <typename AT>
struct Quad;
template <>
struct Quad<bf16_t> {
    using T = uint2;
    __device__ static __forceinline__ float4 unpack(uint2 u) {
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                           __uint_as_float(u.y & 0xFFFF0000u));
    }
    __device__ static __forceinline__ uint2 pack(float4 v) { return make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)); }
};
template <>
struct Quad<float> {
    using T = float4;
    __device__ static __forceinline__ float4 unpack(float4 v) { return v; }
    __device__ static __forceinline__ float4 pack(float4 v) { return v; }
};

// Byte offsets of the dynamic shared memory of a CTA.
struct Layout {
    int scale, roll, rp, y, B, C, bytes;
    __host__ __device__ Layout(int tile, int N, int K, int as) {
        scale = tile * N;                // the new scales
        rp = scale + tile * 4;           // per row {dt*x, scale*dA}
        y = rp + tile * 8;               // D*x, later y
        B = y + tile * 4;
        C = B + N * 4;
        roll = C + N * 4;                // [K-1][2][N]: the group's rolled B and C conv rows (cluster rank 0)
        bytes = roll + 2 * (K - 1) * N * as;
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
    constexpr int AS = sizeof(AT);
    using Q = Quad<AT>;
    using V4 = typename Q::T;

    extern __shared__ __align__(128) uint8_t s_dyn[];
    __shared__ __align__(8) uint64_t s_bar[kMaxCopies];
    __shared__ float s_dt[kMaxHeads], s_dA[kMaxHeads], s_D[kMaxHeads];
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
    float2* s_rp = reinterpret_cast<float2*>(s_dyn + L.rp);
    float* s_y = reinterpret_cast<float*>(s_dyn + L.y);
    float* s_B = reinterpret_cast<float*>(s_dyn + L.B);
    float* s_C = reinterpret_cast<float*>(s_dyn + L.C);
    V4* s_roll = reinterpret_cast<V4*>(s_dyn + L.roll);

    constexpr int COPY = PASS * kCopyPasses;  // rows of one copy
    const int passes = (nrows + PASS - 1) / PASS;
    const int copies = (nrows + COPY - 1) / COPY;
    if (tid == 0) {
        for (int c = 0; c < copies; ++c) mbar_init(&s_bar[c], 1);
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
    // its latency hides behind the slot's and the codes'. A thread's first four
    // conv channels (of the tile's x, then the group's B and C):
    const int nx = nrows / 4, n_quads = nx + N / 2;
    const AT* w = static_cast<const AT*>(a.conv_w);
    const AT* bias = static_cast<const AT*>(a.conv_b);
    auto quad_channel = [&](int q) -> int {
        const int j = (q - nx) * 4;
        return static_cast<int>(q < nx ? r0 + q * 4 : (j < N ? cB + j : cC + (j - N)));
    };
    auto quad_of = [](const AT* p) -> V4 { return *reinterpret_cast<const V4*>(p); };
    struct Taps {
        uint4 v[AS];  // 4 channels x 4 taps
    };
    auto taps_of = [&](int c0) {
        Taps t;
#pragma unroll
        for (int i = 0; i < AS; ++i) t.v[i] = __ldg(reinterpret_cast<const uint4*>(w + static_cast<int64_t>(c0) * 4) + i);
        return t;
    };
    const int c_first = quad_channel(tid);
    const bool q_first = tid < n_quads;
    V4 raw_in{}, bias_in{}, z_in{}, old_in[3]{};
    Taps w_in{};
    float4 scale_in = make_float4(0.f, 0.f, 0.f, 0.f);
    if (q_first) {
        raw_in = quad_of(xrow + c_first);
        if (bias) bias_in = quad_of(bias + c_first);
        if (K == 4) w_in = taps_of(c_first);
        if (zrow && tid < nx) z_in = quad_of(zrow + c_first);
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
        for (int c = 0; c < copies; ++c) {
            const int rows = min(COPY, nrows - c * COPY);
            mbar_arrive_expect_tx(&s_bar[c], rows * N);
            bulk_g2s(s_dyn + c * COPY * N, tile + static_cast<int64_t>(c) * COPY * N, rows * N, &s_bar[c]);
        }
    }
    auto old_quad = [&](int k, int c) -> V4 { return quad_of(conv0 + k * cd + c); };
    if (q_first) {
        if (K == 4) {
#pragma unroll
            for (int k = 0; k < 3; ++k) old_in[k] = old_quad(k, c_first);
        }
        if (tid < nx) scale_in = *reinterpret_cast<const float4*>(scales + tid * 4);
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (tid < n_heads) {
        const float dt = softplus_f32(hs_dt + hs_bias);
        s_dt[tid] = dt;
        s_dA[tid] = expf(dt * -expf(hs_alog));
        s_D[tid] = hs_D;
    }
    __syncthreads();

    // ---- conv: four channels at a time, x of the tile, then B and C
    {
        auto conv_quad = [&](int q, int c0, V4 raw, V4 bias_v, const Taps& taps, const V4 (&old)[3], float4 sc) {
            const bool is_x = q < nx;
            const int j = is_x ? q * 4 : (q - nx) * 4;  // channel within x, or within (B, C)
            const float4 b4 = Q::unpack(bias_v);
            float2 out01 = make_float2(b4.x, b4.y), out23 = make_float2(b4.z, b4.w);
            auto tap = [&](V4 row, const float (&wk)[4]) {
                const float4 r = Q::unpack(row);
                out01 = __ffma2_rn(make_float2(wk[0], wk[1]), make_float2(r.x, r.y), out01);
                out23 = __ffma2_rn(make_float2(wk[2], wk[3]), make_float2(r.z, r.w), out23);
            };
            if (K == 4) {
                float f[16];
#pragma unroll
                for (int i = 0; i < AS; ++i) unpack16<AT>(taps.v[i], f + i * Vec16<AT>::n);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float wk[4] = {f[k], f[4 + k], f[8 + k], f[12 + k]};
                    tap(k < 3 ? old[k] : raw, wk);
                }
            } else {
                const AT* wc = w + static_cast<int64_t>(c0) * K;
                for (int k = 0; k < K; ++k) {
                    const float wk[4] = {to_f32(__ldg(wc + k)), to_f32(__ldg(wc + K + k)), to_f32(__ldg(wc + 2 * K + k)),
                                         to_f32(__ldg(wc + 3 * K + k))};
                    tap(k < K - 1 ? old_quad(k, c0) : raw, wk);
                }
            }
            if (a.activation) {
                out01 = silu2_f32(out01);
                out23 = silu2_f32(out23);
            }
            // the rolled conv rows: this CTA's own into the cache, the group's aside for the end
            auto roll_into = [&](V4* row, int64_t pitch) {
                if (K == 4) {
                    row[0] = old[1];
                    row[pitch] = old[2];
                    row[2 * pitch] = raw;
                } else {
                    for (int k = 0; k < K - 1; ++k) row[k * pitch] = k < K - 2 ? old_quad(k + 1, c0) : raw;
                }
            };
            if (is_x) {
                roll_into(reinterpret_cast<V4*>(conv0 + c0), cd / 4);
                const int hl = head_of(rr0 + j);  // 4 channels lie in one head
                const float2 dtv = make_float2(s_dt[hl], s_dt[hl]), Dv = make_float2(s_D[hl], s_D[hl]);
                const float dAv = s_dA[hl];
                const float2 u01 = __fmul2_rn(dtv, out01), u23 = __fmul2_rn(dtv, out23);
                float4* rp = reinterpret_cast<float4*>(s_rp + j);
                rp[0] = make_float4(u01.x, sc.x * dAv, u01.y, sc.y * dAv);
                rp[1] = make_float4(u23.x, sc.z * dAv, u23.y, sc.w * dAv);
                const float2 y01 = __fmul2_rn(Dv, out01), y23 = __fmul2_rn(Dv, out23);
                *reinterpret_cast<float4*>(s_y + j) = make_float4(y01.x, y01.y, y23.x, y23.y);
            } else {
                float* dst = j < N ? s_B + bc_place<LPR>(j) : s_C + bc_place<LPR>(j - N);
                *reinterpret_cast<float4*>(dst) = make_float4(out01.x, out01.y, out23.x, out23.y);
                if (cluster_rank() == 0) roll_into(s_roll + j / 4, N / 2);
            }
        };
        if (q_first) conv_quad(tid, c_first, raw_in, bias_in, w_in, old_in, scale_in);
        for (int q = kThreads + tid; q < n_quads; q += kThreads) {
            const int c0 = quad_channel(q);
            V4 old[3]{};
            if (K == 4) {
#pragma unroll
                for (int k = 0; k < 3; ++k) old[k] = old_quad(k, c0);
            }
            conv_quad(q, c0, quad_of(xrow + c0), bias ? quad_of(bias + c0) : V4{}, K == 4 ? taps_of(c0) : Taps{}, old,
                      q < nx ? *reinterpret_cast<const float4*>(scales + q * 4) : make_float4(0.f, 0.f, 0.f, 0.f));
        }
    }
    __syncthreads();
    // This CTA has read the group's B/C conv rows: what it computed from them lies in
    // shared memory behind the barrier above. (A release would wait for the
    // conv rows just stored, too: 41.4 us in place of 34.9 for 64 rows.)
    cluster_arrive_relaxed();
    bool ok = true;

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
    for (int first = 0; first < passes; first += kCopyPasses) {
        if (!mbar_wait_bounded(&s_bar[first / kCopyPasses], 0, kWaitLimitNs)) {
            record_error(a.error, M2_ERR_TIMEOUT);
            ok = false;
            break;
        }
#pragma unroll 1
        for (int c = first; c < min(first + kCopyPasses, passes); ++c) {
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
    }
    if (!ok) {  // let this CTA's copies land before its shared memory goes
        for (int c = 0; c < copies; ++c) mbar_wait_bounded(&s_bar[c], 0, kWaitLimitNs);
    }
    __syncthreads();

    if (ok) {  // by the threads that have fewer rows of y
        for (int i = kThreads - 1 - tid; i < nx; i += kThreads)
            reinterpret_cast<float4*>(scales)[i] = reinterpret_cast<const float4*>(s_scale)[i];
    }
    // four rows' gated y
    auto gated = [&](int q) -> float4 {
        float4 v = reinterpret_cast<const float4*>(s_y)[q];
        if (zrow) {
            const float4 z4 = Q::unpack(q == tid ? z_in : quad_of(zrow + r0 + q * 4));
            const float2 g01 = silu2_f32(make_float2(z4.x, z4.y)), g23 = silu2_f32(make_float2(z4.z, z4.w));
            v = make_float4(v.x * g01.x, v.y * g01.y, v.z * g23.x, v.w * g23.y);
        }
        return v;
    };
    if constexpr (!NORM) {
        if (ok) {
            for (int q = tid; q < nx; q += kThreads) reinterpret_cast<V4*>(yrow + r0)[q] = Q::pack(gated(q));
        }
    } else {
        // gated RMSNorm over the group's rows, which are this cluster's
        float ss = 0.f;
        if (ok) {
            for (int q = tid; q < nx; q += kThreads) {
                const float4 v = gated(q);
                reinterpret_cast<float4*>(s_y)[q] = v;
                ss += (v.x * v.x + v.y * v.y) + (v.z * v.z + v.w * v.w);
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
        for (int q = tid; q < N / 2; q += kThreads) {
            V4* row = reinterpret_cast<V4*>(conv0 + quad_channel(nx + q));
            for (int k = 0; k < K - 1; ++k) row[k * (cd / 4)] = s_roll[k * (N / 2) + q];
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
    int tile = std::min(kTileCodes / a.N, max_tile(a.N));
    if (group_rows < tile) tile = (group_rows + pass_rows(a.N) - 1) / pass_rows(a.N) * pass_rows(a.N);
    while ((group_rows + tile - 1) / tile > kMaxCluster) tile *= 2;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 148;
    // few rows: halve the tiles as long as that brings idle SMs in, to clusters of
    // 8 up to three CTAs an SM (Nemotron-H, 256 rows a tile and 128: one row 4.9
    // and 3.9 us, five 6.2 and 5.4, twelve 11.5 and 10.6, sixteen 12.5 and 12.9),
    // to clusters of 16 up to one (64 heads of 64 x 64 in one group, clusters
    // of 8 and 16: one row 6.2 and 4.2 us, sixteen 7.0 and 5.6; 128 heads in eight
    // groups, where 8 make 256 CTAs: four rows 4.2 and 4.9)
    for (;;) {
        const int ctas = (group_rows + tile - 1) / tile;
        const int64_t all = static_cast<int64_t>(a.G) * ctas * a.batch;
        if (tile % (2 * pass_rows(a.N)) != 0 || 2 * ctas > kMaxCluster || all >= (2 * ctas <= 8 ? 3 : 1) * sms) break;
        tile /= 2;
    }
    a.group_rows = group_rows;
    a.hpg = a.H / a.G;
    a.inv_P = ((1u << 22) + a.P - 1) / a.P;
    a.tile_rows = tile;
    a.group_ctas = (group_rows + tile - 1) / tile;
    return a.act_bf16 ? by_n<bf16_t>(a, stream) : by_n<float>(a, stream);
}

}  // namespace m2
