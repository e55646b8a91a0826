// m2_api_sel.cu -- the C entry points of the per-channel selective scan
// (include/m2.h). Host-side only: argument validation and error mapping.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "m2_host.cuh"
#include "m2_sel.cuh"

using namespace m2::host;

namespace {

// The kernels number a sequence's tokens in 32 bits and step past the last one:
// the conv by up to three strides of its grid, 3 * 65535 * 32 tokens, the scan by
// a tile. Calls stay below 2^31 by more than that.
constexpr int64_t kMaxTokens = (int64_t{1} << 31) - (int64_t{1} << 24);

m2_status sel_shape_status(const m2_sel_shape* s) {
    if (!s) return M2_ERR_INVALID_ARG;
    if (s->channels <= 0 || s->d_state <= 0 || s->ngroups <= 0 || s->d_conv <= 0) return M2_ERR_INVALID_ARG;
    if (s->channels % s->ngroups != 0) return M2_ERR_INVALID_ARG;
    if (!valid_dtype(s->state_dtype) || !valid_dtype(s->act_dtype)) return M2_ERR_INVALID_ARG;
    if (s->d_conv < 2 || s->d_conv > 8 || !m2::sel_state_size_supported(s->d_state)) return M2_ERR_UNSUPPORTED;
    // a group's channels are taken in whole 16-byte vectors
    if (static_cast<int64_t>(s->channels / s->ngroups) * dsize(s->act_dtype) % 16 != 0) return M2_ERR_UNSUPPORTED;
    // groups in a grid dimension, channel and group offsets of a row in 32 bits
    if (s->ngroups > 65535 || s->channels > (1 << 24) || static_cast<int64_t>(s->ngroups) * s->d_state > (1 << 24)) return M2_ERR_UNSUPPORTED;
    return M2_OK;
}

m2_status sel_status(const m2_sel_cache* c) {
    if (!c || !c->ssm || !c->conv || c->num_slots <= 0) return M2_ERR_INVALID_ARG;
    return sel_shape_status(&c->shape);
}

m2_status conv_impl(const m2_sel_cache* c, const m2_conv_params* conv, int32_t batch, int32_t seqlen,
                    const int32_t* cu_seqlens, int64_t total_rows, const void* x, int64_t x_row_stride, void* x_out,
                    int32_t out_dtype, int64_t out_row_stride, const int32_t* slot_idx, m2_stream stream) {
    const m2_status st = sel_status(c);
    if (st != M2_OK) return st;
    if (!conv || !conv->weight || batch < 0 || seqlen < 0 || !valid_buffer_dtype(out_dtype)) return M2_ERR_INVALID_ARG;
    if (conv->activation != 0 && conv->activation != 1) return M2_ERR_INVALID_ARG;
    if (batch == 0 || seqlen == 0) return M2_OK;
    if (!x || !x_out || !slot_idx) return M2_ERR_INVALID_ARG;
    const m2_sel_shape& s = c->shape;
    if (!aligned16(x) || !aligned16(x_out) || !stride_ok(x_row_stride, dsize(s.act_dtype), s.channels) ||
        !stride_ok(out_row_stride, dsize(out_dtype), s.channels) || !aligned16(conv->weight) ||
        (conv->bias && !aligned16(conv->bias)))
        return M2_ERR_INVALID_ARG;
    if (batch > 65535) return M2_ERR_UNSUPPORTED;
    if (!on_current_device(c->device)) return M2_ERR_INVALID_ARG;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (validate_mode()) {
        const m2_status v = validate_slots(slot_idx, batch, c->num_slots, cs);
        if (v != M2_OK) return v;
    }
    m2::ConvArgs a{};
    a.conv = c->conv;
    a.error = c->error;
    a.num_slots = c->num_slots;
    a.K = s.d_conv;
    a.conv_dim = s.channels;
    a.act_bf16 = s.act_dtype == M2_BF16;
    a.out_dtype = out_dtype;
    a.w = conv->weight;
    a.b = conv->bias;
    a.activation = conv->activation;
    a.batch = batch;
    a.seqlen = seqlen;
    a.x = x;
    a.x_stride = x_row_stride;
    a.out = x_out;
    a.out_stride = out_row_stride;
    a.slot_idx = slot_idx;
    a.cu_seqlens = cu_seqlens;
    a.total_rows = total_rows;
    return from_cuda(m2::launch_conv1d_update(a, cs));
}

// What the scan and the one-token step check alike, and their kernel arguments.
m2_status sel_args(const m2_sel_cache* c, const m2_sel_params* p, int32_t nseq, const void* x, int64_t x_row_stride,
                   const void* dt, int64_t dt_row_stride, const void* B, int64_t B_row_stride, const void* C,
                   int64_t C_row_stride, const void* z, int64_t z_row_stride, void* y, int64_t y_row_stride,
                   const int32_t* slot_idx, m2_stream stream, m2::SelArgs* out) {
    if (!x || !dt || !B || !C || !y || !slot_idx) return M2_ERR_INVALID_ARG;
    const m2_sel_shape& s = c->shape;
    const int as = dsize(s.act_dtype);
    const int64_t gn = static_cast<int64_t>(s.ngroups) * s.d_state;
    if (!aligned16(p->A_log)) return M2_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(dt) || !aligned16(B) || !aligned16(C) || !aligned16(y) ||
        !stride_ok(x_row_stride, as, s.channels) || !stride_ok(dt_row_stride, as, s.channels) ||
        !stride_ok(y_row_stride, as, s.channels) || !stride_ok(B_row_stride, as, gn) || !stride_ok(C_row_stride, as, gn))
        return M2_ERR_INVALID_ARG;
    if (z && (!aligned16(z) || !stride_ok(z_row_stride, as, s.channels))) return M2_ERR_INVALID_ARG;
    if (nseq > 65535) return M2_ERR_UNSUPPORTED;
    if (!on_current_device(c->device)) return M2_ERR_INVALID_ARG;
    if (validate_mode()) {
        const m2_status v = validate_slots(slot_idx, nseq, c->num_slots, reinterpret_cast<cudaStream_t>(stream));
        if (v != M2_OK) return v;
    }
    m2::SelArgs a{};
    a.ssm = c->ssm;
    a.error = c->error;
    a.num_slots = c->num_slots;
    a.D = s.channels;
    a.N = s.d_state;
    a.G = s.ngroups;
    a.state_bf16 = s.state_dtype == M2_BF16;
    a.act_bf16 = s.act_dtype == M2_BF16;
    a.A_log = p->A_log;
    a.dt_bias = p->dt_bias;
    a.skip = p->D;
    a.nseq = nseq;
    a.x = x;
    a.x_stride = x_row_stride;
    a.dt = dt;
    a.dt_stride = dt_row_stride;
    a.B = B;
    a.B_stride = B_row_stride;
    a.C = C;
    a.C_stride = C_row_stride;
    a.z = z;
    a.z_stride = z_row_stride;
    a.y = y;
    a.y_stride = y_row_stride;
    a.slot_idx = slot_idx;
    *out = a;
    return M2_OK;
}

bool params_ok(const m2_sel_params* p) { return p && p->A_log && p->dt_bias && p->D; }

}  // namespace

extern "C" {

m2_status m2_sel_shape_check(const m2_sel_shape* s) { return sel_shape_status(s); }

m2_status m2_sel_cache_bytes(const m2_sel_shape* s, int64_t num_slots, int64_t* ssm_bytes, int64_t* conv_bytes) {
    const m2_status st = sel_shape_status(s);
    if (st != M2_OK) return st;
    if (num_slots <= 0) return M2_ERR_INVALID_ARG;
    if (ssm_bytes) *ssm_bytes = static_cast<int64_t>(s->channels) * s->d_state * dsize(s->state_dtype) * num_slots;
    if (conv_bytes) *conv_bytes = static_cast<int64_t>(s->d_conv - 1) * s->channels * dsize(s->act_dtype) * num_slots;
    return M2_OK;
}

m2_status m2_sel_cache_wrap(const m2_sel_shape* s, int64_t num_slots, void* ssm, void* conv, int32_t* error_word,
                            m2_sel_cache* out) {
    if (!out || !ssm || !conv || num_slots <= 0) return M2_ERR_INVALID_ARG;
    if (!aligned16(ssm) || !aligned16(conv)) return M2_ERR_INVALID_ARG;
    if (error_word && (reinterpret_cast<uintptr_t>(error_word) & 3u)) return M2_ERR_INVALID_ARG;
    const m2_status st = sel_shape_status(s);
    if (st != M2_OK) return st;
    int dev = 0;
    cudaGetDevice(&dev);
    cudaGetLastError();
    std::memset(out, 0, sizeof(*out));
    out->ssm = ssm;
    out->conv = conv;
    out->error = error_word;
    out->num_slots = num_slots;
    out->shape = *s;
    out->device = dev;
    return M2_OK;
}

m2_status m2_sel_zero_slots(const m2_sel_cache* c, int32_t n, const int32_t* slot_idx, m2_stream stream) {
    const m2_status st = sel_status(c);
    if (st != M2_OK) return st;
    if (n < 0 || (n > 0 && !slot_idx)) return M2_ERR_INVALID_ARG;
    if (n == 0) return M2_OK;
    if (n > 65535) return M2_ERR_UNSUPPORTED;
    if (!on_current_device(c->device)) return M2_ERR_INVALID_ARG;
    m2::ZeroArgs a{};
    a.ssm = c->ssm;
    a.conv = c->conv;
    a.error = c->error;
    a.num_slots = c->num_slots;
    m2_sel_cache_bytes(&c->shape, 1, &a.ssm_bytes_per_slot, &a.conv_bytes_per_slot);
    a.n = n;
    a.slot_idx = slot_idx;
    return from_cuda(m2::launch_zero_slots(a, reinterpret_cast<cudaStream_t>(stream)));
}

m2_status m2_sel_conv1d_update(const m2_sel_cache* c, const m2_conv_params* conv, int32_t batch, int32_t seqlen,
                               const void* x, int64_t x_row_stride, void* x_out, int32_t out_dtype,
                               int64_t out_row_stride, const int32_t* slot_idx, m2_stream stream) {
    if (batch > 0 && seqlen > 0 && static_cast<int64_t>(batch) * seqlen > kMaxTokens) return M2_ERR_UNSUPPORTED;
    return conv_impl(c, conv, batch, seqlen, nullptr, static_cast<int64_t>(batch) * seqlen, x, x_row_stride, x_out,
                     out_dtype, out_row_stride, slot_idx, stream);
}

m2_status m2_sel_conv1d_update_varlen(const m2_sel_cache* c, const m2_conv_params* conv, int32_t nseq,
                                      const int32_t* cu_seqlens, int64_t total_tokens, int32_t max_seqlen,
                                      const void* x, int64_t x_row_stride, void* x_out, int32_t out_dtype,
                                      int64_t out_row_stride, const int32_t* slot_idx, m2_stream stream) {
    if (nseq < 0 || total_tokens < 0 || max_seqlen < 0) return M2_ERR_INVALID_ARG;
    if (total_tokens > kMaxTokens) return M2_ERR_UNSUPPORTED;
    if (nseq > 0 && total_tokens > 0 && !cu_seqlens) return M2_ERR_INVALID_ARG;
    const int32_t len = (nseq == 0 || total_tokens == 0) ? 0 : std::max(max_seqlen, 1);
    return conv_impl(c, conv, nseq, len, cu_seqlens, total_tokens, x, x_row_stride, x_out, out_dtype, out_row_stride,
                     slot_idx, stream);
}

m2_status m2_sel_state_update(const m2_sel_cache* c, const m2_sel_params* p, int32_t batch, const void* x,
                              int64_t x_row_stride, const void* dt, int64_t dt_row_stride, const void* B,
                              int64_t B_row_stride, const void* C, int64_t C_row_stride, const void* z,
                              int64_t z_row_stride, void* y, int64_t y_row_stride, const int32_t* slot_idx,
                              m2_stream stream) {
    m2_status st = sel_status(c);
    if (st != M2_OK) return st;
    if (!params_ok(p) || batch < 0) return M2_ERR_INVALID_ARG;
    if (batch == 0) return M2_OK;
    m2::SelArgs a{};
    st = sel_args(c, p, batch, x, x_row_stride, dt, dt_row_stride, B, B_row_stride, C, C_row_stride, z, z_row_stride,
                  y, y_row_stride, slot_idx, stream, &a);
    if (st != M2_OK) return st;
    return from_cuda(m2::launch_sel_update(a, reinterpret_cast<cudaStream_t>(stream)));
}

m2_status m2_sel_scan(const m2_sel_cache* c, const m2_sel_params* p, int32_t nseq, const int32_t* cu_seqlens,
                      int64_t total_tokens, int32_t max_seqlen, const void* x, int64_t x_row_stride, const void* dt,
                      int64_t dt_row_stride, const void* B, int64_t B_row_stride, const void* C,
                      int64_t C_row_stride, const void* z, int64_t z_row_stride, void* y, int64_t y_row_stride,
                      const int32_t* slot_idx, const uint8_t* has_initial_state, m2_stream stream) {
    m2_status st = sel_status(c);
    if (st != M2_OK) return st;
    if (!params_ok(p) || nseq < 0 || total_tokens < 0 || max_seqlen < 0) return M2_ERR_INVALID_ARG;
    if (total_tokens > kMaxTokens) return M2_ERR_UNSUPPORTED;
    if (nseq == 0 || total_tokens == 0) return M2_OK;
    if (!cu_seqlens) return M2_ERR_INVALID_ARG;
    m2::SelArgs a{};
    st = sel_args(c, p, nseq, x, x_row_stride, dt, dt_row_stride, B, B_row_stride, C, C_row_stride, z, z_row_stride, y,
                  y_row_stride, slot_idx, stream, &a);
    if (st != M2_OK) return st;
    a.cu_seqlens = cu_seqlens;
    a.total_tokens = total_tokens;
    a.max_seqlen = max_seqlen;
    a.has_init = has_initial_state;
    return from_cuda(m2::launch_sel_scan(a, reinterpret_cast<cudaStream_t>(stream)));
}

m2_status m2_sel_get_device_error(const m2_sel_cache* c, m2_stream stream, int32_t* out_code) {
    if (!c) return M2_ERR_INVALID_ARG;
    m2_cache word{};
    word.error = c->error;
    return m2_get_device_error(&word, stream, out_code);
}

}  // extern "C"
