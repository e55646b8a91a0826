// m2_api_q8.cu -- the C entry points of the 8-bit state cache (include/m2.h).
// Host-side only: argument validation and error mapping.
#include <cuda_runtime.h>

#include <cstring>

#include "m2_host.cuh"
#include "m2_q8.cuh"

using namespace m2::host;

namespace {

m2_status q8_shape_status(const m2_shape* s) {
    if (!s) return M2_ERR_INVALID_ARG;
    if (s->nheads <= 0 || s->head_dim <= 0 || s->d_state <= 0 || s->ngroups <= 0 || s->d_conv <= 0)
        return M2_ERR_INVALID_ARG;
    if (s->nheads % s->ngroups != 0 || !valid_dtype(s->act_dtype)) return M2_ERR_INVALID_ARG;
    if (s->d_conv < 2 || s->d_conv > 8 || s->ngroups > 65535) return M2_ERR_UNSUPPORTED;
    // rows of a slot and channels in 32 bits, as the kernels index them
    if (static_cast<int64_t>(s->nheads) * s->head_dim > INT32_MAX || m2_conv_dim(s) > INT32_MAX) return M2_ERR_UNSUPPORTED;
    return m2::q8_shape_supported(s->nheads, s->head_dim, s->d_state, s->ngroups);
}

m2_status q8_status(const m2_q8_cache* c) {
    if (!c || !c->ssm || !c->scale || !c->conv || c->num_slots <= 0) return M2_ERR_INVALID_ARG;
    return q8_shape_status(&c->shape);
}

int64_t conv_bytes_per_slot(const m2_shape& s) {
    return static_cast<int64_t>(s.d_conv - 1) * m2_conv_dim(&s) * dsize(s.act_dtype);
}

m2_status copy_impl(const m2_cache* full, const m2_q8_cache* q8, bool store, int32_t n, const int32_t* src_idx,
                    const int32_t* dst_idx, m2_stream stream) {
    if (!full || !full->ssm || !full->conv || full->num_slots <= 0) return M2_ERR_INVALID_ARG;
    m2_status st = m2_shape_check(&full->shape);
    if (st != M2_OK) return st;
    st = q8_status(q8);
    if (st != M2_OK) return st;
    const m2_shape &f = full->shape, &q = q8->shape;
    if (f.nheads != q.nheads || f.head_dim != q.head_dim || f.d_state != q.d_state || f.ngroups != q.ngroups ||
        f.d_conv != q.d_conv || f.act_dtype != q.act_dtype)
        return M2_ERR_INVALID_ARG;
    if (n < 0 || (n > 0 && (!src_idx || !dst_idx))) return M2_ERR_INVALID_ARG;
    if (n == 0) return M2_OK;
    if (!on_current_device(q8->device) || !on_current_device(full->device)) return M2_ERR_INVALID_ARG;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (validate_mode()) {
        const m2_status v = validate_slots(dst_idx, n, store ? q8->num_slots : full->num_slots, cs);
        if (v != M2_OK) return v;
    }
    m2::Q8CopyArgs a{};
    a.ssm = full->ssm;
    a.conv = full->conv;
    a.error = full->error;
    a.num_slots = full->num_slots;
    a.q = q8->ssm;
    a.scale = q8->scale;
    a.q_conv = q8->conv;
    a.q_error = q8->error;
    a.q_num_slots = q8->num_slots;
    a.rows = f.nheads * f.head_dim;
    a.N = f.d_state;
    a.state_bf16 = f.state_dtype == M2_BF16;
    a.conv_bytes = conv_bytes_per_slot(f);
    a.n = n;
    a.src_idx = src_idx;
    a.dst_idx = dst_idx;
    return from_cuda(store ? m2::launch_q8_store(a, cs) : m2::launch_q8_load(a, cs));
}

m2_status update_impl(const m2_q8_cache* c, const m2_ssm_params* ssm, const m2_conv_params* conv,
                      const m2_norm_params* norm, int32_t batch, const void* xBC, int64_t xBC_row_stride,
                      const void* dt, int64_t dt_row_stride, const void* z, int64_t z_row_stride, void* y,
                      int64_t y_row_stride, const int32_t* slot_idx, m2_stream stream) {
    const m2_status st = q8_status(c);
    if (st != M2_OK) return st;
    if (!ssm || !ssm->A_log || !ssm->dt_bias || !ssm->D || !conv || !conv->weight || batch < 0)
        return M2_ERR_INVALID_ARG;
    if (conv->activation != 0 && conv->activation != 1) return M2_ERR_INVALID_ARG;
    if (batch == 0) return M2_OK;
    if (!xBC || !dt || !y || !slot_idx) return M2_ERR_INVALID_ARG;
    const m2_shape& s = c->shape;
    const int as = dsize(s.act_dtype);
    const int64_t cd = m2_conv_dim(&s);
    const int64_t hp = static_cast<int64_t>(s.nheads) * s.head_dim;
    if (!aligned16(conv->weight) || (conv->bias && !aligned16(conv->bias))) return M2_ERR_INVALID_ARG;
    if (!aligned16(xBC) || !aligned16(y) || !stride_ok(xBC_row_stride, as, cd) || !stride_ok(y_row_stride, as, hp) ||
        dt_row_stride < s.nheads)
        return M2_ERR_INVALID_ARG;
    if (z && (!aligned16(z) || !stride_ok(z_row_stride, as, hp))) return M2_ERR_INVALID_ARG;
    if (norm && (!norm->weight || !aligned16(norm->weight) || !(norm->eps >= 0.f))) return M2_ERR_INVALID_ARG;
    if (batch > 65535) return M2_ERR_UNSUPPORTED;
    if (!on_current_device(c->device)) return M2_ERR_INVALID_ARG;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    if (validate_mode()) {
        const m2_status v = validate_slots(slot_idx, batch, c->num_slots, cs);
        if (v != M2_OK) return v;
    }
    m2::Q8UpdateArgs a{};
    a.ssm = c->ssm;
    a.scale = c->scale;
    a.conv = c->conv;
    a.error = c->error;
    a.num_slots = c->num_slots;
    a.H = s.nheads;
    a.P = s.head_dim;
    a.N = s.d_state;
    a.G = s.ngroups;
    a.K = s.d_conv;
    a.conv_dim = cd;
    a.act_bf16 = s.act_dtype == M2_BF16;
    a.A_log = ssm->A_log;
    a.dt_bias = ssm->dt_bias;
    a.D = ssm->D;
    a.conv_w = conv->weight;
    a.conv_b = conv->bias;
    a.activation = conv->activation;
    a.batch = batch;
    a.xBC = xBC;
    a.xBC_stride = xBC_row_stride;
    a.dt = dt;
    a.dt_stride = dt_row_stride;
    a.z = z;
    a.z_stride = z_row_stride;
    a.y = y;
    a.y_stride = y_row_stride;
    a.slot_idx = slot_idx;
    a.norm_w = norm ? norm->weight : nullptr;
    a.norm_eps = norm ? norm->eps : 0.f;
    return from_cuda(m2::launch_q8_update(a, cs));
}

}  // namespace

extern "C" {

m2_status m2_q8_shape_check(const m2_shape* s) { return q8_shape_status(s); }

m2_status m2_q8_cache_bytes(const m2_shape* s, int64_t num_slots, int64_t* code_bytes, int64_t* scale_bytes,
                            int64_t* conv_bytes) {
    const m2_status st = q8_shape_status(s);
    if (st != M2_OK) return st;
    if (num_slots <= 0) return M2_ERR_INVALID_ARG;
    const int64_t rows = static_cast<int64_t>(s->nheads) * s->head_dim;
    if (code_bytes) *code_bytes = rows * s->d_state * num_slots;
    if (scale_bytes) *scale_bytes = rows * 4 * num_slots;
    if (conv_bytes) *conv_bytes = conv_bytes_per_slot(*s) * num_slots;
    return M2_OK;
}

m2_status m2_q8_cache_wrap(const m2_shape* s, int64_t num_slots, int8_t* ssm, float* scale, void* conv,
                           int32_t* error_word, m2_q8_cache* out) {
    if (!out || !ssm || !scale || !conv || num_slots <= 0) return M2_ERR_INVALID_ARG;
    if (!aligned16(ssm) || !aligned16(scale) || !aligned16(conv)) return M2_ERR_INVALID_ARG;
    if (error_word && (reinterpret_cast<uintptr_t>(error_word) & 3u)) return M2_ERR_INVALID_ARG;
    const m2_status st = q8_shape_status(s);
    if (st != M2_OK) return st;
    int dev = 0;
    cudaGetDevice(&dev);
    cudaGetLastError();
    std::memset(out, 0, sizeof(*out));
    out->ssm = ssm;
    out->scale = scale;
    out->conv = conv;
    out->error = error_word;
    out->num_slots = num_slots;
    out->shape = *s;
    out->device = dev;
    return M2_OK;
}

m2_status m2_q8_zero_slots(const m2_q8_cache* c, int32_t n, const int32_t* slot_idx, m2_stream stream) {
    const m2_status st = q8_status(c);
    if (st != M2_OK) return st;
    if (n < 0 || (n > 0 && !slot_idx)) return M2_ERR_INVALID_ARG;
    if (n == 0) return M2_OK;
    if (n > 65535) return M2_ERR_UNSUPPORTED;
    if (!on_current_device(c->device)) return M2_ERR_INVALID_ARG;
    const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
    const int64_t rows = static_cast<int64_t>(c->shape.nheads) * c->shape.head_dim;
    m2::ZeroArgs a{};
    a.ssm = c->ssm;
    a.conv = c->conv;
    a.error = c->error;
    a.num_slots = c->num_slots;
    a.ssm_bytes_per_slot = rows * c->shape.d_state;
    a.conv_bytes_per_slot = conv_bytes_per_slot(c->shape);
    a.n = n;
    a.slot_idx = slot_idx;
    const cudaError_t e = m2::launch_zero_slots(a, cs);
    if (e != cudaSuccess) return from_cuda(e);
    a.ssm = c->scale;  // zero states read back as zero with any finite scale; a NaN one has to go
    a.ssm_bytes_per_slot = rows * 4;
    a.conv_bytes_per_slot = 0;
    return from_cuda(m2::launch_zero_slots(a, cs));
}

m2_status m2_q8_store(const m2_cache* src, const m2_q8_cache* dst, int32_t n, const int32_t* src_idx,
                      const int32_t* dst_idx, m2_stream stream) {
    return copy_impl(src, dst, true, n, src_idx, dst_idx, stream);
}

m2_status m2_q8_load(const m2_q8_cache* src, const m2_cache* dst, int32_t n, const int32_t* src_idx,
                     const int32_t* dst_idx, m2_stream stream) {
    return copy_impl(dst, src, false, n, src_idx, dst_idx, stream);
}

m2_status m2_q8_state_update(const m2_q8_cache* c, const m2_ssm_params* ssm, const m2_conv_params* conv,
                             int32_t batch, const void* xBC, int64_t xBC_row_stride, const void* dt,
                             int64_t dt_row_stride, const void* z, int64_t z_row_stride, void* y,
                             int64_t y_row_stride, const int32_t* slot_idx, m2_stream stream) {
    return update_impl(c, ssm, conv, nullptr, batch, xBC, xBC_row_stride, dt, dt_row_stride, z, z_row_stride, y,
                       y_row_stride, slot_idx, stream);
}

m2_status m2_q8_state_update_norm(const m2_q8_cache* c, const m2_ssm_params* ssm, const m2_conv_params* conv,
                                  const m2_norm_params* norm, int32_t batch, const void* xBC,
                                  int64_t xBC_row_stride, const void* dt, int64_t dt_row_stride, const void* z,
                                  int64_t z_row_stride, void* y, int64_t y_row_stride, const int32_t* slot_idx,
                                  m2_stream stream) {
    if (!norm) return M2_ERR_INVALID_ARG;
    return update_impl(c, ssm, conv, norm, batch, xBC, xBC_row_stride, dt, dt_row_stride, z, z_row_stride, y,
                       y_row_stride, slot_idx, stream);
}

m2_status m2_q8_get_device_error(const m2_q8_cache* c, m2_stream stream, int32_t* out_code) {
    if (!c) return M2_ERR_INVALID_ARG;
    m2_cache word{};
    word.error = c->error;
    return m2_get_device_error(&word, stream, out_code);
}

}  // extern "C"
