// C ABI of the feed-forward operators: host-side validation, size queries,
// dispatch to the kernel launchers.  Validation happens before any HIP call.
#include <stddef.h>
#include <stdint.h>

#include "../../include/iq.h"
#include "iq_ffn_launch.h"
#include "iq_launch.h"

namespace {

bool known_dtype(int32_t t) { return t == IQ_F32 || t == IQ_BF16; }
int64_t size_of(int32_t t) { return t == IQ_F32 ? 4 : 2; }
bool known_act(int32_t a) { return a == IQ_ACT_SILU || a == IQ_ACT_GELU || a == IQ_ACT_GELU_TANH; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
iq_status from_hip(hipError_t e) { return e == hipSuccess ? IQ_OK : IQ_EHIP; }

static_assert(iqk::A_SILU == IQ_ACT_SILU && iqk::A_GELU == IQ_ACT_GELU && iqk::A_GELU_TANH == IQ_ACT_GELU_TANH,
              "activations are the public enum values");

constexpr int64_t kMax31 = ((int64_t)1 << 31) - 1;

// Rows of a layer norm: 31 bits; columns: 26, the fold's grid counting threads
// in 32 bits; and a stride whose
// products stay far inside 64 bits.
iq_status check_norm(const iq_desc* d) {
    if (!d) return IQ_EINVAL;
    if (!known_dtype(d->in_dtype)) return IQ_EINVAL;
    if (d->rows < 0 || d->cols < 0 || d->ld_in < d->cols) return IQ_EINVAL;
    if (d->rows > kMax31 || d->cols > ((int64_t)1 << 26) || d->ld_in > ((int64_t)1 << 40)) return IQ_EUNSUPPORTED;
    int64_t span = 0;
    if (__builtin_mul_overflow(d->rows, d->ld_in, &span) || span > ((int64_t)1 << 59)) return IQ_EUNSUPPORTED;
    return IQ_OK;
}

constexpr int64_t kMaxWidth = (int64_t)1 << 20;   // a 256-row tile's byte offsets stay below 2^31

iq_status check_gated(const iq_gated_desc* d) {
    if (!d) return IQ_EINVAL;
    if (!known_act(d->act) || !known_dtype(d->dtype)) return IQ_EINVAL;
    if (d->tokens < 0 || d->cols < 0 || d->features < 0) return IQ_EINVAL;
    if (d->cols % 8 || d->features % 8 || d->ld_x < d->cols) return IQ_EINVAL;
    if (d->dtype != IQ_BF16 || d->flags != 0) return IQ_EUNSUPPORTED;
    if (d->tokens > kMax31 - 1024 || d->cols > kMaxWidth || d->features > kMaxWidth || d->ld_x > kMaxWidth)
        return IQ_EUNSUPPORTED;
    if (d->ld_x % 8) return IQ_EALIGN;
    return IQ_OK;
}

// Launch grids count threads in 32 bits, at most 4 x 256 for 16 rows; byte offsets
// among a workgroup's 32 rows and among 64 tokens stay below 2^31.
constexpr int64_t kMaxRows = (int64_t)1 << 25, kMaxPackedK = (int64_t)1 << 22;

// Rules shared by the packed products; *empty where nothing is to be done.
iq_status check_packed(const iq_desc* d, int32_t x_dtype, int64_t n1, int32_t z_dtype, bool* empty) {
    if (!d) return IQ_EINVAL;
    if (d->fmt != IQ_INT4 && d->fmt != IQ_NVFP4 && d->fmt != IQ_MXFP4) return IQ_EINVAL;
    if (d->gran != IQ_PER_BLOCK || d->rows < 0 || d->cols < 0 || n1 < 0) return IQ_EINVAL;
    if (d->cols % (d->fmt == IQ_INT4 ? 128 : 32)) return IQ_EINVAL;
    if (!known_dtype(x_dtype) || !known_dtype(z_dtype)) return IQ_EINVAL;
    const uint32_t rules = d->fmt == IQ_MXFP4 ? IQ_FLAG_MX_ROUND_NEAREST | IQ_FLAG_MX_ROUND_UP
                           : d->fmt == IQ_NVFP4 ? IQ_FLAG_NV_SCALE_RNE : 0u;
    if (d->flags & ~rules) return IQ_EUNSUPPORTED;   // the rules shape the codes only, so they are not looked at
    if (x_dtype != IQ_BF16 || n1 > iqk::kPackedTokens) return IQ_EUNSUPPORTED;
    if (d->rows > kMaxRows || d->cols > kMaxPackedK) return IQ_EUNSUPPORTED;
    *empty = d->rows == 0 || n1 == 0;
    return IQ_OK;
}

iq_status check_weight(const iq_desc* d, const void* codes, const void* scales, const float* global_scale) {
    if (d->cols == 0) return IQ_OK;
    if (!codes || !scales || (d->fmt == IQ_NVFP4 && !global_scale)) return IQ_EINVAL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || (d->fmt == IQ_NVFP4 && !aligned(global_scale, 4)))
        return IQ_EALIGN;
    return IQ_OK;
}

}  // namespace

extern "C" {

iq_status iq_layer_norm(const iq_desc* d, const void* x, const void* weight, const void* bias, int32_t param_dtype,
                        float eps, void* y, float* mean, float* rstd, hipStream_t stream) {
    iq_status st = check_norm(d);
    if (st != IQ_OK) return st;
    if (!known_dtype(param_dtype)) return IQ_EINVAL;
    if (!(eps >= 0.f) || eps > 3.402823466e+38f) return IQ_EINVAL;
    if (d->rows == 0 || (d->cols == 0 && !mean && !rstd)) return IQ_OK;
    if (d->cols > 0 && (!x || !y)) return IQ_EINVAL;
    const uintptr_t ex = (uintptr_t)size_of(d->in_dtype), ep = (uintptr_t)size_of(param_dtype);
    if (!aligned(x, ex) || !aligned(y, ex) || !aligned(weight, ep) || !aligned(bias, ep) || !aligned(mean, 4) ||
        !aligned(rstd, 4))
        return IQ_EALIGN;
    iqk::NormArgs a;
    a.in_dtype = d->in_dtype; a.param_dtype = param_dtype;
    a.rows = d->rows; a.cols = d->cols; a.ld = d->ld_in; a.eps = eps;
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd;
    return from_hip(iqk::launch_layer_norm(a, stream));
}

size_t iq_layer_norm_workspace_bytes(const iq_desc* d) {
    if (check_norm(d) != IQ_OK) return 0;
    const int64_t parts = d->rows < iqk::kNormParts ? (d->rows > 0 ? d->rows : 1) : iqk::kNormParts;
    const size_t need = (size_t)parts * 2 * (size_t)d->cols * sizeof(float);
    return need < 256 ? 256 : need;
}

iq_status iq_layer_norm_backward(const iq_desc* d, const void* x, const void* dy, const void* weight,
                                 int32_t param_dtype, const float* mean, const float* rstd, void* dx, void* dweight,
                                 void* dbias, void* workspace, hipStream_t stream) {
    iq_status st = check_norm(d);
    if (st != IQ_OK) return st;
    if (!known_dtype(param_dtype)) return IQ_EINVAL;
    if (d->cols == 0) return IQ_OK;
    const bool params = dweight || dbias;
    if (d->rows > 0 && (!x || !dy || !mean || !rstd)) return IQ_EINVAL;
    if (params && d->rows > 0 && !workspace) return IQ_EINVAL;
    const uintptr_t ex = (uintptr_t)size_of(d->in_dtype), ep = (uintptr_t)size_of(param_dtype);
    if (!aligned(x, ex) || !aligned(dy, ex) || !aligned(dx, ex) || !aligned(weight, ep) || !aligned(dweight, ep) ||
        !aligned(dbias, ep) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(workspace, 256))
        return IQ_EALIGN;
    if (!params && (!dx || d->rows == 0)) return IQ_OK;
    iqk::NormGradArgs a;
    a.in_dtype = d->in_dtype; a.param_dtype = param_dtype;
    a.rows = d->rows; a.cols = d->cols; a.ld = d->ld_in;
    a.x = x; a.dy = dy; a.weight = weight; a.mean = mean; a.rstd = rstd;
    a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.partial = static_cast<float*>(workspace);
    return from_hip(iqk::launch_layer_norm_grad(a, stream));
}

size_t iq_gated_saved_bytes(const iq_gated_desc* d) {
    if (check_gated(d) != IQ_OK) return 0;
    return (size_t)d->tokens * (size_t)d->features * 2 * sizeof(float);
}

size_t iq_gated_workspace_bytes(const iq_gated_desc* d) {
    if (check_gated(d) != IQ_OK) return 0;
    const size_t need = iqk::gated_workspace_bytes(d->tokens, d->cols, d->features);
    return need < 256 ? 256 : need;
}

iq_status iq_gated_forward(const iq_gated_desc* d, const void* x, const void* w_gate, const void* w_up, void* h,
                           void* saved, hipStream_t stream) {
    iq_status st = check_gated(d);
    if (st != IQ_OK) return st;
    if (d->tokens == 0 || d->features == 0) return IQ_OK;
    if (!h || (d->cols > 0 && (!x || !w_gate || !w_up))) return IQ_EINVAL;
    if (!aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(h, 16) || !aligned(saved, 16))
        return IQ_EALIGN;
    iqk::GatedArgs a;
    a.act = d->act; a.tokens = d->tokens; a.cols = d->cols; a.features = d->features; a.ldx = d->ld_x;
    a.x = x; a.wg = w_gate; a.wu = w_up; a.h = h; a.saved = static_cast<float*>(saved);
    return from_hip(iqk::launch_gated(a, stream));
}

iq_status iq_gated_backward(const iq_gated_desc* d, const void* dh, const void* x, const void* w_gate,
                            const void* w_up, const void* saved, void* dx, void* dw_gate, void* dw_up,
                            void* workspace, hipStream_t stream) {
    iq_status st = check_gated(d);
    if (st != IQ_OK) return st;
    if (!dw_gate != !dw_up) return IQ_EINVAL;
    const bool some = d->tokens > 0 && d->features > 0 && d->cols > 0;
    if (some && (dx || dw_gate)) {
        if (!dh || !saved || !workspace) return IQ_EINVAL;
        if (dx && (!w_gate || !w_up)) return IQ_EINVAL;
        if (dw_gate && !x) return IQ_EINVAL;
    }
    if (!aligned(dh, 16) || !aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(saved, 16) ||
        !aligned(dx, 16) || !aligned(dw_gate, 16) || !aligned(dw_up, 16) || !aligned(workspace, 256))
        return IQ_EALIGN;
    iqk::GatedGradArgs a;
    a.act = d->act; a.tokens = d->tokens; a.cols = d->cols; a.features = d->features; a.ldx = d->ld_x;
    a.dh = dh; a.x = x; a.wg = w_gate; a.wu = w_up; a.saved = static_cast<const float*>(saved);
    a.dx = dx; a.dwg = dw_gate; a.dwu = dw_up; a.workspace = workspace;
    return from_hip(iqk::launch_gated_grad(a, stream));
}

iq_status iq_packed_gemv(const iq_desc* d, const void* codes, const void* scales, const float* global_scale,
                         const void* x, int32_t x_dtype, int64_t n1, void* z, int32_t z_dtype, hipStream_t stream) {
    bool empty = false;
    iq_status st = check_packed(d, x_dtype, n1, z_dtype, &empty);
    if (st != IQ_OK) return st;
    if (empty) return IQ_OK;
    if (!z || (d->cols > 0 && !x)) return IQ_EINVAL;
    if ((st = check_weight(d, codes, scales, global_scale)) != IQ_OK) return st;
    if (!aligned(x, 16) || !aligned(z, (uintptr_t)size_of(z_dtype))) return IQ_EALIGN;
    iqk::PackedArgs a = {};
    a.fmt = d->fmt; a.gated = false; a.act = 0;
    a.w[0] = {codes, scales, global_scale};
    a.x = x; a.ldx = d->cols; a.out = z; a.out_dtype = z_dtype;
    a.n0 = d->rows; a.n1 = n1; a.K = d->cols;
    return from_hip(iqk::launch_packed(a, stream));
}

iq_status iq_packed_gated(const iq_desc* d, int32_t act, const void* codes_gate, const void* scales_gate,
                          const float* global_gate, const void* codes_up, const void* scales_up,
                          const float* global_up, const void* x, int32_t x_dtype, int64_t n1, void* h,
                          int32_t h_dtype, hipStream_t stream) {
    bool empty = false;
    iq_status st = check_packed(d, x_dtype, n1, h_dtype, &empty);
    if (st != IQ_OK) return st;
    if (!known_act(act)) return IQ_EINVAL;
    if (empty) return IQ_OK;
    if (!h || (d->cols > 0 && !x)) return IQ_EINVAL;
    if ((st = check_weight(d, codes_gate, scales_gate, global_gate)) != IQ_OK) return st;
    if ((st = check_weight(d, codes_up, scales_up, global_up)) != IQ_OK) return st;
    if (!aligned(x, 16) || !aligned(h, (uintptr_t)size_of(h_dtype))) return IQ_EALIGN;
    iqk::PackedArgs a = {};
    a.fmt = d->fmt; a.gated = true; a.act = act;
    a.w[0] = {codes_gate, scales_gate, global_gate};
    a.w[1] = {codes_up, scales_up, global_up};
    a.x = x; a.ldx = d->cols; a.out = h; a.out_dtype = h_dtype;
    a.n0 = d->rows; a.n1 = n1; a.K = d->cols;
    return from_hip(iqk::launch_packed(a, stream));
}

}  // extern "C"
