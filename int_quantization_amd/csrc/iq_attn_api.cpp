// C ABI of the attention operators: host-side validation, size queries,
// dispatch to the kernel launchers.  Validation happens before any HIP call.
#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/iq.h"
#include "iq_attn_launch.h"

namespace {

bool known_dtype(int32_t t) { return t == IQ_F32 || t == IQ_BF16; }
int64_t size_of(int32_t t) { return t == IQ_F32 ? 4 : 2; }
bool known_layout(int32_t l) { return l == IQ_ROTARY_HALF || l == IQ_ROTARY_INTERLEAVED; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
iq_status from_hip(hipError_t e) { return e == hipSuccess ? IQ_OK : IQ_EHIP; }

static_assert(IQ_INT8 == 0 && IQ_FP8_E4M3 == 1 && IQ_F32 == 0 && IQ_BF16 == 1, "kernels take the public enum values");

constexpr int64_t kMostTokens = ((int64_t)1 << 24) - 1, kMostStride = (int64_t)1 << 40;
constexpr int64_t kMostSpan = (int64_t)1 << 59;
constexpr int64_t kMostWork = (int64_t)1 << 23;      // workgroups of a launch, whose threads are counted in 32 bits

bool is_finite(double v) { return v - v == 0; }

// Strides of [n, m] blocks of `dim` elements: not negative, products far inside 64 bits.  Nothing is asked of one that
// leads from the first block to none.
iq_status check_strides(int64_t n, int64_t m, int64_t ld_n, int64_t ld_m) {
    if (n <= 1) ld_n = 0;
    if (m <= 1) ld_m = 0;
    if (ld_n < 0 || ld_m < 0) return IQ_EINVAL;
    if (ld_n > kMostStride || ld_m > kMostStride) return IQ_EUNSUPPORTED;
    if ((ld_n && n > kMostSpan / ld_n) || (ld_m && m > kMostSpan / ld_m)) return IQ_EUNSUPPORTED;
    return IQ_OK;
}

// Whether no two elements of a strided output are one.
bool apart(int64_t n, int64_t m, int64_t dim, int64_t ld_n, int64_t ld_m) {
    if (n == 0 || m == 0 || dim == 0) return true;
    if (n <= 1) return m <= 1 || ld_m >= dim;
    if (m <= 1) return ld_n >= dim;
    return (ld_m >= dim && ld_n >= (m - 1) * ld_m + dim) || (ld_n >= dim && ld_m >= (n - 1) * ld_n + dim);
}

// Whether rows [n, m, dim] with these strides lie as a dense result's do.
bool dense(int64_t n, int64_t m, int64_t dim, int64_t ld_n, int64_t ld_m) { return (n <= 1 || ld_n == m * dim) && (m <= 1 || ld_m == dim); }

iq_status check_rotary(const iq_rotary_desc* d) {
    if (!d) return IQ_EINVAL;
    if (!known_dtype(d->dtype) || !known_layout(d->layout)) return IQ_EINVAL;
    if (d->tokens < 0 || d->heads < 0 || d->dim < 0 || d->rot < 0 || d->rot % 2 || d->rot > d->dim) return IQ_EINVAL;
    if (!is_finite(d->amplitude)) return IQ_EINVAL;
    if (d->flags != 0) return IQ_EUNSUPPORTED;
    if (d->tokens > kMostTokens || d->heads > 4096 || d->dim > 1024 || d->heads * d->dim > ((int64_t)1 << 20)) return IQ_EUNSUPPORTED;
    iq_status st = check_strides(d->tokens, d->heads, d->ld_token, d->ld_head);
    if (st == IQ_OK) st = check_strides(d->tokens, d->heads, d->ld_token_out, d->ld_head_out);
    if (st != IQ_OK) return st;
    return apart(d->tokens, d->heads, d->dim, d->ld_token_out, d->ld_head_out) ? IQ_OK : IQ_EINVAL;
}

iq_status rotate(const iq_rotary_desc* d, const void* x, const int32_t* positions, const double* table, void* y, float way,
                 hipStream_t stream) {
    const iq_status st = check_rotary(d);
    if (st != IQ_OK) return st;
    if (d->tokens == 0 || d->heads == 0 || d->dim == 0) return IQ_OK;
    if (!x || !y || !positions || (d->rot > 0 && !table)) return IQ_EINVAL;
    if (x == y && ((d->tokens > 1 && d->ld_token != d->ld_token_out) || (d->heads > 1 && d->ld_head != d->ld_head_out))) return IQ_EINVAL;
    const uintptr_t e = (uintptr_t)size_of(d->dtype);
    if (!aligned(x, e) || !aligned(y, e) || !aligned(positions, 4) || !aligned(table, 8)) return IQ_EALIGN;
    iqk::RotaryArgs a;
    a.dtype = d->dtype; a.interleaved = d->layout == IQ_ROTARY_INTERLEAVED;
    a.tokens = (int)d->tokens; a.heads = (int)d->heads; a.dim = (int)d->dim; a.rot = d->rot;
    a.ld_token = d->ld_token; a.ld_head = d->ld_head; a.ld_token_out = d->ld_token_out; a.ld_head_out = d->ld_head_out;
    a.amplitude = d->amplitude; a.way = way;
    a.x = x; a.positions = positions; a.table = table; a.y = y;
    return from_hip(iqk::launch_rotary(a, stream));
}

iq_status check_memory(const iq_cache_desc* d) {
    if (!d) return IQ_EINVAL;
    if (d->fmt != IQ_INT8 && d->fmt != IQ_FP8_E4M3) return IQ_EINVAL;
    if (d->heads < 1 || d->dim < 1 || d->pages < 0) return IQ_EINVAL;
    if (d->page < 32 || (d->page & (d->page - 1))) return IQ_EINVAL;
    if (d->flags != 0) return IQ_EUNSUPPORTED;
    if (d->dim != 64 && d->dim != 96 && d->dim != 128 && d->dim != 192 && d->dim != 256) return IQ_EUNSUPPORTED;
    if (d->heads > 1024 || d->page > 4096 || d->pages > ((int64_t)1 << 31) - 1) return IQ_EUNSUPPORTED;
    return IQ_OK;
}

iq_status check_cache(const iq_cache_desc* d, int64_t tokens, const int32_t* starts) {
    const iq_status st = check_memory(d);
    if (st != IQ_OK) return st;
    if (d->batch < 0 || d->width < 0 || tokens < 0) return IQ_EINVAL;
    if (!starts && tokens != d->batch) return IQ_EINVAL;
    if (tokens > kMostTokens || d->batch > ((int64_t)1 << 20)) return IQ_EUNSUPPORTED;
    if (d->width > ((int64_t)1 << 30) / d->page) return IQ_EUNSUPPORTED;
    return IQ_OK;
}

// Slots of a call's blocks of 32 tokens, counted as the kernels' launcher does.
int64_t block_work(const iq_cache_desc* d, int64_t tokens, const int32_t* starts) {
    return (starts ? tokens / 32 + 2 * d->batch : d->batch) * d->heads * 2;
}

// Pointers to the cache; width 0 makes every page absent.
iq_status check_arrays(const iq_cache_desc* d, const void* codes, const void* scales, const int32_t* page_table,
                       const int32_t* lengths, const int32_t* starts) {
    if (!lengths || (d->width > 0 && !page_table) || (d->pages > 0 && (!codes || !scales))) return IQ_EINVAL;
    if (!aligned(codes, 16) || !aligned(scales, 8) || !aligned(page_table, 4) || !aligned(lengths, 4) || !aligned(starts, 4))
        return IQ_EALIGN;
    return IQ_OK;
}

iqk::CacheArgs cache_args(const iq_cache_desc* d, const void* codes, const float* scales, const int32_t* page_table,
                          const int32_t* lengths, const int32_t* starts, int64_t tokens) {
    iqk::CacheArgs c;
    c.fmt = d->fmt; c.heads = d->heads; c.dim = d->dim;
    c.shift = __builtin_ctz((unsigned)d->page) - 5;
    c.batch = (int)d->batch; c.width = (int)d->width; c.pages = d->pages;
    c.codes = static_cast<uint8_t*>(const_cast<void*>(codes)); c.scales = const_cast<float*>(scales);
    c.page_table = page_table; c.lengths = lengths; c.starts = starts; c.tokens = (int)tokens;
    return c;
}

iq_status check_attention(const iq_cache_desc* d, const iq_attention_desc* a, const int32_t* starts) {
    if (!a) return IQ_EINVAL;
    const iq_status st = check_cache(d, a->tokens, starts);
    if (st != IQ_OK) return st;
    if (!known_dtype(a->dtype) || (a->causal != 0 && a->causal != 1)) return IQ_EINVAL;
    if (a->q_heads < 1 || a->q_heads % d->heads || a->window < 0 || (a->window > 0 && !a->causal)) return IQ_EINVAL;
    if (!(a->scale >= 0.f) || !is_finite(a->scale)) return IQ_EINVAL;
    if (a->dtype != IQ_BF16 || a->flags != 0 || a->q_heads > 4096) return IQ_EUNSUPPORTED;
    if (a->tokens * a->q_heads > ((int64_t)1 << 28)) return IQ_EUNSUPPORTED;
    const iq_status strides = check_strides(a->tokens, a->q_heads, a->ld_token, a->ld_head);
    if (strides != IQ_OK) return strides;
    if ((a->tokens > 1 && a->ld_token % 8) || (a->q_heads > 1 && a->ld_head % 8)) return IQ_EALIGN;
    return IQ_OK;
}

iqk::AttendArgs attend_args(const iq_cache_desc* d, const iq_attention_desc* a, const int32_t* starts) {
    iqk::AttendArgs k = {};
    k.c = cache_args(d, nullptr, nullptr, nullptr, nullptr, starts, a->tokens);
    k.q_heads = (int)a->q_heads; k.group = (int)(a->q_heads / d->heads);
    k.causal = a->causal; k.ld_token = a->ld_token; k.ld_head = a->ld_head;
    k.window = a->window > 0 && a->window < (1 << 30) ? (int)a->window : 1 << 30;
    k.scale = a->scale;
    return k;
}

}  // namespace

extern "C" {

iq_status iq_rotary_table(int32_t rot, double base, int32_t scaling, double factor, double context, double low,
                          double high, double* table) {
    if (rot < 0 || rot % 2 || (rot > 0 && !table)) return IQ_EINVAL;
    if (scaling < IQ_ROTARY_PLAIN || scaling > IQ_ROTARY_PARTS) return IQ_EINVAL;
    if (!is_finite(base) || !is_finite(factor) || base <= 0 || factor <= 0) return IQ_EINVAL;
    if (scaling == IQ_ROTARY_PARTS && !(is_finite(context) && is_finite(low) && is_finite(high) && context > 0 && high > low)) return IQ_EINVAL;
    const double tau = 6.283185307179586476925;
    const double b = scaling == IQ_ROTARY_BASE && rot > 2 ? base * pow(factor, (double)rot / (rot - 2)) : base;
    for (int pass = 0; pass < 2; ++pass)               // looked at first, then written
        for (int32_t i = 0; i < rot / 2; ++i) {
            double turns = pow(b, -2.0 * i / rot) / tau;
            if (scaling == IQ_ROTARY_LINEAR) turns /= factor;
            if (scaling == IQ_ROTARY_PARTS) {
                const double w = (turns * context - low) / (high - low), keep = w < 0 ? 0 : w > 1 ? 1 : w;
                turns = turns / factor * (1 - keep) + turns * keep;
            }
            if (!is_finite(turns)) return IQ_EINVAL;
            if (pass) table[i] = turns;
        }
    return IQ_OK;
}

iq_status iq_rotary(const iq_rotary_desc* d, const void* x, const int32_t* positions, const double* table, void* y,
                    hipStream_t stream) {
    return rotate(d, x, positions, table, y, 1.f, stream);
}

iq_status iq_rotary_backward(const iq_rotary_desc* d, const void* dy, const int32_t* positions, const double* table,
                             void* dx, hipStream_t stream) {
    return rotate(d, dy, positions, table, dx, -1.f, stream);
}

size_t iq_cache_codes_bytes(const iq_cache_desc* d) {
    if (check_memory(d) != IQ_OK) return 0;
    return (size_t)d->pages * (size_t)d->heads * (size_t)d->page * 2 * (size_t)d->dim;
}

size_t iq_cache_scales_bytes(const iq_cache_desc* d) {
    if (check_memory(d) != IQ_OK) return 0;
    return (size_t)d->pages * (size_t)d->heads * (size_t)(d->page / 32) * 2 * sizeof(float);
}

iq_status iq_cache_append(const iq_cache_desc* d, const iq_append_desc* a, const void* k, const void* v,
                          const int32_t* page_table, const int32_t* lengths, const int32_t* starts,
                          const double* table, const void* q, void* q_out, void* codes, float* scales,
                          hipStream_t stream) {
    if (!d || !a) return IQ_EINVAL;
    iq_status st = check_cache(d, a->tokens, starts);
    if (st != IQ_OK) return st;
    if (!known_dtype(a->dtype) || !known_layout(a->layout)) return IQ_EINVAL;
    if (a->rot < 0 || a->rot % 2 || a->rot > d->dim || !is_finite(a->amplitude) || a->q_heads < 0) return IQ_EINVAL;
    if (a->flags != 0 || a->q_heads > 4096) return IQ_EUNSUPPORTED;
    if ((st = check_strides(a->tokens, d->heads, a->ld_k_token, a->ld_k_head)) != IQ_OK) return st;
    if ((st = check_strides(a->tokens, d->heads, a->ld_v_token, a->ld_v_head)) != IQ_OK) return st;
    if ((st = check_strides(a->tokens, a->q_heads, a->ld_q_token, a->ld_q_head)) != IQ_OK) return st;
    if (block_work(d, a->tokens, starts) + a->tokens > kMostWork) return IQ_EUNSUPPORTED;
    if (a->tokens == 0 || d->batch == 0) return IQ_OK;
    if (!k || !v || (a->rot > 0 && !table) || (a->q_heads > 0 && (!q || !q_out))) return IQ_EINVAL;
    if (a->q_heads > 0 && q == q_out && !dense(a->tokens, a->q_heads, d->dim, a->ld_q_token, a->ld_q_head)) return IQ_EINVAL;
    if ((st = check_arrays(d, codes, scales, page_table, lengths, starts)) != IQ_OK) return st;
    const uintptr_t e = (uintptr_t)size_of(a->dtype);
    if (!aligned(k, e) || !aligned(v, e) || !aligned(q, e) || !aligned(q_out, e) || !aligned(table, 8)) return IQ_EALIGN;
    iqk::AppendArgs g;
    g.c = cache_args(d, codes, scales, page_table, lengths, starts, a->tokens);
    g.dtype = a->dtype; g.interleaved = a->layout == IQ_ROTARY_INTERLEAVED; g.q_heads = (int)a->q_heads; g.rot = a->rot;
    g.ld_k_token = a->ld_k_token; g.ld_k_head = a->ld_k_head; g.ld_v_token = a->ld_v_token; g.ld_v_head = a->ld_v_head;
    g.ld_q_token = a->ld_q_token; g.ld_q_head = a->ld_q_head; g.amplitude = a->amplitude;
    g.k = k; g.v = v; g.q = a->q_heads > 0 ? q : nullptr; g.q_out = q_out; g.table = table;
    return from_hip(iqk::launch_cache_append(g, stream));
}

iq_status iq_cache_read(const iq_cache_desc* d, const void* codes, const float* scales, const int32_t* page_table,
                        const int32_t* lengths, const int32_t* starts, int64_t tokens, void* k, void* v,
                        int32_t out_dtype, hipStream_t stream) {
    iq_status st = check_cache(d, tokens, starts);
    if (st != IQ_OK) return st;
    if (!known_dtype(out_dtype)) return IQ_EINVAL;
    if (block_work(d, tokens, starts) > kMostWork) return IQ_EUNSUPPORTED;
    if (tokens == 0 || d->batch == 0 || (!k && !v)) return IQ_OK;
    if ((st = check_arrays(d, codes, scales, page_table, lengths, starts)) != IQ_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16)) return IQ_EALIGN;
    if (k == v) return IQ_EINVAL;
    iqk::ReadArgs g;
    g.c = cache_args(d, codes, scales, page_table, lengths, starts, tokens);
    g.dtype = out_dtype; g.k = k; g.v = v;
    return from_hip(iqk::launch_cache_read(g, stream));
}

size_t iq_cache_attention_workspace_bytes(const iq_cache_desc* d, const iq_attention_desc* a) {
    // starts only say how tokens are shared out: the larger of both plans serves either
    const int32_t some = 0;
    size_t need = 256;
    if (check_attention(d, a, &some) != IQ_OK) return 0;
    if (a->tokens == 0 || d->batch == 0) return need;
    size_t n = iqk::attend_workspace_bytes(attend_args(d, a, &some));
    if (n > need) need = n;
    if (a->tokens == d->batch) {
        n = iqk::attend_workspace_bytes(attend_args(d, a, nullptr));
        if (n > need) need = n;
    }
    return need;
}

iq_status iq_cache_attention(const iq_cache_desc* d, const iq_attention_desc* a, const void* codes, const float* scales,
                             const int32_t* page_table, const int32_t* lengths, const int32_t* starts, const void* q,
                             void* o, void* workspace, hipStream_t stream) {
    iq_status st = check_attention(d, a, starts);
    if (st != IQ_OK) return st;
    if (a->tokens == 0 || d->batch == 0) return IQ_OK;
    if (!q || !o || !workspace) return IQ_EINVAL;
    if (q == o && !dense(a->tokens, a->q_heads, d->dim, a->ld_token, a->ld_head)) return IQ_EINVAL;
    if ((st = check_arrays(d, codes, scales, page_table, lengths, starts)) != IQ_OK) return st;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(workspace, 256)) return IQ_EALIGN;
    iqk::AttendArgs k = attend_args(d, a, starts);
    k.c = cache_args(d, codes, scales, page_table, lengths, starts, a->tokens);
    k.q = q; k.o = o; k.workspace = workspace;
    return from_hip(iqk::launch_attend(k, stream));
}

}  // extern "C"
