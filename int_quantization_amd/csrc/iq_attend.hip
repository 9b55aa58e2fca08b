// Attention over the paged 8-bit cache.
//
// A wave takes 32 columns: neighbouring (token, query head) pairs of one key
// head, so that the heads that share a key head read its codes once.  For
// every block of 32 tokens it forms the scores S^T = K Q^T and the running
// output O^T += V^T P^T on the matrix cores (32 x 32 x 16, FP16).  In both
// results a lane holds one column, so maxima, sums and scales are its own, and
// the tokens that a lane holds of S^T are those that it feeds to the second
// product: the order of the cache's values makes them match.
#include <hip/hip_runtime.h>

#include "iq_attn_launch.h"
#include "iq_cache.h"

namespace iqk {
namespace {

constexpr int kThreads = 256, kWaves = 4;

using half2v = __attribute__((ext_vector_type(2))) _Float16;
using half8 = __attribute__((ext_vector_type(8))) _Float16;
using float16v = __attribute__((ext_vector_type(16))) float;
using float4v = __attribute__((ext_vector_type(4))) float;

// Four codes as FP16, exactly.  INT8: 1024 + (q + 128) has q + 128 in its last byte; 1152 is taken off.
template <int FMT> __device__ __forceinline__ void expand4(uint32_t w, half2v* out) {
    if constexpr (FMT == 0) {
        w ^= 0x80808080u;
        const half2v off = {(_Float16)-1152.f, (_Float16)-1152.f};
        out[0] = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x07010700u)) + off;
        out[1] = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0x64646464u, w, 0x07030702u)) + off;
    } else {
        out[0] = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false));
        out[1] = __builtin_bit_cast(half2v, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true));
    }
}

template <int FMT> __device__ __forceinline__ half8 expand8(uint32_t lo, uint32_t hi) {
    union { half2v h[4]; half8 v; } u;
    expand4<FMT>(lo, u.h);
    expand4<FMT>(hi, u.h + 2);
    return u.v;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Probabilities are held times 2^15, so that FP16 keeps all digits of those
// from 2^-29 on; the factor leaves with the division by their sum.
constexpr float kLift = 15.f;

// Parts of split rows: for every (slot, key head, split) the normalized output
// of 32 columns, then their maxima and sums.
__host__ __device__ inline int64_t part_floats(int dim) { return (int64_t)kColumns * (dim + 2); }

struct Plan {
    int64_t slots;
    int splits;
};

template <int D, int FMT> __global__ __launch_bounds__(kThreads) void k_attend(AttendArgs a, Plan plan) {
    constexpr int J = D / 32;                          // pieces of 32 elements
    __shared__ float other[2][kWaves * kColumns];      // maxima and sums of the waves
    __shared__ float pass[2 * (D / 2) * 64];           // outputs on their way to another wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, h = lane >> 5;
    Tile t;
    if (!tile_of(a, blockIdx.x, &t)) return;
    const int head = blockIdx.y, split = blockIdx.z;
    const int keys = (int)min((int64_t)t.s.length, ((int64_t)a.c.width << a.c.shift) * kBlock);
    const int64_t first = (int64_t)t.s.length - t.s.n; // position of token 0 of the call; may be negative

    // what the column sees: tokens [from, to)
    const int f = t.f0 + min(col, t.columns - 1), i = f / a.group, g = f - i * a.group;
    const int64_t p = first + i, p_lo = first + t.f0 / a.group, p_hi = first + (t.f0 + t.columns - 1) / a.group;
    const auto upto = [&](int64_t p) { return (int)(a.causal ? max((int64_t)0, min((int64_t)keys, p + 1)) : keys); };
    const auto since = [&](int64_t p) { return (int)min(max((int64_t)0, p + 1 - a.window), (int64_t)keys); };
    const int to = p < 0 ? 0 : upto(p), from = since(p);
    const int all_to = p_hi < 0 ? 0 : upto(p_hi), all_from = since(p_lo);       // some column sees these
    const int each_to = p_lo < 0 ? 0 : upto(p_lo), each_from = since(p_hi);     // every column sees these

    // the blocks of this split
    const int b_first = all_from / kBlock, b_last = (all_to + kBlock - 1) / kBlock, many = max(b_last - b_first, 0);
    const int chunk = (many + plan.splits - 1) / plan.splits;
    const int b0 = b_first + min(split * chunk, many), b1 = b_first + min((split + 1) * chunk, many);

    // queries: FP16 times a power of two that brings the row's largest into [2^14, 2^15)
    half8 q[2 * J];
    float factor;                                      // of the scores, for exponents of 2
    {
        const uint16_t* row = static_cast<const uint16_t*>(a.q) + (t.s.row + i) * a.ld_token + ((int64_t)head * a.group + g) * a.ld_head;
        uint4 raw[2 * J];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            raw[2 * j] = *reinterpret_cast<const uint4*>(row + 32 * j + 16 * h);
            raw[2 * j + 1] = *reinterpret_cast<const uint4*>(row + 32 * j + 16 * h + 8);
        }
#pragma unroll
        for (int j = 0; j < 2 * J; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = reinterpret_cast<const uint32_t*>(&raw[j])[e];
                top = max(top, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
            }
        top = max(top, (uint32_t)__shfl_xor((int)top, 32));
        int e = (int)(top >> 23);                      // 0 for zeros and subnormals, 255 for infinities and NaN
        e = e == 255 ? 0 : max(e, 1) - 127 - 14;
#pragma unroll
        for (int j = 0; j < 2 * J; ++j)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t w = reinterpret_cast<const uint32_t*>(&raw[j])[k >> 1];
                const float v = __uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16);
                q[j][k] = (_Float16)ldexpf(v, -e);
            }
        factor = ldexpf(a.scale * 1.44269504f, e);
    }

    float16v o[J];
#pragma unroll
    for (int j = 0; j < J; ++j) o[j] = 0.f;
    float m = -INFINITY, l = 0.f;
    int lift = -126;                                   // values' scales are held over 2^lift, the largest so far

    for (int b = b0 + wave; b < b1; b += kWaves) {
        const int64_t at = block_at(a.c, t.seq, b, head);
        if (at < 0) continue;
        const uint4* codes = reinterpret_cast<const uint4*>(a.c.codes + at * (2 * kBlock * (int64_t)D));
        const float2 sc = *reinterpret_cast<const float2*>(a.c.scales + at * 2);
        uint4 kc[J], vc[J];
#pragma unroll
        for (int j = 0; j < J; ++j) kc[j] = codes[(2 * j + h) * 32 + col];
#pragma unroll
        for (int j = 0; j < J; ++j) vc[j] = codes[2 * D + (32 * j + col) * 2 + h];
        float16v s = 0.f;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(kc[j].x, kc[j].y), q[2 * j], s, 0, 0, 0);
            s = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(kc[j].z, kc[j].w), q[2 * j + 1], s, 0, 0, 0);
        }
        const int t0 = b * kBlock;
        const bool masked = t0 + kBlock > each_to || t0 < each_from;
        uint32_t seen = 0xFFFFu;
        if (masked) {
            seen = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int token = t0 + 8 * (r >> 2) + 4 * h + (r & 3);
                seen |= (token >= from && token < to ? 1u : 0u) << r;
            }
        }
        const float fk = factor * sc.x;
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            s[r] *= fk;
            top = (seen >> r) & 1 ? fmaxf(top, s[r]) : top;
        }
        top = fmaxf(top, __shfl_xor(top, 32));
        const float m_new = fmaxf(m, top);
        const float alpha = m_new == m ? 1.f : exp2_fast(m - m_new);
        m = m_new;
        // values' scale as a fraction of 2^lift
        if (sc.y > ldexpf(1.f, lift)) {
            int e;
            frexpf(sc.y, &e);
            const float down = ldexpf(1.f, max(lift - e, -200));
            lift = e;
#pragma unroll
            for (int j = 0; j < J; ++j) o[j] *= down;
        }
        const float fv = ldexpf(sc.y, -lift);
        float sum = 0.f;
        half8 pv[2];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float e = (seen >> r) & 1 ? exp2_fast(s[r] - m + kLift) : 0.f;
            sum += e;
            pv[r >> 3][r & 7] = (_Float16)(e * fv);
        }
        l = l * alpha + sum;
        if (t0 + kBlock > keys) {                      // codes behind the sequence may be anything: zeros
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint32_t* w = reinterpret_cast<uint32_t*>(&vc[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int n = keys - t0 - (8 * i + 4 * h);      // bytes of this word that are the sequence's
                    w[i] &= n <= 0 ? 0u : n >= 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            o[j] *= alpha;
            o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(vc[j].x, vc[j].y), pv[0], o[j], 0, 0, 0);
            o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(vc[j].z, vc[j].w), pv[1], o[j], 0, 0, 0);
        }
    }
    l += __shfl_xor(l, 32);

    // join the four waves: each output over its own sum, weighted by it
    other[0][wave * kColumns + col] = m;
    other[1][wave * kColumns + col] = l;
    __syncthreads();
    float top = -INFINITY, total = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, other[0][w * kColumns + col]);
    const auto weight = [&](float mw) { return mw == top ? 1.f : exp2_fast(mw - top); };
#pragma unroll
    for (int w = 0; w < kWaves; ++w) total += other[1][w * kColumns + col] * weight(other[0][w * kColumns + col]);
    // sums are positive unless nothing was seen; NaN passes through
    const float mine = l == 0.f ? 0.f : weight(m) / total;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[j][r] = l == 0.f ? 0.f : ldexpf(o[j][r] * mine, lift);
#pragma unroll
    for (int round = kWaves / 2; round; round >>= 1) {
        float* mail = pass + (wave & (round - 1)) * (D / 2) * 64;
        if (wave >= round && wave < 2 * round) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) mail[(j * 16 + r) * 64 + lane] = o[j][r];
        }
        __syncthreads();
        if (wave < round) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[j][r] += mail[(j * 16 + r) * 64 + lane];
        }
        __syncthreads();
    }
    if (wave != 0 || col >= t.columns) return;
    if (plan.splits == 1) {
        uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)(t.s.row + i) * a.q_heads + (int64_t)head * a.group + g) * D;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                union { __bf16 b[4]; uint2 w; } u;
#pragma unroll
                for (int e = 0; e < 4; ++e) u.b[e] = (__bf16)o[j][r + e];
                *reinterpret_cast<uint2*>(out + 32 * j + 2 * r + 4 * h) = u.w;
            }
        return;
    }
    float* part = static_cast<float*>(a.workspace) + (((int64_t)blockIdx.x * a.c.heads + head) * plan.splits + split) * part_floats(D);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
            *reinterpret_cast<float4v*>(part + col * D + 32 * j + 2 * r + 4 * h) = (float4v){o[j][r], o[j][r + 1], o[j][r + 2], o[j][r + 3]};
    if (h == 0) {
        part[kColumns * D + col] = top;
        part[kColumns * (D + 1) + col] = total;
    }
}

// Joins the splits of a tile's columns, a wave for each column in turn.
template <int D> __global__ __launch_bounds__(kThreads) void k_join(AttendArgs a, Plan plan) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, head = blockIdx.y;
    Tile t;
    if (!tile_of(a, blockIdx.x, &t)) return;
    const float* parts = static_cast<const float*>(a.workspace) + ((int64_t)blockIdx.x * a.c.heads + head) * plan.splits * part_floats(D);
    for (int col = wave; col < t.columns; col += kWaves) {
        float top = -INFINITY;
        for (int s = 0; s < plan.splits; ++s) top = fmaxf(top, parts[s * part_floats(D) + kColumns * D + col]);
        float total = 0.f, sum[D / 64 + (D % 64 != 0)] = {};
        for (int s = 0; s < plan.splits; ++s) {
            const float* part = parts + s * part_floats(D);
            const float m = part[kColumns * D + col], l = part[kColumns * (D + 1) + col];
            if (l == 0.f) continue;                    // nothing seen there
            const float w = (m == top ? 1.f : exp2_fast(m - top)) * l;
            total += w;
            for (int e = lane, k = 0; e < D; e += 64, ++k) sum[k] += w * part[col * D + e];
        }
        const int f = t.f0 + col, i = f / a.group, g = f - i * a.group;
        uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)(t.s.row + i) * a.q_heads + (int64_t)head * a.group + g) * D;
        for (int e = lane, k = 0; e < D; e += 64, ++k)
            out[e] = __builtin_bit_cast(uint16_t, (__bf16)(total == 0.f ? 0.f : sum[k] / total));
    }
}

Plan plan_of(const AttendArgs& a) {
    Plan p;
    p.slots = tile_slots(a);
    const int64_t tiles = p.slots * a.c.heads, most = ((int64_t)a.c.width << a.c.shift) / 16;
    int64_t splits = (1024 + tiles - 1) / (tiles ? tiles : 1);
    if (splits > most) splits = most;
    if (splits > 128) splits = 128;
    p.splits = (int)(splits < 1 ? 1 : splits);
    return p;
}

template <int D> hipError_t launch(const AttendArgs& a, hipStream_t stream) {
    const Plan p = plan_of(a);
    const dim3 grid((unsigned)p.slots, (unsigned)a.c.heads, (unsigned)p.splits);
    if (a.c.fmt) k_attend<D, 1><<<grid, kThreads, 0, stream>>>(a, p);
    else k_attend<D, 0><<<grid, kThreads, 0, stream>>>(a, p);
    if (p.splits > 1) k_join<D><<<dim3((unsigned)p.slots, (unsigned)a.c.heads), kThreads, 0, stream>>>(a, p);
    return hipGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(const AttendArgs& a) {
    const Plan p = plan_of(a);
    return p.splits == 1 ? 0 : (size_t)(p.slots * a.c.heads * p.splits * part_floats(a.c.dim)) * sizeof(float);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t stream) {
    switch (a.c.dim) {
    case 64: return launch<64>(a, stream);
    case 96: return launch<96>(a, stream);
    case 128: return launch<128>(a, stream);
    case 192: return launch<192>(a, stream);
    default: return launch<256>(a, stream);
    }
}

}  // namespace iqk
