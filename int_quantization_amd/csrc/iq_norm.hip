// Layer norm for gfx950 (MI355X), forward and backward.
//
//   mean = sum x / C, r = 1 / sqrt(sum (x - mean)^2 / C + eps), n = (x - mean) r
//   y  = n w + b
//   dx = r (a - sum a / C - n sum (a n) / C),  a = dy w
//   dw = sum over rows of dy n,  db = sum over rows of dy
//
// HBM bounds both passes: the forward reads x and writes y, the backward
// reads x and dy and writes dx.  A row is therefore held in registers
// between its statistics and its output, and read once; a workgroup holds
// the parameters of its columns, goes over many rows and has the next one
// in flight while it works on this.  The variance is
// taken about the mean, not as a difference of squares, so that an offset
// much larger than the spread costs no digits.
// Measured on 8192 x 8192 BF16: forward 48 us (5.6 TB/s), backward 76 (5.3) and
// the fold of its 256 partial rows 5; with a workgroup to each row and no row
// ahead 73 and 93.  8192 x 8191, whose rows start anywhere: 60 and 142, FP32
// 101 (5.3 TB/s) and 157 (5.1).  One row of 4096: 2.9 us, all of it latency.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "iq_ffn_launch.h"
#include "iq_launch.h"

namespace iqk {
namespace {

typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float as_f(uint32_t u) { return __uint_as_float(u); }

// FP32 to BF16 bits, to nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 b2v __attribute__((ext_vector_type(2)));
    const b2v v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

template <int T> struct Elem;
template <> struct Elem<D_F32> { typedef float type; };
template <> struct Elem<D_BF16> { typedef uint16_t type; };

// Eight consecutive elements as they lie in memory.  A row may start at any
// element, so a load is not aligned to its 16 bytes (the hardware takes global
// loads and stores at any address); of the last vector of a row only the first
// `have` elements are touched, and the others read as zeros.
template <int T> struct Raw { u4v w[T == D_F32 ? 2 : 1]; };
template <int T> __device__ __forceinline__ Raw<T> raw(const void* base, int64_t i, int have) {
    typedef typename Elem<T>::type E;
    const E* p = static_cast<const E*>(base) + i;
    Raw<T> r = {};
    if (have >= 8) {
        __builtin_memcpy(&r, p, 8 * sizeof(E));
    } else {
        E e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) e[k] = k < have ? p[k] : E(0);
        __builtin_memcpy(&r, e, 8 * sizeof(E));
    }
    return r;
}
template <int T> __device__ __forceinline__ void unpack(const Raw<T>& r, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (T == D_F32) {
            v[k] = as_f(r.w[0][k]);
            v[4 + k] = as_f(r.w[1][k]);
        } else {
            v[2 * k] = as_f(r.w[0][k] << 16);
            v[2 * k + 1] = as_f(r.w[0][k] & 0xFFFF0000u);
        }
    }
}
template <int T> __device__ __forceinline__ void load8(const void* base, int64_t i, int have, float (&v)[8]) { unpack<T>(raw<T>(base, i, have), v); }
template <int T> __device__ __forceinline__ void store8(void* base, int64_t i, int have, const float (&v)[8]) {
    typedef typename Elem<T>::type E;
    E* p = static_cast<E*>(base) + i;
    Raw<T> r;
    if constexpr (T == D_F32) {
#pragma unroll
        for (int k = 0; k < 4; ++k) { r.w[0][k] = __float_as_uint(v[k]); r.w[1][k] = __float_as_uint(v[4 + k]); }
    } else {
        r.w[0] = u4v{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7])};
    }
    if (have >= 8) {
        __builtin_memcpy(p, &r, 8 * sizeof(E));
    } else {
        E e[8];
        __builtin_memcpy(e, &r, 8 * sizeof(E));
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < have) p[k] = e[k];
    }
}

__device__ __forceinline__ void load_param(const void* p, int type, int64_t i, int have, float none, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = none;
    } else if (type == D_F32) {
        load8<D_F32>(p, i, have, v);
    } else {
        load8<D_BF16>(p, i, have, v);
    }
}

__device__ __forceinline__ void store_param(void* p, int type, int64_t i, float v) {
    if (type == D_F32) static_cast<float*>(p)[i] = v;
    else static_cast<uint16_t*>(p)[i] = (uint16_t)bf16_pair(v, 0.f);
}
__device__ __forceinline__ void store_param8(void* p, int type, int64_t i, int have, const float (&v)[8]) {
    if (!p) return;
    if (type == D_F32) store8<D_F32>(p, i, have, v);
    else store8<D_BF16>(p, i, have, v);
}

// Sum over the wave; every lane returns it.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
    return v;
}

// Sums of two values over the NW waves of a workgroup or of a group of its
// threads (t: the thread's number there), in wave order.  `red`
// may be written again once every thread has passed a later barrier.
template <int NW> __device__ __forceinline__ void block_sum2(float& a, float& b, float (&red)[NW][2], int t = threadIdx.x) {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (NW > 1) {
        if ((t & 63) == 0) { red[t >> 6][0] = a; red[t >> 6][1] = b; }
        __syncthreads();
        a = red[0][0];
        b = red[0][1];
#pragma unroll
        for (int k = 1; k < NW; ++k) { a += red[k][0]; b += red[k][1]; }
    }
}
template <int NW> __device__ __forceinline__ float block_sum(float a, float (&red)[NW][2]) {
    float b = 0.f;
    block_sum2<NW>(a, b, red);
    return a;
}

// A workgroup of NT threads takes rows blockIdx.x, + gridDim.x, ...; a thread
// holds HOLD vectors of 8 elements of one.
template <int IN, int NT, int HOLD>
__global__ __launch_bounds__(NT) void k_norm(NormArgs a) {
    constexpr int NW = NT / 64;
    __shared__ float red[2][2][NW][2];
    const int t = threadIdx.x, nv = (int)((a.cols + 7) / 8);
    auto have = [&](int64_t c) { return (int)min((int64_t)8, a.cols - 8 * c); };      // elements of vector c
    const float inv = a.cols ? 1.f / (float)a.cols : 0.f;               // rows without elements have statistics too
    Raw<IN> next[HOLD] = {};
    float w[HOLD][8], b[HOLD][8];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (t + k * NT < nv) next[k] = raw<IN>(a.x, row * a.ld + (int64_t)(t + k * NT) * 8, have(t + k * NT));
    };
    fetch(blockIdx.x);
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
        if (t + k * NT < nv) {
            load_param(a.weight, a.param_dtype, (int64_t)(t + k * NT) * 8, have(t + k * NT), 1.f, w[k]);
            load_param(a.bias, a.param_dtype, (int64_t)(t + k * NT) * 8, have(t + k * NT), 0.f, b[k]);
        }
    int odd = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, odd ^= 1) {
        float v[HOLD][8], s = 0.f;
#pragma unroll
        for (int k = 0; k < HOLD; ++k) unpack<IN>(next[k], v[k]);
        if (row + gridDim.x < a.rows) fetch(row + gridDim.x);
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (t + k * NT < nv) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s += v[k][i];
            }
        const float mean = block_sum<NW>(s, red[odd][0]) * inv;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (const int n = have(t + k * NT); n < 8) {              // past the row's end: nothing off the mean
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = i < n ? v[k][i] : mean;
            }
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (t + k * NT < nv) {
#pragma unroll
                for (int i = 0; i < 8; ++i) { v[k][i] -= mean; q = __builtin_fmaf(v[k][i], v[k][i], q); }
            }
        const float rstd = 1.f / sqrtf(block_sum<NW>(q, red[odd][1]) * inv + a.eps);
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (t + k * NT < nv) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf(v[k][i] * rstd, w[k][i], b[k][i]);
                store8<IN>(a.y, row * a.cols + (int64_t)(t + k * NT) * 8, have(t + k * NT), y);
            }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Rows longer than the registers hold, read three times.
template <int IN, int NT>
__global__ __launch_bounds__(NT) void k_norm_long(NormArgs a) {
    constexpr int NW = NT / 64;
    __shared__ float red[2][NW][2];
    const int t = threadIdx.x;
    const int64_t nv = (a.cols + 7) / 8;
    auto have = [&](int64_t c) { return (int)min((int64_t)8, a.cols - 8 * c); };      // elements of vector c
    const float inv = 1.f / (float)a.cols;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t xo = row * a.ld, yo = row * a.cols;
        float e[8], s = 0.f, q = 0.f;
        for (int64_t c = t; c < nv; c += NT) {
            load8<IN>(a.x, xo + c * 8, have(c), e);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += e[i];
        }
        const float mean = block_sum<NW>(s, red[0]) * inv;
        for (int64_t c = t; c < nv; c += NT) {
            load8<IN>(a.x, xo + c * 8, have(c), e);
#pragma unroll
            for (int i = 0; i < 8; ++i) { const float d = i < have(c) ? e[i] - mean : 0.f; q = __builtin_fmaf(d, d, q); }
        }
        const float rstd = 1.f / sqrtf(block_sum<NW>(q, red[1]) * inv + a.eps);
        for (int64_t c = t; c < nv; c += NT) {
            float w[8], b[8], y[8];
            load8<IN>(a.x, xo + c * 8, have(c), e);
            load_param(a.weight, a.param_dtype, c * 8, have(c), 1.f, w);
            load_param(a.bias, a.param_dtype, c * 8, have(c), 0.f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf((e[i] - mean) * rstd, w[i], b[i]);
            store8<IN>(a.y, yo + c * 8, have(c), y);
        }
        if (t == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// Backward: G groups of NT threads take a row each, and a thread the same
// columns of every row of its group, so the sums over rows stay in registers
// until the last one.  The groups' sums are added in LDS in their order, and
// one partial row per workgroup reaches memory; a lone workgroup writes the
// gradients.  (Narrow rows need the groups: 60000 x 1001 FP32 takes 373 us
// with one row at a time to a workgroup.)
template <int IN, int NT, int HOLD, int G>
__global__ __launch_bounds__(NT * G) void k_norm_grad(NormGradArgs a) {
    constexpr int NW = NT / 64;
    constexpr bool AHEAD = NT * HOLD < 2048;     // 1024 threads of two vectors have no registers for the next row
    __shared__ float red[2][G][NW][2];
    __shared__ float sums[G > 1 ? G - 1 : 1][G > 1 ? 2 * HOLD * 8 : 1][NT];
    const int t = threadIdx.x % NT, g0 = threadIdx.x / NT;
    const int nv = (int)((a.cols + 7) / 8);
    auto have = [&](int64_t c) { return (int)min((int64_t)8, a.cols - 8 * c); };      // elements of vector c
    const float inv = 1.f / (float)a.cols;
    float w[HOLD][8], dw[HOLD][8], db[HOLD][8];
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) { w[k][i] = 0.f; dw[k][i] = 0.f; db[k][i] = 0.f; }
        if (t + k * NT < nv) load_param(a.weight, a.param_dtype, (int64_t)(t + k * NT) * 8, have(t + k * NT), 1.f, w[k]);
    }
    Raw<IN> nx[HOLD] = {}, ng[HOLD] = {};
    float next_mean = 0.f, next_rstd = 0.f;
    auto fetch = [&](int64_t row) {
        next_mean = a.mean[row];
        next_rstd = a.rstd[row];
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (t + k * NT < nv) {
                nx[k] = raw<IN>(a.x, row * a.ld + (int64_t)(t + k * NT) * 8, have(t + k * NT));
                ng[k] = raw<IN>(a.dy, row * a.cols + (int64_t)(t + k * NT) * 8, have(t + k * NT));
            }
    };
    // every group makes the same number of turns, for their barriers are one
    const int64_t stride = (int64_t)gridDim.x * G;
    if (AHEAD && (int64_t)blockIdx.x * G + g0 < a.rows) fetch((int64_t)blockIdx.x * G + g0);
    int odd = 0;
    for (int64_t at = (int64_t)blockIdx.x * G; at < a.rows; at += stride, odd ^= 1) {
        const int64_t row = at + g0;
        const bool live = row < a.rows;
        const int64_t yo = row * a.cols;
        const float mean = AHEAD ? next_mean : live ? a.mean[row] : 0.f, rstd = AHEAD ? next_rstd : live ? a.rstd[row] : 0.f;
        float x[HOLD][8], g[HOLD][8], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < HOLD; ++k) {
            if constexpr (AHEAD) {
                unpack<IN>(nx[k], x[k]);
                unpack<IN>(ng[k], g[k]);
            } else if (live && t + k * NT < nv) {
                load8<IN>(a.x, row * a.ld + (int64_t)(t + k * NT) * 8, have(t + k * NT), x[k]);
                load8<IN>(a.dy, yo + (int64_t)(t + k * NT) * 8, have(t + k * NT), g[k]);
            }
        }
        if (AHEAD && row + stride < a.rows) fetch(row + stride);
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (const int n = have(t + k * NT); n < 8) {              // past the row's end: nothing off the mean
#pragma unroll
                for (int i = 0; i < 8; ++i) x[k][i] = i < n ? x[k][i] : mean;
            }
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (live && t + k * NT < nv) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float n = (x[k][i] - mean) * rstd, e = g[k][i] * w[k][i];
                    x[k][i] = n;
                    dw[k][i] = __builtin_fmaf(g[k][i], n, dw[k][i]);
                    db[k][i] += g[k][i];
                    g[k][i] = e;
                    s1 += e;
                    s2 = __builtin_fmaf(e, n, s2);
                }
            }
        if (!a.dx) continue;
        block_sum2<NW>(s1, s2, red[odd][g0], t);
        s1 *= inv;
        s2 *= inv;
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
            if (live && t + k * NT < nv) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = rstd * (g[k][i] - __builtin_fmaf(x[k][i], s2, s1));
                store8<IN>(a.dx, yo + (int64_t)(t + k * NT) * 8, have(t + k * NT), d);
            }
    }
    if (!a.dweight && !a.dbias) return;
    if constexpr (G > 1) {
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (g0) {
                    sums[g0 - 1][16 * k + i][t] = dw[k][i];
                    sums[g0 - 1][16 * k + 8 + i][t] = db[k][i];
                }
        __syncthreads();
        if (g0) return;
#pragma unroll
        for (int k = 0; k < HOLD; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                for (int g = 0; g < G - 1; ++g) {
                    dw[k][i] += sums[g][16 * k + i][t];
                    db[k][i] += sums[g][16 * k + 8 + i][t];
                }
    }
    float* pw = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
        if (t + k * NT < nv) {
            const int64_t c = (int64_t)(t + k * NT) * 8;
            const int n = have(t + k * NT);
            if (gridDim.x == 1) {
                store_param8(a.dweight, a.param_dtype, c, n, dw[k]);
                store_param8(a.dbias, a.param_dtype, c, n, db[k]);
            } else {
                store8<D_F32>(pw, c, n, dw[k]);
                store8<D_F32>(pw + a.cols, c, n, db[k]);
            }
        }
}

// Rows longer than the registers hold: one pass for the sums, one for dx.
// The sums over rows go through the partial rows in memory, each thread
// adding to its own columns.
template <int IN, int NT>
__global__ __launch_bounds__(NT) void k_norm_grad_long(NormGradArgs a) {
    constexpr int NW = NT / 64;
    __shared__ float red[2][NW][2];
    const int t = threadIdx.x;
    const int64_t nv = (a.cols + 7) / 8;
    auto have = [&](int64_t c) { return (int)min((int64_t)8, a.cols - 8 * c); };      // elements of vector c
    const float inv = 1.f / (float)a.cols;
    const bool params = a.dweight || a.dbias;
    float* pw = a.partial + (int64_t)blockIdx.x * 2 * a.cols;
    int odd = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, odd ^= 1) {
        const int64_t xo = row * a.ld, yo = row * a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        const bool first = row == blockIdx.x;
        float x[8], g[8], w[8], s1 = 0.f, s2 = 0.f;
        for (int64_t c = t; c < nv; c += NT) {
            load8<IN>(a.x, xo + c * 8, have(c), x);
            load8<IN>(a.dy, yo + c * 8, have(c), g);
            load_param(a.weight, a.param_dtype, c * 8, have(c), 1.f, w);
            float pdw[8], pdb[8];
            if (params && !first) {
                load8<D_F32>(pw, c * 8, have(c), pdw);
                load8<D_F32>(pw + a.cols, c * 8, have(c), pdb);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n = i < have(c) ? (x[i] - mean) * rstd : 0.f, e = g[i] * w[i];
                s1 += e;
                s2 = __builtin_fmaf(e, n, s2);
                pdw[i] = __builtin_fmaf(g[i], n, first ? 0.f : pdw[i]);
                pdb[i] = first ? g[i] : pdb[i] + g[i];
            }
            if (params) {
                store8<D_F32>(pw, c * 8, have(c), pdw);
                store8<D_F32>(pw + a.cols, c * 8, have(c), pdb);
            }
        }
        if (!a.dx) continue;
        block_sum2<NW>(s1, s2, red[odd]);
        s1 *= inv;
        s2 *= inv;
        for (int64_t c = t; c < nv; c += NT) {
            load8<IN>(a.x, xo + c * 8, have(c), x);
            load8<IN>(a.dy, yo + c * 8, have(c), g);
            load_param(a.weight, a.param_dtype, c * 8, have(c), 1.f, w);
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = rstd * (g[i] * w[i] - __builtin_fmaf((x[i] - mean) * rstd, s2, s1));
            store8<IN>(a.dx, yo + c * 8, have(c), d);
        }
    }
}

// The partial rows' sum: 64 columns per workgroup, 16 waves a sixteenth of
// the rows each, added in row order and then in wave order.
__global__ __launch_bounds__(1024) void k_norm_fold(const float* partial, int parts, int64_t cols, int type, void* dweight,
                                                    void* dbias) {
    __shared__ float red[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;      // of the 2 cols columns of a partial row
    float v[kNormParts / 16];                               // loads of all rows in flight at once
#pragma unroll
    for (int k = 0; k < kNormParts / 16; ++k) v[k] = wave + 16 * k < parts && c < 2 * cols ? partial[(wave + 16 * k) * 2 * cols + c] : 0.f;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kNormParts / 16; ++k) s += v[k];
    red[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= 2 * cols) return;
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[k][lane];
    void* out = c < cols ? dweight : dbias;
    if (out) store_param(out, type, c < cols ? c : c - cols, s);
}

constexpr int64_t kNormHeld = 2048;      // vectors of a row that a workgroup's registers hold

// Workgroups of the forward pass: a row each while they fill the GPU twice
// over at most, then as many as stay resident, each with several rows.
unsigned norm_grid(int64_t rows, int threads) { return (unsigned)std::min<int64_t>(rows, 256 * (2048 / threads)); }

template <int IN> hipError_t pick_norm(const NormArgs& a, hipStream_t s) {
    const int64_t nv = (a.cols + 7) / 8;
    if (nv <= 256) k_norm<IN, 256, 1><<<norm_grid(a.rows, 256), 256, 0, s>>>(a);
    else if (nv <= 512) k_norm<IN, 512, 1><<<norm_grid(a.rows, 512), 512, 0, s>>>(a);
    else if (nv <= 1024) k_norm<IN, 512, 2><<<norm_grid(a.rows, 512), 512, 0, s>>>(a);
    else if (nv <= kNormHeld) k_norm<IN, 1024, 2><<<norm_grid(a.rows, 1024), 1024, 0, s>>>(a);
    else k_norm_long<IN, 512><<<(unsigned)std::min<int64_t>(a.rows, 1 << 20), 512, 0, s>>>(a);
    return hipGetLastError();
}

// Rows that one workgroup takes in less time than the fold's launch, or all at
// once.  BF16, a call by itself and with the fold, in us (on the GPU alone in
// brackets): 4 rows of 4104 columns 8.2 (7.2) and 10.5 (6.3), of 8192 8.8 (8.2)
// and 10.6 (7.1), of 16384 11.5 (11.0) and 10.5 (9.0); 8 rows of 4104 12.5 and 11.3.
constexpr int64_t kNormLone = 4;

// Rows that a workgroup of the backward pass takes at once, in 1024 threads.
int norm_groups(int64_t nv) { return nv <= 64 ? 16 : nv <= 128 ? 8 : nv <= 256 ? 4 : nv <= 512 ? 2 : 1; }

template <int IN> hipError_t pick_grad(const NormGradArgs& a, unsigned grid, hipStream_t s) {
    const int64_t nv = (a.cols + 7) / 8;
    if (nv <= 64) k_norm_grad<IN, 64, 1, 16><<<grid, 1024, 0, s>>>(a);
    else if (nv <= 128) k_norm_grad<IN, 128, 1, 8><<<grid, 1024, 0, s>>>(a);
    else if (nv <= 256) k_norm_grad<IN, 256, 1, 4><<<grid, 1024, 0, s>>>(a);
    else if (nv <= 512) k_norm_grad<IN, 512, 1, 2><<<grid, 1024, 0, s>>>(a);
    else if (nv <= 1024) k_norm_grad<IN, 512, 2, 1><<<grid, 512, 0, s>>>(a);
    else if (nv <= kNormHeld) k_norm_grad<IN, 1024, 2, 1><<<grid, 1024, 0, s>>>(a);
    else k_norm_grad_long<IN, 512><<<grid, 512, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, hipStream_t s) {
    if (a.rows == 0) return hipSuccess;
    return a.in_dtype == D_F32 ? pick_norm<D_F32>(a, s) : pick_norm<D_BF16>(a, s);
}

hipError_t launch_layer_norm_grad(const NormGradArgs& a, hipStream_t s) {
    const int64_t nv = (a.cols + 7) / 8, groups = norm_groups(nv);
    const bool lone = a.rows > 0 && a.rows <= std::max(kNormLone, groups) && nv <= kNormHeld;
    const int parts = lone ? 1 : (int)std::min<int64_t>((a.rows + groups - 1) / groups, kNormParts);
    if (parts > 0) {
        const hipError_t e = a.in_dtype == D_F32 ? pick_grad<D_F32>(a, parts, s) : pick_grad<D_BF16>(a, parts, s);
        if (e != hipSuccess) return e;
    }
    if ((a.dweight || a.dbias) && !lone)
        k_norm_fold<<<(unsigned)((2 * a.cols + 63) / 64), 1024, 0, s>>>(a.partial, parts, a.cols, a.param_dtype, a.dweight,
                                                                      a.dbias);
    return hipGetLastError();
}

}  // namespace iqk
