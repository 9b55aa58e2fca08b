// Rotary positions, and what writes the paged 8-bit cache and reads it back.
#include <hip/hip_bf16.h>
#include <hip/hip_runtime.h>

#include "iq_attn_launch.h"
#include "iq_cache.h"

namespace iqk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float to_float(float v) { return v; }

// FP32 to BF16, nearest even; NaN stays NaN.
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
template <typename T> __device__ __forceinline__ T from_float(float f) {
    if constexpr (sizeof(T) == 2) return to_bf16(f);
    else return f;
}

template <typename T> struct alignas(16) Vec {
    static constexpr int N = 16 / sizeof(T);
    T e[N];
};

// Cosine and sine of 2 pi * position * turns.  The product has up to 31 + 53 bits and is
// reduced to half a turn in 64 bits, so its error is 2^-53 of the angle; what FP32 leaves of the
// reduced angle (up to 2^-25 half turns) turns the result once more, to first order.
__device__ __forceinline__ float2 turn(int position, double turns, float amplitude, float way) {
    double t = (double)position * turns;
    t = 2 * (t - __builtin_rint(t));
    const float near = (float)t, rest = (float)(t - (double)near) * 3.14159265f;
    float s, c;
    sincospif(near, &s, &c);
    const float cosine = __builtin_fmaf(-s, rest, c), sine = __builtin_fmaf(c, rest, s);
    return make_float2(cosine * amplitude, sine * (amplitude * way));
}

// Turns the heads [head0, head1) of one token.  cs: cosine and sine of its pairs, in LDS.
//   VEC: 16-byte units, where strides, bases and the ends of what turns are multiples of them.  Otherwise single
//   elements, but for those from `edge` on, which are copied in such units (dim: none are).
template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ void turn_token(const T* x, T* y, int64_t ldx, int64_t ldy, int head0, int head1, int dim, int rot,
                                           int edge, const float2* cs, int thread, int threads) {
    constexpr int V = VEC ? Vec<T>::N : 1;
    const int pairs = rot >> 1;
    const int turned = INTER ? (VEC ? rot / V : pairs) : pairs / V;     // units that hold pairs
    const int single = (edge - rot) / V;                                  // units to copy: of V, then of 16 bytes
    const int rest = x == y ? 0 : single + (dim - edge) / Vec<T>::N;
    const int units = turned + rest;
    if (units == 0) return;
    const float inv = 1.f / (float)units;
    const int items = (head1 - head0) * units;
    for (int i = thread; i < items; i += threads) {
        // i / units: i + 1/2 is at least half a unit from every multiple, far more than FP32's error below 2^22
        const int head = (int)(((float)i + 0.5f) * inv), u = i - head * units;
        const T* from = x + (head0 + head) * ldx;
        T* to = y + (head0 + head) * ldy;
        if (u >= turned) {
            const int r = u - turned, at = r < single ? rot + r * V : edge + (r - single) * Vec<T>::N;
            if (VEC || r >= single) *reinterpret_cast<Vec<T>*>(to + at) = *reinterpret_cast<const Vec<T>*>(from + at);
            else to[at] = from[at];
        } else if constexpr (INTER && VEC) {
            Vec<T> v = *reinterpret_cast<const Vec<T>*>(from + u * V);
#pragma unroll
            for (int p = 0; p < V / 2; ++p) {
                const float2 w = cs[u * (V / 2) + p];
                const float a = to_float(v.e[2 * p]), b = to_float(v.e[2 * p + 1]);
                v.e[2 * p] = from_float<T>(a * w.x - b * w.y);
                v.e[2 * p + 1] = from_float<T>(b * w.x + a * w.y);
            }
            *reinterpret_cast<Vec<T>*>(to + u * V) = v;
        } else if constexpr (VEC) {
            Vec<T> v = *reinterpret_cast<const Vec<T>*>(from + u * V), w = *reinterpret_cast<const Vec<T>*>(from + pairs + u * V);
#pragma unroll
            for (int p = 0; p < V; ++p) {
                const float2 t = cs[u * V + p];
                const float a = to_float(v.e[p]), b = to_float(w.e[p]);
                v.e[p] = from_float<T>(a * t.x - b * t.y);
                w.e[p] = from_float<T>(b * t.x + a * t.y);
            }
            *reinterpret_cast<Vec<T>*>(to + u * V) = v;
            *reinterpret_cast<Vec<T>*>(to + pairs + u * V) = w;
        } else {
            const int ia = INTER ? 2 * u : u, ib = INTER ? 2 * u + 1 : pairs + u;
            const float2 t = cs[u];
            const float a = to_float(from[ia]), b = to_float(from[ib]);
            to[ia] = from_float<T>(a * t.x - b * t.y);
            to[ib] = from_float<T>(b * t.x + a * t.y);
        }
    }
}

// Bytes bound it: a workgroup takes a token, whose cosines and sines all heads share from LDS.  8192 tokens of 32 heads of
// 128 in BF16 (134 MB) take 24 us there and back each, 5.6 TB/s; 1531 tokens of 12 heads of 96 in FP32 (14 MB) 5.1 us, mostly the
// launch and the 64-bit angles.
constexpr int kMostPairs = 512;

template <typename T, bool INTER, bool VEC> __global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a, int edge) {
    __shared__ float2 cs[kMostPairs];
    const int t = blockIdx.x;
    const int position = a.positions[t];
    for (int p = threadIdx.x; p < a.rot / 2; p += kThreads) cs[p] = turn(position, a.table[p], a.amplitude, a.way);
    __syncthreads();
    turn_token<T, INTER, VEC>(static_cast<const T*>(a.x) + t * a.ld_token, static_cast<T*>(a.y) + t * a.ld_token_out, a.ld_head,
                              a.ld_head_out, 0, a.heads, a.dim, a.rot, edge, cs, threadIdx.x, kThreads);
}

// ---- append -----------------------------------------------------------------------
// 16 elements of a head that a thread holds, two runs of 8: those of `item` of a row, of which there are dim / 16.  Halves
// apart, an item of what turns holds 8 pairs; otherwise 16 neighbours.
__device__ __forceinline__ int second_run(int item, int rot, bool interleaved, int* first) {
    const int at = item * 16;
    if (at >= rot || interleaved) {
        *first = at;
        return at + 8;
    }
    *first = at >> 1;
    return (at >> 1) + (rot >> 1);
}

template <typename T> __device__ __forceinline__ void load8(const T* from, float* v) {
#pragma unroll
    for (int u = 0; u < 8 / Vec<T>::N; ++u) {
        const Vec<T> w = reinterpret_cast<const Vec<T>*>(from)[u];
#pragma unroll
        for (int e = 0; e < Vec<T>::N; ++e) v[u * Vec<T>::N + e] = to_float(w.e[e]);
    }
}

template <int FMT> __device__ __forceinline__ uint32_t code4(const float* v, float scale) {
    if constexpr (FMT == 0) {
        return code_of<0>(v[0] / scale) | code_of<0>(v[1] / scale) << 8 | code_of<0>(v[2] / scale) << 16 | code_of<0>(v[3] / scale) << 24;
    } else {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = v[e] / scale;
            y[e] = y[e] == y[e] ? fminf(fmaxf(y[e], -448.f), 448.f) : 0.f;
        }
        const int low = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], low, true);
    }
}

// Code of each byte over 2^up, rounded.
template <int FMT> __device__ __forceinline__ uint32_t moved4(uint32_t w, int up) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = ldexpf(code_value<FMT>((w >> (8 * e)) & 0xFFu), -up);
    return code4<FMT>(v, 1.f);
}

// Bytes of a word of values that are tokens [lo, hi); the word's first byte is token t.
__device__ __forceinline__ uint32_t bytes_between(int t, int lo, int hi) {
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) m |= t + b >= lo && t + b < hi ? 0xFFu << (8 * b) : 0u;
    return m;
}

// A block's new keys or values.  Every thread holds NI items of 16 elements in registers (heads of up to 128 elements
// have one for each): keys are turned there (cosines and sines from LDS, made once for all heads of the workgroup), the
// largest magnitude is found, and codes are written, so x is read once.  Values change places through LDS, where a row of
// 32 codes has 36 bytes so that rows meet in fewer banks.  Queries are turned in the same launch, a workgroup to a token.
//   VEC: rows that start on 16 bytes, rot a multiple of 16.
// 8192 tokens of 32 + 2 * 8 heads of 128 (184 MB) take 42 us, 4.4 TB/s where a copy reaches 6.1: the vector units are busy 63%
// of the time (a division for each element, conversions, addresses), LDS 28%, most of it conflicts of the values' byte
// stores.  One token of them takes 5.4 us, the launch and a chain of four loads.
constexpr int kPitch = 36;

template <typename T, int FMT, bool VEC, int NI> __global__ __launch_bounds__(kThreads, 4) void k_append(AppendArgs a, int64_t slots, int per, bool vec_q) {
    __shared__ __align__(16) uint8_t turned[256 * kPitch];
    __shared__ float most[kThreads / 64];
    extern __shared__ float2 cs[];                     // [new tokens of the block][pairs]
    const CacheArgs& c = a.c;
    const int dim = c.dim, pairs = a.rot >> 1, tid = threadIdx.x;
    const int groups = (c.heads + per - 1) / per;      // of the key heads, `per` to a workgroup
    const int64_t cache_work = slots * (groups + c.heads);
    if ((int64_t)blockIdx.x >= cache_work) {           // a token's queries
        const int row = (int)(blockIdx.x - cache_work);
        int seq = row;
        if (c.starts) seq = sequence_of(c, row, 1, 1, 0);
        const Span s = span_of(c, seq);
        const int64_t position = (int64_t)s.length - s.n + (row - s.row);
        if (row < s.row || row >= s.row + s.n || position < 0) return;
        for (int p = tid; p < pairs; p += kThreads) cs[p] = turn((int)position, a.table[p], a.amplitude, 1.f);
        __syncthreads();
        const T* x = static_cast<const T*>(a.q) + row * a.ld_q_token;
        T* y = static_cast<T*>(a.q_out) + (int64_t)row * a.q_heads * dim;
        if (vec_q) {
            if (a.interleaved) turn_token<T, true, true>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, dim, cs, tid, kThreads);
            else turn_token<T, false, true>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, dim, cs, tid, kThreads);
        } else {
            if (a.interleaved) turn_token<T, true, false>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, dim, cs, tid, kThreads);
            else turn_token<T, false, false>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, dim, cs, tid, kThreads);
        }
        return;
    }
    const int work = (int)(blockIdx.x % (groups + c.heads));
    const bool which = work >= groups;                 // values
    int seq, block;
    Span s;
    if (!slot_block(c, blockIdx.x / (groups + c.heads), &seq, &s, &block)) return;
    const int64_t place = block_at(c, seq, block, 0);
    if (place < 0) return;
    const int first = s.length - s.n;                  // position of the call's first token; may be negative
    const int lo = max(first - block * kBlock, 0), hi = min(s.length - block * kBlock, kBlock);      // new tokens of the block
    const int row0 = s.row + (block * kBlock - first); // row of the block's token 0
    const int chunks = dim / 16, items = (hi - lo) * chunks;
    const bool turns = !which && pairs > 0;
    if (turns) {
        for (int i = tid; i < (hi - lo) * pairs; i += kThreads) {
            const int r = i / pairs, p = i - r * pairs;
            cs[i] = turn(block * kBlock + lo + r, a.table[p], a.amplitude, 1.f);
        }
        __syncthreads();
    }
    for (int head = which ? work - groups : work * per; head < (which ? work - groups + 1 : min((work + 1) * per, c.heads)); ++head) {
        int id = tid;                                  // known anew for every head: what hangs on it alone would be kept for all
        asm volatile("" : "+v"(id));
        const int64_t at = place + ((int64_t)head << c.shift);
        uint8_t* codes = c.codes + at * (2 * kBlock * (int64_t)dim) + (which ? kBlock * dim : 0);
        float* scale_at = c.scales + at * 2 + which;
        const float had = lo > 0 ? *scale_at : 0.f;
        const T* from = static_cast<const T*>(which ? a.v : a.k) + (int64_t)head * (which ? a.ld_v_head : a.ld_k_head);
        const int64_t ld = which ? a.ld_v_token : a.ld_k_token;
        float v[NI][16], amax = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = id + n * kThreads, r = i / chunks, chunk = i - r * chunks;
            if (i >= items) continue;
            const T* row = from + (row0 + lo + r) * ld;
            int x0;
            const int x1 = second_run(chunk, which ? 0 : a.rot, a.interleaved, &x0);
            if constexpr (VEC) {
                load8(row + x0, v[n]);
                load8(row + x1, v[n] + 8);
            } else if (!turns || a.rot % 16 == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[n][e] = to_float(row[x0 + e]), v[n][8 + e] = to_float(row[x1 + e]);
            }
            if (turns) {
                const float2* w = cs + r * pairs;
                if (!VEC && a.rot % 16) {              // an element and its partner at a time
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int d = chunk * 16 + e;
                        const bool b = a.interleaved ? d & 1 : d >= pairs;
                        const int p = a.interleaved ? d >> 1 : b ? d - pairs : d, other = a.interleaved ? d ^ 1 : b ? p : d + pairs;
                        const float x = to_float(row[d]);
                        v[n][e] = x;
                        if (d < a.rot) {
                            const float y = to_float(row[other]);
                            v[n][e] = b ? x * w[p].x + y * w[p].y : x * w[p].x - y * w[p].y;
                        }
                    }
                } else if (chunk * 16 < a.rot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = w[chunk * 8 + e];
                        if (a.interleaved) {
                            const float x = v[n][2 * e], y = v[n][2 * e + 1];
                            v[n][2 * e] = x * t.x - y * t.y;
                            v[n][2 * e + 1] = y * t.x + x * t.y;
                        } else {
                            const float x = v[n][e], y = v[n][8 + e];
                            v[n][e] = x * t.x - y * t.y;
                            v[n][8 + e] = y * t.x + x * t.y;
                        }
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fabsf(v[n][e]) <= 3.402823466e+38f ? fmaxf(amax, fabsf(v[n][e])) : amax;   // neither NaN nor infinite
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
        __syncthreads();                               // the head before is done with the LDS
        if ((tid & 63) == 0) most[tid >> 6] = amax;
        __syncthreads();
        amax = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));

        float scale = amax / kLargest<FMT>;
        int up = 0;                                    // doublings of the scale that the block had
        if (had > 0.f) {
            if (scale > had) {
                int en, eh;
                const float mn = frexpf(scale, &en), mh = frexpf(had, &eh);
                up = en - eh + (mn > mh);
            }
            scale = ldexpf(had, up);
        }
        if (!which && lo > 0 && up > 0) {              // keys that were there
            for (int i = id; i < lo * chunks; i += kThreads) {
                uint4* p = reinterpret_cast<uint4*>(codes + (i / lo) * 512 + (i % lo) * 16);
                const uint4 w = *p;
                *p = make_uint4(moved4<FMT>(w.x, up), moved4<FMT>(w.y, up), moved4<FMT>(w.z, up), moved4<FMT>(w.w, up));
            }
        }
#pragma unroll
        for (int n = 0; n < NI; ++n) {
            const int i = id + n * kThreads, r = i / chunks, chunk = i - r * chunks;
            if (i >= items) continue;
            uint32_t w[4] = {0, 0, 0, 0};
            if (scale > 0.f) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = code4<FMT>(v[n] + 4 * e, scale);
                    __builtin_amdgcn_sched_barrier(0); // sixteen divisions side by side would take all registers
                }
            }
            int x0;
            const int x1 = second_run(chunk, which || (!VEC && a.rot % 16) ? 0 : a.rot, a.interleaved, &x0);
            if (!which) {
                *reinterpret_cast<uint2*>(codes + (x0 >> 4) * 512 + (lo + r) * 16 + (x0 & 15)) = make_uint2(w[0], w[1]);
                *reinterpret_cast<uint2*>(codes + (x1 >> 4) * 512 + (lo + r) * 16 + (x1 & 15)) = make_uint2(w[2], w[3]);
            } else {
                uint8_t* to = turned + chunk * 16 * kPitch + place_of(lo + r);
#pragma unroll
                for (int e = 0; e < 16; ++e) to[e * kPitch] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
            }
        }
        if (which) {
            __syncthreads();
            for (int i = id; i < 2 * dim; i += kThreads) {            // 16 tokens of element i / 2
                const int h = i & 1;
                const uint32_t* fresh = reinterpret_cast<const uint32_t*>(turned + (i >> 1) * kPitch + h * 16);
                uint4* p = reinterpret_cast<uint4*>(codes) + i;
                uint32_t w[4] = {fresh[0], fresh[1], fresh[2], fresh[3]};
                if (lo > 0 || hi < kBlock) {           // values that were there, and what is no token's
                    const uint4 old = *p;
                    const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int t = token_of(h, 4 * e);
                        const uint32_t now = bytes_between(t, lo, hi), then = bytes_between(t, 0, lo);
                        const uint32_t before = up > 0 && then ? moved4<FMT>(o[e], up) : o[e];
                        w[e] = (w[e] & now) | (before & then) | (o[e] & ~(now | then));
                    }
                }
                *p = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        if (tid == 0) *scale_at = scale;
    }
}

// ---- read -------------------------------------------------------------------------
// Keys and values of a block back to rows, 16 elements of a token to a thread; values change places in LDS.  8192 tokens of
// 8 heads of 128 to BF16 (50 MB, much of it from the last-level cache) take 11 us, 8 at a copy's rate: a short launch's beginning
// and end, for the CUs hold waves 44% of that time.
template <typename T, int FMT> __global__ __launch_bounds__(kThreads) void k_read(ReadArgs a) {
    __shared__ __align__(16) uint8_t turned[256 * kPitch];
    const CacheArgs& c = a.c;
    const int dim = c.dim, tid = threadIdx.x, chunks = dim / 16;
    const int which = blockIdx.x & 1, head = (int)((blockIdx.x >> 1) % c.heads);
    T* to = static_cast<T*>(which ? a.v : a.k);
    if (!to) return;
    int seq, block;
    Span s;
    if (!slot_block(c, (blockIdx.x >> 1) / c.heads, &seq, &s, &block)) return;
    const int first = s.length - s.n;
    const int lo = max(first - block * kBlock, 0), hi = min(s.length - block * kBlock, kBlock);
    const int row0 = s.row + (block * kBlock - first);
    const int64_t at = block_at(c, seq, block, head);
    const uint4* codes = reinterpret_cast<const uint4*>(c.codes + at * (2 * kBlock * (int64_t)dim) + which * (kBlock * dim));
    const float scale = at < 0 ? 0.f : c.scales[at * 2 + which];
    if (which && at >= 0) {
        for (int i = tid; i < 2 * dim; i += kThreads) {
            const uint4 w = codes[i];
            uint32_t* p = reinterpret_cast<uint32_t*>(turned + (i >> 1) * kPitch + (i & 1) * 16);
            p[0] = w.x, p[1] = w.y, p[2] = w.z, p[3] = w.w;
        }
        __syncthreads();
    }
    for (int i = tid; i < (hi - lo) * chunks; i += kThreads) {
        const int r = i / chunks, chunk = i - r * chunks, t = lo + r;
        float v[16];
        if (at < 0) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
        } else {
            uint32_t w[4];
            if (which) {
                const uint8_t* p = turned + chunk * 16 * kPitch + place_of(t);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = p[4 * e * kPitch] | p[(4 * e + 1) * kPitch] << 8 | p[(4 * e + 2) * kPitch] << 16 | (uint32_t)p[(4 * e + 3) * kPitch] << 24;
            } else {
                const uint4 u = codes[chunk * 32 + t];
                w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = code_value<FMT>((w[e >> 2] >> (8 * (e & 3))) & 0xFFu) * scale;
        }
        T* out = to + ((int64_t)(row0 + t) * c.heads + head) * dim + chunk * 16;
#pragma unroll
        for (int u = 0; u < 16 / Vec<T>::N; ++u) {
            Vec<T> y;
#pragma unroll
            for (int e = 0; e < Vec<T>::N; ++e) y.e[e] = from_float<T>(v[u * Vec<T>::N + e]);
            reinterpret_cast<Vec<T>*>(out)[u] = y;
        }
    }
}

bool multiple(int64_t v, int64_t of) { return v % of == 0; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether a head's units of 16 bytes are whole: elements that turn, and their partners.
bool whole_units(int dim, int rot, bool interleaved, int v) {
    return multiple(dim, v) && multiple(interleaved ? rot : rot / 2, v) && multiple(dim - rot, v);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream) {
    const int v = a.dtype ? 8 : 4;
    const bool rows = multiple(a.dim, v) && aligned16(a.x) && aligned16(a.y) && multiple(a.ld_token, v) && multiple(a.ld_head, v) &&
                      multiple(a.ld_token_out, v) && multiple(a.ld_head_out, v);
    const bool vec = rows && whole_units(a.dim, a.rot, a.interleaved, v);
    // few elements that turn leave most to copy: 4 of 192 (3589 tokens of 35 heads BF16, 193 MB there and back)
    // take 50 us, 108 element by element
    const int edge = rows ? (a.rot + v - 1) / v * v : a.dim;
    const dim3 grid((unsigned)a.tokens);
#define IQ_ROTARY(T, INTER)                                                          \
    do {                                                                             \
        if (vec) k_rotary<T, INTER, true><<<grid, kThreads, 0, stream>>>(a, edge);   \
        else k_rotary<T, INTER, false><<<grid, kThreads, 0, stream>>>(a, edge);      \
    } while (0)
    if (a.dtype) {
        if (a.interleaved) IQ_ROTARY(uint16_t, true);
        else IQ_ROTARY(uint16_t, false);
    } else {
        if (a.interleaved) IQ_ROTARY(float, true);
        else IQ_ROTARY(float, false);
    }
#undef IQ_ROTARY
    return hipGetLastError();
}

hipError_t launch_cache_append(const AppendArgs& a, hipStream_t stream) {
    const CacheArgs& c = a.c;
    const int64_t slots = append_slots(c.tokens, c.batch, c.starts != nullptr);
    const int v = a.dtype ? 8 : 4;
    const bool vec_q = whole_units(c.dim, a.rot, a.interleaved, v) && aligned16(a.q) && aligned16(a.q_out) && multiple(a.ld_q_token, v) &&
                       multiple(a.ld_q_head, v);
    const auto whole = [&](const void* p, int64_t token, int64_t head) { return aligned16(p) && multiple(token, v) && multiple(head, v); };
    const bool vec = a.rot % 16 == 0 && whole(a.k, a.ld_k_token, a.ld_k_head) && whole(a.v, a.ld_v_token, a.ld_v_head);
    // Key heads of a workgroup share its cosines and sines: up to 8 where there are workgroups enough without.  8192
    // tokens of 8 key heads take 52.9 us with their read, 63.3 with a head each; one token 12.5, and 23.7 with 8.
    int per = (int)(slots * c.heads / 512);
    per = per < 1 ? 1 : per > 8 ? 8 : per;
    const int groups = (c.heads + per - 1) / per;
    const dim3 grid((unsigned)(slots * (groups + c.heads) + (a.q ? c.tokens : 0)));
    const size_t lds = (size_t)(a.rot / 2) * kBlock * sizeof(float2);
#define IQ_APPEND(T, FMT)                                                                                    \
    do {                                                                                                     \
        if (c.dim <= 128) {                                                                                  \
            if (vec) k_append<T, FMT, true, 1><<<grid, kThreads, lds, stream>>>(a, slots, per, vec_q);       \
            else k_append<T, FMT, false, 1><<<grid, kThreads, lds, stream>>>(a, slots, per, vec_q);          \
        } else {                                                                                             \
            if (vec) k_append<T, FMT, true, 2><<<grid, kThreads, lds, stream>>>(a, slots, per, vec_q);       \
            else k_append<T, FMT, false, 2><<<grid, kThreads, lds, stream>>>(a, slots, per, vec_q);          \
        }                                                                                                    \
    } while (0)
    if (a.dtype) {
        if (c.fmt) IQ_APPEND(uint16_t, 1);
        else IQ_APPEND(uint16_t, 0);
    } else {
        if (c.fmt) IQ_APPEND(float, 1);
        else IQ_APPEND(float, 0);
    }
#undef IQ_APPEND
    return hipGetLastError();
}

hipError_t launch_cache_read(const ReadArgs& a, hipStream_t stream) {
    const CacheArgs& c = a.c;
    const dim3 grid((unsigned)(append_slots(c.tokens, c.batch, c.starts != nullptr) * c.heads * 2));
    if (a.dtype) {
        if (c.fmt) k_read<uint16_t, 1><<<grid, kThreads, 0, stream>>>(a);
        else k_read<uint16_t, 0><<<grid, kThreads, 0, stream>>>(a);
    } else {
        if (c.fmt) k_read<float, 1><<<grid, kThreads, 0, stream>>>(a);
        else k_read<float, 0><<<grid, kThreads, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace iqk
