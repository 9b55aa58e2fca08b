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
// reduced to half a turn in 64 bits, so its error is 2^-53 of the angle, and
// 2^-25 of a turn once it is FP32.
__device__ __forceinline__ float2 turn(int position, double turns, float amplitude, float way) {
    double t = (double)position * turns;
    t -= __builtin_rint(t);
    float s, c;
    sincospif(2.f * (float)t, &s, &c);
    return make_float2(c * amplitude, s * (amplitude * way));
}

// Turns the heads [head0, head1) of one token.  cs: cosine and sine of its pairs, in LDS.
//   VEC: 16-byte units, where strides, bases and the ends of what turns are multiples of them.
template <typename T, bool INTER, bool VEC>
__device__ __forceinline__ void turn_token(const T* x, T* y, int64_t ldx, int64_t ldy, int head0, int head1, int dim, int rot,
                                           const float2* cs, int thread, int threads) {
    constexpr int V = VEC ? Vec<T>::N : 1;
    const int pairs = rot >> 1;
    const int turned = INTER ? (VEC ? rot / V : pairs) : pairs / V;     // units that hold pairs
    const int rest = x == y ? 0 : (dim - rot) / V;                        // units to copy
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
            const int at = rot + (u - turned) * V;
            if constexpr (VEC) *reinterpret_cast<Vec<T>*>(to + at) = *reinterpret_cast<const Vec<T>*>(from + at);
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

constexpr int kMostPairs = 512;

template <typename T, bool INTER, bool VEC> __global__ __launch_bounds__(kThreads) void k_rotary(RotaryArgs a) {
    __shared__ float2 cs[kMostPairs];
    const int t = blockIdx.x;
    const int position = a.positions[t];
    for (int p = threadIdx.x; p < a.rot / 2; p += kThreads) cs[p] = turn(position, a.table[p], a.amplitude, a.way);
    __syncthreads();
    turn_token<T, INTER, VEC>(static_cast<const T*>(a.x) + t * a.ld_token, static_cast<T*>(a.y) + t * a.ld_token_out, a.ld_head,
                              a.ld_head_out, 0, a.heads, a.dim, a.rot, cs, threadIdx.x, kThreads);
}

// ---- append -----------------------------------------------------------------------
template <typename T, int FMT> __global__ __launch_bounds__(kThreads) void k_append(AppendArgs a, int64_t slots, bool vec_q) {
    extern __shared__ __align__(16) float lds[];
    __shared__ float2 cs[128];
    __shared__ float most[kThreads / 64];
    const CacheArgs& c = a.c;
    const int dim = c.dim, pairs = a.rot >> 1, tid = threadIdx.x;
    const int64_t cache_work = slots * c.heads * 2;
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
            if (a.interleaved) turn_token<T, true, true>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, cs, tid, kThreads);
            else turn_token<T, false, true>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, cs, tid, kThreads);
        } else {
            if (a.interleaved) turn_token<T, true, false>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, cs, tid, kThreads);
            else turn_token<T, false, false>(x, y, a.ld_q_head, dim, 0, a.q_heads, dim, a.rot, cs, tid, kThreads);
        }
        return;
    }
    const int which = blockIdx.x & 1, head = (int)((blockIdx.x >> 1) % c.heads);
    int seq, block;
    Span s;
    if (!slot_block(c, (blockIdx.x >> 1) / c.heads, &seq, &s, &block)) return;
    const int64_t at = block_at(c, seq, block, head);
    if (at < 0) return;
    uint8_t* codes = c.codes + at * (2 * kBlock * (int64_t)dim) + which * (kBlock * dim);
    float* scale_at = c.scales + at * 2 + which;
    const int first = s.length - s.n;                  // position of the call's first token; may be negative
    const int lo = max(first - block * kBlock, 0), hi = min(s.length - block * kBlock, kBlock);      // new tokens of the block
    const float had = lo > 0 ? *scale_at : 0.f;

    // new rows to LDS
    const int pitch = dim + 1;
    const T* from = static_cast<const T*>(which ? a.v : a.k) + (int64_t)head * (which ? a.ld_v_head : a.ld_k_head);
    const int64_t ld = which ? a.ld_v_token : a.ld_k_token;
    const int row0 = s.row + (block * kBlock - first);   // row of the block's token 0
    for (int i = tid; i < (hi - lo) * dim; i += kThreads) {
        const int r = lo + i / dim, e = i % dim;
        lds[r * pitch + e] = to_float(from[(row0 + r) * ld + e]);
    }
    __syncthreads();
    if (!which && pairs > 0) {
        for (int i = tid; i < (hi - lo) * pairs; i += kThreads) {
            const int r = lo + i / pairs, p = i % pairs;
            const float2 t = turn(block * kBlock + r, a.table[p], a.amplitude, 1.f);
            float* pa = lds + r * pitch + (a.interleaved ? 2 * p : p);
            float* pb = a.interleaved ? pa + 1 : pa + pairs;
            const float x = *pa, y = *pb;
            *pa = x * t.x - y * t.y;
            *pb = y * t.x + x * t.y;
        }
        __syncthreads();
    }
    float amax = 0.f;
    for (int i = tid; i < (hi - lo) * dim; i += kThreads) {
        const float v = fabsf(lds[(lo + i / dim) * pitch + i % dim]);
        amax = v <= 3.402823466e+38f ? fmaxf(amax, v) : amax;      // neither NaN nor infinite
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) amax = fmaxf(amax, __shfl_xor(amax, d));
    if ((tid & 63) == 0) most[tid >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));

    float scale = amax / kLargest<FMT>;
    int up = 0;                                        // doublings of the scale that the block had
    if (had > 0.f) {
        if (scale > had) {
            int en, eh;
            const float mn = frexpf(scale, &en), mh = frexpf(had, &eh);
            up = en - eh + (mn > mh);
        }
        scale = ldexpf(had, up);
    }
    const auto code = [&](float v) { return scale > 0.f ? code_of<FMT>(v / scale) : 0u; };
    const auto moved = [&](uint32_t byte) { return code_of<FMT>(ldexpf(code_value<FMT>(byte & 0xFFu), -up)); };
    uint4* out = reinterpret_cast<uint4*>(codes);
    for (int i = tid; i < 2 * dim; i += kThreads) {    // 16 bytes each
        uint32_t w[4] = {0, 0, 0, 0};
        if (!which) {                                  // key: 16 elements of token t
            const int t = i & 31, e = (i >> 5) * 16;
            if (t >= hi || (t < lo && up == 0)) continue;
            if (t >= lo) {
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j >> 2] |= code(lds[t * pitch + e + j]) << (8 * (j & 3));
            } else {
                const uint4 old = out[i];
                const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
                for (int j = 0; j < 16; ++j) w[j >> 2] |= moved(o[j >> 2] >> (8 * (j & 3))) << (8 * (j & 3));
            }
        } else {                                       // value: 16 tokens of element e
            const int e = i >> 1, h = i & 1;
            uint4 old = make_uint4(0, 0, 0, 0);
            if (lo > 0 || hi < kBlock) old = out[i];
            const uint32_t o[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int t = token_of(h, j);
                uint32_t byte = (o[j >> 2] >> (8 * (j & 3))) & 0xFFu;
                if (t >= lo && t < hi) byte = code(lds[t * pitch + e]);
                else if (t < lo && up) byte = moved(byte);
                w[j >> 2] |= byte << (8 * (j & 3));
            }
        }
        out[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tid == 0) *scale_at = scale;
}

// ---- read -------------------------------------------------------------------------
template <typename T, int FMT> __global__ __launch_bounds__(kThreads) void k_read(ReadArgs a) {
    __shared__ uint8_t values[256 * 33];
    const CacheArgs& c = a.c;
    const int dim = c.dim, tid = threadIdx.x;
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
    const uint8_t* codes = c.codes + at * (2 * kBlock * (int64_t)dim) + which * (kBlock * dim);
    const float scale = at < 0 ? 0.f : c.scales[at * 2 + which];
    if (which && at >= 0) {
        for (int i = tid; i < kBlock * dim; i += kThreads) values[(i >> 5) * 33 + (i & 31)] = codes[i];
    }
    __syncthreads();
    for (int i = tid; i < (hi - lo) * dim; i += kThreads) {
        const int t = lo + i / dim, e = i % dim;
        uint32_t byte = 0;
        if (at >= 0) byte = which ? values[e * 33 + place_of(t)] : codes[(e >> 4) * 512 + t * 16 + (e & 15)];
        to[((int64_t)(row0 + t) * c.heads + head) * dim + e] = from_float<T>(at < 0 ? 0.f : code_value<FMT>(byte) * scale);
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
    const bool vec = whole_units(a.dim, a.rot, a.interleaved, v) && aligned16(a.x) && aligned16(a.y) && multiple(a.ld_token, v) &&
                     multiple(a.ld_head, v) && multiple(a.ld_token_out, v) && multiple(a.ld_head_out, v);
    const dim3 grid((unsigned)a.tokens);
#define IQ_ROTARY(T, INTER)                                                          \
    do {                                                                             \
        if (vec) k_rotary<T, INTER, true><<<grid, kThreads, 0, stream>>>(a);         \
        else k_rotary<T, INTER, false><<<grid, kThreads, 0, stream>>>(a);            \
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
    const bool vec = whole_units(c.dim, a.rot, a.interleaved, v) && aligned16(a.q) && aligned16(a.q_out) && multiple(a.ld_q_token, v) &&
                     multiple(a.ld_q_head, v);
    const dim3 grid((unsigned)(slots * c.heads * 2 + (a.q ? c.tokens : 0)));
    const size_t lds = (size_t)kBlock * (c.dim + 1) * sizeof(float);
    if (a.dtype) {
        if (c.fmt) k_append<uint16_t, 1><<<grid, kThreads, lds, stream>>>(a, slots, vec);
        else k_append<uint16_t, 0><<<grid, kThreads, lds, stream>>>(a, slots, vec);
    } else {
        if (c.fmt) k_append<float, 1><<<grid, kThreads, lds, stream>>>(a, slots, vec);
        else k_append<float, 0><<<grid, kThreads, lds, stream>>>(a, slots, vec);
    }
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
