// Attention over the paged 8-bit cache.
//
// A wave takes 16 or 32 columns: neighbouring (token, query head) pairs of one
// key head, so that the heads that share a key head read its codes once.  For
// every block of 32 tokens it forms the scores S^T = K Q^T and the running
// output O^T += V^T P^T on the matrix cores (FP16, 32 x 32 x 16 or 16 x 16 x
// 32).  In both results a lane holds one column, so maxima, sums and scales
// are its own, and the tokens that a lane holds of S^T are those that it feeds
// to the second product: the order of the cache's values makes them match.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "iq_attend.h"
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

// Probabilities are relative to a running maximum m that follows the scores
// once one is 2^kSlack past it, so a block rarely costs a rescaling of the
// output.  What the matrix cores take is a probability times its block's values scale, over the largest such product
// 2^(m + z) so far, which is followed as m is: blocks that a column does not see, or sees with next to no probability, take
// no digits from the others.  It is held times 2^kLift: at most 2^15 in FP16, with all digits from 2^-23 of the
// largest product on and steps of 2^-33 of that below.
constexpr float kSlack = 6.f, kLift = 9.f;

// From a maximum of this size on, FP32 steps of an exponent are no small part of 1: scores are taken less the maximum
// before anything is added to them.
constexpr float kFar = 0x1p20f;

// Log2 of a block's values scale over 2^z, at least: what FP16 leaves nothing of, and FP32 enough for the sum, so that
// blocks of small values or none (scale 0) still count in it.
constexpr float kLeastRatio = -60.f, kMostRatio = 1000.f;                 // at most: 2^z is 0 until a value other than 0 is seen

// How the lanes of a wave share a block and C columns.  Lane group g = lane / C
// holds column lane % C.
//   C = 32: scores r = 0 .. 15 are tokens 8 (r / 4) + 4 g + r % 4; fragment f of
//     keys and queries holds elements 32 (f / 2) + 16 g + 8 (f % 2) + 0 .. 7;
//     output tile i, register r is element 32 i + 8 (r / 4) + 4 g + r % 4.
//   C = 16: scores r = 0 .. 7 are tokens 16 (g % 2) + 8 (r / 4) + 4 (g / 2) + r % 4 (the rows of the two
//     score tiles are taken in the order that makes them 8 neighbouring places of the values);
//     fragment f holds elements 64 (f / 2) + 16 g + 8 (f % 2) + 0 .. 7, the last of an odd number 64 (f / 2) + 8 g + 0 .. 7;
//     output tile i, register r is element 16 i + 4 g + r.
template <int D, int C> struct Shape {
    static constexpr int kGroups = 64 / C, kScores = C / 2, kFragments = C == 32 ? D / 16 : D / 32, kSteps = C == 32 ? 2 : 1;
    static constexpr int kTiles = D / C, kPerTile = C * C / 64;      // output tiles and their registers
    using Tile = __attribute__((ext_vector_type(kPerTile))) float;

    static __device__ __forceinline__ int token(int g, int r) {
        return C == 32 ? 8 * (r >> 2) + 4 * g + (r & 3) : 16 * (g & 1) + 8 * (r >> 2) + 4 * (g >> 1) + (r & 3);
    }
    static __device__ __forceinline__ int element(int g, int f) {
        if (C == 32) return 32 * (f >> 1) + 16 * g + 8 * (f & 1);
        return f + 1 == kFragments && kFragments % 2 ? 64 * (f >> 1) + 8 * g : 64 * (f >> 1) + 16 * g + 8 * (f & 1);
    }
    static __device__ __forceinline__ int output(int g, int i, int r) {
        return C == 32 ? 32 * i + 8 * (r >> 2) + 4 * g + (r & 3) : 16 * i + 4 * g + r;
    }
    static __device__ __forceinline__ float over_groups(float v, bool sum) {
#pragma unroll
        for (int d = C; d < 64; d <<= 1) {
            const float u = __shfl_xor(v, d);
            v = sum ? v + u : fmaxf(v, u);
        }
        return v;
    }
};

// The codes of a block that a lane feeds to the matrix cores.
template <int D, int FMT, int C> struct Codes {
    using S = Shape<D, C>;
    static constexpr int kKeys = C == 32 ? D / 32 : 2 * (D / 64), kRest = C == 16 && D % 64 ? 2 : 0, kValues = C == 32 ? D / 32 : D / 16;
    using Value = typename std::conditional<C == 32, uint4, uint2>::type;
    uint4 k[kKeys];
    uint2 rest[kRest + 1];
    Value v[kValues];

    __device__ __forceinline__ void fetch_keys(const uint8_t* block, int lane) {
        const uint4* p = reinterpret_cast<const uint4*>(block);
        const int g = lane / C;
        if constexpr (C == 32) {
#pragma unroll
            for (int j = 0; j < kKeys; ++j) k[j] = p[(2 * j + g) * 32 + (lane & 31)];
        } else {
            const int row = lane & 15, token = 16 * ((row >> 2) & 1) + 4 * (row >> 3) + (row & 3);
#pragma unroll
            for (int j = 0; j < kKeys; ++j) k[j] = p[(4 * (j >> 1) + g) * 32 + 8 * (j & 1) + token];
            if constexpr (kRest) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    rest[t] = reinterpret_cast<const uint2*>(p + (D / 64 * 4 + (g >> 1)) * 32 + 8 * t + token)[g & 1];
            }
        }
    }
    __device__ __forceinline__ void fetch_values(const uint8_t* block, int lane) {
        const Value* p = reinterpret_cast<const Value*>(block + kBlock * D);
#pragma unroll
        for (int j = 0; j < kValues; ++j) v[j] = p[(C * j + (lane & (C - 1))) * S::kGroups + lane / C];
    }
    // Values of tokens from `keep` on (of the block), which may be anything, as zeros.
    __device__ __forceinline__ void keep_values(int g, int keep) {
#pragma unroll
        for (int j = 0; j < kValues; ++j) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&v[j]);
#pragma unroll
            for (int i = 0; i < S::kScores / 4; ++i) {
                const int n = keep - S::token(g, 4 * i);       // bytes of this word that are the sequence's
                w[i] &= n <= 0 ? 0u : n >= 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
            }
        }
    }
    // Scores of the lane's tokens: codes times FP16 queries.
    __device__ __forceinline__ void scores(const half8* q, float* s) const {
        if constexpr (C == 32) {
            float16v x = 0.f;
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(k[j].x, k[j].y), q[2 * j], x, 0, 0, 0);
                x = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(k[j].z, k[j].w), q[2 * j + 1], x, 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = x[r];
        } else {
            float4v x[2] = {0.f, 0.f};
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
                x[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(expand8<FMT>(k[j].x, k[j].y), q[j >> 1 << 1], x[j & 1], 0, 0, 0);
                x[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(expand8<FMT>(k[j].z, k[j].w), q[(j >> 1 << 1) + 1], x[j & 1], 0, 0, 0);
            }
            if constexpr (kRest) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    x[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(expand8<FMT>(rest[t].x, rest[t].y), q[S::kFragments - 1], x[t], 0, 0, 0);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) s[r] = x[r >> 2][r & 3];
        }
    }
    __device__ __forceinline__ void add_values(const half8* p, typename S::Tile* o) const {
#pragma unroll
        for (int j = 0; j < kValues; ++j) {
            if constexpr (C == 32) {
                o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(v[j].x, v[j].y), p[0], o[j], 0, 0, 0);
                o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(v[j].z, v[j].w), p[1], o[j], 0, 0, 0);
            } else {
                o[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(expand8<FMT>(v[j].x, v[j].y), p[0], o[j], 0, 0, 0);
            }
        }
    }
};

// Queries of a column as the matrix cores take them: FP16 times a power of two
// that brings the row's largest into [2^14, 2^15), and the factor that makes
// scores exponents of 2.
template <int D, int C> __device__ __forceinline__ float load_query(float scale, const uint16_t* row, int g, half8* q) {
    using S = Shape<D, C>;
    uint4 raw[S::kFragments];
    uint32_t top = 0;
#pragma unroll
    for (int f = 0; f < S::kFragments; ++f) raw[f] = *reinterpret_cast<const uint4*>(row + S::element(g, f));
#pragma unroll
    for (int f = 0; f < S::kFragments; ++f)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&raw[f])[e];
            top = max(top, max((w << 16) & 0x7FFFFFFFu, w & 0x7FFF0000u));
        }
#pragma unroll
    for (int d = C; d < 64; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d));
    // a query that is not finite answers NaN where it sees anything: all its elements are
    const uint32_t bad = top >= 0x7F800000u ? 0xFFFFFFFFu : 0u;
    int e = (int)(top >> 23);                          // 0 for zeros and subnormals, 255 for infinities and NaN
    e = e == 255 ? 0 : max(e, 1) - 127 - 14;
#pragma unroll
    for (int f = 0; f < S::kFragments; ++f) {
        union { half8 v; uint32_t w[4]; } u;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&raw[f])[k >> 1];
            u.v[k] = (_Float16)ldexpf(__uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16), -e);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) u.w[k] |= bad;
        q[f] = u.v;
    }
    return ldexpf(scale * 1.44269504f, e);
}

// Log2 of a scale, subnormal ones too; -inf of 0.
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(x)) + (float)__builtin_amdgcn_frexp_expf(x); }

// Running state of a column: maximum, sum of this lane's tokens' probabilities over 2^m, output over 2^(m + z - kLift).
template <int D, int C> struct State {
    using S = Shape<D, C>;
    typename S::Tile o[S::kTiles];
    float m, l, z;
    int far;                     // whether some column's m is past kFar

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < S::kTiles; ++j) o[j] = 0.f;
        m = z = -INFINITY;
        l = 0.f;
        far = 0;
    }
    // The largest of the lane's scores, as an exponent of 2.
    static __device__ __forceinline__ float top_of(const float* s, float fk) {
        float top = s[0];
#pragma unroll
        for (int r = 1; r < S::kScores; ++r) top = fmaxf(top, s[r]);
        return top * fk;
    }
    // Whether a maximum is behind the block's; scale_v is the log2 of the block's values scale.  Nothing seen, so far and here, is NaN: no.
    __device__ __forceinline__ bool behind(float top, float scale_v) const {
        const float past = top - m;
        return __any(past > kSlack || past + scale_v > z + kSlack);
    }
    // Brings both up to the block's.  Rare.
    __device__ __forceinline__ void catch_up(float top, float scale_v) {
        top = S::over_groups(top, false);
        const float now = fmaxf(m, top), fall = now == m ? 0.f : m - now, was = z + fall;
        z = fmaxf(was, top - now + scale_v);
        m = now;
        far = __builtin_amdgcn_readfirstlane(__any(fabsf(now) >= kFar && now > -INFINITY));
        l *= exp2_fast(fall);
        const float by = z == was ? 1.f : exp2_fast(was - z);
#pragma unroll
        for (int j = 0; j < S::kTiles; ++j) o[j] *= by;
    }
    static __device__ __forceinline__ float least(float m) { return fmaxf(m, -3.402823466e+38f); }       // m is -inf until a token is seen
    // What turns a block's scores into what the second product takes: factor and offset of the exponents, their running
    // sum, and what makes a sum of probabilities over 2^m of it.
    struct Exponent {
        float factor, offset, weight, sum;
    };
    __device__ __forceinline__ Exponent exponent(float* s, float fk, float scale_v) const {
        const float ratio = __builtin_amdgcn_fmed3f(scale_v - z, kLeastRatio, kMostRatio) + kLift;           // NaN, of 0 and 0: the least
        Exponent x = {fk, ratio - least(m), exp2_fast(-ratio), 0.f};
        if (far) {
#pragma unroll
            for (int r = 0; r < S::kScores; ++r) s[r] = s[r] * fk - least(m);
            x.factor = 1.f;
            x.offset = ratio;
        }
        return x;
    }
    // Elements r and r + 1, in the second product's order.  The sum is of what they are before FP16, which loses
    // those of a block whose values are small beside others'.
    __device__ __forceinline__ void probabilities(const float* s, int r, Exponent& x, half8* p) const {
        const float e0 = exp2_fast(__builtin_fmaf(s[r], x.factor, x.offset)), e1 = exp2_fast(__builtin_fmaf(s[r + 1], x.factor, x.offset));
        x.sum += e0;
        x.sum += e1;
        p[r >> 3][r & 7] = (_Float16)e0;
        p[r >> 3][(r & 7) + 1] = (_Float16)e1;
    }
    __device__ __forceinline__ void add(const Exponent& x) { l = __builtin_fmaf(x.sum, x.weight, l); }
    // What turns the output's registers into values over a sum of probabilities: a factor, and a power of two apart from
    // it, since z may be anything (-inf where all values are 0, and the output with them).
    struct Over {
        float by;
        int power;
    };
    __device__ __forceinline__ Over over(float by) const {
        const float whole = __builtin_rintf(fmaxf(z, -1e4f));
        return {by * exp2_fast(fmaxf(z, -1e4f) - whole), (int)(whole - kLift)};
    }
    static __device__ __forceinline__ float value(float x, const Over& to) { return __builtin_amdgcn_ldexpf(x * to.by, to.power); }
};

// Scores of lane group g whose tokens lie outside [from, to) become -inf; the block's token 0 is t0.
template <int D, int C> __device__ __forceinline__ void hide(float* s, int t0, int g, int from, int to) {
#pragma unroll
    for (int r = 0; r < Shape<D, C>::kScores; ++r) {
        const int token = t0 + Shape<D, C>::token(g, r);
        s[r] = token >= from && token < to ? s[r] : -INFINITY;
    }
}

// The factor of a block's scores, positive and finite, so that hidden ones stay -inf whatever the block's scale is.
__device__ __forceinline__ float factor_of(float fk) { return __builtin_amdgcn_fmed3f(fk, 1e-30f, 3e38f); }

// Values that a wave's lanes share, in scalar registers.
__device__ __forceinline__ int one(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ Tile one(const Tile& t) {
    Tile u;
    u.seq = one(t.seq); u.f0 = one(t.f0); u.columns = one(t.columns);
    u.s.row = one(t.s.row); u.s.n = one(t.s.n); u.s.length = one(t.s.length);
    return u;
}

// A block of a sequence: its number in the memory and its scales, through
// scalar loads, which do not wait for codes in flight.  An absent page's place is block 0,
// of which nothing is to be used.
struct Place {
    int64_t at;
    float raw_k, raw_v;
    bool absent;
    __device__ __forceinline__ float scale_k() const { return absent ? 1.f : raw_k; }
    __device__ __forceinline__ float scale_v() const { return absent ? 0.f : raw_v; }
};
template <typename T> using scalar_t = const __attribute__((address_space(4))) T*;
template <typename T> __device__ __forceinline__ T scalar_load(const T* p, int64_t i) {
    return ((scalar_t<T>)(uintptr_t)p)[i];
}
// The page that holds block b, as the table says.
__device__ __forceinline__ int page_of(const CacheArgs& c, int seq, int b) {
    return scalar_load(c.page_table, (int64_t)seq * c.width + (one(b) >> c.shift));
}
__device__ __forceinline__ Place place_in(const CacheArgs& c, int page, int b, int head) {
    Place p;
    p.absent = (uint32_t)page >= (uint32_t)c.pages;
    p.at = p.absent ? 0 : (((int64_t)page * c.heads + head) << c.shift) | (b & ((1 << c.shift) - 1));
    p.raw_k = scalar_load(c.scales, p.at * 2);
    p.raw_v = scalar_load(c.scales, p.at * 2 + 1);
    return p;
}
__device__ __forceinline__ Place place_at(const CacheArgs& c, int seq, int b, int head) {
    b = one(b);
    return place_in(c, page_of(c, seq, b), b, head);
}

// ---- sharing the work out ----------------------------------------------------------------
struct Share {
    int64_t at, end, per;        // units
    int64_t entry;               // that `at` lies in
    int64_t entry_begin;         // unit that the entry begins with, counting its head's
    int head;
};

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The share of workgroup `worker`; units(e) are those of entry e of `entries` for one head.
template <typename F>
__device__ __forceinline__ Share share_of(int worker, int workers, int heads, int64_t entries, int least, const F& units) {
    __shared__ int64_t sums[kWaves], counts[kWaves], found[2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t first = threadIdx.x < entries ? units(threadIdx.x) : 0, mine = first, some = first > 0;
    for (int64_t e = threadIdx.x + kThreads; e < entries; e += kThreads) {
        const int64_t u = units(e);
        mine += u;
        some += u > 0;
    }
    mine = wave_sum(mine);
    some = wave_sum(some);
    if (lane == 0) sums[wave] = mine, counts[wave] = some;
    __syncthreads();
    const int64_t one_head = sums[0] + sums[1] + sums[2] + sums[3], total = one_head * heads;
    Share s;
    s.per = share_size(total, workers, one_head, counts[0] + counts[1] + counts[2] + counts[3], least);
    s.at = worker * s.per;
    s.end = min(s.at + s.per, total);
    if (s.at >= total) return s;
    s.head = (int)(s.at / one_head);
    const int64_t into = s.at - s.head * one_head;
    int64_t before = 0;                                // units of the entries before the current 256
    for (int64_t base = 0; base < entries; base += kThreads) {
        const int64_t e = base + threadIdx.x, v = base == 0 ? first : e < entries ? units(e) : 0;
        int64_t upto = v;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t u = __shfl_up(upto, d);
            upto += lane >= d ? u : 0;
        }
        __syncthreads();
        if (lane == 63) sums[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; ++w) upto += sums[w];
        upto += before;
        if (into >= upto - v && into < upto) {
            found[0] = e;
            found[1] = upto - v;
        }
        before += sums[0] + sums[1] + sums[2] + sums[3];
        if (into < before) break;
    }
    __syncthreads();
    s.entry = found[0];
    s.entry_begin = s.head * one_head + found[1];
    return s;
}

// ---- few columns: the work is the cache's codes ------------------------------------------
// A workgroup's four waves take a row's blocks in turn, each with the next
// block's codes in flight, and join their outputs through LDS.  Codes go from memory to registers in the order in which
// the matrix cores take them, so LDS holds none, and waves wait for nothing but their own loads.
// HBM bounds it: 64 sequences of 1024 to 16384 tokens (8 key heads of 128, 1.14 GB of codes) take 202 us, 5.6 TB/s
// (a large read: 5.8 to 7.0); one of 131072 tokens (268 MB) 52 us, 5.2 TB/s, and 7 for the join.  Fetching two blocks
// ahead is slower by 1% (its registers), and so are 32 columns where 16 are enough (`few_columns`).

template <int D, int FMT, int C, bool DIRECT> __global__ __launch_bounds__(kThreads, few_waves(D, C)) void k_few(AttendArgs a, Plan plan) {
    using S = Shape<D, C>;
    constexpr int R = D * C / 64;                      // registers of the output
    __shared__ float other[2][kWaves * C];             // maxima and sums of the waves
    __shared__ float pass[2 * R * 64];                 // outputs on their way to another wave
    const int lane = threadIdx.x & 63, wave = one(threadIdx.x >> 6), col = lane & (C - 1), g = lane / C;
    Share share;
    int seq, tile = 0;
    Span span;
    if constexpr (DIRECT) {                            // a workgroup for each row
        seq = blockIdx.x % a.c.batch;                  // tiles that few sequences have come last: they leave no XCD without work
        tile = blockIdx.x / a.c.batch;
        span = span_of(a.c, seq);
        if (!takes(a, plan, span) || (int64_t)tile * C >= (int64_t)span.n * a.group) return;
        share.head = blockIdx.y;
    } else {
        Open* open = reinterpret_cast<Open*>(static_cast<char*>(a.workspace) + plan.opens);
        share = share_of(blockIdx.x, plan.workers, a.c.heads, a.c.batch, kLeastShare, [&](int64_t e) { return units_of<C>(a, plan, (int)e); });
        if (threadIdx.x == 0) open[blockIdx.x].columns = 0;
        if (share.at >= share.end) return;
        seq = one((int)share.entry);
        share.head = one(share.head);
        span = span_of(a.c, seq);
    }
    int64_t row_begin = DIRECT ? 0 : share.entry_begin;                // unit that the row begins with
    bool opening = true;                               // the share's first row

    while (true) {
        if (!DIRECT) {
            if (share.at >= share.end) break;
            if ((int64_t)tile * C >= (int64_t)span.n * a.group || !takes(a, plan, span)) {     // the next sequence, or head
                if (++seq == a.c.batch) {
                    seq = 0;
                    if (++share.head >= a.c.heads) break;              // the arrays changed meanwhile
                }
                tile = 0;
                span = span_of(a.c, seq);
                continue;
            }
        }
        const Tile t = one(tile_at(a, C, seq, span, tile));
        const View v = view_of(a, t);
        const int units = max(v.blocks, 1), head = share.head;
        if (!DIRECT && opening && share.at >= row_begin + units) {     // the share begins in a later row of its sequence
            row_begin += units;
            ++tile;
            continue;
        }
        const int skip = DIRECT ? 0 : one((int)min(max(share.at - row_begin, (int64_t)0), (int64_t)units));
        const int take = DIRECT ? units : one((int)min((int64_t)(units - skip), share.end - share.at));
        const bool whole = take == units;
        const int b0 = v.block + min(skip, v.blocks), b1 = v.block + min(skip + take, v.blocks);

        Codes<D, FMT, C> codes;
        Place now = {};
        const auto block_codes = [&](const Place& p) { return a.c.codes + p.at * (2 * kBlock * (int64_t)D); };
        if (b0 + wave < b1) {
            now = place_at(a.c, t.seq, b0 + wave, head);
            codes.fetch_keys(block_codes(now), lane);
            codes.fetch_values(block_codes(now), lane);
        }
        const Column c = column_of(a, t, v, col);
        half8 q[S::kFragments];
        const float factor = load_query<D, C>(
            a.scale, static_cast<const uint16_t*>(a.q) + c.row * a.ld_token + ((int64_t)head * a.group + c.head) * a.ld_head, g, q);
        State<D, C> st;
        st.clear();
        // Keys of the wave's next block are fetched once the scores of this one are formed, values after its output.
        // Past the last block the last one is fetched again; absent pages stand for a page that nothing is seen of.
        for (int b = b0 + wave; b < b1; b += kWaves) {
            const Place next = place_at(a.c, t.seq, min(b + kWaves, b1 - 1), head);
            const int t0 = b * kBlock;
            const float fk = factor_of(factor * now.scale_k()), scale_v = log2_of(now.scale_v());
            float s[S::kScores];
            codes.scores(q, s);
            codes.fetch_keys(block_codes(next), lane);
            if (now.absent || t0 + kBlock > v.each_to || t0 < v.each_from) hide<D, C>(s, t0, g, c.from, now.absent ? 0 : c.to);
            const float top = st.top_of(s, fk);
            if (st.behind(top, scale_v)) st.catch_up(top, scale_v);
            half8 p[S::kSteps];
            typename State<D, C>::Exponent ex = st.exponent(s, fk, scale_v);
#pragma unroll
            for (int r = 0; r < S::kScores; r += 2) st.probabilities(s, r, ex, p);
            st.add(ex);
            if (now.absent || t0 + kBlock > v.keys) codes.keep_values(g, now.absent ? 0 : v.keys - t0);
            codes.add_values(p, st.o);
            codes.fetch_values(block_codes(next), lane);
            now = next;
        }
        const float l = S::over_groups(st.l, true);

        // join the four waves: each output over the sum of all, weighted by its maximum
        other[0][wave * C + col] = st.m;
        other[1][wave * C + col] = l;
        __syncthreads();
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, other[0][w * C + col]);
        const auto weight = [&](float m) { return m == top ? 1.f : exp2_fast(m - top); };
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += other[1][w * C + col] * weight(other[0][w * C + col]);
        // sums are positive unless nothing was seen; NaN passes through
        const auto part_share = st.over(l == 0.f ? 0.f : weight(st.m) / sum);
#pragma unroll
        for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
            for (int r = 0; r < S::kPerTile; ++r) st.o[j][r] = l == 0.f ? 0.f : st.value(st.o[j][r], part_share);
#pragma unroll
        for (int round = kWaves / 2; round; round >>= 1) {
            float* mail = pass + (wave & (round - 1)) * R * 64;
            if (wave >= round && wave < 2 * round) {
#pragma unroll
                for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
                    for (int r = 0; r < S::kPerTile; ++r) mail[(j * S::kPerTile + r) * 64 + lane] = st.o[j][r];
            }
            __syncthreads();
            if (wave < round) {
#pragma unroll
                for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
                    for (int r = 0; r < S::kPerTile; ++r) st.o[j][r] += mail[(j * S::kPerTile + r) * 64 + lane];
            }
            if (!DIRECT || round > 1) __syncthreads();
        }
        if (wave == 0 && col < t.columns) {
            uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)c.row * a.q_heads + (int64_t)head * a.group + c.head) * D;
            float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan.parts) +
                          (blockIdx.x * 2 + (opening ? 0 : 1)) * part_floats(D, C);
#pragma unroll
            for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
                for (int r = 0; r < S::kPerTile; r += 4) {
                    const int d = S::output(g, j, r);
                    if (DIRECT || whole) {
                        union { __bf16 b[4]; uint2 w; } u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) u.b[e] = (__bf16)st.o[j][r + e];
                        *reinterpret_cast<uint2*>(out + d) = u.w;
                    } else {
                        *reinterpret_cast<float4v*>(part + col * D + d) = (float4v){st.o[j][r], st.o[j][r + 1], st.o[j][r + 2], st.o[j][r + 3]};
                    }
                }
            if (!DIRECT && !whole && g == 0) {
                part[C * D + col] = top;
                part[C * (D + 1) + col] = sum;
            }
        }
        if constexpr (DIRECT) {
            break;
        } else {
            if (!whole && skip == 0 && threadIdx.x == 0) {             // the row begins here and goes on
                Open* open = reinterpret_cast<Open*>(static_cast<char*>(a.workspace) + plan.opens);
                open[blockIdx.x] = {row_begin, share.per, t.s.row, t.f0, t.columns, head, (int)((row_begin + units - 1) / share.per), 0};
            }
            share.at += take;
            row_begin += units;
            ++tile;
            opening = false;
        }
    }
}

// Joins the parts of the row that workgroup blockIdx.x began and others went
// on with, a column at a time: parts' weights in LDS first, then D / 4 threads for each of
// several parts at a time.
template <int D, int C> __global__ __launch_bounds__(kThreads) void k_join(AttendArgs a, Plan plan) {
    constexpr int Q = D / 4, P = kThreads / Q;         // threads of a part, parts at a time
    __shared__ float weights[kThreads], reduced[2][kWaves];
    __shared__ float4v sums[P][Q];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Open open = reinterpret_cast<const Open*>(static_cast<const char*>(a.workspace) + plan.opens)[blockIdx.x];
    const float* parts = reinterpret_cast<const float*>(static_cast<const char*>(a.workspace) + plan.parts);
    const int many = open.last - (int)blockIdx.x + 1;
    const auto part_of = [&](int k) {
        const int64_t w = blockIdx.x + k;
        return parts + (w * 2 + part_index(w, open.per, open.begin)) * part_floats(D, C);
    };
    const int p = threadIdx.x / Q, x = threadIdx.x % Q;
    for (int col = blockIdx.y; col < open.columns; col += gridDim.y) {
        float top = -INFINITY, total = 0.f;
        float4v sum = 0.f;
        for (int base = 0; base < many; base += kThreads) {                // one round up to 256 parts
            const int n = min(many - base, kThreads);
            float m = -INFINITY, l = 0.f;
            if (threadIdx.x < n) {
                const float* q = part_of(base + threadIdx.x);
                m = q[C * D + col];
                l = q[C * (D + 1) + col];
            }
            float now = m;
#pragma unroll
            for (int d = 32; d; d >>= 1) now = fmaxf(now, __shfl_xor(now, d));
            if (lane == 0) reduced[0][wave] = now;
            __syncthreads();
            now = fmaxf(top, fmaxf(fmaxf(reduced[0][0], reduced[0][1]), fmaxf(reduced[0][2], reduced[0][3])));
            const float weight = l == 0.f ? 0.f : (m == now ? 1.f : exp2_fast(m - now)) * l;       // 0: nothing seen there
            weights[threadIdx.x] = weight;
            float added = weight;
#pragma unroll
            for (int d = 32; d; d >>= 1) added += __shfl_xor(added, d);
            if (lane == 0) reduced[1][wave] = added;
            __syncthreads();
            const float alpha = now == top ? 1.f : exp2_fast(top - now);
            top = now;
            total = total * alpha + (reduced[1][0] + reduced[1][1] + reduced[1][2] + reduced[1][3]);
            sum *= alpha;
            if (p < P) {
#pragma unroll 8
                for (int k = p; k < n; k += P) {
                    const float w = weights[k];
                    const float4v o = *reinterpret_cast<const float4v*>(part_of(base + k) + col * D + 4 * x);
                    sum += w == 0.f ? (float4v)0.f : o * w;
                }
            }
            __syncthreads();
        }
        if (p < P) sums[p][x] = sum;
        __syncthreads();
        if (p == 0) {
#pragma unroll
            for (int k = 1; k < P; ++k) sum += sums[k][x];
            const int f = open.f0 + col, i = f / a.group, gh = f - i * a.group, row = open.row + i;
            uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)row * a.q_heads + (int64_t)open.head * a.group + gh) * D;
            union { __bf16 b[4]; uint2 w; } u;
#pragma unroll
            for (int e = 0; e < 4; ++e) u.b[e] = (__bf16)(total == 0.f ? 0.f : sum[e] / total);
            *reinterpret_cast<uint2*>(out + 4 * x) = u.w;
        }
        __syncthreads();
    }
}

// ---- many columns: the work is products ----------------------------------------------------
// A workgroup takes 128 columns, 32 to a wave.  Its waves turn a block's codes
// into FP16 once, in LDS and in the order in which the matrix cores take them; two blocks are there, one read, one made.
// The issue of instructions bounds it: for a block of 32 tokens a wave of 128 elements has 16 products (512 cycles of a
// SIMD's matrix core) and about 125 vector instructions beside them (570 cycles: conversion, maxima, exponentials,
// rounding), and takes 1240 cycles.  So the matrix cores are busy 41% of the time and the vector units 45%: the two waves of a SIMD
// hardly overlap one's products with the other's vector work.  A prompt of 8192 tokens (32 heads of 128 on 8; 550 GFLOP)
// takes 590 to 650 us from card to card, 0.85 to 0.93 PFLOP/s, and 20 for the join.  Priority for the wave in its products gains 5%; rows
// in the order of `row_at` 12%; 64 columns a wave cost their output registers' copies (1506 us), three LDS buffers 690 to 723 against 698.
template <int D, int FMT> __global__ __launch_bounds__(kThreads, many_waves(D)) void k_many(AttendArgs a, Plan plan) {
    using S = Shape<D, 32>;
    constexpr int C = kManyColumns, J = D / 32, F = D / 16, N = (J + kWaves - 1) / kWaves;
    constexpr int kAhead = 3;                          // fragments read before their products (with 5: 1% slower)
    __shared__ Tile tiles[64];
    __shared__ half8 stage[2][2][F][64];               // [buffer][keys, values][fragment][lane]
    const int lane = threadIdx.x & 63, wave = one(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    Open* open = reinterpret_cast<Open*>(static_cast<char*>(a.workspace) + plan.opens);
    // workgroups of one XCD, every eighth, take neighbouring shares: of few key heads, whose codes then stay in its L2
    const int worker = (blockIdx.x % 8) * (plan.workers / 8) + blockIdx.x / 8;
    Share share = share_of(worker, plan.workers, a.c.heads, plan.slots, kLeastManyShare, [&](int64_t e) -> int64_t {
        Tile t;
        return row_at(a, plan, e, &t) ? max(view_of(a, t).blocks, 1) : 0;
    });
    if (threadIdx.x == 0) open[worker].columns = 0;
    if (share.at >= share.end) return;
    int64_t entry = share.entry, row_begin = share.entry_begin;        // an entry is one row
    int64_t known = entry - 64;                        // 64 entries from here on are in `tiles`
    uint64_t rows = 0;
    int head = one(share.head);
    bool opening = true;

    while (share.at < share.end) {
        // the next entry that is a row: of 64 at a time, looked up together; sequences of few columns have entries that are none
        if (entry >= known + 64) {
            known = entry;
            Tile u;
            const bool some = known + lane < plan.slots && row_at(a, plan, known + lane, &u);
            rows = __ballot(some);
            __syncthreads();                           // the row before is done with what it read
            if (wave == 0 && some) tiles[lane] = u;
            __syncthreads();
        }
        const uint64_t left = rows >> (entry - known);
        if (!left) {
            entry = known + 64;
            if (entry >= plan.slots) {
                entry = 0;
                known = -64;
                if (++head >= a.c.heads) break;        // the arrays changed meanwhile
            }
            continue;
        }
        entry += __builtin_ctzll(left);
        const Tile t = one(tiles[entry - known]);
        const View v = view_of(a, t);
        const int units = max(v.blocks, 1), skip = one((int)min(max(share.at - row_begin, (int64_t)0), (int64_t)units));
        const int take = one((int)min((int64_t)(units - skip), share.end - share.at));
        const bool whole = take == units;
        const int b0 = v.block + min(skip, v.blocks), b1 = v.block + min(skip + take, v.blocks);

        // the wave's columns, and what they see
        const int c0 = wave * 32;
        Tile mine = t;
        mine.f0 += c0;
        mine.columns = min(t.columns - c0, 32);
        View w = {};
        if (mine.columns > 0) w = view_of(a, mine);
        const int each_from = one(w.each_from), each_to = one(w.each_to), keys = one(v.keys);
        const Column c = column_of(a, t, v, c0 + col);

        uint4 kc[N], vc[N];
        const auto fetch = [&](const Place& p) {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                const int j = wave + kWaves * n;
                if (J % kWaves == 0 || j < J) {
                    const uint4* codes = reinterpret_cast<const uint4*>(a.c.codes + p.at * (2 * kBlock * (int64_t)D));
                    kc[n] = codes[(2 * j + h) * 32 + col];
                    vc[n] = codes[2 * D + (32 * j + col) * 2 + h];
                }
            }
        };
        // Codes that are no token's may be anything: zeros.
        const auto keep_tail = [&](int b, const Place& p) {
            const int keep = p.absent ? 0 : keys - b * kBlock;
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = keep - S::token(h, 4 * i);
                    reinterpret_cast<uint32_t*>(&vc[n])[i] &= m <= 0 ? 0u : m >= 4 ? 0xFFFFFFFFu : (1u << (8 * m)) - 1u;
                }
        };
        // Eight codes of the wave's part: a quarter of each of its N pieces.
        const auto turn = [&](int buffer, int u) {
            const int n = u >> 2, j = wave + kWaves * n, e = u & 1;
            if (J % kWaves == 0 || j < J) {
                const uint4& w = u & 2 ? vc[n] : kc[n];
                stage[buffer][(u >> 1) & 1][2 * j + e][lane] = e ? expand8<FMT>(w.z, w.w) : expand8<FMT>(w.x, w.y);
            }
        };
        const auto fill = [&](int buffer, int b, const Place& p) {
            if (p.absent || keys < (b + 1) * kBlock) keep_tail(b, p);
#pragma unroll
            for (int u = 0; u < 4 * N; ++u) turn(buffer, u);
        };
        Place now = {}, next = {};
        if (b0 < b1) {
            now = place_at(a.c, t.seq, b0, head);
            fetch(now);
        }
        half8 q[F];
        const float factor = load_query<D, 32>(
            a.scale, static_cast<const uint16_t*>(a.q) + c.row * a.ld_token + ((int64_t)head * a.group + c.head) * a.ld_head, h, q);
        State<D, 32> st;
        st.clear();
        if (b0 < b1) {
            fill(0, b0, now);
            next = place_at(a.c, t.seq, min(b0 + 1, b1 - 1), head);
            fetch(next);
            int page = page_of(a.c, t.seq, min(b0 + 2, b1 - 1));
            __syncthreads();
            int buffer = 0;
            for (int b = b0; b < b1; ++b) {
                const int t0 = b * kBlock;
                const float fk = factor_of(factor * now.scale_k()), scale_v = log2_of(now.scale_v());
                half8 y[2 * F];                        // fragments of keys, then of values
                const auto read = [&](int i) { y[i] = stage[buffer][i >= F][i >= F ? i - F : i][lane]; };
#pragma unroll
                for (int i = 0; i < kAhead; ++i) read(i);
                if (next.absent || keys < (b + 2) * kBlock) keep_tail(b + 1, next);
                __builtin_amdgcn_s_setprio(1);
                float16v x = 0.f;
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    if (i + kAhead < 2 * F) read(i + kAhead);
                    x = __builtin_amdgcn_mfma_f32_32x32x16_f16(y[i], q[i], x, 0, 0, 0);
#pragma unroll
                    for (int u = 4 * N * i / F; u < 4 * N * (i + 1) / F; ++u) turn(buffer ^ 1, u);
                    __builtin_amdgcn_sched_barrier(0);
                }
                __builtin_amdgcn_s_setprio(0);
                int ahead = min(b + 2, b1 - 1);
                asm volatile("" : "+s"(ahead));
                const Place last = place_in(a.c, page, ahead, head);
                fetch(last);
                page = page_of(a.c, t.seq, min(ahead + 1, b1 - 1));
                float s[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = x[r];
                if (now.absent || t0 + kBlock > each_to || t0 < each_from) hide<D, 32>(s, t0, h, c.from, now.absent ? 0 : c.to);
                const float top = st.top_of(s, fk);
                if (st.behind(top, scale_v)) st.catch_up(top, scale_v);
                half8 p[2];
                typename State<D, 32>::Exponent ex = st.exponent(s, fk, scale_v);
#pragma unroll
                for (int r = 0; r < 16; r += 2) st.probabilities(s, r, ex, p);
                st.add(ex);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int i = 0; i < F; ++i) {
                    if (i + F + kAhead < 2 * F) read(i + F + kAhead);
                    st.o[i >> 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(y[F + i], p[i & 1], st.o[i >> 1], 0, 0, 0);
                    if (i + F + kAhead < 2 * F) __builtin_amdgcn_sched_barrier(0);
                }
                __builtin_amdgcn_s_setprio(0);
                now = next;
                next = last;
                __syncthreads();
                buffer ^= 1;
            }
        }

        const float l = S::over_groups(st.l, true);
        const int column = c0 + col;
        if (column < t.columns) {
            const auto over = st.over(l == 0.f ? 0.f : 1.f / l);       // nothing seen: zeros
            uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)c.row * a.q_heads + (int64_t)head * a.group + c.head) * D;
            float* part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + plan.parts) + (worker * 2 + (opening ? 0 : 1)) * part_floats(D, C);
#pragma unroll
            for (int j = 0; j < S::kTiles; ++j)
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const int d = S::output(h, j, r);
                    float x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = l == 0.f ? 0.f : st.value(st.o[j][r + e], over);
                    if (whole) {
                        union { __bf16 b[4]; uint2 w; } y;
#pragma unroll
                        for (int e = 0; e < 4; ++e) y.b[e] = (__bf16)x[e];
                        *reinterpret_cast<uint2*>(out + d) = y.w;
                    } else {
                        *reinterpret_cast<float4v*>(part + column * D + d) = (float4v){x[0], x[1], x[2], x[3]};
                    }
                }
            if (!whole && h == 0) {
                part[C * D + column] = st.m;
                part[C * (D + 1) + column] = l;
            }
        }
        if (!whole && skip == 0 && threadIdx.x == 0)   // the row begins here and goes on
            open[worker] = {row_begin, share.per, t.s.row, t.f0, t.columns, head, (int)((row_begin + units - 1) / share.per), 0};
        share.at += take;
        row_begin += units;
        ++entry;
        opening = false;
    }
}

// Joins the parts of a row of many columns: D / 4 threads for each of several columns.  The parts' bytes bound it, written
// and read once each: 14 to 20 us after prompts.  Eight parts are loaded together (one row of 63 parts: 121 to 108 us in all).
template <int D> __global__ __launch_bounds__(kThreads) void k_join_many(AttendArgs a, Plan plan) {
    constexpr int Q = D / 4, P = kThreads / Q, C = kManyColumns;
    const Open open = reinterpret_cast<const Open*>(static_cast<const char*>(a.workspace) + plan.opens)[blockIdx.x];
    const int x = threadIdx.x % Q, lane_column = threadIdx.x / Q, col = blockIdx.y * P + lane_column;
    if (lane_column >= P || col >= open.columns) return;
    const float* parts = reinterpret_cast<const float*>(static_cast<const char*>(a.workspace) + plan.parts);
    const int many = open.last - (int)blockIdx.x + 1;
    const auto part_of = [&](int k) {
        const int64_t w = blockIdx.x + k;
        return parts + (w * 2 + part_index(w, open.per, open.begin)) * part_floats(D, C);
    };
    float top = -INFINITY, total = 0.f;
#pragma unroll 8
    for (int k = 0; k < many; ++k) top = fmaxf(top, part_of(k)[C * D + col]);
    float4v sum = 0.f;
#pragma unroll 8
    for (int k = 0; k < many; ++k) {
        const float* p = part_of(k);
        const float m = p[C * D + col], l = p[C * (D + 1) + col];
        const float w = l == 0.f ? 0.f : (m == top ? 1.f : exp2_fast(m - top)) * l;            // 0: nothing seen there
        const float4v o = *reinterpret_cast<const float4v*>(p + col * D + 4 * x);
        total += w;
        sum += w == 0.f ? (float4v)0.f : o * w;
    }
    const int f = open.f0 + col, i = f / a.group, gh = f - i * a.group, row = open.row + i;
    uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)row * a.q_heads + (int64_t)open.head * a.group + gh) * D;
    union { __bf16 b[4]; uint2 w; } u;
#pragma unroll
    for (int e = 0; e < 4; ++e) u.b[e] = (__bf16)(total == 0.f ? 0.f : sum[e] / total);
    *reinterpret_cast<uint2*>(out + 4 * x) = u.w;
}

// ---- launches ----------------------------------------------------------------------------
template <int D, int FMT, int C> void launch_few(const AttendArgs& a, const Plan& p, hipStream_t stream) {
    if (direct(a)) {
        k_few<D, FMT, C, true><<<dim3((unsigned)direct_rows(a, C), (unsigned)a.c.heads), kThreads, 0, stream>>>(a, p);
        return;
    }
    k_few<D, FMT, C, false><<<p.workers, kThreads, 0, stream>>>(a, p);
    k_join<D, C><<<dim3(p.workers, a.c.starts || a.group > 8 ? 8 : a.group), kThreads, 0, stream>>>(a, p);
}

template <int D, int FMT> hipError_t launch(const AttendArgs& a, hipStream_t stream) {
    const Plans p = plans_of(a);
    if (p.few.workers) {
        if (few_columns(a) == 16) launch_few<D, FMT, 16>(a, p.few, stream);
        else launch_few<D, FMT, 32>(a, p.few, stream);
    }
    if (p.many.workers) {
        constexpr int P = kThreads / (D / 4);
        k_many<D, FMT><<<p.many.workers, kThreads, 0, stream>>>(a, p.many);
        k_join_many<D><<<dim3(p.many.workers, (kManyColumns + P - 1) / P), kThreads, 0, stream>>>(a, p.many);
    }
    return hipGetLastError();
}

template <int D> hipError_t launch(const AttendArgs& a, hipStream_t stream) {
    return a.c.fmt ? launch<D, 1>(a, stream) : launch<D, 0>(a, stream);
}

}  // namespace

size_t attend_workspace_bytes(const AttendArgs& a) { return plans_of(a).bytes; }

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
