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

// Probabilities are relative to a running maximum m that follows the scores
// once one is 2^kSlack past it, so a block rarely costs a rescaling of the
// output.  They are held times 2^kLift: at most 2^15 in FP16, with all digits
// from 2^-23 on and steps of 2^-33 below.  The factor leaves with the division by their sum.
constexpr float kSlack = 6.f, kLift = 9.f;

// The block's values scale enters the exponent, as a fraction of the largest
// so far, 2^lift; a fraction below 2^-60 counts as 2^-60, where values are 2^-50 of
// what the row holds already.
constexpr float kLeastFraction = 0x1p-60f;

// What a tile's columns see.  Columns are sorted by position, so the first and
// the last bound them all.
struct View {
    int keys;                    // tokens that the table has entries for
    int64_t first;               // position of token 0 of the call; may be negative
    int all_from, all_to;        // some column sees some of these
    int each_from, each_to;      // every column sees all of these
    int block, blocks;           // blocks that hold some
};

__device__ __forceinline__ int seen_to(const AttendArgs& a, int64_t p, int keys) {
    return p < 0 ? 0 : a.causal ? (int)min((int64_t)keys, p + 1) : keys;
}
__device__ __forceinline__ int seen_from(const AttendArgs& a, int64_t p, int keys) {
    return (int)min(max((int64_t)0, p + 1 - a.window), (int64_t)keys);
}

__device__ __forceinline__ View view_of(const AttendArgs& a, const Tile& t) {
    View v;
    v.keys = a.c.pages > 0 ? (int)min((int64_t)t.s.length, ((int64_t)a.c.width << a.c.shift) * kBlock) : 0;
    v.first = (int64_t)t.s.length - t.s.n;
    const int64_t lo = v.first + t.f0 / a.group, hi = v.first + (t.f0 + t.columns - 1) / a.group;
    v.all_to = seen_to(a, hi, v.keys); v.all_from = seen_from(a, lo, v.keys);
    v.each_to = seen_to(a, lo, v.keys); v.each_from = seen_from(a, hi, v.keys);
    v.block = v.all_from / kBlock;
    v.blocks = max((v.all_to + kBlock - 1) / kBlock - v.block, 0);
    return v;
}

// Queries of a column as the matrix cores take them: FP16 times a power of two
// that brings the row's largest into [2^14, 2^15), and the factor that makes
// scores exponents of 2.
template <int J> __device__ __forceinline__ float load_query(const AttendArgs& a, const uint16_t* row, int h, half8* q) {
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
    int e = (int)(top >> 23);                          // 0 for zeros and subnormals, 255 for infinities and NaN
    e = e == 255 ? 0 : max(e, 1) - 127 - 14;
#pragma unroll
    for (int j = 0; j < 2 * J; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(&raw[j])[k >> 1];
            q[j][k] = (_Float16)ldexpf(__uint_as_float(k & 1 ? w & 0xFFFF0000u : w << 16), -e);
        }
    return ldexpf(a.scale * 1.44269504f, e);
}

// Running state of a column: maximum, sum of this lane's tokens, output.
template <int J> struct State {
    float16v o[J];
    float m, l;
    int lift;                    // values' scales are held over 2^lift, the largest so far

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < J; ++j) o[j] = 0.f;
        m = -INFINITY;
        l = 0.f;
        lift = -126;
    }
    __device__ __forceinline__ void scale(float by) {
#pragma unroll
        for (int j = 0; j < J; ++j) o[j] *= by;
    }
    // From scores (codes times FP16 queries) to probabilities: pv[step][e] is
    // that of the e-th of the 8 tokens of matrix product `step`.  seen: bit r for score r.
    __device__ __forceinline__ void probabilities(const float16v& s, float fk, float scale_v, uint32_t seen, bool masked, half8* pv) {
        float top = -INFINITY;
        if (!masked) {
#pragma unroll
            for (int r = 0; r < 16; ++r) top = fmaxf(top, s[r]);
        } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) top = (seen >> r) & 1 ? fmaxf(top, s[r]) : top;
        }
        top = top == -INFINITY ? top : top * fk;
        if (__any(top > m + kSlack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float now = fmaxf(m, top), alpha = now == m ? 1.f : exp2_fast(m - now);
            m = now;
            l *= alpha;
            scale(alpha);
        }
        if (scale_v > ldexpf(1.f, lift)) {             // the same for the whole wave
            int e;
            frexpf(scale_v, &e);
            scale(ldexpf(1.f, max(lift - e, -200)));
            lift = e;
        }
        const float fraction = fmaxf(ldexpf(scale_v, -lift), kLeastFraction);
        const float off = kLift + __builtin_amdgcn_logf(fraction) - m;
        float sum = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float e = exp2_fast(__builtin_fmaf(s[r], fk, off));
            if (masked) e = (seen >> r) & 1 ? e : 0.f;
            sum += e;
            pv[r >> 3][r & 7] = (_Float16)e;
        }
        l = __builtin_fmaf(sum, 1.f / fraction, l);
    }
};

// Bits of the scores of lane half h whose tokens lie in [from, to); the block's token 0 is t0.
__device__ __forceinline__ uint32_t seen_bits(int t0, int h, int from, int to) {
    uint32_t seen = 0;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        const int token = t0 + 8 * (r >> 2) + 4 * h + (r & 3);
        seen |= (token >= from && token < to ? 1u : 0u) << r;
    }
    return seen;
}

// Codes of 16 values of lane half h with those from token `keys` on, which may be anything, as zeros.
__device__ __forceinline__ void keep_values(uint4* v, int t0, int h, int keys) {
    uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = keys - t0 - (8 * i + 4 * h);     // bytes of this word that are the sequence's
        w[i] &= n <= 0 ? 0u : n >= 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1u;
    }
}

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
    float scale_k, scale_v;
    bool absent;
};
template <typename T> using scalar_t = const __attribute__((address_space(4))) T*;
template <typename T> __device__ __forceinline__ T scalar_load(const T* p, int64_t i) {
    return ((scalar_t<T>)(uintptr_t)p)[i];
}
__device__ __forceinline__ Place place_at(const CacheArgs& c, int seq, int b, int head) {
    Place p;
    b = one(b);
    const int64_t page = scalar_load(c.page_table, (int64_t)seq * c.width + (b >> c.shift));
    p.absent = page < 0 || page >= c.pages;
    p.at = p.absent ? 0 : ((page * c.heads + head) << c.shift) | (b & ((1 << c.shift) - 1));
    p.scale_k = scalar_load(c.scales, p.at * 2);
    p.scale_v = scalar_load(c.scales, p.at * 2 + 1);
    return p;
}

// ---- few columns: the work is the cache's codes ------------------------------------------
// All (tile, key head, block) triples in order are shared out evenly among a
// fixed number of workgroups, so sequences of any lengths keep every CU busy.
// A row that more than one workgroup has a share of is joined by a second launch.
//
// A workgroup's four waves take its blocks in turn, each with the next block's
// codes in flight, and join their outputs through LDS.
constexpr int kLeastShare = 8;   // blocks of a workgroup, at least

__host__ __device__ inline int64_t part_floats(int dim) { return (int64_t)kColumns * (dim + 2); }

struct Plan {
    int64_t slots;
    int workers;
    int64_t parts;               // where the parts begin in the workspace, in floats
};
// The workspace begins with the share and the running sums of blocks of all
// slots, int64 [2 + slots]; parts follow, two for every workgroup: of the row
// that its share begins in (0), and of the one that it ends in (1).

__device__ __forceinline__ int units_of(const AttendArgs& a, const Plan& plan, int64_t slot) {
    Tile t;
    if (slot >= plan.slots || !tile_of(a, slot, &t)) return 0;
    return max(view_of(a, t).blocks, 1);               // a row that sees nothing is written by someone
}

// The share of a workgroup: sum over slots, then the slot that unit `at` lies in.
struct Shares {
    int64_t total, per;
};

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

template <int D, int FMT> __global__ __launch_bounds__(kThreads, D <= 128 ? 2 : 1) void k_few(AttendArgs a, Plan plan) {
    constexpr int J = D / 32;                          // pieces of 32 elements
    __shared__ float other[2][kWaves * kColumns];      // maxima and sums of the waves
    __shared__ float pass[2 * (D / 2) * 64];           // outputs on their way to another wave
    __shared__ int64_t sums[kWaves + 1];
    __shared__ int64_t found[2];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, h = lane >> 5;
    int64_t* header = static_cast<int64_t*>(a.workspace);

    // the workgroup's share of all units
    int64_t mine = 0;
    for (int64_t s = threadIdx.x; s < plan.slots; s += kThreads) mine += units_of(a, plan, s);
    mine = wave_sum(mine);
    if (lane == 0) sums[wave] = mine;
    __syncthreads();
    const int64_t total = (sums[0] + sums[1] + sums[2] + sums[3]) * a.c.heads;
    int64_t per = (total + plan.workers - 1) / plan.workers;
    per = per < kLeastShare ? kLeastShare : per;
    int64_t at = blockIdx.x * per;
    const int64_t end = min(at + per, total);
    if (blockIdx.x == 0 && threadIdx.x == 0) header[0] = per;
    if (at >= total) return;
    int64_t before = 0;                                // units of the slots before the current 256, one head
    for (int64_t base = 0; base < plan.slots; base += kThreads) {
        const int v = units_of(a, plan, base + threadIdx.x);
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
        if (blockIdx.x == 0 && base + threadIdx.x < plan.slots) header[1 + base + threadIdx.x] = upto - v;
        if (at >= (upto - v) * a.c.heads && at < upto * a.c.heads) {
            found[0] = base + threadIdx.x;
            found[1] = upto - v;
        }
        before += sums[0] + sums[1] + sums[2] + sums[3];
        if (blockIdx.x != 0 && at < before * a.c.heads) break;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) header[1 + plan.slots] = before;
    __syncthreads();
    int64_t slot = found[0];
    const int64_t into = at - found[1] * a.c.heads;
    bool opening = true;                               // the share's first row
    int head = -1, skip = 0;

    while (at < end) {
        Tile t;
        if (!tile_of(a, slot, &t)) {
            ++slot;
            continue;
        }
        t = one(t);
        const View v = view_of(a, t);
        const int units = max(v.blocks, 1);
        if (opening) {
            head = one((int)(into / units));
            skip = one((int)(into - (int64_t)head * units));
        } else {
            if (++head == a.c.heads) {
                head = -1;
                ++slot;
                continue;
            }
            skip = 0;
        }
        const int take = one((int)min((int64_t)(units - skip), end - at));
        const bool whole = take == units;
        const int b0 = v.block + min(skip, v.blocks), b1 = v.block + min(skip + take, v.blocks);

        // what this column sees: tokens [from, to)
        const int f = t.f0 + min(col, t.columns - 1), i = f / a.group, g = f - i * a.group;
        const int from = seen_from(a, v.first + i, v.keys), to = seen_to(a, v.first + i, v.keys);
        half8 q[2 * J];
        const float factor = load_query<J>(
            a, static_cast<const uint16_t*>(a.q) + (t.s.row + i) * a.ld_token + ((int64_t)head * a.group + g) * a.ld_head, h, q);

        State<J> st;
        st.clear();
        // Codes of the wave's next block: keys are fetched once the scores of this one are formed, values after its output.
        // Past the last block the last one is fetched again; absent pages stand for a page that nothing is seen of.
        uint4 kc[J], vc[J];
        if (b0 + wave < b1) {
            Place now = place_at(a.c, t.seq, b0 + wave, head), next = now;
            const auto fetch_keys = [&](int64_t at) {
                const uint4* codes = reinterpret_cast<const uint4*>(a.c.codes + at * (2 * kBlock * (int64_t)D));
#pragma unroll
                for (int j = 0; j < J; ++j) kc[j] = codes[(2 * j + h) * 32 + col];
            };
            const auto fetch_values = [&](int64_t at) {
                const uint4* codes = reinterpret_cast<const uint4*>(a.c.codes + at * (2 * kBlock * (int64_t)D)) + 2 * D;
#pragma unroll
                for (int j = 0; j < J; ++j) vc[j] = codes[(32 * j + col) * 2 + h];
            };
            fetch_keys(now.at);
            fetch_values(now.at);
            for (int b = b0 + wave; b < b1; b += kWaves) {
                next = place_at(a.c, t.seq, min(b + kWaves, b1 - 1), head);
                float16v s = 0.f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(kc[j].x, kc[j].y), q[2 * j], s, 0, 0, 0);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(kc[j].z, kc[j].w), q[2 * j + 1], s, 0, 0, 0);
                }
                fetch_keys(next.at);
                const int t0 = b * kBlock;
                half8 pv[2];
                const bool masked = now.absent || t0 + kBlock > v.each_to || t0 < v.each_from;
                uint32_t seen = 0xFFFFu;
                if (masked) seen = seen_bits(t0, h, from, now.absent ? 0 : to);
                st.probabilities(s, factor * now.scale_k, now.scale_v, seen, masked, pv);
                if (now.absent || t0 + kBlock > v.keys) {
#pragma unroll
                    for (int j = 0; j < J; ++j) keep_values(&vc[j], t0, h, now.absent ? 0 : v.keys);
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    st.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(vc[j].x, vc[j].y), pv[0], st.o[j], 0, 0, 0);
                    st.o[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(expand8<FMT>(vc[j].z, vc[j].w), pv[1], st.o[j], 0, 0, 0);
                }
                fetch_values(next.at);
                now = next;
            }
        }
        float l = st.l + __shfl_xor(st.l, 32);

        // join the four waves: each output over the sum of all, weighted by its maximum
        other[0][wave * kColumns + col] = st.m;
        other[1][wave * kColumns + col] = l;
        __syncthreads();
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, other[0][w * kColumns + col]);
        const auto weight = [&](float m) { return m == top ? 1.f : exp2_fast(m - top); };
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += other[1][w * kColumns + col] * weight(other[0][w * kColumns + col]);
        // sums are positive unless nothing was seen; NaN passes through
        const float share = l == 0.f ? 0.f : weight(st.m) / sum;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) st.o[j][r] = l == 0.f ? 0.f : ldexpf(st.o[j][r] * share, st.lift);
#pragma unroll
        for (int round = kWaves / 2; round; round >>= 1) {
            float* mail = pass + (wave & (round - 1)) * (D / 2) * 64;
            if (wave >= round && wave < 2 * round) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) mail[(j * 16 + r) * 64 + lane] = st.o[j][r];
            }
            __syncthreads();
            if (wave < round) {
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) st.o[j][r] += mail[(j * 16 + r) * 64 + lane];
            }
            __syncthreads();
        }
        if (wave == 0 && col < t.columns) {
            if (whole) {
                uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)(t.s.row + i) * a.q_heads + (int64_t)head * a.group + g) * D;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        union { __bf16 b[4]; uint2 w; } u;
#pragma unroll
                        for (int e = 0; e < 4; ++e) u.b[e] = (__bf16)st.o[j][r + e];
                        *reinterpret_cast<uint2*>(out + 32 * j + 2 * r + 4 * h) = u.w;
                    }
            } else {
                float* part = static_cast<float*>(a.workspace) + plan.parts + (blockIdx.x * 2 + (opening ? 0 : 1)) * part_floats(D);
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int r = 0; r < 16; r += 4)
                        *reinterpret_cast<float4v*>(part + col * D + 32 * j + 2 * r + 4 * h) =
                            (float4v){st.o[j][r], st.o[j][r + 1], st.o[j][r + 2], st.o[j][r + 3]};
                if (h == 0) {
                    part[kColumns * D + col] = top;
                    part[kColumns * (D + 1) + col] = sum;
                }
            }
        }
        at += take;
        opening = false;
    }
}

// Joins the parts of rows that several workgroups had a share of: a wave for
// each column, its lanes the parts for the weights and the elements for the sums.
template <int D> __global__ __launch_bounds__(kThreads) void k_join(AttendArgs a, Plan plan) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, head = blockIdx.y, col = blockIdx.z * kWaves + wave;
    const int64_t* header = static_cast<const int64_t*>(a.workspace);
    const int64_t per = header[0], slot = blockIdx.x, units = header[2 + slot] - header[1 + slot];
    if (units == 0) return;
    const int64_t u0 = header[1 + slot] * a.c.heads + head * units, u1 = u0 + units;
    const int64_t w0 = u0 / per, w1 = (u1 - 1) / per;
    if (w0 == w1) return;                              // one workgroup had it all and wrote it
    Tile t;
    if (!tile_of(a, slot, &t) || col >= t.columns) return;
    const float* parts = static_cast<const float*>(a.workspace) + plan.parts;
    const auto part_of = [&](int64_t w) { return parts + (w * 2 + (w * per < u0 ? 1 : 0)) * part_floats(D); };
    float top = -INFINITY;
    for (int64_t w = w0 + lane; w <= w1; w += 64) top = fmaxf(top, part_of(w)[kColumns * D + col]);
#pragma unroll
    for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    constexpr int E = (D + 63) / 64;
    float total = 0.f, sum[E] = {};
    for (int64_t base = w0; base <= w1; base += 64) {
        const int n = (int)min((int64_t)64, w1 + 1 - base);
        float mine = 0.f;
        if (lane < n) {
            const float* p = part_of(base + lane);
            const float m = p[kColumns * D + col], l = p[kColumns * (D + 1) + col];
            mine = l == 0.f ? 0.f : (m == top ? 1.f : exp2_fast(m - top)) * l;        // 0: nothing seen there
        }
        for (int k = 0; k < n; ++k) {
            const float w = __shfl(mine, k);
            total += w;
            const float* p = part_of(base + k) + col * D;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (D % 64 == 0 || e * 64 + lane < D) sum[e] += w * p[e * 64 + lane];
        }
    }
    const int f = t.f0 + col, i = f / a.group, g = f - i * a.group;
    uint16_t* out = static_cast<uint16_t*>(a.o) + ((int64_t)(t.s.row + i) * a.q_heads + (int64_t)head * a.group + g) * D;
#pragma unroll
    for (int e = 0; e < E; ++e)
        if (D % 64 == 0 || e * 64 + lane < D)
            out[e * 64 + lane] = __builtin_bit_cast(uint16_t, (__bf16)(total == 0.f ? 0.f : sum[e] / total));
}

Plan plan_of(const AttendArgs& a) {
    Plan p;
    p.slots = tile_slots(a);
    p.workers = a.c.dim <= 128 ? 512 : 256;            // what the GPU holds at once: two or one on a CU
    p.parts = ((p.slots + 2) * 2 + 63) / 64 * 64;
    return p;
}

template <int D> hipError_t launch(const AttendArgs& a, hipStream_t stream) {
    const Plan p = plan_of(a);
    if (a.c.fmt) k_few<D, 1><<<p.workers, kThreads, 0, stream>>>(a, p);
    else k_few<D, 0><<<p.workers, kThreads, 0, stream>>>(a, p);
    k_join<D><<<dim3((unsigned)p.slots, (unsigned)a.c.heads, kColumns / kWaves), kThreads, 0, stream>>>(a, p);
    return hipGetLastError();
}

}  // namespace

size_t attend_workspace_bytes(const AttendArgs& a) {
    const Plan p = plan_of(a);
    return (size_t)(p.parts + p.workers * 2 * part_floats(a.c.dim)) * sizeof(float);
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
