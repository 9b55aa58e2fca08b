// A few tokens against weights that are read from memory once, for gfx950
// (MI355X).
//
//   z[t, j] = sum_k x[t, k] w[j, k]                      one matrix
//   h[t, j] = act(sum_k x[t, k] wg[j, k]) * sum_k x[t, k] wu[j, k]   gated
//
// Weights are packed in 4 bits (INT4 with an FP16 scale per 128, NVFP4 with
// an E4M3 scale per 16 and one FP32 scale, MXFP4 with an E8M0 scale per 32)
// or are BF16.  HBM bounds the call: a weight costs half a byte and 2 n1
// flops, so up to 64 tokens the matrix cores have time to spare, and the
// work per weight on the vector units is what has to be kept small.
//
// A workgroup takes 16 FR rows of each matrix and up to 16 tokens; its
// four waves take a quarter of k each, in steps of 128, and add their sums in
// LDS in wave order, so every call returns the same bits.  Tokens are the
// MFMA's rows and weight rows its columns: lane l holds weight row l % 16 at k
// block l / 16 and receives results of that same row for tokens 4 (l / 16) ..
// + 3, so its group scale is its own.  Codes go from memory to registers to
// the matrix cores, the next batch of steps in flight while one is multiplied:
// a wave's steps follow each other in memory, so a batch is whole 128-byte
// lines.  Scales and up to 16 tokens are copied to LDS by the wave that needs
// them, so that nothing but the sums is shared and no wave waits for another.
//
// Measured on weights that come from memory: INT4 28672 x 8192, one token 28 us
// (4.3 TB/s); gated NVFP4 28672 x 8192, 8 tokens 58 (4.6 TB/s); gated BF16
// 14336 x 4096, 16 tokens 48 (4.9 TB/s).  With a single read of the codes and
// nothing else these take 21, 44 and 45: what is left is the start of a
// workgroup and, for NVFP4, 70 vector instructions per 2048 weights.  At 14336 x
// 4096 the start weighs more: gated INT4, one token 17; NVFP4, 16 tokens 13.6.
// 64 tokens take 31 there in every format, for each tile of 16 tokens converts
// the codes again.  More steps in flight, 32 rows of
// both matrices to a workgroup and starting each workgroup at another k made no
// difference or cost a little.
//
// Every code becomes exact BF16:
//   E2M1   one convert per pair, the E8M0 scale applied by the convert;
//   NVFP4  code times E4M3 has 6 significant bits: two FP32 values per
//          convert, a product each, upper halves packed by a byte permute;
//   INT4   a two's-complement nibble is 4 a + b, a = its upper two bits as a
//          signed number, b = its lower two: both are E2M1 codes of halves
//          (b: 0, 1/2, 1, 3/2; a: sign and 0, 1/2, 1), so the FP4 convert
//          serves here too and two MFMAs add the parts.  14 instructions per
//          8 weights, where unsigned converts and subtractions take 23.  The
//          parts may have opposite signs, so an infinite activation, or one
//          near 2^125 whose multiple overflows, gives NaN.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "iq_ffn_launch.h"
#include "iq_gate.h"
#include "iq_launch.h"

namespace iqk {
namespace {

using namespace gate;

struct PackedK {
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    const float* gscale[2];
    const uint16_t* x;
    void* out;
    float* saved;
    int64_t ldx;
    int32_t n0, n1, K;
    int32_t f32_out, act;
    int32_t scale_words;          // rows of scales are whole 4-byte words
};

constexpr int kStep = 128;            // k of one step: 64 code bytes per row
constexpr uint32_t kOutside = 0x80000000u;     // an offset beyond every buffer: loads zeros
constexpr int kChunkSteps = 64;       // steps whose scales are in LDS at once, 16 for each wave

// Scale bytes per row and step.
template <int FMT> constexpr int scale_bytes() { return FMT == F_INT4 ? 2 : FMT == F_NVFP4 ? 8 : FMT == F_MXFP4 ? 4 : 0; }

template <int FMT> __device__ __forceinline__ int64_t row_bytes(int K) { return FMT == F_BF16W ? 2 * (int64_t)K : K / 2; }

// 8 E2M1 codes times a power of two.
__device__ __forceinline__ u4v fp4_bf16x8(uint32_t w, float sc) {
    const bf2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1);
    const bf2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3);
    return u4v{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
               __builtin_bit_cast(uint32_t, d)};
}

// 8 E2M1 codes times an E4M3 scale: at most 2 + 4 significant bits, so the
// upper half of each FP32 product is the whole of it.
__device__ __forceinline__ u4v fp4_scaled_bf16x8(uint32_t w, float s) {
    typedef float f2v __attribute__((ext_vector_type(2)));
    u4v o;
    const f2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
    const f2v c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
    auto pack = [&](f2v v) {
        return __builtin_amdgcn_perm(__float_as_uint(v.y * s), __float_as_uint(v.x * s), 0x07060302u);
    };
    o.x = pack(a); o.y = pack(b); o.z = pack(c); o.w = pack(d);
    return o;
}

// The upper parts of 8 two's-complement nibbles as E2M1 codes of halves.
__device__ __forceinline__ uint32_t int4_upper(uint32_t w) {
    const uint32_t b2 = (w >> 2) & 0x11111111u;                       // weight 4
    const uint32_t b3 = (w >> 2) & ~(w >> 1) & 0x22222222u;           // weight -8 where b2 is clear
    return (w & 0x88888888u) | b2 | b3;                               // sign, 10 (-2), 01 (+-1)
}

// One step's codes of one fragment, as loaded.
template <int FMT> struct Codes { u4v v[FMT == F_BF16W ? 4 : 1]; };

// XR: token rows that a wave copies to LDS for every step: 4, 8 or 16.
template <int FMT, int FR, int XR, bool GATED>
__global__ __launch_bounds__(256, XR > 4 && FMT != F_BF16W ? 3 : 4) void k_packed(PackedK a) {
    constexpr int M = GATED ? 2 : 1;
    constexpr int kRows = 16 * FR, SB = scale_bytes<FMT>();
    constexpr int kScRow = 128;                                       // bytes of a row's scales for a wave's share of a chunk
    constexpr int D = (XR == 4 || XR == 8) && FMT != F_BF16W ? 2 : 1; // steps of a batch: 2 where their tokens fit
    constexpr int NC = D * M * FR * (FMT == F_BF16W ? 4 : 1), NX = D * XR / 4;      // loads of a batch's codes, copies of its tokens
    constexpr int XW = D * XR * 16;                          // 16-byte words of a batch's tokens
    struct Sums { f4v of[4][M * FR][64]; };
    // scales, a wave's own share (16-byte word w of row r at word w ^ r % 8, as the
    // rows' words of one step would else be in one bank), then sums
    __shared__ __align__(16) uint8_t s_sc[std::max<int>(SB ? 4 * M * kRows * kScRow : 16, sizeof(Sums))];
    // tokens of the batch at hand and of the next, a wave's own each: word w of
    // row r at word w ^ turn(r) of its 256 bytes, so that the lanes that the
    // LDS serves together (0-3, 12-15, 20-23, 24-27 and so on) are in
    // different banks
    __shared__ u4v s_x0[4][XW], s_x1[4][XW];
    const int t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int i = lane & 15, h = lane >> 4;
    // consecutive workgroups of an XCD take the token tiles of the same rows,
    // whose codes come from its L2 after the first
    const uint32_t tiles = (uint32_t)(a.n1 + 15) >> 4, turn8 = blockIdx.x >> 3;
    const int64_t jt = ((int64_t)(turn8 / tiles) * 8 + (blockIdx.x & 7)) * kRows;
    if (jt >= a.n0) return;
    const int j0 = (int)jt, t0 = (int)(turn8 % tiles) * 16;
    const int steps = (a.K + kStep - 1) / kStep;
    const int64_t rb = row_bytes<FMT>(a.K);

    // Rows past n0 and tokens past n1 read the last one: their lanes feed
    // only outputs that are not stored.  Offsets from the workgroup's first
    // row and token fit 32 bits.
    __amdgpu_buffer_rsrc_t cbuf[M];
    uint32_t coff[FR];
#pragma unroll
    for (int m = 0; m < M; ++m)
        cbuf[m] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.codes[m] + j0 * rb), 0, (int)(min(kRows, a.n0 - j0) * rb), 0x00020000);
#pragma unroll
    for (int f = 0; f < FR; ++f) coff[f] = (uint32_t)min(16 * f + i, a.n0 - 1 - j0) * (uint32_t)rb + 16 * h;
    const auto xbuf = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(a.x + t0 * a.ldx), 0, (int)kOutside, 0x00020000);

    f4v acc[M][FR];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int f = 0; f < FR; ++f) acc[m][f] = f4v{0.f, 0.f, 0.f, 0.f};

    // Lane h's 32 elements of a packed step start at 32 h, whole or not at
    // all; of a BF16 step, 8 elements at 32 q + 8 h.  From `limit` on, the
    // wave's last k or the row's, tokens are given an offset beyond their
    // buffer and return zeros, and so are BF16 weights, which need not be
    // finite; codes there are finite and meet zeros, and past the last row
    // their buffer ends.  A step past the matrix stands for its end, and its
    // offset is part of the lane's: the range check takes a scalar offset off
    // the buffer's size, which a row shorter than a step (K = 32 .. 96, a
    // workgroup's only row) does not have.  The loop has no branch: the copies are
    // waited for by counting what was issued after them, and the compiler
    // would move loads into a branch that alone uses them.
    auto k_of = [&](int s, int q) { return s * kStep + (FMT == F_BF16W ? 32 * q + 8 * h : 32 * h); };
    struct Batch { Codes<FMT> c[D][M][FR]; };
    struct Tokens { u4v v[D][4]; };
    auto load = [&](Batch& o, int s, int limit) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const uint32_t at = (uint32_t)min(s + d, steps) * (FMT == F_BF16W ? 256 : 64);
#pragma unroll
            for (int q = 0; q < (FMT == F_BF16W ? 4 : 1); ++q)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int f = 0; f < FR; ++f) {
                        const uint32_t off = FMT != F_BF16W || k_of(s + d, q) < limit ? coff[f] + 64 * q + at : kOutside;
                        o.c[d][m][f].v[q] = __builtin_amdgcn_raw_buffer_load_b128(cbuf[m], off, 0, 0);
                    }
        }
    };
    // instruction c copies rows 4 c .. + 3 of a step, word lane % 16 of row 4 c + lane / 16
    auto turn = [](int r) { return 4 * ((0x78 >> ((r >> 1) & 6)) & 3) + (r & 3); };     // 0, 2, 3, 1 by fours of rows
    auto copy_x = [&](u4v (&to)[4][XW], int s, int limit) {
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int c = 0; c < XR / 4; ++c) {
                const int r = 4 * c + h, w = i ^ turn(r);
                const uint32_t off = t0 + r < a.n1 && (s + d) * kStep + 8 * w < limit ? (uint32_t)r * (uint32_t)(2 * a.ldx) + 16 * w : kOutside;
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xbuf, (__attribute__((address_space(3))) void*)&to[wave][(d * XR + 4 * c) * 16], 16, off,
                                                         (uint32_t)(s + d) * (2 * kStep), 0, 0);
            }
    };
    const int xr = min(i, min(XR, a.n1 - t0) - 1);
    auto read_x = [&](Tokens& x, const u4v (&from)[4][XW]) {
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                x.v[d][q] = from[wave][(d * XR + xr) * 16 + ((FMT == F_BF16W ? 4 * q + h : 4 * h + q) ^ turn(xr))];
    };
    // `at`: the wave's first step of the chunk
    auto multiply = [&](const Batch& o, const Tokens& x, int s, int at, int limit) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const bool live = (s + d) * kStep + 32 * h < limit;       // packed lanes past it have no scale
            const uint32_t byte = (uint32_t)min(s + d - at, 16 - 1) * SB;
            uint32_t sc_at = (uint32_t)((wave * M * kRows + i) * kScRow + (FMT == F_NVFP4 ? 2 * h : FMT == F_MXFP4 ? h : 0)) +
                                   ((byte >> 4) ^ (uint32_t)(i & 7)) * 16 + (byte & 15);
            // kept whole: of an address in several parts the compiler no longer tells
            // which array it is in, and waits for the copies under way into others
            asm("" : "+v"(sc_at));
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    const Codes<FMT>& c = o.c[d][m][f];
                    const uint32_t sc = sc_at + (uint32_t)((m * kRows + 16 * f) * kScRow);
                    if constexpr (FMT == F_BF16W) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[m][f] = mfma(__builtin_bit_cast(bf8v, x.v[d][q]), __builtin_bit_cast(bf8v, c.v[q]), acc[m][f]);
                    } else if constexpr (FMT == F_INT4) {
                        const float stored = (float)*reinterpret_cast<const _Float16*>(s_sc + sc);
                        const float scale = live ? stored : 0.f;
                        f4v part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t w = c.v[0][q];
                            const bf8v lo = __builtin_bit_cast(bf8v, fp4_bf16x8(w & 0x33333333u, 2.f));
                            const bf8v up = __builtin_bit_cast(bf8v, fp4_bf16x8(int4_upper(w), 8.f));
                            part = mfma(__builtin_bit_cast(bf8v, x.v[d][q]), lo, part);
                            part = mfma(__builtin_bit_cast(bf8v, x.v[d][q]), up, part);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[m][f][e] = __builtin_fmaf(scale, part[e], acc[m][f][e]);
                    } else {
                        const uint32_t stored = FMT == F_NVFP4 ? *reinterpret_cast<const uint16_t*>(s_sc + sc) : s_sc[sc];
                        const uint32_t b = live ? stored : 0u;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            u4v v;
                            if constexpr (FMT == F_NVFP4) {
                                v = fp4_scaled_bf16x8(c.v[0][q], q < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)b, 0)
                                                                      : __builtin_amdgcn_cvt_f32_fp8((int)b, 1));
                            } else {
                                // 2^(b - 127): b = 0 is the subnormal 2^-127; 255 is NaN
                                v = fp4_bf16x8(c.v[0][q], __uint_as_float(b ? b << 23 : 0x00400000u));
                                if (b == 255u) v = u4v{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
                            }
                            acc[m][f] = mfma(__builtin_bit_cast(bf8v, x.v[d][q]), __builtin_bit_cast(bf8v, v), acc[m][f]);
                        }
                    }
                }
        }
    };

    constexpr int kChunk = SB ? kChunkSteps : 1 << 30;
    for (int s0 = 0; s0 < steps; s0 += kChunk) {
        const int s1 = min(steps, s0 > steps - kChunk ? steps : s0 + kChunk);
        const int unit = FMT == F_INT4 ? 2 : D;                       // whole batches, and whole 4-byte words of scales
        const int share = (s1 - s0 + 4 * unit - 1) / (4 * unit) * unit;
        const int first = s0 + wave * share, end = min(s1, first + share);      // past s1: no steps
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): the last chunk's scales have been read
        if constexpr (SB > 0) {
            const uint32_t per_row = (uint32_t)(FMT == F_INT4 ? a.K / 128 * 2 : FMT == F_NVFP4 ? a.K / 16 : a.K / 32);
            const uint32_t most = (uint32_t)min(kRows, a.n0 - j0);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const uint8_t* from = a.scales[m] + (int64_t)j0 * per_row;
                if (a.scale_words) {
                    const auto buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(from), 0, (int)(most * per_row), 0x00020000);
#pragma unroll
                    for (int c = 0; c < kRows / 8; ++c) {
                        const uint32_t r = 8 * c + (lane >> 3);
                        __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (__attribute__((address_space(3))) void*)(s_sc + ((wave * M + m) * kRows + 8 * c) * kScRow), 16,
                                                                 min(r, most - 1) * per_row + first * SB + 16 * ((lane & 7) ^ (r & 7)), 0, 0, 0);
                    }
                } else {                                              // rows that 4-byte words do not divide
                    const int take = max(0, min((end - first) * SB, (int)per_row - first * SB));
                    for (int r = lane; r < kRows; r += 64) {
                        const uint8_t* row = from + (int64_t)min((uint32_t)r, most - 1) * per_row + first * SB;
                        for (int b = 0; b < take; ++b) s_sc[((wave * M + m) * kRows + r) * kScRow + ((b >> 4) ^ (r & 7)) * 16 + (b & 15)] = row[b];
                    }
                }
            }
        }
        Batch now, next;
        const int limit = min(a.K, end * kStep);
        copy_x(s_x0, first, limit);
        __builtin_amdgcn_sched_barrier(0);
        load(now, first, limit);
        // The wave's copies are waited for here and in `batch` by their
        // number: the compiler's own waits for them may come out too weak.
        if constexpr (SB > 0) wait_for_all_but<NX + NC>();
        // tokens, which come from the caches, before codes, so that waiting for
        // them does not wait for memory
        auto batch = [&](Batch& o, Batch& ahead, u4v (&xo)[4][XW], u4v (&xa)[4][XW], int s) {
            Tokens x;
            __builtin_amdgcn_sched_barrier(0);        // what was read of xa has been multiplied
            copy_x(xa, s + D, limit);
            __builtin_amdgcn_sched_barrier(0);        // in this order, and not put off
            load(ahead, s + D, limit);
            __builtin_amdgcn_sched_barrier(0);
            wait_for_all_but<2 * NC + NX>();
            read_x(x, xo);
            multiply(o, x, s, first, limit);
        };
        for (int s = first; s < end; s += 2 * D) {
            batch(now, next, s_x0, s_x1, s);
            batch(next, now, s_x1, s_x0, s + D);
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);                               // copies past the last step write LDS too
    auto& red = reinterpret_cast<Sums*>(s_sc)->of;
    if constexpr (SB > 0) __syncthreads();                            // scales are no longer read
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int f = 0; f < FR; ++f) red[wave][m * FR + f][lane] = acc[m][f];
    __syncthreads();
    // the first FR waves add and store a fragment each
    if (wave >= FR) return;
    const int f = wave, j = j0 + 16 * f + i;
    if (j >= a.n0) return;
    f4v v[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        const float gs = FMT == F_NVFP4 && a.K > 0 ? *a.gscale[m] : 1.f;
        v[m] = (((red[0][m * FR + f][lane] + red[1][m * FR + f][lane]) + red[2][m * FR + f][lane]) + red[3][m * FR + f][lane]) * gs;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int tok = t0 + 4 * h + e;
        if (tok >= a.n1) continue;
        const int64_t o = (int64_t)tok * a.n0 + j;
        float z = v[0][e];
        if constexpr (GATED) {
            if (a.saved) {
                a.saved[o] = v[0][e];
                a.saved[(int64_t)a.n1 * a.n0 + o] = v[1][e];
            }
            z = (a.act == A_SILU ? act<A_SILU>(z) : a.act == A_GELU ? act<A_GELU>(z) : act<A_GELU_TANH>(z)) * v[1][e];
        }
        if (a.f32_out) static_cast<float*>(a.out)[o] = z;
        else static_cast<uint16_t*>(a.out)[o] = (uint16_t)bf16_pair(z, 0.f);
    }
}

template <int FMT, int FR, int XR, bool GATED> hipError_t run(const PackedK& k, hipStream_t s) {
    const int64_t rows = (k.n0 + 16 * FR - 1) / (16 * FR), tiles = (k.n1 + 15) / 16;
    k_packed<FMT, FR, XR, GATED><<<(unsigned)((rows + 7) / 8 * 8 * tiles), 256, 0, s>>>(k);
    return hipGetLastError();
}

template <int FMT, int FR, bool GATED> hipError_t pick_tokens(const PackedK& k, hipStream_t s) {
    if (k.n1 <= 4) return run<FMT, FR, 4, GATED>(k, s);
    if (k.n1 <= 8) return run<FMT, FR, 8, GATED>(k, s);
    return run<FMT, FR, 16, GATED>(k, s);
}

// 32 rows of one matrix to a workgroup share its tokens; while workgroups of 16
// rows are too few to give every CU two, these end sooner.  K = 4096, INT4, by 16
// and by 32 rows, in us: one token, 1024 rows 4.8 and 6.1, 4096 rows 5.0 and
// 6.3, 6144 rows 6.2 and 6.5, 14336 rows 10.8 and 10.6; 16 tokens, 4096 rows 6.0
// and 7.2, 6144 rows 7.6 and 7.3, 14336 rows 16.6 and 13.6; 64 tokens, 1024 rows
// 5.9 and 7.1, 2048 rows 7.6 and 7.3, 4096 rows 12.2 and 10.3.  NVFP4 and MXFP4
// cross near the same sizes.
constexpr int64_t kFewWorkgroups = 384;
template <int FMT, bool GATED> hipError_t pick(const PackedK& k, hipStream_t s) {
    if constexpr (GATED) return pick_tokens<FMT, 1, true>(k, s);
    else if ((int64_t)((k.n0 + 15) / 16) * ((k.n1 + 15) / 16) < kFewWorkgroups) return pick_tokens<FMT, 1, false>(k, s);
    else return pick_tokens<FMT, 2, false>(k, s);
}

template <int FMT> hipError_t pick(bool gated, const PackedK& k, hipStream_t s) {
    return gated ? pick<FMT, true>(k, s) : pick<FMT, false>(k, s);
}

}  // namespace

hipError_t launch_packed(const PackedArgs& a, hipStream_t s) {
    PackedK k = {};
    for (int m = 0; m < (a.gated ? 2 : 1); ++m) {
        k.codes[m] = static_cast<const uint8_t*>(a.w[m].codes);
        k.scales[m] = static_cast<const uint8_t*>(a.w[m].scales);
        k.gscale[m] = a.w[m].global_scale;
    }
    k.x = static_cast<const uint16_t*>(a.x); k.out = a.out; k.saved = a.saved; k.ldx = a.ldx;
    k.n0 = (int32_t)a.n0; k.n1 = (int32_t)a.n1; k.K = (int32_t)a.K;
    k.f32_out = a.out_dtype == D_F32;
    k.scale_words = a.K % (a.fmt == F_INT4 ? 256 : a.fmt == F_NVFP4 ? 64 : 128) == 0;
    k.act = a.act;
    switch (a.fmt) {
    case F_INT4: return pick<F_INT4>(a.gated, k, s);
    case F_NVFP4: return pick<F_NVFP4>(a.gated, k, s);
    case F_MXFP4: return pick<F_MXFP4>(a.gated, k, s);
    default: return a.gated ? pick<F_BF16W, true>(k, s) : hipErrorInvalidValue;
    }
}

}  // namespace iqk
