// The gated block's matrix products for gfx950 (MI355X), BF16 operands.
//
//   forward   g = x Wg^T, u = x Wu^T, h = act(g) u
//   backward  dg = dh u act'(g), du = dh act(g)
//             dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
//
// Each product is C[m][n] = sum_k P[n][k] Q[m][k]: P is the MFMA's row
// operand, so that a lane holds four consecutive n of one m, n being the
// contiguous dimension of C.
//
//   mode    m         n         k                 P             Q
//   FWD     tokens    features  cols              Wg, Wu        x
//   DX      tokens    cols      2 x features      Wg, Wu ^T     dg, du
//   DW      features  cols      tokens            x ^T          dg, du ^T
//
// An operand is "k-contiguous" (its rows are the product's rows) or
// "k-strided" (its rows are the sum's index, marked ^T).  Both kinds are
// copied to LDS as they lie in memory by buffer loads that write LDS
// directly, and k-strided tiles are turned round on the way to the matrix
// cores by the transposing LDS read, so no operand is transposed in memory.
// Elements past the end of a row, a column or k are given an offset beyond
// the buffer's range, which loads zeros.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <utility>

#include "iq_ffn_launch.h"
#include "iq_gate.h"
#include "iq_launch.h"

namespace iqk {
namespace {

using namespace gate;

typedef __attribute__((address_space(3))) void lds_void;
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

enum { FWD = 0, DX = 1, DW = 2 };

constexpr int BK = 64;                         // k of one step: a 128-byte line of a k-contiguous row
constexpr uint32_t kOutside = 0x80000000u;     // an offset beyond every buffer: loads zeros

struct GemmArgs {
    const uint16_t* p[2];
    const uint16_t* q[2];
    int64_t ldp, ldq;
    int32_t N, M, K;              // of one of the two weights
    int32_t tiles_n, tiles_m;     // tiles_m counts both weights in DW
    uint32_t tiles;
    int32_t per_xcd;
    int32_t split_steps;          // DX: steps of one part of k
    int32_t parts;                // DX: parts of k; above 1 the sums go to `partial`
    uint16_t* out[2];
    float* saved;                 // FWD: g and u [2][M][N], may be null
    float* partial;               // DX: [parts][M][N]
};

// A tile of 128 rows (or columns) by 64 k in LDS: 16 KB.
//   k-contiguous: 16-byte slot s of row r at slot s ^ (r & 7) of its 128 bytes;
//   k-strided:    32-byte slot c of row k at slot c ^ (k & 3 | k >> 1 & 4) of
//                 its 256 bytes: the 8 rows that half a wave reads at a time
//                 fall into the 8 different slots.
struct Half { u4v w[1024]; };

// One wave's share of the copies of a Half: NI instructions of 64 x 16 bytes.
template <bool KC, int NI> struct Copy {
    uint32_t off[NI];     // byte offset from the tile's first element
    int32_t kk;           // first k that the lane's word holds (KC: of every instruction; else of instruction 0)
    // `left`: rows (KC) or columns (else) from the tile's first to the matrix's last
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t left) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int q = wave * NI + i;
            if constexpr (KC) {
                const int r = 8 * q + (lane >> 3), slot = (lane & 7) ^ (lane >> 3);
                off[i] = r < left ? (uint32_t)(r * ld * 2) + slot * 16u : kOutside;
            } else {
                const int k = 4 * q + (lane >> 4), col = 8 * ((lane & 15) ^ (2 * ((k & 3) | ((k >> 1) & 4))));
                off[i] = col < left ? (uint32_t)(k * ld * 2) + col * 2u : kOutside;
            }
        }
        kk = KC ? 8 * ((lane & 7) ^ (lane >> 3)) : 4 * wave * NI + (lane >> 4);
    }
    // `base`: the tile's first element at this step; `left`: k from there to the end
    __device__ __forceinline__ void issue(const uint16_t* base, int left, int wave, Half& to) const {
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base), 0, (int)kOutside, 0x00020000);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const uint32_t o = kk + (KC ? 0 : 4 * i) < left ? off[i] : kOutside;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)&to.w[(wave * NI + i) * 64], 16, o, 0, 0, 0);
        }
    }
};

// MFMA operand of rows (columns) rb .. rb + 15 at k 32 ks .. + 31 of the Half
// that starts `at` bytes into LDS object T: lane l has row rb + l % 16 and
// k 32 ks + 8 (l / 16) .. + 7.  The address is one offset from the object,
// not a chain of members: past a few links the compiler no longer sees which
// object a read is from and lets it wait for copies into the others.
template <bool KC, class T> __device__ __forceinline__ bf8v fragment(const T& t, uint32_t at, int rb, int ks, int lane) {
    const uint32_t i = lane & 15, h = lane >> 4;
    const char* base = reinterpret_cast<const char*>(&t);
    if constexpr (KC) {
        return *reinterpret_cast<const bf8v*>(base + (at + (rb + i) * 128 + ((4 * ks + h) ^ (i & 7)) * 16));
    } else {
        // the transposing read gives lane i of 16 element i of the four rows
        // that its group's lanes 4 j + c name by column 4 c of row j
        const uint32_t k = 32 * ks + 8 * h + (i >> 2), slot = (rb >> 4) ^ ((i >> 2) | ((h & 1) << 2));
        const uint32_t o = at + k * 256 + slot * 32 + (i & 3) * 8;
        const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(base + o));
        const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(base + (o + 4 * 256)));
        return __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// Two neighbouring 16 x 16 results (n 0..15 in a, 16..31 in b; the lane's m)
// to BF16 memory: the lanes of even and odd 16s exchange halves so that each
// stores 8 consecutive n.
__device__ __forceinline__ void store_pair(uint16_t* row, int n0, int N, int lane, f4v a, f4v b) {
    const int h = lane >> 4, n = n0 + 16 * (h & 1) + 8 * (h >> 1);
    const u2v lo = __builtin_bit_cast(u2v, __builtin_amdgcn_permlane16_swap(bf16_pair(a[0], a[1]), bf16_pair(b[0], b[1]),
                                                                           false, false));
    const u2v hi = __builtin_bit_cast(u2v, __builtin_amdgcn_permlane16_swap(bf16_pair(a[2], a[3]), bf16_pair(b[2], b[3]),
                                                                           false, false));
    if (row && n < N) *reinterpret_cast<u4v*>(row + n) = u4v{lo.x, hi.x, lo.y, hi.y};
}
__device__ __forceinline__ void store_f4(float* row, int n, int N, f4v v) {
    if (row && n < N) *reinterpret_cast<f4v*>(row + n) = v;
}

// Tile order: consecutive tiles of one XCD's slice run down `kGroup` columns
// of tiles, so that the tiles in flight on an XCD share operands in its L2.
constexpr int kGroup = 8;
__device__ __forceinline__ bool tile_of(const GemmArgs& a, int& tn, int& tm) {
    const uint32_t b = blockIdx.x, idx = (b & 7u) * (uint32_t)a.per_xcd + (b >> 3);
    if (idx >= a.tiles) return false;
    const uint32_t band = (uint32_t)kGroup * (uint32_t)a.tiles_m, g = idx / band, in = idx - g * band;
    const uint32_t width = min((uint32_t)kGroup, (uint32_t)a.tiles_n - g * kGroup);
    tn = (int)(g * kGroup + in % width);
    tm = (int)(in / width);
    return true;
}

// 128 x 128 tiles (FWD: 64 features of each weight), 4 waves of 64 x 64, two
// LDS stages: the copies of step s + 1 are in flight during step s.
template <int MODE, int ACT> __global__ __launch_bounds__(256, 2) void k_gemm(GemmArgs a) {
    constexpr bool PK = MODE == FWD, QK = MODE != DW;
    constexpr int kTileN = MODE == FWD ? 64 : 128;
    __shared__ Half P0, P1, Q0, Q1;
    int tn, tm;
    if (!tile_of(a, tn, tm)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int sel = MODE == DW && tm >= a.tiles_m / 2 ? 1 : 0;        // which weight's gradient
    const int n0 = tn * kTileN, m0 = (MODE == DW ? tm - sel * (a.tiles_m / 2) : tm) * 128;
    const int seg_steps = (a.K + BK - 1) / BK;
    const int all = MODE == DX ? 2 * seg_steps : seg_steps;
    const int first = MODE == DX ? (int)blockIdx.y * a.split_steps : 0;
    const int last = MODE == DX ? min(all, first + a.split_steps) : all;

    Copy<PK, 4> cp;
    Copy<QK, 4> cq;
    // FWD: waves 0 and 1 copy the gate's 64 rows, 2 and 3 the up projection's
    if (MODE == FWD) {
        cp.init(wave, lane, a.ldp, (wave >= 2 ? 64 : 0) + (int64_t)a.N - n0);
        if (wave < 2)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (8 * (4 * wave + i) + (lane >> 3) >= a.N - n0) cp.off[i] = kOutside;
    } else {
        cp.init(wave, lane, a.ldp, (int64_t)a.N - n0);
    }
    cq.init(wave, lane, a.ldq, (int64_t)a.M - m0);

    auto issue = [&](int s, Half& P, Half& Q) {
        const int seg = MODE == DX && s >= seg_steps ? 1 : 0;
        const int k0 = (s - seg * seg_steps) * BK, left = a.K - k0;
        const uint16_t* pb;
        if (MODE == FWD) pb = wave < 2 ? a.p[0] + (int64_t)n0 * a.ldp + k0 : a.p[1] + ((int64_t)n0 - 64) * a.ldp + k0;
        else pb = a.p[MODE == DX ? seg : 0] + (int64_t)k0 * a.ldp + n0;
        const uint16_t* qb = QK ? a.q[seg] + (int64_t)m0 * a.ldq + k0 : a.q[sel] + (int64_t)k0 * a.ldq + m0;
        cp.issue(pb, left, wave, P);
        cq.issue(qb, left, wave, Q);
    };
    auto row_of = [&](int t) { return MODE == FWD ? (t >> 1) * 64 + wn * 32 + (t & 1) * 16 : wn * 64 + t * 16; };

    f4v acc[4][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[n][m] = f4v{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int s, const Half& P, const Half& Q, Half& nP, Half& nQ) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0F70);           // vmcnt(0): this wave's copies of step s have landed
        lds_barrier();                                // every wave's have; step s - 1's tiles are free
        if (s + 1 < last) issue(s + 1, nP, nQ);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            bf8v pf[4], qf[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) pf[n] = fragment<PK>(P, 0, row_of(n), ks, lane);
#pragma unroll
            for (int m = 0; m < 4; ++m) qf[m] = fragment<QK>(Q, 0, wm * 64 + m * 16, ks, lane);
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 4; ++m) acc[n][m] = mfma(pf[n], qf[m], acc[n][m]);
        }
    };
    if (first < last) issue(first, P0, Q0);
    for (int s = first; s < last; s += 2) {
        step(s, P0, Q0, P1, Q1);
        if (s + 1 < last) step(s + 1, P1, Q1, P0, Q0);
    }

#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int row = m0 + wm * 64 + m * 16 + (lane & 15);
        const bool in = row < a.M;
        if constexpr (MODE == FWD) {
            const int nb = n0 + wn * 32;
            uint16_t* hr = in ? a.out[0] + (int64_t)row * a.N : nullptr;
            f4v h[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (a.saved) {
                    float* gr = in ? a.saved + (int64_t)row * a.N : nullptr;
                    float* ur = in ? a.saved + ((int64_t)a.M + row) * a.N : nullptr;
                    store_f4(gr, nb + 16 * t + 4 * (lane >> 4), a.N, acc[t][m]);
                    store_f4(ur, nb + 16 * t + 4 * (lane >> 4), a.N, acc[2 + t][m]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) h[t][e] = act<ACT>(acc[t][m][e]) * acc[2 + t][m][e];
            }
            store_pair(hr, nb, a.N, lane, h[0], h[1]);
        } else {
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                const int nb = n0 + wn * 64 + t * 16;
                if (MODE == DX && a.parts > 1) {
                    float* pr = in ? a.partial + ((int64_t)blockIdx.y * a.M + row) * a.N : nullptr;
                    store_f4(pr, nb + 4 * (lane >> 4), a.N, acc[t][m]);
                    store_f4(pr, nb + 16 + 4 * (lane >> 4), a.N, acc[t + 1][m]);
                } else {
                    store_pair(in ? a.out[sel] + (int64_t)row * a.N : nullptr, nb, a.N, lane, acc[t][m], acc[t + 1][m]);
                }
            }
        }
    }
}

// ---- 256 x 256 tiles ----------------------------------------------------------
// Four waves of 128 x 128 results, one to a SIMD: the results fill 256
// registers of a lane and every operand fragment serves 8 products, so that
// the reads from LDS take half as long as the products.  (Waves of 64 x 64
// read as long as they multiply.)  A lone wave hides nothing by itself, so the
// instructions are laid out by hand between single products.  A step of 64 k:
//   products of its k 0..31   | reads of its k 32..63, copies of Q of step s + 2
//   wait for step s + 1, barrier
//   products of its k 32..63  | reads of k 0..31 of step s + 1, copies of P of
//                               step s + 2 over P of step s
// LDS holds two stages of P and three of Q, all of its 160 KB: the third lets
// the copies run evenly, one in eight products.  (Sixteen in 64 products stall
// the wave at the copies; steps of 32 k with four stages of both operands read
// k-contiguous rows in halves of 128-byte lines, which costs as much.)
constexpr uint32_t kStage = 32768;                 // 256 rows or columns of one operand, 64 k
constexpr int kStagesP = 2, kStagesQ = 3;

// One wave's share of the copies of a stage: instructions 4 wave .. + 3 of
// each half, a half being 128 rows or columns, laid out like a Half.
template <bool KC> struct WideCopy {
    uint32_t off[8];      // byte offset from the tile's first element of the step
    int32_t kk;           // KC: first k that the lane's words hold
    uint64_t base;        // address of the step's first element
    int32_t left;         // k from there to the end
    int32_t ld2;          // bytes of a row
    // `rest` as `left` of Copy.  `pair`: the halves are 64 gate rows and 64 up
    // rows each, and the wave's are from one of the two matrices.
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t rest, bool pair) {
        ld2 = (int32_t)(2 * ld);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int half = i >> 2, q = 4 * wave + (i & 3);
            if constexpr (KC) {
                const int r0 = 8 * q + (lane >> 3), r = pair ? 64 * half + (r0 & 63) : 128 * half + r0;
                off[i] = r < rest ? (uint32_t)(r * ld * 2) + 16u * ((lane & 7) ^ (lane >> 3)) : kOutside;
            } else {
                const int k = 4 * q + (lane >> 4), col = 128 * half + 8 * ((lane & 15) ^ (2 * ((k & 3) | ((k >> 1) & 4))));
                off[i] = col < rest ? (uint32_t)(k * ld * 2) + col * 2u : kOutside;
            }
        }
        kk = 8 * ((lane & 7) ^ (lane >> 3));
    }
    __device__ __forceinline__ void start(const uint16_t* first, int k, int to_end) {
        base = reinterpret_cast<uint64_t>(first) + (KC ? 2 * (int64_t)k : (int64_t)k * ld2);
        left = to_end;
    }
    __device__ __forceinline__ void advance() {
        base += KC ? 2 * BK : (int64_t)BK * ld2;
        left -= BK;
    }
    // Buffer of the step: a k-strided operand's rows past k are beyond its range.
    __device__ __forceinline__ u4v buffer() const {
        const int range = KC || left >= BK ? (int)kOutside : max(left, 0) * ld2;
        return u4v{(uint32_t)base, (uint32_t)(base >> 32), (uint32_t)range, 0x00020000u};
    }
    // The lane's offset in copy i; a k-contiguous operand's words past k are outside.
    __device__ __forceinline__ uint32_t at(int i) const { return !KC || kk < left ? off[i] : kOutside; }
};

// Copies are written out, for the compiler would take every later read of LDS
// to depend on them; they have no output register, and the step's wait and
// barrier stand between them and the reads.  Lane l's 16 bytes go to byte
// `to` + 16 l of LDS.
__device__ __forceinline__ void copy_1k(uint32_t off, u4v buf, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(buf) : "memory");
}

// LDS addresses of a wave's fragments of one operand in a stage: rows
// (columns) 16 t .. + 15 of its half, k 32 ks .. + 31, as `fragment` has them.
template <bool KC> struct WideRead {
    uint32_t at[KC ? 2 : 8];       // KC: by ks; else by t, which the turn of a row's slots mixes with the lane
    __device__ __forceinline__ void init(uint32_t stage, int half, int lane) {
        const uint32_t i = lane & 15, h = lane >> 4;
#pragma unroll
        for (uint32_t e = 0; e < (KC ? 2 : 8); ++e)
            at[e] = stage + half * 16384u + (KC ? i * 128 + ((4 * e + h) ^ (i & 7)) * 16
                                                : (8 * h + (i >> 2)) * 256 + (e ^ ((i >> 2) | ((h & 1) << 2))) * 32 + (i & 3) * 8);
    }
    // part e of 8 of the way to another stage
    __device__ __forceinline__ void move(int e, uint32_t by) { if (e < (KC ? 2 : 8)) at[e] += by; }
    __device__ __forceinline__ bf8v get(int t, int ks) const {
        if constexpr (KC) {
            return *(__attribute__((address_space(3))) const bf8v*)(uintptr_t)(at[ks] + t * 2048);
        } else {
            const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(uintptr_t)(at[t] + ks * 8192));
            const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(uintptr_t)(at[t] + ks * 8192 + 1024));
            return __builtin_bit_cast(bf8v, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        }
    }
};

// A product whose sum stays where it is, in the upper half of the registers:
// left to itself the compiler moves results between the halves in every step.
// It does not see inside, so what the matrix cores ask for is kept here: an
// operand comes from LDS reads alone (which are waited for; an operand written
// by the vector units would need two wait states), and from the last product
// to a read of its result pass at least 18 states.
__device__ __forceinline__ void mfma_in_place(f4v& c, bf8v p, bf8v q) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(p), "v"(q));
}
// With a copy behind it, the product being the state that lies between a write
// of m0 and its use.
template <uint32_t TO> __device__ __forceinline__ void mfma_and_copy(f4v& c, bf8v p, bf8v q, uint32_t off, u4v buf, uint32_t to) {
    asm volatile("s_add_u32 m0, %3, %4\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\tbuffer_load_dwordx4 %5, %6, 0 offen lds"
                 : "+a"(c) : "v"(p), "v"(q), "s"(to), "i"(TO), "v"(off), "s"(buf) : "memory", "scc");
}
__device__ __forceinline__ void settle(f4v (&acc)[8][8]) {
    asm volatile("s_nop 15\ns_nop 15" ::: "memory");
#pragma unroll
    for (int n = 0; n < 8; ++n)
        asm volatile("" : "+a"(acc[n][0]), "+a"(acc[n][1]), "+a"(acc[n][2]), "+a"(acc[n][3]), "+a"(acc[n][4]), "+a"(acc[n][5]),
                     "+a"(acc[n][6]), "+a"(acc[n][7]));
    __builtin_amdgcn_sched_barrier(0);
}

// f of the constants 0, 1, ... in turn.
template <class F, int... I> __device__ __forceinline__ void in_turn(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

template <int MODE, int ACT> __global__ __launch_bounds__(256, 1) void k_gemm_wide(GemmArgs a) {
    constexpr bool PK = MODE == FWD, QK = MODE != DW;
    constexpr int kTileN = MODE == FWD ? 128 : 256;
    __shared__ __align__(1024) char lds[(kStagesP + kStagesQ) * kStage];
    int tn, tm;
    if (!tile_of(a, tn, tm)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int sel = MODE == DW && tm >= a.tiles_m / 2 ? 1 : 0;        // which weight's gradient
    const int n0 = tn * kTileN, m0 = (MODE == DW ? tm - sel * (a.tiles_m / 2) : tm) * 256;
    const int seg_steps = (a.K + BK - 1) / BK;
    const int all = MODE == DX ? 2 * seg_steps : seg_steps;
    const int first = MODE == DX ? (int)blockIdx.y * a.split_steps : 0;
    const int last = MODE == DX ? min(all, first + a.split_steps) : all;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;

    WideCopy<PK> cp;
    WideCopy<QK> cq;
    cp.init(wave, lane, a.ldp, (int64_t)a.N - n0, MODE == FWD);
    cq.init(wave, lane, a.ldq, (int64_t)a.M - m0, false);
    // first elements of both operands; DX goes on to the second pair where the first ends
    const uint16_t* p0 = a.p[MODE == FWD && wave >= 2 ? 1 : 0] + (PK ? (int64_t)n0 * a.ldp : n0);
    const uint16_t* q0 = a.q[sel] + (QK ? (int64_t)m0 * a.ldq : m0);
    const uint16_t* p1 = a.p[1] + (PK ? (int64_t)n0 * a.ldp : n0);
    const uint16_t* q1 = a.q[1] + (QK ? (int64_t)m0 * a.ldq : m0);
    {
        const int seg = MODE == DX && first >= seg_steps ? 1 : 0, k0 = (first - seg * seg_steps) * BK;
        cp.start(seg ? p1 : p0, k0, a.K - k0);
        cq.start(seg ? q1 : q0, k0, a.K - k0);
    }
    int sp = first, sq = first;                                       // the steps that cp and cq are at
    auto advance_p = [&] {
        cp.advance();
        if (MODE == DX && ++sp == seg_steps) cp.start(p1, 0, a.K);
    };
    auto advance_q = [&] {
        cq.advance();
        if (MODE == DX && ++sq == seg_steps) cq.start(q1, 0, a.K);
    };

    f4v acc[8][8];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int m = 0; m < 8; ++m) acc[n][m] = f4v{0.f, 0.f, 0.f, 0.f};
    bf8v pa[8], qa[8], pb[8], qb[8];
    uint32_t p = 0, q = kStagesP * kStage, q2 = q + 2 * kStage;       // stages of this step; of Q two steps on
    WideRead<PK> rp;
    WideRead<QK> rq;
    rp.init(lds0 + p, wn, lane);
    rq.init(lds0 + q, wm, lane);
    auto read = [&](int i, int ks, bf8v (&pf)[8], bf8v (&qf)[8]) {    // i: 0 .. 15
        if (i & 1) qf[i >> 1] = rq.get(i >> 1, ks);
        else pf[i >> 1] = rp.get(i >> 1, ks);
    };
    const uint32_t to0 = lds0 + (uint32_t)wave * 4096u;               // byte of LDS that the wave's copies start at
    auto copy_all = [&](const auto& c, uint32_t stage) {
        const u4v buf = c.buffer();
#pragma unroll
        for (int i = 0; i < 8; ++i) copy_1k(c.at(i), buf, to0 + stage + (i >> 2) * 16384u + (i & 3) * 1024u);
    };
    copy_all(cp, p);
    copy_all(cq, q);
    advance_q();
    copy_all(cq, q + kStage);
    advance_p();
    copy_all(cp, p + kStage);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x4F70);               // vmcnt(16): this wave's copies of the first step have landed
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 16; ++i) read(i, 0, pa, qa);

    // Product i of 64, in blocks of 2 x 2: a fragment's first use comes after
    // its read in the order of `read`.  One in eight has a copy behind it.
    auto products = [&](const bf8v (&pf)[8], const bf8v (&qf)[8], const auto& copies, const u4v& buf, uint32_t stage, auto&& between) {
        auto one = [&](auto index) {
            constexpr int i = decltype(index)::value, c = i >> 3;
            constexpr int n = 2 * (i >> 4) + ((i >> 1) & 1), m = 2 * ((i >> 2) & 3) + (i & 1);
            between(i);
            if constexpr (i % 8 == 5) mfma_and_copy<(c >> 2) * 16384u + (c & 3) * 1024u>(acc[n][m], pf[n], qf[m], copies.at(c), buf, to0 + stage);
            else mfma_in_place(acc[n][m], pf[n], qf[m]);
            __builtin_amdgcn_sched_barrier(0);
        };
        in_turn(one, std::make_integer_sequence<int, 64>{});
    };
    advance_q();
    u4v bufp, bufq = cq.buffer();
    for (int s = first; s < last; ++s) {
        const uint32_t np = p ^ kStage, nq = q == (kStagesP + kStagesQ - 1) * kStage ? kStagesP * kStage : q + kStage;
        products(pa, qa, cq, bufq, q2, [&](int i) {
            if (i % 3 == 0 && i < 48) read(i / 3, 1, pb, qb);
            if (i == 50) advance_p();
            if (i == 54) bufp = cp.buffer();
            if (i >= 56) { rp.move(i - 56, np - p); rq.move(i - 56, nq - q); }
        });
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0078);           // vmcnt(8), lgkmcnt(0): step s + 1 has landed, step s is read
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        products(pb, qb, cp, bufp, p, [&](int i) {
            if (i % 4 == 0) read(i / 4, 0, pa, qa);
            if (i == 42) advance_q();
            if (i == 50) bufq = cq.buffer();
        });
        q2 = q;                                       // step s + 3 takes the stage of step s
        p = np;
        q = nq;
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);               // the copies past the last step write LDS too
    settle(acc);

#pragma unroll
    for (int m = 0; m < 8; ++m) {
        const int row = m0 + wm * 128 + m * 16 + (lane & 15);
        const bool in = row < a.M;
        if constexpr (MODE == FWD) {
            const int nb = n0 + wn * 64;
            uint16_t* hr = in ? a.out[0] + (int64_t)row * a.N : nullptr;
            float* gr = in && a.saved ? a.saved + (int64_t)row * a.N : nullptr;
            float* ur = in && a.saved ? a.saved + ((int64_t)a.M + row) * a.N : nullptr;
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                f4v h[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    store_f4(gr, nb + 16 * (t + e) + 4 * (lane >> 4), a.N, acc[t + e][m]);
                    store_f4(ur, nb + 16 * (t + e) + 4 * (lane >> 4), a.N, acc[4 + t + e][m]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[e][j] = act<ACT>(acc[t + e][m][j]) * acc[4 + t + e][m][j];
                }
                store_pair(hr, nb + 16 * t, a.N, lane, h[0], h[1]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 8; t += 2) {
                const int nb = n0 + wn * 128 + t * 16;
                if (MODE == DX && a.parts > 1) {
                    float* pr = in ? a.partial + ((int64_t)blockIdx.y * a.M + row) * a.N : nullptr;
                    store_f4(pr, nb + 4 * (lane >> 4), a.N, acc[t][m]);
                    store_f4(pr, nb + 16 + 4 * (lane >> 4), a.N, acc[t + 1][m]);
                } else {
                    store_pair(in ? a.out[sel] + (int64_t)row * a.N : nullptr, nb, a.N, lane, acc[t][m], acc[t + 1][m]);
                }
            }
        }
    }
}

// dg = dh u act'(g), du = dh act(g), 8 elements per thread.  HBM bounds it:
// 10 bytes read and 4 written per element.
template <int ACT> __global__ __launch_bounds__(256) void k_gate_grad(const uint16_t* dh, const float* saved, uint16_t* dg, uint16_t* du,
                                                                      int64_t n) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        const u4v d = *reinterpret_cast<const u4v*>(dh + i);
        f4v g[2], u[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            g[k] = *reinterpret_cast<const f4v*>(saved + i + 4 * k);
            u[k] = *reinterpret_cast<const f4v*>(saved + n + i + 4 * k);
        }
        u4v og, ou;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float rg[2], ru[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float x = __uint_as_float(e ? d[k] & 0xFFFF0000u : d[k] << 16);
                float f, df;
                act_slope<ACT>(g[k >> 1][2 * (k & 1) + e], f, df);
                rg[e] = x * u[k >> 1][2 * (k & 1) + e] * df;
                ru[e] = x * f;
            }
            og[k] = bf16_pair(rg[0], rg[1]);
            ou[k] = bf16_pair(ru[0], ru[1]);
        }
        *reinterpret_cast<u4v*>(dg + i) = og;
        *reinterpret_cast<u4v*>(du + i) = ou;
    }
}

// The parts of dx added in order and rounded, 8 elements per thread.
__global__ __launch_bounds__(256) void k_join(const float* partial, int parts, int64_t n, uint16_t* out) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        f4v s0 = *reinterpret_cast<const f4v*>(partial + i), s1 = *reinterpret_cast<const f4v*>(partial + i + 4);
        for (int p = 1; p < parts; ++p) {
            s0 += *reinterpret_cast<const f4v*>(partial + p * n + i);
            s1 += *reinterpret_cast<const f4v*>(partial + p * n + i + 4);
        }
        *reinterpret_cast<u4v*>(out + i) = u4v{bf16_pair(s0[0], s0[1]), bf16_pair(s0[2], s0[3]), bf16_pair(s1[0], s1[1]),
                                              bf16_pair(s1[2], s1[3])};
    }
}

__global__ __launch_bounds__(256) void k_clear(uint16_t* out, int64_t n) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8)
        *reinterpret_cast<u4v*>(out + i) = u4v{0u, 0u, 0u, 0u};
}

unsigned wide_grid(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n / 8 + 255) / 256, 8192)); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 256 where they fill the GPU.
#ifndef FORCE
#define FORCE -1
#endif
bool wide_tiles(int64_t N, int64_t M, int mode) {
    if (FORCE >= 0) return FORCE;
    return ceil_div(N, mode == FWD ? 128 : 256) * ceil_div(M, 256) * (mode == DW ? 2 : 1) >= 224;
}

hipError_t clear(void* p, int64_t n, hipStream_t s) {
    if (!p || n == 0) return hipSuccess;
    k_clear<<<wide_grid(n), 256, 0, s>>>(static_cast<uint16_t*>(p), n);
    return hipGetLastError();
}

template <int MODE, int ACT> hipError_t run_gemm(GemmArgs& a, hipStream_t s) {
    const int64_t side = wide_tiles(a.N, a.M, MODE) ? 256 : 128;
    const int64_t tiles_n = ceil_div(a.N, MODE == FWD ? side / 2 : side), tiles_m = ceil_div(a.M, side) * (MODE == DW ? 2 : 1);
    const int64_t tiles = tiles_n * tiles_m;
    if (tiles > ((int64_t)1 << 31) - 64) return hipErrorInvalidConfiguration;
    a.tiles_n = (int32_t)tiles_n;
    a.tiles_m = (int32_t)tiles_m;
    a.tiles = (uint32_t)tiles;
    a.per_xcd = (int32_t)ceil_div(tiles, 8);
    const dim3 grid((unsigned)(8 * (int64_t)a.per_xcd), MODE == DX ? a.parts : 1);
    if (side == 256) k_gemm_wide<MODE, ACT><<<grid, 256, 0, s>>>(a);
    else k_gemm<MODE, ACT><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

// Parts of dx's sum: enough workgroups for two per CU, at least 8 steps each.
int dx_parts(int64_t tokens, int64_t cols, int64_t features) {
    const bool wide = wide_tiles(cols, tokens, DX);
    const int64_t side = wide ? 256 : 128, tiles = ceil_div(tokens, side) * ceil_div(cols, side), steps = 2 * ceil_div(features, BK);
    return (int)std::max<int64_t>(1, std::min<int64_t>({(wide ? 256 : 512) / std::max<int64_t>(1, tiles), steps / 8, 16}));
}

constexpr int64_t kAlign = 256;
int64_t plane_bytes(int64_t tokens, int64_t features) { return ceil_div(tokens * features * 2, kAlign) * kAlign; }

}  // namespace

size_t gated_workspace_bytes(int64_t tokens, int64_t cols, int64_t features) {
    const int parts = dx_parts(tokens, cols, features);
    return (size_t)(2 * plane_bytes(tokens, features) + (parts > 1 ? parts * tokens * cols * 4 : 0));
}

hipError_t launch_gated(const GatedArgs& g, hipStream_t s) {
    if (g.tokens <= kPackedTokens) {
        PackedArgs p = {};
        p.fmt = F_BF16W; p.gated = true; p.act = g.act;
        p.w[0].codes = g.wg; p.w[1].codes = g.wu;
        p.x = g.x; p.ldx = g.ldx; p.out = g.h; p.out_dtype = D_BF16; p.saved = g.saved;
        p.n0 = g.features; p.n1 = g.tokens; p.K = g.cols;
        return launch_packed(p, s);
    }
    GemmArgs a = {};
    a.p[0] = static_cast<const uint16_t*>(g.wg); a.p[1] = static_cast<const uint16_t*>(g.wu);
    a.q[0] = a.q[1] = static_cast<const uint16_t*>(g.x);
    a.ldp = g.cols; a.ldq = g.ldx;
    a.N = (int32_t)g.features; a.M = (int32_t)g.tokens; a.K = (int32_t)g.cols;
    a.out[0] = static_cast<uint16_t*>(g.h);
    a.saved = g.saved;
    if (g.act == A_SILU) return run_gemm<FWD, A_SILU>(a, s);
    if (g.act == A_GELU) return run_gemm<FWD, A_GELU>(a, s);
    return run_gemm<FWD, A_GELU_TANH>(a, s);
}

hipError_t launch_gated_grad(const GatedGradArgs& g, hipStream_t s) {
    const int64_t tf = g.tokens * g.features;
    if (tf == 0 || g.cols == 0) {           // sums of nothing
        hipError_t e = clear(g.dx, g.tokens * g.cols, s);
        if (e == hipSuccess) e = clear(g.dwg, g.features * g.cols, s);
        return e == hipSuccess ? clear(g.dwu, g.features * g.cols, s) : e;
    }
    if (!g.dx && !g.dwg) return hipSuccess;
    char* ws = static_cast<char*>(g.workspace);
    uint16_t* dg = reinterpret_cast<uint16_t*>(ws);
    uint16_t* du = reinterpret_cast<uint16_t*>(ws + plane_bytes(g.tokens, g.features));
    const uint16_t* dh = static_cast<const uint16_t*>(g.dh);
    if (g.act == A_SILU) k_gate_grad<A_SILU><<<wide_grid(tf), 256, 0, s>>>(dh, g.saved, dg, du, tf);
    else if (g.act == A_GELU) k_gate_grad<A_GELU><<<wide_grid(tf), 256, 0, s>>>(dh, g.saved, dg, du, tf);
    else k_gate_grad<A_GELU_TANH><<<wide_grid(tf), 256, 0, s>>>(dh, g.saved, dg, du, tf);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (g.dx) {
        GemmArgs a = {};
        a.p[0] = static_cast<const uint16_t*>(g.wg); a.p[1] = static_cast<const uint16_t*>(g.wu);
        a.q[0] = dg; a.q[1] = du;
        a.ldp = g.cols; a.ldq = g.features;
        a.N = (int32_t)g.cols; a.M = (int32_t)g.tokens; a.K = (int32_t)g.features;
        a.out[0] = static_cast<uint16_t*>(g.dx);
        a.parts = dx_parts(g.tokens, g.cols, g.features);
        a.split_steps = (int32_t)ceil_div(2 * ceil_div(g.features, BK), a.parts);
        a.partial = reinterpret_cast<float*>(ws + 2 * plane_bytes(g.tokens, g.features));
        e = run_gemm<DX, 0>(a, s);
        if (e != hipSuccess) return e;
        if (a.parts > 1) {
            const int64_t n = g.tokens * g.cols;
            k_join<<<wide_grid(n), 256, 0, s>>>(a.partial, a.parts, n, a.out[0]);
            if ((e = hipGetLastError()) != hipSuccess) return e;
        }
    }
    if (g.dwg) {
        GemmArgs a = {};
        a.p[0] = static_cast<const uint16_t*>(g.x);
        a.q[0] = dg; a.q[1] = du;
        a.ldp = g.ldx; a.ldq = g.features;
        a.N = (int32_t)g.cols; a.M = (int32_t)g.features; a.K = (int32_t)g.tokens;
        a.out[0] = static_cast<uint16_t*>(g.dwg); a.out[1] = static_cast<uint16_t*>(g.dwu);
        e = run_gemm<DW, 0>(a, s);
    }
    return e;
}

}  // namespace iqk
