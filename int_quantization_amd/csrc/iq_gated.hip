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
//
// Measured at 4096 tokens, 4096 x 14336, back to back, BF16: forward 650 us
// (1.48 PFLOP/s), with g and u saved in FP32 740 (the stores of 587 MB come
// at the end of every tile), dx 620 (1.55), both weight gradients 660 (1.46);
// a large library product reaches 1.4 to 1.6 here.  The matrix cores are busy
// four fifths of the cycles, and the clock gives way under that load, from 2.4
// to 1.85 - 2.1 GHz, so power bounds these and fewer stalls no longer show.
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
    int32_t N, M, K;              // of one of the two weights; N of this launch's columns
    int64_t ldo;                  // elements of a row of C
    int32_t tiles_n, tiles_m;     // tiles_m counts both weights in DW
    uint32_t tiles;
    int32_t per_xcd;
    int32_t split_steps;          // DX, DW: steps of one part of k
    int32_t parts;                // DX, DW: parts of k; above 1 the sums go to `partial`
    uint16_t* out[2];
    float* saved;                 // FWD: g and u [2][M][N], may be null
    float* partial;               // DX: [parts][M][N], DW: [parts][2][M][N]
};

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

// Tiles of 2 W x 2 W results, W = 16 T: four waves of W x W.
//
// T = 8, one workgroup on a CU: the results fill 256 registers of a lane and
// every operand fragment serves 8 products, so that the reads from LDS take
// half as long as the products.  A lone wave on a SIMD hides nothing by
// itself, so the instructions are laid out by hand between single products.
// A step of 64 k, with copies A = AHEAD steps ahead:
//   products of its k 0..31   | reads of its k 32..63, copies of Q of step s + A
//   wait for step s + 1, barrier
//   products of its k 32..63  | reads of k 0..31 of step s + 1, copies of P of
//                               step s + A over P of step s
// A is 2: LDS holds two stages of P and three of Q, all of its 160 KB.  The
// third lets the copies run evenly, one in eight products.  (Sixteen in 64 products stall
// the wave at the copies; steps of 32 k with four stages of both operands read
// k-contiguous rows in halves of 128-byte lines, which costs as much.)
//
// T = 4, two workgroups on a CU (or one, and A = 4): the same for grids that
// T = 8 leaves too small; the reads take as long as the products.  (1024 tokens, 1024 x 1024,
// forward: 10 us, and 26 with T = 8, whose prologue alone takes 10.)

// A half of a stage: W rows (columns) by 64 k of one operand.
//   k-contiguous: 16-byte slot s of row r at slot s ^ (r & 7) of its 128 bytes;
//   k-strided:    32-byte slot c of row k at slot c ^ turn(k) of its 2 W
//                 bytes, so that the 8 rows that half a wave reads at a time
//                 (k 0-3 and 8-11 and so on) are in different banks.
template <int T> constexpr uint32_t kHalf = 2048 * T;
template <int T> __device__ __forceinline__ int turn(int k) {
    return T == 8 ? (k & 3) | ((k >> 1) & 4) : ((k >> 1) & 1) | ((k >> 2) & 2);
}

// One wave's share of the copies of a stage: T / 2 instructions of each half.
template <bool KC, int T> struct Copy {
    static constexpr int NI = T / 2;
    uint32_t off[T];      // byte offset from the tile's first element of the step
    int32_t kk;           // KC: first k that the lane's words hold
    uint64_t base;        // address of the step's first element
    int32_t left;         // k from there to the end
    int32_t ld2;          // bytes of a row
    // `rest`: rows (KC) or columns (else) from the tile's first to the
    // matrix's last.  `pair`: the halves are W / 2 gate rows and W / 2 up rows
    // each, and the wave's are from one of the two matrices.
    __device__ __forceinline__ void init(int wave, int lane, int64_t ld, int64_t rest, bool pair) {
        ld2 = (int32_t)(2 * ld);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int half = i / NI, q = NI * wave + i % NI;
            if constexpr (KC) {
                const int r0 = 8 * q + (lane >> 3), r = pair ? 8 * T * half + (r0 & (8 * T - 1)) : 16 * T * half + r0;
                off[i] = r < rest ? (uint32_t)(r * ld * 2) + 16u * ((lane & 7) ^ (lane >> 3)) : kOutside;
            } else {
                const int k = (32 / T) * q + lane / (2 * T), col = 16 * T * half + 8 * ((lane & (2 * T - 1)) ^ (2 * turn<T>(k)));
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
    // The byte of copy i in a stage, from that of the wave's first.
    static constexpr uint32_t to(int i) { return (i / NI) * kHalf<T> + (i % NI) * 1024u; }
};

// Copies are written out, for the compiler would take every later read of LDS
// to depend on them; they have no output register, and the step's wait and
// barrier stand between them and the reads.  Lane l's 16 bytes go to byte
// `to` + 16 l of LDS.
// m0 is the compiler's reserved register and cannot be named as overwritten:
// every copy sets it anew, and nothing else in the kernel may use it.
__device__ __forceinline__ void copy_1k(uint32_t off, u4v buf, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(buf) : "memory");
}

// LDS addresses of a wave's fragments of one operand in a stage: fragment t is
// rows (columns) 16 t .. + 15 of its half; lane l has row 16 t + l % 16 and
// k 32 ks + 8 (l / 16) .. + 7.
template <bool KC, int T> struct Read {
    uint32_t at[KC ? 2 : T];       // KC: by ks; else by t, which the turn of a row's slots mixes with the lane
    __device__ __forceinline__ void init(uint32_t stage, int half, int lane) {
        const uint32_t i = lane & 15, h = lane >> 4;
#pragma unroll
        for (uint32_t e = 0; e < (KC ? 2 : T); ++e)
            at[e] = stage + half * kHalf<T> + (KC ? i * 128 + ((4 * e + h) ^ (i & 7)) * 16
                                                  : (8 * h + (i >> 2)) * (32 * T) + (e ^ turn<T>(8 * h + (i >> 2))) * 32 + (i & 3) * 8);
    }
    // part e of T of the way to another stage
    __device__ __forceinline__ void move(int e, uint32_t by) { if (e < (KC ? 2 : T)) at[e] += by; }
    __device__ __forceinline__ bf8v get(int t, int ks) const {
        if constexpr (KC) {
            return *(__attribute__((address_space(3))) const bf8v*)(uintptr_t)(at[ks] + t * 2048);
        } else {
            // the transposing read gives lane i of 16 element i of the four
            // rows that its group's lanes 4 j + c name by column 4 c of row j;
            // four rows on, a row's slots are turned alike
            const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(uintptr_t)(at[t] + ks * 1024 * T));
            const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(uintptr_t)(at[t] + ks * 1024 * T + 128 * T));
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
template <int T> __device__ __forceinline__ void settle(f4v (&acc)[T][T]) {
    asm volatile("s_nop 15\ns_nop 15" ::: "memory");
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
        for (int m = 0; m < T; m += 4) asm volatile("" : "+a"(acc[n][m]), "+a"(acc[n][m + 1]), "+a"(acc[n][m + 2]), "+a"(acc[n][m + 3]));
    __builtin_amdgcn_sched_barrier(0);
}

// f of the constants 0, 1, ... in turn.
template <class F, int... I> __device__ __forceinline__ void in_turn(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

template <int MODE, int ACT, int T, int AHEAD> __global__ __launch_bounds__(256, T == 8 || AHEAD > 2 ? 1 : 2) void k_gemm(GemmArgs a) {
    constexpr bool PK = MODE == FWD, QK = MODE != DW;
    constexpr int W = 16 * T, kTileN = MODE == FWD ? W : 2 * W;
    constexpr uint32_t kStage = 2 * kHalf<T>;
    constexpr int kStagesP = AHEAD, kStagesQ = AHEAD + 1;
    __shared__ __align__(1024) char lds[(kStagesP + kStagesQ) * kStage];
    int tn, tm;
    if (!tile_of(a, tn, tm)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wm = wave >> 1;
    const int sel = MODE == DW && tm >= a.tiles_m / 2 ? 1 : 0;        // which weight's gradient
    const int n0 = tn * kTileN, m0 = (MODE == DW ? tm - sel * (a.tiles_m / 2) : tm) * 2 * W;
    const int seg_steps = (a.K + BK - 1) / BK;
    const int all = MODE == DX ? 2 * seg_steps : seg_steps;
    const int first = MODE == FWD ? 0 : (int)blockIdx.y * a.split_steps;
    const int last = MODE == FWD ? all : min(all, first + a.split_steps);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_void*)lds;

    Copy<PK, T> cp;
    Copy<QK, T> cq;
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

    f4v acc[T][T];
#pragma unroll
    for (int n = 0; n < T; ++n)
#pragma unroll
        for (int m = 0; m < T; ++m) acc[n][m] = f4v{0.f, 0.f, 0.f, 0.f};
    bf8v pa[T], qa[T], pb[T], qb[T];
    uint32_t p = 0, q = kStagesP * kStage, q2 = q + AHEAD * kStage;   // stages of this step; of Q's copies
    Read<PK, T> rp;
    Read<QK, T> rq;
    rp.init(lds0 + p, wn, lane);
    rq.init(lds0 + q, wm, lane);
    auto read = [&](int i, int ks, bf8v (&pf)[T], bf8v (&qf)[T]) {    // i: 0 .. 2 T - 1
        if (i & 1) qf[i >> 1] = rq.get(i >> 1, ks);
        else pf[i >> 1] = rp.get(i >> 1, ks);
    };
    const uint32_t to0 = lds0 + (uint32_t)wave * (512u * T);              // byte of LDS that the wave's copies start at
    auto copy_all = [&](const auto& c, uint32_t stage) {
        const u4v buf = c.buffer();
#pragma unroll
        for (int i = 0; i < T; ++i) copy_1k(c.at(i), buf, to0 + stage + c.to(i));
    };
    copy_all(cp, p);
    copy_all(cq, q);
#pragma unroll
    for (int d = 1; d < AHEAD; ++d) {
        advance_q();
        copy_all(cq, q + d * kStage);
        advance_p();
        copy_all(cp, p + d * kStage);
    }
    wait_for_all_but<2 * (AHEAD - 1) * T>();          // this wave's copies of the first step have landed
    lds_barrier();
#pragma unroll
    for (int i = 0; i < 2 * T; ++i) read(i, 0, pa, qa);

    // Product i of T^2, in blocks of 2 x 2: a fragment's first use comes after
    // its read in the order of `read`.  One in T has a copy behind it.
    auto products = [&](const bf8v (&pf)[T], const bf8v (&qf)[T], const auto& copies, const u4v& buf, uint32_t stage, auto&& between) {
        auto one = [&](auto index) {
            constexpr int i = decltype(index)::value, c = i / T;
            constexpr int n = 2 * (i / (2 * T)) + ((i >> 1) & 1), m = 2 * ((i >> 2) % (T / 2)) + (i & 1);
            between(i);
            if constexpr (i % T == T - 3) mfma_and_copy<Copy<true, T>::to(c)>(acc[n][m], pf[n], qf[m], copies.at(c), buf, to0 + stage);
            else mfma_in_place(acc[n][m], pf[n], qf[m]);
            __builtin_amdgcn_sched_barrier(0);
        };
        in_turn(one, std::make_integer_sequence<int, T * T>{});
    };
    // reads: all of a step's before its wait, and spread over what follows it
    constexpr int kBefore = T == 8 ? 3 : 1, kAfter = T == 8 ? 4 : 1, kEnd = T * T;
    advance_q();
    u4v bufp, bufq = cq.buffer();
    // One step at least: a part without any adds zeros, and the results reach
    // `settle` from the loop alone, without copies that would read them early.
    int s = first;
    do {
        const uint32_t np = p == (kStagesP - 1) * kStage ? 0 : p + kStage, nq = q == (kStagesP + kStagesQ - 1) * kStage ? kStagesP * kStage : q + kStage;
        products(pa, qa, cq, bufq, q2, [&](int i) {
            if (i % kBefore == 0 && i < 2 * T * kBefore) read(i / kBefore, 1, pb, qb);
            if (i == kEnd - T - 6) advance_p();
            if (i == kEnd - T - 2) bufp = cp.buffer();
            if (i >= kEnd - T) { rp.move(i - kEnd + T, np - p); rq.move(i - kEnd + T, nq - q); }
        });
        __builtin_amdgcn_s_waitcnt(0xC07F);           // lgkmcnt(0): step s is read
        wait_for_all_but<(2 * AHEAD - 3) * T>();      // step s + 1 has landed
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        products(pb, qb, cp, bufp, p, [&](int i) {
            if (i % kAfter == 0 && i < 2 * T * kAfter) read(i / kAfter, 0, pa, qa);
            if (i == kEnd - T - 6) advance_q();
            if (i == kEnd - T - 2) bufq = cq.buffer();
        });
        q2 = q;                                       // the next step's copies of Q take the stage of this
        p = np;
        q = nq;
    } while (++s < last);
    settle<T>(acc);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70);               // the copies past the last step write LDS too

#pragma unroll
    for (int m = 0; m < T; ++m) {
        const int row = m0 + wm * W + m * 16 + (lane & 15);
        const bool in = row < a.M;
        if constexpr (MODE == FWD) {
            const int nb = n0 + wn * (W / 2);
            uint16_t* hr = in ? a.out[0] + (int64_t)row * a.ldo : nullptr;
            float* gr = in && a.saved ? a.saved + (int64_t)row * a.ldo : nullptr;
            float* ur = in && a.saved ? a.saved + ((int64_t)a.M + row) * a.ldo : nullptr;
#pragma unroll
            for (int t = 0; t < T / 2; t += 2) {
                f4v h[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    store_f4(gr, nb + 16 * (t + e) + 4 * (lane >> 4), a.N, acc[t + e][m]);
                    store_f4(ur, nb + 16 * (t + e) + 4 * (lane >> 4), a.N, acc[T / 2 + t + e][m]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[e][j] = act<ACT>(acc[t + e][m][j]) * acc[T / 2 + t + e][m][j];
                }
                store_pair(hr, nb + 16 * t, a.N, lane, h[0], h[1]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < T; t += 2) {
                const int nb = n0 + wn * W + t * 16;
                if (a.parts > 1) {
                    float* pr = in ? a.partial + (((int64_t)blockIdx.y * (MODE == DW ? 2 : 1) + sel) * a.M + row) * a.ldo : nullptr;
                    store_f4(pr, nb + 4 * (lane >> 4), a.N, acc[t][m]);
                    store_f4(pr, nb + 16 + 4 * (lane >> 4), a.N, acc[t + 1][m]);
                } else {
                    store_pair(in ? a.out[sel] + (int64_t)row * a.ldo : nullptr, nb, a.N, lane, acc[t][m], acc[t + 1][m]);
                }
            }
        }
    }
}

// dg = dh u act'(g), du = dh act(g), 8 elements per thread.  HBM bounds it:
// 10 bytes read and 4 written per element (4096 x 14336: 155 us, 5.3 TB/s).
// Both are rounded to BF16, the type that the matrix cores take; two BF16 parts
// of each would double the products.  The gradients are off by 0.0023 of their
// norm that way, 0.0017 of which their own rounding to BF16 costs already.
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

// The parts of a product added in order and rounded, 8 elements per thread;
// elements from `first` on go to the second output.
__global__ __launch_bounds__(256) void k_join(const float* partial, int parts, int64_t n, int64_t first, uint16_t* out, uint16_t* second) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8) {
        f4v s0 = *reinterpret_cast<const f4v*>(partial + i), s1 = *reinterpret_cast<const f4v*>(partial + i + 4);
        for (int p = 1; p < parts; ++p) {
            s0 += *reinterpret_cast<const f4v*>(partial + p * n + i);
            s1 += *reinterpret_cast<const f4v*>(partial + p * n + i + 4);
        }
        *reinterpret_cast<u4v*>(i < first ? out + i : second + (i - first)) =
            u4v{bf16_pair(s0[0], s0[1]), bf16_pair(s0[2], s0[3]), bf16_pair(s1[0], s1[1]), bf16_pair(s1[2], s1[3])};
    }
}

__global__ __launch_bounds__(256) void k_clear(uint16_t* out, int64_t n) {
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (int64_t)gridDim.x * 256 * 8)
        *reinterpret_cast<u4v*>(out + i) = u4v{0u, 0u, 0u, 0u};
}

unsigned wide_grid(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n / 8 + 255) / 256, 8192)); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

hipError_t clear(void* p, int64_t n, hipStream_t s) {
    if (!p || n == 0) return hipSuccess;
    k_clear<<<wide_grid(n), 256, 0, s>>>(static_cast<uint16_t*>(p), n);
    return hipGetLastError();
}

// Tiles of one product and the parts of its sum.  T = 8 where its tiles fill
// the GPU (2048 tokens, 2048 x 8192, forward, 512 tiles: 110 us, 123 with
// T = 4; 1024 tokens, 4096 x 4096, 128 tiles: 78 and 61).  Else T = 4 and, for
// the gradients, the sum split into parts of 8 steps and more until every CU
// has a workgroup (8192 tokens, 256 x 512, the weights' gradients: 88 us in one
// part, 31 in 16; two workgroups to a CU: x's gradient at 512 tokens, 8192 x
// 1024, 33 us, 23 with one).
//
// T = 4 tiles that have their CU alone keep four steps ahead instead of two
// where the sum is long enough to gain from it (512 tokens, 8192 x 1024,
// forward, 128 steps: 44 us, 56 with two; 1024 tokens, 1024 x 1024, 16 steps:
// 10.3 and 9.8).
//
// T = 8 tiles take a CU each, so 256 of them are a round.  Where the last round
// would be half full or less, its columns go to T = 4 tiles, a quarter as large
// and two to a CU, in a launch of their own (1000 tokens, 4096 x 10000,
// forward: 129 us, 159 without; 2048 tokens, 4096 x 14336: 354 and 361).
struct Plan {
    int T, parts, ahead;
    int32_t tail;          // columns left to T = 4
};
Plan plan(int mode, int64_t N, int64_t M, int64_t K) {
    const int64_t width = mode == FWD ? 128 : 256, both = mode == DW ? 2 : 1;
    const int64_t tiles_n = ceil_div(N, width), tiles_m = ceil_div(M, 256) * both, tiles = tiles_n * tiles_m;
    const int64_t steps = ceil_div(K, BK) * (mode == DX ? 2 : 1);
    Plan p = {8, 1, 2, 0};
    if (tiles >= 224) {
        const int64_t over = tiles % 256;
        if (tiles > 256 && over > 0 && over <= 128) {
            const int64_t first = (tiles - over) / tiles_m * width, rest = N - first;
            if (first > 0 && ceil_div(rest, width / 2) * ceil_div(M, 128) * both <= 512) p.tail = (int32_t)rest;
        }
    } else {
        p.T = 4;
        const int64_t small = std::max<int64_t>(1, ceil_div(N, width / 2) * ceil_div(M, 128) * both);
        if (mode != FWD) p.parts = (int)std::max<int64_t>(1, std::min<int64_t>({256 / small, steps / 8, 16}));
        if (small * p.parts <= 256 && steps / p.parts >= 20) p.ahead = 4;
    }
    return p;
}

// Bytes of the parts' sums.
int64_t part_bytes(int mode, int64_t N, int64_t M, int64_t K) {
    const int parts = plan(mode, N, M, K).parts;
    return parts > 1 ? parts * M * N * 4 * (mode == DW ? 2 : 1) : 0;
}

template <int MODE, int ACT, int T, int AHEAD> hipError_t run_tiles(GemmArgs a, int64_t parts, hipStream_t s) {
    const int64_t tiles_n = ceil_div(a.N, (MODE == FWD ? 16 : 32) * T), tiles_m = ceil_div(a.M, 32 * T) * (MODE == DW ? 2 : 1);
    const int64_t tiles = tiles_n * tiles_m;
    if (tiles > ((int64_t)1 << 24) - 64) return hipErrorInvalidConfiguration;      // 256 threads each, counted in 32 bits
    a.tiles_n = (int32_t)tiles_n;
    a.tiles_m = (int32_t)tiles_m;
    a.tiles = (uint32_t)tiles;
    a.per_xcd = (int32_t)ceil_div(tiles, 8);
    k_gemm<MODE, ACT, T, AHEAD><<<dim3((unsigned)(8 * (int64_t)a.per_xcd), (unsigned)parts), 256, 0, s>>>(a);
    return hipGetLastError();
}

template <int MODE, int ACT> hipError_t run_gemm(GemmArgs& a, hipStream_t s) {
    const Plan p = plan(MODE, a.N, a.M, a.K);
    const int64_t steps = ceil_div(a.K, BK) * (MODE == DX ? 2 : 1), n = (int64_t)a.M * a.N;
    a.parts = p.parts;
    a.split_steps = (int32_t)ceil_div(steps, p.parts);
    a.ldo = a.N;
    hipError_t e;
    if (p.T == 4) {
        e = p.ahead == 4 ? run_tiles<MODE, ACT, 4, 4>(a, p.parts, s) : run_tiles<MODE, ACT, 4, 2>(a, p.parts, s);
    } else if (p.tail == 0) {
        e = run_tiles<MODE, ACT, 8, 2>(a, p.parts, s);
    } else {
        const int32_t first = a.N - p.tail;
        GemmArgs t = a;
        a.N = first;
        if ((e = run_tiles<MODE, ACT, 8, 2>(a, 1, s)) != hipSuccess) return e;
        t.N = p.tail;
        for (int w = 0; w < 2; ++w) {
            t.p[w] += MODE == FWD ? first * t.ldp : first;
            if (t.out[w]) t.out[w] += first;
        }
        if (t.saved) t.saved += first;
        return run_tiles<MODE, ACT, 4, 2>(t, 1, s);
    }
    if (e != hipSuccess || p.parts == 1) return e;
    k_join<<<wide_grid(n * (MODE == DW ? 2 : 1)), 256, 0, s>>>(a.partial, p.parts, n * (MODE == DW ? 2 : 1), n, a.out[0], a.out[1]);
    return hipGetLastError();
}

constexpr int64_t kAlign = 256;
int64_t plane_bytes(int64_t tokens, int64_t features) { return ceil_div(tokens * features * 2, kAlign) * kAlign; }

}  // namespace

// dg and du, then the parts of dx, and after it those of dw_gate and dw_up.
size_t gated_workspace_bytes(int64_t tokens, int64_t cols, int64_t features) {
    return (size_t)(2 * plane_bytes(tokens, features) +
                    std::max(part_bytes(DX, cols, tokens, features), part_bytes(DW, cols, features, tokens)));
}

hipError_t launch_gated(const GatedArgs& g, hipStream_t s) {
    // A few tokens go with the weights' rows, 16 to a workgroup.  Beyond one
    // tile of 16 tokens, 64 to a workgroup are faster once they fill the GPU
    // (33 tokens, 4096 x 14336: 59 us by 16 rows, 37 by 64; 8192 x 28672: 253
    // and 182; 8192 x 8192: 61 and 83).
    if (g.tokens <= 16 || (g.tokens <= kPackedTokens && ceil_div(g.features, 64) < 192)) {
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
    float* partial = reinterpret_cast<float*>(ws + 2 * plane_bytes(g.tokens, g.features));
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
        a.partial = partial;
        e = run_gemm<DX, 0>(a, s);
        if (e != hipSuccess) return e;
    }
    if (g.dwg) {
        GemmArgs a = {};
        a.p[0] = static_cast<const uint16_t*>(g.x);
        a.q[0] = dg; a.q[1] = du;
        a.ldp = g.ldx; a.ldq = g.features;
        a.N = (int32_t)g.cols; a.M = (int32_t)g.features; a.K = (int32_t)g.tokens;
        a.out[0] = static_cast<uint16_t*>(g.dwg); a.out[1] = static_cast<uint16_t*>(g.dwu);
        a.partial = partial;
        e = run_gemm<DW, 0>(a, s);
    }
    return e;
}

}  // namespace iqk
