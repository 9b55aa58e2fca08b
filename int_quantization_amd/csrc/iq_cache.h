// Device-side view of the paged cache, shared by the kernels that append to
// it, read it back and attend over it: where sequences and blocks lie, and the
// 8-bit codes.
#pragma once

#include <hip/hip_runtime.h>

#include "iq_attn_launch.h"

namespace iqk {

constexpr int kBlock = 32;       // tokens of a block, which share a scale

// The call's tokens of one sequence: rows [row, row + n), positions
// [length - n, length).  What starts and lengths hold is not trusted: rows
// stay inside [0, tokens) and n and length are not negative.
struct Span {
    int row, n, length;
};

__host__ __device__ inline Span span_of(const CacheArgs& c, int seq) {
    Span s;
    s.length = max(c.lengths[seq], 0);
    if (c.starts) {
        s.row = min(max(c.starts[seq], 0), c.tokens);
        s.n = max(min(max(c.starts[seq + 1], 0), c.tokens) - s.row, 0);
    } else {
        s.row = seq;
        s.n = 1;
    }
    return s;
}

// Largest sequence whose first slot is at most `slot`, where sequence s begins
// at slot floor(starts[s] * scale / unit) + extra * s.
__host__ __device__ inline int sequence_of(const CacheArgs& c, int64_t slot, int64_t scale, int64_t unit, int extra) {
    int lo = 0, hi = c.batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)max(c.starts[mid], 0) * scale / unit + (int64_t)extra * mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Number of block b of a sequence in the cache's memory, for head 0 of its
// page; -1 where the page is absent.  b is at least 0.
__host__ __device__ inline int64_t block_at(const CacheArgs& c, int seq, int b, int head) {
    const int entry = b >> c.shift;
    if (entry >= c.width) return -1;
    const int64_t page = c.page_table[(int64_t)seq * c.width + entry];
    if (page < 0 || page >= c.pages) return -1;
    return ((page * c.heads + head) << c.shift) | (b & ((1 << c.shift) - 1));
}

// Slots of a sequence: floor(starts / 32) + 2 s onwards, which is never fewer
// than the blocks that its n tokens touch, at most floor((n + 62) / 32).
__host__ __device__ inline int64_t append_slots(int64_t tokens, int64_t batch, bool starts) {
    return starts ? tokens / kBlock + 2 * batch : batch;
}

__host__ __device__ inline bool slot_block(const CacheArgs& c, int64_t slot, int* seq, Span* s, int* block) {
    int64_t first = slot;
    *seq = (int)slot;
    if (c.starts) {
        *seq = sequence_of(c, slot, 1, kBlock, 2);
        first = (int64_t)max(c.starts[*seq], 0) / kBlock + 2 * (int64_t)*seq;
    }
    *s = span_of(c, *seq);
    const int64_t begin = max(s->length - s->n, 0);
    const int64_t b = begin / kBlock + (slot - first);
    *block = (int)b;
    return s->n > 0 && slot >= first && b * kBlock < s->length;
}

// Place of token t in a block's values: its bits 2, 4, 3, 1, 0 from the top.  A
// lane of the score's matrix holds tokens 8 g + 4 h + r (h its half of the wave); this
// order makes them 16 neighbouring bytes, 8 for each of two matrix products.
__host__ __device__ inline int place_of(int t) { return ((t >> 2) & 1) * 16 + (t >> 4) * 8 + ((t >> 3) & 1) * 4 + (t & 3); }

// The token of byte i of the 16 at half h: the inverse.
__host__ __device__ inline int token_of(int h, int i) { return (i >> 2) * 8 + h * 4 + (i & 3); }

template <int FMT> __device__ __forceinline__ float code_value(uint32_t byte) {
    if constexpr (FMT == 0) return (float)(int8_t)byte;
    else return __builtin_amdgcn_cvt_f32_fp8((int)byte, 0);
}

template <int FMT> constexpr float kLargest = FMT == 0 ? 127.f : 448.f;

// The code nearest y (ties to even), saturating; NaN gives 0.
template <int FMT> __device__ __forceinline__ uint32_t code_of(float y) {
    y = y == y ? fminf(fmaxf(y, -kLargest<FMT>), kLargest<FMT>) : 0.f;
    if constexpr (FMT == 0) return (uint32_t)(int)rintf(y) & 0xFFu;
    else return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, y, 0, false) & 0xFFu;
}

// ---- attention: tiles of columns ------------------------------------------------------
// The columns of a sequence and key head are its (token, query head of that
// head) pairs in order.  With tiles of `unit` columns sequence s has the slots from floor(starts[s] * group
// / unit) + s on, never fewer than the tiles that it needs.
__host__ __device__ inline int64_t tile_slots(const AttendArgs& a, int unit) {
    return a.c.starts ? (int64_t)a.c.tokens * a.group / unit + a.c.batch : (int64_t)a.c.batch * ((a.group + unit - 1) / unit);
}

struct Tile {
    int seq, f0, columns;        // first flattened column of the tile, valid columns
    Span s;
};

__host__ __device__ inline bool tile_of(const AttendArgs& a, int unit, int64_t slot, Tile* t) {
    const int per = (a.group + unit - 1) / unit;
    int64_t index;
    if (a.c.starts) {
        t->seq = sequence_of(a.c, slot, a.group, unit, 1);
        index = slot - ((int64_t)max(a.c.starts[t->seq], 0) * a.group / unit + t->seq);
    } else {
        t->seq = (int)(slot / per);
        index = slot % per;
    }
    t->s = span_of(a.c, t->seq);
    const int64_t left = (int64_t)t->s.n * a.group - index * unit;
    t->f0 = (int)(index * unit);
    t->columns = (int)(left < unit ? left : unit);
    return index >= 0 && left > 0;
}

}  // namespace iqk
