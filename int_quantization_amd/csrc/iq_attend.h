// How attention's work is shared out: what columns see, rows and their units, and which kernels a call launches.  Compiled
// for the host too, where the check of the indexing runs it on arrays of any content.
#pragma once

#include "iq_cache.h"

namespace iqk {

// What a tile's columns see.  Columns are sorted by position, so the first and
// the last bound them all.
struct View {
    int keys;                    // tokens that the table has entries for
    int first;                   // position of token 0 of the call; may be negative
    int each_from, each_to;      // every column sees all of these
    int block, blocks;           // blocks that hold some that some column sees
};

__host__ __device__ inline int seen_to(const AttendArgs& a, int p, int keys) { return p < 0 ? 0 : a.causal ? min(keys - 1, p) + 1 : keys; }
__host__ __device__ inline int seen_from(const AttendArgs& a, int p, int keys) { return min(max(0, p - (a.window - 1)), keys); }

__host__ __device__ inline View view_of(const AttendArgs& a, const Tile& t) {
    View v;
    v.keys = a.c.pages > 0 ? min(t.s.length, (a.c.width << a.c.shift) * kBlock) : 0;
    v.first = t.s.length - t.s.n;
    const int lo = v.first + t.f0 / a.group, hi = v.first + (t.f0 + t.columns - 1) / a.group;
    v.each_to = seen_to(a, lo, v.keys); v.each_from = seen_from(a, hi, v.keys);
    v.block = seen_from(a, lo, v.keys) / kBlock;
    v.blocks = max((seen_to(a, hi, v.keys) + kBlock - 1) / kBlock - v.block, 0);
    return v;
}

// Columns of a lane's column `col`, of a tile that begins with flattened column f0.
struct Column {
    int row, head;               // of q and o; head among those of the key head
    int from, to;                // tokens that it sees
};
__host__ __device__ inline Column column_of(const AttendArgs& a, const Tile& t, const View& v, int col) {
    const int f = t.f0 + min(col, t.columns - 1), i = f / a.group;
    return {t.s.row + i, f - i * a.group, seen_from(a, v.first + i, v.keys), seen_to(a, v.first + i, v.keys)};
}

// ---- sharing the work out ----------------------------------------------------------------
// A row is a tile of columns of one sequence and key head; its units are the
// blocks that some column sees (one where there are none: someone writes its
// zeros).  The units of all rows, key head by key head, are shared out evenly among
// the workgroups that the GPU holds at once, so sequences of any lengths keep
// every CU busy.  A row that more than one workgroup has a share of is joined by another launch.

// Sequences of few columns are k_few's, the others k_many's.
enum { kAny = 0, kFew = 1, kMany = 2 };        // which of them a kernel takes: all where the other is not launched

// A row's parts: the normalized output of its columns, their maxima and sums.
__host__ __device__ inline int64_t part_floats(int dim, int columns) { return (int64_t)columns * (dim + 2); }

// Units of a workgroup's share of `total`, which are `one_head` for each key head, in `rows` rows of that head.  `least` spares
// short rows the join.  Rows shorter than that take a workgroup each, since a row costs several
// blocks' time to begin with: 5 prompts of 18 to 25 tokens take 24 us, 122 with 16 rows to a workgroup.
__host__ __device__ inline int64_t share_size(int64_t total, int workers, int64_t one_head, int64_t rows, int least) {
    const int64_t even = (total + workers - 1) / workers, row = one_head / (rows > 1 ? rows : 1), floor = row < least ? row : least;
    return even > floor ? (even > 1 ? even : 1) : floor > 1 ? floor : 1;
}

// Which of a row's two parts worker w's share of it is: 1 if the row begins inside the share, 0 if the share begins with it or in it.
__host__ __device__ inline int part_index(int64_t w, int64_t per, int64_t begin) { return w * per < begin ? 1 : 0; }

// The row that a workgroup's share ends in, if it began there and does not end
// there: the join's work.  columns is 0 if there is none.
struct Open {
    int64_t begin;               // unit that the row begins with
    int64_t per;                 // units of a share
    int row, f0, columns, head;  // row: of q and o, of the sequence's first token
    int last, unused;            // workgroup that has the row's end
};

struct Plan {
    int kind, workers;
    int few;                     // columns that are few
    int slots;                   // of k_many: tiles' slots
    int64_t opens, parts;        // where the Opens and the parts begin in the workspace, in bytes: an Open and two
                                 // parts for every workgroup, of the row that its share begins in (0) and ends in (1)
};

__host__ __device__ inline bool takes(const AttendArgs& a, const Plan& plan, const Span& s) {
    const bool few = (int64_t)s.n * a.group <= plan.few;
    return s.n > 0 && (plan.kind == kAny || (plan.kind == kFew) == few);
}

// ---- few columns --------------------------------------------------------------------------
// Blocks of a workgroup, at least.  One sequence of 8000 tokens takes 19.4 us, 23.2 with 4 and 19.6 with 16; one of 2000
// takes 17.3, and 18.6 with 16.
constexpr int kLeastShare = 8;

// Waves of a SIMD, and so workgroups of a CU: as many as registers allow, but for 16 columns of 96 elements and more,
// where two take 212 us for the 64 sequences above and 61 for the long one, three 212 and 66, four 217 and 69: more
// workgroups mean more parts to join, and two have enough codes in flight.
constexpr int few_waves(int dim, int columns) {
    return columns == 16 ? (dim <= 64 ? 3 : 2) : dim <= 64 ? 4 : dim <= 96 ? 3 : dim <= 128 ? 2 : 1;
}

__host__ __device__ inline Tile tile_at(const AttendArgs& a, int unit, int seq, const Span& s, int k) {
    const int64_t left = (int64_t)s.n * a.group - (int64_t)k * unit;
    return {seq, k * unit, (int)min(left, (int64_t)unit), s};
}

template <int C> __host__ __device__ inline int64_t units_of(const AttendArgs& a, const Plan& plan, int seq) {
    const Span s = span_of(a.c, seq);
    if (!takes(a, plan, s)) return 0;
    const int tiles = (int)(((int64_t)s.n * a.group + C - 1) / C);
    if (s.n == 1) return (int64_t)tiles * max(view_of(a, tile_at(a, C, seq, s, 0)).blocks, 1);      // tiles of one token see the same
    int64_t sum = 0;
    for (int k = 0; k < tiles; ++k) sum += max(view_of(a, tile_at(a, C, seq, s, k)).blocks, 1);
    return sum;
}

// ---- many columns -------------------------------------------------------------------------
constexpr int kManyColumns = 128;

// Blocks of a workgroup, at least: prompts of 77 to 2047 tokens (12 heads of 64) take 71 us, 74 with 24.
constexpr int kLeastManyShare = 16;

// Waves of a SIMD, and so workgroups of a CU: as many as LDS and registers allow.  Prompts of 4096 tokens of 64 elements
// take 129 us with 3 and 135 with 2; of 2048 tokens of 192 elements 112 with 2 and 136 with 1.
constexpr int many_waves(int dim) { return dim <= 64 ? 3 : dim <= 192 ? 2 : 1; }

// Row `e` of a key head: the slots in an order that takes one from the front and one from the back by turns, for a prompt's
// first rows see few tokens and its last ones many, and a share of either alone would hold many rows or few.
__host__ __device__ inline bool row_at(const AttendArgs& a, const Plan& plan, int64_t e, Tile* t) {
    const int64_t slot = e & 1 ? plan.slots - 1 - (e >> 1) : e >> 1;
    return tile_of(a, kManyColumns, slot, t) && takes(a, plan, t->s);
}

// ---- plans ----------------------------------------------------------------------------------
// Columns of a sequence that are few: two tiles of k_few read the codes as often as one of k_many and start sooner.
// 64: 12 tokens of 4 heads (48 columns) at 2000 tokens take 29 us, 39 in k_many; at 32000 48 and 113.
// 128 where all sequences are pieces of that size and their blocks are few for the GPU, for k_many's waves then wait for
// their codes alone: 24 tokens (96 columns) at 8000 tokens take 37 us, 60 in k_many; four such 61 and 66; past 8192 blocks
// eight such take 95, and 80 in k_many, 32 of them 335 and 205.  Heads of 192 elements and more have one wave a SIMD in
// k_few: 16 prompts of 20 to 30 tokens (256 elements) 31 us, and 25 in k_many.
constexpr int kFewColumns = 64, kFewColumnsShort = 128, kShortUnits = 8192;
inline int few_limit(const AttendArgs& a) {
    const int64_t units = ((int64_t)a.c.width << a.c.shift) * a.c.heads * a.c.batch;
    return a.c.dim <= 128 && (int64_t)a.c.tokens * a.group <= (int64_t)kFewColumnsShort * a.c.batch && units <= kShortUnits ? kFewColumnsShort : kFewColumns;
}

// 16 columns to a wave where that holds a sequence's columns: half the work on them.  8 sequences of 4 tokens of 4 heads
// at 8000 tokens take 44 us, 47 with 32 columns; with 8 tokens (32 columns) 64 in two tiles of 16, 53 in one of 32.
inline int few_columns(const AttendArgs& a) {
    const int64_t columns = a.c.starts ? (int64_t)a.c.tokens * a.group / (a.c.batch > 0 ? a.c.batch : 1) : a.group;
    return columns <= 16 ? 16 : 32;
}

// A row of this many blocks is not worth sharing (blocks that the table has entries for, since the host does not know the
// lengths: one token at 500 tokens takes 6.9 us, 12.9 with a table for 131072): its workgroup takes it whole, without a search for its share and
// without the join's launch.  One sequence of 2000 tokens takes 14.4 us, 17.6 shared; of 4000 tokens 23.0 and 18.2.  Where
// rows fill half the CUs twice as many blocks are not worth it: 16 sequences of 4000 tokens 26.8 and 34.0, 64 of 100 to 4000 tokens 62
// and 78, but 4 of 4000 24.1 and 21.9.  kDirectRows bounds the launch where most sequences have no tokens.
constexpr int64_t kDirectBlocks = 64, kDirectManyBlocks = 128, kDirectManyRows = 128, kDirectRows = 1 << 20;
inline int64_t direct_rows(const AttendArgs& a, int columns) {
    return (int64_t)a.c.batch * (a.c.starts ? few_limit(a) / columns : (a.group + columns - 1) / columns);
}
inline bool direct(const AttendArgs& a) {
    const int64_t blocks = (int64_t)a.c.width << a.c.shift;
    return blocks <= ((int64_t)a.c.batch * a.c.heads < kDirectManyRows ? kDirectBlocks : kDirectManyBlocks) &&
           direct_rows(a, few_columns(a)) * a.c.heads <= kDirectRows;
}

struct Plans {
    Plan few, many;
    size_t bytes;
};

inline Plans plans_of(const AttendArgs& a) {
    Plans p = {};
    const int64_t rows = (int64_t)a.c.tokens * a.group;
    int64_t at = 0;
    const auto room = [&](int64_t bytes) { const int64_t here = at; at += (bytes + 255) / 256 * 256; return here; };
    // Which kernels some sequence may be for; of one sequence the host knows nothing better than that it has all rows.  Without
    // starts all is k_few's, whatever the group: 128 heads on each of 1 key head, 8 sequences of 4000 tokens 33 us and 39 in
    // k_many, of 32000 50 and 56; on each of 8 key heads 67 and 74, but of 32000 tokens 322 and 211.
    const int limit = few_limit(a);
    const bool many = a.c.starts && rows > limit, few = !many || a.c.batch > 1;
    p.few.few = p.many.few = limit;
    if (few) {
        const int columns = few_columns(a);
        p.few.kind = many ? kFew : kAny;
        p.few.workers = 256 * few_waves(a.c.dim, columns);             // what the GPU holds at once
        if (!direct(a)) {
            p.few.opens = room(p.few.workers * (int64_t)sizeof(Open));
            p.few.parts = room(p.few.workers * 2 * part_floats(a.c.dim, columns) * (int64_t)sizeof(float));
        }
    }
    if (many) {
        p.many.kind = few ? kMany : kAny;
        p.many.workers = 256 * many_waves(a.c.dim);    // what the GPU holds at once
        p.many.slots = (int)tile_slots(a, kManyColumns);
        p.many.opens = room(p.many.workers * (int64_t)sizeof(Open));
        p.many.parts = room(p.many.workers * 2 * part_floats(a.c.dim, kManyColumns) * (int64_t)sizeof(float));
    }
    p.bytes = (size_t)at;
    return p;
}

}  // namespace iqk
