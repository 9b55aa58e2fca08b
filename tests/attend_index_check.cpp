// How attention shares its work out, on the host, by the functions that the kernels call: whatever lengths and starts
// hold, blocks and rows stay inside the arrays, shares are all taken, and no two rows of a workgroup want one place of the
// workspace; for ascending starts every column is answered exactly once.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../int_quantization_amd/csrc/iq_attend.h"

using namespace iqk;

static uint64_t state = 1;
static int64_t pick(int64_t lo, int64_t hi) {
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return lo + (int64_t)((state >> 33) % (uint64_t)(hi - lo + 1));
}
#define EXPECT(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)

static std::vector<int> answered;                      // of every (token, head of all key heads)

// A row of `unit` columns: what it reads and writes.  Returns its units.
static int64_t row_in_range(const AttendArgs& a, int unit, const Tile& t, int head) {
    EXPECT(t.seq >= 0 && t.seq < a.c.batch && head >= 0 && head < a.c.heads && t.f0 >= 0 && t.columns >= 1 && t.columns <= unit);
    const View v = view_of(a, t);
    EXPECT(v.keys >= 0 && v.block >= 0 && v.blocks >= 0);
    if (v.blocks > 0) EXPECT(a.c.pages > 0 && (int64_t)v.block + v.blocks <= (int64_t)a.c.width << a.c.shift);
    for (int col = 0; col < unit; ++col) {
        const Column c = column_of(a, t, v, col);
        EXPECT(c.row >= 0 && c.row < a.c.tokens && c.head >= 0 && c.head < a.group && c.from >= 0);
        if (c.from < c.to) EXPECT(c.to <= v.keys && c.from / kBlock >= v.block && (c.to - 1) / kBlock < v.block + v.blocks);
        EXPECT(!(v.each_from < v.each_to) || col >= t.columns || (c.from <= v.each_from && c.to >= v.each_to));
        if (col < t.columns) ++answered[((int64_t)c.row * a.c.heads + head) * a.group + c.head];
    }
    return v.blocks > 1 ? v.blocks : 1;
}

// Rows one after another, as shares cut them.
struct Cut {
    const Plan& plan;
    int64_t per, total, at = 0;
    std::vector<int> parts, opens;
    Cut(const Plan& p, int64_t per, int64_t total) : plan(p), per(per), total(total), parts(2 * p.workers), opens(p.workers) {
        EXPECT(per >= 1 && (total + per - 1) / per <= p.workers);
    }
    void row(int64_t units) {
        const int64_t first = at / per, last = (at + units - 1) / per;
        EXPECT(last < plan.workers);
        if (first != last) {
            EXPECT(!opens[first]++);
            for (int64_t w = first; w <= last; ++w) {
                const bool opening = at <= w * per;    // the share's first row: the part that a kernel writes
                EXPECT(part_index(w, per, at) == !opening && !parts[2 * w + !opening]++);
            }
        }
        at += units;
    }
};

template <int C> static void few_rows(const AttendArgs& a, const Plan& plan) {
    if (direct(a)) {
        EXPECT(direct_rows(a, C) * a.c.heads <= kDirectRows);
        for (int head = 0; head < a.c.heads; ++head)
            for (int64_t block = 0; block < direct_rows(a, C); ++block) {
                const int seq = (int)(block % a.c.batch), tile = (int)(block / a.c.batch);
                const Span s = span_of(a.c, seq);
                if (takes(a, plan, s) && (int64_t)tile * C < (int64_t)s.n * a.group) row_in_range(a, C, tile_at(a, C, seq, s, tile), head);
            }
        return;
    }
    int64_t one_head = 0, rows = 0;
    for (int seq = 0; seq < a.c.batch; ++seq) {
        const int64_t u = units_of<C>(a, plan, seq);
        EXPECT(u >= 0);
        one_head += u;
        rows += u > 0;
    }
    Cut cut(plan, share_size(one_head * a.c.heads, plan.workers, one_head, rows, kLeastShare), one_head * a.c.heads);
    for (int head = 0; head < a.c.heads; ++head)
        for (int seq = 0; seq < a.c.batch; ++seq) {
            const Span s = span_of(a.c, seq);
            const int64_t before = cut.at;
            for (int tile = 0; takes(a, plan, s) && (int64_t)tile * C < (int64_t)s.n * a.group; ++tile) cut.row(row_in_range(a, C, tile_at(a, C, seq, s, tile), head));
            EXPECT(cut.at - before == units_of<C>(a, plan, seq));
        }
    EXPECT(cut.at == cut.total);
}

static void many_rows(const AttendArgs& a, const Plan& plan) {
    EXPECT(plan.workers % 8 == 0);                     // workgroups are numbered by XCD
    int64_t one_head = 0, rows = 0;
    for (int64_t e = 0; e < plan.slots; ++e) {
        Tile t;
        if (!row_at(a, plan, e, &t)) continue;
        const int blocks = view_of(a, t).blocks;
        one_head += blocks > 1 ? blocks : 1;
        ++rows;
    }
    Cut cut(plan, share_size(one_head * a.c.heads, plan.workers, one_head, rows, kLeastManyShare), one_head * a.c.heads);
    for (int head = 0; head < a.c.heads; ++head)
        for (int64_t e = 0; e < plan.slots; ++e) {
            Tile t;
            if (row_at(a, plan, e, &t)) cut.row(row_in_range(a, kManyColumns, t, head));
        }
    EXPECT(cut.at == cut.total);
}

static int kinds[4];                                   // calls seen: few direct, few shared, many, both

static void run(bool sound, bool with_starts) {
    AttendArgs a = {};
    CacheArgs& c = a.c;
    const int dims[] = {64, 96, 128, 192, 256};
    c.heads = (int)pick(1, 4); c.dim = dims[pick(0, 4)]; c.shift = (int)pick(0, 3); c.batch = (int)pick(1, 9);
    c.width = pick(0, 2) ? (int)pick(0, 6) : (int)pick(60, 3000) >> c.shift;
    c.pages = pick(0, 9) ? pick(1, 20) : 0;
    std::vector<int32_t> lengths(c.batch), starts(c.batch + 1);
    const int longest = (c.width << c.shift) * kBlock;
    const int32_t odd[] = {-1, INT32_MIN, INT32_MAX, 1 << 30, 0};
    const int most = pick(0, 2) ? 20 : 300;
    starts[0] = sound ? 0 : (int32_t)pick(-3, 50);
    for (int s = 0; s < c.batch; ++s) {
        const int n = pick(0, 4) ? (int)pick(0, most) : (int)pick(0, 1);
        starts[s + 1] = sound ? starts[s] + n : pick(0, 2) ? (int32_t)pick(-5, 400) : odd[pick(0, 4)];
        lengths[s] = sound ? n + (int)pick(0, longest) : pick(0, 2) ? (int32_t)pick(-5, longest + 100) : odd[pick(0, 4)];
    }
    c.lengths = lengths.data(); c.starts = with_starts ? starts.data() : nullptr;
    c.tokens = !with_starts ? c.batch : sound ? starts[c.batch] + (int)pick(0, 40) : (int)pick(0, 600);
    if (c.tokens == 0) return;
    a.group = (int)pick(0, 2) ? (int)pick(1, 9) : (int)pick(10, 70);
    a.q_heads = a.group * c.heads;
    a.causal = pick(0, 3) > 0;
    a.window = a.causal && pick(0, 1) ? (int)pick(1, 400) : 1 << 30;
    answered.assign((size_t)c.tokens * a.q_heads, 0);

    const Plans p = plans_of(a);
    int64_t end = 0;
    const auto room = [&](const Plan& plan, int columns) {           // Opens and parts one after the other, on 16 bytes
        EXPECT(plan.opens >= end && plan.opens % 16 == 0 && plan.parts % 16 == 0);
        EXPECT(plan.parts >= plan.opens + plan.workers * (int64_t)sizeof(Open));
        end = plan.parts + plan.workers * 2 * part_floats(c.dim, columns) * (int64_t)sizeof(float);
    };
    if (p.few.workers) {
        ++kinds[direct(a) ? 0 : 1];
        if (!direct(a)) room(p.few, few_columns(a));
        if (few_columns(a) == 16) few_rows<16>(a, p.few);
        else few_rows<32>(a, p.few);
    }
    if (p.many.workers) {
        ++kinds[p.few.workers ? 3 : 2];
        room(p.many, kManyColumns);
        many_rows(a, p.many);
    }
    EXPECT(end <= (int64_t)p.bytes);
    if (sound)
        for (int s = 0; s < c.batch; ++s) {
            const Span span = span_of(c, s);
            for (int64_t i = 0; i < (int64_t)span.n * a.q_heads; ++i) EXPECT(answered[(size_t)span.row * a.q_heads + i] == 1);
        }
}

int main() {
    for (int i = 0; i < 6000; ++i) run(i & 1, i & 6);
    for (int k : kinds) EXPECT(k > 100);
    printf("ok\n");
    return 0;
}
