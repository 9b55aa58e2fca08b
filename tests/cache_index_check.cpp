// The cache's indexing on the host, the functions that the kernels call: whatever
// lengths, starts and the page table hold, rows and blocks stay inside their
// arrays; for ascending starts every new token has exactly one slot.
#include <stdio.h>
#include <stdlib.h>

#include <vector>

#include "../int_quantization_amd/csrc/iq_cache.h"

using namespace iqk;

static uint64_t state = 1;
static int64_t pick(int64_t lo, int64_t hi) {
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return lo + (int64_t)((state >> 33) % (uint64_t)(hi - lo + 1));
}
#define EXPECT(x) do { if (!(x)) { printf("line %d: %s\n", __LINE__, #x); exit(1); } } while (0)

static void block_in_range(const CacheArgs& c, int seq, int block) {
    for (int head : {0, c.heads - 1}) {
        const int64_t at = block_at(c, seq, block, head);
        EXPECT(at >= -1 && at < c.pages * c.heads << c.shift);
        if (at >= 0) {
            const int32_t page = c.page_table[(int64_t)seq * c.width + (block >> c.shift)];
            EXPECT(at >> c.shift == (int64_t)page * c.heads + head && (at & ((1 << c.shift) - 1)) == (block & ((1 << c.shift) - 1)));
        }
    }
}

static void run(bool sound, bool with_starts) {
    CacheArgs c = {};
    c.heads = (int)pick(1, 5); c.dim = 64; c.shift = (int)pick(0, 3); c.batch = (int)pick(1, 9); c.width = (int)pick(0, 6);
    c.pages = pick(0, 20);
    std::vector<int32_t> lengths(c.batch), starts(c.batch + 1), table((size_t)c.batch * c.width);
    const int longest = (c.width << c.shift) * kBlock;
    const int32_t odd[] = {-1, INT32_MIN, INT32_MAX, 1 << 30, 0};
    starts[0] = sound ? 0 : (int32_t)pick(-3, 50);
    for (int s = 0; s < c.batch; ++s) {
        const int n = (int)pick(0, 4) ? (int)pick(0, 100) : 0;
        starts[s + 1] = sound ? starts[s] + n : pick(0, 2) ? (int32_t)pick(-5, 400) : odd[pick(0, 4)];
        lengths[s] = sound ? n + (int)pick(0, 300) : pick(0, 2) ? (int32_t)pick(-5, longest + 100) : odd[pick(0, 4)];
    }
    for (auto& p : table) p = pick(0, 4) ? (int32_t)pick(-2, c.pages + 1) : odd[pick(0, 4)];
    c.lengths = lengths.data(); c.page_table = table.data(); c.starts = with_starts ? starts.data() : nullptr;
    c.tokens = !with_starts ? c.batch : sound ? starts[c.batch] + (int)pick(0, 40) : (int)pick(0, 300);

    std::vector<int> written(c.tokens);
    for (int64_t slot = 0; slot < append_slots(c.tokens, c.batch, with_starts); ++slot) {
        int seq, block;
        Span s;
        const bool some = slot_block(c, slot, &seq, &s, &block);
        EXPECT(seq >= 0 && seq < c.batch);
        if (!some) continue;
        EXPECT(s.row >= 0 && s.n >= 0 && s.row + s.n <= c.tokens && block >= 0);
        block_in_range(c, seq, block);
        const int first = s.length - s.n, lo = std::max(first - block * kBlock, 0), hi = std::min(s.length - block * kBlock, kBlock);
        EXPECT(lo >= 0 && lo < hi && hi <= kBlock);
        for (int t = lo; t < hi; ++t) {
            const int row = s.row + (block * kBlock - first) + t;
            EXPECT(row >= 0 && row < c.tokens && row >= s.row && row < s.row + s.n);
            ++written[row];
        }
    }
    if (sound)
        for (int s = 0; s < c.batch; ++s) {
            const Span p = span_of(c, s);
            for (int i = 0; i < p.n; ++i) EXPECT(written[p.row + i] == (p.length - p.n + i >= 0 ? 1 : 0));
        }

    AttendArgs a = {};
    a.c = c;
    a.group = (int)pick(0, 2) ? (int)pick(1, 9) : (int)pick(10, 70);
    const int unit = 1 << pick(3, 8);
    std::vector<int> answered((size_t)c.tokens * a.group);
    for (int64_t slot = 0; slot < tile_slots(a, unit); ++slot) {
        Tile t;
        const bool some = tile_of(a, unit, slot, &t);
        EXPECT(t.seq >= 0 && t.seq < c.batch);
        if (!some) continue;
        EXPECT(t.columns >= 1 && t.columns <= unit && t.f0 >= 0);
        for (int col = 0; col < t.columns; ++col) {
            const int64_t row = t.s.row + (t.f0 + col) / a.group;
            EXPECT(row >= 0 && row < c.tokens);
            ++answered[row * a.group + (t.f0 + col) % a.group];
        }
    }
    if (sound)
        for (int s = 0; s < c.batch; ++s) {
            const Span p = span_of(c, s);
            for (int i = 0; i < p.n * a.group; ++i) EXPECT(answered[(size_t)p.row * a.group + i] == 1);
        }
}

int main() {
    for (int t = 0; t < 32; ++t) EXPECT(token_of(place_of(t) >> 4, place_of(t) & 15) == t);
    for (int i = 0; i < 20000; ++i) run(i & 1, i & 2);
    printf("ok\n");
    return 0;
}
