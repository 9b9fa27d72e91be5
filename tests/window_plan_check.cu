// Host-only check of the launch plan of the windowed calls on GPUs that hold
// other numbers of clusters at once than the one its constants were measured on.
// Prints "ok" and exits 0 when every plan can be launched as it stands.
#include <cstdint>
#include <cstdio>

#include "pa_window_plan.cuh"

using namespace pa;

static int bad = 0;
static void expect(bool ok, const char *what, long long a, long long b) {
    if (!ok && ++bad < 20) std::printf("%s: %lld %lld\n", what, a, b);
}

int main() {
    // a GPU as measured; one that launches no cluster beyond the 8 CTAs every
    // GPU has to allow; one without clusters; half of the SMs; few large ones
    const WindowDevice portable = {{0, 148, 74, 45, 33, 26, 22, 15, 15}};
    const WindowDevice none = {{0, 132}};
    const WindowDevice half = {{0, 74, 37, 22, 16, 13, 11, 7, 7, 7, 5, 3, 3, 3, 3, 3, 3}};
    const WindowDevice holes = {{0, 100, 50, 0, 20, 0, 12, 0, 9, 0, 0, 0, 0, 0, 0, 0, 2}};
    const WindowDevice devs[] = {kMeasuredDevice, portable, none, half, holes};

    // one user's long window: 2 runs of 188 blocks
    auto one_user = [](const WindowDevice &d) { return window_plan(d, 1, 1, 1, 8, 2, 200, 3000, 0).cluster; };
    expect(one_user(kMeasuredDevice) == 16, "measured", one_user(kMeasuredDevice), 16);
    expect(one_user(portable) == 8, "portable", one_user(portable), 8);
    expect(one_user(none) == 1, "none", one_user(none), 1);
    expect(one_user(half) == 16, "half", one_user(half), 16);
    expect(one_user(holes) == 16, "holes", one_user(holes), 16);
    // 8 runs of 513 blocks
    auto long_window = [](const WindowDevice &d) { return window_plan(d, 1, 1, 1, 32, 8, 1024, 8192, 4); };
    expect(long_window(kMeasuredDevice).cluster == 10, "measured", long_window(kMeasuredDevice).cluster, 10);
    expect(long_window(portable).cluster == 8, "portable", long_window(portable).cluster, 8);
    expect(long_window(none).cluster == 0 && long_window(none).parts > 1, "none", long_window(none).cluster, 0);
    expect(long_window(half).cluster == 6, "half", long_window(half).cluster, 6);
    expect(long_window(holes).cluster == 8, "holes", long_window(holes).cluster, 8);

    uint64_t x = 88172645463325252ull;
    auto next = [&](int64_t n) {
        x ^= x << 13; x ^= x >> 7; x ^= x << 17;
        return (int64_t)(x % (uint64_t)n);
    };
    for (int i = 0; i < 400000; ++i) {
        const WindowDevice &d = devs[next(5)];
        const int kv = 1 << next(6), group = 1 + (int)next(next(2) ? 8 : 16);
        const int64_t seqs = 1 + next(1 << next(11));
        const int max_query = next(2) ? 1 : 1 + (int)next(1 << next(11));
        const int width = 1 + (int)next(1 << (1 + next(17))), window = 1 + (int)next(1 << (1 + next(20)));
        const int sinks = (int)next(1 << next(10));
        const WindowPlan p = window_plan(d, seqs, (int)(seqs * max_query), max_query, kv * group, kv, width,
                                         window, sinks);
        expect(p.tile_tokens >= 1 && p.parts >= 1, "plan", p.tile_tokens, p.parts);
        if (p.umma) continue;
        const int64_t runs = seqs * kv * ((max_query + p.tile_tokens - 1) / p.tile_tokens);
        const int64_t blocks = window_visible_blocks(width, p.tile_tokens, window, sinks);
        expect(p.tile_tokens * group <= kChunkRows, "rows of a run", p.tile_tokens, group);
        if (p.cluster > 0) {
            expect(p.cluster == 1 || d.room[p.cluster] >= runs, "room", p.cluster, runs);
            expect((blocks + p.cluster - 1) / p.cluster <= kFewBlocks, "blocks of a CTA", p.cluster, blocks);
            expect(p.parts == 1, "no workspace", p.cluster, p.parts);
        } else if (p.warp_runs) {
            expect(blocks <= 32 && p.parts == 1, "a warp's run", blocks, p.parts);
        } else if (p.part_blocks == 0) {
            expect(blocks <= kManyBlocks && p.parts == 1, "a CTA's run", blocks, p.parts);
        } else {
            expect(p.part_blocks <= kManyBlocks && p.parts * p.part_blocks >= blocks, "parts", p.parts, blocks);
        }
    }
    if (bad == 0) std::printf("ok\n");
    return bad != 0;
}
