// How the windowed calls run: the choice between the kernels and their launch
// shapes, from the sizes of a call and what the GPU holds at once.
#pragma once

#include <algorithm>
#include <cstdint>

#include "pa_prefill_umma.cuh"
#include "pa_window.cuh"

namespace pa {

// Positions stay below 2^30 (the table's width is checked), so a longer
// window or sink run means "all" and is cut to that.
constexpr int32_t kWindowMax = 1 << 30;

// Most blocks a call may have to read for one run of `queries` consecutive
// query tokens: the sinks' and those any placement of the window touches.
inline int64_t window_visible_blocks(int32_t max_blocks_per_seq, int32_t queries, int32_t window,
                                     int32_t num_sinks) {
    const int64_t w = ((int64_t)window + queries - 1 + 2 * (kBlock - 1)) / kBlock;
    const int64_t k = ((int64_t)num_sinks + kBlock - 1) / kBlock;
    return std::min<int64_t>(max_blocks_per_seq, w + k);
}

// How a windowed call runs: on decode_window_kernel (runs of tile_tokens query
// tokens; few rows: `cluster` CTAs each, many: `parts` partitions each), or on
// prefill_umma_kernel (umma; `parts` ranges of split_tiles key tiles).
struct WindowPlan {
    bool umma;
    bool warp_runs;
    int tile_tokens, cluster, part_blocks, qtiles, split_tiles;
    int64_t parts;
    // rows of the workspace, each with `parts` partial results
    int64_t ws_rows;
};

// What a GPU holds at once of CTAs that take an SM each: room[c] clusters of c
// of them (their SMs have to lie in one partition of the GPU), room[1] SMs;
// 0 where it launches none of that size.
struct WindowDevice {
    int room[kMaxCluster + 1];
};
// The GPU the plan's constants were measured on; for a size query on a machine
// without one.
constexpr WindowDevice kMeasuredDevice = {{0, 148, 74, 45, 33, 26, 22, 15, 15, 15, 11, 7, 7, 7, 7, 7, 7}};

constexpr int kChunkRows = 16;  // rows of a run on decode_window_kernel
// Shapes of decode_window_kernel (see there): warps per CTA and blocks in
// flight per warp.  Few rows at head_dim 128: 6 warps x 4 blocks, up to 8 %
// faster than 8 x 3; at 64: 8 x 6, 6 % faster than 6 x 8.  A lane holds one
// block id, so a CTA takes 32 blocks per warp at most.
template <int D>
constexpr int kFewWarps = D == 128 ? 6 : 8;
template <int D>
constexpr int kFewStages = D == 128 ? 4 : 6;
constexpr int kMinFewWarps = 6, kManyWarps = 4, kManyStages = 3;
constexpr int kWarpRunBlocks = 6;
constexpr int kFewBlocks = 32 * kMinFewWarps, kManyBlocks = 32 * kManyWarps;

// The heads, window and widths were checked: 1 <= group <= kUmmaRows.
inline WindowPlan window_plan(const WindowDevice &dev, int64_t num_seqs, int32_t num_q_tokens,
                              int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t max_blocks_per_seq, int32_t window, int32_t num_sinks) {
    const int sms = dev.room[1];
    const int group = num_q_heads / num_kv_heads;
    WindowPlan p = {};
    p.ws_rows = (int64_t)num_q_tokens * num_q_heads;
    // decode_window_kernel: runs of at most kChunkRows rows
    const int64_t run_tokens =
        max_query_len * (int64_t)group <= 8 ? max_query_len : std::max(kChunkRows / group, 1);
    const int64_t runs = num_seqs * num_kv_heads * ((max_query_len + run_tokens - 1) / run_tokens);
    const int64_t blocks =
        window_visible_blocks(max_blocks_per_seq, (int32_t)run_tokens, window, num_sinks);
    // prefill_umma_kernel: items of two query tiles (halved below where that is
    // faster), walked in tiles of 128 keys
    constexpr int kTileBlocks = kUmmaKeys / kBlock;
    const int64_t item_tokens = kUmmaQTiles * (kUmmaRows / group);
    const int64_t items = num_seqs * num_kv_heads * ((max_query_len + item_tokens - 1) / item_tokens);
    const int64_t tiles =
        (window_visible_blocks(max_blocks_per_seq, (int32_t)std::min<int64_t>(max_query_len, item_tokens),
                               window, num_sinks) + kTileBlocks - 1) / kTileBlocks;
    // one query tile per item: both warpgroups share its key tiles
    const bool one = max_query_len <= kUmmaRows / group;
    // Few rows keep most of a 256-row item empty.  The decode kernel takes about
    // 1.5 ns per (run, block) while the GPU holds the runs at once, the other
    // about 2.1 us per key tile on each SM (half for one query tile) and 6 us more at its ends.  Of 90 measured shapes this takes the faster
    // one or one at most 20 % slower (40 tokens, window 100: 6.3 us here, 10.3
    // there; 32 tokens of 4 heads, window 4096: 25.5 us here, 17.6 there).
    // Beyond one wave of runs only those of few blocks (a warp each) may stay
    // there: 4 + 0.9 ns per block a run against 5 or 7 us an item and its tiles (31
    // x 32 heads x 48 tokens: 21 us here, 43 there).
    const bool wave = runs <= sms * PA_DECODE_MIN_CTAS;
    const bool warp_runs = !wave && blocks <= kWarpRunBlocks;
    const double rounds = (double)((items + sms - 1) / sms);
    const bool slower =
        wave ? 2 * runs * blocks > 8400 + (one ? 11 : 22) * items * tiles
             : !warp_runs || 1e-3 * runs * (4 + 0.9 * blocks) >
                                 rounds * (one ? 5 + 0.9 * tiles : 7 + 2.1 * tiles);
    p.umma = group > kChunkRows ||
             (max_query_len > 1 && (int64_t)max_query_len * group > 8 && slower);
    if (p.umma) {
        // Query tiles and key ranges per item: the fewest microseconds over the
        // rounds that the SMs need (2.1 per key tile, half for one query tile, and
        // 3 per item), plus the launch of the join and its traffic.  Measured: 8
        // items of 33 tiles 70 us unsplit, 43 in 2 ranges, 28 in 4, 20.3 in 11, 23
        // in 17; 64 items of 33 tiles 72 us, 51 in 2 ranges, 47 as 128 of one
        // query tile.
        double best = 0;
        for (int qtiles = kUmmaQTiles; qtiles >= 1; --qtiles) {
            const int64_t tokens = qtiles * (kUmmaRows / group);
            const int64_t count =
                num_seqs * num_kv_heads * ((max_query_len + tokens - 1) / tokens);
            const int64_t t = (window_visible_blocks(max_blocks_per_seq,
                                                     (int32_t)std::min<int64_t>(max_query_len, tokens),
                                                     window, num_sinks) + kTileBlocks - 1) / kTileBlocks;
            const bool single = one || qtiles == 1;
            const double per_tile = single ? 1.05 : 2.1, per_range = single ? 0.03 : 0.06;
            for (int64_t n = 1; n <= 64 && n <= t; ++n) {
                const int64_t per = (t + n - 1) / n, used = (t + per - 1) / per;
                const double cost =
                    (double)((count * used + sms - 1) / sms) * (per_tile * per + 3.0) +
                    (used > 1 ? 3.0 + per_range * count * used + 0.25 * used : 0.0);
                if (p.parts == 0 || cost < best) {
                    best = cost;
                    p.qtiles = qtiles;
                    p.tile_tokens = (int)tokens;
                    p.parts = used;
                    p.split_tiles = (int)per;
                    p.ws_rows = count * kUmmaQTiles * kUmmaRows;
                }
            }
            if (one) break;  // a second query tile would be empty either way
        }
        return p;
    }
    p.tile_tokens = (int)run_tokens;
    p.parts = 1;
    if (runs <= sms && blocks > kManyWarps) {
        // A cluster as large as finds room for every run at once, while each
        // warp keeps a block: a second wave doubles the time.
        int ctas = (int)std::min<int64_t>(kMaxCluster, (blocks + kMinFewWarps - 1) / kMinFewWarps);
        while (ctas > 1 && dev.room[ctas] < runs) --ctas;
        // (up to three blocks per warp the next shape's one CTA is done before a
        // cluster has joined its sums: 9 blocks 3.0 us, 3.7 in a cluster of two;
        // 20 blocks 5.3 and 4.5)
        if ((blocks + ctas - 1) / ctas <= kFewBlocks && (ctas == 1 || blocks > 3 * kManyWarps)) {
            p.cluster = ctas;
            return p;
        }
    }
    if (runs <= 2 * sms && blocks > kManyWarps && blocks <= kManyBlocks) {
        p.part_blocks = 0;  // one CTA per run, all at once (256 runs of 64 blocks: 24.3 us, split 28.5)
        return p;
    }
    // more runs than a wave of CTAs holds, of a few blocks each (7360 runs: 1 block
    // 18 us, 40 as a CTA per run; 2 blocks 26 and 42, 6 blocks 57 and 65, 8 blocks
    // 84 and 74)
    if (warp_runs) {
        p.warp_runs = true;
        return p;
    }
    // 512-token partitions, or 1024 where that still makes several of a run:
    // 320, 512 and 1024 runs of equal length, and of lengths up to twice the
    // window.  Of 258 to 560 blocks the longer ones take 0.97 to 1.01 of the
    // shorter ones' time (320 ragged runs of 258: 1.08); of 132 to 250 blocks 0.98
    // to 1.09 (512 runs of 132: 89.5 us, 95.3 with the longer ones; 320 ragged
    // runs of 132: 46.2 and 42.7).
    p.part_blocks = blocks >= 8 * kPartBlocks ? 2 * kPartBlocks : kPartBlocks;
    p.parts = (blocks + p.part_blocks - 1) / p.part_blocks;
    return p;
}

}  // namespace pa
