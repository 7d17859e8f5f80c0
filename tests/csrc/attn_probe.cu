// Test-only probe of parts of the attention kernels, from the kernels' own source.
#include <stdint.h>

#include "../../gated_delta_rule_86_b200/csrc/attn_decode_mma.cuh"

using namespace kda::attn;

namespace {

// The places of the line from (b, vh, 0) on, `count` of them, as a warp of the bf16 decode step walks them;
// returns how often the page that it was given is `marker`.
template <int TILE> int64_t walk(const DecodeArgs &a, int b, int vh, int64_t count, int warp, int32_t marker) {
    Walk<TILE> w = {};
    w.b = b;
    w.vh = vh;
    w.len = decode_len(a, b);
    w.tiles = (w.len + TILE - 1) / TILE;
    w.last = count;
    int64_t hits = 0;
    if (!w.more()) return 0;
    for (int page = first_page(a, w, warp);; page = next_page(a, w, warp)) {
        hits += page == marker;
        if (!w.more()) return hits;
    }
}

}  // namespace

// On the host, over host memory.
extern "C" int64_t attn_probe_walk(const int32_t *lens, int n, int vheads, const int32_t *table, int64_t row, int width,
                                   int page_log2, int b, int vh, int64_t count, int warp, int32_t marker) {
    DecodeArgs a = {};
    a.lens = lens;
    a.n = n;
    a.vheads = vheads;
    a.cache.table = table;
    a.cache.row = row;
    a.cache.width = width;
    a.cache.page_log2 = page_log2;
    return walk<DecodeMmaCfg<128, 8>::kTile>(a, b, vh, count, warp, marker);
}
