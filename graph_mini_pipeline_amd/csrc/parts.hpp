// How a summed length is cut into the parts of the dense layers' products.  Host and device, no includes of either.
#pragma once

#include <cstdint>

namespace gnnmb {

struct SumPart {
    int64_t first, steps;      // tiles of the sum before the part, and in it (none, where the parts before have all)
    int32_t seg;               // segment of its first tile, and the tile within that: places of the sum in any case
    int64_t tile;
};

// Part `part` of `parts` of a sum over `segs` segments of `seg_tiles` tiles each.
constexpr SumPart part_of_sum(int64_t seg_tiles, int32_t segs, int64_t parts, int64_t part) {
    SumPart p{0, seg_tiles * segs, 0, 0};
    if (parts > 1) {
        const int64_t share = (p.steps + parts - 1) / parts;
        p.first = part * share < p.steps ? part * share : p.steps;
        p.steps = p.steps - p.first < share ? p.steps - p.first : share;
    }
    if (p.steps > 0) {      // (an empty part would start past the last segment)
        p.seg = static_cast<int32_t>(p.first / seg_tiles);
        p.tile = p.first - p.seg * seg_tiles;
    }
    return p;
}

}  // namespace gnnmb
