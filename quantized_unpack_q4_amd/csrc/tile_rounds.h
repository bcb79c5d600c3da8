// tile_rounds.h -- how many of a launch's workgroup tiles are cut in two (mxfp4_tile.h).  Host only.
#pragma once

#include <stdint.h>

namespace gq {

// How many of the tiles are not cut, and the workgroups of the launch.
inline int tiles_whole(int64_t total, int64_t cus)
{
    const int64_t rest = total % cus;
    return (int)(rest > 0 && 2 * rest <= cus ? total - rest : total);
}
inline unsigned tile_grid(int64_t total, int64_t whole)
{
    return (unsigned)((whole + 7) / 8 * 8 + (2 * (total - whole) + 7) / 8 * 8);
}

} // namespace gq
