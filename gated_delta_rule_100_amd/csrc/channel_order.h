// channel_order.h -- which tile of a column a workgroup of the channel scan takes (channel.hip).
// Plain C++, so that a host program can check that every ticket stays inside the column.
#pragma once

#include <cstdint>

namespace gdr {

// Whether a workgroup with this ticket has a tile.  In a pass of its own workspace tickets run
// from 0 to tiles - 1; where calls that run at the same time share a workspace, against the
// rules, a ticket may be anything, and a tile from it behind the rows and the workspace.
constexpr bool has_tile(uint32_t ticket, int tiles) { return ticket < static_cast<uint32_t>(tiles); }

// Its tile, of `tiles` in time: from the first on, or from the last on (the gradient).
constexpr int tile_of_ticket(uint32_t ticket, int tiles, bool back) {
  return back ? tiles - 1 - static_cast<int>(ticket) : static_cast<int>(ticket);
}

}  // namespace gdr
