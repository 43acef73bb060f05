// When a tile's MMA thread may wait for a tile of the K/V ring (host code too: a
// model of the ring is checked with it).
//
// Fill f of a ring of N slots lies in slot f % N and completes phase f / N of the
// slot's barriers: `full` when its copies have landed, `fixed` when its values
// have been looked over, `empty` when all of its readers have let go of it.  A
// wait tells phases by their parity, so it must not be made while phase f / N - 1
// is open: phase f / N - 2, long complete, would satisfy it.
//
// The fill before f in its slot is certainly through once the producer has begun
// f, for it waited for `empty` first.  A thread that took that fill itself knows
// too, but a query tile takes some fills only: the other tile's of a unit of two
// heads are not its own, nor those of a unit without a second tile, of steps that
// only the later tile's tokens see, or of a part for which the first tile is through.
// Copies land in any order, so nothing that it did take tells of those.
#pragma once

namespace sv {

// Whether a thread asks that a fill has begun before it waits for it; in_order: the
// fills of the ring complete in order (codes that warps widen one fill after the
// other), so that the first one of a part, found complete, stands for all before it.
constexpr bool chunk_ring_asks(bool in_order, bool first_of_part) { return !in_order || first_of_part; }

}  // namespace sv
