// Which of an expert's tiles a number stands for (plain C++, so that a host program can go through all of them).
#pragma once

namespace moe {

struct TileIn {
  bool ok;
  int q, p;
};

// Tile `within` of an expert's q_tiles x p_tiles: they lie in groups of up to `most_q` q-tiles, within a group p-tile by
// p-tile.  (Groups of about the same size: with 9 q-tiles, 8 and 1 would leave a group whose p panels are read by one
// workgroup each.)  within comes of two readings of the plan's starts: the sum of the tiles up to this expert's last, and
// q_tiles.  Where they changed meanwhile it may lie ahead of the expert's first tile; there is no such tile then.
constexpr TileIn tile_in(int within, int q_tiles, int p_tiles, int most_q) {
  if (within < 0) return TileIn{false, 0, 0};
  const int groups = (q_tiles + most_q - 1) / most_q, each = (q_tiles + groups - 1) / groups;
  const int q0 = within / (each * p_tiles) * each, left = q_tiles - q0, size = each < left ? each : left;
  const int in = within - q0 * p_tiles, p = in / size;
  return TileIn{true, q0 + in - p * size, p};
}

}  // namespace moe
