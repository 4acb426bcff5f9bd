// gate.h -- how many tokens the gate takes (not installed).
#pragma once

namespace coli {

constexpr int GATE_TILE = 64;                       // tokens of a tile; tiles lie along grid.y
constexpr int GATE_MAX_TOKENS = 65535 * GATE_TILE;  // the largest grid.y

}  // namespace coli
