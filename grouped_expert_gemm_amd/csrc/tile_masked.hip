// The dgrad kernels whose adapter delta is masked (dropout of the adapter's input), and nothing
// else of tile.hip: a unit of their own, so that the plain kernels keep their registers.
#define GEG_TILE_MASKED
#include "tile.hip"
