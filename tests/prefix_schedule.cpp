// The host side of csrc/prefix_sched.h as C functions, for tests/test_prefix_schedule.py.
#include "prefix_sched.h"

using namespace h3b;

extern "C" {

int t_tile_piece(int row, int piece) { return tile_piece(row, piece); }
}
