// norm_shapes.cpp -- prints the launch shape of the residual norm at one size:
// lanes of a group, rows of a block at a time, and row blocks.
// Arguments: forward|backward, rows, channels, groups.
#include <stdio.h>
#include <stdlib.h>

#include "engram_layer_host.h"

int main(int argc, char **argv) {
  if (argc != 5) return 1;
  const int64_t rows = atoll(argv[2]), channels = atoll(argv[3]), groups = atoll(argv[4]);
  const engram::NormShape s = argv[1][0] == 'f'
                                  ? engram::norm_forward_shape(rows, channels, groups)
                                  : engram::norm_backward_shape(rows, channels, groups);
  printf("%d %d %lld\n", s.lanes, s.trows, (long long)s.rowblocks);
  return 0;
}
