"""Shapes at which a block of the residual norm's kernels holds one wide group and
takes several rows in turn: [rows, channels] with one group a row."""

# the forward takes rows in turn past 32,768 (8192 past 8192 channels)
FORWARD = [(32_900, 2056), (8300, 8200)]
# the backward past 512 (192 past 4096 channels)
BACKWARD = [(1000, 1024), (1100, 1032), (1537, 2048), (1026, 4096), (500, 6144), (400, 8192),
            (300, 8200), (200, 16384)]
