"""Sizes at which linear attention takes each form of its kernels, as (sizes, the form): the
state's columns of a workgroup and the cut over time are chosen by size, and so is whether a
gradient's three recurrences share a launch.  test_block_layout.py holds every form to the
library's own rules, and the GPU tests compare every form with float64."""

# (Bt, T, H, G, K, V), columns, segments
ATTN_FWD = [
    ((2, 70, 3, 3, 64, 64), 64, 1), ((2, 70, 3, 1, 128, 128), 64, 1),
    ((40, 45, 5, 5, 64, 128), 128, 1), ((50, 45, 4, 2, 128, 72), 128, 1),
    ((16, 33, 16, 16, 64, 80), 128, 1), ((13, 33, 15, 5, 16, 128), 128, 1),
    ((25, 40, 4, 4, 64, 256), 128, 1), ((25, 40, 4, 2, 128, 200), 128, 1),
    ((25, 40, 4, 2, 200, 200), 64, 1),
    ((65, 40, 4, 4, 64, 128), 64, 1), ((48, 40, 4, 1, 128, 128), 64, 1),
    ((2, 600, 2, 2, 64, 64), 64, 2), ((1, 1100, 4, 2, 128, 128), 64, 4),
    ((1, 800, 2, 1, 256, 192), 64, 3),
]
# (Bt, T, H, G, K, V), columns, segments, recurrences in one launch
ATTN_BWD = [
    ((2, 70, 3, 3, 64, 96), 64, 1, True), ((2, 70, 3, 1, 128, 64), 64, 1, True),
    ((2, 40, 4, 2, 40, 200), 64, 1, True),
    ((14, 45, 5, 5, 64, 128), 128, 1, False), ((14, 45, 5, 1, 64, 128), 128, 1, False),
    ((17, 45, 4, 4, 128, 128), 128, 1, False), ((17, 45, 4, 2, 128, 96), 128, 1, False),
    ((9, 40, 4, 4, 256, 64), 128, 1, False), ((9, 40, 4, 2, 136, 200), 64, 1, False),
    ((22, 40, 4, 4, 64, 64), 64, 1, False), ((22, 40, 4, 2, 48, 128), 64, 1, False),
    ((24, 40, 4, 1, 128, 128), 64, 1, False), ((24, 40, 4, 4, 128, 72), 64, 1, False),
    ((9, 40, 4, 1, 120, 200), 128, 1, False),
    ((1, 600, 2, 2, 64, 64), 64, 2, True), ((1, 1100, 4, 2, 128, 64), 64, 4, True),
    ((1, 1100, 6, 3, 64, 200), 64, 4, False), ((1, 800, 2, 1, 256, 192), 64, 3, True),
]
