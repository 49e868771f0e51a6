"""Sizes at which the convolution and the selective scan take each form of their kernels, as
(sizes, the form): the states, tokens, sequences or channels of a lane and the cut over time
are chosen by size.  test_layer_layout.py holds every form to the library's own rules, and
the GPU tests compare every form with float64."""

# (Bt, T, Dm, N), states per lane, cut over time
SCAN_FWD = [
    ((1025, 41, 33, 8), 4, False), ((1025, 41, 36, 8), 4, False),
    ((512, 41, 65, 16), 4, False), ((512, 41, 68, 16), 4, False),
    ((512, 41, 33, 32), 4, False), ((512, 41, 36, 32), 4, False),
    ((2, 41, 33, 64), 4, False), ((2, 41, 36, 64), 4, False),
    ((199, 400, 33, 8), 4, True), ((199, 400, 36, 8), 4, True),
    ((100, 400, 65, 16), 4, True), ((100, 400, 68, 16), 4, True),
    ((100, 400, 33, 32), 4, True), ((100, 400, 36, 32), 4, True),
    ((2, 140, 33, 64), 4, True), ((2, 140, 36, 64), 4, True),
    ((3, 41, 129, 8), 2, False), ((3, 41, 132, 8), 2, False),
    ((3, 41, 65, 16), 2, False), ((3, 41, 68, 16), 2, False),
    ((3, 41, 33, 32), 2, False), ((3, 41, 36, 32), 2, False),
    ((2, 140, 129, 8), 2, True), ((2, 140, 132, 8), 2, True),
    ((2, 140, 65, 16), 2, True), ((2, 140, 68, 16), 2, True),
    ((2, 140, 33, 32), 2, True), ((2, 140, 36, 32), 2, True),
]

SCAN_BWD = [
    ((130, 41, 65, 8), 2, False), ((130, 41, 68, 8), 2, False),
    ((2, 41, 65, 8), 2, True), ((2, 41, 68, 8), 2, True),
    ((130, 50, 33, 16), 2, False), ((130, 50, 36, 16), 2, False),
    ((2, 70, 33, 16), 2, True), ((2, 70, 36, 16), 2, True),
    ((260, 50, 33, 16), 4, False), ((260, 50, 36, 16), 4, False),
    ((96, 41, 33, 16), 4, True), ((96, 41, 36, 16), 4, True),
    ((96, 41, 33, 32), 2, False), ((96, 41, 36, 32), 2, False),
    ((2, 70, 33, 32), 2, True), ((2, 70, 36, 32), 2, True),
    ((192, 41, 33, 32), 4, False), ((192, 41, 36, 32), 4, False),
    ((64, 41, 33, 32), 4, True), ((64, 41, 36, 32), 4, True),
    ((96, 50, 33, 64), 4, False), ((96, 50, 36, 64), 4, False),
    ((2, 70, 33, 64), 4, True), ((2, 70, 36, 64), 4, True),
]

# (Bt, Dm, N), channels per lane; three blocks of channels, the last one short
SCAN_STEP = [((350, 300, 8), 2), ((350, 131, 16), 2), ((350, 70, 32), 2), ((350, 35, 64), 2),
             ((7, 300, 8), 1), ((7, 131, 16), 1), ((7, 70, 32), 1), ((7, 35, 64), 1)]

EVEN, ODD = (4000, 52, 52), (4001, 50, 51)
# (Bt, T, splits), tokens per lane
CONV_FWD = [((Bt, 77, s), run) for Bt, run in ((86, 32), (26, 16), (13, 8), (2, 4))
            for s in (EVEN, ODD)]
CONV_BWD = [((Bt, 77, s), run) for Bt, run in ((43, 32), (26, 16), (13, 8), (2, 4))
            for s in (EVEN, ODD)]
# (Bt, splits), sequences per lane
CONV_STEP = [((259, (2048, 64, 64)), 4), ((259, (2050, 63, 65)), 4), ((259, (513, 2, 1)), 1)]
