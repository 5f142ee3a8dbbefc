"""Shapes (tokens, ids, hidden) of the GPU tests of the losses over a vocabulary."""

# tokens around the tiles' 32, 64, 128 and 256, ids around 64 and 256 (and below a wave's 32), K
# around the copies' 64 and with ends inside them
SMALL = [(1, 1, 8), (1, 256, 64), (2, 7, 16), (31, 255, 56), (32, 257, 72), (33, 300, 128), (64, 1000, 136),
         (65, 511, 64), (100, 700, 200), (128, 256, 264), (129, 513, 72), (200, 33, 8), (256, 512, 128),
         (257, 769, 136), (300, 1031, 520), (513, 300, 64)]

# enough ids for the wide tiles, each with a last tile that is not whole
LARGE = [(32, 100001, 520), (64, 66000, 72), (127, 40001, 584), (129, 70000, 264), (500, 70001, 520),
         (700, 40300, 648), (60, 20001, 1160), (128, 5003, 2056), (1000, 3001, 264)]
