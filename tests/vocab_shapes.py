"""Shapes (tokens, ids, hidden) of the GPU tests of the losses over a vocabulary."""

# tokens around the tiles' 32, 64, 128 and 256, ids around 64 and 256 (and below a wave's 32), K
# around the copies' 64 and with ends inside them
SMALL = [(1, 1, 8), (1, 256, 64), (2, 7, 16), (31, 255, 56), (32, 257, 72), (33, 300, 128), (64, 1000, 136),
         (65, 511, 64), (100, 700, 200), (128, 256, 264), (129, 513, 72), (200, 33, 8), (256, 512, 128),
         (257, 769, 136), (300, 1031, 520), (513, 300, 64)]

# enough ids for the wide tiles, each with a last tile that is not whole
LARGE = [(32, 100001, 520), (64, 66000, 72), (127, 40001, 584), (129, 70000, 264), (500, 70001, 520),
         (700, 40300, 648), (60, 20001, 1160), (128, 5003, 2056), (1000, 3001, 264)]

# every tile of the logits with few K steps (one, two, five or nine copies of 64) and a last tile of one id or
# one short, one token, one short or whole; the last member: tokens that count
TILES = [(31, 255, 72, 31), (63, 257, 8, 63), (33, 255, 520, 33),
         (63, 16385, 8, 63), (65, 11263, 72, 65), (128, 8447, 520, 128),
         (127, 16385, 8, 127), (129, 13311, 264, 129), (640, 3327, 72, 640), (639, 3327, 520, 639),
         (31, 32769, 8, 31), (65, 17407, 72, 65), (32, 33791, 520, 32),
         (63, 32769, 8, 63), (129, 17407, 72, 129), (64, 33791, 520, 64),
         (127, 32769, 8, 127), (129, 26623, 72, 129), (128, 32769, 264, 128), (639, 6655, 520, 639),
         (255, 32769, 8, 255), (257, 26623, 72, 257), (256, 33791, 520, 256), (300, 40001, 136, 127),
         (300, 40001, 136, 129), (700, 40300, 72, 100), (700, 40300, 72, 300)]

# heads beyond the 256 MiB up to which the logits' second pass leaves them in the cache, and beyond the 32
# MiB up to which dX does
STREAMED = [(33, 131001, 1032, 33), (200, 131001, 1032, 200), (200, 131001, 1032, 100), (60, 20001, 1160, 60),
            (300, 131001, 1032, 300), (16, 131001, 1032, 16), (127, 131001, 1032, 127), (64, 131001, 1032, 64)]


# more tokens than those whose G is held in two parts, on every tile, one more than a tile's among them, and
# both sides of that number among masked ones
HALF = [(5603, 89, 6272, 5603), (5067, 334, 1808, 5067), (5787, 377, 1408, 5787), (602, 3280, 3016, 602),
        (1301, 6081, 480, 1301), (1260, 7826, 416, 1024), (3924, 24490, 32, 3924), (769, 10241, 1032, 769),
        (641, 12801, 520, 641), (513, 40001, 264, 513), (1100, 3001, 1160, 128), (1100, 3001, 1160, 129),
        (1000, 33333, 520, 128), (1000, 33333, 520, 129), (257, 100003, 392, 257), (2000, 9001, 1032, 414)]


TWICE = 128  # tokens that count up to which a gradient holds G in two parts of bf16; beyond, in fp16


def bodies(plan, M, N, K, live, need_dX=True, need_dW=True):
    """(product, ids, tokens or rows, hint, fp16) of the kernel bodies that a call of the losses and one of
    the gradients run; `plan` as binding.vocab_plan. "hint": W's copies, dW's stores, leave the caches alone."""
    def ceil(a, b):
        return -(-a // b)

    if live == 0:
        return set()
    half = live > TWICE

    def logits(what, ids, stream, half):
        bn, bm = plan(M, ids, K)[:2]
        if bm == 256:  # where tiles of 128 tokens take fewer rounds, they run
            a, grid = ceil(ids, 256), max(256, ceil(ceil(ids, 256) * ceil(M, 256), 8) * 8)
            part, whole = a * ceil(live, 128), a * ceil(live, 256)
            if part <= grid and ceil(part, 256) * 2 < ceil(whole, 256) * 3:
                bm = 128
            what += " wide"
        return (what, bn, bm, stream and live <= bm, half)

    out = {logits("sums", N, True, False)}
    dx_rows, piece = plan(M, N, K)[2:]
    rows = live if half else 2 * live
    for id0 in range(0, N, piece):
        ids = min(piece, N - id0)
        out.add(logits("G", ids, not need_dX or ids * K * 2 > 1 << 28, half))
        if need_dX:
            out.add(("dX" if need_dW else "dX alone", 256, dx_rows, ids * K * 2 > 1 << 25 and rows <= dx_rows, half))
        if need_dW:
            out.add(("dW", 256, 256, rows <= 256, half))
    return out
