"""Sizes of the routed-expert tests that are to reach a kernel, checked on the CPU against the plans."""

# Rows per expert that make entries of exactly the heights where row tiles change (64, 128, 192,
# 256), one more, one less; products of few k-tiles (whole ones, and with a last one of 32).
HEIGHTS = [(256, 192, 128, 64), (255, 257, 193, 191, 129, 127, 65, 63), (512, 448, 384, 320)]
HEIGHT_KS = [(32, 32), (96, 32), (128, 128), (320, 64)]
HEIGHT_INNER, HEIGHT_N = 4512, 8768

# (T, E, topk, K, inner, N, g) of a whole MLP, and whether its first and second products stream.
FAMILIES = [
    ((1500, 4, 2, 96, 1056, 2080, 32), 0, 0),
    ((1500, 4, 2, 64, 1088, 2048, 64), 0, 0),
    ((1500, 4, 2, 160, 1056, 96, 32), 0, 1),
    ((1500, 4, 2, 128, 1024, 256, 64), 0, 1),
    ((1500, 4, 2, 288, 96, 2080, 32), 1, 0),
    ((1500, 4, 2, 64, 64, 2048, 64), 1, 0),
]
