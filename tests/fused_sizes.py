"""Sizes (M, K, N, g) with which awq_gemm_fused's tests reach the row tiles, by their height and whether K is split;
N counts the outputs.  That they do is a test of the plans on the CPU."""

# Whole k-tiles and half ones, groups that begin at even k-tiles, any, and inside one; a last tile that is shorter, and
# columns that end inside a tile.
TILES = {
    (64, False): [(100, 64, 22016, 32), (75, 96, 22016, 32), (75, 320, 22016, 64)],
    (128, False): [(75, 160, 44128, 32), (600, 192, 11008, -1)],
    (192, False): [(130, 96, 33056, 32), (380, 512, 22528, 128)],
    (256, False): [(250, 160, 33056, 32), (391, 1024, 22016, -1)],
    (64, True): [(130, 4128, 2112, 32)],
    (128, True): [(75, 4128, 8256, 32), (75, 8160, 11008, 96), (600, 8192, 4096, -1)],
    (192, True): [(130, 4096, 8256, 64), (700, 6144, 4096, 384)],
    (256, True): [(250, 8160, 8256, 96), (250, 8192, 8224, -1)],
}
GATED_TILES = {
    (64, False): [(260, 4096, 5504, 64)],
    (128, False): [(75, 160, 22048, 32), (600, 1024, 5504, -1)],
    (192, False): [(130, 96, 16544, 32), (180, 128, 22016, 128)],
    (256, False): [(250, 320, 16544, 64), (391, 1024, 11008, -1)],
    (64, True): [(75, 8160, 544, 96)],
    (128, True): [(130, 4128, 2048, 32), (500, 8192, 544, -1)],
    (192, True): [(130, 4096, 4128, 64)],
    (256, True): [(700, 8192, 1056, -1), (250, 6144, 4128, 384)],
}
