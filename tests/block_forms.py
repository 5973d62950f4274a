"""Sizes of the block-scaled products by the kernel form that they take.

The form is chosen on the host (``wq_block_form``, csrc/wq_block_plan.cpp);
tests assert it for every size here, so that a change of the rule shows up as a
failure instead of leaving a kernel without a test.  Each LDS-tiled form is met
with whole scale blocks of K and with a short last one (two kernels), an odd
and an even number of blocks, and more than 16 of them for each group of waves
(the scales are fetched 8 blocks at a time into two buffers)."""

import ctypes

from weight_only_bit_dequant_amd import wq

# (form, M, N, K)
PLAIN = [
    ("stream 16x16", 3, 1000, 1168), ("stream 16x16", 20, 2000, 2560),
    ("stream 16x16 deep", 30, 1000, 7424), ("stream 16x16 deep", 2, 2500, 6160),
    ("stream 32x16 eight", 32, 4096, 3072), ("stream 32x16 eight", 50, 3002, 2192),
    ("stream 32x16", 5, 4500, 1040), ("stream 32x16", 37, 3000, 1920),
    ("stream 32x32", 60, 5000, 640), ("stream 32x32", 45, 8190, 1168), ("stream 32x32", 100, 1224, 3120),
    ("tile 64x64 one", 86, 7771, 2128), ("tile 64x64 one", 86, 7776, 2176),
    ("tile 64x64", 256, 4096, 4096), ("tile 64x64", 200, 3000, 4480), ("tile 64x64", 97, 4010, 4448), ("tile 64x64", 70, 5650, 4544),
    ("tile 128x64", 300, 6152, 4096), ("tile 128x64", 131, 5788, 4480), ("tile 128x64", 139, 5489, 4688), ("tile 128x64", 150, 5480, 4496),
    ("tile 128x128", 334, 5534, 2176), ("tile 128x128", 258, 6593, 2272),
    ("tile 256x128", 538, 7266, 2176), ("tile 256x128", 726, 5649, 2128),
    ("tile 256x256", 1684, 4621, 2176), ("tile 256x256", 1684, 4624, 2144),
]


def _uneven(E, T):
    """E counts of sum T, every fifth expert without rows, the others up to five times each other."""
    w = [0 if e % 5 == 2 else 1 + 4 * (e * 7 % 11) / 10 for e in range(E)]
    n = [int(T * x / sum(w)) for x in w]
    n[0] += T - sum(n)
    return n


# (form, rows of each expert, N, K, gathered from this many rows or None, rows past the last expert's)
GROUPED = [
    ("stream 16x16", [1, 0, 2], 1000, 2064, 70, 3), ("stream 16x16", [7, 0, 3, 30], 1000, 2560, None, 0),
    ("stream 16x16 deep", [1, 0, 2], 600, 5776, 70, 3), ("stream 16x16 deep", [10, 20, 2], 1100, 6144, None, 0),
    ("stream 32x16", [17, 0, 5, 1] * 5, 392, 528, 70, 3), ("stream 32x16", _uneven(32, 64), 2048, 2048, 16, 0),
    ("stream 64x16", [16, 0, 40, 3, 1] * 26, 648, 272, 70, 3), ("stream 64x16", _uneven(70, 600), 1530, 1152, None, 0),
    ("stream 32x32", _uneven(3, 60), 504, 1024, None, 0), ("stream 32x32", _uneven(70, 1300), 24, 912, 70, 5),
    ("tile 64x64 one", _uneven(3, 74), 4438, 2144, 40, 2), ("tile 64x64 one", _uneven(70, 1290), 392, 2048, None, 0),
    ("tile 64x64", _uneven(3, 66), 3519, 4464, 40, 0), ("tile 64x64", _uneven(70, 1707), 386, 4608, None, 0),
    ("tile 128x64", _uneven(3, 67), 4595, 4560, 40, 0), ("tile 128x64", _uneven(70, 1261), 208, 4480, None, 0),
    ("tile 128x128", _uneven(3, 67), 8068, 3968, 40, 0), ("tile 128x128", _uneven(70, 1302), 379, 2784, 500, 9),
    ("tile 256x128", _uneven(3, 501), 7327, 2176, 300, 0), ("tile 256x128", _uneven(70, 1208), 632, 2256, None, 0),
    ("tile 256x256", _uneven(3, 925), 7463, 2176, 600, 0), ("tile 256x256", _uneven(8, 770), 6530, 144, 500, 30),
    ("tile 256x256", _uneven(70, 7020), 672, 384, 3000, 0),
]


def form(T, N, K, E=0):
    """The form of a call with T rows of Y (E = 0: a plain Linear)."""
    f = wq.lib().wq_block_form
    f.restype, f.argtypes = ctypes.c_char_p, [ctypes.c_int64] * 4
    return f(T, E, N, K).decode()


ROUND, MOST_REST = 256, 128  # tiles in a round of the chip; the largest rest of one that is split
_SPLIT_TILES = {"tile 256x256": (256, 256), "tile 256x128": (256, 128)}


def rest(form, counts, N):
    """Tiles of the last round that are computed in 128 x 128 pieces, for the rows of each expert ([M]: plain)."""
    if form not in _SPLIT_TILES:
        return 0
    bn, bm = _SPLIT_TILES[form]
    tiles = -(-N // bn) * sum(-(-c // bm) for c in counts)
    return tiles % ROUND if tiles >= ROUND and tiles % ROUND <= MOST_REST else 0


# As PLAIN and GROUPED, with a last round that is split.
PLAIN_SPLIT = [
    ("tile 256x128", 2573, 7577, 2176), ("tile 256x128", 2833, 6734, 2208), ("tile 256x128", 3387, 5699, 16),
    ("tile 256x256", 2362, 6940, 2176), ("tile 256x256", 2317, 6696, 2096), ("tile 256x256", 4300, 4096, 528),
]
GROUPED_SPLIT = [
    ("tile 256x128", [260, 260, 293], 7190, 2096, 500, 0), ("tile 256x128", [270, 260, 300], 7184, 2176, None, 0),
    ("tile 256x128", _uneven(70, 1240), 1111, 2288, None, 0), ("tile 256x128", _uneven(70, 1192), 1144, 2048, 700, 0),
    ("tile 256x256", [520, 522, 600], 7642, 2096, None, 0), ("tile 256x256", [600, 518, 514], 7184, 2176, 900, 0),
]
