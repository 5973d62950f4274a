"""Sizes of the 8-bit integer products by the kernel form that they take.

The form is chosen on the host (``wq_int8_form``, csrc/wq_int8_plan.cpp); tests
assert it for every size here, so that a change of the rule shows up as a failure
instead of leaving a kernel without a test.  Each form is met with whole steps of
K and with a short last one (two kernels of each LDS-tiled form), with more steps
than its ring of operands has places, with fewer, and with odd widths."""

import ctypes

from block_forms import ROUND, MOST_REST, _uneven
from weight_only_bit_dequant_amd import wq

FORMS = ("dot 2", "dot 4", "dot 8", "stream 16x16", "stream 16x16 deep", "stream 32x16", "stream 16x32", "tile 256x256", "tile 256x128",
         "tile 128x128", "tile 128x64", "tile 64x64", "tile 32x64")

# (form, M, N, K)
PLAIN = [
    ("dot 2", 3, 248, 4352), ("dot 2", 3, 165, 4592), ("dot 2", 3, 56, 6240),
    ("dot 4", 2, 152, 1408), ("dot 4", 1, 2413, 5936), ("dot 4", 1, 112, 1344),
    ("dot 4", 2, 24, 448), ("dot 8", 3, 3752, 1536), ("dot 8", 2, 2358, 1584),
    ("dot 8", 2, 2992, 1488), ("dot 8", 1, 5344, 192), ("stream 16x16", 4, 5328, 2560),
    ("stream 16x16", 20, 3730, 2512), ("stream 16x16", 34, 936, 1200), ("stream 16x16", 3, 2648, 448),
    ("stream 16x16 deep", 20, 160, 1664), ("stream 16x16 deep", 16, 389, 4928), ("stream 16x16 deep", 14, 16, 4640),
    ("stream 16x16 deep", 8, 32, 208), ("stream 32x16", 4, 8192, 512), ("stream 32x16", 14, 3338, 224),
    ("stream 32x16", 3, 8192, 448), ("stream 32x16", 5, 424, 16), ("stream 16x32", 159, 248, 2304),
    ("stream 16x32", 122, 543, 1264), ("stream 16x32", 129, 16, 1200), ("stream 16x32", 142, 192, 688),
    ("tile 256x256", 2655, 3616, 2176), ("tile 256x256", 1657, 5054, 1712), ("tile 256x256", 1985, 4408, 1328),
    ("tile 256x256", 3128, 4856, 32), ("tile 256x128", 2495, 2000, 1792), ("tile 256x128", 939, 4507, 2336),
    ("tile 256x128", 1619, 2888, 1904), ("tile 256x128", 783, 6480, 16), ("tile 128x128", 1795, 1408, 1152),
    ("tile 128x128", 715, 2813, 2880), ("tile 128x128", 528, 3936, 960), ("tile 128x128", 2576, 1272, 32),
    ("tile 128x64", 1708, 1104, 2048), ("tile 128x64", 2436, 538, 4496), ("tile 128x64", 1035, 1352, 3152),
    ("tile 128x64", 1342, 1264, 208), ("tile 64x64", 209, 3384, 1280), ("tile 64x64", 3509, 308, 1104),
    ("tile 64x64", 181, 2744, 1008), ("tile 64x64", 627, 1552, 48), ("tile 32x64", 2835, 112, 1920),
    ("tile 32x64", 1219, 323, 1360), ("tile 32x64", 550, 48, 3216), ("tile 32x64", 2047, 16, 416),
]

# (form, rows of each expert, N, K, gathered from this many rows or None, rows past the last expert's)
GROUPED = [
    ("dot 4", _uneven(8, 3), 136, 2432, 1, 0),
    ("dot 4", _uneven(70, 25), 530, 2096, 8, 0),
    ("dot 4", _uneven(3, 1), 592, 32, 1, 0),
    ("dot 8", _uneven(70, 5), 704, 1792, 1, 0),
    ("dot 8", _uneven(40, 4), 3184, 1088, 1, 3),
    ("dot 8", _uneven(40, 40), 157, 1200, 11, 0),
    ("stream 16x16", _uneven(70, 202), 105, 1792, None, 0),
    ("stream 16x16", _uneven(8, 110), 600, 720, None, 3),
    ("stream 16x16", _uneven(40, 435), 120, 416, 145, 0),
    ("stream 16x16 deep", _uneven(3, 28), 490, 1024, None, 0),
    ("stream 16x16 deep", _uneven(3, 52), 17, 1728, None, 3),
    ("stream 16x16 deep", _uneven(8, 39), 58, 464, 4, 0),
    ("stream 32x16", _uneven(70, 572), 1286, 896, 190, 0),
    ("stream 32x16", _uneven(40, 407), 1132, 3376, 100, 0),
    ("stream 32x16", _uneven(40, 822), 394, 832, 274, 0),
    ("stream 32x16", _uneven(70, 60), 791, 240, None, 3),
    ("stream 16x32", _uneven(8, 281), 243, 1024, None, 3),
    ("stream 16x32", _uneven(3, 111), 961, 960, 37, 0),
    ("stream 16x32", _uneven(70, 3192), 38, 64, None, 0),
    ("tile 256x256", _uneven(8, 2445), 3062, 1792, 815, 3),
    ("tile 256x256", _uneven(40, 5686), 2952, 864, 1635, 0),
    ("tile 256x256", _uneven(3, 4224), 3065, 272, 1408, 3),
    ("tile 256x128", _uneven(70, 2880), 1544, 1152, None, 3),
    ("tile 256x128", _uneven(8, 4898), 1528, 1104, None, 0),
    ("tile 256x128", _uneven(40, 1981), 1410, 448, None, 3),
    ("tile 128x128", _uneven(3, 3398), 856, 2304, 1132, 3),
    ("tile 128x128", _uneven(40, 2228), 3081, 960, None, 3),
    ("tile 128x128", _uneven(70, 5873), 1600, 64, 1957, 0),
    ("tile 128x64", _uneven(8, 1206), 1128, 1152, None, 3),
    ("tile 128x64", _uneven(40, 5012), 248, 2480, None, 3),
    ("tile 128x64", _uneven(8, 174), 3761, 240, None, 0),
    ("tile 64x64", _uneven(40, 983), 408, 1280, 327, 0),
    ("tile 64x64", _uneven(3, 5872), 320, 992, None, 0),
    ("tile 64x64", _uneven(8, 1645), 313, 16, 748, 0),
    ("tile 32x64", _uneven(3, 1611), 32, 1280, None, 0),
    ("tile 32x64", _uneven(8, 546), 112, 1616, None, 3),
    ("tile 32x64", _uneven(3, 778), 24, 176, None, 0),
]

_SPLIT_TILES = {"tile 256x256": (256, 256), "tile 256x128": (256, 128)}


def form(T, N, K, E=0):
    """The form of a call with T rows of Y (E = 0: a plain Linear)."""
    f = wq.lib().wq_int8_form
    f.restype, f.argtypes = ctypes.c_char_p, [ctypes.c_int64] * 4
    return f(T, E, N, K).decode()


def rest(form, counts, N):
    """Tiles of the last round that are computed in 128 x 128 pieces, for the rows of each expert ([M]: plain)."""
    if form not in _SPLIT_TILES:
        return 0
    bn, bm = _SPLIT_TILES[form]
    tiles = -(-N // bn) * sum(-(-c // bm) for c in counts)
    return tiles % ROUND if tiles >= ROUND and tiles % ROUND <= MOST_REST else 0


# As PLAIN and GROUPED, with a last round that is split.
PLAIN_SPLIT = [
    ("tile 256x128", 2527, 8192, 1024), ("tile 256x128", 8192, 2426, 752), ("tile 256x128", 7754, 2416, 1152),
    ("tile 256x256", 8192, 6418, 1408), ("tile 256x256", 6488, 5160, 528), ("tile 256x256", 2390, 7080, 592),
]
GROUPED_SPLIT = [
    ("tile 256x128", _uneven(3, 3075), 2425, 512, 768, 0),
    ("tile 256x128", _uneven(3, 3253), 4848, 560, None, 0),
    ("tile 256x256", _uneven(3, 6048), 3987, 768, 1332, 0),
    ("tile 256x256", _uneven(8, 5540), 2760, 528, None, 0),
]
