"""Sizes of grouped products that take the form "dot 2" (single rows of long weights), laid out as int8_forms.GROUPED:
gathered rows and not, several rows of one expert, experts without rows, odd widths, rows past the last expert's."""

from block_forms import _uneven

GROUPED = [
    ("dot 2", _uneven(3, 2), 16, 9984, 1, 0),
    ("dot 2", _uneven(8, 5), 17, 5072, None, 3),
    ("dot 2", _uneven(8, 8), 40, 13696, 3, 0),
    ("dot 2", _uneven(4, 3), 2363, 9024, 2, 0),
    ("dot 2", [2, 0, 0, 1], 18, 4944, None, 1),
    ("dot 2", _uneven(16, 14), 17, 5504, 5, 0),
    ("dot 2", _uneven(70, 53), 29, 6528, 11, 0),
    ("dot 2", _uneven(70, 44), 24, 8064, None, 3),
    ("dot 2", [0, 0, 2, 0, 0, 0, 0, 0], 4096, 7168, 9, 2),
]
