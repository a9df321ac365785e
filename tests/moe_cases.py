"""Grouped products by the kernel that takes them on a GB300 of 152 SMs: for few rows, CTA pairs on narrow tiles, on wide ones.
A case: operation, kernel, the experts' rows, rows behind the last, K, N (gated: the packed columns), gathered rows."""
EVEN = [40, 1, 0, 16, 17, 33, 64, 5]                         # few rows on eight experts
MANY = [0, 1, 15, 16, 17, 0, 63, 64, 65, 30] + [0] * 54      # most experts without any
MIXED = [0, 1, 15, 16, 17, 0, 129, 255, 256, 257, 300, 513, 0]
LONG = [1300, 0, 1801]
SKEWED = [0] * 40 + [2000, 3] + [0] * 22                     # rows taken as spread, but on one expert
SKEWED_FEW = [0] * 60 + [600, 0, 0, 1]
SMALL = [(37 * i) % 129 for i in range(256)]                 # 256 small experts, 64 rows each on average
MOST = [(11 * i) % 33 for i in range(1024)]                  # the most experts

CASES = [
    ("forward", "few", EVEN, 37, 136, 520, False), ("forward", "few", EVEN, 0, 1032, 264, True),
    ("forward", "few", MANY, 37, 200, 1000, False), ("forward", "few", MANY, 37, 4104, 520, True),
    ("forward", "few", SKEWED_FEW, 5, 136, 264, True), ("forward", "few", [1], 0, 4104, 8, False),
    ("forward", "narrow", MIXED, 37, 200, 520, False), ("forward", "narrow", MIXED, 37, 1032, 520, True),
    ("forward", "narrow", SKEWED, 9, 72, 1000, False), ("forward", "narrow", SMALL, 3, 136, 264, False),
    ("forward", "wide", MIXED, 37, 200, 1544, True), ("forward", "wide", LONG, 37, 4104, 2000, False),
    ("forward", "wide", SKEWED, 9, 136, 1544, True), ("forward", "wide", SMALL, 3, 200, 1544, True),
    ("forward", "wide", MOST, 1, 72, 520, True),
    ("gated", "few", EVEN, 37, 136, 768, False), ("gated", "few", EVEN, 0, 1032, 512, True),
    ("gated", "few", MANY, 37, 200, 1024, True), ("gated", "few", SKEWED_FEW, 5, 136, 256, False),
    ("gated", "narrow", MIXED, 37, 200, 768, False), ("gated", "narrow", MIXED, 37, 1032, 768, True),
    ("gated", "narrow", SKEWED, 9, 72, 1024, False), ("gated", "narrow", SMALL, 3, 136, 512, False),
    ("gated", "wide", MIXED, 37, 200, 1792, True), ("gated", "wide", LONG, 37, 2056, 2560, False),
    ("gated", "wide", SKEWED, 9, 136, 1792, True), ("gated", "wide", SMALL, 3, 200, 1536, True),
    ("dx", "few", EVEN, 37, 520, 136, False), ("dx", "few", MANY, 37, 1000, 4104, False), ("dx", "few", SKEWED_FEW, 5, 264, 136, False),
    ("dx", "narrow", MIXED, 37, 520, 200, False), ("dx", "narrow", SKEWED, 9, 1000, 72, False), ("dx", "narrow", SMALL, 3, 264, 136, False),
    ("dx", "wide", LONG, 37, 2000, 4104, False), ("dx", "wide", SMALL, 3, 1032, 4104, False),
    ("gated dx", "few", [0, 1, 15, 16, 17, 0, 33, 5], 0, 384, 200, False), ("gated dx", "few", SKEWED_FEW[:-4] + [100, 0, 0, 1], 5, 128, 4104, False),
    ("gated dx", "narrow", MIXED, 37, 640, 200, False), ("gated dx", "narrow", SKEWED, 9, 384, 72, False), ("gated dx", "narrow", SMALL, 3, 256, 136, False),
    ("dw", "narrow", MIXED, 37, 200, 520, False), ("dw", "narrow", MIXED, 37, 264, 136, True), ("dw", "narrow", SKEWED, 9, 136, 264, False),
    ("dw", "narrow", SMALL, 3, 72, 520, False),
    ("dw", "wide", MIXED, 37, 1032, 1544, True), ("dw", "wide", [2700, 61], 37, 2056, 4616, False), ("dw", "wide", SKEWED, 9, 136, 1544, True),
    ("dw", "wide", SMALL, 3, 200, 1544, True), ("dw", "wide", MOST, 1, 72, 520, True),
]


def name(case):
    op, kernel, counts, behind, K, N, gathered = case
    return f"{op}-{kernel}-{len(counts)}x{sum(counts) + behind}-{K}-{N}{'-gathered' if gathered else ''}"
