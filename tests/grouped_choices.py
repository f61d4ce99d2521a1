"""Sizes of the grouped products for every way in which they are computed."""
import torch

BF16, F32 = torch.bfloat16, torch.float32

# (product, type of the result, slices of the contraction or 0: pairs of CTAs, rows, experts, N (fc1: n), K)
CASES = [
    ("fc1", BF16, 0, 1500, 5, 1288, 1288), ("fc1", BF16, 0, 700, 5, 2056, 136), ("fc1", BF16, 0, 7, 7, 2760, 8),
    ("fc1", BF16, 1, 200, 5, 1160, 880), ("fc1", BF16, 1, 3, 3, 8, 8), ("fc1", BF16, 2, 51, 3, 1568, 1144),
    ("fc1", BF16, 2, 4, 4, 1280, 3912), ("fc1", BF16, 4, 150, 5, 72, 664), ("fc1", BF16, 4, 3, 3, 8, 680),
    ("fc1", BF16, 8, 90, 5, 136, 1352), ("fc1", BF16, 8, 3, 3, 8, 1512),
    ("mm", BF16, 0, 1500, 5, 1288, 1288), ("mm", BF16, 0, 1200, 5, 2056, 520), ("mm", BF16, 1, 700, 5, 2056, 136),
    ("mm", BF16, 1, 3, 3, 8, 8), ("mm", BF16, 2, 51, 3, 1568, 1144), ("mm", BF16, 2, 5, 3, 3200, 1296),
    ("mm", BF16, 4, 150, 5, 72, 664), ("mm", BF16, 4, 3, 3, 8, 680), ("mm", BF16, 8, 90, 5, 136, 1352),
    ("mm", BF16, 8, 3, 3, 8, 1512),
    ("dgrad", BF16, 0, 1500, 5, 1288, 1288), ("dgrad", BF16, 0, 1200, 5, 520, 2056),
    ("dgrad", BF16, 1, 700, 5, 136, 2056), ("dgrad", BF16, 1, 3, 3, 8, 8), ("dgrad", BF16, 2, 51, 3, 1144, 1568),
    ("dgrad", BF16, 2, 5, 3, 1296, 3200), ("dgrad", BF16, 4, 150, 5, 664, 72), ("dgrad", BF16, 4, 3, 3, 680, 8),
    ("dgrad", BF16, 8, 90, 5, 1352, 136), ("dgrad", BF16, 8, 3, 3, 1512, 8),
    ("wgrad", BF16, 0, 1500, 5, 1288, 1288), ("wgrad", BF16, 0, 700, 5, 776, 1032),
    ("wgrad", BF16, 1, 300, 5, 520, 1160), ("wgrad", BF16, 2, 1925, 5, 72, 72), ("wgrad", BF16, 4, 2600, 4, 136, 72),
    ("wgrad", BF16, 8, 6000, 4, 136, 264),
    ("wgrad", F32, 0, 500, 5, 1032, 1288), ("wgrad", F32, 0, 1500, 5, 1288, 1288),
    ("wgrad", F32, 0, 7000, 3, 1288, 1288), ("wgrad", F32, 1, 300, 5, 520, 1160), ("wgrad", F32, 1, 4197, 7, 8, 1304),
    ("wgrad", F32, 2, 1000, 3, 72, 72), ("wgrad", F32, 2, 1925, 5, 72, 72), ("wgrad", F32, 4, 2000, 3, 136, 136),
    ("wgrad", F32, 4, 2600, 4, 136, 72), ("wgrad", F32, 8, 3900, 3, 136, 264), ("wgrad", F32, 8, 6000, 4, 136, 264),
]


def counts_of(rows, experts):
    """Rows per expert, uneven: the second has none, the third at least one; and the rows
    of no expert."""
    tail = rows // 12
    parts = [(5, 0, 2, 1, 3)[e % 5] for e in range(experts)]
    counts = [(rows - tail) * p // sum(parts) for p in parts]
    counts[2] = max(counts[2], 1)
    counts[0] += rows - tail - sum(counts)
    return counts, tail
