"""Shapes of 8-bit products and the form of the kernels that each of them takes:
(kind, rows, columns) with tiled forms in units of 64 rows and columns, and the
split and ring forms in units of 16."""

# Groups of no rows, of one, and of a row more than whole 16-row fragments,
# waves and tiles hold; what follows the last group.
UNEVEN = [1, 17, 0, 33, 65, 97, 129, 300, 2, 128]
SMALL = [1, 0, 3, 5, 16, 2, 17, 8] * 8
TAIL = 70

# rows at any byte, dense: (M, N, K)
DENSE = [
    ((70, 900, 257), ("split", 1, 1)),
    ((130, 1500, 1), ("staged", 1, 1)),
    ((130, 1500, 15), ("staged", 1, 1)),
    ((257, 4001, 7), ("staged", 2, 1)),
    ((257, 4001, 130), ("staged", 2, 1)),
    ((400, 5003, 17), ("staged", 2, 2)),
    ((511, 5003, 1041), ("staged", 2, 2)),
    ((400, 5003, 1), ("staged", 2, 2)),
    ((1100, 4001, 333), ("staged", 2, 4)),
    ((1000, 5003, 15), ("staged", 2, 4)),
]

# rows at any byte, by expert: (sizes, N, K)
GROUPS = [
    ((UNEVEN, 300, 257), ("split", 1, 2)),
    ((UNEVEN, 300, 7), ("split", 1, 2)),
    ((UNEVEN, 700, 333), ("staged", 1, 1)),
    ((UNEVEN, 513, 15), ("staged", 1, 1)),
    ((UNEVEN, 1001, 257), ("staged", 2, 1)),
    ((UNEVEN, 1001, 1), ("staged", 2, 1)),
    ((UNEVEN, 2047, 1041), ("staged", 2, 2)),
    ((UNEVEN, 2047, 17), ("staged", 2, 2)),
    ((UNEVEN, 4001, 333), ("staged", 2, 4)),
    ((UNEVEN, 4001, 7), ("staged", 2, 4)),
    ((UNEVEN * 2, 1600, 257), ("staged", 2, 4)),
    ((SMALL, 513, 130), ("staged", 2, 4)),
    ((SMALL, 1500, 333), ("staged", 2, 2)),
]

# rows 2^23 codes apart or more (A's where M is the smaller, else B's): (M, N, K)
FAR = [
    ((17, 70, 1041), ("split", 1, 1)),
    ((17, 6200, 1041), ("split", 1, 2)),
    ((6200, 17, 64), ("split", 1, 2)),
    ((9, 12300, 7), ("split", 1, 2)),
]

# whole pieces, dense: (M, N, K)
DENSE_PIECES = [
    ((4000, 4040, 240), ("pipe", 4, 4)),
    ((2000, 4040, 240), ("pipe", 2, 4)),
    ((2001, 2040, 240), ("pipe", 2, 2)),
    ((1000, 2039, 240), ("pipe", 2, 1)),
    ((970, 1001, 240), ("pipe", 1, 1)),
    ((17, 50, 16), ("pipe", 1, 1)),
    ((16, 8185, 1040), ("ring", 1, 1)),
    ((3, 8200, 1040), ("ring", 1, 2)),
    ((1, 16400, 1040), ("ring", 1, 4)),
]

# whole pieces, by expert: (sizes, N, K)
GROUP_PIECES = [
    ((SMALL, 513, 1040), ("pipe", 1, 4)),
    ((UNEVEN, 513, 1040), ("pipe", 2, 4)),
    (([700, 0, 3, 513, 256], 300, 272), ("pipe", 4, 4)),
    (([300, 17, 0, 1, 65, 640], 300, 16), ("pipe", 4, 4)),
]
