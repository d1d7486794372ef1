"""Sizes of adapters without a projection, (rows, width in, width out, rank, adapters), that between them take every way through the second
product's kernel: K ranges of the first product that it joins itself, that a kernel of their own joins, or none; workgroups
of 16 and of 64 rows; ranks in one pass of 64 or in several."""
ALONE = [(256, 7168, 1100, 64, 16), (1000, 2056, 515, 136, 5), (2047, 1032, 264, 256, 9), (70, 8200, 203, 24, 3), (1025, 1032, 97, 8, 40),
         (2100, 4104, 1100, 64, 4), (2048, 2056, 330, 128, 3), (200, 520, 141, 200, 4), (130, 776, 328, 64, 9), (3000, 520, 259, 72, 6),
         (5000, 520, 136, 16, 7)]
