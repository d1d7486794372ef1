"""Sizes (M, N, K) that reach each kernel of moe_mx_linear, by the kernel's name in
csrc/mx_linear_rule.hpp. test_mx_linear_rule_cpu.py asks the rule itself whether they do."""

# Whole products. The two-buffer kernels (TILE_LARGEST) fetch scales for 1024 (MXFP8) or 2048 K values at a
# time: up to three fetches, odd and even numbers of stages of 128 or 256, ragged and whole ends, N that is
# and is not a multiple of 8.
LARGEST = {
    "mxfp8": [(1537, 3848, 1056), (1600, 4096, 2304), (1500, 4100, 2336), (1664, 3841, 128)],
    "mxfp4": [(3585, 3592, 2080), (3400, 3840, 4608), (3400, 3840, 4128), (3600, 3500, 4384), (3584, 3585, 256)],
}
OTHERS = [
    ("SKINNY_8_1_1_LITE", 3, 2048, 7168), ("SKINNY_4_1_1_LITE", 2, 4112, 4096), ("SKINNY_8_1_1", 13, 90, 20000),
    ("SKINNY_4_2_1", 12, 4200, 4128), ("SKINNY_4_1_2", 30, 2048, 9120), ("SKINNY_X_2_2", 25, 8200, 4096),
    ("TILE_64_64", 130, 4000, 4160), ("TILE_64_128", 8192, 256, 7168), ("TILE_128_128", 300, 7000, 2336),
]
# N that takes 16-byte accesses, and N that does not
EPILOGUE = [
    ("TILE_LARGEST", "mxfp8", 1500, (4104, 4100)), ("TILE_LARGEST", "mxfp4", 3600, (3504, 3500)),
    ("TILE_128_128", "mxfp8", 300, (7000, 7003)), ("TILE_128_128", "mxfp4", 300, (7000, 7003)),
    ("TILE_64_128", "mxfp8", 200, (5200, 5201)), ("TILE_64_128", "mxfp4", 200, (5200, 5201)),
    ("TILE_64_64", "mxfp8", 130, (4000, 4002)), ("TILE_64_64", "mxfp4", 130, (4000, 4002)),
]
EPILOGUE_K = 352
# one small case of each kernel that multiplies MXFP8 rows exactly
EXACT = [
    ("SKINNY_8_1_1_LITE", 3, 2048), ("SKINNY_4_1_1_LITE", 2, 4112), ("SKINNY_8_1_1", 13, 90), ("SKINNY_4_2_1", 12, 4200),
    ("SKINNY_4_1_2", 30, 2048), ("SKINNY_X_2_2", 25, 4200), ("TILE_64_64", 130, 4000), ("TILE_64_128", 200, 5200),
    ("TILE_128_128", 300, 7000),
]
EXACT_K = 640
