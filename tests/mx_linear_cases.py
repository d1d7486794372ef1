"""Sizes (M, N, K) that reach each kernel of moe_mx_linear, by the kernel's name in
csrc/mx_linear_rule.hpp. test_mx_linear_rule_cpu.py asks the rule itself whether they do."""

# Whole products. The two-buffer kernels (TILE_LARGEST) fetch scales for 1024 (MXFP8) or 2048 K values at a
# time: up to three fetches, odd and even numbers of stages of 128 or 256, ragged and whole ends, N that is
# and is not a multiple of 8.
LARGEST = {
    "mxfp8": [(1537, 3848, 1056), (1600, 4096, 2304), (1500, 4100, 2336), (1664, 3841, 128)],
    "mxfp4": [(3585, 3592, 2080), (3400, 3840, 4608), (3400, 3840, 4128), (3600, 3500, 4384), (3584, 3585, 256)],
}
# N that takes 16-byte accesses, and N that does not
EPILOGUE = [
    ("TILE_LARGEST", "mxfp8", 1500, (4104, 4100)), ("TILE_LARGEST", "mxfp4", 3600, (3504, 3500)),
    ("TILE_128_128", "mxfp8", 300, (7000, 7003)), ("TILE_128_128", "mxfp4", 300, (7000, 7003)),
    ("TILE_64_128", "mxfp8", 200, (5200, 5201)), ("TILE_64_128", "mxfp4", 200, (5200, 5201)),
    ("TILE_64_64", "mxfp8", 130, (4000, 4002)), ("TILE_64_64", "mxfp4", 130, (4000, 4002)),
]
EPILOGUE_K = 352
