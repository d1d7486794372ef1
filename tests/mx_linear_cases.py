"""Sizes (M, N, K) that reach each kernel of moe_mx_linear, by the kernel's name in
csrc/mx_linear_rule.hpp. test_mx_linear_rule_cpu.py asks the rule itself whether they do."""

# Whole products. The two-buffer kernels (TILE_LARGEST) fetch scales for 1024 (MXFP8) or 2048 K values at a
# time: up to three fetches, odd and even numbers of stages of 128 or 256, ragged and whole ends, N that is
# and is not a multiple of 8.
LARGEST = {
    "mxfp8": [(1537, 3848, 1056), (1600, 4096, 2304), (1500, 4100, 2336), (1664, 3841, 128)],
    "mxfp4": [(3585, 3592, 2080), (3400, 3840, 4608), (3400, 3840, 4128), (3600, 3500, 4384), (3584, 3585, 256)],
}
