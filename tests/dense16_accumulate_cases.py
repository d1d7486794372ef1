"""Sizes, (rows, width in, width out), of gradients that are added to earlier ones beyond the few rows held at once."""
ACCUMULATE = [(129, 136, 200), (257, 776, 328), (300, 2048, 64), (8200, 72, 2120), (4099, 2056, 2088), (8200, 1528, 1496)]
