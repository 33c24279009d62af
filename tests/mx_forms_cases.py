"""Cases of the 4-bit products that reach every form a call may take, for the GPU tests that
run them and for the host test that holds the rules to them."""

MANY = (64, 128, 8, 16, "skew", 0.1)      # a few rows on each of many experts
SERIES = (400, 128, 8, 1, "skew", 0.1)    # the same, more tiles than run at once
MIDDLE = (700, 64, 8, 16, "skew", 0.1)    # about 100 rows an expert, more 128-wide tiles than run at once
FOUR = (260, 4, 2, 16, "random", 0.0)
EIGHT = (520, 8, 4, 16, "skew", 0.0)
LONG = (2100, 16, 4, 16, "skew", 0.0)     # runs of every length
SHORT = (40, 8, 2, 16, "skew", 0.1)

# depths: a multiple of 128 that ends inside a stage of weights, and one that is no multiple of 128
DEPTHS = (384, 224)

# form, rows (as in the products' tests), N, and which rows take it
FORWARD = [
    ("split", 20, 96, "both"), ("split", SHORT, 96, "both"),  # 16 columns a workgroup, 32 for MXFP4 rows out
    ("split32by2", 16, 16416, "both"), ("split32by2", SHORT, 800, "both"),
    ("32x128", MANY, 288, "both"), ("32x128", SERIES, 544, "both"),
    ("64x128", 300, 544, "mxfp4"), ("64x128", FOUR, 544, "mxfp4"),
    ("32x64", 300, 544, "bf16"), ("32x64", FOUR, 544, "bf16"),
    ("64x64", 1100, 1056, "bf16"), ("64x64", EIGHT, 800, "bf16"),
    ("128x128", 2100, 2080, "both"), ("128x128", MIDDLE, 800, "both"),
    ("256x256", LONG, 2080, "both"),
]

# form, rows, N (of the depth), K
BACKWARD = [
    ("32x128", MANY, 72, 288), ("32x128", SERIES, 200, 544), ("64x128", 300, 72, 544), ("64x128", FOUR, 200, 544),
    ("128x128", 2100, 72, 2080), ("128x128", MIDDLE, 200, 800), ("256x256", LONG, 136, 2080),
]
