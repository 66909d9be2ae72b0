"""More calls as in head_cases.CASES, of weights as wide as a vocabulary or as long as an int8 row may be: what runs there and in
no case of that list."""

CASES = [
    ("x in LDS i8 1 8 2", "i8", 10, 33032, 4096),
    ("x in LDS i8 2 8 2", "i8", 20, 33032, 4096),
    ("rows loss 1 2 4 4, k shared; join 2", "loss", 10, 520, 66048),
]

# the parts of x in LDS outgrow the workspace, or there are more tiles than arrival counts: run as tiles. (Up to 17 GB of w:
# looked at without running them; the GPU runs the same kernels in smaller calls.)
OUTGROWN = [
    ("tiles 128 logits dynamic; join 16", "loss", 16, 1 << 20, 8192),
    ("tiles 128 logits dynamic; join 2", "loss", 4, 1 << 20, 8192),
    ("tiles 128 logits dynamic, split; join 2", "loss", 8, 400000, 16384),
    ("rows i8 1 2 4 4", "i8", 12, 1 << 20, 16384),
]
