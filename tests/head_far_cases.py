"""More calls as in head_cases.CASES, of weights as wide as a vocabulary or as long as an int8 row may be: what runs there and in
no case of that list."""

CASES = [
    ("x in LDS i8 1 8 2", "i8", 10, 33032, 4096),
    ("x in LDS i8 2 8 2", "i8", 20, 33032, 4096),
    ("rows loss 1 2 4 4, k shared; join 2", "loss", 10, 520, 66048),
]
