"""Products of the layer operators, one for each kernel, split and way of running them that the choice of tiles and rows
(256 CUs) makes: on the CPU the choice is asserted, on the GPU each is compared with the oracle. A refit of the choice that
moves a case to another kernel fails the first test, so that no kernel loses its comparison unseen.

(what runs, kind, m, n, k): kind is the operands' type of layer_linear, or dx or dw of layer_linear_backward."""

LINEAR = [
    # rows <type>, blocks of x, blocks of w, waves; "shared": several workgroups share a tile's k
    ("rows bf16 1 1 4", "bf16", 1, 16584, 520),
    ("rows bf16 1 1 8", "bf16", 3, 264, 136),
    ("rows bf16 1 1 8 shared", "bf16", 4, 264, 8200),
    ("rows bf16 1 2 4", "bf16", 12, 10248, 3296),
    ("rows bf16 1 2 4 shared", "bf16", 9, 2824, 12928),
    ("rows bf16 2 2 4", "bf16", 21, 5000, 264),
    ("rows bf16 2 2 4 shared", "bf16", 18, 264, 2056),
    ("rows bf16 4 2 4", "bf16", 35, 5000, 264),
    ("rows bf16 4 2 4 shared", "bf16", 64, 264, 2056),
    ("rows e4m3 1 1 4", "e4m3", 1, 16584, 528),
    ("rows e4m3 1 1 8", "e4m3", 5, 264, 144),
    ("rows e4m3 1 1 8 shared", "e4m3", 2, 264, 8208),
    ("rows e4m3 1 2 4", "e4m3", 16, 9640, 3504),
    ("rows e4m3 1 2 4 shared", "e4m3", 7, 3976, 9168),
    ("rows e4m3 2 2 4", "e4m3", 31, 5000, 272),
    ("rows e4m3 2 2 4 shared", "e4m3", 17, 264, 4112),
    ("rows e4m3 2 4 4", "e4m3", 24, 16392, 2736),
    ("rows e4m3 2 4 4 shared", "e4m3", 29, 2552, 13680),
    ("rows e4m3 4 2 4", "e4m3", 33, 5000, 272),
    ("rows e4m3 4 2 4 shared", "e4m3", 61, 264, 4112),
    # tiles <edge>, layout, one workgroup a unit ("one wave") or the dynamic scheduler; which of them are split along k
    ("tiles 128 NT one wave", "bf16", 130, 1032, 136),
    ("tiles 128 NT one wave, all split", "bf16", 101, 520, 4104),
    ("tiles 128 NT dynamic", "bf16", 2049, 4104, 72),
    ("tiles 128 NT dynamic, all split", "bf16", 6, 11296, 7688),
    ("tiles 128 NT dynamic, last wave split", "bf16", 1066, 3600, 600),
    ("tiles 256 NT one wave", "bf16", 1237, 10392, 312),
    ("tiles 256 NT one wave, all split", "bf16", 300, 8200, 8208),
    ("tiles 256 NT dynamic", "bf16", 8418, 8912, 136),
    ("tiles 256 NT dynamic, last wave split", "bf16", 4104, 4104, 1032),
    ("tiles 128 E8 one wave", "e4m3", 130, 1032, 144),
    ("tiles 128 E8 one wave, all split", "e4m3", 101, 520, 4112),
    ("tiles 128 E8 dynamic", "e4m3", 2049, 4104, 80),
    ("tiles 128 E8 dynamic, all split", "e4m3", 36, 10928, 14992),
    ("tiles 128 E8 dynamic, last wave split", "e4m3", 142, 16520, 1280),
    ("tiles 256 E8 one wave", "e4m3", 1348, 9216, 800),
    ("tiles 256 E8 one wave, all split", "e4m3", 129, 8616, 7568),
    ("tiles 256 E8 dynamic", "e4m3", 6419, 4504, 528),
    ("tiles 256 E8 dynamic, last wave split", "e4m3", 1249, 13472, 1456),
]

BACKWARD = [
    ("tiles 128 NN one wave", "dx", 130, 264, 1032),
    ("tiles 128 NN one wave, all split", "dx", 9, 4104, 520),
    ("tiles 128 NN dynamic", "dx", 333, 72, 16456),
    ("tiles 128 NN dynamic, all split", "dx", 1, 4976, 16768),
    ("tiles 128 NN dynamic, last wave split", "dx", 4610, 584, 816),
    ("tiles 256 NN one wave", "dx", 969, 344, 12544),
    ("tiles 256 NN one wave, all split", "dx", 300, 8200, 4104),
    ("tiles 256 NN dynamic", "dx", 8963, 136, 8280),
    ("tiles 256 NN dynamic, last wave split", "dx", 6866, 688, 2360),
    ("tiles 128 TN one wave", "dw", 33, 264, 1032),
    ("tiles 128 TN one wave, all split", "dw", 2049, 264, 520),
    ("tiles 128 TN dynamic", "dw", 45, 4104, 8200),
    ("tiles 256 TN one wave", "dw", 1144, 3640, 4304),
    ("tiles 256 TN one wave, all split", "dw", 8200, 1032, 4104),
    ("tiles 256 TN dynamic", "dw", 193, 15424, 6400),
    ("tiles 256 TN dynamic, last wave split", "dw", 355, 7296, 13440),
]
