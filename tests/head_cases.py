"""int8 products, cross entropies and their gradients, one for each kernel, split and way of running them that the choices (256
CUs) make: on the CPU the choice is asserted, on the GPU each is compared with the oracle. A refit of a choice that moves a case
to another kernel fails the first test, so that no kernel loses its comparison unseen.

(what runs, kind, m, n, k): i8 is layer_linear, loss layer_cross_entropy, dx and dw layer_cross_entropy_backward in one piece."""

# what a call launches, in words; for hip_stand_in.run, after `assert lib.layer_create(...)`
WHAT_RUNS = r"""
import re
assert lib.layer_create(ctypes.byref(plan), 0) == 0
hip.stand_in_launches()
FORMS = {"7": "logits", "8": "logit gradients", "5": "NN", "6": "TN"}
MODES = {("4", "0"): "one wave", ("4", "2"): "dynamic", ("8", "0"): "one a CU"}
def what_runs(kind, m, n, k):
    if kind == "i8":
        a = layer.LinearArgs(x=P, w=P, out=P, m=m, n=n, k=k, ldx=k, ldw=k, ldo=n, in_type=3, out_type=1)
        assert call(lib.layer_linear, a) == 0, (kind, m, n, k)
    elif kind == "loss":
        a = layer.CrossEntropyArgs(x=P, w=P, label=P, lse=P, m=m, n=n, k=k, ldx=k, ldw=k)
        assert call(lib.layer_cross_entropy, a) == 0, (kind, m, n, k)
    else:
        a = layer.CrossEntropyGradArgs(x=P, w=P, label=P, lse=P, dx=P if kind == "dx" else None, dw=P if kind == "dw" else None, scratch=P,
                                       scratch_bytes=2 * m * n, m=m, n=n, k=k, ldx=k, ldw=k, lddx=k, lddw=k, dx_type=1, dw_type=1)
        assert call(lib.layer_cross_entropy_backward, a) == 0, (kind, m, n, k)
    words = []
    for line in hip.stand_in_launches().decode().splitlines():
        name, gx, gy, block, first, chunks = line.split()
        kernel, numbers = re.match(r"_ZN3ptg\d+ptg_(\w+?)_kernelI(.*?)EEv", name).groups()
        d = re.findall(r"L[ib](\d+)E?", numbers)
        shares = ", k shared" if int(gy) > 1 else ""
        if kernel == "product_i8":
            words.append("tiles %s int8 %s" % (d[0], MODES[d[1], d[2]]))
        elif kernel in ("product_scaled", "loss"):
            words.append("tiles %s %s %s" % (d[0], FORMS[d[1]], MODES[d[2], d[3]]))
        elif kernel in ("product_i8_reduce", "product_scaled_reduce"):
            words[-1] += ", all split" if first == "0" else ", last wave split"
        elif kernel == "loss_chunks":
            words[-1] += ", split"
        elif kernel.startswith("rows_shared"):
            words.append("x in LDS %s %s%s" % (kernel.split("_")[2], " ".join(d), shares))
        elif kernel.startswith("rows"):
            words.append("rows %s %s%s" % (kernel.split("_")[1], " ".join(d), shares))
        elif kernel == "loss_join":
            words.append("join %s" % d[0])
        else:
            words.append(kernel)
    return "; ".join(words)
"""

CASES = [
    ("rows i8 1 1 4 4", "i8", 1, 16512, 80),
    ("rows i8 1 1 8 4", "i8", 2, 64, 64),
    ("rows i8 1 1 8 4, k shared", "i8", 1, 72, 4224),
    ("rows i8 1 2 4 4", "i8", 3, 5056, 6656),
    ("rows i8 1 2 4 4, k shared", "i8", 2, 3336, 10096),
    ("rows i8 2 1 4 2", "i8", 18, 4096, 80),
    ("rows i8 2 1 8 2", "i8", 21, 64, 80),
    ("rows i8 2 1 8 2, k shared", "i8", 18, 64, 4512),
    ("rows i8 4 1 4 2", "i8", 34, 4096, 112),
    ("rows i8 4 1 8 2", "i8", 33, 64, 128),
    ("rows i8 4 1 8 2, k shared", "i8", 37, 64, 4816),
    ("tiles 128 int8 dynamic", "i8", 1029, 13656, 64),
    ("tiles 128 int8 dynamic, last wave split", "i8", 13323, 576, 9344),
    ("tiles 128 int8 one a CU", "i8", 78, 72, 64),
    ("tiles 128 int8 one a CU, all split", "i8", 66, 64, 1472),
    ("tiles 128 int8 one wave", "i8", 158, 16536, 240),
    ("tiles 128 int8 one wave, all split", "i8", 6000, 160, 10768),
    ("tiles 128 int8 one wave, last wave split", "i8", 8414, 408, 4864),
    ("tiles 256 int8 dynamic", "i8", 9653, 2056, 64),
    ("tiles 256 int8 dynamic, last wave split", "i8", 10406, 1632, 1104),
    ("tiles 256 int8 one wave", "i8", 7522, 1056, 112),
    ("tiles 256 int8 one wave, all split", "i8", 6371, 168, 16208),
    ("x in LDS i8 1 4 4", "i8", 10, 16448, 2048),
    ("x in LDS i8 1 4 4, k shared", "i8", 11, 3296, 10208),
    ("x in LDS i8 1 8 2, k shared", "i8", 9, 13264, 10240),
    ("x in LDS i8 2 4 4", "i8", 17, 13632, 2480),
    ("x in LDS i8 2 4 4, k shared", "i8", 32, 4120, 4080),
    ("x in LDS i8 2 8 2, k shared", "i8", 17, 10952, 12704),
    ("x in LDS i8 4 8 2", "i8", 62, 16440, 1088),
    ("x in LDS i8 4 8 2, k shared", "i8", 33, 2968, 5712),
    ("rows loss 1 1 4 4; join 2", "loss", 2, 16808, 88),
    ("rows loss 1 1 8 4, k shared; join 16", "loss", 16, 64, 2056),
    ("rows loss 1 1 8 4; join 1", "loss", 1, 96, 80),
    ("rows loss 1 2 4 4; join 2", "loss", 15, 46720, 768),
    ("rows loss 2 2 4 2, k shared; join 16", "loss", 24, 72, 1008),
    ("rows loss 2 2 4 2; join 16", "loss", 17, 64, 128),
    ("rows loss 4 2 4 2, k shared; join 16", "loss", 41, 88, 1072),
    ("rows loss 4 2 4 2; join 16", "loss", 36, 72, 72),
    ("tiles 128 logits dynamic, split; join 16", "loss", 19, 66176, 640),
    ("tiles 128 logits dynamic; join 2", "loss", 5, 105328, 208),
    ("tiles 128 logits one a CU, split; join 16", "loss", 74, 88, 504),
    ("tiles 128 logits one a CU; join 16", "loss", 86, 64, 104),
    ("tiles 128 logits one wave, split; join 16", "loss", 5657, 248, 4632),
    ("tiles 128 logits one wave; join 2", "loss", 10, 47216, 376),
    ("tiles 256 logits dynamic, split; join 16", "loss", 212, 66304, 640),
    ("tiles 256 logits dynamic; join 16", "loss", 160, 94432, 64),
    ("tiles 256 logits one wave, split; join 16", "loss", 5078, 432, 5416),
    ("tiles 256 logits one wave; join 16", "loss", 166, 34048, 128),
    ("x in LDS loss 1 4 4, k shared; join 2", "loss", 11, 4736, 7808),
    ("x in LDS loss 1 4 4; join 2", "loss", 14, 16328, 2144),
    ("x in LDS loss 1 8 2, k shared; join 2", "loss", 6, 9728, 6984),
    ("x in LDS loss 1 8 2; join 2", "loss", 2, 20872, 3240),
    ("x in LDS loss 2 4 4, k shared; join 16", "loss", 21, 3136, 5376),
    ("x in LDS loss 2 4 4; join 16", "loss", 19, 9200, 1928),
    ("x in LDS loss 2 8 2, k shared; join 16", "loss", 17, 16720, 4208),
    ("x in LDS loss 4 8 2, k shared; join 16", "loss", 33, 3144, 5392),
    ("x in LDS loss 4 8 2; join 16", "loss", 42, 17280, 1024),
    ("tiles 128 logit gradients dynamic, split; tiles 128 NN one a CU, all split", "dx", 9, 66168, 496),
    ("tiles 128 logit gradients one a CU, split; tiles 128 NN dynamic", "dx", 3171, 72, 5048),
    ("tiles 128 logit gradients one a CU, split; tiles 128 NN one wave", "dx", 937, 88, 5696),
    ("tiles 128 logit gradients one a CU, split; tiles 256 NN dynamic", "dx", 4701, 72, 4992),
    ("tiles 128 logit gradients one a CU, split; tiles 256 NN one wave", "dx", 1253, 64, 8000),
    ("tiles 128 logit gradients one a CU; tiles 128 NN one a CU", "dx", 3, 80, 72),
    ("tiles 128 logit gradients one a CU; tiles 256 NN dynamic, last wave split", "dx", 3740, 704, 4608),
    ("tiles 128 logit gradients one a CU; tiles 256 NN one wave, all split", "dx", 956, 3504, 2176),
    ("tiles 128 logit gradients one wave, split; tiles 128 NN one wave, all split", "dx", 211, 5424, 5480),
    ("tiles 128 logit gradients one wave, split; tiles 128 NN one wave, last wave split", "dx", 2355, 1784, 1680),
    ("tiles 128 logit gradients one wave; tiles 128 NN one a CU, all split", "dx", 3, 40328, 72),
    ("tiles 256 logit gradients dynamic; tiles 128 NN one a CU, all split", "dx", 136, 89904, 120),
    ("tiles 256 logit gradients one wave; tiles 128 NN dynamic, last wave split", "dx", 1358, 6432, 6128),
    ("tiles 128 logit gradients dynamic; tiles 128 TN dynamic", "dw", 1, 71528, 72),
    ("tiles 128 logit gradients one a CU, split; tiles 256 TN one wave", "dw", 638, 2408, 3736),
    ("tiles 128 logit gradients one a CU; tiles 128 TN one wave", "dw", 2, 80, 64),
    ("tiles 128 logit gradients one a CU; tiles 128 TN one wave, all split", "dw", 735, 72, 96),
    ("tiles 256 logit gradients dynamic, split; tiles 128 TN dynamic", "dw", 170, 67664, 664),
    ("tiles 256 logit gradients one wave, split; tiles 256 TN dynamic", "dw", 1256, 4072, 7624),
    ("tiles 256 logit gradients one wave, split; tiles 256 TN dynamic, last wave split", "dw", 2227, 2488, 7720),
    ("tiles 256 logit gradients one wave, split; tiles 256 TN one wave, all split", "dw", 4357, 672, 5496),
]
