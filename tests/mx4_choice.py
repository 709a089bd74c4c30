"""Which kernel a product of microscaled 4-bit values runs, worked out as csrc/mx4.hip does (choose_mx4 and
launch_product), and what of it a size reaches.  The estimate's constants are read from the source."""

import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_group_quantized_w4_amd", "csrc",
                      "mx4.hip")
MiB = 1 << 20

# What the functions below repeat, as it stands in the source (white space aside).
REPEATED = [
    "if (rows <= 16) return nb < 256 ? Mx4::kStream1x4 : nb < 384 ? Mx4::kStream2x4 : nb < 1024 ? Mx4::kStream2x2 : "
    "Mx4::kStream2x1;",
    "const int64_t spread = M / s.BM + busy / 2; const int64_t tiles = busy == 1 ? (M + s.BM - 1) / s.BM : spread > busy ? "
    "spread : busy; const int64_t blocks = tiles * ((N + s.BN - 1) / s.BN); double load = (double)blocks / s.slots;",
    "load = (double)(blocks / kCus) + (left == 0 ? 0 : left <= kMostCut ? 0.45 : 1);",
    "const double full = s.start + (double)steps * (load * s.all > s.one ? load * s.all : s.one); const double few = s.bare + "
    "(double)steps * s.step, cost = full > few ? full : few;",
    "constexpr int kCus = 256, kMostCut = kCus / 4;",
    "const int64_t busy = a.experts < a.M ? a.experts : a.M, bytes = busy * a.N * a.K / 2; if (bytes >= (busy == 1 ? 12 : 32) * "
    "(int64_t(1) << 20))",
]


def source():
    with open(SOURCE) as f:
        return f.read()


def shapes():
    """(kind, BM, BN, threads, slots, start, one, all, bare, step) of the estimate's kernels."""
    found = re.findall(r"\{Mx4::k(\w+)" + r", (\d+)" * 4 + r", ([\d.]+)" * 5 + r"\}", source())
    return [(f[0], *map(int, f[1:5]), *map(float, f[5:])) for f in found]


def up(a, b):
    return -(-a // b)


def kernel(M, N, K, experts=1):
    """The kernel's name; a streaming one past the caches ends in "Past"."""
    busy = min(experts, M)
    rows, nb, steps = up(M, busy), up(N, 16) * busy, up(K, 256)
    if rows <= 16:
        best = "Stream1x4" if nb < 256 else "Stream2x4" if nb < 384 else "Stream2x2" if nb < 1024 else "Stream2x1"
    else:
        least = None
        for kind, BM, BN, _, slots, start, one, every, bare, step in shapes():
            if not slots:
                continue
            tiles = up(M, BM) if busy == 1 else max(M // BM + busy // 2, busy)
            blocks = tiles * up(N, BN)
            load = blocks / slots
            if kind == "Tile256":
                left = blocks % 256
                load = blocks // 256 + (0 if left == 0 else 0.45 if left <= 64 else 1)
            cost = max(start + steps * max(load * every, one), bare + steps * step)
            if least is None or cost < least:
                least, best = cost, kind
    if best == "Stream2x1" and busy * N * K // 2 >= (12 if busy == 1 else 32) * MiB:
        best += "Past"
    return best


# Sizes that reach each kernel, with ends inside a tile of rows, of outputs and of K: (M, N, K) of dense calls, and
# (rows of each expert, N, K) of calls by expert, 5 rows of none before and 3 behind.
DENSE = {
    "Stream1x4": [(13, 2001, 4736), (1, 17, 128)],
    "Stream2x4": [(15, 5003, 1152)],
    "Stream2x2": [(3, 9217, 2688), (26, 124, 896), (70, 33, 13440)],
    "Stream2x1": [(13, 20001, 640), (152, 102, 128), (69, 5672, 2304)],
    "Stream2x1Past": [(1, 65537, 384), (16, 28673, 1152), (20, 65537, 384), (17, 30001, 896)],
    "Deep32x64": [(19, 4555, 1664), (154, 1133, 4224)],
    "Deep64": [(251, 1774, 5248), (311, 8545, 128)],
    "Deep64x128": [(500, 2561, 9088), (263, 3140, 11392)],
    "Deep128": [(327, 8264, 1152), (273, 7413, 2816)],
    "Tile256": [(260, 7521, 128), (633, 4908, 2176)],
}
GROUPED = {
    "Stream1x4": [([1, 16, 0, 3], 146, 640)],
    "Stream2x4": [([0, 7], 2150, 640)],
    "Stream2x2": [([50, 0, 42], 581, 9472)],
    "Stream2x1": [([2, 31, 0, 33, 4], 3833, 1152)],
    "Stream2x1Past": [([3, 0, 16, 1, 9, 17, 40, 0, 2, 5, 1, 7], 2561, 2432), ([20, 0, 16, 52, 30, 2], 4867, 3456)],
    "Deep32x64": [([20, 2, 49, 0, 72], 1130, 5248)],
    "Deep64": [([130, 0, 1, 100, 66], 1547, 5376)],
    "Deep64x128": [([433, 0, 458], 1746, 6784), ([200, 0, 170, 233, 264], 1352, 8576)],
    "Deep128": [([70, 128, 0, 131, 11, 123], 3703, 2176)],
    "Tile256": [([257, 0, 300, 15], 3481, 128)],
}
NONE_BEFORE, NONE_BEHIND = 5, 3
