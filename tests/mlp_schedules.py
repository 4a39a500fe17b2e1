"""One size for every schedule that a feed-forward product can be planned as
(152 SMs): tile shape; tiles claimed from a counter ("ticket"), more than a wave
of them ("waves") or at most one ("under"); and whether the last tiles are cut
into K segments.  The plan is checked where a size is used, so that a retuned
constant cannot leave a schedule without a test."""

from __future__ import annotations

import re

SCHEDULES = [
    # product, M, N, K, tile shape, order, split tail
    ("linear", 3892, 7528, 3040, "pair 256x256", "ticket", True),
    ("linear", 8443, 3336, 1008, "pair 256x256", "ticket", False),
    ("linear", 144, 4920, 5208, "pair 256x256", "under", True),
    ("linear", 132, 9888, 928, "pair 256x256", "under", False),
    ("linear", 262, 12992, 3264, "pair 256x256", "waves", True),
    ("linear", 2229, 11948, 67, "pair 256x256", "waves", False),
    ("linear", 154, 64, 1912, "single 128x128", "under", True),
    ("linear", 139, 64, 64, "single 128x128", "under", False),
    ("linear", 135, 9816, 64, "single 128x128", "waves", False),
    ("linear", 4406, 7608, 1056, "single 128x256", "ticket", False),
    ("linear", 317, 3344, 5720, "single 128x256", "under", True),
    ("linear", 264, 10088, 1048, "single 128x256", "under", False),
    ("linear", 289, 15392, 4048, "single 128x256", "waves", True),
    ("linear", 5968, 3869, 134, "single 128x256", "waves", False),
    ("gated", 5113, 2832, 2936, "pair 256x256", "ticket", True),
    ("gated", 1346, 9704, 1048, "pair 256x256", "ticket", False),
    ("gated", 5065, 71, 5316, "pair 256x256", "under", True),
    ("gated", 137, 5248, 752, "pair 256x256", "under", False),
    ("gated", 133, 10304, 3112, "pair 256x256", "waves", True),
    ("gated", 145, 14696, 392, "pair 256x256", "waves", False),
    ("gated", 132, 64, 1920, "single 128x128", "under", True),
    ("gated", 142, 64, 64, "single 128x128", "under", False),
    ("gated", 134, 4920, 64, "single 128x128", "waves", False),
    ("gated", 1396, 12976, 3272, "single 128x256", "ticket", True),
    ("gated", 2175, 7840, 976, "single 128x256", "ticket", False),
    ("gated", 270, 1698, 5885, "single 128x256", "under", True),
    ("gated", 266, 4960, 976, "single 128x256", "under", False),
    ("gated", 294, 7328, 4104, "single 128x256", "waves", True),
    ("gated", 278, 10072, 472, "single 128x256", "waves", False),
    ("linear_dx", 8527, 3096, 3584, "pair 256x256", "ticket", True),
    ("linear_dx", 4690, 1024, 6112, "pair 256x256", "ticket", False),
    ("linear_dx", 139, 5248, 5664, "pair 256x256", "under", True),
    ("linear_dx", 643, 64, 80, "pair 256x256", "under", False),
    ("linear_dx", 1034, 2928, 4288, "pair 256x256", "waves", True),
    ("linear_dx", 5149, 72, 5176, "pair 256x256", "waves", False),
    ("linear_dx", 129, 3488, 64, "single 128x128", "under", True),
    ("linear_dx", 133, 129, 64, "single 128x128", "under", False),
    ("linear_dx", 6936, 64, 264, "single 128x128", "waves", False),
    ("linear_dx", 7187, 1208, 3976, "single 128x256", "ticket", False),
    ("linear_dx", 266, 7348, 3371, "single 128x256", "under", True),
    ("linear_dx", 264, 72, 6464, "single 128x256", "under", False),
    ("linear_dx", 1093, 4824, 6152, "single 128x256", "waves", True),
    ("linear_dx", 2865, 136, 8088, "single 128x256", "waves", False),
    ("gated_dx", 6186, 1432, 5384, "pair 256x256", "ticket", True),
    ("gated_dx", 4990, 456, 6232, "pair 256x256", "ticket", False),
    ("gated_dx", 132, 2672, 5568, "pair 256x256", "under", True),
    ("gated_dx", 751, 64, 80, "pair 256x256", "under", False),
    ("gated_dx", 7767, 1528, 600, "pair 256x256", "waves", True),
    ("gated_dx", 2704, 72, 4448, "pair 256x256", "waves", False),
    ("gated_dx", 140, 1552, 64, "single 128x128", "under", True),
    ("gated_dx", 133, 72, 64, "single 128x128", "under", False),
    ("gated_dx", 6624, 64, 312, "single 128x128", "waves", False),
    ("gated_dx", 7526, 456, 4504, "single 128x256", "ticket", False),
    ("gated_dx", 266, 2872, 3232, "single 128x256", "under", True),
    ("gated_dx", 289, 64, 5320, "single 128x256", "under", False),
    ("gated_dx", 5661, 2456, 1064, "single 128x256", "waves", True),
    ("gated_dx", 5907, 72, 3864, "single 128x256", "waves", False),
    ("linear_dw", 2917, 14936, 1880, "pair 256x256", "ticket", True),
    ("linear_dw", 970, 10560, 2840, "pair 256x256", "ticket", False),
    ("linear_dw", 5417, 136, 5072, "pair 256x256", "under", True),
    ("linear_dw", 132, 824, 64, "pair 256x256", "under", False),
    ("linear_dw", 3112, 9808, 424, "pair 256x256", "waves", True),
    ("linear_dw", 1, 13208, 4304, "pair 256x256", "waves", False),
    ("linear_dw", 2990, 64, 64, "single 128x128", "under", True),
    ("linear_dw", 1, 64, 64, "single 128x128", "under", False),
    ("linear_dw", 6281, 14896, 296, "single 128x128", "waves", True),
    ("linear_dw", 1, 9730, 136, "single 128x128", "waves", False),
    ("linear_dw", 1569, 7448, 4520, "single 128x256", "ticket", False),
    ("linear_dw", 6761, 299, 3224, "single 128x256", "under", True),
    ("linear_dw", 302, 72, 8072, "single 128x256", "under", False),
    ("linear_dw", 5688, 1056, 5720, "single 128x256", "waves", True),
    ("linear_dw", 138, 3688, 6456, "single 128x256", "waves", False),
    ("gated_dw", 2891, 4640, 3216, "pair 256x256", "ticket", True),
    ("gated_dw", 1031, 14888, 784, "pair 256x256", "ticket", False),
    ("gated_dw", 5399, 136, 2712, "pair 256x256", "under", True),
    ("gated_dw", 135, 424, 72, "pair 256x256", "under", False),
    ("gated_dw", 3542, 10341, 132, "pair 256x256", "waves", True),
    ("gated_dw", 1, 5024, 5600, "pair 256x256", "waves", False),
    ("gated_dw", 2731, 64, 88, "single 128x128", "under", True),
    ("gated_dw", 1, 64, 64, "single 128x128", "under", False),
    ("gated_dw", 1803, 10080, 64, "single 128x128", "waves", True),
    ("gated_dw", 1, 10376, 64, "single 128x128", "waves", False),
    ("gated_dw", 1032, 2400, 7136, "single 128x256", "ticket", False),
    ("gated_dw", 5944, 80, 4896, "single 128x256", "under", True),
    ("gated_dw", 164, 69, 5058, "single 128x256", "under", False),
    ("gated_dw", 4166, 296, 7696, "single 128x256", "waves", True),
    ("gated_dw", 154, 1304, 8584, "single 128x256", "waves", False),
    ("gated_dw", 129, 66, 66, "pair 256x128", "under", False),
    ("gated_dx", 142, 64, 64, "pair 256x128", "under", False),
    ("linear_dw", 137, 197, 83, "pair 256x128", "under", False),
    ("linear_dx", 129, 64, 64, "pair 256x128", "under", False),
]

ROW = re.compile(r"((?:pair|single) \d+x\d+) tiles=(\d+) k_blocks=\d+ grid=\d+ raster=\d+ "
                 r"split=(\d+)x\d+ schedule=(ticket|static) beside=[01]")


def schedule(text, sms):
    """(tile shape, order, split tail) of a tg_product_plan_describe line."""
    m = ROW.fullmatch(text)
    assert m, text
    teams = sms // 2 if m[1].startswith("pair") else sms
    order = "ticket" if m[4] == "ticket" else "under" if int(m[2]) <= teams else "waves"
    return m[1], order, int(m[3]) > 0
