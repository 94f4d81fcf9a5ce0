"""Sizes of the products that the few-row kernel answers with clusters of CTAs, by the number of CTAs and the
rounds of units that each cluster walks on a GB300; test_linear_plan.py holds them against the plan."""

# clusters of so many of these CTAs that an idle GB300 with 152 SMs holds at once, one CTA to an SM
ROOM = {1: 152, 2: 76, 3: 46, 4: 36, 5: 28, 6: 23, 7: 15, 8: 15}

# (rows, or rows of each group; K, N, activation, e4m3, CTAs of a cluster, rounds)
CLUSTERS = [
    (33, 4000, 204, "none", False, 8, 1), (9, 3880, 204, "none", False, 7, 1),
    (5, 2760, 1536, "silu_mul", False, 5, 1), (7, 2576, 256, "silu_mul", False, 7, 1),
    (3, 4736, 1930, "none", True, 5, 1), (11, 4352, 201, "none", True, 7, 1),
    (2, 4864, 3072, "silu_mul", True, 5, 1), (10, 4352, 256, "silu_mul", True, 7, 1),
]
ROUNDS = [
    (3163, 36488, 141, "none", False, 5, 2), (54, 14968, 19968, "silu_mul", False, 2, 3),
    (647, 85872, 1024, "silu_mul", False, 5, 2),
    (2495, 15616, 139, "none", True, 3, 2), (41, 14208, 20133, "none", True, 2, 3),
    (2978, 34304, 130, "none", True, 4, 3), (3645, 128768, 210, "none", True, 6, 5),
    (2796, 12288, 256, "silu_mul", True, 3, 2), (32, 11776, 19968, "silu_mul", True, 3, 4),
    (3648, 95872, 256, "silu_mul", True, 6, 5),
    ((124, 22, 119), 17632, 1433, "none", False, 3, 2),
    ((1, 1, 1, 1, 1, 26, 1), 21688, 597, "none", False, 4, 2),
    ((112, 101, 1, 79, 116, 6, 72), 36712, 409, "none", False, 5, 3),
    ((5, 7), 19576, 2816, "silu_mul", False, 3, 2),
    ((3, 146, 206, 1, 180, 0, 0, 215, 1), 27504, 512, "silu_mul", False, 5, 3),
    ((216, 0, 150, 137, 117, 0, 1), 26752, 702, "none", True, 4, 3),
    ((13, 3), 26240, 4735, "none", True, 2, 2),
    ((96, 57, 4, 92), 11392, 1536, "silu_mul", True, 3, 2),
    ((11, 1, 1), 15616, 7936, "silu_mul", True, 2, 5),
    ((1,), 25216, 19712, "silu_mul", True, 3, 7),
]

# gated e4m3 calls of many rows: (rows, or rows of each group; K, N)
GATED_FP8 = [(300, 384, 4096), (777, 1024, 2048), ((400, 0, 257, 131), 384, 512)]
