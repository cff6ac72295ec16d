"""Attention calls of the paged cache, named after the way in which the host
cuts them: the call (nq, nkv, hd, page, P, lens, new, window), its rows of
padding, and what the host has to choose for it on 148 SMs."""

H32 = (40, 8, 128)
FEW, PASS, NONE, AHEAD = "with the rows of few_kernel", "a pass of its own", "no prefix", "ahead of the own keys"

PATHS = {
    # one or a few requests behind a prompt: the prefix as a last sequence of few_kernel
    "one row behind a prompt": ((*H32, 64, 5000, [3], [1], 0), 0, dict(prefix=FEW)),
    "three rows behind a prompt": ((*H32, 64, 5000, [1, 70, 300], [1] * 3, 0), 0, dict(prefix=FEW)),
    "a window that ends inside the prompt": ((*H32, 64, 5000, [1, 70, 300], [1] * 3, 2000), 0, dict(prefix=FEW)),
    "a window that hides the prompt from some": ((*H32, 16, 5001, [10, 700, 90], [1] * 3, 100), 0, dict(prefix=FEW)),
    "a window that hides the prompt": ((*H32, 64, 5000, [300, 200, 400], [1] * 3, 64), 0, dict(prefix=FEW)),
    "48 rows behind a prompt": ((8, 2, 64, 16, 5003, [20, 9], [9, 2], 0), 1, dict(prefix=FEW, few=48)),
    "48 rows, a window": ((8, 2, 64, 16, 5003, [20, 700], [9, 2], 3000), 1, dict(prefix=FEW, few=48)),
    "one row of 16 heads": ((16, 1, 128, 32, 4500, [5, 0], [1, 0], 0), 0, dict(prefix=FEW, few=16)),
    "drafted rows of 16 heads": ((16, 1, 64, 128, 4500, [5], [2], 0), 0, dict(prefix=FEW, few=32)),
    # a pass over the prefix, its window's end inside it (rows of a tile see different parts)
    "a tile of rows, window": ((*H32, 64, 1000, list(range(10, 910, 45)), [1, 2, 3, 1] * 5, 700),
                               1, dict(prefix=PASS, few=16, gap=False)),
    "a pair and a rest, window": ((*H32, 64, 1000, list(range(10, 910, 15)), [1] * 60, 700),
                                  3, dict(prefix=PASS, gap=True)),
    "small heads, window": ((8, 2, 64, 16, 1003, list(range(10, 710, 10)), [1] * 70, 650), 1, dict(prefix=PASS, gap=True)),
    # a rest of rows in fewer pieces than the whole pair tiles
    "a pair and a rest": ((*H32, 64, 4000, [30 + i for i in range(64)], [1] * 64, 0), 0, dict(prefix=PASS, gap=True)),
    "small heads, a pair and a rest": ((8, 2, 64, 16, 3001, [30 + i for i in range(70)], [1] * 70, 0),
                                       0, dict(prefix=PASS, gap=True)),
    "long window over a pair and a rest": ((*H32, 32, 3000, [30 + i for i in range(64)], [1] * 64, 2500),
                                           0, dict(prefix=PASS, gap=True)),
    # sequences with many rows behind a prefix with pieces of its own
    "own pieces and the prefix's": ((*H32, 64, 4500, [160, 70, 300, 61], [60] * 4, 0),
                                    1, dict(prefix=PASS, many=True, final=False)),
    "finished behind two pieces": ((*H32, 64, 4500, [200, 150, 130, 101], [100] * 4, 0),
                                   1, dict(prefix=PASS, many=True, final=True, pieces=2)),
    "finished behind three pieces": ((*H32, 16, 4500, [300, 250, 151, 150], [150] * 4, 0),
                                     0, dict(prefix=PASS, many=True, final=True, pieces=3)),
    "finished behind three pieces, a few rows among them": ((*H32, 64, 4500, [700, 30, 1], [600, 8, 1], 0),
                                                         0, dict(prefix=PASS, many=True, final=True, pieces=3)),
    "finished, window inside the prefix": ((*H32, 64, 4500, [200, 150, 900, 101], [100] * 4, 800),
                                           0, dict(prefix=PASS, many=True, final=True, pieces=2)),
    "finished without a prefix": ((*H32, 64, 0, [300] * 4, [300, 200, 299, 100], 0),
                                  2, dict(prefix=NONE, many=True, final=True)),
    "ahead and finished": ((*H32, 64, 1000, [620, 500, 530], [600, 450, 520], 0), 0, dict(prefix=AHEAD, many=True, final=True)),
    "ahead and finished, window": ((*H32, 64, 1000, [500, 300, 400], [400, 250, 320], 600),
                                   0, dict(prefix=AHEAD, many=True, final=True)),
}
