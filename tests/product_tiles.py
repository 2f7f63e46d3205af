"""Sizes that reach every kernel of the bf16 products, by its name on 256 compute units: last tiles short
of rows, of columns and of K; one K block, two and more; and, for each tile that large products take,
more tiles than compute units, so that a workgroup goes from one to the next."""

GATED = ("silu_mul", "swiglu_clamp")
UNGATED = (None, "silu", "gelu_tanh")

# (kernel, gated): [(M, K, Ns, S)]
DENSE = {
    ("gemm_rows_kernel 16x16", False): [(1, 8, 8, 1), (13, 1032, 200, 3), (16, 264, 4104, 1)],
    ("gemm_rows_kernel 16x32", True): [(1, 72, 8, 2), (11, 520, 1032, 2)],
    ("gemm_tile_kernel 32x32", False): [(33, 912, 40, 1), (100, 2888, 328, 1), (1, 16400, 16, 2)],
    ("gemm_tile_kernel 32x32", True): [(35, 952, 24, 2), (75, 2888, 392, 2)],
    ("gemm_tile_kernel 32x128", False): [(65, 8, 2848, 3), (66, 72, 4280, 2), (68, 152, 4168, 2), (333, 2888, 2888, 1),
                                         (66, 136, 5584, 3)],
    ("gemm_tile_kernel 32x128", True): [(66, 8, 4216, 2), (72, 136, 4104, 2), (135, 136, 5584, 2)],
    ("gemm_tile_kernel 64x64", False): [(65, 8, 72, 1), (66, 72, 24, 3), (73, 392, 136, 2), (8349, 144, 48, 3)],
    ("gemm_tile_kernel 64x64", True): [(65, 8, 40, 2), (68, 136, 40, 2), (8776, 144, 72, 2)],
    ("gemm_tile_kernel 64x128", False): [(66, 8, 5488, 2), (68, 80, 3752, 3), (5561, 136, 48, 3), (396, 152, 2360, 3)],
    ("gemm_tile_kernel 64x128", True): [(65, 8, 5592, 2), (132, 72, 3304, 2), (258, 136, 5368, 2)],
    ("gemm_tile_kernel 128x128", False): [(8362, 136, 200, 1), (395, 72, 4704, 3), (4985, 8, 2824, 1)],
    ("gemm_tile_kernel 128x128", True): [(166, 144, 5480, 2), (7147, 136, 392, 2), (3151, 8, 2248, 2)],
    ("gemm_tile_kernel 128x256", False): [(8212, 464, 480, 1), (211, 568, 5472, 3), (1380, 456, 3608, 3)],
    ("gemm_tile_kernel 128x256", True): [(321, 472, 5512, 2), (1566, 504, 4728, 2)],
    ("gemm_tile_kernel 256x256", False): [(1184, 336, 5128, 2), (4000, 1336, 4072, 1), (7318, 328, 1928, 2)],
    ("gemm_tile_kernel 256x256", True): [(4512, 336, 1368, 2), (1671, 336, 3704, 2), (3810, 328, 3864, 2)],
}

# (kernel, gated): [(M, topk, E, K, Ns, S, block_m)]
GROUPED = {
    ("gemm_rows_kernel 16x32", False): [(16, 4, 32, 2880, 200, 1, 16), (33, 2, 8, 136, 72, 2, 32)],
    ("gemm_rows_kernel 16x32", True): [(64, 6, 6, 1032, 40, 2, 16)],
    ("gemm_rows_kernel 16x64", False): [(300, 4, 8, 200, 264, 2, 64), (513, 2, 4, 328, 520, 1, 128)],
    ("gemm_rows_kernel 16x64", True): [(8, 4, 128, 520, 264, 2, 16), (100, 8, 16, 264, 264, 2, 64)],
    ("gemm_tile_kernel 64x256", False): [(207, 4, 24, 8, 944, 1, 64), (212, 4, 24, 72, 1016, 1, 16),
                                         (1974, 1, 24, 88, 1184, 2, 16)],
    ("gemm_tile_kernel 64x256", True): [(387, 2, 24, 72, 544, 2, 64), (1388, 1, 24, 80, 1688, 2, 32)],
    ("gemm_tile_kernel 128x256", False): [(304, 2, 8, 8, 1424, 1, 128), (868, 2, 24, 80, 544, 1, 128),
                                          (7798, 4, 24, 80, 144, 2, 128)],
    ("gemm_tile_kernel 128x256", True): [(1732, 2, 8, 72, 136, 2, 128), (983, 4, 24, 80, 1160, 2, 32)],
    ("gemm_tile_kernel 256x256", False): [(4910, 4, 24, 88, 264, 1, 16), (4874, 4, 5, 72, 816, 1, 32),
                                          (7155, 4, 24, 72, 528, 1, 128)],
    ("gemm_tile_kernel 256x256", True): [(4120, 4, 8, 80, 136, 2, 128), (4853, 4, 8, 80, 392, 2, 32)],
}


def flat(table, only=None):
    """[(kernel, activation's kind, size)] with an id for each, or those of one kind."""
    rows = [(name, gated, size) for (name, gated), sizes in table.items() for size in sizes if only in (None, gated)]
    return dict(argvalues=rows, ids=["-".join([n.split()[1], *(["gated"] if g else []), "x".join(map(str, s))])
                                     for n, g, s in rows])
