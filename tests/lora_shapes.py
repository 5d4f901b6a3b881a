"""Shapes (M, N, K, bits, group size, rank) of qmv_lora_run whose launch plans are tight:
the GPU tests run them, and the plan's test says that they cover what plans differ in."""

# more vectors than a pass over projections of full width, every weight form
PASSES = [(M, N, K, bits, gs, R)
          for (N, K), Ms in (((15360, 3840), (17, 33, 64)), ((14336, 4096), (17, 32, 64)), ((3840, 15360), (17, 33, 64)), ((4096, 14336), (32,)))
          for M in Ms for bits, gs, R in ((4, 64, 16), (4, 128, 27), (2, 64, 16), (2, 128, 64))]
# high ranks, and more than one round of tiles
PASSES += [(50, 17408, 4096, 4, 64, 200), (48, 20008, 1984, 4, 64, 24), (40, 39000, 4096, 2, 64, 8), (70, 1000, 8192, 4, 64, 256)]

# one pass whose ring has three slots
THREE_SLOTS = [(16, 15360, 3840, 4, 64, 16), (13, 14336, 4096, 2, 64, 64), (16, 17408, 4096, 4, 64, 64)]

# several passes in a CTA over fewer slots of K than there are worker groups
FEW_SLOTS = [(100, 20008, 256, 4, 64, 16), (64, 20000, 512, 4, 128, 8), (40, 19500, 128, 2, 64, 27), (200, 19456, 1024, 2, 128, 64)]
